// Cutting a cache down: per sequence and kv head, the `keep` tokens that stay are the first
// `sinks`, the last `recent` and, of those between, the ones of the largest accumulated
// weight (ties: the earlier); they move to the slots 0 .. keep - 1, in their order.
//
// Choosing (select_kernel): one block per (sequence, head) finds the weight of rank
// `heavy` by three passes over 11, 11 and 10 bits of the weights' ordered patterns, counted in one
// histogram in shared memory, then goes once through the slots, four in a row to a thread, and writes
// the staying ones by their rank, a prefix sum over the block. The first kCache patterns stay in shared
// memory. The longest row bounds it, 24 us for 30,515 tokens of which 4,096 stay (3 to load, 10 to count and search, 9
// to place, 2 for the zeros behind), 47 us for 65,531: so 1,024 threads a block, patterns formed once and counted four at a time. (The last pass with
// a range of the slots per warp, twice, and one sum over the block: the same.)
// The moves' launch comes when all blocks have chosen: blocks that wait for it on SMs with room made a
// call 27 us longer.
//
// Moving (move_kernel): a chunk is 2,048 pieces of 16 bytes, eight per thread, whose loads
// are in flight together, and those of the next chunk before this one's are stored. To
// other pages, a CTA takes a part of the line of all sequences' slots. In place, slot i
// takes that of kept[i] >= i, so whoever writes slot i must know that all that lies there
// is read: a CTA takes the slots of one (sequence, head, K or V) in order, of which it may store a
// chunk as soon as its own loads of it are through, since later chunks read later slots; with few
// sequences CTAs share a row's bytes, not its slots, and nobody waits for another CTA. Short rows
// are moved by the block that has chosen them, in one launch (FUSED). Bound by HBM: 952 MB in 147 us, 6.5 TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_cache.cuh"
#include "kda_common.cuh"

namespace kda {
namespace cache {

struct EvictArgs {
    Table src, dst;
    const int32_t *lens, *keep;
    const int32_t *refs;  // or NULL
    int sinks, recent;
    int Hkv, cap, page, page_bits, pages;
    const float *w;       // [rows, Hkv, cap]
    float *w_out;
    int32_t *kept;
    int32_t *state;       // [rows]: slots that move, 0: none
    int in_place;
    int ranked;           // at most kRanked rows, the longest first
    uint32_t *status;
    uint4 *kp, *vp;
    int row_bits;         // 16-byte pieces of a row: 16 or 32
    __device__ __forceinline__ int row(const Table &t, int b, int h, int slot) const {
        return (t.row(b)[slot >> page_bits] * Hkv + h) * page + (slot & (page - 1));
    }
};

// ---- the slots that stay ---------------------------------------------------------
// Patterns that order as the weights do: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t ordered(uint32_t bits) {
    const float x = __uint_as_float(bits);
    if (x != x) return 0xffffffffu;
    const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
    return u >> 31 ? ~u : u | 0x80000000u;
}
// Whether a pattern tells its weight, and which.
__device__ __forceinline__ bool tells(uint32_t key) { return key != 0xffffffffu && key != 0x80000000u; }
__device__ __forceinline__ float weight_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }

constexpr int kSelThreads = 1024, kSelWarps = 32;
constexpr int kCache = 49152;
constexpr int kRanked = 128;  // rows that are ranked at the most
constexpr int kBins = 2048, kBinsEach = kBins / kSelThreads;
constexpr int kRound = 4 * kSelThreads;  // slots of a round of the last pass

// The moves of a fused block: four pieces per thread, all of them in flight.
constexpr int kFusedFlight = 4, kFusedBytes = kSelThreads * kFusedFlight * 16;  // K and V of a head at the most

__device__ __forceinline__ void fused_moves(const EvictArgs &a, int b, int h, int n, const int32_t *kept) {
    __shared__ int2 where[kFusedBytes / 512];  // (from, to) rows of the pools, (-1, ..): none
    const int tid = threadIdx.x, slot_bits = a.row_bits + 1, pieces = n << slot_bits;
    __syncthreads();  // `kept` is written
    if (tid < n) {
        int2 p = make_int2(a.row(a.src, b, h, kept[tid]), a.row(a.dst, b, h, tid));
        if (p.x == p.y) p.x = -1;
        where[tid] = p;
    }
    __syncthreads();
    uint4 y[kFusedFlight];
    auto each = [&](auto f) {  // (piece, rows, the pool, its piece of a row)
#pragma unroll
        for (int q = 0; q < kFusedFlight; ++q) {
            const int x = q * kSelThreads + tid, at = x & ((1 << slot_bits) - 1);
            if (x >= pieces) continue;
            const int2 p = where[x >> slot_bits];
            if (p.x >= 0) f(y[q], p, at >> a.row_bits ? a.vp : a.kp, at & ((1 << a.row_bits) - 1));
        }
    };
    each([&](uint4 &z, int2 p, const uint4 *pool, int at) { z = pool[((size_t)p.x << a.row_bits) + at]; });
    __syncthreads();  // in place: all is read
    each([&](const uint4 &z, int2 p, uint4 *pool, int at) { pool[((size_t)p.y << a.row_bits) + at] = z; });
}

template <bool FUSED>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ __align__(16) uint32_t patterns[];
    __shared__ int warp_sums[2][32];
    __shared__ int hist[kBins];
    __shared__ int found[2];  // the digit, and how many above it there are
    wait_before();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Where not all blocks start at once, long rows first: the last ones to start are then the shortest (25.7 us
    // instead of 35.0 for 32 sequences of 966 to 30,515 tokens on 8 heads). Each thread ranks a row.
    __shared__ int lens[kRanked], row_of_rank;
    int b = blockIdx.x / a.Hkv;
    const int h = blockIdx.x - b * a.Hkv;
    if (a.ranked) {
        if (tid < a.src.rows) lens[tid] = a.lens[tid];
        __syncthreads();
        if (tid < a.src.rows) {
            int rank = 0;
            for (int i = 0; i < a.src.rows; ++i) rank += lens[i] > lens[tid] || (lens[i] == lens[tid] && i < tid);
            if (rank == b) row_of_rank = tid;
        }
        __syncthreads();
        b = row_of_rank;
    }
    const int len = a.lens[b], budget = a.keep[b];
    if (budget < 0) {
        if (!FUSED && h == 0 && tid == 0) a.state[b] = 0;
        return;
    }
    const int n = min(len, budget);
    const bool moves = !a.in_place || len > budget;
    bool bad = len < 0 || len > a.cap || (long long)len > (long long)a.src.cols * a.page ||
               (long long)n > (long long)a.dst.cols * a.page;
    const size_t first = ((size_t)b * a.Hkv + h) * a.cap;
    const float *const w = a.w + first;
    const int cached = min(len, kCache);
    if (!bad && len > budget) {  // (on their way while the pages are looked at)
        const int whole = (reinterpret_cast<uintptr_t>(w) & 15) == 0 ? cached & ~3 : 0;
        for (int i = 4 * tid; i < whole; i += 4 * kSelThreads)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(patterns + i)), "l"(w + i) : "memory");
        for (int i = whole + tid; i < cached; i += kSelThreads)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_u32(patterns + i)), "l"(w + i) : "memory");
    }
    if (!bad) {
        const int32_t *const from = a.src.row(b), *const to = a.dst.row(b);
        for (int j = tid; j < (int)(((unsigned)len + a.page - 1) >> a.page_bits); j += kSelThreads)
            bad = bad || from[j] < 0 || from[j] >= a.pages;
        for (int j = tid; j < (int)(((unsigned)n + a.page - 1) >> a.page_bits); j += kSelThreads) {
            const int pg = to[j];
            bad = bad || pg < 0 || pg >= a.pages;
            if (!bad && moves && a.refs != nullptr) bad = a.refs[pg] != 1;  // others read what is there
        }
    }
    const int sinks = min(a.sinks, n), recent = min(a.recent, n - sinks), end = len - recent;
    int need = n - sinks - recent;  // of [sinks, end)
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    if (__syncthreads_or(bad)) {
        if (tid == 0 && h == 0) {
            if (!FUSED) a.state[b] = 0;
            atomicOr(a.status, kStatusBadSeqlens);
        }
        return;
    }
    if (!FUSED && h == 0 && tid == 0) a.state[b] = moves ? n : 0;
    float *const w_out = a.w_out + first;
    int32_t *const kept = a.kept + first;
    if (len <= budget) {
        for (int i = tid; i < len; i += kSelThreads) {
            kept[i] = i;
            if (w_out != w) w_out[i] = w[i];
        }
        if (FUSED && moves) fused_moves(a, b, h, n, kept);
        return;
    }
    uint32_t top = 0xffffffffu;  // what is above it stays, and the first `need` equal ones
    const bool ranked = need > 0;  // else the weights do not count, and their patterns are not formed
    if (ranked) {
        top = 0;
        for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {  // 21, 10, 0
#pragma unroll
            for (int e = 0; e < kBinsEach; ++e) hist[tid + kSelThreads * e] = 0;
            __syncthreads();
            const uint32_t mask = shift == 21 ? 0u : (shift == 10 ? ~0u << 21 : ~0u << 10), digits = shift == 0 ? 1023 : 2047;
            auto count = [&](uint32_t key) {
                if ((key & mask) == top) atomicAdd(&hist[key >> shift & digits], 1);
            };
#pragma unroll 2
            for (int i = 4 * tid; i < cached; i += 4 * kSelThreads) {
                uint4 x = *reinterpret_cast<const uint4 *>(patterns + i);  // (behind `cached`: anything)
                if (shift == 21) {
                    x = make_uint4(ordered(x.x), ordered(x.y), ordered(x.z), ordered(x.w));
                    *reinterpret_cast<uint4 *>(patterns + i) = x;
                }
                if (i >= sinks && i + 4 <= min(end, cached)) {
                    count(x.x);
                    count(x.y);
                    count(x.z);
                    count(x.w);
                } else {
                    const int last = min(end, cached);
                    if (i >= sinks && i < last) count(x.x);
                    if (i + 1 >= sinks && i + 1 < last) count(x.y);
                    if (i + 2 >= sinks && i + 2 < last) count(x.z);
                    if (i + 3 >= sinks && i + 3 < last) count(x.w);
                }
            }
#pragma unroll 4
            for (int i = max(sinks, kCache) + tid; i < end; i += kSelThreads) count(ordered(__float_as_uint(w[i])));
            __syncthreads();
            int mine = 0, c[kBinsEach], total;  // the digits from the top
#pragma unroll
            for (int e = 0; e < kBinsEach; ++e) mine += c[e] = hist[kBins - 1 - kBinsEach * tid - e];
            int above = block_exclusive<kSelWarps>(mine, warp_sums[0], total);
#pragma unroll
            for (int e = 0; e < kBinsEach; ++e) {
                if (above < need && above + c[e] >= need) {
                    found[0] = kBins - 1 - kBinsEach * tid - e;
                    found[1] = above;
                }
                above += c[e];
            }
            __syncthreads();
            top |= (uint32_t)found[0] << shift;
            need -= found[1];
        }
    }
    // Weights in place: a step writes no slot past those that it or earlier ones have read.
    int above = 0, equal = 0;
    for (int i0 = 0, round = 0; i0 < len; i0 += kRound, ++round) {
        const int at = i0 + 4 * tid;
        uint32_t key[4] = {0, 0, 0, 0};
        if (at < cached) *reinterpret_cast<uint4 *>(key) = *reinterpret_cast<const uint4 *>(patterns + at);
        uint32_t stays = 0, ties = 0;
        float x[4];
        // Most warps: no end of anything, no equal one, every staying weight told by its pattern.
        bool plain = ranked && at >= sinks && at + 4 <= end && at + 4 <= cached;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            stays |= (uint32_t)(key[e] > top) << e;
            plain = plain && key[e] != top && !(key[e] > top && !tells(key[e]));
            x[e] = weight_of(key[e]);
        }
        if (!__all_sync(0xffffffffu, plain)) {
            stays = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = at + e;
                if (i >= len) continue;
                if (ranked && i >= cached) key[e] = ordered(__float_as_uint(w[i]));
                const bool stay = i < sinks || i >= end || (ranked && key[e] > top), tie = ranked && !stay && key[e] == top;
                stays |= (uint32_t)stay << e;
                ties |= (uint32_t)tie << e;
                if (stay || tie) x[e] = w[i];
            }
        }
        // staying ones ahead of this thread's, and equal ones in the upper half
        int mine = __popc(stays) + (__popc(ties) << 16), incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sums[round & 1][warp] = incl;
        __syncthreads();  // (so that all of this step's weights are read; the other sums are the last one's)
        const int theirs = warp_sums[round & 1][lane];
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0) + incl - mine;
        const int total = __reduce_add_sync(0xffffffffu, theirs);
        int s = above + (before & 0xffff), t = equal + (before >> 16);
        if (ties == 0) {
            s += min(t, need);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (stays >> e & 1) {
                    kept[s] = at + e;
                    w_out[s++] = x[e];
                }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool tie = ties >> e & 1;
                if ((stays >> e & 1) || (tie && t < need)) {
                    const int to = s + min(t, need);
                    kept[to] = at + e;
                    w_out[to] = x[e];
                }
                s += stays >> e & 1;
                t += tie;
            }
        }
        above += total & 0xffff;
        equal += total >> 16;
    }
    let_next_start();
    __syncthreads();
    for (int i = n + tid; i < len; i += kSelThreads) w_out[i] = 0.f;
    if (FUSED) fused_moves(a, b, h, n, kept);
}

// ---- the rows that move ------------------------------------------------------------
constexpr int kMoveThreads = 256, kFlight = 8, kChunk = kMoveThreads * kFlight;
constexpr int kMoveRows = kChunk / 4;  // rows of a chunk at the most: four pieces of each

struct MoveArgs {
    int rows;        // of the table
    int piece_bits;  // pieces of a slot in a chunk: in place those of a CTA's slice, else those of K and V
    int parts;       // in place: CTAs of a (sequence, head)
};

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a, const MoveArgs m) {
    __shared__ int2 where[3][kMoveRows];  // (from, to) rows of the pools, (-1, ..): none
    wait_before();
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31;
    const int per_chunk = kChunk >> m.piece_bits;  // slots
    // The chunks of this CTA: (b, h, chunk), `left` of them.
    int b, h = 0, chunk = 0, n = 0;
    long long left;
    auto chunks = [&](int slots) { return (int)(((unsigned)slots + per_chunk - 1) / (unsigned)per_chunk); };
    if (IN_PLACE) {
        const int bh = blockIdx.x / m.parts;
        b = bh / a.Hkv;
        h = bh - b * a.Hkv;
        n = a.state[b];
        left = chunks(n);
    } else {
        long long total = 0;
        for (int i = lane; i < m.rows; i += 32) total += chunks(a.state[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= a.Hkv;
        long long x = total * blockIdx.x / gridDim.x;
        left = total * (blockIdx.x + 1LL) / gridDim.x - x;
        if (left == 0) return;
        for (b = 0; b < m.rows; b += 32) {
            const int mine_n = b + lane < m.rows ? a.state[b + lane] : 0;
            const long long mine = (long long)chunks(mine_n) * a.Hkv;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const long long sum = __shfl_sync(0xffffffffu, incl, 31);
            if (x >= sum) {
                x -= sum;
                continue;
            }
            const int at = __ffs(__ballot_sync(0xffffffffu, x < incl)) - 1;
            x -= __shfl_sync(0xffffffffu, incl - mine, at);
            n = __shfl_sync(0xffffffffu, mine_n, at);
            b += at;
            h = (int)(x / chunks(n));
            chunk = (int)(x - (long long)h * chunks(n));
            break;
        }
    }
    if (left == 0) return;
    const int32_t *kept = a.kept + ((size_t)b * a.Hkv + h) * a.cap;
    // Where the next chunk's rows are and go, and on to the one after it. (Behind the last: none.)
    auto look = [&](int2 *to) {
        const bool any = left > 0;
        for (int r = tid; r < per_chunk; r += kMoveThreads) {
            const int i = chunk * per_chunk + r;
            int2 p = make_int2(-1, -1);
            if (any && i < n) {
                p = make_int2(a.row(a.src, b, h, kept[i]), a.row(a.dst, b, h, i));
                if (p.x == p.y) p.x = -1;
            }
            to[r] = p;
        }
        if (!any) return;
        --left;
        ++chunk;
        if (!IN_PLACE && left > 0 && chunk == chunks(n)) {
            chunk = 0;
            if (++h == a.Hkv) {
                h = 0;
                do n = ++b < m.rows ? a.state[b] : 0;
                while (n == 0 && b < m.rows);
            }
            kept = a.kept + ((size_t)b * a.Hkv + h) * a.cap;
        }
    };
    const int part = IN_PLACE ? blockIdx.x % m.parts : 0;
    // piece x of a slot: of K or V, and which of its row
    auto piece = [&](int x, int row, bool &is_v) -> size_t {
        const int at = IN_PLACE ? (part << m.piece_bits) + x : x;
        is_v = at >> a.row_bits;
        return ((size_t)row << a.row_bits) + (at & ((1 << a.row_bits) - 1));
    };
    auto load = [&](const int2 *rows, uint4 *y) {
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int x = f * kMoveThreads + tid, from = rows[x >> m.piece_bits].x;
            bool is_v;
            const size_t at = piece(x & ((1 << m.piece_bits) - 1), from, is_v);
            if (from >= 0) y[f] = (is_v ? a.vp : a.kp)[at];
        }
    };
    auto store = [&](const int2 *rows, const uint4 *y) {
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int x = f * kMoveThreads + tid;
            const int2 p = rows[x >> m.piece_bits];
            bool is_v;
            const size_t at = piece(x & ((1 << m.piece_bits) - 1), p.y, is_v);
            if (p.x >= 0) (is_v ? a.vp : a.kp)[at] = y[f];
        }
    };
    uint4 y[2][kFlight];
    long long todo = left;
    look(where[0]);
    look(where[1]);
    __syncthreads();
    load(where[0], y[0]);
    __syncthreads();
    int at = 0;  // todo chunks from this buffer on
    for (; todo > 0; todo -= 2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int next = at == 2 ? 0 : at + 1, after = next == 2 ? 0 : next + 1;
            load(where[next], y[1 - half]);
            look(where[after]);
            // this chunk's loads of all threads are through (the barrier before), and so
            // are those of every slot that it writes
            if (half == 0 || todo > 1) store(where[at], y[half]);
            __syncthreads();
            at = next;
        }
    }
}

// ---- pages behind the end ------------------------------------------------------------
__global__ void __launch_bounds__(256)
    trim_kernel(Table table, int32_t *lens, int32_t *refs, int pages, int page, const int32_t *__restrict__ want,
                uint32_t *status) {
    wait_before();
    let_next_start();
    for (int r = blockIdx.x; r < table.rows; r += gridDim.x) {
        const int n = want[r];
        if (n < 0) continue;
        int32_t *row = table.row(r);
        const int first = (int)(((unsigned)n + page - 1) / (unsigned)page);
        for (int j = first + blockIdx.y * blockDim.x + threadIdx.x; j < table.cols; j += gridDim.y * blockDim.x) {
            const int pg = row[j];
            if (!in_use(pg)) continue;
            if (pg >= 0 && pg < pages) atomicSub(refs + pg, 1);
            else if (pg >= 0 && status) atomicOr(status, kStatusBadSeqlens);
            row[j] = -1;
        }
        if (blockIdx.y == 0 && threadIdx.x == 0 && lens[r] > n) lens[r] = n;
    }
}

// ---- host ------------------------------------------------------------------------------
cudaError_t launch_evict(void *kp, void *vp, int pages, int page, int32_t *table, int64_t ld, int rows, int cols,
                         int32_t *dst, int64_t dst_ld, int dst_cols, const int32_t *refs, const int32_t *lens,
                         const int32_t *keep, int sinks, int recent, int Hkv, int es, const float *w, float *w_out,
                         int32_t *kept, int cap, int32_t *state, uint32_t *status, int sms, cudaStream_t stream) {
    EvictArgs a = {};
    a.src = Table{table, ld, rows, cols};
    a.in_place = dst == nullptr;
    a.dst = a.in_place ? a.src : Table{dst, dst_ld, rows, dst_cols};
    a.lens = lens;
    a.keep = keep;
    a.refs = refs;
    a.sinks = sinks;
    a.recent = recent;
    a.Hkv = Hkv;
    a.cap = cap;
    a.page = page;
    a.pages = pages;
    while ((1 << a.page_bits) < page) ++a.page_bits;
    a.w = w;
    a.w_out = w_out;
    a.kept = kept;
    a.state = state;
    a.status = status;
    const long long heads = (long long)rows * Hkv;
    a.ranked = rows <= kRanked && heads > sms;
    a.kp = static_cast<uint4 *>(kp);
    a.vp = static_cast<uint4 *>(vp);
    a.row_bits = es == 2 ? 4 : 5;
    // (shared memory for the longest possible row; past kCache weights the others are read from L2)
    const int cached = cap < kCache ? (cap + 3) & ~3 : kCache;
    // The block that has chosen moves the rows too where they are few: 8.4 us instead of 11.3 for 50 rows of
    // 512 bytes (K and V), but 16.5 instead of 14.4 for 200 of 1,024.
    const long long room = a.in_place ? cap : (long long)dst_cols * page;
    const bool fused = ((room < cap ? room : cap) << (a.row_bits + 5)) <= kFusedBytes;
    static std::atomic<uint64_t> ready{0};  // devices whose limits are raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCache * 4);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCache * 4);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    e = launch_early(fused ? select_kernel<true> : select_kernel<false>, dim3((unsigned)heads), kSelThreads, (size_t)cached * 4,
                     stream, a);
    if (e != cudaSuccess || fused) return e;
    MoveArgs m = {rows, 0, 1};
    m.piece_bits = a.row_bits;
    if (a.in_place) {
        // Slices of a row down to 64 bytes, until two CTAs per SM have work.
        while (m.piece_bits > 2 && (heads * 2 << (a.row_bits - m.piece_bits)) < 2LL * sms) --m.piece_bits;
        m.parts = 2 << (a.row_bits - m.piece_bits);
        return launch_early(move_kernel<true>, dim3((unsigned)(heads * m.parts)), kMoveThreads, 0, stream, a, m);
    }
    m.piece_bits = a.row_bits + 1;
    const long long per = kChunk >> m.piece_bits, most = heads * (((long long)cap + per - 1) / per), ctas = 4LL * sms;
    return launch_early(move_kernel<false>, dim3((unsigned)(most < ctas ? most : ctas)), kMoveThreads, 0, stream, a, m);
}

cudaError_t launch_trim(int32_t *table, int64_t ld, int rows, int cols, int32_t *lens, int32_t *refs, int pages, int page,
                        const int32_t *want, uint32_t *status, cudaStream_t stream) {
    const int y = (cols + 255) / 256;
    return launch_early(trim_kernel, dim3((unsigned)(rows < 65535 ? rows : 65535), (unsigned)(y < 64 ? y : 64)), 256, 0,
                        stream, Table{table, ld, rows, cols}, lens, refs, pages, page, want, status);
}

}  // namespace cache
}  // namespace kda
