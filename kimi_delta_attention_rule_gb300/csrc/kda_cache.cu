// The pages of a key/value cache: appending rows, and allocating, forking,
// freeing, compacting and copying pages.
//
// A cache is a pool of pages [pages][Hkv][page][128] for K and one for V (of any
// number of layers), a block table int32 [rows][cols] (row b: the pages of a
// sequence in order, -1 past its end) and refs int32 [pages], the number of table
// entries on each page (0: free). A page is chosen lowest number first, so that a
// call's result is a function of its inputs.
//
// The calls that choose pages need, for every page, its rank among the free (or
// live) ones: a prefix sum over refs. They run as one cluster of eight CTAs,
// each with an eighth of refs, that exchange their counts through distributed
// shared memory: one launch, no workspace for the sum, no spinning. Bound: the
// latency of a handful of dependent loads and cluster barriers (refs itself, 4
// bytes per page, is 0.3 us of one SM's bandwidth at 8,192 pages).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_cache.cuh"
#include "kda_common.cuh"

namespace kda {
namespace cache {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;  // the largest portable cluster
constexpr int kMaxPools = 16;

// ---- append -----------------------------------------------------------------
// A warp per row: it issues the loads of the row's first 2 KB (which need no look-up,
// but for accepted drafts), then finds where the row goes, a chain of dependent loads
// that those of other warps and its own data hide, then stores. Bound by HBM: 16,385 rows of
// 8 heads, 134 MB each way together, in 20.6 to 23 us, 5.8 to 6.5 TB/s (8 pieces in flight
// instead of 4: the same; several rows per warp or a block per page: slower).
constexpr int kAppendWarps = 8, kAppendFlight = 4;

// The last sequence that starts at or before row r, by one converged warp.
__device__ __forceinline__ int find_sequence(const int32_t *__restrict__ cu, int N, int64_t r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, count = N;  // in [lo, lo + count)
    while (count > 1) {
        const int step = (count + 31) >> 5, at = lo + lane * step;
        const bool before = lane == 0 || (lane * step < count && cu[at] <= r);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, before));
        count = min(step, count - k * step);
        lo += k * step;
    }
    return lo;
}

__global__ void __launch_bounds__(32 * kAppendWarps)
    append_kernel(const uint4 *__restrict__ k, const uint4 *__restrict__ v, int64_t ldk, int64_t ldv,
                  const int32_t *__restrict__ cu, int N, int T, int64_t rows, const int32_t *__restrict__ index,
                  const int32_t *__restrict__ count, const int32_t *__restrict__ start, Table table, int pages,
                  int page, int Hkv, int piece_bits, uint4 *__restrict__ kp, uint4 *__restrict__ vp,
                  uint32_t *status) {
    wait_before();
    let_next_start();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    if (r >= rows) return;
    // the sequence, the row's number in it, and the row to read
    int n = 0, i = 0;
    bool ok = true;
    int64_t from = r;
    if (cu == nullptr) {
        n = (int)(r / T);
        i = (int)(r - (int64_t)n * T);
        int have = T;
        if (count != nullptr) {
            have = count[n];
            if (have < 0 || have > T) {
                if (status && i == 0 && lane == 0) atomicOr(status, kStatusBadSeqlens);
                return;
            }
        }
        if (i >= have) return;
        if (index != nullptr) {
            const int x = index[r];
            ok = x >= 0 && x < T;
            if (ok) from = (int64_t)n * T + x;
        }
    }
    const int per_row = Hkv << piece_bits, work = 2 * per_row;  // 16-byte pieces of a row, of K and V
    auto piece = [&](int x) { return x < per_row ? k[from * ldk + x] : v[from * ldv + (x - per_row)]; };
    uint4 y[kAppendFlight];
#pragma unroll
    for (int f = 0; f < kAppendFlight; ++f)
        if (lane + 32 * f < work) y[f] = piece(lane + 32 * f);
    if (cu != nullptr) {
        n = find_sequence(cu, N, r);
        i = (int)(r - cu[n]);
        ok = cu[0] == 0 && cu[n + 1] > r;  // else the offsets do not cover this row
    }
    int64_t dst = -1;  // first piece of (page, head 0, offset)
    if (ok) {
        const int64_t pos = (int64_t)start[n] + i, slot = pos / page;
        const int pg = pos >= 0 && slot < table.cols ? table.row(n)[slot] : -1;
        if (pg >= 0 && pg < pages) dst = ((int64_t)pg * Hkv * page + pos % page) << piece_bits;
    }
    if (dst < 0) {
        if (status && lane == 0) atomicOr(status, kStatusBadSeqlens);
        return;
    }
    const int64_t head_step = (int64_t)page << piece_bits;
    auto store = [&](int x, uint4 z) {
        const bool is_v = x >= per_row;
        const int w = is_v ? x - per_row : x;
        (is_v ? vp : kp)[dst + (w >> piece_bits) * head_step + (w & ((1 << piece_bits) - 1))] = z;
    };
    for (int x0 = lane; x0 < work; x0 += 32 * kAppendFlight) {
        if (x0 != lane) {
#pragma unroll
            for (int f = 0; f < kAppendFlight; ++f)
                if (x0 + 32 * f < work) y[f] = piece(x0 + 32 * f);
        }
#pragma unroll
        for (int f = 0; f < kAppendFlight; ++f)
            if (x0 + 32 * f < work) store(x0 + 32 * f, y[f]);
    }
}

// ---- copy ---------------------------------------------------------------------
// A block takes 32 KB of one entry at a time: eight 16-byte pieces in flight per
// thread before the first is stored. Bound by HBM: 1.95 GB in 299 us, 6.5 TB/s (four pieces:
// 10 us more).
struct Pools {
    uint4 *base[kMaxPools];
};
constexpr int kCopyThreads = 256, kCopyFlight = 8, kCopyChunk = kCopyThreads * kCopyFlight;

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const Pools pools, int n_pools, int64_t entry, int entries, const int2 *__restrict__ pairs, int n,
                const int32_t *__restrict__ count) {
    wait_before();
    let_next_start();
    if (count != nullptr) {
        const int have = *count;
        n = have < 0 ? 0 : (have < n ? have : n);
    }
    const int64_t chunks = (entry + kCopyChunk - 1) / kCopyChunk, per_pair = chunks * n_pools;
    for (int64_t w = blockIdx.x; w < per_pair * n; w += gridDim.x) {
        const int j = (int)(w / per_pair);
        const int2 p = pairs[j];
        if (p.x < 0 || p.y < 0 || p.x >= entries || p.y >= entries || p.x == p.y) continue;
        const int rest = (int)(w - j * per_pair), pool = (int)(rest / chunks);
        const int64_t at = (rest - pool * chunks) * kCopyChunk + threadIdx.x;
        const uint4 *src = pools.base[pool] + p.x * entry;
        uint4 *dst = pools.base[pool] + p.y * entry;
        uint4 y[kCopyFlight];
#pragma unroll
        for (int f = 0; f < kCopyFlight; ++f)
            if (at + f * kCopyThreads < entry) y[f] = __ldcs(src + at + f * kCopyThreads);
#pragma unroll
        for (int f = 0; f < kCopyFlight; ++f)
            if (at + f * kCopyThreads < entry) __stcs(dst + at + f * kCopyThreads, y[f]);
    }
}

// ---- free -----------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    free_kernel(Table table, int32_t *lens, int32_t *refs, int pages, const int32_t *__restrict__ rows,
                uint32_t *status) {
    wait_before();
    let_next_start();
    const int r = rows[blockIdx.x];
    if (r < 0 || r >= table.rows) {
        if (r >= 0 && status && threadIdx.x == 0) atomicOr(status, kStatusBadSeqlens);
        return;
    }
    int32_t *row = table.row(r);
    for (int j = blockIdx.y * blockDim.x + threadIdx.x; j < table.cols; j += gridDim.y * blockDim.x) {
        const int pg = row[j];
        if (!in_use(pg)) continue;
        if (pg >= 0 && pg < pages) atomicSub(refs + pg, 1);
        else if (pg >= 0 && status) atomicOr(status, kStatusBadSeqlens);
        row[j] = -1;
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) lens[r] = 0;
}

// ---- cluster sums ------------------------------------------------------------
// The slice of refs of one CTA: a multiple of four pages, read as int4.
struct Slice {
    int lo, hi;
};
__device__ __forceinline__ Slice slice_of(int pages, int rank) {
    const int per = ((pages + kCtas - 1) / kCtas + 3) & ~3;
    Slice s;
    s.lo = min(pages, rank * per);
    s.hi = min(pages, s.lo + per);
    return s;
}
// refs[p .. p + 3] as four live bits (pages past hi: neither live nor free)
__device__ __forceinline__ void flags4(const int32_t *refs, int p, int hi, int &live, int &free) {
    live = free = 0;
    if (p + 4 <= hi) {
        const int4 x = *reinterpret_cast<const int4 *>(refs + p);
        live = (x.x > 0) | (x.y > 0) << 1 | (x.z > 0) << 2 | (x.w > 0) << 3;
        free = 15 ^ live;
        return;
    }
    for (int e = 0; e < 4 && p + e < hi; ++e) {
        const int x = refs[p + e];
        live |= (x > 0) << e;
        free |= (x <= 0) << e;
    }
}

struct Shared {
    int warp_sums[32];
    int mine;   // this CTA's count, read by the others
    int mine2;
};

// Sum of a count over the CTAs before this one, and over all. `which` is a
// member of Shared that holds this CTA's count.
__device__ __forceinline__ void cluster_prefix(cg::cluster_group &cl, int *mine, int rank, int &before, int &total) {
    cl.sync();
    before = total = 0;
#pragma unroll
    for (int i = 0; i < kCtas; ++i) {
        const int x = *cl.map_shared_rank(mine, i);
        total += x;
        before += i < rank ? x : 0;
    }
}

// The free pages among the four of a thread's first look at its CTA's slice.
struct First {
    Slice s;
    int p, free;
};
__device__ __forceinline__ First first_free(const int32_t *refs, int pages, int rank) {
    First f;
    int live;
    f.s = slice_of(pages, rank);
    f.p = f.s.lo + 4 * (int)threadIdx.x;
    f.free = 0;
    if (f.p < f.s.hi) flags4(refs, f.p, f.s.hi, live, f.free);
    return f;
}
// The free pages of rank < need, lowest first, into list; returns the number of
// free pages. Ends with the cluster in step: list is complete for every CTA, and no
// CTA reads another's shared memory any more.
__device__ __forceinline__ int list_free(cg::cluster_group &cl, Shared &sh, const int32_t *refs, const First &f, int need,
                                         int32_t *list) {
    const int rank = (int)cl.block_rank();
    const Slice s = f.s;
    int mine = __popc(f.free), live, fr;
    for (int p = f.p + 4 * kThreads; p < s.hi; p += 4 * kThreads) {
        flags4(refs, p, s.hi, live, fr);
        mine += __popc(fr);
    }
    int total, before, all;
    const int ahead = block_exclusive(mine, sh.warp_sums, total);
    if (threadIdx.x == 0) sh.mine = total;
    cluster_prefix(cl, &sh.mine, rank, before, all);
    if (need <= all) {
        auto put = [&](int p, int free, int j) {
            for (int e = 0; e < 4; ++e)
                if (free >> e & 1) {
                    if (j < need) list[j] = p + e;
                    ++j;
                }
        };
        if (s.hi - s.lo <= 4 * kThreads) {  // one look has been all
            put(f.p, f.free, before + ahead);
        } else {
            int at = before;
            for (int p0 = s.lo; p0 < s.hi && at < need; p0 += 4 * kThreads) {
                const int p = p0 + 4 * (int)threadIdx.x;
                int round;
                fr = 0;
                if (p < s.hi) flags4(refs, p, s.hi, live, fr);
                const int j = at + block_exclusive(__popc(fr), sh.warp_sums, round);
                put(p, fr, j);
                at += round;
            }
        }
    }
    cl.sync();
    return all;
}

// ---- fork -------------------------------------------------------------------------
// Each CTA ranks all forks that need a page (their lengths end inside one) and
// lists its slice's free pages; then a warp per fork copies the table row. All that does
// not depend on the list is read ahead of it: what bounds the call is the number of
// dependent reads and barriers (free, fork and copy of 61 forks, 8,192 pages: 15.8 us, of
// 5 forks, 1,024 pages: 9.3; 17.3 and 11.1 when the rows were read after it).
constexpr int kForksAhead = kThreads;  // whose (rank, src, dst, length) and last page stay in shared memory
constexpr int kEntriesAhead = 4;       // table entries per lane

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(Table table, int32_t *lens, int32_t *refs, int pages, int page, const int32_t *__restrict__ src,
                const int32_t *__restrict__ dst, int n, int2 *copies, int32_t *list, int32_t *ranks,
                uint32_t *status) {
    __shared__ Shared sh;
    __shared__ int4 forks[kForksAhead];
    __shared__ int tails[kForksAhead];  // the partly filled last page of the source
    cg::cluster_group cl = cg::this_cluster();
    wait_before();
    let_next_start();
    const int rank = (int)cl.block_rank();
    const First first = first_free(refs, pages, rank);
    // a fork's rank: -2 = not a fork (or a malformed one: it takes no page), -1 = no partial
    // page, else its rank among the fresh pages
    int need = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + (int)threadIdx.x;
        int state = -2, a = -1, z = -1, len = 0, tail = -1;
        if (i < n) {
            a = src[i];
            z = dst[i];
            if (a >= 0 && z >= 0) {
                bool ok = a < table.rows && z < table.rows && a != z;
                if (ok) {
                    const int taken = table.row(z)[0];
                    len = lens[a];
                    ok = len >= 0 && (long long)len <= (long long)table.cols * page && !in_use(taken);
                    state = len % page != 0;
                }
                if (ok && state == 1) {  // a page to copy from
                    tail = table.row(a)[len / page];
                    ok = tail >= 0 && tail < pages;
                }
                if (!ok) {
                    state = -2;
                    if (rank == 0 && status) atomicOr(status, kStatusBadSeqlens);
                }
            }
        }
        int round;
        const int j = need + block_exclusive(state == 1, sh.warp_sums, round);
        state = state == 1 ? j : (state == 0 ? -1 : -2);
        if (i < kForksAhead) {
            forks[i] = make_int4(state, a, z, len);
            tails[i] = tail;
        } else if (rank == 0 && i < n) {
            ranks[i] = state;
        }
        need += round;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, first_fork = rank * (kThreads / 32) + (int)(threadIdx.x >> 5);
    auto fork_of = [&](int i) {
        if (i < kForksAhead) return forks[i];
        const int state = ranks[i];
        return make_int4(state, src[i], dst[i], state != -2 ? lens[src[i]] : 0);
    };
    int4 f = make_int4(-2, -1, -1, 0);
    int ahead[kEntriesAhead], partial = -1;
    if (first_fork < n && first_fork < kForksAhead) f = forks[first_fork];
    if (f.x != -2) {
#pragma unroll
        for (int e = 0; e < kEntriesAhead; ++e) {
            const int j = lane + 32 * e;
            if (j < f.w / page) ahead[e] = table.row(f.y)[j];
        }
        partial = tails[first_fork];
    }
    const int have = list_free(cl, sh, refs, first, need, list);
    if (need > have && rank == 0 && threadIdx.x == 0 && status) atomicOr(status, kStatusNoSpace);
    for (int i = first_fork; i < n; i += kCtas * kThreads / 32) {
        const bool read = i == first_fork && i < kForksAhead;
        if (!read) f = fork_of(i);
        int2 pair = make_int2(-1, -1);
        if (f.x != -2 && need <= have) {
            const int32_t *from = table.row(f.y);
            int32_t *to = table.row(f.z);
            const int full = f.w / page;
            auto share = [&](int j, int pg) {
                to[j] = pg;
                if (pg >= 0 && pg < pages) atomicAdd(refs + pg, 1);
                else if (pg != kPageGone && status) atomicOr(status, kStatusBadSeqlens);
            };
            if (read) {
#pragma unroll
                for (int e = 0; e < kEntriesAhead; ++e)
                    if (lane + 32 * e < full) share(lane + 32 * e, ahead[e]);
            }
#pragma unroll 4
            for (int j = lane + (read ? 32 * kEntriesAhead : 0); j < full; j += 32) share(j, from[j]);
            if (f.x >= 0) {
                pair = make_int2(read ? partial : from[full], list[f.x]);
                if (lane == 0) {
                    to[full] = pair.y;
                    refs[pair.y] = 1;
                }
            }
            if (lane == 0) lens[f.z] = f.w;
        }
        if (lane == 0) copies[i] = pair;
    }
}

// ---- alloc ------------------------------------------------------------------------
// The entries in use of a row: up to the first -1, by a 32-way search of one warp.
__device__ __forceinline__ int row_used(const int32_t *row, int cols) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = cols;  // the answer lies in [lo, hi]
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool used = at < hi && in_use(row[at]);
        const unsigned b = __ballot_sync(0xffffffffu, used);
        const int k = b == 0xffffffffu ? 32 : __ffs(~b) - 1;  // probes in use
        if (k == 0) return lo;
        const int last = lo + (k - 1) * step;  // in use; the next probe is not
        hi = min(hi, last + step);
        lo = last + 1;
    }
    return lo;
}
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    alloc_kernel(Table table, const int32_t *__restrict__ want, int32_t *refs, int pages, int page, int32_t *list,
                 int2 *rows_state, uint32_t *status) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    wait_before();
    let_next_start();
    const int rank = (int)cl.block_rank(), lane = threadIdx.x & 31;
    const First first = first_free(refs, pages, rank);
    const int warp = rank * (kThreads / 32) + (int)(threadIdx.x >> 5), warps = kCtas * kThreads / 32;
    for (int r = warp; r < table.rows; r += warps) {  // (pages in use, pages to add)
        const int used = row_used(table.row(r), table.cols);
        const long long w = want[r];
        const bool ok = w >= 0 && w <= (long long)table.cols * page;
        if (!ok && lane == 0 && status) atomicOr(status, kStatusBadSeqlens);
        const int to = ok ? (int)((w + page - 1) / page) : 0;
        if (lane == 0) rows_state[r] = make_int2(used, max(0, to - used));
    }
    cl.sync();
    int need = 0;
    for (int r0 = 0; r0 < table.rows; r0 += kThreads) {
        const int r = r0 + (int)threadIdx.x;
        int round;
        block_exclusive(r < table.rows ? rows_state[r].y : 0, sh.warp_sums, round);
        need += round;
    }
    const int have = list_free(cl, sh, refs, first, need, list);
    if (need > have) {
        if (rank == 0 && threadIdx.x == 0 && status) atomicOr(status, kStatusNoSpace);
    } else if (need > 0) {
        int at = 0;
        for (int r0 = 0; r0 < table.rows; r0 += kThreads) {
            const int r = r0 + (int)threadIdx.x;
            const int2 s = r < table.rows ? rows_state[r] : make_int2(0, 0);
            int round;
            const int j = at + block_exclusive(s.y, sh.warp_sums, round);
            at += round;
            if (threadIdx.x % kCtas != rank) continue;
            int32_t *row = r < table.rows ? table.row(r) : nullptr;
            for (int e = 0; e < s.y; ++e) {
                const int pg = list[j + e];
                row[s.x + e] = pg;
                refs[pg] = 1;
            }
        }
    }
}

// ---- compact ----------------------------------------------------------------------
// n = live pages. The j-th live page >= n moves to the j-th free page < n.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    compact_kernel(int32_t *refs, int pages, int2 *copies, int32_t *count, int32_t *name, int32_t *n_live) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    wait_before();
    let_next_start();
    const int rank = (int)cl.block_rank();
    const Slice s = slice_of(pages, rank);
    int mine = 0, total, before, n;
    for (int p = s.lo + 4 * (int)threadIdx.x; p < s.hi; p += 4 * kThreads) {
        int live, fr;
        flags4(refs, p, s.hi, live, fr);
        mine += __popc(live);
    }
    block_exclusive(mine, sh.warp_sums, total);
    if (threadIdx.x == 0) sh.mine = total;
    cluster_prefix(cl, &sh.mine, rank, before, n);
    // holes below n (as many as live pages from n on), by slice
    mine = 0;
    for (int p = s.lo + 4 * (int)threadIdx.x; p < min(s.hi, n); p += 4 * kThreads) {
        int live, fr;
        flags4(refs, p, min(s.hi, n), live, fr);
        mine += __popc(fr);
    }
    block_exclusive(mine, sh.warp_sums, total);
    if (threadIdx.x == 0) sh.mine2 = total;
    int holes_before, holes;
    cluster_prefix(cl, &sh.mine2, rank, holes_before, holes);
    // live pages before this slice that are >= n: all live before less those below n
    const int low_before = min(s.lo, n) - holes_before;
    int hole_at = holes_before, move_at = before - low_before;
    for (int p0 = s.lo; p0 < s.hi; p0 += 4 * kThreads) {
        const int p = p0 + 4 * (int)threadIdx.x;
        int live = 0, fr = 0, round;
        if (p < s.hi) flags4(refs, p, s.hi, live, fr);
        const int low = p + 4 <= n ? 15 : (p >= n ? 0 : (1 << (n - p)) - 1);
        const int hole = fr & low, mover = live & ~low;
        int j = hole_at + block_exclusive(__popc(hole), sh.warp_sums, round);
        hole_at += round;
        for (int e = 0; e < 4; ++e)
            if (hole >> e & 1) copies[j++].y = p + e;
        j = move_at + block_exclusive(__popc(mover), sh.warp_sums, round);
        move_at += round;
        for (int e = 0; e < 4; ++e)
            if (mover >> e & 1) copies[j++].x = p + e;
            else if (p + e >= n && p + e < s.hi) name[p + e] = p + e;
    }
    cl.sync();
    for (int j = rank * kThreads + (int)threadIdx.x; j < pages; j += kCtas * kThreads) {
        if (j < holes) {
            const int2 p = copies[j];
            name[p.x] = p.y;
            refs[p.y] = refs[p.x];
            refs[p.x] = 0;
        } else {
            copies[j] = make_int2(-1, -1);
        }
    }
    if (rank == 0 && threadIdx.x == 0) {
        *count = holes;
        *n_live = n;
    }
}
// Table entries of the pages that moved (those from n_live on) get their new names.
__global__ void __launch_bounds__(256)
    rename_kernel(Table table, int pages, const int32_t *__restrict__ name, const int32_t *__restrict__ n_live,
                  uint32_t *status) {
    wait_before();
    let_next_start();
    const int n = *n_live;
    for (int r = blockIdx.x; r < table.rows; r += gridDim.x) {
        int32_t *row = table.row(r);
        for (int j = blockIdx.y * blockDim.x + threadIdx.x; j < table.cols; j += gridDim.y * blockDim.x) {
            const int pg = row[j];
            if (pg < n) continue;
            if (pg < pages) row[j] = name[pg];
            else if (status) atomicOr(status, kStatusBadSeqlens);
        }
    }
}

// ---- host -------------------------------------------------------------------------
cudaError_t launch_append(const void *k, const void *v, int64_t ldk, int64_t ldv, const int32_t *cu, int N, int T,
                          int64_t rows, const int32_t *index, const int32_t *count, const int32_t *start,
                          const int32_t *table, int64_t table_ld, int cols, int pages, int page, int Hkv, int es,
                          void *kp, void *vp, uint32_t *status, cudaStream_t stream) {
    const int piece_bits = es == 2 ? 4 : 5;  // 16-byte pieces of a head's row: 16 or 32
    const int64_t per = 16 / es;
    const Table t = {const_cast<int32_t *>(table), table_ld, N, cols};
    return launch_early(append_kernel, dim3((unsigned)((rows + kAppendWarps - 1) / kAppendWarps)), 32 * kAppendWarps, 0,
                        stream, static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), ldk / per, ldv / per, cu, N,
                        T, rows, index, count, start, t, pages, page, Hkv, piece_bits, static_cast<uint4 *>(kp),
                        static_cast<uint4 *>(vp), status);
}

cudaError_t launch_copy(void *const *pools, int n_pools, int64_t entry_bytes, int entries, const int32_t *pairs, int n,
                        const int32_t *count, int sms, cudaStream_t stream) {
    for (int at = 0; at < n_pools; at += kMaxPools) {
        Pools p = {};
        const int here = n_pools - at < kMaxPools ? n_pools - at : kMaxPools;
        for (int i = 0; i < here; ++i) p.base[i] = static_cast<uint4 *>(pools[at + i]);
        const int64_t entry = entry_bytes / 16, work = (entry + kCopyChunk - 1) / kCopyChunk * here * n;
        const int64_t most = (int64_t)sms * 8;
        const cudaError_t e = launch_early(copy_kernel, dim3((unsigned)(work < most ? work : most)), kCopyThreads, 0, stream,
                                           p, here, entry, entries, reinterpret_cast<const int2 *>(pairs), n, count);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

static dim3 table_grid(int rows, int cols) {  // about one entry per thread, within reason
    const int y = (cols + 255) / 256;
    return dim3((unsigned)rows, (unsigned)(y < 64 ? y : 64));
}

cudaError_t launch_free(int32_t *table, int64_t ld, int rows, int cols, int32_t *lens, int32_t *refs, int pages,
                        const int32_t *which, int n, uint32_t *status, cudaStream_t stream) {
    return launch_early(free_kernel, table_grid(n, cols), 256, 0, stream, Table{table, ld, rows, cols}, lens, refs, pages,
                        which, status);
}

cudaError_t launch_fork(int32_t *table, int64_t ld, int rows, int cols, int32_t *lens, int32_t *refs, int pages, int page,
                        const int32_t *src, const int32_t *dst, int n, int32_t *copies, int32_t *scratch,
                        uint32_t *status, cudaStream_t stream) {
    return launch_early(fork_kernel, dim3(kCtas), kThreads, 0, stream, Table{table, ld, rows, cols}, lens, refs, pages, page,
                        src, dst, n, reinterpret_cast<int2 *>(copies), scratch, scratch + pages, status);
}

cudaError_t launch_alloc(int32_t *table, int64_t ld, int rows, int cols, const int32_t *want, int32_t *refs, int pages,
                         int page, int32_t *scratch, uint32_t *status, cudaStream_t stream) {
    return launch_early(alloc_kernel, dim3(kCtas), kThreads, 0, stream, Table{table, ld, rows, cols}, want, refs, pages,
                        page, scratch + 2 * (int64_t)rows, reinterpret_cast<int2 *>(scratch), status);
}

cudaError_t launch_compact(int32_t *table, int64_t ld, int rows, int cols, int32_t *refs, int pages, int32_t *copies,
                           int32_t *count, int32_t *scratch, uint32_t *status, cudaStream_t stream) {
    cudaError_t e = launch_early(compact_kernel, dim3(kCtas), kThreads, 0, stream, refs, pages,
                                 reinterpret_cast<int2 *>(copies), count, scratch + 4, scratch);
    if (e != cudaSuccess || rows == 0 || cols == 0) return e;
    return launch_early(rename_kernel, table_grid(rows < 65535 ? rows : 65535, cols), 256, 0, stream,
                        Table{table, ld, rows, cols}, pages, static_cast<const int32_t *>(scratch + 4),
                        static_cast<const int32_t *>(scratch), status);
}

}  // namespace cache
}  // namespace kda
