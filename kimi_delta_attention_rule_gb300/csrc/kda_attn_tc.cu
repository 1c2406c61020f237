// Softmax attention in bf16 on the tensor cores: causal attention over packed
// prompts, and attention of new (drafted) tokens over a paged cache.
//
//   s_ij = scale q_i . k_j,  o_i = sum_j e^{s_ij - m_i} v_j / l_i,
//   m_i = max_j s_ij (kept in fp32, over the keys seen so far),
//   l_i = sum_j e^{s_ij - m_i} (fp32)
//
// in one pass over the keys. A CTA holds two row tiles of 128 (token, head of the
// group) rows, its streams: S = Q K^T and O += P V run as M128 N128 tcgen05.mma
// with S, P and O in TMEM (S 2 x 128 columns, P over S, O 2 x 128). Roles of the
// 12 warps: 8 softmax warps (216 registers, four to a stream), one that issues the
// products, one that fills a ring of 128-key K and V tiles by TMA, one that walks the
// CTA's parts ahead of the others, one that zeroes V rows past a sequence's end. While
// one stream forms P from its S, the tensor core runs the other's products.
//
// Each softmax thread owns one row (a TMEM lane), so no row statistic ever crosses
// threads. Per stream S, P and the products form one serial chain, which is what
// bounds the kernel: so P goes to the tensor core in two parts (96 keys' products run
// while the last 32 keys' exponentials do), and a part's first Q K^T
// follows the last P V of the part before it, under that part's epilogue. O is
// rescaled only when a row's maximum grows by more than 2^8: P is then 2^8 at most, far
// inside the range of bf16 (to which it is rounded, 2^-8 of it at most, for the product),
// and l sums the unrounded terms in fp32.
// With at most 128 rows per kv head (decode) both streams take the same row tile
// and alternate key tiles; their results are joined at the end (DUAL).
//
// Measured (GB300; copy 6,782 GB/s, cuBLAS bf16 1,917 TFLOP/s): causal attention of 8,192
// tokens, 32 heads on 8: 320 us, 1,718 TFLOP/s in a short run in a graph, 355 us in calls back to
// back (at the power cap); the tensor pipe is busy 74 % of the time and the
// exponentials' 37 %; a step of two row tiles takes some 2,700 cycles, 2,048 of them products.
// One token each of 128 sequences, 400,003 cached tokens: 251 us, 6.5 TB/s (loads).
// Through a window (instances of their own): 15,001 tokens behind 1,383, window 4,096: 570 us in a graph, 1.66
// PFLOP/s of visible keys; 128 sequences, window 1,024: 96.5 us, 5.4 TB/s, as caches of that length. Some
// 11,000 cycles pass before the first softmax (5,500 of a direct call): the search for the
// CTA's work, the page's number, the first tile, each from a cold cache. Tried without gain: 16
// softmax warps of two threads a row (spills), halves of 64 keys with a maximum ahead of
// the second (340 us instead of 328), a third of the exponentials as polynomials (344 to 357
// instead of 335), more Q tiles and fewer K tiles in the ring (458 instead of 425 for a long prefix), one fused step of both
// products per vote of the issuing warp (no change).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_attn.cuh"
#include "kda_common.cuh"
#include "kda_tcgen05.cuh"
#include "kda_tensormap.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace attn {

constexpr int kSoftmaxWarps = 8;
constexpr int kWarpMma = 8, kWarpTma = 9, kWarpSched = 10, kWarpFix = 11;
constexpr int kThreads = 384;
constexpr int kMinPart = kTcMinPart;
constexpr int kTile = 128;      // rows of a row tile, keys of a key tile
constexpr uint32_t kTileBytes = 32768;  // 128 rows x 128 channels bf16, two 64-channel halves
constexpr uint32_t kHalf = 16384;
constexpr long long kWaitNs = 2000000000, kTestWaitNs = 20000000;
constexpr float kRescale = 8.f;  // log2 growth of a maximum that rescales O
constexpr int kJobRing = 8;  // more than the ring has slots: a job holds its slot until it is done

constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: S/P of stream s at 128 s, O at 256 + 128 s

struct Maps {
    CUtensorMap q, k, v, kn, vn, out;
    CUtensorMap k16, v16;  // prefill through a window: 16 rows at a time, for tiles of sinks and others
};

// A part as the roles need it, in shared memory.
constexpr int kDescs = 4;
struct Desc {
    int last;              // no further part
    int n, h, q0, k0, Lk;
    int first_tok;         // the item's first token within its sequence
    int ta, nt;            // the part's first tile; tiles of the item
    int whole, slot;       // the part is the item; else its workspace slot
    int open;              // the item goes on in the next CTA
    int writer;            // DUAL: the stream with the first tile, which joins and writes
    int seen;              // prefill: keys that the item's first token sees; decode: cached keys
    int q[2];              // running number of each stream's Q tile
    int count[2];          // key tiles of each stream
    int start[2];          // its first tile (DUAL: every second from there)
    int tokens[2];         // valid tokens of its row tile
    Span span;             // WIN
};

// Shared memory: two Q tiles of RT rows, 32 KB for the way out (DUAL: the box for the
// join of the two streams, RT rows x 64 channels fp32, and the rows are staged in the
// Q tile; else both streams stage there, and their Q tiles are free for the next part
// once the last Q K^T is through), the ring of K and V tiles, barriers, descriptors.
// With RT = 32 (a decode step's rows, as a rule) the ring has six tiles: 192 KB in
// flight instead of 128 hide the latency of a chain of short sequences (128 of 500 tokens:
// 66.6 us instead of 72.6 when it was taken; of 3,125: 255 instead of 250). The products
// read 128 rows of Q all the same; what lies behind the tile gives rows of S and O
// that nobody looks at.
template <bool DUAL, int RT>
struct Smem {
    static constexpr int kQs = 2, kRing = RT == 32 ? 6 : 4;
    static constexpr uint32_t kQTile = RT * 256, kQHalf = RT * 128;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kJoin = kQs * kQTile;   // DUAL only
    static constexpr uint32_t kStage = kQs * kQTile;  // not DUAL: 64 channels of each stream's row tile
    static constexpr uint32_t kKv = 3 * kQTile;
    static constexpr uint32_t kBars = kKv + kRing * kTileBytes;
    static constexpr uint32_t kMl = kBars + 1024;  // DUAL: the second stream's m and l
    static constexpr uint32_t kBytes = kMl + (DUAL ? 1024 : 0);
};

struct Bars {  // shared-memory addresses
    uint32_t base;
    __device__ uint32_t qfull(int i) const { return base + 8 * i; }
    __device__ uint32_t qempty(int i) const { return base + 32 + 8 * i; }
    __device__ uint32_t sfull(int s) const { return base + 64 + 8 * s; }
    __device__ uint32_t pready(int s, int half) const { return base + 80 + 16 * half + 8 * s; }
    __device__ uint32_t ofull(int s) const { return base + 112 + 8 * s; }
    __device__ uint32_t kvfull(int i) const { return base + 128 + 8 * i; }
    __device__ uint32_t kvempty(int i) const { return base + 176 + 8 * i; }
    __device__ uint32_t vraw(int i) const { return base + 224 + 8 * i; }
    __device__ uint32_t dfull(int i) const { return base + 272 + 8 * i; }
    __device__ uint32_t dempty(int i) const { return base + 304 + 8 * i; }
    __device__ uint32_t jfull(int i) const { return base + 336 + 8 * i; }
    static constexpr uint32_t kTmem = 400;
    static constexpr uint32_t kDead = 404;  // a role gave up
    static constexpr uint32_t kJobs = 408;  // kJobRing times (slot, valid rows)
    static constexpr uint32_t kEnd = 472;   // Point: the end of the CTA's work
    static constexpr uint32_t kEarly = 488;  // the next CTA's early part is there
    static constexpr uint32_t kDesc = 496;  // kDescs descriptors
    // Between the softmax warps, at a part's end. (As mbarriers: a named barrier waits
    // without a limit for a warp that has given up. But see hand_over.)
    static constexpr uint32_t kPartEnd = 880;
    __device__ uint32_t early() const { return base + kPartEnd; }          // kEarly is written
    __device__ uint32_t drained() const { return base + kPartEnd + 8; }    // all products are through
    __device__ uint32_t stage_free(int s) const { return base + kPartEnd + 16 + 8 * s; }  // twice a staged part
    __device__ uint32_t staged(int s) const { return base + kPartEnd + 32 + 8 * s; }      // likewise
    static constexpr uint32_t kGone = 928;  // DUAL, four quads: a warp of these rows has given up
};
static_assert(Bars::kDesc + kDescs * sizeof(Desc) <= Bars::kPartEnd && Bars::kGone + 16 <= 1024, "barrier area");

// shared memory (128-byte swizzle) to global; the issuing thread's bulk group
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, int c0, int c1, int c2, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(m),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// A bounded wait: true once the phase is through, false after `NS` nanoseconds (two
// seconds). (The clock is read once in 1024 tries: a read takes as long as much of what is
// waited for. Written out, since it stands in many places and all code here is fetched cold.)
template <long long NS>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n, r;\n .reg .u64 t0, t;\n"
        " mov.u32 n, 0;\n mov.u64 t0, 0;\n"
        "WAIT:\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " @p bra DONE;\n"
        " add.u32 n, n, 1;\n and.b32 r, n, 1023;\n setp.ne.u32 q, r, 0;\n @q bra WAIT;\n"
        " mov.u64 t, %%globaltimer;\n"
        " setp.eq.u64 q, t0, 0;\n @q mov.u64 t0, t;\n"
        " sub.u64 t, t, t0;\n setp.lt.u64 q, t, %3;\n @q bra WAIT;\n"
        "DONE:\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(NS)
        : "memory");
    return ok != 0;
}
// whether a phase is through, without waiting
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// a wait of a whole warp, which leaves it converged
template <long long NS>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait<NS>(bar, parity));
}
// DUAL: the two warps of the same 32 rows meet, four times a joined part. (A named barrier:
// with mbarriers here 128 sequences of 500 tokens take 72.5 us instead of 69.6.) Such a barrier
// waits for both, so it must not wait for a warp that is gone: a warp gives up only ahead of
// a part's first meeting, and as it leaves it says so in kGone and arrives (hand_over_gone)
// for that one. Its partner, should it come there, looks at kGone after the first meeting of a
// part, and leaves too.
__device__ __forceinline__ void hand_over(int quad) { asm volatile("barrier.sync %0, 64;\n" ::"r"(1 + quad) : "memory"); }
__device__ __forceinline__ void hand_over_gone(int quad) {
    asm volatile("barrier.arrive %0, 64;\n" ::"r"(1 + quad) : "memory");
}
// z = z f + y g
__device__ __forceinline__ void join4(uint32_t *z, float f, float4 y, float g) {
    z[0] = __float_as_uint(join_sum(__uint_as_float(z[0]), f, y.x, g));
    z[1] = __float_as_uint(join_sum(__uint_as_float(z[1]), f, y.y, g));
    z[2] = __float_as_uint(join_sum(__uint_as_float(z[2]), f, y.z, g));
    z[3] = __float_as_uint(join_sum(__uint_as_float(z[3]), f, y.w, g));
}

// The scheduler's state over a CTA's parts: Q tiles and (DUAL) key tiles so far.
struct Run {
    int q, tiles;
};
template <bool PAGED, bool DUAL, bool WIN>
__device__ __forceinline__ void describe(const Args &a, const Part &p, int cta, Run &run, Desc &d) {
    d.last = 0;
    d.n = p.n;
    d.h = p.h;
    d.q0 = p.q0;
    d.k0 = p.k0;
    d.Lk = p.Lk;
    d.first_tok = p.first_tok;
    d.ta = p.ta;
    d.nt = p.nt;
    d.whole = p.whole();
    d.slot = part_slot(cta, p);
    d.open = p.tb < p.nt;
    d.writer = DUAL ? run.tiles & 1 : 0;
    d.seen = PAGED ? p.Lk : p.Lk - p.Lq + p.first_tok + 1;
    if (WIN) d.span = p.span;
    if (DUAL) {  // tiles alternate between the streams, across parts too
        const int tiles = p.tb - p.ta;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int second = s != d.writer;
            d.tokens[s] = p.tokens;
            d.count[s] = (tiles + 1 - second) / 2;
            d.start[s] = p.ta + second;
            d.q[s] = run.q;
        }
        run.tiles += tiles;
        run.q += tiles > 0;
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int left = p.tokens - s * a.tile_tokens;
            const int tokens = left < 0 ? 0 : (left < a.tile_tokens ? left : a.tile_tokens);
            int end = p.tb;
            if (!PAGED) {  // the keys that the row tile's last token sees
                const int seen = d.seen + s * a.tile_tokens + tokens - 1;
                const int nt = seen <= 0 ? 0 : (int)(((unsigned)(WIN ? seen - p.span.shift : seen) + kTile - 1) / kTile);
                end = end < nt ? end : nt;
            }
            d.tokens[s] = tokens;
            d.count[s] = tokens == 0 || end < p.ta ? 0 : end - p.ta;
            d.start[s] = p.ta;
            d.q[s] = run.q;
            run.q += d.count[s] > 0;
        }
    }
}

// The rows of an item that see no key: zeros, and -inf. A converged warp.
__device__ __forceinline__ void write_nothing(const Args &a, const Part &p) {
#pragma unroll 1
    for (int t = 0; t < p.tokens; ++t) {
        const size_t row = (size_t)(p.q0 + t) * a.Hq + p.h * a.G;
#pragma unroll 1
        for (int x = threadIdx.x & 31; x < a.G * 16; x += 32) {  // 16 pieces of a row
            static_cast<uint4 *>(a.out)[row * 16 + x] = make_uint4(0, 0, 0, 0);
            if (a.lse != nullptr && x < a.G) a.lse[row + x] = -INFINITY;
        }
    }
}

// Every wait has a limit. A role whose wait runs out goes to the kernel's end, the others
// follow as theirs run out or they see kDead, and the status tells; the copies and products
// in flight are waited for first. TEST (kda_testing_attn_*): waits of 20 ms, and warp
// a.lose - 1 gives up at its wait number a.lose_at.
template <bool PAGED, bool DUAL, int RT, bool WIN, bool TEST>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
    using L = Smem<DUAL, RT>;
    constexpr long long kLimit = TEST ? kTestWaitNs : kWaitNs;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_u32(sm);
    const Bars bars{base + L::kBars};
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int cta = blockIdx.x;
    if (base & 1023u) {  // (the swizzled tiles need it)
        if (tid == 0) atomicOr(status_word(a), kStatusTimeout);
        return;
    }

    Point p0;
    Seq s0;
    bool any = false;
    if (warp == kWarpSched || warp == kWarpFix) {  // where this CTA's work starts; kWarpFix: where it ends
        const int end = warp == kWarpFix;
        wait_before();
        if (!a.direct) {
            any = split_point<PAGED, kTile, WIN>(a, cta + end, p0, s0) && p0.n < a.N;
            if (end && lane == 0) {
                *reinterpret_cast<Point *>(sm + L::kBars + Bars::kEnd) = p0;
                part_header(a, 2 * cta)->valid = 0;
                part_header(a, 2 * cta + 1)->valid = 0;
            }
        }
    } else if (warp == kWarpTma) {
        if (lane == 0) {
            for (int i = 0; i < L::kQs; ++i) {
                tc::mbar_init(bars.qfull(i), 1);
                tc::mbar_init(bars.qempty(i), DUAL ? 4 : 1);  // DUAL: the writer's warps; else the products
            }
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(bars.sfull(i), 1);
                tc::mbar_init(bars.pready(i, 0), 4);
                tc::mbar_init(bars.pready(i, 1), 4);
                tc::mbar_init(bars.ofull(i), 1);
            }
            for (int i = 0; i < L::kRing; ++i) {
                tc::mbar_init(bars.kvfull(i), 1);
                tc::mbar_init(bars.kvempty(i), 1);
                tc::mbar_init(bars.vraw(i), 1);
            }
            for (int i = 0; i < kDescs; ++i) {
                tc::mbar_init(bars.dfull(i), 1);
                tc::mbar_init(bars.dempty(i), kSoftmaxWarps + 2);  // and TMA, MMA
            }
            for (int i = 0; i < kJobRing; ++i) tc::mbar_init(bars.jfull(i), 1);
            tc::mbar_init(bars.drained(), 1);
            if (DUAL) {
                *reinterpret_cast<int4 *>(sm + L::kBars + Bars::kGone) = make_int4(0, 0, 0, 0);
            } else {
                tc::mbar_init(bars.early(), 1);
                for (int i = 0; i < 2; ++i) {
                    tc::mbar_init(bars.stage_free(i), 1);
                    tc::mbar_init(bars.staged(i), 4);
                }
            }
            *reinterpret_cast<int *>(sm + L::kBars + Bars::kDead) = 0;
            tc::fence_mbar_init();
        }
    } else if (warp == kWarpMma) {
        tc::tmem_alloc(bars.base + Bars::kTmem, 512);
        tc::tmem_relinquish();
        if (lane == 0) {
            prefetch_map(&maps.q);
            prefetch_map(&maps.k);
            prefetch_map(&maps.v);
            if (PAGED && a.has_new) {
                prefetch_map(&maps.kn);
                prefetch_map(&maps.vn);
            }
        }
    }
    wait_before();
    // (Blocks of the join kernel that wait on SMs whose work is done first cost the others 1 us of
    // 51 for one long sequence; a direct call has none, and the next call may start.)
    if (a.direct) let_next_start();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *reinterpret_cast<uint32_t *>(sm + L::kBars + Bars::kTmem);
    const Desc *const descs = reinterpret_cast<const Desc *>(sm + L::kBars + Bars::kDesc);
    volatile int *const dead = reinterpret_cast<volatile int *>(sm + L::kBars + Bars::kDead);
    volatile int *const early_there = reinterpret_cast<volatile int *>(sm + L::kBars + Bars::kEarly);
    bool alive = true;
    uint32_t nd = 0;  // descriptors taken
    int waits = 0;
    auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if constexpr (TEST) {
            if (warp == a.lose - 1 && waits++ >= a.lose_at) return false;
        }
        return wait_warp<kLimit>(bar, parity);
    };
    // a wait that may last for a whole part: limited too, and ends when another role gives up
    auto long_wait = [&](uint32_t bar, uint32_t parity) -> bool {
        for (int i = 0; i < 100; ++i) {
            if (warp_wait(bar, parity)) return true;
            if (*dead) return false;
        }
        return false;
    };
    // the next descriptor (NULL: no further part, or a wait ran out)
    auto next_desc = [&]() -> const Desc * {
        alive = warp_wait(bars.dfull(nd % kDescs), (nd / kDescs) & 1);
        const Desc *d = descs + nd % kDescs;
        return alive && !d->last ? d : nullptr;
    };

    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
        // ---- softmax warps: thread = row (TMEM lane) ---------------------------------
        const int s = warp >> 2, quad = warp & 3, r = 32 * quad + lane;
        const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
        const uint32_t tS = tl + kColS + 128 * s, tO = tl + kColO + 128 * s;
        const uint32_t inv_g = (65536u + a.G - 1) / a.G;  // x / G = x inv_g >> 16, exact for x < 1024
        const int tok = (int)(r * inv_g >> 16), g = r - tok * a.G;
        const float c = a.scale * kLog2e;
        volatile int *const gone = reinterpret_cast<volatile int *>(sm + L::kBars + Bars::kGone);
        uint32_t ns = 0, no = 0;
        while (const Desc *d = next_desc()) {
            const int steps = d->count[s];
            const bool row_ok = tok < d->tokens[s];
            const bool warp_ok = __any_sync(0xffffffffu, row_ok);
            float m = -INFINITY, l = 0.f;
            unsigned long long bits = 0;
            int fresh = 1;  // WIN: the new tokens that it sees, itself counted in any case
            if (PAGED && row_ok) {
                const int t = d->first_tok + (DUAL ? 0 : s * a.tile_tokens) + tok;
                bits = a.mask != nullptr ? a.mask[(size_t)d->n * a.T + t]
                                         : (t >= 63 ? ~0ull : (2ull << t) - 1);
                if (WIN) {
                    if (a.T < 64) bits &= (1ull << a.T) - 1;
                    fresh = __popcll(bits | 1ull << t);
                }
            }
            // keys that the row tile's first row and this row see
            const int seen0 = d->seen + (PAGED ? 0 : s * a.tile_tokens);
            const int seen = PAGED ? seen0 : seen0 + tok;
            const int draft_tile = PAGED && a.has_new ? d->nt - 1 : -1;
            // WIN: where this row's window starts, and where the last one of the row tile does (decode: at
            // most), among the item's keys; so are `seen` and `seen0` from there on
            const int shift = WIN ? d->span.shift : 0;
            const int from = WIN ? window_start(a, PAGED && a.has_new ? seen + fresh : seen) - shift : 0;
            const int from_last = WIN ? window_start(a, seen0 + (PAGED ? a.has_new * a.T : d->tokens[s] - 1)) - shift : 0;
            int t = d->start[s];
            for (int j = 0; j < steps; ++j, t += DUAL ? 2 : 1) {
                if (!warp_wait(bars.sfull(s), ns++ & 1)) {
                    alive = false;
                    break;
                }
                tc::fence_after_sync();
                if (warp_ok) {
                    uint32_t x[8][16];
                    tc::tmem_ld_cols<8>(tS, x);
                    const bool drafts = PAGED && t == draft_tile;
                    const int t0 = t * kTile;  // the tile's first key
                    if (drafts || seen0 - shift < t0 + kTile || (WIN && from_last > t0 && a.sinks - kTile < t0)) {
                        // the keys that this row sees, a bit each
                        if (PAGED && drafts && a.T < 64) bits &= (1ull << a.T) - 1;
                        const int lim = seen - shift - t0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            auto below = [&](int n) { return __funnelshift_lc(~0u, 0u, (uint32_t)max(n - 32 * i, 0)); };  // (by 32 at most)
                            uint32_t see = below(lim);
                            if (WIN) see &= ~below(from - t0) | below(a.sinks - t0);
                            if (PAGED && drafts) see = i == 0 ? (uint32_t)bits : (i == 1 ? (uint32_t)(bits >> 32) : 0u);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see >> e & 1)) x[2 * i + e / 16][e % 16] = 0xff800000u;
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kTile; i += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(x[i / 16][i % 16 + e]),
                                                       __uint_as_float(x[i / 16][i % 16 + 4 + e])));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (j == 0) {
                        m = top;
                    } else {
                        // (-inf - -inf is NaN: not greater, no rescale. Rows past the tile's own
                        // hold anything: they have no say, or the bits would depend on it.)
                        const bool grow = row_ok && (top - m) * c > kRescale;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float up = fmaxf(m, top);
                            const float f = m == -INFINITY ? 0.f : ex2((m - up) * c);
                            m = up;
                            l *= f;
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                uint32_t o[1][16];
                                tc::tmem_ld_cols<1>(tO + 16 * q, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    o[0][i] = __float_as_uint(f * __uint_as_float(o[0][i]));
                                tc::tmem_st16u(tO + 16 * q, o[0]);
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int k = 32 * q + 2 * i;
                            float2 y = make_float2(__uint_as_float(x[k / 16][k % 16]),
                                                   __uint_as_float(x[k / 16][k % 16 + 1]));
                            y = fma2(y, c2, mc2);
                            y.x = ex2(y.x);
                            y.y = ex2(y.y);
                            sum[i & 1] = add2(sum[i & 1], y);
                            w[i] = pack_bf16(y.x, y.y);
                        }
                        tc::tmem_st16u(tS + 16 * q, w);
                        if (q == 2) {  // the products of the first 96 keys may start
                            tc::tmem_wait_st();
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bars.pready(s, 0));
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc::tmem_wait_st();
                } else if (lane == 0) {
                    mbar_arrive(bars.pready(s, 0));
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.pready(s, 1));
            }
            if (!alive) break;
            // ---- the part's end ----
            const int others = d->count[1 - s];
            bool early = false;  // the next CTA has the item's last part ready
            if (!DUAL && d->open) {
                if (tid == 0) {
                    uint32_t flags;
                    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(flags) : "l"(early_flag(a, cta + 1)) : "memory");
                    *early_there = flags >> ((cta + 1) & 31) & 1;
                    if (*early_there) {
                        PartHeader *const h = part_header(a, d->slot);
                        if (d->ta == 0) h->valid = 0;
                        else h->ends = kEndsJoined;
                    }
                    mbar_arrive(bars.early());
                }
                if (!(alive = warp_wait(bars.early(), 0))) break;  // (the last part of a CTA)
                early = *early_there != 0;
            }
            const bool whole = d->whole || (early && d->ta == 0);
            // the stage is free when its last copy has read it (seen to before O is there)
            const bool staged = !DUAL && whole && (steps > 0 || early), leader = quad == 0 && lane == 0;
            if (staged) {
                if (leader) {
                    tc::bulk_wait_read();
                    mbar_arrive(bars.stage_free(s));
                }
                if (!(alive = warp_wait(bars.stage_free(s), 0))) break;
            }
            const float *const next_o = part_o(a, 2 * (cta + 1));
            if (steps > 0) {
                if (!warp_wait(bars.ofull(s), no++ & 1)) {
                    alive = false;
                    break;
                }
                tc::fence_after_sync();
            }
            const bool writer = !DUAL || s == d->writer, joins = DUAL && steps > 0 && others > 0;
            if ((warp_ok || staged) && (writer || joins)) {
                // In two parts of 64 channels: O from TMEM; the second stream of a join
                // hands it over in shared memory; the writer stores the sum, or stages it
                // for whole rows to leave together.
                float4 *const box = reinterpret_cast<float4 *>(sm + L::kJoin) + r;
                float2 *const box_ml = reinterpret_cast<float2 *>(sm + L::kMl) + r;
                const int q0 = d->q0 + (DUAL ? 0 : s * a.tile_tokens), row0 = d->h * a.G;
                // A full row tile goes out by tensor copies, in the layout of Q; the rows of a
                // short one (next to them may lie another sequence's) by the warps.
                const bool full = !DUAL && d->tokens[s] == a.tile_tokens;
                const uint32_t stage_at = DUAL ? L::kQ + d->q[s] % L::kQs * L::kQTile : L::kStage + s * kHalf;
                unsigned char *const stage = sm + stage_at;
                const int rows = d->tokens[s] * a.G;
                __nv_bfloat16 *const out = static_cast<__nv_bfloat16 *>(a.out);
                auto write_lse = [&]() {
                    if (whole && row_ok && a.lse != nullptr)
                        a.lse[(size_t)(q0 + tok) * a.Hq + row0 + g] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
                };
                float f = 1.f, f1 = 0.f;
#pragma unroll 1
                for (int p = 0; p < 2; ++p) {
                    if (!DUAL && p == 1) write_lse();  // (while the first half's copy reads the stage)
                    uint32_t o[4][16] = {};
                    if (steps > 0) tc::tmem_ld_cols<4>(tO + 64 * p, o);
                    if (!writer) {
                        if (p == 0) *box_ml = make_float2(m, l);
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            box[RT * q] = make_float4(
                                __uint_as_float(o[q / 4][4 * (q % 4)]), __uint_as_float(o[q / 4][4 * (q % 4) + 1]),
                                __uint_as_float(o[q / 4][4 * (q % 4) + 2]), __uint_as_float(o[q / 4][4 * (q % 4) + 3]));
                        hand_over(quad);  // handed over
                        if (p == 0 && gone[quad] != 0) {
                            alive = false;
                            break;
                        }
                        hand_over(quad);  // taken
                        continue;
                    }
                    if (joins) {
                        hand_over(quad);
                        if (p == 0 && gone[quad] != 0) {
                            alive = false;
                            break;
                        }
                        if (p == 0) {
                            const float2 ml = *box_ml;
                            const float2 fs = join_factors(m, ml.x, c);
                            f = fs.x;
                            f1 = fs.y;
                            m = fmaxf(m, ml.x);
                            l = join_sum(l, f, ml.y, f1);
                        }
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float4 y = box[RT * q];
                            uint32_t *z = &o[q / 4][4 * (q % 4)];
                            join4(z, f, y, f1);
                        }
                        hand_over(quad);
                    }
                    if (!DUAL && early && row_ok) {
                        const float4 *const y4 = reinterpret_cast<const float4 *>(next_o) + 128 * s + r;
                        if (p == 0) {
                            const float2 ml = __ldcg(part_ml(a, 2 * (cta + 1)) + 128 * s + r);
                            const float2 fs = join_factors(m, ml.x, c);
                            f = fs.x;
                            f1 = fs.y;
                            m = fmaxf(m, ml.x);
                            l = join_sum(l, f, ml.y, f1);
                        }
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            join4(&o[q / 4][4 * (q % 4)], f, __ldcg(y4 + (size_t)(16 * p + q) * a.part_rows), f1);
                    }
                    if (!whole) {
                        if (row_ok) {
                            float4 *o4 = reinterpret_cast<float4 *>(part_o(a, d->slot)) + (DUAL ? r : 128 * s + r);
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                o4[(size_t)(16 * p + q) * a.part_rows] = make_float4(
                                    __uint_as_float(o[q / 4][4 * (q % 4)]), __uint_as_float(o[q / 4][4 * (q % 4) + 1]),
                                    __uint_as_float(o[q / 4][4 * (q % 4) + 2]), __uint_as_float(o[q / 4][4 * (q % 4) + 3]));
                        }
                        continue;
                    }
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    if (steps == 0 && !early) {  // rows that see nothing (no Q tile is theirs): zeros
                        if (row_ok) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                                   ((size_t)(q0 + tok) * a.Hq + row0 + g) * kD + 64 * p);
#pragma unroll
                            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
                        }
                        continue;
                    }
                    if (!DUAL && p == 1) {
                        if (leader) {
                            tc::bulk_wait_read();
                            mbar_arrive(bars.stage_free(s));
                        }
                        if (!(alive = warp_wait(bars.stage_free(s), 1))) break;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16(inv * __uint_as_float(o[i / 2][8 * (i % 2) + 2 * e]),
                                             inv * __uint_as_float(o[i / 2][8 * (i % 2) + 2 * e + 1]));
                        const int at = DUAL ? r * 256 + (((8 * p + i) ^ (r & 15)) * 16) : r * 128 + ((i ^ (r & 7)) * 16);
                        *reinterpret_cast<uint4 *>(stage + at) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (DUAL) continue;
                    // The stream's four warps have staged their rows (short tile: and are done with
                    // them): the leader waits for that before it frees the stage again.
                    auto all_staged = [&]() -> bool {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bars.staged(s));
                        return quad != 0 || warp_wait(bars.staged(s), p);
                    };
                    if (full) {
                        tc::fence_async_smem();
                        if (!(alive = all_staged())) break;
                        if (leader) {
                            tma_store_3d(&maps.out, 64 * p, row0, q0, base + stage_at);
                            tc::bulk_commit();
                        }
                    } else {
                        __syncwarp();
                        const int ch = lane & 7;  // eight lanes write 128 bytes of a row
#pragma unroll 4
                        for (int i = 0; i < 32; i += 4) {
                            const int row = 32 * quad + i + (lane >> 3), tk = (int)(row * inv_g >> 16);
                            const uint4 y = *reinterpret_cast<const uint4 *>(stage + row * 128 + ((ch ^ (row & 7)) * 16));
                            if (row < rows)
                                reinterpret_cast<uint4 *>(out + ((size_t)(q0 + tk) * a.Hq + row0 + (row - tk * a.G)) * kD + 64 * p)[ch] = y;
                        }
                        if (!(alive = all_staged())) break;
                    }
                }
                if (!alive) break;
                if (writer && !whole) {
                    if (row_ok) part_ml(a, d->slot)[DUAL ? r : 128 * s + r] = make_float2(m, l);
                } else if (writer) {
                    if (DUAL) write_lse();
                    if (DUAL && steps > 0) {
                        __syncwarp();
                        const int ch = lane & 15;  // sixteen lanes write a row's 256 bytes
#pragma unroll 4
                        for (int i = 0; i < 32; i += 2) {
                            const int row = 32 * quad + i + (lane >> 4), tk = (int)(row * inv_g >> 16);
                            if (32 * quad + i >= rows) break;
                            const uint4 y = *reinterpret_cast<const uint4 *>(stage + row * 256 + ((ch ^ (row & 15)) * 16));
                            if (row < rows)
                                reinterpret_cast<uint4 *>(out + ((size_t)(q0 + tk) * a.Hq + row0 + (row - tk * a.G)) * kD)[ch] = y;
                        }
                    }
                }
            }
            // O is read: the MMA warp's next P V waits for this warp's next P.
            // DUAL: the Q tile (the staging's too) goes back to the TMA warp.
            tc::fence_before_sync();
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (DUAL && steps > 0 && writer) mbar_arrive(bars.qempty(d->q[s] % L::kQs));
                mbar_arrive(bars.dempty(nd % kDescs));
            }
            ++nd;
        }
        if (DUAL && !alive && __all_sync(0xffffffffu, gone[quad] == 0)) {
            if (lane == 0) gone[quad] = 1;
            __syncwarp();
            hand_over_gone(quad);
        }
        if (lane == 0) tc::bulk_wait_all();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
        if (warp == kWarpSched) {
            // ---- scheduler warp: walks the CTA's parts ahead of the others ------------
            Part p;
            Walk<PAGED, kTile, WIN> walk;
            if (any && !a.direct) walk.init(p0, *reinterpret_cast<const Point *>(sm + L::kBars + Bars::kEnd), s0);
            Run run = {0, 0};
            bool todo = a.direct ? direct_part<PAGED, kTile, WIN>(a, cta, p) : any;
            bool tells = false;  // the CTA before may take the first part
            auto tell = [&]() {  // (its descriptor is back: all of it is written)
                if (tells && lane == 0)
                    asm volatile("red.release.gpu.global.or.b32 [%0], %1;\n" ::"l"(early_flag(a, cta)), "r"(1u << (cta & 31))
                                 : "memory");
            };
            while (true) {
                const bool more = todo && (a.direct || walk.next(a, p));
                todo = more && !a.direct;
                // Items that see nothing get their rows here. As descriptors they would stop all: a part's
                // last P V runs with the next part's first Q K^T, which would lie behind more of them than
                // there are descriptors, and these come back in order.
                if (more && p.nt == 0) {
                    write_nothing(a, p);
                    continue;
                }
                if (nd == 0) tells = !DUAL && more && p.ta > 0 && p.tb == p.nt;
                if (nd >= kDescs && !(alive = long_wait(bars.dempty(nd % kDescs), (nd / kDescs - 1) & 1))) break;
                if (nd == kDescs) tell();
                if (lane == 0) {
                    Desc *d = const_cast<Desc *>(descs) + nd % kDescs;
                    // The others wait for the descriptor: the header of a part comes after it,
                    // but ahead of it where the softmax warps may change it at the part's end.
                    const bool open = more && p.tb < p.nt;
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        if ((k == 0) != open) {
                            if (more) describe<PAGED, DUAL, WIN>(a, p, cta, run, *d);
                            else d->last = 1;
                            mbar_arrive(bars.dfull(nd % kDescs));
                        } else if (more && !p.whole()) {
                            PartHeader *h = part_header(a, part_slot(cta, p));
                            h->ends = open ? 0 : kEnds;
                            h->token0 = p.q0;
                            h->tokens = p.tokens;
                            h->kvh = p.h;
                            h->valid = 1;
                        }
                    }
                }
                ++nd;
                if (!more) break;
            }
            if (tells && alive && nd <= kDescs) {
                alive = long_wait(bars.dempty(0), 0);
                if (alive) tell();
            }
        } else if (warp == kWarpTma) {
            // ---- TMA warp ------------------------------------------------------
            // K tile g, then V tile g - kLag: in the order in which the products take
            // them, through the ends of parts.
            constexpr int kLag = DUAL ? 2 : 1;
            struct Load {
                int n, h, k0, Lk, t, draft, pg;
                Span span;
            };
            uint32_t kv = 0, jobs = 0, g = 0;
            uint32_t sent = 0;  // bit i: the parity of Q slot i's copies
            const uint32_t qbytes = (uint32_t)(a.tile_tokens * a.G) * 256u;
            const int rows = a.page < kTile ? a.page : kTile;  // decode: rows of one copy
            const int row_bits = 31 - __clz(rows), page_bits = 31 - __clz(a.page);
            const uint32_t lead = tc::elect_one();
            // decode: the page of this lane's copy of tile t
            auto page_of = [&](const Span &span, int n, int Lk, int t) -> int {
                const int v = t * kTile + (lane << row_bits), pos = WIN ? span.key(v) : v;
                if (!PAGED || (lane << row_bits) >= kTile || pos >= Lk) return -1;
                return __ldg(a.table + (size_t)n * a.table_ld + (pos >> page_bits));
            };
            auto load = [&](const Load x, bool is_v) {
                const uint32_t slot = kv % L::kRing;
                const uint32_t dst = base + L::kKv + slot * kTileBytes;
                if (kv >= (uint32_t)L::kRing && !warp_wait(bars.kvempty(slot), (kv / L::kRing - 1) & 1)) {
                    alive = false;
                    return;
                }
                ++kv;
                // rows of this tile that are the sequence's own
                const int t0 = x.t * kTile, first = WIN && t0 >= x.span.sinks ? t0 + x.span.shift : t0;  // the tile's first key
                const int left = x.draft ? a.T : x.Lk - (WIN ? x.span.shift : 0) - t0, valid = left < kTile ? left : kTile;
                // rows past the end hold other sequences' values or nothing at all:
                // P is 0 there, but 0 times a NaN is not, so V gets zeros
                const bool fix = is_v && valid < kTile;
                const uint32_t bar = fix ? bars.vraw(slot) : bars.kvfull(slot);
                const CUtensorMap *m = is_v ? &maps.v : &maps.k;
                if (!PAGED && WIN && t0 < x.span.sinks && t0 + kTile > x.span.sinks) {  // sinks, then others
                    const CUtensorMap *m16 = is_v ? &maps.v16 : &maps.k16;
                    expect_tx(lead, bar, kTileBytes);
#pragma unroll 1
                    for (int i = 0; i < kTile; i += 16) {
                        const int row = x.k0 + x.span.key(t0 + i);
                        tma_3d(lead, dst + i * 128, m16, 0, x.h, row, bar);
                        tma_3d(lead, dst + kHalf + i * 128, m16, 64, x.h, row, bar);
                    }
                } else if (!PAGED) {
                    expect_tx(lead, bar, kTileBytes);
                    tma_3d(lead, dst, m, 0, x.h, x.k0 + first, bar);
                    tma_3d(lead, dst + kHalf, m, 64, x.h, x.k0 + first, bar);
                } else if (x.draft) {
                    const CUtensorMap *mn = is_v ? &maps.vn : &maps.kn;
                    expect_tx(lead, bar, (uint32_t)((a.T + 7) & ~7) * 256u);
                    tma_3d(lead, dst, mn, 0, x.h, x.n * a.T, bar);
                    tma_3d(lead, dst + kHalf, mn, 64, x.h, x.n * a.T, bar);
                } else {
                    const int copies = (valid + rows - 1) >> row_bits;
                    expect_tx(lead, bar, (uint32_t)(copies << row_bits) * 256u);
                    int row = max(a.pages * a.Hkv * a.page, 1);  // past the map's last row (an empty pool's has one): zeros
                    if (x.pg >= 0 && x.pg < a.pages)
                        row = (x.pg * a.Hkv + x.h) * a.page + ((WIN ? x.span.key(t0 + (lane << row_bits)) : t0 + (lane << row_bits)) & (a.page - 1));
                    else if (lane < copies)
                        atomicOr(status_word(a), kStatusBadSeqlens);
                    for (int i = 0; i < copies; ++i) {
                        const int ri = __shfl_sync(0xffffffffu, row, i);
                        tma_2d(lead, dst + (i << (row_bits + 7)), m, 0, ri, bar);
                        tma_2d(lead, dst + kHalf + (i << (row_bits + 7)), m, 64, ri, bar);
                    }
                }
                if (fix && lane == 0) {  // the fixing warp waits for the copy and hands the slot on
                    int2 *job = reinterpret_cast<int2 *>(sm + L::kBars + Bars::kJobs) + jobs % kJobRing;
                    *job = make_int2((int)slot, valid);
                    mbar_arrive(bars.jfull(jobs % kJobRing));
                }
                if (fix) ++jobs;
                __syncwarp();
            };
            auto load_q = [&](int i, int tok, int h) {
                const uint32_t slot = (uint32_t)i % L::kQs, use = (uint32_t)i / L::kQs;
                if (use > 0 && !warp_wait(bars.qempty(slot), (use - 1) & 1)) {
                    alive = false;
                    return;
                }
                sent ^= 1u << slot;
                const uint32_t dst = base + L::kQ + slot * L::kQTile, bar = bars.qfull(slot);
                expect_tx(lead, bar, qbytes);
                tma_3d(lead, dst, &maps.q, 0, h * a.G, tok, bar);
                tma_3d(lead, dst + L::kQHalf, &maps.q, 64, h * a.G, tok, bar);
                __syncwarp();
            };
            Load x = {}, x1 = {}, x2 = {};  // this K tile and the last two
            uint32_t peeked = 0;  // descriptors whose first pages are looked up
            int peek_pg = -1, peek_pg2 = -1, next_pg = -1, next_pg2 = -1;
            int left = 0, flush = kLag, draft_tile = -1, q_first = 0;
            const Desc *d = nullptr;
            bool more = true;
            while (alive) {
                while (left == 0 && more) {  // the next part
                    d = next_desc();
                    more = d != nullptr;
                    if (!more) break;
                    const int n0 = d->count[0], n1 = d->count[1];
                    left = DUAL ? n0 + n1 : (n0 > n1 ? n0 : n1);  // (one at least)
                    x.n = d->n;
                    x.h = d->h;
                    x.k0 = d->k0;
                    x.Lk = d->Lk;
                    x.t = d->ta - 1;
                    if (WIN) x.span = d->span;
                    draft_tile = PAGED && a.has_new ? d->nt - 1 : -1;
                    q_first = 1;
                    next_pg = peek_pg;
                    next_pg2 = peek_pg2;
                    if (PAGED && peeked != nd + 1) {
                        next_pg = page_of(x.span, x.n, x.Lk, d->ta);
                        next_pg2 = page_of(x.span, x.n, x.Lk, d->ta + 1);
                    }
                }
                if (!alive || (left == 0 && flush-- == 0)) break;
                const bool has_k = left > 0;
                if (has_k) {
                    ++x.t;
                    x.draft = PAGED && x.t == draft_tile;
                    x.pg = next_pg;  // looked up two tiles ahead
                    next_pg = next_pg2;
                    next_pg2 = page_of(x.span, x.n, x.Lk, x.t + 2);
                    if (PAGED && left == 1 &&
                        __all_sync(0xffffffffu, mbar_test(bars.dfull((nd + 1) % kDescs), ((nd + 1) / kDescs) & 1))) {
                        const Desc *e = descs + (nd + 1) % kDescs;
                        if (!e->last) {
                            const Span span = WIN ? e->span : Span{0, 0};
                            peek_pg = page_of(span, e->n, e->Lk, e->ta);
                            peek_pg2 = page_of(span, e->n, e->Lk, e->ta + 1);
                            peeked = nd + 2;
                        }
                    }
                }
                // V of kLag tiles ago, then this K tile, a part's Q tiles around its first
#pragma unroll 1
                for (int is_k = g < (uint32_t)kLag; is_k < 1 + has_k && alive; ++is_k) {
                    if (is_k && q_first && (DUAL || d->count[0] > 0)) load_q(d->q[0], d->q0, x.h);
                    if (alive) load(is_k ? x : (DUAL ? x2 : x1), !is_k);
                }
                if (!DUAL && q_first && alive && d->count[1] > 0) load_q(d->q[1], d->q0 + a.tile_tokens, x.h);
                q_first = 0;
                x2 = x1;
                x1 = x;
                ++g;
                if (has_k && --left == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars.dempty(nd % kDescs));
                    ++nd;
                }
            }
            if (lane == 0) {  // no further job
                reinterpret_cast<int2 *>(sm + L::kBars + Bars::kJobs)[jobs % kJobRing] = make_int2(-1, 0);
                mbar_arrive(bars.jfull(jobs % kJobRing));
            }
            // The last copy into each slot has landed before the CTA ends, whoever takes it or not.
            // (Of n copies the last one's parity is n - 1's; of none it is that of no wait. A copy that
            // the fixing warp would have handed on has landed when the limit is over.)
            bool landed = true;
#pragma unroll 1
            for (uint32_t i = 0; i < (uint32_t)L::kRing; ++i)
                landed = wait_warp<kLimit>(bars.kvfull(i), ((kv + L::kRing - 1 - i) / L::kRing - 1) & 1) && landed;
#pragma unroll 1
            for (uint32_t i = 0; i < (uint32_t)L::kQs; ++i)
                landed = wait_warp<kLimit>(bars.qfull(i), ~sent >> i & 1) && landed;
            alive = alive && landed;
        } else if (warp == kWarpFix) {
            // ---- fixing warp: zeros in the V rows past a sequence's end ----------------
            uint32_t fixed = 0;
            for (uint32_t jobs = 0;; ++jobs) {
                if (!(alive = long_wait(bars.jfull(jobs % kJobRing), (jobs / kJobRing) & 1))) break;
                const int2 job = reinterpret_cast<const int2 *>(sm + L::kBars + Bars::kJobs)[jobs % kJobRing];
                const int slot = job.x;
                if (slot < 0) break;
                // the slot's V copies that end here: one phase of vraw each
                if (!(alive = warp_wait(bars.vraw(slot), (fixed >> slot) & 1))) break;
                fixed ^= 1u << slot;
                for (int r = job.y + (lane >> 3); r < kTile; r += 4) {
                    const uint32_t at = L::kKv + slot * kTileBytes + r * 128 + (lane & 7) * 16;
                    *reinterpret_cast<uint4 *>(sm + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(sm + at + kHalf) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.kvfull(slot));
            }
        } else {
            // ---- MMA warp: the whole warp walks along, one lane issues --------------
            constexpr uint32_t kIdQK = tc::idesc_f16(128, 128, 0, 0, 0);
            constexpr uint32_t kIdPV = tc::idesc_f16(128, 128, 0, 0, 1);
            const uint32_t lead = tc::elect_one();
            const uint64_t q_desc = tc::smem_desc_sw128(base + L::kQ, 16, 1024);
            const uint64_t k_desc = tc::smem_desc_sw128(base + L::kKv, 16, 1024);
            const uint64_t v_desc = tc::smem_desc_sw128(base + L::kKv, kHalf, 1024);
            uint32_t kv = 0, np0 = 0, np1 = 0;
            auto wait_kv = [&](uint32_t at) {
                if (alive) alive = warp_wait(bars.kvfull(at % L::kRing), (at / L::kRing) & 1);
            };
            auto free_kv = [&](uint32_t at) { tc::mma_commit_lead(lead, bars.kvempty(at % L::kRing)); };
            // S_s = Q K^T with Q tile i; then the row tile's softmax may read it
            auto qk = [&](int s, int i, bool first, bool last, uint32_t at) {
                const uint32_t slot = (uint32_t)i % L::kQs;
                if (first && alive) alive = warp_wait(bars.qfull(slot), ((uint32_t)i / L::kQs) & 1);
                if (!alive) return;
                const uint64_t qd = q_desc + slot * (L::kQTile >> 4);
                const uint64_t kd = k_desc + (at % L::kRing) * (kTileBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t k16 = (kk & 3) * 32, half = kk >> 2;
                    tc::mma_f16_lead(lead, tm + kColS + 128 * s, qd + ((half * L::kQHalf + k16) >> 4),
                                     kd + ((half * kHalf + k16) >> 4), kIdQK, kk > 0);
                }
                tc::mma_commit_lead(lead, bars.sfull(s));
                if (!DUAL && last) tc::mma_commit_lead(lead, bars.qempty(slot));
            };
            // O_s (+)= P V, keys 0 .. 95 and 96 .. 127 once their P is there
            auto pv = [&](int s, uint32_t at, bool first, bool last) {
                const uint64_t vd = v_desc + (at % L::kRing) * (kTileBytes >> 4);
                const uint32_t parity = (s ? np1++ : np0++) & 1;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (alive) alive = warp_wait(bars.pready(s, half), parity);
                    if (!alive) return;
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = half ? 6 : 0; kk < (half ? 8 : 6); ++kk)
                        tc::mma_f16_ta_lead(lead, tm + kColO + 128 * s, tm + kColS + 128 * s + 8 * kk,
                                            vd + ((kk * 2048) >> 4), kIdPV, !first || kk > 0);
                }
                if (last) tc::mma_commit_lead(lead, bars.ofull(s));
            };
            if (!DUAL) {
                // step g: per stream, P V of step g - 1, then Q K^T of step g (of the next
                // part when the last one is through: its S is there when its O is read)
                int n0 = 0, n1 = 0, at_j = -1;  // of step g - 1
                while (alive) {
                    const Desc *d = next_desc();
                    if (!alive) break;
                    int c0 = 0, c1 = 0, q0 = 0, q1 = 0;
                    if (d != nullptr) {
                        c0 = d->count[0];
                        c1 = d->count[1];
                        q0 = d->q[0];
                        q1 = d->q[1];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bars.dempty(nd % kDescs));
                        ++nd;
                    }
                    const int n = d == nullptr ? 1 : (c0 > c1 ? c0 : c1);
                    for (int j = 0; j < n && alive; ++j) {
                        const uint32_t v = kv, k = kv + (at_j >= 0);
                        kv = k + (d != nullptr);
                        if (at_j >= 0) wait_kv(v);
                        bool waited = false;
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {
                            const int before = s ? n1 : n0, now = s ? c1 : c0;
                            if (at_j >= 0 && at_j < before) pv(s, v, at_j == 0, at_j + 1 == before);
                            if (j < now) {
                                if (!waited) wait_kv(k);
                                waited = true;
                                qk(s, s ? q1 : q0, j == 0, j + 1 == now, k);
                            }
                        }
                        if (!alive) break;
                        if (at_j >= 0) free_kv(v);
                        if (d != nullptr) free_kv(k);
                        at_j = j;
                        n0 = c0;
                        n1 = c1;
                    }
                    if (d == nullptr) break;
                }
            } else {
                // tile g is stream g % 2's: its P V of tile g - 2, then Q K^T of tile g
                uint32_t g = 0, flags = 0;  // per stream: its last tile was its part's first, last
                int left = 0, j = 0, q = 0, tiles = 0, flush = 2;
                bool more = true;
                while (alive) {
                    while (left == 0 && more) {  // the next part
                        const Desc *d = next_desc();
                        more = d != nullptr;
                        if (!more) break;
                        tiles = left = d->count[0] + d->count[1];
                        q = d->q[0];
                        j = 0;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bars.dempty(nd % kDescs));
                        ++nd;
                    }
                    if (!alive || (left == 0 && flush-- == 0)) break;
                    const int s = g & 1;
                    if (g >= 2) {
                        const uint32_t v = kv++;
                        wait_kv(v);
                        pv(s, v, flags >> (2 * s) & 1, flags >> (2 * s + 1) & 1);
                        if (!alive) break;
                        free_kv(v);
                    }
                    if (left > 0) {
                        const uint32_t k = kv++;
                        wait_kv(k);
                        qk(s, q, j < 2, false, k);
                        if (!alive) break;
                        free_kv(k);
                        flags = (flags & ~(3u << (2 * s))) | ((uint32_t)(j < 2) | (uint32_t)(j + 2 >= tiles) << 1) << (2 * s);
                        --left;
                        ++j;
                    }
                    ++g;
                }
            }
            tc::mma_commit_lead(lead, bars.drained());  // no product outlives the CTA, or its TMEM
            alive = wait_warp<kLimit>(bars.drained(), 0) && alive;
        }
    }
    __syncwarp();
    if (!alive && lane == 0) {
        *dead = 1;
        atomicOr(status_word(a), kStatusTimeout);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) tc::tmem_dealloc(tm, 512);
}

cudaError_t launch_attn_combine(const Args &a, bool bf16, bool joins_early, cudaStream_t stream);

// ---- host -----------------------------------------------------------------
namespace {
// Through a window: whether each item goes to a CTA of its own. That takes as long as its tiles; shared
// evenly there are fewer to each, but a search ahead and the parts' way out and back in, which cost
// as much as some tiles more (of one row tile 7, of two 11, of prompts, whose parts mostly have
// no second pass, 4). Direct and split, us: one token, 64 items of 9 tiles 14.7, 16.7, of 17
// 21.5, 20.0; 64 drafts, 64 items of 17 tiles 31.2, 35.3, of 33 52.0, 44.5; prompts, 128
// items of 18 tiles 32.9, 38.4, of 34 53.3, 50.5.
// The host knows how long an item may be, not whether they are. One sequence of 65,000 tokens and many of 100
// leave most SMs idle for as long as its items take, so items of more than kLongest tiles are always shared: up to there
// even batches gain as much as uneven ones lose. Direct and split, us, even and uneven: 152 items of one token, 17 tiles 31.2,
// 34.1 and 20.6, 17.2, of 33 53.3, 56.6 and 33.9, 18.1, of 510 222, 225 and 426, 51.4; 128 items of 24 tiles 36.5, 43.3
// and 27.2, 18.1; 64 drafts, 144 items of 17 tiles 25.2, 38.1 and 24.6, 19.6, of 24 33.1, 43.1 and 32.3, 19.8.
template <bool PAGED, bool DUAL>
bool window_direct(const Args &a, long long slots, long long keys) {
    constexpr int kTiles = PAGED ? (DUAL ? 7 : 11) : 4, kLongest = 20;
    const long long own = (long long)a.window + a.sinks + (PAGED ? kTile : a.block), longest = keys < own ? keys : own;
    return slots <= a.sms && longest <= kLongest * kTile && longest * (a.sms - slots) <= (long long)kTiles * kTile * a.sms;
}
template <bool PAGED, bool DUAL, int RT, bool WIN, bool TEST>
cudaError_t launch_form(Args &a, const Maps &maps, long long slots, long long keys, cudaStream_t stream) {
    a.streams = DUAL ? 1 : 2;
    // An item's start and end cost about as much as 1.2 key tiles of 256 rows, and a tile that is
    // cut short half of one (extra 192, 256, 320 on ragged prompts: 51.8, 53.0, 55.5 us); a
    // decode's are hidden by the loads of long items, but not of short ones (192 alone,
    // 320 alone, 192 and 512: 71.0, 66.8, 66.5 us for 128 sequences of 500 tokens, 254.0,
    // 256.5, 254.1 for 3,125). Pieces of fewer than two tiles do not pay for their join (cut
    // 1, 2, 3 on ragged prompts: 52.9, 51.8, 53.3 us).
    a.extra = 192;
    a.extra_short = PAGED ? 512 : 0;
    a.min_part = kMinPart;
    set_block(a);
    // Where a tile's rows come from other places than one stretch, they come 16 rows (prefill) or a
    // page's at a time.
    if (WIN) keys = PAGED ? set_window(a, keys, a.page < kTile ? a.page : kTile, a.page < kTile ? a.page : kTile) : set_window(a, keys, 16, 1);
    // every item's keys, its start and end and, at the most, its drafts' tile
    set_unit(a, (double)slots * ((double)keys + 512 + kTile));
    a.cut = 2;
    // (a CTA each for four short prompts: 9.1 us instead of 14.4)
    a.direct = slots <= a.sms && keys <= 5 * kTile;
    if (WIN) a.direct = window_direct<PAGED, DUAL>(a, slots, keys);
    constexpr int bytes = Smem<DUAL, RT>::kBytes;
    static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(attn_tc_kernel<PAGED, DUAL, RT, WIN, TEST>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    e = launch_early(attn_tc_kernel<PAGED, DUAL, RT, WIN, TEST>, dim3(a.direct ? (unsigned)slots : (unsigned)a.ctas), kThreads,
                     bytes, stream, a, maps);
    return e == cudaSuccess && !a.direct ? launch_attn_combine(a, true, !DUAL, stream) : e;
}
template <bool PAGED, bool DUAL, int RT>
cudaError_t launch(Args &a, const Maps &maps, long long slots, long long keys, cudaStream_t stream) {
    if (a.window > 0)
        return a.lose > 0 ? launch_form<PAGED, DUAL, RT, true, true>(a, maps, slots, keys, stream)
                          : launch_form<PAGED, DUAL, RT, true, false>(a, maps, slots, keys, stream);
    return a.lose > 0 ? launch_form<PAGED, DUAL, RT, false, true>(a, maps, slots, keys, stream)
                      : launch_form<PAGED, DUAL, RT, false, false>(a, maps, slots, keys, stream);
}
}  // namespace

cudaError_t launch_attn_prefill_tc(Args a, const void *q, const void *k, const void *v, long long ldq,
                                   long long ldk, long long ldv, cudaStream_t stream) {
    a.tile_tokens = kTile / a.G;
    Maps m{};
    if (!map3(&m.q, q, a.Hq, a.Tq_total, ldq, a.G, a.tile_tokens) ||
        !map3(&m.k, k, a.Hkv, a.Tk_total, ldk, 1, kTile) ||
        !map3(&m.v, v, a.Hkv, a.Tk_total, ldv, 1, kTile) ||
        !map3(&m.out, a.out, a.Hq, a.Tq_total, (long long)a.Hq * kD, a.G, a.tile_tokens))
        return cudaErrorInvalidValue;
    if (a.window > 0 && (!map3(&m.k16, k, a.Hkv, a.Tk_total, ldk, 1, 16) || !map3(&m.v16, v, a.Hkv, a.Tk_total, ldv, 1, 16)))
        return cudaErrorInvalidValue;
    const long long slots = ((long long)a.Tq_total / (2 * a.tile_tokens) + a.N) * a.Hkv;
    return launch<false, false, 128>(a, m, slots, a.Tk, stream);
}

cudaError_t launch_attn_decode_tc(Args a, const void *q, const void *kp, const void *vp, const void *kn,
                                  const void *vn, long long ldq, long long ldk, long long ldv,
                                  cudaStream_t stream) {
    // (one row tile for both streams instead of a second, empty one: 128 sequences of 500
    // tokens, when it was taken, 66.6 us instead of 79.3, one of 65,531 51.5 instead of 52.3)
    bool dual = a.T * a.G <= kTile;
    a.tile_tokens = dual ? a.T : kTile / a.G;
    const long long keys = (long long)a.table_cols * a.page + kTile;
    // Through a window also where every row tile can be an item with a CTA of its own: 27 us instead of 33 for 64
    // drafts of 8 users, 128 items of 17 tiles.
    if (!dual && a.window > 0)
        dual = window_direct<true, true>(a, (long long)a.N * a.Hkv * ((a.T + a.tile_tokens - 1) / a.tile_tokens), keys);
    const long long rows = (long long)a.pages * a.Hkv * a.page, toks = (long long)a.N * a.T;
    Maps m{};
    if (!map3(&m.q, q, a.Hq, toks, ldq, a.G, a.tile_tokens) ||
        !map2(&m.k, kp, rows, a.page < kTile ? a.page : kTile) ||
        !map2(&m.v, vp, rows, a.page < kTile ? a.page : kTile))
        return cudaErrorInvalidValue;
    if (!dual && !map3(&m.out, a.out, a.Hq, toks, (long long)a.Hq * kD, a.G, a.tile_tokens)) return cudaErrorInvalidValue;
    const int drafts = (a.T + 7) & ~7;  // whole groups of eight rows of the swizzle
    if (a.has_new && (!map3(&m.kn, kn, a.Hkv, toks, ldk, 1, drafts) || !map3(&m.vn, vn, a.Hkv, toks, ldv, 1, drafts)))
        return cudaErrorInvalidValue;
    const int block = a.tile_tokens * (dual ? 1 : 2);
    const long long slots = (long long)a.N * a.Hkv * ((a.T + block - 1) / block);
    if (!dual) return launch<true, false, 128>(a, m, slots, keys, stream);
    if (a.T * a.G <= 32) return launch<true, true, 32>(a, m, slots, keys, stream);
    return launch<true, true, 128>(a, m, slots, keys, stream);
}

}  // namespace attn
}  // namespace kda
