// Attention weights in bf16 on the tensor cores (the formula and the work split are those of
// kda_attn_weights.cuh).
//
// A tile is S = K Q^T of 128 keys and up to 512 (token, head) rows: the keys are the
// product's M, so that a key is a TMEM lane, its exponentials and their sum belong to one
// thread, and nothing crosses threads. The rows' lse goes through the product too, as 16
// further channels: keys have ones there, rows the three bf16 parts of -lse / scale (24 bits), so that
// S leaves the tensor core as q.k - lse / scale in fp32 and costs a thread one product, one
// exponential and one sum per element. A CTA
// (one per SM) streams K tiles through a ring by TMA; the rows' Q lies in shared memory
// for as long as the CTA stays with a (sequence, head), and the next one's is copied meanwhile.
// Roles of the 22 warps: 16 for the exponentials (four groups of four, each with 128 columns
// of TMEM), one issues the products, one fills the ring, four copy Q and lse, of which the
// first walks the CTA's parts ahead of the others.
//
// Up to 128 rows the groups take the tiles in turn. Up to 256 (PARTS = 2) a product is two groups
// wide, so that K is read once for both, and up to 512 (PARTS = 4) a tile is two products, of each of which all four
// groups take a quarter (a half each of one of them: 1.73 us a tile instead of 1.62, since two warps a scheduler
// hide less); the groups of a tile hand their sums to its first one. With 512 rows the Q tile
// takes the room of two, and a CTA waits for the next part's rows: they come in two copies, the first of which
// starts under the last part's last products and is all that the part's first ones need (27.5 us instead of 28.7
// in a graph for the prompts below).
//
// Measured (GB300; copy 6,790 GB/s): one token of 32 heads on 8 over 65,531 cached ones 26.8 us (5.1 TB/s with 5 us
// of start), four drafts of 128 sequences on 400,003 134 us (6.3 TB/s): bound by HBM. 64 tokens of 8
// prompts, 512 rows per kv head, 40,009 cached: 27.5 us, 24 with all inputs in L2, 1.62 us a tile and SM where its products alone take
// 1.24 and its exponentials with one of nine products 1.49 (1.0 of the exponentials' pipe). Tried on those 512 rows: two groups of
// warps that take 128 columns into registers at once 2.2 us, four that take their 64 at once 1.7, the next 16
// columns while these are summed 1.83, products of 128 rows instead of 256 2.0 (their own
// time 1.49), -lse from shared memory with a product and a sum more per element 2.2, two launches of 256 rows 2.2.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_attn.cuh"
#include "kda_attn_weights.cuh"
#include "kda_common.cuh"
#include "kda_tcgen05.cuh"
#include "kda_tensormap.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace weights {

using attn::add2;
using attn::ex2;
using attn::mbar_arrive;

constexpr int kGroups = 4, kExpWarps = 4 * kGroups, kWarpMma = 16, kWarpTma = 17, kWarpRows = 18, kRowWarps = 4;
constexpr int kTcThreads = 32 * (kWarpRows + kRowWarps);
constexpr int kTile = 128, kMaxRows = 512;
constexpr uint32_t kTileBytes = 32768, kHalf = 16384;
constexpr int kDescs = 4, kMaxRing = 6;
constexpr uint64_t kWaitNs = 2000000000, kTestWaitNs = 20000000;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;\n"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

// A part as the roles need it.
struct Desc {
    int last;      // no further part
    int b, h, len;
    int ta, tb;
    int seen;      // keys that its first row sees
    int tokens;
};

// Shared memory: two Q tiles (PARTS = 4: one) of `nq` rows (in halves of 64 channels), the ring of K tiles, the further
// channels of the rows of each Q tile and of the keys (8 x 8 blocks of 128 bytes, two to eight
// rows), then:
struct Shared {
    int seen[kDescs][kMaxRows];  // keys that a row sees; 0: it gives nothing
    Desc desc[kDescs];
    int4 least[kDescs];  // keys that all rows of each of the four warps see (0: some give nothing)
    uint64_t qfull[2], qempty[2];  // of a Q tile; PARTS = 4: of the first copy's rows, of the others
    uint64_t landed[2];  // its tensor copies: a phase ends with them alone, whichever warp has given up
    uint64_t sfull[kGroups], sempty[kGroups];  // of a group's S, or of two groups'
    uint64_t kfull[kMaxRing], kempty[kMaxRing];
    uint64_t dfull[kDescs], rfull[kDescs], dempty[kDescs];
    uint64_t drained;
    uint64_t pfull[kGroups][4], pempty[kGroups][4];  // the sums of a warp that hands them over
    float sums[kGroups][kTile];
    uint32_t tmem;
    int dead;
};
constexpr int kSmemMost = 232448;
struct Shape {
    int ns;    // rows of a group: 16, or a multiple of 32 up to 128
    int nq;    // rows of a Q tile: PARTS ns
    int tiles;  // Q tiles
    int ring;  // K tiles
    int box, boxes;  // Q by tensor copies: tokens of one, how many; box = 0: by the warps' own
    __host__ __device__ uint32_t q_tile() const { return (uint32_t)nq * 256; }
    __host__ __device__ uint32_t ring_at() const { return tiles * q_tile(); }
    __host__ __device__ uint32_t q_more_at() const { return ring_at() + ring * kTileBytes; }
    __host__ __device__ uint32_t q_more() const { return (uint32_t)nq * 32; }
    __host__ __device__ uint32_t k_more_at() const { return q_more_at() + tiles * q_more(); }
    __host__ __device__ uint32_t shared_at() const { return k_more_at() + kTile * 32; }
    __host__ __device__ uint32_t bytes() const { return shared_at() + (uint32_t)sizeof(Shared); }
};

// A wait of a whole warp, at most LIMIT nanoseconds.
template <uint64_t LIMIT>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    bool ok = false;
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if ((ok = tc::mbar_try_wait(bar, parity))) break;
        if ((n & 1023) != 0) continue;
        const uint64_t t = tc::globaltimer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > LIMIT) break;
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// Byte of (row, channel) of the further channels.
__device__ __forceinline__ uint32_t more_at(int row, int ch) { return tc::kmajor_off(row, ch, 128, 256); }

// The sum of 2^(c s) over N columns of S from column `at` on.
template <int N, bool MASKED>
__device__ __forceinline__ float2 exp_sum(uint32_t x[N / 16][16], const int *seen, int at, int pos, float c, float2 sum) {
    const float2 c2 = make_float2(c, c);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __uint_as_float(x[(i + e) / 16][(i + e) % 16]);
        if (MASKED) {
            const int4 n = *reinterpret_cast<const int4 *>(seen + at + i);
            y[0] = pos < n.x ? y[0] : -INFINITY;
            y[1] = pos < n.y ? y[1] : -INFINITY;
            y[2] = pos < n.z ? y[2] : -INFINITY;
            y[3] = pos < n.w ? y[3] : -INFINITY;
        }
        float2 u = mul2(make_float2(y[0], y[1]), c2), v = mul2(make_float2(y[2], y[3]), c2);
        u.x = ex2(u.x);
        u.y = ex2(u.y);
        v.x = ex2(v.x);
        v.y = ex2(v.y);
        sum = add2(sum, add2(u, v));
    }
    return sum;
}

// PARTS groups share a tile; SMALL: 16 rows at the most. Every wait has a limit: a role whose wait
// runs out goes to the kernel's end, the others follow as theirs run out or they see `dead`, and the
// status tells; the copies and products in flight are waited for first. TEST
// (kda_testing_attn_weights_timeout): waits of 20 ms, and warp a.lose - 1 gives up at its wait number a.lose_at.
template <int PARTS, bool SMALL, bool TEST>
__global__ void __launch_bounds__(kTcThreads, 1)
    weights_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map,
                      const Shape shape) {
    constexpr int kQTiles = PARTS == 4 ? 1 : 2;
    constexpr uint64_t kLimit = TEST ? kTestWaitNs : kWaitNs;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_u32(sm);
    Shared &sh = *reinterpret_cast<Shared *>(sm + shape.shared_at());
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (base & 1023u) {  // (the swizzled tiles need it)
        if (tid == 0 && a.status != nullptr) atomicOr(a.status, kStatusTimeout);
        return;
    }
    auto bar = [](const uint64_t &x) { return smem_u32(&x); };
    if (warp == kWarpTma && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(sh.qfull[i]), kRowWarps);
            tc::mbar_init(bar(sh.qempty[i]), 1);
            tc::mbar_init(bar(sh.landed[i]), 1);
        }
        for (int i = 0; i < kMaxRing; ++i) {
            tc::mbar_init(bar(sh.kfull[i]), 1);
            tc::mbar_init(bar(sh.kempty[i]), 1);
        }
        for (int i = 0; i < kDescs; ++i) {
            tc::mbar_init(bar(sh.dfull[i]), 1);
            tc::mbar_init(bar(sh.rfull[i]), kRowWarps);
            tc::mbar_init(bar(sh.dempty[i]), kExpWarps + 2 + kRowWarps - 1);  // and TMA, MMA
        }
        tc::mbar_init(bar(sh.drained), 1);
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(bar(sh.sfull[i]), 1);
            tc::mbar_init(bar(sh.sempty[i]), 4 * PARTS);
            for (int j = 0; j < 4; ++j) {
                tc::mbar_init(bar(sh.pfull[i][j]), 1);
                tc::mbar_init(bar(sh.pempty[i][j]), 1);
            }
        }
        sh.dead = 0;
        tc::fence_mbar_init();
        attn::prefetch_map(&map);
        attn::prefetch_map(&q_map);
    } else if (warp == kWarpMma) {
        tc::tmem_alloc(smem_u32(&sh.tmem), 512);
        tc::tmem_relinquish();
    }
    if (tid < kTile) {  // the keys' further channels: 1, 1, 1, 0, ..
        uint4 *const to = reinterpret_cast<uint4 *>(sm + shape.k_more_at() + more_at(tid, 0));
        to[0] = make_uint4(pack_bf16(1.f, 1.f), pack_bf16(1.f, 0.f), 0u, 0u);
        to[8] = make_uint4(0u, 0u, 0u, 0u);
        tc::fence_async_smem();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sh.tmem;
    volatile int *const dead = &sh.dead;
    wait_before();
    let_next_start();
    bool alive = true;
    uint32_t nd = 0;  // descriptors taken
    int waits = 0;
    auto warp_wait = [&](uint32_t at, uint32_t parity) -> bool {
        if constexpr (TEST) {
            if (warp == a.lose - 1 && waits++ >= a.lose_at) return false;
        }
        return wait_warp<kLimit>(at, parity);
    };
    // a wait that may last as long as a part does: it ends when another role gives up
    auto long_wait = [&](uint32_t at, uint32_t parity) -> bool {
        for (int i = 0; i < 100; ++i) {
            if (warp_wait(at, parity)) return true;
            if (*dead) return false;
        }
        return false;
    };
    auto next_desc = [&]() -> const Desc * {
        alive = long_wait(bar(sh.dfull[nd % kDescs]), (nd / kDescs) & 1);
        const Desc *const d = &sh.desc[nd % kDescs];
        return alive && !d->last ? d : nullptr;
    };
    auto done_desc = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.dempty[nd % kDescs]));
        ++nd;
    };

    if (warp < kExpWarps) {
        // ---- exponentials: thread = key -------------------------------------------------
        const int group = warp >> 2, quad = warp & 3, r = 32 * quad + lane;
        const int part = group % PARTS, lead = group - part;  // which rows of a tile; the group that writes
        const int buffer = PARTS == 1 ? group : (PARTS == 2 ? group >> 1 : 0);
        const int cols = PARTS == 4 ? shape.ns / 2 : shape.ns;  // of this group in a product
        const uint32_t tS = tm + ((uint32_t)(32 * quad) << 16) + (PARTS == 1 ? 128 : 256) * buffer + part * cols;
        const float c = a.scale * attn::kLog2e;
        constexpr int kTurns = kGroups / PARTS;  // every so many tiles are this group's
        uint32_t tiles = 0, mine = 0;  // of the CTA, of this group
        while (const Desc *d = next_desc()) {
            const uint32_t slot = nd % kDescs;
            const int *const seen = sh.seen[slot] + part * cols;
            const int ta = d->ta, tb = d->tb, len = d->len, rows = d->tokens * a.G - part * cols;
            float *const w = a.w + ((size_t)d->b * a.Hkv + d->h) * a.cap;
            if (!(alive = warp_wait(bar(sh.rfull[slot]), (nd / kDescs) & 1))) break;
            const int4 four = sh.least[slot];
            const int least = min(min(four.x, four.y), min(four.z, four.w));
            for (int t = ta + (int)((group / PARTS - tiles) % kTurns); t < tb; t += kTurns, ++mine) {
                const int pos = t * kTile + r;
                const bool ok = pos < len && part == 0;
                const float before = ok ? w[pos] : 0.f;
                const bool masked = least < (t + 1) * kTile;
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int e = 0; e < (PARTS == 4 ? 2 : 1); ++e) {  // products of a tile
                    if (!(alive = warp_wait(bar(sh.sfull[buffer + e]), mine & 1))) break;
                    tc::fence_after_sync();
                    if (SMALL) {
                        uint32_t x[1][16];
                        tc::tmem_ld_cols<1>(tS, x);
                        sum = exp_sum<16, true>(x, seen, 0, pos, c, sum);
                    } else {
                        const int row0 = 2 * shape.ns * e;
                        int at = 0;
                        for (; at + 32 <= cols; at += 32) {
                            uint32_t x[2][16];
                            tc::tmem_ld_cols<2>(tS + 256 * e + at, x);
                            if (masked || row0 + at + 32 > rows) sum = exp_sum<32, true>(x, seen, row0 + at, pos, c, sum);
                            else sum = exp_sum<32, false>(x, seen, row0 + at, pos, c, sum);
                        }
                        if (PARTS == 4 && at < cols) {  // 48 columns
                            uint32_t x[1][16];
                            tc::tmem_ld_cols<1>(tS + 256 * e + at, x);
                            sum = exp_sum<16, true>(x, seen, row0 + at, pos, c, sum);
                        }
                    }
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.sempty[buffer + e]));
                }
                if (!alive) break;
                float total = sum.x + sum.y;
                if (part > 0) {
                    if (mine > 0 && !(alive = warp_wait(bar(sh.pempty[group][quad]), (mine - 1) & 1))) break;
                    sh.sums[group][r] = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.pfull[group][quad]));
                    continue;
                }
#pragma unroll
                for (int e = 1; e < PARTS; ++e) {
                    if (alive) alive = warp_wait(bar(sh.pfull[lead + e][quad]), mine & 1);
                    if (!alive) break;
                    total += sh.sums[lead + e][r];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.pempty[lead + e][quad]));
                }
                if (!alive) break;
                if (ok) w[pos] = before + total;
            }
            if (!alive) break;
            tiles += tb - ta;
            done_desc();
        }
    } else if (warp >= kWarpRows) {
        // ---- the CTA's parts (the first of the warps), their Q and lse -----------------------
        const int wr = warp - kWarpRows;
        Walk<kTile> walk;
        if (wr == 0) walk.init(a, blockIdx.x, gridDim.x);
        const __nv_bfloat16 *const q = static_cast<const __nv_bfloat16 *>(a.q);
        const uint32_t inv_g = (65536u + a.G - 1) / a.G;  // r / G = r inv_g >> 16 for r < 1024
        const int Hq = a.Hkv * a.G;
        uint32_t sent[2] = {0, 0};  // copies into each Q tile, or of each half
        while (true) {
            const uint32_t slot = nd % kDescs, tile = nd % kQTiles;
            if (wr == 0) {
                Part p;
                const bool more = walk.next(a, p);
                if (nd >= kDescs && !(alive = long_wait(bar(sh.dempty[slot]), (nd / kDescs - 1) & 1))) break;
                if (lane == 0) {
                    Desc *const d = &sh.desc[slot];
                    d->last = !more;
                    if (more) {
                        d->b = p.b;
                        d->h = p.h;
                        d->len = p.s.len;
                        d->ta = p.ta;
                        d->tb = p.tb;
                        d->seen = p.s.len - p.s.count + a.t0 + 1;
                        d->tokens = p.s.tokens;
                    }
                    mbar_arrive(bar(sh.dfull[slot]));
                }
                __syncwarp();
            }
            const Desc *const d = next_desc();
            if (d == nullptr) break;
            const int b = d->b, tokens = d->tokens, rows = tokens * a.G, seen0 = d->seen, head = d->h * a.G;
            const size_t token0 = (size_t)b * a.T;
            // the tokens' numbers in q, two to a lane
            int tok[2] = {a.t0 + lane, a.t0 + lane + 32};
            if (a.index != nullptr) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (lane + 32 * e < tokens) tok[e] = token_of(a, b, a.t0 + lane + 32 * e);
            }
            auto token = [&](int i) {
                const int lo = __shfl_sync(0xffffffffu, tok[0], i & 31), hi = __shfl_sync(0xffffffffu, tok[1], i & 31);
                return i < 32 ? lo : hi;
            };
            const uint32_t dst = base + tile * shape.q_tile();
            const bool copies = shape.box > 0;
            // (PARTS = 4: what the last part's first products have read may be overwritten while the others run)
            for (uint32_t i = 0; i < (PARTS == 4 ? 2u : 1u) && alive; ++i) {
                const uint32_t half = PARTS == 4 ? i : tile;
                if (nd >= kQTiles) alive = long_wait(bar(sh.qempty[half]), (nd / kQTiles - 1) & 1);
                if (!alive || !copies || wr != 0) continue;
                // (tokens past the part's own come along, whose columns nobody looks at)
                const uint32_t lead = tc::elect_one(), full = bar(sh.landed[half]), bytes = (uint32_t)(shape.box * a.G) * 128u;
                const int token = b * a.T + a.t0 + (int)i * shape.box;
                attn::expect_tx(lead, full, 2 * bytes);
                attn::tma_3d(lead, dst + i * bytes, &q_map, 0, head, token, full);
                attn::tma_3d(lead, dst + (uint32_t)shape.nq * 128 + i * bytes, &q_map, 64, head, token, full);
                sent[0] += half == 0;
                sent[1] += half == 1;
                __syncwarp();
            }
            if (!alive) break;
            const int c = lane & 15;  // a row's 16 pieces, two rows at a time
#pragma unroll 4
            for (int r0 = copies ? rows : 2 * wr; r0 < rows; r0 += 2 * kRowWarps) {
                const int row = r0 + (lane >> 4), i = (int)(row * inv_g >> 16);
                const int tk = token(min(i, 63));
                if (row < rows && tk >= 0)
                    cp16(dst + (c >> 3) * (uint32_t)shape.nq * 128 + row * 128 + (((c & 7) ^ (row & 7)) * 16),
                         q + (token0 + tk) * a.ldq + (size_t)(head + row - i * a.G) * kD + 8 * c);
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            constexpr int kEach = PARTS;  // rows of lse of a lane
            float l[kEach];
            int sees[kEach];
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int row = 32 * (wr + kRowWarps * k) + lane, i = (int)(row * inv_g >> 16), tk = token(min(i, 63));
                l[k] = -INFINITY;
                sees[k] = seen0 + i;
                if (row < rows && tk >= 0) l[k] = a.lse[(token0 + tk) * Hq + head + row - i * a.G];
            }
            bool nothing = false;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int row = 32 * (wr + kRowWarps * k) + lane;
                const bool none = l[k] == -INFINITY;
                if (row < shape.nq) {
                    // (finite, since what is infinite times the keys' zeros is NaN: 2^(c x) is 0 or infinite far before)
                    float x = none ? 0.f : -l[k] / a.scale;
                    if (!(x != x)) x = fminf(fmaxf(x, -3e38f), 3e38f);
                    const float hi = __bfloat162float(__float2bfloat16_rn(x)), mid = __bfloat162float(__float2bfloat16_rn(x - hi));
                    unsigned char *const to = sm + shape.q_more_at() + tile * shape.q_more() + more_at(row, 0);
                    *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16(hi, mid), pack_bf16(x - hi - mid, 0.f), 0u, 0u);
                    *reinterpret_cast<uint4 *>(to + 128) = make_uint4(0u, 0u, 0u, 0u);
                }
                sh.seen[slot][row] = none ? 0 : sees[k];
                nothing = nothing || (none && row < rows);
            }
            nothing = __any_sync(0xffffffffu, nothing);
            if (lane == 0) (&sh.least[slot].x)[wr] = nothing ? 0 : seen0;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sh.rfull[slot]));
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(sh.qfull[tile]));
                if (PARTS == 4) mbar_arrive(bar(sh.qfull[1]));
                if (wr != 0) mbar_arrive(bar(sh.dempty[slot]));
            }
            ++nd;
        }
        // (as the ring's copies below; none: the parity of the phase before the first)
        if (wr == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i) alive = wait_warp<kLimit>(bar(sh.landed[i]), (sent[i] - 1) & 1) && alive;
    } else if (warp == kWarpTma) {
        // ---- K tiles -------------------------------------------------------------------------
        // A copy is at most a page's rows of a tile; a lane each looks up the pages of the next 32
        // copies, while those of the last 32 are issued.
        const int rows = a.page < kTile ? a.page : kTile, row_bits = 31 - __clz(rows), page_bits = 31 - __clz(a.page);
        const int per_tile = kTile >> row_bits, tiles_ahead = 32 / per_tile;
        const uint32_t lead = tc::elect_one();
        uint32_t kv = 0;
        while (const Desc *d = next_desc()) {
            const int b = d->b, h = d->h, len = d->len, tb = d->tb;
            const int32_t *const table = a.table + (size_t)b * a.table_ld;
            auto page_of = [&](int t) -> int {
                const long long pos = (long long)t * kTile + ((long long)lane << row_bits);
                return pos < len ? table[pos >> page_bits] : -1;
            };
            int pages = page_of(d->ta);
            for (int t0 = d->ta; t0 < tb && alive; t0 += tiles_ahead) {
                const int here = pages;
                if (t0 + tiles_ahead < tb) pages = page_of(t0 + tiles_ahead);
                const int pos = (int)min((long long)t0 * kTile + ((long long)lane << row_bits), 0x7fffffffLL);
                int row = max(a.pages * a.Hkv * a.page, 1);  // past the map's last row: zeros
                if (here >= 0 && here < a.pages) row = (here * a.Hkv + h) * a.page + (pos & (a.page - 1));
                else if (pos < len && pos < tb * kTile) flag(a);
                for (int t = t0; t < tb && t < t0 + tiles_ahead; ++t) {
                    const uint32_t slot = kv % shape.ring;
                    if (kv >= (uint32_t)shape.ring && !(alive = warp_wait(bar(sh.kempty[slot]), (kv / shape.ring - 1) & 1))) break;
                    ++kv;
                    const int copies = (min(len - t * kTile, kTile) + rows - 1) >> row_bits;
                    const uint32_t full = bar(sh.kfull[slot]), dst = base + shape.ring_at() + slot * kTileBytes;
                    attn::expect_tx(lead, full, (uint32_t)(copies << row_bits) * 256u);
                    for (int i = 0; i < copies; ++i) {
                        const int ri = __shfl_sync(0xffffffffu, row, (t - t0) * per_tile + i);
                        attn::tma_2d(lead, dst + (i << (row_bits + 7)), &map, 0, ri, full);
                        attn::tma_2d(lead, dst + kHalf + (i << (row_bits + 7)), &map, 64, ri, full);
                    }
                    __syncwarp();
                }
            }
            if (!alive) break;
            done_desc();
        }
        // the last copy into each slot has landed before the CTA ends, whoever takes it or not
        for (uint32_t i = 0; i < (uint32_t)shape.ring; ++i)
            alive = wait_warp<kLimit>(bar(sh.kfull[i]), ((kv + shape.ring - 1 - i) / shape.ring - 1) & 1) && alive;
    } else {
        // ---- products ------------------------------------------------------------------------
        const uint64_t k_more = tc::smem_desc(base + shape.k_more_at(), 128, 256), q_more = tc::smem_desc(base + shape.q_more_at(), 128, 256);
        const uint32_t lead = tc::elect_one(), idesc = tc::idesc_f16(kTile, (PARTS == 1 ? 1 : 2) * shape.ns, 0, 0, 0);
        const uint64_t q_desc = tc::smem_desc_sw128(base, 16, 1024), k_desc = tc::smem_desc_sw128(base + shape.ring_at(), 16, 1024);
        uint32_t kv = 0;
        while (const Desc *d = next_desc()) {
            const int n = d->tb - d->ta;
            const uint32_t tile = nd % kQTiles;
            auto rows_there = [&](uint32_t half) -> bool {
                const uint32_t parity = (nd / kQTiles) & 1;
                return warp_wait(bar(sh.qfull[half]), parity) && (shape.box == 0 || warp_wait(bar(sh.landed[half]), parity));
            };
            if (!(alive = rows_there(tile))) break;
            // PARTS = 4: the first products may need the second copy's rows too
            bool all = PARTS < 4;
            auto need_all = [&]() {
                if (alive && !all) alive = rows_there(1);
                all = true;
            };
            if (PARTS == 4 && shape.box * a.G < 2 * shape.ns) need_all();
            for (int t = 0; t < n && alive; ++t) {
                const uint32_t slot = kv % shape.ring;
                if (!(alive = warp_wait(bar(sh.kfull[slot]), (kv / shape.ring) & 1))) break;
                const uint64_t kd = k_desc + slot * (kTileBytes >> 4);
#pragma unroll
                for (int e = 0; e < (PARTS == 4 ? 2 : 1); ++e) {
                    const uint32_t s = PARTS == 1 ? kv & 3 : (PARTS == 2 ? kv & 1 : e);
                    const uint32_t used = PARTS == 1 ? kv >> 2 : (PARTS == 2 ? kv >> 1 : kv);  // times that this S has been
                    if (alive && used > 0) alive = warp_wait(bar(sh.sempty[s]), (used - 1) & 1);
                    if (e == 1) need_all();
                    if (!alive) break;
                    tc::fence_after_sync();
                    const uint32_t tS = tm + (PARTS == 1 ? 128 : 256) * s, row = e * 2 * shape.ns;
                    const uint64_t qd = q_desc + ((tile * shape.q_tile() + row * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t k16 = (kk & 3) * 32, half = kk >> 2;
                        tc::mma_f16_lead(lead, tS, kd + ((half * kHalf + k16) >> 4),
                                         qd + ((half * (uint32_t)shape.nq * 128 + k16) >> 4), idesc, kk > 0);
                    }
                    tc::mma_f16_lead(lead, tS, k_more, q_more + ((tile * shape.q_more() + row * 32) >> 4), idesc, 1);
                    tc::mma_commit_lead(lead, bar(sh.sfull[s]));
                    if (PARTS == 4 && t + 1 == n) tc::mma_commit_lead(lead, bar(sh.qempty[e]));
                }
                if (!alive) break;
                ++kv;
                tc::mma_commit_lead(lead, bar(sh.kempty[slot]));
            }
            if (!alive) break;
            if (PARTS < 4) tc::mma_commit_lead(lead, bar(sh.qempty[tile]));
            done_desc();
        }
        tc::mma_commit_lead(lead, bar(sh.drained));  // no product outlives the CTA, or its TMEM
        alive = wait_warp<kLimit>(bar(sh.drained), 0) && alive;
    }
    __syncwarp();
    if (!alive && lane == 0) {
        *dead = 1;
        if (a.status != nullptr) atomicOr(a.status, kStatusTimeout);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) tc::tmem_dealloc(tm, 512);
}

template <int PARTS, bool SMALL, bool TEST>
static cudaError_t launch_kernel(const Args &a, const CUtensorMap &map, const CUtensorMap &q_map, const Shape &shape, unsigned ctas,
                                 cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(weights_tc_kernel<PARTS, SMALL, TEST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_early(weights_tc_kernel<PARTS, SMALL, TEST>, dim3(ctas), kTcThreads, shape.bytes(), stream, a, map, q_map, shape);
}

template <int PARTS, bool SMALL>
static cudaError_t launch_form(const Args &a, const CUtensorMap &map, const CUtensorMap &q_map, const Shape &shape, unsigned ctas,
                               cudaStream_t stream) {
    return a.lose > 0 ? launch_kernel<PARTS, SMALL, true>(a, map, q_map, shape, ctas, stream)
                      : launch_kernel<PARTS, SMALL, false>(a, map, q_map, shape, ctas, stream);
}

cudaError_t launch_weights_tc(Args a, int sms, cudaStream_t stream) {
    CUtensorMap map;
    if (!attn::map2(&map, a.kp, (long long)a.pages * a.Hkv * a.page, a.page < kTile ? a.page : kTile))
        return cudaErrorInvalidValue;
    // tokens of a launch: as many as have 512 rows, evenly shared
    const int most = kMaxRows / a.G, T = a.T, launches = (T + most - 1) / most, per = (T + launches - 1) / launches;
    const long long tiles = (long long)a.B * a.Hkv * (((long long)a.cols * a.page + kTile - 1) / kTile);
    for (int t0 = 0; t0 < T; t0 += per) {
        a.t0 = t0;
        a.t1 = t0 + per < T ? t0 + per : T;
        Shape shape;
        const int rows = (a.t1 - a.t0) * a.G;
        const int parts = rows <= 128 ? 1 : (rows <= 256 ? 2 : 4);
        shape.ns = rows <= 16 ? 16 : ((rows + parts - 1) / parts + 31) / 32 * 32;
        shape.nq = parts * shape.ns;
        shape.tiles = parts == 4 ? 1 : 2;
        // Tokens in a row come by one tensor copy of each half of the channels, or two past 256 rows, the first
        // of which ends at a multiple of eight rows, where the swizzle starts over, if that leaves room.
        shape.boxes = rows <= 256 ? 1 : 2;
        shape.box = (a.t1 - a.t0 + shape.boxes - 1) / shape.boxes;
        while (shape.boxes > 1 && shape.box * a.G % 8 != 0) ++shape.box;
        if (a.index != nullptr || shape.boxes * shape.box * a.G > shape.nq) shape.box = 0;
        CUtensorMap q_map = {};
        if (shape.box > 0 && !attn::map3(&q_map, a.q, a.Hkv * a.G, (long long)a.B * T, a.ldq, a.G, shape.box))
            return cudaErrorInvalidValue;
        shape.ring = 0;
        shape.ring = (kSmemMost - (int)shape.bytes()) / (int)kTileBytes;
        if (shape.ring > kMaxRing) shape.ring = kMaxRing;
        const unsigned ctas = (unsigned)(tiles < sms ? tiles : sms);
        const cudaError_t e = rows <= 16   ? launch_form<1, true>(a, map, q_map, shape, ctas, stream)
                              : parts == 1 ? launch_form<1, false>(a, map, q_map, shape, ctas, stream)
                              : parts == 2 ? launch_form<2, false>(a, map, q_map, shape, ctas, stream)
                                           : launch_form<4, false>(a, map, q_map, shape, ctas, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace weights
}  // namespace kda
