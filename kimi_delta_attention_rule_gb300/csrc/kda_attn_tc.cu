// Softmax attention in bf16 on the tensor cores: causal attention over packed
// prompts, and attention of new (drafted) tokens over a paged cache.
//
//   s_ij = scale q_i . k_j,  o_i = sum_j e^{s_ij - m_i} v_j / l_i,
//   m_i = max_j s_ij (kept in fp32, over the keys seen so far),
//   l_i = sum_j e^{s_ij - m_i} (fp32)
//
// in one pass over the keys. A CTA (12 warps) holds two row tiles of 128
// (token, head of the group) rows, one per softmax warpgroup: S = Q K^T and
// O += P V run as M128 N128 tcgen05.mma with S, P and O in TMEM (S 2 x 128
// columns, P over S, O 2 x 128); one thread of an MMA warp issues, a TMA warp
// fills a ring of 128-key K and V tiles, and each softmax thread owns one row
// (a TMEM lane), so no row statistic ever crosses threads. While one
// warpgroup forms P from its S, the tensor core runs the other's products.
// O is rescaled only when a row's maximum grows by more than 2^8, which P in
// bf16 (rounded to nearest, relative step 2^-8) and l in fp32 hold without loss.
// With at most 128 rows per kv head (decode) both warpgroups take the same row
// tile and alternate key tiles; their results are joined at the end (DUAL).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn.cuh"
#include "kda_common.cuh"
#include "kda_tcgen05.cuh"
#include "kda_tensormap.cuh"

namespace kda {
namespace attn {

constexpr int kThreads = 384;   // 2 softmax warpgroups, MMA warp, TMA warp, 2 idle
constexpr int kTile = 128;      // rows of a row tile, keys of a key tile
constexpr uint32_t kTileBytes = 32768;  // 128 rows x 128 channels bf16, two 64-channel halves
constexpr uint32_t kHalf = 16384;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kRescale = 8.f;  // log2 growth of a maximum that rescales O

constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: S/P of stream s at 128 s, O at 256 + 128 s

struct Maps {
    CUtensorMap q, k, v, kn, vn;
};

// Shared memory. Not DUAL: Q [2 buffers][2 tiles], ring of 3. DUAL: Q [2
// buffers], 32 KB for the join of the two streams, ring of 4.
template <bool DUAL>
struct Smem {
    static constexpr int kRing = DUAL ? 4 : 3;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kJoin = 2 * kTileBytes;  // DUAL only
    static constexpr uint32_t kKv = (DUAL ? 3 : 4) * kTileBytes;
    static constexpr uint32_t kBars = kKv + kRing * kTileBytes;
    static constexpr uint32_t kBytes = kBars + 1024 + 1024;  // + barriers and descriptors, + alignment
};

struct Bars {  // shared-memory addresses
    uint32_t base;
    __device__ uint32_t qfull(int i) const { return base + 8 * i; }
    __device__ uint32_t qempty(int i) const { return base + 16 + 8 * i; }
    __device__ uint32_t sfull(int s) const { return base + 32 + 8 * s; }
    __device__ uint32_t pready(int s) const { return base + 48 + 8 * s; }
    __device__ uint32_t ofull(int s) const { return base + 64 + 8 * s; }
    __device__ uint32_t tail() const { return base + 80; }
    __device__ uint32_t kvfull(int i) const { return base + 96 + 8 * i; }
    __device__ uint32_t kvempty(int i) const { return base + 128 + 8 * i; }
    __device__ uint32_t tmem() const { return base + 160; }
    __device__ uint32_t dfull(int i) const { return base + 168 + 8 * i; }
    __device__ uint32_t dempty(int i) const { return base + 200 + 8 * i; }
    static constexpr uint32_t kDesc = 256;  // kDescs descriptors
};

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *m, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(m), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;\n"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
// a wait of a whole warp, which leaves it converged
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, kWaitNs));
}
__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("barrier.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// A part as the roles need it, in shared memory. The scheduler warp walks the
// CTA's parts ahead of the others (its dependent loads of lengths are off their
// path, and their registers hold no walk) and puts them in a ring.
constexpr int kDescs = 4;
struct Desc {
    int last;              // no further part
    int n, h, q0, k0, Lk;
    int first_tok;         // the item's first token within its sequence
    int ta, step;          // stream s takes the tiles ta + s (step - 1), then every step-th
    int nt;                // tiles of the item
    int whole, ends, slot; // the part is the item; it is the item's last; its workspace slot
    int part_tokens;
    int count[2];          // tiles of each stream
    int tokens[2];         // valid tokens of its row tile
    int seen;              // prefill: keys that the item's first token sees; decode: cached keys
};
template <bool PAGED, bool DUAL>
__device__ __forceinline__ void describe(const Args &a, const Part &p, int cta, Desc &d) {
    d.last = 0;
    d.n = p.n;
    d.h = p.h;
    d.q0 = p.q0;
    d.k0 = p.k0;
    d.Lk = p.Lk;
    d.first_tok = p.first_tok;
    d.ta = p.ta;
    d.step = DUAL ? 2 : 1;
    d.nt = p.nt;
    d.whole = p.whole();
    d.ends = p.tb == p.nt;
    d.slot = part_slot(cta, p);
    d.part_tokens = p.tokens;
    d.seen = PAGED ? p.Lk : p.Lk - p.Lq + p.first_tok + 1;
    for (int s = 0; s < 2; ++s) {
        if (DUAL) {
            d.tokens[s] = p.tokens;
            d.count[s] = (p.tb - p.ta - s + 1) / 2;
            continue;
        }
        const int left = p.tokens - s * a.tile_tokens;
        const int tokens = left < 0 ? 0 : (left < a.tile_tokens ? left : a.tile_tokens);
        int end = p.tb;
        if (!PAGED) {  // the keys that the row tile's last token sees
            const int seen = d.seen + s * a.tile_tokens + tokens - 1;
            const int nt = seen <= 0 ? 0 : (seen + kTile - 1) / kTile;
            end = end < nt ? end : nt;
        }
        d.tokens[s] = tokens;
        d.count[s] = tokens == 0 || end < p.ta ? 0 : end - p.ta;
    }
}

template <bool PAGED, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const Args a, const __grid_constant__ Maps maps) {
    using L = Smem<DUAL>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sm = smem_raw + (base - smem_u32(smem_raw));
    const Bars bars{base + L::kBars};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;

    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (warp == 9) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(bars.qfull(i), 1);
                tc::mbar_init(bars.qempty(i), 8);
                tc::mbar_init(bars.sfull(i), 1);
                tc::mbar_init(bars.pready(i), 4);
                tc::mbar_init(bars.ofull(i), 1);
            }
            tc::mbar_init(bars.tail(), 1);
            for (int i = 0; i < kDescs; ++i) {
                tc::mbar_init(bars.dfull(i), 1);
                tc::mbar_init(bars.dempty(i), 10);  // TMA, MMA, 8 softmax warps
            }
            for (int i = 0; i < L::kRing; ++i) {
                tc::mbar_init(bars.kvfull(i), 1);
                tc::mbar_init(bars.kvempty(i), 1);
            }
            tc::fence_mbar_init();
        }
    } else if (warp == 10) {
        tc::tmem_alloc(bars.tmem(), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *reinterpret_cast<uint32_t *>(sm + L::kBars + 160);
    const Desc *const descs = reinterpret_cast<const Desc *>(sm + L::kBars + Bars::kDesc);
    bool alive = true;
    uint32_t nd = 0;  // descriptors taken
    // the next descriptor (NULL: no further part, or a wait ran out)
    auto next_desc = [&]() -> const Desc * {
        alive = tc::mbar_wait(bars.dfull(nd % kDescs), (nd / kDescs) & 1, kWaitNs);
        const Desc *d = descs + nd % kDescs;
        return alive && !d->last ? d : nullptr;
    };
    auto free_desc = [&]() { mbar_arrive(bars.dempty(nd++ % kDescs)); };

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n");
        // ---- softmax warpgroups: thread = row (TMEM lane) ------------------------
        const int s = warp >> 2, r = tid & 127;
        const uint32_t tl = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tS = tl + kColS + 128 * s, tO = tl + kColO + 128 * s;
        const int tok = r / a.G, g = r - tok * a.G;
        const float c = a.scale * kLog2e;
        uint32_t ns = 0, no = 0, items = 0;
        while (const Desc *d = next_desc()) {
            const int steps = d->count[s], others = d->count[1 - s], tokens = d->tokens[s];
            const bool row_ok = tok < tokens;
            const bool warp_ok = __any_sync(0xffffffffu, row_ok);
            float m = -INFINITY, l = 0.f;
            unsigned long long bits = 0;
            if (PAGED && row_ok) {
                const int t = d->first_tok + (DUAL ? 0 : s * a.tile_tokens) + tok;
                bits = a.mask != nullptr ? a.mask[(size_t)d->n * a.T + t]
                                         : (t >= 63 ? ~0ull : (2ull << t) - 1);
                if (a.T < 64) bits &= (1ull << a.T) - 1;
            }
            // keys that the row tile's first row and this row see
            const int seen0 = d->seen + (PAGED ? 0 : s * a.tile_tokens);
            const int seen = PAGED ? seen0 : seen0 + tok;
            const int last_tile = d->nt - 1, step = d->step;
            int t = d->ta + s * (step - 1);
            for (int j = 0; j < steps; ++j, t += step) {
                if (!warp_wait(bars.sfull(s), ns++ & 1)) {
                    alive = false;
                    break;
                }
                tc::fence_after_sync();
                if (warp_ok) {
                    uint32_t x[8][16];
                    tc::tmem_ld_cols<8>(tS, x);
                    const bool drafts = PAGED && a.has_new && t == last_tile;
                    if (drafts) {
#pragma unroll
                        for (int i = 0; i < kTile; ++i)
                            if (i >= kMaxDrafts || !((bits >> i) & 1)) x[i / 16][i % 16] = 0xff800000u;
                    } else if (seen0 < (t + 1) * kTile) {
                        const int lim = seen - t * kTile;
#pragma unroll
                        for (int i = 0; i < kTile; ++i)
                            if (i >= lim) x[i / 16][i % 16] = 0xff800000u;
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
                        // -inf - -inf is NaN: not greater, no rescale
                        const bool grow = (top - m) * c > kRescale;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float up = fmaxf(m, top);
                            const float f = m == -INFINITY ? 0.f : ex2((m - up) * c);
                            m = up;
                            l *= f;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint32_t o[2][16];
                                tc::tmem_ld_cols<2>(tO + 32 * q, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i / 16][i % 16] = __float_as_uint(f * __uint_as_float(o[i / 16][i % 16]));
                                tc::tmem_st16u(tO + 32 * q, o[0]);
                                tc::tmem_st16u(tO + 32 * q + 16, o[1]);
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
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc::tmem_wait_st();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.pready(s));
            }
            if (!alive) break;
            // ---- the part's end ----
            if (steps > 0) {
                if (!warp_wait(bars.ofull(s), no++ & 1)) {
                    alive = false;
                    break;
                }
                tc::fence_after_sync();
            }
            const uint32_t qb = items & 1;
            if (steps == 0 && others > 0 && !warp_wait(bars.qfull(qb), (items >> 1) & 1)) {
                // (without this wait an idle stream would run ahead and release the
                // buffer of the item after next in the other stream's stead)
                alive = false;
                break;
            }
            if (steps + others > 0) ++items;
            float f = 1.f, f1 = 0.f;  // weights of this stream's and (DUAL) the other's O
            if (DUAL && others > 0 && steps > 0) {
                // join: stream 1 hands over (m, l), then O in two halves of 64 channels
                float *box = reinterpret_cast<float *>(sm + L::kJoin);
                if (s == 1) reinterpret_cast<float2 *>(box)[r] = make_float2(m, l);
                named_bar(1, 256);
                if (s == 0) {
                    const float2 ml = reinterpret_cast<float2 *>(box)[r];
                    const float up = fmaxf(m, ml.x);
                    f = m == -INFINITY ? 0.f : ex2((m - up) * c);
                    f1 = ml.x == -INFINITY ? 0.f : ex2((ml.x - up) * c);
                    m = up;
                    l = l * f + ml.y * f1;
                }
                named_bar(1, 256);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (s == 1 && warp_ok) {
                        uint32_t o[4][16];
                        tc::tmem_ld_cols<4>(tO + 64 * h, o);
                        float4 *b4 = reinterpret_cast<float4 *>(box) + r;
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            b4[128 * q] = make_float4(
                                __uint_as_float(o[q / 4][4 * (q % 4)]), __uint_as_float(o[q / 4][4 * (q % 4) + 1]),
                                __uint_as_float(o[q / 4][4 * (q % 4) + 2]), __uint_as_float(o[q / 4][4 * (q % 4) + 3]));
                    }
                    named_bar(1, 256);
                    if (s == 0 && warp_ok) {
                        uint32_t o[4][16];
                        tc::tmem_ld_cols<4>(tO + 64 * h, o);
                        const float4 *b4 = reinterpret_cast<const float4 *>(box) + r;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float4 y = b4[128 * q];
                            uint32_t *z = &o[q / 4][4 * (q % 4)];
                            z[0] = __float_as_uint(f * __uint_as_float(z[0]) + f1 * y.x);
                            z[1] = __float_as_uint(f * __uint_as_float(z[1]) + f1 * y.y);
                            z[2] = __float_as_uint(f * __uint_as_float(z[2]) + f1 * y.z);
                            z[3] = __float_as_uint(f * __uint_as_float(z[3]) + f1 * y.w);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) tc::tmem_st16u(tO + 64 * h + 16 * q, o[q]);
                        tc::tmem_wait_st();
                    }
                    named_bar(1, 256);
                }
            }
            const bool writes = warp_ok && (!DUAL || s == 0);
            if (writes && !d->whole) {
                const int slot = d->slot, row = DUAL ? r : 128 * s + r;
                float4 *o4 = reinterpret_cast<float4 *>(part_o(a, slot)) + row;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[2][16];
                    if (steps > 0) tc::tmem_ld_cols<2>(tO + 32 * q, o);
                    if (row_ok) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (steps > 0)
                                y = make_float4(__uint_as_float(o[i / 4][4 * (i % 4)]),
                                                __uint_as_float(o[i / 4][4 * (i % 4) + 1]),
                                                __uint_as_float(o[i / 4][4 * (i % 4) + 2]),
                                                __uint_as_float(o[i / 4][4 * (i % 4) + 3]));
                            o4[(size_t)(8 * q + i) * kPartRows] = y;
                        }
                    }
                }
                if (row_ok) part_ml(a, slot)[row] = make_float2(m, l);
            } else if (writes) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int q0 = d->q0 + (DUAL ? 0 : s * a.tile_tokens);
                unsigned char *stage = sm + L::kQ + (DUAL ? qb : 2 * qb + s) * kTileBytes;
                if (row_ok && a.lse != nullptr)
                    a.lse[(size_t)(q0 + tok) * a.Hq + d->h * a.G + g] =
                        l == 0.f ? -INFINITY : m * a.scale + logf(l);
                if (steps == 0) {  // rows that see nothing
                    if (row_ok) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                               ((size_t)(q0 + tok) * a.Hq + d->h * a.G + g) * kD);
#pragma unroll
                        for (int i = 0; i < 16; ++i) dst[i] = make_uint4(0, 0, 0, 0);
                    }
                } else {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[2][16];
                        tc::tmem_ld_cols<2>(tO + 32 * q, o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack_bf16(inv * __uint_as_float(o[i / 2][8 * (i % 2) + 2 * e]),
                                                 inv * __uint_as_float(o[i / 2][8 * (i % 2) + 2 * e + 1]));
                            const int ch = 4 * q + i;
                            *reinterpret_cast<uint4 *>(stage + r * 256 + ((ch ^ (r & 15)) * 16)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    __syncwarp();
                    // 16 lanes write one row of 256 bytes
                    const int rows = tokens * a.G;
                    for (int i = lane >> 4; i < 32; i += 2) {
                        const int row = 32 * (warp & 3) + i;
                        if (row >= rows) break;
                        const int ch = lane & 15, tk = row / a.G;
                        const uint4 y = *reinterpret_cast<const uint4 *>(stage + row * 256 + ((ch ^ (row & 15)) * 16));
                        reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                  ((size_t)(q0 + tk) * a.Hq + d->h * a.G + (row - tk * a.G)) * kD)[ch] = y;
                    }
                }
            }
            // O is read: the MMA warp's next P V waits for this warp's next P.
            // The Q buffer (the staging's too) goes back to the TMA warp.
            tc::fence_before_sync();
            if (steps + others > 0) {
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.qempty(qb));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.dempty(nd % kDescs));
            ++nd;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;\n");
        if (warp == 10) {
            // ---- scheduler warp ---------------------------------------------------
            Point p0, p1;
            const bool any = split_points<PAGED>(a, cta, p0, p1);
            if (lane == 0) {
                part_header(a, 2 * cta)->valid = 0;
                part_header(a, 2 * cta + 1)->valid = 0;
                Walk<PAGED> walk;
                Part p;
                if (any) walk.init(p0, p1);
                bool more = true;
                while (more && alive) {
                    if (nd >= kDescs) alive = tc::mbar_wait(bars.dempty(nd % kDescs), (nd / kDescs - 1) & 1, kWaitNs);
                    if (!alive) break;
                    Desc *d = const_cast<Desc *>(descs) + nd % kDescs;
                    more = any && walk.next(a, p);
                    if (more) {
                        describe<PAGED, DUAL>(a, p, cta, *d);
                        if (!d->whole) {
                            PartHeader *h = part_header(a, d->slot);
                            h->ends = d->ends;
                            h->token0 = p.q0;
                            h->tokens = p.tokens;
                            h->kvh = p.h;
                            h->valid = 1;
                        }
                    } else {
                        d->last = 1;
                    }
                    mbar_arrive(bars.dfull(nd++ % kDescs));
                }
            }
        } else if (warp == 9) {
            // ---- TMA warp ------------------------------------------------------
            const int G = a.G;
            uint32_t kv = 0, items = 0, tails = 0;
            const uint32_t qbytes = (uint32_t)a.tile_tokens * G * 256u;
            // one K (is_v = false) or V tile into the next ring slot
            auto load = [&](const Desc &pt, int t, bool is_v) {
                const uint32_t slot = kv % L::kRing;
                const uint32_t dst = base + L::kKv + slot * kTileBytes;
                if (kv >= (uint32_t)L::kRing &&
                    !warp_wait(bars.kvempty(slot), (kv / L::kRing - 1) & 1)) {
                    alive = false;
                    return;
                }
                ++kv;
                int valid;  // rows of this tile that are the sequence's own
                bool drafts = false;
                if (PAGED) {
                    drafts = a.has_new && t == pt.nt - 1;
                    valid = drafts ? a.T : pt.Lk - t * kTile;
                } else {
                    valid = pt.Lk - t * kTile;
                }
                valid = valid < kTile ? valid : kTile;
                // rows past the end hold other sequences' values or nothing at all:
                // P is 0 there, but 0 times a NaN is not, so V gets zeros
                const bool fix = is_v && valid < kTile;
                const uint32_t bar = fix ? bars.tail() : bars.kvfull(slot);
                if (!PAGED) {
                    if (lane == 0) {
                        const CUtensorMap *m = is_v ? &maps.v : &maps.k;
                        tc::mbar_arrive_expect_tx(bar, kTileBytes);
                        tma_3d(dst, m, 0, pt.h, pt.k0 + t * kTile, bar);
                        tma_3d(dst + kHalf, m, 64, pt.h, pt.k0 + t * kTile, bar);
                    }
                } else if (drafts) {
                    if (lane == 0) {
                        const CUtensorMap *m = is_v ? &maps.vn : &maps.kn;
                        tc::mbar_arrive_expect_tx(bar, 64 * 256);
                        tma_3d(dst, m, 0, pt.h, pt.n * a.T, bar);
                        tma_3d(dst + kHalf, m, 64, pt.h, pt.n * a.T, bar);
                    }
                } else {
                    const int rows = a.page < kTile ? a.page : kTile;  // rows of one copy
                    const int copies = (valid + rows - 1) / rows;
                    if (lane == 0) tc::mbar_arrive_expect_tx(bar, (uint32_t)copies * rows * 256u);
                    __syncwarp();
                    if (lane < copies) {
                        const CUtensorMap *m = is_v ? &maps.v : &maps.k;
                        const int pos = t * kTile + lane * rows;
                        const int pg = a.table[(size_t)pt.n * a.table_ld + pos / a.page];
                        int row;
                        if (pg < 0 || pg >= a.pages) {  // zeros instead (past the pool's last row)
                            atomicOr(status_word(a), kStatusBadSeqlens);
                            row = a.pages * a.Hkv * a.page;
                        } else {
                            row = (pg * a.Hkv + pt.h) * a.page + pos % a.page;
                        }
                        tma_2d(dst + lane * rows * 128, m, 0, row, bar);
                        tma_2d(dst + kHalf + lane * rows * 128, m, 64, row, bar);
                    }
                }
                if (fix) {
                    __syncwarp();
                    if (!warp_wait(bars.tail(), tails++ & 1)) {
                        alive = false;
                        return;
                    }
                    for (int r = valid + (lane >> 3); r < kTile; r += 4) {
                        const uint32_t at = L::kKv + slot * kTileBytes + r * 128 + (lane & 7) * 16;
                        *reinterpret_cast<uint4 *>(sm + at) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(sm + at + kHalf) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars.kvfull(slot));
                }
                __syncwarp();
            };
            while (const Desc *d = next_desc()) {
                const int n0 = d->count[0], n1 = d->count[1];
                if (n0 + n1 > 0) {
                    const uint32_t qb = items & 1;
                    if (items >= 2 && !warp_wait(bars.qempty(qb), ((items >> 1) - 1) & 1)) {
                        alive = false;
                        break;
                    }
                    ++items;
                    if (lane == 0) {
                        const int tiles = DUAL ? 1 : (d->tokens[1] > 0 ? 2 : 1);
                        tc::mbar_arrive_expect_tx(bars.qfull(qb), tiles * qbytes);
                        for (int i = 0; i < tiles; ++i) {
                            const uint32_t dst = base + L::kQ + (DUAL ? qb : 2 * qb + i) * kTileBytes;
                            const int tok = d->q0 + i * a.tile_tokens;
                            tma_3d(dst, &maps.q, 0, d->h * G, tok, bars.qfull(qb));
                            tma_3d(dst + kHalf, &maps.q, 64, d->h * G, tok, bars.qfull(qb));
                        }
                    }
                    __syncwarp();
                    // In the order in which the MMA warp takes them: one K tile ahead of
                    // the V tiles (DUAL: one of each stream).
                    const int tiles = DUAL ? n0 + n1 : (n0 > n1 ? n0 : n1), ahead = DUAL ? 2 : 1;
                    for (int j = 0; j < tiles + ahead && alive; ++j) {
                        if (j >= ahead) load(*d, d->ta + j - ahead, true);
                        if (alive && j < tiles) load(*d, d->ta + j, false);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.dempty(nd % kDescs));
                ++nd;
            }
        } else if (warp == 8) {
            // ---- MMA warp (one thread) -------------------------------------------
            if (lane == 0) {
                constexpr uint32_t kIdQK = tc::idesc_f16(128, 128, 0, 0, 0);
                constexpr uint32_t kIdPV = tc::idesc_f16(128, 128, 0, 0, 1);
                uint32_t kv = 0, items = 0, np[2] = {0, 0};
                auto wait_kv = [&](uint32_t at) {
                    if (!alive) return;
                    alive = tc::mbar_wait(bars.kvfull(at % L::kRing), (at / L::kRing) & 1, kWaitNs);
                };
                auto qk = [&](int s, uint32_t qb, uint32_t at) {
                    const uint32_t qa = base + L::kQ + (DUAL ? qb : 2 * qb + s) * kTileBytes;
                    const uint32_t ka = base + L::kKv + (at % L::kRing) * kTileBytes;
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        tc::mma_f16(tm + kColS + 128 * s, tc::smem_desc_sw128(qa + off, 16, 1024),
                                    tc::smem_desc_sw128(ka + off, 16, 1024), kIdQK, kk > 0);
                    }
                    tc::mma_commit(bars.sfull(s));
                };
                auto pv = [&](int s, uint32_t at, bool first) {
                    const uint32_t va = base + L::kKv + (at % L::kRing) * kTileBytes;
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_f16_ta(tm + kColO + 128 * s, tm + kColS + 128 * s + 8 * kk,
                                       tc::smem_desc_sw128(va + kk * 2048, kHalf, 1024), kIdPV,
                                       !first || kk > 0);
                };
                auto free_kv = [&](uint32_t at) { tc::mma_commit(bars.kvempty(at % L::kRing)); };
                auto wait_p = [&](int s) {
                    if (!alive) return;
                    alive = tc::mbar_wait(bars.pready(s), np[s]++ & 1, kWaitNs);
                    tc::fence_after_sync();
                };
                while (const Desc *d = next_desc()) {
                    const int n0 = d->count[0], n1 = d->count[1];
                    free_desc();
                    if (n0 + n1 == 0) continue;
                    const int n = n0 > n1 ? n0 : n1;
                    const uint32_t qb = items & 1;
                    alive = tc::mbar_wait(bars.qfull(qb), (items >> 1) & 1, kWaitNs);
                    ++items;
                    if (!DUAL) {
                        wait_kv(kv);
                        if (!alive) break;
                        if (n0 > 0) qk(0, qb, kv);
                        if (n1 > 0) qk(1, qb, kv);
                        free_kv(kv++);
                        for (int j = 0; j < n && alive; ++j) {
                            const uint32_t v = kv++;
                            const bool more = j + 1 < n;
                            const uint32_t k = more ? kv++ : 0;
                            wait_kv(v);
                            for (int s = 0; s < 2; ++s) {
                                const int ns = s ? n1 : n0;
                                if (j < ns) {
                                    wait_p(s);
                                    if (!alive) break;
                                    pv(s, v, j == 0);
                                    if (j + 1 == ns) tc::mma_commit(bars.ofull(s));
                                }
                                if (j + 1 < ns) {
                                    if (s == 0 || n0 <= j + 1) wait_kv(k);
                                    if (!alive) break;
                                    qk(s, qb, k);
                                }
                            }
                            free_kv(v);
                            if (more) free_kv(k);
                        }
                    } else {
                        // tiles 0, 1, 2, .. go to streams 0, 1, 0, ..; K runs two tiles ahead of V
                        const int tiles = n0 + n1;
                        for (int j = 0; j < tiles + 2 && alive; ++j) {
                            const int s = j & 1;
                            if (j >= 2) {
                                wait_kv(kv);
                                wait_p(s);
                                if (!alive) break;
                                pv(s, kv, j < 4);
                                if (j >= tiles) tc::mma_commit(bars.ofull(s));
                                free_kv(kv++);
                            }
                            if (j < tiles) {
                                wait_kv(kv);
                                if (!alive) break;
                                qk(s, qb, kv);
                                free_kv(kv++);
                            }
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    if (!alive && lane == 0) atomicOr(status_word(a), kStatusTimeout);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 10) tc::tmem_dealloc(tm, 512);
}

// ---- host -----------------------------------------------------------------
namespace {
// [rows][heads][128] bf16 with `ld` elements between rows; box = 64 channels x bh heads x br rows
bool map3(CUtensorMap *m, const void *p, int heads, long long rows, long long ld, int bh, int br) {
    const EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)(rows > 0 ? rows : 1)};
    const cuuint64_t strides[2] = {256, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)bh, (cuuint32_t)br};
    const cuuint32_t es[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map2(CUtensorMap *m, const void *p, long long rows, int br) {
    const EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {128, (cuuint64_t)(rows > 0 ? rows : 1)};
    const cuuint64_t strides[1] = {256};
    const cuuint32_t box[2] = {64u, (cuuint32_t)br};
    const cuuint32_t es[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <bool PAGED, bool DUAL>
cudaError_t launch(const Args &a, const Maps &maps, cudaStream_t stream) {
    constexpr int bytes = Smem<DUAL>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<PAGED, DUAL>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    attn_tc_kernel<PAGED, DUAL><<<a.ctas, kThreads, bytes, stream>>>(a, maps);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_attn_combine(const Args &a, bool bf16, cudaStream_t stream);

cudaError_t launch_attn_prefill_tc(Args a, const void *q, const void *k, const void *v, long long ldq,
                                   long long ldk, long long ldv, cudaStream_t stream) {
    a.kt = kTile;
    a.tile_tokens = kTile / a.G;
    a.streams = 2;
    a.extra = 256;
    a.min_part = 768;
    Maps m{};
    if (!map3(&m.q, q, a.Hq, a.Tq_total, ldq, a.G, a.tile_tokens) ||
        !map3(&m.k, k, a.Hkv, a.Tk_total, ldk, 1, kTile) ||
        !map3(&m.v, v, a.Hkv, a.Tk_total, ldv, 1, kTile))
        return cudaErrorInvalidValue;
    cudaError_t e = launch<false, false>(a, m, stream);
    return e == cudaSuccess ? launch_attn_combine(a, true, stream) : e;
}

cudaError_t launch_attn_decode_tc(Args a, const void *q, const void *kp, const void *vp, const void *kn,
                                  const void *vn, long long ldq, long long ldk, long long ldv,
                                  cudaStream_t stream) {
    const bool dual = a.T * a.G <= kTile;
    a.kt = kTile;
    a.streams = dual ? 1 : 2;
    a.tile_tokens = dual ? a.T : kTile / a.G;
    a.extra = 256;
    a.min_part = 768;
    const long long rows = (long long)a.pages * a.Hkv * a.page, toks = (long long)a.N * a.T;
    Maps m{};
    if (!map3(&m.q, q, a.Hq, toks, ldq, a.G, a.tile_tokens) ||
        !map2(&m.k, kp, rows, a.page < kTile ? a.page : kTile) ||
        !map2(&m.v, vp, rows, a.page < kTile ? a.page : kTile))
        return cudaErrorInvalidValue;
    if (a.has_new && (!map3(&m.kn, kn, a.Hkv, toks, ldk, 1, kMaxDrafts) ||
                      !map3(&m.vn, vn, a.Hkv, toks, ldv, 1, kMaxDrafts)))
        return cudaErrorInvalidValue;
    cudaError_t e = dual ? launch<true, true>(a, m, stream) : launch<true, false>(a, m, stream);
    return e == cudaSuccess ? launch_attn_combine(a, true, stream) : e;
}

}  // namespace attn
}  // namespace kda
