// Attention weights in bf16 on the tensor cores (the formula and the work split are those of
// kda_attn_weights.cuh).
//
// A tile is S = K Q^T of 128 keys and up to 256 (token, head) rows: the keys are the
// product's M, so that a key is a TMEM lane, its exponentials and their sum belong to one
// thread, and nothing crosses threads; a row's -lse is the same word for all of them. A CTA
// (one per SM) streams K tiles through a ring by TMA; the rows' Q lies in shared memory
// for as long as the CTA stays with a (sequence, head), and the next one's is copied meanwhile.
// Roles of the 14 warps: 8 for the exponentials (two groups of four, which take the tiles in
// turn, each with its own 256 columns of TMEM), one issues the products, one fills the ring, four
// copy Q and lse, of which the first walks the CTA's parts ahead of the others.
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
using attn::fma2;
using attn::mbar_arrive;

constexpr int kExpWarps = 8, kWarpMma = 8, kWarpTma = 9, kWarpRows = 10, kRowWarps = 4, kTcThreads = 448;
constexpr int kTile = 128, kMaxRows = 256;
constexpr uint32_t kTileBytes = 32768, kHalf = 16384;
constexpr int kDescs = 4, kMaxRing = 6;
constexpr uint64_t kWaitNs = 2000000000;

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

// Shared memory: two Q tiles of `nq` rows (in halves of 64 channels), the ring of K tiles, then:
struct Shared {
    float minus_lse[kDescs][kMaxRows];
    int seen[kDescs][kMaxRows];  // keys that a row sees; 0: it gives nothing
    Desc desc[kDescs];
    int4 least[kDescs];  // keys that all rows of each of the four warps see (0: some give nothing)
    uint64_t qfull[2], qempty[2], sfull[2], sempty[2];
    uint64_t kfull[kMaxRing], kempty[kMaxRing];
    uint64_t dfull[kDescs], rfull[kDescs], dempty[kDescs];
    uint64_t drained;
    uint32_t tmem;
    int dead;
};
constexpr int kSmemMost = 232448;
struct Shape {
    int nq;    // rows of a Q tile: 16, or a multiple of 32
    int ring;  // K tiles
    __host__ __device__ uint32_t q_tile() const { return (uint32_t)nq * 256; }
    __host__ __device__ uint32_t ring_at() const { return 2 * q_tile(); }
    __host__ __device__ uint32_t shared_at() const { return ring_at() + ring * kTileBytes; }
    __host__ __device__ uint32_t bytes() const { return shared_at() + (uint32_t)sizeof(Shared); }
};

// A wait with a limit, of a whole warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    bool ok = false;
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if ((ok = tc::mbar_try_wait(bar, parity))) break;
        if ((n & 1023) != 0) continue;
        const uint64_t t = tc::globaltimer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > kWaitNs) break;
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// The sum of exp(scale s - lse) over N columns of S from column c on.
template <int N, bool MASKED>
__device__ __forceinline__ float2 exp_sum(uint32_t x[N / 16][16], const float *minus_lse, const int *seen, int c, int pos,
                                          float scale, float2 sum) {
    const float2 scale2 = make_float2(scale, scale), log2e = make_float2(attn::kLog2e, attn::kLog2e);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(minus_lse + c + i);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __uint_as_float(x[(i + e) / 16][(i + e) % 16]);
        if (MASKED) {
            const int4 n = *reinterpret_cast<const int4 *>(seen + c + i);
            y[0] = pos < n.x ? y[0] : -INFINITY;
            y[1] = pos < n.y ? y[1] : -INFINITY;
            y[2] = pos < n.z ? y[2] : -INFINITY;
            y[3] = pos < n.w ? y[3] : -INFINITY;
        }
        float2 u = mul2(fma2(make_float2(y[0], y[1]), scale2, make_float2(l.x, l.y)), log2e);
        float2 v = mul2(fma2(make_float2(y[2], y[3]), scale2, make_float2(l.z, l.w)), log2e);
        u.x = ex2(u.x);
        u.y = ex2(u.y);
        v.x = ex2(v.x);
        v.y = ex2(v.y);
        sum = add2(sum, add2(u, v));
    }
    return sum;
}

// SMALL: nq = 16.
template <bool SMALL>
__global__ void __launch_bounds__(kTcThreads, 1)
    weights_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map, const Shape shape) {
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
            tc::mbar_init(bar(sh.sfull[i]), 1);
            tc::mbar_init(bar(sh.sempty[i]), 4);
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
        sh.dead = 0;
        tc::fence_mbar_init();
        attn::prefetch_map(&map);
    } else if (warp == kWarpMma) {
        tc::tmem_alloc(smem_u32(&sh.tmem), 512);
        tc::tmem_relinquish();
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
    // a wait that may last as long as a part does: it ends when another role gives up
    auto long_wait = [&](uint32_t at, uint32_t parity) -> bool {
        for (int i = 0; i < 100; ++i) {
            if (wait_warp(at, parity)) return true;
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
        const int group = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t tS = tm + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * group;
        uint32_t tiles = 0, mine = 0;  // of the CTA, of this group
        while (const Desc *d = next_desc()) {
            const uint32_t slot = nd % kDescs;
            const float *const minus_lse = sh.minus_lse[slot];
            const int *const seen = sh.seen[slot];
            const int ta = d->ta, tb = d->tb, len = d->len, rows = d->tokens * a.G;
            float *const w = a.w + ((size_t)d->b * a.Hkv + d->h) * a.cap;
            if (!(alive = wait_warp(bar(sh.rfull[slot]), (nd / kDescs) & 1))) break;
            const int4 four = sh.least[slot];
            const int least = min(min(four.x, four.y), min(four.z, four.w));
            for (int t = ta + (int)((tiles ^ group) & 1); t < tb; t += 2) {
                const int pos = t * kTile + r;
                const bool ok = pos < len;
                const float before = ok ? w[pos] : 0.f;
                if (!(alive = wait_warp(bar(sh.sfull[group]), mine++ & 1))) break;
                tc::fence_after_sync();
                const bool masked = least < (t + 1) * kTile;
                float2 sum = make_float2(0.f, 0.f);
                if (SMALL) {
                    uint32_t x[1][16];
                    tc::tmem_ld_cols<1>(tS, x);
                    sum = exp_sum<16, true>(x, minus_lse, seen, 0, pos, a.scale, sum);
                } else {
                    uint32_t x[2][2][16];  // the next columns come while these are summed
                    auto fetch = [&](int c, uint32_t y[2][16]) {
                        tc::tmem_ld16_raw(tS + c, y[0]);
                        tc::tmem_ld16_raw(tS + c + 16, y[1]);
                    };
                    fetch(0, x[0]);
                    for (int c0 = 0; c0 < shape.nq; c0 += 64) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int c = c0 + 32 * e;
                            if (c >= shape.nq) break;
                            tc::tmem_wait_ld();
                            tc::reg_fence16(x[e][0]);
                            tc::reg_fence16(x[e][1]);
                            if (c + 32 < shape.nq) fetch(c + 32, x[1 - e]);
                            if (masked || c + 32 > rows) sum = exp_sum<32, true>(x[e], minus_lse, seen, c, pos, a.scale, sum);
                            else sum = exp_sum<32, false>(x[e], minus_lse, seen, c, pos, a.scale, sum);
                        }
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sh.sempty[group]));
                if (ok) w[pos] = before + (sum.x + sum.y);
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
        while (true) {
            const uint32_t slot = nd % kDescs, tile = nd & 1;
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
            if (nd >= 2 && !(alive = long_wait(bar(sh.qempty[tile]), (nd / 2 - 1) & 1))) break;
            const uint32_t dst = base + tile * shape.q_tile();
            const int c = lane & 15;  // a row's 16 pieces, two rows at a time
#pragma unroll 4
            for (int r0 = 2 * wr; r0 < rows; r0 += 2 * kRowWarps) {
                const int row = r0 + (lane >> 4), i = (int)(row * inv_g >> 16);
                const int tk = token(min(i, 63));
                if (row < rows && tk >= 0)
                    cp16(dst + (c >> 3) * (uint32_t)shape.nq * 128 + row * 128 + (((c & 7) ^ (row & 7)) * 16),
                         q + (token0 + tk) * a.ldq + (size_t)(head + row - i * a.G) * kD + 8 * c);
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            constexpr int kEach = kMaxRows / (32 * kRowWarps);  // rows of lse of a lane
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
                sh.minus_lse[slot][row] = none ? 0.f : -l[k];
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
                if (wr != 0) mbar_arrive(bar(sh.dempty[slot]));
            }
            ++nd;
        }
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
                    if (kv >= (uint32_t)shape.ring && !(alive = wait_warp(bar(sh.kempty[slot]), (kv / shape.ring - 1) & 1))) break;
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
            alive = wait_warp(bar(sh.kfull[i]), ((kv + shape.ring - 1 - i) / shape.ring - 1) & 1) && alive;
    } else {
        // ---- products ------------------------------------------------------------------------
        const uint32_t lead = tc::elect_one(), idesc = tc::idesc_f16(kTile, shape.nq, 0, 0, 0);
        const uint64_t q_desc = tc::smem_desc_sw128(base, 16, 1024), k_desc = tc::smem_desc_sw128(base + shape.ring_at(), 16, 1024);
        uint32_t kv = 0;
        while (const Desc *d = next_desc()) {
            const int n = d->tb - d->ta;
            const uint32_t tile = nd & 1;
            if (!(alive = wait_warp(bar(sh.qfull[tile]), (nd >> 1) & 1))) break;
            const uint64_t qd = q_desc + tile * (shape.q_tile() >> 4);
            for (int t = 0; t < n; ++t) {
                const uint32_t slot = kv % shape.ring, s = kv & 1;
                if (!(alive = wait_warp(bar(sh.kfull[slot]), (kv / shape.ring) & 1))) break;
                if (kv >= 2 && !(alive = wait_warp(bar(sh.sempty[s]), ((kv >> 1) - 1) & 1))) break;
                ++kv;
                tc::fence_after_sync();
                const uint64_t kd = k_desc + slot * (kTileBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t k16 = (kk & 3) * 32, half = kk >> 2;
                    tc::mma_f16_lead(lead, tm + 256 * s, kd + ((half * kHalf + k16) >> 4),
                                     qd + ((half * (uint32_t)shape.nq * 128 + k16) >> 4), idesc, kk > 0);
                }
                tc::mma_commit_lead(lead, bar(sh.kempty[slot]));
                tc::mma_commit_lead(lead, bar(sh.sfull[s]));
            }
            if (!alive) break;
            tc::mma_commit_lead(lead, bar(sh.qempty[tile]));
            done_desc();
        }
        tc::mma_commit_lead(lead, bar(sh.drained));  // no product outlives the CTA, or its TMEM
        alive = wait_warp(bar(sh.drained), 0) && alive;
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

template <bool SMALL>
static cudaError_t launch_form(const Args &a, const CUtensorMap &map, const Shape &shape, unsigned ctas, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(weights_tc_kernel<SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_early(weights_tc_kernel<SMALL>, dim3(ctas), kTcThreads, shape.bytes(), stream, a, map, shape);
}

cudaError_t launch_weights_tc(Args a, int sms, cudaStream_t stream) {
    CUtensorMap map;
    if (!attn::map2(&map, a.kp, (long long)a.pages * a.Hkv * a.page, a.page < kTile ? a.page : kTile))
        return cudaErrorInvalidValue;
    // tokens of a launch: as many as have 256 rows (a second launch reads K again, mostly from L2, and
    // with so many rows the exponentials take as long as a tile's way from HBM), evenly shared
    const int most = kMaxRows / a.G, T = a.T, launches = (T + most - 1) / most, per = (T + launches - 1) / launches;
    const long long tiles = (long long)a.B * a.Hkv * (((long long)a.cols * a.page + kTile - 1) / kTile);
    for (int t0 = 0; t0 < T; t0 += per) {
        a.t0 = t0;
        a.t1 = t0 + per < T ? t0 + per : T;
        Shape shape;
        const int rows = (a.t1 - a.t0) * a.G;
        shape.nq = rows <= 16 ? 16 : (rows + 31) / 32 * 32;
        shape.ring = ((int)kSmemMost - (int)sizeof(Shared) - (int)shape.ring_at()) / (int)kTileBytes;
        if (shape.ring > kMaxRing) shape.ring = kMaxRing;
        const unsigned ctas = (unsigned)(tiles < sms ? tiles : sms);
        const cudaError_t e = shape.nq == 16 ? launch_form<true>(a, map, shape, ctas, stream)
                                             : launch_form<false>(a, map, shape, ctas, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace weights
}  // namespace kda
