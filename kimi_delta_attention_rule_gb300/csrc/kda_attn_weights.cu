// Attention weights in fp32 on CUDA cores (the formula and the work split are those of
// kda_attn_weights.cuh), in tiles of 64 keys.
//
// Up to eight rows (few_kernel) a warp reads sixteen keys of a tile straight into registers, a
// lane four channels of each, and multiplies them with its four of every row; the 32 sums of four
// keys and eight rows (or eight and four) cross the warp in 31 steps, after which a lane has one of them.
// Through shared memory K would be read once for each of the eight threads of a key, which bounded it (86
// us for one token of four heads on 65,531 x 8; 56 so).
//
// With more rows (weights_kernel) a thread of 128 forms a 4 x 4 piece of S = K Q^T for 32 rows at a time, two
// products per instruction, its exponentials, and their sum over its rows; the eight threads of a key add up
// in shared memory in a fixed order. Up to 64 rows stay in shared memory while the CTA stays with a (sequence,
// head). More of them are loaded in turn for every tile where a CTA has few (185 rows, one tile: 55 us, in four
// launches 76; 512 rows, three tiles: 358, 379), or take further launches where it has many: K, mostly from L2, then
// costs less than the rows (116 rows, five tiles: 183 in one, 166 in two; 128 rows on 65,531 tokens 481 us instead
// of 562, 0.48 of the FMA pipe). Several CTAs per SM hide one another's loads.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn.cuh"
#include "kda_attn_weights.cuh"
#include "kda_common.cuh"

namespace kda {
namespace weights {

constexpr int kThreads = 128, kKeys = 64, kRows = 32, kRpt = 4, kMostRows = 64;
// Rows of K and Q are read by neighbouring threads: the 16-byte pieces of a row stand in the order
// of (piece xor row % 8).
constexpr int smem_of(int rows) { return (kKeys + rows) * kD * 4 + 8 * kKeys * 4 + rows * 8; }

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

__device__ __forceinline__ void cp16(float *dst, const float *src, bool ok) {  // (not ok: zeros)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}

__global__ void __launch_bounds__(kThreads, 4) weights_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) float sm[];
    const int held = (a.t1 - a.t0) * a.G > kRows ? kMostRows : kRows;  // rows that there is room for
    const int most = held / a.G;                                     // tokens
    float *const Ks = sm, *const Qs = Ks + kKeys * kD, *const sums = Qs + held * kD, *const minus_lse = sums + 8 * kKeys;
    int *const seen = reinterpret_cast<int *>(minus_lse + held);  // keys that a row sees
    wait_before();
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
    const float *const q = static_cast<const float *>(a.q), *const kp = static_cast<const float *>(a.kp);
    const int Hq = a.Hkv * a.G, page_bits = 31 - __clz(a.page);
    Walk<kKeys> walk;
    walk.init(a, blockIdx.x, gridDim.x);
    Part p;
    while (walk.next(a, p)) {
        // rows of the tokens from `first` on, as many as there is room for
        auto load_rows = [&](int first) {
            const int rows = min(p.s.tokens - first, most) * a.G, padded = (rows + kRows - 1) & ~(kRows - 1);
#pragma unroll 4
            for (int r = warp; r < padded; r += kThreads / 32) {
                const int i = r / a.G, g = r - i * a.G, tok = r < rows ? token_of(a, p.b, a.t0 + first + i) : -1;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                float l = -INFINITY;
                if (tok >= 0) {
                    x = load4(q + ((size_t)p.b * a.T + tok) * a.ldq + (size_t)(p.h * a.G + g) * kD + 4 * lane);
                    l = a.lse[((size_t)p.b * a.T + tok) * Hq + p.h * a.G + g];
                }
                *reinterpret_cast<float4 *>(Qs + r * kD + 4 * (lane ^ (r & 7))) = x;
                if (lane == 0) {
                    minus_lse[r] = -l;
                    seen[r] = l == -INFINITY ? 0 : p.s.len - p.s.count + a.t0 + first + i + 1;
                }
            }
            return padded;
        };
        __syncthreads();  // the last part is through
        int padded = load_rows(0);
        const bool stay = p.s.tokens <= most;
        for (int t = p.ta; t < p.tb; ++t) {
            if (t > p.ta) __syncthreads();  // the last tile is through
            {  // a warp copies the rows warp, warp + 4, ..: lane i knows where row warp + 4 i is
                const int pos = t * kKeys + warp + 4 * (lane & 15);
                bool in = pos < p.s.len;
                long long off = 0;
                if (in) {
                    const int pg = a.table[(size_t)p.b * a.table_ld + (pos >> page_bits)];
                    in = pg >= 0 && pg < a.pages;
                    if (in) off = (((long long)pg * a.Hkv + p.h) * a.page + (pos & (a.page - 1))) * kD;
                    else flag(a);  // zeros instead
                }
                const unsigned rows_ok = __ballot_sync(0xffffffffu, in);
#pragma unroll 4
                for (int i = 0; i < kKeys / 4; ++i) {
                    const int r = warp + 4 * i;
                    cp16(Ks + r * kD + 4 * (lane ^ (r & 7)), kp + __shfl_sync(0xffffffffu, off, i) + 4 * lane, rows_ok >> i & 1);
                }
                asm volatile("cp.async.commit_group;\n" ::: "memory");
            }
            float sum[4] = {0.f, 0.f, 0.f, 0.f};  // keys tx + 16 e
            if (!stay && t > p.ta) padded = load_rows(0);
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
            __syncthreads();
            for (int first = 0, r0 = 0;; r0 += kRows) {
                if (r0 >= padded) {  // on to the next rows
                    first += most;
                    if (first >= p.s.tokens) break;
                    __syncthreads();
                    padded = load_rows(first);
                    __syncthreads();
                    r0 = 0;
                }
                float2 s2[4][kRpt] = {};
#pragma unroll 4
                for (int d = 0; d < kD; d += 4) {
                    float4 kk[4], qq[kRpt];
#pragma unroll
                    for (int e = 0; e < 4; ++e) kk[e] = load4(Ks + (tx + 16 * e) * kD + (d ^ ((tx & 7) * 4)));
#pragma unroll
                    for (int i = 0; i < kRpt; ++i) qq[i] = load4(Qs + (r0 + ty + 8 * i) * kD + (d ^ (ty * 4)));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < kRpt; ++i) {
                            s2[e][i] = attn::fma2(make_float2(kk[e].x, kk[e].y), make_float2(qq[i].x, qq[i].y), s2[e][i]);
                            s2[e][i] = attn::fma2(make_float2(kk[e].z, kk[e].w), make_float2(qq[i].z, qq[i].w), s2[e][i]);
                        }
                }
#pragma unroll
                for (int i = 0; i < kRpt; ++i) {
                    const int r = r0 + ty + 8 * i;
                    const float l = minus_lse[r];
                    const int n = seen[r];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t * kKeys + tx + 16 * e < n) sum[e] += expf(fmaf(s2[e][i].x + s2[e][i].y, a.scale, l));
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[ty * kKeys + tx + 16 * e] = sum[e];
            __syncthreads();
            const int pos = t * kKeys + tid;
            if (tid < kKeys && pos < p.s.len) {
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) y += sums[i * kKeys + tid];
                a.w[((size_t)p.b * a.Hkv + p.h) * a.cap + pos] += y;
            }
        }
    }
}

// 32 values of every lane, v[i]: the sum of all lanes' v[lane].
__device__ __forceinline__ float reduce_32(float *v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 16; half > 0; half >>= 1) {
        const bool upper = lane & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {  // keep one half of the values, give the other one away
            const float mine = upper ? v[i + half] : v[i], theirs = upper ? v[i] : v[i + half];
            v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, half);
        }
    }
    return v[0];
}

// ROWS = 4 or 8.
template <int ROWS>
__global__ void __launch_bounds__(kThreads, ROWS == 8 ? 3 : 4) few_kernel(const __grid_constant__ Args a) {
    constexpr int kEach = kKeys / (kThreads / 32), kBatch = 32 / ROWS;  // keys of a warp, and of 32 sums
    wait_before();
    let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane % ROWS;
    const float *const q = static_cast<const float *>(a.q), *const kp = static_cast<const float *>(a.kp);
    const int Hq = a.Hkv * a.G, page_bits = 31 - __clz(a.page);
    Walk<kKeys> walk;
    walk.init(a, blockIdx.x, gridDim.x);
    Part p;
    while (walk.next(a, p)) {
        const int rows = p.s.tokens * a.G;
        float4 qq[ROWS];
        float minus_lse = 0.f;  // of this lane's row, and the keys that it sees
        int seen = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int t = i / a.G, tok = i < rows ? token_of(a, p.b, a.t0 + t) : -1;
            qq[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tok < 0) continue;
            const size_t token = (size_t)p.b * a.T + tok;
            const int head = p.h * a.G + i - t * a.G;
            qq[i] = load4(q + token * a.ldq + (size_t)head * kD + 4 * lane);
            if (i == r) {
                const float l = a.lse[token * Hq + head];
                minus_lse = -l;
                seen = l == -INFINITY ? 0 : p.s.len - p.s.count + a.t0 + t + 1;
            }
        }
        float *const w = a.w + ((size_t)p.b * a.Hkv + p.h) * a.cap;
        for (int t = p.ta; t < p.tb; ++t) {
            const int first = t * kKeys + kEach * warp;  // this warp's keys
            const int pos = first + (lane & (kEach - 1));
            bool in = pos < p.s.len;
            long long off = 0;
            if (in) {
                const int pg = a.table[(size_t)p.b * a.table_ld + (pos >> page_bits)];
                in = pg >= 0 && pg < a.pages;
                if (in) off = (((long long)pg * a.Hkv + p.h) * a.page + (pos & (a.page - 1))) * kD;
                else flag(a);  // zeros instead
            }
            const unsigned keys_ok = __ballot_sync(0xffffffffu, in);
            float4 kk[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const long long at = __shfl_sync(0xffffffffu, off, i);
                kk[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (keys_ok >> i & 1) kk[i] = load4(kp + at + 4 * lane);
            }
            const int mine = lane / ROWS;  // of a batch's keys
#pragma unroll
            for (int i = 0; i < kEach; i += kBatch) {
                const int key = first + i + mine;
                const bool writes = r == 0 && key < p.s.len;
                const float before = writes ? w[key] : 0.f;
                float v[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    const float4 k4 = kk[i + x / ROWS], q4 = qq[x % ROWS];
                    v[x] = fmaf(k4.x, q4.x, fmaf(k4.y, q4.y, fmaf(k4.z, q4.z, k4.w * q4.w)));
                }
                const float s = reduce_32(v);
                float y = key < seen ? expf(fmaf(s, a.scale, minus_lse)) : 0.f;
#pragma unroll
                for (int o = 1; o < ROWS; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (writes) w[key] = before + y;
            }
        }
    }
}

static long long tiles_of(const Args &a) { return (long long)a.B * a.Hkv * (((long long)a.cols * a.page + kKeys - 1) / kKeys); }

template <int ROWS>
static cudaError_t launch_few(const Args &a, int sms, cudaStream_t stream) {
    const long long tiles = tiles_of(a), most = (ROWS == 8 ? 3LL : 4LL) * sms;
    return launch_early(few_kernel<ROWS>, dim3((unsigned)(tiles < most ? tiles : most)), kThreads, 0, stream, a);
}

cudaError_t launch_weights_f32(Args a, int sms, cudaStream_t stream) {
    if (a.T * a.G <= 8) return a.T * a.G <= 4 ? launch_few<4>(a, sms, stream) : launch_few<8>(a, sms, stream);
    const cudaError_t e = cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(kMostRows));
    if (e != cudaSuccess) return e;
    // One launch where a CTA has four tiles at the most, else tokens of as many rows as stay in shared memory to each.
    const int most = kMostRows / a.G, T = a.T;
    const long long tiles = tiles_of(a);
    const int launches = tiles <= 12LL * sms ? 1 : (T + most - 1) / most, per = (T + launches - 1) / launches;
    const long long ctas = (per * a.G > kRows ? 3LL : 4LL) * sms;
    for (int t0 = 0; t0 < T; t0 += per) {
        a.t0 = t0;
        a.t1 = t0 + per < T ? t0 + per : T;
        const int rows = (a.t1 - a.t0) * a.G > kRows ? kMostRows : kRows;
        const cudaError_t x = launch_early(weights_kernel, dim3((unsigned)(tiles < ctas ? tiles : ctas)), kThreads, smem_of(rows),
                                           stream, a);
        if (x != cudaSuccess) return x;
    }
    return cudaSuccess;
}

}  // namespace weights
}  // namespace kda
