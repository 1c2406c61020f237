// Attention weights in fp32 on CUDA cores (the formula and the work split are those of
// kda_attn_weights.cuh): 128 threads take tiles of 64 keys; a thread forms a 4 x RPT piece
// of S = K Q^T for 8 RPT rows at a time (RPT = 1 where there are no more than eight, else 4), its
// exponentials, and their sum over its rows; the eight threads of a key add up in shared memory in a
// fixed order. Several CTAs per SM hide one another's loads.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn_weights.cuh"
#include "kda_common.cuh"

namespace kda {
namespace weights {

constexpr int kThreads = 128, kKeys = 64;
// Rows of K and Q are read by neighbouring threads: the 16-byte pieces of a row stand in the order
// of (piece xor row % 8).
constexpr int smem_of(int rows) { return (kKeys + rows) * kD * 4 + 8 * kKeys * 4 + rows * 8; }

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

__device__ __forceinline__ void cp16(float *dst, const float *src, bool ok) {  // (not ok: zeros)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}

template <int RPT>
__global__ void __launch_bounds__(kThreads, 4) weights_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int kRows = 8 * RPT;
    float *const Ks = sm, *const Qs = Ks + kKeys * kD, *const sums = Qs + kRows * kD, *const minus_lse = sums + 8 * kKeys;
    int *const seen = reinterpret_cast<int *>(minus_lse + kRows);  // keys that a row sees
    wait_before();
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
    const float *const q = static_cast<const float *>(a.q), *const kp = static_cast<const float *>(a.kp);
    const int Hq = a.Hkv * a.G, page_bits = 31 - __clz(a.page);
    Walk<kKeys> walk;
    walk.init(a, blockIdx.x, gridDim.x);
    Part p;
    while (walk.next(a, p)) {
        const int rows = p.s.tokens * a.G;
        for (int t = p.ta; t < p.tb; ++t) {
            __syncthreads();  // the last tile is through
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
            for (int r0 = 0; r0 < rows; r0 += kRows) {
                if (r0 > 0) __syncthreads();  // the last rows are read
                if (rows > kRows || t == p.ta) {
                    for (int r = warp; r < kRows; r += kThreads / 32) {
                        const int i = (r0 + r) / a.G, g = r0 + r - i * a.G;
                        int tok = r0 + r < rows ? token_of(a, p.b, a.t0 + i) : -1;
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                        float l = -INFINITY;
                        if (tok >= 0) {
                            x = load4(q + ((size_t)p.b * a.T + tok) * a.ldq + (size_t)(p.h * a.G + g) * kD + 4 * lane);
                            l = a.lse[((size_t)p.b * a.T + tok) * Hq + p.h * a.G + g];
                        }
                        *reinterpret_cast<float4 *>(Qs + r * kD + 4 * (lane ^ (r & 7))) = x;
                        if (lane == 0) {
                            minus_lse[r] = -l;
                            seen[r] = l == -INFINITY ? 0 : p.s.len - p.s.count + a.t0 + i + 1;
                        }
                    }
                }
                asm volatile("cp.async.wait_group 0;\n" ::: "memory");
                __syncthreads();
                float s[4][RPT] = {};
#pragma unroll 4
                for (int d = 0; d < kD; d += 4) {
                    float4 kk[4], qq[RPT];
#pragma unroll
                    for (int e = 0; e < 4; ++e) kk[e] = load4(Ks + (tx + 16 * e) * kD + (d ^ ((tx & 7) * 4)));
#pragma unroll
                    for (int i = 0; i < RPT; ++i) qq[i] = load4(Qs + (ty + 8 * i) * kD + (d ^ (ty * 4)));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < RPT; ++i) {
                            s[e][i] = fmaf(kk[e].x, qq[i].x, s[e][i]);
                            s[e][i] = fmaf(kk[e].y, qq[i].y, s[e][i]);
                            s[e][i] = fmaf(kk[e].z, qq[i].z, s[e][i]);
                            s[e][i] = fmaf(kk[e].w, qq[i].w, s[e][i]);
                        }
                }
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int r = ty + 8 * i;
                    const float l = minus_lse[r];
                    const int n = seen[r];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t * kKeys + tx + 16 * e < n) sum[e] += expf(fmaf(s[e][i], a.scale, l));
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

template <int RPT>
static cudaError_t launch_form(const Args &a, int sms, cudaStream_t stream) {
    constexpr int bytes = smem_of(8 * RPT);
    const cudaError_t e = cudaFuncSetAttribute(weights_kernel<RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.B * a.Hkv * (((long long)a.cols * a.page + kKeys - 1) / kKeys), most = 4LL * sms;
    return launch_early(weights_kernel<RPT>, dim3((unsigned)(tiles < most ? tiles : most)), kThreads, bytes, stream, a);
}

cudaError_t launch_weights_f32(const Args &a, int sms, cudaStream_t stream) {
    return a.T * a.G <= 8 ? launch_form<1>(a, sms, stream) : launch_form<4>(a, sms, stream);
}

}  // namespace weights
}  // namespace kda
