// Joins the parts of items that more than one CTA worked on: for each row, over
// the parts in CTA order,
//   M = max_p m_p,  L = sum_p l_p e^{c (m_p - M)},  O = sum_p O_p e^{c (m_p - M)} / L.
// A block takes a share of the item that starts (unfinished) in CTA c = blockIdx.x;
// thread = (row, four channels), rows fastest, as the parts are laid out. The
// order of the sum is fixed, so a call gives the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn.cuh"
#include "kda_common.cuh"

namespace kda {
namespace attn {

constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 4;  // blocks per item

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 y) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}
__device__ __forceinline__ void store4(float *p, float4 y) { *reinterpret_cast<float4 *>(p) = y; }

template <typename IO>
__global__ void __launch_bounds__(kJoinThreads) attn_combine_kernel(const Args a, const int tile_rows) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int c0 = blockIdx.x;
    const PartHeader h = *part_header(a, 2 * c0 + 1);
    if (!h.valid) return;
    // the item's other parts are the first ones of the CTAs that follow
    int n = 1;
    while (c0 + n < a.ctas) {
        const PartHeader *x = part_header(a, 2 * (c0 + n));
        if (!x->valid) break;
        ++n;
        if (x->ends) break;
    }
    const float c = a.scale * kLog2e;
    // rows in the parts: stream s at tile_rows s
    const int first = h.tokens < a.tile_tokens ? h.tokens : a.tile_tokens;
    const int rows0 = first * a.G, rows = h.tokens * a.G;
    for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < rows * 32; i += kJoinBlocks * kJoinThreads) {
        const int q = i / rows, row = i - q * rows;
        const int at = row < rows0 ? row : tile_rows + row - rows0;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const int slot = k == 0 ? 2 * c0 + 1 : 2 * (c0 + k);
            const float2 ml = part_ml(a, slot)[at];
            const float4 y = reinterpret_cast<const float4 *>(part_o(a, slot))[(size_t)q * kPartRows + at];
            const float up = fmaxf(m, ml.x);
            if (up == -INFINITY) {  // nothing seen yet: l and O are 0, or NaN
                l += ml.y;
                continue;
            }
            const float f0 = exp2f((m - up) * c), f1 = exp2f((ml.x - up) * c);
            m = up;
            l = l * f0 + ml.y * f1;
            o.x = o.x * f0 + y.x * f1;
            o.y = o.y * f0 + y.y * f1;
            o.z = o.z * f0 + y.z * f1;
            o.w = o.w * f0 + y.w * f1;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int tok = row / a.G, head = h.kvh * a.G + row - tok * a.G;
        const size_t dst = (size_t)(h.token0 + tok) * a.Hq + head;
        store4(static_cast<IO *>(a.out) + dst * kD + 4 * q,
               make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (q == 0 && a.lse != nullptr) a.lse[dst] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
    }
}

cudaError_t launch_attn_combine(const Args &a, bool bf16, cudaStream_t stream) {
    if (a.ctas < 2) return cudaSuccess;
    // may start while the attention kernel still runs (it waits for its end)
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas, kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<__nv_bfloat16>, a, 128)
                : cudaLaunchKernelEx(&cfg, attn_combine_kernel<float>, a, 128);
}

}  // namespace attn
}  // namespace kda
