// Joins the parts of items that more than one CTA worked on: for each row, over
// the parts in CTA order,
//   M = max_p m_p,  L = sum_p l_p e^{c (m_p - M)},  O = sum_p O_p e^{c (m_p - M)} / L.
// A block takes a share of the item that starts (unfinished) in CTA c = blockIdx.x;
// thread = (row, four channels), rows fastest, as the parts are laid out; the loads
// of four parts are in flight at a time. With many parts (few rows over a long
// cache) eight lanes share a thread's work. The
// order of the sum is fixed, so a call gives the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn.cuh"
#include "kda_common.cuh"

namespace kda {
namespace attn {

constexpr int kJoinThreads = 128;

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 y) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}
__device__ __forceinline__ void store4(float *p, float4 y) { *reinterpret_cast<float4 *>(p) = y; }

struct Acc {
    float m, l;
    float4 o;
};
// x = x + y, both relative to their own maxima
__device__ __forceinline__ void join(Acc &x, const Acc &y, float c) {
    const float up = fmaxf(x.m, y.m);
    // (-inf: no key seen; l and O are 0, or NaN)
    const float f = x.m == -INFINITY ? 1.f : exp2f((x.m - up) * c), g = y.m == -INFINITY ? 1.f : exp2f((y.m - up) * c);
    x.m = up;
    x.l = x.l * f + y.l * g;
    x.o.x = x.o.x * f + y.o.x * g;
    x.o.y = x.o.y * f + y.o.y * g;
    x.o.z = x.o.z * f + y.o.z * g;
    x.o.w = x.o.w * f + y.o.w * g;
}

// SUB neighbouring lanes share a (row, quad), each with every SUB-th part.
template <typename IO, int SUB>
__device__ __forceinline__ void join_rows(const Args &a, const PartHeader &h, int c0, int n, int tile_rows) {
    const float c = a.scale * kLog2e;
    const int first = h.tokens < a.tile_tokens ? h.tokens : a.tile_tokens;
    const int rows0 = first * a.G, rows = h.tokens * a.G;  // rows in the parts: stream s at tile_rows s
    const int sub = threadIdx.x % SUB;
    const int groups = kJoinThreads / SUB * (int)gridDim.y;
    for (int i0 = blockIdx.y * (kJoinThreads / SUB); i0 < rows * 32; i0 += groups) {
        const int i = i0 + (int)threadIdx.x / SUB;
        const bool in = i < rows * 32;
        const int q = in ? i / rows : 0, row = in ? i - q * rows : 0;
        const int at = row < rows0 ? row : tile_rows + row - rows0;
        Acc x = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        constexpr int kFlight = 4;  // parts whose loads are issued together
        for (int k0 = sub; k0 < n; k0 += kFlight * SUB) {
            Acc y[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const int k = k0 + f * SUB, slot = k == 0 ? 2 * c0 + 1 : 2 * (c0 + k);
                y[f] = Acc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
                if (k < n) {
                    const float2 ml = part_ml(a, slot)[at];
                    y[f].m = ml.x;
                    y[f].l = ml.y;
                    y[f].o = reinterpret_cast<const float4 *>(part_o(a, slot))[(size_t)q * a.part_rows + at];
                }
            }
#pragma unroll
            for (int f = 0; f < kFlight; ++f) join(x, y[f], c);
        }
#pragma unroll
        for (int w = 1; w < SUB; w <<= 1) {
            Acc y;
            y.m = __shfl_xor_sync(0xffffffffu, x.m, w);
            y.l = __shfl_xor_sync(0xffffffffu, x.l, w);
            y.o.x = __shfl_xor_sync(0xffffffffu, x.o.x, w);
            y.o.y = __shfl_xor_sync(0xffffffffu, x.o.y, w);
            y.o.z = __shfl_xor_sync(0xffffffffu, x.o.z, w);
            y.o.w = __shfl_xor_sync(0xffffffffu, x.o.w, w);
            join(x, y, c);
        }
        if (!in || sub != 0) continue;
        const float inv = x.l == 0.f ? 0.f : 1.f / x.l;
        const int tok = row / a.G, head = h.kvh * a.G + row - tok * a.G;
        const size_t dst = (size_t)(h.token0 + tok) * a.Hq + head;
        store4(static_cast<IO *>(a.out) + dst * kD + 4 * q,
               make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv));
        if (q == 0 && a.lse != nullptr) a.lse[dst] = x.l == 0.f ? -INFINITY : x.m * a.scale + logf(x.l);
    }
}

template <typename IO>
__global__ void __launch_bounds__(kJoinThreads) attn_combine_kernel(const Args a, const int tile_rows) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int c0 = blockIdx.x;
    const PartHeader h = *part_header(a, 2 * c0 + 1);
    if (!h.valid) return;
    // the item's other parts are the first ones of the CTAs that follow: every
    // warp looks at 32 of them at a time
    const int lane = threadIdx.x & 31;
    int n = 1;
    while (true) {
        const int k = c0 + n + lane;
        int ends = 1;
        if (k < a.ctas) {
            const PartHeader *x = part_header(a, 2 * k);
            ends = !x->valid || x->ends;
        }
        const unsigned who = __ballot_sync(0xffffffffu, ends);
        if (who != 0) {
            n += __ffs(who);
            break;
        }
        n += 32;
    }
    if (c0 + n > a.ctas) n = a.ctas - c0;
    if (n <= 8 || h.tokens * a.G > 32) join_rows<IO, 1>(a, h, c0, n, tile_rows);
    else join_rows<IO, 8>(a, h, c0, n, tile_rows);
}

cudaError_t launch_attn_combine(const Args &a, bool bf16, cudaStream_t stream) {
    if (a.ctas < 2) return cudaSuccess;
    // may start while the attention kernel still runs (it waits for its end)
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // a thread per (row, quad) of an item where the rows are few, two items of a
    // row's quads per thread at most where they are many
    const int rows = a.tile_tokens * a.streams * a.G;
    cfg.gridDim = dim3((unsigned)a.ctas, (unsigned)(rows <= 32 ? 8 : rows / 8 < 32 ? rows / 8 + 1 : 32));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<__nv_bfloat16>, a, 128)
                : cudaLaunchKernelEx(&cfg, attn_combine_kernel<float>, a, 128);
}

}  // namespace attn
}  // namespace kda
