// Joins the parts of items that more than one CTA worked on: for each row, over
// the parts in CTA order,
//   M = max_p m_p,  L = sum_p l_p e^{c (m_p - M)},  O = sum_p O_p e^{c (m_p - M)} / L.
//
// Every block looks through the parts' headers (one load per thread), which gives it
// all split items and how many threads' worth of rows they have, and takes every
// gridDim-th chunk of that: a call may have one split item of a hundred parts or a
// hundred of two, and all SMs share either evenly. Thread = (row, four channels), eight rows
// and four quads to a warp, so that reads are 128 bytes (the parts are laid out rows
// fastest) and writes whole sectors; the loads of four parts are in flight at a time.
// With many parts (few rows over a long cache) eight lanes share a thread's work. The
// order of the sum is fixed, so a call gives the same bits every time.
//
// Bound by the parts' way through L2 and a chain of latencies (the headers, the search, a
// part): 7 us for 152 parts of 4 rows, 12 us for the 28 MB of a step of 64 drafts by eight
// users (cold caches). A grid with a column of blocks per CTA, most of them empty, took 12 us
// more for 24 items of 13 parts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn.cuh"
#include "kda_common.cuh"

namespace kda {
namespace attn {

constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 3;  // per SM (2, 3, 4: 37.7, 37.2, 38.4 us for an fp32 tree of 11 drafts on 6 short caches)

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
    const float2 f = join_factors(x.m, y.m, c);
    x.m = fmaxf(x.m, y.m);
    x.l = join_sum(x.l, f.x, y.l, f.y);
    x.o.x = join_sum(x.o.x, f.x, y.o.x, f.y);
    x.o.y = join_sum(x.o.y, f.x, y.o.y, f.y);
    x.o.z = join_sum(x.o.z, f.x, y.o.z, f.y);
    x.o.w = join_sum(x.o.w, f.x, y.o.w, f.y);
}

// Eight lanes per (row, quad), each with every eighth part? (One long sequence 51.5 us
// instead of 55.2, fp32 65.0 instead of 77.2; from four parts on: no better, 34.9 instead
// of 33.0 for an fp32 tree.)
__device__ __forceinline__ bool shared_work(int n, int rows) { return n > 8 && rows <= 32; }

// Chunk `chunk` of an item of n terms, the last of which is two parts with `pair`:
// kJoinThreads / SUB (row, quad) pairs. SUB neighbouring lanes share one, each with
// every SUB-th term.
template <typename IO, int SUB>
__device__ __forceinline__ void join_rows(const Args &a, const PartHeader &h, int c0, int n, bool pair, int tile_rows,
                                          int chunk) {
    const float c = a.scale * kLog2e;
    const int first = h.tokens < a.tile_tokens ? h.tokens : a.tile_tokens;
    const int rows0 = first * a.G, rows = h.tokens * a.G;  // rows in the parts: stream s at tile_rows s
    const int sub = threadIdx.x % SUB;
    const int i = chunk * (kJoinThreads / SUB) + (int)threadIdx.x / SUB;
    const int eights = (rows + 7) >> 3, block = i >> 5;
    const int q = block / eights * 4 + (i >> 3 & 3), row = block % eights * 8 + (i & 7);
    const bool in = q < 32 && row < rows;
    const int at = row < rows0 ? row : tile_rows + row - rows0;
    auto load = [&](int k) {
        const int slot = k == 0 ? 2 * c0 + 1 : 2 * (c0 + k);
        const float2 ml = part_ml(a, slot)[at];
        return Acc{ml.x, ml.y, reinterpret_cast<const float4 *>(part_o(a, slot))[(size_t)q * a.part_rows + at]};
    };
    Acc x = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    constexpr int kFlight = 4;  // parts whose loads are issued together
    for (int k0 = sub; k0 < n; k0 += kFlight * SUB) {
        Acc y[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int k = k0 + f * SUB;
            y[f] = Acc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            if (in && k < n) y[f] = load(k);
        }
        Acc z = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        const int f_last = pair && in && (n - 1 - k0) % SUB == 0 ? (n - 1 - k0) / SUB : -1;
        if (f_last >= 0 && f_last < kFlight) z = load(n);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            if (f == f_last) join(y[f], z, c);
            join(x, y[f], c);
        }
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
    if (!in || sub != 0) return;
    const float inv = x.l == 0.f ? 0.f : 1.f / x.l;
    const int tok = row / a.G, head = h.kvh * a.G + row - tok * a.G;
    const size_t dst = (size_t)(h.token0 + tok) * a.Hq + head;
    store4(static_cast<IO *>(a.out) + dst * kD + 4 * q, make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv));
    if (q == 0 && a.lse != nullptr) a.lse[dst] = x.l == 0.f ? -INFINITY : x.m * a.scale + logf(x.l);
}

template <typename IO>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) attn_combine_kernel(const Args a, const int tile_rows,
                                                                     const bool joins_early) {
    constexpr int kWords = kMaxCtas / 32;
    __shared__ uint32_t ends[kWords];  // bit c: CTA c's first part is an item's last one, or it has none
    __shared__ int sums[kJoinThreads / 32];
    __shared__ int starts[kMaxCtas + 1];  // chunks of the items that start before CTA c
    __shared__ int terms[kMaxCtas];       // of the item that starts in CTA c; bit 16: the last one is two parts
    __shared__ uint32_t joined[kWords];   // bit c: CTA c's first part holds the item's last one too
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_before();
    let_next_start();
    if (blockIdx.x == 0 && tid < kFlagWords) *early_flag(a, 32 * tid) = 0;
    constexpr int kRounds = kMaxCtas / kJoinThreads;
    int rows[kRounds];  // of the item that starts in CTA tid + kJoinThreads i, 0: none
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int c = tid + kJoinThreads * i;
        int end = kEnds;
        rows[i] = 0;
        if (c < a.ctas) {
            const PartHeader *x = part_header(a, 2 * c);
            if (x[0].valid) end = x[0].ends;
            if (x[1].valid) rows[i] = x[1].tokens * a.G;
        }
        const unsigned who = __ballot_sync(0xffffffffu, end != 0), both = __ballot_sync(0xffffffffu, end == kEndsJoined);
        if (lane == 0) {
            ends[c >> 5] = who;
            joined[c >> 5] = both;
        }
    }
    int any = 0;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) any |= rows[i];
    if (!__syncthreads_or(any)) return;
    int total = 0;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int c = tid + kJoinThreads * i;
        if (kJoinThreads * i >= a.ctas) {  // (nor do the rounds after this one have any)
            starts[c] = total;
            continue;
        }
        int n = 1, chunks = 0;
        if (rows[i] > 0) {  // its other parts are the first ones of the CTAs that follow
            int e = c + 1, w = e >> 5;
            uint32_t bits = w < kWords ? ends[w] & (~0u << (e & 31)) : 0u;
            while (bits == 0 && ++w < kWords) bits = ends[w];
            e = bits != 0 ? 32 * w + __ffs(bits) - 1 : a.ctas - 1;
            e = min(e, a.ctas - 1);
            n = e - c + 1;
            if (joins_early && !(joined[e >> 5] >> (e & 31) & 1) && n > 1) n = (n - 1) | 1 << 16;
            const int pairs = ((rows[i] + 7) & ~7) * 32 * (shared_work(n & 0xffff, rows[i]) ? 8 : 1);
            chunks = (pairs + kJoinThreads - 1) / kJoinThreads;
        }
        int incl = chunks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        terms[c] = n;
        starts[c] = total + before + incl - chunks;
        total += all;
        __syncthreads();  // sums is free
    }
    if (tid == 0) starts[kMaxCtas] = total;
    __syncthreads();
    for (int chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
        int lo = 0, hi = kMaxCtas;  // the last CTA whose chunks start at or before this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= chunk) lo = mid;
            else hi = mid;
        }
        const PartHeader h = *part_header(a, 2 * lo + 1);
        const int n = terms[lo] & 0xffff;
        const bool pair = terms[lo] >> 16;
        if (shared_work(n, h.tokens * a.G)) join_rows<IO, 8>(a, h, lo, n, pair, tile_rows, chunk - starts[lo]);
        else join_rows<IO, 1>(a, h, lo, n, pair, tile_rows, chunk - starts[lo]);
    }
}

cudaError_t launch_attn_combine(const Args &a, bool bf16, bool joins_early, cudaStream_t stream) {
    if (a.ctas < 2) return cudaSuccess;
    // at most the chunks that a.ctas items of all the rows that a part holds have
    const long long most = (long long)a.ctas * a.part_rows * 32 / kJoinThreads, blocks = (long long)kJoinBlocks * a.sms;
    return launch_early(bf16 ? attn_combine_kernel<__nv_bfloat16> : attn_combine_kernel<float>,
                        dim3((unsigned)(most < blocks ? most : blocks)), kJoinThreads, 0, stream, a, 128, joins_early);
}

}  // namespace attn
}  // namespace kda
