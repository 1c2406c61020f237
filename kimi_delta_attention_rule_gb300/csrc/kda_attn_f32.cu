// Softmax attention in fp32 on CUDA cores (the formulas and the work split are
// those of kda_attn.cuh): 128 threads hold 64 (token, head) rows, or 32, 24 or 8 where a
// kv head has no more (RPT = 8, 4, 3 or 1 rows per thread); per tile of 64 keys a thread
// forms an RPT x 4 piece of S = Q K^T and an RPT x 8 piece of O += P V, two products per
// instruction. With RPT = 8 a step of four channels loads 192 bytes per thread for 128
// FMAs, one of four keys 256 bytes for 256, so shared memory and the FMA pipe bound it
// alike: 173 us for 5.7 GFLOP of causal attention over 2,011 tokens, 33 TFLOP/s of the
// 75 that the FMA pipe has. With few rows it is the loads: 65 us for one token on 40,000 cached
// ones (164 MB, 2.5 TB/s), in a chain of copies that come while the tile before is multiplied
// (79 us when they did not). Two CTAs per SM.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kda_attn.cuh"
#include "kda_common.cuh"

namespace kda {
namespace attn {

constexpr int kF32Threads = 128;
constexpr int kF32Tile = 64;          // keys; rows: 8 RPT
// Q, K, V and P. Rows that a warp reads together would lie on the same banks: the 16-byte
// pieces of a K row stand in the order of (piece xor row % 8), of a Q row of (piece xor
// its thread row % 8), the 16-key groups of a P row of (group xor thread row % 2).
constexpr int f32_smem(int rpt) { return (8 * rpt * (kD + kF32Tile) + 2 * kF32Tile * kD) * 4; }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

struct F32Ptrs {
    const float *q, *k, *v, *kn, *vn;  // decode: k, v = pages
    long long ldq, ldk, ldv;           // decode: of kn, vn
};

template <bool PAGED, int RPT, bool WIN>
__global__ void __launch_bounds__(kF32Threads, 2) attn_f32_kernel(const __grid_constant__ Args a, const F32Ptrs io) {
    extern __shared__ __align__(16) float smf[];
    constexpr int kRows = 8 * RPT;
    float *const Qs = smf, *const Ks = Qs + kRows * kD, *const Vs = Ks + kF32Tile * kD, *const Ps = Vs + kF32Tile * kD;
    __shared__ Point pts[2];
    __shared__ Seq seq0;
    __shared__ int any;
    wait_before();
    if (a.direct) let_next_start();
    const int tid = threadIdx.x, cta = blockIdx.x;
    __shared__ Part direct;
    if (tid < 64) {  // one warp finds where this CTA's work starts, one where it ends
        const int w = tid >> 5;
        Point pt;
        Seq s0;
        Part p;
        bool ok = false;
        if (!a.direct) ok = split_point<PAGED, kF32Tile, WIN>(a, cta + w, pt, s0) && (w != 0 || pt.n < a.N);
        else if (w == 0) ok = direct_part<PAGED, kF32Tile, WIN>(a, cta, p);
        if ((tid & 31) == 0) {
            pts[w] = pt;
            if (w == 0) {
                if (a.direct) direct = p;
                else seq0 = s0;
                any = ok;
            } else if (!a.direct) {
                part_header(a, 2 * cta)->valid = 0;
                part_header(a, 2 * cta + 1)->valid = 0;
            }
        }
    }
    __syncthreads();
    if (!any) return;
    Walk<PAGED, kF32Tile, WIN> walk;
    if (!a.direct) walk.init(pts[0], pts[1], seq0);
    const int ty = tid >> 4, tx = tid & 15, lane = tid & 31, warp = tid >> 5;  // rows RPT ty + i; keys tx + 16 e, channels 4 tx + 64 e
    const float c = a.scale * kLog2e;
    const uint32_t inv_g = (65536u + a.G - 1) / a.G;  // r / G = r inv_g >> 16 for r < 1024
    const int G = a.G, page_bits = PAGED ? 31 - __clz(a.page) : 0;
    Part p = direct;
    for (bool more = a.direct || walk.next(a, p); more; more = !a.direct && walk.next(a, p)) {
        const int rows = p.tokens * G;
        __syncthreads();  // the last part's reads are done
        for (int x = tid; x < kRows * 32; x += kF32Threads) {
            const int r = x >> 5, ch = (x & 31) * 4, tok = (int)(r * inv_g >> 16);
            const bool ok = r < rows;
            const float *src = io.q + (ok ? (long long)(p.q0 + tok) * io.ldq + (p.h * G + r - tok * G) * kD + ch : 0);
            cp16(smem_u32(Qs + r * kD + (ch ^ (r / RPT % 8 * 4))), src, ok);
        }
        cp_commit();
        float m[RPT], l[RPT];
        float4 o[RPT][2];
        int seen[RPT];  // keys that the row sees (of the cache: all)
        unsigned long long bits[RPT];
        int from[RPT];  // WIN: the first key of the row's window
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            o[i][0] = o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int r = RPT * ty + i, t = p.first_tok + (int)(r * inv_g >> 16);
            seen[i] = PAGED ? p.Lk : p.Lk - p.Lq + t + 1;
            bits[i] = 0;
            int fresh = 1;  // WIN: the new tokens that it sees, itself counted in any case
            if (PAGED && r < rows) {
                bits[i] = a.mask != nullptr ? a.mask[(size_t)p.n * a.T + t]
                                            : (t >= 63 ? ~0ull : (2ull << t) - 1);
                if (a.T < 64) bits[i] &= (1ull << a.T) - 1;
                if (WIN) fresh = __popcll(bits[i] | 1ull << t);
            }
            if (WIN) from[i] = window_start(a, PAGED && a.has_new ? p.Lk + fresh : seen[i]);
        }
        // the first key of all rows' windows: those before it, the sinks apart, are not read
        const int first = WIN ? window_start(a, PAGED ? p.Lk + a.has_new : p.Lk - p.Lq + p.first_tok + 1) : 0;
        // WIN: keys of the item. Behind them a tile is not multiplied, as its items are short: 57 us instead of 63 for
        // 2,011 tokens and a window of 64, 116 instead of 122 for one of 300. (The plain calls' long prompts would
        // take 2 % more.)
        const int keys = (PAGED ? p.Lk : p.Lk - p.Lq + p.first_tok + p.tokens) - p.span.shift;
        // A warp copies the rows warp, warp + 4, ..: lane i knows where row warp + 4 i is.
        struct Where {
            long long k, v;
            unsigned rows_ok;
            bool drafts;
        };
        const int mine = warp + 4 * (lane & 15);
        auto locate = [&](int t) {
            Where w = {0, 0, 0, PAGED && a.has_new && t == p.nt - 1};
            const int pos = WIN ? p.span.key(t * kF32Tile + mine) : t * kF32Tile + mine;  // of this lane's row
            // keys past the end load as zeros (0 times what is there could be NaN)
            bool ok = w.drafts ? mine < a.T : pos < p.Lk;
            if (WIN && !w.drafts) ok = ok && (pos >= first || pos < a.sinks);
            if (!PAGED) {
                w.k = (long long)(p.k0 + pos) * io.ldk;
                w.v = (long long)(p.k0 + pos) * io.ldv;
            } else if (w.drafts) {
                w.k = (long long)(p.n * a.T + mine) * io.ldk;
                w.v = (long long)(p.n * a.T + mine) * io.ldv;
            } else if (ok) {
                const int pg = a.table[(size_t)p.n * a.table_ld + (pos >> page_bits)];
                ok = pg >= 0 && pg < a.pages;
                if (!ok) atomicOr(status_word(a), kStatusBadSeqlens);  // zeros instead
                else w.k = w.v = (((long long)pg * a.Hkv) * a.page + (pos & (a.page - 1))) * kD;
            }
            w.rows_ok = __ballot_sync(0xffffffffu, ok);
            return w;
        };
        auto copy = [&](const Where &w, bool is_v) {
            const long long head = (PAGED && !w.drafts ? (long long)p.h * a.page : p.h) * kD + 4 * lane;
            const float *const src = (is_v ? (w.drafts ? io.vn : io.v) : (w.drafts ? io.kn : io.k)) + head;
            float *const dst = is_v ? Vs : Ks;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const bool in = w.rows_ok >> i & 1;
                const long long off = __shfl_sync(0xffffffffu, is_v ? w.v : w.k, i);
                const int r = warp + 4 * i;
                cp16(smem_u32(dst + r * kD + (is_v ? 4 * lane : 4 * (lane ^ (r & 7)))), in ? src + off : io.q, in);
            }
        };
        // K of the next tile comes while this one's P V is formed, its V during the next Q K^T.
        Where next = {};
        if (p.ta < p.tb) {
            next = locate(p.ta);
            copy(next, false);
            cp_commit();
            copy(next, true);
            cp_commit();
        }
        for (int t = p.ta; t < p.tb; ++t) {
            const bool drafts = next.drafts;
            if (t + 1 < p.tb) next = locate(t + 1);
            cp_wait<1>();
            __syncthreads();
            // (two terms of a dot product per instruction, as two sums: half the issue slots)
            float2 s2[RPT][4] = {};
            const int valid = !WIN ? kF32Tile : (drafts ? a.T : min(keys - t * kF32Tile, kF32Tile));
            auto multiply = [&](auto groups) {  // of 16 keys
                constexpr int E = decltype(groups)::value;
#pragma unroll 4
                for (int d = 0; d < kD; d += 4) {
                    float4 kk[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) kk[e] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * e) * kD + (d ^ (tx % 8 * 4)));
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float4 qq = *reinterpret_cast<const float4 *>(Qs + (RPT * ty + i) * kD + (d ^ (ty % 8 * 4)));
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            s2[i][e] = fma2(make_float2(qq.x, qq.y), make_float2(kk[e].x, kk[e].y), s2[i][e]);
                            s2[i][e] = fma2(make_float2(qq.z, qq.w), make_float2(kk[e].z, kk[e].w), s2[i][e]);
                        }
                    }
                }
            };
            if (valid > 32) multiply(std::integral_constant<int, 4>());
            else multiply(std::integral_constant<int, 2>());
            float s[RPT][4];
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = s2[i][e].x + s2[i][e].y;
            __syncthreads();  // K is read
            if (t + 1 < p.tb) copy(next, false);
            cp_commit();
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = tx + 16 * e;
                    const int pos = WIN ? p.span.key(t * kF32Tile + key) : t * kF32Tile + key;
                    bool see = drafts ? (bits[i] >> key & 1) != 0 : seen[i] > pos;
                    if (WIN && !drafts) see = see && (pos >= from[i] || pos < a.sinks);
                    if (!see) s[i][e] = -INFINITY;
                    top = fmaxf(top, s[i][e]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float up = fmaxf(m[i], top);
                const float f = m[i] == -INFINITY ? 0.f : exp2f((m[i] - up) * c);
                const float uc = up == -INFINITY ? 0.f : up * c;
                m[i] = up;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = exp2f(fmaf(s[i][e], c, -uc));
                    sum += y;
                    Ps[(RPT * ty + i) * kF32Tile + tx + 16 * (e ^ (ty & 1))] = y;
                }
                l[i] = l[i] * f + sum;  // this lane's keys; joined at the end
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[i][e].x *= f;
                    o[i][e].y *= f;
                    o[i][e].z *= f;
                    o[i][e].w *= f;
                }
            }
            cp_wait<1>();
            __syncthreads();
            auto add_keys = [&](int key) {  // four of them
                float4 vv[4][2];
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        vv[x][e] = *reinterpret_cast<const float4 *>(Vs + (key + x) * kD + 4 * tx + 64 * e);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float4 pp = *reinterpret_cast<const float4 *>(Ps + (RPT * ty + i) * kF32Tile + (key ^ (ty % 2 * 16)));
                    const float w[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float2 w2 = make_float2(w[x], w[x]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 lo = fma2(w2, make_float2(vv[x][e].x, vv[x][e].y), make_float2(o[i][e].x, o[i][e].y));
                            const float2 hi = fma2(w2, make_float2(vv[x][e].z, vv[x][e].w), make_float2(o[i][e].z, o[i][e].w));
                            o[i][e] = make_float4(lo.x, lo.y, hi.x, hi.y);
                        }
                    }
                }
            };
            if constexpr (WIN) {
#pragma unroll 1
                for (int key = 0; key < valid; key += 8) {
                    add_keys(key);
                    add_keys(key + 4);
                }
            } else {
#pragma unroll 2
                for (int key = 0; key < kF32Tile; key += 4) add_keys(key);
            }
            __syncthreads();  // V and P are read
            if (t + 1 < p.tb) copy(next, true);
            cp_commit();
        }
        if (p.ta >= p.tb) cp_wait<0>();  // Q of a part without keys
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
            const int r = RPT * ty + i;
            if (r >= rows) continue;
            if (!p.whole()) {
                const int slot = part_slot(cta, p);
                float4 *o4 = reinterpret_cast<float4 *>(part_o(a, slot)) + r;
                o4[(size_t)tx * a.part_rows] = o[i][0];
                o4[(size_t)(16 + tx) * a.part_rows] = o[i][1];
                if (tx == 0) part_ml(a, slot)[r] = make_float2(m[i], l[i]);
                continue;
            }
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
            const int tok = (int)(r * inv_g >> 16);
            const size_t dst = (size_t)(p.q0 + tok) * a.Hq + p.h * G + r - tok * G;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + dst * kD + 4 * tx + 64 * e) =
                    make_float4(o[i][e].x * inv, o[i][e].y * inv, o[i][e].z * inv, o[i][e].w * inv);
            if (tx == 0 && a.lse != nullptr) a.lse[dst] = l[i] == 0.f ? -INFINITY : m[i] * a.scale + logf(l[i]);
        }
        if (tid == 0 && !p.whole()) {
            PartHeader *h = part_header(a, part_slot(cta, p));
            h->ends = p.tb == p.nt ? kEnds : 0;
            h->token0 = p.q0;
            h->tokens = p.tokens;
            h->kvh = p.h;
            h->valid = 1;
        }
    }
}

cudaError_t launch_attn_combine(const Args &a, bool bf16, bool joins_early, cudaStream_t stream);

// Through a window: whether each item goes to a CTA of its own, as many as there are. That leaves SMs idle in
// the last wave for as long as its items take; shared evenly the work costs a search and a join, as much as some
// more keys (144 for 64 rows, for fewer rows 256). Direct and split, us: 2,011 tokens of three prompts, 12
// heads on 4, window 64: 48, 57, 128: 70, 74, 200: 95, 91; 7 prompts of 50 tokens 14, 27; 4 drafts of 16 sequences,
// 32 heads on 8, window 128: 19, 25, 400: 37, 39; 11 of 6 sequences, 12 on 4, window 64: 24.1, 24.6, 128: 34, 29. (Items of more than 8 tiles differ too much; a prompt's CTA looks at all sequences; the
// division of slots is exact below 2^20.)
template <bool PAGED, int RPT>
static bool window_direct(const Args &a, long long slots, long long keys) {
    const long long room = 2LL * a.sms, waves = (slots + room - 1) / room;
    const long long own = (long long)a.window + a.sinks + (PAGED ? kF32Tile : a.block), longest = keys < own ? keys : own;
    return slots < (1 << 20) && (PAGED || a.N <= 256) && longest <= 8 * kF32Tile &&
           longest * (waves * room - slots) <= (RPT < 8 ? 256 : 144) * room;
}

template <bool PAGED, int RPT, bool WIN>
static cudaError_t launch_form(Args a, const F32Ptrs &io, cudaStream_t stream) {
    constexpr int rows = 8 * RPT;
    a.streams = 1;
    a.tile_tokens = PAGED && a.T * a.G < rows ? a.T : rows / a.G;
    a.extra = 64;  // (more of it, and cuts at two or three tiles: slower; through a window the same: 124, 144 us)
    a.extra_short = 0;
    a.min_part = kF32MinPart;
    set_block(a);
    a.cut = 1;
    const long long slots = PAGED ? (long long)a.N * a.Hkv * ((a.T + a.tile_tokens - 1) / a.tile_tokens)
                                  : ((long long)a.Tq_total / a.tile_tokens + a.N) * a.Hkv;
    long long keys = PAGED ? (long long)a.table_cols * a.page + kF32Tile : a.Tk;
    const bool own = WIN && window_direct<PAGED, RPT>(a, slots, keys);
    if (WIN) keys = set_window(a, keys, 1, 1);
    set_unit(a, (double)slots * ((double)keys + a.extra + kF32Tile));
    // (a CTA each for four prompts of 25 tokens: 14.3 us instead of 35.6)
    a.direct = own || (slots <= 2 * a.sms && keys <= 2 * kF32Tile);
    cudaError_t e = cudaFuncSetAttribute(attn_f32_kernel<PAGED, RPT, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         f32_smem(RPT));
    if (e != cudaSuccess) return e;
    e = launch_early(attn_f32_kernel<PAGED, RPT, WIN>, dim3(a.direct ? (unsigned)slots : (unsigned)a.ctas), kF32Threads,
                     f32_smem(RPT), stream, a, io);
    return e == cudaSuccess && !a.direct ? launch_attn_combine(a, false, false, stream) : e;
}

template <bool PAGED, int RPT>
static cudaError_t launch_f32(const Args &a, const F32Ptrs &io, cudaStream_t stream) {
    return a.window > 0 ? launch_form<PAGED, RPT, true>(a, io, stream) : launch_form<PAGED, RPT, false>(a, io, stream);
}

cudaError_t launch_attn_prefill_f32(const Args &a, const void *q, const void *k, const void *v, long long ldq,
                                    long long ldk, long long ldv, cudaStream_t stream) {
    const F32Ptrs io = {static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v),
                        nullptr, nullptr, ldq, ldk, ldv};
    return launch_f32<false, 8>(a, io, stream);
}
cudaError_t launch_attn_decode_f32(const Args &a, const void *q, const void *kp, const void *vp, const void *kn,
                                   const void *vn, long long ldq, long long ldk, long long ldv,
                                   cudaStream_t stream) {
    const F32Ptrs io = {static_cast<const float *>(q), static_cast<const float *>(kp), static_cast<const float *>(vp),
                        static_cast<const float *>(kn), static_cast<const float *>(vn), ldq, ldk, ldv};
    const int rows = a.T * a.G;
    // (RPT 8 or 1 for one token per kv head on 40,000: 95, 65 us; 8, 4 or 3 for the 22 rows of a tree of
    // 11 drafts on six caches of 1,500: 99, 36.0, 33.2 us)
    return rows <= 8    ? launch_f32<true, 1>(a, io, stream)
           : rows <= 24 ? launch_f32<true, 3>(a, io, stream)
           : rows <= 32 ? launch_f32<true, 4>(a, io, stream)
                        : launch_f32<true, 8>(a, io, stream);
}

}  // namespace attn
}  // namespace kda
