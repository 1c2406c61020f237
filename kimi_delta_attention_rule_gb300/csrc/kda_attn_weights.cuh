// The attention weight that cached tokens get from the last queries: the arguments and
// the work split that the kernels for bf16 and fp32 share.
//
//   w[b, h, j] += sum_i sum_g exp(scale q_ig . k_j - lse_ig),   j <= L - count + i,
//
// over the accepted tokens i of sequence b (the last `count` of its L cached ones) and
// the G query heads g of kv head h. With the lse of an attention call over these very keys (none
// through a window) the terms are its probabilities, so nothing is normalised here and every key is on its own.
//
// Work. All sequences' (kv head, key tile) pairs form one line, of which CTA c takes
// the part [U c / C, U (c + 1) / C): every CTA has as many tiles whatever the lengths
// are, and each weight is read, added to and written by one thread, so that a call gives the same
// bits every time.
#pragma once

#include <stdint.h>

#include "kda_common.cuh"

namespace kda {
namespace weights {

struct Args {
    const void *q;       // [B, T, Hq, 128], ldq elements from token to token
    long long ldq;
    const void *kp;      // [pages, Hkv, page, 128]
    const float *lse;    // [B, T, Hq]
    float *w;            // [B, Hkv, cap]
    const int32_t *index, *count;  // [B, T], [B], or NULL
    const int32_t *table, *lens;
    long long table_ld;
    int B, T, G, Hkv, cap, page, pages, cols;
    int t0, t1;          // the accepted tokens of this launch
    float scale;
    uint32_t *status;    // or NULL
    int lose, lose_at;   // tests: 1 + the warp that gives up, and at which of its waits (0: none does)
};

__device__ __forceinline__ void flag(const Args &a) {
    if (a.status != nullptr) atomicOr(a.status, kStatusBadSeqlens);
}

// One sequence: cached tokens, accepted tokens, those of this launch.
struct Seq {
    int len, count, tokens;
};
// tokens = 0: nothing to do (malformed: said so).
__device__ __forceinline__ Seq load_seq(const Args &a, int b, bool says) {
    Seq s;
    s.len = a.lens[b];
    s.count = a.count != nullptr ? a.count[b] : a.T;
    const bool ok = s.len >= 0 && s.len <= a.cap && (long long)s.len <= (long long)a.cols * a.page && s.count >= 0 &&
                    s.count <= a.T;
    if (!ok && says) flag(a);
    s.tokens = ok && s.len > 0 ? max(0, min(a.t1, s.count) - a.t0) : 0;
    return s;
}
__device__ __forceinline__ int seq_tiles(const Seq &s, int kt) { return s.tokens > 0 ? (int)(((unsigned)s.len + kt - 1) / kt) : 0; }

// Tiles [ta, tb) of (b, h).
struct Part {
    int b, h, ta, tb;
    Seq s;
};
// The parts of a CTA, one after the other; the same for all lanes of a converged warp.
template <int KT>
struct Walk {
    long long left;  // tiles that this CTA still has
    int b, h, tile;
    Seq s;
    __device__ __forceinline__ void init(const Args &a, int c, int ctas) {
        const int lane = threadIdx.x & 31;
        long long total = 0;
        for (int n = lane; n < a.B; n += 32) total += seq_tiles(load_seq(a, n, c == 0), KT);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= a.Hkv;
        long long x = total * c / ctas;
        left = total * (c + 1) / ctas - x;
        b = h = tile = 0;
        if (left == 0) return;
        for (int n0 = 0; n0 < a.B; n0 += 32) {  // (x is below the total)
            Seq mine = {0, 0, 0};
            if (n0 + lane < a.B) mine = load_seq(a, n0 + lane, false);
            const long long tiles = (long long)seq_tiles(mine, KT) * a.Hkv;
            long long incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const long long sum = __shfl_sync(0xffffffffu, incl, 31);
            if (x >= sum) {
                x -= sum;
                continue;
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, x < incl)) - 1;
            x -= __shfl_sync(0xffffffffu, incl - tiles, src);
            b = n0 + src;
            s.len = __shfl_sync(0xffffffffu, mine.len, src);
            s.count = __shfl_sync(0xffffffffu, mine.count, src);
            s.tokens = __shfl_sync(0xffffffffu, mine.tokens, src);
            const int per = seq_tiles(s, KT);
            h = (int)(x / per);
            tile = (int)(x - (long long)h * per);
            return;
        }
        left = 0;  // (lengths that changed under the call)
    }
    __device__ __forceinline__ bool next(const Args &a, Part &p) {
        if (left == 0) return false;
        while (tile == 0 && h == 0 && seq_tiles(s, KT) == 0) {
            if (++b >= a.B) return false;  // (lengths that changed under the call)
            s = load_seq(a, b, false);
        }
        const int per = seq_tiles(s, KT), here = (int)min((long long)(per - tile), left);
        p.b = b;
        p.h = h;
        p.ta = tile;
        p.tb = tile + here;
        p.s = s;
        left -= here;
        tile = 0;
        if (p.tb == per && ++h == a.Hkv) {
            h = 0;
            s.tokens = 0;  // the next sequence, if any tile is left
        }
        return true;
    }
};

// The token of q that accepted token i (of t0 + i) is; -1: malformed.
__device__ __forceinline__ int token_of(const Args &a, int b, int i) {
    if (a.index == nullptr) return i;
    const int t = a.index[(size_t)b * a.T + i];
    if (t >= 0 && t < a.T) return t;
    flag(a);
    return -1;
}

}  // namespace weights
}  // namespace kda
