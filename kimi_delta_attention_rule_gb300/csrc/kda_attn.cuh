// Softmax attention: the arguments and the work split that the tensor-core
// kernel (bf16, kda_attn_tc.cu), the CUDA-core kernel (fp32, kda_attn_f32.cu)
// and the kernel that joins split rows (kda_attn_combine.cu) share.
//
// Work. An item is (sequence, kv head, row block): the rows of a block are
// (token, query head of the group) pairs, token major, so that the G query
// heads that share a kv head share every K and V tile that is loaded. A row
// block is `streams` tiles of `tile_tokens` tokens (tile_tokens * G rows at
// most per tile). An item's keys are cut into tiles of `kt` keys; with drafts,
// the last tile holds the drafts alone.
//
// Split. All items, in order, form one line of weighted work (their visible
// keys plus a fixed share for an item's start and end); CTA c takes the part
// [U c / C, U (c + 1) / C) of it, cut at key tiles. So every CTA has the same
// load whatever the lengths are, one long sequence spreads over all SMs, and a
// CTA has at most two parts of items: its first (which starts inside an item)
// and its last (which ends inside one). Those write (O, m, l) to the workspace and
// the join kernel adds them up in CTA order; all others write their rows. (A join by
// the CTA that finishes an item last saves a launch, 4 us of host time, but one SM
// waits for all the parts' loads: 5 to 20 us more on calls with many parts.) Few and
// short items go to a CTA each (`direct`), without the search and without a join.
//
// Early parts. A CTA's first part is done long before its neighbour's last one, so
// where it ends the item, the neighbour adds it to its own rows as it writes them
// (`joins_early`, row tiles of 128): items of two parts, nearly all of them with long
// prompts, then need no second pass. Nobody waits: a part that is not there yet is left to
// the join kernel, which adds the last two parts first, so that the bits are the same.
#pragma once

#include <stdint.h>

#include "kda_common.cuh"

namespace kda {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// The factors that bring two partial sums (of maxima m0 and m1) to their common maximum.
// (-inf: no key seen; l and O are 0, or NaN)
__device__ __forceinline__ float2 join_factors(float m0, float m1, float c) {
    const float up = fmaxf(m0, m1);
    return make_float2(m0 == -INFINITY ? 1.f : ex2((m0 - up) * c), m1 == -INFINITY ? 1.f : ex2((m1 - up) * c));
}
// x f + y g, rounded alike wherever two parts are joined
__device__ __forceinline__ float join_sum(float x, float f, float y, float g) {
    return __fmaf_rn(x, f, __fmul_rn(y, g));
}

constexpr int kMaxDrafts = 64;  // a row's draft mask has 64 bits
// Keys of work (an item's start and end included) below which no further CTA is used.
constexpr int kTcMinPart = 384, kF32MinPart = 128;
constexpr int kMaxCtas = 512;  // CTAs of a call

// Workspace: status word, the early parts' flags and padding (256 bytes), the parts'
// headers, then per part slot O (fp32, [32 channel quads][part_rows][4]) and m, l
// ([part_rows] each).
constexpr size_t kWsHeader = 256;
// Bit c: CTA c's first part ends its item and is written. All zero between calls: the
// join kernel clears them.
constexpr int kFlagsAt = 64, kFlagWords = kMaxCtas / 32;
static_assert(kFlagsAt + 4 * kFlagWords <= (int)kWsHeader, "the flags");
constexpr int kEnds = 1, kEndsJoined = 2;
struct PartHeader {
    int32_t valid;      // this slot holds a part of an item
    int32_t ends;       // kEnds: the item's last part; kEndsJoined: with the last part added
    int32_t token0;     // first token row of the item in q / out
    int32_t tokens;     // valid tokens of the item
    int32_t kvh;        // kv head
    int32_t pad[3];
};
__host__ __device__ inline size_t part_stride(int part_rows) { return (size_t)part_rows * (kD * 4 + 8); }
__host__ __device__ inline size_t headers_bytes(int ctas) {
    return ((size_t)2 * ctas * sizeof(PartHeader) + 255) / 256 * 256;
}
__host__ __device__ inline size_t workspace_bytes(int ctas, int part_rows) {
    return kWsHeader + headers_bytes(ctas) + (size_t)2 * ctas * part_stride(part_rows);
}

// Arguments shared by the kernels (prefill: packed rows; decode: pages).
struct Args {
    // sizes
    int N, Hq, Hkv, G;       // sequences, heads, Hq / Hkv
    int T;                   // decode: new tokens per sequence; prefill: query rows of an equal-length sequence
    int Tk;                  // prefill: keys of an equal-length sequence
    int Tq_total, Tk_total;  // prefill: packed totals
    int page, pages, table_cols;
    long long table_ld;
    int has_new;             // decode: k_new / v_new given
    int tile_tokens;         // tokens of a row tile
    int streams;             // row tiles of an item: 2, or 1 when both streams share one row tile
    int extra;               // an item's start and end, in keys: decode: at least
    int extra_short;         // extra_short less half of the item's own keys
    int min_part;            // keys of work below which no further CTA is used
    int cut;                 // tiles that a part of an item has at least
    int direct;              // one CTA for each slot of an item, nothing is split
    float unit, inv_unit;    // keys per unit of weight, and its inverse
    int block;               // tokens of an item: tile_tokens * streams
    uint32_t block_mul;      // x / block = x block_mul >> block_shift, for x < 2^31
    int block_shift;
    float inv_block, inv_min_part;
    float scale;
    // device pointers
    const int32_t *cu_q, *cu_k;      // prefill offsets (NULL: equal lengths)
    const int32_t *table, *lens;     // decode
    const unsigned long long *mask;  // decode, NULL: the chain
    void *out;
    float *lse;
    unsigned char *ws;
    int ctas, sms;           // CTAs that share the work; SMs of the device
    int part_rows;           // rows of a part in the workspace: those of an item at the most
    int lose, lose_at;       // tests: 1 + the warp that gives up, and at which of its waits (0: none does)
};

// The unit of weight: `keys` is an upper bound of a call's work in keys, of at most
// kMaxItems items.
constexpr long long kMaxItems = 1LL << 29;
inline void set_unit(Args &a, double keys) {
    a.unit = 1.f;
    while (keys / a.unit > 5e8) a.unit *= 2.f;
    a.inv_unit = 1.f / a.unit;
}

// What divides by tile_tokens * streams. The search for a CTA's work is a chain of
// dependent operations ahead of everything else, so none of it is a division of a
// hundred cycles. With s = floor(log2 block) and m = ceil(2^(32 + s) / block), the quotient of x is
// exact if x (m block - 2^(32 + s)) < 2^(32 + s): the bracket is below block < 2^(s + 1), x below 2^31.
inline void set_block(Args &a) {
    a.block = a.tile_tokens * a.streams;
    int s = 0;
    while ((2 << s) <= a.block) ++s;
    const bool power = (1 << s) == a.block;  // then block_mul would have 33 bits
    a.block_shift = power ? 31 + s : 32 + s;
    a.block_mul = (uint32_t)((((uint64_t)1 << a.block_shift) + a.block - 1) / a.block);
    a.inv_block = 1.f / (float)a.block;
    a.inv_min_part = 1.f / (float)a.min_part;
}
__device__ __forceinline__ int div_block(const Args &a, int x) {  // x >= 0
    return (int)(((uint64_t)(uint32_t)x * a.block_mul) >> a.block_shift);
}
// x / d for x < 2^30 and a quotient below 2^20: the estimate is off by one at most.
__device__ __forceinline__ uint32_t quick_div(uint32_t x, uint32_t d, uint32_t &rest) {
    uint32_t q = (uint32_t)__fdividef((float)x, (float)d);
    rest = x - q * d;
    if ((int)rest < 0) {
        --q;
        rest += d;
    } else if (rest >= d) {
        ++q;
        rest -= d;
    }
    return q;
}

__device__ __forceinline__ uint32_t *status_word(const Args &a) {
    return reinterpret_cast<uint32_t *>(a.ws);
}
__device__ __forceinline__ uint32_t *early_flag(const Args &a, int cta) {  // bit cta % 32 of it
    return reinterpret_cast<uint32_t *>(a.ws + kFlagsAt) + (cta >> 5);
}
__device__ __forceinline__ PartHeader *part_header(const Args &a, int slot) {
    return reinterpret_cast<PartHeader *>(a.ws + kWsHeader) + slot;
}
__device__ __forceinline__ float *part_o(const Args &a, int slot) {
    return reinterpret_cast<float *>(a.ws + kWsHeader + headers_bytes(a.ctas) +
                                     (size_t)slot * part_stride(a.part_rows));
}
__device__ __forceinline__ float2 *part_ml(const Args &a, int slot) {
    return reinterpret_cast<float2 *>(part_o(a, slot) + (size_t)a.part_rows * kD);
}

// One sequence. ok = false: malformed lengths.
struct Seq {
    int q0, Lq;  // first query row, query tokens
    int k0, Lk;  // prefill: first key row, keys; decode: Lk = cached tokens
    int ni;      // items per kv head
};
template <bool PAGED>
__device__ __forceinline__ bool load_seq(const Args &a, int n, Seq &s) {
    bool ok = true;
    if (PAGED) {
        s.q0 = n * a.T;
        s.Lq = a.T;
        s.k0 = 0;
        s.Lk = a.lens[n];
        ok = s.Lk >= 0 && (long long)s.Lk <= (long long)a.table_cols * a.page;
    } else {
        int q1, k1;
        if (a.cu_q != nullptr) {
            s.q0 = a.cu_q[n];
            q1 = a.cu_q[n + 1];
        } else {
            s.q0 = n * a.T;
            q1 = s.q0 + a.T;
        }
        if (a.cu_k != nullptr) {
            s.k0 = a.cu_k[n];
            k1 = a.cu_k[n + 1];
        } else {
            s.k0 = n * a.Tk;
            k1 = s.k0 + a.Tk;
        }
        ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.Tq_total && s.k0 >= 0 && k1 >= s.k0 &&
             k1 <= a.Tk_total && (n != 0 || (s.q0 == 0 && s.k0 == 0));
        s.Lq = q1 - s.q0;
        s.Lk = k1 - s.k0;
    }
    if (!ok) s.Lq = 0;
    s.ni = div_block(a, s.Lq) + (s.Lq - div_block(a, s.Lq) * a.block > 0);
    return ok;
}
// Keys that the last row of item i sees (prefill), or all keys (decode).
template <bool PAGED>
__device__ __forceinline__ int item_keys(const Args &a, const Seq &s, int i) {
    if (PAGED) return s.Lk;
    const int left = (int)((unsigned)s.Lq - (unsigned)(i + 1) * (unsigned)a.block);  // tokens after the item
    const int v = left > 0 ? s.Lk - left : s.Lk;
    return v > 0 ? v : 0;
}
template <bool PAGED, int KT>
__device__ __forceinline__ int item_tiles(const Args &a, const Seq &s, int i) {
    return (int)(((unsigned)item_keys<PAGED>(a, s, i) + KT - 1) / KT) + (PAGED ? a.has_new : 0);
}
// An item's start and end, in keys. (Decode: an item of few tiles is a chain of
// latencies, one of many is bound by its loads.)
template <bool PAGED, int KT>
__device__ __forceinline__ int item_extra(const Args &a, int nt) {
    return PAGED ? max(a.extra, a.extra_short - nt * (KT / 2)) : a.extra;
}
// Weight of items 0 .. i - 1 of one kv head: an arithmetic series of visible keys and
// the items' starts and ends, in units of a.unit keys, which the host chooses so that a
// call's total stays below 2^30, and one unit per item, so that no item weighs
// nothing. Formed in fp32: every operation rounds monotonically, so the weights rise
// with i, and all that follows is in whole units.
template <bool PAGED, int KT>
__device__ __forceinline__ uint32_t items_weight(const Args &a, const Seq &s, int i) {
    float w;
    if (PAGED) {
        const int nt = item_tiles<PAGED, KT>(a, s, 0);
        w = (float)i * (float)(item_extra<PAGED, KT>(a, nt) + nt * KT);
    } else {
        const int d = s.Lk - s.Lq, full = i < s.ni ? i : s.ni - 1;  // items without the sequence's last token
        const float block = (float)a.block;
        const float unseen = fmaxf(0.f, floorf((float)-d * a.inv_block));  // items that see nothing
        const float count = fmaxf(0.f, (float)full - unseen);
        // the last rows of items `unseen` .. full - 1 see d + block (unseen + 1) .. keys
        w = (float)i * (float)a.extra + count * fmaf(0.5f * block, (float)full + unseen + 1.f, (float)d);
        if (i >= s.ni) w += (float)s.Lk;
    }
    return (uint32_t)(fmaxf(w, 0.f) * a.inv_unit) + (uint32_t)i;
}

// A point on the line of work: before tile `tile` of item (n, h, i).
struct Point {
    int n, h, i, tile;
};
__device__ __forceinline__ bool same_item(const Point &x, const Point &y) {
    return x.n == y.n && x.h == y.h && x.i == y.i;
}

// The point at distance x into sequence n (of this weight per head, x below all heads');
// a converged warp with the same arguments in all lanes.
template <bool PAGED, int KT>
__device__ __forceinline__ Point point_in_seq(const Args &a, const Seq &s, int n, uint32_t per_head, uint32_t x) {
    const int lane = threadIdx.x & 31;
    Point p;
    p.n = n;
    p.h = (int)quick_div(x, per_head, x);
    int lo = 0, count = s.ni;  // the last item that starts at or before x is in [lo, lo + count)
    while (count > 1) {
        const int step = (count + 31) >> 5, at = lo + lane * step;
        const bool before = lane * step < count && items_weight<PAGED, KT>(a, s, at) <= x;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, before));  // (lane 0 always is)
        count = min(step, count - k * step);
        lo += k * step;
    }
    p.i = lo;
    const int nt = item_tiles<PAGED, KT>(a, s, lo);
    const float y = (float)(x - items_weight<PAGED, KT>(a, s, lo)) * a.unit - 0.5f * (float)item_extra<PAGED, KT>(a, nt);
    const int t = (int)fminf(fmaxf(0.f, y * (1.f / KT) + 0.5f), (float)nt);
    // short pieces are not worth their join: such a cut moves to the item's edge
    p.tile = t < a.cut ? 0 : (t > nt - a.cut ? nt : t);
    return p;
}

// Finds, with one converged warp, the point at U c / C (at the line's end: n = N).
// Returns false when CTA c has no part, or the offsets are malformed (which sets the
// status bit; the whole call is then skipped). A decode sequence with a malformed
// length is flagged and skipped alone. s0 gets the point's sequence. (It runs once,
// before everything else that a CTA does, from a cold instruction cache: short code
// counts more than few operations. A kernel calls it in one place, inlined, so that the
// arguments are read from the constant bank.)
template <bool PAGED, int KT>
__device__ __forceinline__ bool split_point(const Args &a, int c, Point &p0, Seq &s0) {
    const int lane = threadIdx.x & 31;
    constexpr int kFlight = PAGED ? 4 : 1;  // groups of 32 sequences whose loads are in flight together
    uint32_t w[kFlight], total = 0, per_head = 1;  // w: a head's
    auto weigh = [&](int n0) {
        bool ok = true;
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int n = n0 + 32 * u + lane;
            Seq s;
            w[u] = 0;
            if (n < a.N) {
                ok = load_seq<PAGED>(a, n, s) && ok;
                if (s.ni > 0) w[u] = items_weight<PAGED, KT>(a, s, s.ni);
            }
        }
        return ok;
    };
    bool good = true;
#pragma unroll 1
    for (int n0 = 0; n0 < a.N; n0 += 32 * kFlight) {
        good = weigh(n0) && good;
#pragma unroll
        for (int u = 0; u < kFlight; ++u) total += w[u];
    }
    total = __reduce_add_sync(0xffffffffu, total) * (uint32_t)a.Hkv;
    if (!__all_sync(0xffffffffu, good)) {
        if (lane == 0) atomicOr(status_word(a), kStatusBadSeqlens);
        if (!PAGED) return false;
    }
    if (total == 0) return false;
    // (single precision: a cut may lie anywhere, but for all CTAs at the same place)
    const float units = (float)total;
    // at least min_part keys and two units each: the cuts inside an item are at
    // different tiles, and every CTA from an item's first to its last has a part of it
    const int ctas = max(1, (int)fminf((float)a.ctas, fminf(units * a.unit * a.inv_min_part, 0.5f * units)));
    if (c > ctas) return false;
    p0.n = a.N;
    p0.h = p0.i = p0.tile = 0;
    if (c == ctas) return true;
    // (a product with one factor for all: rising with c)
    uint32_t x = (uint32_t)(units * ((float)c * __fdividef(1.f, (float)ctas)));
#pragma unroll 1
    for (int n0 = 0; n0 < a.N; n0 += 32 * kFlight) {
        if (a.N > 32 * kFlight) weigh(n0);  // (else the loop above left them in place)
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const uint32_t sum = __reduce_add_sync(0xffffffffu, w[u]) * (uint32_t)a.Hkv;
            if (x >= sum) {
                x -= sum;
                continue;
            }
            const uint32_t mine = w[u] * (uint32_t)a.Hkv;
            uint32_t incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, x < incl)) - 1;
            x -= __shfl_sync(0xffffffffu, incl - mine, src);
            per_head = __shfl_sync(0xffffffffu, w[u], src);
            p0.n = n0 + 32 * u + src;
            n0 = a.N;  // found
            break;
        }
    }
    load_seq<PAGED>(a, p0.n, s0);
    p0 = point_in_seq<PAGED, KT>(a, s0, p0.n, per_head, x);
    return true;
}

// A part of an item: the key tiles [ta, tb) of (n, h, i).
struct Part {
    int n, h, i;
    int ta, tb, nt;   // tiles of this part, tiles of the item
    int q0, tokens;   // first token row, valid tokens of the item
    int first_tok;    // the item's first token within its sequence
    int Lq, Lk, k0;
    __device__ __forceinline__ bool whole() const { return ta == 0 && tb == nt; }
};
template <bool PAGED, int KT>
__device__ __forceinline__ void item_part(const Args &a, const Seq &s, Part &p) {
    p.nt = item_tiles<PAGED, KT>(a, s, p.i);
    p.first_tok = p.i * a.block;
    p.q0 = s.q0 + p.first_tok;
    p.tokens = min(a.block, s.Lq - p.first_tok);
    p.Lq = s.Lq;
    p.Lk = s.Lk;
    p.k0 = s.k0;
}

// `direct`: the item of slot x, whole. A head's slots: those of sequence n start at
// (its first token) / block + n, which leaves each sequence at least as many slots
// as it has items. A converged warp. False: an empty slot or malformed offsets.
template <bool PAGED, int KT>
__device__ __forceinline__ bool direct_part(const Args &a, int x, Part &p) {
    const int lane = threadIdx.x & 31;
    Seq s;
    bool good = true;
    if (PAGED) {
        uint32_t i, h;
        const uint32_t nh = quick_div((uint32_t)x, (uint32_t)(div_block(a, a.T - 1) + 1), i);
        p.n = (int)quick_div(nh, (uint32_t)a.Hkv, h);
        p.i = (int)i;
        p.h = (int)h;
        good = load_seq<PAGED>(a, p.n, s);
    } else {
        uint32_t in_head;
        p.h = (int)quick_div((uint32_t)x, (uint32_t)(div_block(a, a.Tq_total) + a.N), in_head);
        const int slot = (int)in_head;
        p.n = -1;
        for (int n0 = 0; n0 < a.N; n0 += 32) {
            Seq t;
            bool here = false;
            if (n0 + lane < a.N) {
                good = load_seq<PAGED>(a, n0 + lane, t) && good;
                here = div_block(a, t.q0) + n0 + lane <= slot;
            }
            const unsigned who = __ballot_sync(0xffffffffu, here);
            if (who == 0) continue;
            const int src = 31 - __clz(who);
            p.n = n0 + src;
            s.q0 = __shfl_sync(0xffffffffu, t.q0, src);
            s.Lq = __shfl_sync(0xffffffffu, t.Lq, src);
            s.k0 = __shfl_sync(0xffffffffu, t.k0, src);
            s.Lk = __shfl_sync(0xffffffffu, t.Lk, src);
            s.ni = __shfl_sync(0xffffffffu, t.ni, src);
        }
        good = __all_sync(0xffffffffu, good);
        p.i = slot - (div_block(a, s.q0) + p.n);
    }
    if (!good) {
        if (lane == 0) atomicOr(status_word(a), kStatusBadSeqlens);
        return false;
    }
    if (p.n < 0 || p.i >= s.ni) return false;
    item_part<PAGED, KT>(a, s, p);
    p.ta = 0;
    p.tb = p.nt;
    return true;
}

// Walks the parts of [at, end).
template <bool PAGED, int KT>
struct Walk {
    Point at, end;
    Seq s;
    int seq_n;
    __device__ __forceinline__ void init(const Point &p0, const Point &p1, const Seq &s0) {
        at = p0;
        end = p1;
        s = s0;
        seq_n = p0.n;
    }
    __device__ __forceinline__ bool next(const Args &a, Part &p) {
        while (true) {
            if (at.n >= a.N || (same_item(at, end) && at.tile >= end.tile)) return false;
            if (seq_n != at.n) {
                load_seq<PAGED>(a, at.n, s);
                seq_n = at.n;
            }
            if (s.ni == 0) {
                ++at.n;
                at.h = at.i = at.tile = 0;
                continue;
            }
            p.n = at.n;
            p.h = at.h;
            p.i = at.i;
            item_part<PAGED, KT>(a, s, p);
            p.ta = at.tile;
            p.tb = same_item(at, end) ? end.tile : p.nt;
            if (same_item(at, end)) {
                at.tile = end.tile;
            } else {
                at.tile = 0;
                if (++at.i == s.ni) {
                    at.i = 0;
                    if (++at.h == a.Hkv) {
                        at.h = 0;
                        ++at.n;
                    }
                }
            }
            // a part without tiles is one only for rows that see nothing
            if (p.tb > p.ta || p.nt == 0) return true;
        }
    }
};
// The workspace slot of CTA c's unfinished part.
__device__ __forceinline__ int part_slot(int c, const Part &p) { return 2 * c + (p.ta == 0); }


}  // namespace attn
}  // namespace kda
