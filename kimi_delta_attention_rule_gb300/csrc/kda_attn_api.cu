// C ABI of the attention and page-cache entry points (declared in
// include/kda.h): argument validation and dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include <nvtx3/nvToolsExt.h>

#include "kda.h"
#include "kda_attn.cuh"
#include "kda_testing.h"

namespace kda {
namespace attn {
cudaError_t launch_attn_prefill_tc(Args a, const void *q, const void *k, const void *v, long long ldq,
                                   long long ldk, long long ldv, cudaStream_t stream);
cudaError_t launch_attn_decode_tc(Args a, const void *q, const void *kp, const void *vp, const void *kn,
                                  const void *vn, long long ldq, long long ldk, long long ldv,
                                  cudaStream_t stream);
cudaError_t launch_attn_prefill_f32(const Args &a, const void *q, const void *k, const void *v, long long ldq,
                                    long long ldk, long long ldv, cudaStream_t stream);
cudaError_t launch_attn_decode_f32(const Args &a, const void *q, const void *kp, const void *vp, const void *kn,
                                   const void *vn, long long ldq, long long ldk, long long ldv,
                                   cudaStream_t stream);
}  // namespace attn
namespace cache {
cudaError_t launch_append(const void *k, const void *v, int64_t ldk, int64_t ldv, const int32_t *cu, int N, int T,
                          int64_t rows, const int32_t *index, const int32_t *count, const int32_t *start,
                          const int32_t *table, int64_t table_ld, int cols, int pages, int page, int Hkv, int es,
                          void *kp, void *vp, uint32_t *status, cudaStream_t stream);
cudaError_t launch_copy(void *const *pools, int n_pools, int64_t entry_bytes, int entries, const int32_t *pairs, int n,
                        const int32_t *count, int sms, cudaStream_t stream);
cudaError_t launch_free(int32_t *table, int64_t ld, int rows, int cols, int32_t *lens, int32_t *refs, int pages,
                        const int32_t *which, int n, uint32_t *status, cudaStream_t stream);
cudaError_t launch_fork(int32_t *table, int64_t ld, int rows, int cols, int32_t *lens, int32_t *refs, int pages,
                        int page, const int32_t *src, const int32_t *dst, int n, int32_t *copies, int32_t *scratch,
                        uint32_t *status, cudaStream_t stream);
cudaError_t launch_alloc(int32_t *table, int64_t ld, int rows, int cols, const int32_t *want, int32_t *refs,
                         int pages, int page, int32_t *scratch, uint32_t *status, cudaStream_t stream);
cudaError_t launch_compact(int32_t *table, int64_t ld, int rows, int cols, int32_t *refs, int pages,
                           int32_t *copies, int32_t *count, int32_t *scratch, uint32_t *status,
                           cudaStream_t stream);
}  // namespace cache
}  // namespace kda

namespace {

using kda::attn::Args;

constexpr int kMaxGroup = 64;
constexpr int kMaxTokens = kda::attn::kMaxDrafts;
constexpr long long kMaxKeys = (1LL << 31) - 1024;  // (positions two key tiles past a sequence's end are formed)
constexpr size_t kHeader = 256;  // of a cache workspace: the status word
// Pages, and entries of a block table: their kernels step past the last one by less than 2^16
// and add up the pages that all rows lack, in 32 bits.
constexpr long long kMaxPages = (1LL << 31) - (1LL << 16);

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    const bool any = cudaGetDevice(&dev) == cudaSuccess;
    if (any && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (!any || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();  // no device: sizes for a full GB300
        return 152;
    }
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}
// CTAs of one attention call: all that fit on the device at once, fewer when
// an upper bound of the work (in keys) cannot fill them.
int attn_ctas(int32_t io, long long keys) {
    const int most = std::min((io == KDA_F32 ? 2 : 1) * sm_count(), kda::attn::kMaxCtas);
    const long long n = keys / (io == KDA_F32 ? kda::attn::kF32MinPart : kda::attn::kTcMinPart);
    return (int)(n < 1 ? 1 : (n < most ? n : most));
}
// Rows of an item at the most: a row tile (fp32), or two of 128 rows, which a decode
// of at most 128 rows per kv head does not need.
int part_rows(int32_t io, int rows) { return io == KDA_F32 ? 64 : (rows <= 128 ? 128 : 256); }
int check_heads(int32_t Hq, int32_t Hkv, int32_t D, int32_t io) {
    if (Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return KDA_ERR_INVALID_ARG;
    if (io != KDA_BF16 && io != KDA_F32) return KDA_ERR_UNSUPPORTED;
    if (D != kda::kD || Hq / Hkv > kMaxGroup) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
bool page_ok(int32_t page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }
// Upper bounds of the work, in keys (each item: its keys and at most 512 more)
long long prefill_keys(int32_t N, long long Tq, long long Tk, int32_t Hq, int32_t Hkv, int32_t io) {
    const long long g = Hq / Hkv, block = io == KDA_F32 ? 64 / g : 2 * (128 / g);
    long long items = (Tq / block + N) * Hkv;
    const long long cap = 1LL << 20;  // enough for any device
    return items > cap ? cap * 1024 : items * (Tk < cap ? Tk + 512 : cap);
}
long long decode_keys(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t page, int32_t cols, int32_t io) {
    if (T == 0) return 0;
    const long long g = Hq / Hkv, block = io == KDA_F32 ? 64 / g : (T * g <= 128 ? T : 2 * (128 / g));
    const long long items = (long long)B * Hkv * ((T + block - 1) / block), cap = 1LL << 20;
    const long long keys = (long long)page * cols + 512;
    return items > cap ? cap * 1024 : items * (keys < cap ? keys : cap);
}
// Items of a call at the most (the fp32 kernel's, which are the smaller ones).
long long prefill_items(int32_t N, long long Tq, int32_t Hq, int32_t Hkv) {
    return (Tq / (64 / (Hq / Hkv)) + N) * Hkv;
}
bool ld_ok(int64_t ld, int32_t heads, int32_t io) {
    return ld >= (int64_t)heads * kda::kD && ld % (io == KDA_BF16 ? 8 : 4) == 0 && ld < (1LL << 36);
}
bool scale_ok(float s) { return isfinite(s) && s > 0.f; }
// A warp of the bf16 kernel that gives up at one of its waits (tests).
struct Lose {
    int32_t warp = -1, at = 0;
    bool ok(int32_t io) const { return io == KDA_BF16 && warp >= 0 && warp < 12 && at >= 0; }
};

int prefill_impl(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                 const int32_t *cu_q, const int32_t *cu_k, int32_t N, int32_t Tq, int32_t Tk, int32_t Hq,
                 int32_t Hkv, int32_t D, int32_t io, void *out, float *lse, void *workspace, size_t workspace_bytes,
                 const Lose &lose, void *stream) {
    const int rc = check_heads(Hq, Hkv, D, io);
    if (rc != KDA_OK) return rc;
    if (N < 0 || Tq < 0 || Tk < 0 || !scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if (cu_q == nullptr && cu_k != nullptr) return KDA_ERR_INVALID_ARG;
    const bool packed = cu_q != nullptr;
    if (packed && cu_k == nullptr) {
        if (Tk != Tq) return KDA_ERR_INVALID_ARG;
        cu_k = cu_q;
    }
    const long long tq = packed ? Tq : (long long)N * Tq, tk = packed ? Tk : (long long)N * Tk;
    if (tq > 0x7fffffffLL || tk > 0x7fffffffLL || tq * Hq > (1LL << 40) || tk * Hkv > (1LL << 40) ||
        prefill_items(N, tq, Hq, Hkv) > kda::attn::kMaxItems)
        return KDA_ERR_INVALID_ARG;
    if (N == 0 || tq == 0) return KDA_OK;
    if (q == nullptr || out == nullptr || (tk > 0 && (k == nullptr || v == nullptr)) || workspace == nullptr)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    if (!ld_ok(ldq, Hq, io) || !ld_ok(ldk, Hkv, io) || !ld_ok(ldv, Hkv, io)) return KDA_ERR_INVALID_ARG;
    Args a = {};
    a.ctas = attn_ctas(io, prefill_keys(N, tq, tk, Hq, Hkv, io));
    a.part_rows = part_rows(io, 256);
    if (workspace_bytes < kda::attn::workspace_bytes(a.ctas, a.part_rows)) return KDA_ERR_INVALID_ARG;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.T = Tq;
    a.Tk = Tk;
    a.sms = sm_count();
    a.Tq_total = (int)tq;
    a.Tk_total = (int)tk;
    a.scale = scale;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.out = out;
    a.lse = lse;
    a.ws = static_cast<unsigned char *>(workspace);
    a.lose = lose.warp + 1;
    a.lose_at = lose.at;
    if (tk == 0) k = v = q;  // never read, but a tensor map needs an address
    Range range("kda_attn_prefill");
    return done((io == KDA_BF16 ? kda::attn::launch_attn_prefill_tc(a, q, k, v, ldq, ldk, ldv, static_cast<cudaStream_t>(stream))
                                : kda::attn::launch_attn_prefill_f32(a, q, k, v, ldq, ldk, ldv, static_cast<cudaStream_t>(stream))));
}

int decode_impl(const void *q, int64_t ldq, const void *k_new, const void *v_new, int64_t ldk, int64_t ldv,
                const void *k_pages, const void *v_pages, int32_t num_pages, int32_t page_size,
                const int32_t *block_table, int64_t table_ld, int32_t table_cols, const int32_t *seq_lens,
                const uint64_t *tree_mask, float scale, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
                int32_t io, void *out, float *lse, void *workspace, size_t workspace_bytes, const Lose &lose,
                void *stream) {
    const int rc = check_heads(Hq, Hkv, D, io);
    if (rc != KDA_OK) return rc;
    if (B < 0 || T < 0 || num_pages < 0 || table_cols < 0 || table_ld < table_cols || !scale_ok(scale))
        return KDA_ERR_INVALID_ARG;
    if (T > kMaxTokens || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if ((k_new == nullptr) != (v_new == nullptr) || (tree_mask != nullptr && k_new == nullptr))
        return KDA_ERR_INVALID_ARG;
    if ((long long)num_pages * Hkv * page_size > 0x7fffffffLL || (long long)B * T > 0x7fffffffLL ||
        (long long)B * T * Hq > (1LL << 40) || (long long)table_cols * page_size > kMaxKeys ||
        (long long)B * T * Hkv > kda::attn::kMaxItems)
        return KDA_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return KDA_OK;
    if (q == nullptr || out == nullptr || seq_lens == nullptr || workspace == nullptr ||
        (table_cols > 0 && block_table == nullptr) || (num_pages > 0 && (k_pages == nullptr || v_pages == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pages, 16) ||
        !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(tree_mask, 8) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    if (!ld_ok(ldq, Hq, io) || (k_new != nullptr && (!ld_ok(ldk, Hkv, io) || !ld_ok(ldv, Hkv, io))))
        return KDA_ERR_INVALID_ARG;
    Args a = {};
    a.ctas = attn_ctas(io, decode_keys(B, T, Hq, Hkv, page_size, table_cols, io));
    a.part_rows = part_rows(io, T * (Hq / Hkv));
    if (workspace_bytes < kda::attn::workspace_bytes(a.ctas, a.part_rows)) return KDA_ERR_INVALID_ARG;
    a.N = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.T = T;
    a.page = page_size;
    a.sms = sm_count();
    a.pages = num_pages;
    a.table_cols = table_cols;
    a.table_ld = table_ld;
    a.has_new = k_new != nullptr;
    a.scale = scale;
    a.table = block_table;
    a.lens = seq_lens;
    a.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
    a.out = out;
    a.lse = lse;
    a.ws = static_cast<unsigned char *>(workspace);
    a.lose = lose.warp + 1;
    a.lose_at = lose.at;
    if (num_pages == 0) k_pages = v_pages = q;  // a tensor map needs an address; its only row is never read
    Range range("kda_attn_decode");
    return done((io == KDA_BF16 ? kda::attn::launch_attn_decode_tc(a, q, k_pages, v_pages, k_new, v_new, ldq, ldk, ldv, static_cast<cudaStream_t>(stream))
                                : kda::attn::launch_attn_decode_f32(a, q, k_pages, v_pages, k_new, v_new, ldq, ldk, ldv, static_cast<cudaStream_t>(stream))));
}

}  // namespace

extern "C" {

size_t kda_attn_prefill_workspace_size(int32_t N, int32_t Tq_total, int32_t Tk_total, int32_t Hq, int32_t Hkv,
                                       int32_t D, int32_t io) {
    if (N < 0 || Tq_total < 0 || Tk_total < 0 || check_heads(Hq, Hkv, D, io) != KDA_OK) return 0;
    return kda::attn::workspace_bytes(attn_ctas(io, prefill_keys(N, Tq_total, Tk_total, Hq, Hkv, io)),
                                     part_rows(io, 256));
}

int kda_attn_prefill(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                     const int32_t *cu_q, const int32_t *cu_k, int32_t N, int32_t Tq, int32_t Tk, int32_t Hq,
                     int32_t Hkv, int32_t D, int32_t io, void *out, float *lse, void *workspace,
                     size_t workspace_bytes, void *stream) {
    return prefill_impl(q, k, v, ldq, ldk, ldv, scale, cu_q, cu_k, N, Tq, Tk, Hq, Hkv, D, io, out, lse, workspace,
                        workspace_bytes, Lose(), stream);
}

int kda_testing_attn_prefill_timeout(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk, int64_t ldv,
                                     float scale, const int32_t *cu_q, const int32_t *cu_k, int32_t N, int32_t Tq,
                                     int32_t Tk, int32_t Hq, int32_t Hkv, int32_t D, int32_t io, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, int32_t warp, int32_t at, void *stream) {
    const Lose lose = {warp, at};
    if (!lose.ok(io)) return KDA_ERR_INVALID_ARG;
    return prefill_impl(q, k, v, ldq, ldk, ldv, scale, cu_q, cu_k, N, Tq, Tk, Hq, Hkv, D, io, out, lse, workspace,
                        workspace_bytes, lose, stream);
}

size_t kda_attn_decode_workspace_size(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                      int32_t table_cols, int32_t io) {
    if (B < 0 || T < 0 || T > kMaxTokens || table_cols < 0 || !page_ok(page_size) || check_heads(Hq, Hkv, D, io) != KDA_OK)
        return 0;
    return kda::attn::workspace_bytes(attn_ctas(io, decode_keys(B, T, Hq, Hkv, page_size, table_cols, io)),
                                     part_rows(io, T * (Hq / Hkv)));
}

int kda_attn_decode(const void *q, int64_t ldq, const void *k_new, const void *v_new, int64_t ldk, int64_t ldv,
                    const void *k_pages, const void *v_pages, int32_t num_pages, int32_t page_size,
                    const int32_t *block_table, int64_t table_ld, int32_t table_cols, const int32_t *seq_lens,
                    const uint64_t *tree_mask, float scale, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
                    int32_t io, void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    return decode_impl(q, ldq, k_new, v_new, ldk, ldv, k_pages, v_pages, num_pages, page_size, block_table, table_ld,
                       table_cols, seq_lens, tree_mask, scale, B, T, Hq, Hkv, D, io, out, lse, workspace,
                       workspace_bytes, Lose(), stream);
}

int kda_testing_attn_decode_timeout(const void *q, int64_t ldq, const void *k_new, const void *v_new, int64_t ldk,
                                    int64_t ldv, const void *k_pages, const void *v_pages, int32_t num_pages,
                                    int32_t page_size, const int32_t *block_table, int64_t table_ld, int32_t table_cols,
                                    const int32_t *seq_lens, const uint64_t *tree_mask, float scale, int32_t B, int32_t T,
                                    int32_t Hq, int32_t Hkv, int32_t D, int32_t io, void *out, float *lse,
                                    void *workspace, size_t workspace_bytes, int32_t warp, int32_t at, void *stream) {
    const Lose lose = {warp, at};
    if (!lose.ok(io)) return KDA_ERR_INVALID_ARG;
    return decode_impl(q, ldq, k_new, v_new, ldk, ldv, k_pages, v_pages, num_pages, page_size, block_table, table_ld,
                       table_cols, seq_lens, tree_mask, scale, B, T, Hq, Hkv, D, io, out, lse, workspace,
                       workspace_bytes, lose, stream);
}

// Scratch of the calls that choose pages: the free pages' list and a state per
// fork (at most num_pages and rows of them), or names, or two words per row.
size_t kda_cache_workspace_size(int32_t num_pages, int32_t rows) {
    if (num_pages < 0 || rows < 0) return 0;
    return (kHeader + ((size_t)num_pages + 2 * (size_t)rows + 4) * 4 + 255) / 256 * 256;
}

// The checks that the table calls share.
static int check_cache(const int32_t *table, int64_t ld, int32_t rows, int32_t cols, const int32_t *refs,
                       int32_t num_pages, const void *ws, size_t ws_bytes) {
    if (rows < 0 || cols < 0 || ld < cols || num_pages < 0) return KDA_ERR_INVALID_ARG;
    if (num_pages > kMaxPages || (long long)rows * cols > kMaxPages) return KDA_ERR_INVALID_ARG;
    if ((rows > 0 && cols > 0 && table == nullptr) || (num_pages > 0 && refs == nullptr) || ws == nullptr)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(table, 4) || !aligned(refs, 16) || !aligned(ws, 256) ||
        ws_bytes < kda_cache_workspace_size(num_pages, rows))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}
static uint32_t *status_of(void *ws) { return static_cast<uint32_t *>(ws); }
static int32_t *scratch_of(void *ws) {
    return reinterpret_cast<int32_t *>(static_cast<unsigned char *>(ws) + kHeader);
}

int kda_cache_alloc(int32_t *table, int64_t ld, int32_t rows, int32_t cols, const int32_t *want, int32_t *refs,
                    int32_t num_pages, int32_t page_size, void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_cache(table, ld, rows, cols, refs, num_pages, ws, ws_bytes);
    if (rc != KDA_OK) return rc;
    if (page_size <= 0) return KDA_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return KDA_OK;
    if (want == nullptr || !aligned(want, 4)) return KDA_ERR_INVALID_ARG;
    Range range("kda_cache_alloc");
    return done(kda::cache::launch_alloc(table, ld, rows, cols, want, refs, num_pages, page_size, scratch_of(ws),
                                         status_of(ws), static_cast<cudaStream_t>(stream)));
}

int kda_cache_fork(int32_t *table, int64_t ld, int32_t rows, int32_t cols, int32_t *seq_lens, int32_t *refs,
                   int32_t num_pages, int32_t page_size, const int32_t *src, const int32_t *dst, int32_t n,
                   int32_t *copies, void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_cache(table, ld, rows, cols, refs, num_pages, ws, ws_bytes);
    if (rc != KDA_OK) return rc;
    if (page_size <= 0 || n < 0 || n > rows) return KDA_ERR_INVALID_ARG;  // every dst is a row of its own
    if (n == 0) return KDA_OK;
    if (cols == 0 || seq_lens == nullptr || src == nullptr || dst == nullptr || copies == nullptr)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(seq_lens, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(copies, 8))
        return KDA_ERR_INVALID_ARG;
    Range range("kda_cache_fork");
    return done(kda::cache::launch_fork(table, ld, rows, cols, seq_lens, refs, num_pages, page_size, src, dst, n,
                                        copies, scratch_of(ws), status_of(ws), static_cast<cudaStream_t>(stream)));
}

int kda_cache_free(int32_t *table, int64_t ld, int32_t rows, int32_t cols, int32_t *seq_lens, int32_t *refs,
                   int32_t num_pages, const int32_t *which, int32_t n, void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_cache(table, ld, rows, cols, refs, num_pages, ws, ws_bytes);
    if (rc != KDA_OK) return rc;
    if (n < 0) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    if (cols == 0 || seq_lens == nullptr || which == nullptr || !aligned(seq_lens, 4) || !aligned(which, 4))
        return KDA_ERR_INVALID_ARG;
    Range range("kda_cache_free");
    return done(kda::cache::launch_free(table, ld, rows, cols, seq_lens, refs, num_pages, which, n, status_of(ws),
                                        static_cast<cudaStream_t>(stream)));
}

int kda_cache_compact(int32_t *table, int64_t ld, int32_t rows, int32_t cols, int32_t *refs, int32_t num_pages,
                      int32_t *copies, int32_t *count, void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_cache(table, ld, rows, cols, refs, num_pages, ws, ws_bytes);
    if (rc != KDA_OK) return rc;
    if (count == nullptr || (num_pages > 0 && copies == nullptr) || !aligned(copies, 8) || !aligned(count, 4))
        return KDA_ERR_INVALID_ARG;
    Range range("kda_cache_compact");
    return done(kda::cache::launch_compact(table, ld, rows, cols, refs, num_pages, copies, count, scratch_of(ws),
                                           status_of(ws), static_cast<cudaStream_t>(stream)));
}

int kda_cache_copy(void *const *pools, int32_t n_pools, int64_t entry_bytes, int32_t num_entries,
                   const int32_t *pairs, int32_t n, const int32_t *count, void *stream) {
    if (n_pools < 0 || n < 0 || num_entries < 0 || entry_bytes < 0 || entry_bytes % 16 != 0) return KDA_ERR_INVALID_ARG;
    if (entry_bytes / 16 > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (n_pools == 0 || n == 0 || num_entries == 0 || entry_bytes == 0) return KDA_OK;
    if (pools == nullptr || pairs == nullptr || !aligned(pairs, 8) || !aligned(count, 4)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < n_pools; ++i)
        if (pools[i] == nullptr || !aligned(pools[i], 16)) return KDA_ERR_INVALID_ARG;
    Range range("kda_cache_copy");
    return done(kda::cache::launch_copy(pools, n_pools, entry_bytes, num_entries, pairs, n, count, sm_count(),
                                        static_cast<cudaStream_t>(stream)));
}

int kda_cache_append(const void *k, const void *v, int64_t ldk, int64_t ldv, const int32_t *cu, int32_t N, int32_t T,
                     const int32_t *index, const int32_t *count, const int32_t *start, const int32_t *table,
                     int64_t table_ld, int32_t cols, int32_t num_pages, int32_t page_size, int32_t Hkv, int32_t D,
                     int32_t io, void *k_pages, void *v_pages, void *workspace, void *stream) {
    const int rc = check_heads(Hkv, Hkv, D, io);
    if (rc != KDA_OK) return rc;
    if (N < 0 || T < 0 || num_pages < 0 || cols < 0 || table_ld < cols) return KDA_ERR_INVALID_ARG;
    if (!page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (cu != nullptr && (index != nullptr || count != nullptr)) return KDA_ERR_INVALID_ARG;
    const long long rows = cu != nullptr ? T : (long long)N * T;
    if (rows > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (N == 0 || rows == 0) return KDA_OK;
    if (k == nullptr || v == nullptr || start == nullptr || table == nullptr || k_pages == nullptr ||
        v_pages == nullptr || cols == 0)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(cu, 4) ||
        !aligned(index, 4) || !aligned(count, 4) || !aligned(start, 4) || !aligned(table, 4) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    if (!ld_ok(ldk, Hkv, io) || !ld_ok(ldv, Hkv, io)) return KDA_ERR_INVALID_ARG;
    Range range("kda_cache_append");
    return done(kda::cache::launch_append(k, v, ldk, ldv, cu, N, T, rows, index, count, start, table, table_ld, cols,
                                          num_pages, page_size, Hkv, io == KDA_BF16 ? 2 : 4, k_pages, v_pages,
                                          status_of(workspace), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
