// C entry points of the paged 4-bit cache: argument validation and launches.
// The contract of every function is documented in include/kda.h.
#include <math.h>
#include <string.h>

#include "kda_internal.h"

namespace {

bool dtype_ok(int dt) { return dt == KDA_DTYPE_BF16 || dt == KDA_DTYPE_FP16; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
// log2 of a page size of 16 .. 256 tokens, or -1
int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}
// a power of two whose reciprocal is one too
bool power_of_two(float x) {
    int e;
    return x > 0.f && isfinite(x) && isfinite(1.f / x) && frexpf(x, &e) == 0.5f;
}
bool row_stride_ok(const void *p, long long stride, long long row) {
    return aligned16(p) && stride >= row && stride % 8 == 0;
}

int fill_cache_args(kda::KvCacheArgs &a, int dt, int B, int total_tokens, int H, int D, const int32_t *cu,
                    const int32_t *start, const int32_t *page_table, int max_pages, int page_size, const void *pool,
                    int num_pages, float k_scale, float v_scale, int32_t *dev_err) {
    if (!dtype_ok(dt) || (D != 64 && D != 128)) return KDA_ERR_UNSUPPORTED;
    const int shift = page_shift_of(page_size);
    if (B < 0 || total_tokens < 0 || H < 1 || max_pages < 1 || num_pages < 1 || shift < 0 ||
        !power_of_two(k_scale) || !power_of_two(v_scale) || (B == 0 && total_tokens > 0))
        return KDA_ERR_INVALID_ARG;
    if ((long long)total_tokens * H > 0x7fffffffLL || (long long)H * D > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0) return KDA_OK;
    if (!cu || !start || !page_table || !pool || !aligned16(pool)) return KDA_ERR_INVALID_ARG;
    memset(&a, 0, sizeof(a));
    a.dt = dt; a.B = B; a.T = total_tokens; a.H = H; a.D = D;
    a.max_pages = max_pages; a.page_shift = shift; a.num_pages = num_pages;
    a.cu = cu; a.start = start; a.page_table = page_table; a.pool = (uint8_t *)pool;
    a.k_scale = k_scale; a.v_scale = v_scale; a.k_inv = 1.f / k_scale; a.v_inv = 1.f / v_scale;
    a.err = dev_err;
    return KDA_OK;
}

int fill_page_args(kda::PageArgs &a, int B, int max_pages, int page_size, int num_pages, int32_t *refs,
                   int32_t *page_table, int32_t *lens, int32_t *dev_err) {
    const int shift = page_shift_of(page_size);
    if (B < 0 || max_pages < 1 || num_pages < 1 || shift < 0) return KDA_ERR_INVALID_ARG;
    if ((long long)max_pages << shift > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (!refs || (B > 0 && (!page_table || !lens))) return KDA_ERR_INVALID_ARG;
    a.B = B; a.max_pages = max_pages; a.page_shift = shift; a.num_pages = num_pages;
    a.refs = refs; a.page_table = page_table; a.lens = lens; a.err = dev_err;
    return KDA_OK;
}

int fill_copy_params(kda::PageCopyParams &p, int num_pools, void *const *pools, size_t page_bytes, int num_pages,
                     int32_t *dev_err) {
    if (num_pools < 1 || num_pools > KDA_MAX_LAYERS || !pools || page_bytes == 0 || page_bytes % 16 != 0 ||
        num_pages < 1)
        return KDA_ERR_INVALID_ARG;
    memset(&p, 0, sizeof(p));
    for (int i = 0; i < num_pools; ++i) {
        if (!pools[i] || !aligned16(pools[i])) return KDA_ERR_INVALID_ARG;
        p.pool[i] = (uint8_t *)pools[i];
    }
    p.P = num_pools; p.page_bytes = page_bytes; p.num_pages = num_pages; p.err = dev_err;
    return KDA_OK;
}

int attention(kda_dtype dt, int B, int total_tokens, int max_q, int H_q, int H_kv, int D, const void *q,
              long long q_stride, const int32_t *cu_seqlens, const int32_t *kv_lens, const int32_t *page_table,
              int max_pages, int page_size, const void *pool, int num_pages, int window, float scale, float k_scale,
              float v_scale, void *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_err,
              uint64_t wait_ns, int starve, void *stream, const int32_t *picked = nullptr, int count = 0) {
    if (!dtype_ok(dt) || (D != 64 && D != 128)) return KDA_ERR_UNSUPPORTED;
    const int shift = page_shift_of(page_size);
    if (B < 0 || total_tokens < 0 || max_q < 0 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || max_pages < 1 ||
        num_pages < 1 || shift < 0 || window < 0 || !isfinite(scale) || !power_of_two(k_scale) ||
        !power_of_two(v_scale) || (B == 0 && total_tokens > 0))
        return KDA_ERR_INVALID_ARG;
    if ((long long)total_tokens * H_q > 0x7fffffffLL || (long long)H_q * D > 0x7fffffffLL ||
        ((long long)max_pages << shift) > 0x40000000LL)
        return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0 || max_q == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    if (!q || !cu_seqlens || !kv_lens || !page_table || !pool || !o || !workspace) return KDA_ERR_INVALID_ARG;
    if (!row_stride_ok(q, q_stride, (long long)H_q * D) || !aligned16(pool) || !aligned16(o) ||
        !aligned16(workspace) || workspace_bytes < kda_kv4_workspace_bytes())
        return KDA_ERR_INVALID_ARG;
    kda::KvAttentionArgs a;
    memset(&a, 0, sizeof(a));
    a.dt = dt; a.B = B; a.T = total_tokens; a.max_q = max_q; a.Hq = H_q; a.Hkv = H_kv; a.D = D;
    a.max_pages = max_pages; a.page_shift = shift; a.num_pages = num_pages;
    // a window that no cache of this table can fill is none: positions minus a window then stay in 32 bits
    a.window = window < (max_pages << shift) ? window : 0;
    a.q = q; a.q_stride = q_stride; a.cu = cu_seqlens; a.kv_lens = kv_lens; a.page_table = page_table;
    a.pool = (const uint8_t *)pool;
    a.scale_k = (float)((double)scale * k_scale * 1.4426950408889634); a.v_scale = v_scale;
    a.o = o; a.lse = lse; a.ws = (uint8_t *)workspace; a.err = dev_err;
    a.wait_ns = wait_ns; a.starve = starve;
    a.picked = picked; a.count = count;
    if (picked) return from_cuda(kda::launch_kv4_attention_picked(a, (cudaStream_t)stream));
    return from_cuda(kda::launch_kv4_attention(a, (cudaStream_t)stream));
}

int pick(kda_dtype dt, int B, int total_tokens, int max_q, int H_q, int H_kv, int D, const void *q, long long q_stride,
         const int32_t *cu_seqlens, const int32_t *kv_lens, const int32_t *page_table, int max_pages, int page_size,
         const int8_t *bounds, int num_pages, int count, int first, int recent, int32_t *picked, void *workspace,
         size_t workspace_bytes, int32_t *dev_err, uint64_t wait_ns, int starve, void *stream) {
    if (!dtype_ok(dt) || (D != 64 && D != 128)) return KDA_ERR_UNSUPPORTED;
    const int shift = page_shift_of(page_size);
    if (B < 0 || total_tokens < 0 || max_q < 0 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || max_pages < 1 ||
        num_pages < 1 || shift < 0 || (B == 0 && total_tokens > 0) || count < 1 || first < 0 || recent < 1 ||
        (long long)first + recent > count)
        return KDA_ERR_INVALID_ARG;
    if ((long long)total_tokens * H_q > 0x7fffffffLL || (long long)H_q * D > 0x7fffffffLL ||
        ((long long)max_pages << shift) > 0x40000000LL)
        return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0 || max_q == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    if (!q || !cu_seqlens || !kv_lens || !page_table || !bounds || !picked || !workspace) return KDA_ERR_INVALID_ARG;
    if (!row_stride_ok(q, q_stride, (long long)H_q * D) || !aligned16(bounds) || !aligned16(workspace) ||
        workspace_bytes < kda_kv4_pick_workspace_bytes(total_tokens, H_kv, max_pages))
        return KDA_ERR_INVALID_ARG;
    // the scores' grid: blocks of 8 tokens a request, groups of 8 or 2 heads
    const int most = max_q < total_tokens ? max_q : total_tokens;
    if (max_pages > count && (B * ((most + 7LL) / 8) > 0x7fffffffLL || H_kv > (most == 1 ? 8 : 2) * 65535)) return KDA_ERR_INVALID_ARG;
    kda::KvPickArgs a;
    memset(&a, 0, sizeof(a));
    a.dt = dt; a.B = B; a.T = total_tokens; a.max_q = max_q < total_tokens ? max_q : total_tokens;
    a.Hq = H_q; a.Hkv = H_kv; a.D = D; a.max_pages = max_pages; a.page_shift = shift; a.num_pages = num_pages; a.count = count; a.first = first;
    a.recent = recent; a.q = q; a.q_stride = q_stride; a.cu = cu_seqlens; a.kv_lens = kv_lens;
    a.page_table = page_table; a.bounds = bounds; a.picked = picked; a.keys = (uint32_t *)workspace;
    a.key_stride = max_pages; a.err = dev_err; a.wait_ns = wait_ns; a.starve = starve;
    return from_cuda(kda::launch_kv4_pick(a, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

KDA_API int kda_kv4_append(kda_dtype dt, int B, int total_tokens, int H_kv, int D, const void *k,
                           long long k_stride, const void *v, long long v_stride,
                           const int32_t *cu_seqlens, const int32_t *start,
                           const int32_t *page_table, int max_pages, int page_size, void *pool,
                           int num_pages, float k_scale, float v_scale, int32_t *dev_err,
                           void *stream) {
    kda::KvCacheArgs a;
    const int st = fill_cache_args(a, dt, B, total_tokens, H_kv, D, cu_seqlens, start, page_table, max_pages,
                                   page_size, pool, num_pages, k_scale, v_scale, dev_err);
    if (st != KDA_OK || total_tokens == 0) return st;
    if (!k || !v || !row_stride_ok(k, k_stride, (long long)H_kv * D) ||
        !row_stride_ok(v, v_stride, (long long)H_kv * D))
        return KDA_ERR_INVALID_ARG;
    a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride;
    return from_cuda(kda::launch_kv4_cache(a, true, (cudaStream_t)stream));
}

KDA_API int kda_kv4_append_rope(kda_dtype dt, int B, int total_tokens, int H_q, int H_kv, int D,
                                int R, int pairs, const void *q, long long q_stride,
                                const void *k, long long k_stride, const void *v,
                                long long v_stride, const float *rope, int positions,
                                const int32_t *cu_seqlens, const int32_t *start,
                                const int32_t *page_table, int max_pages, int page_size,
                                void *pool, int num_pages, float k_scale, float v_scale,
                                void *q_out, long long q_out_stride, int32_t *dev_err,
                                void *stream) {
    kda::KvCacheArgs c;
    const int st = fill_cache_args(c, dt, B, total_tokens, H_kv, D, cu_seqlens, start, page_table, max_pages,
                                   page_size, pool, num_pages, k_scale, v_scale, dev_err);
    if (st != KDA_OK) return st;
    if (R < 32 || R > D || R % 32 != 0 || H_q < 1 || positions < 1) return KDA_ERR_INVALID_ARG;
    const long long heads = (long long)H_q + 2LL * H_kv;
    if (heads * D > 0x7fffffffLL || heads * total_tokens > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0) return KDA_OK;
    if (!q || !k || !v || !rope || !q_out || !aligned16(rope) || !row_stride_ok(q, q_stride, (long long)H_q * D) ||
        !row_stride_ok(k, k_stride, (long long)H_kv * D) || !row_stride_ok(v, v_stride, (long long)H_kv * D) ||
        !row_stride_ok(q_out, q_out_stride, (long long)H_q * D) || (q == q_out && q_stride != q_out_stride))
        return KDA_ERR_INVALID_ARG;
    kda::KvRopeArgs a;
    memset(&a, 0, sizeof(a));
    a.dt = dt; a.B = B; a.T = total_tokens; a.Hq = H_q; a.Hkv = H_kv; a.D = D; a.max_pages = max_pages;
    a.page_shift = c.page_shift; a.num_pages = num_pages; a.R = R; a.positions = positions; a.pairs = pairs != 0;
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.qo_stride = q_out_stride; a.rope = rope; a.cu = cu_seqlens; a.start = start; a.page_table = page_table;
    a.pool = c.pool; a.q_out = q_out; a.k_inv = c.k_inv; a.v_inv = c.v_inv; a.err = dev_err;
    return from_cuda(kda::launch_kv4_rope(a, (cudaStream_t)stream));
}

KDA_API int kda_kv4_bounds(int B, int total_tokens, int H_kv, int D, const int32_t *cu_seqlens,
                           const int32_t *start, const int32_t *page_table, int max_pages,
                           int page_size, const void *pool, int num_pages, int8_t *bounds,
                           int32_t *dev_err, void *stream) {
    kda::KvCacheArgs c;
    const int st = fill_cache_args(c, KDA_DTYPE_BF16, B, total_tokens, H_kv, D, cu_seqlens, start, page_table, max_pages,
                                   page_size, pool, num_pages, 1.f, 1.f, dev_err);
    if (st != KDA_OK || total_tokens == 0) return st;
    if (!bounds || !aligned16(bounds)) return KDA_ERR_INVALID_ARG;
    kda::KvBoundsArgs a;
    memset(&a, 0, sizeof(a));
    a.B = B; a.T = total_tokens; a.H = H_kv; a.D = D; a.max_pages = max_pages; a.page_shift = c.page_shift;
    a.num_pages = num_pages; a.cu = cu_seqlens; a.start = start; a.page_table = page_table; a.pool = c.pool;
    a.bounds = bounds; a.err = dev_err;
    return from_cuda(kda::launch_kv4_bounds(a, (cudaStream_t)stream));
}

KDA_API size_t kda_kv4_pick_workspace_bytes(int total_tokens, int H_kv, int max_pages) {
    if (total_tokens < 0 || H_kv < 1 || max_pages < 1 || (long long)total_tokens * H_kv > 0x7fffffffLL) return 0;
    return 16 + ((size_t)total_tokens * H_kv * max_pages * 4 + 15) / 16 * 16;
}

KDA_API int kda_kv4_pick(kda_dtype dt, int B, int total_tokens, int max_q, int H_q, int H_kv, int D,
                         const void *q, long long q_stride, const int32_t *cu_seqlens,
                         const int32_t *kv_lens, const int32_t *page_table, int max_pages,
                         int page_size, const int8_t *bounds, int num_pages, int count, int first,
                         int recent, int32_t *picked, void *workspace, size_t workspace_bytes,
                         int32_t *dev_err, void *stream) {
    return pick(dt, B, total_tokens, max_q, H_q, H_kv, D, q, q_stride, cu_seqlens, kv_lens, page_table, max_pages, page_size,
                bounds, num_pages, count, first, recent, picked, workspace, workspace_bytes, dev_err, KDA_KV4_WAIT_NS, 0, stream);
}

KDA_API int kda_selftest_kv4_pick_wait(kda_dtype dt, int B, int total_tokens, int max_q, int H_q,
                                       int H_kv, int D, const void *q, long long q_stride, const int32_t *cu_seqlens,
                                       const int32_t *kv_lens, const int32_t *page_table, int max_pages,
                                       int page_size, const int8_t *bounds, int num_pages, int count, int first,
                                       int recent, int32_t *picked, void *workspace, size_t workspace_bytes,
                                       int32_t *dev_err, int wait_us, void *stream) {
    if (!dev_err || wait_us < 1 || wait_us > 2000000 || total_tokens < 1 || max_q != 1 || count >= max_pages) return KDA_ERR_INVALID_ARG;
    return pick(dt, B, total_tokens, max_q, H_q, H_kv, D, q, q_stride, cu_seqlens, kv_lens, page_table, max_pages, page_size,
                bounds, num_pages, count, first, recent, picked, workspace, workspace_bytes, dev_err, (uint64_t)wait_us * 1000ull, 1, stream);
}

KDA_API int kda_kv4_attention_picked(kda_dtype dt, int B, int total_tokens, int max_q, int H_q,
                                     int H_kv, int D, const void *q, long long q_stride,
                                     const int32_t *cu_seqlens, const int32_t *kv_lens,
                                     const int32_t *page_table, int max_pages, int page_size,
                                     const int32_t *picked, int count, const void *pool,
                                     int num_pages, float scale, float k_scale, float v_scale,
                                     void *o, float *lse, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_err, void *stream) {
    if (count < 1 || (!picked && total_tokens > 0)) return KDA_ERR_INVALID_ARG;
    return attention(dt, B, total_tokens, max_q, H_q, H_kv, D, q, q_stride, cu_seqlens, kv_lens, page_table, max_pages,
                     page_size, pool, num_pages, 0, scale, k_scale, v_scale, o, lse, workspace, workspace_bytes,
                     dev_err, KDA_KV4_WAIT_NS, 0, stream, picked, count);
}

KDA_API int kda_kv4_gather(kda_dtype dt, int B, int total_tokens, int H_kv, int D, void *k,
                           void *v, const int32_t *cu_seqlens, const int32_t *start,
                           const int32_t *page_table, int max_pages, int page_size,
                           const void *pool, int num_pages, float k_scale, float v_scale,
                           int32_t *dev_err, void *stream) {
    kda::KvCacheArgs a;
    const int st = fill_cache_args(a, dt, B, total_tokens, H_kv, D, cu_seqlens, start, page_table, max_pages,
                                   page_size, pool, num_pages, k_scale, v_scale, dev_err);
    if (st != KDA_OK || total_tokens == 0) return st;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return KDA_ERR_INVALID_ARG;
    a.k_out = k; a.v_out = v;
    return from_cuda(kda::launch_kv4_cache(a, false, (cudaStream_t)stream));
}

KDA_API size_t kda_kv4_workspace_bytes(void) { return KDA_KV4_WORKSPACE; }

KDA_API int kda_kv4_attention(kda_dtype dt, int B, int total_tokens, int max_q, int H_q, int H_kv,
                              int D, const void *q, long long q_stride, const int32_t *cu_seqlens,
                              const int32_t *kv_lens, const int32_t *page_table, int max_pages,
                              int page_size, const void *pool, int num_pages, int window,
                              float scale, float k_scale, float v_scale, void *o, float *lse,
                              void *workspace, size_t workspace_bytes, int32_t *dev_err,
                              void *stream) {
    return attention(dt, B, total_tokens, max_q, H_q, H_kv, D, q, q_stride, cu_seqlens, kv_lens, page_table, max_pages,
                     page_size, pool, num_pages, window, scale, k_scale, v_scale, o, lse, workspace, workspace_bytes,
                     dev_err, KDA_KV4_WAIT_NS, 0, stream);
}

KDA_API int kda_selftest_kv4_wait(kda_dtype dt, int B, int total_tokens, int max_q, int H_q,
                                  int H_kv, int D, const void *q, long long q_stride,
                                  const int32_t *cu_seqlens, const int32_t *kv_lens,
                                  const int32_t *page_table, int max_pages, int page_size,
                                  const void *pool, int num_pages, void *o, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_err, int wait_us,
                                  void *stream) {
    if (!dev_err || wait_us < 1 || wait_us > 2000000 || total_tokens < 1) return KDA_ERR_INVALID_ARG;
    return attention(dt, B, total_tokens, max_q, H_q, H_kv, D, q, q_stride, cu_seqlens, kv_lens, page_table, max_pages,
                     page_size, pool, num_pages, 0, 1.f, 1.f, 1.f, o, nullptr, workspace, workspace_bytes, dev_err,
                     (uint64_t)wait_us * 1000ull, 1, stream);
}

KDA_API int kda_page_alloc(int B, int max_pages, int page_size, int num_pages, int32_t *refs,
                           int32_t *page_table, int32_t *lens, const int32_t *grow,
                           int32_t *dev_err, void *stream) {
    kda::PageArgs a;
    const int st = fill_page_args(a, B, max_pages, page_size, num_pages, refs, page_table, lens, dev_err);
    if (st != KDA_OK || B == 0) return st;
    if (!grow) return KDA_ERR_INVALID_ARG;
    return from_cuda(kda::launch_page_alloc(a, grow, (cudaStream_t)stream));
}

KDA_API int kda_page_fork(int num_pools, void *const *pools, size_t page_bytes, int B,
                          int max_pages, int page_size, int num_pages, int32_t *refs,
                          int32_t *page_table, int32_t *lens, const int32_t *src,
                          const int32_t *dst, int n, int32_t *workspace, size_t workspace_ints,
                          int32_t *dev_err, void *stream) {
    kda::PageArgs a;
    kda::PageCopyParams p;
    int st = fill_page_args(a, B, max_pages, page_size, num_pages, refs, page_table, lens, dev_err);
    if (st == KDA_OK) st = fill_copy_params(p, num_pools, pools, page_bytes, num_pages, dev_err);
    if (st != KDA_OK) return st;
    if (n < 0) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    if (!src || !dst || !workspace || workspace_ints < 2 * (size_t)n) return KDA_ERR_INVALID_ARG;
    return from_cuda(kda::launch_page_fork(a, src, dst, n, p, workspace, (cudaStream_t)stream));
}

KDA_API int kda_page_free(int B, int max_pages, int page_size, int num_pages, int32_t *refs,
                          int32_t *page_table, int32_t *lens, const int32_t *rows, int n,
                          int32_t *dev_err, void *stream) {
    kda::PageArgs a;
    const int st = fill_page_args(a, B, max_pages, page_size, num_pages, refs, page_table, lens, dev_err);
    if (st != KDA_OK) return st;
    if (n < 0) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    if (!rows) return KDA_ERR_INVALID_ARG;
    return from_cuda(kda::launch_page_free(a, rows, n, (cudaStream_t)stream));
}

KDA_API int kda_page_compact(int num_pools, void *const *pools, size_t page_bytes, int B,
                             int max_pages, int num_pages, int32_t *refs, int32_t *page_table,
                             int32_t *live, int32_t *workspace, size_t workspace_ints,
                             int32_t *dev_err, void *stream) {
    kda::PageCopyParams p;
    const int st = fill_copy_params(p, num_pools, pools, page_bytes, num_pages, dev_err);
    if (st != KDA_OK) return st;
    if (B < 0 || max_pages < 1 || !refs || (B > 0 && !page_table) || !live || !workspace ||
        workspace_ints < 3 * (size_t)num_pages + 16)
        return KDA_ERR_INVALID_ARG;
    kda::PageArgs a;
    memset(&a, 0, sizeof(a));
    a.B = B; a.max_pages = max_pages; a.num_pages = num_pages; a.refs = refs; a.page_table = page_table;
    a.err = dev_err;
    return from_cuda(kda::launch_page_compact(a, p, workspace, live, (cudaStream_t)stream));
}

KDA_API int kda_page_copy(int num_pools, void *const *pools, size_t page_bytes, int num_pages,
                          const int32_t *src, const int32_t *dst, int n, int32_t *dev_err,
                          void *stream) {
    kda::PageCopyParams p;
    const int st = fill_copy_params(p, num_pools, pools, page_bytes, num_pages, dev_err);
    if (st != KDA_OK) return st;
    if (n < 0) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    if (!src || !dst) return KDA_ERR_INVALID_ARG;
    p.n = n; p.src = src; p.dst = dst; p.step = 1;
    return from_cuda(kda::launch_page_copy(p, (cudaStream_t)stream));
}

}  // extern "C"
