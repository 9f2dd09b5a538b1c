// Internal launch interface between the C entry points (kda_api.cu) and the
// kernel translation units.  Host-side only; no device code here.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

// Bytes of the cache attention's workspace: a counter and two partial results a CTA.
#define KDA_KV4_WORKSPACE (16u << 20)
// Limit of the cache attention's waits.
#define KDA_KV4_WAIT_NS 2000000000ull

namespace kda {

struct DecodeArgs {
    int dt, B, H, num_slots;
    const void *q, *k, *v, *gk, *beta;
    const int32_t *slot_ids;
    float *pool;
    void *o;
    float scale;
    int32_t *err;
};

struct VerifyArgs {
    int dt, B, G, H, num_slots, ring_len;
    const void *q, *k, *v, *gk, *beta;
    const int32_t *slot_ids, *ring_base;
    // ragged drafts: request b's tokens are cu_drafts[b] .. cu_drafts[b+1]-1 of
    // [total_tokens][H][..] and number at most G; NULL: uniform [B][G][H][..]
    const int32_t *cu_drafts;
    int total_tokens;
    const float *pool;
    void *rk, *rv;
    float *rdecay, *rbeta;
    void *o;
    float scale;
    int32_t *err;
};

// One layer of a fold: its state pool and ring buffers.
struct FoldLayer {
    float *pool;
    void *rk, *rv;
    float *rdecay, *rbeta;
};

struct FoldParams {
    int L, B, H, num_slots, max_accept, ring_len;
    const int32_t *slot_ids, *accept, *ring_base;
    int32_t *err;
    FoldLayer layer[KDA_MAX_LAYERS];
};

struct CopyParams {
    int P, n, num_slots, chunks_per_copy;
    size_t slot_elems;
    const int32_t *src, *dst;
    int32_t *err;
    float *pool[KDA_MAX_LAYERS];
};

struct PrefillArgs {
    int dt, N, T_total, H, num_slots;
    const void *q, *k, *v, *gk, *beta;
    const int32_t *cu;            // device
    const int32_t *cu_host;       // host (validated)
    float *pool;
    const int32_t *init_slot, *out_slot, *snap_slot;
    void *o;
    float scale;
    int32_t *err;
    int ckpt_interval;             // 0: no checkpoints
    int max_ckpts;
    const int32_t *ckpt_slots;     // device [N][max_ckpts]
    uint64_t wait_ns = 0;          // limit of the kernel's waits (0: its default)
    int skip_first_load = 0;       // self-test only: the first chunk's q, k, gk are never requested
};

// Snapshot-per-step verify: the state after every draft step into a
// snapshot buffer [num_snap_slots][G][H][K][V].
struct SnapVerifyArgs {
    int dt, B, G, H, num_slots, num_snap_slots;
    const void *q, *k, *v, *gk, *beta;
    const int32_t *slot_ids, *snap_ids;
    const float *pool;
    float *snaps;
    void *o;
    float scale;
    int32_t *err;
};

// Commit of the snapshot baseline: snapshot accept-1 -> the request's slot,
// every layer, one launch.
struct SnapCommitParams {
    int L, B, H, G, num_slots, num_snap_slots, chunks_per_copy;
    const int32_t *slot_ids, *snap_ids, *accept;
    int32_t *err;
    float *pool[KDA_MAX_LAYERS];
    const float *snaps[KDA_MAX_LAYERS];
};

// Conv prologue over a packed varlen batch: grid (N x max_tiles, H).
struct PrologueArgs {
    int dt, N, T_total, H, num_slots, max_tiles;
    const void *q_raw, *k_raw, *v_raw, *b_raw;
    long long raw_stride;
    const void *conv_w;
    void *conv_state;
    const int32_t *init_slot, *out_slot, *cu;
    void *q, *k, *v, *beta;
    float eps;
    int32_t *err;
};

struct NormArgs {
    int dt, tokens, H;
    const void *o;
    long long o_token_stride, o_head_stride;
    const void *gate, *w_norm;
    float eps;
    void *out;
};

struct FusedDecodeArgs {
    int dt, B, H, num_slots;
    const void *q_raw, *k_raw, *v_raw;
    long long raw_stride;
    const void *gk, *b_raw, *conv_w;
    void *conv_state;
    const void *gate, *w_norm;
    const int32_t *slot_ids;
    float *pool;
    void *out;
    float scale, eps_l2, eps_norm;
    int32_t *err;
};

// Append to and gather from one layer's 4-bit pool (kda_kv4.cuh: its layout).
struct KvCacheArgs {
    int dt, B, T, H, D, max_pages, page_shift, num_pages;
    const void *k, *v;             // append: [T][H][D], tokens k_stride / v_stride elements apart
    long long k_stride, v_stride;
    void *k_out, *v_out;           // gather: [T][H][D]
    const int32_t *cu, *start, *page_table;
    uint8_t *pool;
    float k_scale, v_scale, k_inv, v_inv;
    int32_t *err;
};

struct KvAttentionArgs {
    int dt, B, T, max_q, Hq, Hkv, D, max_pages, page_shift, num_pages, window;
    const void *q;                 // [T][Hq][D], tokens q_stride elements apart
    long long q_stride;
    const int32_t *cu, *kv_lens, *page_table;
    const uint8_t *pool;
    float scale_k, v_scale;        // scale x k_scale x log2(e)
    void *o;
    float *lse;
    uint8_t *ws;
    int32_t *err;
    const int32_t *picked;         // [T][Hkv][count] of a row's pages, or NULL: all of them
    int count;
    uint64_t wait_ns;              // limit of the kernels' waits
    int starve;                    // self-test: the first codes never arrive
};

// Append with rotation: KvCacheArgs' sizes, q beside k and v, and the angles' table.
struct KvRopeArgs {
    int dt, B, T, Hq, Hkv, D, max_pages, page_shift, num_pages, R, positions, pairs;
    int q_groups, kv_groups, q_each, kv_each;      // groups of a token's heads, a thread each, and heads a group (set by the launch)
    unsigned q_blocks, kv_blocks;  // CTAs
    float minus_zero;
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride, qo_stride;
    const float *rope;             // [positions][R]: R / 2 cosines, R / 2 sines
    const int32_t *cu, *start, *page_table;
    uint8_t *pool;
    void *q_out;
    float k_inv, v_inv;
    int32_t *err;
};

// The bounds of the pages that new tokens lie in.
struct KvBoundsArgs {
    int B, T, H, D, max_pages, page_shift, num_pages;
    int slice;                     // tokens a warp looks at (set by the launch)
    const int32_t *cu, *start, *page_table;
    const uint8_t *pool;
    int8_t *bounds;
    int32_t *err;
};

// The pages that each token attends to.
struct KvPickArgs {
    int dt, B, T, max_q, Hq, Hkv, D, max_pages, page_shift, num_pages, count, first, recent;
    int blocks, chunks;            // of tokens a request, of pages (set by the launch)
    const void *q;
    long long q_stride;
    const int32_t *cu, *kv_lens, *page_table;
    const int8_t *bounds;
    int32_t *picked;
    uint32_t *keys;                // [T][Hkv][key_stride]
    long long key_stride;
    int32_t *err;
    uint64_t wait_ns;              // limit of the scores' waits
    int starve;                    // self-test: the first records never all arrive
};

// out = (x + residual) normed, in dtype or in e4m3 with scales.
struct AddNormArgs {
    int dt, tokens, C, mode;
    const void *x, *residual, *w_norm;
    long long x_stride, residual_stride, sum_stride;
    float eps;
    void *sum, *out;
    float *scales;
};

// The page table's state: refs [num_pages], page_table [B][max_pages], lens [B].
struct PageArgs {
    int B, max_pages, page_shift, num_pages;
    int32_t *refs, *page_table, *lens;
    int32_t *err;
};

struct PageCopyParams {
    int P, n, num_pages, step, chunks;
    size_t page_bytes;
    const int32_t *n_dev;          // the number of pairs on the device, or NULL: n
    const int32_t *src, *dst;
    long long cells;               // a compaction's page table entries, sent through map; or 0
    int32_t *table;
    const int32_t *map;
    int32_t *err;
    uint8_t *pool[KDA_MAX_LAYERS];
};

cudaError_t launch_kv4_cache(const KvCacheArgs &a, bool append, cudaStream_t s);
cudaError_t launch_kv4_attention(const KvAttentionArgs &a, cudaStream_t s);
// The same with the rows' picked pages alone.
cudaError_t launch_kv4_attention_picked(const KvAttentionArgs &a, cudaStream_t s);
cudaError_t launch_kv4_rope(const KvRopeArgs &a, cudaStream_t s);
cudaError_t launch_kv4_bounds(KvBoundsArgs a, cudaStream_t s);
cudaError_t launch_kv4_pick(const KvPickArgs &a, cudaStream_t s);
cudaError_t launch_add_rmsnorm(const AddNormArgs &a, cudaStream_t s);
cudaError_t launch_page_alloc(const PageArgs &a, const int32_t *grow, cudaStream_t s);
cudaError_t launch_page_fork(const PageArgs &a, const int32_t *src, const int32_t *dst, int n, PageCopyParams p,
                             int32_t *ws, cudaStream_t s);
cudaError_t launch_page_free(const PageArgs &a, const int32_t *rows, int n, cudaStream_t s);
cudaError_t launch_page_compact(const PageArgs &a, PageCopyParams p, int32_t *ws, int32_t *live, cudaStream_t s);
cudaError_t launch_page_copy(const PageCopyParams &p, cudaStream_t s);
cudaError_t launch_conv_prologue(const PrologueArgs &a, cudaStream_t s);
cudaError_t launch_gated_rmsnorm(const NormArgs &a, cudaStream_t s);
cudaError_t launch_decode_fused(const FusedDecodeArgs &a, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t s);
cudaError_t launch_verify_snapshot(const SnapVerifyArgs &a, cudaStream_t s);
cudaError_t launch_snapshot_commit(const SnapCommitParams &p, cudaStream_t s);
cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s);
cudaError_t launch_fold(const FoldParams &p, int dt, cudaStream_t s);
cudaError_t launch_slot_copy(const CopyParams &p, cudaStream_t s);
// Exact fp32 CUDA-core prefill (token by token, state in registers).
cudaError_t launch_prefill_recurrent(const PrefillArgs &a, cudaStream_t s);
// Chunked tensor-core prefill (bf16 inputs).
cudaError_t launch_prefill_chunked(const PrefillArgs &a, cudaStream_t s);

// One CTA waiting on a barrier nothing arrives at, for wait_us microseconds.
cudaError_t launch_selftest_wait(int32_t *err, int wait_us, cudaStream_t s);

}  // namespace kda
