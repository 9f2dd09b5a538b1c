// Attention of each request's newest tokens over its paged 4-bit cache.
//
// Row i of a request with n new tokens and len tokens cached (the new ones
// among them) sees positions j <= len - n + i, and j > len - n + i - window
// where a window is given:
//     o_i = sum_j softmax_j(scale q_i . k_j) v_j,   lse_i = ln sum_j exp(scale q_i . k_j)
// A row that sees nothing has o = 0 and lse = -inf.
//
// One CTA per (token, query head): scores of 128 tokens at a time, then their
// values, with the running maximum and sum of the softmax.
#include "kda_internal.h"
#include "kda_kv4.cuh"

namespace kda {
namespace {

constexpr int THREADS = 128;

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) attention_kernel(const KvAttentionArgs a) {
    using L = KvTile<D>;
    __shared__ float q_s[D], p_s[THREADS], red[4];
    __shared__ const uint8_t *tile_s[THREADS / KV_TILE];
    const int t = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, hk = hq / (a.Hq / a.Hkv), x = threadIdx.x;
    const int b = owner_of(a.cu, a.B, t);
    if (b < 0) return;
    const int n = a.cu[b + 1] - a.cu[b], len = a.kv_lens[b];
    if (n > a.max_q || len < 0 || (long long)len > ((long long)a.max_pages << a.page_shift)) {
        if (x == 0) report(a.err, DEVERR_SEQLENS);
        return;
    }
    const int last = len - n + (t - a.cu[b]);
    const int first = a.window > 0 ? max(0, last + 1 - a.window) : 0;
    for (int d = x; d < D; d += THREADS) q_s[d] = (float)((const T *)a.q)[t * a.q_stride + hq * D + d];
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int j0 = first & ~(KV_TILE - 1); j0 <= last; j0 += THREADS) {
        __syncthreads();
        if (x < THREADS / KV_TILE) {
            const int j = j0 + x * KV_TILE;
            tile_s[x] = nullptr;
            if (j <= last) {
                const int page = a.page_table[(size_t)b * a.max_pages + (j >> a.page_shift)];
                if (page < 0 || page >= a.num_pages) report(a.err, DEVERR_PAGE_RANGE);
                else
                    tile_s[x] = a.pool + ((((size_t)page * a.Hkv + hk) << (a.page_shift - 4)) +
                                          ((j & ((1 << a.page_shift) - 1)) >> 4)) * L::BYTES;
            }
        }
        __syncthreads();
        const int j = j0 + x, tok = x & 15;
        const uint8_t *tile = tile_s[x >> 4];
        float s = -INFINITY;
        if (j >= first && j <= last && tile) {
            s = 0.f;
            for (int blk = 0; blk < D / 16; ++blk) {
                const float sc = f16x2_to_float2(e4m3x2_to_f16x2(tile[L::KS + tok * (D / 16) + blk])).x;
                float part = 0.f;
                for (int i = 0; i < 8; ++i) {
                    const float2 c = f16x2_to_float2(e2m1x2_to_f16x2(tile[tok * (D / 2) + blk * 8 + i]));
                    part += c.x * q_s[blk * 16 + 2 * i] + c.y * q_s[blk * 16 + 2 * i + 1];
                }
                s += part * sc;
            }
            s *= a.scale_k;
        }
        float top = s;
        for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
        if ((x & 31) == 0) red[x >> 5] = top;
        __syncthreads();
        top = max_nan(max_nan(max_nan(red[0], red[1]), max_nan(red[2], red[3])), m);
        const float ref = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(m - ref);
        p_s[x] = exp2f(s - ref);
        __syncthreads();
        acc *= keep;
        l *= keep;
        m = top;
        for (int i = 0; i < THREADS; ++i) {
            const uint8_t *vt = tile_s[i >> 4];
            const int ji = j0 + i;
            if (ji < first || ji > last || !vt) continue;
            l += p_s[i];
            if (x < D) {
                const uint32_t byte = vt[L::VC + (i & 15) * (D / 2) + x / 2];
                const float2 c = f16x2_to_float2(e2m1x2_to_f16x2(byte));
                const float sc = f16x2_to_float2(e4m3x2_to_f16x2(vt[L::VS + x / 16 * KV_TILE + (i & 15)])).x;
                acc += p_s[i] * ((x & 1) ? c.y : c.x) * sc;
            }
        }
    }
    if (x < D) ((T *)a.o)[((size_t)t * a.Hq + hq) * D + x] = (T)(l == 0.f ? 0.f : acc / l * a.v_scale);
    if (x == 0 && a.lse) a.lse[(size_t)t * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D, typename T>
cudaError_t launch(const KvAttentionArgs &a, cudaStream_t s) {
    attention_kernel<D, T><<<(unsigned)(a.T * a.Hq), THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_attention(const KvAttentionArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch<128, __nv_bfloat16>(a, s) : launch<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch<128, __half>(a, s) : launch<64, __half>(a, s);
}

}  // namespace kda
