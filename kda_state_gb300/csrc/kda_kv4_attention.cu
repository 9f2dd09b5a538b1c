// Attention of each request's newest tokens over its paged 4-bit cache.
//
// Row i of a request with n new tokens and len tokens cached (the new ones
// among them) sees positions j <= len - n + i, and j > len - n + i - window
// where a window is given:
//     o_i = sum_j softmax_j(scale q_i . k_j) v_j,   lse_i = ln sum_j exp(scale q_i . k_j)
// A row that sees nothing has o = 0 and lse = -inf.
#include "kda_kv4_decode.cuh"
#include "kda_kv4_tiles.cuh"

namespace kda {
namespace {

template <int D, typename T>
cudaError_t launch(const KvAttentionArgs &a, cudaStream_t s) {
    const long long rows = (long long)a.max_q * (a.Hq / a.Hkv);
    // Few rows: the kernel that reads the cache once, 8 or 16 rows at a time.  64 requests of 0.5 to 6 K tokens, D = 128,
    // 8 kv heads: 16 rows 89 us against 136 us in tiles, 24 rows 149 against 137, 64 rows 280 against 143.
    if (rows <= 8) return kv4::launch_decode_attention<D, 1, T>(a, s);
    if (rows <= 16) return kv4::launch_decode_attention<D, 2, T>(a, s);
    // Tiles with 256 rows a part make half as many parts, which take 1.4 times as long (3.7 K cycles a tile against 2.7 K)
    // and are not cut.  One request: as the waves of parts come out, at 1.3 (300 new tokens of 8 x 8 heads over 3259: 44 us
    // with 128 rows, one wave, 62 with 256; 340: 61 with 256 rows, 79 with 128 in two waves).  Several, of unknown lengths:
    // 256 rows where the average request fills them and there are a quarter more parts than SMs (4 requests of 0.5 to 6 K,
    // 218 parts: 99 us against 119; 109 parts: 76 against 73; between them, 163 parts: 80 against 92, which are left to 128).
    const long long all = (long long)a.T * (a.Hq / a.Hkv);
    bool wide;
    if (a.B == 1) {
        const long long w1 = ((all + 127) / 128 * a.Hkv + kv4::SMS - 1) / kv4::SMS, w2 = ((all + 255) / 256 * a.Hkv + kv4::SMS - 1) / kv4::SMS;
        wide = 13 * w2 < 10 * w1;
    } else {
        wide = all >= 256LL * a.B && all / 256 * a.Hkv >= kv4::SMS * 5 / 4;
    }
    return wide ? kv4::launch_tile_attention<D, 2, T>(a, s) : kv4::launch_tile_attention<D, 1, T>(a, s);
}

// A token's rows of one kv head, 8 or 16 at a time.  Its pages are read for it alone: of drafts that share three quarters of
// theirs, two tokens' rows together (16, in the kernel that has room for one CTA an SM) would read 0.63 of the pages at 1.7
// times the cost each.  96 requests, 64 pages of 32, 64 / 8 heads of 128: 55 us at 4.1 TB/s; 32 requests of 6 drafts, 32
// pages of 64: 94 us, 33 tokens and kv heads a ns as with dense caches.
template <int D, typename T>
cudaError_t launch_picked(const KvAttentionArgs &a, cudaStream_t s) {
    return a.Hq / a.Hkv <= 8 ? kv4::launch_decode_attention<D, 1, T, true>(a, s) : kv4::launch_decode_attention<D, 2, T, true>(a, s);
}

}  // namespace

cudaError_t launch_kv4_attention_picked(const KvAttentionArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch_picked<128, __nv_bfloat16>(a, s) : launch_picked<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch_picked<128, __half>(a, s) : launch_picked<64, __half>(a, s);
}

cudaError_t launch_kv4_attention(const KvAttentionArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch<128, __nv_bfloat16>(a, s) : launch<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch<128, __half>(a, s) : launch<64, __half>(a, s);
}

}  // namespace kda
