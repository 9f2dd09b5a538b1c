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
    if (rows <= 8) return kv4::launch_decode_attention<D, 1, T>(a, s);
    if (rows <= 16) return kv4::launch_decode_attention<D, 2, T>(a, s);
    // 256 rows a part where that still makes enough parts for the SMs
    const long long parts = (long long)a.T * (a.Hq / a.Hkv) / 256 * a.Hkv;
    if (parts >= 2 * kv4::SMS) return kv4::launch_tile_attention<D, 2, T>(a, s);
    return kv4::launch_tile_attention<D, 1, T>(a, s);
}

}  // namespace

cudaError_t launch_kv4_attention(const KvAttentionArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch<128, __nv_bfloat16>(a, s) : launch<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch<128, __half>(a, s) : launch<64, __half>(a, s);
}

}  // namespace kda
