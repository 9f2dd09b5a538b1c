// Append to and read back from the paged 4-bit cache.
//
// Append: for each 16 channels of a token's key or value
//     s = e4m3(max|x| / 6),   code = e2m1(x / s)   (0 where s = 0)
// One thread holds one block of 16 channels: 32 bytes in, 8 bytes of codes and
// one scale out, no communication.  Both directions are bound by HBM for
// prompts and by the launch for single tokens.
#include "kda_internal.h"
#include "kda_kv4_store.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256;

// Where token t's head h lies: its tile, and its token in the tile; null with a bit set on bad input.
template <int D>
__device__ __forceinline__ uint8_t *locate(const KvCacheArgs &a, int t, int h, int &tok) {
    const int b = owner_of(a.cu, a.B, t);
    if (t >= a.T) return nullptr;
    if (b < 0) {
        report(a.err, DEVERR_SEQLENS);
        return nullptr;
    }
    const long long pos = (long long)a.start[b] + (t - a.cu[b]);
    if (pos < 0 || (pos >> a.page_shift) >= a.max_pages) {
        report(a.err, DEVERR_SEQLENS);
        return nullptr;
    }
    const int page = a.page_table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) {
        report(a.err, DEVERR_PAGE_RANGE);
        return nullptr;
    }
    const int in_page = (int)pos & ((1 << a.page_shift) - 1);
    tok = in_page & (KV_TILE - 1);
    return a.pool + ((((size_t)page * a.H + h) << (a.page_shift - 4)) + (in_page >> 4)) * KvTile<D>::BYTES;
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) append_kernel(const KvCacheArgs a) {
    constexpr int NB = D / 16;
    // (token, head) pairs have 31 bits; a CTA holds a whole number of them
    constexpr int PAIRS = THREADS / (2 * NB);
    const int blk = threadIdx.x % NB, side = threadIdx.x / NB & 1;
    const unsigned pair = blockIdx.x * (unsigned)PAIRS + threadIdx.x / (2 * NB);
    const int t = (int)(pair / (unsigned)a.H), h = (int)(pair - (unsigned)t * a.H);
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (t < a.T) {
        const T *src = (side ? (const T *)a.v + t * a.v_stride : (const T *)a.k + t * a.k_stride) + h * D + blk * 16;
        w0 = __ldg(reinterpret_cast<const uint4 *>(src));
        w1 = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
    }
    int tok;
    uint8_t *tile = locate<D>(a, t, h, tok);
    if (!tile) return;
    float x[16];
    unpack16(w0, x, T());
    unpack16(w1, x + 8, T());
    store_block<D>(tile, tok, blk, side, x, side ? a.v_inv : a.k_inv);
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS) gather_kernel(const KvCacheArgs a) {
    constexpr int NB = D / 16;
    using L = KvTile<D>;
    // (token, head) pairs have 31 bits; a CTA holds a whole number of them
    constexpr int PAIRS = THREADS / (2 * NB);
    const int blk = threadIdx.x % NB, side = threadIdx.x / NB & 1;
    const unsigned pair = blockIdx.x * (unsigned)PAIRS + threadIdx.x / (2 * NB);
    const int t = (int)(pair / (unsigned)a.H), h = (int)(pair - (unsigned)t * a.H);
    int tok;
    const uint8_t *tile = locate<D>(a, t, h, tok);
    if (t >= a.T) return;
    uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (tile) {
        const uint2 code = *reinterpret_cast<const uint2 *>(tile + (side ? L::VC : L::KC) + tok * (D / 2) + blk * 8);
        const uint32_t sb = tile[side ? L::VS + blk * KV_TILE + tok : L::KS + tok * NB + blk];
        // code times scale first, exact in fp16: scale times tensor scale alone may leave fp32's range
        const uint32_t ss = e4m3x2_to_f16x2(sb | sb << 8);
        const __half2 s = *reinterpret_cast<const __half2 *>(&ss);
        const float by = side ? a.v_scale : a.k_scale;
        uint32_t h[8];
        e2m1x8_to_f16x2(code.x, *reinterpret_cast<uint32_t(*)[4]>(h));
        e2m1x8_to_f16x2(code.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = __half22float2(__hmul2_rn(*reinterpret_cast<const __half2 *>(&h[i]), s));
            out[i] = pack2(f.x * by, f.y * by, T());
        }
    }
    T *dst = (side ? (T *)a.v_out : (T *)a.k_out) + ((size_t)t * a.H + h) * D + blk * 16;
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

template <int D, typename T>
cudaError_t launch(const KvCacheArgs &a, bool append, cudaStream_t s) {
    constexpr int PAIRS = THREADS / (2 * (D / 16));
    const long long grid = ((long long)a.T * a.H + PAIRS - 1) / PAIRS;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (append) append_kernel<D, T><<<(unsigned)grid, THREADS, 0, s>>>(a);
    else gather_kernel<D, T><<<(unsigned)grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_cache(const KvCacheArgs &a, bool append, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16)
        return a.D == 128 ? launch<128, __nv_bfloat16>(a, append, s) : launch<64, __nv_bfloat16>(a, append, s);
    return a.D == 128 ? launch<128, __half>(a, append, s) : launch<64, __half>(a, append, s);
}

}  // namespace kda
