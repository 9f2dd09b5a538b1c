// Append to the paged 4-bit cache with the position rotation on the way.
//
// Of a token at position p, the first R channels of each head of q and k are turned by p's angles, in pairs (c, c + R / 2)
// or (2 c, 2 c + 1):
//     x1' = x1 cos - x2 sin,   x2' = x2 cos + x1 sin
// each product and sum rounded to fp32, the result to the type that an unfused rotation would store.  q leaves as it is,
// k and v become codes as the append makes them, so the bytes are those of a rotation followed by kda_kv4_append.
//
// A thread holds one block of 16 channels of a head; the partner's of a (c, c + R / 2) pair comes by shuffles from R / 32
// lanes on, so that each value is read once and q may be turned in place.  cos and sin stay in registers while the thread
// walks over several heads of its token.  Bound by HBM for prompts, by the launch for single tokens.
#include "kda_internal.h"
#include "kda_kv4_store.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256;

template <int D, typename T, bool PAIRS>
__global__ void __launch_bounds__(THREADS) append_rope_kernel(const KvRopeArgs a) {
    constexpr int NB = D / 16, SLOTS = THREADS / NB;
    const int blk = threadIdx.x % NB, heads = a.Hq + 2 * a.Hkv;
    // (token, group of heads) slots; heads * T has 31 bits
    const unsigned slot = blockIdx.x * (unsigned)SLOTS + threadIdx.x / NB;
    const int t = (int)(slot / (unsigned)a.groups), g = (int)(slot - (unsigned)t * a.groups);
    uint4 next[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    auto ask = [&](int h) {                // (what is read here is written by this thread's warp after it, or by none)
        if (t >= a.T || h >= heads) return;
        const T *src = h < a.Hq ? (const T *)a.q + t * a.q_stride + h * D
                                : h < a.Hq + a.Hkv ? (const T *)a.k + t * a.k_stride + (h - a.Hq) * D : (const T *)a.v + t * a.v_stride + (h - a.Hq - a.Hkv) * D;
        next[0] = reinterpret_cast<const uint4 *>(src + blk * 16)[0];
        next[1] = reinterpret_cast<const uint4 *>(src + blk * 16)[1];
    };
    ask(g);
    const Owner own = owner_with(a.cu, a.start, a.B, a.T, t);
    const bool mine = own.b >= 0;
    long long pos = -1;
    uint8_t *page_at = nullptr;            // the token's tile of head 0
    int tok = 0;
    if (mine) {
        pos = (long long)own.more + (t - own.q0);
        if (pos < 0 || pos >= a.positions || (pos >> a.page_shift) >= a.max_pages) {
            report(a.err, DEVERR_SEQLENS);
        } else {
            const int page = a.page_table[(size_t)own.b * a.max_pages + (pos >> a.page_shift)];
            const int in_page = (int)pos & ((1 << a.page_shift) - 1);
            tok = in_page & (KV_TILE - 1);
            if (page < 0 || page >= a.num_pages) report(a.err, DEVERR_PAGE_RANGE);
            else page_at = a.pool + (((size_t)page * a.Hkv << (a.page_shift - 4)) + (in_page >> 4)) * KvTile<D>::BYTES;
        }
    } else if (t < a.T) {
        report(a.err, DEVERR_SEQLENS);
    }
    const bool turns = pos >= 0 && pos < a.positions;
    const int turn = a.R / 32;             // blocks of half a rotation
    const bool first = blk < turn;
    float cs[16], sn[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (turns && blk < 2 * turn) {
        const float *row = a.rope + pos * a.R + (PAIRS ? blk * 8 : (first ? blk : blk - turn) * 16);
#pragma unroll
        for (int i = 0; i < (PAIRS ? 8 : 16); i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(row + i)), y = __ldg(reinterpret_cast<const float4 *>(row + a.R / 2 + i));
            cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
            sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
        }
    }
    const int partner = (int)(threadIdx.x & 31) + (first ? turn : -turn);
    const int steps = (heads + a.groups - 1) / a.groups;
    const size_t head_bytes = (size_t)KvTile<D>::BYTES << (a.page_shift - 4);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
        const int h = g + i * a.groups;
        const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
        const bool have = mine && h < heads;
        const uint4 w[2] = {next[0], next[1]};
        ask(h + a.groups);
        float x[16];
        if constexpr (PAIRS) {
            unpack16(w[0], x, T());
            unpack16(w[1], x + 8, T());
            if ((is_q || is_k) && blk < 2 * turn) {
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const float lo = x[2 * p], hi = x[2 * p + 1];
                    x[2 * p] = __fsub_rn(__fmul_rn(lo, cs[p]), __fmul_rn(hi, sn[p]));
                    x[2 * p + 1] = __fadd_rn(__fmul_rn(hi, cs[p]), __fmul_rn(lo, sn[p]));
                }
            }
        } else {
            uint4 z[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                z[p].x = __shfl_sync(~0u, w[p].x, partner);
                z[p].y = __shfl_sync(~0u, w[p].y, partner);
                z[p].z = __shfl_sync(~0u, w[p].z, partner);
                z[p].w = __shfl_sync(~0u, w[p].w, partner);
            }
            unpack16(w[0], x, T());
            unpack16(w[1], x + 8, T());
            if ((is_q || is_k) && blk < 2 * turn) {
                float y[16];
                unpack16(z[0], y, T());
                unpack16(z[1], y + 8, T());
#pragma unroll
                for (int p = 0; p < 16; ++p) {
                    const float c = __fmul_rn(x[p], cs[p]), s = __fmul_rn(y[p], sn[p]);
                    x[p] = first ? __fsub_rn(c, s) : __fadd_rn(c, s);
                }
            }
        }
        if (!have) continue;
        if (is_q) {
            uint32_t o[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) o[p] = turns ? pack2(x[2 * p], x[2 * p + 1], T()) : 0u;
            uint4 *dst = reinterpret_cast<uint4 *>((T *)a.q_out + t * a.qo_stride + h * D + blk * 16);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        } else if (page_at) {
            if (is_k) {                    // rounded to the type, as an unfused rotation would leave it
                uint32_t o[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) o[p] = pack2(x[2 * p], x[2 * p + 1], T());
                unpack16(make_uint4(o[0], o[1], o[2], o[3]), x, T());
                unpack16(make_uint4(o[4], o[5], o[6], o[7]), x + 8, T());
            }
            const int kv = is_k ? h - a.Hq : h - a.Hq - a.Hkv;
            store_block<D>(page_at + kv * head_bytes, tok, blk, is_k ? 0 : 1, x, is_k ? a.k_inv : a.v_inv);
        }
    }
}

template <int D, typename T>
cudaError_t launch(KvRopeArgs a, cudaStream_t s) {
    constexpr int SLOTS = THREADS / (D / 16);
    const int heads = a.Hq + 2 * a.Hkv;
    // One head a thread while that does not fill the GPU, then up to eight, whose cos and sin are read once.
    const long long fill = (long long)a.T * heads / (SLOTS * 152 * 8);
    const int each = (int)(fill < 1 ? 1 : fill > 8 ? 8 : fill);
    a.groups = (heads + each - 1) / each;
    const long long grid = ((long long)a.T * a.groups + SLOTS - 1) / SLOTS;
    if (a.pairs) append_rope_kernel<D, T, true><<<(unsigned)grid, THREADS, 0, s>>>(a);
    else append_rope_kernel<D, T, false><<<(unsigned)grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_rope(const KvRopeArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch<128, __nv_bfloat16>(a, s) : launch<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch<128, __half>(a, s) : launch<64, __half>(a, s);
}

}  // namespace kda
