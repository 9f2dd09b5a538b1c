// Append to the paged 4-bit cache with the position rotation on the way.
//
// Of a token at position p, the first R channels of each head of q and k are turned by p's angles, in pairs (c, c + R / 2)
// or (2 c, 2 c + 1):
//     x1' = x1 cos - x2 sin,   x2' = x2 cos + x1 sin
// each product and sum rounded to fp32, the result to the type that an unfused rotation would store.  q leaves as it is,
// k and v become codes as the append makes them, so the bytes are those of a rotation followed by kda_kv4_append.
//
// A thread holds 8 channels of a head; the other of a (c, c + R / 2) pair comes by shuffles from R / 16 lanes on, and the
// largest of a block of 16 from the lane beside, so that each value is read once and q may be turned in place.  cos and
// sin stay in registers while the thread walks over several heads of its token, with the next ones' loads in flight.
// Products and sums run on channel pairs, each half rounded as the scalar instruction does.  CTAs have queries or keys
// and values, not both.  Bound by HBM for prompts, by the launch for single tokens.
#include "kda_internal.h"
#include "kda_kv4_store.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int AT_ONCE = 2;     // heads whose loads are in flight together

__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
// x c + y s of two channels, three roundings each.  Products and sums of pairs are merged into fused ones even where both
// ask for rounding to nearest; a fused x c + z whose z is not known to be -0 cannot be merged any further.
__device__ __forceinline__ float2 turned(float2 x, float2 y, float2 c, float2 s, float minus_zero) {
    uint64_t a, b;
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a) : "l"(pair(x.x, x.y)), "l"(pair(c.x, c.y)), "l"(pair(minus_zero, minus_zero)));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(b) : "l"(pair(y.x, y.y)), "l"(pair(s.x, s.y)), "l"(pair(minus_zero, minus_zero)));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}

template <int D, typename T, bool PAIRS>
__global__ void __launch_bounds__(THREADS) append_rope_kernel(const KvRopeArgs a) {
    constexpr int NL = D / 8, SLOTS = THREADS / NL;
    using L = KvTile<D>;
    const int j = threadIdx.x % NL;        // channels 8 j ..
    const bool is_q = blockIdx.x < a.q_blocks;
    const int heads = is_q ? a.Hq : 2 * a.Hkv, groups = is_q ? a.q_groups : a.kv_groups;
    const unsigned slot = (blockIdx.x - (is_q ? 0u : a.q_blocks)) * (unsigned)SLOTS + threadIdx.x / NL;
    const int t = (int)(slot / (unsigned)groups), g = (int)(slot - (unsigned)t * groups);
    uint4 next[AT_ONCE];
    auto ask = [&](int i, int h) {         // (what is read here is written by this thread's warp after it, or by none)
        if (t >= a.T || h >= heads) return;
        const T *src = is_q ? (const T *)a.q + t * a.q_stride + h * D
                            : h < a.Hkv ? (const T *)a.k + t * a.k_stride + h * D : (const T *)a.v + t * a.v_stride + (h - a.Hkv) * D;
        next[i] = *reinterpret_cast<const uint4 *>(src + j * 8);
    };
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) next[i] = make_uint4(0, 0, 0, 0), ask(i, g + i * groups);
    const Owner own = owner_with(a.cu, a.start, a.B, a.T, t);
    const bool mine = own.b >= 0;
    const long long pos = mine ? (long long)own.more + (t - own.q0) : -1;
    const bool angles = pos >= 0 && pos < a.positions, placed = angles && (pos >> a.page_shift) < a.max_pages;
    if (t < a.T && !placed) report(a.err, DEVERR_SEQLENS);
    uint8_t *tile = nullptr;               // the token's tile of head 0
    int tok = 0;
    if (!is_q && placed) {
        const int page = a.page_table[(size_t)own.b * a.max_pages + (pos >> a.page_shift)];
        const int in_page = (int)pos & ((1 << a.page_shift) - 1);
        tok = in_page & (KV_TILE - 1);
        if (page < 0 || page >= a.num_pages) report(a.err, DEVERR_PAGE_RANGE);
        else tile = a.pool + (((size_t)page * a.Hkv << (a.page_shift - 4)) + (in_page >> 4)) * L::BYTES;
    }
    const int turn = a.R / 16;             // lanes of half a rotation
    const bool turns = j < 2 * turn, lower = j < turn;
    float2 c[4], s[4];                     // of each two channels; the sine with its sign
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = s[i] = make_float2(0.f, 0.f);
    if (angles && turns) {
        const float *row = a.rope + pos * a.R;
        if constexpr (PAIRS) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(row + 4 * j)), y = __ldg(reinterpret_cast<const float4 *>(row + a.R / 2 + 4 * j));
            c[0] = make_float2(x.x, x.x), c[1] = make_float2(x.y, x.y), c[2] = make_float2(x.z, x.z), c[3] = make_float2(x.w, x.w);
            s[0] = make_float2(-y.x, y.x), s[1] = make_float2(-y.y, y.y), s[2] = make_float2(-y.z, y.z), s[3] = make_float2(-y.w, y.w);
        } else {
            row += 8 * (lower ? j : j - turn);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(row + 2 * i)), y = __ldg(reinterpret_cast<const float4 *>(row + a.R / 2 + 2 * i));
                c[i] = make_float2(x.x, x.y), c[i + 1] = make_float2(x.z, x.w);
                s[i] = lower ? make_float2(-y.x, -y.y) : make_float2(y.x, y.y);
                s[i + 1] = lower ? make_float2(-y.z, -y.w) : make_float2(y.z, y.w);
            }
        }
    }
    const int partner = PAIRS || !turns ? (int)(threadIdx.x & 31) : (int)(threadIdx.x & 31) + (lower ? turn : -turn);
    const size_t head_bytes = (size_t)L::BYTES << (a.page_shift - 4);
#pragma unroll 1
    for (int h0 = g; h0 - g < heads; h0 += AT_ONCE * groups) {       // (the same number of turns for a whole warp)
        uint4 now[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) now[i] = next[i];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) ask(i, h0 + (i + AT_ONCE) * groups);
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int h = h0 + i * groups;
            uint4 w = now[i], z = w;
            if constexpr (!PAIRS) {
                z.x = __shfl_sync(~0u, w.x, partner);
                z.y = __shfl_sync(~0u, w.y, partner);
                z.z = __shfl_sync(~0u, w.z, partner);
                z.w = __shfl_sync(~0u, w.w, partner);
            }
            if (turns && (is_q || h < a.Hkv)) {
                float x[8], y[8], r[8];
                unpack16(w, x, T());
                unpack16(z, y, T());
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 o = turned(make_float2(x[2 * k], x[2 * k + 1]), PAIRS ? make_float2(y[2 * k + 1], y[2 * k]) : make_float2(y[2 * k], y[2 * k + 1]), c[k], s[k], a.minus_zero);
                    r[2 * k] = o.x, r[2 * k + 1] = o.y;
                }
                w = make_uint4(pack2(r[0], r[1], T()), pack2(r[2], r[3], T()), pack2(r[4], r[5], T()), pack2(r[6], r[7], T()));
            }
            if (is_q) {
                if (mine && h < heads)
                    *reinterpret_cast<uint4 *>((T *)a.q_out + t * a.qo_stride + h * D + j * 8) = angles ? w : make_uint4(0, 0, 0, 0);
            } else {
                const bool v = h >= a.Hkv;
                const float inv = v ? a.v_inv : a.k_inv;
                float x[8], top = 0.f, one_over;
                unpack16(w, x, T());
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= inv, top = max_nan(top, fabsf(x[k]));
                top = max_nan(top, __shfl_xor_sync(~0u, top, 1));
                const uint32_t sb = scale_of(top, one_over), code = codes_of(x, sb, one_over);
                if (tile && h < heads) {
                    uint8_t *const at = tile + (v ? h - a.Hkv : h) * head_bytes;
                    const int blk = j >> 1;
                    *reinterpret_cast<uint32_t *>(at + (v ? L::VC : L::KC) + tok * (D / 2) + j * 4) = code;
                    if ((j & 1) == 0) at[v ? L::VS + blk * KV_TILE + tok : L::KS + tok * L::BLOCKS + blk] = (uint8_t)sb;
                }
            }
        }
    }
}

template <int D, typename T>
cudaError_t launch(KvRopeArgs a, cudaStream_t s) {
    constexpr int SLOTS = THREADS / (D / 8);
    // One head a thread while that does not fill the GPU, then up to 8 of q and 4 of k and v, whose cos and sin are read once.
    auto each = [&](int heads, int most) {
        const long long fill = (long long)a.T * heads / (SLOTS * 152 * 8);
        return (int)(fill < 1 ? 1 : fill > most ? most : fill);
    };
    a.minus_zero = -0.f;
    const int eq = each(a.Hq, 8), ekv = each(2 * a.Hkv, 4);
    a.q_groups = (a.Hq + eq - 1) / eq, a.kv_groups = (2 * a.Hkv + ekv - 1) / ekv;
    a.q_blocks = (unsigned)(((long long)a.T * a.q_groups + SLOTS - 1) / SLOTS);
    const unsigned grid = a.q_blocks + (unsigned)(((long long)a.T * a.kv_groups + SLOTS - 1) / SLOTS);
    if (a.pairs) append_rope_kernel<D, T, true><<<grid, THREADS, 0, s>>>(a);
    else append_rope_kernel<D, T, false><<<grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_rope(const KvRopeArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch<128, __nv_bfloat16>(a, s) : launch<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch<128, __half>(a, s) : launch<64, __half>(a, s);
}

}  // namespace kda
