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
// Products and sums run on channel pairs, each half rounded as the scalar instruction does.  A CTA has queries, keys or
// values.  Prompts of 9.6 K tokens, 64 / 8 heads: 62 us, 5.8 TB/s (0.86 of the copy bandwidth measured), the queries' bytes
// alone 46; the rest is the arithmetic of keys' and values' codes.  384 single tokens: 4.5 us, the launch and three rounds
// of loads.
#include "kda_async.cuh"
#include "kda_internal.h"
#include "kda_kv4_store.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int THREADS = 256;

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

enum Role { QUERIES, KEYS, VALUES };

// Block `block` of those that have this role: (token, group of heads) slots.  AT_ONCE: heads whose loads are in flight together.
template <int D, typename T, bool PAIRS, Role ROLE, int AT_ONCE>
__device__ __forceinline__ void run(const KvRopeArgs &a, unsigned block) {
    constexpr int NL = D / 8, SLOTS = THREADS / NL;
    using L = KvTile<D>;
    const int j = threadIdx.x % NL;        // channels 8 j ..
    const int heads = ROLE == QUERIES ? a.Hq : a.Hkv, groups = ROLE == QUERIES ? a.q_groups : a.kv_groups;
    const int turns_of_loop = ROLE == QUERIES ? a.q_each : a.kv_each;      // the same for a whole warp
    const unsigned slot = block * (unsigned)SLOTS + threadIdx.x / NL;
    const int t = (int)(slot / (unsigned)groups), g = (int)(slot - (unsigned)t * groups);
    int left = t < a.T ? (heads - g + groups - 1) / groups : 0;           // heads still to be asked for
    const long long stride = ROLE == QUERIES ? a.q_stride : ROLE == KEYS ? a.k_stride : a.v_stride;
    const T *src = (const T *)(ROLE == QUERIES ? a.q : ROLE == KEYS ? a.k : a.v) + (size_t)min(t, a.T - 1) * stride + g * D + j * 8;
    const int step = groups * D;
    auto ask = [&]() {                     // (what is read here is written by this thread's warp after it, or by none)
        uint4 w = make_uint4(0, 0, 0, 0);
        if (left-- > 0) w = *reinterpret_cast<const uint4 *>(src);
        src += step;
        return w;
    };
    uint4 next[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) next[i] = ask();
    const Owner own = owner_with(a.cu, a.start, a.B, a.T, t);
    const bool mine = own.b >= 0;
    const long long pos = mine ? (long long)own.more + (t - own.q0) : -1;
    const bool angles = pos >= 0 && pos < a.positions, placed = angles && (pos >> a.page_shift) < a.max_pages;
    if (t < a.T && !placed) report(a.err, DEVERR_SEQLENS);
    uint8_t *out = nullptr;                // null: nothing is written
    int tok = 0;
    if (ROLE == QUERIES) {
        if (mine) out = (uint8_t *)((T *)a.q_out + t * a.qo_stride + g * D + j * 8);
    } else if (placed) {
        const int page = a.page_table[(size_t)own.b * a.max_pages + (pos >> a.page_shift)];
        const int in_page = (int)pos & ((1 << a.page_shift) - 1);
        tok = in_page & (KV_TILE - 1);
        if (page < 0 || page >= a.num_pages) report(a.err, DEVERR_PAGE_RANGE);
        else out = a.pool + ((((size_t)page * a.Hkv + g) << (a.page_shift - 4)) + (in_page >> 4)) * L::BYTES;
    }
    const size_t out_step = ROLE == QUERIES ? (size_t)step * sizeof(T) : (size_t)groups * L::BYTES << (a.page_shift - 4);
    const int turn = a.R / 16;             // lanes of half a rotation
    const bool turns = ROLE != VALUES && j < 2 * turn, lower = j < turn;
    float2 c[4], s[4];                     // of each two channels; the sine with its sign
    if constexpr (ROLE != VALUES) {
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
    }
    const int partner = PAIRS || !turns ? (int)(threadIdx.x & 31) : (int)(threadIdx.x & 31) + (lower ? turn : -turn);
    const float inv = ROLE == KEYS ? a.k_inv : a.v_inv;
    int n = out ? (heads - g + groups - 1) / groups : 0;                  // heads of this thread that are still to be written
    if (ROLE == QUERIES && !angles) {      // (out: the token is a request's)
        for (; n > 0; --n, out += out_step) *reinterpret_cast<uint4 *>(out) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll 1
    for (int done = 0; done < turns_of_loop; done += AT_ONCE) {
        uint4 now[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) now[i] = next[i];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) next[i] = ask();
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            uint4 w = now[i];
            if constexpr (ROLE != VALUES) {
                uint4 z = w;
                if constexpr (!PAIRS) {
                    z.x = __shfl_sync(~0u, w.x, partner);
                    z.y = __shfl_sync(~0u, w.y, partner);
                    z.z = __shfl_sync(~0u, w.z, partner);
                    z.w = __shfl_sync(~0u, w.w, partner);
                }
                if (turns) {
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
            }
            if constexpr (ROLE == QUERIES) {
                if (n > 0) *reinterpret_cast<uint4 *>(out) = w;
            } else {
                float x[8], top = 0.f, one_over;
                unpack16(w, x, T());
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= inv, top = max_nan(top, fabsf(x[k]));
                top = max_nan(top, __shfl_xor_sync(~0u, top, 1));
                const uint32_t sb = scale_of(top, one_over), code = codes_of(x, sb, one_over);
                if (n > 0) {
                    *reinterpret_cast<uint32_t *>(out + (ROLE == VALUES ? L::VC : L::KC) + tok * (D / 2) + j * 4) = code;
                    if ((j & 1) == 0) out[ROLE == VALUES ? L::VS + (j >> 1) * KV_TILE + tok : L::KS + tok * L::BLOCKS + (j >> 1)] = (uint8_t)sb;
                }
            }
            out += out_step;
            --n;
        }
    }
}

template <int D, typename T, bool PAIRS, int Q_AT_ONCE, int KV_AT_ONCE>
__global__ void __launch_bounds__(THREADS) append_rope_kernel(const KvRopeArgs a) {
    wait_for_earlier_kernels();
    let_later_kernels_in();
    const unsigned b = blockIdx.x;
    if (b < a.q_blocks) run<D, T, PAIRS, QUERIES, Q_AT_ONCE>(a, b);
    else if (b - a.q_blocks < a.kv_blocks) run<D, T, PAIRS, KEYS, KV_AT_ONCE>(a, b - a.q_blocks);
    else run<D, T, PAIRS, VALUES, KV_AT_ONCE>(a, b - a.q_blocks - a.kv_blocks);
}

template <int D, typename T>
cudaError_t launch(KvRopeArgs a, cudaStream_t s) {
    constexpr int SLOTS = THREADS / (D / 8);
    // Heads a thread: as many as leave a CTA an SM, up to 8, and as leave two beyond, up to 32; its cos and sin are read once,
    // and one start's chain of loads serves them all.  64 / 8 heads of 128, single tokens of 128 requests 3.4 us, one head a
    // thread 4.8; of 384 4.5 (8 a thread), 7.6 (1); 1.3 K tokens 9.6 (16 a thread), 13.7 (32: a CTA an SM), 13.6 (8 of q, 1 of
    // k and v); 9.6 K tokens 62 (32), 64 (16), 76 (8 and 4).
    auto each = [&](int heads, int most) {
        const long long all = (long long)a.T * heads / (SLOTS * 152), fill = all < 8 ? all : all / 2 < 8 ? 8 : all / 2;
        return (int)(fill < 1 ? 1 : fill > most ? most : fill);
    };
    a.minus_zero = -0.f;
    const int eq = each(a.Hq, 32), ekv = each(a.Hkv, 8);
    a.q_groups = (a.Hq + eq - 1) / eq, a.kv_groups = (a.Hkv + ekv - 1) / ekv;
    a.q_each = (a.Hq + a.q_groups - 1) / a.q_groups, a.kv_each = (a.Hkv + a.kv_groups - 1) / a.kv_groups;
    a.q_blocks = (unsigned)(((long long)a.T * a.q_groups + SLOTS - 1) / SLOTS);
    a.kv_blocks = (unsigned)(((long long)a.T * a.kv_groups + SLOTS - 1) / SLOTS);
    const unsigned grid = a.q_blocks + 2 * a.kv_blocks;
    const bool q1 = a.q_each == 1, kv1 = a.kv_each == 1;
    const auto kernel = a.pairs ? (q1 ? (kv1 ? append_rope_kernel<D, T, true, 1, 1> : append_rope_kernel<D, T, true, 1, 2>)
                                      : (kv1 ? append_rope_kernel<D, T, true, 2, 1> : append_rope_kernel<D, T, true, 2, 2>))
                                : (q1 ? (kv1 ? append_rope_kernel<D, T, false, 1, 1> : append_rope_kernel<D, T, false, 1, 2>)
                                      : (kv1 ? append_rope_kernel<D, T, false, 2, 1> : append_rope_kernel<D, T, false, 2, 2>));
    return launch_early(kernel, dim3(grid), dim3(THREADS), 0, s, a);
}

}  // namespace

cudaError_t launch_kv4_rope(const KvRopeArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return a.D == 128 ? launch<128, __nv_bfloat16>(a, s) : launch<64, __nv_bfloat16>(a, s);
    return a.D == 128 ? launch<128, __half>(a, s) : launch<64, __half>(a, s);
}

}  // namespace kda
