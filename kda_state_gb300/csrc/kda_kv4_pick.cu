// Which pages of a long cache a token attends to, by a score that is cheap and exact.
//
// Of every page and kv head a record holds the largest and smallest value of each channel of its keys, rounded outwards to
// whole numbers of a unit 2^e: hi_c = ceil(max_t k_tc / 2^e), lo_c = floor(min_t k_tc / 2^e), with e the least that keeps
// them in [-127, 127].  For the queries q_h of a kv head,
//     sum_h q_h . k_t <= sum_c up_c max_t k_tc - down_c min_t k_tc,   up = sum_h max(q_h, 0), down = sum_h max(-q_h, 0)
// for each token t of the page.  u and d are up and down as whole numbers 0 .. 127 of a unit that is the row's own, and the
// score is 2^e sum_c (u_c hi_c - d_c lo_c): a whole number below 2^23 times a power of two, exact in fp32.  So the pages
// picked do not depend on the order of a sum, and equal scores are equal: the lower page is taken.
//
// Records are int8 [num_pages][Hkv][2 D + 16]: hi, lo, e, zeros.  e = 127 marks a page with a NaN (its score is infinite).
//
// Single tokens are bound by the records' bytes and, as these are few, by a chain of dependent loads in each of three
// kernels: 96 requests of 900 to 16 K tokens in pages of 32 take 29 us with the bounds before them (5 to 7 us bounds, 16
// scores at 3.5 TB/s, 3 to 4 behind them for the rows' picks; floor 9), one of 131 K tokens in pages of 64 takes 13.  Prompts are
// bound by issue: 1552 tokens, 8 kv heads, up to 384 pages 35 us (5, 18, 11 behind them).
#include "kda_async.cuh"
#include "kda_internal.h"
#include "kda_kv4.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int UNBOUNDED = 127;
constexpr int SMS = 152;

// The least e with top <= 127 x 2^e, of a finite top > 0 that is a normal number.
__device__ __forceinline__ int unit_of(float top) {
    const uint32_t u = __float_as_uint(top);
    return (int)(u >> 23) - 127 + 1 - 7 + ((u & 0x7fffffu) > 0x7e0000u);     // 127/64 = 1.984375
}
__device__ __forceinline__ float power_of(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
    const __half2 r = __hmin2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t scaled(uint32_t codes, uint32_t scale) {
    const __half2 r = __hmul2_rn(*reinterpret_cast<__half2 *>(&codes), *reinterpret_cast<__half2 *>(&scale));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// ---------------------------------------------------------------------------
// the bounds of the pages that new tokens lie in
// ---------------------------------------------------------------------------

// Lanes that differ in the bit FROM join what they hold of N pairs of channels, and keep a half each: from `at` on.
template <int N, int FROM>
__device__ __forceinline__ void fold(uint32_t (&hi)[16], uint32_t (&lo)[16], int &at) {
    constexpr int H = N / 2;
    const bool upper = threadIdx.x & FROM;
    at += upper ? H : 0;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const uint32_t gh = __shfl_xor_sync(~0u, upper ? hi[i] : hi[i + H], FROM), gl = __shfl_xor_sync(~0u, upper ? lo[i] : lo[i + H], FROM);
        hi[i] = hmax2(upper ? hi[i + H] : hi[i], gh);
        lo[i] = hmin2(upper ? lo[i + H] : lo[i], gl);
    }
}

// One page of one head: fill tokens (>= 1) of its tiles.  Code x scale is exact in fp16, so that the bounds are the values'
// own.
template <int D>
__device__ __forceinline__ void bound_page(const uint8_t *tiles, int fill, int8_t *record) {
    using L = KvTile<D>;
    constexpr int CHUNKS = D / 32, ROWS = 32 / CHUNKS;     // lanes that hold a token, 32 channels each; tokens at a time
    const int lane = threadIdx.x & 31, c = lane % CHUNKS;
    uint32_t hi[16], lo[16], nan = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) hi[i] = 0xfc00fc00u, lo[i] = 0x7c007c00u;
#pragma unroll 2
    for (int t = lane / CHUNKS; t < fill; t += ROWS) {
        const uint8_t *tile = tiles + (t >> 4) * L::BYTES;
        const uint4 w = *reinterpret_cast<const uint4 *>(tile + L::KC + (t & 15) * (D / 2) + c * 16);
        const uint32_t pair = *reinterpret_cast<const uint16_t *>(tile + L::KS + (t & 15) * L::BLOCKS + c * 2);
        nan |= ((pair & 0x7f) == 0x7f) | ((pair & 0x7f00) == 0x7f00);
        const uint32_t s = e4m3x2_to_f16x2(pair), s0 = __byte_perm(s, s, 0x1010), s1 = __byte_perm(s, s, 0x3232);
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t f[4];
            e2m1x8_to_f16x2(word[q], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = scaled(f[i], q < 2 ? s0 : s1);
                hi[4 * q + i] = hmax2(hi[4 * q + i], x);
                lo[4 * q + i] = hmin2(lo[4 * q + i], x);
            }
        }
    }
    int at = 0;
    fold<16, 16>(hi, lo, at);
    fold<8, 8>(hi, lo, at);
    fold<4, 4>(hi, lo, at);
    if constexpr (D == 64) fold<2, 2>(hi, lo, at);
    constexpr int OWN = D == 64 ? 1 : 2;                    // pairs of channels that the lane is left with
    float top = 0.f;
    float2 h[OWN], l[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        h[i] = f16x2_to_float2(hi[i]), l[i] = f16x2_to_float2(lo[i]);
        top = fmaxf(top, fmaxf(fmaxf(fabsf(h[i].x), fabsf(h[i].y)), fmaxf(fabsf(l[i].x), fabsf(l[i].y))));
    }
    top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
    const bool any_nan = __any_sync(~0u, nan != 0);
    const int e = any_nan ? UNBOUNDED : top > 0.f ? unit_of(top) : 0;
    const float per = power_of(any_nan ? 0 : -e);
    uint32_t bh = 0, bl = 0;
#pragma unroll
    for (int i = 0; i < OWN && !any_nan; ++i) {
        bh |= ((uint32_t)(int)ceilf(h[i].x * per) & 255u) << (16 * i) | ((uint32_t)(int)ceilf(h[i].y * per) & 255u) << (16 * i + 8);
        bl |= ((uint32_t)(int)floorf(l[i].x * per) & 255u) << (16 * i) | ((uint32_t)(int)floorf(l[i].y * per) & 255u) << (16 * i + 8);
    }
    const int ch = c * 32 + 2 * at;
    if constexpr (D == 128) {
        *reinterpret_cast<uint32_t *>(record + ch) = bh;
        *reinterpret_cast<uint32_t *>(record + D + ch) = bl;
    } else {
        *reinterpret_cast<uint16_t *>(record + ch) = (uint16_t)bh;
        *reinterpret_cast<uint16_t *>(record + D + ch) = (uint16_t)bl;
    }
    if (lane == 0) *reinterpret_cast<uint4 *>(record + 2 * D) = make_uint4((uint32_t)e & 255u, 0, 0, 0);
}

// A warp takes one head of `slice` tokens (1 to 32), and of those the ones that are their request's first in a page.
template <int D>
__global__ void __launch_bounds__(THREADS) bounds_kernel(const KvBoundsArgs a) {
    wait_for_earlier_kernels();
    let_later_kernels_in();
    const int lane = threadIdx.x & 31;
    const unsigned unit = blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
    const int h = (int)(unit % (unsigned)a.H);
    const long long t0 = (long long)(unit / (unsigned)a.H) * a.slice;
    if (t0 >= a.T) return;
    const int t = (int)min(t0 + min(lane, a.slice - 1), (long long)a.T);
    const Owner own = owner_with(a.cu, a.start, a.B, a.T, t);
    int page = -1, fill = 0;
    if (lane < a.slice && t < a.T) {
        const int i = t - own.q0, P = 1 << a.page_shift;
        const long long pos = (long long)own.more + i, end = (long long)own.more + (own.end - own.q0);
        if (own.b < 0 || pos < 0 || (pos >> a.page_shift) >= a.max_pages) {
            report(a.err, DEVERR_SEQLENS);
        } else if (i == 0 || (pos & (P - 1)) == 0) {
            page = a.page_table[(size_t)own.b * a.max_pages + (pos >> a.page_shift)];
            if (page < 0 || page >= a.num_pages) {
                report(a.err, DEVERR_PAGE_RANGE);
                page = -1;
            }
            fill = (int)min((long long)P, end - (pos & ~(long long)(P - 1)));
        }
    }
    for (uint32_t todo = __ballot_sync(~0u, page >= 0); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, p = __shfl_sync(~0u, page, from), f = __shfl_sync(~0u, fill, from);
        const size_t at = (size_t)p * a.H + h;
        bound_page<D>(a.pool + (at << (a.page_shift - 4)) * KvTile<D>::BYTES, f, a.bounds + at * (2 * D + 16));
    }
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------

constexpr int HEADS_1 = 8, HEADS = 2;      // kv heads that a CTA takes with single tokens, and with several
constexpr int TOKENS = 8;                  // several
constexpr int MISSING = 1000;              // in place of a unit: a page out of range, whose key is 1 (below every score; 0 is no page)

// The bits of a finite or infinite float as a number that orders as it does.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// What request b has of new tokens and cache; n = 0 where it is malformed.
struct Tokens {
    int q0, n, len;
};
__device__ __forceinline__ void check(const KvPickArgs &a, Tokens &r, bool tell) {
    if (r.q0 < 0 || r.n < 0 || r.n > a.max_q || (long long)r.q0 + r.n > a.T || r.len < 0 ||
        (long long)r.len > ((long long)a.max_pages << a.page_shift)) {
        if (tell) report(a.err, DEVERR_SEQLENS);
        r.n = 0;
    }
}

template <typename T> __device__ __forceinline__ float2 halves(uint32_t w);
template <> __device__ __forceinline__ float2 halves<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 halves<__half>(uint32_t w) { return f16x2_to_float2(w); }

// A value of T, without its sign, as m 2^(place - 133) (finite).
__device__ __forceinline__ uint32_t whole_of(uint32_t bits, __nv_bfloat16, int &place) {
    const int e = bits >> 7 & 255;
    place = max(e, 1) - 1;
    return (bits & 127) | (e ? 128 : 0);
}
__device__ __forceinline__ uint32_t whole_of(uint32_t bits, __half, int &place) {
    const int e = bits >> 10 & 31;
    place = max(e, 1) + 108;
    return (bits & 1023) | (e ? 1024 : 0);
}

// The sign of sum_h x_h - m 2^e, exact; x_h is max(v, 0), max(-v, 0) or |v| (side 1, -1, 0) of a head's value v, the first of
// them at `at`.  m < 2^24, -101 <= e <= 122.
template <int D, typename T>
__device__ __forceinline__ int against(const uint16_t *at, int G, int side, uint32_t m, int e) {
    float sum = 0.f;                       // off by less than G 2^-23 of itself
    for (int g = 0; g < G; ++g) {
        const float v = halves<T>(at[(size_t)g * D]).x;
        sum += side == 0 ? fabsf(v) : fmaxf((float)side * v, 0.f);
    }
    const float mark = (float)m * power_of(e), off = sum * ((float)G * 0x1p-23f);
    if (G < 1 << 20 && sum - mark > off) return 1;
    if (G < 1 << 20 && mark - sum > off) return -1;
    long long s = 0;                       // 16 bits at a time, from the lowest on
    bool some = false;
    for (int i = 0; i < 18; ++i) {
        for (int g = 0; g < G; ++g) {
            const uint32_t v = at[(size_t)g * D];
            int place;
            const uint32_t w = whole_of(v, T(), place);
            if (place >> 4 == i && (side == 0 || (side < 0) == (v >> 15 != 0))) s += (long long)w << (place & 15);
        }
        if ((e + 133) >> 4 == i) s -= (long long)m << ((e + 133) & 15);
        some |= (s & 0xffff) != 0;
        s >>= 16;
    }
    return s < 0 ? -1 : s > 0 || some;
}

// The whole number that sum_h x_h / 2^f rounds to (x_h as above, side 1 or -1), known to be k or k + 1: up to 41 bits below
// the border between them, and what the rest may add.
template <int D, typename T>
__device__ __noinline__ int settled(const uint16_t *at, int G, int side, int k, int f) {
    long long s = -((long long)(2 * k + 1) << 40);
    int parts = 0;                         // values that have bits below, less than 1 each
    for (int g = 0; g < G; ++g) {
        const uint32_t v = at[(size_t)g * D];
        if ((side < 0) != (v >> 15 != 0)) continue;
        int place;
        const uint32_t w = whole_of(v, T(), place);
        const int by = place - (f + 92);
        if (by >= 0) {
            s += (long long)w << by;
        } else {
            s += w >> min(-by, 31);
            parts += (w & ((1u << min(-by, 31)) - 1)) != 0;
        }
    }
    const int x = s >= 0 ? s > 0 || parts : s + parts <= 0 ? -1 : against<D, T>(at, G, side, 2 * k + 1, f - 1);
    return k + (x > 0 || (x == 0 && (k & 1)));
}

// u and d of the lane's D / 32 channels, a byte each, from exact sums; a warp's work, where fp32 sums do not tell the unit.  f:
// about the unit.
template <int D, typename T>
__device__ __noinline__ uint2 asked_exactly(const T *q, int G, int f) {
    constexpr int N = D / 32;
    const uint16_t *const at = reinterpret_cast<const uint16_t *>(q) + (threadIdx.x & 31) * N;
    bool good = true;                      // finite, and |q| adds up to a finite fp32
    for (int i = 0; i < N; ++i)
        for (int g = 0; g < G; ++g) good = good && isfinite(halves<T>(at[(size_t)g * D + i]).x);
    for (int i = 0; i < N; ++i) good = good && against<D, T>(at + i, G, 0, 0xffffffu, 104) <= 0;
    if (!__all_sync(~0u, good)) return make_uint2(0, 0);
    auto past = [&](int e) {
        bool any = false;
        for (int i = 0; i < N; ++i)
            for (int side = -1; side <= 1; side += 2) any = any || against<D, T>(at + i, G, side, 127, e) > 0;
        return __any_sync(~0u, any);
    };
    f = max(f - 1, -100);
    while (f > -100 && !past(f - 1)) --f;
    while (past(f)) ++f;
    uint32_t r[2] = {0, 0};
    for (int i = 0; i < 2 * N; ++i) {
        const uint16_t *const c = at + (i >> 1);
        const int side = i & 1 ? -1 : 1;
        float sum = 0.f;
        for (int g = 0; g < G; ++g) sum += fmaxf((float)side * halves<T>(c[(size_t)g * D]).x, 0.f);
        auto above = [&](int k) {          // the nearest whole number is k + 1 or more
            const int x = against<D, T>(c, G, side, 2 * k + 1, f - 1);
            return x > 0 || (x == 0 && (k & 1));
        };
        int k = min(__float2int_rn(sum * power_of(-f)), 127);
        while (k < 127 && above(k)) ++k;
        while (k > 0 && !above(k - 1)) --k;
        r[i & 1] |= (uint32_t)k << (8 * (i >> 1));
    }
    return make_uint2(r[0], r[1]);
}

// Half the sum of a channel's magnitudes up to which its fp32 sums are exact: 2^23 times the lowest bit that its values can
// have, by the least of them that is not 0 (bits - 1 of it, or 0x7fff; 0 of a subnormal, which is not looked into).
__device__ __forceinline__ float exact_to(uint32_t least, __nv_bfloat16) { return __uint_as_float((least + 1 & 0x7f80u) << 16) * 0x1p16f; }
__device__ __forceinline__ float exact_to(uint32_t least, __half) {
    const uint32_t e = least + 1 & 0x7c00u;
    return e ? __uint_as_float((e << 13) + (112u << 23)) * 0x1p13f : 0.f;
}

// u and -d of a token and kv head; a warp's work, N of them at once so that their loads are in flight together.  q(n) is where
// number n's queries lie; put(n, channel, x, y) gets D / 32 of each, from `channel` on.
//
// They are the exact sums' whole numbers.  fp32 sums are exact where a channel's values do not lie further apart than its 24
// bits, and settle what is not near a tie or the border of a unit; the few channels where neither holds (of normal queries one
// row of 8 heads in 600 has one) are looked at exactly.
template <int D, int N, typename T, typename Q, typename Put>
__device__ __forceinline__ void ask_of(const Q &q, int G, const Put &put) {
    constexpr int W = D / 64;              // words of the lane: 2 W channels
    const int lane = threadIdx.x & 31;
    // up = (sum |f| + sum f) / 2 and down = (sum |f| - sum f) / 2, an addition less a value than from their parts; halves
    // are exact, and an infinity or a NaN stays one
    float all[N][2 * W], net[N][2 * W];
    uint32_t least[N][W];                  // of each two channels the least |f| but 0: bits - 1 with the sign set, compared as signed
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) all[n][i] = net[n][i] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) least[n][i] = 0x7fff7fffu;
    }
    for (int g0 = 0; g0 < G; g0 += 8) {    // eight heads' loads at once
        uint32_t w[N][8][W];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const T *const src = q(n);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                if constexpr (W == 2) {
                    const uint2 x = g0 + g < G ? __ldg(reinterpret_cast<const uint2 *>(src + (g0 + g) * D + lane * 4)) : make_uint2(0, 0);
                    w[n][g][0] = x.x, w[n][g][W - 1] = x.y;
                } else {
                    w[n][g][0] = g0 + g < G ? __ldg(reinterpret_cast<const uint32_t *>(src + (g0 + g) * D + lane * 2)) : 0u;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int g = 0; g < 8; ++g)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float2 f = halves<T>(w[n][g][i]);
                    all[n][2 * i] += fabsf(f.x), net[n][2 * i] += f.x;
                    all[n][2 * i + 1] += fabsf(f.y), net[n][2 * i + 1] += f.y;
                    least[n][i] = __vmins2(least[n][i], (w[n][g][i] | 0x80008000u) - 0x00010001u);
                }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float top = 0.f;
        uint32_t open = 0;                 // channels whose sums may have lost bits
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            all[n][i] *= 0.5f, net[n][i] *= 0.5f;
            top = max_nan(top, all[n][i] + fabsf(net[n][i]));
            if (!(all[n][i] <= exact_to(least[n][i / 2] >> (16 * (i & 1)), T()))) open |= 1u << i;
        }
        const uint32_t bits = __reduce_max_sync(~0u, __float_as_uint(top) & 0x7fffffffu);       // (a NaN is above all)
        // nothing to go by: all pages score 0
        const int f = max(unit_of(__uint_as_float(bits)), -100);
        const float per = bits >= 0x7f800000u || bits < 0x00800000u ? 0.f : power_of(-f);
        int u[2 * W], d[2 * W];
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            u[i] = per == 0.f ? 0 : __float2int_rn((all[n][i] + net[n][i]) * per);
            d[i] = per == 0.f ? 0 : __float2int_rn((net[n][i] - all[n][i]) * per);
        }
        bool unit_open = bits >= 0x7e800000u;          // (2^126: |q| may add up to more than fp32 has)
        if (open) {
            unit_open = unit_open || G > 4096 || abs((int)(bits & 0x7fffffu) - 0x7e0000) <= 8 * (G + 2);
            const float half = 0.5f - (float)(G + 2) * 0x1p-15f;       // (sums are off by G + 1 times 254 2^-24 of a unit)
            const uint16_t *const at = reinterpret_cast<const uint16_t *>(q(n)) + lane * 2 * W;
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) {
                const float x = (all[n][i] + net[n][i]) * per, y = (all[n][i] - net[n][i]) * per;
                if (!(open >> i & 1)) continue;
                if (fabsf(x - rintf(x)) >= half) u[i] = settled<D, T>(at + i, G, 1, (int)x, f);
                if (fabsf(y - rintf(y)) >= half) d[i] = -settled<D, T>(at + i, G, -1, (int)y, f);
            }
        }
        if (__any_sync(~0u, unit_open)) {
            const uint2 x = asked_exactly<D, T>(q(n), G, f);
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) u[i] = x.x >> (8 * i) & 255, d[i] = -(int)(x.y >> (8 * i) & 255);
        }
        put(n, lane * 2 * W, u, d);
    }
}

// What a CTA scores: up to `tokens` tokens of one request, with a run of its pages, for up to `heads` kv heads.
struct Share {
    int b, q0, nt, h0, heads, p0, p1;      // p0 >= p1: nothing
};
__device__ __forceinline__ Share share_of(const KvPickArgs &a, int tokens, int heads) {
    Share s;
    const int chunk = blockIdx.y;
    s.h0 = blockIdx.z * heads, s.heads = min(heads, a.Hkv - s.h0);
    s.b = tokens == 1 ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)a.blocks);
    const int i0 = tokens == 1 ? 0 : (int)(blockIdx.x % (unsigned)a.blocks) * tokens;
    Tokens rq{a.cu[s.b], 0, a.kv_lens[s.b]};
    rq.n = a.cu[s.b + 1] - rq.q0;
    check(a, rq, false);                   // (told by pick_kernel)
    s.p0 = s.p1 = 0;
    if (i0 >= rq.n) return s;
    s.q0 = rq.q0 + i0, s.nt = min(tokens, rq.n - i0);
    const int last = rq.len - rq.n + i0 + s.nt - 1;        // the last token's position
    const int pages = last < 0 ? 0 : (last >> a.page_shift) + 1;
    if (pages <= a.count) return s;        // all of them are taken
    const int run = 32 * ((THREADS / 32) / s.heads);       // what the CTA's warps take at a time
    const int per = a.chunks * run >= a.max_pages ? run : ((pages + a.chunks - 1) / a.chunks + run - 1) / run * run;
    s.p0 = (int)min((long long)chunk * per, (long long)pages), s.p1 = min(pages, s.p0 + per);
    return s;
}
__device__ __forceinline__ uint32_t key_of(float sum, int unit) {
    return unit == MISSING ? 1u : unit == UNBOUNDED ? 0xff800000u : ordered(sum * power_of(unit));
}
// pg, or 0 with `bad` set where it is out of range
__device__ __forceinline__ int page_or_0(const KvPickArgs &a, int pg, bool &bad) {
    bad = pg < 0 || pg >= a.num_pages;
    if (bad) report(a.err, DEVERR_PAGE_RANGE);
    return bad ? 0 : pg;
}

template <int D>
struct OneShape {
    // a page's records lie 16 bytes further than they are long, so that neighbouring lanes' 16-byte words meet no bank twice
    static constexpr int RECORD = 2 * D + 16, STAGE = 32 * (HEADS_1 * RECORD + 8 * 16), SMEM = STAGE + HEADS_1 * 2 * D + 16;
};

// Single tokens.  A run of pages' records, each one block of all the CTA's heads, comes by bulk copies while the queries are
// added up; then a lane multiplies one page's on the integer units.  (An 8-bit MMA of 16 pages and 32 channels takes 64
// cycles a scheduler here; the same products of one token take 4 of these instructions, 8 cycles.)
template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 3) score_one_kernel(const KvPickArgs a) {
    using S = OneShape<D>;
    constexpr int RECORD = S::RECORD;
    extern __shared__ __align__(128) uint8_t smem[];
    int8_t *const ask = reinterpret_cast<int8_t *>(smem + S::STAGE);
    const uint32_t bar = shared_addr(smem + S::STAGE + HEADS_1 * 2 * D);
    wait_for_earlier_kernels();
    let_later_kernels_in();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // where a chunk is one run, this lane's page is asked for beside the request's numbers
    const int heads0 = min(HEADS_1, a.Hkv - (int)blockIdx.z * HEADS_1), run0 = 32 * ((THREADS / 32) / heads0);
    const bool one_run = a.chunks * run0 >= a.max_pages;
    const int early_at = (int)min((long long)blockIdx.y * run0 + 32 * (w / heads0) + lane, 0x7fffffffLL);
    const int early = one_run && early_at < a.max_pages ? a.page_table[(size_t)blockIdx.x * a.max_pages + early_at] : 0;
    const Share z = share_of(a, 1, HEADS_1);
    if (z.p0 >= z.p1) return;
    // the warps are dealt over the heads, and those of a head over the runs of 32 pages
    const int parts = (THREADS / 32) / z.heads, part = w / z.heads, h = w - part * z.heads, stride = 32 * parts;
    const bool works = part < parts;
    const int page_bytes = z.heads * RECORD, apart = page_bytes + 16;       // an odd number of 16 bytes for 8, 4, 2 heads
    uint8_t *const stage = smem + 32 * part * apart;
    if (threadIdx.x == 0) {
        barrier_init(bar, parts);
        if (a.starve) barrier_await(bar, 16);      // (a self-test: bytes that nobody copies)
    }
    __syncthreads();
    bool good = false;                     // page p + lane
    auto fetch = [&](int p) {
        if (!works) return;
        const bool asked = p + lane < z.p1;
        const int page = !asked || one_run ? early : a.page_table[(size_t)z.b * a.max_pages + p + lane];
        good = asked && page >= 0 && page < a.num_pages;
        if (asked && !good) report(a.err, DEVERR_PAGE_RANGE);
        if (h != 0) return;
        const uint32_t there = __ballot_sync(~0u, good);
        if (lane == 0) barrier_expect(bar, __popc(there) * page_bytes);
        __syncwarp();
        if (good) bulk_copy(stage + lane * apart, a.bounds + ((size_t)page * a.Hkv + z.h0) * RECORD, page_bytes, bar);
    };
    int p = z.p0 + 32 * part;
    fetch(p);
    const int G = a.Hq / a.Hkv;
    for (int i = w; i < z.heads; i += THREADS / 32)
        ask_of<D, 1, T>([&](int) { return (const T *)a.q + (long long)z.q0 * a.q_stride + (z.h0 + i) * G * D; }, G, [&](int, int ch, const int *u, const int *d) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) ask[i * 2 * D + ch + k] = (int8_t)u[k], ask[i * 2 * D + D + ch + k] = (int8_t)d[k];
        });
    __syncthreads();
    uint32_t *const keys = a.keys + ((size_t)z.q0 * a.Hkv + z.h0 + h) * a.key_stride;
    for (int turn = 0, q0 = z.p0;; ++turn) {       // (q0: of the CTA)
        const bool landed = __all_sync(~0u, barrier_wait_for(bar, turn & 1, a.wait_ns));       // (each lane looks at its own clock)
        if (!landed) {
            if (lane == 0) report(a.err, DEVERR_TIMEOUT);
            barrier_wait_for(bar, turn & 1, a.wait_ns);            // (copies that are under way land in this CTA's memory)
        }
        if (works && landed) {
            const uint4 *x = reinterpret_cast<const uint4 *>(stage + lane * apart + h * RECORD), *y = reinterpret_cast<const uint4 *>(ask + h * 2 * D);
            int s[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint4 u = x[i], v = y[i];
                s[i & 1] = __dp4a((int)u.x, (int)v.x, s[i & 1]);
                s[i & 1] = __dp4a((int)u.y, (int)v.y, s[i & 1]);
                s[i & 1] = __dp4a((int)u.z, (int)v.z, s[i & 1]);
                s[i & 1] = __dp4a((int)u.w, (int)v.w, s[i & 1]);
            }
            if (p + lane < z.p1) keys[p + lane] = key_of((float)(s[0] + s[1]), good ? (int)*reinterpret_cast<const int8_t *>(x + D / 8) : MISSING);
        }
        q0 += stride, p += stride;
        if (q0 >= z.p1) break;
        if (!__syncthreads_and(landed)) return;                    // all have read the stage
        fence_async_shared();
        fetch(p);
    }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four signed bytes as fp16: 1024 + 128 + byte has them in its low bits.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t v = w ^ 0x80808080u, bias = 0x64806480u;
    uint32_t l = __byte_perm(v, 0x64646464u, 0x4140), h = __byte_perm(v, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&l), *reinterpret_cast<const __half2 *>(&bias));
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&h), *reinterpret_cast<const __half2 *>(&bias));
    lo = *reinterpret_cast<const uint32_t *>(&x), hi = *reinterpret_cast<const uint32_t *>(&y);
}

// Up to 8 tokens of a request.  Pages stand on the 16 rows of an fp16 MMA and tokens on its 8 columns: whole numbers up to
// 127 are exact, and so are their sums below 2^23.  The contraction may be permuted if both operands agree, so that a
// lane's share of a record is whole 16-byte words, four lanes beside each other.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS, D == 64 ? 3 : 2) score_kernel(const KvPickArgs a) {
    constexpr int RECORD = 2 * D + 16, PARTS = D / 32;     // runs of 64 bytes of a record
    constexpr int ROW = 4 * D + 64;        // bytes of one token's asked numbers: rows that follow each other meet no bank twice
    __shared__ __align__(16) uint8_t ask[HEADS * TOKENS * ROW];
    wait_for_earlier_kernels();
    let_later_kernels_in();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const Share z = share_of(a, TOKENS, HEADS);
    if (z.p0 >= z.p1) return;
    const int parts = (THREADS / 32) / z.heads, part = w / z.heads, h = w - part * z.heads, stride = 32 * parts;
    uint4 x[2][2][PARTS];                  // of pages p + 16 s + 8 k + r: this lane's quarter of each 64 bytes
    int unit[2];                           // of page p + 16 s + (lane & 15)
    auto look = [&](int p) { return p + lane < z.p1 ? a.page_table[(size_t)z.b * a.max_pages + p + lane] : 0; };
    auto record = [&](int pg) { return a.bounds + ((size_t)pg * a.Hkv + z.h0 + h) * RECORD; };
    auto load = [&](int s, int pages) {    // half of a run, of 32 looked up
        bool bad;
        const int pg = page_or_0(a, __shfl_sync(~0u, pages, 16 * s + (lane & 15)), bad);
        unit[s] = bad ? MISSING : __ldg(record(pg) + 2 * D);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 *src = reinterpret_cast<const uint4 *>(record(__shfl_sync(~0u, pg, 8 * k + r))) + c;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) x[s][k][i] = __ldg(src + 4 * i);
        }
    };
    int p = z.p0 + 32 * part, pages = 0, next = 0;
    const bool works = part < parts && p < z.p1;
    if (works) {
        pages = look(p);
        next = look(p + stride);
        if constexpr (D == 64) load(0, pages), load(1, pages);
    }
    const int G = a.Hq / a.Hkv;
    // the CTA's rows (head, token), two at a time; rows of no token stay what they are: no column of theirs is looked at
    for (int i = 2 * w; i < TOKENS * z.heads; i += 2 * (THREADS / 32)) {
        const int hh = i / TOKENS, k0 = i % TOKENS;
        if (k0 >= z.nt) continue;
        ask_of<D, 2, T>([&](int n) { return (const T *)a.q + (long long)(z.q0 + min(k0 + n, z.nt - 1)) * a.q_stride + (z.h0 + hh) * G * D; }, G,
                        [&](int n, int ch, const int *u, const int *d) {
                            uint8_t *const row = ask + (i + n) * ROW;
                            // channel ch of a record: 64-byte run ch / 64, lane's quarter ch / 16 % 4, half of it ch / 8 % 2
                            auto place = [&](int c) { return reinterpret_cast<__half2 *>(row + (((c >> 6) * 2 + (c >> 3 & 1)) * 4 + (c >> 4 & 3)) * 16 + (c & 7) * 2); };
#pragma unroll
                            for (int m = 0; m < D / 32; m += 2) {
                                *place(ch + m) = __floats2half2_rn((float)u[m], (float)u[m + 1]);
                                *place(D + ch + m) = __floats2half2_rn((float)d[m], (float)d[m + 1]);
                            }
                        });
    }
    __syncthreads();
    if (!works) return;
    if constexpr (D == 128) load(0, pages), load(1, pages);        // (registers are short before)
    const uint4 *const y = reinterpret_cast<const uint4 *>(ask + (h * TOKENS + r) * ROW) + c;
    uint32_t *const keys = a.keys + ((size_t)(z.q0 + 2 * c) * a.Hkv + z.h0 + h) * a.key_stride;      // of tokens 2 c and 2 c + 1
    const size_t row = (size_t)a.Hkv * a.key_stride;
    const bool has[2] = {2 * c < z.nt, 2 * c + 1 < z.nt};
    for (; p < z.p1; p += stride) {
        const int later = look(p + 2 * stride);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const uint4 y0 = y[8 * i], y1 = y[8 * i + 4];
                const uint32_t xa[4] = {x[s][0][i].x, x[s][0][i].y, x[s][0][i].z, x[s][0][i].w}, xb[4] = {x[s][1][i].x, x[s][1][i].y, x[s][1][i].z, x[s][1][i].w};
                const uint32_t b[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    uint32_t a0, a1, a2, a3;
                    s8x4_to_f16(xa[n], a0, a2);
                    s8x4_to_f16(xb[n], a1, a3);
                    mma_f16(d, a0, a1, a2, a3, b[2 * n], b[2 * n + 1]);
                }
            }
            const int e = unit[s];
            if (p + stride < z.p1) load(s, next);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int of = p + 16 * s + 8 * k + r, pe = __shfl_sync(~0u, e, 8 * k + r);
                const float per = power_of(pe);
                const bool plain = pe < UNBOUNDED, there = of < z.p1;
                const uint32_t other = key_of(0.f, pe);
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    if (has[n] && there) keys[n * row + of] = plain ? ordered(d[2 * k + n] * per) : other;
            }
        }
        next = later;
    }
}

// ---------------------------------------------------------------------------
// the best of a row's scores
// ---------------------------------------------------------------------------

// One row (token, kv head) is W warps' work, each with 32 K neighbouring pages in its lanes' registers (K = 0: read again at
// every step).  The count-th best key is found by narrowing an interval of keys: lo has at least as many pages at or above
// it as are wanted, hi fewer; it ends early once there are exactly as many.
template <int W, int K>
__global__ void __launch_bounds__(W == 1 ? THREADS : 32 * W) pick_kernel(const KvPickArgs a) {
    constexpr int ROWS = W == 1 ? THREADS / 32 : 1;
    __shared__ uint32_t box[2][32];
    wait_for_earlier_kernels();
    let_later_kernels_in();
    const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const unsigned row = blockIdx.x * (unsigned)ROWS + (W == 1 ? w : 0);
    const int t = (int)min(row / (unsigned)a.Hkv, (unsigned)a.T);
    const Owner own = owner_with(a.cu, a.kv_lens, a.B, a.T, t);
    if (own.b < 0) return;
    Tokens r{own.q0, own.end - own.q0, own.more};
    check(a, r, true);
    if (r.n == 0) return;
    int32_t *const out = a.picked + (size_t)row * a.count;
    const int pos = r.len - r.n + (t - r.q0), pages = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
    if (pages <= a.count) {
        for (unsigned i = tid; i < (unsigned)a.count; i += 32 * W) out[i] = i < (unsigned)pages ? (int)i : -1;     // (count may be 2^31 - 1)
        return;
    }
    const int want = a.count - a.first - a.recent, from = a.first, to = pages - a.recent;    // candidates from .. to - 1, more than want
    for (int i = tid; i < a.first; i += 32 * W) out[i] = i;
    for (int i = tid; i < a.recent; i += 32 * W) out[a.count - a.recent + i] = to + i;
    if (want == 0) return;
    const uint32_t *const keys = a.keys + (size_t)row * a.key_stride;
    const int span = K ? K : (a.max_pages + 32 * W - 1) / (32 * W);          // pages a lane, 32 apart
    const int p0 = (W == 1 ? 0 : w * 32 * span) + lane;
    uint32_t key[K ? K : 1];
    auto at = [&](int i) -> uint32_t {     // 0: no candidate
        const int p = p0 + 32 * i;
        return p >= from && p < to ? __ldcg(keys + p) : 0u;
    };
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) key[i] = at(i);
    }
    const int ours = to - (p0 - lane);     // pages of the warp's that there are
    auto each = [&](const auto &f) {       // f(number, key)
        if constexpr (K > 0) {
#pragma unroll
            for (int b = 0; b < K; b += 4) {
                if (32 * b >= ours) break;
#pragma unroll
                for (int i = b; i < b + 4; ++i) f(i, key[i]);
            }
        } else {
            for (int i = 0; i < span; ++i) f(i, at(i));
        }
    };
    int step = 0;
    // all threads' x, added up, or the largest
    auto total = [&](uint32_t x, bool largest) -> uint32_t {
        x = largest ? __reduce_max_sync(~0u, x) : __reduce_add_sync(~0u, x);
        if constexpr (W > 1) {
            if (lane == 0) box[step & 1][w] = x;
            __syncthreads();
            x = lane < W ? box[step & 1][lane] : 0u;
            x = largest ? __reduce_max_sync(~0u, x) : __reduce_add_sync(~0u, x);
            ++step;
        }
        return x;
    };
    uint32_t high = 0, low = 0;            // low: of the keys' complements
    each([&](int, uint32_t k) { high = max(high, k), low = max(low, k ? ~k : 0u); });
    uint32_t lo = ~total(low, true), hi = total(high, true) + 1, have = (uint32_t)(to - from), fewer = 0;
    for (bool even = true; hi - lo > 1 && have != (uint32_t)want; even = !even) {
        // in turn where the counts at both ends would have it, and in the middle, so that it ends soon on any keys
        const float part = even ? __fdividef((float)(have - want), (float)(have - fewer)) : 0.5f;
        const uint32_t mid = lo + min(max((uint32_t)((float)(hi - lo) * part), 1u), hi - lo - 1);
        uint32_t n = 0;
        each([&](int, uint32_t k) { n += k >= mid; });
        n = total(n, false);
        if (n >= (uint32_t)want) lo = mid, have = n;
        else hi = mid, fewer = n;
    }
    // those above lo, and of those at lo the first `extra`
    const uint32_t extra = have == (uint32_t)want ? have : (uint32_t)want - fewer;
    uint32_t put = a.first, tied = 0;      // in the warps before
    if constexpr (W > 1) {
        uint32_t sure = 0, ties = 0;
        each([&](int, uint32_t k) { sure += k > lo, ties += k == lo; });
        auto before = [&](uint32_t x) -> uint32_t {
            x = __reduce_add_sync(~0u, x);
            if (lane == 0) box[step & 1][w] = x;
            __syncthreads();
            x = __reduce_add_sync(~0u, lane < w ? box[step & 1][lane] : 0u);
            ++step;
            return x;
        };
        sure = before(sure), ties = before(ties);
        tied = ties;
        put += sure + min(extra, ties);
    }
    const uint32_t below = (1u << lane) - 1;
    each([&](int i, uint32_t k) {
        const uint32_t at_lo = __ballot_sync(~0u, k == lo);
        const bool take = k > lo || (k == lo && tied + __popc(at_lo & below) < extra);
        const uint32_t taken = __ballot_sync(~0u, take);
        if (take) out[put + __popc(taken & below)] = p0 + 32 * i;
        put += __popc(taken), tied += __popc(at_lo);
    });
}

template <int W, int K>
cudaError_t pick_rows(const KvPickArgs &a, cudaStream_t s) {
    const long long rows = (long long)a.T * a.Hkv, per = W == 1 ? THREADS / 32 : 1;
    const dim3 grid((unsigned)((rows + per - 1) / per)), block(W == 1 ? THREADS : 32 * W);
    return launch_early(pick_kernel<W, K>, grid, block, 0, s, a);
}

template <int D, typename T>
cudaError_t score(KvPickArgs a, cudaStream_t s) {
    const int tokens = a.max_q == 1 ? 1 : TOKENS, heads = tokens == 1 ? HEADS_1 : HEADS, groups = (a.Hkv + heads - 1) / heads;
    a.blocks = (a.max_q + tokens - 1) / tokens;
    const long long units = (long long)a.B * a.blocks * groups;
    // One run of pages a CTA, unless that were more than some dozens an SM (with tables far wider than their rows most have
    // nothing); several tokens: a few CTAs an SM, as each adds up its queries.  Picks by CTAs an SM, us: 384 single tokens on 1000
    // pages 114 (4), 105 (16), 111 (32), 130 (128), on 200 pages 31, 34, 36, 36; 64 x 16 tokens on 1000 98 (1 to 4), 109 (16);
    // 2 x 800 on 384 70 (1 to 8), 84 (16).  CTAs of tokens that a request does not have find out and leave: 255 single tokens
    // and a piece of 2048 in one call take 422 us, 26 and 95 in two.
    const int run = 32 * ((THREADS / 32) / min(heads, a.Hkv));
    a.chunks = (int)max(1LL, min(SMS * (tokens == 1 ? 32LL : 4LL) / units, ((long long)a.max_pages + run - 1) / run));
    const dim3 grid((unsigned)(a.B * a.blocks), (unsigned)a.chunks, (unsigned)groups);     // (what the call takes fits)
    if (tokens == 1) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_shared(reinterpret_cast<const void *>(score_one_kernel<D, T>), OneShape<D>::SMEM, done);
        if (e != cudaSuccess) return e;
        return launch_early(score_one_kernel<D, T>, grid, dim3(THREADS), OneShape<D>::SMEM, s, a);
    }
    return launch_early(score_kernel<D, T>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace

cudaError_t launch_kv4_bounds(KvBoundsArgs a, cudaStream_t s) {
    // single tokens and drafts begin a page each or nearly; of prompts one token in a page does
    a.slice = a.T >= 16LL * a.B ? 16 : 1;
    const long long units = ((long long)a.T + a.slice - 1) / a.slice * a.H;
    const unsigned grid = (unsigned)((units + THREADS / 32 - 1) / (THREADS / 32));
    return launch_early(a.D == 128 ? bounds_kernel<128> : bounds_kernel<64>, dim3(grid), dim3(THREADS), 0, s, a);
}

cudaError_t launch_kv4_pick(const KvPickArgs &a, cudaStream_t s) {
    if (a.max_pages > a.count) {           // (else every row takes all that it sees)
        cudaError_t e;
        if (a.dt == KDA_DTYPE_BF16) e = a.D == 128 ? score<128, __nv_bfloat16>(a, s) : score<64, __nv_bfloat16>(a, s);
        else e = a.D == 128 ? score<128, __half>(a, s) : score<64, __half>(a, s);
        if (e != cudaSuccess) return e;
    }
    // A warp a row where its lanes hold the candidates (pages before the last `recent`) and rows fill the GPU, else a CTA with
    // the fewest keys a lane.  Picks by both forms, us, a warp and a CTA: 12288 rows of 250 pages 59 and 78, of 500 78 and 99, of
    // 1000 124 and 170; 7168 rows of single tokens 93 and 103, 137 and 149, 232 and 257; 3584 42 and 45, 66 and 69, 112 and 124
    // (already ahead, as it is from about 1800 on); 128 8.0 and 8.6, 11.5 and 10.6, 15.4 and 13.2.  1900 pages with 8 warps
    // 8.4 (8 rows) and 402 (7168), with 32 10 and 512.
    const bool many = (long long)a.T * a.Hkv >= SMS * 24;
    const int width = a.max_pages - a.recent;
    if (many && width <= 256) return pick_rows<1, 8>(a, s);
    if (many && width <= 512) return pick_rows<1, 16>(a, s);
    if (many && width <= 1024) return pick_rows<1, 32>(a, s);
    if (width <= 512) return pick_rows<4, 4>(a, s);
    if (width <= 2048) return pick_rows<8, 8>(a, s);
    if (width <= 8192) return pick_rows<32, 8>(a, s);
    if (width <= 32768) return pick_rows<32, 32>(a, s);
    return pick_rows<32, 0>(a, s);
}

}  // namespace kda
