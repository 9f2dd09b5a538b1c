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
#include "kda_internal.h"
#include "kda_kv4.cuh"

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

// One page of one head: fill tokens (>= 1) of its tiles.
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
    const int lane = threadIdx.x & 31;
    const unsigned unit = blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
    const int h = (int)(unit % (unsigned)a.H);
    const long long t0 = (long long)(unit / (unsigned)a.H) * a.slice;
    if (t0 >= a.T) return;
    const int t = (int)min(t0 + min(lane, a.slice - 1), (long long)a.T);
    const int b = owner_of(a.cu, a.B, t);
    int page = -1, fill = 0;
    if (lane < a.slice && t < a.T) {
        if (b < 0) {
            report(a.err, DEVERR_SEQLENS);
        } else {
            const int i = t - a.cu[b], P = 1 << a.page_shift;
            const long long pos = (long long)a.start[b] + i, end = (long long)a.start[b] + (a.cu[b + 1] - a.cu[b]);
            if (pos < 0 || (pos >> a.page_shift) >= a.max_pages) {
                report(a.err, DEVERR_SEQLENS);
            } else if (i == 0 || (pos & (P - 1)) == 0) {
                page = a.page_table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
                if (page < 0 || page >= a.num_pages) {
                    report(a.err, DEVERR_PAGE_RANGE);
                    page = -1;
                }
                fill = (int)min((long long)P, end - (pos & ~(long long)(P - 1)));
            }
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

constexpr int HEADS = 8;       // kv heads that a CTA takes

// The bits of a finite or infinite float as a number that orders as it does.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// What request b has of new tokens and cache; n = 0 where it is malformed.
struct Tokens {
    int q0, n, len;
};
__device__ __forceinline__ Tokens tokens_of(const KvPickArgs &a, int b, bool tell) {
    Tokens r;
    r.q0 = a.cu[b];
    r.n = a.cu[b + 1] - r.q0;
    r.len = a.kv_lens[b];
    if (r.q0 < 0 || r.n < 0 || r.n > a.max_q || (long long)r.q0 + r.n > a.T || r.len < 0 ||
        (long long)r.len > ((long long)a.max_pages << a.page_shift)) {
        if (tell) report(a.err, DEVERR_SEQLENS);
        r.n = 0;
    }
    return r;
}

template <typename T> __device__ __forceinline__ float2 halves(uint32_t w);
template <> __device__ __forceinline__ float2 halves<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 halves<__half>(uint32_t w) { return f16x2_to_float2(w); }

// u and -d of one token and kv head, as 2 D bytes laid out as a record is; a warp's work.
template <int D, typename T>
__device__ __forceinline__ void ask_of(const T *q, int G, int8_t *out) {
    constexpr int W = D / 64;              // words of the lane: 2 W channels
    const int lane = threadIdx.x & 31;
    float up[2 * W], down[2 * W];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) up[i] = down[i] = 0.f;
#pragma unroll 8
    for (int g = 0; g < G; ++g) {
        uint32_t w[W];
        if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(q + g * D + lane * 4);
            w[0] = x.x, w[W - 1] = x.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(q + g * D + lane * 2);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 f = halves<T>(w[i]);
            up[2 * i] = __fadd_rn(up[2 * i], max_nan(f.x, 0.f)), down[2 * i] = __fadd_rn(down[2 * i], max_nan(-f.x, 0.f));
            up[2 * i + 1] = __fadd_rn(up[2 * i + 1], max_nan(f.y, 0.f)), down[2 * i + 1] = __fadd_rn(down[2 * i + 1], max_nan(-f.y, 0.f));
        }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) top = max_nan(top, max_nan(up[i], down[i]));
    const uint32_t bits = __reduce_max_sync(~0u, __float_as_uint(top) & 0x7fffffffu);       // (a NaN is above all)
    // nothing to go by: all pages score 0
    const float per = bits >= 0x7f800000u || bits < 0x00800000u ? 0.f : power_of(-max(unit_of(__uint_as_float(bits)), -100));
    uint32_t u = 0, d = 0;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
        const int x = per == 0.f ? 0 : __float2int_rn(up[i] * per), y = per == 0.f ? 0 : -__float2int_rn(down[i] * per);
        u |= ((uint32_t)x & 255u) << (8 * i), d |= ((uint32_t)y & 255u) << (8 * i);
    }
    if constexpr (W == 2) {
        *reinterpret_cast<uint32_t *>(out + lane * 4) = u;
        *reinterpret_cast<uint32_t *>(out + D + lane * 4) = d;
    } else {
        *reinterpret_cast<uint16_t *>(out + lane * 2) = (uint16_t)u;
        *reinterpret_cast<uint16_t *>(out + D + lane * 2) = (uint16_t)d;
    }
}

// Scores of up to NT tokens of one request with a run of its pages, for up to HEADS kv heads.  A record is held by eight
// lanes, 16 or 32 bytes each, so that its loads are whole lines; four pages a warp at a time.
template <int D, int NT, typename T>
__global__ void __launch_bounds__(THREADS) score_kernel(const KvPickArgs a) {
    constexpr int RECORD = 2 * D + 16, LOADS = D / 64;
    __shared__ __align__(16) int8_t ask[NT * HEADS * 2 * D];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane & 7, four = lane >> 3;
    const int groups = (a.Hkv + HEADS - 1) / HEADS, G = a.Hq / a.Hkv;
    unsigned at = blockIdx.x;
    const int chunk = (int)(at % (unsigned)a.chunks);
    at /= (unsigned)a.chunks;
    const int h0 = (int)(at % (unsigned)groups) * HEADS, heads = min(HEADS, a.Hkv - h0);
    at /= (unsigned)groups;
    const int b = (int)(at / (unsigned)a.blocks), i0 = (int)(at % (unsigned)a.blocks) * NT;
    const Tokens r = tokens_of(a, b, false);
    if (i0 >= r.n) return;
    const int nt = min(NT, r.n - i0), last = r.len - r.n + i0 + nt - 1;      // the last token's position
    const int pages = last < 0 ? 0 : (last >> a.page_shift) + 1;
    if (pages <= a.count) return;          // all of them are taken
    const int per = ((pages + a.chunks - 1) / a.chunks + 31) & ~31, p0 = chunk * per, p1 = min(pages, p0 + per);
    if (p0 >= p1) return;
    for (int x = w; x < nt * heads; x += THREADS / 32) {
        const int k = x / heads, h = x % heads;
        ask_of<D, T>((const T *)a.q + (long long)(r.q0 + i0 + k) * a.q_stride + (h0 + h) * G * D, G, ask + (k * HEADS + h) * 2 * D);
    }
    __syncthreads();
    // the warps are dealt over the heads, and those of a head over the runs of 32 pages
    const int parts = (THREADS / 32) / heads, h = w % heads, part = w / heads;
    if (part >= parts) return;
    for (int p = p0 + 32 * part; p < p1; p += 32 * parts) {
        int page = p + lane < p1 ? a.page_table[(size_t)b * a.max_pages + p + lane] : 0;
        if (page < 0 || page >= a.num_pages) {
            report(a.err, DEVERR_PAGE_RANGE);
            page = -1;
        }
        uint32_t mine = 0;                 // NT == 1: the key of page p + lane
#pragma unroll 2
        for (int step = 0; step < 8; ++step) {
            // pages 8 four + step: the lane that has the step's number keeps the result
            const int local = 8 * four + step, pg = __shfl_sync(~0u, page, local);
            const bool good = p + local < p1 && pg >= 0;
            const int8_t *rec = a.bounds + ((size_t)max(pg, 0) * a.Hkv + h0 + h) * RECORD;
            uint4 x[LOADS];
            int e = 0;
#pragma unroll
            for (int k = 0; k < LOADS; ++k) x[k] = good ? __ldg(reinterpret_cast<const uint4 *>(rec) + j + 8 * k) : make_uint4(0, 0, 0, 0);
            if (good) e = __ldg(rec + 2 * D);
            int sum[NT];
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                sum[k] = 0;
                if (k < nt) {
                    const uint4 *y = reinterpret_cast<const uint4 *>(ask + (k * HEADS + h) * 2 * D);
#pragma unroll
                    for (int z = 0; z < LOADS; ++z) {
                        const uint4 v = y[j + 8 * z];
                        sum[k] = __dp4a((int)x[z].x, (int)v.x, sum[k]);
                        sum[k] = __dp4a((int)x[z].y, (int)v.y, sum[k]);
                        sum[k] = __dp4a((int)x[z].z, (int)v.z, sum[k]);
                        sum[k] = __dp4a((int)x[z].w, (int)v.w, sum[k]);
                    }
                }
            }
            auto key_of = [&](int s) {     // 1: below every score (a page that is not there); 0 is no page
                return !good ? 1u : e == UNBOUNDED ? 0xff800000u : ordered((float)s * power_of(e));
            };
            if constexpr (NT == 1) {
                int s = sum[0];
                s += __shfl_xor_sync(~0u, s, 1);
                s += __shfl_xor_sync(~0u, s, 2);
                s += __shfl_xor_sync(~0u, s, 4);
                if (j == step) mine = key_of(s);
            } else {
                // lane j is left with token j's sum
                static_assert(NT == 8, "one token a lane");
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool u = j & 4;
                    const int give = u ? sum[k] : sum[k + 4], keep = u ? sum[k + 4] : sum[k];
                    sum[k] = keep + __shfl_xor_sync(~0u, give, 4);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool u = j & 2;
                    const int give = u ? sum[k] : sum[k + 2], keep = u ? sum[k + 2] : sum[k];
                    sum[k] = keep + __shfl_xor_sync(~0u, give, 2);
                }
                const bool u = j & 1;
                const int give = u ? sum[0] : sum[1], keep = u ? sum[1] : sum[0];
                const int s = keep + __shfl_xor_sync(~0u, give, 1);
                if (j < nt && p + local < p1)
                    a.keys[((size_t)(r.q0 + i0 + j) * a.Hkv + h0 + h) * a.key_stride + p + local] = key_of(s);
            }
        }
        if constexpr (NT == 1)
            if (p + lane < p1) a.keys[((size_t)(r.q0 + i0) * a.Hkv + h0 + h) * a.key_stride + p + lane] = mine;
    }
}

// ---------------------------------------------------------------------------
// the best of a row's scores
// ---------------------------------------------------------------------------

// One row (token, kv head) is W warps' work, each thread's K neighbouring pages in registers (K = 0: read again at every
// step).  The count-th best key is found by halving an interval of keys: lo has at least as many pages at or above it as
// are wanted, hi fewer; it ends early once there are exactly as many.
template <int W, int K>
__global__ void __launch_bounds__(W == 1 ? THREADS : 32 * W) pick_kernel(const KvPickArgs a) {
    constexpr int ROWS = W == 1 ? THREADS / 32 : 1;
    __shared__ uint32_t box[2][32];
    const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const unsigned row = blockIdx.x * (unsigned)ROWS + (W == 1 ? w : 0);
    if (row >= (unsigned)a.T * (unsigned)a.Hkv) return;
    const int t = (int)(row / (unsigned)a.Hkv);
    const int b = owner_of(a.cu, a.B, t);
    if (b < 0) return;
    const Tokens r = tokens_of(a, b, true);
    if (r.n == 0) return;
    int32_t *const out = a.picked + (size_t)row * a.count;
    const int pos = r.len - r.n + (t - r.q0), pages = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
    if (pages <= a.count) {
        for (int i = tid; i < a.count; i += 32 * W) out[i] = i < pages ? i : -1;
        return;
    }
    const int want = a.count - a.first - a.recent, from = a.first, to = pages - a.recent;    // candidates from .. to - 1, more than want
    for (int i = tid; i < a.first; i += 32 * W) out[i] = i;
    for (int i = tid; i < a.recent; i += 32 * W) out[a.count - a.recent + i] = to + i;
    if (want == 0) return;
    const uint32_t *const keys = a.keys + (size_t)row * a.key_stride;
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
    const int span = K ? K : (a.max_pages + 32 * W - 1) / (32 * W);          // pages a thread
    const int i0 = tid * span;
    uint32_t key[K ? K : 1];
    auto at = [&](int i) -> uint32_t {     // 0: no candidate
        const int p = i0 + i;
        return p >= from && p < to ? __ldcg(keys + p) : 0u;
    };
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) key[i] = at(i);
    }
    auto get = [&](int i) -> uint32_t {
        if constexpr (K > 0) return key[i];
        else return at(i);
    };
    auto above = [&](uint32_t x) -> uint32_t {       // candidates with a key of x or more
        uint32_t n = 0;
        if constexpr (K > 0) {
#pragma unroll
            for (int i = 0; i < K; ++i) n += key[i] >= x;
        } else {
            for (int i = 0; i < span; ++i) n += at(i) >= x;
        }
        return total(n, false);
    };
    uint32_t high = 0, low = 0;            // low: of the keys' complements
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) high = max(high, key[i]), low = max(low, key[i] ? ~key[i] : 0u);
    } else {
        for (int i = 0; i < span; ++i) {
            const uint32_t k = at(i);
            high = max(high, k), low = max(low, k ? ~k : 0u);
        }
    }
    uint32_t lo = ~total(low, true), hi = total(high, true) + 1, have = (uint32_t)(to - from);
    while (hi - lo > 1 && have != (uint32_t)want) {
        const uint32_t mid = lo + (hi - lo) / 2, n = above(mid);
        if (n >= (uint32_t)want) lo = mid, have = n;
        else hi = mid;
    }
    // those above lo, and of those at lo the first that are still wanted
    const uint32_t extra = have == (uint32_t)want ? 0u : (uint32_t)want - above(hi);
    const bool exact = have == (uint32_t)want;
    uint32_t sure = 0, ties = 0;
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) sure += exact ? key[i] >= lo : key[i] > lo, ties += !exact && key[i] == lo;
    } else {
        for (int i = 0; i < span; ++i) {
            const uint32_t k = at(i);
            sure += exact ? k >= lo : k > lo, ties += !exact && k == lo;
        }
    }
    // what the threads before have
    auto before = [&](uint32_t x) -> uint32_t {
        uint32_t in = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, in, o);
            if (lane >= o) in += y;
        }
        uint32_t base = 0;
        if constexpr (W > 1) {
            if (lane == 31) box[step & 1][w] = in;
            __syncthreads();
            const uint32_t y = lane < w ? box[step & 1][lane] : 0u;
            base = __reduce_add_sync(~0u, y);
            ++step;
        }
        return base + in - x;
    };
    uint32_t tied = before(ties);
    const uint32_t taken = min(extra, tied + ties) - min(extra, tied);
    uint32_t put = before(sure + taken) + a.first;
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const uint32_t k = key[i];
            const bool tie = !exact && k == lo;
            if ((exact ? k >= lo : k > lo) || (tie && tied < extra)) out[put++] = i0 + i;
            tied += tie;
        }
    } else {
        for (int i = 0; i < span; ++i) {
            const uint32_t k = get(i);
            const bool tie = !exact && k == lo;
            if ((exact ? k >= lo : k > lo) || (tie && tied < extra)) out[put++] = i0 + i;
            tied += tie;
        }
    }
}

template <int W, int K>
cudaError_t pick_rows(const KvPickArgs &a, cudaStream_t s) {
    const long long rows = (long long)a.T * a.Hkv, per = W == 1 ? THREADS / 32 : 1;
    pick_kernel<W, K><<<(unsigned)((rows + per - 1) / per), W == 1 ? THREADS : 32 * W, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D, typename T>
cudaError_t score(KvPickArgs a, cudaStream_t s) {
    const int nt = a.max_q == 1 ? 1 : 8, groups = (a.Hkv + HEADS - 1) / HEADS;
    a.blocks = (a.max_q + nt - 1) / nt;
    const long long units = (long long)a.B * a.blocks * groups;
    a.chunks = (int)max(1LL, min((SMS * 4LL + units - 1) / units, (a.max_pages + 31LL) / 32));
    if (units * a.chunks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (nt == 1) score_kernel<D, 1, T><<<(unsigned)(units * a.chunks), THREADS, 0, s>>>(a);
    else score_kernel<D, 8, T><<<(unsigned)(units * a.chunks), THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_bounds(KvBoundsArgs a, cudaStream_t s) {
    // single tokens and drafts begin a page each or nearly; of prompts one token in a page does
    a.slice = a.T >= 16LL * a.B ? 16 : 1;
    const long long units = ((long long)a.T + a.slice - 1) / a.slice * a.H;
    const unsigned grid = (unsigned)((units + THREADS / 32 - 1) / (THREADS / 32));
    if (a.D == 128) bounds_kernel<128><<<grid, THREADS, 0, s>>>(a);
    else bounds_kernel<64><<<grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv4_pick(const KvPickArgs &a, cudaStream_t s) {
    if (a.max_pages > a.count) {           // (else every row takes all that it sees)
        cudaError_t e;
        if (a.dt == KDA_DTYPE_BF16) e = a.D == 128 ? score<128, __nv_bfloat16>(a, s) : score<64, __nv_bfloat16>(a, s);
        else e = a.D == 128 ? score<128, __half>(a, s) : score<64, __half>(a, s);
        if (e != cudaSuccess) return e;
    }
    if (a.max_pages <= 256) return pick_rows<1, 8>(a, s);
    if (a.max_pages <= 1024) return pick_rows<1, 32>(a, s);
    if (a.max_pages <= 2048) return pick_rows<8, 8>(a, s);
    if (a.max_pages <= 8192) return pick_rows<8, 32>(a, s);
    if (a.max_pages <= 32768) return pick_rows<32, 32>(a, s);
    return pick_rows<32, 0>(a, s);
}

}  // namespace kda
