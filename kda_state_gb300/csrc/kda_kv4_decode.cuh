// Attention over the 4-bit cache for few query rows: single tokens, drafts.
//
// The cache is read once and its bytes bound the work, so tokens stand on the
// 16 rows of an MMA and query rows on its 8 columns (no padding up to 8 rows of
// a kv head):  S^T = K Q^T,  O^T = V^T P^T.  Both A operands are made in
// registers from the codes as they lie in the tile: an MMA's contraction index
// may be permuted freely if both operands agree, so a lane's share of a K row is
// 16 neighbouring bytes, and of V the 8 bytes of one scale block for each of 4
// neighbouring tokens.  V's fragments pair two tokens: their nibbles are
// interleaved before the conversion, four logic operations for 16 values.
//
// A code becomes fp16 by one conversion and one product with its scale, exactly
// (6 significant bits).  A query row is scaled by a power of two so that its
// largest value is in [1, 2): exact to 2^-25 of it in fp16 whatever its type's
// range.  Weights are rounded to fp16 (2^-11 of a weight, against 2^-9 and more
// of bf16), and held 2^9 above the running maximum, which moves only when a
// score passes it by 2^6: a weight is a normal fp16 number down to 2^-23 of the
// largest, and most steps rescale nothing.
//
// Work is the list of all (request, block of rows, kv head, 32 tokens), cut into
// equal contiguous ranges, one a CTA: a ragged batch and one long request are
// balanced alike.  A range that ends inside a (request, rows, head) leaves a
// partial result; the last of its CTAs to arrive joins them in order, so results
// do not depend on timing.
//
// Each warp takes every eighth 32 tokens of its CTA's range through a ring of its
// own, filled by bulk copies (one contiguous block of 18 D bytes for 16 tokens).
#pragma once

#include "kda_async.cuh"
#include "kda_internal.h"
#include "kda_kv4.cuh"

namespace kda {
namespace kv4 {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int CHUNK = 32;              // tokens of one step of a warp
constexpr int MAX_CTAS = 152 * 2;
constexpr float HEADROOM = 9.f;        // log2 of a weight at the running maximum
constexpr float MOVE = HEADROOM + 6.f; // a score this far above m makes the maximum move
constexpr float NOTHING = -1e30f;      // the running maximum before any score

template <int D, int NT>
struct DecodeShape {
    static constexpr int ROWS = 8 * NT;
    static constexpr int STAGES = 2;
    static constexpr int STAGE_BYTES = 2 * KvTile<D>::BYTES;
    static constexpr int OSTRIDE = D + 4;
    static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
    static constexpr int OUT = WARPS * ROWS * OSTRIDE * 4;
    static constexpr int SMEM = RING + OUT + WARPS * ROWS * 8 + WARPS * STAGES * 8 + 64;
    static constexpr int PARTIAL = ROWS * (D + 2);         // floats
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair_of<__half>(uint32_t w) {
    return f16x2_to_float2(w);
}
template <typename T>
__device__ __forceinline__ uint32_t pack_of(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_of<__nv_bfloat16>(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_of<__half>(float a, float b) {
    return half_pair(a, b);
}

// What one request asks for; chunks = 0 where it asks for nothing or is malformed.
struct Request {
    int q0, n, len, first_chunk, chunks, row_blocks;
};
__device__ __forceinline__ Request request_of(const KvAttentionArgs &a, int b, int rows, bool tell) {
    Request r;
    r.q0 = a.cu[b];
    r.n = a.cu[b + 1] - r.q0;
    r.len = a.kv_lens[b];
    r.first_chunk = r.chunks = r.row_blocks = 0;
    if (r.q0 < 0 || r.n < 0 || r.n > a.max_q || (long long)r.q0 + r.n > a.T || r.len < 0 ||
        (long long)r.len > ((long long)a.max_pages << a.page_shift)) {
        if (tell) report(a.err, DEVERR_SEQLENS);
        r.n = 0;
        return r;
    }
    if (r.n == 0) return r;
    const int first = a.window > 0 ? max(0, min(r.len, r.len - r.n + 1) - a.window) : 0;
    r.first_chunk = first / CHUNK;
    r.chunks = max(1, (r.len + CHUNK - 1) / CHUNK - r.first_chunk);
    r.row_blocks = (r.n * (a.Hq / a.Hkv) + rows - 1) / rows;
    return r;
}

template <int D, int NT, typename T>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 2 : 1) decode_attention_kernel(const KvAttentionArgs a) {
    using L = KvTile<D>;
    using S = DecodeShape<D, NT>;
    constexpr int KS = D / 16;             // MMA steps of a score; also V's tiles of 16 channels
    constexpr int LW = D / 32;             // 32-bit words of a lane's share of a K row
    extern __shared__ __align__(128) uint8_t smem[];
    float *const out_s = reinterpret_cast<float *>(smem + S::RING);                  // [WARPS][ROWS][OSTRIDE]
    float2 *const ml_s = reinterpret_cast<float2 *>(smem + S::RING + S::OUT);        // [WARPS][ROWS]
    uint8_t *const bars = smem + S::RING + S::OUT + WARPS * S::ROWS * 8;
    int *const shared = reinterpret_cast<int *>(bars + WARPS * S::STAGES * 8);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int G = a.Hq / a.Hkv;

    // ---- the work's total and this CTA's range -------------------------------------------------
    long long begin, end, per, base;       // base: where request b's work begins
    int b;
    {
        __shared__ long long scan_s[WARPS + 1];
        __shared__ long long found_s[2];
        const int share = (a.B + THREADS - 1) / THREADS;
        long long mine = 0;
        for (int i = 0; i < share; ++i) {
            const int bb = tid * share + i;
            if (bb >= a.B) break;
            const Request q = request_of(a, bb, S::ROWS, blockIdx.x == 0);
            mine += (long long)q.chunks * q.row_blocks * a.Hkv;
        }
        long long in = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, in, o);
            if (lane >= o) in += y;
        }
        if (lane == 31) scan_s[w] = in;
        if (lane == 0) {
#pragma unroll
            for (int s = 0; s < S::STAGES; ++s) barrier_init(shared_addr(bars + (w * S::STAGES + s) * 8), 1);
        }
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            if (i < w) before += scan_s[i];
            total += scan_s[i];
        }
        before += in - mine;
        per = max((total + gridDim.x - 1) / gridDim.x, (long long)WARPS);
        begin = blockIdx.x * per;
        end = min(begin + per, total);
        if (begin >= total) return;
        if (begin >= before && begin < before + mine) {
            for (int i = 0; i < share; ++i) {
                const int bb = tid * share + i;
                const Request q = request_of(a, bb, S::ROWS, false);
                const long long here = (long long)q.chunks * q.row_blocks * a.Hkv;
                if (begin < before + here) {
                    found_s[0] = bb;
                    found_s[1] = before;
                    break;
                }
                before += here;
            }
        }
        __syncthreads();
        b = (int)found_s[0];
        base = found_s[1];
    }

    uint8_t *const ring = smem + w * S::STAGES * S::STAGE_BYTES;
    const uint32_t bar0 = shared_addr(bars + w * S::STAGES * 8);
    uint32_t phases = 0;                   // the parity that each stage waits for next
    bool dead = false;                     // a wait gave up: nothing more is read
    const int tA = 4 * (r >> 1) + (r & 1), tB = tA + 2;    // the tokens of this lane's MMA rows r and r + 8

    Request rq = request_of(a, b, S::ROWS, false);
    long long at = begin;
    while (at < end) {
        // ---- the next (request, rows, head) of the range ---------------------------------------
        while (at >= base + (long long)rq.chunks * rq.row_blocks * a.Hkv) {
            base += (long long)rq.chunks * rq.row_blocks * a.Hkv;
            rq = request_of(a, ++b, S::ROWS, false);
        }
        const int unit = (int)((at - base) / rq.chunks);
        const long long unit_begin = base + (long long)unit * rq.chunks, unit_end = unit_begin + rq.chunks;
        const int h = unit % a.Hkv, row0 = unit / a.Hkv * S::ROWS, rows = min(S::ROWS, rq.n * G - row0);
        const int c0 = rq.first_chunk + (int)(at - unit_begin);
        const int c1 = rq.first_chunk + (int)(min(end, unit_end) - unit_begin);
        const int32_t *const pages = a.page_table + (size_t)b * a.max_pages;

        // ---- queries, as B fragments, and what their rows see -----------------------------------
        uint32_t qf[NT][2 * KS];
        float factor[NT][2];
        int last[NT][2];
        int last_min, first_max;
        {
            const int i0 = row0 / G, i1 = (row0 + rows - 1) / G;
            last_min = rq.len - rq.n + i0;
            first_max = a.window > 0 ? rq.len - rq.n + i1 + 1 - a.window : 0;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = row0 + t * 8 + r;
            float top = 0.f, x[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
            if (t * 8 + r < rows) {
                const uint4 *src = reinterpret_cast<const uint4 *>((const T *)a.q + (long long)(rq.q0 + row / G) * a.q_stride +
                                                                   (h * G + row % G) * D + c * (D / 4));
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 v = __ldg(src + i);
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = pair_of<T>(u[k]);
                        x[8 * i + 2 * k] = f.x;
                        x[8 * i + 2 * k + 1] = f.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 4; ++i) top = max_nan(top, fabsf(x[i]));
            }
            top = max_nan(top, __shfl_xor_sync(~0u, top, 1));
            top = max_nan(top, __shfl_xor_sync(~0u, top, 2));
            const int e = min(max((int)(__float_as_uint(top) >> 23 & 255), 1), 253);
            const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) qf[t][i] = half_pair(x[2 * i] * down, x[2 * i + 1] * down);
            // scores come back by columns: this lane holds those of rows 2 c and 2 c + 1
            const float f = a.scale_k * up;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                factor[t][k] = __shfl_sync(~0u, f, (2 * c + k) * 4);
                const int col = t * 8 + 2 * c + k;
                last[t][k] = col < rows ? rq.len - rq.n + (row0 + col) / G : -1;
            }
        }

        float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < KS; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
            m[t][0] = m[t][1] = NOTHING;
            l[t][0] = l[t][1] = 0.f;
        }

        // ---- this warp's chunks: c0 + w, c0 + w + WARPS, ... ------------------------------------
        const int count = c1 - c0 > w ? (c1 - c0 - w + WARPS - 1) / WARPS : 0;
        int page0 = -1, page1 = -1;        // pages of the two tiles of chunk (32-fold part) + lane
        uint32_t here = 0;                 // two bits a stage: which tiles of it were loaded
        auto fetch = [&](int k) {
            if ((k & 31) == 0) {
                const int kk = k + lane, t0 = (c0 + w + kk * WARPS) * CHUNK, t1 = t0 + KV_TILE;
                page0 = kk < count && t0 < rq.len ? pages[t0 >> a.page_shift] : -2;
                page1 = kk < count && t1 < rq.len ? pages[t1 >> a.page_shift] : -2;
                if ((page0 != -2 && (page0 < 0 || page0 >= a.num_pages)) ||
                    (page1 != -2 && (page1 < 0 || page1 >= a.num_pages)))
                    report(a.err, DEVERR_PAGE_RANGE);
            }
            const int s = k % S::STAGES;
            const int p0 = __shfl_sync(~0u, page0, k & 31), p1 = __shfl_sync(~0u, page1, k & 31);
            const bool ok0 = p0 >= 0 && p0 < a.num_pages, ok1 = p1 >= 0 && p1 < a.num_pages;
            here = (here & ~(3u << (2 * s))) | ((ok0 ? 1u : 0u) | (ok1 ? 2u : 0u)) << (2 * s);
            if (lane == 0) {
                const int t0 = (c0 + w + k * WARPS) * CHUNK, in_page = t0 & ((1 << a.page_shift) - 1);
                const uint32_t bar = bar0 + 8 * s;
                uint8_t *dst = ring + s * S::STAGE_BYTES;
                const uint8_t *src0 = a.pool + ((((size_t)p0 * a.Hkv + h) << (a.page_shift - 4)) + (in_page >> 4)) * L::BYTES;
                barrier_expect(bar, (ok0 ? L::BYTES : 0) + (ok1 ? L::BYTES : 0));
                if (ok0 && ok1 && p0 == p1 && a.page_shift > 4) {
                    bulk_copy(dst, src0, 2 * L::BYTES, bar);
                } else {
                    if (ok0) bulk_copy(dst, src0, L::BYTES, bar);
                    if (ok1) {
                        const int in1 = (t0 + KV_TILE) & ((1 << a.page_shift) - 1);
                        bulk_copy(dst + L::BYTES,
                                  a.pool + ((((size_t)p1 * a.Hkv + h) << (a.page_shift - 4)) + (in1 >> 4)) * L::BYTES,
                                  L::BYTES, bar);
                    }
                }
            }
        };
        if (!dead) {
#pragma unroll
            for (int s = 0; s < S::STAGES; ++s)
                if (s < count) fetch(s);
        }

        for (int k = 0; k < count && !dead; ++k) {
            const int s = k % S::STAGES, t0 = (c0 + w + k * WARPS) * CHUNK;
            if (!__all_sync(~0u, barrier_test(bar0 + 8 * s, phases >> s & 1) || barrier_wait(bar0 + 8 * s, phases >> s & 1))) {
                barrier_wait(bar0 + 8 * (1 - s), phases >> (1 - s) & 1);
                if (lane == 0) report(a.err, DEVERR_TIMEOUT);
                dead = true;
                break;
            }
            phases ^= 1u << s;
            const uint8_t *stage = ring + s * S::STAGE_BYTES;
            const uint32_t loaded = here >> (2 * s) & 3u;
            const bool whole = loaded == 3u && t0 >= first_max && t0 + CHUNK - 1 <= last_min;

            // scores of 32 tokens
            float y[2][NT][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *tile = stage + i * L::BYTES;
                uint32_t ka[LW], kb[LW], sa[2], sb[2];
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(tile + tA * 64 + c * 16);
                    const uint4 z = *reinterpret_cast<const uint4 *>(tile + tB * 64 + c * 16);
                    ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
                    kb[0] = z.x, kb[1] = z.y, kb[2] = z.z, kb[3] = z.w;
                    const uint32_t fa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(tile + L::KS + tA * 8 + c * 2));
                    const uint32_t fb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(tile + L::KS + tB * 8 + c * 2));
                    sa[0] = __byte_perm(fa, 0, 0x1010), sa[1] = __byte_perm(fa, 0, 0x3232);
                    sb[0] = __byte_perm(fb, 0, 0x1010), sb[1] = __byte_perm(fb, 0, 0x3232);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(tile + tA * 32 + c * 8);
                    const uint2 z = *reinterpret_cast<const uint2 *>(tile + tB * 32 + c * 8);
                    ka[0] = x.x, ka[1] = x.y;
                    kb[0] = z.x, kb[1] = z.y;
                    sa[0] = sa[1] = __byte_perm(e4m3x2_to_f16x2(tile[L::KS + tA * 4 + c]), 0, 0x1010);
                    sb[0] = sb[1] = __byte_perm(e4m3x2_to_f16x2(tile[L::KS + tB * 4 + c]), 0, 0x1010);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) y[i][t][0] = y[i][t][1] = y[i][t][2] = y[i][t][3] = 0.f;
#pragma unroll
                for (int q = 0; q < LW; ++q) {
                    uint32_t fa[4], fb[4];
                    e2m1x8_to_f16x2(ka[q], fa);
                    e2m1x8_to_f16x2(kb[q], fb);
                    const int blk = D == 128 ? q / 2 : 0;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t a0 = hmul2(fa[2 * z], sa[blk]), a1 = hmul2(fb[2 * z], sb[blk]);
                        const uint32_t a2 = hmul2(fa[2 * z + 1], sa[blk]), a3 = hmul2(fb[2 * z + 1], sb[blk]);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            mma_16816(y[i][t], a0, a1, a2, a3, qf[t][4 * q + 2 * z], qf[t][4 * q + 2 * z + 1]);
                    }
                }
            }
            // y <- the scores, in units of log2; the maximum moves if a weight is too large
            bool move = false;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[i][t][e] *= factor[t][e & 1];
                        if (!whole) {
                            const int pos = t0 + i * KV_TILE + (e < 2 ? tA : tB), end_at = last[t][e & 1];
                            if (!(loaded >> i & 1) || pos > end_at || (a.window > 0 && pos <= end_at - a.window))
                                y[i][t][e] = -INFINITY;
                        }
                        move |= y[i][t][e] - m[t][e & 1] > MOVE;
                    }
            if (__any_sync(~0u, move)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        float top = fmaxf(fmaxf(y[0][t][k2], y[0][t][k2 + 2]), fmaxf(y[1][t][k2], y[1][t][k2 + 2]));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                        const float to = fmaxf(m[t][k2], top - HEADROOM), keep = exp2_fast(m[t][k2] - to);
                        m[t][k2] = to;
                        l[t][k2] *= keep;
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            o[t][j][k2] *= keep;
                            o[t][j][k2 + 2] *= keep;
                        }
                    }
            }
            // values of 32 tokens
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *tile = stage + i * L::BYTES;
                uint32_t pb[NT][2], seen_b[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = exp2_fast(y[i][t][e] - m[t][e & 1]);
                        l[t][e & 1] += p[e];
                    }
                    pb[t][0] = transpose8(half_pair(p[0], p[1]));
                    pb[t][1] = transpose8(half_pair(p[2], p[3]));
                }
                uint32_t sc = *reinterpret_cast<const uint32_t *>(tile + L::VS + (D == 128 ? r : r >> 1) * KV_TILE + 4 * c);
                if (!whole) {
                    // a NaN scale (0x7f) reaches only the rows that see its token
                    const uint32_t nan4 = (((sc & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                    if (__any_sync(~0u, nan4 != 0)) {
                        sc &= ~(nan4 * 255u);
                        const uint32_t one = 0x3c00u;
                        const uint32_t n01 = ((nan4 & 1) ? one : 0) | ((nan4 >> 8 & 1) ? one << 16 : 0);
                        const uint32_t n23 = ((nan4 >> 16 & 1) ? one : 0) | ((nan4 >> 24 & 1) ? one << 16 : 0);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float hit[4] = {0.f, 0.f, 0.f, 0.f}, sees[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) sees[e] = y[i][t][e] == -INFINITY ? 0.f : 1.f;
                            seen_b[t][0] = transpose8(half_pair(sees[0], sees[1]));
                            seen_b[t][1] = transpose8(half_pair(sees[2], sees[3]));
                            mma_16816(hit, n01, n01, n23, n23, seen_b[t][0], seen_b[t][1]);
#pragma unroll
                            for (int j = 0; j < KS; ++j)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (hit[e] > 0.f) o[t][j][e] = __uint_as_float(0x7fc00000u);
                        }
                    }
                }
                const uint32_t s01 = e4m3x2_to_f16x2(sc & 0xffffu), s23 = e4m3x2_to_f16x2(sc >> 16);
                constexpr int VW = D / 64;   // words of a lane's share of a V row
                uint32_t v[4][VW];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    if constexpr (D == 128) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(tile + L::VC + (4 * c + z) * 64 + r * 8);
                        v[z][0] = u.x;
                        v[z][VW - 1] = u.y;
                    } else {
                        v[z][0] = *reinterpret_cast<const uint32_t *>(tile + L::VC + (4 * c + z) * 32 + r * 4);
                    }
                }
#pragma unroll
                for (int q = 0; q < VW; ++q) {
                    constexpr uint32_t LOW = 0x0f0f0f0fu;
                    const uint32_t lo01 = (v[0][q] & LOW) | ((v[1][q] << 4) & ~LOW), hi01 = ((v[0][q] >> 4) & LOW) | (v[1][q] & ~LOW);
                    const uint32_t lo23 = (v[2][q] & LOW) | ((v[3][q] << 4) & ~LOW), hi23 = ((v[2][q] >> 4) & LOW) | (v[3][q] & ~LOW);
                    uint32_t f0[4], f1[4], f2[4], f3[4];
                    e2m1x8_to_f16x2(lo01, f0);
                    e2m1x8_to_f16x2(hi01, f1);
                    e2m1x8_to_f16x2(lo23, f2);
                    e2m1x8_to_f16x2(hi23, f3);
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const uint32_t a0 = hmul2(f0[z], s01), a1 = hmul2(f1[z], s01), a2 = hmul2(f2[z], s23), a3 = hmul2(f3[z], s23);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma_16816(o[t][4 * q + z], a0, a1, a2, a3, pb[t][0], pb[t][1]);
                    }
                }
            }
            __syncwarp();                  // all lanes have read the stage
            if (k + S::STAGES < count) {
                fence_async_shared();
                fetch(k + S::STAGES);
            }
        }

        // ---- join the warps ---------------------------------------------------------------------
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                float sum = l[t][k2];
                sum += __shfl_xor_sync(~0u, sum, 4);
                sum += __shfl_xor_sync(~0u, sum, 8);
                sum += __shfl_xor_sync(~0u, sum, 16);
                const int col = t * 8 + 2 * c + k2;
                if (r == 0) ml_s[w * S::ROWS + col] = make_float2(m[t][k2], sum);
                float *dst = out_s + (w * S::ROWS + col) * S::OSTRIDE + r * (D / 8);
#pragma unroll
                for (int j = 0; j < KS; j += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * j) =
                        make_float4(o[t][j][k2], o[t][j][k2 + 2], o[t][j + 1][k2], o[t][j + 1][k2 + 2]);
            }
        __syncthreads();
        const bool complete = unit_begin >= begin && unit_end <= end;
        const int cta0 = (int)(unit_begin / per), cta1 = (int)((unit_end - 1) / per);
        float *const partials = reinterpret_cast<float *>(a.ws + MAX_CTAS * 4);
        constexpr int QUADS = S::ROWS * D / 4;
        auto finish = [&](int col, int d, float4 v, float top, float sum) {
            const int row = row0 + col;
            const size_t at_row = (size_t)(rq.q0 + row / G) * a.Hq + h * G + row % G;
            const float f = sum == 0.f ? 0.f : a.v_scale / sum;
            uint32_t *dst = reinterpret_cast<uint32_t *>((T *)a.o + at_row * D + d);
            *reinterpret_cast<uint2 *>(dst) = sum == 0.f ? make_uint2(0, 0) : make_uint2(pack_of<T>(v.x * f, v.y * f), pack_of<T>(v.z * f, v.w * f));
            if (d == 0 && a.lse) a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        };
        for (int i = tid; i < QUADS; i += THREADS) {
            const int col = i / (D / 4), d = i % (D / 4) * 4;
            float top = NOTHING;
#pragma unroll
            for (int x = 0; x < WARPS; ++x) top = max_nan(top, ml_s[x * S::ROWS + col].x);
            float sum = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < WARPS; ++x) {
                const float2 ml = ml_s[x * S::ROWS + col];
                const float keep = exp2_fast(ml.x - top);
                const float4 u = *reinterpret_cast<const float4 *>(out_s + (x * S::ROWS + col) * S::OSTRIDE + d);
                sum += ml.y * keep;
                v.x += u.x * keep, v.y += u.y * keep, v.z += u.z * keep, v.w += u.w * keep;
            }
            if (complete) {
                if (col < rows) finish(col, d, v, top, sum);
            } else {
                float *dst = partials + (size_t)(2 * blockIdx.x + (at == unit_begin)) * S::PARTIAL;
                __stcg(reinterpret_cast<float4 *>(dst + col * D + d), v);
                if (d == 0) __stcg(reinterpret_cast<float2 *>(dst + S::ROWS * D + 2 * col), make_float2(top, sum));
            }
        }
        if (!complete) {
            // the last of the unit's CTAs to arrive joins their results, in order
            __threadfence();
            __syncthreads();
            int *const counter = reinterpret_cast<int *>(a.ws) + cta0;
            if (tid == 0) {
                const int arrived = atomicAdd(counter, 1) == cta1 - cta0;
                if (arrived) *counter = 0;     // as the next call needs it
                *shared = arrived;
            }
            __syncthreads();
            if (*shared) {
                __threadfence();
                for (int i = tid; i < QUADS; i += THREADS) {
                    const int col = i / (D / 4), d = i % (D / 4) * 4;
                    if (col >= rows) continue;
                    float top = NOTHING, sum = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int x = cta0; x <= cta1; ++x) {
                        const float *src = partials + (size_t)(2 * x + (x == cta0)) * S::PARTIAL;
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + S::ROWS * D + 2 * col));
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(src + col * D + d));
                        const float to = max_nan(top, ml.x), keep = exp2_fast(top - to), add = exp2_fast(ml.x - to);
                        top = to;
                        sum = sum * keep + ml.y * add;
                        v.x = v.x * keep + u.x * add, v.y = v.y * keep + u.y * add;
                        v.z = v.z * keep + u.z * add, v.w = v.w * keep + u.w * add;
                    }
                    finish(col, d, v, top, sum);
                }
            }
        }
        __syncthreads();                   // the joined results are read; the next segment writes over them
        at = min(end, unit_end);
    }
}

template <int D, int NT, typename T>
cudaError_t launch_decode_attention(const KvAttentionArgs &a, cudaStream_t s) {
    using Sh = DecodeShape<D, NT>;
    static_assert((size_t)MAX_CTAS * (4 + 2 * Sh::PARTIAL * 4) <= KDA_KV4_WORKSPACE, "workspace");
    static const cudaError_t set = cudaFuncSetAttribute(decode_attention_kernel<D, NT, T>,
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (set != cudaSuccess) return set;
    decode_attention_kernel<D, NT, T><<<NT == 1 ? MAX_CTAS : MAX_CTAS / 2, THREADS, Sh::SMEM, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace kda
