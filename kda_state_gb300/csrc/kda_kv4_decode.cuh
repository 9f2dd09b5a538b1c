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
// largest, and most steps rescale nothing.  The maximum m is held as a product
// y = q . k before the row's factor f, and the exponent is (y - m) f + 9, two packed
// operations for two scores: with y f - (m f - 9) the rounding of m f alone would pass
// 2^6 from scores of 2^28 on (the weights then leave fp16, or are all 0).  128 requests:
// 131 us with either.
//
// Work is the list of all (request, block of rows, kv head, 32 tokens), cut into
// equal contiguous ranges, one a warp: a ragged batch and one long request are
// balanced alike, and a warp writes out by itself every (request, rows, head) that
// lies in its range.  One that it shares leaves a partial result, joined by the CTA
// once all its warps are done, or, where several CTAs share it, by the last of them
// to arrive; in order, so results do not depend on timing.
//
// A warp's tokens come through a ring of its own, filled by bulk copies (one
// contiguous block of 18 D bytes for 16 tokens); the next unit's are asked for
// before the last one's result leaves.
//
// With PICKED each token is a request of its own, whose cache is the list of pages that was picked for it and a kv head:
// position j of it is token j % P of the page in the list's place j / P.  The last place is the token's own page, so that
// the list's length and what the token sees of it follow from its position alone, whatever the head; an entry of -1 is a
// page without tokens.
#pragma once

#include "kda_async.cuh"
#include "kda_internal.h"
#include "kda_launch.h"
#include "kda_kv4.cuh"

namespace kda {
namespace kv4 {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int MAX_CTAS = 152 * 2;
constexpr float HEADROOM = 9.f;        // log2 of a weight at the running maximum
constexpr float MOVE = HEADROOM + 6.f; // a score this far above m makes the maximum move
constexpr float NOTHING = -1e30f;      // the running maximum before any product (they lie within 2^21)
constexpr float LOWEST = -3.4028234e38f;   // the maximum of a partial result without weights, as a score

constexpr float LN2 = 0.69314718055994531f;

// What a warp leaves of a unit that it does not have all of (rows = 0: none).
struct Piece {
    long long begin, end;
    int q0, h, row0, rows;
};
struct WarpPieces {
    Piece first, last;
};

template <int D, int NT>
struct DecodeShape {
    static constexpr int ROWS = 8 * NT;
    static constexpr int TILES = D == 128 ? 2 : 4;       // of 16 tokens: a chunk, one step of a warp
    static constexpr int CHUNK = TILES * KV_TILE;
    static constexpr int STAGES = 2;
    static constexpr int STAGE_BYTES = TILES * KvTile<D>::BYTES;
    static constexpr int OSTRIDE = D + 4;
    static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
    static constexpr int OUT = WARPS * ROWS * OSTRIDE * 4;
    static constexpr int ML = 2 * WARPS * ROWS * 8;
    static constexpr int SMEM = RING + OUT + ML + WARPS * STAGES * 8 + 16 + WARPS * sizeof(WarpPieces);
    static_assert(STAGES == 2 && ROWS * OSTRIDE * 4 <= STAGES * STAGE_BYTES, "a warp's last piece lies over its ring");
    static constexpr int PARTIAL = ROWS * (D + 2);         // floats
};

// Whether the phase with the given parity is complete (it may wait a short time).
__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}
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
// a times one half of b
__device__ __forceinline__ uint32_t hmul2_by(uint32_t a, uint32_t b, bool high) {
    const __half2 x = *reinterpret_cast<const __half2 *>(&a), y = *reinterpret_cast<const __half2 *>(&b);
    const __half2 d = __hmul2_rn(x, high ? __high2half2(y) : __low2half2(y));
    return *reinterpret_cast<const uint32_t *>(&d);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
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
// What a row's products are scaled by to be scores, up a power of two.  Neither 0 nor infinite: a difference of 0 and a
// masked -inf stay what they are.
__device__ __forceinline__ float factor_of(float scale, float up) {
    return fminf(fmaxf(fabsf(scale) * up, 1.1754944e-38f), -LOWEST);
}
// f, or NaN for a row whose largest query is infinite or NaN: all its products are then NaN, and so are the results of
// what it sees (infinite scores of one sign would be taken for masked ones).
__device__ __forceinline__ float finite_or_nan(float top, float f) {
    return top <= -LOWEST ? f : __uint_as_float(0x7fc00000u);
}
// The score at which a weight is 1, of a row whose maximum is m and whose weights add up to sum: finite, so that
// results can be joined.
__device__ __forceinline__ float base_of(float m, float factor, float sum) {
    return sum == 0.f ? LOWEST : fminf(fmaxf(fmaf(m, factor, -HEADROOM), LOWEST), -LOWEST);
}
__device__ __forceinline__ uint64_t pair_of_floats(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
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
    int row, own;                          // PICKED: the request that token q0 is of, and the page that it lies in
};
// Token t and the pages picked for it, as a request; a thread's work.  One request is guessed, the right one where all
// have as many tokens, and all of its numbers are asked for at once.
__device__ __forceinline__ Request request_of_picked(const KvAttentionArgs &a, int t, int rows, int chunk, bool tell) {
    Request r;
    r.q0 = t;
    r.n = r.len = r.first_chunk = r.chunks = r.row_blocks = r.own = 0;
    r.row = min((int)(((float)t + 0.5f) * ((float)a.B / (float)a.T)), a.B - 1);
    int q0 = a.cu[r.row], n = a.cu[r.row + 1] - q0, len = a.kv_lens[r.row];
    if (q0 > t || t - q0 >= n) {
        int lo = 0, hi = a.B;              // the first request with cu[b + 1] > t
        while (lo < hi) {
            const int b = lo + (hi - lo) / 2;
            if (a.cu[b + 1] > t) hi = b;
            else lo = b + 1;
        }
        if (lo >= a.B || a.cu[lo] > t) return r;
        r.row = lo;
        q0 = a.cu[lo], n = a.cu[lo + 1] - q0, len = a.kv_lens[lo];
    }
    if (q0 < 0 || n > a.max_q || (long long)q0 + n > a.T || len < 0 || (long long)len > ((long long)a.max_pages << a.page_shift)) {
        if (tell) report(a.err, DEVERR_SEQLENS);
        return r;
    }
    const int pos = len - n + (t - q0);
    r.n = 1;
    if (pos >= 0) {
        r.own = pos >> a.page_shift;
        r.len = (min(a.count, r.own + 1) - 1 << a.page_shift) + (pos & ((1 << a.page_shift) - 1)) + 1;
    }
    r.chunks = max(1, (r.len + chunk - 1) / chunk);
    r.row_blocks = (a.Hq / a.Hkv + rows - 1) / rows;
    return r;
}
__device__ __forceinline__ Request request_of(const KvAttentionArgs &a, int b, int rows, int chunk, bool tell) {
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
    r.first_chunk = first / chunk;
    r.chunks = max(1, (int)(((long long)r.len + chunk - 1) / chunk) - r.first_chunk);
    r.row_blocks = (r.n * (a.Hq / a.Hkv) + rows - 1) / rows;
    return r;
}

// x / y (x >= 0, y > 0), which is short where x has 32 bits
__device__ __forceinline__ long long divide(long long x, int y) {
    return x >> 32 == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
}

template <int D, int NT, typename T, bool PICKED>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 2 : 1) decode_attention_kernel(const KvAttentionArgs a) {
    using L = KvTile<D>;
    using S = DecodeShape<D, NT>;
    constexpr int KS = D / 16;             // MMA steps of a score; also V's tiles of 16 channels
    constexpr int TILES = S::TILES, CHUNK = S::CHUNK;
    constexpr int LW = D / 32;             // 32-bit words of a lane's share of a K row
    extern __shared__ __align__(128) uint8_t smem[];
    if constexpr (PICKED) {
        wait_for_earlier_kernels();
        let_later_kernels_in();
    }
    float *const out_s = reinterpret_cast<float *>(smem + S::RING);                  // [WARPS][ROWS][OSTRIDE]
    float2 *const ml_s = reinterpret_cast<float2 *>(smem + S::RING + S::OUT);        // [2][WARPS][ROWS]
    uint8_t *const bars = smem + S::RING + S::OUT + S::ML;
    int *const shared = reinterpret_cast<int *>(bars + WARPS * S::STAGES * 8);
    WarpPieces *const pieces = reinterpret_cast<WarpPieces *>(bars + WARPS * S::STAGES * 8 + 16);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int G = a.Hq / a.Hkv;
    const int requests = PICKED ? a.T : a.B;
    auto request = [&](int i, bool tell) {
        if constexpr (PICKED) return request_of_picked(a, i, S::ROWS, CHUNK, tell);
        else return request_of(a, i, S::ROWS, CHUNK, tell);
    };

    // ---- the work's total and this CTA's range -------------------------------------------------
    long long begin, end, per, base;       // base: where request b's work begins
    int b;
    Request rq;                            // request b
    {
        __shared__ long long scan_s[WARPS + 1];
        __shared__ long long found_s;
        __shared__ int found_b;
        __shared__ Request found_rq;
        const int share = (requests + THREADS - 1) / THREADS;
        long long mine = 0;
        for (int i = 0; i < share; ++i) {
            const int bb = tid * share + i;
            if (bb >= requests) break;
            const Request q = request(bb, blockIdx.x == 0);
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
            if (a.starve) barrier_await(shared_addr(bars + w * S::STAGES * 8), 16);    // (a self-test: bytes that nobody copies)
        }
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            if (i < w) before += scan_s[i];
            total += scan_s[i];
        }
        before += in - mine;
        per = max(divide(total + gridDim.x - 1, gridDim.x), (long long)WARPS);
        begin = blockIdx.x * per;
        end = min(begin + per, total);
        if (begin >= total) return;
        if (begin >= before && begin < before + mine) {
            for (int i = 0; i < share; ++i) {
                const int bb = tid * share + i;
                const Request q = request(bb, false);
                const long long here = (long long)q.chunks * q.row_blocks * a.Hkv;
                if (begin < before + here) {
                    found_b = bb;
                    found_s = before;
                    found_rq = q;
                    break;
                }
                before += here;
            }
        }
        __syncthreads();
        b = found_b;
        base = found_s;
        rq = found_rq;
    }

    uint8_t *const ring = smem + w * S::STAGES * S::STAGE_BYTES;
    const uint32_t bar0 = shared_addr(bars + w * S::STAGES * 8);
    uint32_t asked = 0, taken = 0;         // chunks that went through the ring
    bool dead = false;                     // a wait gave up: nothing more is read or written
    const int tA = 4 * (r >> 1) + (r & 1), tB = tA + 2;    // the tokens of this lane's MMA rows r and r + 8

    // ---- this warp's share of the range: contiguous, so that most of its units are its own ------
    long long at = begin + (end - begin) * w / WARPS;
    const long long stop = begin + (end - begin) * (w + 1) / WARPS;
    // A unit: the rows of one (request, block of rows, kv head), and the chunks of it that are this warp's.
    struct Unit {
        long long begin, end;
        int b, q0, n, len, h, row0, rows, c0, count, own;
    } u;
    auto plan = [&]() {                    // of the unit at `at`
        while (at >= base + (long long)rq.chunks * rq.row_blocks * a.Hkv) {
            base += (long long)rq.chunks * rq.row_blocks * a.Hkv;
            rq = request(++b, false);
        }
        const int index = (int)divide(at - base, rq.chunks);
        u.begin = base + (long long)index * rq.chunks;
        u.end = u.begin + rq.chunks;
        u.b = PICKED ? rq.row : b, u.q0 = rq.q0, u.n = rq.n, u.len = rq.len;
        if constexpr (PICKED) u.own = rq.own;
        u.h = index % a.Hkv;
        u.row0 = index / a.Hkv * S::ROWS;
        u.rows = min(S::ROWS, rq.n * G - u.row0);
        u.c0 = rq.first_chunk + (int)(at - u.begin);
        u.count = (int)(min(stop, u.end) - at);
    };
    uint32_t q_raw[NT][D / 8];             // this lane's quarter of row r of each 8, as it was given
    auto ask_q = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = u.row0 + t * 8 + r;
            const uint4 *src = reinterpret_cast<const uint4 *>((const T *)a.q + (long long)(u.q0 + row / G) * a.q_stride +
                                                               (u.h * G + row % G) * D + c * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = t * 8 + r < u.rows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                q_raw[t][4 * i] = v.x, q_raw[t][4 * i + 1] = v.y, q_raw[t][4 * i + 2] = v.z, q_raw[t][4 * i + 3] = v.w;
            }
        }
    };
    // Pages are looked up for 32 tiles at a time, one by a lane, and 32 ahead; each lane asks for its own tile
    // when its chunk's turn comes, or one lane for all of a chunk that lies in one page.
    constexpr int WINDOW = 32 / TILES;     // chunks
    const bool one_copy = 1 << a.page_shift >= CHUNK;
    int page_next = -2;                    // -2: past the end (a negative entry of the table counts as -1)
    const uint8_t *source = nullptr;
    uint32_t oks = 0, here = 0;            // tiles of the window whose page is good; of each stage, those loaded
    auto look = [&](int k) -> int {
        const long long t = ((long long)(u.c0 + k) * TILES + lane) * KV_TILE;
        if constexpr (PICKED) {
            if (k + lane / TILES >= u.count || t >= u.len) return -2;
            const int place = (int)(t >> a.page_shift);
            const int entry = a.picked[((size_t)u.q0 * a.Hkv + u.h) * a.count + place];
            if (entry == -1) return -2;
            const bool good = place == (u.len - 1) >> a.page_shift ? entry == u.own : entry >= 0 && entry < u.own;
            return good ? max(a.page_table[(size_t)u.b * a.max_pages + entry], -1) : -1;
        } else {
            return k + lane / TILES < u.count && t < u.len ? max(a.page_table[(size_t)u.b * a.max_pages + (t >> a.page_shift)], -1) : -2;
        }
    };
    auto fetch = [&](int k) {              // the unit's k-th chunk
        const int j = k % WINDOW;
        if (j == 0) {
            const int page = k == 0 ? look(0) : page_next;
            page_next = look(k + WINDOW);
            const bool ok = page >= 0 && page < a.num_pages;
            oks = __ballot_sync(~0u, ok);
            if (!ok && page != -2) report(a.err, DEVERR_PAGE_RANGE);
            const int in_page = (int)((unsigned)((u.c0 + k) * TILES + lane) * KV_TILE) & ((1 << a.page_shift) - 1);
            source = a.pool + ((((size_t)page * a.Hkv + u.h) << (a.page_shift - 4)) + (in_page >> 4)) * L::BYTES;
        }
        const int s = asked++ % S::STAGES;
        const uint32_t run = oks >> (TILES * j) & ((1u << TILES) - 1), bar = bar0 + 8 * s;
        here = (here & ~(((1u << TILES) - 1) << (TILES * s))) | run << (TILES * s);
        uint8_t *const dst = ring + s * S::STAGE_BYTES;
        if (lane == TILES * j) {
            barrier_expect(bar, __popc(run) * L::BYTES);
            if (one_copy && run) bulk_copy(dst, source, __popc(run) * L::BYTES, bar);
        }
        if (!one_copy) {
            __syncwarp();
            const int i = lane - TILES * j;
            if (i >= 0 && i < TILES && (run >> i & 1)) bulk_copy(dst + i * L::BYTES, source, L::BYTES, bar);
        }
    };
    // A result that is part of its unit's: maximum, sum and weighted values of its rows.  Of a warp's
    // range only the first unit (begun by another warp) and the last (not ended) are such: the first
    // goes to out_s, the last over the ring, which is empty by then.
    auto row_of = [&](const Unit &x, int col) {
        const int row = x.row0 + col;
        return (size_t)(x.q0 + row / G) * a.Hq + x.h * G + row % G;
    };
    if (lane == 0) pieces[w].first.rows = pieces[w].last.rows = 0;

    bool more = at < stop;
    if (more) {
        plan();
        ask_q();
#pragma unroll
        for (int i = 0; i < S::STAGES; ++i)
            if (i < u.count) fetch(i);
    }
    while (more) {
        // ---- queries, as B fragments, and what their rows see -----------------------------------
        uint32_t qf[NT][2 * KS];
        float factor[NT][2];
        int last[NT][2];
        int last_min, first_max;
        {
            const int i0 = u.row0 / G, i1 = (u.row0 + u.rows - 1) / G;
            last_min = u.len - u.n + i0;
            first_max = a.window > 0 ? u.len - u.n + i1 + 1 - a.window : 0;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 f = pair_of<T>(q_raw[t][i]);
                top = max_nan(top, max_nan(fabsf(f.x), fabsf(f.y)));
            }
            top = max_nan(top, __shfl_xor_sync(~0u, top, 1));
            top = max_nan(top, __shfl_xor_sync(~0u, top, 2));
            const int e = min(max((int)(__float_as_uint(top) >> 23 & 255), 1), 253);
            const float down = copysignf(finite_or_nan(top, __uint_as_float((uint32_t)(254 - e) << 23)), a.scale_k), up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 f = pair_of<T>(q_raw[t][i]);
                qf[t][i] = half_pair(f.x * down, f.y * down);
            }
            // scores come back by columns: this lane holds those of rows 2 c and 2 c + 1
            const float f = factor_of(a.scale_k, up);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                factor[t][k] = __shfl_sync(~0u, f, (2 * c + k) * 4);
                const int col = t * 8 + 2 * c + k;
                last[t][k] = col < u.rows ? u.len - u.n + (u.row0 + col) / G : -1;
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


        for (int k = 0; k < u.count && !dead; ++k) {
            const int s = taken & 1, t0 = (u.c0 + k) * CHUNK;
            const uint32_t parity = taken >> 1 & 1;
            if (!__all_sync(~0u, barrier_test(bar0 + 8 * s, parity) || barrier_wait_for(bar0 + 8 * s, parity, a.wait_ns))) {
                if (asked - taken > 1) barrier_wait_for(bar0 + 8 * (1 - s), (taken + 1) >> 1 & 1, a.wait_ns);
                if (lane == 0) report(a.err, DEVERR_TIMEOUT);
                dead = true;
                break;
            }
            ++taken;
            const uint8_t *stage = ring + s * S::STAGE_BYTES;
            const uint32_t loaded = here >> (TILES * s) & ((1u << TILES) - 1);
            const bool whole = loaded == (1u << TILES) - 1 && t0 >= first_max && t0 + CHUNK - 1 <= last_min;

            // scores: the tiles' products alternate, so that none waits for its own sums
            float y[TILES][NT][4];
            {
                uint32_t ka[TILES][LW], kb[TILES][LW], sa[TILES], sb[TILES];
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    const uint8_t *tile = stage + i * L::BYTES;
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(tile + tA * 64 + c * 16);
                        const uint4 z = *reinterpret_cast<const uint4 *>(tile + tB * 64 + c * 16);
                        ka[i][0] = x.x, ka[i][1] = x.y, ka[i][LW - 2] = x.z, ka[i][LW - 1] = x.w;
                        kb[i][0] = z.x, kb[i][1] = z.y, kb[i][LW - 2] = z.z, kb[i][LW - 1] = z.w;
                        sa[i] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(tile + L::KS + tA * 8 + c * 2));
                        sb[i] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(tile + L::KS + tB * 8 + c * 2));
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(tile + tA * 32 + c * 8);
                        const uint2 z = *reinterpret_cast<const uint2 *>(tile + tB * 32 + c * 8);
                        ka[i][0] = x.x, ka[i][1] = x.y;
                        kb[i][0] = z.x, kb[i][1] = z.y;
                        sa[i] = e4m3x2_to_f16x2(tile[L::KS + tA * 4 + c]);
                        sb[i] = e4m3x2_to_f16x2(tile[L::KS + tB * 4 + c]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) y[i][t][0] = y[i][t][1] = y[i][t][2] = y[i][t][3] = 0.f;
                }
#pragma unroll
                for (int q = 0; q < LW; ++q) {
                    uint32_t fa[TILES][4], fb[TILES][4];
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        e2m1x8_to_f16x2(ka[i][q], fa[i]);
                        e2m1x8_to_f16x2(kb[i][q], fb[i]);
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int i = 0; i < TILES; ++i) {
                            const uint32_t a0 = hmul2_by(fa[i][2 * z], sa[i], D == 128 && q >= 2), a1 = hmul2_by(fb[i][2 * z], sb[i], D == 128 && q >= 2);
                            const uint32_t a2 = hmul2_by(fa[i][2 * z + 1], sa[i], D == 128 && q >= 2), a3 = hmul2_by(fb[i][2 * z + 1], sb[i], D == 128 && q >= 2);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                mma_16816(y[i][t], a0, a1, a2, a3, qf[t][4 * q + 2 * z], qf[t][4 * q + 2 * z + 1]);
                        }
                }
            }
            // x: log2 of the weights; the maximum moves if one is too large
            uint32_t seen = ~0u;               // a bit a score
            if (!whole) {
                seen = 0;
#pragma unroll
                for (int i = 0; i < TILES; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int pos = t0 + i * KV_TILE + (e < 2 ? tA : tB), end_at = last[t][e & 1];
                            if ((loaded >> i & 1) && pos <= end_at && (a.window <= 0 || pos > end_at - a.window))
                                seen |= 1u << ((i * NT + t) * 4 + e);
                        }
            }
            float x[TILES][NT][4];
            auto weigh = [&]() {
#pragma unroll
                for (int i = 0; i < TILES; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            uint64_t v = pair_of_floats(y[i][t][e], y[i][t][e + 1]);
                            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(pair_of_floats(-m[t][0], -m[t][1])));
                            asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(pair_of_floats(factor[t][0], factor[t][1])), "l"(pair_of_floats(HEADROOM, HEADROOM)));
                            asm("mov.b64 {%0, %1}, %2;" : "=f"(x[i][t][e]), "=f"(x[i][t][e + 1]) : "l"(v));
                        }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < TILES; ++i)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!(seen >> ((i * NT + t) * 4 + e) & 1)) x[i][t][e] = -INFINITY;
                }
            };
            weigh();
            float high = -INFINITY;
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) high = max3(high, x[i][t][e], x[i][t][e + 1]);
            if (__any_sync(~0u, high > MOVE)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 0; i < TILES; ++i)
#pragma unroll
                            for (int e = k2; e < 4; e += 2)
                                if (seen >> ((i * NT + t) * 4 + e) & 1) top = fmaxf(top, y[i][t][e]);
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                        const float to = fmaxf(m[t][k2], top), keep = exp2_fast((m[t][k2] - to) * factor[t][k2]);
                        m[t][k2] = to;
                        l[t][k2] *= keep;
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            o[t][j][k2] *= keep;
                            o[t][j][k2 + 2] *= keep;
                        }
                    }
                weigh();
            }
            // values
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                const uint8_t *tile = stage + i * L::BYTES;
                uint32_t pb[NT][2], seen_b[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = exp2_fast(x[i][t][e]);
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
                            for (int e = 0; e < 4; ++e) sees[e] = seen >> ((i * NT + t) * 4 + e) & 1 ? 1.f : 0.f;
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
            if (k + S::STAGES < u.count) {
                fence_async_shared();
                fetch(k + S::STAGES);
            }
        }

        // ---- the unit's end: the next one's codes are asked for, then its results leave ----------
        const Unit x = u;
        const bool begun = at == x.begin, ended = at + x.count == x.end;
        at += x.count;
        more = at < stop;
        if (more) {
            plan();
            if (!dead) {
                fence_async_shared();
#pragma unroll
                for (int i = 0; i < S::STAGES; ++i)
                    if (i < u.count) fetch(i);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                float sum = l[t][k2];
                sum += __shfl_xor_sync(~0u, sum, 4);
                sum += __shfl_xor_sync(~0u, sum, 8);
                sum += __shfl_xor_sync(~0u, sum, 16);
                const float base = base_of(m[t][k2], factor[t][k2], sum);
                const int col = t * 8 + 2 * c + k2;
                if (begun && ended) {
                    if (col >= x.rows || dead) continue;
                    const size_t row = row_of(x, col);
                    const float f = sum == 0.f ? 0.f : 1.f / sum;      // (apart from v_scale: their quotient may underflow)
                    if (r == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * LN2;
                    uint32_t y[KS];
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        y[j] = sum == 0.f ? 0u : pack_of<T>(o[t][j][k2] * f * a.v_scale, o[t][j][k2 + 2] * f * a.v_scale);
                    uint4 *dst = reinterpret_cast<uint4 *>((T *)a.o + row * D + r * (D / 8));
#pragma unroll
                    for (int j = 0; j < KS / 4; ++j) dst[j] = make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                } else {
                    if (r == 0) ml_s[((begun ? WARPS : 0) + w) * S::ROWS + col] = make_float2(base, sum);
                    float *dst = (begun ? reinterpret_cast<float *>(ring) : out_s + w * S::ROWS * S::OSTRIDE) + col * S::OSTRIDE + r * (D / 8);
#pragma unroll
                    for (int j = 0; j < KS; j += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * j) =
                            make_float4(o[t][j][k2], o[t][j][k2 + 2], o[t][j + 1][k2], o[t][j + 1][k2 + 2]);
                }
            }
        if (!(begun && ended) && lane == 0) {
            Piece &y = begun ? pieces[w].last : pieces[w].first;
            y.begin = x.begin, y.end = x.end, y.q0 = x.q0, y.h = x.h, y.row0 = x.row0, y.rows = x.rows;
        }
        if (more) ask_q();
    }

    // ---- join what the warps have of one unit ------------------------------------------------------
    // A unit begins with a warp's last piece, or before this CTA (then the first warp with a share has its
    // first piece of it), and goes on in the first pieces of the warps behind.
    __syncthreads();
    constexpr int QUADS = S::ROWS * D / 4;
    auto finish = [&](const Piece &x, int col, int d, float4 v, float top, float sum) {
        const int row = x.row0 + col;
        const size_t at_row = (size_t)(x.q0 + row / G) * a.Hq + x.h * G + row % G;
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>((T *)a.o + at_row * D + d) =
            sum == 0.f ? make_uint2(0, 0) : make_uint2(pack_of<T>(v.x * f * a.v_scale, v.y * f * a.v_scale), pack_of<T>(v.z * f * a.v_scale, v.w * f * a.v_scale));
        if (d == 0 && a.lse) a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * LN2;
    };
    auto add = [](float4 &v, float &top, float &sum, const float4 &z, const float2 &ml) {
        const float to = max_nan(top, ml.x), keep = exp2_fast(top - to), by = exp2_fast(ml.x - to);
        top = to;
        sum = sum * keep + ml.y * by;
        v.x = v.x * keep + z.x * by, v.y = v.y * keep + z.y * by;
        v.z = v.z * keep + z.z * by, v.w = v.w * keep + z.w * by;
    };
    // four channels of a row over this CTA's pieces of the unit x that begins in warp w0's first or last piece
    auto gather = [&](const Piece &x, int w0, bool with_last, int col, int d, float &top, float &sum) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        top = LOWEST, sum = 0.f;
        if (with_last)
            add(v, top, sum, *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w0 * S::STAGES * S::STAGE_BYTES) +
                                                               col * S::OSTRIDE + d),
                ml_s[(WARPS + w0) * S::ROWS + col]);
        for (int y = with_last ? w0 + 1 : w0; y < WARPS; ++y)
            if (pieces[y].first.rows && pieces[y].first.begin == x.begin)
                add(v, top, sum, *reinterpret_cast<const float4 *>(out_s + (y * S::ROWS + col) * S::OSTRIDE + d), ml_s[y * S::ROWS + col]);
        return v;
    };
    // the two that other CTAs share: four warps each, one for the unit that began before, one for that which goes on
    const int side = w >> 2, st = tid & 127;
    int w0 = -1;
    if (side == 0) {
        for (int y = WARPS - 1; y >= 0; --y)
            if (pieces[y].first.rows || pieces[y].last.rows) w0 = y;
        if (w0 >= 0 && !(pieces[w0].first.rows && pieces[w0].first.begin < begin)) w0 = -1;
    } else {
        for (int y = 0; y < WARPS; ++y)
            if (pieces[y].last.rows && pieces[y].last.end > end) w0 = y;
    }
    float *const partials = reinterpret_cast<float *>(a.ws + MAX_CTAS * 4);
    Piece x;
    x.rows = 0;
    if (w0 >= 0) {
        x = side ? pieces[w0].last : pieces[w0].first;
        float *const dst = partials + (size_t)(2 * blockIdx.x + side) * S::PARTIAL;
        for (int i = st; i < x.rows * (D / 4); i += 128) {
            const int col = i / (D / 4), d = i % (D / 4) * 4;
            float top, sum;
            const float4 v = gather(x, w0, side, col, d, top, sum);
            __stcg(reinterpret_cast<float4 *>(dst + col * D + d), v);
            if (d == 0) __stcg(reinterpret_cast<float2 *>(dst + S::ROWS * D + 2 * col), make_float2(top, sum));
        }
    }
    __syncthreads();
    const int cta0 = w0 >= 0 ? (int)divide(x.begin, (int)per) : 0, cta1 = w0 >= 0 ? (int)divide(x.end - 1, (int)per) : 0;
    if (st == 0) {
        bool arrived = false;
        if (w0 >= 0) {
            // the last of the unit's CTAs to arrive joins their results, in order
            int *const counter = reinterpret_cast<int *>(a.ws) + cta0;
            __threadfence();
            arrived = atomicAdd(counter, 1) == cta1 - cta0;
            if (arrived) {
                *counter = 0;              // as the next call needs it
                __threadfence();
            }
        }
        shared[side] = arrived;
    }
    // units that begin and end in this CTA, four channels a thread of all of them side by side
    uint32_t inside = 0;                   // the warps where they begin, four bits each
    int units = 0, most = 0;
    for (int y = 0; y < WARPS; ++y)
        if (pieces[y].last.rows && pieces[y].last.end <= end) {
            inside |= (uint32_t)y << (4 * units++);
            most = max(most, pieces[y].last.rows);
        }
    for (int i = tid; i < units * most * (D / 4); i += THREADS) {
        const int unit = i / (most * (D / 4)), y = inside >> (4 * unit) & 15, col = i / (D / 4) - unit * most, d = i % (D / 4) * 4;
        const Piece x = pieces[y].last;
        if (col >= x.rows) continue;
        float top, sum;
        const float4 v = gather(x, y, true, col, d, top, sum);
        finish(x, col, d, v, top, sum);
    }
    __syncthreads();
    if (!shared[side]) return;
    // each warp takes every fourth result, a lane QUADS / 32 times four channels of it
    {
        constexpr int N = QUADS / 32;
        float4 v[N];
        float top[N], sum[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f), top[k] = LOWEST, sum[k] = 0.f;
#pragma unroll 2
        for (int y = cta0 + (w & 3); y <= cta1; y += 4) {
            const float *src = partials + (size_t)(2 * y + (y == cta0)) * S::PARTIAL;
            float4 z[N];
            float2 ml[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int i = 32 * k + lane, col = i / (D / 4);
                z[k] = make_float4(0.f, 0.f, 0.f, 0.f), ml[k] = make_float2(LOWEST, 0.f);
                if (col < x.rows) {
                    z[k] = __ldcg(reinterpret_cast<const float4 *>(src) + i);
                    ml[k] = __ldcg(reinterpret_cast<const float2 *>(src + S::ROWS * D) + col);
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k) add(v[k], top[k], sum[k], z[k], ml[k]);
        }
        // (both sides' pieces in out_s have been read)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = 32 * k + lane, col = i / (D / 4), d = i % (D / 4) * 4;
            *reinterpret_cast<float4 *>(out_s + (w * S::ROWS + col) * S::OSTRIDE + d) = v[k];
            if (d == 0) ml_s[w * S::ROWS + col] = make_float2(top[k], sum[k]);
        }
    }
    asm volatile("bar.sync %0, 128;" ::"r"(1 + side) : "memory");
    for (int i = st; i < x.rows * (D / 4); i += 128) {
        const int col = i / (D / 4), d = i % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = LOWEST, sum = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            add(v, top, sum, *reinterpret_cast<const float4 *>(out_s + ((4 * side + y) * S::ROWS + col) * S::OSTRIDE + d),
                ml_s[(4 * side + y) * S::ROWS + col]);
        finish(x, col, d, v, top, sum);
    }
}

template <int D, int NT, typename T, bool PICKED = false>
cudaError_t launch_decode_attention(const KvAttentionArgs &a, cudaStream_t s) {
    using Sh = DecodeShape<D, NT>;
    static_assert((size_t)MAX_CTAS * (4 + 2 * Sh::PARTIAL * 4) <= KDA_KV4_WORKSPACE, "workspace");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(decode_attention_kernel<D, NT, T, PICKED>), Sh::SMEM, done);
    if (e != cudaSuccess) return e;
    if (PICKED) return launch_early(decode_attention_kernel<D, NT, T, PICKED>, dim3(NT == 1 ? MAX_CTAS : MAX_CTAS / 2), dim3(THREADS), Sh::SMEM, s, a);
    decode_attention_kernel<D, NT, T, PICKED><<<NT == 1 ? MAX_CTAS : MAX_CTAS / 2, THREADS, Sh::SMEM, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace kda
