// Attention over the 4-bit cache for many query rows: prompts, long drafts.
//
// One CTA an SM works on 128 query rows of a kv head at a time (QT = 1) or 256
// (QT = 2), a row being one (token, query head of the group), against tiles of
// 128 cached tokens.  Four kinds of warps hand work on through mbarriers:
//
//   load    (warp 17)     claims the next part of the work and describes it to the
//                         others; looks up pages and asks for their codes by bulk
//                         copies, 64 tokens to a stage of a ring
//   unpack  (warps 8-15)  codes to fp16 K [token][channel] and V^T [channel][token],
//                         both K-major with the 128-byte swizzle: one conversion and
//                         one product with the scale for two values, exact.  V is
//                         turned by transposing matrix stores; a lane takes its
//                         bytes in an order of its own, so that the eight rows of
//                         each stored matrix lie in different banks
//   product (warp 16)     S = Q K^T and O += P V on tcgen05 (fp16, fp32 sums): S, P
//                         and O stay in TMEM, with D = 128 P over S's columns
//   softmax (warps 0-7)   two groups of four warps, a thread a row: the running
//                         maximum (it moves only when a score passes it by 2^6, so O
//                         is seldom rescaled), the weights as fp16 into TMEM, the sum
//
// The two groups alternate on the tensor cores: one's softmax runs beside the
// other's products.  With QT = 2 they hold different rows and share each tile
// (two products for each unpacked tile); with QT = 1 the same rows and every other
// tile, joined at the end.  Queries are scaled by powers of two and weights held
// 2^9 above the maximum as in the kernel for few rows.  The exponent of a weight is
// one fused operation, y f - (m f - 9), while a warp's maxima are below 2^10 as
// scores (m f is then rounded by 2^-14 or less), and (y - m) f + 9 beyond.  (With the second form
// everywhere prompts of 2048 tokens take 870 us instead of 862, with 64 channels 662 instead of 643.)
//
// If there are fewer (request, rows, head) than SMs, each is cut along the tokens;
// the last part to arrive joins the results in order, so they do not depend on
// which CTA claimed what.
#pragma once

#include "kda_kv4_decode.cuh"

namespace kda {
namespace kv4 {

constexpr int TT = 128;                // tokens of a tile
constexpr int BOX = 64;                // tokens of a stage of codes: half a tile
constexpr int TILE_THREADS = 20 * 32;  // warps 18 and 19 are idle: registers are dealt by four warps
constexpr int REGS_SOFTMAX = 168, REGS_UNPACK = 40, REGS_OTHER = 64;   // 640 threads are launched with 96
static_assert(256 * REGS_SOFTMAX + 256 * REGS_UNPACK + 128 * REGS_OTHER <= TILE_THREADS * 96, "register split");
constexpr int SMS = 152;
constexpr float FAR = 1024.f;          // a maximum, as a score, from which on differences are taken before the factor
constexpr int MAX_SLOTS = 252;         // partial results, as the workspace holds
constexpr int NEXT_PART = MAX_SLOTS, CTAS_DONE = NEXT_PART + 1;        // counters behind the joins'
static_assert(CTAS_DONE < MAX_CTAS, "counters");

// A piece of work: rows of one kv head of one request against tiles of its cache.
struct Part {
    int b, h, row0, rows, q0, n, len;
    int tile0, tiles;                  // of TT tokens; tiles may be 0, and is -1 after the last part
    int pieces, slot0, piece;          // how many parts share the rows; their first slot
};

template <int D, int QT>
struct TileShape {
    static constexpr int RAW = QT == 1 ? 6 : 3;          // stages of BOX tokens' codes
    static constexpr int RAW_BYTES = BOX / KV_TILE * KvTile<D>::BYTES;
    static constexpr int QBYTES = 128 * D * 2;
    static constexpr int KBYTES = TT * D * 2;            // of a tile of K, and of V^T: two stages each
    static constexpr int K_AT = QT * QBYTES, V_AT = K_AT + 2 * KBYTES, RAW_AT = V_AT + 2 * KBYTES;
    static constexpr int META = RAW_AT + RAW * RAW_BYTES;
    static constexpr int PARTIAL = 128 * (D + 2);        // floats
    // Columns of TMEM: S, O, and P, a column for two tokens' weights.  If there is room, P has columns of its own; else
    // it lies over S, and the next S waits for the product that reads P: products of different accumulators are
    // not ordered among themselves.  When it came the wait cost prompts of 2048 tokens 7% (791 -> 851 us), drafts of 8
    // tokens 2% (136 -> 138); a product warp for each group instead of one that alternates took 913, half tiles in turn,
    // so that the next scores are always there, 1035, weights handed on by halves 869 (whole: 859).
    static constexpr bool OWN_P = D == 64;
    // Then, with QT = 2, the next S is asked for as soon as the softmax has this one in registers (2 x 2048 tokens on
    // up to 6 K, D = 64: 141 -> 132 us).
    static constexpr bool EARLY = OWN_P && QT == 2;
    static constexpr uint32_t O_COL = 256, P_COL = OWN_P ? O_COL + 2 * D : 0, P_STEP = OWN_P ? TT / 2 : TT;
};

// The small shared arrays behind the tiles.
struct alignas(16) TileMeta {
    float2 ml[2][128];                 // maximum and sum of the groups' rows (QT = 1)
    uint8_t nan_row[2][128];           // scale blocks in which a row met a NaN value (QT = 1)
    uint8_t nan_value[4][16][8];       // by tile & 3, group of 8 tokens, block: tokens whose V scale is NaN
    uint8_t nan_group[4][16];          // whether that group has any (else its bytes above are old)
    uint8_t missing[4][16];            // 255: the group's page is out of range
    Part parts[4];
    int2 raw_about[8];                 // by stage of codes: tokens before the end; a bit a run of 16 out of range
    uint32_t tmem;
    uint2 asked;                       // the stage of codes to be filled next, and how often that ring went round
    int last, dead, cut;
    uint64_t bars[27 + 2 * 6];
};

__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) {   // K-major, 128-byte swizzle, 8-row groups 1 KB apart
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)64 << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
constexpr uint32_t idesc_f16(int M, int N) {                      // fp16 operands, fp32 sums, both K-major
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_done(uint32_t bar) {          // arrives when every MMA issued so far is complete
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of this thread's lane; the registers hold them after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32_async(uint32_t at, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
// The wait names the registers, so that nothing reads them before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
    tmem_ld32_async(at, r);
    tmem_ld_wait(r);
}
// (x0, x1) * f + c, on pairs of fp32
__device__ __forceinline__ void fma_pair(uint32_t &x0, uint32_t &x1, uint64_t f, uint64_t c) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x0), "r"(x1));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(f), "l"(c));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x0), "=r"(x1) : "l"(v));
}
// What is added to y f for the exponent of a weight, up to FAR; finite before any product, so that a masked -inf stays.
__device__ __forceinline__ float offset_of(float m, float factor) {
    return fminf(fmaf(-m, factor, HEADROOM), -LOWEST);
}
__device__ __forceinline__ bool is_far(float m, float factor) {
    return m != NOTHING && fabsf(m * factor) >= FAR;
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
template <int N>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One lane of the warp, chosen so that the compiler knows it is one.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one;
}
__device__ __forceinline__ void group_sync(uint32_t id, uint32_t count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// A warp's bounded wait; once one has given up (*dead), none waits any longer and the CTA runs out on what it has.
__device__ __forceinline__ void wait_or_dead(uint32_t bar, uint32_t parity, volatile int *dead) {
    if (!barrier_test(bar, parity)) {
        const uint64_t t0 = global_timer();
        while (!*dead && !barrier_test(bar, parity))
            if (global_timer() - t0 > ASYNC_WAIT_NS) *dead = 1;
    }
    __syncwarp();
}
// The same, and whether the phase is complete: the loading and unpacking warps end where it is not.  They leave what others
// may still use as it is, a part's description (its readers meet at barriers by it) and a stage whose copies may be under
// way (its barrier takes no second arrival before they land).
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *dead, uint64_t limit_ns = ASYNC_WAIT_NS) {
    bool ok = barrier_test(bar, parity);
    if (__all_sync(~0u, ok)) return true;
    const uint64_t t0 = global_timer();
    while (!ok && !*dead) {
        ok = barrier_test(bar, parity);
        if (global_timer() - t0 > limit_ns) *dead = 1;
    }
    return __all_sync(~0u, ok);
}
// Whether any thread of the named barrier's says so.
__device__ __forceinline__ bool group_any(uint32_t id, uint32_t count, bool mine) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)mine), "r"(id), "r"(count)
                 : "memory");
    return r;
}

__device__ __forceinline__ int tiles_of(int tokens) { return tokens / TT + (tokens % TT != 0); }

// Finds parts by number, in ascending order, 32 requests at a time; every lane of a warp calls it.
// Up to 128 requests come by classes of their length, the longest first, so that the last parts
// claimed are short ones (64 requests of 0.5 to 6 K tokens, 8 new each: 172 -> 157 us); what is
// needed of them is kept, a lane a request of each 32.
template <int QT>
struct Walker {
    static constexpr int GROUPS = 4;
    int b0, before, slots_before, cut, classes, cls;
    int parts[GROUPS], cls_of[GROUPS];     // of requests lane, lane + 32, ...: parts (negative: cut ones), class
    int mine, my_slots, incl, slots_incl;

    // Tiles that no part of the request exceeds.
    __device__ __forceinline__ static int most_tiles(const KvAttentionArgs &a, int len) {
        const int all = tiles_of(len);
        if (a.window <= 0) return max(all, 1);
        const long long near = ((long long)a.window + 128 * QT) / TT + 2;
        return max((int)min((long long)all, near), 1);
    }
    __device__ __forceinline__ int pieces_of(const KvAttentionArgs &a, int len) const {
        return cut > 0 ? (most_tiles(a, len) + cut - 1) / cut : 1;
    }
    __device__ __forceinline__ int parts_of(const KvAttentionArgs &a, const Request &q) const {
        const int pieces = pieces_of(a, q.len), n = q.row_blocks * a.Hkv * pieces;
        return pieces > 1 ? -n : n;
    }
    __device__ __forceinline__ void load(const KvAttentionArgs &a) {
        const int lane = threadIdx.x & 31;
        int n = 0;
        if (classes > 1) {
#pragma unroll
            for (int i = 0; i < GROUPS; ++i)
                if (b0 == 32 * i && cls_of[i] == cls) n = parts[i];
        } else if (b0 + lane < a.B) {
            n = parts_of(a, request_of(a, b0 + lane, 128 * QT, TT, blockIdx.x == 0));
        }
        mine = abs(n);
        my_slots = n < 0 ? -n : 0;
        incl = mine, slots_incl = my_slots;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, incl, o), y = __shfl_up_sync(~0u, slots_incl, o);
            if (lane >= o) incl += x, slots_incl += y;
        }
    }
    __device__ __forceinline__ void start(const KvAttentionArgs &a, int cut_) {
        cut = cut_;
        classes = a.B > 1 && a.B <= 32 * GROUPS ? 8 : 1;
        b0 = before = slots_before = cls = 0;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int b = 32 * i + (threadIdx.x & 31);
            parts[i] = cls_of[i] = 0;
            if (classes > 1 && b < a.B) {
                const Request q = request_of(a, b, 128 * QT, TT, blockIdx.x == 0);
                parts[i] = parts_of(a, q);
                cls_of[i] = q.row_blocks ? most_tiles(a, q.len) : 0;      // tiles first
            }
        }
        int longest = 1;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) longest = max(longest, cls_of[i]);
        longest = __reduce_max_sync(~0u, longest);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
            cls_of[i] = cls_of[i] ? (int)((long long)(longest - cls_of[i]) * classes / longest) : 0;
        load(a);
    }
    __device__ __forceinline__ bool find(const KvAttentionArgs &a, int p, Part &out) {
        while (true) {
            const int total = __shfl_sync(~0u, incl, 31);
            if (p < before + total) break;
            b0 += 32;
            if (b0 >= a.B) {
                if (cls + 1 >= classes) return false;
                ++cls;
                b0 = 0;
            }
            before += total;
            slots_before += __shfl_sync(~0u, slots_incl, 31);
            load(a);
        }
        const int src = __ffs(__ballot_sync(~0u, before + incl > p)) - 1;
        const int index = p - (before + __shfl_sync(~0u, incl - mine, src));
        out.b = b0 + src;
        const Request q = request_of(a, out.b, 128 * QT, TT, false);
        const int blocks = q.row_blocks;
        out.q0 = q.q0, out.n = q.n, out.len = q.len;
        out.pieces = pieces_of(a, q.len);
        out.piece = index % out.pieces;
        const int unit = index / out.pieces;
        out.slot0 = slots_before + __shfl_sync(~0u, slots_incl - my_slots, src) + unit * out.pieces;
        out.h = unit / blocks;
        // the rows that see most come first
        out.row0 = (blocks - 1 - unit % blocks) * 128 * QT;
        const int G = a.Hq / a.Hkv;
        out.rows = min(128 * QT, out.n * G - out.row0);
        const int i0 = out.row0 / G, i1 = (out.row0 + out.rows - 1) / G;
        const int lo = a.window > 0 ? max(0, out.len - out.n + i0 + 1 - a.window) / TT : 0;
        const int hi = tiles_of(max(out.len - out.n + i1 + 1, 0));
        const long long tiles = max(hi - lo, 1);
        out.tile0 = lo + (int)(tiles * out.piece / out.pieces);
        out.tiles = lo + (int)(tiles * (out.piece + 1) / out.pieces) - out.tile0;
        return true;
    }
};

// How the work is cut along the tokens (0: not at all); a whole warp calls it.
// Only fewer units than SMs are cut, into the shortest pieces (of two tiles at least) that make one part an SM at most:
// with more parts some SMs would work on two while others wait (one request of 100 new tokens over 3259, 56 units: 168 parts
// 54 us, 112 parts 41 us).
template <int QT>
__device__ __noinline__ int cut_of(const KvAttentionArgs &a) {
    constexpr int GROUPS = 5;              // larger batches are not cut
    const int lane = threadIdx.x & 31;
    int n_of[GROUPS], tiles_in[GROUPS];
    long long units = 0, all = 0;
    int longest = 1;
    for (int i = 0; i < GROUPS; ++i) n_of[i] = 0, tiles_in[i] = 1;
    for (int b = lane, i = 0; b < a.B; b += 32, ++i) {
        const Request q = request_of(a, b, 128 * QT, TT, false);
        if (!q.row_blocks) continue;
        const int tiles = Walker<QT>::most_tiles(a, q.len);
        units += (long long)q.row_blocks * a.Hkv;
        all += (long long)q.row_blocks * a.Hkv * tiles;
        longest = max(longest, tiles);
#pragma unroll
        for (int k = 0; k < GROUPS; ++k)
            if (i == k) n_of[k] = q.row_blocks * a.Hkv, tiles_in[k] = tiles;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        units += __shfl_xor_sync(~0u, units, o);
        all += __shfl_xor_sync(~0u, all, o);
        longest = max(longest, __shfl_xor_sync(~0u, longest, o));
    }
    if (units >= SMS || a.B > 32 * GROUPS) return 0;
    int cut = (int)max((all + SMS - 1) / SMS, 2LL);
    for (; cut < longest; cut += max(cut / 8, 1)) {
        int parts = 0;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) parts += n_of[k] * ((tiles_in[k] + cut - 1) / cut);
        if (__reduce_add_sync(~0u, parts) <= SMS) break;
    }
    return cut;
}

// Byte of the 16-byte chunk (8 fp16 of the contraction axis) of a row in a K-major tile of `rows` rows.
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk, int rows) {
    return (uint32_t)((chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// The first and last tokens row `row` of a part sees (last < first: none).
__device__ __forceinline__ int2 sight(const KvAttentionArgs &a, const Part &p, int row) {
    if (row >= p.rows) return make_int2(0, -1);
    const int last = p.len - p.n + (p.row0 + row) / (a.Hq / a.Hkv);
    return make_int2(a.window > 0 ? max(0, last + 1 - a.window) : 0, last);
}

// Four 8 x 8 matrices of fp16, each stored transposed; lane 8 m + r gives the address of row r of matrix m.
__device__ __forceinline__ void store_transposed(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

template <int D, int QT, typename T>
__global__ void __launch_bounds__(TILE_THREADS, 1) tile_attention_kernel(const KvAttentionArgs a) {
    using L = KvTile<D>;
    using S = TileShape<D, QT>;
    extern __shared__ __align__(1024) uint8_t tile_smem[];
    uint8_t *const smem = tile_smem;
    TileMeta &meta = *reinterpret_cast<TileMeta *>(smem + S::META);
    volatile int *const dead = &meta.dead;
    const uint32_t bar = shared_addr(meta.bars);
    const uint32_t PART_FULL = bar, PART_FREE = bar + 32, Q_FULL = bar + 64, S_FULL = bar + 80, P_FULL = bar + 96, PV_DONE = bar + 112,
                   K_FULL = bar + 128, K_FREE = bar + 144, V_FULL = bar + 160, V_FREE = bar + 176, FINISHED = bar + 192,
                   S_FREE = bar + 200, RAW_FULL = bar + 216, RAW_FREE = RAW_FULL + 8 * S::RAW;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int G = a.Hq / a.Hkv;

    if (w == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(shared_addr(&meta.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            barrier_init(PART_FULL + 8 * i, 1);
            barrier_init(PART_FREE + 8 * i, 9);        // the softmax and product warps
        }
        for (int i = 0; i < 2; ++i) {
            barrier_init(Q_FULL + 8 * i, 4);
            barrier_init(S_FULL + 8 * i, 1);
            barrier_init(P_FULL + 8 * i, 4);
            barrier_init(S_FREE + 8 * i, 4);
            barrier_init(PV_DONE + 8 * i, 1);
            barrier_init(K_FULL + 8 * i, 8);
            barrier_init(K_FREE + 8 * i, 1);
            barrier_init(V_FULL + 8 * i, 8);
            barrier_init(V_FREE + 8 * i, 1);
        }
        for (int i = 0; i < S::RAW; ++i) {
            barrier_init(RAW_FULL + 8 * i, 1);
            barrier_init(RAW_FREE + 8 * i, 8);
        }
        barrier_init(FINISHED, 1);
        if (a.starve) barrier_await(RAW_FULL, 16);     // (a self-test: bytes that nobody copies)
        meta.dead = 0;
    }
    if (QT == 1 && w == 17) {
        const int cut = cut_of<QT>(a);
        if (lane == 0) meta.cut = cut;
    }
    tmem_before_sync();
    __syncthreads();
    tmem_after_sync();
    const uint32_t tmem = meta.tmem;

    if (w < 8) {
        take_registers<REGS_SOFTMAX>();
        // ================================ softmax ======================================================
        const int g = w >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(w & 3) << 21);
        const uint32_t s_col = lanes + g * 128, o_col = lanes + S::O_COL + g * D, p_col = lanes + S::P_COL + g * S::P_STEP;
        uint8_t *const q_tile = smem + (QT == 2 ? g : 0) * S::QBYTES;
        const int my_row = (QT == 2 ? g * 128 : 0) + row;      // of the part
        uint32_t done = 0;             // this group's tiles so far
        uint32_t kv = 0;               // tiles so far
        // The next part: its queries go out, and its tiles are returned, or -1 after the last one.
        float factor = 0.f, next_factor = 0.f;
        auto take = [&](uint32_t part, float &factor) {
            wait_or_dead(PART_FULL + 8 * (part & 3), part >> 2 & 1, dead);
            const Part &p = meta.parts[part & 3];
            const int tiles = __shfl_sync(~0u, p.tiles, 0);
            // all that meet at a barrier below leave together
            const bool leave = tiles < 0 || *dead;
            if (QT == 1 ? group_any(1, 256, leave) : (bool)__any_sync(~0u, leave)) return -1;
            // queries: scaled by a power of two, so that the largest of a row is in [1, 2)
            {
                uint32_t qw[D / 2], most = 0;
                const int rr = p.row0 + min(my_row, p.rows - 1);       // (rows past the last are computed like it)
                const uint4 *src = reinterpret_cast<const uint4 *>((const T *)a.q + (long long)(p.q0 + rr / G) * a.q_stride +
                                                                   (p.h * G + rr % G) * D);
                if ((my_row & ~31) < p.rows) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 v = __ldg(src + i);
                        qw[4 * i] = v.x, qw[4 * i + 1] = v.y, qw[4 * i + 2] = v.z, qw[4 * i + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) qw[i] = 0;
                }
                // magnitudes of both types order as their bits do, NaN last
#pragma unroll
                for (int i = 0; i < D / 2; ++i) most = __vmaxu2(most, qw[i] & 0x7fff7fffu);
                const float2 tops = pair_of<T>(most);
                const float top = max_nan(tops.x, tops.y);
                const int e = min(max((int)(__float_as_uint(top) >> 23 & 255), 1), 253);
                const float down = copysignf(finite_or_nan(top, __uint_as_float((uint32_t)(254 - e) << 23)), a.scale_k);
                factor = factor_of(a.scale_k, __uint_as_float((uint32_t)e << 23));
                if (QT == 2 || (g == 0 && tiles > 0)) {        // (a piece without tiles hands over none)
                    if ((my_row & ~31) < p.rows)
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        uint32_t x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = pair_of<T>(qw[4 * i + k]);
                            x[k] = half_pair(f.x * down, f.y * down);
                        }
                        *reinterpret_cast<uint4 *>(q_tile + chunk_at(row, i, 128)) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(Q_FULL + 8 * g);
                }
            }
            return tiles;
        };
        int tiles = take(0, factor), next_tiles = -1;
        for (uint32_t part = 0; tiles >= 0; ++part, tiles = next_tiles, factor = next_factor) {
            const Part &p = meta.parts[part & 3];
            const int tile0 = p.tile0;
            const int2 see = sight(a, p, my_row);
            // every row of this group sees a tile whole if it lies between these
            int all_first, all_last;
            {
                const int2 x = sight(a, p, QT == 2 ? g * 128 : 0);
                const int2 y = sight(a, p, min(QT == 2 ? g * 128 + 127 : 127, p.rows - 1));
                all_first = y.x, all_last = x.y;
            }
            // a warp without rows leaves its lanes of Q and P as they are: they reach nothing but its lanes of O
            const bool no_rows = QT == 1 && (my_row & ~31) >= p.rows;
            float m = NOTHING, l = 0.f;
            bool far = false;          // some row's maximum is
            uint32_t nan_blocks = 0;
            int mine = 0;              // tiles of this part that this group has done
#pragma unroll 1
            for (int j = QT == 2 ? 0 : g; j < tiles; j += QT == 2 ? 1 : 2) {
                const int pos0 = (tile0 + j) * TT, ring = (kv + j) & 3;
                wait_or_dead(S_FULL + 8 * g, done & 1, dead);
                tmem_after_sync();
                if (no_rows) {
                    if (lane == 0) barrier_arrive(P_FULL + 8 * g);
                    ++done;
                    ++mine;
                    continue;
                }
                const uint4 miss = *reinterpret_cast<const uint4 *>(meta.missing[ring]);
                const uint4 nans = *reinterpret_cast<const uint4 *>(meta.nan_group[ring]);
                const bool any_nan = (nans.x | nans.y | nans.z | nans.w) != 0;
                const bool some = pos0 < all_first || pos0 + TT - 1 > all_last || (miss.x | miss.y | miss.z | miss.w) != 0;
                auto visible = [&](int c) -> uint32_t {        // of tokens 32 c .. 32 c + 31
                    const int lo = see.x - (pos0 + 32 * c), hi = see.y - (pos0 + 32 * c);
                    uint32_t v = hi < 0 ? 0u : hi >= 31 ? ~0u : (2u << hi) - 1;
                    v &= lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
                    const uint32_t gone = reinterpret_cast<const uint32_t *>(meta.missing[ring])[c];
                    return v & ~gone;
                };
                uint32_t x[TT];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_async(s_col + 32 * c, x + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_wait(x + 32 * c);
                if constexpr (S::EARLY) {
                    tmem_before_sync();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(S_FREE + 8 * g);
                }
                if (some) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t v = visible(c);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(v >> e & 1)) x[32 * c + e] = 0xff800000u;
                    }
                }
                float tops[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tops[c] = __uint_as_float(x[c]);
#pragma unroll
                    for (int e = c + 4; e < TT; e += 8)
                        tops[c] = max3(tops[c], __uint_as_float(x[e]), e + 4 < TT ? __uint_as_float(x[e + 4]) : -INFINITY);
                }
                const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
                if (__any_sync(~0u, (top - m) * factor > MOVE - HEADROOM)) {
                    const float to = fmaxf(m, top), keep = exp2_fast((m - to) * factor);
                    m = to;
                    far |= __any_sync(~0u, is_far(m, factor));
                    l *= keep;
                    if (mine > 0) {
                        wait_or_dead(PV_DONE + 8 * g, (done - 1) & 1, dead);
                        tmem_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t y[16];
                            tmem_ld16(o_col + 16 * c, y);
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
                            tmem_st16(o_col + 16 * c, y);
                        }
                    }
                }
                float add = offset_of(m, factor);
                if (far) {
                    add = HEADROOM;
#pragma unroll
                    for (int e = 0; e < TT; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) - m);
                }
                const uint64_t ff = pair_of_floats(factor, factor), aa = pair_of_floats(add, add);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        uint64_t u0, u1;
                        uint32_t *const z = x + 16 * c + e;
                        fma_pair(z[0], z[1], ff, aa);
                        fma_pair(z[2], z[3], ff, aa);
                        const float p0 = exp2_fast(__uint_as_float(z[0])), p1 = exp2_fast(__uint_as_float(z[1]));
                        const float p2 = exp2_fast(__uint_as_float(z[2])), p3 = exp2_fast(__uint_as_float(z[3]));
                        u0 = pair_of_floats(p0, p1), u1 = pair_of_floats(p2, p3);
                        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum0) : "l"(u0));
                        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum1) : "l"(u1));
                        pk[e / 2] = half_pair(p0, p1);
                        pk[e / 2 + 1] = half_pair(p2, p3);
                    }
                    if (S::EARLY && c == 0 && mine > 0) {      // the last weights have been read
                        wait_or_dead(PV_DONE + 8 * g, (done - 1) & 1, dead);
                        tmem_after_sync();
                    }
                    tmem_st8(p_col + 8 * c, pk);
                }
                l += (__uint_as_float((uint32_t)sum0) + __uint_as_float((uint32_t)(sum0 >> 32))) +
                     (__uint_as_float((uint32_t)sum1) + __uint_as_float((uint32_t)(sum1 >> 32)));
                if (any_nan) {                                 // NaN values: they reach the rows that see them
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t v = visible(c);
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            if (!meta.nan_group[ring][4 * c + i]) continue;
#pragma unroll 1
                            for (int blk = 0; blk < D / 16; ++blk)
                                if (v >> (8 * i) & meta.nan_value[ring][4 * c + i][blk]) nan_blocks |= 1u << blk;
                        }
                    }
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tmem_before_sync();
                __syncwarp();
                if (lane == 0) barrier_arrive(P_FULL + 8 * g);
                ++done;
                ++mine;
            }
            kv += tiles;
            if (mine > 0) wait_or_dead(PV_DONE + 8 * g, (done - 1) & 1, dead);
            tmem_after_sync();

            const float base = base_of(m, factor, l);
            const int rr = p.row0 + my_row;
            const size_t at_row = (size_t)(p.q0 + rr / G) * a.Hq + p.h * G + rr % G;
            if (QT == 2) {
                const float f = l == 0.f ? 0.f : 1.f / l;              // (apart from v_scale: their quotient may underflow)
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(o_col + 32 * c, x);
                    if (my_row < p.rows && !*dead) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            const bool bad = nan_blocks >> (2 * c + e / 16) & 1;
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float u = __uint_as_float(x[e + 2 * k]) * f * a.v_scale, v = __uint_as_float(x[e + 2 * k + 1]) * f * a.v_scale;
                                y[k] = bad ? 0x7fff7fffu : l == 0.f ? 0u : pack_of<T>(u, v);
                            }
                            *reinterpret_cast<uint4 *>((T *)a.o + at_row * D + 32 * c + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                if (my_row < p.rows && a.lse && !*dead) a.lse[at_row] = l == 0.f ? -INFINITY : (base + log2f(l)) * LN2;
                tmem_before_sync();
            } else {
                // both groups hold the same rows: each joins half of the channels
                meta.ml[g][row] = make_float2(base, l);
                meta.nan_row[g][row] = (uint8_t)nan_blocks;
                tmem_before_sync();
                group_sync(1, 256);
                tmem_after_sync();
                const float2 ml0 = meta.ml[0][row], ml1 = meta.ml[1][row];
                nan_blocks = meta.nan_row[0][row] | meta.nan_row[1][row];
                const float both = fmaxf(ml0.x, ml1.x);
                const float k0 = exp2_fast(ml0.x - both), k1 = exp2_fast(ml1.x - both), sum = ml0.y * k0 + ml1.y * k1;
                const bool split = p.pieces > 1;
                const float f = split ? 1.f : sum == 0.f ? 0.f : 1.f / sum, f0 = k0 * f, f1 = k1 * f;
                float *const partials = reinterpret_cast<float *>(a.ws + MAX_CTAS * 4);
                float *const my_part = partials + (size_t)(p.slot0 + p.piece) * S::PARTIAL;
#pragma unroll 1
                for (int c = no_rows ? D / 32 : g * (D / 64); c < (g + 1) * (D / 64); ++c) {
                    uint32_t x0[32], x1[32];
                    tmem_ld32_async(lanes + S::O_COL + 32 * c, x0);
                    tmem_ld32_async(lanes + S::O_COL + D + 32 * c, x1);
                    tmem_ld_wait(x0);
                    tmem_ld_wait(x1);
                    if (tiles < 2) {       // a group without a tile has made no O
#pragma unroll
                        for (int e = 0; e < 32; ++e) x0[e] = tiles < 1 ? 0 : x0[e], x1[e] = 0;
                    }
                    if (my_row >= p.rows || *dead) continue;
#pragma unroll
                    for (int e = 0; e < 32; ++e) x0[e] = __float_as_uint(fmaf(__uint_as_float(x0[e]), f0, __uint_as_float(x1[e]) * f1));
                    if (nan_blocks >> (2 * c) & 3) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (nan_blocks >> (2 * c + e / 16) & 1) x0[e] = 0x7fffffffu;
                    }
                    if (split) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            __stcg(reinterpret_cast<uint4 *>(my_part + row * D + 32 * c + e), make_uint4(x0[e], x0[e + 1], x0[e + 2], x0[e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = pack_of<T>(__uint_as_float(x0[e + 2 * k]) * a.v_scale, __uint_as_float(x0[e + 2 * k + 1]) * a.v_scale);
                            *reinterpret_cast<uint4 *>((T *)a.o + at_row * D + 32 * c + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                if (g == 0 && my_row < p.rows && !*dead) {
                    if (split) __stcg(reinterpret_cast<float2 *>(my_part + 128 * D + 2 * row), make_float2(both, sum));
                    else if (a.lse) a.lse[at_row] = sum == 0.f ? -INFINITY : (both + log2f(sum)) * LN2;
                }
                if (split) {
                    __threadfence();
                    group_sync(1, 256);
                    if (tid == 0) {
                        int *const counter = reinterpret_cast<int *>(a.ws) + p.slot0;
                        const bool last = atomicAdd(counter, 1) == p.pieces - 1;
                        if (last) *counter = 0;                // as the next call needs it
                        meta.last = last;
                    }
                    group_sync(1, 256);
                    if (*(volatile int *)&meta.last && !*dead) {
                        __threadfence();
                        // four times four channels a thread, so that many loads are on their way
                        constexpr int N = 4;
                        for (int i0 = tid; i0 < p.rows * (D / 4); i0 += N * 256) {
                            float to[N], total[N];
                            float4 v[N];
#pragma unroll
                            for (int k = 0; k < N; ++k) to[k] = LOWEST, total[k] = 0.f, v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                            for (int x = 0; x < p.pieces; ++x) {
                                const float *src = partials + (size_t)(p.slot0 + x) * S::PARTIAL;
#pragma unroll
                                for (int k = 0; k < N; ++k) {
                                    const int i = min(i0 + k * 256, p.rows * (D / 4) - 1);
                                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + 128 * D) + i / (D / 4));
                                    const float4 u = __ldcg(reinterpret_cast<const float4 *>(src) + i);
                                    const float up = fmaxf(to[k], ml.x), keep = exp2_fast(to[k] - up), add = exp2_fast(ml.x - up);
                                    to[k] = up;
                                    total[k] = total[k] * keep + ml.y * add;
                                    v[k].x = v[k].x * keep + u.x * add, v[k].y = v[k].y * keep + u.y * add;
                                    v[k].z = v[k].z * keep + u.z * add, v[k].w = v[k].w * keep + u.w * add;
                                }
                            }
#pragma unroll
                            for (int k = 0; k < N; ++k) {
                                const int i = i0 + k * 256, col = i / (D / 4), d = i % (D / 4) * 4;
                                if (col >= p.rows) continue;
                                const int orow = p.row0 + col;
                                const size_t at = (size_t)(p.q0 + orow / G) * a.Hq + p.h * G + orow % G;
                                const float fo = total[k] == 0.f ? 0.f : 1.f / total[k];
                                *reinterpret_cast<uint2 *>((T *)a.o + at * D + d) =
                                    total[k] == 0.f ? make_uint2(0, 0)
                                                    : make_uint2(pack_of<T>(v[k].x * fo * a.v_scale, v[k].y * fo * a.v_scale), pack_of<T>(v[k].z * fo * a.v_scale, v[k].w * fo * a.v_scale));
                                if (d == 0 && a.lse) a.lse[at] = total[k] == 0.f ? -INFINITY : (to[k] + log2f(total[k])) * LN2;
                            }
                        }
                    }
                }
                tmem_before_sync();
                group_sync(1, 256);    // both have read O, the maxima and sums
            }
            __syncwarp();
            if (lane == 0) barrier_arrive(PART_FREE + 8 * (part & 3));
            next_tiles = take(part + 1, next_factor);
        }
    } else if (w < 16) {
        give_registers<REGS_UNPACK>();
        // ================================ unpack =======================================================
        // A lane holds, of token 8 uw + lane / 4 of each half tile, a quarter of the channels of K and of V: all of a
        // tile's codes are in registers, and their stages free again, before the first is converted.
        constexpr int W = D / 32;                              // words of a lane
        const int uw = w - 8, c = lane & 3, tok = uw * 8 + (lane >> 2);
        const uint8_t *const codes = smem + S::RAW_AT + (tok >> 4) * L::BYTES;
        const int in_tile = tok & 15;
        const uint32_t base = shared_addr(smem);
        // V: row r of stored matrix m is the channel that lane quarter r / 2 put there
        const int am = lane >> 3, ac = lane >> 1 & 3;
        const int v_channel = 8 * W * ac + 2 * ((am + ac) & 3) + (lane & 1);
        uint32_t raw = 0, raw_parity = 0;
        for (uint32_t n = 0;; ++n) {                           // tiles
            const uint32_t stage = n & 1, round = n >> 1, ring = n & 3;
            uint32_t k[2][W], v[2][W], ks[2], vs[2], gone = 0;
            bool end = false;
#pragma unroll
            for (int box = 0; box < 2; ++box) {
                if (!wait_all(RAW_FULL + 8 * raw, raw_parity, dead, a.wait_ns)) goto unpacked;
                const int2 about = meta.raw_about[raw];        // tokens before the end; runs of 16 out of range
                end |= about.x < 0;
                const uint8_t *t = codes + raw * S::RAW_BYTES;
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(t + in_tile * 64 + c * 16);
                    const uint4 y = *reinterpret_cast<const uint4 *>(t + L::VC + in_tile * 64 + c * 16);
                    ks[box] = *reinterpret_cast<const uint16_t *>(t + L::KS + in_tile * 8 + c * 2);
                    vs[box] = t[L::VS + 2 * c * KV_TILE + in_tile] | (uint32_t)t[L::VS + (2 * c + 1) * KV_TILE + in_tile] << 8;
                    // lanes 2 and 3 of four take K's words in the order 2, 3, 0, 1: no bank conflicts below
                    k[box][0] = c & 2 ? x.z : x.x, k[box][1] = c & 2 ? x.w : x.y;
                    k[box][W - 2] = c & 2 ? x.x : x.z, k[box][W - 1] = c & 2 ? x.y : x.w;
                    v[box][0] = y.x, v[box][1] = y.y, v[box][W - 2] = y.z, v[box][W - 1] = y.w;
                    if (c & 2) ks[box] = __byte_perm(ks[box], 0, 0x4401);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(t + in_tile * 32 + c * 8);
                    const uint2 y = *reinterpret_cast<const uint2 *>(t + L::VC + in_tile * 32 + c * 8);
                    ks[box] = t[L::KS + in_tile * 4 + c];
                    vs[box] = t[L::VS + c * KV_TILE + in_tile];
                    k[box][0] = x.x, k[box][1] = x.y;
                    v[box][0] = y.x, v[box][1] = y.y;
                }
                const bool away = about.y >> (tok >> 4) & 1;
                gone |= (uint32_t)away << box;
                if (away || tok >= about.x) vs[box] = 0;       // nothing that no row sees goes into a product
                __syncwarp();
                if (lane == 0) barrier_arrive(RAW_FREE + 8 * raw);
                if (++raw == S::RAW) raw = 0, raw_parity ^= 1;
            }
            if (__any_sync(~0u, end || *dead)) break;
            // what the softmax has to know of these tokens: a page out of range, NaN values (their scales: 0 here)
            const uint32_t both = vs[0] | vs[1] << 16, nan4 = (((both & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
            const bool any = __any_sync(~0u, nan4 != 0);
            if (round > 0) wait_or_dead(K_FREE + 8 * stage, (round - 1) & 1, dead);
            if (any) {
#pragma unroll
                for (int box = 0; box < 2; ++box) {
                    const uint32_t n0 = __ballot_sync(~0u, nan4 >> (16 * box) & 1), n1 = __ballot_sync(~0u, nan4 >> (16 * box + 8) & 1);
                    if (lane < 4) {
                        uint32_t x0 = 0, x1 = 0;
                        for (int i = 0; i < 8; ++i) {
                            x0 |= (n0 >> (4 * i + c) & 1) << i;
                            x1 |= (n1 >> (4 * i + c) & 1) << i;
                        }
                        meta.nan_value[ring][box * 8 + uw][D == 128 ? 2 * c : c] = (uint8_t)x0;
                        if (D == 128) meta.nan_value[ring][box * 8 + uw][2 * c + 1] = (uint8_t)x1;
                    }
                }
                vs[0] &= ~(nan4 * 255u);
                vs[1] &= ~((nan4 >> 16) * 255u);
            }
            if (lane < 2) {                                    // a lane a half tile
                meta.nan_group[ring][lane * 8 + uw] = any;
                meta.missing[ring][lane * 8 + uw] = gone >> lane & 1 ? 255 : 0;
            }
#pragma unroll
            for (int box = 0; box < 2; ++box) {
                const uint32_t two = e4m3x2_to_f16x2(ks[box]);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const int chunk = W * c + (D == 128 ? i ^ (c & 2) : i);
                    uint32_t f[4];
                    e2m1x8_to_f16x2(k[box][i], f);
                    *reinterpret_cast<uint4 *>(smem + S::K_AT + stage * S::KBYTES + chunk_at(box * BOX + tok, chunk, TT)) =
                        make_uint4(hmul2_by(f[0], two, i >= 2), hmul2_by(f[1], two, i >= 2), hmul2_by(f[2], two, i >= 2), hmul2_by(f[3], two, i >= 2));
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) barrier_arrive(K_FULL + 8 * stage);

            if (round > 0) wait_or_dead(V_FREE + 8 * stage, (round - 1) & 1, dead);
            const uint32_t v_tile = base + S::V_AT + stage * S::KBYTES;
#pragma unroll
            for (int box = 0; box < 2; ++box) {
                const uint32_t two = e4m3x2_to_f16x2(vs[box]);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    uint32_t f[4];
                    e2m1x8_to_f16x2(__funnelshift_r(v[box][i], v[box][i], 8 * c), f);
                    store_transposed(v_tile + chunk_at(v_channel + 8 * i, box * 8 + uw, D), hmul2_by(f[0], two, i >= 2), hmul2_by(f[1], two, i >= 2),
                                     hmul2_by(f[2], two, i >= 2), hmul2_by(f[3], two, i >= 2));
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) barrier_arrive(V_FULL + 8 * stage);
        }
    unpacked:;
    } else {
        give_registers<REGS_OTHER>();
        if (w == 16) {
            // ============================ products =====================================================
            constexpr uint32_t ID_S = idesc_f16(128, TT), ID_O = idesc_f16(128, D);
            const uint32_t base = shared_addr(smem);
            uint32_t done[2] = {0, 0}, kv = 0, queries = 0;
            for (uint32_t part = 0;; ++part) {
                wait_or_dead(PART_FULL + 8 * (part & 3), part >> 2 & 1, dead);
                const int tiles = __shfl_sync(~0u, meta.parts[part & 3].tiles, 0);
                if (__any_sync(~0u, tiles < 0 || *dead)) break;
                if (lane == 0) barrier_arrive(PART_FREE + 8 * (part & 3));
                auto scores = [&](int g, int j, bool frees) {
                    const uint32_t n = kv + j;
                    const uint64_t dq = tile_desc(base + (QT == 2 ? g : 0) * S::QBYTES), dk = tile_desc(base + S::K_AT + (n & 1) * S::KBYTES);
                    tmem_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < D / 16; ++s) {
                            const uint64_t at = (uint64_t)(((s >> 2) * 16384 + (s & 3) * 32) >> 4);
                            mma_f16_ss(tmem + g * 128, dq + at, dk + at, ID_S, s > 0);
                        }
                        mma_done(S_FULL + 8 * g);
                        if (frees) mma_done(K_FREE + 8 * (n & 1));
                    }
                    __syncwarp();
                };
                auto values = [&](int g, int j, bool first, bool frees) {
                    const uint32_t n = kv + j;
                    wait_or_dead(P_FULL + 8 * g, done[g] & 1, dead);
                    ++done[g];
                    const uint64_t dv = tile_desc(base + S::V_AT + (n & 1) * S::KBYTES);
                    tmem_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < TT / 16; ++s) {
                            const uint64_t at = (uint64_t)(((s >> 2) * D * 128 + (s & 3) * 32) >> 4);
                            mma_f16_ts(tmem + S::O_COL + g * D, tmem + S::P_COL + g * S::P_STEP + 8 * s, dv + at, ID_O, s > 0 || !first);
                        }
                        mma_done(PV_DONE + 8 * g);
                        if (frees) mma_done(V_FREE + 8 * (n & 1));
                    }
                    __syncwarp();
                };
                // the weights of the group's last tile have been read
                auto p_wait = [&](int g) {
                    if (!S::OWN_P) wait_or_dead(PV_DONE + 8 * g, (done[g] - 1) & 1, dead);
                };
                auto k_wait = [&](int j) { wait_or_dead(K_FULL + 8 * ((kv + j) & 1), (kv + j) >> 1 & 1, dead); };
                auto v_wait = [&](int j) { wait_or_dead(V_FULL + 8 * ((kv + j) & 1), (kv + j) >> 1 & 1, dead); };
                if (QT == 2 || tiles > 0) wait_or_dead(Q_FULL, queries & 1, dead);
                if (QT == 2) {
                    wait_or_dead(Q_FULL + 8, queries & 1, dead);
                    k_wait(0);
                    scores(0, 0, false);
                    scores(1, 0, true);
#pragma unroll 1
                    for (int j = 0; j < tiles; ++j) {
                        const bool more = j + 1 < tiles;
                        if constexpr (S::EARLY) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                if (more) {
                                    wait_or_dead(S_FREE + 8 * g, done[g] & 1, dead);
                                    if (g == 0) k_wait(j + 1);
                                    scores(g, j + 1, g == 1);
                                }
                                if (g == 0) v_wait(j);
                                values(g, j, j == 0, g == 1);
                            }
                            continue;
                        }
                        v_wait(j);
                        values(0, j, j == 0, false);
                        if (more) {
                            k_wait(j + 1);
                            p_wait(0);
                            scores(0, j + 1, false);
                        }
                        values(1, j, j == 0, true);
                        if (more) {
                            p_wait(1);
                            scores(1, j + 1, true);
                        }
                    }
                } else {
                    for (int j = 0; j < min(tiles, 2); ++j) {
                        k_wait(j);
                        scores(j, j, true);
                    }
#pragma unroll 1
                    for (int j = 0; j < tiles; ++j) {
                        v_wait(j);
                        values(j & 1, j, j < 2, true);
                        if (j + 2 < tiles) {
                            k_wait(j + 2);
                            p_wait(j & 1);
                            scores(j & 1, j + 2, true);
                        }
                    }
                }
                kv += tiles;
                queries += QT == 2 || tiles > 0;
            }
            if (elect_one()) {
                mma_done(FINISHED);
                barrier_wait(FINISHED, 0);
            }
            __syncwarp();
        } else if (w == 17) {
            // ============================ load =========================================================
            int *const counters = reinterpret_cast<int *>(a.ws);
            Walker<QT> walk;
            walk.start(a, QT == 1 ? meta.cut : 0);
            uint32_t raw = 0, raw_round = 0;
            for (uint32_t part = 0;; ++part) {
                int pi = 0;
                if (lane == 0) pi = atomicAdd(counters + NEXT_PART, 1);
                pi = __shfl_sync(~0u, pi, 0);
                Part p;
                const bool found = walk.find(a, pi, p) && !__any_sync(~0u, *dead);
                if (part >= 4 && !wait_all(PART_FREE + 8 * (part & 3), ((part >> 2) - 1) & 1, dead)) break;
                if (lane == 0) {
                    if (found) meta.parts[part & 3] = p;
                    else meta.parts[part & 3].tiles = -1;
                    barrier_arrive(PART_FULL + 8 * (part & 3));
                }
                __syncwarp();
                if (!found) break;
                const int32_t *const pages = a.page_table + (size_t)p.b * a.max_pages;
                const int boxes = 2 * p.tiles, from = p.tile0 * TT;
                // a lane looks up one run of 16 tokens of each 8 stages, and asks for it when its stage's turn comes
                const int runs_in = min(boxes * 4, (max(p.len - from, 0) + KV_TILE - 1) / KV_TILE);    // that are to be read
                auto look = [&](int i) {               // the page of the part's i-th run
                    return i < runs_in ? pages[((long long)from + (long long)i * KV_TILE) >> a.page_shift] : -1;
                };
                const bool one_copy = a.page_shift >= 6;       // a stage lies in one page
                int then = look(lane);
                for (int i0 = 0; i0 < boxes; i0 += 8) {
                    const int page = then;
                    then = look((i0 + 8) * 4 + lane);
                    const bool ok = page >= 0 && page < a.num_pages;
                    const uint32_t oks = __ballot_sync(~0u, ok), gone = __ballot_sync(~0u, !ok && i0 * 4 + lane < runs_in);
                    if (gone && lane == 0) report(a.err, DEVERR_PAGE_RANGE);
                    const int in_page = (from + (i0 * 4 + lane) * KV_TILE) & ((1 << a.page_shift) - 1);
                    const uint8_t *const src = a.pool + ((((size_t)page * a.Hkv + p.h) << (a.page_shift - 4)) + (in_page >> 4)) * L::BYTES;
                    const int mine = lane & 3, left = p.len - from - i0 * BOX;
                    for (int i = 0; i < min(8, boxes - i0); ++i) {
                        if (raw_round > 0 && !wait_all(RAW_FREE + 8 * raw, (raw_round - 1) & 1, dead)) goto gave_up;
                        const int runs = __popc(oks >> (4 * i) & 15u);
                        if (lane == 4 * i) {
                            meta.raw_about[raw] = make_int2(min(max(left - i * BOX, 0), BOX), gone >> (4 * i) & 15u);
                            barrier_expect(RAW_FULL + 8 * raw, runs * L::BYTES);
                        }
                        __syncwarp();
                        if (lane >> 2 == i && ok && (mine == 0 || !one_copy))
                            bulk_copy(smem + S::RAW_AT + raw * S::RAW_BYTES + mine * L::BYTES, src, one_copy ? runs * L::BYTES : L::BYTES,
                                      RAW_FULL + 8 * raw);
                        if (++raw == S::RAW) raw = 0, ++raw_round;
                    }
                }
            }
        gave_up:
            // the end, for the unpacking warps; the last CTA leaves the counters as the next call needs them
            for (int i = 0; i < 2; ++i) {              // (they look at two stages at a time)
                if (raw_round > 0 && !wait_all(RAW_FREE + 8 * raw, (raw_round - 1) & 1, dead)) break;
                if (lane == 0) {
                    meta.raw_about[raw] = make_int2(-1, 0);
                    barrier_arrive(RAW_FULL + 8 * raw);
                }
                if (++raw == S::RAW) raw = 0, ++raw_round;
            }
            if (lane == 0) {
                meta.asked = make_uint2(raw, raw_round);
                if (atomicAdd(counters + CTAS_DONE, 1) == (int)gridDim.x - 1) {
                    counters[NEXT_PART] = 0;
                    counters[CTAS_DONE] = 0;
                }
            }
        }
    }

    tmem_before_sync();
    __syncthreads();
    if (w == 17 && *dead) {                            // the copies that were asked for may still be on their way
        const uint2 upto = meta.asked;
        for (uint32_t i = 0; i < S::RAW; ++i)
            if (i < upto.x || upto.y > 0) barrier_wait_for(RAW_FULL + 8 * i, (i < upto.x ? upto.y : upto.y - 1) & 1, a.wait_ns);
        if (lane == 0) report(a.err, DEVERR_TIMEOUT);
    }
    if (w == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int D, int QT, typename T>
cudaError_t launch_tile_attention(const KvAttentionArgs &a, cudaStream_t s) {
    using Sh = TileShape<D, QT>;
    constexpr int SMEM = Sh::META + sizeof(TileMeta);
    static_assert(SMEM <= 232448, "shared memory");
    static_assert((size_t)MAX_CTAS * 4 + MAX_SLOTS * (size_t)Sh::PARTIAL * 4 <= KDA_KV4_WORKSPACE, "workspace");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(tile_attention_kernel<D, QT, T>), SMEM, done);
    if (e != cudaSuccess) return e;
    tile_attention_kernel<D, QT, T><<<SMS, TILE_THREADS, SMEM, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace kda
