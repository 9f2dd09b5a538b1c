// The paged 4-bit key/value cache: its layout, and the conversions of its types.
//
// A pool is uint8 [num_pages][Hkv][P / 16][18 D]: within a page and head, tiles
// of 16 tokens, each
//
//     K codes [16][D/2] | K scales [16][D/16] | V codes [16][D/2] | V scales [D/16][16]
//
// Codes are e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), the even
// channel in the low nibble; scales are e4m3, one for 16 channels of a token.
// A value is code x scale x tensor scale, and code x scale has at most 2 + 4
// significant bits: exact in fp16, bf16 and fp32.
//
// A tile is one contiguous block, so any run of 16 tokens is one bulk copy
// whatever the page size, and a page of one layer is one contiguous block for
// copies.  V's scales are stored by block so that one 32-bit load gives the
// scales of four neighbouring tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

enum { DEVERR_PAGE_RANGE = 32, DEVERR_PAGES = 64 };

constexpr int KV_TILE = 16;     // tokens
template <int D>
struct KvTile {
    static constexpr int KC = 0, KS = 8 * D, VC = 9 * D, VS = 17 * D, BYTES = 18 * D;
    static constexpr int BLOCKS = D / 16;
};

// Two e2m1 codes (a byte, low nibble first) as fp16.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
    uint32_t r;
    asm("{\n .reg .b8 b, x, y, z;\n mov.b32 {b, x, y, z}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}" : "=r"(r) : "r"(byte));
    return r;
}
// The four bytes of a word, each two e2m1 codes, as fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Two e4m3 scales (the low 16 bits) as fp16; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
    uint32_t r;
    asm("{\n .reg .b16 p, q;\n mov.b32 {p, q}, %1;\n cvt.rn.f16x2.e4m3x2 %0, p;\n}" : "=r"(r) : "r"(pair));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}
// To e2m1, nearest even, saturating; lo in the low nibble.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n .reg .b8 b;\n .reg .b16 z;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u16.u8 z, b;\n cvt.u32.u16 %0, z;\n}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// To e4m3, nearest even, saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The request b of B with cu[b] <= t < cu[b + 1], or -1; a whole warp calls it, with its lanes' t ascending.
// 32 places are looked at in one step, so that a search is two or three loads deep.
__device__ __forceinline__ int owner_of(const int32_t *cu, int B, int t) {
    const int lane = threadIdx.x & 31, t0 = __shfl_sync(~0u, t, 0);
    int lo = 0, hi = B;          // the first b in [lo, hi] with cu[b + 1] > t0, hi standing for none
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;     // the last of each 32nd
        const uint32_t past = __ballot_sync(~0u, at >= hi || cu[at + 1] > t0);
        const int k = past ? __ffs(past) - 1 : 32;
        hi = min(lo + (k + 1) * step - 1, hi);
        lo += k * step;
        if (step == 1) break;
    }
    lo = min(lo, B);
    while (lo < B && cu[lo + 1] <= t) ++lo;
    return lo < B && cu[lo] <= t ? lo : -1;
}

// The owner of token t of T and what is known of it; a whole warp calls it, with its lanes' t ascending.  One request is
// guessed, the right one where all have as many tokens (single tokens among them), and what is asked of it is asked for
// beside the check: one round of loads, not the three or four of a search.
struct Owner {
    int b, q0, end, more;                  // request or -1, its first token and the one behind its last, per[b]
};
__device__ __forceinline__ Owner owner_with(const int32_t *cu, const int32_t *per, int B, int T, int t) {
    Owner o;
    o.b = min((int)(((float)t + 0.5f) * ((float)B / (float)T)), B - 1);        // (0 <= t; off by one at worst, which is looked for)
    o.q0 = cu[o.b], o.end = cu[o.b + 1], o.more = per[o.b];
    if (!__all_sync(~0u, t >= T || (o.q0 <= t && t < o.end))) {
        o.b = owner_of(cu, B, t);
        if (o.b >= 0) o.q0 = cu[o.b], o.end = cu[o.b + 1], o.more = per[o.b];
    }
    if (t >= T) o.b = -1;
    return o;
}

}  // namespace kda
