// What the calls that write and read back the 4-bit cache share: where a token
// lies, and how 16 channels of it become codes and a scale:
//     s = e4m3(max|x| / 6),   code = e2m1(x / s)   (0 where s = 0)
//
// The quotients are products with a reciprocal, rounded to 18 bits.  What comes of
// them changes only at ties of the two small types, values of at most 5 bits: an
// exact quotient of x (8 or 11 bits) that is no tie is at least 2^-16 of it away
// from one, and the product is off by less than 2^-22, so rounding to 18 bits puts
// ties on themselves and takes nothing across.
#pragma once

#include "kda_kv4.cuh"

namespace kda {

__device__ __forceinline__ void unpack16(const uint4 &w, float *x, __nv_bfloat16) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack16(const uint4 &w, float *x, __half) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = f16x2_to_float2(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ float to_18_bits(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x20u) & ~0x3fu);
}

// The scale (its byte) of a block whose largest magnitude is top, and what its values are multiplied by to be codes.
__device__ __forceinline__ uint32_t scale_of(float top, float &one_over) {
    const uint32_t sb = to_e4m3(isnan(top) ? top : to_18_bits(top * (1.f / 6.f)));
    one_over = sb != 0 ? __frcp_rn(f16x2_to_float2(e4m3x2_to_f16x2(sb)).x) : 0.f;
    return sb;
}
// Eight values as codes; sb is their scale's byte.
__device__ __forceinline__ uint32_t codes_of(const float *x, uint32_t sb, float one_over) {
    uint32_t code = 0;
    if (sb != 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code |= to_e2m1x2(to_18_bits(x[2 * i] * one_over), to_18_bits(x[2 * i + 1] * one_over)) << (8 * i);
    }
    return code;
}

// Channels 16 blk .. 16 blk + 15 of token tok of a tile, as V (side 1) or K; x is what was given, of 8 or 11 bits, and
// inv the reciprocal of the tensor scale, a power of two.
template <int D>
__device__ __forceinline__ void store_block(uint8_t *tile, int tok, int blk, int side, float (&x)[16], float inv) {
    using L = KvTile<D>;
    float top = 0.f, one_over;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] *= inv;
        top = max_nan(top, fabsf(x[i]));
    }
    const uint32_t sb = scale_of(top, one_over);
    *reinterpret_cast<uint2 *>(tile + (side ? L::VC : L::KC) + tok * (D / 2) + blk * 8) =
        make_uint2(codes_of(x, sb, one_over), codes_of(x + 8, sb, one_over));
    tile[side ? L::VS + blk * KV_TILE + tok : L::KS + tok * L::BLOCKS + blk] = (uint8_t)sb;
}

}  // namespace kda
