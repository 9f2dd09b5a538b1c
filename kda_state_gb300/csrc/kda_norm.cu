// Residual addition and RMS norm in one pass, with the output in the type or in 8 bits.
//
//     h = x + residual, rounded to the type      (the new residual; h = x where there is none)
//     y = h w / sqrt(mean h^2 + eps)
// Output y, or e4m3 codes with scales of a row or of 128 channels: s = max|y| / 448, code = e4m3(y / s), 0 where s = 0.
// With r = 1 / sqrt(..) the same for a row, max|y| = r max|h w| and y / s = h w (448 / max|h w|): the row's sum and its
// maximum are taken together, with one exchange between threads, and codes do not wait for r.  That holds while the products
// and the scale are normal numbers; a row or block where they are not (faint or zero, NaN, products past fp32) goes by y.
//
// A row is one warp's or one CTA's, in registers from its one read on: bound by HBM (bf16: 4 bytes read, 3 or 4 written a
// channel), and by the launch and two round trips for a row alone.  16384 rows of 8192 channels with a scale for 128: 139 us,
// 6.8 TB/s (the copy bandwidth measured is 6.7; a twentieth of the bytes stays in L2); 5003 rows of 2560 in fp16: 17.2 us, 6.0
// TB/s; one row: 3.1 us.
#include "kda_async.cuh"
#include "kda_internal.h"
#include "kda_kv4_store.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr float TOP = 448.f;           // the largest e4m3

template <typename T> struct Vec8;     // eight channels
template <> struct Vec8<__nv_bfloat16> { uint4 w; };
template <> struct Vec8<__half> { uint4 w; };
template <> struct Vec8<float> { float4 a, b; };

template <typename T>
__device__ __forceinline__ void unpack8(const Vec8<T> &v, float (&x)[8]) { unpack16(v.w, x, T()); }
__device__ __forceinline__ void unpack8(const Vec8<float> &v, float (&x)[8]) {
    x[0] = v.a.x, x[1] = v.a.y, x[2] = v.a.z, x[3] = v.a.w, x[4] = v.b.x, x[5] = v.b.y, x[6] = v.b.z, x[7] = v.b.w;
}
template <typename T>
__device__ __forceinline__ void pack8(const float (&x)[8], Vec8<T> &v) {
    v.w = make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
}
__device__ __forceinline__ void pack8(const float (&x)[8], Vec8<float> &v) {
    v.a = make_float4(x[0], x[1], x[2], x[3]), v.b = make_float4(x[4], x[5], x[6], x[7]);
}
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T *p) { return *reinterpret_cast<const Vec8<T> *>(p); }
template <typename T>
__device__ __forceinline__ void store8(T *p, const Vec8<T> &v) { *reinterpret_cast<Vec8<T> *>(p) = v; }

// To e4m3, lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Whether codes are h w (448 / top), top the largest |h w|, y = r top: within [2^-100, 2^125] no product that counts has lost
// bits and the factor is finite, within [2^-117, FLT_MAX] the scale y / 448 has all of its bits.  False for NaN.
__device__ __forceinline__ bool by_products(float top, float y) {
    return __float_as_uint(top) - 0x0d800000u <= 0x7e000000u - 0x0d800000u && __float_as_uint(y) - 0x05000000u < 0x7f800000u - 0x05000000u;
}
// The scale of a largest |y|; NaN for an infinity, which no scale brings into range.
__device__ __forceinline__ float scale_of_y(float top) { return isinf(top) ? __uint_as_float(0x7fffffffu) : top / TOP; }

// The 8-bit output of a row, or with scales of 128 channels of a warp's part of it, by y itself.  h is read again (a thread
// its own channels), as this is rare: faint or zero rows and blocks, NaN, products past fp32.
template <typename T, int WARPS, int N>
__device__ __noinline__ void codes_of_y(const AddNormArgs &a, int row, float r) {
    constexpr int THREADS = 32 * WARPS;
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, vectors = a.C / 8;
    auto y_of = [&](int i, float (&y)[8]) {
        const int c = tid + i * THREADS;
        float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, top = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = 0.f;
        if (c < vectors) {
            Vec8<T> v = load8(a.sum ? (const T *)a.sum + row * a.sum_stride + c * 8 : (const T *)a.x + row * a.x_stride + c * 8);
            unpack8(v, y);
            if (a.residual && !a.sum) {
                unpack8(load8((const T *)a.residual + row * a.residual_stride + c * 8), g);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] += g[k];
                pack8(y, v);
                unpack8(v, y);
            }
            unpack8(load8((const T *)a.w_norm + c * 8), g);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = y[k] * r * g[k], top = max_nan(top, fabsf(y[k]));
        return c < vectors ? top : 0.f;    // (0 r is NaN where r is infinite)
    };
    const bool by_block = a.mode == KDA_NORM_E4M3_BLOCK;
    float y[8], s = 0.f;
    if (!by_block) {
        float t = 0.f;
#pragma unroll 1
        for (int i = 0; i < N; ++i) t = max_nan(t, y_of(i, y));
#pragma unroll
        for (int o = 16; o; o >>= 1) t = max_nan(t, __shfl_xor_sync(~0u, t, o));
        if constexpr (WARPS > 1) {
            __shared__ float part[WARPS];
            if (lane == 0) part[threadIdx.x >> 5] = t;
            __syncthreads();
            t = lane < WARPS ? part[lane] : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) t = max_nan(t, __shfl_xor_sync(~0u, t, o));
        }
        s = scale_of_y(t);
        if (tid == 0) a.scales[row] = s;
    }
    const int blocks = (a.C + 127) / 128;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        const int c = tid + i * THREADS;
        float t = y_of(i, y);
        if (by_block) {
#pragma unroll
            for (int o = 8; o; o >>= 1) t = max_nan(t, __shfl_xor_sync(~0u, t, o));
            s = scale_of_y(t);
            if ((lane & 15) == 0 && c < vectors) a.scales[(size_t)row * blocks + c / 16] = s;
        }
        if (c >= vectors) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = s == 0.f ? 0.f : y[k] / s;
        *reinterpret_cast<uint2 *>((uint8_t *)a.out + (size_t)row * a.C + c * 8) =
            make_uint2(to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16, to_e4m3x2(y[4], y[5]) | to_e4m3x2(y[6], y[7]) << 16);
    }
}

// WARPS warps a row, N vectors of 8 channels a thread.
template <typename T, int WARPS, int N>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS) add_rmsnorm_kernel(const __grid_constant__ AddNormArgs a) {
    constexpr int ROWS = WARPS == 1 ? 4 : 1, THREADS = 32 * WARPS;
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x * ROWS + (WARPS == 1 ? w : 0);
    wait_for_earlier_kernels();
    let_later_kernels_in();
    if (row >= a.tokens) return;
    const int vectors = a.C / 8;
    const T *const x_at = (const T *)a.x + row * a.x_stride, *const w_at = (const T *)a.w_norm;
    const T *const r_at = (const T *)a.residual + row * a.residual_stride;
    Vec8<T> xv[N], rv[N], wv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = tid + i * THREADS;
        if (c < vectors) {
            xv[i] = load8(x_at + c * 8);
            if (a.residual) rv[i] = load8(r_at + c * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (tid + i * THREADS < vectors) wv[i] = load8(w_at + (tid + i * THREADS) * 8);
    float sum = 0.f, top = 0.f, block_top[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = tid + i * THREADS;
        block_top[i] = 0.f;
        if (c < vectors) {
            float h[8], g[8];
            unpack8(xv[i], h);
            if (a.residual) {
                unpack8(rv[i], g);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[k] += g[k];
                pack8(h, xv[i]);
                if (a.sum) store8((T *)a.sum + row * a.sum_stride + c * 8, xv[i]);
                unpack8(xv[i], h);
            }
            unpack8(wv[i], g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum = fmaf(h[k], h[k], sum);
                block_top[i] = max_nan(block_top[i], fabsf(h[k] * g[k]));
            }
        }
        top = max_nan(top, block_top[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        top = max_nan(top, __shfl_xor_sync(~0u, top, o));
    }
    if constexpr (WARPS > 1) {
        __shared__ float2 part[WARPS];
        if (lane == 0) part[w] = make_float2(sum, top);
        __syncthreads();
        const float2 p = lane < WARPS ? part[lane] : make_float2(0.f, 0.f);
        sum = p.x, top = p.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(~0u, sum, o);
            top = max_nan(top, __shfl_xor_sync(~0u, top, o));
        }
    }
    const float r = rsqrtf(sum / (float)a.C + a.eps);
    if (a.mode == KDA_NORM_TYPE) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = tid + i * THREADS;
            if (c >= vectors) continue;
            float h[8], g[8];
            unpack8(xv[i], h);
            unpack8(wv[i], g);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = h[k] * r * g[k];
            pack8(h, xv[i]);
            store8((T *)a.out + (size_t)row * a.C + c * 8, xv[i]);
        }
        return;
    }
    const bool by_block = a.mode == KDA_NORM_E4M3_BLOCK;
    bool plain = by_products(top, r * top);            // (the same for all of the row's threads)
    if (by_block) {
        plain = true;
#pragma unroll
        for (int i = 0; i < N; ++i) {      // 16 neighbouring lanes hold a block
#pragma unroll
            for (int o = 8; o; o >>= 1) block_top[i] = max_nan(block_top[i], __shfl_xor_sync(~0u, block_top[i], o));
            plain = plain && (tid + i * THREADS >= vectors || by_products(block_top[i], r * block_top[i]));
        }
        plain = __all_sync(~0u, plain);
    }
    if (!plain) return codes_of_y<T, WARPS, N>(a, row, r);
    float s = r * top / TOP, per = TOP / top;
    if (!by_block && tid == 0) a.scales[row] = s;
    const int blocks = (a.C + 127) / 128;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = tid + i * THREADS;
        if (c >= vectors) continue;
        if (by_block) {
            s = r * block_top[i] / TOP, per = TOP / block_top[i];
            if ((lane & 15) == 0) a.scales[(size_t)row * blocks + c / 16] = s;
        }
        float h[8], g[8];
        unpack8(xv[i], h);
        unpack8(wv[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = h[k] * g[k] * per;
        *reinterpret_cast<uint2 *>((uint8_t *)a.out + (size_t)row * a.C + c * 8) =
            make_uint2(to_e4m3x2(h[0], h[1]) | to_e4m3x2(h[2], h[3]) << 16, to_e4m3x2(h[4], h[5]) | to_e4m3x2(h[6], h[7]) << 16);
    }
}

template <typename T, int WARPS, int N>
cudaError_t go(const AddNormArgs &a, cudaStream_t s) {
    constexpr int ROWS = WARPS == 1 ? 4 : 1;
    return launch_early(add_rmsnorm_kernel<T, WARPS, N>, dim3(((unsigned)a.tokens + ROWS - 1) / ROWS), dim3(WARPS == 1 ? 128 : 32 * WARPS), 0, s, a);
}

template <typename T>
cudaError_t launch(const AddNormArgs &a, cudaStream_t s) {
    // A warp a row while its lanes hold it in four vectors, then as many warps as that takes: the loads of a row are all in
    // flight at once, and what rows share is done by few warps.  Measured with scales of 128, us for 2^27 channels in bf16 and
    // for one row, warps x vectors: 512 channels 1 x 2 141 and 2.0, 2 x 1 264 and 1.7; 1024 1 x 4 135 and 2.7, 2 x 2 139 and
    // 2.0, 4 x 1 164 and 1.7; 2048 4 x 2 140 and 2.1, 2 x 4 139 and 2.7, 8 x 1 166 and 1.7; 4096 4 x 4 141 and 2.8, 8 x 2 142
    // and 2.3, 16 x 4 298 and 2.5; 8192 8 x 4 140 and 3.1, 16 x 2 147 and 2.6; 16384 16 x 4 147 and 3.9, 32 x 2 191 and 3.7.
    const int v = a.C / 8;
    if (v <= 32) return go<T, 1, 1>(a, s);
    if (v <= 64) return go<T, 1, 2>(a, s);
    if (v <= 128) return go<T, 1, 4>(a, s);
    if (v <= 256) return go<T, 4, 2>(a, s);
    if (v <= 512) return go<T, 4, 4>(a, s);
    if (v <= 1024) return go<T, 8, 4>(a, s);
    if (v <= 2048) return go<T, 16, 4>(a, s);
    return go<T, 32, 4>(a, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs &a, cudaStream_t s) {
    if (a.dt == KDA_DTYPE_BF16) return launch<__nv_bfloat16>(a, s);
    if (a.dt == KDA_DTYPE_FP16) return launch<__half>(a, s);
    return launch<float>(a, s);
}

}  // namespace kda
