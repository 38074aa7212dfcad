// quantize_tokens.hip -- hidden states to 8- and 4-bit codes with one scale per
// token, the residual sum and the norm before them in the same pass; and back; for gfx950.
//
// The norm's factor 1 / sqrt(mean + eps) is common to a token, so it cancels in
// y_k / max |y| and the codes depend on h * weight alone: two fp16 factors, whose
// product fp32 holds exactly. A code is the rounded quotient y L / m of exact numbers;
// it is found in fp32 and, where that lies within 10^-4 of a border between two codes,
// decided by comparing 2 L |y| with (2 k + 1) m, both exact in fp64 (at most 30 bits).
// So codes do not depend on the order of any sum, and equal the definition's.
//
// One pass: a token's values stay in registers between the sums and the codes (up to
// 16384 channels; longer tokens are read twice).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "bitmap_spmm.h"
#include "device_common.h"

namespace {

typedef uint32_t qt_u4 __attribute__((ext_vector_type(4)));
typedef uint32_t qt_u2 __attribute__((ext_vector_type(2)));
typedef _Float16 qt_h8 __attribute__((ext_vector_type(8)));

struct QtArgs {
    const uint16_t *x, *residual, *weight;
    uint16_t *hidden, *x16;
    int64_t xs, rs, hs, x16s, cs;
    float *scale;
    uint8_t *codes;
    int64_t n;
    int K, K16;             // K16: channels with the zeroed ones behind them
    float eps;
};

template <bool VEC>
__device__ __forceinline__ qt_h8 qt_load(const uint16_t *p, int k, int K) {
    if constexpr (VEC) return __builtin_bit_cast(qt_h8, *reinterpret_cast<const qt_u4 *>(p + k));
    qt_h8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < K ? __builtin_bit_cast(_Float16, p[k + e]) : (_Float16)0.0f;
    return v;
}

template <bool VEC>
__device__ __forceinline__ void qt_store(uint16_t *p, int k, int K, qt_h8 v) {
    if constexpr (VEC) {
        *reinterpret_cast<qt_u4 *>(p + k) = __builtin_bit_cast(qt_u4, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const _Float16 f = v[e];      // (a bit cast of a vector's element takes its first)
            if (k + e < K) p[k + e] = __builtin_bit_cast(uint16_t, f);
        }
    }
}

// round-half-even(y L / m), inv = fp32(L / m)
__device__ __forceinline__ int qt_code(float y, float m, float inv, int L) {
    const float t = y * inv, q = rintf(t);
    if (__builtin_expect(fabsf(t - q) > 0.4999f, 0)) {
        const int k = (int)fabsf(t);
        const double a = 2.0 * L * (double)fabsf(y), b = (2.0 * k + 1.0) * (double)m;
        const int r = k + ((a > b || (a == b && (k & 1))) ? 1 : 0);
        return y < 0.0f ? -r : r;
    }
    return (int)q;
}

// A token over WPR wavefronts, C pieces of 8 channels a lane in registers (C = 0: any
// number, read again for the codes); 4 / WPR tokens a workgroup where WPR < 4.
template <int DTYPE, bool VEC, int WPR, int C>
__global__ __launch_bounds__(WPR < 4 ? 256 : WPR * 64) void k_quantize(const QtArgs a) {
    constexpr int RPB = WPR < 4 ? 4 / WPR : 1, STEP = WPR * 64 * 8, HOLD = C > 0 ? C : 1;
    constexpr int L = DTYPE == BSP_INT8 ? 127 : 7;
    __shared__ float sums[RPB * WPR];
    __shared__ uint32_t tops[RPB * WPR];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * RPB + wave / WPR;
    const bool live = t < a.n;
    const int64_t row = live ? t : a.n - 1;
    const int k0 = ((wave % WPR) * 64 + lane) * 8;
    const uint16_t *x = a.x + row * a.xs;
    const uint16_t *res = a.residual == nullptr ? nullptr : a.residual + row * a.rs;
    auto load = [&](int k) {
        qt_h8 h = qt_load<VEC>(x, k, a.K);
        if (res != nullptr) {
            const qt_h8 r = qt_load<VEC>(res, k, a.K);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = (_Float16)((float)h[e] + (float)r[e]);
        }
        return h;
    };
    auto values = [&](qt_h8 h, int k, float (&y)[8]) {
        if (a.weight != nullptr) {
            const qt_h8 w = qt_load<VEC>(a.weight, k, a.K);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (float)h[e] * (float)w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (float)h[e];
        }
    };
    qt_h8 held[HOLD];
    float sum = 0.0f;
    uint32_t top = 0;
    auto take = [&](qt_h8 h, int k) {
        float y[8];
        values(h, k, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum = __builtin_fmaf((float)h[e], (float)h[e], sum);
            top = max(top, __builtin_bit_cast(uint32_t, y[e]) & 0x7FFFFFFFu);
        }
        if (a.hidden != nullptr && live && C > 0) qt_store<VEC>(a.hidden + row * a.hs, k, a.K, h);
    };
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * STEP < a.K) held[c] = load(k0 + c * STEP);
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * STEP < a.K) take(held[c], k0 + c * STEP);
    } else {
        for (int k = k0; k < a.K; k += STEP) take(load(k), k);
    }
    sum = bsp_wave_sum(sum);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
    if constexpr (WPR > 1) {
        if (lane == 0) sums[wave] = sum, tops[wave] = top;
        __syncthreads();
        const int w0 = wave / WPR * WPR;
        sum = sums[w0], top = tops[w0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) sum += sums[w0 + w], top = max(top, tops[w0 + w]);
    }
    if (!live) return;
    float r = 1.0f;
    if (a.weight != nullptr) {
        const float mean = sum / (float)a.K + a.eps;
        r = mean == 0.0f ? 0.0f : 1.0f / sqrtf(mean);
    }
    const bool bad = top >= 0x7F800000u;
    const float m = __builtin_bit_cast(float, top), inv = top == 0 || bad ? 0.0f : (float)L / m;
    if (k0 == 0) a.scale[t] = bad ? __builtin_nanf("") : m * r / (float)L;
    uint8_t *codes = a.codes + t * a.cs;
    auto give = [&](qt_h8 h, int k) {
        float y[8];
        int u[8];
        values(h, k, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = bad ? 0 : qt_code(y[e], m, inv, L);
        if (C == 0 && a.hidden != nullptr) qt_store<VEC>(a.hidden + t * a.hs, k, a.K, h);
        if (a.x16 != nullptr) {
            qt_h8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (_Float16)bsp_rounded(y[e] * r);
            qt_store<VEC>(a.x16 + t * a.x16s, k, a.K, o);
        }
        if constexpr (DTYPE == BSP_INT8) {
            if constexpr (VEC) {
                qt_u2 c;
                c.x = (u[0] & 255) | ((u[1] & 255) << 8) | ((u[2] & 255) << 16) | ((uint32_t)u[3] << 24);
                c.y = (u[4] & 255) | ((u[5] & 255) << 8) | ((u[6] & 255) << 16) | ((uint32_t)u[7] << 24);
                *reinterpret_cast<qt_u2 *>(codes + k) = c;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < a.K) codes[k + e] = (uint8_t)u[e];
            }
        } else {
            if constexpr (VEC) {
                uint32_t c = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) c |= (uint32_t)(u[e] & 15) << (4 * e);
                *reinterpret_cast<uint32_t *>(codes + k / 2) = c;
            } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    if (k + e < a.K)
                        codes[(k + e) / 2] = (uint8_t)((u[e] & 15) | (k + e + 1 < a.K ? (u[e + 1] & 15) << 4 : 0));
            }
        }
    };
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * STEP < a.K) give(held[c], k0 + c * STEP);
    } else {
        for (int k = k0; k < a.K; k += STEP) give(load(k), k);
    }
    if constexpr (DTYPE == BSP_INT8)
        if (k0 < 16 && a.K + k0 / 8 < a.K16)       // at most 15 bytes: lane 0 the even ones, lane 1 the odd ones
            for (int k = a.K + k0 / 8; k < a.K16; k += 2) codes[k] = 0;
}

template <int DTYPE, bool VEC>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t *codes, int64_t cs, const float *scale, int64_t n,
                                                    int K, uint32_t pieces, uint16_t *x, int64_t xs) {
    const int64_t first = (int64_t)blockIdx.x * 256;
    int64_t t = first / pieces;
    const uint32_t at = (uint32_t)(first - t * pieces) + threadIdx.x;
    t += at / pieces;
    if (t >= n) return;
    const int k = (int)(at % pieces) * 8;
    const float s = scale[t];
    const uint8_t *c = codes + t * cs;
    qt_h8 o;
    if constexpr (VEC) {
        if constexpr (DTYPE == BSP_INT8) {
            const qt_u2 v = *reinterpret_cast<const qt_u2 *>(c + k);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (_Float16)bsp_rounded(s * (float)(int8_t)((e < 4 ? v.x : v.y) >> (8 * (e & 3))));
        } else {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(c + k / 2);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (_Float16)bsp_rounded(s * (float)bsp_sext4(v >> (4 * e)));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int u = 0;
            if (k + e < K)
                u = DTYPE == BSP_INT8 ? (int)(int8_t)c[k + e] : bsp_sext4((uint32_t)c[(k + e) / 2] >> (4 * (e & 1)));
            o[e] = (_Float16)bsp_rounded(s * (float)u);
        }
    }
    qt_store<VEC>(x + t * xs, k, K, o);
}

template <int DTYPE, bool VEC, int WPR, int C>
void qt_run(const QtArgs &a, hipStream_t stream) {
    constexpr int RPB = WPR < 4 ? 4 / WPR : 1;
    hipLaunchKernelGGL((k_quantize<DTYPE, VEC, WPR, C>), dim3((unsigned)((a.n + RPB - 1) / RPB)),
                       dim3(WPR < 4 ? 256 : WPR * 64), 0, stream, a);
}

template <int DTYPE, bool VEC>
void qt_launch(const QtArgs &a, hipStream_t stream) {
    if (a.K <= 512)
        qt_run<DTYPE, VEC, 1, 1>(a, stream);
    else if (a.K <= 8192)
        qt_run<DTYPE, VEC, 4, 4>(a, stream);
    else if (a.K <= 16384)
        qt_run<DTYPE, VEC, 8, 4>(a, stream);
    else
        qt_run<DTYPE, VEC, 8, 0>(a, stream);
}

bool qt_sizes(int64_t n, int64_t K) { return K < (INT64_C(1) << 25) && n < (INT64_C(1) << 31) && n < (INT64_C(1) << 40) / std::max<int64_t>(K, 1); }

}  // namespace

extern "C" int quantize_tokens_f16(const bsp_tokens *tokens, int dtype, uint8_t *codes, int64_t code_stride,
                                   hipStream_t stream) {
    const bsp_tokens *d = tokens;
    if (d == nullptr || (dtype != BSP_INT8 && dtype != BSP_INT4)) return BSP_E_ARG;
    if (d->n < 0 || d->K < 0 || !(d->eps >= 0.0f) || std::isinf(d->eps)) return BSP_E_ARG;
    if (!qt_sizes(d->n, d->K)) return BSP_E_OVERFLOW;
    if ((d->residual != nullptr) != (d->hidden != nullptr)) return BSP_E_ARG;
    if (d->n == 0 || d->K == 0) return BSP_OK;
    const int64_t bytes = dtype == BSP_INT8 ? d->K : (d->K + 1) / 2;
    if (d->X == nullptr || codes == nullptr || d->scale == nullptr) return BSP_E_ARG;
    if (d->x_stride < d->K || code_stride < bytes) return BSP_E_ARG;
    uintptr_t bits = (uintptr_t)d->X | (uintptr_t)d->weight;
    int64_t strides = d->x_stride;
    if (d->residual != nullptr) {
        if (d->residual_stride < d->K || d->hidden_stride < d->K) return BSP_E_ARG;
        bits |= (uintptr_t)d->residual | (uintptr_t)d->hidden, strides |= d->residual_stride | d->hidden_stride;
    }
    if (d->x16 != nullptr) {
        if (d->x16_stride < d->K) return BSP_E_ARG;
        bits |= (uintptr_t)d->x16, strides |= d->x16_stride;
    }
    if ((bits & 1u) != 0 || ((uintptr_t)d->scale & 3u) != 0) return BSP_E_ARG;
    QtArgs a{};
    a.x = d->X, a.residual = d->residual, a.weight = d->weight, a.hidden = d->hidden, a.x16 = d->x16;
    a.xs = d->x_stride, a.rs = d->residual_stride, a.hs = d->hidden_stride, a.x16s = d->x16_stride, a.cs = code_stride;
    a.scale = d->scale, a.codes = codes, a.n = d->n, a.K = (int)d->K, a.eps = d->eps;
    a.K16 = (int)std::min<int64_t>((d->K + 15) / 16 * 16, code_stride);
    // whole pieces of 8 channels, unless a row or its end is off their boundary
    const uintptr_t cmask = dtype == BSP_INT8 ? 7u : 3u;
    const bool vec = (bits & 15u) == 0 && (strides & 7) == 0 && d->K % 8 == 0 && ((uintptr_t)codes & cmask) == 0 &&
                     (code_stride & (int64_t)cmask) == 0;
    if (dtype == BSP_INT8)
        vec ? qt_launch<BSP_INT8, true>(a, stream) : qt_launch<BSP_INT8, false>(a, stream);
    else
        vec ? qt_launch<BSP_INT4, true>(a, stream) : qt_launch<BSP_INT4, false>(a, stream);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}

extern "C" int dequantize_tokens_f16(const uint8_t *codes, int64_t code_stride, int dtype, const float *scale,
                                     int64_t n, int64_t K, uint16_t *X, int64_t x_stride, hipStream_t stream) {
    if (dtype != BSP_INT8 && dtype != BSP_INT4) return BSP_E_ARG;
    if (n < 0 || K < 0) return BSP_E_ARG;
    if (!qt_sizes(n, K)) return BSP_E_OVERFLOW;
    if (n == 0 || K == 0) return BSP_OK;
    const int64_t bytes = dtype == BSP_INT8 ? K : (K + 1) / 2;
    if (codes == nullptr || scale == nullptr || X == nullptr) return BSP_E_ARG;
    if (code_stride < bytes || x_stride < K) return BSP_E_ARG;
    if (((uintptr_t)X & 1u) != 0 || ((uintptr_t)scale & 3u) != 0) return BSP_E_ARG;
    const uintptr_t cmask = dtype == BSP_INT8 ? 7u : 3u;
    const bool vec = ((uintptr_t)X & 15u) == 0 && (x_stride & 7) == 0 && K % 8 == 0 &&
                     ((uintptr_t)codes & cmask) == 0 && (code_stride & (int64_t)cmask) == 0;
    const uint32_t pieces = (uint32_t)((K + 7) / 8);
    const dim3 grid((unsigned)((n * pieces + 255) / 256)), block(256);
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, codes, code_stride, scale, n, (int)K, pieces, X, x_stride);
    };
    if (dtype == BSP_INT8)
        vec ? run(k_dequantize<BSP_INT8, true>) : run(k_dequantize<BSP_INT8, false>);
    else
        vec ? run(k_dequantize<BSP_INT4, true>) : run(k_dequantize<BSP_INT4, false>);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
