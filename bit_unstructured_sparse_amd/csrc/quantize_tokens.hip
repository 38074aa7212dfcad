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
// 16384 channels; longer tokens are read twice). Rounding is by adding 1.5 * 2^23, which leaves a code in
// the low bits; the exact comparison is one branch for 8 channels.
//
// Bound by memory where tokens are many and long: 8191 x 8192 with residual and norm to int8, and back, 671 MB in 111 to 116 us
// (6.0 TB/s, part of it the last-level cache's; the sums' inputs are read past it, which leaves the codes there: 133 us
// otherwise), to int4 77 of them and back 26. Odd rows cost more, their pieces are read and written whole at any address: 4096 x
// 11007, normed, 50 us, 4096 x 11008 39 (146 with single values). Many short tokens have one or two pieces a lane on their way,
// and read the weight again for each: 16384 x 164 with residual and norm 7.5 us, 32768 x 300 23, where the bytes take 3.9
// and 14.4 at the rate of a copy (4.77 TB/s). Few tokens are launch latency: one token of 4096 2.9 us, back 2.0 (3.3 and
// 2.5 in a graph).
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
    int K;
    float eps;
};

// 8 values at p + k of a row of K, zeros past its end. The memory takes 16 bytes at any address: odd rows are
// read and written in whole pieces too, all but the one at their end. ONCE: nobody reads it again (it need not push
// the codes out of the last-level cache).
template <bool ONCE>
__device__ __forceinline__ qt_h8 qt_load(const uint16_t *p, int k, int K) {
    struct __attribute__((packed, aligned(2))) piece {
        qt_u4 v;
    };
    if (k + 8 <= K) {
        if constexpr (ONCE) return __builtin_bit_cast(qt_h8, __builtin_nontemporal_load(&reinterpret_cast<const piece *>(p + k)->v));
        return __builtin_bit_cast(qt_h8, reinterpret_cast<const piece *>(p + k)->v);
    }
    qt_h8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < K ? __builtin_bit_cast(_Float16, p[k + e]) : (_Float16)0.0f;
    return v;
}

__device__ __forceinline__ void qt_store(uint16_t *p, int k, int K, qt_h8 v) {
    if (k + 8 <= K) {
        __builtin_memcpy(p + k, &v, 16);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const _Float16 f = v[e];      // (a bit cast of a vector's element takes its first)
        if (k + e < K) p[k + e] = __builtin_bit_cast(uint16_t, f);
    }
}

// 1.5 * 2^23: added to a number below 2^22 it leaves its rounded value in the low bits
#define QT_MAGIC 12582912.0f

// round-half-even(y L / m) decided exactly, for a quotient next to a border
__device__ __forceinline__ int qt_code_exact(float y, float t, float m, int L) {
    const int k = (int)fabsf(t);
    const double a = 2.0 * L * (double)fabsf(y), b = (2.0 * k + 1.0) * (double)m;
    const int r = k + ((a > b || (a == b && (k & 1))) ? 1 : 0);
    return y < 0.0f ? -r : r;
}

// A token over TPR threads, C pieces of 8 channels a thread in registers (C = 0: any number, read again
// for the codes); 256 / TPR tokens a workgroup where TPR is less.
template <int DTYPE, int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_quantize(const QtArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1, STEP = TPR * 8, HOLD = C > 0 ? C : 1, WPR = TPR / 64;
    constexpr int L = DTYPE == BSP_INT8 ? 127 : 7;
    __shared__ float sums[WPR > 1 ? WPR : 1];
    __shared__ uint32_t tops[WPR > 1 ? WPR : 1];
    static_assert(TPR >= 256 || TPR <= 64, "a token's wavefronts are those of its workgroup");
    const int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const bool live = t < a.n;
    const int64_t row = live ? t : a.n - 1;
    const int k0 = (int)(threadIdx.x % TPR) * 8;
    const uint16_t *x = a.x + row * a.xs;
    const uint16_t *res = a.residual == nullptr ? nullptr : a.residual + row * a.rs;
    auto load = [&](int k) {
        qt_h8 h = qt_load<(C > 0)>(x, k, a.K);
        if (res != nullptr) {
            const qt_h8 r = qt_load<(C > 0)>(res, k, a.K);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = (_Float16)((float)h[e] + (float)r[e]);
        }
        return h;
    };
    auto values = [&](qt_h8 h, int k, float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (float)h[e];
        if (a.weight != nullptr) {
            const qt_h8 w = qt_load<false>(a.weight, k, a.K);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= (float)w[e];
        }
    };
    float sum = 0.0f, held[HOLD][8];
    uint32_t top = 0;
    auto take = [&](qt_h8 h, int k, float (&y)[8]) {
        values(h, k, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.weight != nullptr) sum = __builtin_fmaf((float)h[e], (float)h[e], sum);
            top = max(top, __builtin_bit_cast(uint32_t, y[e]) & 0x7FFFFFFFu);
        }
        if (a.hidden != nullptr && live && C > 0) qt_store(a.hidden + row * a.hs, k, a.K, h);
    };
    if constexpr (C > 0) {
        qt_h8 h[HOLD];
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * STEP < a.K) h[c] = load(k0 + c * STEP);
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * STEP < a.K) take(h[c], k0 + c * STEP, held[c]);
    } else {
        for (int k = k0; k < a.K; k += STEP) take(load(k), k, held[0]);
    }
#pragma unroll
    for (int d = (TPR < 64 ? TPR : 64) / 2; d >= 1; d >>= 1) {
        sum += __shfl_xor(sum, d, 64);
        top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
    }
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) sums[wave] = sum, tops[wave] = top;
        __syncthreads();
        sum = sums[0], top = tops[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) sum += sums[w], top = max(top, tops[w]);
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
    auto give = [&](const float (&y)[8], int k) {
        uint32_t u[8];
        float worst = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = y[e] * inv, s = q + QT_MAGIC;
            u[e] = __builtin_bit_cast(uint32_t, s);
            worst = fmaxf(worst, fabsf(q - (s - QT_MAGIC)));
        }
        if (__builtin_expect(worst > 0.4999f, 0)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q = y[e] * inv;
                if (fabsf(q - rintf(q)) > 0.4999f) u[e] = (uint32_t)qt_code_exact(y[e], q, m, L);
            }
        }
        if (bad) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = 0;
        }
        if (a.x16 != nullptr) {
            qt_h8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (_Float16)bsp_rounded(y[e] * r);
            qt_store(a.x16 + t * a.x16s, k, a.K, o);
        }
        if constexpr (DTYPE == BSP_INT8) {
            qt_u2 c;
            c.x = (u[0] & 255) | ((u[1] & 255) << 8) | ((u[2] & 255) << 16) | (u[3] << 24);
            c.y = (u[4] & 255) | ((u[5] & 255) << 8) | ((u[6] & 255) << 16) | (u[7] << 24);
            if (k + 8 <= a.K) {
                __builtin_memcpy(codes + k, &c, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < a.K) codes[k + e] = (uint8_t)u[e];
            }
        } else {
            uint32_t c = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) c |= (k + e < a.K ? u[e] & 15u : 0u) << (4 * e);
            if (k + 8 <= a.K) {
                __builtin_memcpy(codes + k / 2, &c, 4);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    if (k + e < a.K) codes[(k + e) / 2] = (uint8_t)(c >> (4 * e));
            }
        }
    };
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * STEP < a.K) give(held[c], k0 + c * STEP);
    } else {
        for (int k = k0; k < a.K; k += STEP) {
            const qt_h8 h = load(k);
            values(h, k, held[0]);
            if (a.hidden != nullptr) qt_store(a.hidden + t * a.hs, k, a.K, h);
            give(held[0], k);
        }
    }
}

template <int DTYPE>
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
    int u[8];
    if (k + 8 <= K) {
        if constexpr (DTYPE == BSP_INT8) {
            int8_t v[8];
            __builtin_memcpy(v, c + k, 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = v[e];
        } else {
            uint32_t v;
            __builtin_memcpy(&v, c + k / 2, 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = bsp_sext4(v >> (4 * e));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            u[e] = k + e >= K ? 0 : DTYPE == BSP_INT8 ? (int)(int8_t)c[k + e] : bsp_sext4((uint32_t)c[(k + e) / 2] >> (4 * (e & 1)));
    }
    qt_h8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (_Float16)bsp_rounded(s * (float)u[e]);
    qt_store(x + t * xs, k, K, o);
}

// A launch holds fewer than 2^32 threads: more tokens go in several.
template <int DTYPE, int TPR, int C>
void qt_run(const QtArgs &all, hipStream_t stream) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const int64_t most = (INT64_C(1) << 31) / TPR;
    for (int64_t t = 0; t < all.n; t += most) {
        QtArgs a = all;
        a.n = std::min(all.n - t, most);
        a.x += t * a.xs, a.scale += t, a.codes += t * a.cs;
        if (a.residual != nullptr) a.residual += t * a.rs, a.hidden += t * a.hs;
        if (a.x16 != nullptr) a.x16 += t * a.x16s;
        hipLaunchKernelGGL((k_quantize<DTYPE, TPR, C>), dim3((unsigned)((a.n + RPB - 1) / RPB)), dim3(TPR < 256 ? 256 : TPR),
                           0, stream, a);
    }
}

// One piece a thread while tokens are few (one token of 4096: 3.5 us over 512 threads, 4.4 over 256): most
// wavefronts on the card. Many tokens keep it full anyway; two pieces a thread then halve the barriers
// and turns of workgroups: 16384 x 4096 46 us with 256 threads a token, 65 with 512; 16384 x 1024 16 us
// with a wavefront each, 27 with 256 threads (at 1024 tokens 5.1 against 4.6: the border lies at 2048).
// Short tokens share a wavefront, as many as leave its lanes work: 117258 x 164 43 us with 16 lanes a token, 50 with 32, 83
// with 64 (2048 x 256 5.2, 4.2, 4.4); 32768 x 300 24 with 32 and 28 with 64, 16384 x 512 14.4 and 15.2 (2048 5.6 and 4.9).
template <int DTYPE>
void qt_launch(const QtArgs &a, hipStream_t stream) {
    const bool many = a.n >= 2048, lots = a.n >= 16384;
    if (a.K <= 128)
        qt_run<DTYPE, 16, 1>(a, stream);
    else if (a.K <= 256 && lots)
        qt_run<DTYPE, 16, 2>(a, stream);
    else if (a.K <= 256)
        qt_run<DTYPE, 32, 1>(a, stream);
    else if (a.K <= 512 && lots)
        qt_run<DTYPE, 32, 2>(a, stream);
    else if (a.K <= 512)
        qt_run<DTYPE, 64, 1>(a, stream);
    else if (a.K <= 1024 && many)
        qt_run<DTYPE, 64, 2>(a, stream);
    else if (a.K <= 2048)
        qt_run<DTYPE, 256, 1>(a, stream);
    else if (a.K <= 4096 && many)
        qt_run<DTYPE, 256, 2>(a, stream);
    else if (a.K <= 4096)
        qt_run<DTYPE, 512, 1>(a, stream);
    else if (a.K <= 8192)
        qt_run<DTYPE, 512, 2>(a, stream);
    else if (a.K <= 16384)
        qt_run<DTYPE, 1024, 2>(a, stream);
    else
        qt_run<DTYPE, 1024, 0>(a, stream);
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
    if (d->residual != nullptr) {
        if (d->residual_stride < d->K || d->hidden_stride < d->K) return BSP_E_ARG;
        bits |= (uintptr_t)d->residual | (uintptr_t)d->hidden;
    }
    if (d->x16 != nullptr) {
        if (d->x16_stride < d->K) return BSP_E_ARG;
        bits |= (uintptr_t)d->x16;
    }
    if ((bits & 1u) != 0 || ((uintptr_t)d->scale & 3u) != 0) return BSP_E_ARG;
    QtArgs a{};
    a.x = d->X, a.residual = d->residual, a.weight = d->weight, a.hidden = d->hidden, a.x16 = d->x16;
    a.xs = d->x_stride, a.rs = d->residual_stride, a.hs = d->hidden_stride, a.x16s = d->x16_stride, a.cs = code_stride;
    a.scale = d->scale, a.codes = codes, a.n = d->n, a.K = (int)d->K, a.eps = d->eps;
    if (dtype == BSP_INT8)
        qt_launch<BSP_INT8>(a, stream);
    else
        qt_launch<BSP_INT4>(a, stream);
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
    const uint32_t pieces = (uint32_t)((K + 7) / 8);
    const int64_t most = (INT64_C(1) << 31) / pieces;      // fewer than 2^32 threads a launch
    auto run = [&](auto kernel) {
        for (int64_t t = 0; t < n; t += most) {
            const int64_t m = std::min(n - t, most);
            hipLaunchKernelGGL(kernel, dim3((unsigned)((m * pieces + 255) / 256)), dim3(256), 0, stream, codes + t * code_stride,
                               code_stride, scale + t, m, (int)K, pieces, X + t * x_stride, x_stride);
        }
    };
    if (dtype == BSP_INT8)
        run(k_dequantize<BSP_INT8>);
    else
        run(k_dequantize<BSP_INT4>);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
