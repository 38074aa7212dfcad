// kv_cache.h -- what the kernels that write or read the cache share: the
// scale word of a quantised row, the quantisation of a row held 8 channels to a
// lane, and the checks of a cache descriptor.
#pragma once
#include <stdint.h>

#include "bitmap_spmm.h"
#include "device_common.h"

typedef uint32_t kv_u4 __attribute__((ext_vector_type(4)));
typedef uint32_t kv_u2 __attribute__((ext_vector_type(2)));
typedef _Float16 kv_h8 __attribute__((ext_vector_type(8)));
typedef _Float16 kv_h2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ kv_h2 kv_pair(uint32_t v) { return __builtin_bit_cast(kv_h2, v); }

// 1.5 * 2^23: added to a number below 2^22 it leaves its rounded value in the low bits
#define KV_MAGIC 12582912.0f

// A row's scale word: step as bfloat16 (high half), offset as fp16 (low half).
__device__ __forceinline__ float kv_word_step(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ __forceinline__ float kv_word_offset(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
}

// 8 fp16 values at p; element loads when p may be off a 16-byte boundary.
template <bool VEC>
__device__ __forceinline__ kv_u4 kv_load8(const uint16_t *p) {
    if constexpr (VEC) return *reinterpret_cast<const kv_u4 *>(p);
    kv_u4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return v;
}

template <bool VEC>
__device__ __forceinline__ void kv_store8(uint16_t *p, kv_u4 v) {
    if constexpr (VEC) {
        *reinterpret_cast<kv_u4 *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[2 * i] = (uint16_t)v[i];
            p[2 * i + 1] = (uint16_t)(v[i] >> 16);
        }
    }
}

template <int CTRL>
__device__ __forceinline__ float kv_dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The value of the neighbouring run of d lanes, where all lanes of a run hold the same: the steps of a reduction over
// a row's lanes. Up to 16 lanes a move within the vector unit, not a trip through LDS.
__device__ __forceinline__ float kv_other(float v, int d) {
    switch (d) {
        case 1: return kv_dpp<0xB1>(v);       // within four lanes
        case 2: return kv_dpp<0x4E>(v);
        case 4: return kv_dpp<0x141>(v);      // eight lanes mirrored
        case 8: return kv_dpp<0x140>(v);      // sixteen mirrored
        default: return __shfl_xor(v, d, 64);
    }
}

// Quantise the 8 values of a lane; the row's lanes are LPR neighbours.
// (x - o) / s is needed correctly rounded, so that a value half way between
// two codes goes to the even one: with r the correctly rounded reciprocal of
// s, q = fma(fma(-q0, s, n), r, q0), q0 = n r, is the correctly rounded
// quotient (Markstein's theorem), at three operations instead of a division.
template <int LPR>
__device__ __forceinline__ void kv_quantise(kv_u4 raw, float levels, uint32_t (&u)[8], uint32_t &word) {
    // minimum and negated maximum in one word of two halves: two values an instruction, and one reduction over the
    // lanes (a third of the instructions: 8192 tokens x 32 heads to int8 39.5 us, in fp32 45). (These keep a NaN, and take -0 for less than +0, as the fp32 ones do.)
    kv_h2 least = kv_pair(raw[0]), most = least;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        least = __builtin_elementwise_minimum(least, kv_pair(raw[i]));
        most = __builtin_elementwise_maximum(most, kv_pair(raw[i]));
    }
    const uint32_t lb = __builtin_bit_cast(uint32_t, least), mb = __builtin_bit_cast(uint32_t, most) ^ 0x80008000u;
    kv_h2 range = __builtin_elementwise_minimum(kv_pair((lb & 0xFFFFu) | (mb << 16)), kv_pair((lb >> 16) | (mb & 0xFFFF0000u)));
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1)
        range = __builtin_elementwise_minimum(
            range, kv_pair(__builtin_bit_cast(uint32_t, kv_other(__builtin_bit_cast(float, range), d))));
    const uint32_t ends = __builtin_bit_cast(uint32_t, range);
    if ((ends & 0x7C00u) == 0x7C00u || (ends & 0x7C000000u) == 0x7C000000u) {      // an infinity or a NaN in the row
        word = 0x7FC07E00u;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = 0;
        return;
    }
    const kv_h8 h = __builtin_bit_cast(kv_h8, raw);
    const float lo = (float)range.x, hi = -(float)range.y;
    const uint32_t sb = (__builtin_bit_cast(uint32_t, (hi - lo) / levels) + 0xFFFFu) & 0xFFFF0000u;
    const float s = __builtin_bit_cast(float, sb);
    word = sb | (ends & 0xFFFFu);
    const float r = sb != 0 ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float nmr = (float)h[i] - lo;
        const float q0 = nmr * r;
        const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, nmr), r, q0);
        u[i] = __builtin_bit_cast(uint32_t, fminf(q + KV_MAGIC, levels + KV_MAGIC));
    }
}

// The codes (the low bits of u) of channels ch .. ch + 7 of a row, `at` = row * D + ch.
template <int KIND>
__device__ __forceinline__ void kv_store_codes(uint8_t *codes, int64_t at, const uint32_t (&u)[8]) {
    kv_u2 c;      // a code a byte
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = __builtin_amdgcn_perm(u[4 * i + 1], u[4 * i], 0x0C0C0400u) |
               __builtin_amdgcn_perm(u[4 * i + 3], u[4 * i + 2], 0x04000C0Cu);
    if constexpr (KIND == BSP_INT8) {
        *reinterpret_cast<kv_u2 *>(codes + at) = c;
    } else {      // a byte's code beside its neighbour's, then every other byte
        c.x |= c.x >> 4, c.y |= c.y >> 4;
        *reinterpret_cast<uint32_t *>(codes + at / 2) = __builtin_amdgcn_perm(c.y, c.x, 0x06040200u);
    }
}

// Bytes of one cache row.
static inline int64_t kv_row_bytes(int dtype, int64_t head_dim) {
    return dtype == BSP_FP16 ? 2 * head_dim : dtype == BSP_INT8 ? head_dim : head_dim / 2;
}

// Host-side checks of a descriptor; runs before any HIP call.
static inline int kv_check_cache(const bsp_kv_cache *c) {
    if (c == nullptr) return BSP_E_ARG;
    if (c->dtype != BSP_FP16 && c->dtype != BSP_INT8 && c->dtype != BSP_INT4) return BSP_E_ARG;
    if (c->num_pages < 0 || c->kv_heads < 0 || c->page_size < 16 || c->page_size > 4096) return BSP_E_ARG;
    if ((c->page_size & (c->page_size - 1)) != 0) return BSP_E_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return BSP_E_UNSUPPORTED;
    if (c->kv_heads > 65535) return BSP_E_OVERFLOW;
    if (c->num_pages > INT32_MAX / c->page_size) return BSP_E_OVERFLOW;
    if (c->num_pages == 0 || c->kv_heads == 0) return BSP_OK;
    if (c->k == nullptr || c->v == nullptr) return BSP_E_ARG;
    if ((((uintptr_t)c->k | (uintptr_t)c->v) & 15u) != 0) return BSP_E_ARG;
    if (c->dtype != BSP_FP16) {
        if (c->k_scale == nullptr || c->v_scale == nullptr) return BSP_E_ARG;
        if ((((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 15u) != 0) return BSP_E_ARG;
    }
    return BSP_OK;
}
