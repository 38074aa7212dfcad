// kv_cache.h -- what the cache kernels and the attention kernels share: the
// scale word of a quantised row and the checks of a cache descriptor.
#pragma once
#include <stdint.h>

#include "bitmap_spmm.h"

// A row's scale word: step as bfloat16 (high half), offset as fp16 (low half).
__device__ __forceinline__ float kv_word_step(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ __forceinline__ float kv_word_offset(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
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
