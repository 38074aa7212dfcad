// attention_tree.hip -- attention of drafted token trees over the paged
// key/value cache, for gfx950.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "bitmap_spmm.h"
#include "device_common.h"
#include "kv_cache.h"

namespace {

struct AtArgs {
    const uint16_t *Q;
    int64_t q_stride;
    const uint8_t *k, *v;
    const uint32_t *kw, *vw;
    const int32_t *table;
    int64_t table_width;
    const int32_t *kv_lens, *q_start;
    const uint64_t *mask;
    uint16_t *O;
    int64_t o_stride;
    int total_q, max_q, hq, hkv, num_pages, page_shift;
    float scale;
};

// Channel d of cache row `row` (K or V).
template <int KIND, int D>
__device__ __forceinline__ float at_value(const uint8_t *codes, const uint32_t *words, int64_t row, int d) {
    if constexpr (KIND == BSP_FP16) {
        return bsp_h2f(reinterpret_cast<const uint16_t *>(codes)[row * D + d]);
    } else {
        const uint32_t w = words[row];
        uint32_t u;
        if constexpr (KIND == BSP_INT8)
            u = codes[row * D + d];
        else
            u = (codes[row * (D / 2) + (d >> 1)] >> (4 * (d & 1))) & 15u;
        return kv_word_step(w) * (float)u + kv_word_offset(w);
    }
}

// One wavefront per (drafted token, query head). 64 tokens at a time: lane j
// scores token j (its row against the query in LDS), the running maximum and
// sum are updated, then each lane adds its D / 64 channels of the 64 rows.
template <int KIND, int D>
__global__ __launch_bounds__(64) void k_at_row(const AtArgs a) {
    const int lane = threadIdx.x, h = blockIdx.x % a.hq, b = blockIdx.y, i = blockIdx.x / a.hq;
    const int q0 = min(max(a.q_start[b], 0), a.total_q), q1 = min(max(a.q_start[b + 1], q0), a.total_q);
    const int T = min(q1 - q0, a.max_q);
    if (i >= T) return;
    const int64_t cap = a.table_width << a.page_shift;
    const int len = (int)min((int64_t)max(a.kv_lens[b], 0), cap);
    const int past = len - T;
    const uint64_t seen = a.mask != nullptr ? a.mask[q0 + i] : (uint64_t)-1 >> (63 - i);
    const int kvh = h / (a.hq / a.hkv);
    __shared__ float q[D];
    for (int d = lane; d < D; d += 64) q[d] = bsp_h2f(a.Q[(int64_t)(q0 + i) * a.q_stride + (int64_t)h * D + d]);
    __syncthreads();
    float m = -1e30f, l = 0.f, acc[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) acc[c] = 0.f;
    for (int j0 = 0; j0 < len; j0 += 64) {
        const int j = j0 + lane;
        float x = -INFINITY;
        int64_t row = 0;
        const int dj = j - past;
        const bool ok = j < len && (dj < 0 || (dj < T && (seen >> dj & 1)));
        if (ok) {
            int page = a.table[b * a.table_width + (j >> a.page_shift)];
            if ((unsigned)page >= (unsigned)a.num_pages) page = 0;
            row = (((int64_t)page * a.hkv + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
            float s = 0.f;
            for (int d = 0; d < D; ++d) s += q[d] * at_value<KIND, D>(a.k, a.kw, row, d);
            x = s * a.scale;
        }
        float mt = x;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d, 64));
        const float mn = fmaxf(m, mt), f = expf(m - mn);
        const float p = expf(x - mn);
        l = l * f + bsp_wave_sum(p);
        m = mn;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) acc[c] *= f;
        for (int t = 0; t < 64; ++t) {
            const float pt = __shfl(p, t, 64);
            const int64_t rt = __shfl((long long)row, t, 64);
            if (!__shfl((int)ok, t, 64)) continue;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) acc[c] += pt * at_value<KIND, D>(a.v, a.vw, rt, lane + 64 * c);
        }
    }
    uint16_t *o = a.O + (int64_t)(q0 + i) * a.o_stride + (int64_t)h * D;
    // a NaN score leaves NaN in l: not an empty row
#pragma unroll
    for (int c = 0; c < D / 64; ++c) o[lane + 64 * c] = bsp_f2h(l == 0.f ? 0.f : acc[c] / l);
}

template <int KIND>
void at_launch(const AtArgs &a, int64_t D, int64_t B, hipStream_t stream) {
    const dim3 grid((unsigned)(a.max_q * a.hq), (unsigned)B);
    if (D == 64)
        hipLaunchKernelGGL((k_at_row<KIND, 64>), grid, dim3(64), 0, stream, a);
    else if (D == 128)
        hipLaunchKernelGGL((k_at_row<KIND, 128>), grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL((k_at_row<KIND, 256>), grid, dim3(64), 0, stream, a);
}

// Checks shared by the call and its workspace size.
int at_check(const bsp_kv_cache *c, int64_t table_width, int64_t B, int64_t max_q, int64_t hq) {
    const int rc = kv_check_cache(c);
    if (rc != BSP_OK) return rc;
    if (table_width < 0 || B < 0 || max_q < 0 || max_q > BSP_TREE_MAX || hq < 0) return BSP_E_ARG;
    if (hq > 0 && (c->kv_heads == 0 || hq % c->kv_heads != 0)) return BSP_E_ARG;
    if (B > 65535 || hq > 65535) return BSP_E_OVERFLOW;
    if (table_width > INT32_MAX / c->page_size) return BSP_E_OVERFLOW;
    return BSP_OK;
}

}  // namespace

extern "C" int attention_tree_workspace_bytes(const bsp_kv_cache *cache, int64_t table_width, int64_t B, int64_t max_q,
                                              int64_t q_heads, int64_t *bytes) {
    if (bytes == nullptr) return BSP_E_ARG;
    const int rc = at_check(cache, table_width, B, max_q, q_heads);
    if (rc != BSP_OK) return rc;
    *bytes = 0;
    return BSP_OK;
}

extern "C" int attention_tree_f16(const uint16_t *Q, int64_t q_stride, const bsp_kv_cache *cache,
                                  const int32_t *block_table, int64_t table_width, const int32_t *kv_lens,
                                  const int32_t *q_start, int64_t B, int64_t total_q, int64_t max_q, int64_t q_heads,
                                  const uint64_t *tree_mask, float scale, uint16_t *O, int64_t o_stride,
                                  void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    const int rc = at_check(cache, table_width, B, max_q, q_heads);
    if (rc != BSP_OK) return rc;
    if (total_q < 0 || workspace_bytes < 0 || !std::isfinite(scale)) return BSP_E_ARG;
    if (total_q > INT32_MAX) return BSP_E_OVERFLOW;
    if (workspace == nullptr && workspace_bytes != 0) return BSP_E_ARG;
    if (workspace != nullptr && ((uintptr_t)workspace & 255u) != 0) return BSP_E_ARG;
    if (B == 0 || max_q == 0 || q_heads == 0 || total_q == 0) return BSP_OK;
    if (Q == nullptr || O == nullptr || kv_lens == nullptr || q_start == nullptr) return BSP_E_ARG;
    if (table_width > 0 && (block_table == nullptr || cache->num_pages == 0)) return BSP_E_ARG;
    if (q_stride < q_heads * cache->head_dim || o_stride < q_heads * cache->head_dim) return BSP_E_ARG;
    if ((((uintptr_t)Q | (uintptr_t)O) & 1u) != 0 || ((uintptr_t)tree_mask & 7u) != 0) return BSP_E_ARG;
    AtArgs a{};
    a.Q = Q, a.q_stride = q_stride;
    a.k = (const uint8_t *)cache->k, a.v = (const uint8_t *)cache->v;
    a.kw = cache->k_scale, a.vw = cache->v_scale;
    a.table = block_table, a.table_width = table_width;
    a.kv_lens = kv_lens, a.q_start = q_start, a.mask = tree_mask;
    a.O = O, a.o_stride = o_stride;
    a.total_q = (int)total_q, a.max_q = (int)max_q, a.hq = (int)q_heads, a.hkv = (int)cache->kv_heads;
    a.num_pages = (int)cache->num_pages;
    a.page_shift = __builtin_ctzll((unsigned long long)cache->page_size);
    a.scale = scale;
    if (cache->dtype == BSP_FP16)
        at_launch<BSP_FP16>(a, cache->head_dim, B, stream);
    else if (cache->dtype == BSP_INT8)
        at_launch<BSP_INT8>(a, cache->head_dim, B, stream);
    else
        at_launch<BSP_INT4>(a, cache->head_dim, B, stream);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
