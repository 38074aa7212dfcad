// kv_cache.hip -- writing the paged key/value cache (quantising as it goes)
// and reading it back, for gfx950.
//
// Both kernels move bytes: a row is read once and written once, and the
// arithmetic between (the row's minimum and maximum, then four VALU operations
// per value) hides under it. One lane holds 8 channels of a row (a 16-byte piece
// of its fp16 form), so a row is 8, 16 or 32 lanes and a wavefront holds 8, 4 or
// 2 rows: consecutive tokens of one kv head, whose cache rows are neighbours
// whenever the slots are.
//
// Bound by HBM for long calls: 8192 tokens x 32 heads of 128, int8, written
// and read back, 407 MB in 74.5 us (5.46 TB/s, the codes read back among them, which
// the last-level cache may serve); 65537 tokens x 8 heads, int4, read back, 340 MB
// in 75.2 us (4.52 TB/s). Four rows in flight per lane made that: with
// one (three dependent loads of 4 to 16 bytes per lane) 92 and 106 us; a row's minimum and maximum two values an
// instruction took the first from 85.4 (writing alone 45 to 39.5). Short calls
// are launch latency (32 tokens, write and read: 4.8 us for the two kernels).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitmap_spmm.h"
#include "device_common.h"
#include "kv_cache.h"

namespace {

struct KvArgs {
    const uint16_t *K, *V;       // append: source rows
    uint16_t *Ko, *Vo;           // gather: destination rows
    int64_t ks, vs;              // their token strides in elements
    const int64_t *slots;
    uint8_t *kc, *vc;            // cache codes
    uint32_t *kw, *vw;           // cache words
    int64_t n, nslots;           // tokens of the call; slots of the cache
    int hkv, page_shift;
};

#define KV_BLOCK 256
#define KV_MANY 65536      // (token, head) rows

// Rows of one lane: U token groups of a (head, K / V), so that a lane has U
// independent chains of loads (slot, row, codes) in flight. Items run over (run
// of groups, head, K / V), K / V fastest; a group is the rows a wavefront holds,
// consecutive tokens.
struct KvItem {
    int64_t token;     // of the first group
    int head;
    bool is_v;
    int ch;            // the lane's first channel
};

template <int D, int U>
__device__ __forceinline__ KvItem kv_item(const KvArgs &a, uint32_t item) {
    constexpr int LPR = D / 8, RPW = 64 / LPR;
    const int lane = threadIdx.x & 63;
    const uint32_t th = item >> 1, run = th / (uint32_t)a.hkv;
    KvItem it;
    it.is_v = (item & 1) != 0;
    it.head = (int)(th - run * (uint32_t)a.hkv);
    it.token = (int64_t)run * (RPW * U) + lane / LPR;
    it.ch = (lane % LPR) * 8;
    return it;
}

// Row index of a slot in the cache ([page][head][offset]).
__device__ __forceinline__ int64_t kv_row(const KvArgs &a, int64_t slot, int head) {
    const int64_t page = slot >> a.page_shift;
    const int64_t off = slot & (((int64_t)1 << a.page_shift) - 1);
    return (((page * a.hkv + head) << a.page_shift)) + off;
}

// The fp16 value a code stands for. s * u + o may pass the largest finite fp16
// (a step rounded up, on a row that reaches it): saturated, so that finite
// rows read back finite. (The comparison keeps a NaN.)
__device__ __forceinline__ uint32_t kv_value(float s, float o, uint32_t u) {
    const float v = s * (float)u + o;
    return bsp_f2h(v > 65504.0f ? 65504.0f : v);
}

template <int KIND, int D, bool VEC, int U>
__global__ __launch_bounds__(KV_BLOCK) void k_kv_append(const KvArgs a, uint32_t items) {
    constexpr int RPW = 64 / (D / 8);
    const uint32_t item = blockIdx.x * (KV_BLOCK / 64) + (threadIdx.x >> 6);
    if (item >= items) return;
    const KvItem it = kv_item<D, U>(a, item);
    kv_u4 raw[U];
    int64_t slot[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        // rows past the end are read as row 0 of the call, so that every lane
        // of the shuffles holds a value
        const int64_t token = it.token + i * RPW;
        const bool in = token < a.n;
        slot[i] = in ? a.slots[token] : -1;
        const int64_t t = in ? token : 0;
        raw[i] = kv_load8<VEC>((it.is_v ? a.V + t * a.vs : a.K + t * a.ks) + (int64_t)it.head * D + it.ch);
    }
    uint8_t *codes = it.is_v ? a.vc : a.kc;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const bool ok = slot[i] >= 0 && slot[i] < a.nslots;
        const int64_t row = kv_row(a, ok ? slot[i] : 0, it.head);
        if constexpr (KIND == BSP_FP16) {
            if (ok) *reinterpret_cast<kv_u4 *>(codes + row * (2 * D) + 2 * it.ch) = raw[i];
        } else {
            uint32_t u[8], word;
            kv_quantise<D / 8>(raw[i], KIND == BSP_INT8 ? 255.0f : 15.0f, u, word);
            if (!ok) continue;
            kv_store_codes<KIND>(codes, row * D + it.ch, u);
            if (it.ch == 0) (it.is_v ? a.vw : a.kw)[row] = word;
        }
    }
}

template <int KIND, int D, bool VEC, int U>
__global__ __launch_bounds__(KV_BLOCK) void k_kv_gather(const KvArgs a, uint32_t items) {
    constexpr int RPW = 64 / (D / 8);
    constexpr int CW = KIND == BSP_FP16 ? 4 : KIND == BSP_INT8 ? 2 : 1;      // dwords of a lane's codes
    const uint32_t item = blockIdx.x * (KV_BLOCK / 64) + (threadIdx.x >> 6);
    if (item >= items) return;
    const KvItem it = kv_item<D, U>(a, item);
    const uint8_t *codes = it.is_v ? a.vc : a.kc;
    const uint32_t *words = it.is_v ? a.vw : a.kw;
    int64_t slot[U];
    uint32_t c[U][CW], w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t token = it.token + i * RPW;
        slot[i] = token < a.n ? a.slots[token] : -1;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const bool ok = slot[i] >= 0 && slot[i] < a.nslots;
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < CW; ++j) c[i][j] = 0;
        if (ok) {
            const int64_t row = kv_row(a, slot[i], it.head);
            const uint32_t *p = reinterpret_cast<const uint32_t *>(codes + (row * D + it.ch) * CW / 2);
            if constexpr (CW == 4) {
                const kv_u4 v = *reinterpret_cast<const kv_u4 *>(p);
                c[i][0] = v.x, c[i][1] = v.y, c[i][2] = v.z, c[i][3] = v.w;
            } else if constexpr (CW == 2) {
                const kv_u2 v = *reinterpret_cast<const kv_u2 *>(p);
                c[i][0] = v.x, c[i][1] = v.y;
            } else {
                c[i][0] = *p;
            }
            if constexpr (KIND != BSP_FP16) w[i] = words[row];
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t token = it.token + i * RPW;
        if (token >= a.n) continue;
        kv_u4 out;
        if constexpr (KIND == BSP_FP16) {
            out = kv_u4{c[i][0], c[i][1], c[i][2], c[i][3]};
        } else {
            // (a slot outside the cache: word and codes 0, value 0)
            const float s = kv_word_step(w[i]), o = kv_word_offset(w[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t u0, u1;
                if constexpr (KIND == BSP_INT8)
                    u0 = (c[i][e >> 1] >> (16 * (e & 1))) & 255u, u1 = (c[i][e >> 1] >> (16 * (e & 1) + 8)) & 255u;
                else
                    u0 = (c[i][0] >> (8 * e)) & 15u, u1 = (c[i][0] >> (8 * e + 4)) & 15u;
                out[e] = kv_value(s, o, u0) | (kv_value(s, o, u1) << 16);
            }
        }
        kv_store8<VEC>((it.is_v ? a.Vo + token * a.vs : a.Ko + token * a.ks) + (int64_t)it.head * D + it.ch, out);
    }
}

template <int KIND, int D, bool VEC, int U>
void kv_launch_u(const KvArgs &a, bool append, hipStream_t stream) {
    constexpr int RUN = 64 / (D / 8) * U;
    const uint32_t items = (uint32_t)((a.n + RUN - 1) / RUN * a.hkv * 2);
    const unsigned grid = (items + KV_BLOCK / 64 - 1) / (KV_BLOCK / 64);
    if (append)
        hipLaunchKernelGGL((k_kv_append<KIND, D, VEC, U>), dim3(grid), dim3(KV_BLOCK), 0, stream, a, items);
    else
        hipLaunchKernelGGL((k_kv_gather<KIND, D, VEC, U>), dim3(grid), dim3(KV_BLOCK), 0, stream, a, items);
}

// Four groups a lane once that leaves enough wavefronts to fill the card
// (65536 rows: 8192 wavefronts at 4 rows each).
template <int KIND, int D, bool VEC>
void kv_launch(const KvArgs &a, bool append, hipStream_t stream) {
    if (a.n * a.hkv >= KV_MANY)
        kv_launch_u<KIND, D, VEC, 4>(a, append, stream);
    else
        kv_launch_u<KIND, D, VEC, 1>(a, append, stream);
}

template <int KIND, bool VEC>
void kv_launch_d(const KvArgs &a, int64_t D, bool append, hipStream_t stream) {
    if (D == 64)
        kv_launch<KIND, 64, VEC>(a, append, stream);
    else if (D == 128)
        kv_launch<KIND, 128, VEC>(a, append, stream);
    else
        kv_launch<KIND, 256, VEC>(a, append, stream);
}

template <bool VEC>
void kv_launch_k(const KvArgs &a, int dtype, int64_t D, bool append, hipStream_t stream) {
    if (dtype == BSP_FP16)
        kv_launch_d<BSP_FP16, VEC>(a, D, append, stream);
    else if (dtype == BSP_INT8)
        kv_launch_d<BSP_INT8, VEC>(a, D, append, stream);
    else
        kv_launch_d<BSP_INT4, VEC>(a, D, append, stream);
}

int kv_common(const bsp_kv_cache *c, const uint16_t *K, int64_t ks, const uint16_t *V, int64_t vs,
              const int64_t *slots, int64_t n, bool append, hipStream_t stream) {
    const int rc = kv_check_cache(c);
    if (rc != BSP_OK) return rc;
    if (n < 0) return BSP_E_ARG;
    // a launch holds fewer than 2^32 threads (16 rows at least per workgroup of 256)
    if (n >= (INT64_C(1) << 28) / std::max<int64_t>(c->kv_heads, 1)) return BSP_E_OVERFLOW;
    if (n == 0 || c->kv_heads == 0) return BSP_OK;
    if (K == nullptr || V == nullptr || slots == nullptr) return BSP_E_ARG;
    if (ks < c->kv_heads * c->head_dim || vs < c->kv_heads * c->head_dim) return BSP_E_ARG;
    if ((((uintptr_t)K | (uintptr_t)V) & 1u) != 0 || ((uintptr_t)slots & 7u) != 0) return BSP_E_ARG;
    if (append && c->num_pages == 0) return BSP_OK;        // every slot is outside
    KvArgs a{};
    a.K = K, a.V = V, a.Ko = const_cast<uint16_t *>(K), a.Vo = const_cast<uint16_t *>(V);
    a.ks = ks, a.vs = vs, a.slots = slots;
    a.kc = (uint8_t *)c->k, a.vc = (uint8_t *)c->v, a.kw = c->k_scale, a.vw = c->v_scale;
    a.n = n, a.nslots = c->num_pages * c->page_size;
    a.hkv = (int)c->kv_heads;
    a.page_shift = __builtin_ctzll((unsigned long long)c->page_size);
    // whole 16-byte pieces of the rows, unless the rows are off that boundary
    const bool vec = (((uintptr_t)K | (uintptr_t)V) & 15u) == 0 && ((ks | vs) & 7) == 0;
    if (vec)
        kv_launch_k<true>(a, c->dtype, c->head_dim, append, stream);
    else
        kv_launch_k<false>(a, c->dtype, c->head_dim, append, stream);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}

}  // namespace

extern "C" int kv_cache_append(const bsp_kv_cache *cache, const uint16_t *K, int64_t k_stride, const uint16_t *V,
                               int64_t v_stride, const int64_t *slots, int64_t n, hipStream_t stream) {
    return kv_common(cache, K, k_stride, V, v_stride, slots, n, true, stream);
}

extern "C" int kv_cache_gather(const bsp_kv_cache *cache, const int64_t *slots, int64_t n, uint16_t *K,
                               int64_t k_stride, uint16_t *V, int64_t v_stride, hipStream_t stream) {
    return kv_common(cache, K, k_stride, V, v_stride, slots, n, false, stream);
}
