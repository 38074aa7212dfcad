// qk_heads.hip -- query and key heads normed and rotated, and (with the values)
// written to the paged cache, for gfx950.
//
// One lane holds 8 channels of a head (a 16-byte piece), as in the cache kernels: a
// head is 8, 16 or 32 lanes and a wavefront holds 8, 4 or 2 of them, neighbouring
// heads of one token and one kind (query, key or value; of several where heads are few), in U such groups.
//
// The angle of pair i at position p is p * freq[i] turns, freq in units of 2^-64
// turns: the product mod 2^64 is the angle mod one turn, exactly. Split into a multiple
// of a quarter turn and a rest x of at most an eighth, its sine and cosine are Taylor
// sums to x^13 and x^12 (the first terms left out are 2^-45 and 2^-41), the leading
// terms in 64 bits, the others, under 2^-14, in 32: both come out as the nearest float
// but where they lie within 2^-11 of a step from the middle of two. A wavefront
// computes each of its token's angles once, a pair a lane, and shares them through LDS.
//
// Everything between the input and the result is 32-bit, each operation rounded once and none contracted, in the
// order of the definition: y = x / sqrt(mean + eps), a correctly rounded quotient (rc = 1 / r,
// q = fma(fma(-q0, r, x), rc, q0), q0 = x rc, Markstein), times w, then y1 c - y2 s and y2 c + y1 s. A key whose
// fp16 neighbour would do as well still lands in another code of an int4 row, a sixteenth of the row's range: an
// evaluation in the plain order gives the same codes but for one result in 10^7. (A form with w and the norm folded
// into the sines, within 2^-24 of the definition too, differed from it in 1.3 results of 10^4, at the same speed.)
// The mean's squares are added as a 16-byte piece holds them, its halves of four in turn (heads of 64: neighbours
// first), then the lanes' sums neighbours first.
//
// Bound by memory where tokens and heads are many: 8192 tokens, 32 query and 32 key heads of 128, 268 MB in 48 to 53 us
// (5.1 to 5.6 TB/s); with values into an fp16 cache 403 MB in 76 us (5.3 TB/s). Into an int8 cache 338 MB take 79 to 83 us,
// into an int4 one 304 MB 80: a row's codes cost about as many vector instructions as the rotation, and no longer all hide
// (86 with its minimum and maximum in fp32). (With each lane its own 8 angles a group: 84 and 127 us. With 64-bit sines
// throughout 55 and 91.) Few heads a token fill a part of a wavefront, which evaluates all of the token's angles all the same:
// 60000 tokens x (1 + 1) heads of 64 25 us, of 128 38, 8192 x (8 + 1, with values) of 256 into an int8 cache 26, where the bytes
// take 6.4, 12.9 and 16.7 us at the rate of a copy (4.77 TB/s). Few tokens are launch latency: 3.8 us, 3.9 with an int8 cache.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "bitmap_spmm.h"
#include "device_common.h"
#include "kv_cache.h"

namespace {

#define QK_BLOCK 256

struct QkArgs {
    const uint16_t *x[3];         // query, key, value heads
    uint16_t *o[2];               // their results (cached: o[0] alone)
    int64_t xs[3], os[2];         // token strides in elements
    const uint16_t *weight[2];
    const uint64_t *freq;
    const int32_t *positions;
    const int64_t *slots;
    uint8_t *codes[2];            // the cache
    uint32_t *words[2];
    int64_t nslots;
    float eps;
    int heads[3];                 // heads of each kind; values: 0 without a cache
    uint32_t parts[3];            // running number of a token's items: queries, keys, values (MIX: the last is all)
    uint32_t n;
    int kind, page_shift, rot, interleaved;
    bool cached;                  // keys and values go to the cache
};

// sin and cos of t * 2^-64 turns, rounded to 32 bits.
__device__ __forceinline__ void qk_sincos(uint64_t t, float &s, float &c) {
    const uint32_t q = (uint32_t)((t + (UINT64_C(1) << 61)) >> 62);              // nearest quarter
    const double x = (double)(int64_t)(t - ((uint64_t)q << 62)) * 3.4061215800865545e-19;      // 2 pi / 2^64
    const double z = x * x;
    const float y = (float)z;
    float ps = __builtin_fmaf(y, 1.6059043836821613e-10f, -2.505210838544172e-8f);
    ps = __builtin_fmaf(y, ps, 2.7557319223985893e-6f);
    ps = __builtin_fmaf(y, ps, -1.984126984126984e-4f);
    double sn = __builtin_fma(z, (double)ps, 8.333333333333333e-3);
    sn = __builtin_fma(z, sn, -0.16666666666666666);
    sn = __builtin_fma(z * x, sn, x);
    float pc = __builtin_fmaf(y, 2.08767569878681e-9f, -2.755731922398589e-7f);
    pc = __builtin_fmaf(y, pc, 2.48015873015873e-5f);
    pc = __builtin_fmaf(y, pc, -1.388888888888889e-3f);
    double cs = __builtin_fma(z, (double)pc, 4.1666666666666664e-2);
    cs = __builtin_fma(z, cs, -0.5);
    cs = __builtin_fma(z, cs, 1.0);
    s = (float)((q & 1) ? cs : sn);
    c = (float)((q & 1) ? sn : cs);
    if (q & 2) s = -s;
    if ((q + 1) & 2) c = -c;
}

// 8 values at any 2-byte address: the memory takes 16 bytes anywhere.
__device__ __forceinline__ kv_u4 qk_load(const uint16_t *p) {
    kv_u4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

__device__ __forceinline__ void qk_store(uint16_t *p, kv_u4 v) { __builtin_memcpy(p, &v, 16); }

typedef float qk_f4 __attribute__((ext_vector_type(4)));

// MIX: queries, keys and values follow each other without a gap, and a wavefront may hold some of two kinds or all.
template <int D, int U, bool MIX>
__global__ __launch_bounds__(QK_BLOCK) void k_qk_heads(const QkArgs a, uint32_t items) {
    constexpr int LPR = D / 8, RPW = 64 / LPR;
    __shared__ __align__(16) float turns[QK_BLOCK / 64][2][D / 2];      // each wavefront's cosines and sines
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * (QK_BLOCK / 64) + wave);
    if (item >= items) return;
    const uint32_t token = item / a.parts[2], part = item - token * a.parts[2];
    const int h1 = a.heads[0], h2 = h1 + a.heads[1];
    const int one = part < a.parts[0] ? 0 : part < a.parts[1] ? 1 : 2;      // the kind of all rows, unless MIX
    const int first = MIX ? (int)part * (RPW * U)
                          : one == 0 ? (int)part * (RPW * U)
                          : one == 1 ? h1 + (int)(part - a.parts[0]) * (RPW * U)
                                     : h2 + (int)(part - a.parts[1]) * (RPW * U);
    const int rows = !MIX && one == 0 ? h1 : !MIX && one == 1 ? h2 : h2 + a.heads[2];
    auto kind_of = [&](int r) { return !MIX ? one : r < h1 ? 0 : r < h2 ? 1 : 2; };
    const int ch = (lane % LPR) * 8;
    // where row r would lie if it were a query, a key, a value
    const uint16_t *const qs = a.x[0] + (int64_t)token * a.xs[0], *const ks = a.x[1] + (int64_t)token * a.xs[1] - (int64_t)h1 * D,
                   *const vs = a.x[2] + (int64_t)token * a.xs[2] - (int64_t)h2 * D;
    int place[U];
    kv_u4 raw[U];
    kv_h8 w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        // rows past the last are read as the item's first, so that every lane of the reductions holds a value
        place[i] = first + i * RPW + lane / LPR;
        const int r = place[i] < rows ? place[i] : first;
        const int kind = kind_of(r);
        raw[i] = qk_load((kind == 0 ? qs : kind == 1 ? ks : vs) + (int64_t)r * D + ch);
        const uint16_t *weight = kind == 0 ? a.weight[0] : kind == 1 ? a.weight[1] : nullptr;
        if (weight != nullptr) w[i] = __builtin_bit_cast(kv_h8, *reinterpret_cast<const kv_u4 *>(weight + ch));
    }
    const int rot = first < h2 ? a.rot : 0, half = rot / 2;
    float cs[8], sn[8];
    int partner = lane;
    const bool turned = ch < rot;
    if (rot > 0) {
        // each pair's angle once for the wavefront, by way of its own LDS
        const int32_t p = a.positions[token];
#pragma unroll
        for (int i = 0; i < D / 2; i += 64) {
            const int j = i + lane;
            if (j < half) qk_sincos((uint64_t)(int64_t)p * a.freq[j], turns[wave][1][j], turns[wave][0][j]);
        }
        __builtin_amdgcn_wave_barrier();
        const bool upper = !a.interleaved && ch >= half;
        if (turned && a.interleaved) {
            const qk_f4 c = *reinterpret_cast<const qk_f4 *>(&turns[wave][0][ch / 2]);
            const qk_f4 s = *reinterpret_cast<const qk_f4 *>(&turns[wave][1][ch / 2]);
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] = c[e / 2], sn[e] = (e & 1) ? s[e / 2] : -s[e / 2];
        } else if (turned) {
            partner = upper ? lane - half / 8 : lane + half / 8;
            const int i0 = upper ? ch - half : ch;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const qk_f4 c = *reinterpret_cast<const qk_f4 *>(&turns[wave][0][i0 + 4 * q]);
                const qk_f4 s = *reinterpret_cast<const qk_f4 *>(&turns[wave][1][i0 + 4 * q]);
#pragma unroll
                for (int e = 0; e < 4; ++e) cs[4 * q + e] = c[e], sn[4 * q + e] = upper ? s[e] : -s[e];
            }
        }
    }
    // (an item of queries alone has no slot to read: without kv heads there need be none)
    const int64_t slot = a.cached && min(first + RPW * U, rows) > h1 ? a.slots[token] : -1;
    const bool stored = slot >= 0 && slot < a.nslots;
    const int64_t page = (stored ? slot : 0) >> a.page_shift;
    const int64_t off = (stored ? slot : 0) & (((int64_t)1 << a.page_shift) - 1);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const bool live = place[i] < rows;
        const int r = live ? place[i] : first, kind = kind_of(r);
        if (kind < 2) {
#pragma clang fp contract(off)
            const kv_h8 x = __builtin_bit_cast(kv_h8, raw[i]);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (float)x[e];
            if ((kind == 0 ? a.weight[0] : a.weight[1]) != nullptr) {
                float sum;
                if constexpr (D == 64)
                    sum = ((y[0] * y[0] + y[1] * y[1]) + (y[2] * y[2] + y[3] * y[3])) +
                          ((y[4] * y[4] + y[5] * y[5]) + (y[6] * y[6] + y[7] * y[7]));
                else
                    sum = (((y[0] * y[0] + y[1] * y[1]) + y[2] * y[2]) + y[3] * y[3]) +
                          (((y[4] * y[4] + y[5] * y[5]) + y[6] * y[6]) + y[7] * y[7]);
#pragma unroll
                for (int d = 1; d < LPR; d <<= 1) sum += kv_other(sum, d);
                const float root = sqrtf(sum * (1.0f / D) + a.eps), rc = 1.0f / root, rz = root < INFINITY ? root : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float q0 = y[e] * rc;
                    y[e] = __builtin_fmaf(__builtin_fmaf(-q0, rz, y[e]), rc, q0) * (float)w[i][e];
                }
            }
            if (rot > 0 && !a.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float other = __shfl(y[e], partner, 64);
                    if (turned) y[e] = y[e] * cs[e] + other * sn[e];
                }
            } else if (turned) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float y1 = y[e], y2 = y[e + 1];
                    y[e] = y1 * cs[e] + y2 * sn[e];
                    y[e + 1] = y2 * cs[e + 1] + y1 * sn[e + 1];
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                raw[i][e] = bsp_f2h(bsp_rounded(y[2 * e])) | ((uint32_t)bsp_f2h(bsp_rounded(y[2 * e + 1])) << 16);
        }
        if (kind == 0 || !a.cached) {
            uint16_t *o = kind == 0 ? a.o[0] + (int64_t)token * a.os[0] : a.o[1] + (int64_t)token * a.os[1] - (int64_t)h1 * D;
            if (live) qk_store(o + (int64_t)r * D + ch, raw[i]);
            continue;
        }
        const bool value = kind == 2;
        const int64_t row = ((page * a.heads[1] + (r - (value ? h2 : h1))) << a.page_shift) + off;
        uint8_t *codes = value ? a.codes[1] : a.codes[0];
        if (a.kind == BSP_FP16) {
            if (live && stored) *reinterpret_cast<kv_u4 *>(codes + row * (2 * D) + 2 * ch) = raw[i];
        } else {
            uint32_t u[8], word;
            kv_quantise<LPR>(raw[i], a.kind == BSP_INT8 ? 255.0f : 15.0f, u, word);
            if (!(live && stored)) continue;
            if (a.kind == BSP_INT8)
                kv_store_codes<BSP_INT8>(codes, row * D + ch, u);
            else
                kv_store_codes<BSP_INT4>(codes, row * D + ch, u);
            if (ch == 0) (value ? a.words[1] : a.words[0])[row] = word;
        }
    }
}

// A launch holds fewer than 2^32 threads: more tokens go in several.
template <int D, int U, bool MIX>
void qk_launch_u(const QkArgs &all, hipStream_t stream) {
    constexpr int RUN = 64 / (D / 8) * U;
    uint32_t parts[3], total = 0;
    for (int k = 0; k < 3; ++k) parts[k] = total += (uint32_t)((all.heads[k] + RUN - 1) / RUN);
    if (MIX) parts[2] = total = (uint32_t)((all.heads[0] + all.heads[1] + all.heads[2] + RUN - 1) / RUN);
    const uint32_t most = std::max<uint32_t>((UINT32_C(1) << 25) / total, 1);
    for (uint32_t t = 0; t < all.n; t += std::min(most, all.n - t)) {
        QkArgs a = all;
        a.n = std::min(most, all.n - t);
        for (int k = 0; k < 3; ++k) {
            a.parts[k] = parts[k];
            if (a.heads[k] > 0) a.x[k] += t * a.xs[k];
            if (k < 2 && a.o[k] != nullptr) a.o[k] += t * a.os[k];
        }
        if (a.positions != nullptr) a.positions += t;
        if (a.slots != nullptr) a.slots += t;
        const uint32_t items = a.n * total;
        const unsigned grid = (items + QK_BLOCK / 64 - 1) / (QK_BLOCK / 64);
        hipLaunchKernelGGL((k_qk_heads<D, U, MIX>), dim3(grid), dim3(QK_BLOCK), 0, stream, a, items);
    }
}

// Heads of 128, many of them: two groups a wavefront (8192 tokens x 64 heads 51.8 us against 61.3, into an int8 cache
// 79 against 94; 512 x 64 6.8 against 7.1, 512 x 80 7.5 against 7.7; 128 x 80 5.0 against 4.4). Heads of 64, 8 to
// a group, gain nothing (8192 x 40 20.5 against 20.6, with an int8 cache 28.4 against 26.2), nor do those of 256 (23.7
// against 25.5, 32.1 against 30.9).
//
// Kinds mixed in a wavefront where that takes over a twelfth fewer of them: 8192 tokens x (5 + 1) heads of 128 10.3 us against 14.2,
// (28 + 4, with values, into an int8 cache) 33.5 against 37.8, (8 + 2 + 2) heads of 64 x 6120 9.2 against 10.3. Where it
// takes as many, what is then found out lane by lane costs more: (32 + 32) 56.3 against 51.8.
template <int D, int U>
void qk_launch_mix(const QkArgs &a, hipStream_t stream) {
    constexpr int RUN = 64 / (D / 8) * U;
    int apart = 0, all = 0;
    for (int k = 0; k < 3; ++k) apart += (a.heads[k] + RUN - 1) / RUN, all += a.heads[k];
    if (12 * ((all + RUN - 1) / RUN) < 11 * apart)
        qk_launch_u<D, U, true>(a, stream);
    else
        qk_launch_u<D, U, false>(a, stream);
}

template <int D>
void qk_launch(const QkArgs &a, hipStream_t stream) {
    if (D == 128 && (int64_t)a.n * (a.heads[0] + a.heads[1] + a.heads[2]) >= 32768)
        qk_launch_mix<128, 2>(a, stream);
    else
        qk_launch_mix<D, 1>(a, stream);
}

int qk_common(QkArgs &a, int64_t n, int64_t hq, int64_t hkv, int64_t D, const bsp_rotation *r, bool values,
              hipStream_t stream) {
    if (D != 64 && D != 128 && D != 256) return BSP_E_UNSUPPORTED;
    if (hq > INT64_C(1) << 20 || hkv > INT64_C(1) << 20) return BSP_E_OVERFLOW;
    if (n >= (INT64_C(1) << 28) / std::max<int64_t>(hq + 2 * hkv, 1)) return BSP_E_OVERFLOW;
    if (r->rot < 0 || r->rot > D || r->rot % 16 != 0) return BSP_E_UNSUPPORTED;
    if (!(r->eps >= 0.0f) || std::isinf(r->eps)) return BSP_E_ARG;
    if ((((uintptr_t)r->q_weight | (uintptr_t)r->k_weight) & 15u) != 0) return BSP_E_ARG;
    if (n == 0 || hq + hkv == 0) return BSP_OK;
    const int64_t heads[3] = {hq, hkv, values ? hkv : 0};
    a.cached = values;
    uintptr_t bits = 0;
    for (int k = 0; k < 3; ++k) {
        a.heads[k] = (int)heads[k];
        if (heads[k] == 0) continue;
        const bool out = k == 0 || (k == 1 && !values);
        if (a.x[k] == nullptr || (out && a.o[k] == nullptr)) return BSP_E_ARG;
        if (a.xs[k] < heads[k] * D || (out && a.os[k] < heads[k] * D)) return BSP_E_ARG;
        bits |= (uintptr_t)a.x[k];
        if (out) bits |= (uintptr_t)a.o[k];
    }
    if ((bits & 1u) != 0) return BSP_E_ARG;
    if (r->rot > 0) {
        if (r->freq == nullptr || r->positions == nullptr) return BSP_E_ARG;
        if (((uintptr_t)r->freq & 7u) != 0 || ((uintptr_t)r->positions & 3u) != 0) return BSP_E_ARG;
    }
    a.weight[0] = r->q_weight, a.weight[1] = r->k_weight;
    a.freq = r->freq, a.positions = r->positions;
    a.eps = r->eps, a.rot = (int)r->rot, a.interleaved = r->interleaved != 0;
    a.n = (uint32_t)n;
    if (D == 64)
        qk_launch<64>(a, stream);
    else if (D == 128)
        qk_launch<128>(a, stream);
    else
        qk_launch<256>(a, stream);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}

}  // namespace

extern "C" int qk_norm_rope_f16(const uint16_t *Q, int64_t q_stride, const uint16_t *K, int64_t k_stride, int64_t n,
                                int64_t q_heads, int64_t kv_heads, int64_t head_dim, const bsp_rotation *rotation,
                                uint16_t *Qo, int64_t qo_stride, uint16_t *Ko, int64_t ko_stride,
                                hipStream_t stream) {
    if (rotation == nullptr || n < 0 || q_heads < 0 || kv_heads < 0) return BSP_E_ARG;
    QkArgs a{};
    a.x[0] = Q, a.x[1] = K, a.xs[0] = q_stride, a.xs[1] = k_stride;
    a.o[0] = Qo, a.o[1] = Ko, a.os[0] = qo_stride, a.os[1] = ko_stride;
    return qk_common(a, n, q_heads, kv_heads, head_dim, rotation, false, stream);
}

extern "C" int qk_norm_rope_append_f16(const uint16_t *Q, int64_t q_stride, const uint16_t *K, int64_t k_stride,
                                       const uint16_t *V, int64_t v_stride, int64_t n, int64_t q_heads,
                                       const bsp_rotation *rotation, const bsp_kv_cache *cache, const int64_t *slots,
                                       uint16_t *Qo, int64_t qo_stride, hipStream_t stream) {
    const int rc = kv_check_cache(cache);
    if (rc != BSP_OK) return rc;
    if (rotation == nullptr || n < 0 || q_heads < 0) return BSP_E_ARG;
    if (n > 0 && cache->kv_heads > 0 && (slots == nullptr || ((uintptr_t)slots & 7u) != 0)) return BSP_E_ARG;
    QkArgs a{};
    a.x[0] = Q, a.x[1] = K, a.x[2] = V, a.xs[0] = q_stride, a.xs[1] = k_stride, a.xs[2] = v_stride;
    a.o[0] = Qo, a.os[0] = qo_stride;
    a.slots = slots;
    a.codes[0] = (uint8_t *)cache->k, a.codes[1] = (uint8_t *)cache->v;
    a.words[0] = cache->k_scale, a.words[1] = cache->v_scale;
    a.nslots = cache->num_pages * cache->page_size;
    a.kind = cache->dtype;
    a.page_shift = __builtin_ctzll((unsigned long long)cache->page_size);
    return qk_common(a, n, q_heads, cache->kv_heads, cache->head_dim, rotation, true, stream);
}
