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
    int total_q, max_q, hq, hkv, num_pages, page_shift, B;
    int q_vec, o_vec;              // Q / O rows on 16-byte boundaries
    int row_blocks;                // blocks of query rows
    int chunks, min_per, max_chunks;   // pieces aimed at (0: one per sequence), least tiles of one, most pieces
    float scale;
    float *part;                   // partial sums of the pieces
    uint32_t *counters;            // arrivals per (sequence, kv head, row block), zero between calls
};

typedef float at_f4 __attribute__((ext_vector_type(4)));
typedef uint32_t at_u4 __attribute__((ext_vector_type(4)));

// 8 channels of a finished row: sums times inv, rounded to fp16.
__device__ __forceinline__ void at_write(const AtArgs &a, int q0, int kvh, int G, int row, int d, int D, at_f4 y0,
                                         at_f4 y1, float inv) {
    const int t = row / G, g = row - t * G;
    uint16_t *o = a.O + (int64_t)(q0 + t) * a.o_stride + (int64_t)(kvh * G + g) * D + d;
    uint16_t h[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = bsp_f2h(y0[e] * inv), h[4 + e] = bsp_f2h(y1[e] * inv);
    if (a.o_vec) {
        at_u4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (uint32_t)h[2 * e] | ((uint32_t)h[2 * e + 1] << 16);
        *reinterpret_cast<at_u4 *>(o) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = h[e];
    }
}

typedef _Float16 at_h8 __attribute__((ext_vector_type(8)));
typedef _Float16 at_h2 __attribute__((ext_vector_type(2)));

#define AT_WAVES 4
#define AT_TILE 32                 // cached tokens per wavefront and step
#define AT_BOOST 6.0f              // log2: the weights' scale, 2^6 at the running maximum
#define AT_SLACK 8.0f              // log2: how far a score may pass the running maximum before it is moved
#define AT_LOW -1e30f              // the running maximum before any score

// Bytes a lane reads of a K row (its quarter of the channels) and of a V row
// (its sixteenth), in dwords (V: at least one).
template <int KIND, int D>
struct AtShape {
    static constexpr int ROW = KIND == BSP_FP16 ? 2 * D : KIND == BSP_INT8 ? D : D / 2;
    static constexpr int KW = ROW / 16;                      // dwords per K row and lane
    static constexpr int VB = ROW / 16;                      // bytes per V row and lane
    static constexpr int VW = VB < 4 ? 1 : VB / 4;
    static constexpr int NT = D / 16;                        // 16-channel blocks of the output
    static constexpr int STEPS = D / 32;                     // MFMAs along the channels
};

template <int N>
__device__ __forceinline__ void at_load(const uint8_t *p, uint32_t (&r)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const at_u4 v = reinterpret_cast<const at_u4 *>(p)[i];
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// Agent-scope 16-byte stores and loads of the partial sums: they go to the
// coherence point all XCDs share, so partials are visible to the workgroup
// that joins them once the stores have completed (aux 16: sc1).
__device__ __forceinline__ void at_ws_store(__amdgpu_buffer_rsrc_t rs, uint32_t off, at_f4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(at_u4, v), rs, off, 0, 16);
}
__device__ __forceinline__ at_f4 at_ws_load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    return __builtin_bit_cast(at_f4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 16));
}

// Bytes 2k, 2k + 1 of a dword, or byte k of two dwords, as the low bytes of
// two 16-bit lanes: fp16 subnormals u * 2^-24, which the MFMA takes exactly.
__device__ __forceinline__ uint32_t at_bytes(uint32_t hi, uint32_t lo, uint32_t sel) {
    return __builtin_amdgcn_perm(hi, lo, sel);
}

// The A operand of step `s` of the scores: 8 channels of this lane's K row.
// int4: even steps hold the even channels of 16, odd steps the odd ones times
// 16 (the codes stay where they are in their bytes).
template <int KIND>
__device__ __forceinline__ at_h8 at_k_frag(const uint32_t *k, int s) {
    at_u4 f;
    if constexpr (KIND == BSP_FP16) {
        f = at_u4{k[4 * s], k[4 * s + 1], k[4 * s + 2], k[4 * s + 3]};
    } else if constexpr (KIND == BSP_INT8) {
        const uint32_t a = k[2 * s], b = k[2 * s + 1];
        f = at_u4{at_bytes(a, a, 0x0C010C00u), at_bytes(a, a, 0x0C030C02u), at_bytes(b, b, 0x0C010C00u),
                  at_bytes(b, b, 0x0C030C02u)};
    } else {
        const uint32_t a = k[s & ~1], b = k[s | 1];
        const uint32_t m = (s & 1) ? 0x00F000F0u : 0x000F000Fu;
        f = at_u4{a & m, (a >> 8) & m, b & m, (b >> 8) & m};
    }
    return __builtin_bit_cast(at_h8, f);
}

// The B operand of step `s`: the matching channels of a query row, from its
// quarter of the row in channel order.
template <int KIND>
__device__ __forceinline__ at_h8 at_q_frag(const uint32_t *q, int s) {
    if constexpr (KIND == BSP_INT4) {
        // 16 channels of steps s & ~1 and s | 1: dword i holds channels 2i, 2i + 1
        const uint32_t *p = q + 8 * (s >> 1);
        const uint32_t sel = (s & 1) ? 0x07060302u : 0x05040100u;
        const at_u4 f = {at_bytes(p[2], p[0], sel), at_bytes(p[3], p[1], sel), at_bytes(p[6], p[4], sel),
                         at_bytes(p[7], p[5], sel)};
        return __builtin_bit_cast(at_h8, f);
    } else {
        return __builtin_bit_cast(at_h8, at_u4{q[4 * s], q[4 * s + 1], q[4 * s + 2], q[4 * s + 3]});
    }
}

// The A operand of output block `t`: channel t of this lane's channels over
// its 8 tokens. v[c] holds the lane's channels of token c.
template <int KIND, int VW>
__device__ __forceinline__ at_h8 at_v_frag(const uint32_t (&v)[8][VW], int t) {
    at_u4 f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        if constexpr (KIND == BSP_FP16) {
            f[p] = at_bytes(v[2 * p + 1][t >> 1], v[2 * p][t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
        } else if constexpr (KIND == BSP_INT8) {
            f[p] = at_bytes(v[2 * p + 1][t >> 2], v[2 * p][t >> 2], 0x0C040C00u + 0x00010001u * (t & 3));
        } else {
            const uint32_t b = at_bytes(v[2 * p + 1][t >> 3], v[2 * p][t >> 3], 0x0C040C00u + 0x00010001u * ((t >> 1) & 3));
            f[p] = b & ((t & 1) ? 0x00F000F0u : 0x000F000Fu);
        }
    }
    return __builtin_bit_cast(at_h8, f);
}

__device__ __forceinline__ float at_group_sum(float v) {      // over the four lanes of a query row
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float at_group_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

template <int KIND, int D, int RT>
struct AtWave {
    using Sh = AtShape<KIND, D>;
    static constexpr bool QUANT = KIND != BSP_FP16;
    const AtArgs &a;
    int lane, col, grp;
    int kvh, len, past, T;
    const int32_t *table;
    // per query row (the lane's column)
    at_h8 q[RT][Sh::STEPS];
    float qc[RT];                  // sum of the row's q, times the score factor
    uint64_t seen[RT];
    float m[RT], l[RT], osum[RT], psum[RT];
    at_f4 acc[RT][Sh::NT];
    float sig, rsig;               // the value steps' common power of two, and 1 / it
    float c;                       // score factor: scale * log2(e)
    // the tile in flight
    uint32_t k[2][Sh::KW], v[8][Sh::VW], kw[8], vw[8];
    int pk, pv;                    // its pages: of the lane's K rows, of its V rows

    __device__ AtWave(const AtArgs &args) : a(args) {}

    __device__ __forceinline__ int page_of(int j) const {
        const int p = table[min(j, len - 1) >> a.page_shift];
        return (unsigned)p < (unsigned)a.num_pages ? p : 0;
    }
    __device__ __forceinline__ int64_t row_of(int page, int j) const {
        return (((int64_t)page * a.hkv + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
    }
    // S tile u, A row i: token 8 (i / 4) + 4 u + i % 4, so that the scores of a
    // lane (C rows 4 g .. 4 g + 3 of both tiles) are those of 8 neighbouring
    // tokens, 8 g .. 8 g + 7: its part of the second product's B operand.
    __device__ __forceinline__ void load_pages(int j0) {
        pk = page_of(j0 + 8 * (col >> 2));
        pv = page_of(j0 + 8 * grp);
    }
    __device__ __forceinline__ void load_k(int j0) {
        const int64_t r = row_of(pk, j0 + 8 * (col >> 2) + (col & 3));
#pragma unroll
        for (int u = 0; u < 2; ++u) at_load(a.k + (r + 4 * u) * Sh::ROW + grp * (Sh::ROW / 4), k[u]);
        if constexpr (QUANT) at_load(reinterpret_cast<const uint8_t *>(a.kw + row_of(pv, j0 + 8 * grp)), kw);
    }
    __device__ __forceinline__ void load_v(int j0) {
        const int64_t r = row_of(pv, j0 + 8 * grp);
        const uint8_t *p = a.v + r * Sh::ROW + col * Sh::VB;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if constexpr (Sh::VB == 2)
                v[t][0] = *reinterpret_cast<const uint16_t *>(p + t * Sh::ROW);
            else
                at_load(p + t * Sh::ROW, v[t]);
        }
        if constexpr (QUANT) at_load(reinterpret_cast<const uint8_t *>(a.vw + r), vw);
    }

    // One tile: scores, running maximum, weights, output. MASKED: the tile
    // holds drafted tokens or the end of the sequence. The next tile's loads
    // are issued as the registers they fill fall free.
    template <bool MASKED>
    __device__ __forceinline__ void tile(int j0, int jn) {
        at_f4 x[RT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) x[rt][u] = at_f4{0.f, 0.f, 0.f, 0.f};
            if constexpr (KIND == BSP_INT4) {
                at_f4 hi[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) hi[rt] = at_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < Sh::STEPS; s += 2) {
                    const at_h8 f0 = at_k_frag<KIND>(k[u], s), f1 = at_k_frag<KIND>(k[u], s + 1);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        x[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f0, q[rt][s], x[rt][u], 0, 0, 0);
                        hi[rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f1, q[rt][s + 1], hi[rt], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[rt][u][r] = fmaf(hi[rt][r], 0.0625f, x[rt][u][r]);
            } else {
#pragma unroll
                for (int s = 0; s < Sh::STEPS; ++s) {
                    const at_h8 f = at_k_frag<KIND>(k[u], s);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        x[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, q[rt][s], x[rt][u], 0, 0, 0);
                }
            }
        }
        // scores in log2 units: scale * log2(e) * (s u.q 2^-24 2^24 + o sum(q))
        float ks[8], ko[8];
        if constexpr (QUANT) {
            const float cc = c * 16777216.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ks[e] = kv_word_step(kw[e]) * cc, ko[e] = kv_word_offset(kw[e]);
        }
        load_pages(jn);
        load_k(jn);
        uint32_t ok[RT];
        float top[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            ok[rt] = 0xFFu;
            top[rt] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y = x[rt][e >> 2][e & 3];
                if constexpr (QUANT)
                    y = fmaf(y, ks[e], ko[e] * qc[rt]);
                else
                    y *= c;
                if constexpr (MASKED) {
                    const int j = j0 + 8 * grp + e, dj = j - past;
                    const bool see = j < len && (dj < 0 || (dj < BSP_TREE_MAX && (seen[rt] >> (dj & 63) & 1)));
                    y = see ? y : -INFINITY;
                    if (!see) ok[rt] &= ~(1u << e);
                }
                x[rt][e >> 2][e & 3] = y;
                top[rt] = fmaxf(top[rt], y);
            }
        }
        float vs[8], vo[8];
        float smax = 0.f;
        if constexpr (QUANT) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t w = vw[e];
                if constexpr (MASKED) w = j0 + 8 * grp + e < len ? w : 0u;
                vs[e] = kv_word_step(w), vo[e] = kv_word_offset(w);
                smax = fmaxf(smax, vs[e] < INFINITY ? vs[e] : 0.f);
            }
        }
        // Move the running maximum only when a score passes it by more than
        // the slack (the weights stay fp16: 2^(6 + 8) at most), and the value
        // steps' scale when a step passes it.
        bool move = QUANT && smax > sig;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) move |= top[rt] > m[rt] + AT_SLACK;
        if (__ballot(move) != 0) {
            float f[RT], fs = 1.f;
            if constexpr (QUANT) {
                const float sm = fmaxf(at_group_max(smax), sig);
                const uint32_t b = (__builtin_bit_cast(uint32_t, sm) + 0x7FFFFFu) & 0x7F800000u;
                fs = sig * __builtin_bit_cast(float, 0x7F000000u - b);
                sig = __builtin_bit_cast(float, b);
                rsig = __builtin_bit_cast(float, 0x7F000000u - b);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float mn = fmaxf(m[rt], at_group_max(top[rt]));
                f[rt] = __builtin_amdgcn_exp2f(m[rt] - mn);
                m[rt] = mn;
                l[rt] *= f[rt], osum[rt] *= f[rt];
                f[rt] *= fs;
                psum[rt] *= f[rt];
#pragma unroll
                for (int t = 0; t < Sh::NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[rt][t][r] *= f[rt];
            }
        }
        at_h8 p[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float mb = m[rt] - AT_BOOST;
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float ex = __builtin_amdgcn_exp2f(x[rt][e >> 2][e & 3] - mb);
                l[rt] += ex;
                if constexpr (QUANT) {
                    constexpr float mid = KIND == BSP_INT8 ? 128.0f : 8.0f;
                    float wt = ex * (vs[e] * rsig), wo = ex * fmaf(mid, vs[e], vo[e]);
                    if constexpr (MASKED) {      // a masked row's word may be NaN
                        const bool see = ok[rt] >> e & 1;
                        wt = see ? wt : 0.f, wo = see ? wo : 0.f;
                    }
                    osum[rt] += wo;
                    w[e] = wt;
                } else {
                    w[e] = ex;
                }
            }
            // to fp16, nearest even: 11 bits of each weight, which average out over the tokens
#pragma unroll
            for (int e = 0; e < 8; ++e) p[rt][e] = (_Float16)w[e];
            if constexpr (QUANT) {
                const at_h2 one = {(_Float16)1.f, (_Float16)1.f};
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    psum[rt] = __builtin_amdgcn_fdot2(at_h2{p[rt][e], p[rt][e + 1]}, one, psum[rt], false);
            }
        }
        bool bad = false;
        if constexpr (MASKED && !QUANT) {
            // rows past the end: whatever lies there is not a number to multiply with zero
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int i = 0; i < Sh::VW; ++i) {
                    v[t][i] = j0 + 8 * grp + t < len ? v[t][i] : 0u;
                    bad |= (v[t][i] & 0x7C00u) == 0x7C00u || (v[t][i] & 0x7C000000u) == 0x7C000000u;
                }
            bad = __ballot(bad) != 0;
        }
        if (MASKED && !QUANT && bad) {
            // An infinite or NaN value: out of the product, and NaN in that
            // channel for the rows that see its token.
#pragma unroll
            for (int t = 0; t < Sh::NT; ++t) {
                at_h8 f = at_v_frag<KIND>(v, t), g;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const _Float16 fe = f[e];
                    const bool nf = (__builtin_bit_cast(uint16_t, fe) & 0x7C00u) == 0x7C00u;
                    g[e] = nf ? (_Float16)1.f : (_Float16)0.f;
                    f[e] = nf ? (_Float16)0.f : fe;
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    at_h8 see;
#pragma unroll
                    for (int e = 0; e < 8; ++e) see[e] = (ok[rt] >> e & 1) ? (_Float16)1.f : (_Float16)0.f;
                    acc[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, p[rt], acc[rt][t], 0, 0, 0);
                    const at_f4 n = __builtin_amdgcn_mfma_f32_16x16x32_f16(g, see, at_f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[rt][t][r] = n[r] > 0.f ? __builtin_nanf("") : acc[rt][t][r];
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < Sh::NT; ++t) {
                const at_h8 f = at_v_frag<KIND>(v, t);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    acc[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, p[rt], acc[rt][t], 0, 0, 0);
            }
        }
        load_v(jn);
    }
};

// Which sequence and which of its chunks workgroup `ch` of a (kv head, row
// block) has. A chunk is per tiles of AT_TILE tokens; per follows from all the
// sequences' lengths, so that chunks are alike whatever the lengths are.
struct AtPlace {
    int b, first, count, per;      // sequence; its first chunk's number; its chunks; tiles per chunk
};

__device__ __forceinline__ int at_len(const AtArgs &a, int b) {
    return (int)min((int64_t)max(a.kv_lens[b], 0), a.table_width << a.page_shift);
}

__device__ __forceinline__ AtPlace at_place(const AtArgs &a, int ch) {
    const int lane = threadIdx.x & 63;
    AtPlace p{-1, 0, 1, 1 << 30};
    if (a.chunks == 0) {           // no split
        p.b = ch < a.B ? ch : -1;
        p.first = ch;
        return p;
    }
    int total = 0;
    for (int b = lane; b < a.B; b += 64) total += (at_len(a, b) + AT_TILE - 1) / AT_TILE;
    total = bsp_wave_sum(total);
    p.per = max(a.min_per, (total + a.chunks - 1) / a.chunks);
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        const int n = b < a.B ? max(1, ((at_len(a, b) + AT_TILE - 1) / AT_TILE + p.per - 1) / p.per) : 0;
        int s = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d, 64);
            if (lane >= d) s += o;
        }
        const uint64_t hit = __ballot(ch < before + s);
        if (hit != 0) {
            const int at = __builtin_ctzll(hit);
            p.b = b0 + at;
            p.count = __shfl(n, at, 64);
            p.first = before + __shfl(s, at, 64) - p.count;
            return p;
        }
        before += __shfl(s, 63, 64);
    }
    return p;
}

template <int KIND, int D, int RT>
__global__ __launch_bounds__(64 * AT_WAVES) void k_at(const AtArgs a) {
    using Sh = AtShape<KIND, D>;
    extern __shared__ __attribute__((aligned(16))) float at_smem[];
    constexpr int LD = D + 4;                      // floats per row of a wavefront's output in LDS
    float *s_acc = at_smem;                        // [AT_WAVES][16][LD]
    float *s_m = s_acc + AT_WAVES * 16 * LD;       // [AT_WAVES][16]
    float *s_l = s_m + AT_WAVES * 16;
    int *s_flag = reinterpret_cast<int *>(s_l + AT_WAVES * 16);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // workgroups 8 apart share an XCD and its L2: the row blocks of one piece
    // of the cache are 8 apart
    const int group = blockIdx.x / (8 * a.row_blocks), in = blockIdx.x % (8 * a.row_blocks);
    const int rb = in >> 3, piece = group * 8 + (in & 7);
    const int ch = piece / a.hkv;
    if (ch >= a.max_chunks) return;
    AtWave<KIND, D, RT> w(a);
    w.kvh = piece - ch * a.hkv;
    const AtPlace pl = at_place(a, ch);
    if (pl.b < 0) return;
    const int b = __builtin_amdgcn_readfirstlane(pl.b);
    const int q0 = min(max(a.q_start[b], 0), a.total_q), q1 = min(max(a.q_start[b + 1], q0), a.total_q);
    const int G = a.hq / a.hkv;
    const int rows = min(q1 - q0, a.max_q) * G;    // query rows of this kv head
    const int r0 = rb * 16 * RT;
    if (r0 >= rows) return;
    w.lane = threadIdx.x & 63, w.col = w.lane & 15, w.grp = w.lane >> 4;
    w.len = at_len(a, b);
    w.T = q1 - q0;
    w.past = w.len - w.T;
    w.table = a.table + (int64_t)b * a.table_width;
    w.c = a.scale * 1.44269504088896341f;
    w.sig = 0x1p-100f, w.rsig = 0x1p100f;
    const int nt = (w.len + AT_TILE - 1) / AT_TILE;
    const int t0 = min(nt, (ch - pl.first) * pl.per), t1 = min(nt, t0 + min(pl.per, nt));
    const int tile0 = t0 + wave;
    if (tile0 < t1) {
        w.load_pages(tile0 * AT_TILE);
        w.load_k(tile0 * AT_TILE);
        w.load_v(tile0 * AT_TILE);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = r0 + 16 * rt + w.col;
        const bool in_rows = row < rows;
        const int t = in_rows ? row / G : 0, g = in_rows ? row - t * G : 0;
        const uint16_t *src = a.Q + (int64_t)(q0 + t) * a.q_stride + (int64_t)(w.kvh * G + g) * D + w.grp * (D / 4);
        uint32_t qr[D / 8];
        if (a.q_vec) {
            at_load(reinterpret_cast<const uint8_t *>(src), qr);
        } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) qr[i] = (uint32_t)src[2 * i] | ((uint32_t)src[2 * i + 1] << 16);
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            if (!in_rows) qr[i] = 0u;
            const at_h2 h = __builtin_bit_cast(at_h2, qr[i]);
            sum += (float)h.x + (float)h.y;
        }
        w.qc[rt] = at_group_sum(sum) * w.c;
#pragma unroll
        for (int s = 0; s < Sh::STEPS; ++s) w.q[rt][s] = at_q_frag<KIND>(qr, s);
        w.seen[rt] = a.mask != nullptr ? a.mask[q0 + t] : (uint64_t)-1 >> (63 - min(t, 63));
        w.m[rt] = AT_LOW, w.l[rt] = 0.f, w.osum[rt] = 0.f, w.psum[rt] = 0.f;
#pragma unroll
        for (int i = 0; i < Sh::NT; ++i) w.acc[rt][i] = at_f4{0.f, 0.f, 0.f, 0.f};
    }
    for (int t = tile0; t < t1; t += AT_WAVES) {
        const int j0 = t * AT_TILE, jn = (t + AT_WAVES < t1 ? t + AT_WAVES : t) * AT_TILE;
        if (j0 + AT_TILE <= w.past)
            w.template tile<false>(j0, jn);
        else
            w.template tile<true>(j0, jn);
    }

    // Join the wavefronts, row tile by row tile; then write the rows, or post
    // them for the last workgroup of the sequence to join.
    const int unit = (b * a.hkv + w.kvh) * a.row_blocks + rb;
    const uint32_t slot_bytes = 16u * RT * (D + 4) * 4u;     // [row][D] sums, then [row] (m, l, 0, 0)
    const int64_t slot = (int64_t)ch * a.hkv * a.row_blocks + w.kvh * a.row_blocks + rb;
    const bool split = pl.count > 1;
    const int chunk = 16 * D / 8;                            // 8-channel pieces of a row tile
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if (r0 + 16 * rt >= rows) break;
        if (rt > 0) __syncthreads();
        const float l = at_group_sum(w.l[rt]);
        float os = 0.f, ps = 0.f, up = 1.f;
        if constexpr (AtWave<KIND, D, RT>::QUANT) {
            os = at_group_sum(w.osum[rt]);
            ps = at_group_sum(w.psum[rt]) * (KIND == BSP_INT8 ? 128.0f : 8.0f);
            up = 16777216.0f;
        }
        if (w.grp == 0) s_m[wave * 16 + w.col] = w.m[rt], s_l[wave * 16 + w.col] = l;
        float *o = s_acc + (wave * 16 + w.col) * LD;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int t = 0; t < Sh::NT; t += 4) {
                at_f4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float z = w.acc[rt][t + i][r];
                    if constexpr (AtWave<KIND, D, RT>::QUANT) {
                        const float h = KIND == BSP_INT4 && (i & 1) ? up * 0.0625f : up;
                        z = fmaf(w.sig, fmaf(z, h, -ps), os);
                    }
                    y[i] = z;
                }
                *reinterpret_cast<at_f4 *>(o + (4 * w.grp + r) * Sh::NT + t) = y;
            }
        __syncthreads();
        for (int i = threadIdx.x; i < chunk; i += 64 * AT_WAVES) {
            const int row = i / (D / 8), d = (i % (D / 8)) * 8;
            const int ri = r0 + 16 * rt + row;
            if (ri >= rows) continue;
            float mx = s_m[row];
#pragma unroll
            for (int k = 1; k < AT_WAVES; ++k) mx = fmaxf(mx, s_m[k * 16 + row]);
            at_f4 y0 = {0.f, 0.f, 0.f, 0.f}, y1 = y0;
            float lt = 0.f;
#pragma unroll
            for (int k = 0; k < AT_WAVES; ++k) {
                const float f = __builtin_amdgcn_exp2f(s_m[k * 16 + row] - mx);
                lt = fmaf(s_l[k * 16 + row], f, lt);
                const at_f4 *src = reinterpret_cast<const at_f4 *>(s_acc + (k * 16 + row) * LD + d);
                const at_f4 z0 = src[0], z1 = src[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) y0[e] = fmaf(z0[e], f, y0[e]), y1[e] = fmaf(z1[e], f, y1[e]);
            }
            if (split) {
                const __amdgpu_buffer_rsrc_t rs = bsp_rsrc(a.part + slot * (slot_bytes / 4), slot_bytes);
                const uint32_t at = ((uint32_t)(16 * rt + row) * D + d) * 4u;
                at_ws_store(rs, at, y0), at_ws_store(rs, at + 16, y1);
                if (d == 0) at_ws_store(rs, (16u * RT * D + 4u * (16 * rt + row)) * 4u, at_f4{mx, lt, 0.f, 0.f});
            } else {
                const float inv = lt == 0.f ? 0.f : 1.0f / lt;
                at_write(a, q0, w.kvh, G, ri, d, D, y0, y1, inv);
            }
        }
    }
    if (!split) return;
    __builtin_amdgcn_s_waitcnt(0);      // this thread's partial stores completed
    __syncthreads();
    if (threadIdx.x == 0)
        *s_flag = (int)__hip_atomic_fetch_add(&a.counters[unit], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*s_flag != pl.count - 1) return;
    const int64_t stride = (int64_t)a.hkv * a.row_blocks * (slot_bytes / 4);
    const float *base = a.part + (int64_t)pl.first * stride + (int64_t)(w.kvh * a.row_blocks + rb) * (slot_bytes / 4);
    for (int i = threadIdx.x; i < min(16 * RT, rows - r0) * (D / 8); i += 64 * AT_WAVES) {
        const int row = i / (D / 8), d = (i % (D / 8)) * 8;
        const uint32_t at = ((uint32_t)row * D + d) * 4u, at_ml = (16u * RT * D + 4u * row) * 4u;
        at_f4 y0 = {0.f, 0.f, 0.f, 0.f}, y1 = y0;
        float mx = AT_LOW, lt = 0.f;
        for (int s = 0; s < pl.count; ++s) {      // in chunk order
            const __amdgpu_buffer_rsrc_t rs = bsp_rsrc(base + s * stride, slot_bytes);
            const at_f4 ml = at_ws_load(rs, at_ml), z0 = at_ws_load(rs, at), z1 = at_ws_load(rs, at + 16);
            const float mn = fmaxf(mx, ml.x);
            const float f = __builtin_amdgcn_exp2f(mx - mn), g = __builtin_amdgcn_exp2f(ml.x - mn);
            mx = mn;
            lt = lt * f + ml.y * g;
#pragma unroll
            for (int e = 0; e < 4; ++e) y0[e] = y0[e] * f + z0[e] * g, y1[e] = y1[e] * f + z1[e] * g;
        }
        at_write(a, q0, w.kvh, G, r0 + row, d, D, y0, y1, lt == 0.f ? 0.f : 1.0f / lt);
    }
    if (threadIdx.x == 0) __hip_atomic_store(&a.counters[unit], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The plan of a call: query rows per workgroup, row blocks, and how many
// pieces the cached tokens of all sequences are cut into.
struct AtPlan {
    int rt, row_blocks, chunks, min_per, max_chunks;
    int64_t ws_bytes;
};

#define AT_WS_COUNTERS 16384           // arrival counters at the start of a workspace
#define AT_GROUPS 768                  // workgroups aimed at: three a CU

AtPlan at_plan(const bsp_kv_cache *c, int64_t table_width, int64_t B, int64_t max_q, int64_t hq, bool split) {
    AtPlan p{};
    const int64_t rows = max_q * (hq / c->kv_heads);
    p.rt = rows <= 16 || c->head_dim == 256 ? 1 : 2;
    p.row_blocks = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    p.max_chunks = (int)B;
    p.min_per = 8;
    const int64_t per_chunk = c->kv_heads * p.row_blocks;
    const int64_t tiles = (table_width * c->page_size + AT_TILE - 1) / AT_TILE;      // of the longest sequence
    if (split && B * per_chunk <= AT_WS_COUNTERS && tiles > p.min_per) {
        const int64_t want = (AT_GROUPS + per_chunk - 1) / per_chunk;
        const int64_t most = B * ((tiles + p.min_per - 1) / p.min_per);
        if (2 * want > B) {
            p.chunks = (int)std::min(want, most);
            p.max_chunks = (int)(p.chunks + B);
            p.ws_bytes = AT_WS_COUNTERS * 4 + (int64_t)p.max_chunks * per_chunk * 16 * p.rt * (c->head_dim + 4) * 4;
        }
    }
    return p;
}

template <int KIND, int D, int RT>
void at_launch_t(const AtArgs &a, hipStream_t stream) {
    const size_t lds = (size_t)(AT_WAVES * 16 * (D + 4) + 2 * AT_WAVES * 16 + 4) * 4;
    const int64_t pieces = ((int64_t)a.max_chunks * a.hkv + 7) / 8 * 8;
    (void)hipFuncSetAttribute((const void *)k_at<KIND, D, RT>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL((k_at<KIND, D, RT>), dim3((unsigned)(pieces * a.row_blocks)), dim3(64 * AT_WAVES), lds, stream, a);
}

template <int KIND>
void at_launch(const AtArgs &a, int64_t D, int rt, hipStream_t stream) {
    if (D == 64) {
        if (rt == 1) at_launch_t<KIND, 64, 1>(a, stream); else at_launch_t<KIND, 64, 2>(a, stream);
    } else if (D == 128) {
        if (rt == 1) at_launch_t<KIND, 128, 1>(a, stream); else at_launch_t<KIND, 128, 2>(a, stream);
    } else {
        at_launch_t<KIND, 256, 1>(a, stream);
    }
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
    *bytes = B == 0 || max_q == 0 || q_heads == 0 ? 0 : at_plan(cache, table_width, B, max_q, q_heads, true).ws_bytes;
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
    const AtPlan p = at_plan(cache, table_width, B, max_q, q_heads, workspace != nullptr);
    if (p.ws_bytes > workspace_bytes) return BSP_E_CAPACITY;
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
    a.B = (int)B;
    a.q_vec = ((uintptr_t)Q & 15u) == 0 && (q_stride & 7) == 0;
    a.o_vec = ((uintptr_t)O & 15u) == 0 && (o_stride & 7) == 0;
    a.row_blocks = p.row_blocks, a.chunks = p.chunks, a.min_per = p.min_per, a.max_chunks = p.max_chunks;
    a.counters = (uint32_t *)workspace;
    a.part = p.ws_bytes > 0 ? (float *)((uint8_t *)workspace + AT_WS_COUNTERS * 4) : nullptr;
    if (cache->dtype == BSP_FP16)
        at_launch<BSP_FP16>(a, cache->head_dim, p.rt, stream);
    else if (cache->dtype == BSP_INT8)
        at_launch<BSP_INT8>(a, cache->head_dim, p.rt, stream);
    else
        at_launch<BSP_INT4>(a, cache->head_dim, p.rt, stream);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
