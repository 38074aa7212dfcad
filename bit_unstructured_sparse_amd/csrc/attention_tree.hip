// attention_tree.hip -- attention of drafted token trees over the paged
// key/value cache, for gfx950.
//
// Mathematics. For one kv head, with query rows r (drafted token, query head)
// and cached tokens j, x_rj = scale log2(e) q_r.k_j and
//     O_r = sum_j 2^(x_rj - m_r) v_j / sum_j 2^(x_rj - m_r)
// over the tokens r sees, in one pass over the cache: m_r is a running maximum,
// and sums made before it moved are scaled by 2^(old - new). A quantised row
// is s u + o (u unsigned codes), so
//     q.k_j = s_j (q.u_j) + o_j sum(q),
//     sum_j w_j v_j = sum_j (w_j s_j) u_j + sum_j w_j o_j :
// the codes go through the products as they are, and steps and offsets are
// applied to scores and weights, per token and not per channel.
//
// Both products are v_mfma_f32_16x16x32_f16. Scores are computed transposed (A =
// 16 cached tokens, B = 16 query rows), so that a lane ends with the scores of
// 8 neighbouring tokens for one query row: exactly its part of the second
// product's B operand (32 tokens x 16 rows), whose A operand is V transposed, put
// together in registers by byte permutes. No score, weight or V passes through
// LDS. Codes enter as fp16 subnormals (u 2^-24: the code in the low byte of a
// 16-bit lane; int4 16 u 2^-24), which the MFMA multiplies exactly.
//
// Numbers. Weights are scaled by 2^6 and the maximum is moved only when a score
// passes it by 2^8, so they stay below 2^14 and are normal fp16 numbers down to
// 2^-20 of the maximum; their 11 bits are the one rounding between the products,
// independent from token to token. For quantised values weight times step is
// what enters, and its maximum over the tokens a row sees is the running one (a
// maximum of the scores, with one scale for the steps beside it, lets a single
// large step, of a negligible weight or not seen at all, push the others' weights
// below the normal numbers: 500 int8 tokens of size 1e-3 beside one unseen row of
// 3e4 came out 2.8e-3 off in norm, against 3.3e-4). The sum of the rounded weights
// times the middle code is taken off again: what is rounded counts from the middle
// of the codes, not from their end. Sums, maxima and normalisations are fp32.
//
// What bounds it. With few query rows, the cache's bytes: 131072 tokens x 8 kv
// heads, one token, on caches not used before, fp16 105 us (5.1 TB/s; a copy
// reaches 5.3 counting both ways), int8 63 (4.4 TB/s), int4 40 (3.5 TB/s). Past 32
// query rows per kv head instructions and their latency, at two wavefronts per
// SIMD: per 32 tokens and 32 rows 321 VALU instructions (half of them the decoding
// of codes, masks and addresses, done by each wavefront of the rows) beside 32
// MFMAs; 65536 int8 tokens, 128 rows, 83 us (414 TFLOP/s; counters: vector unit
// about half of the time busy, matrix cores 18 %, so a good part of it neither;
// partial sums, their joining and the start take about 15 us). Short calls are bound by
// latency: launch, lengths, block table, first tile, join, about 6 us for 16 tokens.
//
// Taken and dropped, measured at the same sizes: 4 row tiles per wavefront (one
// wavefront per SIMD: trees of 16 at 8192 tokens 169 us against 112), the last
// workgroup of a sequence joining all parts of 64 rows (218 us against 128 with a
// kernel of its own), masks as comparisons (16 pairs of scalar registers in
// flight, spilled), rows written from registers without LDS (16-byte pieces at
// 512-byte strides: trees 87 us against 63), tiles of codes moved to LDS by DMA and
// read there by the wavefronts side by side, each of which still decodes them (trees 61.5 us against 62.7, but a batch of
// 32 31.5 against 30.0 and trees of 61 42.8 against 40.0; the same with one tile's
// output beside the next one's scores 61.9, 35.5 and 44.3; decoding a tile once for
// all of them has not been built), workgroups of 8 wavefronts for 32 rows each (half the partial sums: 131072 fp16 tokens 119 us
// against 124, but 4 x 2000 30 against 25).
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
    int unit_rows;                 // query rows a wavefront takes
    int row_blocks, slot_rows;     // blocks of query rows; rows of one in the partial sums
    int chunks, min_per, max_chunks;   // chunks (0: one per sequence), least work of one, chunks launched
    float scale, inv_group;        // inv_group: 1 / (query heads per kv head)
    int join;                      // partial sums are joined by k_at_join, not by the last chunk
    float *part;                   // partial sums, two places per chunk, kv head and row block
    uint32_t *counters;            // arrivals per (sequence, kv head, row block), zero between calls
};

typedef float at_f4 __attribute__((ext_vector_type(4)));
typedef uint32_t at_u4 __attribute__((ext_vector_type(4)));

// The kernel's arguments, read again where they are needed: what only the ends
// of a sequence's part use must not hold scalar registers through its tiles.
typedef const __attribute__((address_space(4))) AtArgs *AtLate;
__device__ __forceinline__ AtLate at_late() {
    AtLate p = (AtLate)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

// The quotient of a query row by the group size, by the host's reciprocal:
// exact below 2^21 rows.
__device__ __forceinline__ int at_div(int row, float inv) { return (int)(((float)row + 0.5f) * inv); }

// 8 channels of a finished row: sums times inv, rounded to fp16.
__device__ __forceinline__ void at_write(AtLate ap, int q0, int kvh, int G, int row, int d, int D, at_f4 y0,
                                         at_f4 y1, float inv) {
    const int t = at_div(row, ap->inv_group), g = row - t * G;
    uint16_t *o = ap->O + (int64_t)(q0 + t) * ap->o_stride + (int64_t)(kvh * G + g) * D + d;
    uint16_t h[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = bsp_f2h(y0[e] * inv), h[4 + e] = bsp_f2h(y1[e] * inv);
    if (ap->o_vec) {
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
#define AT_CUS 256
#define AT_TILE 32                 // cached tokens per wavefront and step
#define AT_AHEAD (32 * AT_WAVES * AT_TILE)   // tokens past the end that indexes may reach
#define AT_BOOST 6.0f              // log2: the weights' scale, 2^6 at the running maximum
#define AT_SLACK 8.0f              // log2: how far a score may pass the running maximum before it is moved
// Query rows of a row block: 16 where a call has no more, else four wavefronts of 16 RT.
#define AT_ROWS(RT) ((RT) == 1 ? (D == 256 ? 64 : 16) : 64 * (RT))
#define AT_LOW -1e30f              // stands for the maximum of no scores when sums are joined
#define AT_NONE -3e38f             // `limit` of a row without a score yet
// Bits of the least value step the maximum counts, 2^-40 (a row of equal
// values has step 0; the least other step is 2^-24 / 255): weights relative to
// a maximum with steps this small stay in range.
#define AT_STEP_LOW 0x2B800000u

// Workgroups per CU that the kernels are compiled for and the work is cut to
// (their registers; a wavefront each per SIMD): one round, no workgroup waits
// for another. D = 128: aiming at 448 workgroups, trees 65.8 us against 63.4
// and long fp16 135 against 124; at 768, 75 and 132; int4 with few rows fits
// three, and 768 then took 28.0 against 30.2 for the batch of uneven lengths but
// 39.8 against 34.8 for 32 sequences of 4096. D = 256, 512 against 256: int8
// 30,000 tokens x 2 44.3 us against 38.3.
constexpr int at_per_cu(int dim) { return dim == 256 ? 1 : 2; }

// What a lane reads of a K row and of a V row. A K row goes to the four lanes
// of its A row in pieces of PIECE bytes in turn, so that one load instruction
// takes whole 64-byte stretches of 16 rows (with a contiguous quarter of the
// row per lane each of its loads touches every line of the rows: 131072 fp16
// tokens 224 us against 218). A V row goes to 16 lanes, a sixteenth each.
template <int KIND, int D>
struct AtShape {
    static constexpr int ROW = KIND == BSP_FP16 ? 2 * D : KIND == BSP_INT8 ? D : D / 2;
    static constexpr int KW = ROW / 16;                      // dwords per K row and lane
    static constexpr int PIECE = ROW < 64 ? ROW / 4 : 16;
    static constexpr int PIECES = ROW / (4 * PIECE);
    static constexpr int PCH = PIECE * D / ROW;              // channels of a piece
    static constexpr int VB = ROW / 16;                      // bytes per V row and lane
    static constexpr int VW = VB < 4 ? 1 : VB / 4;
    static constexpr int NT = D / 16;                        // 16-channel blocks of the output
    static constexpr int STEPS = D / 32;                     // MFMAs along the channels
    static constexpr float UNIT = KIND == BSP_INT8 ? 0x1p24f : 0x1p20f;      // a code over what stands for it
};

// Agent-scope 16-byte stores and loads of the partial sums: they go to the
// coherence point all XCDs share, so partials are visible to the workgroup
// that joins them once the stores have completed (aux 16: sc1).
__device__ __forceinline__ void at_ws_store(__amdgpu_buffer_rsrc_t rs, uint32_t off, at_f4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(at_u4, v), rs, off, 0, 16);
}
__device__ __forceinline__ at_f4 at_ws_load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    return __builtin_bit_cast(at_f4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 16));
}

// Eight channels of a row summed over chunks: sums and normalisation relative
// to the largest of the chunks' maxima so far.
struct AtSum {
    at_f4 y0 = {0.f, 0.f, 0.f, 0.f}, y1 = {0.f, 0.f, 0.f, 0.f};
    float m = AT_LOW, l = 0.f;
    __device__ __forceinline__ void add(at_f4 z0, at_f4 z1, float zm, float zl) {
        const float mn = fmaxf(m, zm);
        const float f = __builtin_amdgcn_exp2f(m - mn), g = __builtin_amdgcn_exp2f(zm - mn);
        m = mn;
        l = l * f + zl * g;
#pragma unroll
        for (int e = 0; e < 4; ++e) y0[e] = y0[e] * f + z0[e] * g, y1[e] = y1[e] * f + z1[e] * g;
    }
    // a posted part: the place's first float, its bytes, where the channels and (m, l) lie
    __device__ __forceinline__ void add(const float *place, uint32_t bytes, uint32_t at, uint32_t at_ml) {
        const __amdgpu_buffer_rsrc_t rs = bsp_rsrc(place, bytes);
        const at_f4 ml = at_ws_load(rs, at_ml), z0 = at_ws_load(rs, at), z1 = at_ws_load(rs, at + 16);
        add(z0, z1, ml.x, ml.y);
    }
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

// Bytes 2k, 2k + 1 of a dword, or byte k of two dwords, as the low bytes of
// two 16-bit lanes: fp16 subnormals u * 2^-24. The MFMA multiplies them exactly,
// and lines products up by the exponents of their factors, so a subnormal's
// leading zeros are bits its sums lose: int4 codes sit in bits 4 .. 7 for that
// (as 16 u; in bits 0 .. 3, 606409 int4 tokens came out 7.8e-4 off in norm, half
// of it a bias, against 2.6e-4).
__device__ __forceinline__ uint32_t at_bytes(uint32_t hi, uint32_t lo, uint32_t sel) {
    return __builtin_amdgcn_perm(hi, lo, sel);
}

// The A operand of step `s` of the scores: 8 channels of this lane's K row.
// int4: even steps hold the even channels of 16, odd steps the odd ones, all
// times 16.
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
        constexpr uint32_t m = 0x00F000F0u;
        f = (s & 1) ? at_u4{a & m, (a >> 8) & m, b & m, (b >> 8) & m}
                    : at_u4{(a << 4) & m, (a >> 4) & m, (b << 4) & m, (b >> 4) & m};
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
            f[p] = ((t & 1) ? b : b << 4) & 0x00F000F0u;
        }
    }
    return __builtin_bit_cast(at_h8, f);
}

// Over the four lanes of a query row (16 apart): swaps of halves and of
// 16-lane rows leave a lane's value and its partner's in the two results.
template <class F>
__device__ __forceinline__ float at_group(float v, F f) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t h0 = h[0], h1 = h[1];
    const uint32_t w = __builtin_bit_cast(uint32_t, f(__builtin_bit_cast(float, h0), __builtin_bit_cast(float, h1)));
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    const uint32_t q0 = q[0], q1 = q[1];
    return f(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
}
__device__ __forceinline__ float at_group_sum(float v) {
    return at_group(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float at_group_max(float v) {
    return at_group(v, [](float a, float b) { return fmaxf(a, b); });
}

__device__ __forceinline__ int at_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// All ones where bit e of m is set, else zero.
__device__ __forceinline__ uint32_t at_spread(uint32_t m, int e) { return (uint32_t)((int32_t)(m << (31 - e)) >> 31); }

// 1 in each half of a dword of two fp16 numbers that is an infinity or a NaN:
// an exponent of all ones carries into the bit above it.
__device__ __forceinline__ uint32_t at_odd(uint32_t h) { return (((h & 0x7C007C00u) + 0x04000400u) >> 15) & 0x00010001u; }

// One wavefront's share: 16 RT query rows, every wt_n-th tile.
template <int KIND, int D, int RT>
struct AtWave {
    using Sh = AtShape<KIND, D>;
    static constexpr bool QUANT = KIND != BSP_FP16;
    const AtArgs &a;
    int lane, col, grp;
    int kvh, len, past;
    int wt_n;                      // wavefronts that take the tiles in turn
    const int32_t *table;
    // per query row (the lane's column); q in registers, or in LDS where those
    // are short: [RT][STEPS][64 lanes], the workgroup's wavefronts share the rows
    static constexpr bool Q_LDS = RT > 1 || D == 256;
    at_h8 q[Q_LDS ? 1 : RT][Q_LDS ? 1 : Sh::STEPS];
    const at_h8 *q_lds;
    float qc[RT];                  // sum of the row's q, times the score factor
    uint64_t seen[RT];
    // the running maximum less AT_BOOST (of scores, or of scores + log2(value
    // step)), and the sums of the weights 2^(x - mb)
    float mb[RT], l[RT], osum[RT], psum[RT];
    float limit[RT];               // a score past it moves the maximum (AT_NONE: the row has none yet)
    at_f4 acc[RT][Sh::NT];
    float c;                       // score factor: scale * log2(e)
    // the tile in flight
    uint32_t k[2][Sh::KW], v[8][Sh::VW], kw[8], vw[8];
    // Cache pages of the wavefront's next 32 tiles, looked up at once: lane
    // 2 i + h has the page of the i-th tile's 16 tokens h (a page holds whole
    // groups of 16).
    int pages;
    int64_t base0, base1;          // rows of the next tile's two groups (uniform)

    __device__ AtWave(const AtArgs &args) : a(args) {}

    __device__ __forceinline__ at_h8 q_frag(int rt, int s) const {
        if constexpr (Q_LDS)
            return q_lds[(rt * Sh::STEPS + s) * 64 + lane];
        else
            return q[rt][s];
    }

    __device__ __forceinline__ void load_pages(int tile) {
        const int j = min((tile + wt_n * (lane >> 1)) * AT_TILE + 16 * (lane & 1), len - 1);
        const int p = table[j >> a.page_shift];
        pages = (unsigned)p < (unsigned)a.num_pages ? p : 0;
    }
    // The row of the wavefront's tile i (mod 32), at token j0 of the sequence.
    __device__ __forceinline__ void set_tile(int i, int j0) {
        const int in = (1 << a.page_shift) - 1;
        const int p0 = __builtin_amdgcn_readlane(pages, 2 * (i & 31)), p1 = __builtin_amdgcn_readlane(pages, 2 * (i & 31) + 1);
        base0 = (((int64_t)p0 * a.hkv + kvh) << a.page_shift) + (j0 & in);
        base1 = (((int64_t)p1 * a.hkv + kvh) << a.page_shift) + ((j0 + 16) & in);
    }
    // S tile u, A row i: token 8 (i / 4) + 4 u + i % 4, so that the scores of a
    // lane (C rows 4 g .. 4 g + 3 of both tiles) are those of 8 neighbouring
    // tokens, 8 g .. 8 g + 7: its part of the second product's B operand.
    __device__ __forceinline__ void load_k() {
        const uint8_t *p = a.k + ((col >> 3) ? base1 : base0) * Sh::ROW + (8 * ((col >> 2) & 1) + (col & 3)) * Sh::ROW +
                           grp * Sh::PIECE;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < Sh::PIECES; ++j) {
                uint32_t r[Sh::PIECE / 4];
                at_load(p + 4 * u * Sh::ROW + 64 * j, r);
#pragma unroll
                for (int i = 0; i < Sh::PIECE / 4; ++i) k[u][j * (Sh::PIECE / 4) + i] = r[i];
            }
        if constexpr (QUANT)
            at_load(reinterpret_cast<const uint8_t *>(a.kw + ((grp >> 1) ? base1 : base0) + 8 * (grp & 1)), kw);
    }
    __device__ __forceinline__ void load_v() {
        const int64_t r = ((grp >> 1) ? base1 : base0) + 8 * (grp & 1);
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

    // Bits 0 .. 7: whether a row that sees drafted tokens `bits` sees the 8
    // tokens from the drafted one d on (negative: before them) on.
    __device__ __forceinline__ uint32_t visible(int d, uint64_t bits) const {
        const int b = min(max(-d, 0), 8);          // tokens before the drafted ones
        const uint32_t m = d < 64 ? (uint32_t)(bits >> max(d, 0)) : 0u;
        return (m << b) | ((1u << b) - 1u);
    }

    // Values that are not finite: how many infinities (a NaN is one of each
    // sign) a row sees per channel is a product of ones; they are added to the
    // sums, and taken out of v.
    __device__ __forceinline__ void add_odd(const uint32_t (&ok)[RT]) {
#pragma unroll
        for (int t = 0; t < Sh::NT; ++t) {
            const at_u4 f = __builtin_bit_cast(at_u4, at_v_frag<KIND>(v, t));
            at_u4 pos, neg;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t nf = at_odd(f[p]), sign = f[p] >> 15;
                const uint32_t nan = ((f[p] & 0x03FF03FFu) + 0x03FF03FFu) >> 10;
                pos[p] = (nf & (~sign | nan)) * 0x3C00u, neg[p] = (nf & (sign | nan)) * 0x3C00u;
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                at_u4 see;
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    see[p] = ((at_spread(ok[rt], 2 * p) & 0xFFFFu) | (at_spread(ok[rt], 2 * p + 1) << 16)) & 0x3C003C00u;
                const at_f4 none = {0.f, 0.f, 0.f, 0.f};
                const at_h8 b = __builtin_bit_cast(at_h8, see);
                const at_f4 up = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(at_h8, pos), b, none, 0, 0, 0);
                const at_f4 dn = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(at_h8, neg), b, none, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[rt][t][i] += up[i] > 0.f ? INFINITY : 0.f;
                    acc[rt][t][i] -= dn[i] > 0.f ? INFINITY : 0.f;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int i = 0; i < Sh::VW; ++i) v[e][i] &= ~(at_odd(v[e][i]) * 0xFFFFu);
    }

    // One tile: scores, running maximum, weights, output. The next tile's loads
    // (base0, base1: set_tile) are issued as the registers they fill fall free.
    __device__ __forceinline__ void tile(int j0) {
        at_f4 x[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) x[rt][0] = x[rt][1] = at_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < Sh::STEPS; ++s) {
            const at_h8 f = at_k_frag<KIND>(k[0], s), g = at_k_frag<KIND>(k[1], s);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const at_h8 qs = q_frag(rt, s);
                x[rt][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, qs, x[rt][0], 0, 0, 0);
                x[rt][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(g, qs, x[rt][1], 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // scores in log2 units, less the running maximum (mb):
        // scale * log2(e) * (s u.q + o sum(q)) - mb
        float top[RT];
        const float cc = c * Sh::UNIT;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) top[rt] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float ks, ko;
            if constexpr (QUANT) ks = kv_word_step(kw[e]) * cc, ko = kv_word_offset(kw[e]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float y = x[rt][e >> 2][e & 3];
                if constexpr (QUANT)
                    y = fmaf(y, ks, fmaf(ko, qc[rt], -mb[rt]));
                else
                    y = fmaf(y, c, -mb[rt]);
                x[rt][e >> 2][e & 3] = y;
                top[rt] = fmaxf(top[rt], y);
            }
        }
        load_k();
        if (j0 + AT_TILE > past) {
            // Drafted tokens or the end of the sequence: what a row does not
            // see scores -inf; rows past the end hold anything, NaN too, and
            // count as zeros. A value that is not finite counts as zero in the
            // product, where a weight of zero would not keep it out, and is
            // added for the query rows that see it; a quantised row whose word
            // is not finite makes them NaN. (Masks are spread over registers:
            // comparisons would hold 16 pairs of scalar registers at a time.)
            const int n = min(max(len - (j0 + 8 * grp), 0), 8);     // tokens there are
            const uint32_t in = (1u << n) - 1u;
            uint32_t ok[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                ok[rt] = visible(j0 + 8 * grp - past, seen[rt]) & in;
                top[rt] = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x0 = x[rt][e >> 2][e & 3];
                    const uint32_t m = at_spread(ok[rt], e), y = __builtin_bit_cast(uint32_t, x0);
                    const float z = __builtin_bit_cast(float, (m & y) | (~m & 0xFF800000u));
                    x[rt][e >> 2][e & 3] = z;
                    top[rt] = fmaxf(top[rt], z);
                }
            }
            uint32_t odd = 0;              // quantised: bit e: token e's word is not finite; else any value of the lane's
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = at_spread(in, e);
                if constexpr (QUANT) {
                    // an exponent of all ones carries into the bit above it
                    const uint32_t w = vw[e] & m;
                    const uint32_t nf = ((((w & 0x7F800000u) + 0x00800000u) >> 31) | (((w & 0x7C00u) + 0x0400u) >> 15)) & 1u;
                    vw[e] = w & (nf - 1u);
                    odd |= nf << e;
                } else {
                    uint32_t any = 0;
#pragma unroll
                    for (int i = 0; i < Sh::VW; ++i) {
                        v[e][i] &= m;
                        any |= at_odd(v[e][i]);
                    }
                    odd |= any;
                }
            }
            if (__ballot(odd != 0) != 0) {
                if constexpr (QUANT) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) l[rt] = (ok[rt] & odd) != 0u ? __builtin_nanf("") : l[rt];
                } else {
                    add_odd(ok);
                }
            }
        }
        // Move the running maximum only when a score passes it by more than
        // the slack (the weights stay fp16: 2^(6 + 8) at most). What enters the
        // second product of a quantised cache is weight times step, so there
        // the maximum is that of score + log2(step), over the tokens the row
        // sees: a large step counts with its weight alone. The largest step of
        // the lane's tokens and the largest score bound it from above.
        float lg = 0.f;
        if constexpr (QUANT) {
            uint32_t smax = AT_STEP_LOW;                   // (positive floats order as integers)
#pragma unroll
            for (int e = 0; e < 8; ++e) smax = max(smax, vw[e]);
            lg = __builtin_amdgcn_logf(__builtin_bit_cast(float, smax));
        }
        bool move = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) move |= (QUANT ? top[rt] + lg : top[rt]) > limit[rt];
        float f[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) f[rt] = 1.f;
        const bool moved = __ballot(move) != 0;
        if (moved) {
            if constexpr (QUANT) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) top[rt] = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float le = __builtin_amdgcn_logf(kv_word_step(max(vw[e], AT_STEP_LOW)));
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) top[rt] = fmaxf(top[rt], x[rt][e >> 2][e & 3] + le);
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                // how far it moves: up only, but for the row's first scores, and
                // by what the row itself sees
                const float most = at_group_max(top[rt]);
                const bool over = most > limit[rt], first = limit[rt] == AT_NONE;
                const float up = over ? most - AT_BOOST : 0.f;
                const float g = over && !first ? __builtin_amdgcn_exp2f(-up) : 1.f;
                limit[rt] = over ? AT_BOOST + AT_SLACK : limit[rt];
                mb[rt] += up;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[rt][e >> 2][e & 3] -= up;
                l[rt] *= g, osum[rt] *= g, psum[rt] *= g;
                f[rt] = g;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (moved) {       // (apart from the block above: the accumulators stay in place)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int t = 0; t < Sh::NT; ++t) acc[rt][t] *= f[rt];
        }
        at_h8 p[RT];
        const at_h2 one = {(_Float16)1.f, (_Float16)1.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float st, vo;
            if constexpr (QUANT) {
                st = kv_word_step(vw[e]);
                vo = fmaf(KIND == BSP_INT8 ? 128.0f : 8.0f, st, kv_word_offset(vw[e]));
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float w = __builtin_amdgcn_exp2f(x[rt][e >> 2][e & 3]);
                if constexpr (QUANT) {
                    l[rt] += w;
                    osum[rt] = fmaf(w, vo, osum[rt]);
                    w *= st;
                }
                p[rt][e] = (_Float16)w;          // nearest even: errors of 11 bits that average out over the tokens
            }
        }
        // the sum of the rounded weights: what the codes' middle is taken off
        // with, and (fp16 cache) the row's normalisation
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const at_h2 pair = {p[rt][e], p[rt][e + 1]};
                if constexpr (QUANT)
                    psum[rt] = __builtin_amdgcn_fdot2(pair, one, psum[rt], false);
                else
                    l[rt] = __builtin_amdgcn_fdot2(pair, one, l[rt], false);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < Sh::NT; ++t) {
            const at_h8 f = at_v_frag<KIND>(v, t);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                acc[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, p[rt], acc[rt][t], 0, 0, 0);
            if (t & 1) __builtin_amdgcn_sched_barrier(0);
        }
        load_v();
    }
};

// Wavefronts side by side that `rows` query rows of a row block take, at `unit`
// (16 RT) rows each.
__device__ __forceinline__ int at_side(int rows, int unit) { return rows <= unit ? 1 : rows <= 2 * unit ? 2 : 4; }

// The sequences, 64 at a time, one a lane: cached tokens, first and last query
// row, and work: tiles (at least one where there are query rows) times the
// wavefronts side by side that take each.
struct AtSeqs {
    int block = -1, len = 0, q0 = 0, q1 = 0, work = 0;

    __device__ __forceinline__ void load(int blk) {
        if (blk == block) return;
        block = blk;
        const AtLate a = at_late();
        const int b = blk * 64 + (threadIdx.x & 63);
        len = q0 = q1 = work = 0;
        if (b < a->B) {
            len = (int)min((int64_t)max(a->kv_lens[b], 0), a->table_width << a->page_shift);
            q0 = min(max(a->q_start[b], 0), a->total_q);
            q1 = min(max(a->q_start[b + 1], q0), a->total_q);
            const int side = at_side(min(q1 - q0, a->max_q) * (a->hq / a->hkv), a->unit_rows);
            work = q1 > q0 ? max(1, (len + AT_TILE - 1) / AT_TILE) * side : 0;
        }
    }
    __device__ __forceinline__ int of(int v, int b) const { return __builtin_amdgcn_readlane(v, b & 63); }
};

// One workgroup: a kv head, a block of query rows, and an equal share of the
// work of all sequences laid end to end (its chunk), which may hold the end of
// one sequence, whole ones, and the start of another. As many wavefronts side
// by side (1, 2 or 4) as the sequence's rows need take 16 RT rows each of the
// same tiles (their reads of the cache meet in the CU's L1); the sets so
// formed take the tiles in turn. RT 1 is for calls of at most 16 rows.
template <int KIND, int D, int RT>
__global__ __launch_bounds__(64 * AT_WAVES, at_per_cu(D)) void k_at(const AtArgs a) {
    using Sh = AtShape<KIND, D>;
    using Wave = AtWave<KIND, D, RT>;
    extern __shared__ __attribute__((aligned(16))) float at_smem[];
    constexpr int LD = D + 4;                      // floats per row of a wavefront's output in LDS
    constexpr int ROWS = AT_ROWS(RT);              // query rows of a row block
    float *s_acc = at_smem;                        // [AT_WAVES][16][LD]
    float *s_m = s_acc + AT_WAVES * 16 * LD;       // [AT_WAVES][16]
    float *s_l = s_m + AT_WAVES * 16;
    int *s_flag = reinterpret_cast<int *>(s_l + AT_WAVES * 16);
    const int wave = at_uniform(threadIdx.x >> 6);
    // workgroups 8 apart share an XCD and its L2: the row blocks of one piece
    // of the cache are 8 apart
    const int group = blockIdx.x / (8 * a.row_blocks), in = blockIdx.x % (8 * a.row_blocks);
    const int rb = in >> 3, piece = group * 8 + (in & 7);
    const int ch = piece / a.hkv;
    if (ch >= a.max_chunks) return;
    Wave w(a);
    w.kvh = piece - ch * a.hkv;
    w.lane = threadIdx.x & 63, w.col = w.lane & 15, w.grp = w.lane >> 4;
    w.c = a.scale * 1.44269504088896341f;
    const int G = a.hq / a.hkv;

    // the chunk's first sequence, and where that one's tiles begin
    AtSeqs seqs;
    int b = ch, begin = 0, per = 0, pos = 0, end = 0;
    if (a.chunks == 0) {                           // no split: a workgroup per sequence
        seqs.load(b >> 6);
        end = seqs.of(seqs.work, b);
        per = max(end, 1);
    } else {
        int total = 0;
        for (int k = (a.B - 1) >> 6; k >= 0; --k) {
            seqs.load(k);
            total += bsp_wave_sum(seqs.work);
        }
        total = at_uniform(total);
        per = max(a.min_per, (total + a.chunks - 1) / a.chunks);
        pos = ch * per, end = min(total, pos + per);
        if (pos >= end) return;
        int before = 0;
        for (int k = 0;; ++k) {
            seqs.load(k);
            int s = seqs.work;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(s, d, 64);
                if (w.lane >= d) s += o;
            }
            const uint64_t hit = __ballot(pos < before + s);
            if (hit != 0) {
                b = __builtin_ctzll(hit);
                begin = before + seqs.of(s, b) - seqs.of(seqs.work, b);
                b += 64 * k;
                break;
            }
            before += seqs.of(s, 63);
        }
    }

    for (; pos < end; ++b) {
        const AtLate as = at_late();
        seqs.load(b >> 6);
        const int work = seqs.of(seqs.work, b);
        if (work == 0) continue;
        const int q0 = seqs.of(seqs.q0, b), T = seqs.of(seqs.q1, b) - q0;
        const int rows = min(T, as->max_q) * G;      // query rows of this kv head
        w.len = seqs.of(seqs.len, b);
        w.past = w.len - T;
        w.table = as->table + (int64_t)b * as->table_width;
        const int nt = (w.len + AT_TILE - 1) / AT_TILE, side = at_side(rows, 16 * RT);
        const int t0 = min(nt, (pos - begin) / side), t1 = min(nt, (end - begin) / side);
        // chunks that hold work of the sequence, and this one's place for its part
        const int c0 = begin / per, count = as->chunks == 0 ? 1 : (begin + work - 1) / per - c0 + 1;
        begin += work;
        pos = begin;
        const int rows_here = min(rows - rb * ROWS, ROWS);
        if (rows_here <= 0) continue;
        // wavefronts side by side, the wavefront's place among them, its first row
        const int wr_n = at_side(rows_here, 16 * RT);
        const int wr = wave & (wr_n - 1), wt = wave / wr_n, r0 = rb * ROWS + wr * 16 * RT;
        w.wt_n = AT_WAVES / wr_n;
        w.q_lds = reinterpret_cast<at_h8 *>(at_smem) + wr * (RT * Sh::STEPS * 64);
        const int tile0 = t0 + wt;
        if (tile0 < t1) {
            w.load_pages(tile0);
            w.set_tile(0, tile0 * AT_TILE);
            w.load_k();
            w.load_v();
        }
        if constexpr (Wave::Q_LDS) __syncthreads();      // the LDS area's last readers
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int row = r0 + 16 * rt + w.col;
            const bool in_rows = row < rows;
            const int t = in_rows ? at_div(row, as->inv_group) : 0, g = in_rows ? row - t * G : 0;
            const uint16_t *src = as->Q + (int64_t)(q0 + t) * as->q_stride + (int64_t)(w.kvh * G + g) * D;
            uint32_t qr[D / 8];                    // the channels of the lane's K pieces
#pragma unroll
            for (int j = 0; j < Sh::PIECES; ++j) {
                const uint16_t *sp = src + (4 * j + w.grp) * Sh::PCH;
                uint32_t piece[Sh::PCH / 2];
                if (as->q_vec) {
                    at_load(reinterpret_cast<const uint8_t *>(sp), piece);
                } else {
#pragma unroll
                    for (int i = 0; i < Sh::PCH / 2; ++i) piece[i] = (uint32_t)sp[2 * i] | ((uint32_t)sp[2 * i + 1] << 16);
                }
#pragma unroll
                for (int i = 0; i < Sh::PCH / 2; ++i) qr[j * (Sh::PCH / 2) + i] = piece[i];
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
            for (int s = 0; s < Sh::STEPS; ++s) {
                if constexpr (Wave::Q_LDS) {
                    if (rt % w.wt_n == wt)               // shared by the wavefronts of these rows
                        const_cast<at_h8 *>(w.q_lds)[(rt * Sh::STEPS + s) * 64 + w.lane] = at_q_frag<KIND>(qr, s);
                } else {
                    w.q[rt][s] = at_q_frag<KIND>(qr, s);
                }
            }
            w.seen[rt] = as->mask != nullptr ? as->mask[q0 + t] : (uint64_t)-1 >> (63 - min(t, 63));
            w.mb[rt] = 0.f, w.limit[rt] = AT_NONE, w.l[rt] = 0.f, w.osum[rt] = 0.f, w.psum[rt] = 0.f;
#pragma unroll
            for (int i = 0; i < Sh::NT; ++i) w.acc[rt][i] = at_f4{0.f, 0.f, 0.f, 0.f};
        }
        if constexpr (Wave::Q_LDS) __syncthreads();
        const int te = r0 < rows ? t1 : tile0;           // (no rows: no tiles)
        for (int t = tile0, i = 1; t < te; t += w.wt_n, ++i) {
            if (t + w.wt_n < t1) {     // (past the last tile its own rows are loaded again, unused)
                if ((i & 31) == 0) w.load_pages(t + w.wt_n);
                w.set_tile(i, (t + w.wt_n) * AT_TILE);
            }
            w.tile(t * AT_TILE);
        }

        const AtLate ap = at_late();
        // Join the wavefronts of each row tile, one row tile of each at a time;
        // then write the rows, or post them for the sequence's last chunk to join.
        const bool split = count > 1;
        const uint32_t slot_floats = ap->slot_rows * (D + 4);     // [row][D] sums, then [row] (m, l, 0, 0)
        const int64_t head = (int64_t)w.kvh * ap->row_blocks + rb, heads = (int64_t)ap->hkv * ap->row_blocks;
        const auto put = [&](int rl, int d, at_f4 y0, at_f4 y1, float mx, float lt) {
            if (split) {
                float *place = ap->part + ((2 * (int64_t)ch + (ch == c0)) * heads + head) * slot_floats;
                if (ap->join) {                          // for another kernel: plain stores
                    at_f4 *y = reinterpret_cast<at_f4 *>(place + rl * D + d);
                    y[0] = y0, y[1] = y1;
                    if (d == 0) *reinterpret_cast<float2 *>(place + ap->slot_rows * D + 4 * rl) = float2{mx, lt};
                    return;
                }
                const __amdgpu_buffer_rsrc_t rs = bsp_rsrc(place, slot_floats * 4);
                const uint32_t at = ((uint32_t)rl * D + d) * 4u;
                at_ws_store(rs, at, y0), at_ws_store(rs, at + 16, y1);
                if (d == 0) at_ws_store(rs, (uint32_t)(ap->slot_rows * D + 4 * rl) * 4u, at_f4{mx, lt, 0.f, 0.f});
            } else {
                at_write(ap, q0, w.kvh, G, rb * ROWS + rl, d, D, y0, y1, lt == 0.f ? 0.f : 1.0f / lt);
            }
        };
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float l = at_group_sum(w.l[rt]), m = w.limit[rt] == AT_NONE ? AT_LOW : w.mb[rt];
            float os = 0.f, ps = 0.f;
            if constexpr (Wave::QUANT) {
                os = at_group_sum(w.osum[rt]);
                ps = at_group_sum(w.psum[rt]) * (KIND == BSP_INT8 ? 128.0f : 8.0f);
            }
            // the lane's channels: NT from (4 grp + r) NT on, for r = 0 .. 3
            const auto y_of = [&](int r, int t) {
                at_f4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float z = w.acc[rt][t + i][r];
                    if constexpr (Wave::QUANT) z = fmaf(z, Sh::UNIT, -ps) + os;
                    y[i] = z;
                }
                return y;
            };
            __syncthreads();                             // the LDS area's last readers
            if (w.grp == 0) s_m[wave * 16 + w.col] = m, s_l[wave * 16 + w.col] = l;
            float *o = s_acc + (wave * 16 + w.col) * LD;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int t = 0; t < Sh::NT; t += 4) *reinterpret_cast<at_f4 *>(o + (4 * w.grp + r) * Sh::NT + t) = y_of(r, t);
            __syncthreads();
            for (int i = threadIdx.x; i < wr_n * 16 * (D / 8); i += 64 * AT_WAVES) {
                const int d = (i % (D / 8)) * 8, row = i / (D / 8) % 16, g = i / (D / 8) / 16;   // g: the row group
                const int rl = g * 16 * RT + 16 * rt + row;
                if (rl >= rows_here) continue;
                AtSum sum;
                for (int k = 0; k < w.wt_n; ++k) {
                    const int at = (k * wr_n + g) * 16 + row;
                    const at_f4 *src = reinterpret_cast<const at_f4 *>(s_acc + at * LD + d);
                    sum.add(src[0], src[1], s_m[at], s_l[at]);
                }
                put(rl, d, sum.y0, sum.y1, sum.m, sum.l);
            }
        }
        if (!split || ap->join) continue;
        const int64_t unit = (int64_t)b * heads + head;
        __builtin_amdgcn_s_waitcnt(0);      // this thread's partial stores completed
        __syncthreads();
        if (threadIdx.x == 0)
            *s_flag = (int)__hip_atomic_fetch_add(&ap->counters[unit], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (*s_flag != count - 1) continue;
        for (int i = threadIdx.x; i < rows_here * (D / 8); i += 64 * AT_WAVES) {
            const int row = i / (D / 8), d = (i % (D / 8)) * 8;
            const uint32_t at = ((uint32_t)row * D + d) * 4u, at_ml = (uint32_t)(ap->slot_rows * D + 4 * row) * 4u;
            AtSum sum;
            for (int s = 0; s < count; ++s)        // in chunk order
                sum.add(ap->part + ((2 * (int64_t)(c0 + s) + (s == 0)) * heads + head) * slot_floats, slot_floats * 4, at, at_ml);
            at_write(ap, q0, w.kvh, G, rb * ROWS + row, d, D, sum.y0, sum.y1, sum.l == 0.f ? 0.f : 1.0f / sum.l);
        }
        if (threadIdx.x == 0) __hip_atomic_store(&ap->counters[unit], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// Joins the posted parts of split sequences: a workgroup takes 4 rows of a
// (sequence, kv head), its wavefronts every fourth chunk; their sums meet in
// LDS, in wavefront order.
template <int D>
__global__ __launch_bounds__(64 * AT_WAVES) void k_at_join(const AtArgs a, int block_rows) {
    constexpr int P = D / 8, RW = 64 / P;          // 8-channel pieces of a row; rows of a wavefront's 64 lanes
    __shared__ __attribute__((aligned(16))) float s_y[AT_WAVES][64][8];
    __shared__ float s_ml[AT_WAVES][64][2];
    const int lane = threadIdx.x & 63, wave = at_uniform(threadIdx.x >> 6);
    const int b = blockIdx.z, kvh = blockIdx.y, row = blockIdx.x * RW + lane / P, d = (lane % P) * 8;
    // the sequence's chunks, as the main kernel cuts them
    AtSeqs seqs;
    int total = 0, begin = 0;
    for (int k = (a.B - 1) >> 6; k >= 0; --k) {
        seqs.load(k);
        total += bsp_wave_sum(seqs.work);
        begin += bsp_wave_sum(k * 64 + lane < b ? seqs.work : 0);
    }
    seqs.load(b >> 6);
    const int work = seqs.of(seqs.work, b), q0 = seqs.of(seqs.q0, b), T = seqs.of(seqs.q1, b) - q0;
    const int G = a.hq / a.hkv, rows = min(T, a.max_q) * G;
    total = at_uniform(total), begin = at_uniform(begin);
    const int per = max(a.min_per, (total + a.chunks - 1) / a.chunks);
    const int c0 = begin / per, count = work == 0 ? 0 : (begin + work - 1) / per - c0 + 1;
    if (count <= 1 || (int)blockIdx.x * RW >= rows) return;
    const int64_t heads = (int64_t)a.hkv * a.row_blocks, head = (int64_t)kvh * a.row_blocks + row / block_rows;
    const uint32_t slot_floats = (uint32_t)a.slot_rows * (D + 4), rl = (uint32_t)(row % block_rows);
    AtSum sum;
    if (row < rows) {
        // (a kernel of its own: plain loads)
#pragma unroll 4
        for (int s = wave; s < count; s += AT_WAVES) {
            const float *place = a.part + ((2 * (int64_t)(c0 + s) + (s == 0)) * heads + head) * slot_floats;
            const float2 ml = *reinterpret_cast<const float2 *>(place + a.slot_rows * D + 4 * rl);
            const at_f4 *z = reinterpret_cast<const at_f4 *>(place + rl * D + d);
            sum.add(z[0], z[1], ml.x, ml.y);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s_y[wave][lane][e] = sum.y0[e], s_y[wave][lane][4 + e] = sum.y1[e];
    s_ml[wave][lane][0] = sum.m, s_ml[wave][lane][1] = sum.l;
    __syncthreads();
    if (wave != 0 || row >= rows) return;
#pragma unroll
    for (int k = 1; k < AT_WAVES; ++k) {
        at_f4 z0, z1;
#pragma unroll
        for (int e = 0; e < 4; ++e) z0[e] = s_y[k][lane][e], z1[e] = s_y[k][lane][4 + e];
        sum.add(z0, z1, s_ml[k][lane][0], s_ml[k][lane][1]);
    }
    at_write(at_late(), q0, kvh, G, row, d, D, sum.y0, sum.y1, sum.l == 0.f ? 0.f : 1.0f / sum.l);
}

// The plan of a call: row tiles per wavefront, rows of a row block and of its
// partial sums, row blocks, and how many chunks the work is cut into.
struct AtPlan {
    int rt, block_rows, slot_rows, row_blocks, chunks, min_per, max_chunks, join;
    int64_t ws_bytes;
};

#define AT_WS_COUNTERS 16384           // arrival counters at the start of a workspace

AtPlan at_plan(const bsp_kv_cache *c, int64_t table_width, int64_t B, int64_t max_q, int64_t hq, bool split) {
    AtPlan p{};
    const int64_t rows = max_q * (hq / c->kv_heads);
    const int64_t D = c->head_dim;
    p.rt = rows <= 16 || D == 256 ? 1 : 2;
    p.block_rows = (int)(p.rt == 1 ? AT_ROWS(1) : AT_ROWS(2));
    p.row_blocks = (int)((rows + p.block_rows - 1) / p.block_rows);
    p.slot_rows = (int)std::min<int64_t>(p.block_rows, rows);
    p.max_chunks = (int)B;
    // four tiles per wavefront at least (two: one token at 500 cached 9.8 us
    // against 9.3; longer calls alike)
    p.min_per = 4 * AT_WAVES;
    const int64_t heads = c->kv_heads * p.row_blocks;
    const int64_t tiles = (table_width * c->page_size + AT_TILE - 1) / AT_TILE;      // of the longest sequence
    // all work in 32 bits (sequences may share pages, so B * tiles is not bounded by
    // the cache): up to 4 wavefronts side by side per tile, or for a sequence of
    // none, and what rounding it up to whole chunks adds (at most 2 AT_CUS of them)
    const int64_t most_work = 4 * B * std::max<int64_t>(1, tiles);
    if (split && B * heads <= AT_WS_COUNTERS && most_work <= INT32_MAX - 2 * AT_CUS * p.min_per) {
        const int64_t want = std::max<int64_t>(1, (int64_t)AT_CUS * at_per_cu((int)D) / heads);
        const int64_t side = p.slot_rows <= 16 * p.rt ? 1 : p.slot_rows <= 32 * p.rt ? 2 : 4;
        const int64_t most = B * std::max<int64_t>(1, (tiles * side + p.min_per - 1) / p.min_per);
        p.chunks = p.max_chunks = (int)std::min(want, most);
        // Few parts of few rows are joined by the last of them to arrive, others
        // by a kernel of their own: joining is 3 loads a part and 8 channels, one
        // part after another, on one workgroup per row block.
        p.join = p.chunks > B && (rows > 16 || p.chunks > 8 * B);
        p.ws_bytes = AT_WS_COUNTERS * 4 + 2 * p.chunks * heads * p.slot_rows * (D + 4) * 4;
    }
    return p;
}

template <int KIND, int D, int RT>
void at_launch_t(const AtArgs &a, hipStream_t stream) {
    const size_t lds = (size_t)(AT_WAVES * 16 * (D + 4) + 2 * AT_WAVES * 16 + 4) * 4;
    const int64_t pieces = ((int64_t)a.max_chunks * a.hkv + 7) / 8 * 8;
    if (lds > 65536)
        (void)hipFuncSetAttribute((const void *)k_at<KIND, D, RT>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL((k_at<KIND, D, RT>), dim3((unsigned)(pieces * a.row_blocks)), dim3(64 * AT_WAVES), lds, stream, a);
    if (a.join) {
        const int rw = 64 / (D / 8), rows = a.max_q * (a.hq / a.hkv);
        hipLaunchKernelGGL((k_at_join<D>), dim3((rows + rw - 1) / rw, a.hkv, a.B), dim3(64 * AT_WAVES), 0, stream, a,
                           AT_ROWS(RT));
    }
}

template <int KIND, int D>
void at_launch_r(const AtArgs &a, const AtPlan &p, hipStream_t stream) {
    if (p.rt == 1)
        at_launch_t<KIND, D, 1>(a, stream);
    else if constexpr (D != 256)
        at_launch_t<KIND, D, 2>(a, stream);
}

template <int KIND>
void at_launch(const AtArgs &a, int64_t D, const AtPlan &p, hipStream_t stream) {
    if (D == 64)
        at_launch_r<KIND, 64>(a, p, stream);
    else if (D == 128)
        at_launch_r<KIND, 128>(a, p, stream);
    else
        at_launch_r<KIND, 256>(a, p, stream);
}

// Checks shared by the call and its workspace size.
int at_check(const bsp_kv_cache *c, int64_t table_width, int64_t B, int64_t max_q, int64_t hq) {
    const int rc = kv_check_cache(c);
    if (rc != BSP_OK) return rc;
    if (table_width < 0 || B < 0 || max_q < 0 || max_q > BSP_TREE_MAX || hq < 0) return BSP_E_ARG;
    if (hq > 0 && (c->kv_heads == 0 || hq % c->kv_heads != 0)) return BSP_E_ARG;
    if (B > 65535 || hq > 65535) return BSP_E_OVERFLOW;
    if (hq > 0 && hq / c->kv_heads > 16384) return BSP_E_UNSUPPORTED;
    // token indexes are 32 bits wide, and a wavefront looks pages up to 32 of its
    // tiles ahead: 4 x 31 tiles and one more past the last token
    if (table_width > (INT32_MAX - AT_AHEAD) / c->page_size) return BSP_E_OVERFLOW;
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
    // a launch holds fewer than 2^32 threads
    if (((int64_t)p.max_chunks * cache->kv_heads + 7) * p.row_blocks >= (int64_t)1 << 24) return BSP_E_OVERFLOW;
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
    a.inv_group = 1.0f / (float)(q_heads / cache->kv_heads);
    a.B = (int)B;
    a.q_vec = ((uintptr_t)Q & 15u) == 0 && (q_stride & 7) == 0;
    a.o_vec = ((uintptr_t)O & 15u) == 0 && (o_stride & 7) == 0;
    a.unit_rows = 16 * p.rt, a.row_blocks = p.row_blocks, a.slot_rows = p.slot_rows, a.chunks = p.chunks, a.min_per = p.min_per, a.max_chunks = p.max_chunks, a.join = p.join;
    a.counters = (uint32_t *)workspace;
    a.part = p.ws_bytes > 0 ? (float *)((uint8_t *)workspace + AT_WS_COUNTERS * 4) : nullptr;
    if (cache->dtype == BSP_FP16)
        at_launch<BSP_FP16>(a, cache->head_dim, p, stream);
    else if (cache->dtype == BSP_INT8)
        at_launch<BSP_INT8>(a, cache->head_dim, p, stream);
    else
        at_launch<BSP_INT4>(a, cache->head_dim, p, stream);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
