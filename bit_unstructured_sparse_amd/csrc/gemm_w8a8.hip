// gemm_w8a8.hip -- dense 8-bit product with scales per channel and token, for gfx950.
//
// v_mfma_i32_16x16x64_i8: a lane brings 16 bytes of one row of W (its tile in memory is
// in lane order) and 16 bytes of one token, and holds 4 neighbouring channels of
// one token of the result. Sums are int32 and exact, so the order in which parts of K
// meet changes nothing: K is split over wavefronts and workgroups wherever that is faster,
// and every plan gives the same bits.
//
// Three kernels. For at most 4 tokens and weights of 32 MB and more W streams past LDS into registers
// (k_w8_stream). Up to a few hundred tokens a tile is small and its wavefronts share K: each fills and reads a
// ring of its own in LDS by DMA, so that no barrier stands between memory and the matrix instructions
// (k_w8_ring). Past that a workgroup's wavefronts share the tile and a ring (k_w8_tiles).
//
// What bounds them. The time of all but the largest tiles is (bands + blocks) KB per 64 columns at about 57 KB/us a CU
// (N = 128, 4096 x 4096, 64 x 64 tiles: 8 KB a step, 0.14 us; deeper rings gain under 3 %). It is why tiles are
// chosen by their bytes, and why four bands and two blocks beat one and four. That rate is measured on the
// tiles, a mean over where their operands come from, and not what a CU can take: with each wavefront reading lines of its own and
// all 256 CUs at it, one takes in 98 to 134 KB/us from its L2, 20 to 28 from the last-level cache and 19 to 23 from memory,
// in pieces of 64 bytes, 128 or 1 KB (within a quarter of each other, neither form the fastest throughout). 32 tokens x
// 4096 x 11008: the 45 MB of W alone are 7 of the 10 us at the last-level cache's 6.5 TB/s.
//
// The 256 x 256 tiles: 8192 tokens x 12288 x 4096 in 328 to 349 us back to back, 369 in the middle of 50 traced launches
// (from machine to machine and with the power drawn; 2,230 to 2,510 TOP/s), 66 % of the cycles in matrix instructions, LDS
// reads and the DMA's writes taking as many cycles as those. Of that time the matrix instructions alone would take 256 us,
// with the reads from LDS 285, the loads and reads without them 235: it is their meeting. What brought them there from 600:
// operands read one step ahead into a second set of registers
// (with the scheduler told to spread the reads: left alone it sinks them behind all matrix instructions),
// a swizzle that leaves the operands' reads no bank conflict (440 to 385 us), three stages rather than four (less power), the
// result through LDS in whole rows (366 to 332). 4 wavefronts of 128 x 128 read a
// third less LDS, but need all 512 registers and hide no latency: 490 us, 368 with the accumulators held in place. A
// workgroup that stays and loads its next tile under the results' stores took 354.
#include <hip/hip_runtime.h>

#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "bitmap_spmm.h"
#include "device_common.h"

namespace {

typedef int w8_i4 __attribute__((ext_vector_type(4)));
typedef uint32_t w8_u2 __attribute__((ext_vector_type(2)));
typedef float w8_f4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void w8_lds_void;
typedef __attribute__((address_space(3))) const w8_i4 w8_lds_i4;
typedef __attribute__((address_space(3))) w8_u2 w8_lds_u2;

struct W8Args {
    const uint8_t *tiles;
    const int8_t *x;
    int64_t xs;
    const float *scale_w, *scale_x;
    uint16_t *y;
    int64_t ys, n;
    int M, bands, ktiles;
    int splits, per;         // workgroups that share a tile, column tiles of each (the last may have fewer)
    uint32_t *counters;      // splits > 1: arrivals at each tile, zero between calls
    uint8_t *parts;          // and their sums
    int last;                // last 16-byte piece of a token's row, as a byte offset
    uint32_t mtiles, ntiles; // tiles of the result
    bool once;               // W is read once, and too large to be there for the next call
};

// 4 neighbouring channels m .. m + 3 of token n.
__device__ __forceinline__ void w8_store(const W8Args &a, int64_t n, int m, w8_i4 v) {
    if (n >= a.n || m >= a.M) return;
    const float sx = a.scale_x[n];
    uint16_t *y = a.y + n * a.ys + m;
    if (m + 3 < a.M) {
        uint16_t h[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = bsp_f2h(bsp_rounded((float)v[r] * a.scale_w[m + r] * sx));
        __builtin_memcpy(y, h, 8);      // (at any 2-byte address)
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (m + r < a.M) y[r] = bsp_f2h(bsp_rounded((float)v[r] * a.scale_w[m + r] * sx));
    }
}

// The workgroup's tile. Consecutive workgroups go to the 8 dies in turn: where W is read more than once each
// die is given a run of neighbouring tiles, `deep` rows of tiles at a time, so that it reads few bands and tokens at
// once. (m = mtiles: none, the grid is a multiple of 8.)
struct W8Tile {
    uint32_t m, n, split;
};

__device__ __forceinline__ W8Tile w8_tile(const W8Args &a, uint32_t deep) {
    const uint32_t total = a.mtiles * a.ntiles * (uint32_t)a.splits, per = (total + 7) / 8;
    if (a.ntiles == 1 && a.splits == 1) return W8Tile{min(blockIdx.x, a.mtiles), 0, 0};
    const uint32_t at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (at >= total) return W8Tile{a.mtiles, 0, 0};
    const uint32_t tile = at / (uint32_t)a.splits, split = at - tile * (uint32_t)a.splits;
    const uint32_t strip = tile / (deep * a.ntiles), rest = tile - strip * (deep * a.ntiles);
    const uint32_t rows = min(deep, a.mtiles - strip * deep);
    return W8Tile{strip * deep + rest % rows, rest / rows, split};
}

// Agent-scope 16-byte stores and loads (aux 16: sc1): they go to the point of coherence that all dies share, so
// that a part is there for the workgroup that adds it once its store has completed.
__device__ __forceinline__ void w8_part_store(void *base, uint32_t bytes, uint32_t off, w8_i4 v) {
    typedef unsigned u4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), bsp_rsrc(base, bytes), off, 0, 16);
}
__device__ __forceinline__ w8_i4 w8_part_load(const void *base, uint32_t bytes, uint32_t off) {
    return __builtin_bit_cast(w8_i4, __builtin_amdgcn_raw_buffer_load_b128(bsp_rsrc(base, bytes), off, 0, 16));
}

// The e-th of the tile's splits after this one, e < splits.
__device__ __forceinline__ uint32_t w8_other(const W8Args &a, const W8Tile &tile, int e) {
    const uint32_t s = tile.split + (uint32_t)e;
    return s < (uint32_t)a.splits ? s : s - (uint32_t)a.splits;
}

// Whether this workgroup is the last to come to its tile (every thread gets the same answer). Each thread's part
// is stored before the call and complete before the barrier, the arrival follows it: the last one finds all parts.
__device__ __forceinline__ bool w8_last(const W8Args &a, const W8Tile &tile) {
    __shared__ uint32_t arrived;
    uint32_t *counter = a.counters + tile.m * a.ntiles + tile.n;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0) arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != (uint32_t)a.splits - 1) return false;
    if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// ---- at most 4 tokens: W streams from memory straight into registers ----

// A workgroup owns a band of 16 channels and 16 tokens; its W wavefronts take every W-th column tile of K, U of them
// on their way at once, and meet in LDS. W is read once: marked so, it costs the last-level cache nothing (one
// token x 12288 x 4096, cold: 10.0 us, through a ring 11.5).
template <int W, int U>
__global__ __launch_bounds__(64 * W) void k_w8_stream(const W8Args a) {
    __shared__ int32_t sums[256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const W8Tile tile = w8_tile(a, 1);
    if (tile.m >= a.mtiles) return;
    const int64_t n = (int64_t)tile.n * 16 + (lane & 15);
    const uint8_t *w = a.tiles + ((int64_t)tile.m * a.ktiles << 10) + lane * 16;
    const int8_t *x = a.x + min(n, a.n - 1) * a.xs;
    const int piece = (lane >> 4) * 16;
    w8_i4 acc = {0, 0, 0, 0};
    if (threadIdx.x < 256) sums[threadIdx.x] = 0;
    auto step = [&](int t, auto count) {
        constexpr int C = decltype(count)::value;
        w8_i4 A[C], B[C];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int k = t + u * W;
            A[u] = __builtin_nontemporal_load(reinterpret_cast<const w8_i4 *>(w + ((int64_t)k << 10)));
            // past the row's last piece W is zero: any value will do
            B[u] = *reinterpret_cast<const w8_i4 *>(x + min(k * 64 + piece, a.last));
        }
#pragma unroll
        for (int u = 0; u < C; ++u) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[u], B[u], acc, 0, 0, 0);
    };
    int t = wave;
    for (; t + (U - 1) * W < a.ktiles; t += U * W) step(t, std::integral_constant<int, U>{});
    for (; t < a.ktiles; t += W) step(t, std::integral_constant<int, 1>{});
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) atomicAdd(&sums[r * 64 + lane], acc[r]);
    __syncthreads();
    if (wave != 0) return;
    w8_i4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = sums[r * 64 + lane];
    w8_store(a, n, (int)tile.m * 16 + (lane >> 4) * 4, v);
}

// ---- more tokens: both operands through LDS ----

__device__ __forceinline__ void w8_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits until at most N pieces of this wavefront are on their way, and its reads of LDS are done.
template <int N>
__device__ __forceinline__ void w8_wait_vm() {
    static_assert(N >= 0 && N < 64, "the counter's range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}

// 1 KB from [base, base + bytes) to LDS, 16 bytes a lane from off + more; nothing is read past the end.
__device__ __forceinline__ void w8_dma(const void *base, uint32_t bytes, uint32_t dst, uint32_t off, uint32_t more) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(bsp_rsrc(base, bytes), (w8_lds_void *)(uintptr_t)dst, 16, off, more, 0, 0);
}

// The same of what is read once, past the last-level cache (aux 2: nt).
__device__ __forceinline__ void w8_dma_once(const void *base, uint32_t bytes, uint32_t dst, uint32_t off, uint32_t more) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(bsp_rsrc(base, bytes), (w8_lds_void *)(uintptr_t)dst, 16, off, more, 0, 2);
}

// Few tokens, through LDS: as k_w8_stream, each wavefront with a ring of P stages of its own (MB bands and NB
// blocks of tokens, 128 columns), which it alone fills and reads. A token's 128 columns come in one piece, whole lines
// of memory: with stages of 64 columns 32 tokens x 4096 x 11008 took 11.3 us in place of 10.4 (cold 17.2, 15.7). Two
// stages do as well as three (10.4, 10.6): the other wavefronts' loads are on their way beside a wavefront's own.
template <int NB, int MB, int W, int P>
__global__ __launch_bounds__(64 * W) void k_w8_ring(const W8Args a) {
    constexpr int PIECES = 2 * (MB + NB);
    constexpr uint32_t STAGE = PIECES * 1024u;
    extern __shared__ __attribute__((aligned(128))) uint8_t w8_lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const W8Tile tile = w8_tile(a, 1);
    if (tile.m >= a.mtiles) return;
    const int band = (int)tile.m * MB, nb = min(MB, a.bands - band);
    const int64_t n0 = (int64_t)tile.n * (NB * 16);
    const int ntok = (int)min((int64_t)(NB * 16), a.n - n0);
    const int k0 = (int)tile.split * a.per, kn = min(a.per, a.ktiles - k0), pairs = (kn + 1) / 2;
    const uint8_t *wbase = a.tiles + (((int64_t)band * a.ktiles + k0) << 10);
    const int8_t *xbase = a.x + n0 * a.xs + k0 * 64;
    const uint32_t wbytes = ((uint32_t)nb * (uint32_t)a.ktiles - k0) << 10, xbytes = (uint32_t)ntok * (uint32_t)a.xs - k0 * 64;
    const uint32_t lds = (uint32_t)(uintptr_t)(w8_lds_void *)w8_lds + wave * (P * STAGE);
    // a stage: MB bands of the first 64 columns, of the second, then 8 tokens a piece. Lane l brings piece
    // (l % 8) ^ (row / 2) of token l / 8, row its place among the block's 16: 16 lanes that read 16 tokens' pieces
    // from LDS together find them on different banks
    uint32_t woff[MB], xoff[2 * NB];
#pragma unroll
    for (int c = 0; c < MB; ++c) woff[c] = ((uint32_t)min(c, nb - 1) * (uint32_t)a.ktiles << 10) + lane * 16;
#pragma unroll
    for (int c = 0; c < 2 * NB; ++c) {
        const int row = (c & 1) * 8 + (lane >> 3);
        xoff[c] = (uint32_t)min((c >> 1) * 16 + row, ntok - 1) * (uint32_t)a.xs + (((lane & 7) ^ (row >> 1)) << 4);
    }
    auto fetch = [&](int t, uint32_t slot) {
        const uint32_t dst = lds + slot * STAGE;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t k = (uint32_t)min(2 * t + q, kn - 1) << 10;
#pragma unroll
            for (int c = 0; c < MB; ++c) {
                if (a.once)
                    w8_dma_once(wbase, wbytes, dst + (q * MB + c) * 1024u, woff[c], k);
                else
                    w8_dma(wbase, wbytes, dst + (q * MB + c) * 1024u, woff[c], k);
            }
        }
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) w8_dma(xbase, xbytes, dst + (2 * MB + c) * 1024u, xoff[c], (uint32_t)t << 7);
    };
    const uint32_t abase = lds + lane * 16, brow = lane & 15, bpiece = lane >> 4,
                   bbase = lds + 2 * MB * 1024u + brow * 128u;
    w8_i4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = w8_i4{0, 0, 0, 0};
    uint32_t fill = 0, use = 0;
#pragma unroll
    for (int s = 0; s < P - 1; ++s)
        if (wave + s * W < pairs) fetch(wave + s * W, fill++);
    for (int t = wave; t < pairs; t += W) {
        const bool more = t + (P - 1) * W < pairs;
        if (more)
            w8_wait_vm<(P - 2) * PIECES>();
        else
            w8_wait_vm<0>();
        w8_i4 A[2][MB], B[2][NB];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int i = 0; i < MB; ++i) A[q][i] = *(w8_lds_i4 *)(uintptr_t)(abase + use * STAGE + (q * MB + i) * 1024u);
#pragma unroll
            for (int j = 0; j < NB; ++j)
                B[q][j] = *(w8_lds_i4 *)(uintptr_t)(bbase + use * STAGE + j * 2048u + (((4 * q + bpiece) ^ (brow >> 1)) << 4));
        }
        use = use + 1 == P ? 0 : use + 1;
        if (more) {
            fetch(t + (P - 1) * W, fill);
            fill = fill + 1 == P ? 0 : fill + 1;
        }
        // past the last column tile W's second half is its first again, and not added
        const bool both = 2 * t + 1 < kn;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (q == 0 || both)
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[q][i], B[q][j], acc[i][j], 0, 0, 0);
    }
    w8_wait_vm<0>();
    __syncthreads();
    int32_t *sums = reinterpret_cast<int32_t *>(w8_lds);
    for (int i = threadIdx.x; i < MB * NB * 256; i += 64 * W) sums[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) atomicAdd(&sums[((i * NB + j) * 4 + r) * 64 + lane], acc[i][j][r]);
    __syncthreads();
    // the wavefront's blocks of the tile: f = wave, wave + W, ...
    constexpr uint32_t PART = MB * NB * 1024u;
    auto block = [&](int f) {
        w8_i4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = sums[(f * 4 + r) * 64 + lane];
        return v;
    };
    uint8_t *parts = a.parts + (int64_t)(tile.m * a.ntiles + tile.n) * a.splits * PART;
    if (a.splits > 1) {
        for (int f = wave; f < MB * NB; f += W)
            w8_part_store(parts, PART * (uint32_t)a.splits, tile.split * PART + f * 1024u + lane * 16, block(f));
        if (!w8_last(a, tile)) return;
    }
    for (int f = wave; f < MB * NB; f += W) {
        w8_i4 v = block(f);
        // the others' parts, eight on their way at once
        for (int s = 1; s < a.splits; s += 8) {
            w8_i4 p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = w8_i4{0, 0, 0, 0};
                if (s + e < a.splits)
                    p[e] = w8_part_load(parts, PART * (uint32_t)a.splits, w8_other(a, tile, s + e) * PART + f * 1024u + lane * 16);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v += p[e];
        }
        if (band + f / NB < a.bands)
            w8_store(a, n0 + f % NB * 16 + (lane & 15), (band + f / NB) * 16 + (lane >> 4) * 4, v);
    }
}

// A workgroup's result is (WM TM 16) channels x (WN TN 16) tokens; a wavefront's TM x TN
// blocks of 16 x 16. Stages of KS x 64 columns of K pass through a ring of R in LDS.
template <int WM, int WN, int TM, int TN, int KS, int R>
__global__ __launch_bounds__(64 * WM * WN) void k_w8_tiles(const W8Args a) {
    constexpr int W = WM * WN, MBANDS = WM * TM, NBLOCKS = WN * TN, CHUNKS = MBANDS + NBLOCKS, CW = CHUNKS / W;
    static_assert(CHUNKS % W == 0, "every wavefront moves as many pieces");
    static_assert(KS == 1 || KS % 2 == 0, "the operands' two sets of registers change places");
    constexpr uint32_t STEP = CHUNKS * 1024u, STAGE = KS * STEP;
    extern __shared__ __attribute__((aligned(128))) uint8_t w8_lds[];
    const uint32_t lds = (uint32_t)(uintptr_t)(w8_lds_void *)w8_lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const W8Tile tile = w8_tile(a, 8);
    if (tile.m >= a.mtiles) return;
    const int band0 = (int)tile.m * MBANDS;
    const int64_t n0 = (int64_t)tile.n * (NBLOCKS * 16);
    const int ntok = (int)min((int64_t)(NBLOCKS * 16), a.n - n0);
    const int nb = min(MBANDS, a.bands - band0);
    const int k0 = (int)tile.split * a.per, kn = min(a.per, a.ktiles - k0);
    const uint8_t *wbase = a.tiles + (((int64_t)band0 * a.ktiles + k0) << 10);
    const int8_t *xbase = a.x + n0 * a.xs + k0 * 64;
    const uint32_t wbytes = ((uint32_t)nb * (uint32_t)a.ktiles - k0) << 10, xbytes = (uint32_t)ntok * (uint32_t)a.xs - k0 * 64;
    // the pieces of 1 KB this wavefront moves for each 64 columns: chunks wave, wave + W, ...
    uint32_t off[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) {
        const int chunk = wave + c * W;
        if (chunk < MBANDS) {
            off[c] = ((uint32_t)min(chunk, nb - 1) * (uint32_t)a.ktiles << 10) + lane * 16;
        } else {
            // lane l brings piece (l % 4) ^ (-(l / 16) % 4) of token l / 4: 64 bytes a token together, and the
            // lanes that read LDS in the same cycle on different banks
            const int row = min((chunk - MBANDS) * 16 + (lane >> 2), ntok - 1);
            off[c] = (uint32_t)row * (uint32_t)a.xs + (((lane & 3) ^ (-(lane >> 4) & 3)) << 4);
        }
    }
    auto fetch = [&](int t, uint32_t slot) {
#pragma unroll
        for (int q = 0; q < KS; ++q) {
            const uint32_t k = (uint32_t)min(t * KS + q, kn - 1);
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                const int chunk = wave + c * W;
                const uint32_t dst = lds + slot * STAGE + q * STEP + (uint32_t)chunk * 1024u;
                if (chunk < MBANDS)
                    w8_dma(wbase, wbytes, dst, off[c], k << 10);
                else
                    w8_dma(xbase, xbytes, dst, off[c], k << 6);
            }
        }
    };
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t abase = lds + (uint32_t)(wm * TM) * 1024u + lane * 16;
    const uint32_t brow = lane & 15, bbase = lds + (uint32_t)(MBANDS + wn * TN) * 1024u +
                                            (brow * 4 + ((lane >> 4) ^ (-(brow >> 2) & 3))) * 16;
    w8_i4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = w8_i4{0, 0, 0, 0};
    // The operands of 64 columns are in registers when their turn comes: the next ones are read from
    // LDS under their matrix instructions, and at the last ones of stage t stage t + R takes its place.
    w8_i4 A[2][TM], B[2][TN];
    uint32_t slot = 0;
    auto read = [&](uint32_t at, w8_i4 (&x)[TM], w8_i4 (&y)[TN]) {
#pragma unroll
        for (int j = 0; j < TN; ++j) y[j] = *(w8_lds_i4 *)(uintptr_t)(bbase + at + j * 1024u);
#pragma unroll
        for (int i = 0; i < TM; ++i) x[i] = *(w8_lds_i4 *)(uintptr_t)(abase + at + i * 1024u);
    };
    auto multiply = [&](w8_i4 (&x)[TM], w8_i4 (&y)[TN], auto pieces) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[i], y[j], acc[i][j], 0, 0, 0);
        // reads and pieces spread over the matrix instructions
        constexpr int READS = TM + TN, VM = decltype(pieces)::value, PER = TM * TN / (READS + VM) > 0 ? TM * TN / (READS + VM) : 1;
#pragma unroll
        for (int c = 0; c < READS; ++c) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, PER, 0);
        }
#pragma unroll
        for (int c = 0; c < VM; ++c) {
            __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, PER, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto turn = [&](int t, w8_i4 (&x)[TM], w8_i4 (&y)[TN], w8_i4 (&x1)[TM], w8_i4 (&y1)[TN]) {
#pragma unroll
        for (int q = 0; q + 1 < KS; ++q) {
            const bool odd = q & 1;
            read(slot * STAGE + (q + 1) * STEP, odd ? x : x1, odd ? y : y1);
            if (q == 0 || t * KS + q < kn) multiply(odd ? x1 : x, odd ? y1 : y, std::integral_constant<int, 0>{});
        }
        w8_wait_vm<(R - 2) * CW * KS>();      // this wavefront's pieces of stage t + 1, and its reads of stage t
        w8_barrier();                         // every wavefront's
        fetch(t + R, slot);
        slot = slot + 1 == R ? 0 : slot + 1;
        constexpr bool last = KS > 1;         // (KS even: the last operands lie in the second set, the next in the first)
        read(slot * STAGE, last ? x : x1, last ? y : y1);
        if (KS == 1 || t * KS + KS - 1 < kn) multiply(last ? x1 : x, last ? y1 : y, std::integral_constant<int, CW * KS>{});
    };
#pragma unroll
    for (int s = 0; s < R; ++s) fetch(s, s);
    w8_wait_vm<(R - 1) * CW * KS>();
    w8_barrier();
    read(0, A[0], B[0]);
    int t = 0;
    if constexpr (KS > 1) {
        for (; t * KS < kn; ++t) turn(t, A[0], B[0], A[1], B[1]);
    } else {
        for (; t + 1 < kn; t += 2) {
            turn(t, A[0], B[0], A[1], B[1]);
            turn(t + 1, A[1], B[1], A[0], B[0]);
        }
        if (t < kn) turn(t, A[0], B[0], A[1], B[1]);
    }
    w8_wait_vm<0>();
    w8_barrier();
    if (a.splits > 1) {
        constexpr uint32_t PART = MBANDS * NBLOCKS * 1024u;
        uint8_t *parts = a.parts + (int64_t)(tile.m * a.ntiles + tile.n) * a.splits * PART;
        const uint32_t all = PART * (uint32_t)a.splits, mine = (uint32_t)(wave * TM * TN) * 1024u + lane * 16;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                w8_part_store(parts, all, tile.split * PART + mine + (i * TN + j) * 1024u, acc[i][j]);
        if (!w8_last(a, tile)) return;
        // the others' parts, as many on their way at once as registers hold
        constexpr int AT_ONCE = TM * TN <= 4 ? 8 : TM * TN <= 8 ? 4 : TM * TN <= 16 ? 2 : 1;
        for (int s = 1; s < a.splits; s += AT_ONCE) {
            w8_i4 p[AT_ONCE][TM][TN];
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e) {
                const uint32_t from = w8_other(a, tile, s + e) * PART + mine;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        p[e][i][j] = w8_i4{0, 0, 0, 0};
                        if (s + e < a.splits) p[e][i][j] = w8_part_load(parts, all, from + (i * TN + j) * 1024u);
                    }
            }
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] += p[e][i][j];
        }
    }
    // The result by way of LDS, 16 tokens at a time in the wavefront's own part of it: a token's TM x 16 channels
    // leave together, 16 bytes a lane.
    constexpr int PITCH = TM * 16 + 8, LPR = TM * 2, RPI = 64 / LPR;      // halves a token, lanes a token, tokens at once
    static_assert(W * 16 * PITCH * 2 <= (int)(R * STAGE), "the ring holds it");
    const uint32_t out = lds + (uint32_t)(wave * 16 * PITCH * 2);
    const int m0 = (band0 + wm * TM) * 16;
    w8_f4 sw[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + i * 16 + (lane >> 4) * 4;
        if (m + 3 < a.M) {
            __builtin_memcpy(&sw[i], a.scale_w + m, 16);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) sw[i][r] = m + r < a.M ? a.scale_w[m + r] : 0.0f;
        }
    }
    const int piece = m0 + lane % LPR * 8;      // the lane's 8 channels
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int first = (wn * TN + j) * 16;
        const float sx = a.scale_x[n0 + min(first + (lane & 15), ntok - 1)];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            uint16_t h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = bsp_f2h(bsp_rounded((float)acc[i][j][r] * sw[i][r] * sx));
            *(w8_lds_u2 *)(uintptr_t)(out + (uint32_t)((lane & 15) * PITCH + i * 16 + (lane >> 4) * 4) * 2) =
                w8_u2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int c = 0; c < 16 / RPI; ++c) {
            const int row = c * RPI + lane / LPR;
            const w8_i4 v = *(w8_lds_i4 *)(uintptr_t)(out + (uint32_t)(row * PITCH + lane % LPR * 8) * 2);
            if (first + row >= ntok) continue;
            uint16_t *y = a.y + (n0 + first + row) * a.ys + piece;
            if (piece + 8 <= a.M) {
                __builtin_memcpy(y, &v, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (piece + e < a.M) y[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

#define W8_MOST_LDS (160u * 1024u - 256u)      // beside the kernels' own words

// Allows a kernel its LDS, once for each device.
template <class Kernel>
void w8_allow(Kernel *kernel, unsigned lds, std::atomic<uint64_t> &done) {
    int device = 0;
    if (lds <= 65536 || hipGetDevice(&device) != hipSuccess) return;
    const uint64_t bit = UINT64_C(1) << (device & 63);
    if (device < 64 && (done.load(std::memory_order_relaxed) & bit) != 0) return;
    if (hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) == hipSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
}

// Launches are for a grid of whole eights (w8_tile).
unsigned w8_grid(W8Args &a, int bands, int blocks) {
    a.mtiles = (uint32_t)((a.bands + bands - 1) / bands), a.ntiles = (uint32_t)((a.n + blocks * 16 - 1) / (blocks * 16));
    return (a.mtiles * a.ntiles * (uint32_t)a.splits + 7) / 8 * 8;
}

template <int W, int U>
void w8_stream(W8Args &a, hipStream_t stream) {
    const unsigned grid = w8_grid(a, 1, 1);
    hipLaunchKernelGGL((k_w8_stream<W, U>), dim3(grid), dim3(64 * W), 0, stream, a);
}

// Weights of 96 MB and more, read once a call, are mostly gone from the last-level cache (256 MB, shared with all else)
// by the next one: marked so. 8 tokens x 128256 x 4096 87 us (unmarked 98), 32000 x 4096 cold 23.1 (27.2), on nothing but
// itself 22.2 (21.7). Smaller ones may still be there: 12288 x 4096 cold 10.5 (11.9), on itself 10.0 (8.3).
#define W8_ONCE (INT64_C(96) << 10)      // in tiles of 1 KB

template <int NB, int MB, int W, int P>
void w8_ring(W8Args &a, hipStream_t stream) {
    constexpr unsigned LDS = 2 * (MB + NB) * 1024u * P * W;
    static_assert(LDS <= W8_MOST_LDS, "a workgroup's LDS");
    static std::atomic<uint64_t> done{0};
    w8_allow(k_w8_ring<NB, MB, W, P>, LDS, done);
    const unsigned grid = w8_grid(a, MB, NB);
    a.once = a.ntiles == 1 && (int64_t)a.bands * a.ktiles >= W8_ONCE;
    hipLaunchKernelGGL((k_w8_ring<NB, MB, W, P>), dim3(grid), dim3(64 * W), LDS, stream, a);
}

template <int WM, int WN, int TM, int TN, int KS, int R>
void w8_tiles(W8Args &a, hipStream_t stream) {
    constexpr unsigned LDS = (WM * TM + WN * TN) * 1024u * KS * R;
    static_assert(LDS <= W8_MOST_LDS, "a workgroup's LDS");
    static std::atomic<uint64_t> done{0};
    w8_allow(k_w8_tiles<WM, WN, TM, TN, KS, R>, LDS, done);
    const unsigned grid = w8_grid(a, WM * TM, WN * TN);
    hipLaunchKernelGGL((k_w8_tiles<WM, WN, TM, TN, KS, R>), dim3(grid), dim3(64 * WM * WN), LDS, stream, a);
}

typedef void (*W8Run)(W8Args &, hipStream_t);

struct W8Shape {
    int bands, blocks;       // a workgroup's tile, in 16s
    W8Run run;
    const char *name;
};

#define W8_STREAM(W, U) {1, 1, w8_stream<W, U>, "k_w8_stream<" #W ", " #U ">"}
#define W8_RING(NB, MB, W, P) {MB, NB, w8_ring<NB, MB, W, P>, "k_w8_ring<" #NB ", " #MB ", " #W ", " #P ">"}
#define W8_TILES(WM, WN, TM, TN, KS, R) \
    {WM * TM, WN * TN, w8_tiles<WM, WN, TM, TN, KS, R>, "k_w8_tiles<" #WM ", " #WN ", " #TM ", " #TN ", " #KS ", " #R ">"}

// The first six split K over their wavefronts, the others the tile.
const W8Shape W8_SHAPES[] = {
    W8_RING(1, 1, 16, 2), W8_RING(2, 1, 8, 2), W8_RING(2, 2, 8, 2), W8_RING(4, 1, 4, 3), W8_RING(2, 4, 6, 2),
    W8_RING(4, 2, 6, 2), W8_TILES(2, 2, 2, 2, 4, 3), W8_TILES(2, 2, 4, 2, 2, 3), W8_TILES(2, 4, 4, 2, 1, 4),
    W8_TILES(2, 4, 8, 2, 1, 4), W8_TILES(2, 4, 8, 4, 1, 3),
};
// For few tokens alone (w8_plan).
const W8Shape W8_STREAM_16 = W8_STREAM(16, 2), W8_STREAM_8 = W8_STREAM(8, 4), W8_RING_4 = W8_RING(1, 1, 4, 2);

#define W8_COUNTERS 16384      // arrival counters at the head of a workspace (64 KB, as everywhere in the library)
#define W8_SPLIT_TILES 256     // more tiles fill the card without splits
static_assert(W8_SPLIT_TILES <= W8_COUNTERS, "an arrival counter a tile");
#define W8_MOST_TILES ((INT64_C(1) << 22) - 8)      // of a launch: fewer than 2^32 threads

#define W8_MOST_ROWS (W8_MOST_TILES * 16)

struct W8Plan {
    const W8Shape *shape;
    int splits, per;
    int64_t part_bytes;      // of all tiles and splits
};

// A tile's time is that of its operands' way into the CU (a KB of them every 1 / 57 us, the rate that tiles reach) or of its
// matrix instructions (a 16 x 16 x 64 block every 1 / 330 us), whichever is longer; the tiles of
// a CU come one after the other. Splitting K shares a tile among workgroups, which then store and one of which
// adds the parts: 2.5 us, 1.3 for each, and their bytes at 4 TB/s.
//
// Few tokens are tiles of one band, and how many wavefronts share its columns is a matter of how many bands there are
// (us on the same W again and again / past the last-level cache):
// - up to 4 tokens and 32 MB of weights W streams past LDS: 1 x 4096 x 8192 4.8 / 7.1, through the ring of 16 wavefronts
//   5.2 / 9.0; 1 x 12288 x 4096 7.7 / 9.8, through that of 4 7.7 / 11.5; with less the rings do as well (1 x 4096 x 4096 4.0).
//   Two workgroups of 16 wavefronts are on a CU at once, four of 8: past 512 bands those have no second round (12288 x 4096
//   7.7, of 16 8.8; 32768 x 1024 5.9 and 7.5; at 512 bands alike, 4.7). Long rows want the wavefronts (12288 x 8192 of 8 14.2,
//   of 16 13.9; 4096 x 11008 8.5 and 6.6): the border is 128 column tiles (just below it, at 513 bands, 16 would be better:
//   8208 x 8128 11.9 and 10.6).
// - up to 16 tokens past 256 bands: the ring of 16 wavefronts fills a CU's LDS, so band 257 waits for a second
//   round; five of 4 wavefronts fit (8 x 12288 x 4096 7.8 / 11.6, of 16 11.2 / 14.4; 8 x 4112 x 1024 2.7 and 3.8; at 256
//   bands 8 x 4096 x 4096 5.6, of 16 4.1). Few bands past 256 and long rows lose by it (8 x 4112 x 11008 12.8, of 16 11.3), and
//   16 x 128256 x 4096 takes 97 for the 88 of the tiles below.
W8Plan w8_plan(int64_t bands, int64_t ktiles, int64_t n, bool split) {
    const int k = (int)ktiles;
    if (k == 0 || (n <= 4 && bands * ktiles >= 32768))
        return {bands > 512 && ktiles < 128 ? &W8_STREAM_8 : &W8_STREAM_16, 1, k, 0};
    if (n <= 16 && bands > 256) return {&W8_RING_4, 1, k, 0};
    W8Plan best{nullptr, 1, k, 0};
    double least = 0.0;
    for (const W8Shape &p : W8_SHAPES) {
        const int64_t tiles = (bands + p.bands - 1) / p.bands * ((n + p.blocks * 16 - 1) / (p.blocks * 16));
        const double one = std::max((p.bands + p.blocks) / 57.0, p.bands * p.blocks / 330.0);
        for (int splits = 1; splits <= 16; splits *= 2) {
            const int per = ((k + splits - 1) / splits + 1) & ~1, used = (k + per - 1) / per;
            double t = (double)((tiles * used + 255) / 256) * one * per;
            int64_t bytes = 0;
            if (splits > 1) {
                if (!split || per < 8 || tiles > W8_SPLIT_TILES) break;
                bytes = tiles * used * p.bands * p.blocks * 1024;
                t += 2.5 + 1.3 * splits + (double)bytes * 0.25e-6;
            }
            if (best.shape == nullptr || t < least) best = W8Plan{&p, used, per, bytes}, least = t;
        }
    }
    return best;
}

// The tokens of one launch: so many that tiles of 16 could pass a launch's go in runs.
int64_t w8_most_tokens(int64_t bands) { return W8_MOST_TILES / bands * 16; }

}  // namespace

extern "C" int gemm_w8a8_describe(int64_t M, int64_t K, int64_t N, int with_workspace, char *buf, size_t n) {
    if (M < 0 || K < 0 || N < 0 || buf == nullptr || n == 0) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > W8_MOST_ROWS || N > INT32_MAX) return BSP_E_OVERFLOW;
    const int at = snprintf(buf, n, "dtype=int8 M=%lld K=%lld N=%lld", (long long)M, (long long)K, (long long)N);
    if (M == 0 || N == 0 || at < 0 || (size_t)at >= n) return BSP_OK;
    const int64_t bands = (M + 15) / 16, most = w8_most_tokens(bands);
    const W8Plan p = w8_plan(bands, (K + 63) / 64, std::min(N, most), with_workspace != 0 && N <= most);
    snprintf(buf + at, n - at, " -> kernel=%s tile=%dx%d splits=%d", p.shape->name, p.shape->bands * 16, p.shape->blocks * 16,
             p.splits);
    return BSP_OK;
}

extern "C" int gemm_w8a8_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t *bytes) {
    if (bytes == nullptr || M < 0 || K < 0 || N < 0) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > W8_MOST_ROWS || N > INT32_MAX) return BSP_E_OVERFLOW;
    *bytes = 0;
    if (M == 0 || K == 0) return BSP_OK;
    // plans change with every 16 tokens (and after 4), and more of them can take less
    const int64_t bands = (M + 15) / 16, ktiles = (K + 63) / 64;
    for (int64_t n = 1; n <= N; n = n == 1 ? 5 : n == 5 ? 17 : n + 16) {
        if ((bands + 15) / 16 * ((n + 255) / 256) > W8_SPLIT_TILES) break;
        const W8Plan p = w8_plan(bands, ktiles, n, true);
        if (p.splits > 1) *bytes = std::max(*bytes, W8_COUNTERS * 4 + p.part_bytes);
    }
    return BSP_OK;
}

extern "C" int gemm_w8a8_dq(const uint8_t *tiles, int64_t M, int64_t K, const int8_t *X, int64_t x_stride, int64_t N,
                            const float *scale_w, const float *scale_x, uint16_t *Y, int64_t y_stride,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (M < 0 || K < 0 || N < 0 || workspace_bytes < 0) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > W8_MOST_ROWS || N > INT32_MAX) return BSP_E_OVERFLOW;
    if (M == 0 || N == 0) return BSP_OK;
    if (Y == nullptr || scale_w == nullptr || scale_x == nullptr || y_stride < M) return BSP_E_ARG;
    if (K > 0 && (tiles == nullptr || X == nullptr || x_stride < K || x_stride % 16 != 0)) return BSP_E_ARG;
    if ((((uintptr_t)tiles | (uintptr_t)X) & 15u) != 0 || ((uintptr_t)Y & 1u) != 0) return BSP_E_ARG;
    if ((((uintptr_t)scale_w | (uintptr_t)scale_x) & 3u) != 0) return BSP_E_ARG;
    if ((workspace == nullptr) != (workspace_bytes == 0) || ((uintptr_t)workspace & 255u) != 0) return BSP_E_ARG;
    // the tokens of a tile (256 at most) are reached by 32-bit offsets
    if (K > 0 && x_stride >= INT64_C(1) << 23) return BSP_E_OVERFLOW;
    W8Args a{};
    a.tiles = tiles, a.xs = x_stride, a.scale_w = scale_w, a.ys = y_stride;
    a.M = (int)M, a.bands = (int)((M + 15) / 16), a.ktiles = (int)((K + 63) / 64);
    a.last = (int)std::max<int64_t>(x_stride - 16, 0);
    const int64_t most = w8_most_tokens(a.bands);
    for (int64_t t = 0; t < N; t += most) {
        a.n = std::min(N - t, most);
        a.x = X + t * x_stride, a.scale_x = scale_x + t, a.y = Y + t * y_stride;
        const W8Plan p = w8_plan(a.bands, a.ktiles, a.n, workspace != nullptr && N <= most);
        a.splits = p.splits, a.per = p.per;
        if (p.splits > 1) {
            if (workspace_bytes < W8_COUNTERS * 4 + p.part_bytes) return BSP_E_CAPACITY;
            a.counters = (uint32_t *)workspace, a.parts = (uint8_t *)workspace + W8_COUNTERS * 4;
        }
        p.shape->run(a, stream);
    }
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
