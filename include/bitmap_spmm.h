/*
 * bitmap_spmm.h -- C ABI of the bitmap-tiled sparse x dense matmul for AMD
 * Instinct MI355X (gfx950).
 *
 * Computes Y = W_sparse * X, the problem statement of SPDP ("Unified
 * Static-Dynamic Pruning for Efficient LLM Inference", Sec. 2.2) and of the
 * UnionSparse SpMM kernel ("UnionSparse: An Index-Efficient Sparsity
 * Framework for Low-Bit Sparse LLM Inference on Edge", IEEE TCAD, Sec. VI),
 * for the decode-phase shapes those pages study: W is M x K with 30-70 %
 * unstructured sparsity, X is a skinny K x N activation matrix, N = 1..32.
 *
 * ---------------------------------------------------------------------------
 * Encoded format ("BT64"): UnionSparse Sec. V-A, "IE-BME Representation",
 * with one area per tile (R_A = C_A = 1, Q = 1) on 1 x 64 row tiles.
 *   T = ceil(K/64) tiles per row; G = M*T tiles; tile g = m*T + t covers
 *   columns 64t .. 64t+63 of row m (row-major tile order).
 *   bitmaps[g]   uint64. Bit j is set iff W[m][64t+j] != 0; bit 0 is the
 *                first column (the LSB-first packing of the Fig. 7 example).
 *                Bits of columns >= K are zero.
 *   offsets[g]   uint32, the number of nonzeros in tiles 0..g-1 ("Union Value
 *                Offsets" with Q = 1); offsets[G] = nnz. G+1 entries.
 *   payload      the nonzeros in tile order and, inside a tile, in column
 *                order: value (m, 64t+j) is element offsets[g] + rank, rank =
 *                popcount(bitmaps[g] & ((1<<j)-1)) ("Compressed Values").
 *                int4: element e is byte e>>1, low nibble when e is even, a
 *                4-bit two's-complement code; ceil(nnz/2) bytes, an odd count
 *                leaves the final high nibble zero.
 *                fp16: element e is uint16 e (IEEE binary16 bits); 2*nnz bytes.
 * Activations: X is K x N stored column by column, i.e. an [N][K] array.
 *   int4: packed along K, two per byte, low nibble = even k, row stride
 *   ceil(K/2) bytes. fp16: row stride K elements.
 * Output: Y is M x N stored column by column, i.e. [N][M]; int32 for the int4
 *   path, fp16 for the fp16 path. Y is fully overwritten, never accumulated.
 * ---------------------------------------------------------------------------
 *
 * Conventions
 *   - Every entry point returns a bsp_status. No C++ exception crosses the ABI.
 *   - Arguments are checked on the host before any HIP call, so a bad call
 *     returns an error code without touching the GPU.
 *   - SpMM calls are asynchronous on `stream` (NULL = the null stream); a fault
 *     inside a kernel surfaces at the caller's next synchronisation. The
 *     content of the encoded stream is not validated on the device (that
 *     would cost a full extra pass over HBM): a corrupt stream gives a wrong
 *     Y, never an out-of-bounds access, because every payload read is bounded
 *     by `payload_bytes` in hardware (buffer-resource loads).
 *   - The calls hold no state between calls, allocate no memory and are
 *     reentrant; concurrent calls on different streams are allowed.
 */
#ifndef BITMAP_SPMM_H
#define BITMAP_SPMM_H

#include <stdint.h>
#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum bsp_status {
    BSP_OK = 0,
    BSP_E_ARG = 1,       /* null pointer, negative size, N > 32, ldw < K, unknown dtype/algo */
    BSP_E_RANGE = 2,     /* a weight outside its type's range: int4 [-8, 7], int2 [-2, 1] */
    BSP_E_CAPACITY = 3,  /* payload buffer smaller than the encoded payload, a workspace smaller than the call needs */
    BSP_E_OVERFLOW = 4,  /* nnz >= 2^32, K >= 2^25 (int32 sums could overflow), an index beyond 2^31, or a size past what
                            an entry point names */
    BSP_E_HIP = 5,       /* a HIP launch error (hipGetLastError after the launch) */
    BSP_E_UNSUPPORTED = 6 /* a kernel forced through an *_algo entry point cannot run this shape, or a form that has no
                             kernel (head_dim, rot, sequences) */
} bsp_status;

/* BSP_INT8 is a type of caches (bsp_kv_cache) and token codes (quantize_tokens_f16) only; BSP_INT2 of weights only. */
typedef enum bsp_dtype { BSP_INT4 = 0, BSP_FP16 = 1, BSP_INT2 = 2, BSP_INT8 = 3 } bsp_dtype;

/* Kernel choice for the *_algo entry points. BSP_ALGO_AUTO applies the
 * library's shape-aware selection (by N, density, M, K). A forced choice
 * that cannot run the shape returns BSP_E_UNSUPPORTED and launches nothing;
 * it never falls back to another kernel. */
typedef enum bsp_algo {
    BSP_ALGO_AUTO = 0,
    BSP_ALGO_ROWWAVE = 1,   /* one wavefront per output row; plain per-nonzero decode (any shape) */
    BSP_ALGO_MFMA = 2,      /* lane-per-tile decode from LDS-staged 16-row blocks over all of K + int8 / fp16
                               MFMA (int4: K <= 16384; fp16: K <= 4096, K % 8 == 0) */
    BSP_ALGO_SPLITK = 3     /* the same decode and MFMA over K ranges of block sets (UnionSparse Sec. VI-C,
                               Alg. 2: partial tiles, then a reduction): any K (fp16: K % 8 == 0); with a
                               workspace (the *_ws entry points) a block set's K ranges run on several
                               workgroups and meet in it */
} bsp_algo;

/* The device payload allocation handed to the SpMM calls is a whole number
 * of 16-byte units (zero-filled past the encoded payload): kernels read it in
 * whole dwords, and the hardware range check is applied to whole dwords. */
#define BSP_PAYLOAD_ALIGN 16

/* Largest N the SpMM entry points accept. */
#define BSP_MAX_N 32
/* K bound that keeps every int4 x int4 sum inside int32: |Y| <= 64*K < 2^31. */
#define BSP_MAX_K ((int64_t)1 << 25)

/*
 * encode_bitmap_tiles -- host-side encoder (UnionSparse Sec. V-A, Q = 1 on
 * 1 x 64 tiles; the encoded form is produced offline and cached, Sec. V-B).
 *
 *   dtype    BSP_INT4: W is const int8_t*, values in [-8, 7];
 *            BSP_INT2: W is const int8_t*, values in [-2, 1] (the W2A4 weights
 *            of UnionSparse Sec. VII, Fig. 11): payload element e is the 2-bit
 *            two's-complement code in byte e>>2 at bits 2*(e&3), lowest first;
 *            BSP_FP16: W is const uint16_t* holding IEEE binary16 bits
 *            (+0 and -0 are zero; every other pattern, NaN included, is stored).
 *   W        HOST memory, row-major M x K with leading dimension ldw >= K.
 *   bitmaps  HOST, caller-allocated, M*T entries (T = ceil(K/64)), or NULL.
 *   offsets  HOST, caller-allocated, M*T+1 entries, or NULL.
 *   payload  HOST, caller-allocated, payload_capacity_bytes bytes, or NULL for
 *            a size query (then bitmaps/offsets may also be NULL).
 *   nnz_out, payload_bytes_out  written on BSP_OK and on BSP_E_CAPACITY
 *            (either may be NULL). payload_bytes = ceil(nnz/2) (int4),
 *            ceil(nnz/4) (int2) or 2*nnz (fp16).
 * Returns BSP_E_ARG, BSP_E_RANGE (nothing written), BSP_E_OVERFLOW
 * (nnz >= 2^32), BSP_E_CAPACITY (counts written, arrays untouched) or BSP_OK.
 * Multi-threaded over rows; the output does not depend on the thread count.
 */
int encode_bitmap_tiles(int dtype, const void *W, int64_t M, int64_t K, int64_t ldw,
                        uint64_t *bitmaps, uint32_t *offsets,
                        void *payload, int64_t payload_capacity_bytes,
                        int64_t *nnz_out, int64_t *payload_bytes_out);

/*
 * pack_int4_activations -- host helper that writes int4 activations in the
 * layout the SpMM reads: X (values in [-8, 7], HOST [N][K] int8, row stride
 * ldx >= K) -> Xp (HOST, N * ceil(K/2) bytes). Returns BSP_E_RANGE for a
 * value outside [-8, 7] (Xp then undefined).
 */
int pack_int4_activations(const int8_t *X, int64_t N, int64_t K, int64_t ldx, uint8_t *Xp);

/*
 * spmm_bitmap_w4a4 -- Y = W * X with int4 W (BT64 stream) and int4 X, exact
 * int32 result (UnionSparse Sec. VI; W4A4 decode shapes of Sec. VII-A).
 *
 *   bitmaps, offsets, payload   DEVICE, the encoded W (M*T, M*T+1 entries and
 *                               payload_bytes bytes); payload may be NULL only
 *                               if payload_bytes == 0.
 *   payload_bytes               size of the payload allocation: a multiple of
 *                               BSP_PAYLOAD_ALIGN, >= ceil(nnz/2), bytes past the
 *                               encoded payload zero. No byte at or past it is read.
 *   M, K                        0 <= M < 2^31, 0 <= K < 2^25, M*ceil(K/64) < 2^31.
 *   X                           DEVICE, [N][ceil(K/2)] packed int4. The MFMA and split-K
 *                               kernels need X on a 4-byte boundary (any allocation is;
 *                               fp16: 16 bytes); an X off it runs the plain kernel
 *                               (BSP_ALGO_AUTO) or is refused with BSP_E_UNSUPPORTED.
 *   N                           0..32. N == 0 or M == 0: nothing is launched.
 *   Y                           DEVICE, [N][M] int32, fully overwritten (K == 0 gives zeros).
 *   stream                      HIP stream (NULL = null stream).
 * Exact: int32 sums are associative and cannot overflow under the K bound,
 * so every kernel gives the same bits.
 */
int spmm_bitmap_w4a4(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                     int64_t payload_bytes, int64_t M, int64_t K,
                     const uint8_t *X, int64_t N, int32_t *Y, hipStream_t stream);

/* As spmm_bitmap_w4a4 with an explicit kernel choice (bsp_algo). */
int spmm_bitmap_w4a4_algo(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                          int64_t payload_bytes, int64_t M, int64_t K,
                          const uint8_t *X, int64_t N, int32_t *Y, int algo, hipStream_t stream);

/*
 * spmm_bitmap_f16 -- fp16 variant (SPDP Sec. 4: FP16 values in a bitmap
 * format, decoded with a masked-popcount rank): payload is uint16[nnz]
 * (payload_bytes >= 2*nnz, a multiple of BSP_PAYLOAD_ALIGN), X is fp16 [N][K],
 * Y is fp16 [N][M]. Products and
 * sums in fp32 (any order), one round-to-nearest-even to fp16 at the end.
 * Other arguments as spmm_bitmap_w4a4.
 */
int spmm_bitmap_f16(const uint64_t *bitmaps, const uint32_t *offsets, const uint16_t *payload,
                    int64_t payload_bytes, int64_t M, int64_t K,
                    const uint16_t *X, int64_t N, uint16_t *Y, hipStream_t stream);

int spmm_bitmap_f16_algo(const uint64_t *bitmaps, const uint32_t *offsets, const uint16_t *payload,
                         int64_t payload_bytes, int64_t M, int64_t K,
                         const uint16_t *X, int64_t N, uint16_t *Y, int algo, hipStream_t stream);

/*
 * Split-K with a workspace (UnionSparse Sec. VI-C, Alg. 2: each workgroup
 * stores its partial tile, a reduction adds them; the N:M co-design page,
 * Sec. 4.3, bounds the split count). The library allocates nothing; callers
 * that want the split plans pass a workspace:
 *
 *   bsp_workspace_bytes -- bytes of workspace the *_ws entry points want for
 *     a problem (their automatic plan and the forced BSP_ALGO_SPLITK plan),
 *     0 when no plan of the shape uses one. nnz may be -1 when unknown.
 *     Returns BSP_E_ARG / BSP_E_OVERFLOW for invalid shapes. Host only.
 *
 *   spmm_bitmap_w4a4_ws / spmm_bitmap_f16_ws -- as the *_algo entry points
 *     with a workspace: DEVICE memory, 256-byte aligned, workspace_bytes long,
 *     owned by the caller, ZERO-FILLED before its first use (its first 64 KiB
 *     hold arrival counters; every call leaves them at zero again, so one
 *     workspace serves calls of any shapes in turn). workspace may be NULL
 *     with workspace_bytes 0 (then no plan needs one). A plan that needs more
 *     than workspace_bytes returns BSP_E_CAPACITY and launches nothing; a
 *     workspace off a 256-byte boundary returns BSP_E_ARG. Calls that share a
 *     workspace must be ordered (one stream, or events): concurrent calls on
 *     one workspace race. fp16 results do not depend on timing (partials are
 *     added in a fixed order).
 */
int bsp_workspace_bytes(int dtype, int64_t M, int64_t K, int64_t N, int64_t nnz, int64_t *bytes);

int spmm_bitmap_w4a4_ws(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                        int64_t payload_bytes, int64_t M, int64_t K, const uint8_t *X, int64_t N, int32_t *Y,
                        void *workspace, int64_t workspace_bytes, int algo, hipStream_t stream);

int spmm_bitmap_f16_ws(const uint64_t *bitmaps, const uint32_t *offsets, const uint16_t *payload,
                       int64_t payload_bytes, int64_t M, int64_t K, const uint16_t *X, int64_t N, uint16_t *Y,
                       void *workspace, int64_t workspace_bytes, int algo, hipStream_t stream);

/*
 * spmm_bitmap_f16_noalloc -- for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): spmm_bitmap_f16_ws with the library's own scratch as the
 * workspace instead of a caller's. The scratch is a static device array of
 * bsp_noalloc_scratch_bytes() bytes (8 MiB), one per GPU, held until the
 * process ends; its device address is looked up on a device's first call
 * (which also clears it with a fill kernel on `stream`). No call allocates.
 * A plan that needs more scratch returns BSP_E_CAPACITY (a 4096-row fp16
 * problem needs at most 1 MiB; the need grows with M and N). Every call on a
 * GPU shares that GPU's scratch: calls that overlap on one GPU (different
 * streams without ordering) race, and must not be made. Other arguments,
 * results and errors as spmm_bitmap_f16_ws.
 */
int spmm_bitmap_f16_noalloc(const uint64_t *bitmaps, const uint32_t *offsets, const uint16_t *payload,
                            int64_t payload_bytes, int64_t M, int64_t K, const uint16_t *X, int64_t N,
                            uint16_t *Y, int algo, hipStream_t stream);

/* Size in bytes of the per-GPU scratch of spmm_bitmap_f16_noalloc. */
int64_t bsp_noalloc_scratch_bytes(void);

/*
 * bsp_select -- the kernel BSP_ALGO_AUTO picks for a problem (shape-aware
 * selection; UnionSparse Sec. I names it, without a rule). nnz may be -1 when
 * unknown. Returns a bsp_algo value, or -1 for invalid arguments. Host only.
 */
int bsp_select(int dtype, int64_t M, int64_t K, int64_t N, int64_t nnz);

/* Human-readable description of bsp_select's choice and launch shape (the
 * plain and *_algo entry points, no workspace), written NUL-terminated into
 * buf (at most n bytes). Returns bsp_status. Host only. */
int bsp_describe_selection(int dtype, int64_t M, int64_t K, int64_t N, int64_t nnz, char *buf, size_t n);

/* The same for the automatic plan of the *_ws entry points given a
 * workspace of bsp_workspace_bytes. */
int bsp_describe_selection_ws(int dtype, int64_t M, int64_t K, int64_t N, int64_t nnz, char *buf, size_t n);

/* The plan an explicit kernel choice takes: `algo` (a bsp_algo) through the
 * *_algo entry points (with_workspace 0) or the *_ws ones given a workspace
 * of bsp_workspace_bytes (with_workspace 1), described as above. Returns
 * BSP_E_UNSUPPORTED (and a description saying so) when that choice cannot
 * run the shape, BSP_E_ARG for an unknown dtype or algo. Host only. */
int bsp_describe_plan(int dtype, int64_t M, int64_t K, int64_t N, int64_t nnz, int algo, int with_workspace,
                      char *buf, size_t n);

/*
 * spmm_bitmap_w2a4 -- Y = W * X with W's values 2-bit (encoded with dtype
 * BSP_INT2: the W2A4 setting of UnionSparse Sec. VII, Fig. 11) and X packed
 * int4 as for spmm_bitmap_w4a4; Y int32 [N][M], exact. payload_bytes >=
 * ceil(nnz/4), a multiple of BSP_PAYLOAD_ALIGN. The automatic choice runs the
 * MFMA block kernels (streaming up to K = 4096, the ring kernel up to 16384;
 * X on a 4-byte boundary) and the plain kernel elsewhere; _algo forces
 * BSP_ALGO_MFMA (BSP_E_UNSUPPORTED outside it) or BSP_ALGO_ROWWAVE;
 * BSP_ALGO_SPLITK returns BSP_E_UNSUPPORTED. bsp_describe_selection and
 * bsp_describe_plan with dtype BSP_INT2 describe these plans.
 */
int spmm_bitmap_w2a4(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                     int64_t payload_bytes, int64_t M, int64_t K, const uint8_t *X, int64_t N,
                     int32_t *Y, hipStream_t stream);
int spmm_bitmap_w2a4_algo(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                          int64_t payload_bytes, int64_t M, int64_t K, const uint8_t *X, int64_t N,
                          int32_t *Y, int algo, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Dequant epilogue and grouped launch (the Quant -> SpMM -> Dequant pipeline
 * of UnionSparse Fig. 2, with the Dequant step fused into the SpMM's final
 * write, and several matrices in one launch).
 * With the epilogue, output element (n, m) is
 *     Yh[n*M + m] = fp16( fp32( fp32(y) * scale_w[m] ) * scale_x[n] )
 * y being the int32 sum of spmm_bitmap_w4a4: the sum converted to fp32
 * (round to nearest even), multiplied by the output channel's scale, then by
 * the token's scale, each product rounded to nearest even in fp32, and one
 * round to nearest even to fp16 (overflow gives +-inf). Scales are fp32, in
 * the normal range (no subnormal products).
 * --------------------------------------------------------------------------- */

/*
 * spmm_bitmap_w4a4_dq -- spmm_bitmap_w4a4 with the dequant epilogue.
 *   scale_w    DEVICE float[M], one scale per output row (channel).
 *   scale_x    DEVICE float[N], one scale per activation column (token).
 *   Yh         DEVICE uint16 [N][M] (fp16 bits), fully overwritten.
 * Runs the int4 MFMA kernels (K <= 16384, X on a 4-byte boundary); other
 * shapes return BSP_E_UNSUPPORTED. K == 0 gives fp16(0 * scale_w * scale_x)
 * (signed zeros). Other arguments as spmm_bitmap_w4a4.
 */
int spmm_bitmap_w4a4_dq(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                        int64_t payload_bytes, int64_t M, int64_t K, const uint8_t *X, int64_t N,
                        const float *scale_w, const float *scale_x, uint16_t *Yh, hipStream_t stream);

/* Most matrices in one grouped launch. */
#define BSP_GROUP_MAX 8

/* One matrix of a grouped launch: its BT64 stream, its X, and exactly one of
 * Y (int32 [N][M]) or Yh (fp16 [N][M] through the dequant epilogue, with
 * scale_w[M] and scale_x[N]). All pointers DEVICE; M, N, payload_bytes as for
 * spmm_bitmap_w4a4. An item with M == 0 or N == 0 is skipped. */
typedef struct bsp_w4a4_item {
    const uint64_t *bitmaps;
    const uint32_t *offsets;
    const uint8_t *payload;
    int64_t payload_bytes;
    int64_t M;
    const uint8_t *X;
    int64_t N;
    int32_t *Y;
    uint16_t *Yh;
    const float *scale_w;
    const float *scale_x;
} bsp_w4a4_item;

/*
 * spmm_bitmap_w4a4_grouped -- Y_i = W_i * X_i for `count` (1..BSP_GROUP_MAX)
 * matrices sharing one K (e.g. the Q, K and V projections of a layer, or an
 * FFN's gate and up projections) in ONE kernel launch on `stream`; the
 * workgroups are shared out over the items in proportion to their rows.
 *   items      HOST array of `count` descriptors (read during the call only).
 * Results equal spmm_bitmap_w4a4 / spmm_bitmap_w4a4_dq per item, bit for bit.
 * The items must all run the streaming int4 kernel (1 <= K <= 4096, X on a
 * 4-byte boundary), else BSP_E_UNSUPPORTED and nothing is launched. Errors
 * in any item are reported before anything is launched.
 */
int spmm_bitmap_w4a4_grouped(const bsp_w4a4_item *items, int count, int64_t K, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Union-mask format ("IE-BME"): UnionSparse Sec. V-A, Fig. 7, with 16 x 64
 * local tiles (LTs) and bitmap-aware row reordering (Sec. V-B, Eq. 3-5,
 * Algorithm 1).
 *   bands = ceil(M/16), T = ceil(K/64), nlt = bands*T LTs in row-major order
 *   (LT t = band*T + column covers rows 16*band .. +15, columns 64*column ..
 *   +63; past M or K the tile is padded with zeros).
 *   An LT is cut into ra x ca areas of (16/ra) x (64/ca); area q = a*ca + c
 *   holds tile rows a*16/ra .. and columns c*64/ca ... Logical position (i, j)
 *   of the (16/ra) x (64/ca) union mask is set iff any area has a nonzero at
 *   (i, j) (after the LT's row permutation).
 *   ubitmaps[t*W .. t*W+W-1]  uint64, W = 16/(ra*ca) words: the mask scanned
 *                row-major, position f in bit f%64 of word f/64 (leftmost
 *                position of a row in the lowest bit, as in Fig. 7).
 *   offsets[t]   uint32, number of values before LT t ("Union Value Offsets":
 *                the sum of Q*P over earlier LTs, Q = ra*ca, P = set mask
 *                bits); offsets[nlt] = nvals. nlt+1 entries.
 *   rowpos[t]    uint64, nibble r = position of tile row r in the LT's
 *                reordered row order (identity without reordering). The
 *                reordered tile lists, area row by area row, row p of every
 *                row group found by the reordering.
 *   payload      int4 values ("Compressed Values"): for each set position of
 *                rank rho (set positions before it, row-major), area q's value
 *                (zero or not) is element offsets[t] + q*P + rho. Element e is
 *                byte e>>1, low nibble when e is even. ceil(nvals/2) bytes.
 * Row reordering, per LT: rows are grouped into 16/ra groups of ra rows so
 * that the number of set mask positions is minimal (subset DP over row sets,
 * each step taking a group with the smallest remaining row); among equal
 * costs the first group in ascending lexicographic order is kept.
 * --------------------------------------------------------------------------- */
#define BSP_LT_ROWS 16
#define BSP_LT_COLS 64

/* Number of LTs of an M x K matrix (ceil(M/16)*ceil(K/64)); -1 for negative sizes. */
int64_t union_tile_count(int64_t M, int64_t K);

/* 64-bit mask words per LT for an ra x ca partition: 16/(ra*ca). 0 when the
 * partition is not supported (ra, ca powers of two with ra*ca <= 16). */
int union_mask_words(int ra, int ca);

/*
 * encode_union_tiles -- host-side encoder of the union-mask format.
 *   W          HOST int8 [M][ldw], values in [-8, 7] (BSP_E_RANGE otherwise).
 *   ra, ca     area partition (union_mask_words(ra, ca) > 0, else BSP_E_ARG).
 *   reorder    nonzero: bitmap-aware row reordering of every LT; 0: identity.
 *   ubitmaps, offsets, rowpos   HOST, caller-allocated: nlt*W, nlt+1 and nlt
 *              entries; all three NULL for a size query.
 *   payload    HOST, payload_capacity_bytes >= ceil(nvals/2), or NULL (size
 *              query, or words/offsets/rowpos only).
 *   nvals_out, payload_bytes_out  written on BSP_OK, BSP_E_CAPACITY and
 *              BSP_E_OVERFLOW (either may be NULL).
 * Returns BSP_E_OVERFLOW when nvals >= 2^32. Deterministic for a given input.
 */
int encode_union_tiles(const int8_t *W, int64_t M, int64_t K, int64_t ldw, int ra, int ca, int reorder,
                       uint64_t *ubitmaps, uint32_t *offsets, uint64_t *rowpos,
                       uint8_t *payload, int64_t payload_capacity_bytes,
                       int64_t *nvals_out, int64_t *payload_bytes_out);

/* K bound of the union-mask SpMM. */
#define BSP_UNION_MAX_K 32768

/*
 * spmm_union_w4a4 -- Y = W * X with W in the union-mask format (int4 values,
 * int32 Y), asynchronous on `stream`. All pointers are DEVICE memory.
 *   ubitmaps, offsets, rowpos, payload   as encode_union_tiles wrote them;
 *              payload_bytes is the payload allocation (a multiple of
 *              BSP_PAYLOAD_ALIGN, zero past the encoded bytes).
 *   ra, ca     the encoding's partition. The kernel runs ra = ca = 2 (the
 *              pages' 2 x 2 areas); another valid partition returns
 *              BSP_E_UNSUPPORTED, an invalid one BSP_E_ARG.
 *   M, K       0 <= M < 2^31, 0 <= K <= BSP_UNION_MAX_K (larger K: BSP_E_UNSUPPORTED).
 *   X          [N][ceil(K/2)] packed int4 as for spmm_bitmap_w4a4, on a 4-byte
 *              boundary (BSP_E_UNSUPPORTED otherwise).
 *   N          0..32; N == 0 or M == 0 launches nothing.
 *   Y          [N][M] int32, fully overwritten (K == 0 gives zeros).
 */
int spmm_union_w4a4(const uint64_t *ubitmaps, const uint32_t *offsets, const uint64_t *rowpos,
                    const uint8_t *payload, int64_t payload_bytes, int ra, int ca, int64_t M, int64_t K,
                    const uint8_t *X, int64_t N, int32_t *Y, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Tiled-CBC format and dynamic activation pruning (SPDP, Sec. 4.1 "Tiled-CBC",
 * Fig. 4(a); Sec. 4.2, the decode-phase spMspV kernel).
 *   GTiles of BSP_CBC_TILE_M x BSP_CBC_TILE_K (256 x 64) in row-major order
 *   over the matrix (n_gt = cbc_gtile_count(M, K); zero-padded past M and K).
 *   tile_offsets[g]   uint32, GTile g's first value; n_gt+1 entries, the last NNZ.
 *   colinfo[g*64 + c] uint32, (first value of column c inside the GTile << 16)
 *                     | (nonzeros of column c).
 *   bitmaps[(g*64 + c)*4 + w]  uint64: bit j is row 64w+j of column c.
 *   values            fp16 bits: GTile by GTile, column by column, rows ascending.
 * Storage: 4(n_gt+1) + 4 n_gt 64 + 8 (n_gt 64 4) + 2 NNZ bytes.
 * --------------------------------------------------------------------------- */
#define BSP_CBC_TILE_M 256
#define BSP_CBC_TILE_K 64
/* Largest N of spmspv_cbc_f16 (decode widths). */
#define BSP_CBC_MAX_N 8

/* GTiles of an M x K matrix; -1 for negative sizes. */
int64_t cbc_gtile_count(int64_t M, int64_t K);

/*
 * encode_cbc_f16 -- host-side Tiled-CBC encoder. W: HOST uint16 (fp16 bits)
 * [M][ldw]; +0 and -0 are zero. tile_offsets/colinfo/bitmaps: HOST arrays of
 * n_gt+1, n_gt*64 and n_gt*256 entries, all NULL for a size query; values:
 * HOST, values_capacity elements (>= NNZ), or NULL. nnz_out written on BSP_OK,
 * BSP_E_CAPACITY and BSP_E_OVERFLOW (NNZ >= 2^32).
 */
int encode_cbc_f16(const uint16_t *W, int64_t M, int64_t K, int64_t ldw, uint32_t *tile_offsets,
                   uint32_t *colinfo, uint64_t *bitmaps, uint16_t *values, int64_t values_capacity,
                   int64_t *nnz_out);

/* Workspace bytes spmspv_cbc_f16 uses to split K over workgroups (0: none). */
int spmspv_cbc_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t *bytes);

/*
 * spmspv_cbc_f16 -- Y = W * X' on `stream`, X' = X with every activation of
 * magnitude <= threshold set to zero (dynamic pruning); the columns of W
 * whose activations are all pruned are not read. fp32 products and sums, one
 * round to nearest even to fp16.
 *   tile_offsets, colinfo, bitmaps, values  DEVICE, as encode_cbc_f16 wrote
 *            them; values_bytes: the values allocation, a multiple of
 *            BSP_PAYLOAD_ALIGN, zero past the encoded values.
 *   X        DEVICE fp16 [N][K]; N 0..BSP_CBC_MAX_N.
 *   threshold  fp32, finite, >= 0 (0: the plain product); compared with |x| in fp32.
 *   Y        DEVICE fp16 [N][M], fully overwritten (K == 0 gives zeros).
 *   workspace  DEVICE, NULL (one workgroup per 256-row band) or
 *            spmspv_cbc_workspace_bytes() bytes, 256-byte aligned, zero-filled
 *            before its first use (its first 64 KiB are arrival counters,
 *            left zero by every call); calls that share a workspace must be
 *            ordered on one stream. Too small: BSP_E_CAPACITY.
 */
int spmspv_cbc_f16(const uint32_t *tile_offsets, const uint32_t *colinfo, const uint64_t *bitmaps,
                   const uint16_t *values, int64_t values_bytes, int64_t M, int64_t K, const uint16_t *X,
                   int64_t N, float threshold, uint16_t *Y, void *workspace, int64_t workspace_bytes,
                   hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Paged key/value cache, quantised as it is written.
 *   A cache holds the K and V rows (one per token and kv head, head_dim
 *   channels) of many sequences in pages of page_size token slots. Slot
 *   page * page_size + offset is token `offset` of page `page`; which pages a
 *   sequence owns is the caller's block table.
 *   k, v         [num_pages][kv_heads][page_size][row], a row being head_dim fp16
 *                values (BSP_FP16), head_dim code bytes (BSP_INT8) or head_dim / 2
 *                bytes (BSP_INT4: two codes per byte, low nibble = even channel).
 *   k_scale, v_scale   uint32 [num_pages][kv_heads][page_size], one word per
 *                row: the step s as bfloat16 in the high half, the offset o as
 *                fp16 in the low half (NULL for BSP_FP16). The row stands for
 *                s * u + o, u its unsigned codes (0..255 or 0..15).
 *   Quantising a row x (fp16, as given):
 *                o = min x;  s = fp32((max x - o) / L) rounded up to bfloat16,
 *                L = 255 or 15;  u = round-half-even((x - o) / s), at most L
 *                (u = 0 where s = 0; x - o and the quotient as fp32). A row holding
 *                an infinity or a NaN gets s = o = NaN and codes 0: it reads back as NaN.
 *   s is rounded up so that L steps reach the maximum; the error of a value is
 *   at most s / 2, plus its rounding to fp16 where it is read back.
 * --------------------------------------------------------------------------- */
typedef struct bsp_kv_cache {
    int dtype;              /* BSP_FP16, BSP_INT8 or BSP_INT4 */
    int64_t num_pages;      /* num_pages * page_size < 2^31 */
    int64_t kv_heads;
    int64_t page_size;      /* a power of two, 16 .. 4096 */
    int64_t head_dim;       /* 64, 128 or 256 (BSP_E_UNSUPPORTED otherwise) */
    void *k, *v;            /* DEVICE, 16-byte aligned */
    uint32_t *k_scale, *v_scale;   /* DEVICE, 16-byte aligned; NULL for BSP_FP16 */
} bsp_kv_cache;

/*
 * kv_cache_append -- quantise n tokens' K and V rows into their slots, on `stream`.
 *   cache     HOST descriptor (read during the call only).
 *   K, V      DEVICE fp16 [n][kv_heads][head_dim], token t starting at element
 *             t * k_stride (v_stride): a slice of a fused QKV projection's
 *             output will do. Strides >= kv_heads * head_dim.
 *   slots     DEVICE int64 [n]. A slot outside [0, num_pages * page_size) is
 *             skipped; two tokens of one call must not share a slot.
 * n == 0 or kv_heads == 0 launches nothing; n * kv_heads >= 2^28 is refused
 * (BSP_E_OVERFLOW), here and in kv_cache_gather.
 */
int kv_cache_append(const bsp_kv_cache *cache, const uint16_t *K, int64_t k_stride, const uint16_t *V,
                    int64_t v_stride, const int64_t *slots, int64_t n, hipStream_t stream);

/*
 * kv_cache_gather -- the K and V rows of n slots as fp16 (the sum s * u + o in
 * fp32, at most 65504, one round to nearest even), [n][kv_heads][head_dim] with token strides
 * as above. A slot outside the cache gives zeros. The same slot may repeat.
 */
int kv_cache_gather(const bsp_kv_cache *cache, const int64_t *slots, int64_t n, uint16_t *K, int64_t k_stride,
                    uint16_t *V, int64_t v_stride, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of drafted token trees over the paged cache (decode: one token per
 * sequence is a tree of one).
 *   Sequence b has kv_lens[b] tokens in the cache, the last T_b of them this
 *   step's drafted tokens (appended before the call); their queries are rows
 *   q_start[b] .. q_start[b+1]-1 of Q, T_b = q_start[b+1] - q_start[b].
 *   Drafted token i sees every token before the drafted ones, and drafted token
 *   j iff bit j of tree_mask[q_start[b] + i] is set (its ancestors and itself);
 *   without a mask, j <= i (a chain).
 *   O[row][h] = sum_j softmax_j(scale * Q[row][h] . k_j) v_j over the visible
 *   tokens j, k_j and v_j the rows of kv head h / (q_heads / kv_heads) as the
 *   cache stands for them. A row that sees no token gives zeros. What lies in
 *   the cache at tokens a row does not see, NaN included, has no effect on it.
 *   An infinity or a NaN in a v row that a row sees makes that channel of its
 *   output infinite or NaN (a quantised row that held one stands for NaN in
 *   every channel), one in a k row the score of that token.
 * Scores, softmax statistics and sums are fp32, the exponentials (times the
 * value row's step, where it is quantised) enter the second product as fp16
 * (their scale chosen so that they stay normal numbers down to 2^-20 of the
 * largest the row sees), one rounding to fp16 at the end. Partial sums
 * are joined in a fixed order: results do not depend on timing.
 * --------------------------------------------------------------------------- */

/* Most drafted tokens of a sequence in one call (bits of a mask word). */
#define BSP_TREE_MAX 64

/*
 * attention_tree_workspace_bytes -- bytes of workspace attention_tree_f16 uses
 * to split the cached tokens over workgroups; table_width as in the call. Host
 * only. 0 when B, max_q, q_heads or kv_heads is 0.
 */
int attention_tree_workspace_bytes(const bsp_kv_cache *cache, int64_t table_width, int64_t B, int64_t max_q,
                                   int64_t q_heads, int64_t *bytes);

/*
 * attention_tree_f16 -- the attention above, asynchronous on `stream`.
 *   Q            DEVICE fp16, token row r at element r * q_stride, [q_heads][head_dim] there.
 *   cache        HOST descriptor (read during the call only).
 *   block_table  DEVICE int32 [B][table_width]: page of tokens p * page_size ...
 *                of sequence b at [b][p]. Entries outside the cache are read as page 0.
 *                table_width * page_size is below 2^31 - 4096 (BSP_E_OVERFLOW past that).
 *   kv_lens      DEVICE int32 [B], at most table_width * page_size (clamped to it).
 *   q_start      DEVICE int32 [B+1], non-decreasing, q_start[B] <= total_q. Rows
 *                of Q no sequence owns leave O as it is.
 *   max_q        most drafted tokens of a sequence, 0..BSP_TREE_MAX; rows past it are
 *                not computed.
 *   tree_mask    DEVICE uint64 [total_q], or NULL for chains.
 *   q_heads      a multiple of kv_heads, at most 16384 of them per kv head
 *                (BSP_E_UNSUPPORTED past that).
 *   scale        finite.
 *   O            DEVICE fp16, token row r at element r * o_stride. Must not overlap Q.
 *   workspace    DEVICE, NULL (one workgroup walks all of a sequence) or
 *                attention_tree_workspace_bytes() bytes, 256-byte aligned, zero-filled
 *                before its first use (its first 64 KiB hold arrival counters, left zero by
 *                every call: a workspace of the other entry points will do). Too
 *                small: BSP_E_CAPACITY. Calls that share one must be ordered.
 */
int attention_tree_f16(const uint16_t *Q, int64_t q_stride, const bsp_kv_cache *cache, const int32_t *block_table,
                       int64_t table_width, const int32_t *kv_lens, const int32_t *q_start, int64_t B,
                       int64_t total_q, int64_t max_q, int64_t q_heads, const uint64_t *tree_mask, float scale,
                       uint16_t *O, int64_t o_stride, void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside one shared sparse projection:
 *   Y[n] = W x_n + scale[a] * B_a (A_a x_n),  a = index[n]   (a < 0: W x_n alone)
 * with A_a [rank][K] and B_a [M][rank] fp16. A_a x_n is summed and kept in
 * fp32, W x_n and the adapter's part meet in fp32, one rounding to fp16 at the end.
 * --------------------------------------------------------------------------- */
typedef struct bsp_lora {
    int64_t adapters;       /* adapters held; an index at or past it counts as -1 */
    int64_t rank;           /* the storage rank R: a multiple of 8, 8..256 */
    const uint16_t *A;      /* DEVICE fp16 [adapters][R][K], 16-byte aligned */
    const uint16_t *B;      /* DEVICE fp16 [adapters][M][R], 16-byte aligned */
    const float *scale;     /* DEVICE [adapters], or NULL for 1 */
    const int32_t *ranks;   /* DEVICE [adapters], the rows of A_a in use (0..R, clamped), or
                               NULL for R; what lies past them is not used */
    const int32_t *index;   /* DEVICE [N], the adapter of each token */
} bsp_lora;

/*
 * lora_workspace_bytes -- bytes of workspace the calls below need for an M x K
 * product of N tokens and storage rank R; dtype BSP_FP16 or BSP_INT4. Host only.
 */
int lora_workspace_bytes(int dtype, int64_t M, int64_t K, int64_t N, int64_t nnz, int64_t rank, int64_t *bytes);

/*
 * spmm_bitmap_f16_lora -- spmm_bitmap_f16_ws with adapters. The workspace is
 * required (256-byte aligned, zero-filled before its first use, as for the _ws entry
 * points, and of lora_workspace_bytes); BSP_E_CAPACITY when it is too small.
 */
int spmm_bitmap_f16_lora(const uint64_t *bitmaps, const uint32_t *offsets, const uint16_t *payload,
                         int64_t payload_bytes, int64_t M, int64_t K, const uint16_t *X, int64_t N,
                         const bsp_lora *lora, uint16_t *Y, void *workspace, int64_t workspace_bytes,
                         hipStream_t stream);

/*
 * spmm_bitmap_w4a4_dq_lora -- spmm_bitmap_w4a4_dq with adapters: W x_n is the
 * dequantised int4 product (packed X, scale_w, scale_x); the adapters take the
 * fp16 activations X16 [N][K] the packed ones came from. Yh = fp16(fp32(y) *
 * scale_w[m] * scale_x[n] + the adapter's part), in fp32. Any K
 * spmm_bitmap_w4a4 takes; the workspace as for spmm_bitmap_f16_lora.
 */
int spmm_bitmap_w4a4_dq_lora(const uint64_t *bitmaps, const uint32_t *offsets, const uint8_t *payload,
                             int64_t payload_bytes, int64_t M, int64_t K, const uint8_t *X, const uint16_t *X16,
                             int64_t N, const float *scale_w, const float *scale_x, const bsp_lora *lora,
                             uint16_t *Yh, void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Block tables, slots and positions of a step, made on the GPU.
 *   The pages of a cache are handed to sequences from a list of free ones. All
 *   of it is device memory that a step reads and updates in place, so a captured
 *   step needs nothing from the host.
 *   block_table  int32 [sequences][table_width], as attention_tree_f16 takes it;
 *                entries past a sequence's held pages mean nothing.
 *   lens         int32 [sequences], tokens a sequence has in the cache.
 *   held         int32 [sequences], pages it holds: entries 0 .. held-1 of its row
 *                (ceil(lens / page_size), or more after it had to wait).
 *   free_pages   int32 [2 + pool]: the number of free pages, a counter of the call's
 *                own (zero before its first use, left zero), then the pages,
 *                the next to be taken last.
 * Values that cannot be (lens past the table, a count past the pool, ...) are
 * taken as the nearest that can: nothing outside the arrays is touched.
 * --------------------------------------------------------------------------- */
typedef struct bsp_kv_pages {
    int64_t sequences;      /* 0 .. BSP_PAGES_MAX_SEQUENCES */
    int64_t table_width;    /* sequences * table_width + pool < 2^31 */
    int64_t page_size;      /* a power of two, 16 .. 4096; table_width * page_size < 2^31 - 4096 */
    int64_t pool;           /* pages the list can hold */
    int32_t *block_table, *lens, *held, *free_pages;   /* DEVICE */
} bsp_kv_pages;

#define BSP_PAGES_MAX_SEQUENCES 4096

/*
 * kv_pages_step -- one step of all sequences, asynchronous on `stream`: sequence
 * b keeps the first keep[b] of its tokens (a rejected draft goes, a finished
 * request keeps none) and appends new_tokens[b].
 *   keep, new_tokens  DEVICE int32 [sequences]; keep NULL: all kept. Clamped to
 *                0 .. lens[b], and to 0 from below.
 *   tree_mask    DEVICE uint64 [rows], or NULL: attention_tree_f16's words.
 *   rows         rows of the step's token arrays (0 .. 2^28 - 1), sequence b's from q_start[b].
 *   slots        DEVICE int64 [rows]: the slot of each new token, for kv_cache_append.
 *   positions    DEVICE int32 [rows]: keep + i for the i-th new token; with tree_mask,
 *                in sequences of at most BSP_TREE_MAX new tokens, keep + the number of
 *                bits below i in its word (its ancestors).
 *   sequences    DEVICE int32 [rows]: the sequence of each row.
 *   q_start      DEVICE int32 [sequences + 1]: new tokens before each sequence, at most rows.
 *   kv_lens      DEVICE int32 [sequences]: the new length, what attention takes.
 * Rows behind the last sequence get slot -1, position 0 and sequence -1. A
 * sequence then needs ceil(length / page_size) pages. Pages given back are numbered
 * in order of sequence and place, pages taken likewise: the n-th taken is the n-th
 * given back, past those the list's last, last but one, ...; what was given back and
 * not taken is put onto the list's end, the first given back last (so that a step and
 * the one that undoes it restore every entry).
 * A sequence waits when its rows pass `rows`, its pages pass table_width, or it
 * takes pages and the pages taken up to it are more than there are (then so do the
 * later ones that take pages): it keeps its pages and its kept tokens, appends none,
 * gets slots -1 and kv_lens 0 (attention then gives zeros for its rows).
 * Calls on the same pages must be ordered on one stream. An output that overlaps an
 * input, the pages' arrays or another output is refused (BSP_E_ARG); keep may be lens.
 */
int kv_pages_step(const bsp_kv_pages *pages, const int32_t *keep, const int32_t *new_tokens,
                  const uint64_t *tree_mask, int64_t rows, int64_t *slots, int32_t *positions, int32_t *sequences,
                  int32_t *q_start, int32_t *kv_lens, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Queries and keys normed head by head and rotated to their positions.
 *   y = x / sqrt(mean(x^2) + eps) * weight over a head's channels (no weight: y = x);
 *   then pairs (y1, y2) of its first `rot` channels become
 *   (y1 cos a - y2 sin a, y2 cos a + y1 sin a), pair i at the angle of position
 *   p: a = p * freq[i] turns. Pair i is channels (i, i + rot / 2), or (2 i, 2 i + 1)
 *   where interleaved. fp32 throughout, one rounding to fp16 at the end.
 *   freq holds turns per position as fractions of 2^64, so that p * freq[i] mod
 *   2^64 is the angle mod one turn without a rounding, however far the position.
 * --------------------------------------------------------------------------- */
typedef struct bsp_rotation {
    int64_t rot;                 /* rotated channels: a multiple of 16, 0 .. head_dim (BSP_E_UNSUPPORTED otherwise) */
    int interleaved;             /* 0: pairs (i, i + rot / 2); 1: pairs (2 i, 2 i + 1) */
    const uint64_t *freq;        /* DEVICE [rot / 2] */
    const int32_t *positions;    /* DEVICE [n] */
    const uint16_t *q_weight;    /* DEVICE fp16 [head_dim], 16-byte aligned, or NULL: queries not normed */
    const uint16_t *k_weight;    /* the same for keys */
    float eps;                   /* finite, >= 0 */
} bsp_rotation;

/*
 * qk_norm_rope_f16 -- n tokens' query and key heads, asynchronous on `stream`.
 *   Q, K         DEVICE fp16 [n][q_heads][head_dim], [n][kv_heads][head_dim], token t at
 *                element t * stride (a slice of a fused projection's output will do).
 *   Qo, Ko       the results, with strides of their own; may be Q, K with their strides,
 *                and must not overlap the inputs otherwise.
 *   head_dim     64, 128 or 256 (BSP_E_UNSUPPORTED otherwise).
 * n * (q_heads + 2 kv_heads) >= 2^28 and more than 2^20 heads are refused (BSP_E_OVERFLOW),
 * here and below.
 */
int qk_norm_rope_f16(const uint16_t *Q, int64_t q_stride, const uint16_t *K, int64_t k_stride, int64_t n,
                     int64_t q_heads, int64_t kv_heads, int64_t head_dim, const bsp_rotation *rotation, uint16_t *Qo,
                     int64_t qo_stride, uint16_t *Ko, int64_t ko_stride, hipStream_t stream);

/*
 * qk_norm_rope_append_f16 -- the same, with the keys (rounded to fp16) and the
 * values V written to the cache's slots: bit for bit what qk_norm_rope_f16 and
 * kv_cache_append leave there, in one pass. slots as for kv_cache_append. Without kv heads (here and above) the queries
 * alone are worked on, and what belongs to keys and values may be NULL, slots among it.
 */
int qk_norm_rope_append_f16(const uint16_t *Q, int64_t q_stride, const uint16_t *K, int64_t k_stride,
                            const uint16_t *V, int64_t v_stride, int64_t n, int64_t q_heads,
                            const bsp_rotation *rotation, const bsp_kv_cache *cache, const int64_t *slots,
                            uint16_t *Qo, int64_t qo_stride, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Hidden states quantised token by token, with the residual sum and the norm
 * before it, for spmm_bitmap_w4a4_dq (packed int4) and gemm_w8a8_dq (int8).
 *   h = fp16(x + residual) (or x), y = h * weight (or h), m = max_k |y_k|, L = 127 or 7
 *   code_k = round-half-even(y_k * L / m), of the exact quotient (0 where m = 0)
 *   scale  = m / sqrt(mean(h^2) + eps) / L with a weight, m / L without, fp32
 *   x16    = fp16(y / sqrt(mean(h^2) + eps)) with a weight, h without: what the codes stand
 *            for, unquantised (the adapters' activations)
 *   A token with an infinity or a NaN in y gets codes 0 and scale NaN.
 * --------------------------------------------------------------------------- */
typedef struct bsp_tokens {
    int64_t n, K;                /* n * K < 2^40, K < 2^25 */
    const uint16_t *X;           /* DEVICE fp16 [n][K], token t at element t * x_stride */
    int64_t x_stride;
    const uint16_t *residual;    /* DEVICE fp16, or NULL */
    int64_t residual_stride;
    const uint16_t *weight;      /* DEVICE fp16 [K], or NULL: no norm */
    float eps;                   /* finite, >= 0 */
    uint16_t *hidden;            /* DEVICE fp16, h; required with a residual (may be X or residual, with its
                                    stride), NULL without */
    int64_t hidden_stride;
    uint16_t *x16;               /* DEVICE fp16, or NULL */
    int64_t x16_stride;
    float *scale;                /* DEVICE [n] */
} bsp_tokens;

/*
 * quantize_tokens_f16 -- asynchronous on `stream`.
 *   tokens       HOST descriptor (read during the call only).
 *   dtype        BSP_INT8: codes int8, token t at byte t * code_stride; BSP_INT4: packed as
 *                pack_int4_activations does (an odd K leaves the last high nibble zero).
 *   codes        DEVICE; code_stride >= K (int8) or ceil(K / 2) (int4). What lies between a token's
 *                codes and the next token's is left as it is.
 * n == 0 or K == 0 launches nothing (and writes no scales). No output may overlap an input but hidden, as above, nor
 * another output.
 */
int quantize_tokens_f16(const bsp_tokens *tokens, int dtype, uint8_t *codes, int64_t code_stride, hipStream_t stream);

/*
 * dequantize_tokens_f16 -- the values the codes stand for, fp16(scale[t] * code), into
 * X fp16 [n][K] with token stride x_stride.
 */
int dequantize_tokens_f16(const uint8_t *codes, int64_t code_stride, int dtype, const float *scale, int64_t n,
                          int64_t K, uint16_t *X, int64_t x_stride, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Dense 8-bit product, for layers left unpruned and for prompts (any N):
 *   Y[n][m] = fp16(fp32(sum_k W[m][k] X[n][k]) * scale_w[m] * scale_x[n])
 * with int32 sums (exact: K <= BSP_W8_MAX_K). W is laid out once on the host in
 * the order the matrix instruction takes it: tiles of 16 rows x 64 columns, row band
 * by row band, 1 KiB each, 16-byte piece l of a tile holding row l % 16, columns
 * 16 (l / 16) ..; zeros past M and K.
 * --------------------------------------------------------------------------- */
#define BSP_W8_MAX_K 131071

/* Bytes of the laid-out form: ceil(M/16) * ceil(K/64) * 1024; -1 for sizes that encode_int8_tiles refuses. */
int64_t int8_tiles_bytes(int64_t M, int64_t K);

/*
 * encode_int8_tiles -- W HOST int8 [M][ldw] -> tiles HOST (int8_tiles_bytes bytes). K > BSP_W8_MAX_K, M >= 2^31:
 * BSP_E_OVERFLOW.
 */
int encode_int8_tiles(const int8_t *W, int64_t M, int64_t K, int64_t ldw, uint8_t *tiles);

/* Bytes of workspace gemm_w8a8_dq uses to split K over workgroups, for any number of tokens up to N (0: none). Host
 * only. */
int gemm_w8a8_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t *bytes);

/* The kernel, its tile (channels x tokens) and over how many workgroups K is split, as gemm_w8a8_dq chooses them
 * without a workspace (0) or with one of gemm_w8a8_workspace_bytes() (1), written NUL-terminated into buf (at most n bytes).
 * Host only. */
int gemm_w8a8_describe(int64_t M, int64_t K, int64_t N, int with_workspace, char *buf, size_t n);

/*
 * gemm_w8a8_dq -- asynchronous on `stream`.
 *   tiles        DEVICE, 16-byte aligned, as encode_int8_tiles wrote them.
 *   X            DEVICE int8, token n at byte n * x_stride, 16-byte aligned; x_stride a multiple of
 *                16, >= K. All N * x_stride bytes are readable; what lies past K is not used.
 *   scale_w, scale_x   DEVICE fp32 [M], [N].
 *   Y            DEVICE fp16 [N][M], row n at element n * y_stride >= M. Must not overlap X.
 *   workspace    DEVICE, NULL (K not split over workgroups) or gemm_w8a8_workspace_bytes()
 *                bytes, 256-byte aligned, zero-filled before its first use (its first 64 KiB hold
 *                arrival counters, left zero by every call: a workspace of the other entry points
 *                will do). Too small: BSP_E_CAPACITY. Calls that share one must be ordered.
 * K > BSP_W8_MAX_K, M > 2^26 - 128, N >= 2^31, x_stride >= 2^23: BSP_E_OVERFLOW. K == 0 gives zeros. The result does not
 * depend on timing or on the workspace.
 */
int gemm_w8a8_dq(const uint8_t *tiles, int64_t M, int64_t K, const int8_t *X, int64_t x_stride, int64_t N,
                 const float *scale_w, const float *scale_x, uint16_t *Y, int64_t y_stride, void *workspace,
                 int64_t workspace_bytes, hipStream_t stream);

/* Static string for a bsp_status code. */
const char *bsp_status_string(int status);

/* Library version as "major.minor.patch". */
const char *bsp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BITMAP_SPMM_H */
