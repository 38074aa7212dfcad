// kernels_lora.hip -- low-rank adapters of many requests beside a shared
// sparse projection: Y[n] = W x_n + scale[a] B_a (A_a x_n), a = index[n].
//
// Two small products around the sparse one: t_n = scale[a] A_a x_n (rank
// values per token, fp32, through the workspace) ahead of it, and B_a t_n in
// the final write, where W x_n is still an fp32 (or int32) sum: one rounding.

struct LoraArgs {
    const uint16_t *A, *B;
    const float *scale;
    const int32_t *ranks, *index;
    float *t;          // [N][R]
    int adapters, R;
};

// What a kernel adds to its sum for output (n, m) before rounding it. The
// plain entry points add nothing.
struct NoAdd {
    template <int ROWS, int PIECES>
    struct Item {};
    template <class I>
    __device__ __forceinline__ void open(I &, int, bool) const {}
    template <class I>
    __device__ __forceinline__ void opened(I &) const {}
    template <class I>
    __device__ __forceinline__ void fetch(I &, int, int) const {}
    template <class I>
    __device__ __forceinline__ void reduce(I &) const {}
    template <class I>
    __device__ __forceinline__ float close(I &, float s, int, int) const { return s; }
    __device__ __forceinline__ float to(float s, int, int, int) const { return s; }
};

// The adapter of token n (-1: none) and its rank.
__device__ __forceinline__ int lora_of(const LoraArgs &a, int n, int *rank) {
    const int i = a.index[n];
    if (i < 0 || i >= a.adapters) {
        *rank = 0;
        return -1;
    }
    *rank = a.ranks != nullptr ? min(max(a.ranks[i], 0), a.R) : a.R;
    return i;
}

typedef _Float16 lora_h8 __attribute__((ext_vector_type(8)));
typedef float lora_f4 __attribute__((ext_vector_type(4)));

// s[k] + B_a[m + k] t_n, 8 rank positions a load; what lies past the rank (any
// bits of B, and t read again where a piece repeats) is left out. Index, rank and rows are loads one after the other
// that the tail of a sparse kernel has too few wavefronts to hide. Where
// registers allow it (N <= 8, and int4) a thread's first item is therefore taken
// in steps beside the kernel's own: its index with the first loads (open), its
// rank and first PIECES positions behind the last payload (fetch), their sum when
// that payload has landed (reduce), the rest in the final write (close): fp16
// 4096 x 4096, N = 1, rank 8 11.3 us against 11.9, int4 12288 x 4096, N = 8, rank
// 16 12.9 against 13.2. (The 1024-thread kernels have 128 registers and spill it:
// fp16 N = 32 29.9 against 24.7. They take all of it at the end, where the one for
// two column blocks still spills 22 registers, with its plain form at 126.)
struct LoraAdd {
    LoraArgs a;

    template <int ROWS, int PIECES>
    struct Item {
        int n, i, rank;
        lora_h8 b[PIECES][ROWS];
        lora_f4 v[PIECES][2];
        float u[ROWS];
    };

    template <int ROWS, int PIECES>
    __device__ __forceinline__ void open(Item<ROWS, PIECES> &e, int n, bool in) const {
        e.n = n, e.i = in ? a.index[n] : -1, e.rank = 0;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) e.u[k] = 0.f;
    }
    // The index is there (waited for here, ahead of the payload, not behind it).
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void opened(Item<ROWS, PIECES> &e) const {
        asm volatile("" : "+v"(e.i));
    }
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void piece(Item<ROWS, PIECES> &e, int p, int r, int m, int M) const {
        const float *t = a.t + (int64_t)e.n * a.R + r;
        const uint16_t *row = a.B + ((int64_t)e.i * M + m) * a.R + r;
        e.v[p][0] = *reinterpret_cast<const lora_f4 *>(t);
        e.v[p][1] = *reinterpret_cast<const lora_f4 *>(t + 4);
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
            e.b[p][k] = *reinterpret_cast<const lora_h8 *>(row + (int64_t)(m + k < M ? k : 0) * a.R);
    }
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void sum(Item<ROWS, PIECES> &e, int r0) const {
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = r0 + 8 * p + j < e.rank;
#pragma unroll
                for (int k = 0; k < ROWS; ++k) {
                    const float u = fmaf((float)e.b[p][k][j], e.v[p][j >> 2][j & 3], e.u[k]);
                    e.u[k] = in ? u : e.u[k];
                }
            }
    }
    // (the first positions are there whatever the rank: R is at least 8; past R the first again)
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void fetch(Item<ROWS, PIECES> &e, int m, int M) const {
        if ((unsigned)e.i >= (unsigned)a.adapters) {
            e.i = -1;
            return;
        }
        e.rank = a.ranks != nullptr ? a.ranks[e.i] : a.R;
#pragma unroll
        for (int p = 0; p < PIECES; ++p) piece(e, p, 8 * p < a.R ? 8 * p : 0, m, M);
    }
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void reduce(Item<ROWS, PIECES> &e) const {
        if (e.i < 0) return;
        e.rank = min(max(e.rank, 0), a.R);
        sum(e, 0);
    }
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void close(Item<ROWS, PIECES> &e, float (&s)[ROWS], int m, int M) const {
        if (e.i < 0) return;
        constexpr int MORE = ROWS == 1 ? 4 : 2;            // positions' pieces per turn: all their loads before the first use
        Item<ROWS, MORE> f;
        f.n = e.n, f.i = e.i, f.rank = e.rank;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) f.u[k] = e.u[k];
        for (int r0 = 8 * PIECES; r0 < f.rank; r0 += 8 * MORE) {
#pragma unroll
            for (int p = 0; p < MORE; ++p) piece(f, p, r0 + 8 * p < f.rank ? r0 + 8 * p : r0, m, M);
            sum(f, r0);
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) s[k] += f.u[k];
    }
    template <int PIECES>
    __device__ __forceinline__ float close(Item<1, PIECES> &e, float s, int m, int M) const {
        float v[1] = {s};
        close(e, v, m, M);
        return v[0];
    }

    // The whole of it at once (a thread's further items).
    template <int ROWS, int PIECES>
    __device__ __forceinline__ void rows(float (&s)[ROWS], int n, int m, int M) const {
        Item<ROWS, PIECES> e;
        open(e, n, true);
        fetch(e, m, M);
        reduce(e);
        close(e, s, m, M);
    }
    __device__ __forceinline__ float to(float s, int n, int m, int M) const {
        float v[1] = {s};
        rows<1, 4>(v, n, m, M);
        return v[0];
    }
};

// t[n][r]: one workgroup per (r, n); its wavefronts take pieces of 512
// channels in turn, so that a row of 4096 is two 16-byte loads a lane, all in
// flight at once. Rows past the rank and tokens without an adapter give zero.
// VEC: the rows of A and X lie on 16-byte boundaries (else element by element).
// Bound by latency (index, rank, row, sum): K = 4096, one token of rank 8 3.2 us,
// 32 tokens of ranks 1 to 64 (8 MB of A) 4.3; reading rows before the rank is
// known, or 8 wavefronts a row, gains 0.1 us for the one and loses 0.5 to 1 for
// the other.
#define LORA_WAVES 4

template <bool VEC>
__global__ __launch_bounds__(64 * LORA_WAVES) void k_lora_down(const LoraArgs a, const uint16_t *__restrict__ X, int K) {
    const int r = blockIdx.x, n = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ float part[LORA_WAVES];
    int rank;
    const int i = lora_of(a, n, &rank);
    const float scale = i >= 0 && a.scale != nullptr ? a.scale[i] : 1.f;
    float s = 0.f;
    if (r < rank) {
        const uint16_t *row = a.A + ((int64_t)i * a.R + r) * K, *x = X + (int64_t)n * K;
        if constexpr (VEC) {
#pragma unroll 4
            for (int k = threadIdx.x * 8; k < K; k += 64 * LORA_WAVES * 8) {
                const lora_h8 u = *reinterpret_cast<const lora_h8 *>(row + k);
                const lora_h8 v = *reinterpret_cast<const lora_h8 *>(x + k);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf((float)u[j], (float)v[j], s);
            }
        } else {
            for (int k = threadIdx.x; k < K; k += 64 * LORA_WAVES) s = fmaf(bsp_h2f(row[k]), bsp_h2f(x[k]), s);
        }
        s = bsp_wave_sum(s);
    }
    if (lane == 0) part[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = part[0];
#pragma unroll
        for (int w = 1; w < LORA_WAVES; ++w) s += part[w];
        a.t[(int64_t)n * a.R + r] = r < rank ? s * scale : 0.f;
    }
}

// The dequantised int32 sums with the adapters' part, rounded once (for every
// int4 plan but the streaming one: K past 4096, more than three 16-row blocks per
// workgroup, an X off a 4-byte boundary; 16384 x 2048, N = 8, rank 16 14.5 us for
// its three kernels).
__global__ __launch_bounds__(256) void k_lora_dq(const LoraAdd add, const int32_t *__restrict__ Y32, int M,
                                                 const float *__restrict__ sw, const float *__restrict__ sx,
                                                 uint16_t *__restrict__ Yh) {
    const int m = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
    if (m >= M) return;
    const int64_t at = (int64_t)n * M + m;
    Yh[at] = bsp_f2h(add.to((float)Y32[at] * sw[m] * sx[n], n, m, M));
}
