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

// s[i] + B_a[m + i] t_n, 8 rank positions a load; what lies past the rank (any
// bits) is replaced by zero. The loads of PIECES positions are issued before
// the first is used: the tail of the sparse kernels has too few wavefronts to
// hide one load after the other.
struct LoraAdd {
    LoraArgs a;

    template <int ROWS, int PIECES>
    __device__ __forceinline__ void rows(float (&s)[ROWS], int n, int m, int M) const {
        int rank;
        const int i = lora_of(a, n, &rank);
        if (i < 0) return;
        const uint16_t *row = a.B + ((int64_t)i * M + m) * a.R;
        const float *t = a.t + (int64_t)n * a.R;
        float u[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) u[k] = 0.f;
        for (int r0 = 0; r0 < rank; r0 += 8 * PIECES) {
            lora_h8 b[PIECES][ROWS];
            lora_f4 v[PIECES][2];
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                // (past the rank: the piece at r0 again)
                const int r = r0 + 8 * p < rank ? r0 + 8 * p : r0;
                v[p][0] = *reinterpret_cast<const lora_f4 *>(t + r);
                v[p][1] = *reinterpret_cast<const lora_f4 *>(t + r + 4);
#pragma unroll
                for (int k = 0; k < ROWS; ++k)
                    b[p][k] = *reinterpret_cast<const lora_h8 *>(row + (int64_t)(m + k < M ? k : 0) * a.R + r);
            }
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool in = r0 + 8 * p + j < rank;
#pragma unroll
                    for (int k = 0; k < ROWS; ++k) u[k] = fmaf(in ? (float)b[p][k][j] : 0.f, v[p][j >> 2][j & 3], u[k]);
                }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) s[k] += u[k];
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
#define LORA_WAVES 4

template <bool VEC>
__global__ __launch_bounds__(64 * LORA_WAVES) void k_lora_down(const LoraArgs a, const uint16_t *__restrict__ X, int K) {
    const int r = blockIdx.x, n = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ float part[LORA_WAVES];
    int rank;
    const int i = lora_of(a, n, &rank);
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
        if (r < rank && a.scale != nullptr) s *= a.scale[i];
        a.t[(int64_t)n * a.R + r] = s;
    }
}

// The dequantised int32 sums with the adapters' part, rounded once (for the
// int4 kernels whose final write does not do it: K past 4096).
__global__ __launch_bounds__(256) void k_lora_dq(const LoraAdd add, const int32_t *__restrict__ Y32, int M,
                                                 const float *__restrict__ sw, const float *__restrict__ sx,
                                                 uint16_t *__restrict__ Yh) {
    const int m = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
    if (m >= M) return;
    const int64_t at = (int64_t)n * M + m;
    Yh[at] = bsp_f2h(add.to((float)Y32[at] * sw[m] * sx[n], n, m, M));
}
