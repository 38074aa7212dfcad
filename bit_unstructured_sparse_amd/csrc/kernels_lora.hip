// kernels_lora.hip -- low-rank adapters of many requests beside a shared
// sparse projection: Y[n] = W x_n + scale[a] B_a (A_a x_n), a = index[n].
//
// Two small products around the sparse one: t_n = scale[a] A_a x_n (rank
// values per token, fp32, through the workspace), then B_a t_n added to W x_n.

struct LoraArgs {
    const uint16_t *A, *B;
    const float *scale;
    const int32_t *ranks, *index;
    float *t;          // [N][R]
    int adapters, R;
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

// t[n][r]: one wavefront per (n, r); rows past the rank and tokens without an
// adapter give zero.
__global__ __launch_bounds__(256) void k_lora_down(const LoraArgs a, const uint16_t *__restrict__ X, int N, int K) {
    const int w = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = w / a.R, r = w - n * a.R;
    if (n >= N) return;
    int rank;
    const int i = lora_of(a, n, &rank);
    float s = 0.f;
    if (r < rank) {
        const uint16_t *row = a.A + ((int64_t)i * a.R + r) * K, *x = X + (int64_t)n * K;
        for (int k = lane; k < K; k += 64) s += bsp_h2f(row[k]) * bsp_h2f(x[k]);
        s = bsp_wave_sum(s);
        if (a.scale != nullptr) s *= a.scale[i];
    }
    if (lane == 0) a.t[(int64_t)n * a.R + r] = s;
}

// Y[n][m] += B_a[m] t_n, a thread per output.
__global__ __launch_bounds__(256) void k_lora_up(const LoraArgs a, int M, uint16_t *__restrict__ Y) {
    const int m = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
    if (m >= M) return;
    int rank;
    const int i = lora_of(a, n, &rank);
    if (i < 0) return;
    const uint16_t *row = a.B + ((int64_t)i * M + m) * a.R;
    float s = 0.f;
    for (int r = 0; r < rank; ++r) s += bsp_h2f(row[r]) * a.t[(int64_t)n * a.R + r];
    uint16_t *y = Y + (int64_t)n * M + m;
    *y = bsp_f2h(bsp_h2f(*y) + s);
}
