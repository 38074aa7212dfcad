// gemm_w8a8.hip -- dense 8-bit product with scales per channel and token, for gfx950.
//
// v_mfma_i32_16x16x64_i8: a lane brings 16 bytes of one row of W (its tile in memory is
// in lane order) and 16 bytes of one token, and holds 4 neighbouring channels of
// one token of the result. Sums are int32 and exact.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitmap_spmm.h"
#include "device_common.h"

namespace {

typedef int w8_i4 __attribute__((ext_vector_type(4)));

struct W8Args {
    const uint8_t *tiles;
    const int8_t *x;
    int64_t xs;
    const float *scale_w, *scale_x;
    uint16_t *y;
    int64_t ys, n;
    int M, bands, ktiles;
    int last;                // last 16-byte piece of a token's row, as a byte offset
};

// One wavefront: 16 channels x 16 tokens over all of K.
__global__ __launch_bounds__(256) void k_w8_plain(const W8Args a) {
    const int lane = threadIdx.x & 63, band = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (band >= a.bands) return;
    const int64_t n = (int64_t)blockIdx.y * 16 + (lane & 15);
    const uint8_t *w = a.tiles + ((int64_t)band * a.ktiles << 10) + lane * 16;
    const int8_t *x = a.x + min(n, a.n - 1) * a.xs;
    w8_i4 acc = {0, 0, 0, 0};
    for (int t = 0; t < a.ktiles; ++t) {
        const w8_i4 A = *reinterpret_cast<const w8_i4 *>(w + ((int64_t)t << 10));
        // past the row's last piece W is zero: any value will do
        const w8_i4 B = *reinterpret_cast<const w8_i4 *>(x + min(t * 64 + (lane >> 4) * 16, a.last));
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(A, B, acc, 0, 0, 0);
    }
    if (n >= a.n) return;
    const float sx = a.scale_x[n];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int m = band * 16 + (lane >> 4) * 4 + r;
        if (m < a.M) a.y[n * a.ys + m] = bsp_f2h(bsp_rounded((float)acc[r] * a.scale_w[m] * sx));
    }
}

}  // namespace

extern "C" int gemm_w8a8_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t *bytes) {
    if (bytes == nullptr || M < 0 || K < 0 || N < 0) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > INT32_MAX || N > INT32_MAX) return BSP_E_OVERFLOW;
    *bytes = 0;
    return BSP_OK;
}

extern "C" int gemm_w8a8_dq(const uint8_t *tiles, int64_t M, int64_t K, const int8_t *X, int64_t x_stride, int64_t N,
                            const float *scale_w, const float *scale_x, uint16_t *Y, int64_t y_stride,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (M < 0 || K < 0 || N < 0 || workspace_bytes < 0) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > INT32_MAX || N > INT32_MAX) return BSP_E_OVERFLOW;
    if (M == 0 || N == 0) return BSP_OK;
    if (Y == nullptr || scale_w == nullptr || scale_x == nullptr || y_stride < M) return BSP_E_ARG;
    if (K > 0 && (tiles == nullptr || X == nullptr || x_stride < K || x_stride % 16 != 0)) return BSP_E_ARG;
    if ((((uintptr_t)tiles | (uintptr_t)X) & 15u) != 0 || ((uintptr_t)Y & 1u) != 0) return BSP_E_ARG;
    if ((((uintptr_t)scale_w | (uintptr_t)scale_x) & 3u) != 0) return BSP_E_ARG;
    if ((workspace == nullptr) != (workspace_bytes == 0) || ((uintptr_t)workspace & 255u) != 0) return BSP_E_ARG;
    W8Args a{};
    a.tiles = tiles, a.x = X, a.xs = x_stride, a.scale_w = scale_w, a.scale_x = scale_x, a.y = Y, a.ys = y_stride;
    a.n = N, a.M = (int)M, a.bands = (int)((M + 15) / 16), a.ktiles = (int)((K + 63) / 64);
    a.last = (int)std::max<int64_t>(x_stride - 16, 0);
    hipLaunchKernelGGL(k_w8_plain, dim3((unsigned)((a.bands + 3) / 4), (unsigned)((N + 15) / 16)), dim3(256), 0, stream,
                       a);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
