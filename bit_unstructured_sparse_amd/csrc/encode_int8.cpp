// encode_int8.cpp -- host side of the dense 8-bit product: W laid out in the order the
// matrix instruction takes it (include/bitmap_spmm.h, encode_int8_tiles).
#include <string.h>

#include <algorithm>

#include "bitmap_spmm.h"

extern "C" int64_t int8_tiles_bytes(int64_t M, int64_t K) {
    if (M < 0 || K < 0) return -1;
    return (M + 15) / 16 * ((K + 63) / 64) * 1024;
}

extern "C" int encode_int8_tiles(const int8_t *W, int64_t M, int64_t K, int64_t ldw, uint8_t *tiles) {
    if (M < 0 || K < 0 || ldw < K) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > INT32_MAX) return BSP_E_OVERFLOW;
    if (M == 0 || K == 0) return BSP_OK;
    if (W == nullptr || tiles == nullptr) return BSP_E_ARG;
    const int64_t ktiles = (K + 63) / 64;
    memset(tiles, 0, (size_t)int8_tiles_bytes(M, K));
    for (int64_t m = 0; m < M; ++m) {
        const int8_t *row = W + m * ldw;
        uint8_t *band = tiles + m / 16 * ktiles * 1024 + m % 16 * 16;
        for (int64_t k = 0; k < K; k += 16)
            memcpy(band + k / 64 * 1024 + k % 64 * 16, row + k, (size_t)std::min<int64_t>(16, K - k));
    }
    return BSP_OK;
}
