// encode_int8.cpp -- host side of the dense 8-bit product: W laid out in the order the
// matrix instruction takes it (include/bitmap_spmm.h, encode_int8_tiles).
#include <string.h>

#include <algorithm>
#include <atomic>
#include <thread>

#include "bitmap_spmm.h"

namespace {

constexpr int64_t BAND_BYTES_PER_THREAD = 1 << 20;

// One band of 16 rows, tile by tile.
void lay_out(const int8_t *W, int64_t M, int64_t K, int64_t ldw, int64_t band, uint8_t *tiles) {
    const int64_t ktiles = (K + 63) / 64;
    const int rows = (int)std::min<int64_t>(16, M - band * 16);
    uint8_t *t = tiles + band * ktiles * 1024;
    for (int64_t k0 = 0; k0 < K; k0 += 64, t += 1024) {
        if (rows < 16 || k0 + 64 > K) memset(t, 0, 1024);
        for (int r = 0; r < rows; ++r)
            for (int64_t k = k0; k < std::min(k0 + 64, K); k += 16)
                memcpy(t + (k - k0) * 16 + r * 16, W + (band * 16 + r) * ldw + k, (size_t)std::min<int64_t>(16, K - k));
    }
}

}  // namespace

extern "C" int64_t int8_tiles_bytes(int64_t M, int64_t K) {
    if (M < 0 || K < 0 || M > INT32_MAX || K > BSP_W8_MAX_K) return -1;
    return (M + 15) / 16 * ((K + 63) / 64) * 1024;
}

extern "C" int encode_int8_tiles(const int8_t *W, int64_t M, int64_t K, int64_t ldw, uint8_t *tiles) {
    if (M < 0 || K < 0 || ldw < K) return BSP_E_ARG;
    if (K > BSP_W8_MAX_K || M > INT32_MAX) return BSP_E_OVERFLOW;
    if (M == 0 || K == 0) return BSP_OK;
    if (W == nullptr || tiles == nullptr) return BSP_E_ARG;
    const int64_t bands = (M + 15) / 16;
    std::atomic<int64_t> next{0};
    auto work = [&] {
        for (int64_t b; (b = next.fetch_add(1, std::memory_order_relaxed)) < bands;) lay_out(W, M, K, ldw, b, tiles);
    };
    const int64_t want = std::min<int64_t>({int8_tiles_bytes(M, K) / BAND_BYTES_PER_THREAD, bands,
                                            (int64_t)std::thread::hardware_concurrency(), 16});
    std::thread others[15];
    for (int64_t i = 0; i + 1 < want; ++i) {
        try {
            others[i] = std::thread(work);
        } catch (...) {      // no thread to be had: this one does the work
            break;
        }
    }
    work();
    for (std::thread &t : others)
        if (t.joinable()) t.join();
    return BSP_OK;
}
