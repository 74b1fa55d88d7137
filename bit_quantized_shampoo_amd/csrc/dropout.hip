// Dropout of a matrix with a mask that is never stored (random.hpp).
//
// A stream: a lane takes eight columns of ROWS rows, all loads in flight before the generator's
// first use.  Bytes bound it: 16384 x 4096 bf16 takes 43-50 us (268 MB), the generator's 40 instructions for
// eight elements beside them.
#include "random.hpp"
#include "train.hpp"

namespace s4 {

namespace {

constexpr int ROWS = 4;

template <class T>
__global__ __launch_bounds__(256) void dropout_kernel(const T* x, int64_t ldx, T* y, int64_t ldy,
                                                      int64_t rows, int64_t cols, uint32_t tiles_n, int64_t ntiles,
                                                      Drop d) {
    const uint32_t tile = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (tile >= ntiles) return;
    const int64_t row0 = (int64_t)(tile / tiles_n) * ROWS, col = (int64_t)(tile % tiles_n) * 512 + (threadIdx.x & 63) * 8;
    const uint64_t call = drop_call(d);
    typename Vec8<T>::Raw r[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) r[i] = load8_near(x + min(row0 + i, rows - 1) * ldx, col, cols);
    const int n = (int)max((int64_t)0, min((int64_t)8, cols - col));
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        finish8<T>(r[i], col, cols);
        if (row0 + i >= rows || n == 0) continue;
        if (d.threshold)
            r[i] = Vec8<T>::put(drop8(Vec8<T>::get(r[i]) * d.scale, drop_keep8(d, call, row0 + i, col >> 3), d));
        store8_n(y + (row0 + i) * ldy + col, r[i], n);
    }
}

}  // namespace

hipError_t launch_dropout(shampoo4_dtype dtype, int64_t rows, int64_t cols, const Drop& d, const void* x, int64_t ldx,
                          void* y, int64_t ldy, hipStream_t stream) {
    if (rows <= 0) return hipSuccess;
    const int64_t tn = (cols + 511) / 512, tiles = (rows + ROWS - 1) / ROWS * tn;
    const dim3 grid((uint32_t)((tiles + 3) / 4));
    by_type(dtype, [&](auto t) {
        using T = decltype(t);
        S4_LAUNCH(dropout_kernel<T>, grid, dim3(256), 0, stream, (const T*)x, ldx, (T*)y, ldy, rows, cols, (uint32_t)tn,
                  tiles, d);
    });
    return hipGetLastError();
}

}  // namespace s4
