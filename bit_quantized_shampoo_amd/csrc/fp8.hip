// Matrices in e4m3 with a scale for each block of 128 columns (shampoo4_train.h).
//
// Rows: a lane takes eight columns, so sixteen lanes hold a block and its maximum takes four
// rotations among them.  Weights: a workgroup takes 128 x 128, keeps it in registers while the
// maximum goes through LDS, and writes the codes as they lie and transposed (4 x 4 codes at a
// time, from LDS).
//
// Bytes bound all of them: 16384 x 4096 bf16 rows are stored in 31-36 us (201 MB, 5.6-6.5 TB/s), a 4096 x 4096 fp32
// weight in both orders in 18.7 (101 MB), one order restored to bf16 in 8.8 (50 MB).  Four rows a lane keep
// enough loads on their way; half a wave writes a whole line of 128 bytes of W^T.
#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

constexpr int ROWS = 4;

template <class T>
__global__ __launch_bounds__(256) void fp8_store_kernel(const T* __restrict__ x, int64_t ldx, uint8_t* codes,
                                                        uint8_t* scales, int64_t rows, int64_t cols, uint32_t tiles_n,
                                                        int64_t ntiles) {
    const uint32_t tile = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (tile >= ntiles) return;
    const int lane = threadIdx.x & 63;
    const int64_t row0 = (int64_t)(tile / tiles_n) * ROWS, col = (int64_t)(tile % tiles_n) * 512 + lane * 8;
    const int64_t pitch = fp8_pitch(cols), sp = fp8_scale_pitch(cols);
    typename Vec8<T>::Raw r[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) r[i] = load8_near(x + min(row0 + i, rows - 1) * ldx, col, cols);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        finish8<T>(r[i], col, cols);
        const floatx8 f = Vec8<T>::get(r[i]);
        const uint32_t e = fp8_exponent(max16(magnitude(f)));
        if (row0 + i >= rows) break;
        if (col < pitch) stg((u32x2*)(codes + (row0 + i) * pitch + col), Fp8Block(e).codes(f));
        // the four blocks of a wave, padding among them, are one word of the row's scales
        if ((lane & 15) == 0) stg(scales + (row0 + i) * sp + (col >> 7), (uint8_t)e);
    }
}

// Rows of codes in LDS: 128 and a gap of 16 bytes.
constexpr int LDS_ROW = 144;

template <class T>
__global__ __launch_bounds__(256) void fp8_weight_kernel(const T* __restrict__ w, int64_t ldw, uint8_t* codes,
                                                         uint8_t* scales, uint8_t* t_codes, uint8_t* t_scales,
                                                         int64_t rows, int64_t cols, uint32_t tiles_n) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[128 * LDS_ROW];
    __shared__ uint32_t wave_max[4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t bm = blockIdx.x / tiles_n, bn = blockIdx.x % tiles_n, row0 = bm * 128, col0 = bn * 128;
    const int c = (tid & 15) * 8, r0 = tid >> 4;
    typename Vec8<T>::Raw r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = load8_near(w + min(row0 + r0 + 16 * i, rows - 1) * ldw, col0 + c, cols);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        finish8<T>(r[i], col0 + c, cols);
        r[i] &= row0 + r0 + 16 * i < rows ? 0xffffffffu : 0u;
        m = max(m, magnitude(Vec8<T>::get(r[i])));
    }
    m = max16(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (lane == 0) wave_max[tid >> 6] = m;
    __syncthreads();
    m = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
    const uint32_t e = fp8_exponent(m);
    const Fp8Block blk(e);
    const int64_t pitch = fp8_pitch(cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const u32x2 q = blk.codes(Vec8<T>::get(r[i]));
        if (row0 + r0 + 16 * i < rows) stg((u32x2*)(codes + (row0 + r0 + 16 * i) * pitch + col0 + c), q);
        if (t_codes) *(u32x2*)(lds + (r0 + 16 * i) * LDS_ROW + c) = q;
    }
    // this block's scale, and behind the last one of a row the padding's
    const int64_t sp = fp8_scale_pitch(cols), tsp = fp8_scale_pitch(rows);
    if (tid == 0) {
        stg(scales + bm * sp + bn, (uint8_t)e);
        if (col0 + 128 >= cols)
            for (int64_t j = bn + 1; j < sp; ++j) stg(scales + bm * sp + j, (uint8_t)1);
        if (t_codes) {
            stg(t_scales + bn * tsp + bm, (uint8_t)e);
            if (row0 + 128 >= rows)
                for (int64_t j = bm + 1; j < tsp; ++j) stg(t_scales + bn * tsp + j, (uint8_t)1);
        }
    }
    if (!t_codes) return;
    __syncthreads();
    // four rows of sixteen columns a thread; neighbouring lanes write neighbouring words of W^T
    const int tr = (tid & 31) * 4, tc = (tid >> 5) * 16;
    u32x4 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = *(const u32x4*)(lds + (tr + i) * LDS_ROW + tc);
    const int64_t tp = fp8_pitch(rows);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo0 = __builtin_amdgcn_perm(q[1][k], q[0][k], 0x05010400u);     // 00 10 01 11
        const uint32_t hi0 = __builtin_amdgcn_perm(q[1][k], q[0][k], 0x07030602u);     // 02 12 03 13
        const uint32_t lo1 = __builtin_amdgcn_perm(q[3][k], q[2][k], 0x05010400u);
        const uint32_t hi1 = __builtin_amdgcn_perm(q[3][k], q[2][k], 0x07030602u);
        const uint32_t t[4] = {__builtin_amdgcn_perm(lo1, lo0, 0x05040100u), __builtin_amdgcn_perm(lo1, lo0, 0x07060302u),
                               __builtin_amdgcn_perm(hi1, hi0, 0x05040100u), __builtin_amdgcn_perm(hi1, hi0, 0x07060302u)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = col0 + tc + 4 * k + j;
            if (at < cols) stg((uint32_t*)(t_codes + at * tp + row0 + tr), t[j]);
        }
    }
}

template <class T>
__global__ __launch_bounds__(256) void fp8_load_kernel(const uint8_t* codes, const uint8_t* scales, T* __restrict__ x,
                                                       int64_t ldx, int64_t rows, int64_t cols, int shift,
                                                       uint32_t tiles_n, int64_t ntiles) {
    const uint32_t tile = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (tile >= ntiles) return;
    const int64_t row0 = (int64_t)(tile / tiles_n) * ROWS, col = (int64_t)(tile % tiles_n) * 512 + (threadIdx.x & 63) * 8;
    const int64_t pitch = fp8_pitch(cols), sp = fp8_scale_pitch(cols);
    const int n = (int)max((int64_t)0, min((int64_t)8, cols - col));
    if (n == 0) return;
    u32x2 q[ROWS];
    uint32_t e[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t row = min(row0 + i, rows - 1);
        q[i] = ldg_u2(codes + row * pitch + col);
        e[i] = ldg(scales + (row >> shift) * sp + (col >> 7));
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (row0 + i >= rows) break;
        // e = 255: infinity times a code 0 is NaN
        const floatx8 f = fp8_values(q[i]) * __uint_as_float(e[i] << 23);
        store8_n(x + (row0 + i) * ldx + col, Vec8<T>::put(saturate<T>(f)), n);
    }
}

}  // namespace

hipError_t launch_fp8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                            uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    if (rows <= 0) return hipSuccess;
    const int64_t tn = (cols + 511) / 512, tiles = (rows + ROWS - 1) / ROWS * tn;
    by_type(dtype, [&](auto t) {
        using T = decltype(t);
        S4_LAUNCH(fp8_store_kernel<T>, dim3((uint32_t)((tiles + 3) / 4)), dim3(256), 0, stream, (const T*)x, ldx, codes,
                  scales, rows, cols, (uint32_t)tn, tiles);
    });
    return hipGetLastError();
}

hipError_t launch_fp8_store_weight(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* w, int64_t ldw,
                                   uint8_t* codes, uint8_t* scales, uint8_t* t_codes, uint8_t* t_scales,
                                   hipStream_t stream) {
    if (rows <= 0) return hipSuccess;
    const int64_t tn = (cols + 127) / 128, tiles = (rows + 127) / 128 * tn;
    by_type(dtype, [&](auto t) {
        using T = decltype(t);
        S4_LAUNCH(fp8_weight_kernel<T>, dim3((uint32_t)tiles), dim3(256), 0, stream, (const T*)w, ldw, codes, scales,
                  t_codes, t_scales, rows, cols, (uint32_t)tn);
    });
    return hipGetLastError();
}

hipError_t launch_fp8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols, int block_rows, const uint8_t* codes,
                           const uint8_t* scales, void* x, int64_t ldx, hipStream_t stream) {
    if (rows <= 0) return hipSuccess;
    const int64_t tn = (cols + 511) / 512, tiles = (rows + ROWS - 1) / ROWS * tn;
    by_type(dtype, [&](auto t) {
        using T = decltype(t);
        S4_LAUNCH(fp8_load_kernel<T>, dim3((uint32_t)((tiles + 3) / 4)), dim3(256), 0, stream, codes, scales, (T*)x, ldx,
                  rows, cols, block_rows == 1 ? 0 : 7, (uint32_t)tn, tiles);
    });
    return hipGetLastError();
}

}  // namespace s4
