// 8-bit activation checkpoints and the activations that keep them.
//
// Format: shampoo4_train.h (blocks of 32 rows x 1 column, scale a power of two, codes in
// two's complement).  All four kernels are HBM streams over the same tiles: a wave takes
// 32 rows x 16 ROWS columns, each lane ROWS rows of eight columns (16 bytes in 16 bits).  A
// lane's row loads are independent and all in flight at once; a block's maximum is ROWS
// maxima in registers, as packed magnitudes, and three cross-lane steps over the row groups,
// so a block's rows are read once and nothing goes through LDS.
//
// Large shapes are bound by HBM: [16384, 4096] bf16 stored in 39.4 us (5.2 TB/s) and loaded
// in 31.6 (6.4 TB/s; part of the codes is still in the last-level cache); gated SiLU of
// [8192, 4096] bf16 with both checkpoints in 58.6 us forward (4.6 TB/s) and 47.6 backward
// (5.7 TB/s).  The counters show each
// input read once and each output written once.  Small shapes take one launch and one trip
// to memory: [16, 1024] bf16 3.0 us stored, 2.5 loaded.  Between them, GELU of [1000, 2309] fp32
// takes 9.0 us forward and 6.6 backward, launches behind each other, where the bytes are 4.6 and
// 4.1; rows that are not aligned are the least of it ([1000, 2304]: 8.8 and 6.2).
//
// ROWS is 8, or 2 while the wide tiles are fewer than one a SIMD, where what counts is how
// long a lane takes and not the 128-byte runs of a row.  Measured with 8 and with 2 rows a
// lane: gated SiLU forward of [16, 1021] bf16 12.0 and 5.6 us, of [1000, 2309] bf16 14.8 and
// 10.1, of [2048, 4096] bf16 15.6 and 19.2, of [16384, 4096] bf16 81 and 124.  Loading to
// fp32 alone gains from 2 rows at every size (32 bytes a lane make long runs by themselves):
// [4096, 4096] 18.9 and 17.7 us, [16384, 4096] 68 and 59.
#include <type_traits>

#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

template <int ROWS>
struct Tile {
    static constexpr int LANES = 2 * ROWS;    // lanes that share a row
    int64_t row0;             // this lane's first row
    int64_t col0;             // this lane's first column
    int64_t rows, cols;
    int nrow, ncol;           // valid rows (0 .. ROWS) and columns (0 .. 8) of the lane
    int64_t block;            // block of 32 rows
    bool full;                // the wave's rows and columns all exist
    bool whole;               // no lane crosses the end of a row
};

template <int ROWS>
__device__ __forceinline__ Tile<ROWS> lane_tile(int64_t rows, int64_t cols, int64_t ntiles, bool& live) {
    const int lane = threadIdx.x & 63;
    const uint32_t tile = blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    live = tile < ntiles;
    const uint32_t ncb = (uint32_t)((cols + 16 * ROWS - 1) / (16 * ROWS));
    Tile<ROWS> t;
    t.rows = rows;
    t.cols = cols;
    t.block = tile / ncb;
    t.row0 = t.block * 32 + lane / t.LANES * ROWS;
    t.col0 = (int64_t)(tile % ncb) * (16 * ROWS) + lane % t.LANES * 8;
    t.nrow = (int)max((int64_t)0, min((int64_t)ROWS, rows - t.row0));
    t.ncol = (int)max((int64_t)0, min((int64_t)8, cols - t.col0));
    t.full = __all(t.nrow == ROWS && t.ncol == 8);
    t.whole = cols >= 8 && __all(t.ncol == 8 || t.ncol == 0);
    return t;
}

// The lane's rows of eight columns, zeros outside the matrix.  No load is under a lane's own
// condition: rows and columns are clamped into the matrix, and masked.
template <class T, int ROWS>
__device__ __forceinline__ void load_tile(typename Vec8<T>::Raw (&r)[ROWS], const T* p, int64_t ld, const Tile<ROWS>& t) {
    if (t.full) {
        p += t.row0 * ld + t.col0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) r[i] = load8(p + i * ld);
        return;
    }
    if (t.whole) {
        p += t.ncol ? t.col0 : 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) r[i] = load8(p + min(t.row0 + i, t.rows - 1) * ld);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) r[i] = load8_edge(p + min(t.row0 + i, t.rows - 1) * ld, t.col0, t.cols);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) r[i] &= i < t.nrow && t.ncol ? 0xffffffffu : 0u;
}

// Row i of the lane, to p (of the lane's first row and column).
template <class T, int ROWS>
__device__ __forceinline__ void store_row(T* p, int64_t ld, int i, typename Vec8<T>::Raw v, const Tile<ROWS>& t) {
    if (t.full)
        store8(p + i * ld, v);
    else if (i < t.nrow)
        store8_n(p + i * ld, v, t.ncol);
}

typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));

// Larger magnitude bits: of one fp32 value, or of two 16-bit ones side by side.
template <class T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, a), __builtin_bit_cast(ushort2v, b)));
}

// The largest over the lanes that hold the same columns (2 ROWS apart): rotations within
// sixteen lanes, then exchanges of sixteen-lane rows and of halves, all without LDS.
template <class T, int ROWS>
__device__ __forceinline__ uint32_t over_groups(uint32_t m) {
    if constexpr (ROWS == 2) {
        m = larger<T>(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, false));    // row_ror:4
        m = larger<T>(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, false));    // row_ror:8
    }
    const auto h = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = larger<T>(h[0], h[1]);
    const auto w = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return larger<T>(w[0], w[1]);
}

// Exponents of the lane's eight columns: maxima over its rows, then over the row groups.
// Values are compared as bits, where NaN is above infinity.
template <class T, int ROWS>
__device__ __forceinline__ void exponents(const typename Vec8<T>::Raw (&r)[ROWS], uint32_t (&e)[8]) {
    constexpr int N = sizeof(r[0]) / 4;
    constexpr uint32_t MAG = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
    typename Vec8<T>::Raw m = {};
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) m[j] = larger<T>(m[j], r[i][j] & MAG);
#pragma unroll
    for (int j = 0; j < N; ++j) m[j] = over_groups<T, ROWS>(m[j]);
    const floatx8 f = Vec8<T>::get(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = act8_exponent(__float_as_uint(f[j]));
}

// Codes and exponents of a loaded tile.  Every lane inside the padded columns writes
// (padding rows and columns hold zeros); the first row group writes the exponents.
template <class T, int ROWS>
__device__ __forceinline__ void encode_tile(typename Vec8<T>::Raw (&r)[ROWS], Act8Ptr out, int64_t pitch,
                                            const Tile<ROWS>& t) {
    uint32_t e[8];
    exponents<T, ROWS>(r, e);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) unpack_again(r[i]);
    if (t.col0 >= pitch) return;
    Act8Block blk;
#pragma unroll
    for (int j = 0; j < 8; ++j) blk.set(j, e[j]);
    int8_t* c = out.codes + t.row0 * pitch + t.col0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        stg((u32x2*)(c + i * pitch), blk.codes(Vec8<T>::get(r[i])));
        unpack_again(r[i]);
    }
    if ((threadIdx.x & 63) < t.LANES) {
        u32x2 p;
        p[0] = e[0] | e[1] << 8 | e[2] << 16 | e[3] << 24;
        p[1] = e[4] | e[5] << 8 | e[6] << 16 | e[7] << 24;
        stg((u32x2*)(out.scales + t.block * pitch + t.col0), p);
    }
}

template <int ROWS>
__device__ __forceinline__ floatx8 load_scales(const uint8_t* scales, int64_t pitch, const Tile<ROWS>& t) {
    return act8_scales(ldg_u2(scales + t.block * pitch + t.col0));
}

template <class T, int ROWS>
__global__ __launch_bounds__(256) void act8_store_kernel(const T* __restrict__ x, int64_t ldx, Act8Ptr out,
                                                         int64_t rows, int64_t cols, int64_t ntiles) {
    bool live;
    const Tile<ROWS> t = lane_tile<ROWS>(rows, cols, ntiles, live);
    if (!live) return;
    typename Vec8<T>::Raw r[ROWS];
    load_tile<T, ROWS>(r, x, ldx, t);
    encode_tile<T, ROWS>(r, out, act8_pitch(cols), t);
}

template <class T, int ROWS>
__global__ __launch_bounds__(256) void act8_load_kernel(Act8Ptr in, T* __restrict__ x, int64_t ldx, int64_t rows,
                                                        int64_t cols, int64_t ntiles) {
    bool live;
    const Tile<ROWS> t = lane_tile<ROWS>(rows, cols, ntiles, live);
    const int64_t pitch = act8_pitch(cols);
    if (!live || t.col0 >= pitch) return;
    const int8_t* c = in.codes + t.row0 * pitch + t.col0;
    u32x2 q[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) q[i] = ldg_u2(c + i * pitch);     // padded rows and columns exist
    const floatx8 s = load_scales(in.scales, pitch, t);
    T* p = x + t.row0 * ldx + t.col0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) store_row<T, ROWS>(p, ldx, i, Vec8<T>::put(saturate<T>(act8_values(q[i], s))), t);
}

// a(x) and a'(x) = sg + x sg (1 - sg) z'(x) with sg = 1 / (1 + exp(-z)): z = x (SiLU) or
// 2 sqrt(2/pi) (x + 0.044715 x^3) (GELU, tanh form).  The hardware's exp2 and reciprocal are
// good to an ulp; what would cost more is the rounding of the argument -z log2 e, |z| 2^-24
// of the result, so its remainder is kept and applied, and the reciprocal takes one Newton
// step.  Past 110 on either side the sigmoid is 0 or 1 in fp32; a NaN comes back with the
// product by x.
template <int KIND>
__device__ __forceinline__ float act_argument(float x) {
    const float z = KIND == SHAMPOO4_ACT_SILU ? x : 1.5957691216f * fmaf(0.044715f * x * x, x, x);
    return __builtin_amdgcn_fmed3f(z, -110.f, 110.f);
}
constexpr float LOG2E = 1.44269502162933349609375f, LOG2E_LO = 1.925963033500e-8f;

// Eight sigmoids, and 1 - sg as e sg, which keeps its digits where the difference would be of
// near numbers.  Below z = -87.3 the exponential, or its reciprocal, leaves the normal range:
// there sg = exp(z), taken 2^64 larger, is brought to the nearest subnormal number (0 from -103.3
// on).  One look for eight values: a wave seldom has one so small.
template <int KIND>
__device__ __forceinline__ floatx8 act_sigmoids(const floatx8& x, floatx8& other) {
    floatx8 sg;
    float low = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float z = act_argument<KIND>(x[j]);
        low = fminf(low, z);
        const float t = z * -LOG2E;
        const float rest = fmaf(z, -LOG2E_LO, fmaf(z, -LOG2E, -t));
        float e = __builtin_amdgcn_exp2f(t);
        e = fmaf(e * 0.693147180559945f, rest, e);
        const float d = 1.f + e;
        const float y = __builtin_amdgcn_rcpf(d);
        sg[j] = fmaf(fmaf(-d, y, 1.f), y, y);
        other[j] = e * sg[j];
    }
    if (__any(low < -87.f)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float z = act_argument<KIND>(x[j]);
            const float t = z * LOG2E;
            const float rest = fmaf(z, LOG2E_LO, fmaf(z, LOG2E, -t));
            float e = __builtin_amdgcn_exp2f(t + 64.f);
            e = fmaf(e * 0.693147180559945f, rest, e);
            sg[j] = z < -87.f ? e * 0x1p-64f : sg[j];
            other[j] = z < -87.f ? 1.f : other[j];
        }
    }
    return sg;
}
// The two terms are of opposite signs for x < 0 and cancel at the derivative's root alone.
template <int KIND>
__device__ __forceinline__ float act_derivative(float x, float sg, float other) {
    // bounded where the sigmoid is 0 or 1 and the product below is 0, so that it stays 0
    const float dz = KIND == SHAMPOO4_ACT_SILU ? 1.f : 1.5957691216f * fmaf(0.134145f, fminf(x * x, 1e8f), 1.f);
    return fmaf(x * sg * other, dz, sg);
}

template <class T, int ROWS, int KIND, bool GATED>
__global__ __launch_bounds__(256) void act_forward_kernel(ActForward a, int64_t ntiles) {
    bool live;
    const Tile<ROWS> t = lane_tile<ROWS>(a.rows, a.cols, ntiles, live);
    if (!live) return;
    const int64_t pitch = act8_pitch(a.cols);
    typename Vec8<T>::Raw g[ROWS], u[ROWS];
    load_tile<T, ROWS>(g, (const T*)a.gate, a.ldgate, t);
    if constexpr (GATED) load_tile<T, ROWS>(u, (const T*)a.up, a.ldup, t);
    if (a.gate8.codes) encode_tile<T, ROWS>(g, a.gate8, pitch, t);
    if constexpr (GATED)
        if (a.up8.codes) encode_tile<T, ROWS>(u, a.up8, pitch, t);
    T* ph = (T*)a.h + t.row0 * a.ldh + t.col0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const floatx8 x = Vec8<T>::get(g[i]);
        floatx8 other;
        floatx8 h = x * act_sigmoids<KIND>(x, other);
        if constexpr (GATED) h *= Vec8<T>::get(u[i]);
        g[i] = Vec8<T>::put(h);
        store_row<T, ROWS>(ph, a.ldh, i, g[i], t);
        __builtin_amdgcn_sched_barrier(0);     // one row's values at a time in registers
    }
    if (a.h8.codes) encode_tile<T, ROWS>(g, a.h8, pitch, t);
}

template <class T, int ROWS, int KIND, bool GATED>
__global__ __launch_bounds__(256) void act_backward_kernel(ActBackward a, int64_t ntiles) {
    bool live;
    const Tile<ROWS> t = lane_tile<ROWS>(a.rows, a.cols, ntiles, live);
    const int64_t pitch = act8_pitch(a.cols);
    if (!live || t.col0 >= pitch) return;
    const int64_t at = t.row0 * pitch + t.col0;
    u32x2 cg[ROWS], cu[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        cg[i] = ldg_u2(a.gate8.codes + at + i * pitch);
        if constexpr (GATED) cu[i] = ldg_u2(a.up8.codes + at + i * pitch);
    }
    typename Vec8<T>::Raw d[ROWS];
    load_tile<T, ROWS>(d, (const T*)a.dh, a.lddh, t);
    const floatx8 sg = load_scales(a.gate8.scales, pitch, t);
    floatx8 su;
    if constexpr (GATED) su = load_scales(a.up8.scales, pitch, t);
    T* pg = (T*)a.dgate + t.row0 * a.lddgate + t.col0;
    T* pu = (T*)a.dup + t.row0 * a.lddup + t.col0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const floatx8 x = act8_values(cg[i], sg);
        const floatx8 dx = Vec8<T>::get(d[i]);
        floatx8 other, dg, du;
        const floatx8 s = act_sigmoids<KIND>(x, other);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dg[j] = dx[j] * act_derivative<KIND>(x[j], s[j], other[j]);
            du[j] = dx[j] * (x[j] * s[j]);
        }
        if constexpr (GATED) dg *= act8_values(cu[i], su);
        store_row<T, ROWS>(pg, a.lddgate, i, Vec8<T>::put(dg), t);
        if constexpr (GATED) store_row<T, ROWS>(pu, a.lddup, i, Vec8<T>::put(du), t);
        __builtin_amdgcn_sched_barrier(0);     // one row's values at a time in registers
    }
}

// Rows a lane takes, and the waves of the launch.
struct Cover {
    int rows;
    int64_t tiles;
    dim3 grid;
};
Cover cover(int64_t rows, int64_t cols, bool narrow = false) {
    Cover c;
    c.rows = act8_tiles(rows, cols) >= 1024 && !narrow ? 8 : 2;
    c.tiles = (rows + 31) / 32 * ((cols + 16 * c.rows - 1) / (16 * c.rows));
    c.grid = dim3((uint32_t)((c.tiles + 3) / 4));
    return c;
}

// Calls f(T{}, rows a lane as a constant) for a type and a cover.
template <class F>
void dispatch(shampoo4_dtype dtype, int rows, F f) {
    const auto with_rows = [&](auto t) {
        if (rows == 8)
            f(t, std::integral_constant<int, 8>{});
        else
            f(t, std::integral_constant<int, 2>{});
    };
    if (dtype == SHAMPOO4_BF16)
        with_rows(__bf16{});
    else if (dtype == SHAMPOO4_F16)
        with_rows(_Float16{});
    else
        with_rows(float{});
}

}  // namespace

hipError_t launch_act8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                             Act8Ptr out, hipStream_t stream) {
    const Cover c = cover(rows, cols);
    if (c.tiles <= 0) return hipSuccess;
    dispatch(dtype, c.rows, [&](auto t, auto r) {
        using T = decltype(t);
        S4_LAUNCH((act8_store_kernel<T, decltype(r)::value>), c.grid, dim3(256), 0, stream, (const T*)x, ldx, out, rows,
                  cols, c.tiles);
    });
    return hipGetLastError();
}

hipError_t launch_act8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols, Act8Ptr in, void* x, int64_t ldx,
                            hipStream_t stream) {
    const Cover c = cover(rows, cols, dtype == SHAMPOO4_F32);
    if (c.tiles <= 0) return hipSuccess;
    dispatch(dtype, c.rows, [&](auto t, auto r) {
        using T = decltype(t);
        constexpr int R = sizeof(T) == 4 ? 2 : decltype(r)::value;
        S4_LAUNCH((act8_load_kernel<T, R>), c.grid, dim3(256), 0, stream, in, (T*)x, ldx, rows, cols,
                  c.tiles);
    });
    return hipGetLastError();
}

hipError_t launch_activation_forward(int kind, shampoo4_dtype dtype, const ActForward& a, hipStream_t stream) {
    const Cover c = cover(a.rows, a.cols);
    if (c.tiles <= 0) return hipSuccess;
    dispatch(dtype, c.rows, [&](auto t, auto r) {
        using T = decltype(t);
        constexpr int R = decltype(r)::value;
        if (kind == SHAMPOO4_ACT_SILU) {
            if (a.up)
                S4_LAUNCH((act_forward_kernel<T, R, SHAMPOO4_ACT_SILU, true>), c.grid, dim3(256), 0, stream, a, c.tiles);
            else
                S4_LAUNCH((act_forward_kernel<T, R, SHAMPOO4_ACT_SILU, false>), c.grid, dim3(256), 0, stream, a, c.tiles);
        } else {
            if (a.up)
                S4_LAUNCH((act_forward_kernel<T, R, SHAMPOO4_ACT_GELU, true>), c.grid, dim3(256), 0, stream, a, c.tiles);
            else
                S4_LAUNCH((act_forward_kernel<T, R, SHAMPOO4_ACT_GELU, false>), c.grid, dim3(256), 0, stream, a, c.tiles);
        }
    });
    return hipGetLastError();
}

hipError_t launch_activation_backward(int kind, shampoo4_dtype dtype, const ActBackward& a, hipStream_t stream) {
    const Cover c = cover(a.rows, a.cols);
    if (c.tiles <= 0) return hipSuccess;
    dispatch(dtype, c.rows, [&](auto t, auto r) {
        using T = decltype(t);
        constexpr int R = decltype(r)::value;
        if (kind == SHAMPOO4_ACT_SILU) {
            if (a.dup)
                S4_LAUNCH((act_backward_kernel<T, R, SHAMPOO4_ACT_SILU, true>), c.grid, dim3(256), 0, stream, a, c.tiles);
            else
                S4_LAUNCH((act_backward_kernel<T, R, SHAMPOO4_ACT_SILU, false>), c.grid, dim3(256), 0, stream, a, c.tiles);
        } else {
            if (a.dup)
                S4_LAUNCH((act_backward_kernel<T, R, SHAMPOO4_ACT_GELU, true>), c.grid, dim3(256), 0, stream, a, c.tiles);
            else
                S4_LAUNCH((act_backward_kernel<T, R, SHAMPOO4_ACT_GELU, false>), c.grid, dim3(256), 0, stream, a, c.tiles);
        }
    });
    return hipGetLastError();
}

}  // namespace s4
