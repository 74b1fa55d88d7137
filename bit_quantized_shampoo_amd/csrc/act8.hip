// 8-bit activation checkpoints and the activations that keep them.
//
// Format: shampoo4_train.h (blocks of 32 rows x 1 column, scale a power of two, codes in
// two's complement).  All four kernels are HBM streams over the same tiles: a wave takes
// 32 rows x 128 columns, lane (rg = lane / 16, cg = lane % 16) the eight rows 8 rg .. 8 rg + 7
// of the eight columns 8 cg ..  A lane's eight row loads are independent and all in flight
// at once (8 KB a wave in 16 bits, in runs of 256 bytes a row); a block's maximum is eight
// maxima in registers and two butterflies over the four row groups, so a block's rows are
// read once and nothing goes through LDS.
#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

struct Tile {
    int64_t row0;             // this lane's first row
    int64_t col0;             // this lane's first column
    int64_t rows, cols;
    int nrow, ncol;           // valid rows and columns of the lane, 0..8
    int64_t block;            // block of 32 rows
    bool full;                // the wave's rows and columns all exist
    bool vectors;             // no lane's columns end inside its eight
};

__device__ __forceinline__ Tile lane_tile(int64_t rows, int64_t cols, int64_t ntiles, bool& live) {
    const int lane = threadIdx.x & 63;
    const uint32_t tile = blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    live = tile < ntiles;
    const uint32_t ncb = (uint32_t)((cols + ACT8_COLS - 1) / ACT8_COLS);
    Tile t;
    t.rows = rows;
    t.cols = cols;
    t.block = tile / ncb;
    t.row0 = t.block * 32 + (lane >> 4) * 8;
    t.col0 = (int64_t)(tile % ncb) * ACT8_COLS + (lane & 15) * 8;
    t.nrow = (int)max((int64_t)0, min((int64_t)8, rows - t.row0));
    t.ncol = (int)max((int64_t)0, min((int64_t)8, cols - t.col0));
    t.full = __all(t.nrow == 8 && t.ncol == 8);
    t.vectors = cols >= 8 && __all(t.ncol == 8 || t.ncol == 0);
    return t;
}

// The lane's eight rows of eight columns, zeros outside the matrix.  No load is under a
// lane's own condition: rows and columns are clamped into the matrix, and masked.
template <class T>
__device__ __forceinline__ void load_tile(typename Vec8<T>::Raw (&r)[8], const T* p, int64_t ld, const Tile& t) {
    if (t.full) {
        p += t.row0 * ld + t.col0;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = load8(p + i * ld);
    } else if (t.vectors) {
        p += t.ncol ? t.col0 : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = load8(p + min(t.row0 + i, t.rows - 1) * ld);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] &= i < t.nrow && t.ncol ? 0xffffffffu : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = load8_clamped(p + min(t.row0 + i, t.rows - 1) * ld, t.col0, t.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] &= i < t.nrow ? 0xffffffffu : 0u;
    }
}

template <class T>
__device__ __forceinline__ void store_tile(const typename Vec8<T>::Raw (&r)[8], T* p, int64_t ld, const Tile& t) {
    p += t.row0 * ld + t.col0;
    if (t.full) {
#pragma unroll
        for (int i = 0; i < 8; ++i) store8(p + i * ld, r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < t.nrow) store8_n(p + i * ld, r[i], t.ncol);
    }
}

// Exponents of the lane's eight columns: maxima over its rows, then over the four row groups
// (lanes 16 and 32 apart).  Values are compared as bits, where NaN is above infinity.
template <class T>
__device__ __forceinline__ void exponents(const typename Vec8<T>::Raw (&r)[8], uint32_t (&e)[8]) {
    uint32_t m[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const floatx8 f = Vec8<T>::get(r[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = max(m[j], __float_as_uint(f[j]) & 0x7fffffffu);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
        m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 32));
        e[j] = act8_exponent(m[j]);
    }
}

// Codes and exponents of a loaded tile.  Every lane inside the padded columns writes
// (padding rows and columns hold zeros); the first row group writes the exponents.
template <class T>
__device__ __forceinline__ void encode_tile(typename Vec8<T>::Raw (&r)[8], Act8Ptr out, int64_t pitch,
                                            const Tile& t) {
    uint32_t e[8];
    exponents<T>(r, e);
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack_again(r[i]);
    if (t.col0 >= pitch) return;
    Act8Block blk;
#pragma unroll
    for (int j = 0; j < 8; ++j) blk.set(j, e[j]);
    int8_t* c = out.codes + t.row0 * pitch + t.col0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        stg((u32x2*)(c + i * pitch), blk.codes(Vec8<T>::get(r[i])));
        unpack_again(r[i]);
    }
    if ((threadIdx.x & 63) < 16) {
        u32x2 p;
        p[0] = e[0] | e[1] << 8 | e[2] << 16 | e[3] << 24;
        p[1] = e[4] | e[5] << 8 | e[6] << 16 | e[7] << 24;
        stg((u32x2*)(out.scales + t.block * pitch + t.col0), p);
    }
}

__device__ __forceinline__ floatx8 load_scales(const uint8_t* scales, int64_t pitch, const Tile& t) {
    return act8_scales(ldg_u2(scales + t.block * pitch + t.col0));
}

template <class T>
__global__ __launch_bounds__(256) void act8_store_kernel(const T* __restrict__ x, int64_t ldx, Act8Ptr out,
                                                         int64_t rows, int64_t cols, int64_t ntiles) {
    bool live;
    const Tile t = lane_tile(rows, cols, ntiles, live);
    if (!live) return;
    typename Vec8<T>::Raw r[8];
    load_tile(r, x, ldx, t);
    encode_tile<T>(r, out, act8_pitch(cols), t);
}

template <class T>
__device__ __forceinline__ floatx8 saturate(floatx8 f) {
    if constexpr (sizeof(T) == 2 && !__is_same(T, __bf16)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // a finite value beyond float16's range; NaN passes (both comparisons are false)
            f[j] = f[j] > 65504.f ? 65504.f : f[j];
            f[j] = f[j] < -65504.f ? -65504.f : f[j];
        }
    }
    return f;
}

template <class T>
__global__ __launch_bounds__(256) void act8_load_kernel(Act8Ptr in, T* __restrict__ x, int64_t ldx, int64_t rows,
                                                        int64_t cols, int64_t ntiles) {
    bool live;
    const Tile t = lane_tile(rows, cols, ntiles, live);
    const int64_t pitch = act8_pitch(cols);
    if (!live || t.col0 >= pitch) return;
    const int8_t* c = in.codes + t.row0 * pitch + t.col0;
    u32x2 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = ldg_u2(c + i * pitch);     // padded rows and columns exist
    const floatx8 s = load_scales(in.scales, pitch, t);
    typename Vec8<T>::Raw r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = Vec8<T>::put(saturate<T>(act8_values(q[i], s)));
    store_tile(r, x, ldx, t);
}

// a(x) and a'(x) = sg + x sg (1 - sg) z'(x) with sg = 1 / (1 + exp(-z)): z = x (SiLU) or
// 2 sqrt(2/pi) (x + 0.044715 x^3) (GELU, tanh form).  No difference of near values, so
// small and large arguments keep their relative precision.  The hardware exp2 and reciprocal
// (1 ulp each) do: the argument's own rounding, |z| 2^-24 of the result, is larger.
template <int KIND>
__device__ __forceinline__ float act_sigmoid(float x) {
    const float z = KIND == SHAMPOO4_ACT_SILU ? x : 1.5957691216f * fmaf(0.044715f * x * x, x, x);
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950409f * z));
}
template <int KIND>
__device__ __forceinline__ float act_derivative(float x, float sg) {
    const float dz = KIND == SHAMPOO4_ACT_SILU ? 1.f : 1.5957691216f * fmaf(0.134145f * x, x, 1.f);
    return fmaf(x * sg * (1.f - sg), dz, sg);
}

template <class T, int KIND, bool GATED>
__global__ __launch_bounds__(256) void act_forward_kernel(ActForward a, int64_t ntiles) {
    bool live;
    const Tile t = lane_tile(a.rows, a.cols, ntiles, live);
    if (!live) return;
    const int64_t pitch = act8_pitch(a.cols);
    typename Vec8<T>::Raw g[8], u[8];
    load_tile(g, (const T*)a.gate, a.ldgate, t);
    if constexpr (GATED) load_tile(u, (const T*)a.up, a.ldup, t);
    if (a.gate8.codes) encode_tile<T>(g, a.gate8, pitch, t);
    if constexpr (GATED)
        if (a.up8.codes) encode_tile<T>(u, a.up8, pitch, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const floatx8 x = Vec8<T>::get(g[i]);
        floatx8 h;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = x[j] * act_sigmoid<KIND>(x[j]);
        if constexpr (GATED) h *= Vec8<T>::get(u[i]);
        g[i] = Vec8<T>::put(h);
        __builtin_amdgcn_sched_barrier(0);     // one row's values at a time in registers
    }
    store_tile(g, (T*)a.h, a.ldh, t);
    if (a.h8.codes) encode_tile<T>(g, a.h8, pitch, t);
}

template <class T, int KIND, bool GATED>
__global__ __launch_bounds__(256) void act_backward_kernel(ActBackward a, int64_t ntiles) {
    bool live;
    const Tile t = lane_tile(a.rows, a.cols, ntiles, live);
    const int64_t pitch = act8_pitch(a.cols);
    if (!live || t.col0 >= pitch) return;
    const int64_t at = t.row0 * pitch + t.col0;
    u32x2 cg[8], cu[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cg[i] = ldg_u2(a.gate8.codes + at + i * pitch);
        if constexpr (GATED) cu[i] = ldg_u2(a.up8.codes + at + i * pitch);
    }
    typename Vec8<T>::Raw d[8];
    load_tile(d, (const T*)a.dh, a.lddh, t);
    const floatx8 sg = load_scales(a.gate8.scales, pitch, t);
    floatx8 su;
    if constexpr (GATED) su = load_scales(a.up8.scales, pitch, t);
    T* pg = (T*)a.dgate + t.row0 * a.lddgate + t.col0;
    T* pu = (T*)a.dup + t.row0 * a.lddup + t.col0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const floatx8 x = act8_values(cg[i], sg);
        const floatx8 dx = Vec8<T>::get(d[i]);
        floatx8 s, dg, du;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = act_sigmoid<KIND>(x[j]);
            dg[j] = dx[j] * act_derivative<KIND>(x[j], s[j]);
            du[j] = dx[j] * (x[j] * s[j]);
        }
        if constexpr (GATED) dg *= act8_values(cu[i], su);
        if (t.full) {
            store8(pg + i * a.lddgate, Vec8<T>::put(dg));
            if constexpr (GATED) store8(pu + i * a.lddup, Vec8<T>::put(du));
        } else if (i < t.nrow) {
            store8_n(pg + i * a.lddgate, Vec8<T>::put(dg), t.ncol);
            if constexpr (GATED) store8_n(pu + i * a.lddup, Vec8<T>::put(du), t.ncol);
        }
        __builtin_amdgcn_sched_barrier(0);     // one row's values at a time in registers
    }
}

dim3 wave_grid(int64_t ntiles) { return dim3((uint32_t)((ntiles + 3) / 4)); }

template <class T, bool GATED>
void forward_of(int kind, const ActForward& a, int64_t nt, hipStream_t stream) {
    if (kind == SHAMPOO4_ACT_SILU)
        S4_LAUNCH((act_forward_kernel<T, SHAMPOO4_ACT_SILU, GATED>), wave_grid(nt), dim3(256), 0, stream, a, nt);
    else
        S4_LAUNCH((act_forward_kernel<T, SHAMPOO4_ACT_GELU, GATED>), wave_grid(nt), dim3(256), 0, stream, a, nt);
}
template <class T, bool GATED>
void backward_of(int kind, const ActBackward& a, int64_t nt, hipStream_t stream) {
    if (kind == SHAMPOO4_ACT_SILU)
        S4_LAUNCH((act_backward_kernel<T, SHAMPOO4_ACT_SILU, GATED>), wave_grid(nt), dim3(256), 0, stream, a, nt);
    else
        S4_LAUNCH((act_backward_kernel<T, SHAMPOO4_ACT_GELU, GATED>), wave_grid(nt), dim3(256), 0, stream, a, nt);
}

}  // namespace

hipError_t launch_act8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                             Act8Ptr out, hipStream_t stream) {
    const int64_t nt = act8_tiles(rows, cols);
    if (nt <= 0) return hipSuccess;
    switch (dtype) {
        case SHAMPOO4_BF16:
            S4_LAUNCH(act8_store_kernel<__bf16>, wave_grid(nt), dim3(256), 0, stream, (const __bf16*)x, ldx, out, rows, cols, nt);
            break;
        case SHAMPOO4_F16:
            S4_LAUNCH(act8_store_kernel<_Float16>, wave_grid(nt), dim3(256), 0, stream, (const _Float16*)x, ldx, out, rows, cols, nt);
            break;
        default:
            S4_LAUNCH(act8_store_kernel<float>, wave_grid(nt), dim3(256), 0, stream, (const float*)x, ldx, out, rows, cols, nt);
    }
    return hipGetLastError();
}

hipError_t launch_act8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols, Act8Ptr in, void* x, int64_t ldx,
                            hipStream_t stream) {
    const int64_t nt = act8_tiles(rows, cols);
    if (nt <= 0) return hipSuccess;
    switch (dtype) {
        case SHAMPOO4_BF16:
            S4_LAUNCH(act8_load_kernel<__bf16>, wave_grid(nt), dim3(256), 0, stream, in, (__bf16*)x, ldx, rows, cols, nt);
            break;
        case SHAMPOO4_F16:
            S4_LAUNCH(act8_load_kernel<_Float16>, wave_grid(nt), dim3(256), 0, stream, in, (_Float16*)x, ldx, rows, cols, nt);
            break;
        default:
            S4_LAUNCH(act8_load_kernel<float>, wave_grid(nt), dim3(256), 0, stream, in, (float*)x, ldx, rows, cols, nt);
    }
    return hipGetLastError();
}

hipError_t launch_activation_forward(int kind, shampoo4_dtype dtype, const ActForward& a, hipStream_t stream) {
    const int64_t nt = act8_tiles(a.rows, a.cols);
    if (nt <= 0) return hipSuccess;
    switch (dtype) {
        case SHAMPOO4_BF16: a.up ? forward_of<__bf16, true>(kind, a, nt, stream) : forward_of<__bf16, false>(kind, a, nt, stream); break;
        case SHAMPOO4_F16: a.up ? forward_of<_Float16, true>(kind, a, nt, stream) : forward_of<_Float16, false>(kind, a, nt, stream); break;
        default: a.up ? forward_of<float, true>(kind, a, nt, stream) : forward_of<float, false>(kind, a, nt, stream);
    }
    return hipGetLastError();
}

hipError_t launch_activation_backward(int kind, shampoo4_dtype dtype, const ActBackward& a, hipStream_t stream) {
    const int64_t nt = act8_tiles(a.rows, a.cols);
    if (nt <= 0) return hipSuccess;
    switch (dtype) {
        case SHAMPOO4_BF16: a.dup ? backward_of<__bf16, true>(kind, a, nt, stream) : backward_of<__bf16, false>(kind, a, nt, stream); break;
        case SHAMPOO4_F16: a.dup ? backward_of<_Float16, true>(kind, a, nt, stream) : backward_of<_Float16, false>(kind, a, nt, stream); break;
        default: a.dup ? backward_of<float, true>(kind, a, nt, stream) : backward_of<float, false>(kind, a, nt, stream);
    }
    return hipGetLastError();
}

}  // namespace s4
