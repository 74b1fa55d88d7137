// Weight gradient G[n, c] = alpha sum_t dY[t, n] X^[t, c] + beta G[n, c] with X^ read from an
// 8-bit checkpoint.
//
// Both operands are contracted over their rows (tokens), so neither has consecutive
// contraction elements in memory.  Tiles are staged in LDS as they lie in memory, token by
// token, in bf16, and gfx950's transposing LDS read (four tokens of sixteen columns a group
// of sixteen lanes) gives each lane the consecutive tokens that a matrix-core operand takes.
// X^ = code * 2^k is a bf16 number exactly, and a bf16 dY is an operand as it stands; an f16
// or f32 dY is split exactly into two or three bf16 pieces, one product each.
#include <algorithm>

#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

typedef short shortx4 __attribute__((ext_vector_type(4)));

constexpr int BM = 128, BN = 128;            // output tile: channels of dY x channels of X
constexpr int KS = 32;                       // tokens a slice: one block of the checkpoint
constexpr int PITCH = 160;                   // LDS row pitch in bf16: 320 bytes, so the four
                                             // token rows of a transposing read are 64 bytes
                                             // apart modulo the 256 bytes of the banks
constexpr int THREADS = 256;                 // 2 x 2 waves of 64 x 64

template <class T>
struct Pieces;
template <>
struct Pieces<__bf16> { static constexpr int N = 1; };
template <>
struct Pieces<_Float16> { static constexpr int N = 2; };
template <>
struct Pieces<float> { static constexpr int N = 3; };

__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// The next piece of eight values: their upper 16 bits, and what is left of them.  An
// infinity leaves nothing.
__device__ __forceinline__ u32x4 take_piece(floatx8& f) {
    u32x4 p;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack_hi(f[2 * i], f[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float hi = __uint_as_float(__float_as_uint(f[i]) & 0xffff0000u);
        f[i] = __builtin_isinf(f[i]) ? 0.f : f[i] - hi;
    }
    return p;
}

template <class T>
__device__ __forceinline__ void split_store(uint16_t* lds, int plane, int at, typename Vec8<T>::Raw r) {
    if constexpr (Pieces<T>::N == 1) {
        *(u32x4*)(lds + at) = r;
    } else {
        floatx8 f = Vec8<T>::get(r);
#pragma unroll
        for (int q = 0; q < Pieces<T>::N; ++q) *(u32x4*)(lds + q * plane + at) = take_piece(f);
    }
}

// Eight consecutive tokens (k0 + 8 (lane / 32) ..) of column n0 + lane % 32.
__device__ __forceinline__ bf16x8 fragment(const uint16_t* lds, int k0, int n0) {
    const int lane = threadIdx.x & 63;
    const uint16_t* p = lds + (k0 + (lane >> 5) * 8 + ((lane >> 2) & 3)) * PITCH + n0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    using L = __attribute__((address_space(3))) shortx4;
    union { shortx4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p);
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p + 4 * PITCH));
    return u.v;
}

template <class T>
__global__ __launch_bounds__(THREADS) void wgrad_kernel(WGrad w, int tiles_m, int64_t rows_per, bool partial) {
    constexpr int NP = Pieces<T>::N;
    constexpr int PLANE = KS * PITCH;
    __shared__ uint16_t lds[(NP + 1) * PLANE];
    uint16_t* la = lds;
    uint16_t* lb = lds + NP * PLANE;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int tile_m = blockIdx.x % tiles_m, tile_n = blockIdx.x / tiles_m;
    const int64_t m0 = (int64_t)tile_m * BM, n0 = (int64_t)tile_n * BN;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per, r1 = min(w.rows, r0 + rows_per);
    const int64_t pitch = act8_pitch(w.cols);
    // staging: thread (row, seg) takes 16 consecutive columns of one token of each tile
    const int srow = tid >> 3, seg = (tid & 7) * 16;
    const int64_t am = m0 + seg, bn = n0 + seg;
    const int an = (int)max((int64_t)0, min((int64_t)16, w.n - am));
    const bool bok = bn < pitch;
    const int wm = (wv & 1) * 64, wn = (wv >> 1) * 64;
    floatx16 acc[2][2] = {};
    for (int64_t k = r0; k < r1; k += KS) {
        typename Vec8<T>::Raw a[2] = {};
        u32x4 c = {}, e = {};
        if (k + srow < r1) {
            const T* p = (const T*)w.dy + (k + srow) * w.lddy + am;
            a[0] = load8_n(p, an);
            a[1] = load8_n(p + 8, max(0, an - 8));
        }
        if (bok) {
            c = ldg((const u32x4*)(w.codes + (k + srow) * pitch + bn));
            e = ldg((const u32x4*)(w.scales + (k / 32) * pitch + bn));
        }
        __syncthreads();
        split_store<T>(la, PLANE, srow * PITCH + seg, a[0]);
        split_store<T>(la, PLANE, srow * PITCH + seg + 8, a[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = act8_scale((e[2 * h + (j >> 2)] >> (8 * (j & 3))) & 0xffu);
            const floatx8 x = act8_values(u32x2{c[2 * h], c[2 * h + 1]}, s);
            u32x4 p;
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = pack_hi(x[2 * j], x[2 * j + 1]);
            *(u32x4*)(lb + srow * PITCH + seg + 8 * h) = p;
        }
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < KS; ks += 16) {
            const bf16x8 b0 = fragment(lb, ks, wn), b1 = fragment(lb, ks, wn + 32);
#pragma unroll
            for (int q = 0; q < NP; ++q)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const bf16x8 av = fragment(la + q * PLANE, ks, wm + 32 * m);
                    acc[m][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, b0, acc[m][0], 0, 0, 0);
                    acc[m][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, b1, acc[m][1], 0, 0, 0);
                }
        }
    }
    float* out = partial ? w.parts + (int64_t)blockIdx.y * w.n * w.cols : w.g;
    const int64_t ld = partial ? w.cols : w.ldg;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t row = m0 + wm + 32 * m + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                const int64_t col = n0 + wn + 32 * n + (lane & 31);
                if (row < w.n && col < w.cols) {
                    float* p = out + row * ld + col;
                    float v = acc[m][n][r];
                    if (!partial) v = w.beta != 0.f ? fmaf(w.alpha, v, w.beta * ldg(p)) : w.alpha * v;
                    stg(p, v);
                }
            }
}

// G = alpha sum_s parts[s] + beta G, the parts in order.
__global__ __launch_bounds__(256) void wgrad_sum_kernel(WGrad w, int splits) {
    const int64_t n = w.n * w.cols;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        float s = 0.f;
        for (int k = 0; k < splits; ++k) s += ldg(w.parts + k * n + i);
        const int64_t r = i / w.cols;
        float* p = w.g + r * w.ldg + (i - r * w.cols);
        stg(p, w.beta != 0.f ? fmaf(w.alpha, s, w.beta * ldg(p)) : w.alpha * s);
    }
}

struct WPlan {
    int64_t tiles_m, tiles_n, rows_per;
    int splits;
};
WPlan wgrad_plan(int64_t rows, int64_t n, int64_t cols) {
    WPlan p;
    p.tiles_m = (n + BM - 1) / BM;
    p.tiles_n = (cols + BN - 1) / BN;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    int64_t s = std::max<int64_t>(1, std::min<int64_t>(512 / std::max<int64_t>(tiles, 1), rows / 256));
    p.rows_per = ((rows + s - 1) / s + KS - 1) / KS * KS;
    p.splits = rows > 0 ? (int)((rows + p.rows_per - 1) / p.rows_per) : 1;
    return p;
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t cols) {
    const WPlan p = wgrad_plan(rows, n, cols);
    return p.splits > 1 ? (size_t)p.splits * n * cols * 4 : 0;
}

hipError_t launch_wgrad(shampoo4_dtype dtype, const WGrad& w, hipStream_t stream) {
    if (w.n <= 0 || w.cols <= 0) return hipSuccess;
    const WPlan p = wgrad_plan(w.rows, w.n, w.cols);
    const dim3 grid((uint32_t)(p.tiles_m * p.tiles_n), (uint32_t)p.splits);
    const bool part = p.splits > 1;
    switch (dtype) {
        case SHAMPOO4_BF16: S4_LAUNCH(wgrad_kernel<__bf16>, grid, dim3(THREADS), 0, stream, w, (int)p.tiles_m, p.rows_per, part); break;
        case SHAMPOO4_F16: S4_LAUNCH(wgrad_kernel<_Float16>, grid, dim3(THREADS), 0, stream, w, (int)p.tiles_m, p.rows_per, part); break;
        default: S4_LAUNCH(wgrad_kernel<float>, grid, dim3(THREADS), 0, stream, w, (int)p.tiles_m, p.rows_per, part);
    }
    if (part) {
        const dim3 sg((uint32_t)std::min<int64_t>((w.n * w.cols + 255) / 256, 4096));
        S4_LAUNCH(wgrad_sum_kernel, sg, dim3(256), 0, stream, w, p.splits);
    }
    return hipGetLastError();
}

}  // namespace s4
