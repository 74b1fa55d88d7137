// The ends of a residual block (shampoo4_train.h): norm behind the block, dropout, gate, residual sum
// and the norm before the next block in one pass, and their gradients in one pass and a short
// launch that joins the sums over rows.
//
// A row is held in registers by one wave or by the waves of a workgroup, as it lies in memory (raw
// 16-bit values stay packed), so every input is read once; the row's sums go across lanes without LDS
// and across waves through it.
#include <algorithm>
#include <type_traits>

#include "random.hpp"
#include "train.hpp"

namespace s4 {

namespace {

// The sum over a wave, the same bits in every lane (each step adds a pair both ways).
__device__ __forceinline__ float wave_sum(float v) {
    const auto ror = [](float x, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    v += ror(v, std::integral_constant<int, 0x128>{});
    v += ror(v, std::integral_constant<int, 0x124>{});
    v += ror(v, std::integral_constant<int, 0x122>{});
    v += ror(v, std::integral_constant<int, 0x121>{});
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
    m = max16(m);
    const auto h = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(h[0], h[1]);
    const auto w = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(w[0], w[1]);
}

// Sums and maxima over the WPR waves of a row.  Consecutive reductions of a kernel take other
// slots: a slot is written again only after a barrier that follows its last read.
template <int WPR>
struct Row {
    float (*red)[WPR];
    int wave;
    __device__ __forceinline__ float sum(float v, int slot) const {
        v = wave_sum(v);
        if constexpr (WPR > 1) {
            red[slot][wave] = v;
            __syncthreads();
            v = red[slot][0];
#pragma unroll
            for (int i = 1; i < WPR; ++i) v += red[slot][i];
        }
        return v;
    }
    __device__ __forceinline__ uint32_t largest(uint32_t m, int slot) const {
        m = wave_max(m);
        if constexpr (WPR > 1) {
            red[slot][wave] = __uint_as_float(m);
            __syncthreads();
            m = 0;
#pragma unroll
            for (int i = 0; i < WPR; ++i) m = max(m, __float_as_uint(red[slot][i]));
        }
        return m;
    }
};

// A thread's columns: vectors of eight, 8 THREADS apart.
template <int THREADS, int VPT>
struct Cols {
    int cols, t;
    bool whole;               // rows of whole vectors
    __device__ __forceinline__ int at(int i) const { return (t + i * THREADS) * 8; }
    __device__ __forceinline__ int n(int i) const { return max(0, min(8, cols - at(i))); }

    template <class T>
    __device__ __forceinline__ void load(typename Vec8<T>::Raw (&r)[VPT], const T* row) const {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (whole) {
                r[i] = load8(row + min(at(i), cols - 8));
                r[i] &= at(i) < cols ? 0xffffffffu : 0u;
            } else {
                r[i] = load8_edge(row, at(i), cols);
            }
        }
    }
    template <class T>
    __device__ __forceinline__ void store(T* row, int i, floatx8 v) const {
        if (n(i)) store8_n(row + at(i), Vec8<T>::put(v), n(i));
    }
    // eight values of a vector that every row shares; `none` where there is no vector
    __device__ __forceinline__ floatx8 shared(const float* p, int i, float none) const {
        floatx8 f;
        if (!p) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = none;
            return f;
        }
        return Vec8<float>::get(load8_edge(p, at(i), cols));
    }
};

// 1 / sqrt(mean v^2 + eps) of a row whose sum of squares is ss.  Where that leaves fp32's range the
// squares are taken again, of the row times 2^-k that brings its largest value to [1, 2).  (What
// squares lose below 2^-149 is nothing beside eps >= 1e-30.)
template <class T, int WPR, int VPT>
__device__ __forceinline__ float reciprocal_norm(const typename Vec8<T>::Raw (&r)[VPT], float ss, int cols, float eps,
                                                 const Row<WPR>& row) {
    float scale = 1.f;
    if (!(ss < 0x1p126f)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) m = max(m, magnitude(Vec8<T>::get(r[i])));
        m = row.largest(m, 2);
        if (m < 0x7f800000u) {
            scale = __uint_as_float((254u - min(m >> 23, 253u)) << 23);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const floatx8 f = Vec8<T>::get(r[i]) * scale;
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
            }
            ss = row.sum(s, 3);
        }
    }
    return scale / sqrtf(ss / (float)cols + eps * scale * scale);
}

constexpr int rows_of(int wpr) { return wpr == 1 ? 4 : 1; }              // of a workgroup
constexpr int threads_of(int wpr) { return 64 * wpr * rows_of(wpr); }

template <class T, int WPR, int VPT>
__global__ __launch_bounds__(threads_of(WPR)) void block_forward_kernel(BlockForward a, Drop d) {
    constexpr int THREADS = 64 * WPR;
    __shared__ float red[4][WPR];
    const int64_t row = (int64_t)blockIdx.x * rows_of(WPR) + (WPR == 1 ? threadIdx.x >> 6 : 0);
    if (row >= a.rows) return;                               // a wave that has its row alone
    const int t = threadIdx.x % THREADS, cols = (int)a.cols;
    const Row<WPR> sums{red, t >> 6};
    const Cols<THREADS, VPT> c{cols, t, (cols & 7) == 0};
    using Raw = typename Vec8<T>::Raw;
    Raw x[VPT], h[VPT], g[VPT];
    c.template load<T>(x, (const T*)a.x + row * a.ldx);
    if (a.h) {
        c.template load<T>(h, (const T*)a.h + row * a.ldh);
        if (a.gate_rows) c.template load<T>(g, (const T*)a.gate + row * a.ldgate);
        float hr = 1.f;
        if (a.post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const floatx8 f = Vec8<T>::get(h[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
            }
            hr = reciprocal_norm<T, WPR, VPT>(h, sums.sum(ss, 0), cols, a.eps, sums);
            if (a.h_rstd && t == 0) stg(a.h_rstd + row, hr);
        }
        const uint64_t call = drop_call(d);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            floatx8 z = Vec8<T>::get(h[i]);
            if (a.post) z = z * hr * c.shared(a.post, i, 1.f);
            if (d.threshold) z = drop8(z, drop_keep8(d, call, row, c.at(i) >> 3), d.scale);
            if (a.gate_rows)
                z *= Vec8<T>::get(g[i]);
            else if (a.gate)
                z *= c.shared((const float*)a.gate, i, 1.f);
            const floatx8 v = Vec8<T>::get(x[i]) * a.rho + z;
            x[i] = Vec8<T>::put(v);
            if (c.n(i)) store8_n((T*)a.out + row * a.ldout + c.at(i), x[i], c.n(i));
        }
    }
    if (!a.weight) return;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const floatx8 f = Vec8<T>::get(x[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
    const float r = reciprocal_norm<T, WPR, VPT>(x, sums.sum(ss, 1), cols, a.eps, sums);
    if (a.rstd && t == 0) stg(a.rstd + row, r);
    const int64_t pitch = fp8_pitch(cols), sp = fp8_scale_pitch(cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const Raw y = Vec8<T>::put(Vec8<T>::get(x[i]) * r * c.shared(a.weight, i, 0.f));
        if (a.y && c.n(i)) store8_n((T*)a.y + row * a.ldy + c.at(i), y, c.n(i));
        if (a.yc) {
            const floatx8 f = Vec8<T>::get(y);
            const uint32_t e = fp8_exponent(max16(magnitude(f)));
            if (c.at(i) < pitch) stg((u32x2*)(a.yc + row * pitch + c.at(i)), Fp8Block(e).codes(f));
            if ((t & 15) == 0 && c.at(i) >> 7 < sp) stg(a.ys + row * sp + (c.at(i) >> 7), (uint8_t)e);
        }
    }
}

// Workgroups of the backward kernel: two a CU, each with a fixed set of rows whose sums it keeps.
constexpr int64_t BACK_GROUPS = 512;
int64_t back_groups(int64_t rows, int wpr) {
    return std::min<int64_t>((rows + rows_of(wpr) - 1) / rows_of(wpr), BACK_GROUPS);
}

template <class T, int WPR, int VPT>
__global__ __launch_bounds__(threads_of(WPR)) void block_backward_kernel(BlockBackward a, Drop d) {
    constexpr int THREADS = 64 * WPR, PER = rows_of(WPR);
    __shared__ float red[2][WPR];
    const int t = threadIdx.x % THREADS, cols = (int)a.cols;
    const Row<WPR> sums{red, t >> 6};
    const Cols<THREADS, VPT> c{cols, t, (cols & 7) == 0};
    using Raw = typename Vec8<T>::Raw;
    const float inv = 1.f / (float)cols;
    const uint64_t call = drop_call(d);
    floatx8 w[VPT], p[VPT], gv[VPT], dw[VPT] = {}, dp[VPT] = {}, dg[VPT] = {};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        w[i] = c.shared(a.weight, i, 0.f);
        p[i] = c.shared(a.post, i, 1.f);
        gv[i] = c.shared(a.gate_rows ? nullptr : (const float*)a.gate, i, 1.f);
    }
    for (int64_t row = (int64_t)blockIdx.x * PER + (WPR == 1 ? threadIdx.x >> 6 : 0); row < a.rows;
         row += (int64_t)gridDim.x * PER) {
        Raw dy[VPT] = {}, dr[VPT] = {}, x[VPT] = {}, h[VPT] = {}, g[VPT] = {};
        float rx = 0.f, hr = 1.f;
        if (a.weight) {
            c.template load<T>(dy, (const T*)a.dy + row * a.lddy);
            c.template load<T>(x, (const T*)a.x + row * a.ldx);
            rx = ldg(a.rstd + row);
        }
        if (a.dres) c.template load<T>(dr, (const T*)a.dres + row * a.lddres);
        if (a.h) {
            c.template load<T>(h, (const T*)a.h + row * a.ldh);
            if (a.post) hr = ldg(a.h_rstd + row);
            if (a.gate_rows) c.template load<T>(g, (const T*)a.gate + row * a.ldgate);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const floatx8 xh = Vec8<T>::get(x[i]) * rx, y = Vec8<T>::get(dy[i]);
            const floatx8 ty = y * w[i];
            dw[i] += y * xh;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(ty[j], xh[j], s);
        }
        s = sums.sum(s, 0) * inv;
        floatx8 u[VPT];
        float s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const floatx8 xh = Vec8<T>::get(x[i]) * rx, ty = Vec8<T>::get(dy[i]) * w[i];
            const floatx8 gx = Vec8<T>::get(dr[i]) + (ty - xh * s) * rx;
            if (a.dx) c.template store<T>((T*)a.dx + row * a.lddx, i, gx * a.rho);
            if (!a.h) continue;
            const floatx8 hh = Vec8<T>::get(h[i]) * hr;
            const uint32_t keep = d.threshold ? drop_keep8(d, call, row, c.at(i) >> 3) : 0xffu;
            const floatx8 z = gx * drop8(hh * p[i], keep, d.scale);
            if (a.gate_rows) {
                if (a.dgate) c.template store<T>((T*)a.dgate + row * a.lddgate, i, z);
            } else {
                dg[i] += z;
            }
            const floatx8 dn = drop8(gx * (a.gate_rows ? Vec8<T>::get(g[i]) : gv[i]), keep, d.scale);
            dp[i] += dn * hh;
            u[i] = dn * p[i];
#pragma unroll
            for (int j = 0; j < 8; ++j) s2 = fmaf(u[i][j], hh[j], s2);
        }
        s2 = sums.sum(s2, 1) * inv;
        if (!a.h || !a.dh) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (a.post) u[i] = (u[i] - Vec8<T>::get(h[i]) * hr * s2) * hr;
            c.template store<T>((T*)a.dh + row * a.lddh, i, u[i]);
        }
    }
    if (!a.parts) return;
    float* out = a.parts + (int64_t)blockIdx.x * 3 * cols;
    const auto write = [&](float* to, floatx8 v, int i) {
        if (c.n(i)) store8_n(to + c.at(i), Vec8<float>::put(v), c.n(i));
    };
    if constexpr (PER == 1) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            write(out, dw[i], i);
            write(out + cols, dp[i], i);
            write(out + 2 * cols, dg[i], i);
        }
    } else {
        // the waves' sums, wave by wave
        __shared__ float all[3][64 * VPT * 8];
        for (int k = 0; k < PER; ++k) {
            if ((int)(threadIdx.x >> 6) == k)
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int at = c.at(i) + j;
                        all[0][at] = k ? all[0][at] + dw[i][j] : dw[i][j];
                        all[1][at] = k ? all[1][at] + dp[i][j] : dp[i][j];
                        all[2][at] = k ? all[2][at] + dg[i][j] : dg[i][j];
                    }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < 3 * cols; i += 64 * PER) stg(out + i, all[i / cols][i % cols]);
    }
}

// out[k][c] = sum over groups of parts[group][k][c], in four runs of groups that are added in order.
struct Join {
    float* out[3];
};
__global__ __launch_bounds__(256) void block_join_kernel(const float* parts, Join j, int groups, int cols) {
    __shared__ float run[4][64];
    float* out = j.out[blockIdx.y];
    if (!out) return;
    const int l = threadIdx.x & 63, q = threadIdx.x >> 6, col = blockIdx.x * 64 + l;
    float s = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int g = q; g < groups; g += 4) s += ldg(parts + ((int64_t)g * 3 + blockIdx.y) * cols + col);
    run[q][l] = s;
    __syncthreads();
    if (q == 0 && col < cols) stg(out + col, ((run[0][l] + run[1][l]) + run[2][l]) + run[3][l]);
}

// Waves and vectors a row takes: up to two vectors a lane (their registers, with the sums over rows, are
// what two waves a SIMD leave), then more waves.
int waves_of(int64_t cols) { return cols <= 1024 ? 1 : cols <= 4096 ? 4 : cols <= 8192 ? 8 : 16; }

template <class F>
void by_row(int64_t cols, F f) {
    const auto vectors = [&](auto w) {
        if (cols <= 512 * decltype(w)::value)
            f(w, std::integral_constant<int, 1>{});
        else
            f(w, std::integral_constant<int, 2>{});
    };
    switch (waves_of(cols)) {
        case 1: return vectors(std::integral_constant<int, 1>{});
        case 4: return vectors(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
        default: return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
    }
}

}  // namespace

hipError_t launch_block_forward(shampoo4_dtype dtype, const BlockForward& a, const Drop& d, hipStream_t stream) {
    if (a.rows <= 0) return hipSuccess;
    by_type(dtype, [&](auto t) {
        using T = decltype(t);
        by_row(a.cols, [&](auto w, auto v) {
            constexpr int W = decltype(w)::value, V = decltype(v)::value;
            S4_LAUNCH((block_forward_kernel<T, W, V>), dim3((uint32_t)((a.rows + rows_of(W) - 1) / rows_of(W))),
                      dim3(threads_of(W)), 0, stream, a, d);
        });
    });
    return hipGetLastError();
}

size_t block_workspace_bytes(int64_t rows, int64_t cols) {
    return (size_t)back_groups(rows, waves_of(cols)) * 3 * cols * 4;
}

hipError_t launch_block_backward(shampoo4_dtype dtype, const BlockBackward& given, const Drop& d, hipStream_t stream) {
    BlockBackward a = given;
    const Join j{{a.dweight, a.dpost, a.gate_rows ? nullptr : (float*)a.dgate}};
    const bool join = j.out[0] || j.out[1] || j.out[2];
    if (!join) a.parts = nullptr;
    const int64_t groups = back_groups(a.rows, waves_of(a.cols));
    if (groups > 0)
        by_type(dtype, [&](auto t) {
            using T = decltype(t);
            by_row(a.cols, [&](auto w, auto v) {
                constexpr int W = decltype(w)::value, V = decltype(v)::value;
                S4_LAUNCH((block_backward_kernel<T, W, V>), dim3((uint32_t)groups), dim3(threads_of(W)), 0, stream, a, d);
            });
        });
    if (join)
        S4_LAUNCH(block_join_kernel, dim3((uint32_t)((a.cols + 63) / 64), 3), dim3(256), 0, stream, a.parts, j, (int)groups,
                  (int)a.cols);
    return hipGetLastError();
}

}  // namespace s4
