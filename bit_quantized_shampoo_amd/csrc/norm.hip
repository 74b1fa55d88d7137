// The ends of a residual block (shampoo4_train.h): norm behind the block, dropout, gate, residual sum
// and the norm before the next block in one pass, and their gradients in one pass and a short
// launch that joins the sums over rows.
//
// A row is held in registers by one wave or by the waves of a workgroup, as it lies in memory (raw
// 16-bit values stay packed), so every input is read once; the row's sums go across lanes without LDS
// and across waves through it.
//
// Bytes bound both.  16384 x 4096 bf16, all options, dropout 0.1: forward 133 us, backward 191, without dropout
// 119 and 164, where a copy of as many bytes takes 105 and 157.  Dropout's generator, 20 wide multiplications for
// eight columns, is most of that difference: it runs while the row is on its way, but with the row's other
// arithmetic it is about as long as the row's loads.
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

// Sums and maxima over the WPR waves of a row.  A reduction's slot is written again only after a
// barrier that follows its last read: the reductions of a row have slots of their own, and rows
// take turns with two sets of them.
template <int WPR>
struct Row {
    float (*red)[WPR];
    int wave;
    // A sum in three steps, so that several share a barrier.
    __device__ __forceinline__ float partial(float v, int slot) const {
        v = wave_sum(v);
        if constexpr (WPR > 1) red[slot][wave] = v;
        return v;
    }
    __device__ __forceinline__ void meet() const {
        // of LDS alone: a row's loads that are on their way, and stores, are not waited for
        if constexpr (WPR > 1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    __device__ __forceinline__ float total(float v, int slot) const {
        if constexpr (WPR > 1) {
            v = red[slot][0];
#pragma unroll
            for (int i = 1; i < WPR; ++i) v += red[slot][i];
        }
        return v;
    }
    __device__ __forceinline__ float sum(float v, int slot) const {
        v = partial(v, slot);
        meet();
        return total(v, slot);
    }
    __device__ __forceinline__ uint32_t largest(uint32_t m, int slot) const {
        m = wave_max(m);
        if constexpr (WPR > 1) {
            red[slot][wave] = __uint_as_float(m);
            meet();
            m = 0;
#pragma unroll
            for (int i = 0; i < WPR; ++i) m = max(m, __float_as_uint(red[slot][i]));
        }
        return m;
    }
};

// A thread's columns: vectors of eight, 8 THREADS apart.  Rows are addressed by the wave (their
// pointers are in scalar registers), columns by 32-bit offsets.
template <int THREADS, int VPT>
struct Cols {
    int cols, t, col0;        // columns of the row, the thread, the first column of all threads
    bool whole;               // rows of whole vectors
    __device__ __forceinline__ Cols(int cols_, int t_, int col0_ = 0) : cols(cols_), t(t_), col0(col0_), whole((cols_ & 7) == 0) {}
    __device__ __forceinline__ int at(int i) const { return col0 + (t + i * THREADS) * 8; }
    __device__ __forceinline__ int n(int i) const { return max(0, min(8, cols - at(i))); }

    // No load is under a lane's own condition: a vector past the row's end is loaded eight from it.  What was
    // loaded is finished where it is used, so that loads are not waited for one by one: shifted, or
    // masked.
    template <class T>
    __device__ __forceinline__ typename Vec8<T>::Raw vector(const T* row, int i) const {
        if (cols < 8) return load8_edge(row, at(i), cols);
        return load8((const T*)((const char*)row + (uint32_t)min(at(i), cols - 8) * (uint32_t)sizeof(T)));
    }
    template <class T>
    __device__ __forceinline__ void finish(typename Vec8<T>::Raw& r, int i) const {
        if (whole)
            r &= at(i) < cols ? 0xffffffffu : 0u;
        else if (cols >= 8)
            r = shift_down<T>(r, min(8, max(0, at(i) - (cols - 8))));
    }
    template <class T>
    __device__ __forceinline__ void store_raw(T* row, int i, typename Vec8<T>::Raw v) const {
        if (at(i) >= cols) return;
        T* p = (T*)((char*)row + (uint32_t)at(i) * (uint32_t)sizeof(T));
        if (whole)
            store8(p, v);
        else
            store8_n(p, v, n(i));
    }
    template <class T>
    __device__ __forceinline__ void store(T* row, int i, floatx8 v) const {
        store_raw(row, i, Vec8<T>::put(v));
    }
    // Zeros past the row's end.
    __device__ __forceinline__ floatx8 own(floatx8 v, int i) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at(i) + j < cols ? v[j] : 0.f;
        return v;
    }
    // Eight values of a vector that every row shares, and how they are finished; ones where there is no
    // vector.
    __device__ __forceinline__ u32x8 shared(const float* p, int i) const {
        if (p) return vector(p, i);
        u32x8 one;
#pragma unroll
        for (int j = 0; j < 8; ++j) one[j] = 0x3f800000u;
        return one;
    }
    __device__ __forceinline__ floatx8 finish_shared(const float* p, u32x8 r, int i) const {
        if (p) finish<float>(r, i);
        return Vec8<float>::get(r);
    }
};

// 1 / sqrt(mean v^2 + eps) of a row whose sum of squares is ss.  Where that leaves fp32's range the
// squares are taken again, of the row times 2^-k that brings its largest value to [1, 2).  (What
// squares lose below 2^-149 is nothing beside eps >= 1e-30.)
template <class T, int WPR, int VPT>
__device__ __forceinline__ float reciprocal_norm(const typename Vec8<T>::Raw (&r)[VPT], float ss, int cols, float eps,
                                                 const Row<WPR>& row, int slot) {
    float scale = 1.f;
    if (!(ss < 0x1p126f)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) m = max(m, magnitude(Vec8<T>::get(r[i])));
        m = row.largest(m, slot);
        if (m < 0x7f800000u) {
            scale = __uint_as_float((254u - min(m >> 23, 253u)) << 23);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const floatx8 f = Vec8<T>::get(r[i]) * scale;
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
            }
            ss = row.sum(s, slot + 1);
        }
    }
    return scale / sqrtf(ss / (float)cols + eps * scale * scale);
}

__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

constexpr int rows_of(int wpr) { return wpr == 1 ? 4 : 1; }              // of a workgroup
constexpr int threads_of(int wpr) { return 64 * wpr * rows_of(wpr); }

// The rows of a workgroup of the backward kernel (of each of its four waves, where a row is a wave's) are
// first, first + stride, and so on.
struct Rows {
    int64_t first, stride;
};
template <int WPR>
__device__ __forceinline__ Rows rows_here() {
    return {(int64_t)blockIdx.x * rows_of(WPR) + (WPR == 1 ? wave_index() : 0), (int64_t)gridDim.x * rows_of(WPR)};
}
// A row's number that the compiler makes addresses of where they are used, in scalar registers, rather
// than keep one for each stream and lane.
__device__ __forceinline__ int64_t here(int64_t row) {
    asm volatile("" : "+s"(row));
    return row;
}

template <class T, int WPR, int VPT, bool DROP, bool TOKEN>
__global__ __launch_bounds__(threads_of(WPR)) void block_forward_kernel(BlockForward a, Drop d) {
    constexpr int THREADS = 64 * WPR;
    __shared__ float red[6][WPR];
    const int64_t row = (int64_t)blockIdx.x * rows_of(WPR) + (WPR == 1 ? wave_index() : 0);
    if (row >= a.rows) return;                               // a wave that has its row alone
    const int t = threadIdx.x % THREADS, cols = (int)a.cols;
    const Row<WPR> sums{red, t >> 6};
    const Cols<THREADS, VPT> c(cols, t);
    using Raw = typename Vec8<T>::Raw;
    Raw x[VPT], h[VPT] = {}, g[VPT] = {};
    u32x8 rw[VPT], rp[VPT], rg[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        x[i] = c.vector((const T*)a.x + row * a.ldx, i);
        if (a.h) {
            h[i] = c.vector((const T*)a.h + row * a.ldh, i);
            if (TOKEN) g[i] = c.vector((const T*)a.gate + row * a.ldgate, i);
        }
    }
    // on their way with the row: behind its sums they would be waited for
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        rp[i] = c.shared(a.post, i);
        if (!TOKEN) rg[i] = c.shared((const float*)a.gate, i);
        rw[i] = c.shared(a.weight, i);
    }
    Keep keep[DROP ? VPT : 1];
    if (DROP) {                                              // while all that is on its way
        const uint64_t call = drop_call(d);
#pragma unroll
        for (int i = 0; i < VPT; ++i) keep[i] = drop_keep8(d, call, row, c.at(i) >> 3);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < VPT; ++i) c.template finish<T>(x[i], i);
    if (a.h) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            c.template finish<T>(h[i], i);
            if (TOKEN) c.template finish<T>(g[i], i);
        }
        float hr = 1.f;
        if (a.post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const floatx8 f = Vec8<T>::get(h[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
            }
            hr = reciprocal_norm<T, WPR, VPT>(h, sums.sum(ss, 0), cols, a.eps, sums, 2);
            if (a.h_rstd && t == 0) stg(a.h_rstd + row, hr);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            floatx8 z = Vec8<T>::get(h[i]) * (DROP ? hr * d.scale : hr) * c.finish_shared(a.post, rp[i], i);
            if (DROP) {
                z = drop8(z, keep[i], d);
                // A norm that is NaN makes it of the zeros past the row's end too.  Where all of the row's own are dropped
                // those must not reach its sum of squares (else the row is NaN by what is its own).
                if (hr != hr) z = c.own(z, i);
            }
            if (TOKEN)
                z *= Vec8<T>::get(g[i]);
            else
                z *= c.finish_shared((const float*)a.gate, rg[i], i);
            x[i] = Vec8<T>::put(Vec8<T>::get(x[i]) * a.rho + z);
            c.template store_raw<T>((T*)a.out + row * a.ldout, i, x[i]);
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
    const float rx = reciprocal_norm<T, WPR, VPT>(x, sums.sum(ss, 1), cols, a.eps, sums, 4);
    if (a.rstd && t == 0) stg(a.rstd + row, rx);
    const int64_t pitch = fp8_pitch(cols), sp = fp8_scale_pitch(cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const Raw y = Vec8<T>::put(Vec8<T>::get(x[i]) * rx * c.finish_shared(a.weight, rw[i], i));
        if (a.y) c.template store_raw<T>((T*)a.y + row * a.ldy, i, y);
        if (a.yc) {
            const floatx8 f = Vec8<T>::get(y);
            // past the row's end a factor that is NaN has made NaN of zeros, which are no part of a block
            const uint32_t e = fp8_exponent(max16(c.at(i) < cols ? magnitude(f) : 0u));
            if (c.at(i) < pitch) stg((u32x2*)(a.yc + row * pitch + c.at(i)), Fp8Block(e).codes(f));
            if ((t & 15) == 0 && c.at(i) >> 7 < sp) stg(a.ys + row * sp + (c.at(i) >> 7), (uint8_t)e);
        }
    }
}

// A whole pass (WHOLE), or, for rows of more than BLOCK_WIDE columns, two: the rows' two sums (SUMS), and the rest by
// ranges of columns, with those sums given (REST): 10 values an element move instead of 6.  Registers hold two
// vectors a lane beside the factors and sums over rows that belong to them; three were spilled, and
// 4096 x 16384 bf16 in one pass took 2940 us, in two 290-296.
enum Pass { WHOLE, SUMS, REST };
template <class T, int WPR, int VPT, bool DROP, bool TOKEN, Pass PASS = WHOLE>
__global__ __launch_bounds__(threads_of(WPR), 2) void block_backward_kernel(BlockBackward a, Drop d) {
    constexpr int THREADS = 64 * WPR, PER = rows_of(WPR);
    constexpr bool AGAIN = PASS == SUMS, AHEAD = VPT == 1;   // a vector at a time; the next row beside this one
    __shared__ float red[6][WPR];
    const int t = threadIdx.x % THREADS, cols = (int)a.cols;
    const Row<WPR> sums{red, t >> 6};
    const Cols<THREADS, VPT> c(cols, t, PASS == REST ? (int)blockIdx.y * (THREADS * VPT * 8) : 0);
    using Raw = typename Vec8<T>::Raw;
    const Rows rows = rows_here<WPR>();
    const float inv = 1.f / (float)cols;
    const uint64_t call = drop_call(d);
    struct In {
        Raw dy, dr, x, h, g;
    };
    const auto load = [&](int64_t row, int i) {
        In in = {};
        if (a.weight) {
            in.dy = c.vector((const T*)a.dy + row * a.lddy, i);
            in.x = c.vector((const T*)a.x + row * a.ldx, i);
        }
        if (a.dres) in.dr = c.vector((const T*)a.dres + row * a.lddres, i);
        if (a.h) {
            in.h = c.vector((const T*)a.h + row * a.ldh, i);
            if (TOKEN) in.g = c.vector((const T*)a.gate + row * a.ldgate, i);
        }
        return in;
    };
    const auto finish = [&](In& in, int i) {
        c.template finish<T>(in.dy, i);
        c.template finish<T>(in.x, i);
        c.template finish<T>(in.dr, i);
        c.template finish<T>(in.h, i);
        if (TOKEN) c.template finish<T>(in.g, i);
    };
    struct Factors {
        float x, h;
    };
    const auto factors = [&](int64_t row) {
        return Factors{a.weight ? ldg(a.rstd + row) : 0.f, a.h && a.post ? ldg(a.h_rstd + row) : 1.f};
    };
    struct Shared {
        floatx8 w, p, g;
    };
    // What is kept of dropout is scaled by way of the gate (a gate by element is scaled itself) and of the sums.
    const float drop_scale = DROP ? d.scale : 1.f;
    const float* gate = TOKEN ? nullptr : (const float*)a.gate;
    const auto shared = [&](int i) {
        const float *pw = a.weight, *pp = a.post, *pg = gate;
        if (AGAIN) asm volatile("" : "+s"(pw), "+s"(pp), "+s"(pg));      // not kept from one row for the next
        const u32x8 w = c.shared(pw, i), p = c.shared(pp, i), g = c.shared(pg, i);
        return Shared{c.finish_shared(pw, w, i), c.finish_shared(pp, p, i), c.finish_shared(pg, g, i) * (TOKEN ? 1.f : drop_scale)};
    };
    In now[AGAIN ? 1 : VPT], next[AHEAD ? VPT : 1];
    Factors f_now = {}, f_next = {};
    Shared vec[AGAIN ? 1 : VPT];
    if (AHEAD && rows.first < a.rows) {
        f_next = factors(rows.first);
        next[0] = load(rows.first, 0);
    }
    if (!AGAIN)
#pragma unroll
        for (int i = 0; i < VPT; ++i) vec[i] = shared(i);
    // A vector gate and the weight behind the block share one sum, da = sum drop(g) hh: dgate = da post, dpost = da gate.
    floatx8 dw[VPT] = {}, da[VPT] = {};
    int set = 0;
    for (int64_t r = rows.first; r < a.rows; r += rows.stride, set ^= 3) {
        const int64_t row = here(r);
        Keep keep[DROP && !AGAIN ? VPT : 1];
        const auto numbers = [&]() {                         // while the row is on its way
            if (DROP)
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    keep[i] = drop_keep8(d, call, row, c.at(i) >> 3);
                    __builtin_amdgcn_sched_barrier(0);
                }
            __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (AHEAD) {
            numbers();
            now[0] = next[0];
            finish(now[0], 0);
            f_now = f_next;
            if (row + rows.stride < a.rows) {                // the next row is on its way while this one is worked on
                f_next = factors(row + rows.stride);
                next[0] = load(row + rows.stride, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        } else {
            f_now = factors(row);
            if (!AGAIN)
#pragma unroll
                for (int i = 0; i < VPT; ++i) now[i] = load(row, i);
            if constexpr (!AGAIN) {
                numbers();
#pragma unroll
                for (int i = 0; i < VPT; ++i) finish(now[i], i);
            }
        }
        const float rx = f_now.x, hr = f_now.h;
        // One reduction for both norms: mean(u hh) = sum q (dres + rstd (t - xh s)) is linear in s = mean(t xh), with
        // q = drop(gate post) hh the same for every term.
        float s = 0.f, qa = 0.f, qb = 0.f;
#pragma unroll(AGAIN ? 1 : VPT)
        for (int i = 0; i < (PASS == REST ? 0 : VPT); ++i) {
            if (AGAIN) {
                now[0] = load(row, i);
                vec[0] = shared(i);
                if (DROP) keep[0] = drop_keep8(d, call, row, c.at(i) >> 3);
                finish(now[0], i);
            }
            In& in = now[AGAIN ? 0 : i];
            const Shared& v = vec[AGAIN ? 0 : i];
            const floatx8 xh = Vec8<T>::get(in.x) * rx, ty = Vec8<T>::get(in.dy) * v.w;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(ty[j], xh[j], s);
            if (a.post) {
                floatx8 q = Vec8<T>::get(in.h) * hr * v.p;
                if (TOKEN)
                    q *= Vec8<T>::get(in.g);
                else
                    q *= v.g;
                if (DROP) q = drop8(q, keep[AGAIN ? 0 : i], d);
                const floatx8 dr = Vec8<T>::get(in.dr);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    qa = fmaf(q[j], fmaf(ty[j], rx, dr[j]), qa);
                    qb = fmaf(q[j], xh[j], qb);
                }
            }
            unpack_again(in.x);
            unpack_again(in.dy);
            unpack_again(in.dr);
            unpack_again(in.h);
            unpack_again(in.g);
            if (DROP) unpack_again(keep[AGAIN ? 0 : i].w);
            if (VPT > 1) __builtin_amdgcn_sched_barrier(0);
        }
        float s2 = 0.f;
        if constexpr (PASS == REST) {
            s = ldg(a.sums + 2 * row);
            s2 = ldg(a.sums + 2 * row + 1);
        } else {
            s = sums.partial(s, set);
            if (a.post) {
                qa = sums.partial(qa, set + 1);
                qb = sums.partial(qb, set + 2);
            }
            sums.meet();
            s = sums.total(s, set) * inv * rx;               // rstd mean(t xh), and h_rstd mean(u hh)
            if (a.post) s2 = (sums.total(qa, set + 1) - s * sums.total(qb, set + 2)) * inv * (TOKEN ? hr * drop_scale : hr);
        }
        if constexpr (PASS == SUMS) {
            if (t == 0) {
                stg(a.sums + 2 * row, s);
                stg(a.sums + 2 * row + 1, s2);
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const In& in = now[AGAIN ? 0 : i];
            const Shared& v = vec[AGAIN ? 0 : i];
            const floatx8 xh = Vec8<T>::get(in.x) * rx, y = Vec8<T>::get(in.dy);
            floatx8 gx = Vec8<T>::get(in.dr);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(y[j], xh[j], dw[i][j]);
                gx[j] = fmaf(xh[j], -s, fmaf(y[j] * v.w[j], rx, gx[j]));
            }
            if (a.dx) c.template store<T>((T*)a.dx + row * a.lddx, i, gx * a.rho);
            if (a.h) {
                floatx8 hh = Vec8<T>::get(in.h) * hr;
                if (DROP) {
                    gx = drop8(gx, keep[i], d);              // dropped: no gradient
                    if (!a.post) hh = drop8(hh, keep[i], d); // and h may be anything
                }
                if (TOKEN) {
                    gx *= drop_scale;
                    if (a.dgate) c.template store<T>((T*)a.dgate + row * a.lddgate, i, gx * (hh * v.p));
                    gx *= Vec8<T>::get(in.g);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) da[i][j] = fmaf(gx[j], hh[j], da[i][j]);
                if (!TOKEN) gx *= v.g;
                if (a.post) {
                    // dh = rstd (u - hh mean(u hh))
#pragma unroll
                    for (int j = 0; j < 8; ++j) gx[j] = fmaf(gx[j] * v.p[j], hr, -hh[j] * s2);
                }
                if (a.dh) c.template store<T>((T*)a.dh + row * a.lddh, i, gx);
            }
            if (VPT > 1) __builtin_amdgcn_sched_barrier(0);  // one vector's values at a time in registers
        }
    }
    if (PASS == SUMS || !a.parts) return;
    const auto dp = [&](int i) { return TOKEN ? da[i] : da[i] * vec[i].g; };
    const auto dg = [&](int i) { return da[i] * (vec[i].p * drop_scale); };
    float* out = a.parts + (int64_t)blockIdx.x * 3 * cols;
    if constexpr (PER == 1) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (a.dweight) c.template store<float>(out, i, dw[i]);
            if (a.dpost) c.template store<float>(out + cols, i, dp(i));
            if (!TOKEN && a.dgate) c.template store<float>(out + 2 * cols, i, dg(i));
        }
    } else {
        // the waves' sums, wave by wave
        __shared__ float all[3][64 * VPT * 8];
        for (int k = 0; k < PER; ++k) {
            if ((int)(threadIdx.x >> 6) == k)
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const floatx8 p = dp(i), g = dg(i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int at = c.at(i) + j;
                        all[0][at] = k ? all[0][at] + dw[i][j] : dw[i][j];
                        all[1][at] = k ? all[1][at] + p[j] : p[j];
                        all[2][at] = k ? all[2][at] + g[j] : g[j];
                    }
                }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < 3 * cols; i += 64 * PER) stg(out + i, all[i / cols][i % cols]);
    }
}

// out[k][c] = sum over groups of parts[group][k][c], in sixteen runs of groups that are added in order.
struct Join {
    float* out[3];
};
constexpr int RUNS = 16;
__global__ __launch_bounds__(64 * RUNS) void block_join_kernel(const float* parts, Join j, int groups, int cols) {
    __shared__ float run[RUNS][64];
    float* out = j.out[blockIdx.y];
    if (!out) return;
    const int l = threadIdx.x & 63, q = threadIdx.x >> 6, col = blockIdx.x * 64 + l;
    float s = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int g = q; g < groups; g += RUNS) s += ldg(parts + ((int64_t)g * 3 + blockIdx.y) * cols + col);
    run[q][l] = s;
    __syncthreads();
    if (q == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < RUNS; ++i) s += run[i][l];
        stg(out + col, s);
    }
}

// Calls f(waves a row takes, vectors a lane takes).  Backward, up to BLOCK_WIDE columns.
// Forward, rows of 16-bit values of more than 2048 columns are two vectors a lane: their arithmetic is as long as
// their loads, and a row's reductions are shared by twice as many (16384 x 4096 bf16 with dropout 133 us where one
// vector takes 143; 8192 x 8192 124 and 138).  Of fp32, whose elements are half as many, one (8192 x 4096 103 and
// 108).  Backward, two of every type: it holds its sums over rows in registers, and few waves fit beside them.
template <class T, bool FORWARD, class F>
void by_row(int64_t cols, F f) {
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, 4> four{};
    constexpr std::integral_constant<int, 8> eight{};
    constexpr std::integral_constant<int, 16> sixteen{};
    if (cols <= 512) return f(one, one);
    if constexpr (FORWARD) {
        if (cols <= 1024) return f(two, one);
        if (cols <= 2048) return f(four, one);
        if constexpr (sizeof(T) == 2) {
            if (cols <= 4096) return f(four, two);
            if (cols <= 8192) return f(eight, two);
        } else {
            if (cols <= 4096) return f(eight, one);
            if (cols <= 8192) return f(sixteen, one);
        }
        f(sixteen, two);
    } else {
        if (cols <= 1024) return f(one, two);
        if (cols <= 2048) return f(two, two);
        if (cols <= 4096) return f(four, two);
        f(eight, two);
    }
}
// Calls f(dropout, gate by element).
template <class F>
void by_form(bool drop, bool token, F f) {
    if (drop)
        token ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
    else
        token ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

int64_t workgroups(int64_t rows, int wpr, int64_t most) {
    return std::min<int64_t>((rows + rows_of(wpr) - 1) / rows_of(wpr), most);
}
// Backward beyond BLOCK_WIDE: ranges of 4096 columns, by four waves with two vectors a lane.
int64_t wide_ranges(int64_t cols) { return (cols + 4095) / 4096; }
// Of the backward kernel: eight waves a CU, each with a fixed set of rows whose sums it keeps.
int64_t back_groups(int64_t rows, int64_t cols) {
    if (cols > BLOCK_WIDE) return workgroups(rows, 4, 512 / wide_ranges(cols));
    int64_t n = 0;
    by_row<float, false>(cols, [&](auto w, auto) {
        constexpr int W = decltype(w)::value;
        n = workgroups(rows, W, 256 * std::max(1, 8 / (W * rows_of(W))));
    });
    return n;
}

}  // namespace

hipError_t launch_block_forward(shampoo4_dtype dtype, const BlockForward& a, const Drop& d, hipStream_t stream) {
    if (a.rows <= 0) return hipSuccess;
    by_type(dtype, [&](auto t) {
        using T = decltype(t);
        by_row<T, true>(a.cols, [&](auto w, auto v) {
            constexpr int W = decltype(w)::value, V = decltype(v)::value;
            by_form(d.threshold && a.h, a.gate_rows, [&](auto drop, auto token) {
                S4_LAUNCH((block_forward_kernel<T, W, V, decltype(drop)::value, decltype(token)::value>),
                          dim3((uint32_t)((a.rows + rows_of(W) - 1) / rows_of(W))), dim3(threads_of(W)), 0, stream, a, d);
            });
        });
    });
    return hipGetLastError();
}

size_t block_workspace_bytes(int64_t rows, int64_t cols) {
    return (size_t)back_groups(rows, cols) * 3 * cols * 4 + (cols > BLOCK_WIDE ? (size_t)rows * 8 : 0);
}

hipError_t launch_block_backward(shampoo4_dtype dtype, const BlockBackward& given, const Drop& d, hipStream_t stream) {
    BlockBackward a = given;
    const Join j{{a.dweight, a.dpost, a.gate_rows ? nullptr : (float*)a.dgate}};
    const bool join = j.out[0] || j.out[1] || j.out[2];
    const int64_t groups = back_groups(a.rows, a.cols);
    if (a.parts) a.sums = a.parts + groups * 3 * a.cols;
    if (!join) a.parts = nullptr;
    if (groups > 0 && a.cols > BLOCK_WIDE)
        by_type(dtype, [&](auto t) {
            using T = decltype(t);
            by_form(d.threshold && a.h, a.gate_rows, [&](auto drop, auto token) {
                constexpr bool D = decltype(drop)::value, G = decltype(token)::value;
                S4_LAUNCH((block_backward_kernel<T, 8, 4, D, G, SUMS>), dim3((uint32_t)workgroups(a.rows, 8, 512)),
                          dim3(threads_of(8)), 0, stream, a, d);
                S4_LAUNCH((block_backward_kernel<T, 4, 2, D, G, REST>), dim3((uint32_t)groups, (uint32_t)wide_ranges(a.cols)),
                          dim3(threads_of(4)), 0, stream, a, d);
            });
        });
    else if (groups > 0)
        by_type(dtype, [&](auto t) {
            using T = decltype(t);
            by_row<T, false>(a.cols, [&](auto w, auto v) {
                constexpr int W = decltype(w)::value, V = decltype(v)::value;
                by_form(d.threshold && a.h, a.gate_rows, [&](auto drop, auto token) {
                    S4_LAUNCH((block_backward_kernel<T, W, V, decltype(drop)::value, decltype(token)::value>),
                              dim3((uint32_t)groups), dim3(threads_of(W)), 0, stream, a, d);
                });
            });
        });
    if (join)
        S4_LAUNCH(block_join_kernel, dim3((uint32_t)((a.cols + 63) / 64), 3), dim3(64 * RUNS), 0, stream, a.parts, j, (int)groups,
                  (int)a.cols);
    return hipGetLastError();
}

}  // namespace s4
