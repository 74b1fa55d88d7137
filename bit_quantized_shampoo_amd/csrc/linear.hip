// Products of linear layers in e4m3: Y[t, n] (+)= sum_k X^[t, k] W^[n, k] (shampoo4_train.h).
#include <algorithm>
#include <type_traits>

#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));

// 32 codes of a lane: of a row (lane % 16) of a 16 x 128 operand, columns 32 (lane / 16) on.
struct Frag {
    u32x4 lo, hi;
};
__device__ __forceinline__ intx8 operand(const Frag& f) {
    return intx8{(int)f.lo[0], (int)f.lo[1], (int)f.lo[2], (int)f.lo[3], (int)f.hi[0], (int)f.hi[1], (int)f.hi[2], (int)f.hi[3]};
}

// acc += W X^T of one block of 128 (D rows: W's, columns: X's).  Any order of the 32 columns
// within a lane will do, as both operands have the same one and a scale covers all of them.
template <bool EXACT>
__device__ __forceinline__ void block_product(floatx4& acc, const Frag& w, const Frag& x, uint32_t we, uint32_t xe) {
    if constexpr (!EXACT) {
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(x), acc, 0, 0, 0, (int)we, 0, (int)xe);
    } else {
        floatx4 part = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const u32x4 a = q < 2 ? w.lo : w.hi, b = q < 2 ? x.lo : x.hi;
            const floatx8 fa = fp8_values(u32x2{a[q % 2 * 2], a[q % 2 * 2 + 1]});
            const floatx8 fb = fp8_values(u32x2{b[q % 2 * 2], b[q % 2 * 2 + 1]});
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_convertvector(fa, bf16x8), __builtin_convertvector(fb, bf16x8),
                                                           part, 0, 0, 0);
        }
        // the scales' product may leave fp32's range where its product with the sum does not
        const int shift = (int)(we + xe) - 254;
        const float one = we == 255u || xe == 255u ? __builtin_nanf("") : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(__builtin_amdgcn_ldexpf(part[i], shift), one, acc[i]);
    }
}

// The largest over the four lanes 16 apart.
__device__ __forceinline__ uint32_t max_of_rows(uint32_t m) {
    const auto h = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(h[0], h[1]);
    const auto w = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(w[0], w[1]);
}

// Y's four consecutive columns of a row, of which n exist.
template <class O>
__device__ __forceinline__ void put4(O* p, floatx4 v, int n, bool accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) stg(p + i, (O)(accumulate ? (float)ldg(p + i) + v[i] : v[i]));
}

// X's element type as a kernel's parameter: uint8_t where it is given as codes.
constexpr int WAVES = 8;

template <class X, class O, int MT>
__global__ __launch_bounds__(64 * WAVES) void linear_rows_kernel(Linear a, uint32_t tiles_n) {
    constexpr bool EXACT = !std::is_same_v<O, __bf16>;
    constexpr int AHEAD = 2;                                 // blocks of k in flight
    __shared__ floatx4 sums[WAVES][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * 16, m0 = (int64_t)(blockIdx.x / tiles_n) * (16 * MT);
    const int64_t pitch = fp8_pitch(a.k), sp = fp8_scale_pitch(a.k);
    const int r = lane & 15, kq = (lane >> 4) * 32;
    const uint8_t* w = a.wc + min(n0 + r, a.n - 1) * pitch + kq;
    const uint8_t* wscale = a.ws + (n0 >> 7) * sp;
    const int nkb = (int)(pitch >> 7);
    floatx4 acc[MT] = {};
    for (int kb0 = wave; kb0 < nkb; kb0 += AHEAD * WAVES) {
        Frag fw[AHEAD], fx[AHEAD][MT];
        uint32_t we[AHEAD], xe[AHEAD][MT];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t kb = min(kb0 + u * WAVES, nkb - 1);
            fw[u].lo = ldg((const u32x4*)(w + kb * 128));
            fw[u].hi = ldg((const u32x4*)(w + kb * 128 + 16));
            we[u] = ldg(wscale + kb);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t row = min(m0 + 16 * t + r, a.rows - 1);
                if constexpr (std::is_same_v<X, uint8_t>) {
                    const uint8_t* x = a.xc + row * pitch + kb * 128 + kq;
                    fx[u][t].lo = ldg((const u32x4*)x);
                    fx[u][t].hi = ldg((const u32x4*)(x + 16));
                    xe[u][t] = ldg(a.xs + row * sp + kb);
                } else {
                    const X* x = (const X*)a.x + row * a.ldx;
                    floatx8 f[4];
                    uint32_t m = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f[q] = Vec8<X>::get(load8_edge(x, kb * 128 + kq + 8 * q, a.k));
                        m = max(m, magnitude(f[q]));
                    }
                    xe[u][t] = fp8_exponent(max_of_rows(m));
                    const Fp8Block blk(xe[u][t]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const u32x2 c = blk.codes(f[q]);
                        u32x4& to = q < 2 ? fx[u][t].lo : fx[u][t].hi;
                        to[q % 2 * 2] = c[0];
                        to[q % 2 * 2 + 1] = c[1];
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (kb0 + u * WAVES < nkb)
#pragma unroll
                for (int t = 0; t < MT; ++t) block_product<EXACT>(acc[t], fw[u], fx[u][t], we[u], xe[u][t]);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) sums[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += WAVES) {
        floatx4 s = sums[0][t][lane];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) s += sums[i][t][lane];
        const int64_t row = m0 + 16 * t + r, col = n0 + 4 * (lane >> 4);
        if (row < a.rows && col < a.n)
            put4((O*)a.y + row * a.ldy + col, s, (int)min((int64_t)4, a.n - col), a.accumulate != 0);
    }
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

template <class X, class O>
hipError_t launch_rows(const Linear& a, hipStream_t stream) {
    const int64_t tn = (a.n + 15) / 16;
    const int mt = a.rows > 16 ? 4 : 1;
    const dim3 grid((uint32_t)((a.rows + 16 * mt - 1) / (16 * mt) * tn));
    if (mt == 4)
        S4_LAUNCH((linear_rows_kernel<X, O, 4>), grid, dim3(64 * WAVES), 0, stream, a, (uint32_t)tn);
    else
        S4_LAUNCH((linear_rows_kernel<X, O, 1>), grid, dim3(64 * WAVES), 0, stream, a, (uint32_t)tn);
    return hipGetLastError();
}

}  // namespace

size_t linear_workspace_bytes(shampoo4_dtype out_dtype, int64_t rows, int64_t n, int64_t k, bool x_quantised) {
    if (rows <= 16 || x_quantised) return 0;
    return up256((size_t)(rows * fp8_pitch(k))) + up256((size_t)(rows * fp8_scale_pitch(k)));
}

hipError_t launch_linear(shampoo4_dtype dtype, shampoo4_dtype out_dtype, const Linear& given, void* workspace,
                         hipStream_t stream) {
    if (given.rows <= 0) return hipSuccess;
    Linear a = given;
    if (a.x && a.rows > 16) {
        uint8_t* codes = (uint8_t*)workspace;
        uint8_t* scales = codes + up256((size_t)(a.rows * fp8_pitch(a.k)));
        const hipError_t e = launch_fp8_store(dtype, a.rows, a.k, a.x, a.ldx, codes, scales, stream);
        if (e != hipSuccess) return e;
        a.x = nullptr;
        a.xc = codes;
        a.xs = scales;
    }
    hipError_t e = hipSuccess;
    by_type(out_dtype, [&](auto o) {
        using O = decltype(o);
        if (!a.x)
            e = launch_rows<uint8_t, O>(a, stream);
        else
            by_type(dtype, [&](auto x) { e = launch_rows<decltype(x), O>(a, stream); });
    });
    return e;
}

}  // namespace s4
