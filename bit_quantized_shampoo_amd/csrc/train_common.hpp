// Device-side pieces shared by the training operators: element types, vectors of eight
// elements at any alignment, and the 8-bit checkpoint's scale and codes.
#pragma once

#include "common.hpp"

namespace s4 {

typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight consecutive elements as raw bits (`Raw`), and their conversion from and to fp32.
// The access types are aligned to the element only: gfx950 loads and stores 16 bytes at any
// element boundary, so odd leading dimensions take the same instructions as even ones.
template <class T>
struct Vec8;

template <>
struct Vec8<__bf16> {
    typedef u32x4 Raw;
    typedef u32x4 Mem __attribute__((aligned(2)));
    static __device__ __forceinline__ floatx8 get(Raw r) {
        floatx8 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(r[i] << 16);
            f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
        return f;
    }
    static __device__ __forceinline__ Raw put(floatx8 f) {
        return __builtin_bit_cast(Raw, __builtin_convertvector(f, bf16x8));
    }
};
template <>
struct Vec8<_Float16> {
    typedef u32x4 Raw;
    typedef u32x4 Mem __attribute__((aligned(2)));
    static __device__ __forceinline__ floatx8 get(Raw r) {
        return __builtin_convertvector(__builtin_bit_cast(f16x8, r), floatx8);
    }
    static __device__ __forceinline__ Raw put(floatx8 f) {
        return __builtin_bit_cast(Raw, __builtin_convertvector(f, f16x8));
    }
};
template <>
struct Vec8<float> {
    typedef u32x8 Raw;
    typedef u32x8 Mem __attribute__((aligned(4)));
    static __device__ __forceinline__ floatx8 get(Raw r) { return __builtin_bit_cast(floatx8, r); }
    static __device__ __forceinline__ Raw put(floatx8 f) { return __builtin_bit_cast(Raw, f); }
};

template <class T>
__device__ __forceinline__ typename Vec8<T>::Raw load8(const T* p) {
    using G = __attribute__((address_space(1))) const typename Vec8<T>::Mem;
    return *(G*)p;
}
template <class T>
__device__ __forceinline__ void store8(T* p, typename Vec8<T>::Raw v) {
    using G = __attribute__((address_space(1))) typename Vec8<T>::Mem;
    *(G*)p = v;
}
// Elements s .. 7 moved to places 0 .. 7 - s, zeros behind them (s = 0 .. 8).
template <class T>
__device__ __forceinline__ typename Vec8<T>::Raw shift_down(typename Vec8<T>::Raw r, int s) {
    constexpr int N = sizeof(r) / 4;
    int d = s;                                               // in dwords
    if constexpr (N == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t up = i + 1 < N ? r[(i + 1) % N] : 0u;
            r[i] = s & 1 ? __builtin_amdgcn_alignbit(up, r[i], 16) : r[i];
        }
        d = s >> 1;
    }
#pragma unroll
    for (int step = 1; step <= N; step *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t up = i + step < N ? r[(i + step) % N] : 0u;
            r[i] = d & step ? up : r[i];
        }
    return r;
}

// Elements c .. c + 7 of a row of `cols` >= 1, zeros beyond its end.  No load is under a lane's
// own condition (it would be waited for before the next is issued): a vector that crosses
// the end is loaded eight from it and shifted, and a row of fewer than eight element by
// element, with indexes clamped into it.
template <class T>
__device__ __forceinline__ typename Vec8<T>::Raw load8_edge(const T* row, int64_t c, int64_t cols) {
    const int n = (int)max((int64_t)0, min((int64_t)8, cols - c));
    if (cols >= 8) return shift_down<T>(load8(row + min(c, cols - 8)), 8 - n);
    typename Vec8<T>::Raw r = {};
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        const int64_t i = min(c + j, cols - 1);
        const uint32_t keep = j < n ? 0xffffffffu : 0u;
        if constexpr (sizeof(T) == 4)
            r[j] = ldg((const uint32_t*)row + i) & keep;
        else
            r[j >> 1] |= ((uint32_t)ldg((const uint16_t*)row + i) & keep) << (16 * (j & 1));
    }
    return r;
}

// The first n (0..8) of eight elements: the whole vector, or pieces of four, two and one.
template <class T>
__device__ __forceinline__ void store8_n(T* p, typename Vec8<T>::Raw v, int n) {
    if (n >= 8) {
        store8(p, v);
        return;
    }
    constexpr int N = sizeof(v) / 4;
    typedef uint32_t H4 __attribute__((ext_vector_type(N / 2)));
    typedef H4 M4 __attribute__((aligned(sizeof(T))));
    if (n & 4) {
        using G = __attribute__((address_space(1))) M4;
        H4 h;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) h[i] = v[i];
        *(G*)p = h;
        v = shift_down<T>(v, 4);
        p += 4;
    }
    if (n & 2) {
        if constexpr (sizeof(T) == 4) {
            typedef u32x2 M2 __attribute__((aligned(4)));
            using G = __attribute__((address_space(1))) M2;
            *(G*)p = u32x2{v[0], v[1]};
        } else {
            typedef uint32_t M2 __attribute__((aligned(2)));
            using G = __attribute__((address_space(1))) M2;
            *(G*)p = v[0];
        }
        v = shift_down<T>(v, 2);
        p += 2;
    }
    if (n & 1) {
        if constexpr (sizeof(T) == 4)
            stg((uint32_t*)p, v[0]);
        else
            stg((uint16_t*)p, (uint16_t)v[0]);
    }
}

// Keeps the compiler from carrying unpacked values from one use of raw registers to the next
// (they would take twice the registers).
template <class R>
__device__ __forceinline__ void unpack_again(R& r) {
    if constexpr (sizeof(R) == 16) asm volatile("" : "+v"(r));
}

// -- the 8-bit checkpoint ----------------------------------------------------------------

// Biased exponent e of a block's scale 2^(e - 127), from the bits of its largest |x|
// (E + mantissa m): a / 2^(E - 6) = 64 m is at most 127 unless the mantissa is above
// 127/64 = 1 + 0x7e0000 / 2^23, where the added 0x1ffff carries into the exponent.
__device__ __forceinline__ uint32_t act8_exponent(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)((amax_bits + 0x1ffffu) >> 23) - 6;
    return (uint32_t)max(e, 1);
}
__device__ __forceinline__ float act8_scale(uint32_t e) { return __uint_as_float(e << 23); }   // e = 255: infinity

// Codes of eight consecutive columns of one row.  inv = 2^(127 - e): x inv is exact, and
// adding 1.5 2^23 rounds it to an integer whose two's complement byte is the sum's low
// byte.  top: 127, or 63 where 64 s is 2^128, or 0 for a block that is not finite.
struct Act8Block {
    float inv[8], top[8];
    __device__ __forceinline__ void set(int j, uint32_t e) {
        inv[j] = __uint_as_float((254u - min(e, 253u)) << 23);
        top[j] = e == 255u ? 0.f : e >= 249u ? 63.f : 127.f;
    }
    __device__ __forceinline__ u32x2 codes(floatx8 x) const {
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // the clamp also turns a NaN, in a block with top = 0, into 0 (of the median's
            // operands a NaN is left out)
            const float y = __builtin_amdgcn_fmed3f(x[j] * inv[j], -top[j], top[j]);
            b[j] = __float_as_uint(y + 12582912.f);
        }
        u32x2 r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x0c0c0400u);
            r[h] = lo | hi << 16;
        }
        return r;
    }
};

// Byte B of a register as a signed number, and shifted into a scale: one instruction each
// (the byte is picked and extended by the instruction's operand selection).
template <int B>
__device__ __forceinline__ float code_value(uint32_t c) {
    float f;
    if constexpr (B == 0)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(c));
    else if constexpr (B == 1)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(c));
    else if constexpr (B == 2)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(c));
    else
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(c));
    return f;
}
template <int B>
__device__ __forceinline__ float byte_scale(uint32_t e) {
    float f;
    const uint32_t sh = 23;
    if constexpr (B == 0)
        asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_0" : "=v"(f) : "v"(sh), "v"(e));
    else if constexpr (B == 1)
        asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_1" : "=v"(f) : "v"(sh), "v"(e));
    else if constexpr (B == 2)
        asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_2" : "=v"(f) : "v"(sh), "v"(e));
    else
        asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_3" : "=v"(f) : "v"(sh), "v"(e));
    return f;
}
// The scales of eight columns from their exponents, and eight codes times them.
__device__ __forceinline__ floatx8 act8_scales(u32x2 e) {
    floatx8 s;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s[4 * h] = byte_scale<0>(e[h]);
        s[4 * h + 1] = byte_scale<1>(e[h]);
        s[4 * h + 2] = byte_scale<2>(e[h]);
        s[4 * h + 3] = byte_scale<3>(e[h]);
    }
    return s;
}
__device__ __forceinline__ floatx8 act8_values(u32x2 c, floatx8 s) {
    floatx8 f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f[4 * h] = code_value<0>(c[h]);
        f[4 * h + 1] = code_value<1>(c[h]);
        f[4 * h + 2] = code_value<2>(c[h]);
        f[4 * h + 3] = code_value<3>(c[h]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= s[j];
    return f;
}

__device__ __forceinline__ u32x2 ldg_u2(const void* p) { return ldg((const u32x2*)p); }

}  // namespace s4
