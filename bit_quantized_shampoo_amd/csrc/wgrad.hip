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

// LDS row pitch in bf16 of a tile `cols` wide: the four token rows that a group of sixteen
// lanes reads at once start 64 bytes apart modulo the 256 bytes of the banks, beside the other group's.
constexpr int tile_pitch(int cols) { return cols + 32; }

// Eight values of one token into the pieces' planes.
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
template <int PITCH>
__device__ __forceinline__ bf16x8 fragment(const uint16_t* lds, int k0, int n0) {
    const int lane = threadIdx.x & 63;
    const uint16_t* p = lds + (k0 + (lane >> 5) * 8 + ((lane >> 2) & 3)) * PITCH + n0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    using L = __attribute__((address_space(3))) shortx4;
    union { shortx4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p);
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p + 4 * PITCH));
    return u.v;
}

// A workgroup of WM x WN waves, each with TM x TN blocks of 32 x 32; slices of KS tokens.
template <class T, int WM, int WN, int TM, int TN, int KS>
struct Shape {
    static constexpr int BM = WM * TM * 32, BN = WN * TN * 32, THREADS = 64 * WM * WN;
    static constexpr int NP = Pieces<T>::N;
    static constexpr int PA = tile_pitch(BM), PB = tile_pitch(BN);
    static constexpr int PLANE = KS * PA;                    // one piece of dY
    static constexpr int STAGE = NP * PLANE + KS * PB;       // bf16 elements of a stage
    static constexpr int STEPS = KS / 16;                    // matrix-core steps of a slice
    static constexpr int VA = KS * BM / 8 / THREADS;         // vectors of dY a thread stages
    static constexpr int VB = KS * BN / 8 / THREADS;         // vectors of codes
    static constexpr size_t LDS_BYTES = 2 * STAGE * 2;
    static_assert(THREADS % (BM / 8) == 0 && THREADS % (BN / 8) == 0, "columns fixed per thread");
};

// Row range and output tile of this workgroup.  Workgroups go to the eight XCDs round robin;
// each XCD takes a contiguous range of the tiles (the remainder, under eight, keeps its
// place), ordered in groups of four tile rows.  The tiles that one L2 serves are then a
// compact region: they share their columns of dY and X, and their neighbouring columns
// spread over the L2's channels where a power-of-two row length would fold a single
// column of tiles onto a few of them.
__device__ __forceinline__ void place(int tiles_m, int tiles_n, int& split, int& tile_m, int& tile_n) {
    const int n = gridDim.x, n8 = n >> 3;
    const int b = (int)blockIdx.x < 8 * n8 ? ((int)blockIdx.x & 7) * n8 + ((int)blockIdx.x >> 3) : (int)blockIdx.x;
    const int tiles = tiles_m * tiles_n;
    split = b / tiles;
    const int t = b - split * tiles;
    const int g = t / (4 * tiles_n);
    const int gh = min(4, tiles_m - 4 * g);
    const int local = t - 4 * g * tiles_n;
    tile_m = 4 * g + local % gh;
    tile_n = local / gh;
}

template <class T, int WM, int WN, int TM, int TN, int KS>
__global__ __launch_bounds__(64 * WM * WN) void wgrad_kernel(WGrad w, int tiles_m, int tiles_n, int64_t rows_per,
                                                             bool partial) {
    using S = Shape<T, WM, WN, TM, TN, KS>;
    using Raw = typename Vec8<T>::Raw;
    constexpr int THREADS = S::THREADS, STEPS = S::STEPS, VA = S::VA, VB = S::VB;
    extern __shared__ uint16_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int split, tile_m, tile_n;
    place(tiles_m, tiles_n, split, tile_m, tile_n);
    const int64_t m0 = (int64_t)tile_m * S::BM, n0 = (int64_t)tile_n * S::BN;
    const int64_t r0 = (int64_t)split * rows_per, r1 = min(w.rows, r0 + rows_per);
    const int64_t pitch = act8_pitch(w.cols);
    const int wm = (wv % WM) * TM * 32, wn = (wv / WM) * TN * 32;

    // staging: thread (row, column group) of both tiles; its vectors are AR (BR) rows apart
    constexpr int AR = THREADS / (S::BM / 8), BR = THREADS / (S::BN / 8);
    const int arow = tid / (S::BM / 8), acol = tid % (S::BM / 8) * 8;
    const int brow = tid / (S::BN / 8), bcol = tid % (S::BN / 8) * 8;
    const int64_t bn = min(n0 + bcol, pitch - 8);            // beyond: columns that are not stored
    // addresses: a base that the workgroup shares (scalar registers) and 32-bit lane offsets
    const char* pa = (const char*)((const T*)w.dy + r0 * w.lddy + m0);
    const char* pc = (const char*)w.codes + r0 * pitch;
    const char* pe = (const char*)w.scales + r0 / 32 * pitch;
    const uint32_t oa = (uint32_t)((arow * w.lddy + acol) * sizeof(T));
    const uint32_t oe = (uint32_t)bn, oc = (uint32_t)(brow * pitch + bn);
    const int64_t sa = AR * w.lddy * (int64_t)sizeof(T), sc = BR * pitch;

    Raw a[VA];
    u32x2 c[VB], e[KS / 32];
    const auto store_a = [&](int buf, int i) {
        split_store<T>(lds + buf * S::STAGE, S::PLANE, (arow + i * AR) * S::PA + acol, a[i]);
    };
    const auto store_b = [&](int buf, int i) {
        // opaque: taken apart where it is loaded, the codes would be waited for there
        asm volatile("" : "+v"(c[i]), "+v"(e[i * BR / 32]));
        const floatx8 v = act8_values(c[i], act8_scales(e[i * BR / 32]));
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = pack_hi(v[2 * j], v[2 * j + 1]);
        *(u32x4*)(lds + buf * S::STAGE + S::NP * S::PLANE + (brow + i * BR) * S::PB + bcol) = q;
    };

    floatx16 acc[TM][TN] = {};
    struct Frags {
        bf16x8 a[S::NP][TM], b[TN];
    };
    const auto read_frags = [&](Frags& f, int buf, int ks) {
        const uint16_t* la = lds + buf * S::STAGE;
        const uint16_t* lb = la + S::NP * S::PLANE;
#pragma unroll
        for (int n = 0; n < TN; ++n) f.b[n] = fragment<S::PB>(lb, 16 * ks, wn + 32 * n);
#pragma unroll
        for (int q = 0; q < S::NP; ++q)
#pragma unroll
            for (int m = 0; m < TM; ++m) f.a[q][m] = fragment<S::PA>(la + q * S::PLANE, 16 * ks, wm + 32 * m);
    };
    const auto products = [&](const Frags& f) {
#pragma unroll
        for (int q = 0; q < S::NP; ++q)
#pragma unroll
            for (int m = 0; m < TM; ++m)
#pragma unroll
                for (int n = 0; n < TN; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[q][m], f.b[n], acc[m][n], 0, 0, 0);
    };

    // Whole slices whose loads all lie inside dY.  A load past a row's end reads the start of
    // the next row, into columns of G that are not stored; only the last rows need care.
    int64_t fast = 0;
    {
        const int64_t x = (w.rows - 1) * w.lddy + w.n - m0 - S::BM;    // last row start that may be loaded
        const int64_t k = x >= 0 ? x / w.lddy - (KS - 1) : -1;         // last slice start
        // lane offsets of 32 bits: AR (BR) rows
        const bool narrow = w.lddy < (1 << 24) && pitch < (1 << 24);
        if (narrow && k >= r0 && r1 > r0) fast = min((r1 - r0) / KS, (k - r0) / KS + 1);
    }
    if (fast > 0) {
        const auto shared_base = [](const char* p) {
            asm("" : "+s"(p));
            return p;
        };
        const auto load_a = [&](int64_t slice, int i) { a[i] = load8((const T*)(shared_base(pa + (slice * VA + i) * sa) + oa)); };
        const auto load_b = [&](int64_t slice, int i) { c[i] = ldg((const u32x2*)(shared_base(pc + (slice * VB + i) * sc) + oc)); };
        const auto load_e = [&](int64_t slice, int i) { e[i] = ldg((const u32x2*)(shared_base(pe + (slice * (KS / 32) + i) * pitch) + oe)); };
        // the scales of a block of 32 tokens follow its last codes
        constexpr int PER_E = 32 / BR;
#pragma unroll
        for (int i = 0; i < VA; ++i) load_a(0, i);
#pragma unroll
        for (int i = 0; i < VB; ++i) load_b(0, i);
#pragma unroll
        for (int i = 0; i < KS / 32; ++i) load_e(0, i);
        const auto stage = [&](int buf, int64_t next, int i0a, int i1a, int i0b, int i1b) {
#pragma unroll
            for (int i = i0a; i < i1a; ++i) {
                store_a(buf, i);
                load_a(next, i);
            }
#pragma unroll
            for (int i = i0b; i < i1b; ++i) {
                store_b(buf, i);
                load_b(next, i);
                if ((i + 1) % PER_E == 0) load_e(next, i / PER_E);
            }
        };
        stage(0, min<int64_t>(1, fast - 1), 0, VA, 0, VB);
        __syncthreads();
        Frags f[2];
        read_frags(f[0], 0, 0);
        for (int64_t s = 0; s < fast; ++s) {
            const int buf = (int)s & 1;
            const int64_t next = min(s + 2, fast - 1);
#pragma unroll
            for (int ks = 0; ks < STEPS; ++ks) {
                // The next slice is whole in LDS before the last step, and this slice's last
                // operands are in registers: the one barrier of a slice, with products to
                // follow it while the next operands are read.
                if (ks == STEPS - 1) __syncthreads();
                read_frags(f[(ks + 1) & 1], ks == STEPS - 1 ? buf ^ 1 : buf, (ks + 1) % STEPS);
                products(f[ks & 1]);
                // a part of the next slice to the other stage, and of the one after it on its way
                constexpr int P = STEPS - 1;
                if (ks < P) stage(buf ^ 1, next, ks * VA / P, (ks + 1) * VA / P, ks * VB / P, (ks + 1) * VB / P);
                // without this the loads gather at the slice's end and are waited for at once
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
    }
    // What is left: the last rows, with every load checked.
    for (int64_t k = r0 + fast * KS; k < r1; k += KS) {
#pragma unroll
        for (int i = 0; i < VA; ++i) {
            const int64_t row = k + arow + i * AR;
            const int n = (int)max((int64_t)0, min((int64_t)8, w.n - m0 - acol));
            a[i] = load8_n((const T*)w.dy + row * w.lddy + m0 + acol, row < r1 ? n : 0);
        }
#pragma unroll
        for (int i = 0; i < KS / 32; ++i) e[i] = k + 32 * i < r1 ? ldg((const u32x2*)(w.scales + (k / 32 + i) * pitch + bn)) : u32x2{0, 0};
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            const int64_t row = k + brow + i * BR;
            c[i] = u32x2{0, 0};
            if (row < r1) c[i] = ldg((const u32x2*)(w.codes + row * pitch + bn));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VA; ++i) store_a(0, i);
#pragma unroll
        for (int i = 0; i < VB; ++i) store_b(0, i);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < STEPS; ++ks) {
            Frags f;
            read_frags(f, 0, ks);
            products(f);
        }
    }

    float* out = partial ? w.parts + (int64_t)split * w.n * w.cols : w.g;
    const int64_t ld = partial ? w.cols : w.ldg;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n)
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
    bool large;               // 256 x 256 tiles, else 128 x 128
    int64_t tiles_m, tiles_n, rows_per;
    int splits;
};
WPlan wgrad_plan(int64_t rows, int64_t n, int64_t cols) {
    WPlan p;
    p.large = ((n + 255) / 256) * ((cols + 255) / 256) >= 128;
    const int64_t tile = p.large ? 256 : 128;
    p.tiles_m = (n + tile - 1) / tile;
    p.tiles_n = (cols + tile - 1) / tile;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t s = p.large ? 1 : std::max<int64_t>(1, std::min<int64_t>(512 / std::max<int64_t>(tiles, 1), rows / 256));
    p.rows_per = ((rows + s - 1) / s + 63) / 64 * 64;
    p.splits = rows > 0 ? (int)((rows + p.rows_per - 1) / p.rows_per) : 1;
    return p;
}

template <class T, int WM, int WN, int TM, int TN, int KS>
hipError_t wgrad_launch(const WGrad& w, const WPlan& p, hipStream_t stream) {
    using S = Shape<T, WM, WN, TM, TN, KS>;
    static const hipError_t attr = hipFuncSetAttribute((const void*)wgrad_kernel<T, WM, WN, TM, TN, KS>,
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)S::LDS_BYTES);
    if (attr != hipSuccess) return attr;
    S4_LAUNCH((wgrad_kernel<T, WM, WN, TM, TN, KS>), dim3((uint32_t)(p.tiles_m * p.tiles_n * p.splits)),
              dim3(S::THREADS), S::LDS_BYTES, stream, w, (int)p.tiles_m, (int)p.tiles_n, p.rows_per, p.splits > 1);
    return hipSuccess;
}

template <class T>
hipError_t wgrad_of(const WGrad& w, const WPlan& p, hipStream_t stream) {
    // three pieces of a 64-token slice would not fit twice into LDS
    constexpr int KS = Pieces<T>::N == 1 ? 64 : 32;
    return p.large ? wgrad_launch<T, 2, 4, 4, 2, KS>(w, p, stream) : wgrad_launch<T, 2, 2, 2, 2, 32>(w, p, stream);
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t cols) {
    const WPlan p = wgrad_plan(rows, n, cols);
    return p.splits > 1 ? (size_t)p.splits * n * cols * 4 : 0;
}

hipError_t launch_wgrad(shampoo4_dtype dtype, const WGrad& w, hipStream_t stream) {
    if (w.n <= 0 || w.cols <= 0) return hipSuccess;
    const WPlan p = wgrad_plan(w.rows, w.n, w.cols);
    const bool part = p.splits > 1;
    hipError_t e;
    switch (dtype) {
        case SHAMPOO4_BF16: e = wgrad_of<__bf16>(w, p, stream); break;
        case SHAMPOO4_F16: e = wgrad_of<_Float16>(w, p, stream); break;
        default: e = wgrad_of<float>(w, p, stream);
    }
    if (e != hipSuccess) return e;
    if (part) {
        const dim3 sg((uint32_t)std::min<int64_t>((w.n * w.cols + 255) / 256, 4096));
        S4_LAUNCH(wgrad_sum_kernel, sg, dim3(256), 0, stream, w, p.splits);
    }
    return hipGetLastError();
}

}  // namespace s4
