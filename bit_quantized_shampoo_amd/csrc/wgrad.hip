// Weight gradient G[n, c] = alpha sum_t dY[t, n] X^[t, c] + beta G[n, c] with X^ read from an
// 8-bit checkpoint.
//
// Both operands are contracted over their rows (tokens), so neither has consecutive
// contraction elements in memory.  Tiles are staged in LDS as they lie in memory, token by
// token, in bf16, and gfx950's transposing LDS read (four tokens of sixteen columns a group of
// sixteen lanes) gives each lane the consecutive tokens that a matrix-core operand takes. X^ =
// code * 2^k is a bf16 number exactly, and a bf16 dY is an operand as it stands; an f16 or f32
// dY is split exactly into two or three bf16 pieces, one product each (what a value has below
// 2^-133, the smallest bf16 number, is dropped: digits of fp32 values under 2^-110).
//
// Bound by the matrix cores.  A workgroup of eight waves holds 256 x 256 outputs in its
// accumulators (128 a lane): the largest tile that two waves a SIMD leave registers for, so an
// operand that is read from L2 once meets 256 others.  Slices of 64 tokens (32 where dY has
// two or three pieces) alternate between two stages of LDS: while one is multiplied, the next
// one's loads, conversion and LDS stores are spread over its products, and each unit's
// operands are read from LDS while the unit before it is multiplied; one barrier a slice.  The
// code bytes become bf16 here, five vector instructions a pair.
//
// 16384 x 4096 x 4096 bf16: 456-472 us, 1165-1205 TFLOP/s, where a library's plain bf16
// product of these shapes (X^ in 16 bits) takes 446-460.  The matrix cores are busy for 63% of
// the CUs' busy clocks, LDS reads take 40%, with no bank conflicts; the operands come through
// L2 2.7 times.  With the staging left out the products and operand reads alone take 352 us,
// so what remains is staging: its vector instructions and LDS stores take the issue slots
// beside the products.  Measured and not better (all within 1%): more registers of loads in
// flight, two units of operands ahead, wave priorities, one scale decoded for two rows, other
// spreads of the staging over the units.  f32 dY 5461 x 4096 x 4096 430 us, f16 8192 x 4096 x
// 4096 432, the same number of matrix-core products; 16384 x 1024 x 4096 bf16 137 us (library
// 156), 8192 x 1024 x 1024 33 (53), 4096 x 4096 x 1024 50 (44), 2048 x 2048 x 2048 28.5 (25.6).
//
// The 128 x 128 tile is bound by what a CU issues, not by a chain of latencies: a slice of 64
// tokens takes 0.60 us for one workgroup on the GPU, 0.71 with one on every CU, and 1.28 for two
// that share a CU (16384 x 4096 x 2048 bf16 in 512 workgroups 329 us, half of it in 256 182;
// kept to one a CU, 355).  Of a CU's busy clocks there LDS is active for 52% (98 KB of operand
// reads and 32 KB of stores a slice), the matrix cores for 42%, and vector instructions issue
// for 49%: the three hide each other little.  Two slices in registers take the same time; four
// waves of 64 x 64 instead of eight of 64 x 32, with two thirds of the LDS reads, take 20% more.
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

// Place in LDS of column `col` (a multiple of 4) of token `row`, in bf16, for a tile `cols`
// wide: rows are dense, and the 64-byte blocks of a row change places by the row's number
// modulo 4.  The four token rows that a transposing read takes at once (64 bytes of each, for
// half a wave) then lie in different quarters of the 256 bytes of the banks.
template <int COLS>
__device__ __forceinline__ int lds_at(int row, int col) {
    return row * COLS + (col ^ ((row & 3) << 5));
}

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

// Eight consecutive tokens (k0 + 8 (lane / 32) ..) of column n0 + lane % 32 (k0 a multiple of
// 16, n0 of 32).
template <int COLS>
__device__ __forceinline__ bf16x8 fragment(const uint16_t* lds, int k0, int n0) {
    const int lane = threadIdx.x & 63;
    const int row = (lane >> 5) * 8 + ((lane >> 2) & 3), col = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    const uint16_t* p = lds + k0 * COLS + lds_at<COLS>(row, n0 + col);
    using L = __attribute__((address_space(3))) shortx4;
    union { shortx4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p);
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p + 4 * COLS));
    return u.v;
}

// A workgroup of WM x WN waves, each with TM x TN blocks of 32 x 32; slices of KS tokens.
template <class T, int WM, int WN, int TM, int TN, int KS>
struct Shape {
    static constexpr int BM = WM * TM * 32, BN = WN * TN * 32, THREADS = 64 * WM * WN;
    static constexpr int NP = Pieces<T>::N;
    static constexpr int PLANE = KS * BM;                    // one piece of dY
    static constexpr int STAGE_A = NP * PLANE, STAGE_B = KS * BN;    // bf16 elements of a stage
    static constexpr int STEPS = KS / 16;                    // matrix-core steps of a slice
    static constexpr int UNITS = STEPS * NP;                 // of one piece of dY each
    static constexpr int VA = KS * BM / 8 / THREADS;         // vectors of dY a thread stages
    static constexpr int VB = KS * BN / 8 / THREADS;         // vectors of codes
    static constexpr size_t LDS_BYTES = 2 * (STAGE_A + STAGE_B) * 2;
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
    constexpr int THREADS = S::THREADS, VA = S::VA, VB = S::VB;
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
    // 32-bit lane offsets, beside bases that the workgroup shares (in scalar registers)
    const uint32_t oa = (uint32_t)((arow * w.lddy + acol) * sizeof(T));
    const uint32_t oe = (uint32_t)bn, oc = (uint32_t)(brow * pitch + bn);
    const int64_t sa = AR * w.lddy * (int64_t)sizeof(T), sc = BR * pitch;

    Raw a[VA];                                               // this thread's part of a slice
    u32x2 c[VB], e[KS / 32];
    const auto store_a = [&](int buf, int i) {
        split_store<T>(lds + buf * S::STAGE_A, S::PLANE, lds_at<S::BM>(arow + i * AR, acol), a[i]);
    };
    const auto store_b = [&](int buf, int i) {
        // opaque: taken apart where it is loaded, the codes would be waited for there
        asm volatile("" : "+v"(c[i]), "+v"(e[i * BR / 32]));
        const floatx8 v = act8_values(c[i], act8_scales(e[i * BR / 32]));
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = pack_hi(v[2 * j], v[2 * j + 1]);
        *(u32x4*)(lds + 2 * S::STAGE_A + buf * S::STAGE_B + lds_at<S::BN>(brow + i * BR, bcol)) = q;
    };

    floatx16 acc[TM][TN] = {};
    // Operands of a unit (one step of 16 tokens, one piece of dY), double buffered: the next
    // unit's are read while this one's products run.
    bf16x8 fa[2][TM], fb[2][TN];
    const auto read_unit = [&](int buf, int u) {
        const uint16_t* la = lds + buf * S::STAGE_A + u % S::NP * S::PLANE;
        const uint16_t* lb = lds + 2 * S::STAGE_A + buf * S::STAGE_B;
        const int ks = u / S::NP;
        if (u % S::NP == 0)
#pragma unroll
            for (int n = 0; n < TN; ++n) fb[ks & 1][n] = fragment<S::BN>(lb, 16 * ks, wn + 32 * n);
#pragma unroll
        for (int m = 0; m < TM; ++m) fa[u & 1][m] = fragment<S::BM>(la, 16 * ks, wm + 32 * m);
    };
    const auto products = [&](int u) {
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int n = 0; n < TN; ++n)
                acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[u & 1][m], fb[u / S::NP & 1][n], acc[m][n], 0, 0, 0);
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
        using Global = __attribute__((address_space(1))) const char;
        Global* na = (Global*)((const T*)w.dy + r0 * w.lddy + m0);       // the slice to load next
        Global* nc = (Global*)(w.codes + r0 * pitch);
        Global* ne = (Global*)(w.scales + r0 / 32 * pitch);
        const auto base = [](Global* p) {
            asm("" : "+s"(p));
            return p;
        };
        const auto load_a = [&](int i) {
            using M = __attribute__((address_space(1))) const typename Vec8<T>::Mem;
            a[i] = *(M*)(base(na + i * sa) + oa);
        };
        const auto load_b = [&](int i) {
            using M = __attribute__((address_space(1))) const u32x2;
            c[i] = *(M*)(base(nc + i * sc) + oc);
            // the scales of a block of 32 tokens follow its last codes
            constexpr int PER_E = 32 / BR;
            if ((i + 1) % PER_E == 0) e[i / PER_E] = *(M*)(base(ne + i / PER_E * pitch) + oe);
        };
        // the last slice is loaded again rather than none
        const auto advance = [&](bool more) {
            na += more ? VA * sa : 0;
            nc += more ? VB * sc : 0;
            ne += more ? KS / 32 * pitch : 0;
        };
        // a part of the loaded slice to LDS, and of the next one on its way
        const auto stage = [&](int buf, int i0a, int i1a, int i0b, int i1b) {
#pragma unroll
            for (int i = i0a; i < i1a; ++i) {
                store_a(buf, i);
                load_a(i);
            }
#pragma unroll
            for (int i = i0b; i < i1b; ++i) {
                store_b(buf, i);
                load_b(i);
            }
        };
#pragma unroll
        for (int i = 0; i < VA; ++i) load_a(i);
#pragma unroll
        for (int i = 0; i < VB; ++i) load_b(i);
        advance(1 < fast);
        stage(0, 0, VA, 0, VB);
        __syncthreads();
        read_unit(0, 0);
        const auto slice = [&](int buf, bool more) {
            advance(more);
#pragma unroll
            for (int u = 0; u < S::UNITS; ++u) {
                // The next slice is whole in LDS before the last unit, and this slice's last
                // operands are in registers: the one barrier of a slice, with products to
                // follow it while the next operands are read.
                if (u == S::UNITS - 1) __syncthreads();
                read_unit(u == S::UNITS - 1 ? buf ^ 1 : buf, (u + 1) % S::UNITS);
                products(u);
                constexpr int P = S::UNITS - 1;
                if (u < P) stage(buf ^ 1, u * VA / P, (u + 1) * VA / P, u * VB / P, (u + 1) * VB / P);
                // operand reads and the staging's arithmetic in the shadow of the products
#pragma unroll
                for (int q = 0; q < TM * TN; ++q) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);       // matrix core
                    __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);       // LDS reads
                    __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);       // vector
                }
                // without this the loads gather at the slice's end and are waited for at once
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // two slices a turn, so that the stage is a constant of every address
        for (int64_t s = 0; s < fast; s += 2) {
            slice(0, s + 2 < fast);
            if (s + 1 < fast) slice(1, s + 3 < fast);
        }
        __syncthreads();
    }
    // What is left: the last rows, with every load checked.
    for (int64_t k = r0 + fast * KS; k < r1; k += KS) {
#pragma unroll
        for (int i = 0; i < VA; ++i) {
            const int64_t row = k + arow + i * AR;
            a[i] = load8_edge((const T*)w.dy + min(row, r1 - 1) * w.lddy, m0 + acol, w.n);
            a[i] &= row < r1 ? 0xffffffffu : 0u;
        }
#pragma unroll
        for (int i = 0; i < KS / 32; ++i)
            e[i] = ldg((const u32x2*)(w.scales + min(k / 32 + i, (r1 - 1) / 32) * pitch + bn));
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            const int64_t row = k + brow + i * BR;
            // past the checkpoint's last block: codes 0, and a scale that is finite
            const bool have = row < (r1 + 31) / 32 * 32;
            c[i] = ldg((const u32x2*)(w.codes + (have ? row : 0) * pitch + bn));
            c[i] &= have ? 0xffffffffu : 0u;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VA; ++i) store_a(0, i);
#pragma unroll
        for (int i = 0; i < VB; ++i) store_b(0, i);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < S::UNITS; ++u) {
            read_unit(0, u);
            products(u);
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

// G = alpha sum_s parts[s] + beta G, the parts in order; V consecutive elements a thread
// (V = 4 where rows are multiples of four long).
template <int V>
__global__ __launch_bounds__(256) void wgrad_sum_kernel(WGrad w, int splits) {
    typedef float Vec __attribute__((ext_vector_type(V)));
    typedef Vec Mem __attribute__((aligned(4)));
    using G = __attribute__((address_space(1))) Mem;
    const int64_t n = w.n * w.cols;
    for (int64_t i = (blockIdx.x * 256ll + threadIdx.x) * V; i < n; i += gridDim.x * 256ll * V) {
        Vec s = *(G*)(w.parts + i);
        int k = 1;
        for (; k + 3 <= splits; k += 3) {
            const Vec a = *(G*)(w.parts + k * n + i), b = *(G*)(w.parts + (k + 1) * n + i), c = *(G*)(w.parts + (k + 2) * n + i);
            s = ((s + a) + b) + c;
        }
        for (; k < splits; ++k) s += *(G*)(w.parts + k * n + i);
        const int64_t r = w.n == 1 ? 0 : i / w.cols;
        G* p = (G*)(w.g + r * w.ldg + (i - r * w.cols));
        s *= w.alpha;
        if (w.beta != 0.f) s += w.beta * *p;
        *p = s;
    }
}

struct WPlan {
    bool large;               // 256 x 256 tiles, else 128 x 128
    int64_t tiles_m, tiles_n, rows_per;
    int splits;
};
// Tile and row ranges by an estimate of the time.  A round of workgroups (one a CU) takes
// 28 ns a token on 256 x 256 tiles and 11 ns on 128 x 128 ones (bf16, measured where the
// rounds are full: 16384 x 4096 x 4096 in 463 us against 663 us in four times the tiles).
// Row ranges beyond one fill the GPU when the output alone cannot, at the cost of writing
// and reading their partial sums (5 TB/s, and 2000 ns for the launch that joins them):
// 16384 x 1024 x 4096 takes 142 us in four ranges of 64 large tiles, 182 us in 256 small
// tiles and 351 us in 64 large ones; 2048 x 2048 x 2048 28 us in 256 small tiles, 44 us in
// four ranges of 64 large ones.  A range has at least 128 tokens.  An f16 or f32 dY is two or
// three products an element.
WPlan wgrad_plan(int64_t rows, int64_t n, int64_t cols, int pieces) {
    WPlan best{};
    double best_ns = 0;
    for (int k = 0; k < 2; ++k) {
        WPlan p;
        p.large = k == 1;
        const int64_t tile = p.large ? 256 : 128;
        p.tiles_m = (n + tile - 1) / tile;
        p.tiles_n = (cols + tile - 1) / tile;
        const int64_t tiles = p.tiles_m * p.tiles_n;
        for (int64_t s = 1; s <= 16 && (s == 1 || (rows / s >= 128 && tiles * s <= 512)); ++s) {
            p.rows_per = ((rows + s - 1) / s + 63) / 64 * 64;
            p.splits = rows > 0 ? (int)((rows + p.rows_per - 1) / p.rows_per) : 1;
            if (p.splits != s) continue;
            double ns = (double)((tiles * s + 255) / 256) * (double)p.rows_per * pieces * (p.large ? 28. : 11.);
            if (s > 1) ns += 2000. + (2. * s + 1) * (double)(n * cols) * 4 / 5e3;
            if (best.splits == 0 || ns < best_ns) {
                best = p;
                best_ns = ns;
            }
        }
    }
    return best;
}

template <class T, int WM, int WN, int TM, int TN, int KS>
hipError_t wgrad_launch(const WGrad& w, const WPlan& p, hipStream_t stream) {
    using S = Shape<T, WM, WN, TM, TN, KS>;
    static LdsLimit limit;
    const hipError_t e = limit.raise((const void*)wgrad_kernel<T, WM, WN, TM, TN, KS>, S::LDS_BYTES);
    if (e != hipSuccess) return e;
    S4_LAUNCH((wgrad_kernel<T, WM, WN, TM, TN, KS>), dim3((uint32_t)(p.tiles_m * p.tiles_n * p.splits)),
              dim3(S::THREADS), S::LDS_BYTES, stream, w, (int)p.tiles_m, (int)p.tiles_n, p.rows_per, p.splits > 1);
    return hipSuccess;
}

template <class T>
hipError_t wgrad_of(const WGrad& w, const WPlan& p, hipStream_t stream) {
    // three pieces of a 64-token slice would not fit twice into LDS
    constexpr int KS = Pieces<T>::N == 1 ? 64 : 32;
    return p.large ? wgrad_launch<T, 2, 4, 4, 2, KS>(w, p, stream) : wgrad_launch<T, 2, 4, 2, 1, KS>(w, p, stream);
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t cols) {
    // the most that any type's plan takes
    size_t most = 0;
    for (int pieces = 1; pieces <= 3; ++pieces) {
        const WPlan p = wgrad_plan(rows, n, cols, pieces);
        if (p.splits > 1) most = std::max(most, (size_t)p.splits * n * cols * 4);
    }
    return most;
}

hipError_t launch_wgrad(shampoo4_dtype dtype, const WGrad& w, hipStream_t stream) {
    if (w.n <= 0 || w.cols <= 0) return hipSuccess;
    const int pieces = dtype == SHAMPOO4_BF16 ? 1 : dtype == SHAMPOO4_F16 ? 2 : 3;
    const WPlan p = wgrad_plan(w.rows, w.n, w.cols, pieces);
    const bool part = p.splits > 1;
    hipError_t e;
    switch (dtype) {
        case SHAMPOO4_BF16: e = wgrad_of<__bf16>(w, p, stream); break;
        case SHAMPOO4_F16: e = wgrad_of<_Float16>(w, p, stream); break;
        default: e = wgrad_of<float>(w, p, stream);
    }
    if (e != hipSuccess) return e;
    if (part) {
        WGrad v = w;
        if (w.ldg == w.cols) {                               // contiguous rows are one
            v.n = 1;
            v.cols = v.ldg = w.n * w.cols;
        }
        const bool four = v.cols % 4 == 0;
        const int64_t threads = v.n * v.cols / (four ? 4 : 1);
        const dim3 sg((uint32_t)std::min<int64_t>((threads + 255) / 256, 4096));
        if (four)
            S4_LAUNCH(wgrad_sum_kernel<4>, sg, dim3(256), 0, stream, v, p.splits);
        else
            S4_LAUNCH(wgrad_sum_kernel<1>, sg, dim3(256), 0, stream, v, p.splits);
    }
    return hipGetLastError();
}

}  // namespace s4
