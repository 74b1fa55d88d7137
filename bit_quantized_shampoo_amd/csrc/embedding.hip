// Embedding lookup and its gradient by sorted tokens.
//
// Lookup: a stream of rows, eight elements a thread.
//
// Gradient: G[v] = scale * sum of dout[t] over the tokens t with id v.
//  1. The positions are sorted by id, stably: least significant digit first, digits of up to
//     9 bits.  A wave ranks 64 ids at a time: a ballot a bit gives each lane the lanes that
//     share its digit, its rank among them and their number.  Up to SMALL_T tokens it is one
//     launch, each workgroup sorting a range of ids in LDS; beyond, a pass is two launches
//     over blocks of SORT_TILE tokens (digit counts, then ranks and scatter).  Up to RANK_T
//     tokens there are no digits: a token's place is counted.
//     Without accumulation the other workgroups of these launches write G's zeros: the fill
//     is bound by HBM and the sort by latency, so the sort costs little beside it.
//  2. Sums of runs of equal ids, cut at every CHUNK sorted positions: one wave per piece (short
//     lists) or per chunk, and 512 columns.  A run inside a chunk is stored as a row of G; a
//     piece of a longer one goes to a partial row.
//  3. Runs over several chunks: a wave adds a short run's partial rows, a workgroup of eight
//     waves a long one's, each every eighth, joined in a fixed order.
// The order of every sum follows from the ids alone: no floating atomics.
//
// Bound by HBM where G is large and by the chain of three dependent launches where it is not.
// 16384 x 1024 bf16 into [65536, 1024]: 78 us, of which the sort beside the zeros takes 39.4
// (268 MB written, 6.8 TB/s: what a plain fill reaches, so the sort is hidden), the sums 21.8
// (33 MB read and 28 MB written by rows of 1 or 2 KB in sorted order), the joins 7.8 (what a launch
// and a chain of three loads take, beside one run of the most frequent id).  The zeros are
// written for all of G and a tenth of them again by the sums: which rows are present is known
// only after the sort.
// 1000 x 577 fp32, added: 15 us, the three kernels 4.0, 6.8 and 3.9.
// Zeros written instead behind the sort, for the rows without a token alone and beside the
// sums and joins, take as long or longer (16384 x 1024 into 65536: 67.4 and 67.7-71 us).
// Beyond SMALL_T tokens (1024 columns bf16 into [65536, 1024]): 32768 tokens 105 us, 65536 141,
// 262144 356 (added to G: 72, 103, 342).  Of the 356 the sums take 176 (537 MB read), the joins
// 90 (the most frequent id's run is one workgroup's), the two scatters 30 each and the counts 13.
// A scatter's workgroup reads every block's counts, which grows with the square of the
// blocks: 79 us a scatter at 1048576 tokens, of 449 with 256 columns.
//
// The lookup of 16384 x 1024 bf16 takes 12.3 us, the copy's time for its 67 MB (13.2).
// Lookup: 8 rows of 1024 bf16 in 2.6 us.
#include <algorithm>

#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

constexpr int RADIX_BITS = 9;                // most bits of a digit
constexpr int BINS = 1 << RADIX_BITS;
constexpr int SMALL_T = 16384;               // tokens of the one-launch sort: 16 waves of up to 16 rounds
constexpr int SMALL_WAVES = 16;
constexpr int RANK_T = 4096;                 // tokens of the sort by counting
constexpr int RANK_LANES = 32;               // lanes that count for an item
constexpr int RANK_ITEMS = 1024 / RANK_LANES;
constexpr int TILE_WAVES = 8;
constexpr int TILE_ROUNDS = 8;
constexpr int SORT_TILE = TILE_WAVES * TILE_ROUNDS * 64;
constexpr int CHUNK = 16;                    // sorted positions per wave
constexpr int COLS = 512;                    // columns per wave
constexpr int JOIN_WAVES = 8;

int bit_length(uint64_t v) {
    int n = 0;
    while (v) { ++n; v >>= 1; }
    return n;
}

__device__ __forceinline__ int64_t id_at(const void* ids, int id64, int64_t i) {
    return id64 ? ldg((const int64_t*)ids + i) : (int64_t)ldg((const int32_t*)ids + i);
}
// Sort key of a token: its id, or `vocab` (behind every row) for one that has none.
__device__ __forceinline__ uint32_t key_at(const void* ids, int id64, int64_t vocab, int64_t i) {
    const int64_t id = id_at(ids, id64, i);
    return (uint32_t)(id >= 0 && id < vocab ? id : vocab);
}

template <class T>
__global__ __launch_bounds__(256) void embedding_kernel(Embed e, uint32_t nvec, uint64_t total) {
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
        const uint64_t t = i / nvec;
        const int64_t c = (int64_t)(i - t * nvec) * 8;
        const int64_t id = id_at(e.ids, e.id64, (int64_t)t);
        const int n = (int)min((int64_t)8, e.dim - c);
        typename Vec8<T>::Raw r = {};
        if (id >= 0 && id < e.vocab) {
            r = load8_edge((const T*)e.table + id * e.ldtable, c, e.dim);
            r = Vec8<T>::put(Vec8<T>::get(r) * e.scale);
        }
        store8_n((T*)e.out + (int64_t)t * e.ldout + c, r, n);
    }
}

// Part `part` of `parts` of the zeros of G, by workgroups 0 .. nblk - 1 of this launch.
struct Fill {
    float* g;                 // NULL: nothing to fill
    int64_t rows, cols, ld;
    int part, parts;
};
__device__ void fill_zeros(const Fill& f, int64_t blk, int64_t nblk) {
    // contiguous rows are one row
    const bool flat = f.ld == f.cols;
    const int64_t cols = flat ? f.rows * f.cols : f.cols;
    const int64_t rows = flat ? 1 : f.rows;
    const int64_t per = (int64_t)blockDim.x * 4;
    const int64_t chunks = (cols + per - 1) / per;           // pieces of a row
    const int64_t n = rows * chunks;
    const int64_t b0 = n * f.part / f.parts, b1 = n * (f.part + 1) / f.parts;
    for (int64_t i = b0 + blk; i < b1; i += nblk) {
        const int64_t r = i / chunks;
        const int64_t c = (i - r * chunks) * per + threadIdx.x * 4;
        float* p = f.g + r * f.ld + c;
        if (c + 4 <= cols) {
            typedef floatx4 M __attribute__((aligned(4)));
            using G = __attribute__((address_space(1))) M;
            *(G*)p = floatx4{0.f, 0.f, 0.f, 0.f};
        } else {
            for (int64_t j = c; j < cols; ++j) stg(f.g + r * f.ld + j, 0.f);
        }
    }
}

// Lanes of this wave with the same digit as this one (live lanes only).  A lane's bit as a
// mask x of ones or zeros keeps the lanes whose bit agrees: m & ~(ballot ^ x).
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool live, int bits) {
    const uint64_t all = __ballot(live);
    uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
    for (int b = 0; b < bits; ++b) {
        const int x = (int)(digit << (31 - b)) >> 31;
        const uint64_t w = __ballot(x < 0);
        lo &= ~((uint32_t)w ^ (uint32_t)x);
        hi &= ~((uint32_t)(w >> 32) ^ (uint32_t)x);
    }
    return (uint64_t)hi << 32 | lo;
}

// Stable ranks of a workgroup's items by digit.  Wave w's item of round r is number
// (w rounds + r) 64 + lane.  cnt [waves][bins] counts each wave's digits; on return rank[r]
// is the item's rank among its wave's items of the same digit.
template <int ROUNDS>
__device__ __forceinline__ void wave_ranks(const uint32_t (&digit)[ROUNDS], const bool (&live)[ROUNDS], int bits,
                                           uint32_t* cnt, uint32_t (&rank)[ROUNDS], int rounds) {
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r < rounds) {
            const uint64_t m = same_digit(digit[r], live[r], bits);
            uint32_t old = 0;
            if (live[r]) old = cnt[digit[r]];
            const uint32_t first = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
            rank[r] = old + first;
            // the next round reads what this one's first lane writes: LDS accesses of a wave
            // execute in order, and the fences keep the compiler to it
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (live[r] && first == 0) cnt[digit[r]] = old + __popcll(m);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
}

// Turns cnt [waves][bins] into each wave's first place per digit, and returns through
// `tot` (LDS, bins) each digit's first place in the workgroup's own order.
template <int WAVES>
__device__ __forceinline__ void digit_places(uint32_t* cnt, int bins, uint32_t* tot, uint32_t* wsum) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    uint32_t s = 0;
    if (tid < bins) {
        uint32_t c[WAVES];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) c[w] = cnt[w * BINS + tid];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            cnt[w * BINS + tid] = s;
            s += c[w];
        }
    }
    uint32_t inc = s;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = (uint32_t)__shfl_up((int)inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 63) wsum[wv] = inc;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wv; ++w) before += wsum[w];
    if (tid < bins) tot[tid] = before + inc - s;
    __syncthreads();
}

// The passes of a small sort: n <= 1024 R items in buf, by the `passes` digits of `bits` bits
// from bit `shift` on.  Items are in registers between the barriers of a pass, so buf is
// sorted in place.
template <int R>
__device__ void sort_in_lds(uint32_t* buf, int n, int shift, int passes, int bits, uint32_t* cnt, uint32_t* tot,
                            uint32_t* wsum) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, bins = 1 << bits;
    const int rounds = (n + 1023) / 1024;
    uint32_t item[R], digit[R], rank[R];
    bool live[R];
    for (int p = 0; p < passes; ++p) {
        for (int i = lane; i < bins; i += 64) cnt[wv * BINS + i] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = (wv * rounds + r) * 64 + lane;
            live[r] = r < rounds && i < n;
            item[r] = buf[min(i, SMALL_T - 1)];
            digit[r] = (item[r] >> (shift + p * bits)) & (uint32_t)(bins - 1);
        }
        wave_ranks<R>(digit, live, bits, cnt + wv * BINS, rank, rounds);
        __syncthreads();
        digit_places<SMALL_WAVES>(cnt, bins, tot, wsum);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (live[r]) buf[tot[digit[r]] + cnt[wv * BINS + digit[r]] + rank[r]] = item[r];
        __syncthreads();
    }
}

// Up to SMALL_T tokens: workgroup k < parts sorts the ids of the k-th range of `range` ids;
// the others fill zeros.  A sorting workgroup reads every id: it counts those below its
// range, which gives the place of its output without a word from the others, and takes its
// own, in order, into LDS (all of them, if all are in one range), as (id - first of the
// range, position) in one word with `pos_bits` low bits of position.  The code runs once,
// so its length counts: a workgroup enters the form of the sort that its items need.
__global__ __launch_bounds__(1024) void sort_small_kernel(const void* ids, int id64, int64_t vocab, int tokens,
                                                          int parts, uint32_t range, int passes, int bits,
                                                          int pos_bits, uint32_t* skey, uint32_t* spos, Fill fill) {
    __shared__ uint32_t buf[SMALL_T];
    __shared__ uint32_t cnt[SMALL_WAVES * BINS];
    __shared__ uint32_t tot[BINS];
    __shared__ uint32_t wsum[SMALL_WAVES], wbelow[SMALL_WAVES];
    if ((int)blockIdx.x >= parts) {
        fill_zeros(fill, blockIdx.x - parts, gridDim.x - parts);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const uint32_t lo = blockIdx.x * range;
    const int rounds = (tokens + 1023) / 1024;
    // item number (wave, round, lane): each wave a contiguous piece; every load is issued
    // before the first is looked at (clamped, so that none is under a condition)
    const int first = wv * rounds * 64 + lane;
    uint32_t key[16], mine = 0, below = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) key[r] = key_at(ids, id64, vocab, min(first + r * 64, tokens - 1));
#pragma unroll
    for (int r = 0; r < 16; ++r)
        if (r < rounds) {
            const bool have = first + r * 64 < tokens;
            below += __popcll(__ballot(have && key[r] < lo));
            mine += __popcll(__ballot(have && key[r] - lo < range));     // below: wraps to a large number
        }
    if (lane == 0) {
        wsum[wv] = mine;
        wbelow[wv] = below;
    }
    __syncthreads();
    uint32_t at = 0, n = 0, out = 0;
    for (int w = 0; w < SMALL_WAVES; ++w) {
        const uint32_t c = wsum[w];
        at += w < wv ? c : 0u;
        n += c;
        out += wbelow[w];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
        if (r < rounds) {
            const bool take = first + r * 64 < tokens && key[r] - lo < range;
            const uint64_t m = __ballot(take);
            if (take)
                buf[at + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u))] =
                    (key[r] - lo) << pos_bits | (uint32_t)(first + r * 64);
            at += __popcll(m);
        }
    // the first pass's barrier comes before any item is read
    if (n <= 1024)
        sort_in_lds<1>(buf, (int)n, pos_bits, passes, bits, cnt, tot, wsum);
    else if (n <= 4096)
        sort_in_lds<4>(buf, (int)n, pos_bits, passes, bits, cnt, tot, wsum);
    else
        sort_in_lds<16>(buf, (int)n, pos_bits, passes, bits, cnt, tot, wsum);
    for (int i = tid; i < (int)n; i += 1024) {
        stg(skey + out + i, lo + (buf[i] >> pos_bits));
        stg(spos + out + i, buf[i] & ((1u << pos_bits) - 1));
    }
}

// Up to RANK_T tokens: an item's place is the number of ids below its own and of equal ones
// before it, counted among all of them in LDS.  A workgroup places RANK_ITEMS items,
// RANK_LANES lanes an item; no passes, and no barrier but the one behind the loads.  Its
// work grows with the tokens' square, so it ends where the digits win.  Measured, by digits
// and by counting: 64 tokens 8.2 and 2.8 us, 1000 9.5 and 4.0, 4096 10.8 and 6.9; with zeros of 33
// MB beside them 4096 14.2 and 11.8, with 268 MB 37.1 and 39.5.
__global__ __launch_bounds__(1024) void sort_rank_kernel(const void* ids, int id64, int64_t vocab, int tokens, int sorters,
                                                         uint32_t* skey, uint32_t* spos, Fill fill) {
    typedef uint32_t U4 __attribute__((ext_vector_type(4)));
    __shared__ U4 keys[RANK_T / 4];
    if ((int)blockIdx.x >= sorters) {
        fill_zeros(fill, blockIdx.x - sorters, gridDim.x - sorters);
        return;
    }
    const int tid = threadIdx.x;
    uint32_t key[RANK_T / 1024];
#pragma unroll
    for (int r = 0; r < RANK_T / 1024; ++r) key[r] = key_at(ids, id64, vocab, min(tid + r * 1024, tokens - 1));
#pragma unroll
    for (int r = 0; r < RANK_T / 1024; ++r)
        // above every id behind the last token
        ((uint32_t*)keys)[tid + r * 1024] = tid + r * 1024 < tokens ? key[r] : 0xffffffffu;
    __syncthreads();
    // ids before the item count if they are below mine + 1, ids behind it below mine; of the
    // four of the read that holds the item, those before it are looked at again
    const int i = blockIdx.x * RANK_ITEMS + tid / RANK_LANES, lane = tid % RANK_LANES;
    const uint32_t mine = ((const uint32_t*)keys)[min(i, RANK_T - 1)];
    uint32_t place = 0;
    static_assert(RANK_T % (16 * RANK_LANES) == 0, "whole turns");
    for (int j0 = 0; j0 < tokens; j0 += 16 * RANK_LANES) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + (u * RANK_LANES + lane) * 4;
            const U4 k = keys[j >> 2];
            const uint32_t below = mine + (j + 3 < i ? 1u : 0u);
#pragma unroll
            for (int q = 0; q < 4; ++q) place += k[q] < below ? 1u : 0u;
        }
    }
    const U4 k = keys[min(i, RANK_T - 1) >> 2];
    if (lane == 0)
#pragma unroll
        for (int q = 0; q < 3; ++q) place += q < (i & 3) && k[q] == mine ? 1u : 0u;
#pragma unroll
    for (int o = RANK_LANES / 2; o >= 1; o >>= 1) place += (uint32_t)__shfl_xor((int)place, o);
    if (lane == 0 && i < tokens) {
        stg(skey + place, mine);
        stg(spos + place, (uint32_t)i);
    }
}

struct SortPass {
    const void* ids;          // pass 0: the ids; else NULL
    const uint32_t* key;
    const uint32_t* pos;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* hist;           // [blocks][bins]
    int64_t vocab, tokens;
    int id64, shift, bits, nblk;
};

__global__ __launch_bounds__(512) void sort_count_kernel(SortPass s, Fill fill) {
    __shared__ uint32_t h[BINS];
    if ((int)blockIdx.x >= s.nblk) {
        fill_zeros(fill, blockIdx.x - s.nblk, gridDim.x - s.nblk);
        return;
    }
    const int tid = threadIdx.x, bins = 1 << s.bits;
    h[tid] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * SORT_TILE;
    uint32_t key[SORT_TILE / 512];
#pragma unroll
    for (int r = 0; r < SORT_TILE / 512; ++r) {
        const int64_t i = min(i0 + r * 512 + tid, s.tokens - 1);
        key[r] = s.ids ? key_at(s.ids, s.id64, s.vocab, i) : ldg(s.key + i);
    }
#pragma unroll
    for (int r = 0; r < SORT_TILE / 512; ++r)
        if (i0 + r * 512 + tid < s.tokens) atomicAdd(&h[(key[r] >> s.shift) & (uint32_t)(bins - 1)], 1u);
    __syncthreads();
    if (tid < bins) stg(s.hist + (int64_t)blockIdx.x * bins + tid, h[tid]);
}

__global__ __launch_bounds__(512) void sort_scatter_kernel(SortPass s, Fill fill) {
    __shared__ uint32_t cnt[TILE_WAVES * BINS];
    __shared__ uint32_t wsum[TILE_WAVES];
    if ((int)blockIdx.x >= s.nblk) {
        fill_zeros(fill, blockIdx.x - s.nblk, gridDim.x - s.nblk);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, bins = 1 << s.bits;
    for (int i = tid; i < TILE_WAVES * BINS; i += 512) cnt[i] = 0;
    __syncthreads();
    uint32_t key[TILE_ROUNDS], pos[TILE_ROUNDS], digit[TILE_ROUNDS], rank[TILE_ROUNDS];
    bool live[TILE_ROUNDS];
    const int64_t i0 = (int64_t)blockIdx.x * SORT_TILE + wv * TILE_ROUNDS * 64 + lane;
#pragma unroll
    for (int r = 0; r < TILE_ROUNDS; ++r) {
        const int64_t i = i0 + r * 64;
        live[r] = i < s.tokens;
        const int64_t in = min(i, s.tokens - 1);
        key[r] = s.ids ? key_at(s.ids, s.id64, s.vocab, in) : ldg(s.key + in);
        pos[r] = s.ids ? (uint32_t)in : ldg(s.pos + in);
        digit[r] = (key[r] >> s.shift) & (uint32_t)(bins - 1);
    }
    wave_ranks<TILE_ROUNDS>(digit, live, s.bits, cnt + wv * BINS, rank, TILE_ROUNDS);
    __syncthreads();
    // places: all tokens of smaller digits, then this digit's in earlier blocks
    uint32_t all = 0, before = 0;
    if (tid < bins)
        for (int b = 0; b < s.nblk; ++b) {
            const uint32_t c = ldg(s.hist + (int64_t)b * bins + tid);
            all += c;
            before += b < (int)blockIdx.x ? c : 0u;
        }
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = (uint32_t)__shfl_up((int)inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 63) wsum[wv] = inc;
    __syncthreads();
    uint32_t prior = 0;
    for (int w = 0; w < wv; ++w) prior += wsum[w];
    if (tid < bins) {
        uint32_t at = prior + inc - all + before;
        for (int w = 0; w < TILE_WAVES; ++w) {
            const uint32_t c = cnt[w * BINS + tid];
            cnt[w * BINS + tid] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < TILE_ROUNDS; ++r)
        if (live[r]) {
            const uint32_t at = cnt[wv * BINS + digit[r]] + rank[r];
            stg(s.key_out + at, key[r]);
            stg(s.pos_out + at, pos[r]);
        }
}

struct RunSum {
    const void* dout;
    const uint32_t* key;      // sorted ids
    const uint32_t* pos;      // their positions
    float* g;
    float* first;             // [chunks][pitch] run that began in an earlier chunk
    float* last;              // [chunks][pitch] run that begins here and goes on
    int64_t tokens, dim, pitch, lddout, ldg;
    uint32_t vocab, chunks, col_tiles;
    float scale;
    int accumulate;
};

// A lane's eight columns of a row; `whole`: no lane of the wave crosses the row's end.
struct Cols {
    int64_t c, dim;
    int n;                    // valid columns, 0..8
    bool whole;
};
__device__ __forceinline__ Cols lane_cols(int64_t tile, int64_t dim) {
    Cols k;
    k.c = tile * COLS + (threadIdx.x & 63) * 8;
    k.dim = dim;
    k.n = (int)max((int64_t)0, min((int64_t)8, dim - k.c));
    k.whole = dim >= 8 && __all(k.n == 8 || k.n == 0);
    return k;
}
template <class T>
__device__ __forceinline__ typename Vec8<T>::Raw load_cols(const T* row, const Cols& k) {
    return k.whole ? load8(row + (k.n ? k.c : 0)) : load8_edge(row, k.c, k.dim);
}

// One wave per sorted position and 512 columns; it has work where a run of equal ids begins, or
// a chunk does inside one, and sums the run's tokens up to the chunk's end.
template <class T, bool ACC>
__global__ __launch_bounds__(256) void run_sums_kernel(RunSum s) {
    const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t i = wave / s.col_tiles;
    if (i >= s.tokens) return;
    const int lane = threadIdx.x & 63;
    // lane l holds sorted position i - 1 + l (the ends again beyond the list)
    const int64_t in = min(max(i - 1 + lane, (int64_t)0), s.tokens - 1);
    const uint32_t k = ldg(s.key + in), p = ldg(s.pos + in);
    const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)k, 1);
    if (key >= s.vocab) return;                              // tokens without a row come last
    const int begin = (int)(i % CHUNK);
    const uint64_t same = __ballot(k == key && i - 1 + lane < s.tokens);
    const bool begun_before = i > 0 && (same & 1);
    if (begun_before && begin != 0) return;
    const int run = __builtin_ctzll(~(same >> 1));           // 63 at most: more than a chunk
    const int count = min(run, CHUNK - begin);
    const bool goes_on = run > count;
    const Cols cols = lane_cols(wave - (uint32_t)i * s.col_tiles, s.dim);
    const auto row = [&](int j) {
        const T* d = (const T*)s.dout + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)p, 1 + j) * s.lddout;
        return load_cols(d, cols);
    };
    const bool whole_run = !begun_before && !goes_on;
    float* g = s.g + (int64_t)key * s.ldg;
    typename Vec8<float>::Raw old = {};
    if (ACC && whole_run) old = load_cols((const float*)g, cols);
    floatx8 acc = Vec8<T>::get(row(0));
    for (int j = 1; j < count; j += 4) {
        typename Vec8<T>::Raw r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = row(min(j + q, count - 1));
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (j + q < count) acc += Vec8<T>::get(r[q]);
    }
    if (cols.n == 0) return;
    if (whole_run) {
        acc *= s.scale;
        if constexpr (ACC) acc += Vec8<float>::get(old);
        store8_n(g + cols.c, Vec8<float>::put(acc), cols.n);
    } else {
        store8((begun_before ? s.first : s.last) + i / CHUNK * s.pitch + cols.c, Vec8<float>::put(acc));
    }
}

constexpr int BATCH = 4;                     // positions processed while the next are on their way

// The same by one wave per chunk and 512 columns, for long lists.  With ACC the rows of G that
// a run is added to are loaded beside its tokens', for every position (those of one run are
// one row).  WHOLE: Cols::whole.
template <class T, bool ACC, bool WHOLE>
__device__ __forceinline__ void chunk_sums(const RunSum& s, const Cols& cols, uint32_t chunk, uint32_t k, uint32_t p) {
    using Raw = typename Vec8<T>::Raw;
    using RawG = typename Vec8<float>::Raw;
    const int64_t c = WHOLE && cols.n == 0 ? 0 : cols.c;
    const auto load = [&](Raw (&r)[BATCH], RawG (&g)[BATCH], int b) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            // positions past the end and tokens without a row load a row that exists
            const uint32_t row = (uint32_t)__builtin_amdgcn_readlane((int)p, b + i);
            const T* d = (const T*)s.dout + (int64_t)row * s.lddout;
            r[i] = WHOLE ? load8(d + c) : load8_edge(d, c, s.dim);
            if constexpr (ACC) {
                const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)k, b + i);
                const float* e = s.g + (int64_t)(key < s.vocab ? key : 0) * s.ldg;
                g[i] = WHOLE ? load8(e + c) : load8_edge(e, c, s.dim);
            }
        }
    };
    floatx8 acc = {};
    // the key before the chunk is on lane CHUNK, the one after it on lane CHUNK + 1
    bool begun_before = __builtin_amdgcn_readlane((int)k, 0) == __builtin_amdgcn_readlane((int)k, CHUNK);
    Raw r[BATCH], r2[BATCH];
    RawG g[BATCH], g2[BATCH];
    load(r, g, 0);
#pragma unroll 1
    for (int b = 0; b < CHUNK; b += BATCH) {
        load(r2, g2, b + BATCH < CHUNK ? b + BATCH : b);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)k, b + i);
            if (key >= s.vocab) return;        // tokens without a row come last
            const bool at_end = b + i + 1 == CHUNK;
            const uint32_t after = (uint32_t)__builtin_amdgcn_readlane((int)k, at_end ? CHUNK + 1 : b + i + 1);
            acc += Vec8<T>::get(r[i]);
            if (key != after || at_end) {
                const bool goes_on = at_end && key == after;
                if (begun_before || goes_on) {
                    float* part = (begun_before ? s.first : s.last) + (int64_t)chunk * s.pitch + cols.c;
                    if (cols.n > 0) store8(part, Vec8<float>::put(acc));
                } else {
                    floatx8 v = acc * s.scale;
                    if constexpr (ACC) v += Vec8<float>::get(g[i]);
                    float* row = s.g + (int64_t)key * s.ldg + cols.c;
                    if (!WHOLE)
                        store8_n(row, Vec8<float>::put(v), cols.n);
                    else if (cols.n > 0)
                        store8(row, Vec8<float>::put(v));
                }
                acc = floatx8{};
                begun_before = false;
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            r[i] = r2[i];
            g[i] = g2[i];
        }
    }
}

template <class T, bool ACC>
__global__ __launch_bounds__(256) void chunk_sums_kernel(RunSum s) {
    const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    const uint32_t chunk = wave / s.col_tiles;
    if (chunk >= s.chunks) return;
    const int lane = threadIdx.x & 63;
    const Cols cols = lane_cols(wave - chunk * s.col_tiles, s.dim);
    const int64_t i0 = (int64_t)chunk * CHUNK;
    const int count = (int)min((int64_t)CHUNK, s.tokens - i0);
    // lane i < CHUNK holds position i0 + i; lanes CHUNK and CHUNK + 1 the keys on either side
    const int64_t at = lane < CHUNK ? i0 + lane : lane == CHUNK ? i0 - 1 : i0 + CHUNK;
    const bool have = (lane < count || lane >= CHUNK) && lane <= CHUNK + 1 && at >= 0 && at < s.tokens;
    const int64_t in = min(max(at, (int64_t)0), s.tokens - 1);
    uint32_t k = ldg(s.key + in), p = ldg(s.pos + in);
    if (!have) k = 0xffffffffu;
    if (cols.whole)
        chunk_sums<T, ACC, true>(s, cols, chunk, k, p);
    else
        chunk_sums<T, ACC, false>(s, cols, chunk, k, p);
}

// Partial rows from, from + step, .. up to `end` of the run that begins in `chunk`, in order,
// four in flight.
__device__ __forceinline__ floatx8 add_parts(const RunSum& s, uint32_t chunk, uint32_t from, uint32_t step, uint32_t end,
                                             int64_t c) {
    floatx8 acc = {};
    for (uint32_t j = from; j <= end; j += 4 * step) {
        typename Vec8<float>::Raw r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t k = min(j + i * step, end);
            r[i] = load8((k == chunk ? s.last : s.first) + (int64_t)k * s.pitch + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i * step <= end) acc += Vec8<float>::get(r[i]);
    }
    return acc;
}

// Runs over several chunks: the partial rows of one, in order.  A wave looks at one chunk and
// 512 columns, and adds a short run by itself; the waves of a workgroup share a long one,
// each taking every JOIN_WAVES-th partial row, joined in the order of the waves.
__global__ __launch_bounds__(64 * JOIN_WAVES) void join_runs_kernel(RunSum s) {
    __shared__ float part[JOIN_WAVES][COLS];
    __shared__ uint32_t ends[JOIN_WAVES];
    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t wave = blockIdx.x * JOIN_WAVES + wv;
    uint32_t chunk = wave / s.col_tiles, key = 0, end = 0;   // end: last chunk of the run, 0: none
    const int64_t i0 = (int64_t)chunk * CHUNK, i1 = i0 + CHUNK;
    if (i1 < s.tokens) {
        // the keys around the chunk's ends, loaded together
        const uint32_t last = ldg(s.key + i1 - 1), after = ldg(s.key + i1), first = ldg(s.key + i0);
        const uint32_t before = ldg(s.key + max(i0 - 1, (int64_t)0));
        const bool begun_before = first == last && i0 > 0 && before == last;
        if (last < s.vocab && after == last && !begun_before) {
            key = last;
            // the chunks after this one that begin with the same id, 64 at a time
            end = chunk;
            uint64_t same;
            do {
                const int64_t i = ((int64_t)end + 1 + lane) * CHUNK;
                same = __ballot(i < s.tokens && ldg(s.key + min(i, s.tokens - 1)) == key);
                end += ~same ? (uint32_t)__builtin_ctzll(~same) : 64u;
            } while (~same == 0);
        }
    }
    const auto put = [&](const Cols& cols, uint32_t row, floatx8 acc) {
        if (cols.n == 0) return;
        acc *= s.scale;
        float* g = s.g + (int64_t)row * s.ldg;
        if (s.accumulate) acc += Vec8<float>::get(load8_edge(g, cols.c, s.dim));
        store8_n(g + cols.c, Vec8<float>::put(acc), cols.n);
    };
    const bool is_long = end > chunk + 2 * JOIN_WAVES;
    if (end && !is_long) {
        const Cols cols = lane_cols(wave - chunk * s.col_tiles, s.dim);
        const int64_t c = cols.n > 0 ? cols.c : 0;           // partial rows are padded to eights
        put(cols, key, add_parts(s, chunk, chunk, 1, end, c));
    }
    if (lane == 0) ends[wv] = is_long ? end : 0;
    __syncthreads();
    for (int v = 0; v < JOIN_WAVES; ++v) {
        const uint32_t last = ends[v];
        if (last == 0) continue;                             // the same for every thread
        const uint32_t w = blockIdx.x * JOIN_WAVES + v;
        chunk = w / s.col_tiles;
        const Cols cols = lane_cols(w - chunk * s.col_tiles, s.dim);
        const int64_t c = cols.n > 0 ? cols.c : 0;
        floatx8 acc = add_parts(s, chunk, chunk + wv, JOIN_WAVES, last, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[wv][i * 64 + lane] = acc[i];
        __syncthreads();
        if (wv == 0) {
            for (int u = 1; u < JOIN_WAVES; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += part[u][i * 64 + lane];
            put(cols, ldg(s.key + (int64_t)(chunk + 1) * CHUNK), acc);
        }
        __syncthreads();
    }
}

template <class T>
void run_sums_of(const RunSum& r, hipStream_t stream) {
    // A wave per position while all of them are resident at once (eight a SIMD), else a wave
    // per chunk.  Measured, position against chunk: 1000 x 577 fp32 added 6.9 and 15.6 us,
    // 1000 x 1024 bf16 7.2 and 8.1, 4000 x 1024 bf16 9.5 and 8.3, 16384 x 1024 bf16 31 and 20.
    if (r.tokens * r.col_tiles <= 8192) {
        const dim3 grid((uint32_t)((r.tokens * r.col_tiles + 3) / 4));
        if (r.accumulate)
            S4_LAUNCH((run_sums_kernel<T, true>), grid, dim3(256), 0, stream, r);
        else
            S4_LAUNCH((run_sums_kernel<T, false>), grid, dim3(256), 0, stream, r);
    } else {
        const dim3 grid((r.chunks * r.col_tiles + 3) / 4);
        if (r.accumulate)
            S4_LAUNCH((chunk_sums_kernel<T, true>), grid, dim3(256), 0, stream, r);
        else
            S4_LAUNCH((chunk_sums_kernel<T, false>), grid, dim3(256), 0, stream, r);
    }
}

struct GradPlan {
    int64_t chunks, nblk;
    int bits, passes, digit, pos_bits, parts;
    uint32_t range;           // ids a part of the small sort
    bool small;
    size_t off_key[2], off_pos[2], off_hist, off_first, off_last, total;
};
GradPlan grad_plan(int64_t tokens, int64_t vocab, int64_t dim) {
    GradPlan p;
    p.chunks = (tokens + CHUNK - 1) / CHUNK;
    p.bits = bit_length((uint64_t)vocab);                    // keys 0 .. vocab
    p.pos_bits = bit_length((uint64_t)(tokens > 0 ? tokens - 1 : 0));
    // a part for every 512 tokens: 16384 tokens into 65536 rows sort in 33 us in one part
    p.parts = (int)std::min<int64_t>(16, std::max<int64_t>(1, tokens / 512));
    p.range = (uint32_t)((vocab + p.parts) / p.parts);
    const int part_bits = std::max(1, bit_length(p.range - 1));
    // id and position in one word: larger tables sort in blocks, whatever the tokens
    p.small = tokens <= SMALL_T && part_bits + p.pos_bits <= 32;
    if (p.small) p.bits = part_bits;
    p.passes = (p.bits + RADIX_BITS - 1) / RADIX_BITS;
    p.digit = (p.bits + p.passes - 1) / p.passes;
    p.nblk = (tokens + SORT_TILE - 1) / SORT_TILE;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    for (int i = 0; i < 2; ++i) {
        p.off_key[i] = take((size_t)tokens * 4);
        p.off_pos[i] = take((size_t)tokens * 4);
    }
    p.off_hist = take(p.small ? 0 : (size_t)p.nblk * BINS * 4);
    p.off_first = take((size_t)p.chunks * ((dim + 7) / 8 * 8) * 4);
    p.off_last = take((size_t)p.chunks * ((dim + 7) / 8 * 8) * 4);
    p.total = at;
    return p;
}

}  // namespace

hipError_t launch_embedding(shampoo4_dtype dtype, const Embed& e, hipStream_t stream) {
    const uint32_t nvec = (uint32_t)((e.dim + 7) / 8);
    const uint64_t total = (uint64_t)e.tokens * nvec;
    if (total == 0) return hipSuccess;
    const dim3 grid((uint32_t)std::min<uint64_t>((total + 255) / 256, 1u << 20));
    switch (dtype) {
        case SHAMPOO4_BF16: S4_LAUNCH(embedding_kernel<__bf16>, grid, dim3(256), 0, stream, e, nvec, total); break;
        case SHAMPOO4_F16: S4_LAUNCH(embedding_kernel<_Float16>, grid, dim3(256), 0, stream, e, nvec, total); break;
        default: S4_LAUNCH(embedding_kernel<float>, grid, dim3(256), 0, stream, e, nvec, total);
    }
    return hipGetLastError();
}

size_t embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    return grad_plan(tokens, vocab, dim).total;
}

hipError_t launch_embedding_grad(shampoo4_dtype dtype, const EmbedGrad& e, void* workspace, hipStream_t stream) {
    const GradPlan p = grad_plan(e.tokens, e.vocab, e.dim);
    char* ws = (char*)workspace;
    Fill fill{e.accumulate ? nullptr : e.g, e.vocab, e.dim, e.ldg, 0, 1};
    // workgroups that fill, 16 KB a turn each: a whole number, up to `each`, for every CU that
    // the sort leaves free (in the small sort its LDS lets one run on a CU at a time, so a
    // remainder would cost a whole turn of them: 46 us against 40 at 65536 x 1024)
    const int64_t fill_bytes = e.accumulate ? 0 : e.vocab * e.dim * 4;
    const auto fill_blocks = [&](int64_t sorters, int launches, int each) {
        const int64_t cus = std::max<int64_t>(64, 256 - sorters);
        const int64_t turns = (fill_bytes / launches + 16383) / 16384;
        return (uint32_t)std::min(turns, std::min<int64_t>(each, (turns + cus - 1) / cus) * cus);
    };
    uint32_t *skey, *spos;
    if (e.tokens == 0 && fill_bytes == 0) return hipSuccess;
    if (e.tokens <= RANK_T || p.small) {
        skey = (uint32_t*)(ws + p.off_key[0]);
        spos = (uint32_t*)(ws + p.off_pos[0]);
    }
    if (e.tokens <= RANK_T) {
        const int sorters = (int)(e.tokens + RANK_ITEMS - 1) / RANK_ITEMS;    // no tokens: nothing is read
        S4_LAUNCH(sort_rank_kernel, dim3(sorters + fill_blocks(sorters, 1, 4)), dim3(1024), 0, stream, e.ids, e.id64,
                  e.vocab, (int)e.tokens, sorters, skey, spos, fill);
    } else if (p.small) {
        S4_LAUNCH(sort_small_kernel, dim3(p.parts + fill_blocks(p.parts, 1, 4)), dim3(1024), 0, stream, e.ids, e.id64,
                  e.vocab, (int)e.tokens, p.parts, p.range, p.passes, p.digit, p.pos_bits, skey, spos, fill);
    } else {
        fill.parts = 2 * p.passes;
        const uint32_t nf = fill_blocks(p.nblk, fill.parts, 4);
        for (int k = 0; k < p.passes; ++k) {
            SortPass s;
            s.ids = k == 0 ? e.ids : nullptr;
            s.key = (uint32_t*)(ws + p.off_key[(k + 1) & 1]);
            s.pos = (uint32_t*)(ws + p.off_pos[(k + 1) & 1]);
            s.key_out = (uint32_t*)(ws + p.off_key[k & 1]);
            s.pos_out = (uint32_t*)(ws + p.off_pos[k & 1]);
            s.hist = (uint32_t*)(ws + p.off_hist);
            s.vocab = e.vocab;
            s.tokens = e.tokens;
            s.id64 = e.id64;
            s.shift = k * p.digit;
            s.bits = p.digit;
            s.nblk = (int)p.nblk;
            fill.part = 2 * k;
            S4_LAUNCH(sort_count_kernel, dim3((uint32_t)p.nblk + nf), dim3(512), 0, stream, s, fill);
            fill.part = 2 * k + 1;
            S4_LAUNCH(sort_scatter_kernel, dim3((uint32_t)p.nblk + nf), dim3(512), 0, stream, s, fill);
        }
        skey = (uint32_t*)(ws + p.off_key[(p.passes - 1) & 1]);
        spos = (uint32_t*)(ws + p.off_pos[(p.passes - 1) & 1]);
    }
    if (e.tokens == 0) return hipGetLastError();
    RunSum r;
    r.dout = e.dout;
    r.key = skey;
    r.pos = spos;
    r.g = e.g;
    r.first = (float*)(ws + p.off_first);
    r.last = (float*)(ws + p.off_last);
    r.tokens = e.tokens;
    r.dim = e.dim;
    r.pitch = (e.dim + 7) / 8 * 8;
    r.lddout = e.lddout;
    r.ldg = e.ldg;
    r.vocab = (uint32_t)e.vocab;
    r.chunks = (uint32_t)p.chunks;
    r.col_tiles = (uint32_t)((e.dim + COLS - 1) / COLS);
    r.scale = e.scale;
    r.accumulate = e.accumulate;
    const uint32_t waves = r.chunks * r.col_tiles;
    switch (dtype) {
        case SHAMPOO4_BF16: run_sums_of<__bf16>(r, stream); break;
        case SHAMPOO4_F16: run_sums_of<_Float16>(r, stream); break;
        default: run_sums_of<float>(r, stream);
    }
    if (r.chunks > 1)
        S4_LAUNCH(join_runs_kernel, dim3((waves + JOIN_WAVES - 1) / JOIN_WAVES), dim3(64 * JOIN_WAVES), 0, stream, r);
    return hipGetLastError();
}

}  // namespace s4
