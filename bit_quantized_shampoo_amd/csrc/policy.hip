// Clipped policy loss with a KL term on logits, forward and backward in one pass over them,
// and the token log-probabilities alone.
//
// A row's softmax statistics are a maximum and a sum of exponentials beside it, in fp32:
// logp = (z_y - m) - log s, and dZ = c ([v = y] - exp(z - m) / s) with one coefficient c a
// row.  Two schedules:
//  * Row kernel: a workgroup keeps a whole row in registers (64 registers of a thread), so
//    the logits are read once and the gradient written once.  Rows up to 1024 threads x 64
//    registers: 131072 16-bit logits, 65536 in fp32.
//  * Split kernels, for few rows (which would leave most of the GPU idle) and for longer
//    ones: a launch of partial statistics over pieces of a row, and a launch that joins a
//    row's pieces and writes its gradient piece by piece (the logits are read again).
// The loss is summed in a fixed order: row terms by one workgroup at the end.
//
// Bound by HBM: 4096 rows of 65536 bf16 logits with their gradient in 198 us (5.4 TB/s for
// 1.07 GB; a plain copy reaches 5.1), the loss's launch 5.1 more, behind it; the log-probabilities
// alone of 2048 rows of 65536 in 40.5 us bf16 (6.6 TB/s) and 95 fp32 (5.6), calls behind each other.  The counters
// show every logit read once (and rows that do not count not at all) and every gradient
// written once.  Few rows are bound by their two launches: 8 rows of 40961 fp32 logits 4.0
// and 4.5 us.
#include <algorithm>

#include "train_common.hpp"
#include "train.hpp"

namespace s4 {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_inff();
constexpr float WHOLE_REF = 1073741824.f;    // 2^30

// The sums' reference point goes by a maximum m.  Up to |m| = 2^30 it is kept in powers of two
// and whole, c = round(m log2e): z - reference = z log2e - c is one fused multiply-add with
// one rounding, two sums are brought together by an exact power of two, and
// logp = ln2 ((z_y log2e - c) - log2 s) meets no rounding of the reference.  c is then off by
// at most half its spacing, 64, so the maximum's own term is within 2^-64 .. 2^64.  For larger
// m the spacing passes the exponent's range, and the reference is m itself, exactly, with
// differences taken as they are: floats beyond 2^30 are 128 or more apart, so exp2(z - m) is
// 1 or 0 (below 2^-127) as exp(z - m) is.  So are two sums of which one has a reference of
// each kind: the smaller one is 0.  A set with no probability (every logit -infinity) has
// m = -infinity and the sum 0.
struct Base {
    float k, c;               // exp(z - reference) = exp2(z k - c)
};
__device__ __forceinline__ Base base_of(float m) {
    if (m == NEG_INF) return {LOG2E, 0.f};
    return fabsf(m) <= WHOLE_REF ? Base{LOG2E, rintf(m * LOG2E)} : Base{1.f, m};
}
__device__ __forceinline__ float exp_at(float z, Base b) {
    return __builtin_amdgcn_exp2f(fmaf(z, b.k, -b.c));
}
// A set's sum s, of maximum m, brought to the reference `to` of a maximum that is not smaller (a
// NaN sum stays NaN).
__device__ __forceinline__ float rebase(float s, float m, Base to) {
    const Base b = base_of(m);
    return s * (m != NEG_INF && b.k == to.k ? __builtin_amdgcn_exp2f(b.c - to.c) : 0.f);
}
__device__ __forceinline__ float log_prob(float zy, Base b, float s) {
    const float l = __builtin_amdgcn_logf(s);
    if (b.k != 1.f && fabsf(zy) <= WHOLE_REF) return LN2 * (fmaf(zy, b.k, -b.c) - l);
    // beyond, z_y log2e may pass fp32's range where logp does not
    return (zy - (b.k == 1.f ? b.c : LN2 * b.c)) - LN2 * l;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Eight logits of -infinity.
template <class T>
__device__ __forceinline__ typename Vec8<T>::Raw no_logits() {
    floatx8 f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = NEG_INF;
    return Vec8<T>::put(f);
}
__device__ __forceinline__ float max8(float m, floatx8 f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, f[j]);
    return m;
}
__device__ __forceinline__ float add_exp8(float s, floatx8 f, Base base) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        a += exp_at(f[j], base);
        b += exp_at(f[j + 1], base);
    }
    return s + (a + b);
}

// Target of a row, or -1: out of range, or a row that does not count.
__device__ __forceinline__ int64_t target_of(const Policy& p, int64_t t) {
    const int64_t y = p.id64 ? ldg((const int64_t*)p.targets + t) : (int64_t)ldg((const int32_t*)p.targets + t);
    if (y < 0 || y >= p.vocab) return -1;
    if (p.train && ldg(p.weights + t) == 0.f) return -1;
    return y;
}

// exp(d) - 1 - d from e = expm1(d).  Near 0, where policies are close to their reference, the
// difference would keep d^2 / 2 to 2^-24 of d only: the series d^2 (1/2 + d/6 + d^2/24 + ..) there,
// whose terms from d^9 on are below 2^-24 of it for |d| <= 1/2.
__device__ __forceinline__ float kl_term(float d, float e) {
    if (!(fabsf(d) <= 0.5f)) return e - d;
    float p = 1.f / 40320.f;                                 // 1 / 8!
    p = fmaf(p, d, 1.f / 5040.f);
    p = fmaf(p, d, 1.f / 720.f);
    p = fmaf(p, d, 1.f / 120.f);
    p = fmaf(p, d, 1.f / 24.f);
    p = fmaf(p, d, 1.f / 6.f);
    return d * d * fmaf(p, d, 0.5f);
}

// The row's weighted loss, and the coefficient of its gradient.
struct RowTerm {
    float loss, coef;
};
__device__ __forceinline__ RowTerm row_term(const Policy& p, int64_t t, float logp) {
    const float w = ldg(p.weights + t), adv = ldg(p.adv + t);
    const float x = logp - ldg(p.old_logp + t);
    const float r = expf(x);
    // no advantage counts for nothing, also where a finite x has a ratio beyond fp32
    const float plain = adv == 0.f && x < -NEG_INF ? 0.f : r * adv;
    const float clipped = fminf(fmaxf(r, 1.f - p.clip_low), 1.f + p.clip_high) * adv;
    // a NaN ratio or advantage stays NaN
    float l = plain <= clipped ? -plain : clipped <= plain ? -clipped : plain + clipped;
    float g = plain <= clipped ? -plain : clipped <= plain ? 0.f : plain + clipped;
    if (p.kl > 0.f) {
        const float d = ldg(p.ref_logp + t) - logp;
        const float e = expm1f(d);
        l += p.kl * kl_term(d, e);
        g -= p.kl * e;
    }
    return {w * l, p.grad_scale * (w * g)};
}

template <class T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void policy_row_kernel(Policy p, float* __restrict__ terms) {
    constexpr int WAVES = THREADS / 64;
    __shared__ float wmax[WAVES], wsum[WAVES], zy;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int64_t t = blockIdx.x;
    const T* z = (const T*)p.logits + t * p.ldz;
    T* dz = p.dlogits ? (T*)p.dlogits + t * p.ldd : nullptr;
    const int nfull = (int)(p.vocab >> 3);                   // whole vectors; the tail is one element a thread
    const int tail = (int)p.vocab & 7;
    const int64_t y = target_of(p, t);
    if (y < 0) {
        if (dz) {
            for (int v = tid; v < nfull; v += THREADS) store8(dz + (int64_t)v * 8, typename Vec8<T>::Raw{});
            if (tid < tail) dz[(int64_t)nfull * 8 + tid] = (T)0.f;
        }
        if (tid == 0) {
            if (p.logp) stg(p.logp + t, 0.f);
            if (p.train) stg(terms + t, 0.f);
        }
        return;
    }
    typename Vec8<T>::Raw r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = j * THREADS + tid;
        r[j] = no_logits<T>();
        if (v < nfull) r[j] = load8(z + (int64_t)v * 8);
    }
    float last = NEG_INF;
    if (tid < tail) last = (float)z[(int64_t)nfull * 8 + tid];
    if (tid == 0) zy = (float)z[y];

    float m = last;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        m = max8(m, Vec8<T>::get(r[j]));
        unpack_again(r[j]);
    }
    m = wave_max(m);
    Base base = base_of(m);
    float s = exp_at(last, base);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        s = add_exp8(s, Vec8<T>::get(r[j]), base);
        unpack_again(r[j]);
    }
    s = wave_add(s);
    if (lane == 0) {
        wmax[wv] = m;
        wsum[wv] = s;
    }
    __syncthreads();
    // every wave joins the waves' sums, lane i taking wave i's
    m = lane < WAVES ? wmax[lane] : NEG_INF;
    s = lane < WAVES ? wsum[lane] : 0.f;
    base = base_of(wave_max(m));
    s = wave_add(rebase(s, m, base));
    const float logp = log_prob(zy, base, s);
    if (tid == 0 && p.logp) stg(p.logp + t, logp);
    if (!p.train) return;
    const RowTerm term = row_term(p, t, logp);
    if (tid == 0) stg(terms + t, term.loss);
    if (!dz) return;
    const float scale = -term.coef / s;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = j * THREADS + tid;
        if (v < nfull) {
            floatx8 f = Vec8<T>::get(r[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = scale * exp_at(f[i], base);
            if (v == (int)(y >> 3)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += i == (int)(y & 7) ? term.coef : 0.f;
            }
            store8(dz + (int64_t)v * 8, Vec8<T>::put(f));
        }
    }
    if (tid < tail) {
        const int64_t v = (int64_t)nfull * 8 + tid;
        dz[v] = (T)(scale * exp_at(last, base) + (v == y ? term.coef : 0.f));
    }
}

// -- split rows --------------------------------------------------------------------------

struct Pieces {
    float* stat;              // [rows][pieces][2]: maximum and sum
    float* zy;                // [rows] target logit
    int64_t pieces;           // per row
    int64_t vecs;             // vectors per piece
};

template <class T>
__global__ __launch_bounds__(256) void policy_part_kernel(Policy p, Pieces q) {
    __shared__ float wmax[4], wsum[4];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int64_t t = blockIdx.x / q.pieces, piece = blockIdx.x - t * q.pieces;
    const int64_t y = target_of(p, t);
    if (y < 0) return;
    const T* z = (const T*)p.logits + t * p.ldz;
    const int64_t nfull = p.vocab >> 3;
    const int tail = (int)p.vocab & 7;
    const int64_t v0 = piece * q.vecs, v1 = min(nfull, v0 + q.vecs);
    float top = NEG_INF, s = 0.f;
    for (int64_t v = v0 + tid; v < v1; v += 1024) {
        typename Vec8<T>::Raw r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = no_logits<T>();
            if (v + j * 256 < v1) r[j] = load8(z + (v + j * 256) * 8);
        }
        float m = top;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max8(m, Vec8<T>::get(r[j]));
        const Base base = base_of(m);
        s = rebase(s, top, base);
        top = m;
#pragma unroll
        for (int j = 0; j < 4; ++j) s = add_exp8(s, Vec8<T>::get(r[j]), base);
    }
    if (piece == q.pieces - 1 && tid < tail) {
        const float x = (float)z[nfull * 8 + tid];
        const float m = fmaxf(top, x);
        const Base base = base_of(m);
        s = rebase(s, top, base) + exp_at(x, base);
        top = m;
    }
    const float m = wave_max(top);
    s = wave_add(rebase(s, top, base_of(m)));
    if (lane == 0) {
        wmax[wv] = m;
        wsum[wv] = s;
    }
    __syncthreads();
    if (tid == 0) {
        float a = wmax[0];
        for (int w = 1; w < 4; ++w) a = fmaxf(a, wmax[w]);
        float b = 0.f;
        for (int w = 0; w < 4; ++w) b += rebase(wsum[w], wmax[w], base_of(a));
        float* o = q.stat + 2 * (t * q.pieces + piece);
        stg(o, a);
        stg(o + 1, b);
        if (piece == 0) stg(q.zy + t, (float)z[y]);
    }
}

struct RowStat {
    Base base;
    float s;
};
// A row's statistics from its pieces, by one wave.
__device__ __forceinline__ RowStat join_pieces(const Pieces& q, int64_t t) {
    const int lane = threadIdx.x & 63;
    const float* st = q.stat + 2 * t * q.pieces;
    float m = NEG_INF;
    for (int64_t i = lane; i < q.pieces; i += 64) m = fmaxf(m, ldg(st + 2 * i));
    const Base base = base_of(wave_max(m));
    float s = 0.f;
    for (int64_t i = lane; i < q.pieces; i += 64) s += rebase(ldg(st + 2 * i + 1), ldg(st + 2 * i), base);
    return {base, wave_add(s)};
}

// Log-probabilities, and the rows' terms when training: one wave a row.
__global__ __launch_bounds__(256) void policy_join_kernel(Policy p, Pieces q, float* __restrict__ terms) {
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.rows) return;
    float logp = 0.f, term = 0.f;
    if (target_of(p, t) >= 0) {
        const RowStat st = join_pieces(q, t);
        logp = log_prob(ldg(q.zy + t), st.base, st.s);
        if (p.train) term = row_term(p, t, logp).loss;
    }
    if ((threadIdx.x & 63) == 0) {
        if (p.logp) stg(p.logp + t, logp);
        if (p.train) stg(terms + t, term);
    }
}

// The loss and the log-probabilities of a few rows, by one workgroup of 256: sixteen lanes a
// row, each row's terms in order.
__device__ void few_rows_loss(const Policy& p, const Pieces& q) {
    __shared__ float part[16];
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    float sum = 0.f;
    for (int64_t t = group; t < p.rows; t += 16) {
        float logp = 0.f;
        if (target_of(p, t) >= 0) {
            const float* st = q.stat + 2 * t * q.pieces;
            float m = NEG_INF;
            for (int64_t i = lane; i < q.pieces; i += 16) m = fmaxf(m, ldg(st + 2 * i));
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
            const Base base = base_of(m);
            float s = 0.f;
            for (int64_t i = lane; i < q.pieces; i += 16) s += rebase(ldg(st + 2 * i + 1), ldg(st + 2 * i), base);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) s += __shfl_xor(s, o);
            logp = log_prob(ldg(q.zy + t), base, s);
            sum += row_term(p, t, logp).loss;
        }
        if (lane == 0 && p.logp) stg(p.logp + t, logp);
    }
    if (lane == 0) part[group] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) sum += part[i];
        stg(p.loss, sum);
    }
}

// A piece of a row's gradient; with LOSS, one more workgroup writes the loss and the
// log-probabilities beside them.
template <class T, bool LOSS>
__global__ __launch_bounds__(256) void policy_grad_kernel(Policy p, Pieces q) {
    if (LOSS && blockIdx.x == gridDim.x - 1) {
        few_rows_loss(p, q);
        return;
    }
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x / q.pieces, piece = blockIdx.x - t * q.pieces;
    const T* z = (const T*)p.logits + t * p.ldz;
    T* dz = (T*)p.dlogits + t * p.ldd;
    const int64_t nfull = p.vocab >> 3;
    const int tail = piece == q.pieces - 1 ? (int)p.vocab & 7 : 0;
    const int64_t v0 = piece * q.vecs, v1 = min(nfull, v0 + q.vecs);
    const int64_t y = target_of(p, t);
    if (y < 0) {
        for (int64_t v = v0 + tid; v < v1; v += 256) store8(dz + v * 8, typename Vec8<T>::Raw{});
        if (tid < tail) dz[nfull * 8 + tid] = (T)0.f;
        return;
    }
    const RowStat st = join_pieces(q, t);
    const float coef = row_term(p, t, log_prob(ldg(q.zy + t), st.base, st.s)).coef;
    const float scale = -coef / st.s;
    const Base base = st.base;
    for (int64_t v = v0 + tid; v < v1; v += 256) {
        floatx8 f = Vec8<T>::get(load8(z + v * 8));
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = scale * exp_at(f[i], base);
        if (v == y >> 3) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += i == (int)(y & 7) ? coef : 0.f;
        }
        store8(dz + v * 8, Vec8<T>::put(f));
    }
    if (tid < tail) {
        const int64_t v = nfull * 8 + tid;
        dz[v] = (T)(scale * exp_at((float)z[v], base) + (v == y ? coef : 0.f));
    }
}

// loss = sum of the rows' terms: strided per thread, then lanes, then waves.
__global__ __launch_bounds__(1024) void loss_sum_kernel(const float* __restrict__ terms, int64_t rows, float* loss) {
    __shared__ float part[16];
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < rows; i += 1024) s += ldg(terms + i);
    s = wave_add(s);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) s += part[w];
        stg(loss, s);
    }
}

// Up to SPLIT_ROWS rows are split.  Measured (split launches against the row kernel and the
// loss's): 8 x 32768 bf16 7.8 us against 11.4, 8 x 40961 fp32 7.9 against 12.2, 63 x 65536
// bf16 11.7 against 14.6, 48 x 131072 bf16 11.2 against 19.9.  Shorter rows are a few
// microseconds either way and take the row kernel; so do the log-probabilities alone, one
// launch instead of two (a call among others: 16 x 65536 bf16 7.0 us against 10.7, 1 and 64 x
// 131072 bf16 8.1 and 8.6 against 10.9 and 10.4).
constexpr int64_t SPLIT_ROWS = 64;
constexpr int64_t SPLIT_GROUPS = 1024;       // workgroups of a split launch, about

struct PolicyPlan {
    bool split;
    int64_t pieces, vecs;
    size_t off_stat, off_zy, total;          // the rows' terms come first
};
PolicyPlan policy_plan(shampoo4_dtype dtype, int64_t rows, int64_t vocab, bool train) {
    PolicyPlan q{};
    const int64_t nvec = vocab >> 3;
    const int64_t most = 1024 * (dtype == SHAMPOO4_F32 ? 8 : 16);    // vectors a workgroup holds
    q.split = nvec > most || (train && rows <= SPLIT_ROWS && nvec > 1024);
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    q.off_stat = up(train ? (size_t)rows * 4 : 0);
    q.total = q.off_stat;
    if (q.split) {
        const int64_t per_row = std::max<int64_t>(1, SPLIT_GROUPS / std::max<int64_t>(rows, 1));
        q.vecs = std::max<int64_t>(256, (nvec + per_row - 1) / per_row);
        q.vecs = std::min<int64_t>((q.vecs + 255) / 256 * 256, 4096);
        q.pieces = (nvec + q.vecs - 1) / q.vecs;
        q.off_zy = q.off_stat + up((size_t)rows * q.pieces * 8);
        q.total = q.off_zy + up((size_t)rows * 4);
    }
    return q;
}

template <class T, int THREADS, int NV>
void row_kernel(const Policy& p, float* terms, hipStream_t stream) {
    S4_LAUNCH((policy_row_kernel<T, THREADS, NV>), dim3((uint32_t)p.rows), dim3(THREADS), 0, stream, p, terms);
}

// Returns whether the rows' terms are left to sum.
template <class T>
bool policy_of(const Policy& p, const PolicyPlan& plan, char* ws, hipStream_t stream) {
    float* terms = (float*)ws;
    constexpr int W = sizeof(T) == 4 ? 1 : 2;                // vectors per 64 data registers: 8 or 16
    const int64_t nvec = p.vocab >> 3;
    if (plan.split) {
        const Pieces q{(float*)(ws + plan.off_stat), (float*)(ws + plan.off_zy), plan.pieces, plan.vecs};
        const uint32_t n = (uint32_t)(p.rows * plan.pieces);
        S4_LAUNCH(policy_part_kernel<T>, dim3(n), dim3(256), 0, stream, p, q);
        if (p.train && p.rows <= SPLIT_ROWS) {
            S4_LAUNCH((policy_grad_kernel<T, true>), dim3(p.dlogits ? n + 1 : 1), dim3(256), 0, stream, p, q);
            return false;
        }
        S4_LAUNCH(policy_join_kernel, dim3((uint32_t)((p.rows + 3) / 4)), dim3(256), 0, stream, p, q, terms);
        if (p.dlogits) S4_LAUNCH((policy_grad_kernel<T, false>), dim3(n), dim3(256), 0, stream, p, q);
    } else if (nvec <= 256 * 2 * W) {
        row_kernel<T, 256, 2 * W>(p, terms, stream);
    } else if (nvec <= 256 * 8 * W) {
        row_kernel<T, 256, 8 * W>(p, terms, stream);
    } else if (nvec <= 512 * 8 * W) {
        row_kernel<T, 512, 8 * W>(p, terms, stream);
    } else {
        row_kernel<T, 1024, 8 * W>(p, terms, stream);
    }
    return p.train;
}

}  // namespace

size_t policy_workspace_bytes(shampoo4_dtype dtype, int64_t rows, int64_t vocab, bool train) {
    return policy_plan(dtype, rows, vocab, train).total;
}

hipError_t launch_policy(shampoo4_dtype dtype, const Policy& p, void* workspace, hipStream_t stream) {
    const PolicyPlan plan = policy_plan(dtype, p.rows, p.vocab, p.train != 0);
    if (p.rows == 0 && !p.train) return hipSuccess;
    bool sum = p.train;
    if (p.rows > 0) {
        switch (dtype) {
            case SHAMPOO4_BF16: sum = policy_of<__bf16>(p, plan, (char*)workspace, stream); break;
            case SHAMPOO4_F16: sum = policy_of<_Float16>(p, plan, (char*)workspace, stream); break;
            default: sum = policy_of<float>(p, plan, (char*)workspace, stream);
        }
    }
    if (sum)
        S4_LAUNCH(loss_sum_kernel, dim3(1), dim3(1024), 0, stream, (const float*)workspace, p.rows, p.loss);
    return hipGetLastError();
}

}  // namespace s4
