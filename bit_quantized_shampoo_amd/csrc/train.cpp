// C ABI of the training operators (shampoo4_train.h): validation on the host, then one
// launcher each.  No call allocates, synchronizes or throws.
#include <cmath>

#include <rocprofiler-sdk-roctx/roctx.h>

#include "train.hpp"

using namespace s4;

namespace {

struct CallRange {
    explicit CallRange(const char* name) { roctxRangePushA(name); }
    ~CallRange() { roctxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 64;

bool dtype_ok(shampoo4_dtype d) { return d == SHAMPOO4_F32 || d == SHAMPOO4_BF16 || d == SHAMPOO4_F16; }
size_t dtype_bytes(shampoo4_dtype d) { return d == SHAMPOO4_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
shampoo4_status launched(hipError_t e) { return e == hipSuccess ? SHAMPOO4_OK : SHAMPOO4_EHIP; }
hipStream_t as_stream(void* s) { return (hipStream_t)s; }

// rows x cols, a positive number of columns, and what one launch covers.
bool shape_ok(int64_t rows, int64_t cols) { return rows >= 0 && cols >= 1 && rows <= kMaxDim && cols <= kMaxDim; }

shampoo4_status matrix_ok(const void* p, shampoo4_dtype d, int64_t rows, int64_t cols, int64_t ld) {
    if (ld < cols) return SHAMPOO4_ESHAPE;
    if (rows == 0) return SHAMPOO4_OK;
    if (!p) return SHAMPOO4_EINVAL;
    return aligned(p, dtype_bytes(d)) ? SHAMPOO4_OK : SHAMPOO4_EALIGN;
}

// A checkpoint pair: both or none; `required`: both.
shampoo4_status act8_ok(const int8_t* codes, const uint8_t* scales, int64_t rows, bool required) {
    if (rows == 0) return SHAMPOO4_OK;
    if (!codes != !scales) return SHAMPOO4_EINVAL;
    if (!codes) return required ? SHAMPOO4_EINVAL : SHAMPOO4_OK;
    return aligned(codes, 16) && aligned(scales, 16) ? SHAMPOO4_OK : SHAMPOO4_EALIGN;
}

shampoo4_status workspace_ok(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return SHAMPOO4_OK;
    if (!ws) return SHAMPOO4_EINVAL;
    if (!aligned(ws, 256)) return SHAMPOO4_EALIGN;
    return bytes >= need ? SHAMPOO4_OK : SHAMPOO4_ESMALLBUF;
}

#define S4_TRY(expr)                                   \
    do {                                               \
        const shampoo4_status st_ = (expr);            \
        if (st_ != SHAMPOO4_OK) return st_;            \
    } while (0)

bool wgrad_shape_ok(int64_t rows, int64_t n, int64_t cols) {
    // output tiles of at least 128 x 128, 512 threads each: below 2^32 in a launch
    return shape_ok(rows, cols) && n >= 1 && n <= kMaxDim && ((n + 127) / 128) * ((cols + 127) / 128) < (int64_t(1) << 23);
}

bool embed_shape_ok(int64_t tokens, int64_t vocab, int64_t dim) {
    if (tokens < 0 || vocab < 1 || dim < 1 || tokens > kMaxDim || vocab > kMaxDim || dim > kMaxDim) return false;
    // chunks of 16 tokens x tiles of 512 columns, 64 threads each in a launch
    return (tokens + 15) / 16 * ((dim + 511) / 512) < (int64_t(1) << 26) - 8;
}

bool policy_shape_ok(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || rows >= (int64_t(1) << 22) || vocab > kMaxDim) return false;
    // pieces of at least 32768 logits, 256 threads each in a launch, once rows fill the GPU
    return rows * ((vocab + 32767) / 32768) < (int64_t(1) << 23);
}

shampoo4_status policy_call(const Policy& p, shampoo4_dtype dtype, int32_t id_bytes, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype) || (id_bytes != 4 && id_bytes != 8)) return SHAMPOO4_EINVAL;
    if (!policy_shape_ok(p.rows, p.vocab)) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(p.logits, dtype, p.rows, p.vocab, p.ldz));
    if (p.rows > 0) {
        if (!p.targets) return SHAMPOO4_EINVAL;
        if (!aligned(p.targets, id_bytes)) return SHAMPOO4_EALIGN;
    }
    S4_TRY(workspace_ok(workspace, workspace_bytes, policy_workspace_bytes(dtype, p.rows, p.vocab, p.train != 0)));
    return launched(launch_policy(dtype, p, workspace, as_stream(stream)));
}

}  // namespace

extern "C" {

shampoo4_status shampoo4_act8_bytes(int64_t rows, int64_t cols, size_t* codes_bytes, size_t* scales_bytes) {
    if (!codes_bytes || !scales_bytes) return SHAMPOO4_EINVAL;
    if (!shape_ok(rows, cols)) return SHAMPOO4_ESHAPE;
    *codes_bytes = (size_t)act8_rows(rows) * act8_pitch(cols);
    *scales_bytes = *codes_bytes / 32;
    return SHAMPOO4_OK;
}

shampoo4_status shampoo4_act8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                    int8_t* codes, uint8_t* scales, void* stream) {
    CallRange range_("shampoo4_act8_store");
    if (!dtype_ok(dtype)) return SHAMPOO4_EINVAL;
    if (!shape_ok(rows, cols) || act8_tiles(rows, cols) > ACT8_MAX_TILES) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(x, dtype, rows, cols, ldx));
    S4_TRY(act8_ok(codes, scales, rows, true));
    return launched(launch_act8_store(dtype, rows, cols, x, ldx, {codes, scales}, as_stream(stream)));
}

shampoo4_status shampoo4_act8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols, const int8_t* codes,
                                   const uint8_t* scales, void* x, int64_t ldx, void* stream) {
    CallRange range_("shampoo4_act8_load");
    if (!dtype_ok(dtype)) return SHAMPOO4_EINVAL;
    if (!shape_ok(rows, cols) ||
        act8_tiles(rows, cols) > (dtype == SHAMPOO4_F32 ? ACT8_MAX_TILES_F32_LOAD : ACT8_MAX_TILES))
        return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(x, dtype, rows, cols, ldx));
    S4_TRY(act8_ok(codes, scales, rows, true));
    return launched(launch_act8_load(dtype, rows, cols, {const_cast<int8_t*>(codes), const_cast<uint8_t*>(scales)}, x,
                                     ldx, as_stream(stream)));
}

shampoo4_status shampoo4_activation_forward(int32_t kind, shampoo4_dtype dtype, int64_t rows, int64_t cols,
                                            const void* gate, int64_t ldgate, const void* up, int64_t ldup, void* h,
                                            int64_t ldh, int8_t* gate_codes, uint8_t* gate_scales, int8_t* up_codes,
                                            uint8_t* up_scales, int8_t* h_codes, uint8_t* h_scales, void* stream) {
    CallRange range_("shampoo4_activation_forward");
    if (!dtype_ok(dtype) || (kind != SHAMPOO4_ACT_SILU && kind != SHAMPOO4_ACT_GELU)) return SHAMPOO4_EINVAL;
    if (!shape_ok(rows, cols) || act8_tiles(rows, cols) > ACT8_MAX_TILES) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(gate, dtype, rows, cols, ldgate));
    if (up) S4_TRY(matrix_ok(up, dtype, rows, cols, ldup));
    S4_TRY(matrix_ok(h, dtype, rows, cols, ldh));
    S4_TRY(act8_ok(gate_codes, gate_scales, rows, false));
    S4_TRY(act8_ok(up_codes, up_scales, rows, false));
    S4_TRY(act8_ok(h_codes, h_scales, rows, false));
    if (!up && up_codes) return SHAMPOO4_EINVAL;
    const ActForward a{gate, up, h, ldgate, ldup, ldh, {gate_codes, gate_scales}, {up_codes, up_scales},
                       {h_codes, h_scales}, rows, cols};
    return launched(launch_activation_forward(kind, dtype, a, as_stream(stream)));
}

shampoo4_status shampoo4_activation_backward(int32_t kind, shampoo4_dtype dtype, int64_t rows, int64_t cols,
                                             const void* dh, int64_t lddh, const int8_t* gate_codes,
                                             const uint8_t* gate_scales, const int8_t* up_codes,
                                             const uint8_t* up_scales, void* dgate, int64_t lddgate, void* dup,
                                             int64_t lddup, void* stream) {
    CallRange range_("shampoo4_activation_backward");
    if (!dtype_ok(dtype) || (kind != SHAMPOO4_ACT_SILU && kind != SHAMPOO4_ACT_GELU)) return SHAMPOO4_EINVAL;
    if (!shape_ok(rows, cols) || act8_tiles(rows, cols) > ACT8_MAX_TILES) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(dh, dtype, rows, cols, lddh));
    S4_TRY(matrix_ok(dgate, dtype, rows, cols, lddgate));
    S4_TRY(act8_ok(gate_codes, gate_scales, rows, true));
    S4_TRY(act8_ok(up_codes, up_scales, rows, dup != nullptr));
    if (dup) S4_TRY(matrix_ok(dup, dtype, rows, cols, lddup));
    if (!dup && up_codes) return SHAMPOO4_EINVAL;
    const ActBackward a{dh, dgate, dup, lddh, lddgate, lddup,
                        {const_cast<int8_t*>(gate_codes), const_cast<uint8_t*>(gate_scales)},
                        {const_cast<int8_t*>(up_codes), const_cast<uint8_t*>(up_scales)}, rows, cols};
    return launched(launch_activation_backward(kind, dtype, a, as_stream(stream)));
}

size_t shampoo4_act8_weight_grad_workspace_bytes(int64_t rows, int64_t n, int64_t cols) {
    if (!wgrad_shape_ok(rows, n, cols)) return 0;
    return wgrad_workspace_bytes(rows, n, cols);
}

shampoo4_status shampoo4_act8_weight_grad(shampoo4_dtype dtype, int64_t rows, int64_t n, int64_t cols, float alpha,
                                          const void* dy, int64_t lddy, const int8_t* codes, const uint8_t* scales,
                                          float beta, float* g, int64_t ldg, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    CallRange range_("shampoo4_act8_weight_grad");
    if (!dtype_ok(dtype) || !std::isfinite(alpha) || !std::isfinite(beta)) return SHAMPOO4_EINVAL;
    if (!wgrad_shape_ok(rows, n, cols)) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(dy, dtype, rows, n, lddy));
    S4_TRY(matrix_ok(g, SHAMPOO4_F32, n, cols, ldg));
    S4_TRY(act8_ok(codes, scales, rows, true));
    S4_TRY(workspace_ok(workspace, workspace_bytes, wgrad_workspace_bytes(rows, n, cols)));
    const WGrad w{dy, codes, scales, g, (float*)workspace, rows, n, cols, lddy, ldg, alpha, beta};
    return launched(launch_wgrad(dtype, w, as_stream(stream)));
}

shampoo4_status shampoo4_embedding(shampoo4_dtype dtype, int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t dim,
                                   const void* table, int64_t ldtable, const void* ids, float scale, void* out,
                                   int64_t ldout, void* stream) {
    CallRange range_("shampoo4_embedding");
    if (!dtype_ok(dtype) || (id_bytes != 4 && id_bytes != 8)) return SHAMPOO4_EINVAL;
    if (!embed_shape_ok(tokens, vocab, dim)) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(table, dtype, vocab, dim, ldtable));
    S4_TRY(matrix_ok(out, dtype, tokens, dim, ldout));
    if (tokens > 0 && !ids) return SHAMPOO4_EINVAL;
    if (!aligned(ids, id_bytes)) return SHAMPOO4_EALIGN;
    const Embed e{table, ids, out, tokens, vocab, dim, ldtable, ldout, scale, id_bytes == 8};
    return launched(launch_embedding(dtype, e, as_stream(stream)));
}

size_t shampoo4_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    return embed_shape_ok(tokens, vocab, dim) ? embedding_grad_workspace_bytes(tokens, vocab, dim) : 0;
}

shampoo4_status shampoo4_embedding_grad(shampoo4_dtype dtype, int32_t id_bytes, int64_t tokens, int64_t vocab,
                                        int64_t dim, const void* dout, int64_t lddout, const void* ids, float scale,
                                        int32_t accumulate, float* g, int64_t ldg, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    CallRange range_("shampoo4_embedding_grad");
    if (!dtype_ok(dtype) || (id_bytes != 4 && id_bytes != 8)) return SHAMPOO4_EINVAL;
    if (!embed_shape_ok(tokens, vocab, dim)) return SHAMPOO4_ESHAPE;
    S4_TRY(matrix_ok(dout, dtype, tokens, dim, lddout));
    S4_TRY(matrix_ok(g, SHAMPOO4_F32, vocab, dim, ldg));
    if (tokens > 0 && !ids) return SHAMPOO4_EINVAL;
    if (!aligned(ids, id_bytes)) return SHAMPOO4_EALIGN;
    S4_TRY(workspace_ok(workspace, workspace_bytes, embedding_grad_workspace_bytes(tokens, vocab, dim)));
    const EmbedGrad e{dout, ids, g, tokens, vocab, dim, lddout, ldg, scale, id_bytes == 8, accumulate != 0};
    return launched(launch_embedding_grad(dtype, e, workspace, as_stream(stream)));
}

size_t shampoo4_policy_loss_workspace_bytes(shampoo4_dtype dtype, int64_t rows, int64_t vocab) {
    return dtype_ok(dtype) && policy_shape_ok(rows, vocab) ? policy_workspace_bytes(dtype, rows, vocab, true) : 0;
}

size_t shampoo4_token_logprobs_workspace_bytes(shampoo4_dtype dtype, int64_t rows, int64_t vocab) {
    return dtype_ok(dtype) && policy_shape_ok(rows, vocab) ? policy_workspace_bytes(dtype, rows, vocab, false) : 0;
}

shampoo4_status shampoo4_policy_loss(const shampoo4_policy_config* cfg, shampoo4_dtype dtype, int32_t id_bytes,
                                     int64_t rows, int64_t vocab, const void* logits, int64_t ldlogits,
                                     const void* targets, const float* old_logp, const float* ref_logp,
                                     const float* advantages, const float* weights, float* loss, float* logp,
                                     void* dlogits, int64_t lddlogits, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    CallRange range_("shampoo4_policy_loss");
    if (!cfg || !loss) return SHAMPOO4_EINVAL;
    if (!(cfg->clip_low >= 0.f && cfg->clip_low <= 1.f && cfg->clip_high >= 0.f && cfg->kl_coef >= 0.f) ||
        !std::isfinite(cfg->clip_high) || !std::isfinite(cfg->kl_coef) || !std::isfinite(cfg->grad_scale))
        return SHAMPOO4_EINVAL;
    if (rows > 0 && (!old_logp || !advantages || !weights || (cfg->kl_coef > 0.f && !ref_logp))) return SHAMPOO4_EINVAL;
    if (!dtype_ok(dtype)) return SHAMPOO4_EINVAL;
    if (dlogits) S4_TRY(matrix_ok(dlogits, dtype, rows, vocab, lddlogits));
    const Policy p{logits, targets, old_logp, ref_logp, advantages, weights, loss, logp, dlogits, rows, vocab,
                   ldlogits, lddlogits, cfg->clip_low, cfg->clip_high, cfg->kl_coef, cfg->grad_scale,
                   id_bytes == 8, 1};
    return policy_call(p, dtype, id_bytes, workspace, workspace_bytes, stream);
}

shampoo4_status shampoo4_token_logprobs(shampoo4_dtype dtype, int32_t id_bytes, int64_t rows, int64_t vocab,
                                        const void* logits, int64_t ldlogits, const void* targets, float* logp,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range_("shampoo4_token_logprobs");
    if (rows > 0 && !logp) return SHAMPOO4_EINVAL;
    Policy p{};
    p.logits = logits;
    p.targets = targets;
    p.logp = logp;
    p.rows = rows;
    p.vocab = vocab;
    p.ldz = ldlogits;
    p.id64 = id_bytes == 8;
    return policy_call(p, dtype, id_bytes, workspace, workspace_bytes, stream);
}

}  // extern "C"
