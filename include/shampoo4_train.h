/*
 * shampoo4_train.h -- C ABI of the training operators beside the 4-bit Shampoo step: what
 * produces the gradients G that shampoo4_step reads, from the first layer of a language
 * model to its loss, with the memory that training keeps between the passes in 8 bits.
 *
 *   8-bit activation checkpoints   shampoo4_act8_store / shampoo4_act8_load
 *   activation, its backward pass reading the checkpoint
 *                                  shampoo4_activation_forward / shampoo4_activation_backward
 *   weight gradient of a linear layer whose input is a checkpoint
 *                                  shampoo4_act8_weight_grad
 *   embedding table                shampoo4_embedding / shampoo4_embedding_grad
 *   clipped policy loss with a KL term, on logits
 *                                  shampoo4_policy_loss / shampoo4_token_logprobs
 *
 * Conventions, beside those of shampoo4.h (ownership, streams, validation before anything
 * is enqueued, status codes):
 *  - No call needs a context, allocates device memory or waits for the device; every call
 *    can be captured into a HIP graph (its host arguments are read during the call).
 *  - Matrices are row-major, with a leading dimension in elements, at least the number of
 *    columns.  Any alignment that the element type allows is accepted.
 *  - Element types are SHAMPOO4_F32, SHAMPOO4_BF16 or SHAMPOO4_F16.  Sums, maxima,
 *    softmax statistics and activations are computed in fp32 (or more) and rounded once.
 *  - Outputs must not overlap inputs, except where an argument says so.
 *  - Zero rows are allowed everywhere (sums over no rows are zero).
 *  - Results do not depend on timing: every sum has a fixed order.
 *  - Workspaces are 256-byte aligned, hold nothing between calls and need no initial value.
 */
#ifndef SHAMPOO4_TRAIN_H
#define SHAMPOO4_TRAIN_H

#include "shampoo4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SHAMPOO4_F32 = 0,
    SHAMPOO4_BF16 = 1,
    SHAMPOO4_F16 = 2
} shampoo4_dtype;

/* 8-bit activation checkpoint of X:[rows, cols].
 *
 * A block is 32 consecutive rows (tokens) of one column (channel); the last one is padded
 * with zeros.  With a = max |x| over the block, its scale is the power of two
 * s = 2^(e - 127), e the smallest value in [1, 254] with a / s <= 127, and a code is
 * c = x / s rounded to the nearest integer (ties to even), so |c| <= 127 and the restored
 * value is c * s: at most s / 2 from x, and a bfloat16 number exactly.  (Where 64 * s is
 * 2^128, |c| stops at 63, so c * s is finite.)  A block that holds an infinity or NaN has
 * e = 255 and codes 0, and is restored as NaN.
 *
 * The scale is a power of two, and shared along the tokens, because the weight gradient
 * sums over tokens: c * s is then an operand of the bf16 matrix cores as it stands.  One
 * channel's outliers cost no other channel precision.
 *
 *   codes   int8  [R, P]        R = rows up to a multiple of 32, P = cols up to one of 16
 *   scales  uint8 [R / 32, P]   the exponents e
 *
 * Padding holds code 0 with e = 1.  Both are contiguous, and 16-byte aligned (EALIGN). */
#define SHAMPOO4_ACT8_ROWS 32
#define SHAMPOO4_ACT8_PITCH 16

/* Bytes of codes and scales.  Host only.  ESHAPE: rows < 0, cols < 1, or above 2^31 - 64.
 * The calls below refuse (ESHAPE) what one launch cannot cover: 2^26 tiles of 32 rows x 128
 * columns, 2^24 where float32 values are loaded (both beyond this GPU's memory or near it). */
SHAMPOO4_API shampoo4_status shampoo4_act8_bytes(int64_t rows, int64_t cols, size_t* codes_bytes,
                                                 size_t* scales_bytes);

SHAMPOO4_API shampoo4_status shampoo4_act8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols,
                                                 const void* x, int64_t ldx, int8_t* codes, uint8_t* scales,
                                                 void* stream);

/* Restores X (any type; values beyond a float16's range become its largest number). */
SHAMPOO4_API shampoo4_status shampoo4_act8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols,
                                                const int8_t* codes, const uint8_t* scales, void* x, int64_t ldx,
                                                void* stream);

/* Activations.  SILU: a(x) = x / (1 + exp(-x)); GELU: the tanh form,
 * a(x) = x / (1 + exp(-2 sqrt(2/pi) (x + 0.044715 x^3))). */
#define SHAMPOO4_ACT_SILU 0
#define SHAMPOO4_ACT_GELU 1

/* H = a(gate) * up, or a(gate) with up NULL, all [rows, cols] of `dtype`, with the
 * checkpoints that training keeps, written in the same pass over the data: of gate
 * (gate_codes / gate_scales), of up, and of H as rounded to `dtype` (the next layer's
 * input).  A NULL pair of codes and scales keeps none (all NULL: the form for inference).
 * EINVAL: only one of a pair is NULL, or a checkpoint of a NULL up. */
SHAMPOO4_API shampoo4_status shampoo4_activation_forward(int32_t kind, shampoo4_dtype dtype, int64_t rows, int64_t cols,
                                                         const void* gate, int64_t ldgate,
                                                         const void* up, int64_t ldup, void* h, int64_t ldh,
                                                         int8_t* gate_codes, uint8_t* gate_scales,
                                                         int8_t* up_codes, uint8_t* up_scales,
                                                         int8_t* h_codes, uint8_t* h_scales, void* stream);

/* With g, u the restored gate and up: dgate = dh * u * a'(g), dup = dh * a(g); without up
 * (its pair and dup NULL), dgate = dh * a'(g).  dgate may be dh itself, with its leading
 * dimension (each element is read before it is written). */
SHAMPOO4_API shampoo4_status shampoo4_activation_backward(int32_t kind, shampoo4_dtype dtype, int64_t rows, int64_t cols,
                                                          const void* dh, int64_t lddh,
                                                          const int8_t* gate_codes, const uint8_t* gate_scales,
                                                          const int8_t* up_codes, const uint8_t* up_scales,
                                                          void* dgate, int64_t lddgate, void* dup, int64_t lddup,
                                                          void* stream);

/* Weight gradient of y = x W^T from the checkpoint of x:
 *     G = alpha * dY^T X^ + beta * G      dY:[rows, n], X^:[rows, cols], G:[n, cols] fp32
 * the block gradient that shampoo4_step takes.  With beta = 0, G is not read.  Products
 * are exact and sums in fp32 on the bf16 matrix cores: X^ and a bf16 dY are operands as
 * they stand, an f16 or f32 dY is split exactly into two or three bf16 pieces (what an fp32
 * value has below 2^-133 is dropped).
 * rows = 0: G = beta * G.  The workspace (NULL when the size is 0) holds partial sums of
 * row ranges when the output alone cannot fill the GPU.
 * ESHAPE also from 2^23 output tiles of 128 x 128 on (512 GiB of G). */
SHAMPOO4_API size_t shampoo4_act8_weight_grad_workspace_bytes(int64_t rows, int64_t n, int64_t cols);
SHAMPOO4_API shampoo4_status shampoo4_act8_weight_grad(shampoo4_dtype dtype, int64_t rows, int64_t n, int64_t cols,
                                                       float alpha, const void* dy, int64_t lddy,
                                                       const int8_t* codes, const uint8_t* scales,
                                                       float beta, float* g, int64_t ldg,
                                                       void* workspace, size_t workspace_bytes, void* stream);

/* Embedding: out[t] = scale * table[ids[t]], table:[vocab, dim], out:[tokens, dim], both of
 * `dtype`; ids is device int32 (id_bytes = 4) or int64 (8).  An id outside [0, vocab) (as
 * -1 for padding) reads nothing and gives a row of zeros. */
SHAMPOO4_API shampoo4_status shampoo4_embedding(shampoo4_dtype dtype, int32_t id_bytes, int64_t tokens, int64_t vocab,
                                                int64_t dim, const void* table, int64_t ldtable, const void* ids,
                                                float scale, void* out, int64_t ldout, void* stream);

/* Its gradient in fp32, G:[vocab, dim]:
 *     G[v] (+)= scale * sum over t with ids[t] = v of dout[t]
 * accumulate = 0 writes every row (zeros where no token is v); accumulate = 1 adds to G and
 * touches the rows of present tokens only.  Ids outside [0, vocab) contribute nothing.
 * The tokens are sorted by id (stable), so a row's sum is taken over its tokens in the
 * order of their positions, split at fixed places of the sorted list.
 * ESHAPE: tokens, vocab or dim above 2^31 - 64, or tokens / 16 * dim / 512 from 2^26 on (also
 * of shampoo4_embedding). */
SHAMPOO4_API size_t shampoo4_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim);
SHAMPOO4_API shampoo4_status shampoo4_embedding_grad(shampoo4_dtype dtype, int32_t id_bytes, int64_t tokens,
                                                     int64_t vocab, int64_t dim, const void* dout, int64_t lddout,
                                                     const void* ids, float scale, int32_t accumulate,
                                                     float* g, int64_t ldg,
                                                     void* workspace, size_t workspace_bytes, void* stream);

/* Clipped policy loss with a KL term, on logits Z:[rows, vocab].  Per row t with y its
 * target, w its weight, A its advantage:
 *     logp = Z[y] - log sum_v exp Z[v],   r = exp(logp - old),   d = ref - logp
 *     l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(d) - d - 1)
 *     loss = sum_t w l
 *     dZ[v] = grad_scale * w * (dl/dlogp) * ([v = y] - softmax(Z)[v])
 * with dl/dlogp = -r A where r A <= clip(r) A (else 0) + kl_coef (1 - exp(d)).  The caller
 * puts the mask and the normalisation into w (a mean over kept tokens: w = mask / sum of
 * mask).  A row with w = 0, or a target outside [0, vocab), is not read at all: its logp
 * and gradient are 0 and it adds nothing, whatever its logits, old, ref and advantage are.
 * Finite logits may be of any size (masks of -1e10 or of the type's lowest value too); one of
 * -infinity has probability 0.
 * Outputs: loss, one fp32; logp, fp32 [rows], or NULL; dlogits [rows, vocab] of `dtype`, or
 * NULL for the loss alone (dlogits may be Z itself, with its leading dimension).  ref may
 * be NULL with kl_coef = 0 (it is then not read).
 * ESHAPE: vocab < 1 or above 2^31 - 64, 2^22 rows or more, or rows * vocab / 32768 from 2^23 on. */
typedef struct {
    float clip_low, clip_high;    /* >= 0; clip_low <= 1 */
    float kl_coef;                /* >= 0 */
    float grad_scale;             /* finite */
} shampoo4_policy_config;

SHAMPOO4_API size_t shampoo4_policy_loss_workspace_bytes(shampoo4_dtype dtype, int64_t rows, int64_t vocab);
SHAMPOO4_API shampoo4_status shampoo4_policy_loss(const shampoo4_policy_config* cfg, shampoo4_dtype dtype,
                                                  int32_t id_bytes, int64_t rows, int64_t vocab,
                                                  const void* logits, int64_t ldlogits, const void* targets,
                                                  const float* old_logp, const float* ref_logp,
                                                  const float* advantages, const float* weights,
                                                  float* loss, float* logp, void* dlogits, int64_t lddlogits,
                                                  void* workspace, size_t workspace_bytes, void* stream);

/* logp[t] alone, for every row (the old and reference log-probabilities of a rollout); 0
 * for a target outside [0, vocab).  Its workspace (NULL when the size is 0) is not larger than
 * shampoo4_policy_loss's. */
SHAMPOO4_API size_t shampoo4_token_logprobs_workspace_bytes(shampoo4_dtype dtype, int64_t rows, int64_t vocab);
SHAMPOO4_API shampoo4_status shampoo4_token_logprobs(shampoo4_dtype dtype, int32_t id_bytes, int64_t rows,
                                                     int64_t vocab, const void* logits, int64_t ldlogits,
                                                     const void* targets, float* logp,
                                                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SHAMPOO4_TRAIN_H */
