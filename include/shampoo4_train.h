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
 *   products of a linear layer in 8-bit floating point, scales for blocks of 128
 *                                  shampoo4_fp8_store / shampoo4_fp8_store_weight / shampoo4_fp8_load /
 *                                  shampoo4_fp8_linear
 *   norms before and after a block, with its gate, residual scale and dropout
 *                                  shampoo4_block_norm_forward / shampoo4_block_norm_backward
 *   dropout from a counter-based generator
 *                                  shampoo4_dropout
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

/* Matrices in 8-bit floating point (e4m3: a sign, four bits of exponent, three of mantissa,
 * largest value 448, no infinity) with a scale for each block of 128 columns.
 *
 * A block is 128 columns of 1 row (block_rows = 1: activations and their gradients) or of 128
 * rows (block_rows = 128: weights).  With a = max |x| over the block, its scale is the power of
 * two s = 2^(e - 127), e the smallest value in [1, 254] with a / s <= 448, and a code is x / s
 * rounded to the nearest e4m3 number (ties to even).  (Where 256 s is 2^128, |x / s| stops at 240,
 * so that the restored value is finite.)  A block that holds an infinity or NaN has e = 255 and
 * codes 0, and stands for NaN.
 *
 * A scale that is a power of two is an operand of this GPU's scaled matrix instructions, and
 * a weight's block is square, so that the transposed weight has the same codes and scales.
 *
 *   codes   [rows, P]                     P = cols up to a multiple of 128
 *   scales  uint8 [rows / block_rows, S]  (rows up to a multiple of block_rows), S = P / 128 up
 *                                         to a multiple of 4
 *
 * Padding holds code 0, and scales of padding e = 1.  Both are contiguous; codes are 16-byte
 * and scales 4-byte aligned (EALIGN). */
#define SHAMPOO4_FP8_BLOCK 128

/* Bytes of codes and scales.  Host only.  EINVAL: block_rows is neither 1 nor 128.  ESHAPE: rows < 0,
 * cols < 1, or above 2^31 - 64.  The calls below refuse (ESHAPE) what one launch cannot cover:
 * 2^24 tiles of 4 rows x 512 columns, or of 128 x 128 in a weight. */
SHAMPOO4_API shampoo4_status shampoo4_fp8_bytes(int64_t rows, int64_t cols, int32_t block_rows, size_t* codes_bytes,
                                                size_t* scales_bytes);

/* Quantises X:[rows, cols], with block_rows = 1. */
SHAMPOO4_API shampoo4_status shampoo4_fp8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* x,
                                                int64_t ldx, uint8_t* codes, uint8_t* scales, void* stream);

/* Quantises a weight W:[rows, cols], with block_rows = 128, and, unless t_codes and t_scales are
 * both NULL, writes W^T:[cols, rows] too (the same codes and scales, for the gradient of the
 * layer's input; EINVAL: into the same memory). */
SHAMPOO4_API shampoo4_status shampoo4_fp8_store_weight(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* w,
                                                       int64_t ldw, uint8_t* codes, uint8_t* scales,
                                                       uint8_t* t_codes, uint8_t* t_scales, void* stream);

/* Restores X (any type; values beyond a float16's range become its largest number). */
SHAMPOO4_API shampoo4_status shampoo4_fp8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols, int32_t block_rows,
                                               const uint8_t* codes, const uint8_t* scales, void* x, int64_t ldx,
                                               void* stream);

/* Product of a linear layer, X^:[rows, k], W^:[n, k] (block_rows = 128), Y:[rows, n]:
 *     Y = X^ W^T          (accumulate = 0: Y is not read)
 *     Y = Y + X^ W^T      (accumulate = 1)
 * X is given by x_codes and x_scales (block_rows = 1; x NULL), or as a matrix x of `dtype`
 * (x_codes and x_scales NULL), which is then quantised within the call as shampoo4_fp8_store
 * does.  Y is of `out_dtype`.  Sums are in fp32 and rounded once.
 *
 * For a bf16 Y the products are the 8-bit matrix cores', which align eight neighbouring products to
 * the largest of them and cut each off 13 bits below its leading one; the groups' sums are added in
 * fp32.  So a sum is within 7 2^-13 of the sum of its terms' sizes, which where they cancel may be many
 * steps of a bf16 result.  (Ordinary operands show 5e-5 of the results' root mean square, a fortieth of bf16's
 * rounding.)  For an fp32 or f16 Y the codes become operands of the bf16 matrix cores: exact products with fp32
 * sums, at about a third of the rate.  Terms and sums below 2^-126 may be lost.
 *
 * k >= 1 and n >= 1; rows = 0: nothing is done.  The workspace (NULL when the size is 0) holds
 * the quantised x and partial sums of ranges of k.  Y must overlap nothing else.
 * ESHAPE: rows, n or k above 2^31 - 64, from 2^23 tiles of 64 rows x 16 columns of Y on, or an X
 * that shampoo4_fp8_store refuses. */
SHAMPOO4_API size_t shampoo4_fp8_linear_workspace_bytes(shampoo4_dtype out_dtype, int64_t rows, int64_t n, int64_t k,
                                                        int32_t x_quantised);
SHAMPOO4_API shampoo4_status shampoo4_fp8_linear(shampoo4_dtype dtype, shampoo4_dtype out_dtype, int64_t rows, int64_t n,
                                                 int64_t k, const void* x, int64_t ldx, const uint8_t* x_codes,
                                                 const uint8_t* x_scales, const uint8_t* w_codes,
                                                 const uint8_t* w_scales, int32_t accumulate, void* y, int64_t ldy,
                                                 void* workspace, size_t workspace_bytes, void* stream);

/* Dropout.  Element (row, col) of a matrix is dropped where the 16 bits r(row, col) are below
 * t = p 65536 rounded to the nearest integer (ties to even); a kept value is multiplied by 65536 / (65536 - t), a
 * dropped one is 0 whatever it was.  No mask is stored: the backward pass is the same call on
 * the gradient.
 *
 * r: the ten-round Philox 4 x 32 generator (Salmon, Moraes, Dror, Shaw, "Parallel random numbers:
 * as easy as 1, 2, 3", 2011) with the key (seed low, seed high 32 bits) and the counter (col / 8,
 * row, call low, call high) gives four words for eight columns: column c takes word (c % 8) / 2,
 * its low half for even c, else its high half.  It depends on nothing else: not on strides, types
 * or the launch.
 *
 * call = offset + *counter (mod 2^64), counter a device uint64 read as the kernel runs (NULL: 0), so that a
 * captured graph draws other numbers in each replay if the program advances it between them.
 * EINVAL: p < 0, or t = 65536, or not a number.  p = 0 keeps everything. */
typedef struct {
    float p;
    int32_t reserved;             /* 0 */
    uint64_t seed, offset;
    const uint64_t* counter;      /* 8-byte aligned, or NULL */
} shampoo4_dropout_config;

/* Y = dropout(X).  Y may be X itself, with its leading dimension.
 * ESHAPE: rows or cols above 2^31 - 64, or from 2^24 tiles of 4 rows x 512 columns on. */
SHAMPOO4_API shampoo4_status shampoo4_dropout(const shampoo4_dropout_config* cfg, shampoo4_dtype dtype, int64_t rows,
                                              int64_t cols, const void* x, int64_t ldx, void* y, int64_t ldy,
                                              void* stream);

/* The ends of a residual block in one pass: the norm behind the block, its dropout, gate and residual
 * sum, and the norm before the next block.  Per row, with rstd(v) = 1 / sqrt(mean(v^2) + eps):
 *     n = h rstd(h) post_weight          (post_weight NULL: n = h)
 *     x' = residual_scale x + gate drop(n)      (gate NULL: 1; h NULL: x' = x, not written)
 *     y = x' rstd(x') weight, of x' as rounded to `dtype`     (weight NULL: no y)
 * x, h, x', y are [rows, cols] of `dtype`; weight and post_weight fp32 [cols].  gate is fp32 [cols]
 * (gate_rows = 0) or a matrix [rows, cols] of `dtype` (gate_rows = 1, leading dimension ldgate).
 * rstd and h_rstd, fp32 [rows], receive the two factors for the backward pass (NULL: none).
 * y_codes and y_scales (both or none) receive y as rounded, quantised as by shampoo4_fp8_store:
 * the next product's operand.  With h NULL, residual_scale must be 1, and post_weight, gate, out
 * and h_rstd NULL.  out may be x or h itself, and y may be h, each with its leading dimension (EINVAL: y is out).
 * With h NULL nothing is dropped.  A gate that is not finite makes NaN where it is dropped too, in x' (0 gate) and
 * in the backward pass, where what is dropped is g.
 * eps: at least 1e-30, finite.  Finite rows of any size have their norm (squares beyond fp32 are taken
 * of the row divided by a power of two).
 * ESHAPE: cols above 16384, or 2^24 rows or more (2^23 from 2049 columns on, 2^22 from 4097 on). */
#define SHAMPOO4_BLOCK_NORM_COLS 16384
typedef struct {
    float eps, residual_scale;
    shampoo4_dropout_config dropout;
} shampoo4_block_norm_config;

SHAMPOO4_API shampoo4_status shampoo4_block_norm_forward(const shampoo4_block_norm_config* cfg, shampoo4_dtype dtype,
                                                         int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                                         const void* h, int64_t ldh, const float* post_weight,
                                                         const void* gate, int32_t gate_rows, int64_t ldgate,
                                                         const float* weight, void* out, int64_t ldout, void* y,
                                                         int64_t ldy, uint8_t* y_codes, uint8_t* y_scales,
                                                         float* h_rstd, float* rstd, void* stream);

/* Its gradients, from dy (of y; NULL with weight NULL), dres (of x' from behind; NULL: 0), x' (out of the
 * forward call; x with h NULL), h and the two factors:
 *     xh = x' rstd;  t = dy weight;  g = dres + rstd (t - xh mean(t xh))      (weight NULL: g = dres)
 *     dx = residual_scale g;  dweight = sum over rows of dy xh
 *     hh = h h_rstd;  z = drop(hh post_weight);  dgate = g z (gate_rows = 1), or its sum over rows
 *     d = gate drop(g);  dpost_weight = sum over rows of d hh;  u = d post_weight
 *     dh = h_rstd (u - hh mean(u hh))     (post_weight NULL: z = drop(h), dh = d)
 * dx, dh and a matrix dgate are of `dtype` and may be NULL; dweight, dpost_weight and a vector dgate
 * are fp32 [cols], written in whole (rows = 0: zeros), and may be NULL.  dx may be dres or dy itself,
 * dh may be h or dy or dres (EINVAL: what dx is, or a matrix dgate), each with its leading dimension.  What is not
 * needed for the outputs asked for may still be read.  The workspace (NULL when the size is 0) holds partial sums.
 * Sums over rows are in fp32, of fixed groups of rows in order. */
SHAMPOO4_API size_t shampoo4_block_norm_workspace_bytes(int64_t rows, int64_t cols);
SHAMPOO4_API shampoo4_status shampoo4_block_norm_backward(const shampoo4_block_norm_config* cfg, shampoo4_dtype dtype,
                                                          int64_t rows, int64_t cols, const void* dy, int64_t lddy,
                                                          const void* dres, int64_t lddres, const void* x, int64_t ldx,
                                                          const float* rstd, const float* weight, const void* h,
                                                          int64_t ldh, const float* h_rstd, const float* post_weight,
                                                          const void* gate, int32_t gate_rows, int64_t ldgate,
                                                          void* dx, int64_t lddx, void* dh, int64_t lddh,
                                                          float* dweight, float* dpost_weight, void* dgate,
                                                          int64_t lddgate, void* workspace, size_t workspace_bytes,
                                                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SHAMPOO4_TRAIN_H */
