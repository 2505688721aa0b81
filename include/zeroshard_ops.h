/*
 * zeroshard_ops.h -- the operators at the two ends and between the layers of a
 * language model, for MI355X (gfx950): what turns token ids into the 16-bit
 * gradient contributions that zero_shard_step (zeroshard.h) reduces.
 *
 *   embedding   rows of a table, scaled; the table's gradient by sorted tokens
 *   norm        root-mean-square norm with the residual's addition, its output
 *               in 16 bits, in 8 bits with scales, or both; its gradient
 *   act8, glu   activations held in 8 bits: packing alone, and the gated unit
 *               that keeps its input so and takes its gradient from it
 *   xent        softmax cross entropy of a linear head, in pieces of the
 *               vocabulary, without keeping the logits; its gradient
 *   layer norm  with the residual's addition, its output in 16, 8 or 4 bits; its
 *               gradient with the sums for the weight and the bias
 *   mx4         matrices in 4 bits, packed along rows, columns or both, and the
 *               product of two such matrices
 *   prefer      a preference loss of pairs of packed sequences on the losses of
 *               xent; its gradient, which is xent's grad_loss
 *   grads       the gradient norm over many tensors, and clipping by it
 *
 * Conventions are those of zeroshard.h: the caller owns every device buffer and
 * the workspaces, calls enqueue kernels on `stream` and return, a negative return
 * is an error found before anything is enqueued (ZS_EHIP excepted) with a message
 * in zero_shard_last_error().  Calls queue kernels only and can be captured in a
 * graph.  Matrices are row-major with a row stride in elements (>= the width);
 * elements of a row are adjacent.  Nothing but element alignment is asked of data
 * pointers; workspaces are 256-byte aligned.  Outputs must not overlap inputs
 * unless a call says so.  Sizes of zero are allowed where
 * a call does not say otherwise, and null pointers for buffers of no elements.
 * Results do not depend on timing: every sum has a fixed order.
 *
 * The 8-bit form.  A row is cut into groups of 32, 64 or 128 elements (the last
 * one may be shorter).  A group has one scale 2^e, e the least integer in
 * -127..127 for which its largest magnitude is at most 1.75 * 2^(8+e) (e4m3) or
 * 1.75 * 2^(15+e) (e5m2), held as the byte e + 127; its codes are the elements
 * times 2^-e rounded to nearest even.  The scaling is exact, so a code is off by
 * that one rounding only.  A group with a NaN or an infinity has scale byte 255
 * and codes 0, and reads back as NaN throughout.
 *
 * The 4-bit form (e2m1).  Groups have 32 elements, zeros behind a row's end, and 2^e is the
 * least scale in the same range for which a group's largest magnitude is at most 6 * 2^e;
 * codes are the elements times 2^-e rounded to 0, 0.5, 1, 1.5, 2, 3, 4 or 6, ties to even.
 * A row has G = ceil(width / 32) groups: 16 * G bytes of codes (element 2i in the low half of
 * byte i).  Scale bytes lie as the matrix instructions take them, sixteen groups of a
 * row together: that of group n of row r at ((n / 16) * rows + r) * 16 + (n % 4) * 4 + n / 4 % 4,
 * ceil(G / 16) * rows * 16 bytes in all; those of groups that do not exist are 127 (a scale
 * of 1).  Codes and scales are 16-byte aligned.
 */
#ifndef ZEROSHARD_OPS_H
#define ZEROSHARD_OPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define ZS_F32 0
#define ZS_BF16 1
#define ZS_F16 2
/* 8-bit forms */
#define ZS_E4M3 0
#define ZS_E5M2 1
/* the 4-bit form */
#define ZS_E2M1 2
/* gated units: act(g) * u */
#define ZS_SILU 0
#define ZS_GELU 1 /* the tanh form */

/*
 * out[t] = scale * table[ids[t] - vocab_start], the product rounded once to
 * `dtype` (table and out).  A token whose local id lies outside [0, vocab) -- a
 * padding id, or an id of another part of a divided table -- gives a row of
 * zeros.  id_bytes: 4 or 8.  1 <= vocab <= 2^24, 1 <= width <= 2^20, n_tokens < 2^23
 * (more up to 1024 columns: what one launch holds).
 */
int zs_embed_forward(const void *table, int64_t table_stride, const void *ids, void *out,
                     int64_t out_stride, int64_t n_tokens, int64_t vocab, int64_t width,
                     int64_t vocab_start, float scale, int32_t dtype, int32_t id_bytes,
                     void *stream);

/* Workspace of zs_embed_backward; 0 when a size is out of range. */
size_t zs_embed_backward_bytes(int64_t n_tokens, int64_t vocab, int64_t width);

/*
 * grad_table[v] = scale * sum of grad_out[t] over the tokens with local id v, in
 * the order of t within fixed runs of sorted tokens, in fp32, rounded once to
 * `table_dtype` (`dtype` or ZS_F32).  Tokens outside [0, vocab) add nothing and
 * their rows are not read.  accumulate = 0 writes every row (zeros where no token
 * fell); accumulate = 1 adds to the rows that tokens fell on and leaves the rest
 * as they are (a tied table whose other gradient was written before).
 * n_tokens < 2^31 and what one launch holds, vocab and width as above.
 */
int zs_embed_backward(const void *grad_out, int64_t grad_stride, const void *ids,
                      void *grad_table, int64_t table_stride, int64_t n_tokens, int64_t vocab,
                      int64_t width, int64_t vocab_start, float scale, int32_t dtype,
                      int32_t table_dtype, int32_t id_bytes, int32_t accumulate, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * s = x + residual (rounded to `dtype`, stored in `sum`; without a residual s is
 * x and `sum` must be NULL), rstd = 1 / sqrt(mean(s^2) + eps) in fp32, and
 * y = s * rstd * weight: in `dtype` to y (NULL: not wanted) and in 8 bits to
 * codes and scales (both NULL: not wanted; ceil(width / group) scale bytes a row,
 * codes rows of `width` bytes).  sum may be x or residual itself.  1 <= width <= 65536,
 * rows < 2^25 up to 512 columns, < 2^23 up to 8192, < 2^22 beyond (one launch's).
 */
int zs_norm_forward(const void *x, int64_t x_stride, const void *residual,
                    int64_t residual_stride, const void *weight, void *sum, int64_t sum_stride,
                    void *y, int64_t y_stride, void *codes, void *scales, float *rstd,
                    int64_t rows, int64_t width, float eps, int32_t dtype, int32_t code,
                    int32_t group, void *stream);

/* Workspace of zs_norm_backward. */
size_t zs_norm_backward_bytes(int64_t rows, int64_t width);

/*
 * With h = s * rstd: grad_x = rstd * (weight*dy - h * mean(weight*dy*h)) +
 * grad_sum (NULL: nothing to add), which is the gradient of x and of the residual
 * alike, and grad_weight = sum over rows of dy * h (in `weight_dtype`: `dtype` or
 * ZS_F32).  Sums in fp32.  grad_x may be dy, sum or grad_sum itself.
 */
int zs_norm_backward(const void *dy, int64_t dy_stride, const void *sum, int64_t sum_stride,
                     const void *weight, const float *rstd, const void *grad_sum,
                     int64_t grad_sum_stride, void *grad_x, int64_t grad_x_stride,
                     void *grad_weight, int64_t rows, int64_t width, int32_t dtype,
                     int32_t weight_dtype, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * x in the 8-bit form, and back (each value rounded once to `dtype`).  Here and in the
 * gated unit 1 <= width <= 2^20 and rows * ceil(width / 2048) < 2^23 (more rows below
 * 1024 columns: what one launch holds).
 */
int zs_act8_pack(const void *x, int64_t x_stride, void *codes, void *scales, int64_t rows,
                 int64_t width, int32_t dtype, int32_t code, int32_t group, void *stream);
int zs_act8_unpack(const void *codes, const void *scales, void *x, int64_t x_stride,
                   int64_t rows, int64_t width, int32_t dtype, int32_t code, int32_t group,
                   void *stream);

/*
 * The gated unit.  gate_up rows hold 2 * width elements, the gate g and then u;
 * out = act(g) * u, computed in fp32 from the unrounded input.  codes (rows of
 * 2 * width bytes) and scales (2 * ceil(width / group) bytes a row, g's and then
 * u's) receive gate_up in the 8-bit form; both NULL: not kept.
 */
int zs_glu_forward(const void *gate_up, int64_t gate_up_stride, void *out, int64_t out_stride,
                   void *codes, void *scales, int64_t rows, int64_t width, int32_t dtype,
                   int32_t act, int32_t code, int32_t group, void *stream);

/*
 * Its gradient from the 8-bit checkpoint: with g, u read back,
 * grad_gate_up = [grad_out * u * act'(g) | grad_out * act(g)], and, unless NULL,
 * out = act(g) * u again (the next product's input, for its weight gradient).
 */
int zs_glu_backward(const void *grad_out, int64_t grad_out_stride, const void *codes,
                    const void *scales, void *grad_gate_up, int64_t grad_gate_up_stride,
                    void *out, int64_t out_stride, int64_t rows, int64_t width, int32_t dtype,
                    int32_t act, int32_t code, int32_t group, void *stream);

/*
 * Workspace of zs_xent_forward (backward = 0) and zs_xent_backward (1) for these
 * matrices: rows that cannot be read 16 bytes at a time are first copied into it.
 * 0 when a size is out of range.
 */
size_t zs_xent_workspace_bytes(const void *hidden, int64_t hidden_stride, const void *weight,
                               int64_t weight_stride, int64_t tokens, int64_t vocab,
                               int64_t width, int32_t backward);

/*
 * logits = hidden weight^T (products of 16-bit values summed in fp32), never
 * stored: lse[t] = log sum_v exp logits[t][v] and loss[t] = lse[t] -
 * logits[t][targets[t]], both fp32.  A target outside [0, vocab) marks a token
 * that does not count: its loss is 0.  dtype: ZS_BF16 or ZS_F16.
 * 1 <= vocab < 2^31 - 512, 1 <= width <= 65536, tokens <= 2^26 - 16, strides <= 2^21.
 */
int zs_xent_forward(const void *hidden, int64_t hidden_stride, const void *weight,
                    int64_t weight_stride, const void *targets, float *loss, float *lse,
                    int64_t tokens, int64_t vocab, int64_t width, int32_t dtype,
                    int32_t target_bytes, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * With G[t][v] = grad_loss[t] * (exp(logits[t][v] - lse[t]) - [v == targets[t]])
 * (zero rows for tokens that do not count, whose hidden rows and grad_loss are not
 * used): grad_hidden = G weight and grad_weight = G^T hidden, each rounded once
 * to `dtype`; either may be NULL.  grad_hidden may be hidden itself.  G is formed a
 * piece of the vocabulary at a time, divided by the largest finite |grad_loss| (and times
 * 2^15 in fp16, whose digits end at 2^-14) and rounded to `dtype` for the two products,
 * which sum in fp32; the factor comes back before the last rounding.
 * tokens <= 2^21 - 64, and tokens * ceil(width / 1024) < 2^24.
 */
int zs_xent_backward(const void *hidden, int64_t hidden_stride, const void *weight,
                     int64_t weight_stride, const void *targets, const float *lse,
                     const float *grad_loss, void *grad_hidden, int64_t grad_hidden_stride,
                     void *grad_weight, int64_t grad_weight_stride, int64_t tokens,
                     int64_t vocab, int64_t width, int32_t dtype, int32_t target_bytes,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * s = x + residual (rounded to `dtype`, stored in `sum`; without a residual s is x and `sum`
 * must be NULL), mean and rstd = 1 / sqrt(mean((s - mean)^2) + eps) of each row in fp32, and
 * y = (s - mean) * rstd * weight + bias (NULL: none): in `dtype` to y (NULL: not wanted), and in
 * 8 bits (code ZS_E4M3 or ZS_E5M2, as zs_norm_forward) or in 4 (ZS_E2M1, group 32) to codes and
 * scales (both NULL: not wanted).  sum may be x or residual itself.  Sizes as zs_norm_forward's.
 */
int zs_layer_norm_forward(const void *x, int64_t x_stride, const void *residual,
                          int64_t residual_stride, const void *weight, const void *bias, void *sum,
                          int64_t sum_stride, void *y, int64_t y_stride, void *codes, void *scales,
                          float *mean, float *rstd, int64_t rows, int64_t width, float eps,
                          int32_t dtype, int32_t code, int32_t group, void *stream);

/* Workspace of zs_layer_norm_backward; 0 when a size is out of range. */
size_t zs_layer_norm_backward_bytes(int64_t rows, int64_t width);

/*
 * With h = (s - mean) * rstd and g = weight*dy: grad_x = rstd * (g - mean(g) - h * mean(g*h)) +
 * grad_sum (NULL: nothing to add), the gradient of x and of the residual alike; grad_weight =
 * sum over rows of dy * h and grad_bias (NULL: not wanted) = sum of dy, in `weight_dtype`:
 * `dtype` or ZS_F32.  Sums in fp32.  grad_x may be dy, sum or grad_sum itself.  Above 8192
 * columns rows < 2^22.
 */
int zs_layer_norm_backward(const void *dy, int64_t dy_stride, const void *sum, int64_t sum_stride,
                           const void *weight, const float *mean, const float *rstd,
                           const void *grad_sum, int64_t grad_sum_stride, void *grad_x,
                           int64_t grad_x_stride, void *grad_weight, void *grad_bias, int64_t rows,
                           int64_t width, int32_t dtype, int32_t weight_dtype, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * x in the 4-bit form: along its rows to codes and scales, along its columns (the form of the
 * transposed matrix, which has `width` rows of `rows` elements) to codes_t and scales_t;
 * either pair may be NULL.  1 <= width <= 2^20, rows <= 2^24 (2^20 along columns), and fewer than
 * 2^24 pieces of 4 rows x 512 (along columns 2^23 of 256 x 256), counting whole spans of 512.
 */
int zs_mx4_pack(const void *x, int64_t x_stride, void *codes, void *scales, void *codes_t,
                void *scales_t, int64_t rows, int64_t width, int32_t dtype, void *stream);

/*
 * Back: each value rounded once to `dtype`.  That is exact in bf16 and fp32 but for 4 * 2^126,
 * the code of magnitudes from 3.5 * 2^126 on, which becomes infinity (zs_mx4_product takes it
 * as it is).
 */
int zs_mx4_unpack(const void *codes, const void *scales, void *x, int64_t x_stride, int64_t rows,
                  int64_t width, int32_t dtype, void *stream);

/*
 * out[t][n] = sum_k x[t][k] * w[n][k] of two matrices in the 4-bit form with rows of `width`
 * elements, summed in fp32 and rounded once to `dtype`.  (A linear layer's three products are
 * this one: y from x and w packed along rows, dx from dy along rows and w along columns, dw from
 * dy and x along columns.)  tokens and features <= 2^24, width <= 2^20, and fewer than 2^24
 * tiles of 256 x 256.
 */
int zs_mx4_product(const void *x_codes, const void *x_scales, const void *w_codes,
                   const void *w_scales, void *out, int64_t out_stride, int64_t tokens,
                   int64_t features, int64_t width, int32_t dtype, void *stream);

/* Workspace of zs_mx4_linear; 0 when a size is out of range. */
size_t zs_mx4_linear_bytes(int64_t tokens, int64_t width);

/* The same for an x of `x_dtype`, which is packed along its rows into the workspace first. */
int zs_mx4_linear(const void *x, int64_t x_stride, const void *w_codes, const void *w_scales,
                  void *out, int64_t out_stride, int64_t tokens, int64_t features, int64_t width,
                  int32_t x_dtype, int32_t dtype, void *workspace, size_t workspace_bytes,
                  void *stream);

/* kinds of preference loss */
#define ZS_SIGMOID 0
#define ZS_HINGE 1
#define ZS_SQUARED 2

/* Workspace of zs_prefer_forward; 0 when a size is out of range, 256 where none is used (it may be
 * NULL then). */
size_t zs_prefer_workspace_bytes(int64_t tokens, int64_t pairs);

/*
 * The preference loss of pairs of sequences that lie one behind the other: sequence i is tokens
 * offsets[i] to offsets[i + 1] - 1 (2 * pairs + 1 offsets that do not fall), pair p has
 * sequence 2p as the chosen one and 2p + 1 as the rejected.  loss is the policy's -log p of
 * each token and ref_loss the reference's (NULL: none); a token whose mask byte is 0 (mask NULL:
 * none) does not count, whatever its losses hold.  With a = -sum(loss - ref_loss) of a sequence,
 * or the mean over its tokens that count where `average`, rewards[2p], [2p+1] = beta * a,
 * margins[p] = m = beta * (a_chosen - a_rejected) - margin, and pair_loss[p] =
 *   ZS_SIGMOID  -(1 - smoothing) * log sigma(m) - smoothing * log sigma(-m)
 *   ZS_HINGE    max(0, 1 - m)
 *   ZS_SQUARED  (m - 1/2)^2 / beta^2
 * which have their limits where m is infinite (a token without probability: its loss or ref_loss
 * is infinite): 0 for the hinge at +infinity and for the sigmoid where smoothing is 0.
 * margins are rounded to nearest, but a hinge's below 1 stays below it.
 * lengths: the tokens that count in each sequence (a sequence of none has a = 0).  Sums in fp64.
 * beta > 0, 0 <= smoothing <= 0.5 (ZS_SIGMOID only); tokens < 2^31, pairs <= 2^22.
 */
int zs_prefer_forward(const float *loss, const float *ref_loss, const void *offsets,
                      const void *mask, float *pair_loss, float *rewards, float *margins,
                      int32_t *lengths, int64_t tokens, int64_t pairs, float beta, float margin,
                      float smoothing, int32_t kind, int32_t average, int32_t offset_bytes,
                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * grad[t] = the derivative of sum_p grad_loss[p] * pair_loss[p] by loss[t], for every token: 0
 * where it does not count or lies in no sequence.  margins and lengths are the forward's; the
 * slope is the one at the margin as it is held there, in fp32.
 */
int zs_prefer_backward(const float *margins, const int32_t *lengths, const void *offsets,
                       const void *mask, const float *grad_loss, float *grad, int64_t tokens,
                       int64_t pairs, float beta, float smoothing, int32_t kind, int32_t average,
                       int32_t offset_bytes, void *stream);

/*
 * A gradient: `rows` rows of `width` adjacent elements of `dtype`, grad_stride elements apart,
 * and where its clipped values go (NULL: nowhere; the gradient itself, with the same strides
 * and type, is allowed).
 */
typedef struct zs_grad_tensor {
  const void *grad;
  void *out;
  int64_t rows, width, grad_stride, out_stride;
  int32_t dtype, out_dtype;
} zs_grad_tensor;

/* How many pieces a list of gradients makes (32 bytes of its table each), or a negative error. */
int64_t zs_grads_pieces(const zs_grad_tensor *list, int64_t n);

/*
 * Fills a list's table, in host memory; the calls below read a copy of it in device memory,
 * 256-byte aligned.  It holds addresses: it is laid out anew when a buffer moves.  An
 * output must not overlap another buffer of the list (its own gradient excepted).
 */
int zs_grads_table(const zs_grad_tensor *list, int64_t n, void *table, size_t table_bytes);

/* Workspace of zs_grads_sumsq and zs_grads_clip; 0 when a size is out of range. */
size_t zs_grads_workspace_bytes(int64_t pieces);

/* *sumsq (device) = the sum of the squares of all elements of the list, in fp64. */
int zs_grads_sumsq(const void *table, int64_t pieces, double *sumsq, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * With the device double *sumsq (of this list, or summed over the ranks; NULL: this list's is taken
 * here, for which alone the workspace is used): norm = sqrt(*sumsq),
 * out = c * grad with c = min(1, max_norm / (norm + 1e-6)) in fp32, rounded once to the
 * output's type; *norm_out (device, may be NULL, not sumsq) = norm.  Every gradient of the list
 * has an output.  One that is its own output is left alone where c is 1.
 */
int zs_grads_clip(const void *table, int64_t pieces, float max_norm, const double *sumsq,
                  double *norm_out, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* ZEROSHARD_OPS_H */
