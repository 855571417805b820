/*
 * gs_tokens.h -- C ABI of the token operators of libgsraster (gfx950): what a decoder that
 * predicts Gaussians from images runs between the images and gs_project.
 *
 * Such a decoder keeps one token for a group of Gaussians and one encoder state for each
 * image tile.  The calls here are the parts of its layer that are not plain matrix products:
 * the norms of queries and keys with the position rotation, the attention of the tokens to the
 * states, and the gated activation of the feed-forward part, which keeps its inputs for the
 * backward pass as 8-bit codes (the fixed-point codes with a (min, max) pair per 256 units of
 * "Training 10M Gaussians in 8 GB: Spirula Studio's VRAM efficiency", here over activations).  What
 * trains such a layer beside them: layer norm, the products of rows with their group's weights
 * (experts), and the optimizer's step over all tensors.
 *
 * The conventions are gs_raster.h's: device pointers owned by the caller unless marked [host],
 * no allocation, scratch from a caller workspace, arguments checked before any HIP call, work
 * enqueued on `stream`, no state between calls, no host wait.  Results do not depend on the
 * order in which workgroups run: no sum goes through atomics, and a call repeated on the same
 * inputs gives the same bits.
 *
 * Element types: GS_BF16 or GS_F32, one for all gs_heads / matrix arguments of a call; norm
 * weights and biases, their gradients, rotation tables, lse and bounds are float32 always.  Sums, norms,
 * softmax statistics and gradients accumulate in float32.
 */
#ifndef GS_TOKENS_H
#define GS_TOKENS_H

#include <stddef.h>
#include <stdint.h>

#include "gs_raster.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GS_BF16 = 0, GS_F32 = 1 };
enum { GS_PAIRS_HALVES = 0, GS_PAIRS_NEIGHBOURS = 1 };
enum { GS_ACT_SILU = 0, GS_ACT_GELU = 1 }; /* x / (1 + e^-x); gelu in its tanh form */

/* Vectors of head_dim elements (dense), one for each (sequence, token, head).  data is 16-byte
 * aligned and the strides, in elements, are multiples of 16 bytes and not negative.  A stride
 * of an axis of length 1 is not used.  Inputs may repeat vectors (a stride of 0); the strides of an
 * output are at least head_dim. */
typedef struct gs_heads {
  void* data;
  int64_t batch_stride, token_stride, head_stride;
} gs_heads;

/* Shape of gs_norm_rotate_*: q[batch][q_len][q_heads][head_dim], k[batch][k_len][k_heads][head_dim].
 * head_dim is a multiple of 8 up to 256; rot_dim, the number of leading elements that are
 * rotated, a multiple of 8 in 0..head_dim.  Pair i (i < rot_dim / 2) is elements (i, i +
 * rot_dim / 2) for GS_PAIRS_HALVES, (2 i, 2 i + 1) for GS_PAIRS_NEIGHBOURS.  n_pos: rows of the
 * rotation tables cos[n_pos][rot_dim / 2] and sin[n_pos][rot_dim / 2]. */
typedef struct gs_norm_rotate {
  int64_t batch, q_len, k_len;
  int32_t q_heads, k_heads, head_dim, rot_dim;
  int32_t pairs, type;
  float eps;
  int64_t n_pos;
} gs_norm_rotate;

/*
 * gs_norm_rotate_fwd -- RMS norm, weight and position rotation of every query and key vector x:
 *   xh = x / sqrt(mean(x^2) + eps),  y = w * xh  (w = wq or wk, [head_dim]),
 *   out = y with each pair (a, b) of its first rot_dim elements replaced by
 *         (a cos - b sin, a sin + b cos), cos and sin those of the token's position.
 *  pos_q[batch][q_len], pos_k[batch][k_len]  table rows (NULL: the token's index in its
 *              sequence); a row outside the table is clamped to its nearest (no read outside)
 *  out_q, out_k  may be the inputs' own buffers with the same strides, and otherwise do not
 *              overlap the inputs
 * Either side may be absent (its length or heads 0: its pointers are not used).
 * Errors: INVALID_ARG, OVERFLOW (2^31 vectors or more), HIP.
 */
gs_status gs_norm_rotate_fwd(const gs_norm_rotate* shape, gs_heads q, gs_heads k, const float* wq, const float* wk,
                             const float* cos, const float* sin, const int32_t* pos_q, const int32_t* pos_k,
                             gs_heads out_q, gs_heads out_k, void* stream);

/*
 * gs_norm_rotate_bwd -- gradients of gs_norm_rotate_fwd from its inputs (nothing is kept from
 * the forward call) and the gradients of its outputs:
 *   g = dout rotated back, dw = sum over vectors of g * xh,
 *   dx = (w g - xh mean(w g xh)) / sqrt(mean(x^2) + eps).
 *  dq, dk      may be dout_q, dout_k's own buffers with the same strides
 *  dwq, dwk    float32 [head_dim], overwritten (0 where a side has no vectors)
 *  workspace   gs_norm_rotate_workspace_bytes(shape) bytes, 16-byte aligned
 * Errors: as the forward call, and WORKSPACE.
 */
size_t gs_norm_rotate_workspace_bytes(const gs_norm_rotate* shape);
gs_status gs_norm_rotate_bwd(const gs_norm_rotate* shape, gs_heads dout_q, gs_heads dout_k, gs_heads q, gs_heads k,
                             const float* wq, const float* wk, const float* cos, const float* sin,
                             const int32_t* pos_q, const int32_t* pos_k, gs_heads dq, gs_heads dk, float* dwq,
                             float* dwk, void* workspace, size_t workspace_bytes, void* stream);

/* Shape and masks of gs_cross_attn_*: q[batch][q_len][q_heads][head_dim], k and v
 * [batch][k_len][kv_heads][head_dim]; q_heads is a multiple of kv_heads, and query head h reads
 * key head h / (q_heads / kv_heads).  head_dim is a multiple of 8 up to 128.  scale is finite, and so is scale *
 * log2(e) in float32 (it is below 2.3e38); 0 and below are scales like the rest.
 *  ranges      int32 pairs [first, last): the keys that a query row may see, cut to [0, k_len);
 *              row (b, i) has the pair at ranges_batch_stride b + ranges_row_stride i (strides
 *              in pairs, 0 = the same for all).  NULL: every key.
 *  key_mask    bytes, 0 = no row of the sequence sees this key; sequence b's are at
 *              key_mask_batch_stride b.  NULL: none masked.
 * Keys and values that no row of a sequence may see are not part of any result, whatever they
 * hold.  (A value that some row sees and another does not has to be finite for the other's
 * result to be: weights of 0 are products like the rest.  So do a row's query and output gradient
 * for the gradients of keys that it does not see and others do; those of a row that sees nothing
 * are not part of any result.)  float32 vectors enter the products as sums of three bfloat16, whose
 * products with an infinity are NaN: where a row sees one (or 3.39e38 and more, which rounds to it), its
 * result may be NaN also where the formula has an infinity or, at a weight of 0, a finite number. */
typedef struct gs_cross_attn {
  int64_t batch, q_len, k_len;
  int32_t q_heads, kv_heads, head_dim, type;
  float scale;
  const int32_t* ranges;
  int64_t ranges_batch_stride, ranges_row_stride;
  const uint8_t* key_mask;
  int64_t key_mask_batch_stride;
} gs_cross_attn;

/*
 * gs_cross_attn_fwd -- attention of every query row to the keys that it may see:
 *   s_j = scale q . k_j,  out = sum_j softmax(s)_j v_j,  lse = log(sum_j e^s_j).
 * A row that sees no key has out = 0 and lse = -inf.
 *  lse         float32 [batch][q_heads][q_len], or NULL
 *  workspace   gs_cross_attn_fwd_workspace_bytes(a) bytes, 16-byte aligned (0 for many shapes:
 *              it holds the parts of a long key axis that is split over workgroups)
 * One query row for each sequence (a token at a time) is the same call with q_len 1.
 * Errors: INVALID_ARG, OVERFLOW (a length of 2^31 or more, or 2^24 blocks of 128 rows or more over all
 * sequences and key heads; a key head has q_len * q_heads / kv_heads rows), WORKSPACE, HIP.
 */
size_t gs_cross_attn_fwd_workspace_bytes(const gs_cross_attn* a);
gs_status gs_cross_attn_fwd(const gs_cross_attn* a, gs_heads q, gs_heads k, gs_heads v, gs_heads out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * gs_cross_attn_bwd -- gradients of gs_cross_attn_fwd, from its inputs, its outputs (out, lse)
 * and the gradient of out.  With p the weights and delta = dout . out:
 *   ds_j = p_j (dout . v_j - delta),  dq = scale sum_j ds_j k_j,
 *   dk_j = scale sum_rows ds_j q,  dv_j = sum_rows p_j dout
 * (rows of every query head that shares the key head).  Everything is overwritten; rows that see
 * nothing and keys that no row sees get 0.
 *  workspace   gs_cross_attn_bwd_workspace_bytes(a) bytes, 16-byte aligned
 * Errors: as the forward call, and OVERFLOW for 2^24 blocks of 128 keys or more.
 */
size_t gs_cross_attn_bwd_workspace_bytes(const gs_cross_attn* a);
gs_status gs_cross_attn_bwd(const gs_cross_attn* a, gs_heads dout, gs_heads q, gs_heads k, gs_heads v, gs_heads out,
                            const float* lse, gs_heads dq, gs_heads dk, gs_heads dv, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * gs_gate8_fwd -- gated activation y = act(gate) * up over rows of `width` units, keeping gate and
 * up for the backward pass as 8-bit codes.
 *  gate, up, y   [rows][width], row strides in elements (at least width)
 *  codes         uint8 [2][rows][width]: gate's, then up's
 *  bounds        float32 [2][rows][ceil(width / 256)][2], 8-byte aligned: (lo, hi) = the minimum
 *                and maximum of each 256 consecutive units of a row (the last block may be
 *                shorter); code = rint((x - lo) * (255 * (1 / (hi - lo)))) with every operation
 *                rounded to float64, 0 where hi == lo.  A block that holds a NaN or an infinity
 *                has NaN bounds and codes 0, so that it stays visible in the gradients.
 * Any width, stride and alignment (of whole elements) is taken; rows that all start at 16-byte
 * boundaries (codes: 8) go faster.
 * Errors: INVALID_ARG, OVERFLOW (2^31 blocks or more), HIP.
 */
gs_status gs_gate8_fwd(int64_t rows, int64_t width, int32_t act, int32_t type, const void* gate, int64_t gate_stride,
                       const void* up, int64_t up_stride, void* y, int64_t y_stride, uint8_t* codes, float* bounds,
                       void* stream);

/*
 * gs_gate8_bwd -- backward pass of gs_gate8_fwd from its codes.  A code stands for
 * lo + code * ((hi - lo) * (1 / 255)), in float32 with every operation rounded, and for NaN where
 * hi - lo is no finite float32.  With g and u these values: dgate = dy * u * act'(g), dup = dy *
 * act(g) and, where y is not NULL, y = act(g) * u again (for the weight gradient of the product
 * that follows: a backward pass that makes that gradient itself need not keep y).
 * Errors: as gs_gate8_fwd.
 */
gs_status gs_gate8_bwd(int64_t rows, int64_t width, int32_t act, int32_t type, const void* dy, int64_t dy_stride,
                       const uint8_t* codes, const float* bounds, void* dgate, int64_t dgate_stride, void* dup,
                       int64_t dup_stride, void* y, int64_t y_stride, void* stream);

/*
 * gs_layer_norm_fwd -- layer norm over rows of `width` units:
 *   xh = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps),  y = w * xh + b.
 *  x, y    [rows][width], row strides in elements (y's at least width; inputs may repeat rows, with a stride of 0);
 *          y may be x's own buffer with the same stride, and otherwise does not overlap x
 *  w, b    float32 [width]; NULL: 1 and 0
 * Any stride and alignment (of whole elements) is taken; width is at most 16384.  The variance is a float32: units up to
 * 1e19 from their row's mean, which is any up to 3e38.  rows or width of 0: nothing is done.
 * Errors: INVALID_ARG, OVERFLOW (a width past 16384, 2^31 rows or more), HIP.
 */
gs_status gs_layer_norm_fwd(int64_t rows, int64_t width, int32_t type, float eps, const void* x, int64_t x_stride,
                            const float* w, const float* b, void* y, int64_t y_stride, void* stream);

/*
 * gs_layer_norm_bwd -- gradients of gs_layer_norm_fwd from its inputs (nothing is kept from the
 * forward call) and the gradient of y.  With g = w * dy and rstd = 1 / sqrt(variance + eps):
 *   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum over rows of dy * xh,  db = sum over rows of dy.
 * The sums over a row are float32s: g, and g times a unit's distance from the mean, up to 1e34.
 *  dx        may be dy's or x's own buffer with the same stride, and otherwise overlaps neither
 *  dw, db    float32 [width], overwritten (0 where there are no rows); NULL: not wanted
 *  workspace gs_layer_norm_workspace_bytes(rows, width) bytes, 16-byte aligned (not looked at where neither dw
 *            nor db is wanted)
 * Errors: as the forward call, and WORKSPACE.
 */
size_t gs_layer_norm_workspace_bytes(int64_t rows, int64_t width);
gs_status gs_layer_norm_bwd(int64_t rows, int64_t width, int32_t type, float eps, const void* dy, int64_t dy_stride,
                            const void* x, int64_t x_stride, const float* w, void* dx, int64_t dx_stride, float* dw,
                            float* db, void* workspace, size_t workspace_bytes, void* stream);

/* Weights of gs_group_mm_*, or their gradients: element (g, i, j) of [groups][k][n] is at
 * g * group_stride + i * k_stride + j * n_stride, in elements; k_stride or n_stride is 1 (an axis of
 * length 1 is not looked at).  The others of an input may be 0: groups, rows or columns that repeat. */
typedef struct gs_weights {
  void* data;
  int64_t group_stride, k_stride, n_stride;
} gs_weights;

/* Shape of gs_group_mm_*: x[rows][k], weights[groups][k][n], y[rows][n], all of one type.  Rows are sorted by
 * group: group g has the rows [offsets[g], offsets[g + 1]).  offsets (device, int32 [groups + 1]) do not
 * decrease; they are cut to [0, rows], and nothing outside of the matrices is read or written whatever they
 * hold.  Rows before the first group's and behind the last one's belong to none.  Groups are looked up 64 at a time: from about 1024 on
 * the time grows with their square (16384 groups: 3.4 ms in bfloat16
 * with rows on 16 bytes, 2.0 ms otherwise). */
typedef struct gs_group_mm {
  int64_t rows, k, n;
  int32_t groups, type;
  const int32_t* offsets;
} gs_group_mm;

/*
 * gs_group_mm_fwd -- the product of every row with its group's weights: y[r] = x[r] W[g(r)].  Rows that
 * belong to no group get 0, whatever x holds there.
 *  x, y        row strides in elements (y's at least n; inputs may repeat rows with a stride of 0); y overlaps
 *              no input
 *  workspace   gs_group_mm_fwd_workspace_bytes(p) bytes, 16-byte aligned (0 for many shapes: it holds the
 *              parts of a long sum that is split over workgroups)
 * Any sizes, strides and alignment (of whole elements) are taken; matrices that all start rows at 16-byte boundaries
 * go faster.  k of 0: y is 0.
 * float32 enters the products as sums of three bfloat16 (see gs_cross_attn: products with an infinity, or with 3.39e38 and more,
 * are NaN).
 * Errors: INVALID_ARG, OVERFLOW (2^31 - 256 rows or more, k or n past 2^24, more than 65536 groups, or 2^23 blocks of 128 x 64 results
 * or more, with one for each group), WORKSPACE, HIP.
 */
size_t gs_group_mm_fwd_workspace_bytes(const gs_group_mm* p);
gs_status gs_group_mm_fwd(const gs_group_mm* p, const void* x, int64_t x_stride, gs_weights w, void* y,
                          int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream);

/*
 * gs_group_mm_bwd -- gradients of gs_group_mm_fwd from its inputs and the gradient of y:
 *   dx[r] = dy[r] W[g(r)]^T,  dW[g] = sum over the group's rows of x[r]^T dy[r].
 * Everything is overwritten; rows of no group and weights of a group without rows get 0.  dx (then w is
 * not looked at) or dw.data may be NULL: not wanted.  Outputs overlap nothing else.
 *  workspace   gs_group_mm_bwd_workspace_bytes(p) bytes, 16-byte aligned
 * Errors: as the forward call.
 */
size_t gs_group_mm_bwd_workspace_bytes(const gs_group_mm* p);
gs_status gs_group_mm_bwd(const gs_group_mm* p, const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                          gs_weights w, void* dx, int64_t dx_stride, gs_weights dw, void* workspace,
                          size_t workspace_bytes, void* stream);

/* A tensor of gs_adamw: n units, dense, aligned to whole elements. */
typedef struct gs_adamw_tensor {
  float* param;       /* updated in place */
  const void* grad;   /* float32 or bfloat16 */
  void* copy;         /* bfloat16: receives the new parameters, rounded; NULL: none */
  int64_t n;
  double decay;       /* its weight decay */
} gs_adamw_tensor;

/* Hyper-parameters of gs_adamw (values, host). */
typedef struct gs_adamw_params {
  double lr, beta1, beta2, eps; /* learning rate, moment decays in [0, 1), epsilon (at least 0) */
  int64_t step;                 /* 1-based step number (bias correction 1 - beta^step) */
} gs_adamw_params;

/*
 * gs_adamw -- one step of AdamW (Loshchilov and Hutter) over `count` tensors at once:
 *   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
 *   p = p (1 - lr decay) - lr (m / (1 - b1^step)) / (sqrt(v / (1 - b2^step)) + eps),
 * computed in float64 (the quotient to float32's accuracy), p rounded once.
 *  tensors     [host] read before the call returns; no two of them overlap
 *  grad_type   GS_F32 or GS_BF16, of all gradients; grad_scale (device, one float32; NULL: 1) multiplies
 *              them: a loss scale's reciprocal, or the factor that clips their norm
 *  bits        32: moments m, v are float32.  8: int8 and uint8 codes with bounds float32 (M, V) for each 256
 *              units of a tensor, the largest |m| and v, rounded: m = M (c / 127)^2 with c's sign, c = rint(127 sqrt(|m| / M)), at
 *              most 127; v = V (c / 255)^4, c = rint(255 (v / V)^(1/4)), at most 255 and, where v > 0 and V > 0, at least 1.  Codes
 *              are decided in float64.  They are rounded to nearest after every step, so that a moment decays by whole codes only.
 *              While another unit holds the block's bound, m's codes of up to 0.5 / (1 - sqrt(beta1)) stay as they are (9 with a beta1
 *              of 0.9: 0.5% of M), and v's of up to 0.5 / (1 - beta2^(1/4)) (199 with a beta2 of 0.99, all with 0.999): a unit whose
 *              gradients end or shrink beside such a one keeps that much of a first moment, and a second one that is too large for
 *              them, for as long as the other lasts.  A block whose gradients end together decays as a whole.  Where units of a
 *              block fare differently for long, 32 bits hold the averages that the formula means.
 *              A block with a moment that is no finite float32 has NaN for its bound and codes 0.
 *  m, v, bounds   the moments of all tensors one after another, each starting at a multiple of 256 units: tensor
 *              i's at 256 * sum over j < i of ceil(n_j / 256); bounds [blocks][2] (8 bits; else not looked at), m and v 16-byte,
 *              bounds 8-byte aligned.  All zeros is the start, and what stands behind a tensor's last unit stays 0.
 * lr and step are values of the call: a captured graph repeats them.
 * Errors: INVALID_ARG (also count < 0, n < 0, hyper-parameters that are not finite or out of range), OVERFLOW (2^34 units or
 * more with every tensor's rounded up to 256), HIP.
 */
gs_status gs_adamw(int32_t count, const gs_adamw_tensor* tensors, int32_t grad_type, int32_t bits, void* m, void* v,
                   float* bounds, const gs_adamw_params* hyper, const float* grad_scale, void* stream);

/*
 * gs_adamw_moments -- what the codes of `blocks` blocks of 256 units stand for: out_m and out_v float32
 * [256 * blocks], 16-byte aligned.
 * Errors: INVALID_ARG, OVERFLOW (2^26 blocks or more, as gs_adamw), HIP.
 */
gs_status gs_adamw_moments(int64_t blocks, const int8_t* m, const uint8_t* v, const float* bounds, float* out_m,
                           float* out_v, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GS_TOKENS_H */
