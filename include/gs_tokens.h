/*
 * gs_tokens.h -- C ABI of the token operators of libgsraster (gfx950): what a decoder that
 * predicts Gaussians from images runs between the images and gs_project.
 *
 * Such a decoder keeps one token for a group of Gaussians and one encoder state for each
 * image tile.  The calls here are the parts of its layer that are not plain matrix products:
 * the norms of queries and keys with the position rotation, the attention of the tokens to the
 * states, and the gated activation of the feed-forward part, which keeps its inputs for the
 * backward pass as 8-bit codes (the fixed-point codes with a (min, max) pair per 256 units of
 * "Training 10M Gaussians in 8 GB: Spirula Studio's VRAM efficiency", here over activations).
 *
 * The conventions are gs_raster.h's: device pointers owned by the caller unless marked [host],
 * no allocation, scratch from a caller workspace, arguments checked before any HIP call, work
 * enqueued on `stream`, no state between calls, no host wait.  Results do not depend on the
 * order in which workgroups run: no sum goes through atomics, and a call repeated on the same
 * inputs gives the same bits.
 *
 * Element types: GS_BF16 or GS_F32, one for all gs_heads / matrix arguments of a call; norm
 * weights, their gradients, rotation tables, lse and bounds are float32 always.  Sums, norms,
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

#ifdef __cplusplus
}
#endif

#endif /* GS_TOKENS_H */
