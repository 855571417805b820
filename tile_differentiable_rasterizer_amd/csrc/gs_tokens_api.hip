// gs_tokens_api.hip -- the extern "C" boundary of the token operators (gs_tokens.h): argument
// checks before any HIP call, the workspace layouts, and the launches on the caller's stream.
#include <math.h>

#include "gs_attn.h"
#include "gs_group.h"

namespace gs {
size_t norm_workspace_bytes(const gs_norm_rotate& p);
hipError_t launch_norm_rotate(const gs_norm_rotate& p, const gs_heads& q, const gs_heads& k, const gs_heads* dq,
                              const gs_heads* dk, const float* wq, const float* wk, const float* cs, const float* sn,
                              const int32_t* pos_q, const int32_t* pos_k, const gs_heads& yq, const gs_heads& yk,
                              float* dwq, float* dwk, void* ws, hipStream_t s);
int attn_padded(int d);
int attn_fwd_splits(const gs_cross_attn& p);
int attn_bwd_q_splits(const gs_cross_attn& p);
int attn_bwd_kv_splits(const gs_cross_attn& p);
int attn_order_items(const gs_cross_attn& p);
hipError_t launch_attn_order(AttnArgs& a, int items, int32_t* space, hipStream_t s);
hipError_t launch_attn_fwd(AttnArgs a, int type, hipStream_t s);
hipError_t launch_attn_bwd(AttnArgs a, int type, int q_splits, int kv_splits, hipStream_t s);
hipError_t launch_gate8_fwd(bool vec, int64_t rows, int64_t width, int act, int type, const void* gate, int64_t gs,
                            const void* up, int64_t us, void* y, int64_t ys, uint8_t* codes, float* bounds,
                            hipStream_t s);
hipError_t launch_gate8_bwd(bool vec, int64_t rows, int64_t width, int act, int type, const void* dy, int64_t dys,
                            const uint8_t* codes, const float* bounds, void* dgate, int64_t gs, void* dup, int64_t us,
                            void* y, int64_t ys, hipStream_t s);
size_t layer_norm_workspace_bytes(int64_t rows, int width);
hipError_t launch_layer_norm(int64_t rows, int width, int type, float eps, const void* dy, int64_t ds, const void* x,
                             int64_t xs, const float* w, const float* b, void* y, int64_t ys, float* dw, float* db,
                             void* ws, hipStream_t s);
int64_t group_tiles(bool over_rows, int64_t rows, int64_t m, int64_t n, int64_t groups);
size_t group_part_bytes(bool over_rows, int type, int64_t rows, int64_t m, int64_t n, int64_t k, int64_t groups);
hipError_t launch_group(bool over_rows, GroupArgs a, int type, void* ws, hipStream_t s);
hipError_t launch_adamw(int count, const gs_adamw_tensor* tensors, int grad_type, int bits, void* m, void* v,
                        float* bounds, const gs_adamw_params& h, const float* grad_scale, hipStream_t s);
hipError_t launch_adamw_moments(int64_t blocks, const int8_t* m, const uint8_t* v, const float* bounds, float* out_m,
                                float* out_v, hipStream_t s);
}  // namespace gs

using namespace gs;

namespace {

constexpr int64_t kMost = (int64_t)1 << 31;    // lengths, vectors, blocks of codes: counted in 31 bits
constexpr int64_t kGrid = (int64_t)1 << 24;    // workgroups of 256 threads: a grid has fewer than 2^32 work items
constexpr int64_t kMostUnits = 1 << 24;        // k and n of a grouped product: with a tile more they are still counted in 31 bits
constexpr int64_t kMostGroups = 1 << 16;

bool on(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t size_of(int type) { return type == GS_BF16 ? 2 : 4; }
gs_status status_of(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }
size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// a * b, or -1 past 2^62.
int64_t times(int64_t a, int64_t b) {
  int64_t r;
  return a < 0 || b < 0 || __builtin_mul_overflow(a, b, &r) || r > ((int64_t)1 << 62) ? -1 : r;
}

// Vectors of `d` elements over [batch][len][heads]: base and strides on 16 bytes.  A stride of an
// axis of length 1 is put to 0, so that no product with it matters.
bool heads_ok(gs_heads* x, int64_t batch, int64_t len, int64_t heads, int type) {
  if (!batch || !len || !heads) return true;
  if (batch == 1) x->batch_stride = 0;
  if (len == 1) x->token_stride = 0;
  if (heads == 1) x->head_stride = 0;
  const int64_t each = 16 / size_of(type);
  return x->data && on(x->data, 16) && x->batch_stride >= 0 && x->token_stride >= 0 && x->head_stride >= 0 &&
         x->batch_stride % each == 0 && x->token_stride % each == 0 && x->head_stride % each == 0;
}

// The same for an output, whose vectors lie apart.
bool heads_out_ok(gs_heads* x, int64_t batch, int64_t len, int64_t heads, int64_t d, int type) {
  if (!heads_ok(x, batch, len, heads, type)) return false;
  if (!batch || !len || !heads) return true;
  return (batch == 1 || x->batch_stride >= d) && (len == 1 || x->token_stride >= d) && (heads == 1 || x->head_stride >= d);
}

gs_status norm_shape(const gs_norm_rotate* p) {
  if (!p) return GS_ERR_INVALID_ARG;
  if (p->batch < 0 || p->q_len < 0 || p->k_len < 0 || p->q_heads < 0 || p->k_heads < 0 || p->n_pos < 0)
    return GS_ERR_INVALID_ARG;
  if (p->head_dim < 8 || p->head_dim > 256 || p->head_dim % 8) return GS_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > p->head_dim || p->rot_dim % 8) return GS_ERR_INVALID_ARG;
  if (p->pairs != GS_PAIRS_HALVES && p->pairs != GS_PAIRS_NEIGHBOURS) return GS_ERR_INVALID_ARG;
  if (p->type != GS_BF16 && p->type != GS_F32) return GS_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !(p->eps < INFINITY)) return GS_ERR_INVALID_ARG;
  const int64_t vq = times(times(p->batch, p->q_len), p->q_heads), vk = times(times(p->batch, p->k_len), p->k_heads);
  if (vq < 0 || vk < 0 || vq >= kMost || vk >= kMost || p->q_len >= kMost || p->k_len >= kMost || p->n_pos >= kMost)
    return GS_ERR_OVERFLOW;
  return GS_OK;
}

gs_status norm_call(const gs_norm_rotate* p, gs_heads dout_q, gs_heads dout_k, gs_heads q, gs_heads k, bool bwd,
                    const float* wq, const float* wk, const float* cs, const float* sn, const int32_t* pos_q,
                    const int32_t* pos_k, gs_heads yq, gs_heads yk, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                    void* stream) {
  const gs_status st = norm_shape(p);
  if (st != GS_OK) return st;
  const bool has_q = p->batch && p->q_len && p->q_heads, has_k = p->batch && p->k_len && p->k_heads;
  if (!heads_ok(&q, p->batch, p->q_len, p->q_heads, p->type) ||
      !heads_out_ok(&yq, p->batch, p->q_len, p->q_heads, p->head_dim, p->type) ||
      !heads_ok(&k, p->batch, p->k_len, p->k_heads, p->type) ||
      !heads_out_ok(&yk, p->batch, p->k_len, p->k_heads, p->head_dim, p->type))
    return GS_ERR_INVALID_ARG;
  if ((has_q && (!wq || !on(wq, 16))) || (has_k && (!wk || !on(wk, 16)))) return GS_ERR_INVALID_ARG;
  if ((has_q || has_k) && p->rot_dim && (!cs || !sn || !on(cs, 16) || !on(sn, 16) || p->n_pos < 1)) return GS_ERR_INVALID_ARG;
  if (!on(pos_q, 4) || !on(pos_k, 4)) return GS_ERR_INVALID_ARG;
  if (bwd) {
    if (!heads_ok(&dout_q, p->batch, p->q_len, p->q_heads, p->type) ||
        !heads_ok(&dout_k, p->batch, p->k_len, p->k_heads, p->type))
      return GS_ERR_INVALID_ARG;
    if (!dwq || !dwk || !on(dwq, 4) || !on(dwk, 4)) return GS_ERR_INVALID_ARG;
    const size_t need = norm_workspace_bytes(*p);
    if (need && (!ws || !on(ws, 16) || ws_bytes < need)) return GS_ERR_WORKSPACE;
  }
  return status_of(launch_norm_rotate(*p, q, k, bwd ? &dout_q : nullptr, bwd ? &dout_k : nullptr, wq, wk, cs, sn, pos_q,
                                      pos_k, yq, yk, dwq, dwk, ws, static_cast<hipStream_t>(stream)));
}

gs_status attn_shape(const gs_cross_attn* p, bool bwd) {
  if (!p) return GS_ERR_INVALID_ARG;
  if (p->batch < 0 || p->q_len < 0 || p->k_len < 0 || p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads)
    return GS_ERR_INVALID_ARG;
  if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8) return GS_ERR_INVALID_ARG;
  if (p->type != GS_BF16 && p->type != GS_F32) return GS_ERR_INVALID_ARG;
  if (!isfinite(p->scale * kLog2e)) return GS_ERR_INVALID_ARG;
  if (p->ranges && (!on(p->ranges, 4) || p->ranges_batch_stride < 0 || p->ranges_row_stride < 0)) return GS_ERR_INVALID_ARG;
  if (p->key_mask && p->key_mask_batch_stride < 0) return GS_ERR_INVALID_ARG;
  const int64_t rows = times(p->q_len, p->q_heads / p->kv_heads);
  const int64_t all = times(p->batch, p->kv_heads);
  if (rows < 0 || rows >= kMost - 128 || p->k_len >= kMost - 128 || all < 0 || all >= kMost) return GS_ERR_OVERFLOW;
  const int64_t vq = times(all, rows), vk = times(all, p->k_len);
  // workgroups: 128 rows, and 128 keys for the gradients (in parts only where there are few)
  const int64_t wide = times(all, ((bwd && p->k_len > rows ? p->k_len : rows) + 127) / 128);
  if (vq < 0 || vk < 0 || wide < 0 || wide >= kGrid || vq / 2 >= kMost || vk / 2 >= kMost) return GS_ERR_OVERFLOW;
  return GS_OK;
}

AttnArgs attn_args(const gs_cross_attn& p) {
  AttnArgs a{};
  a.batch = (int32_t)p.batch;
  a.q_len = (int32_t)p.q_len;
  a.k_len = (int32_t)p.k_len;
  a.kv_heads = p.kv_heads;
  a.group = p.q_heads / p.kv_heads;
  a.d = p.head_dim;
  a.rows = (int32_t)(p.q_len * a.group);
  a.scale = p.scale;
  a.slope = fabsf(p.scale) * kLog2e;  // the kernels take the maximum before they scale: not negative
  a.flip = p.scale < 0.0f ? 0x80008000u : 0u;
  a.ranges = p.ranges;
  a.ranges_b = p.ranges_batch_stride;
  a.ranges_r = p.ranges_row_stride;
  a.mask = p.key_mask;
  a.mask_b = p.key_mask_batch_stride;
  return a;
}

int64_t attn_rows(const gs_cross_attn& p) { return p.batch * p.kv_heads * (p.q_len * (p.q_heads / p.kv_heads)); }

// Tiles of 64 rows of all (sequence, key head)s, and the backward pass's arrays over them.
int64_t attn_row_tiles(const gs_cross_attn& p) {
  return p.batch * p.kv_heads * ((p.q_len * (p.q_heads / p.kv_heads) + 63) / 64);
}
size_t attn_stat_bytes(const gs_cross_attn& p) { return (size_t)attn_row_tiles(p) * 64 * sizeof(float2); }
size_t attn_tile_bytes(const gs_cross_attn& p) { return round16((size_t)attn_row_tiles(p) * sizeof(RowTile)); }

// Bytes of the parts of a sum over `vecs` vectors.
size_t part_bytes(const gs_cross_attn& p, int splits, int64_t vecs) {
  return splits > 1 ? (size_t)splits * vecs * attn_padded(p.head_dim) * sizeof(float) : 0;
}
size_t order_bytes(const gs_cross_attn& p) { return round16((size_t)attn_order_items(p) * 2 * sizeof(int32_t)); }

}  // namespace

extern "C" {

size_t gs_norm_rotate_workspace_bytes(const gs_norm_rotate* shape) {
  return norm_shape(shape) == GS_OK ? norm_workspace_bytes(*shape) : 0;
}

gs_status gs_norm_rotate_fwd(const gs_norm_rotate* shape, gs_heads q, gs_heads k, const float* wq, const float* wk,
                             const float* cos, const float* sin, const int32_t* pos_q, const int32_t* pos_k,
                             gs_heads out_q, gs_heads out_k, void* stream) {
  return norm_call(shape, gs_heads{}, gs_heads{}, q, k, false, wq, wk, cos, sin, pos_q, pos_k, out_q, out_k, nullptr,
                   nullptr, nullptr, 0, stream);
}

gs_status gs_norm_rotate_bwd(const gs_norm_rotate* shape, gs_heads dout_q, gs_heads dout_k, gs_heads q, gs_heads k,
                             const float* wq, const float* wk, const float* cos, const float* sin,
                             const int32_t* pos_q, const int32_t* pos_k, gs_heads dq, gs_heads dk, float* dwq,
                             float* dwk, void* workspace, size_t workspace_bytes, void* stream) {
  return norm_call(shape, dout_q, dout_k, q, k, true, wq, wk, cos, sin, pos_q, pos_k, dq, dk, dwq, dwk, workspace,
                   workspace_bytes, stream);
}

size_t gs_cross_attn_fwd_workspace_bytes(const gs_cross_attn* p) {
  if (attn_shape(p, false) != GS_OK) return 0;
  const int splits = attn_fwd_splits(*p);
  if (splits == 1) return order_bytes(*p);
  return order_bytes(*p) + part_bytes(*p, splits, attn_rows(*p)) + round16((size_t)splits * attn_rows(*p) * sizeof(float2));
}

gs_status gs_cross_attn_fwd(const gs_cross_attn* p, gs_heads q, gs_heads k, gs_heads v, gs_heads out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const gs_status st = attn_shape(p, false);
  if (st != GS_OK) return st;
  if (!heads_ok(&q, p->batch, p->q_len, p->q_heads, p->type) ||
      !heads_out_ok(&out, p->batch, p->q_len, p->q_heads, p->head_dim, p->type) ||
      !heads_ok(&k, p->batch, p->k_len, p->kv_heads, p->type) || !heads_ok(&v, p->batch, p->k_len, p->kv_heads, p->type) ||
      !on(lse, 4))
    return GS_ERR_INVALID_ARG;
  const size_t need = gs_cross_attn_fwd_workspace_bytes(p);
  if (need && (!workspace || !on(workspace, 16) || workspace_bytes < need)) return GS_ERR_WORKSPACE;
  if (attn_rows(*p) == 0) return GS_OK;
  AttnArgs a = attn_args(*p);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  if (a.slope == 0.0f) a.slope = 1.0f;
  a.splits = attn_fwd_splits(*p);
  char* at = static_cast<char*>(workspace) + order_bytes(*p);
  a.part = reinterpret_cast<float*>(at);
  a.part_ml = reinterpret_cast<float2*>(at + part_bytes(*p, a.splits, attn_rows(*p)));
  if (const int items = attn_order_items(*p)) {
    const hipError_t e = launch_attn_order(a, items, static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return GS_ERR_HIP;
  }
  return status_of(launch_attn_fwd(a, p->type, static_cast<hipStream_t>(stream)));
}

size_t gs_cross_attn_bwd_workspace_bytes(const gs_cross_attn* p) {
  if (attn_shape(p, true) != GS_OK) return 0;
  const size_t q = part_bytes(*p, attn_bwd_q_splits(*p), attn_rows(*p));
  const size_t kv = part_bytes(*p, attn_bwd_kv_splits(*p), 2 * p->batch * p->kv_heads * p->k_len);
  return order_bytes(*p) + attn_stat_bytes(*p) + attn_tile_bytes(*p) + (q > kv ? q : kv);
}

gs_status gs_cross_attn_bwd(const gs_cross_attn* p, gs_heads dout, gs_heads q, gs_heads k, gs_heads v, gs_heads out,
                            const float* lse, gs_heads dq, gs_heads dk, gs_heads dv, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const gs_status st = attn_shape(p, true);
  if (st != GS_OK) return st;
  for (gs_heads* x : {&dout, &q, &out})
    if (!heads_ok(x, p->batch, p->q_len, p->q_heads, p->type)) return GS_ERR_INVALID_ARG;
  for (gs_heads* x : {&k, &v})
    if (!heads_ok(x, p->batch, p->k_len, p->kv_heads, p->type)) return GS_ERR_INVALID_ARG;
  if (!heads_out_ok(&dq, p->batch, p->q_len, p->q_heads, p->head_dim, p->type)) return GS_ERR_INVALID_ARG;
  for (gs_heads* x : {&dk, &dv})
    if (!heads_out_ok(x, p->batch, p->k_len, p->kv_heads, p->head_dim, p->type)) return GS_ERR_INVALID_ARG;
  if ((attn_rows(*p) && !lse) || !on(lse, 4)) return GS_ERR_INVALID_ARG;
  const size_t need = gs_cross_attn_bwd_workspace_bytes(p);
  if (need && (!workspace || !on(workspace, 16) || workspace_bytes < need)) return GS_ERR_WORKSPACE;
  AttnArgs a = attn_args(*p);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.lse = const_cast<float*>(lse);
  char* at = static_cast<char*>(workspace) + order_bytes(*p);
  a.stat = reinterpret_cast<float2*>(at);
  a.row_tiles = reinterpret_cast<RowTile*>(at + attn_stat_bytes(*p));
  a.part = reinterpret_cast<float*>(at + attn_stat_bytes(*p) + attn_tile_bytes(*p));
  if (const int items = attn_order_items(*p)) {
    const hipError_t e = launch_attn_order(a, items, static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return GS_ERR_HIP;
  }
  return status_of(launch_attn_bwd(a, p->type, attn_bwd_q_splits(*p), attn_bwd_kv_splits(*p), static_cast<hipStream_t>(stream)));
}

namespace {
gs_status gate_shape(int64_t rows, int64_t width, int32_t act, int32_t type, const float* bounds) {
  if (rows < 0 || width < 0 || (act != GS_ACT_SILU && act != GS_ACT_GELU) || (type != GS_BF16 && type != GS_F32))
    return GS_ERR_INVALID_ARG;
  if (rows && width && (!bounds || !on(bounds, 8))) return GS_ERR_INVALID_ARG;
  const int64_t items = width > ((int64_t)1 << 40) ? -1 : times(rows, (width + 255) / 256);
  return items < 0 || items >= kMost ? GS_ERR_OVERFLOW : GS_OK;
}
// A matrix of `rows` rows: whole elements; *vec stays true where every row starts on 16 bytes.
bool matrix_ok(const void* p, int64_t stride, int64_t rows, int64_t width, int type, bool* vec) {
  if (!p || !on(p, size_of(type))) return false;
  if (rows > 1 && stride < width) return false;
  *vec = *vec && on(p, 16) && (rows == 1 || stride * size_of(type) % 16 == 0);
  return true;
}
}  // namespace

gs_status gs_gate8_fwd(int64_t rows, int64_t width, int32_t act, int32_t type, const void* gate, int64_t gate_stride,
                       const void* up, int64_t up_stride, void* y, int64_t y_stride, uint8_t* codes, float* bounds,
                       void* stream) {
  const gs_status st = gate_shape(rows, width, act, type, bounds);
  if (st != GS_OK) return st;
  if (!rows || !width) return GS_OK;
  bool vec = codes && on(codes, 8) && width % 8 == 0;
  if (!codes || !matrix_ok(gate, gate_stride, rows, width, type, &vec) ||
      !matrix_ok(up, up_stride, rows, width, type, &vec) || !matrix_ok(y, y_stride, rows, width, type, &vec))
    return GS_ERR_INVALID_ARG;
  return status_of(launch_gate8_fwd(vec, rows, width, act, type, gate, gate_stride, up, up_stride, y, y_stride, codes,
                                    bounds, static_cast<hipStream_t>(stream)));
}

gs_status gs_gate8_bwd(int64_t rows, int64_t width, int32_t act, int32_t type, const void* dy, int64_t dy_stride,
                       const uint8_t* codes, const float* bounds, void* dgate, int64_t dgate_stride, void* dup,
                       int64_t dup_stride, void* y, int64_t y_stride, void* stream) {
  const gs_status st = gate_shape(rows, width, act, type, bounds);
  if (st != GS_OK) return st;
  if (!rows || !width) return GS_OK;
  bool vec = codes && on(codes, 8) && width % 8 == 0;
  if (!codes || !matrix_ok(dy, dy_stride, rows, width, type, &vec) ||
      !matrix_ok(dgate, dgate_stride, rows, width, type, &vec) || !matrix_ok(dup, dup_stride, rows, width, type, &vec) ||
      (y && !matrix_ok(y, y_stride, rows, width, type, &vec)))
    return GS_ERR_INVALID_ARG;
  return status_of(launch_gate8_bwd(vec, rows, width, act, type, dy, dy_stride, codes, bounds, dgate, dgate_stride, dup,
                                    dup_stride, y, y_stride, static_cast<hipStream_t>(stream)));
}

namespace {

constexpr int64_t kMostWidth = 16384;  // units of a row that its lanes' registers hold

gs_status layer_norm_shape(int64_t rows, int64_t width, int32_t type, float eps) {
  if (rows < 0 || width < 0 || (type != GS_BF16 && type != GS_F32) || !(eps >= 0.0f) || !(eps < INFINITY)) return GS_ERR_INVALID_ARG;
  return rows >= kMost || width > kMostWidth ? GS_ERR_OVERFLOW : GS_OK;
}

// An input's rows: whole elements, and any stride that is not negative.
bool rows_in_ok(const void* p, int64_t stride, int64_t rows, int type) {
  return p && on(p, size_of(type)) && (rows <= 1 || stride >= 0);
}
// An output's: they do not overlap.
bool rows_ok(const void* p, int64_t stride, int64_t rows, int64_t width, int type) {
  bool vec = true;
  return matrix_ok(p, stride, rows, width, type, &vec);
}

}  // namespace

gs_status gs_layer_norm_fwd(int64_t rows, int64_t width, int32_t type, float eps, const void* x, int64_t x_stride,
                            const float* w, const float* b, void* y, int64_t y_stride, void* stream) {
  const gs_status st = layer_norm_shape(rows, width, type, eps);
  if (st != GS_OK) return st;
  if (!rows || !width) return GS_OK;
  if (!rows_in_ok(x, x_stride, rows, type) || !rows_ok(y, y_stride, rows, width, type) || !on(w, 4) || !on(b, 4))
    return GS_ERR_INVALID_ARG;
  return status_of(launch_layer_norm(rows, (int)width, type, eps, nullptr, 0, x, x_stride, w, b, y, y_stride, nullptr, nullptr,
                                     nullptr, static_cast<hipStream_t>(stream)));
}

size_t gs_layer_norm_workspace_bytes(int64_t rows, int64_t width) {
  return layer_norm_shape(rows, width, GS_F32, 0.0f) == GS_OK ? layer_norm_workspace_bytes(rows, (int)width) : 0;
}

gs_status gs_layer_norm_bwd(int64_t rows, int64_t width, int32_t type, float eps, const void* dy, int64_t dy_stride,
                            const void* x, int64_t x_stride, const float* w, void* dx, int64_t dx_stride, float* dw,
                            float* db, void* workspace, size_t workspace_bytes, void* stream) {
  const gs_status st = layer_norm_shape(rows, width, type, eps);
  if (st != GS_OK) return st;
  if (!width || (!rows && !dw && !db)) return GS_OK;
  if (!on(w, 4) || !on(dw, 4) || !on(db, 4)) return GS_ERR_INVALID_ARG;
  if (rows) {
    if (!rows_in_ok(dy, dy_stride, rows, type) || !rows_in_ok(x, x_stride, rows, type) ||
        !rows_ok(dx, dx_stride, rows, width, type))
      return GS_ERR_INVALID_ARG;
    const size_t need = dw || db ? layer_norm_workspace_bytes(rows, (int)width) : 0;
    if (need && (!workspace || !on(workspace, 16) || workspace_bytes < need)) return GS_ERR_WORKSPACE;
  }
  return status_of(launch_layer_norm(rows, (int)width, type, eps, dy, dy_stride, x, x_stride, w, nullptr, dx, dx_stride, dw, db,
                                     workspace, static_cast<hipStream_t>(stream)));
}

namespace {

gs_status group_shape(const gs_group_mm* p, bool bwd) {
  if (!p || p->rows < 0 || p->k < 0 || p->n < 0 || p->groups < 0 || (p->type != GS_BF16 && p->type != GS_F32)) return GS_ERR_INVALID_ARG;
  if (!p->offsets || !on(p->offsets, 4)) return GS_ERR_INVALID_ARG;
  if (p->rows >= kMost - 256 || p->k > kMostUnits || p->n > kMostUnits || p->groups > kMostGroups) return GS_ERR_OVERFLOW;
  // each factor is below 2^31, the counts below 2^62; a workgroup has 512 threads
  constexpr int64_t kMostTiles = kGrid / 2;
  if (!bwd && group_tiles(false, p->rows, p->rows, p->n, p->groups) >= kMostTiles) return GS_ERR_OVERFLOW;
  if (bwd && (group_tiles(false, p->rows, p->rows, p->k, p->groups) >= kMostTiles ||
              group_tiles(true, p->rows, p->k, p->n, p->groups) >= kMostTiles || group_tiles(true, p->rows, p->n, p->k, p->groups) >= kMostTiles))
    return GS_ERR_OVERFLOW;
  return GS_OK;
}

// Weights [groups][k][n], one of their last two axes dense; an input may repeat along the others (a stride of 0), an output's elements lie
// apart.
bool weights_ok(gs_weights* w, int64_t groups, int64_t k, int64_t n, int type, bool out) {
  if (!groups || !k || !n) return true;
  if (groups == 1) w->group_stride = 0;
  if (k == 1 && n == 1) w->k_stride = w->n_stride = 1;
  else if (k == 1) w->k_stride = w->n_stride == 1 ? n : 1;
  else if (n == 1) w->n_stride = w->k_stride == 1 ? k : 1;
  if (!w->data || !on(w->data, size_of(type)) || w->group_stride < 0 || w->k_stride < 0 || w->n_stride < 0) return false;
  if (w->n_stride != 1 && w->k_stride != 1) return false;
  const bool along_n = w->n_stride == 1;
  const int64_t rows = along_n ? k : n, each = along_n ? n : k, stride = along_n ? w->k_stride : w->n_stride;
  if (rows > 1 && stride < each && (out || stride)) return false;
  const int64_t most = times(rows - 1, stride), between = times(groups - 1, w->group_stride);  // of the last row, of the last group
  if (most < 0 || between < 0) return false;
  // a group's rows one after another, or all groups' first rows, then all their second ones
  return !out || groups == 1 || w->group_stride >= most + each || (w->group_stride >= each && (rows == 1 || stride >= between + each));
}

// A stride of a single row is not used.
int64_t of_rows(int64_t stride, int64_t rows) { return rows > 1 ? stride : 0; }

GroupArgs group_args(const gs_group_mm& p) {
  GroupArgs a{};
  a.rows = (int32_t)p.rows;
  a.groups = p.groups;
  a.offsets = p.offsets;
  return a;
}

}  // namespace

size_t gs_group_mm_fwd_workspace_bytes(const gs_group_mm* p) {
  return group_shape(p, false) == GS_OK ? round16(group_part_bytes(false, p->type, p->rows, p->rows, p->n, p->k, p->groups)) : 0;
}

gs_status gs_group_mm_fwd(const gs_group_mm* p, const void* x, int64_t x_stride, gs_weights w, void* y,
                          int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream) {
  const gs_status st = group_shape(p, false);
  if (st != GS_OK) return st;
  if (!p->rows || !p->n) return GS_OK;
  if (!rows_ok(y, y_stride, p->rows, p->n, p->type) || (p->k && !rows_in_ok(x, x_stride, p->rows, p->type)) ||
      !weights_ok(&w, p->groups, p->k, p->n, p->type, false))
    return GS_ERR_INVALID_ARG;
  const size_t need = gs_group_mm_fwd_workspace_bytes(p);
  if (need && (!workspace || !on(workspace, 16) || workspace_bytes < need)) return GS_ERR_WORKSPACE;
  x_stride = of_rows(x_stride, p->rows);
  y_stride = of_rows(y_stride, p->rows);
  GroupArgs a = group_args(*p);
  a.a = x; a.a_m = x_stride; a.a_k = 1;
  a.b = w.data; a.b_g = w.group_stride; a.b_k = w.k_stride; a.b_n = w.n_stride;
  a.c = y; a.c_m = y_stride; a.c_n = 1;
  a.m = a.rows; a.n = (int32_t)p->n; a.k = (int32_t)p->k;
  return status_of(launch_group(false, a, p->type, workspace, static_cast<hipStream_t>(stream)));
}

size_t gs_group_mm_bwd_workspace_bytes(const gs_group_mm* p) {
  if (group_shape(p, true) != GS_OK) return 0;
  // dx's parts, then in their place dW's, whichever way it lies
  const size_t dx = group_part_bytes(false, p->type, p->rows, p->rows, p->k, p->n, p->groups);
  const size_t dw = group_part_bytes(true, p->type, p->rows, p->k, p->n, p->rows, p->groups), turned = group_part_bytes(true, p->type, p->rows, p->n, p->k, p->rows, p->groups);
  return round16(dx > dw ? dx > turned ? dx : turned : dw > turned ? dw : turned);
}

gs_status gs_group_mm_bwd(const gs_group_mm* p, const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                          gs_weights w, void* dx, int64_t dx_stride, gs_weights dw, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const gs_status st = group_shape(p, true);
  if (st != GS_OK) return st;
  const bool has_dx = dx && p->rows && p->k, has_dw = dw.data && p->groups && p->k && p->n;
  if (p->rows && p->n && (has_dx || has_dw) && !rows_in_ok(dy, dy_stride, p->rows, p->type)) return GS_ERR_INVALID_ARG;
  if (has_dx && (!rows_ok(dx, dx_stride, p->rows, p->k, p->type) || !weights_ok(&w, p->groups, p->k, p->n, p->type, false)))
    return GS_ERR_INVALID_ARG;
  if (has_dw && ((p->rows && !rows_in_ok(x, x_stride, p->rows, p->type)) || !weights_ok(&dw, p->groups, p->k, p->n, p->type, true)))
    return GS_ERR_INVALID_ARG;
  const size_t need = has_dx || has_dw ? gs_group_mm_bwd_workspace_bytes(p) : 0;
  if (need && (!workspace || !on(workspace, 16) || workspace_bytes < need)) return GS_ERR_WORKSPACE;
  dy_stride = of_rows(dy_stride, p->rows);
  x_stride = of_rows(x_stride, p->rows);
  dx_stride = of_rows(dx_stride, p->rows);
  if (has_dx) {
    GroupArgs a = group_args(*p);
    a.a = dy; a.a_m = dy_stride; a.a_k = 1;
    a.b = w.data; a.b_g = w.group_stride; a.b_k = w.n_stride; a.b_n = w.k_stride;
    a.c = dx; a.c_m = dx_stride; a.c_n = 1;
    a.m = a.rows; a.n = (int32_t)p->k; a.k = (int32_t)p->n;
    const gs_status e = status_of(launch_group(false, a, p->type, workspace, static_cast<hipStream_t>(stream)));
    if (e != GS_OK) return e;
  }
  if (!has_dw) return GS_OK;
  // the dense axis of dw is the product's second: dW = x^T dy, or its transpose dy^T x
  GroupArgs a = group_args(*p);
  const bool turned = dw.n_stride != 1;
  a.a = turned ? dy : x; a.a_m = 1; a.a_k = turned ? dy_stride : x_stride;
  a.b = turned ? x : dy; a.b_k = turned ? x_stride : dy_stride; a.b_n = 1;
  a.c = dw.data; a.c_g = dw.group_stride; a.c_m = turned ? dw.n_stride : dw.k_stride; a.c_n = 1;
  a.m = (int32_t)(turned ? p->n : p->k); a.n = (int32_t)(turned ? p->k : p->n); a.k = a.rows;
  return status_of(launch_group(true, a, p->type, workspace, static_cast<hipStream_t>(stream)));
}

gs_status gs_adamw(int32_t count, const gs_adamw_tensor* tensors, int32_t grad_type, int32_t bits, void* m, void* v,
                   float* bounds, const gs_adamw_params* hyper, const float* grad_scale, void* stream) {
  if (count < 0 || (count && !tensors) || !hyper || (grad_type != GS_BF16 && grad_type != GS_F32) || (bits != 8 && bits != 32))
    return GS_ERR_INVALID_ARG;
  const gs_adamw_params h = *hyper;
  if (h.step < 1 || !(h.beta1 >= 0.0 && h.beta1 < 1.0) || !(h.beta2 >= 0.0 && h.beta2 < 1.0) || !(h.eps >= 0.0 && h.eps < INFINITY) ||
      !isfinite(h.lr) || !on(grad_scale, 4))
    return GS_ERR_INVALID_ARG;
  int64_t blocks = 0;
  for (int32_t i = 0; i < count; ++i) {
    const gs_adamw_tensor& x = tensors[i];
    if (x.n < 0 || !isfinite(x.decay)) return GS_ERR_INVALID_ARG;
    if (!x.n) continue;
    if (!x.param || !x.grad || !on(x.param, 4) || !on(x.grad, size_of(grad_type)) || !on(x.copy, 2)) return GS_ERR_INVALID_ARG;
    if (x.n >= (int64_t)1 << 34) return GS_ERR_OVERFLOW;
    blocks += (x.n + 255) / 256;
    if (blocks >= (int64_t)1 << 26) return GS_ERR_OVERFLOW;
  }
  if (!blocks) return GS_OK;
  if (!m || !v || !on(m, 16) || !on(v, 16) || (bits == 8 && (!bounds || !on(bounds, 8)))) return GS_ERR_INVALID_ARG;
  return status_of(launch_adamw(count, tensors, grad_type, bits, m, v, bounds, h, grad_scale, static_cast<hipStream_t>(stream)));
}

gs_status gs_adamw_moments(int64_t blocks, const int8_t* m, const uint8_t* v, const float* bounds, float* out_m,
                           float* out_v, void* stream) {
  if (blocks < 0) return GS_ERR_INVALID_ARG;
  if (blocks >= (int64_t)1 << 26) return GS_ERR_OVERFLOW;
  if (!blocks) return GS_OK;
  if (!m || !v || !bounds || !out_m || !out_v || !on(m, 8) || !on(v, 8) || !on(bounds, 8) || !on(out_m, 16) || !on(out_v, 16))
    return GS_ERR_INVALID_ARG;
  return status_of(launch_adamw_moments(blocks, m, v, bounds, out_m, out_v, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
