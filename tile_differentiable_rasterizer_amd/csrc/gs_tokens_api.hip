// gs_tokens_api.hip -- the extern "C" boundary of the token operators (gs_tokens.h): argument
// checks before any HIP call, the workspace layouts, and the launches on the caller's stream.
#include <math.h>

#include "gs_attn.h"

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
}  // namespace gs

using namespace gs;

namespace {

constexpr int64_t kMost = (int64_t)1 << 31;    // lengths, vectors, blocks of codes: counted in 31 bits
constexpr int64_t kGroups = (int64_t)1 << 24;  // workgroups of 256 threads: a grid has fewer than 2^32 work items

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
  if (vq < 0 || vk < 0 || wide < 0 || wide >= kGroups || vq / 2 >= kMost || vk / 2 >= kMost) return GS_ERR_OVERFLOW;
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

}  // extern "C"
