// gs_attn.hip -- attention of query rows to the keys of another sequence, forward, for gfx950.
//
// softmax in one pass over the keys: with m the running maximum and l the running sum of
// 2^(s - m), a tile that raises m scales l and the output by 2^(m_old - m).
//
// The scores are computed transposed, S^T[key][row] = K Q^T, so that a lane holds scores of one
// row only (its column of the result): maximum and sum are in-lane but for one exchange between
// the halves, the row's statistics are one register, and the weights are at once the B operand of
// O^T[d][row] = V^T P^T.  The weights enter that product in the element type (bfloat16: an error
// of 2^-8 of each weight at most, of the order of the output's own rounding); everything else is float32.
#include "gs_attn.h"

namespace gs {

template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_fwd(AttnArgs a) {
  using Ti = Tile<T, DP>;
  __shared__ __align__(16) char kt[kAttnKeys * Ti::kRowBytes];
  __shared__ __align__(16) char vt[kAttnKeys * Ti::kRowBytes];
  __shared__ int scratch[4][4];
  __shared__ uint64_t words[4];
  const int nbh = a.batch * a.kv_heads;
  const int bh = blockIdx.x % nbh, rest = blockIdx.x / nbh;
  const int split = rest % a.splits, rt = rest / a.splits;
  const int b = bh / a.kv_heads, hk = bh - b * a.kv_heads;
  const int lane = __lane_id(), half = lane >> 5;
  const int row = rt * kAttnRows + (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool valid = row < a.rows;
  const int i = valid ? row / a.group : 0, h = hk * a.group + (valid ? row - i * a.group : 0);
  int2 range = row_range(a, b, i);
  const bool live = valid && range.x < range.y;
  const Seen seen = block_seen(range, live, scratch);

  Frag<T> qf[DP / 16];
  const T* qp = head_ptr<T>(a.q, b, i, h);
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) qf[s] = frag_mem<T>(qp, a.d, s, live);

  f32x16 o[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) o[t] = (f32x16)0.0f;
  float m = -INFINITY, l = 0.0f;

  const int t_lo = seen.first / kAttnKeys, t_n = seen.last > seen.first ? (seen.last + kAttnKeys - 1) / kAttnKeys - t_lo : 0;
  const int t_begin = t_lo + (int)((int64_t)t_n * split / a.splits), t_end = t_lo + (int)((int64_t)t_n * (split + 1) / a.splits);
  for (int t = t_begin; t < t_end; ++t) {
    const int k0 = t * kAttnKeys;
    uint64_t word = key_word(a, b, k0);
    const bool ragged = k0 < seen.all_from || k0 + kAttnKeys > seen.all_to;
    if (ragged) word &= block_word(live ? range_word(range.x, range.y, k0) : 0, words);
    if (word == 0) continue;  // the same for the workgroup
    stage_tokens<T, DP, kAttnKeys>(kt, a.k, b, hk, k0, a.d, word);
    stage_tokens<T, DP, kAttnKeys>(vt, a.v, b, hk, k0, a.d, word);
    __syncthreads();

    f32x16 s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j] = (f32x16)0.0f;
#pragma unroll
      for (int st = 0; st < DP / 16; ++st) s[j] = mma(Ti::frag_rows(kt, 32 * j, st), qf[st], s[j]);
    }
    uint64_t mine = word;
    if (ragged && live) mine &= range_word(range.x, range.y, k0);
    float top = m;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float x = s[j][r] * a.scale_log2;
        if (mine != ~0ull) x = (mine >> (32 * j + crow(r, half))) & 1 ? x : -INFINITY;
        s[j][r] = x;
        top = fmaxf(top, x);
      }
    top = pair_max(top);
    const float base = top == -INFINITY ? 0.0f : top;  // nothing seen yet: every weight 2^-inf = 0
    const float keep = __builtin_amdgcn_exp2f(m - base);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(s[j][r] - base);
        s[j][r] = p;
        sum += p;
      }
    l = l * keep + sum;
    m = top;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt) o[dt] *= keep;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const Frag<T> p = frag_of<T>(s[ks >> 1], ks & 1);
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt) o[dt] = mma(Ti::frag_cols(vt, 16 * ks, 32 * dt), p, o[dt]);
    }
    __syncthreads();
  }

  l = pair_sum(l);
  if (!valid) return;
  if (a.splits == 1) {
    const bool none = !live || l == 0.0f;
    const float inv = none ? 0.0f : 1.0f / l;
    T* op = head_ptr<T>(a.out, b, i, h);
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d = 32 * dt + 8 * c + 4 * half;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = none ? 0.0f : o[dt][4 * c + e] * inv;
        if (d < a.d) store_elems<4>(op + d, x);
      }
    if (a.lse && half == 0)
      a.lse[((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
  } else {
    const int64_t at = ((int64_t)split * nbh + bh) * a.rows + row;
    float* op = a.part + at * DP;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = o[dt][4 * c + e];
        store_elems<4>(op + 32 * dt + 8 * c + 4 * half, x);
      }
    if (half == 0) a.part_ml[at] = make_float2(live ? m : -INFINITY, live ? l : 0.0f);
  }
}

// Joins the splits of a row: weights 2^(m_s - max m).  DP / 4 lanes a row, four elements a lane.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int kPer = 256 / (DP / 4);  // rows of a workgroup
  const int64_t nbh = (int64_t)a.batch * a.kv_heads, n = nbh * a.rows;
  const int64_t at = (int64_t)blockIdx.x * kPer + threadIdx.x / (DP / 4);
  const int d = (threadIdx.x % (DP / 4)) * 4;
  if ((int)threadIdx.x >= kPer * (DP / 4) || at >= n) return;
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[s * n + at].x);
  const float base = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, x[4] = {};
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.part_ml[s * n + at];
    if (ml.x == -INFINITY) continue;  // nothing seen there (or no row: its sums are not written)
    const float w = __builtin_amdgcn_exp2f(ml.x - base);
    l += ml.y * w;
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + (s * n + at) * DP + d);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf(v[e], w, x[e]);
  }
  const bool none = l == 0.0f;
  const float inv = none ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] *= inv;
  const int bh = (int)(at / a.rows), row = (int)(at - (int64_t)bh * a.rows);
  const int b = bh / a.kv_heads, i = row / a.group, h = (bh - b * a.kv_heads) * a.group + row - i * a.group;
  if (d < a.d) store_elems<4>(head_ptr<T>(a.out, b, i, h) + d, x);
  if (a.lse && d == 0)
    a.lse[((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

namespace {

template <typename T, int DP>
hipError_t fwd_launch(const AttnArgs& a, hipStream_t s) {
  const int64_t nbh = (int64_t)a.batch * a.kv_heads;
  const int64_t blocks = nbh * ((a.rows + kAttnRows - 1) / kAttnRows) * a.splits;
  k_attn_fwd<T, DP><<<(unsigned)blocks, 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t per = 256 / (DP / 4);
  k_attn_join<T, DP><<<(unsigned)((nbh * a.rows + per - 1) / per), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// Parts that a long axis of `tiles` tiles is split into when `blocks` workgroups are too few for
// 256 CUs: enough for two workgroups a CU, at least two tiles a part.
int attn_splits(int64_t blocks, int64_t tiles) {
  if (blocks <= 0 || blocks >= 512) return 1;
  const int64_t want = (512 + blocks - 1) / blocks, most = tiles / 2;
  return (int)(want < most ? want : most < 1 ? 1 : most);
}

int attn_padded(int d) { return (d + 31) / 32 * 32; }

int attn_fwd_splits(const gs_cross_attn& p) {
  const int64_t rows = p.q_len * (p.q_heads / p.kv_heads);
  return attn_splits(p.batch * p.kv_heads * ((rows + kAttnRows - 1) / kAttnRows), (p.k_len + kAttnKeys - 1) / kAttnKeys);
}

hipError_t launch_attn_fwd(AttnArgs a, int type, hipStream_t s) {
  switch (attn_padded(a.d) + type) {
    case 32 + GS_BF16: return fwd_launch<__bf16, 32>(a, s);
    case 64 + GS_BF16: return fwd_launch<__bf16, 64>(a, s);
    case 96 + GS_BF16: return fwd_launch<__bf16, 96>(a, s);
    case 128 + GS_BF16: return fwd_launch<__bf16, 128>(a, s);
    case 32 + GS_F32: return fwd_launch<float, 32>(a, s);
    case 64 + GS_F32: return fwd_launch<float, 64>(a, s);
    case 96 + GS_F32: return fwd_launch<float, 96>(a, s);
    default: return fwd_launch<float, 128>(a, s);
  }
}

}  // namespace gs
