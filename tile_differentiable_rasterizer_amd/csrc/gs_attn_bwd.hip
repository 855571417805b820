// gs_attn_bwd.hip -- gradients of the attention, for gfx950.
//
// The weights are made again from the scores and the kept lse: p = e^(s - lse).  Two kernels, each
// with its results in registers from start to end, so that no sum goes through atomics and its
// order is fixed: k_attn_bwd_kv owns 128 keys and walks the rows (of every query head that shares
// them), k_attn_bwd_q owns 128 rows and walks the keys.  That computes the scores twice (7
// products of a tile instead of 5).
//
// kv: S[row][key] = Q K^T and dP[row][key] = dO V^T leave a lane with one key and 16 rows, the B
// operand of dV^T[d][key] = dO^T P and dK^T[d][key] = Q^T dS.  q: as the forward kernel, S^T and
// dP^T = V dO^T, then dQ^T[d][row] = K^T dS^T.
// p and dS enter the products in the element type (bfloat16: rounded once, 2^-8 of each at most).
#include "gs_attn.h"

namespace gs {

constexpr int kBwdRows = 64;  // rows of a tile of the kv kernel

// delta = dout . out for every (sequence, token, head): 16 lanes a vector, eight elements a lane.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_delta(AttnArgs a) {
  const int heads = a.kv_heads * a.group;
  const int64_t n = (int64_t)a.batch * a.q_len * heads;
  const int64_t v = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  if (v >= n) return;
  const int64_t tok = v / heads;
  const int h = (int)(v - tok * heads), b = (int)(tok / a.q_len), i = (int)(tok - (int64_t)b * a.q_len);
  const int d = (threadIdx.x & 15) * 8;
  float sum = 0.0f;
  if (d < a.d) {
    float x[8], y[8];
    load_elems<8>(head_ptr<T>(a.out, b, i, h) + d, x);
    load_elems<8>(head_ptr<T>(a.dout, b, i, h) + d, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
  }
#pragma unroll
  for (int e = 1; e < 16; e <<= 1) sum += __shfl_xor(sum, e, 64);
  if (d == 0) a.delta[((int64_t)b * heads + h) * a.q_len + i] = sum;
}

template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_bwd_kv(AttnArgs a) {
  using Ti = Tile<T, DP>;
  __shared__ __align__(16) char qt[kBwdRows * Ti::kRowBytes];
  __shared__ __align__(16) char gt[kBwdRows * Ti::kRowBytes];
  __shared__ __align__(16) float lse2[kBwdRows], delta[kBwdRows];
  __shared__ __align__(16) int first[kBwdRows], last[kBwdRows];
  const int nbh = a.batch * a.kv_heads;
  const int bh = blockIdx.x % nbh, rest = blockIdx.x / nbh;
  const int split = rest % a.splits, kb = rest / a.splits;
  const int b = bh / a.kv_heads, hk = bh - b * a.kv_heads;
  const int lane = __lane_id(), half = lane >> 5;
  const int k0 = kb * 128, k1 = min(k0 + 128, a.k_len);
  const int key = k0 + (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool open = key < a.k_len && (!a.mask || a.mask[b * a.mask_b + key] != 0);

  Frag<T> kf[DP / 16], vf[DP / 16];
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) {
    kf[s] = frag_flip(frag_mem<T>(head_ptr<T>(a.k, b, key, hk), a.d, s, open), a.flip);
    vf[s] = frag_mem<T>(head_ptr<T>(a.v, b, key, hk), a.d, s, open);
  }
  f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) dk[t] = dv[t] = (f32x16)0.0f;

  const int tiles = (a.rows + kBwdRows - 1) / kBwdRows;
  const int t_begin = (int)((int64_t)tiles * split / a.splits), t_end = (int)((int64_t)tiles * (split + 1) / a.splits);
  for (int t = t_begin; t < t_end; ++t) {
    const int r0 = t * kBwdRows;
    // every wavefront looks at the tile's 64 rows, one a lane
    const int row = r0 + lane;
    const int i = row < a.rows ? row / a.group : 0, h = hk * a.group + (row < a.rows ? row - i * a.group : 0);
    const int2 range = row_range(a, b, i);
    const int64_t at = ((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i;
    const float row_lse = a.lse[at];
    const bool live = row < a.rows && range.x < range.y && row_lse != -INFINITY;
    const uint64_t word = __ballot(live);
    if (__ballot(live && range.x < k1 && range.y > k0) == 0) continue;  // the same for the workgroup
    const bool ragged = __ballot(live && (range.x > k0 || range.y < k1)) != 0;
    if (threadIdx.x < kBwdRows) {
      lse2[lane] = live ? row_lse * kLog2e : INFINITY;  // a row without keys: every weight 2^-inf = 0
      delta[lane] = live ? a.delta[at] : 0.0f;
      first[lane] = range.x;
      last[lane] = range.y;
    }
    for (int c = threadIdx.x; c < kBwdRows * Ti::kChunks; c += 256) {
      const int r = c / Ti::kChunks, ch = c - r * Ti::kChunks;
      f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
      if (((word >> r) & 1) && ch * Ti::kPer < a.d) {
        const int ri = (r0 + r) / a.group, rh = hk * a.group + (r0 + r) - ri * a.group;
        x = *reinterpret_cast<const f32x4*>(head_ptr<T>(a.q, b, ri, rh) + ch * Ti::kPer);
        y = *reinterpret_cast<const f32x4*>(head_ptr<T>(a.dout, b, ri, rh) + ch * Ti::kPer);
      }
      *reinterpret_cast<f32x4*>(qt + Ti::at(r, ch)) = x;
      *reinterpret_cast<f32x4*>(gt + Ti::at(r, ch)) = y;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kBwdRows / 32; ++j) {
      f32x16 s = (f32x16)0.0f, dp = (f32x16)0.0f;
#pragma unroll
      for (int st = 0; st < DP / 16; ++st) {
        s = mma(Ti::frag_rows(qt, 32 * j, st), kf[st], s);
        dp = mma(Ti::frag_rows(gt, 32 * j, st), vf[st], dp);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int r = 32 * j + 8 * c + 4 * half;
        const f32x4 ls = *reinterpret_cast<const f32x4*>(&lse2[r]), de = *reinterpret_cast<const f32x4*>(&delta[r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bool sees = open;
          if (ragged) sees = sees && key >= first[r + e] && key < last[r + e];
          const float p = sees ? __builtin_amdgcn_exp2f(fmaf(s[4 * c + e], a.slope, -ls[e])) : 0.0f;
          s[4 * c + e] = p;
          dp[4 * c + e] = sees ? p * (dp[4 * c + e] - de[e]) : 0.0f;
        }
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const Frag<T> pf = frag_of<T>(s, st), df = frag_of<T>(dp, st);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) {
          dv[dt] = mma(Ti::frag_cols(gt, 32 * j + 16 * st, 32 * dt), pf, dv[dt]);
          dk[dt] = mma(Ti::frag_cols(qt, 32 * j + 16 * st, 32 * dt), df, dk[dt]);
        }
      }
    }
    __syncthreads();
  }

  if (key >= a.k_len) return;
  const bool parts = a.splits > 1;
  const int64_t n = (int64_t)nbh * a.k_len, at = (int64_t)bh * a.k_len + key;
  T* kp = head_ptr<T>(a.dk, b, key, hk);
  T* vp = head_ptr<T>(a.dv, b, key, hk);
  float* kw = a.part + (split * 2 * n + at) * DP;
  float* vw = kw + n * DP;
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = 32 * dt + 8 * c + 4 * half;
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = dk[dt][4 * c + e] * a.scale;
        y[e] = dv[dt][4 * c + e];
      }
      if (parts) {
        store_elems<4>(kw + d, x);
        store_elems<4>(vw + d, y);
      } else if (d < a.d) {
        store_elems<4>(kp + d, x);
        store_elems<4>(vp + d, y);
      }
    }
}

template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_bwd_q(AttnArgs a) {
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
  const int row = rt * 128 + (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool valid = row < a.rows;
  const int i = valid ? row / a.group : 0, h = hk * a.group + (valid ? row - i * a.group : 0);
  int2 range[1] = {row_range(a, b, i)};
  const int64_t at = ((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i;
  const float row_lse = a.lse[at];
  const bool live = valid && range[0].x < range[0].y && row_lse != -INFINITY;
  if (!live) range[0] = make_int2(0, 0);
  const Seen seen = block_seen<1>(range, scratch);
  const float lse2 = live ? row_lse * kLog2e : INFINITY, delta = live ? a.delta[at] : 0.0f;

  Frag<T> qf[DP / 16], gf[DP / 16];
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) {
    qf[s] = frag_flip(frag_mem<T>(head_ptr<T>(a.q, b, i, h), a.d, s, live), a.flip);
    gf[s] = frag_mem<T>(head_ptr<T>(a.dout, b, i, h), a.d, s, live);
  }
  f32x16 dq[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) dq[t] = (f32x16)0.0f;

  const int t_lo = seen.first / kAttnKeys, t_n = seen.last > seen.first ? (seen.last + kAttnKeys - 1) / kAttnKeys - t_lo : 0;
  Tiles tile;
  tile.t = t_lo + (int)((int64_t)t_n * split / a.splits);
  tile.end = t_lo + (int)((int64_t)t_n * (split + 1) / a.splits);
  if (a.d < DP) {
    Stage<T, DP>::clear(kt, sizeof kt);
    Stage<T, DP>::clear(vt, sizeof vt);
    __syncthreads();
  }
  for (;;) {
    tile.next(a, b, seen, range, words);
    if (!tile.word) break;
    const int k0 = tile.k0;
    const uint64_t word = tile.word;
    const bool ragged = tile.ragged;
    Stage<T, DP>::load(kt, head_ptr<T>(a.k, b, 0, hk), a.k.token_stride, k0, a.d, word);
    Stage<T, DP>::load(vt, head_ptr<T>(a.v, b, 0, hk), a.v.token_stride, k0, a.d, word);
    __builtin_amdgcn_s_waitcnt(0x0f70);
    __syncthreads();
    uint64_t mine = word;
    if (ragged) mine &= range_word(range[0].x, range[0].y, k0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f32x16 s = (f32x16)0.0f, dp = (f32x16)0.0f;
#pragma unroll
      for (int st = 0; st < DP / 16; ++st) {
        s = mma(Ti::frag_rows(kt, 32 * j, st), qf[st], s);
        dp = mma(Ti::frag_rows(vt, 32 * j, st), gf[st], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[r], a.slope, -lse2));
        float ds = p * (dp[r] - delta);
        if (mine != ~0ull) ds = (mine >> (32 * j + crow(r, half))) & 1 ? ds : 0.0f;
        dp[r] = ds;
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const Frag<T> df = frag_of<T>(dp, st);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) dq[dt] = mma(Ti::frag_cols(kt, 32 * j + 16 * st, 32 * dt), df, dq[dt]);
      }
    }
    __syncthreads();
  }

  if (!valid) return;
  T* op = head_ptr<T>(a.dq, b, i, h);
  float* pp = a.part + (((int64_t)split * nbh + bh) * a.rows + row) * DP;
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = 32 * dt + 8 * c + 4 * half;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = live ? dq[dt][4 * c + e] * a.scale : 0.0f;
      if (a.splits > 1)
        store_elems<4>(pp + d, x);
      else if (d < a.d)
        store_elems<4>(op + d, x);
    }
}

// Sums of the splits, in order: dq (KV false, over rows) or dk and dv (KV true, over keys; the
// second half of the grid's y axis is dv).
template <typename T, int DP, bool KV>
__global__ __launch_bounds__(256) void k_attn_bwd_join(AttnArgs a) {
  constexpr int kPer = 256 / (DP / 4);
  const int len = KV ? a.k_len : a.rows;
  const int64_t n = (int64_t)a.batch * a.kv_heads * len, step = KV ? 2 * n : n;
  const int64_t at = (int64_t)blockIdx.x * kPer + threadIdx.x / (DP / 4);
  const int d = (threadIdx.x % (DP / 4)) * 4;
  if ((int)threadIdx.x >= kPer * (DP / 4) || at >= n || d >= a.d) return;
  const float* p = a.part + ((KV && blockIdx.y ? n : 0) + at) * DP + d;
  float x[4] = {};
  for (int s = 0; s < a.splits; ++s) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + s * step * DP);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += v[e];
  }
  const int bh = (int)(at / len), j = (int)(at - (int64_t)bh * len);
  const int b = bh / a.kv_heads, hk = bh - b * a.kv_heads;
  if constexpr (KV) {
    store_elems<4>(head_ptr<T>(blockIdx.y ? a.dv : a.dk, b, j, hk) + d, x);
  } else {
    const int i = j / a.group;
    store_elems<4>(head_ptr<T>(a.dq, b, i, hk * a.group + j - i * a.group) + d, x);
  }
}

int attn_splits(int64_t blocks, int64_t tiles);
int attn_padded(int d);

int attn_bwd_kv_splits(const gs_cross_attn& p) {
  const int64_t rows = p.q_len * (p.q_heads / p.kv_heads);
  return attn_splits(p.batch * p.kv_heads * ((p.k_len + 127) / 128), (rows + kBwdRows - 1) / kBwdRows);
}

namespace {

template <typename T, int DP>
hipError_t bwd_launch(AttnArgs a, int q_splits, int kv_splits, hipStream_t s) {
  const int64_t nbh = (int64_t)a.batch * a.kv_heads, vecs = nbh * a.rows, per = 256 / (DP / 4);
  if (nbh == 0 || (a.rows == 0 && a.k_len == 0)) return hipSuccess;
  if (vecs) k_attn_delta<T><<<(unsigned)((vecs + 15) / 16), 256, 0, s>>>(a);
  if (nbh && a.k_len) {
    a.splits = kv_splits;
    k_attn_bwd_kv<T, DP><<<(unsigned)(nbh * ((a.k_len + 127) / 128) * kv_splits), 256, 0, s>>>(a);
    if (kv_splits > 1)
      k_attn_bwd_join<T, DP, true><<<dim3((unsigned)((nbh * a.k_len + per - 1) / per), 2), 256, 0, s>>>(a);
  }
  if (vecs) {
    a.splits = q_splits;
    k_attn_bwd_q<T, DP><<<(unsigned)(nbh * ((a.rows + 127) / 128) * q_splits), 256, 0, s>>>(a);
    if (q_splits > 1) k_attn_bwd_join<T, DP, false><<<(unsigned)((vecs + per - 1) / per), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bwd(AttnArgs a, int type, int q_splits, int kv_splits, hipStream_t s) {
  switch (attn_padded(a.d) + type) {
    case 32 + GS_BF16: return bwd_launch<__bf16, 32>(a, q_splits, kv_splits, s);
    case 64 + GS_BF16: return bwd_launch<__bf16, 64>(a, q_splits, kv_splits, s);
    case 96 + GS_BF16: return bwd_launch<__bf16, 96>(a, q_splits, kv_splits, s);
    case 128 + GS_BF16: return bwd_launch<__bf16, 128>(a, q_splits, kv_splits, s);
    case 32 + GS_F32: return bwd_launch<float, 32>(a, q_splits, kv_splits, s);
    case 64 + GS_F32: return bwd_launch<float, 64>(a, q_splits, kv_splits, s);
    case 96 + GS_F32: return bwd_launch<float, 96>(a, q_splits, kv_splits, s);
    default: return bwd_launch<float, 128>(a, q_splits, kv_splits, s);
  }
}

}  // namespace gs
