// gs_norm.hip -- RMS norm of each head's query and key vector with the position rotation in the
// same pass, and its gradient, for gfx950.
//
// A vector of head_dim D elements belongs to a group of G lanes (D / 8 rounded up to a power of
// two), eight elements a lane, so that a wavefront works on 64 / G vectors at once and no value
// crosses LDS.  For pairs (i, i + rot / 2) a lane takes four elements of the first half and the
// four of the second half that they rotate with; for neighbouring pairs, and in the tail that is
// not rotated, eight in a row.  Either way a lane holds whole pairs, and the only exchange is the
// sum over the group (DPP and permutes inside the wavefront).
//
// Both sides of the call (queries, then keys) go in one launch: the small calls of a decoding
// step are launch latency and nothing else.
//
//   xh = x rstd, y = w xh, (y_a, y_b) turned by the position's angle;
//   back: g = dy turned back, dw = sum g xh, dx = rstd (w g - xh mean(w g xh)).
// About 20 operations an element for 4 to 12 bytes: the memory bounds it.  104k tokens of 16 vectors of 96 in
// float32: forward 232 us, 5.5 TB/s; backward 378 us and 13 for dw, 5.1 TB/s (a copy of 2 GiB: 4.8).  65k vectors of
// 128 in bfloat16: 9.7 us, 3.4 TB/s; back 13.5 us, 3.7 TB/s, and 4; the smallest calls 2.9 us.
#include <algorithm>

#include "gs_device.h"
#include "gs_elem.h"

namespace gs {

constexpr int kNormThreads = 256;

struct NormSide {
  void *x, *y, *dy;  // fwd: x -> y; bwd: (x, dy) -> y = dx
  int64_t xb, xt, xh, yb, yt, yh, db, dt, dh;
  const float* w;
  const int32_t* pos;
  uint32_t heads, len, vecs;  // vecs = batch * len * heads
};

struct NormArgs {
  NormSide side[2];
  const float *cs, *sn;
  int32_t d, rot, n_pos;
  float eps, inv_d;
  uint32_t blocks0;  // workgroups of side 0 (the others take side 1)
};

// Sum over the group's G lanes, in every lane of the group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <typename T, int G, int PAIRS, bool BWD>
__global__ __launch_bounds__(kNormThreads) void k_norm_rotate(NormArgs a, float* __restrict__ part) {
  constexpr int kVecs = kWave / G;  // vectors of a wavefront
  const int which = blockIdx.x >= a.blocks0;
  const NormSide s = a.side[which];
  const uint32_t block = which ? blockIdx.x - a.blocks0 : blockIdx.x;
  const uint32_t blocks = which ? gridDim.x - a.blocks0 : a.blocks0;
  const int lane = threadIdx.x & (G - 1);
  const int D = a.d, half = a.rot >> 1;
  const bool active = lane * 8 < D, turned = lane * 8 < a.rot;
  // the lane's two chunks of four elements
  const int o0 = PAIRS == GS_PAIRS_HALVES && turned ? 4 * lane : 8 * lane;
  const int o1 = PAIRS == GS_PAIRS_HALVES && turned ? half + 4 * lane : 8 * lane + 4;

  float w[8] = {};
  if (active) {
    float t[4];
    load_elems<4>(s.w + o0, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = t[i];
    load_elems<4>(s.w + o1, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 + i] = t[i];
  }
  float dw[8] = {};

  const uint32_t step = blocks * (kNormThreads / G);
  for (uint32_t v = block * (kNormThreads / G) + threadIdx.x / G; v < s.vecs; v += step) {
    const uint32_t tok = v / s.heads, h = v - tok * s.heads;
    const uint32_t b = tok / s.len, t = tok - b * s.len;
    float x[8] = {}, g[8] = {}, c[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 1.0f;
      sn[i] = 0.0f;
    }
    if (active) {
      const T* xp = static_cast<const T*>(s.x) + b * s.xb + t * s.xt + h * s.xh;
      float u[4];
      load_elems<4>(xp + o0, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = u[i];
      load_elems<4>(xp + o1, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 + i] = u[i];
      if constexpr (BWD) {
        const T* gp = static_cast<const T*>(s.dy) + b * s.db + t * s.dt + h * s.dh;
        load_elems<4>(gp + o0, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = u[i];
        load_elems<4>(gp + o1, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[4 + i] = u[i];
      }
      if (turned) {
        int64_t at = s.pos ? s.pos[tok] : (int32_t)t;
        at = at < 0 ? 0 : at >= a.n_pos ? a.n_pos - 1 : at;
        load_elems<4>(a.cs + at * half + 4 * lane, c);
        load_elems<4>(a.sn + at * half + 4 * lane, sn);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float rstd = 1.0f / sqrtf(group_sum<G>(ss) * a.inv_d + a.eps);
    float y[8];
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i] * rstd * w[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& p = PAIRS == GS_PAIRS_HALVES ? y[i] : y[2 * i];
        float& q = PAIRS == GS_PAIRS_HALVES ? y[4 + i] : y[2 * i + 1];
        const float p0 = p, q0 = q;
        p = p0 * c[i] - q0 * sn[i];
        q = p0 * sn[i] + q0 * c[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rotated back
        float& p = PAIRS == GS_PAIRS_HALVES ? g[i] : g[2 * i];
        float& q = PAIRS == GS_PAIRS_HALVES ? g[4 + i] : g[2 * i + 1];
        const float p0 = p, q0 = q;
        p = p0 * c[i] + q0 * sn[i];
        q = q0 * c[i] - p0 * sn[i];
      }
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[i] * rstd;
        dw[i] = fmaf(g[i], xh, dw[i]);
        g[i] *= w[i];
        dot = fmaf(g[i], xh, dot);
        x[i] = xh;
      }
      dot = group_sum<G>(dot) * a.inv_d;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = rstd * (g[i] - x[i] * dot);
    }
    if (active) {
      T* yp = static_cast<T*>(s.y) + b * s.yb + t * s.yt + h * s.yh;
      float u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = y[i];
      store_elems<4>(yp + o0, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = y[4 + i];
      store_elems<4>(yp + o1, u);
    }
  }

  if constexpr (BWD) {
    // the workgroup's sum for each element: lanes of equal place, then the wavefronts, in a fixed order
    __shared__ float sum[kNormThreads / kWave][8 * G];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int d = G; d < kWave; d <<= 1) dw[i] += __shfl_xor(dw[i], d, 64);
      if ((threadIdx.x & (kWave - 1)) < G) sum[threadIdx.x / kWave][(i < 4 ? o0 + i : o1 + i - 4) & (8 * G - 1)] = dw[i];
    }
    __syncthreads();
    if ((int)threadIdx.x < D) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < kNormThreads / kWave; ++i) t += sum[i][threadIdx.x];
      part[(int64_t)blockIdx.x * D + threadIdx.x] = t;
    }
  }
}

// dw[side][e] = sum over the side's workgroups of their parts, in a fixed order: one workgroup for
// each side and 16 elements, 64 threads an element, then a tree.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* __restrict__ part, int D, uint32_t blocks0,
                                                  uint32_t blocks, float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sum[16][16];
  const int e = blockIdx.x * 16 + (threadIdx.x & 15), row = threadIdx.x >> 4;
  const uint32_t b0 = blockIdx.y ? blocks0 : 0, b1 = blockIdx.y ? blocks : blocks0;
  float t = 0.0f;
  if (e < D) {
    const float* p = part + e;
    uint32_t b = b0 + row;
    for (; b + 64 * 7 < b1; b += 64 * 8) {  // eight loads in flight
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[(int64_t)(b + 64 * i) * D];
#pragma unroll
      for (int i = 0; i < 8; ++i) t += x[i];
    }
    for (; b < b1; b += 64) t += p[(int64_t)b * D];
  }
  t += __shfl_xor(t, 16, 64);
  t += __shfl_xor(t, 32, 64);
  if (__lane_id() < 16) sum[threadIdx.x >> 6][threadIdx.x & 15] = t;
  __syncthreads();
  if (threadIdx.x < 16 && e < D) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][threadIdx.x];
    (blockIdx.y ? dwk : dwq)[e] = t;
  }
}

namespace {

// Workgroups of a launch at most.  Forward: one for every 256 / G vectors, as far as a grid should go (float32, 104k
// tokens of 16 vectors of 96: 232 us; eight workgroups a CU that walk the vectors: 263).  Backward, where each leaves a
// part of dw: eight a CU, and more where each still has eight rounds (the same vectors, with the parts' sum: 2048 404 us,
// 8192 391, 13042 392; 65k vectors of 128 in bfloat16: 2048 17.4 us, 1024 17.4, 512 20.6).
constexpr int64_t kNormFwdBlocks = 65536, kNormBwdLeast = 2048, kNormBwdMost = 8192;

int norm_group(int d) {
  int g = 1;
  while (g * 8 < d) g <<= 1;
  return g;
}

// Workgroups of the two sides, in proportion to their vectors.
void norm_blocks(const gs_norm_rotate& p, bool bwd, uint32_t* b0, uint32_t* b1) {
  const int64_t vq = p.batch * p.q_len * p.q_heads, vk = p.batch * p.k_len * p.k_heads;
  const int64_t each = kNormThreads / norm_group(p.head_dim);
  const int64_t nq = (vq + each - 1) / each, nk = (vk + each - 1) / each;
  const int64_t most = bwd ? std::min(kNormBwdMost, std::max(kNormBwdLeast, (nq + nk) / 8)) : kNormFwdBlocks;
  if (nq + nk <= most) {
    *b0 = (uint32_t)nq;
    *b1 = (uint32_t)nk;
    return;
  }
  int64_t q = (int64_t)((double)most * (double)nq / (double)(nq + nk));
  q = nq ? (q < 1 ? 1 : q > nq ? nq : q) : 0;
  int64_t k = most - q;
  k = nk ? (k < 1 ? 1 : k > nk ? nk : k) : 0;
  *b0 = (uint32_t)q;
  *b1 = (uint32_t)k;
}

template <typename T, int G, bool BWD>
void norm_launch(const gs_norm_rotate& p, const NormArgs& a, uint32_t blocks, float* part, hipStream_t s) {
  if (p.pairs == GS_PAIRS_HALVES)
    k_norm_rotate<T, G, GS_PAIRS_HALVES, BWD><<<blocks, kNormThreads, 0, s>>>(a, part);
  else
    k_norm_rotate<T, G, GS_PAIRS_NEIGHBOURS, BWD><<<blocks, kNormThreads, 0, s>>>(a, part);
}

template <typename T, bool BWD>
void norm_pick(const gs_norm_rotate& p, const NormArgs& a, uint32_t blocks, float* part, hipStream_t s) {
  switch (norm_group(p.head_dim)) {
    case 1: norm_launch<T, 1, BWD>(p, a, blocks, part, s); break;
    case 2: norm_launch<T, 2, BWD>(p, a, blocks, part, s); break;
    case 4: norm_launch<T, 4, BWD>(p, a, blocks, part, s); break;
    case 8: norm_launch<T, 8, BWD>(p, a, blocks, part, s); break;
    case 16: norm_launch<T, 16, BWD>(p, a, blocks, part, s); break;
    default: norm_launch<T, 32, BWD>(p, a, blocks, part, s); break;
  }
}

NormSide norm_side(const gs_heads& x, const gs_heads& y, const gs_heads* dy, const float* w, const int32_t* pos,
                   int64_t batch, int64_t len, int64_t heads) {
  NormSide s{};
  s.x = x.data; s.xb = x.batch_stride; s.xt = x.token_stride; s.xh = x.head_stride;
  s.y = y.data; s.yb = y.batch_stride; s.yt = y.token_stride; s.yh = y.head_stride;
  if (dy) { s.dy = dy->data; s.db = dy->batch_stride; s.dt = dy->token_stride; s.dh = dy->head_stride; }
  s.w = w;
  s.pos = pos;
  s.heads = heads > 0 ? (uint32_t)heads : 1;
  s.len = len > 0 ? (uint32_t)len : 1;
  s.vecs = (uint32_t)(batch * len * heads);
  return s;
}

}  // namespace

size_t norm_workspace_bytes(const gs_norm_rotate& p) {
  uint32_t b0, b1;
  norm_blocks(p, true, &b0, &b1);
  return ((size_t)(b0 + b1) * p.head_dim * sizeof(float) + 15) & ~(size_t)15;
}

hipError_t launch_norm_rotate(const gs_norm_rotate& p, const gs_heads& q, const gs_heads& k, const gs_heads* dq,
                              const gs_heads* dk, const float* wq, const float* wk, const float* cs, const float* sn,
                              const int32_t* pos_q, const int32_t* pos_k, const gs_heads& yq, const gs_heads& yk,
                              float* dwq, float* dwk, void* ws, hipStream_t s) {
  NormArgs a{};
  a.side[0] = norm_side(q, yq, dq, wq, pos_q, p.batch, p.q_len, p.q_heads);
  a.side[1] = norm_side(k, yk, dk, wk, pos_k, p.batch, p.k_len, p.k_heads);
  a.cs = cs;
  a.sn = sn;
  a.d = p.head_dim;
  a.rot = p.rot_dim;
  a.n_pos = (int32_t)p.n_pos;
  a.eps = p.eps;
  a.inv_d = 1.0f / (float)p.head_dim;
  uint32_t b1;
  norm_blocks(p, dq != nullptr, &a.blocks0, &b1);
  const uint32_t blocks = a.blocks0 + b1;
  float* part = static_cast<float*>(ws);
  if (blocks) {
    if (p.type == GS_BF16)
      dq ? norm_pick<__bf16, true>(p, a, blocks, part, s) : norm_pick<__bf16, false>(p, a, blocks, part, s);
    else
      dq ? norm_pick<float, true>(p, a, blocks, part, s) : norm_pick<float, false>(p, a, blocks, part, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!dq) return hipSuccess;
  k_norm_dw<<<dim3((p.head_dim + 15) / 16, 2), 1024, 0, s>>>(part, p.head_dim, a.blocks0, blocks, dwq, dwk);
  return hipGetLastError();
}

}  // namespace gs
