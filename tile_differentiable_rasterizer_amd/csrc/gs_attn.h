// gs_attn.h -- what the forward and backward attention kernels share.  Internal to libgsraster.
//
// The query heads that share a key head are rows of one problem: row r of (sequence b, key head
// hk) is query token r / G of head hk G + r % G, so a token's heads are neighbours in memory and
// in a tile, and a tile's rows see nearly the same keys.
#pragma once

#include "gs_device.h"
#include "gs_mfma.h"

namespace gs {

struct AttnArgs {
  gs_heads q, k, v, out, dout, dq, dk, dv;
  int32_t batch, q_len, k_len, kv_heads, group, d;
  int32_t rows;    // q_len * group
  int32_t splits;  // of the long axis: keys (out, dq) or rows (dk, dv)
  float scale, scale_log2;
  const int32_t* ranges;
  int64_t ranges_b, ranges_r;
  const uint8_t* mask;
  int64_t mask_b;
  float* lse;
  float* delta;
  float* part;     // [splits][batch * kv_heads][rows][DP] sums, where splits > 1
  float2* part_ml; // [splits][batch * kv_heads][rows]: running maximum (base 2), sum
};

// One (sequence, key head) with typed, offset pointers.
struct Where {
  int b, hk;
};

template <typename T>
__device__ __forceinline__ T* head_ptr(const gs_heads& x, int b, int t, int h) {
  return static_cast<T*>(x.data) + b * x.batch_stride + t * x.token_stride + h * x.head_stride;
}

// The keys that query row i of sequence b may see, [first, last) inside [0, k_len).
__device__ __forceinline__ int2 row_range(const AttnArgs& a, int b, int i) {
  int2 r = make_int2(0, a.k_len);
  if (a.ranges) {
    const int64_t at = 2 * (b * a.ranges_b + i * a.ranges_r);
    r.x = max(a.ranges[at], 0);
    r.y = min(a.ranges[at + 1], a.k_len);
  }
  return r;
}

// Bits of the 64 keys from k0 that exist and are not masked, the same in every lane.
__device__ __forceinline__ uint64_t key_word(const AttnArgs& a, int b, int k0) {
  const int key = k0 + (int)__lane_id();
  bool ok = key < a.k_len;
  if (ok && a.mask) ok = a.mask[b * a.mask_b + key] != 0;
  return __ballot(ok);
}

// Bits of the 64 keys from k0 that lie in [first, last).
__device__ __forceinline__ uint64_t range_word(int first, int last, int k0) {
  const int lo = max(first - k0, 0), hi = min(last - k0, 64);
  if (lo >= hi) return 0;
  return (~0ull >> (64 - (hi - lo))) << lo;
}

__device__ __forceinline__ int wave_min_i(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = min(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ int wave_max_i(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = max(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ uint64_t wave_or(uint64_t x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x |= __shfl_xor(x, d, 64);
  return x;
}

constexpr int kAttnRows = 128;  // rows of a workgroup: four wavefronts of 32
constexpr int kAttnKeys = 64;   // keys of a tile

// Ends of the keys that the workgroup's rows may see.
struct Seen {
  int first, last;      // some row sees something in here
  int all_from, all_to; // every row that sees anything sees all of this
};
// `mine`: the lane's range; `live`: its row exists and the range is not empty.
__device__ __forceinline__ Seen block_seen(int2 mine, bool live, int (*scratch)[4]) {
  const int w = threadIdx.x >> 6;
  const int a = wave_min_i(live ? mine.x : INT32_MAX), b = wave_max_i(live ? mine.y : 0);
  const int c = wave_max_i(live ? mine.x : 0), d = wave_min_i(live ? mine.y : INT32_MAX);
  if (__lane_id() == 0) {
    scratch[w][0] = a;
    scratch[w][1] = b;
    scratch[w][2] = c;
    scratch[w][3] = d;
  }
  __syncthreads();
  Seen s = {INT32_MAX, 0, 0, INT32_MAX};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s.first = min(s.first, scratch[i][0]);
    s.last = max(s.last, scratch[i][1]);
    s.all_from = max(s.all_from, scratch[i][2]);
    s.all_to = min(s.all_to, scratch[i][3]);
  }
  __syncthreads();
  return s;
}

// Bits of the tile's keys that some row of the workgroup sees (every thread calls it).
__device__ __forceinline__ uint64_t block_word(uint64_t mine, uint64_t* scratch) {
  const uint64_t w = wave_or(mine);
  if (__lane_id() == 0) scratch[threadIdx.x >> 6] = w;
  __syncthreads();
  const uint64_t r = scratch[0] | scratch[1] | scratch[2] | scratch[3];
  __syncthreads();
  return r;
}

// Copies the rows whose bit is set in `word` from head (b, hk) of x, tokens t0.. , to a tile; the
// other rows, and what lies past D, are zeros (nothing there is read).
template <typename T, int DP, int ROWS>
__device__ __forceinline__ void stage_tokens(char* tile, const gs_heads& x, int b, int h, int t0, int d, uint64_t word) {
  using Ti = Tile<T, DP>;
  for (int c = threadIdx.x; c < ROWS * Ti::kChunks; c += 256) {
    const int r = c / Ti::kChunks, ch = c - r * Ti::kChunks;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (((word >> r) & 1) && ch * Ti::kPer < d)
      v = *reinterpret_cast<const f32x4*>(head_ptr<T>(x, b, t0 + r, h) + ch * Ti::kPer);
    *reinterpret_cast<f32x4*>(tile + Ti::at(r, ch)) = v;
  }
}

}  // namespace gs
