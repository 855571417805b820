// gs_group.h -- what the kernels of the products grouped by rows share, gfx950.  Internal to libgsraster.
//
// Rows are sorted by group.  With the rows before the first group's and behind the last one's, which belong
// to none, groups + 2 spans [bound(e), bound(e + 1)) cover all rows; e = 0 and e = groups + 1 are those
// without weights, whose results are 0.
#pragma once

#include "gs_device.h"
#include "gs_elem.h"

namespace gs {

// One product for each group, as C = A B with element strides.
//   by rows (y = x W, dx = dy W^T): M is the span's rows, B the group's weights.
//   over rows (dW = x^T dy): the sum runs over the span's rows, C is the group's.
struct GroupArgs {
  const void *a, *b;
  void* c;
  int64_t a_m, a_k, b_g, b_k, b_n, c_g, c_m, c_n;
  int32_t rows, groups, m, n, k;  // by rows: m = rows; over rows: k = rows
  const int32_t* offsets;
};

__device__ __forceinline__ int group_bound(const GroupArgs& a, int e) {
  if (e <= 0) return 0;
  if (e >= a.groups + 2) return a.rows;
  return min(max(a.offsets[e - 1], 0), a.rows);
}

struct GroupSpan {
  int group;        // -1: none
  int first, last;  // rows; empty: no such tile
};

// The `tile`-th block of BM rows, spans counted one after another.  Every lane of the wavefront calls it.  Offsets that decrease
// make other blocks than there are, never one outside of its span.
template <int BM>
__device__ __forceinline__ GroupSpan group_tile(const GroupArgs& a, uint32_t tile) {
  uint32_t run = 0;
  const int spans = a.groups + 2;
  for (int c = 0; c < spans; c += kWave) {
    const int e = c + (int)__lane_id();
    int lo = 0, hi = 0;
    if (e < spans) {
      lo = group_bound(a, e);
      hi = group_bound(a, e + 1);
    }
    const uint32_t mine = hi > lo ? (uint32_t)(hi - lo + BM - 1) / BM : 0;
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const uint32_t t = __shfl_up(upto, d, 64);
      if ((int)__lane_id() >= d) upto += t;
    }
    const uint64_t hit = __ballot(mine > 0 && tile - (run + upto - mine) < mine);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const uint32_t before = run + __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(mine, l);
      GroupSpan s;
      s.last = __builtin_amdgcn_readlane(hi, l);
      s.first = __builtin_amdgcn_readlane(lo, l) + (int)(tile - before) * BM;
      s.group = c + l == 0 || c + l == spans - 1 ? -1 : c + l - 1;
      return s;
    }
    run += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return {-1, 0, 0};
}

}  // namespace gs
