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
  int32_t splits;  // parts of the sum over k, each made by workgroups of its own
  float* part;     // where there are several: [splits][rows] (over rows: [splits][groups][m]) rows of group_part_width(n)
};

// Blocks of results that a workgroup makes: on the matrix units straight from LDS, and staged through registers.
enum { kGroup256x256, kGroup128x256, kGroup128x128, kGroup32x256, kGroup32x128, kGroupStaged128, kGroupStaged64, kGroupTiles };

inline int64_t tiles(int64_t n, int64_t each) { return (n + each - 1) / each; }
__host__ __device__ constexpr int group_part_width(int n) { return (n + 7) & ~7; }

// Part `split` of k0 .. k_end, in whole steps of `step`.
__device__ __forceinline__ void group_part(const GroupArgs& a, int split, int step, int* k0, int* k_end) {
  if (a.splits == 1) return;
  const int steps = (*k_end - *k0 + step - 1) / step;
  const int first = *k0 + (int)((int64_t)steps * split / a.splits) * step;
  *k_end = min(*k_end, *k0 + (int)((int64_t)steps * (split + 1) / a.splits) * step);
  *k0 = min(first, *k_end);
}

__device__ __forceinline__ int group_bound(const GroupArgs& a, int e) {
  if (e <= 0) return 0;
  if (e >= a.groups + 2) return a.rows;
  return min(max(a.offsets[e - 1], 0), a.rows);
}

// The group with the `rank`-th most rows, so that workgroups of the longest sums start first (up to 64 groups; else by number).
// Every lane of the wavefront calls it.
__device__ __forceinline__ int group_by_length(const GroupArgs& a, int rank) {
  if (a.groups > kWave) return rank;
  const int lane = (int)__lane_id();
  const int rows = lane < a.groups ? max(group_bound(a, lane + 2) - group_bound(a, lane + 1), 0) : -1;
  int before = 0;  // groups that come before the lane's
  for (int i = 0; i < a.groups; ++i) {
    const int other = __builtin_amdgcn_readlane(rows, i);
    before += other > rows || (other == rows && i < lane);
  }
  return __builtin_ctzll(__ballot(lane < a.groups && before == rank));
}

struct GroupSpan {
  int group;        // -1: none
  int first, last;  // rows; empty: no such tile
};

// Blocks of BM rows, spans counted one after another.  Every lane of the wavefront calls these.  Offsets
// that decrease make other blocks than there are, never one outside of its span.
template <int BM>
struct GroupTiles {
  int lo, hi;           // the lane's span of the 64 looked at
  uint32_t mine, upto;  // its blocks, and all up to it

  __device__ __forceinline__ void look(const GroupArgs& a, int c) {
    const int e = c + (int)__lane_id();
    lo = hi = 0;
    if (e < a.groups + 2) {
      lo = group_bound(a, e);
      hi = group_bound(a, e + 1);
    }
    mine = hi > lo ? (uint32_t)(hi - lo + BM - 1) / BM : 0;
    upto = wave_inclusive_scan(mine);
  }
  __device__ __forceinline__ uint32_t last() const { return __builtin_amdgcn_readlane(upto, kWave - 1); }

  // Blocks of all spans; what look(a, 0) found stays where there are no more than 64.
  __device__ __forceinline__ uint32_t count(const GroupArgs& a) {
    look(a, 0);
    uint32_t all = last();
    for (int c = kWave; c < a.groups + 2; c += kWave) {
      look(a, c);
      all += last();
    }
    return all;
  }

  // The `tile`-th block, after count().
  __device__ __forceinline__ GroupSpan find(const GroupArgs& a, uint32_t tile) {
    uint32_t run = 0;
    const int spans = a.groups + 2;
    for (int c = 0; c < spans; c += kWave) {
      if (spans > kWave) look(a, c);
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
      run += last();
    }
    return {-1, 0, 0};
  }
};

}  // namespace gs
