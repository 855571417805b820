// gs_group.hip -- products of rows with their group's weights (experts, or heads of a kind), and their
// gradients, for gfx950.
//
//   y[r] = x[r] W[g(r)],  dx[r] = dy[r] W[g(r)]^T,  dW[g] = sum over the group's rows of x[r]^T dy[r].
#include <algorithm>

#include "gs_group.h"

namespace gs {

hipError_t launch_group_mfma(bool over_rows, const GroupArgs& a, hipStream_t s);

constexpr int kPlainTile = 64, kPlainStep = 16;

// Any strides and sizes: 64 x 64 results a workgroup, 4 x 4 a thread.
template <typename T, bool OVER_ROWS>
__global__ __launch_bounds__(256) void k_group_plain(GroupArgs a) {
  __shared__ float as[kPlainStep][kPlainTile + 4], bs[kPlainStep][kPlainTile + 4];
  const int n_tiles = (a.n + kPlainTile - 1) / kPlainTile;
  int m0, n0, m_end, k0, k_end, g;
  if constexpr (OVER_ROWS) {
    const int m_tiles = (a.m + kPlainTile - 1) / kPlainTile, each = m_tiles * n_tiles;
    g = blockIdx.x / each;
    const int rest = blockIdx.x - g * each;
    m0 = rest / n_tiles * kPlainTile;
    n0 = rest % n_tiles * kPlainTile;
    m_end = a.m;
    k0 = group_bound(a, g + 1);
    k_end = group_bound(a, g + 2);
  } else {
    GroupTiles<kPlainTile> tiles;
    tiles.look(a, 0);
    const GroupSpan s = tiles.find(a, blockIdx.x / n_tiles);
    if (s.first >= s.last) return;
    g = s.group;
    m0 = s.first;
    m_end = s.last;
    n0 = blockIdx.x % n_tiles * kPlainTile;
    k0 = 0;
    k_end = g < 0 ? 0 : a.k;
  }
  const T *A = static_cast<const T*>(a.a), *B = static_cast<const T*>(a.b) + (OVER_ROWS || g < 0 ? 0 : g * a.b_g);
  float acc[4][4] = {};
  const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
  for (int k = k0; k < k_end; k += kPlainStep) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = threadIdx.x + 256 * i;
      // consecutive threads along the axis that lies dense
      const int am = a.a_k == 1 ? at / kPlainStep : at % kPlainTile, ak = a.a_k == 1 ? at % kPlainStep : at / kPlainTile;
      as[ak][am] = m0 + am < m_end && k + ak < k_end ? (float)A[(int64_t)(m0 + am) * a.a_m + (int64_t)(k + ak) * a.a_k] : 0.0f;
      const int bn = a.b_n == 1 ? at % kPlainTile : at / kPlainStep, bk = a.b_n == 1 ? at / kPlainTile : at % kPlainStep;
      bs[bk][bn] = n0 + bn < a.n && k + bk < k_end ? (float)B[(int64_t)(k + bk) * a.b_k + (int64_t)(n0 + bn) * a.b_n] : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kPlainStep; ++kk) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = as[kk][tm + i];
        y[i] = bs[kk][tn + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
  T* C = static_cast<T*>(a.c) + (OVER_ROWS ? g * a.c_g : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (m0 + tm + i < m_end && n0 + tn + j < a.n) C[(int64_t)(m0 + tm + i) * a.c_m + (int64_t)(n0 + tn + j) * a.c_n] = (T)acc[i][j];
}

namespace {

int64_t tiles(int64_t n, int64_t each) { return (n + each - 1) / each; }

// Whether every row of the three matrices starts on 16 bytes and holds whole chunks of 16, at distances that
// a thread's 32-bit offsets reach.
bool group_aligned(bool over_rows, const GroupArgs& a) {
  constexpr int64_t kFar = 1 << 22;
  const int64_t as = over_rows || a.a_k != 1 ? a.a_k : a.a_m, bs = a.b_n == 1 ? a.b_k : a.b_n;
  for (const void* p : {a.a, a.b, static_cast<const void*>(a.c)})
    if ((uintptr_t)p % 16) return false;
  return as % 8 == 0 && bs % 8 == 0 && a.b_g % 8 == 0 && a.c_g % 8 == 0 && a.c_m % 8 == 0 && a.c_n == 1 && as <= kFar && bs <= kFar && a.c_m <= kFar &&
         a.n % 8 == 0 && (over_rows ? a.m : a.k) % 8 == 0;
}

}  // namespace

// Workgroups of a launch (the caller checks that a grid takes them).
int64_t group_tiles(bool over_rows, int64_t rows, int64_t m, int64_t n, int64_t groups) {
  return over_rows ? groups * tiles(m, kPlainTile) * tiles(n, kPlainTile)
                   : (tiles(rows, kPlainTile) + std::min(groups + 2, rows)) * tiles(n, kPlainTile);
}

hipError_t launch_group(bool over_rows, const GroupArgs& a, int type, hipStream_t s) {
  const int64_t blocks = group_tiles(over_rows, a.rows, a.m, a.n, a.groups);
  if (blocks == 0) return hipSuccess;
  if (type == GS_BF16 && group_aligned(over_rows, a)) return launch_group_mfma(over_rows, a, s);
  if (type == GS_BF16)
    over_rows ? k_group_plain<__bf16, true><<<(unsigned)blocks, 256, 0, s>>>(a) : k_group_plain<__bf16, false><<<(unsigned)blocks, 256, 0, s>>>(a);
  else
    over_rows ? k_group_plain<float, true><<<(unsigned)blocks, 256, 0, s>>>(a) : k_group_plain<float, false><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace gs
