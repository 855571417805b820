// gs_group_mfma.hip -- the products of rows with their group's weights on the matrix units, bfloat16, for
// gfx950.
#include <algorithm>

#include "gs_group.h"
#include "gs_lds.h"
#include "gs_mfma.h"

namespace gs {

constexpr int kGroupStep = 32;   // k of a tile in LDS
constexpr int kGroupStages = 3;  // tiles in LDS: one worked on, two on their way

__device__ __forceinline__ void group_barrier() { asm volatile("s_barrier" ::: "memory"); }

// One operand's tile of R rows (or columns) by 32 k in LDS, and the loads of its next one.
//   K dense in memory: 64 bytes of k for each row; 16-byte chunk c of row r lies at c ^ (r / 4 % 4).
//   K not dense: R elements for each k; chunk c of k-row r lies at c ^ (4 (r % 4) + r / 4 % 4).
// Either way what a wavefront reads at once lies in different banks (gs_mfma.h).
template <bool K_DENSE, int R>
struct GroupSide {
  static constexpr int kBytes = R * kGroupStep * 2, kLoads = kBytes / 4096, kChunks = (K_DENSE ? kGroupStep : R) / 8;

  const char* base;     // of the tile at k0
  int64_t step;         // bytes of 32 k
  uint32_t off[kLoads];
  int at;               // where the lane reads, from the start of a tile

  static __device__ __forceinline__ int mix(int r) { return K_DENSE ? (r >> 2) & 3 : ((r & 3) << 2) | ((r >> 2) & 3); }
  static __device__ __forceinline__ int row_of(int i) { return (i * 256 + (int)threadIdx.x) / kChunks; }
  static __device__ __forceinline__ int chunk_of(int i) { return (i * 256 + (int)threadIdx.x) % kChunks ^ mix(row_of(i)); }

  // p: element (row 0, k0); stride: of the axis that is not dense; rows (at least 1) exist.  Those past them are read as the last: what comes
  // of them is not stored.  first: the wavefront's first row.
  __device__ __forceinline__ void plan(const __bf16* p, int64_t stride, int rows, int first) {
    base = reinterpret_cast<const char*>(p);
    step = K_DENSE ? kGroupStep * 2 : kGroupStep * 2 * stride;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = row_of(i), c = chunk_of(i) * 8;
      off[i] = K_DENSE ? (uint32_t)(min(r, rows - 1) * stride + c) * 2u : (uint32_t)(r * stride + min(c, rows - 8)) * 2u;
    }
    const int l = __lane_id(), h = l >> 5, i = l & 15;
    if constexpr (K_DENSE) {
      const int r = l & 31;
      at = (first + r) * (kChunks * 16) + ((h ^ mix(r)) << 4);
    } else {
      const int r = 8 * h + (i >> 2), c = first / 8 + (2 * ((l >> 4) & 1) + ((i & 3) >> 1));
      at = r * (kChunks * 16) + ((c ^ mix(r)) << 4) + 8 * (i & 1);
    }
  }
  __device__ __forceinline__ void load(uint32_t to, int tile) const {
    const char* p = base + tile * step;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_to_lds16(p, off[i], to + i * 4096);
  }
  // The last tile, of which k < left exist: the others are 0.
  __device__ __forceinline__ void load_part(uint32_t to, int tile, int left) const {
    const char* p = base + tile * step;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool there = (K_DENSE ? chunk_of(i) * 8 : row_of(i)) < left;
      load_to_lds16(there ? static_cast<const void*>(p + off[i]) : kZeros, to + i * 4096);
    }
  }
  // The lane's eight k of row `first` + 32 m + l % 32, k = 16 s + 8 (l / 32) + 0..7.
  __device__ __forceinline__ bf16x8 read(const char* tile, int m, int s) const {
    if constexpr (K_DENSE) {
      return *reinterpret_cast<const bf16x8*>(tile + (at ^ (s << 5)) + m * 32 * (kChunks * 16));
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const char* p = tile + 16 * s * (kChunks * 16);
      const int o = at ^ (m << 6);
      union {
        s16x4 q[2];
        bf16x8 v;
      } u;
      u.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + o));
      u.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * (kChunks * 16) + (o ^ 16)));
      return u.v;
    }
  }
};

template <bool A_DENSE, bool B_DENSE, bool OVER_ROWS, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256, 2) void k_group_mfma(GroupArgs a) {
  using SideA = GroupSide<A_DENSE, BM>;
  using SideB = GroupSide<B_DENSE, BN>;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int kStage = SideA::kBytes + SideB::kBytes;
  static_assert(WM * WN == 4, "four wavefronts");
  __shared__ __align__(1024) char lds[kGroupStages * kStage];
  const int n_tiles = (a.n + BN - 1) / BN;
  int m0, m_end, n0, k0, k_end, g;
  const uint32_t pid = blockIdx.x;
  if constexpr (OVER_ROWS) {
    const int m_tiles = (a.m + BM - 1) / BM, each = m_tiles * n_tiles;
    g = pid / each;
    const int rest = pid - g * each;
    m0 = rest % m_tiles * BM;
    n0 = rest / m_tiles * BN;
    m_end = a.m;
    k0 = group_bound(a, g + 1);
    k_end = group_bound(a, g + 2);
  } else {
    GroupTiles<BM> tiles;
    const uint32_t m_tiles = tiles.count(a), all = m_tiles * n_tiles;
    if (pid >= all) return;
    // an XCD's workgroups (every eighth) side by side, in blocks of eight tiles of rows
    const uint32_t xcd = pid % 8, each = all / 8, more = all % 8;
    const uint32_t id = xcd * each + min(xcd, more) + pid / 8;
    const uint32_t patch = id / (8 * n_tiles), rest = id - patch * 8 * n_tiles, high = min(8u, m_tiles - patch * 8);
    const GroupSpan s = tiles.find(a, patch * 8 + rest % high);
    if (s.first >= s.last) return;
    g = s.group;
    m0 = s.first;
    m_end = s.last;
    n0 = rest / high * BN;
    k0 = 0;
    k_end = g < 0 ? 0 : a.k;
  }
  const int wave = threadIdx.x / kWave, wm = wave % WM, wn = wave / WM;
  const int k_tiles = k_end > k0 ? (k_end - k0 + kGroupStep - 1) / kGroupStep : 0;

  f32x16 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[n][m] = (f32x16)0.0f;

  if (k_tiles) {
    SideA sa;
    SideB sb;
    const __bf16 *A = static_cast<const __bf16*>(a.a) + m0 * a.a_m + k0 * a.a_k;
    const __bf16 *B = static_cast<const __bf16*>(a.b) + (OVER_ROWS ? 0 : g * a.b_g) + k0 * a.b_k + n0 * a.b_n;
    sa.plan(A, A_DENSE ? a.a_m : a.a_k, m_end - m0, wm * TM * 32);
    sb.plan(B, B_DENSE ? a.b_n : a.b_k, a.n - n0, wn * TN * 32);
    const uint32_t to = lds_address(lds) + (threadIdx.x / kWave) * 1024;
    auto load = [&](int tile, int stage) {
      const uint32_t at = __builtin_amdgcn_readfirstlane(to + stage * kStage);
      const int left = k_end - k0 - tile * kGroupStep;
      if (left >= kGroupStep) {
        sa.load(at, tile);
        sb.load(at + SideA::kBytes, tile);
      } else {
        sa.load_part(at, tile, left);  // left <= 0: zeros that nothing reads, so that the loads on their way can be counted
        sb.load_part(at + SideA::kBytes, tile, left);
      }
    };
    bf16x8 fa[2][TM], fb[2][TN];
    auto read = [&](int which, int stage, int s) {
      const char* tile = lds + stage * kStage;
#pragma unroll
      for (int n = 0; n < TN; ++n) fb[which][n] = sb.read(tile + SideA::kBytes, n, s);
#pragma unroll
      for (int m = 0; m < TM; ++m) fa[which][m] = sa.read(tile, m, s);
    };
    auto multiply = [&](int which) {
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[which][n], fa[which][m], acc[n][m], 0, 0, 0);
    };
    constexpr int kEach = SideA::kLoads + SideB::kLoads;  // loads of a tile
    load(0, 0);
    load(1, 1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kEach) : "memory");
    group_barrier();
    read(0, 0, 0);
    int stage = 0;
    for (int t = 0; t < k_tiles; ++t) {
      const int next = stage == 2 ? 0 : stage + 1, free = stage == 0 ? 2 : stage - 1;
      load(t + 2, free);  // the tile before was read before the last barrier
      read(1, stage, 1);
      multiply(0);
      asm volatile("s_waitcnt lgkmcnt(0) vmcnt(%0)" ::"n"(kEach) : "memory");
      group_barrier();
      read(0, next, 0);
      multiply(1);
      stage = next;
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load goes to LDS that another workgroup has by then

  __bf16* C = static_cast<__bf16*>(a.c) + (OVER_ROWS ? g * a.c_g : 0);
  const int l = __lane_id(), h = l >> 5;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int row = m0 + (wm * TM + m) * 32 + (l & 31);
    __bf16* to = C + row * a.c_m;
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        union {
          __bf16 x[8];
          uint32_t u[4];
          uint4 v;
        } r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.x[e] = (__bf16)acc[n][m][8 * q + e];
        // a lane and the one 32 on hold fours of columns in turn: now eight in a row each
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const auto w = __builtin_amdgcn_permlane32_swap(r.u[e], r.u[2 + e], false, false);
          r.u[e] = w[0];
          r.u[2 + e] = w[1];
        }
        const int col = n0 + (wn * TN + n) * 32 + 16 * q + 8 * h;
        if (row < m_end && col < a.n) *reinterpret_cast<uint4*>(to + col) = r.v;
      }
  }
}

namespace {
int64_t tiles(int64_t n, int64_t each) { return (n + each - 1) / each; }
}  // namespace

// C's rows dense, A's and B's k dense or not.  The caller has checked alignment, sizes and the grid.
hipError_t launch_group_mfma(bool over_rows, const GroupArgs& a, hipStream_t s) {
  if (over_rows) {
    const int64_t blocks = a.groups * tiles(a.m, 128) * tiles(a.n, 256);
    k_group_mfma<false, false, true, 128, 256, 2, 2><<<(unsigned)blocks, 256, 0, s>>>(a);
  } else {
    const int64_t blocks = (tiles(a.rows, 128) + std::min<int64_t>(a.groups + 2, a.rows)) * tiles(a.n, 256);
    if (a.b_k == 1)
      k_group_mfma<true, true, false, 128, 256, 2, 2><<<(unsigned)blocks, 256, 0, s>>>(a);
    else
      k_group_mfma<true, false, false, 128, 256, 2, 2><<<(unsigned)blocks, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace gs
