// gs_group_mfma.hip -- the products of rows with their group's weights on the matrix units, bfloat16, for
// gfx950: y[r] = x[r] W[g(r)] and dx[r] = dy[r] W[g(r)]^T by rows, dW[g] = x^T dy over them (gs_group.hip chooses the blocks).
//
// What bounds it: with many rows the matrix units, at the clock that their power leaves (78126 rows of 16 groups, 2048 x 8192: forward
// 2145 us, dx 2120, dW 2090, 1220 to 1255 TFLOP/s, units busy 74 to 81% of the time); with few, the weights' way from
// memory (64 rows of 16, 2048 x 4096: 38 us, 6.6 TB/s: a part of them stays in the last cache between calls).  In between, smaller blocks' tiles from the L2 cache, and
// their start and end: 7814 rows of 8, 2048 x 4096: 143, 126 and 137 us, 920 to 1040 TFLOP/s (units busy 50 to 62%); blocks of 192 x 256 took as long.
//
// A workgroup of four wavefronts makes BM x BN results, a quarter each, over tiles of 64 k that come from
// memory straight to LDS: two of A, three of B, so that every tile has three quarters of a tile's time or more to
// arrive.  Between two matrix instructions there is at most one read of LDS or one load, so that neither
// queues up before the matrix unit's next work: reads are of the operands of the next 16 k, loads of the tile after the
// next.  One barrier a tile, placed before the tile's last 16 k: by then all of it is in registers, and
// behind it the next tile's first operands are read under its last products.
//
// The results are computed transposed (a lane holds one row's), so that they leave as 16 bytes a lane.
#include <algorithm>
#include <type_traits>

#include "gs_group.h"
#include "gs_lds.h"
#include "gs_mfma.h"

namespace gs {

constexpr int kGroupK = 64;  // k of a tile in LDS
constexpr int kGroupSteps = kGroupK / 16;

__device__ __forceinline__ void group_barrier() { asm volatile("s_barrier" ::: "memory"); }

// One operand's tile of R rows (or columns) by 64 k in LDS, and the loads of its next one.
//   K dense in memory: rows of 64 k; 16-byte chunk c of row r lies at c ^ (2 (r & 2) + r / 4 % 4).
//   K not dense: R elements for each k; chunk c of k-row r lies at c ^ (4 (r % 4) + r / 4 % 4).
// Either way what a wavefront reads at once lies in different banks (gs_mfma.h).
template <bool K_DENSE, int R>
struct GroupSide {
  static constexpr int kBytes = R * kGroupK * 2, kLoads = kBytes / 4096, kChunks = (K_DENSE ? kGroupK : R) / 8;
  static_assert(kLoads * 4096 == kBytes && (K_DENSE || R >= 128), "whole chunks a thread; sixteen of them a row");

  const char* base;     // of the tile at k0
  int64_t step;         // bytes of 64 k
  uint32_t off[kLoads];
  int at;               // where the lane reads, from the start of a tile

  static __device__ __forceinline__ int mix(int r) {
    return K_DENSE ? ((r & 2) << 1) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
  }
  static __device__ __forceinline__ int row_of(int i) { return (i * 256 + (int)threadIdx.x) / kChunks; }
  static __device__ __forceinline__ int chunk_of(int i) { return (i * 256 + (int)threadIdx.x) % kChunks ^ mix(row_of(i)); }

  // Where the wavefront reads: its rows from `first` on.
  __device__ __forceinline__ void place(int first) {
    const int l = __lane_id(), h = l >> 5, i = l & 15;
    if constexpr (K_DENSE) {
      const int r = l & 31;
      at = (first + r) * (kChunks * 16) + ((h ^ mix(r)) << 4);
    } else {
      const int r = 8 * h + (i >> 2), c = first / 8 + (2 * ((l >> 4) & 1) + ((i & 3) >> 1));
      at = r * (kChunks * 16) + ((c ^ mix(r)) << 4) + 8 * (i & 1);
    }
  }
  // p: element (row 0, k0); stride: of the axis that is not dense; rows (at least 1) exist.  Those past them are read as
  // the last: what comes of them is not stored.
  __device__ __forceinline__ void plan(const __bf16* p, int64_t stride, int rows) {
    base = reinterpret_cast<const char*>(p);
    step = K_DENSE ? kGroupK * 2 : kGroupK * 2 * stride;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = row_of(i), c = chunk_of(i) * 8;
      off[i] = K_DENSE ? (uint32_t)(min(r, rows - 1) * stride + c) * 2u : (uint32_t)(r * stride + min(c, rows - 8)) * 2u;
    }
  }
  // The thread's i-th 16 bytes of the tile at p.  Where it is not whole, k < left exist and the others are 0.
  template <bool WHOLE>
  __device__ __forceinline__ void load(const char* p, uint32_t to, int left, int i) const {
    if constexpr (WHOLE) {
      load_to_lds16(p, off[i], to + i * 4096);
    } else {
      const bool there = (K_DENSE ? chunk_of(i) * 8 : row_of(i)) < left;
      load_to_lds16(there ? static_cast<const void*>(p + off[i]) : kZeros, to + i * 4096);
    }
  }
  __device__ __forceinline__ void load_all(int tile, uint32_t to, int left) const {
    const char* p = base + tile * step;
    if (left >= kGroupK) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load<true>(p, to, left, i);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load<false>(p, to, left, i);
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

// Workgroups that a CU's LDS (160 KB) holds at a time, two at most.
constexpr int group_places(int bm, int bn) { return (2 * bm + 3 * bn) * kGroupK * 2 > 80 * 1024 ? 1 : 2; }

// A block of results: rows m0 .. m_end, columns from n0 on, summed over k0 .. k_end.
struct GroupPlace {
  int g, m0, m_end, n0, k0, k_end, split;
};

template <bool A_DENSE, bool B_DENSE, bool OVER_ROWS, bool PARTS, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256, group_places(BM, BN)) void k_group_mfma(GroupArgs a) {
  using SideA = GroupSide<A_DENSE, BM>;
  using SideB = GroupSide<B_DENSE, BN>;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32, kMma = TM * TN, kReads = TM + TN;
  constexpr int kStores = TM * TN * (PARTS ? 4 : 2);
  static_assert(WM * WN == 4, "four wavefronts");
  __shared__ __align__(1024) char lds[2 * SideA::kBytes + 3 * SideB::kBytes];
  const int n_tiles = (a.n + BN - 1) / BN, columns = PARTS ? n_tiles * a.splits : n_tiles;  // a part's blocks beside the next one's

  // the blocks, an eighth to each XCD (whose workgroups are every eighth), there in patches of a few tiles of rows
  GroupTiles<BM> spans;
  uint32_t m_tiles, id, end;
  if constexpr (OVER_ROWS) {
    m_tiles = (a.m + BM - 1) / BM;
    id = blockIdx.x;
    end = a.groups * m_tiles * columns;
  } else {
    m_tiles = min(spans.count(a), (uint32_t)((a.rows + BM - 1) / BM + min(a.groups + 2, a.rows)));  // (less than it counts: offsets that decrease)
    const uint32_t all = m_tiles * columns, q = all / 8, more = all % 8, xcd = blockIdx.x % 8;
    id = xcd * q + min(xcd, more);
    end = id + q + (xcd < more);
    id += blockIdx.x / 8;
  }
  auto find = [&](uint32_t i) {
    GroupPlace p;
    if constexpr (OVER_ROWS) {  // group by group: an eighth of its blocks to each XCD
      const uint32_t each = m_tiles * columns, rank = i / each, in = i - rank * each, q = each / 8, more = each % 8, slot = in % 8;
      p.g = group_by_length(a, rank);
      i = slot * q + min(slot, more) + in / 8;
    }
    constexpr uint32_t kHigh = BM >= 128 ? 2048 / BM : 16;
    const uint32_t patch = i / (kHigh * columns), rest = i - patch * kHigh * columns, high = min(kHigh, m_tiles - patch * kHigh);
    const uint32_t mt = patch * kHigh + rest % high, column = rest / high;
    p.split = PARTS ? column / n_tiles : 0;
    p.n0 = (PARTS ? column - p.split * n_tiles : column) * BN;
    if constexpr (OVER_ROWS) {
      p.m0 = mt * BM;
      p.m_end = a.m;
      p.k0 = group_bound(a, p.g + 1);
      p.k_end = max(group_bound(a, p.g + 2), p.k0);
    } else {
      const GroupSpan s = spans.find(a, mt);
      p.g = s.group;
      p.m0 = s.first;
      p.m_end = s.last;
      p.k0 = 0;
      p.k_end = s.group < 0 ? 0 : a.k;
    }
    if constexpr (PARTS) group_part(a, p.split, kGroupK, &p.k0, &p.k_end);
    return p;
  };
  if (id >= end) return;
  GroupPlace p = find(id);

  const int wave = threadIdx.x / kWave, wm = wave % WM, wn = wave / WM;
  const uint32_t to = lds_address(lds) + (threadIdx.x / kWave) * 1024;
  auto to_a = [&](int b) { return (uint32_t)__builtin_amdgcn_readfirstlane(to + b * SideA::kBytes); };
  auto to_b = [&](int b) { return (uint32_t)__builtin_amdgcn_readfirstlane(to + 2 * SideA::kBytes + b * SideB::kBytes); };
  SideA sa;
  SideB sb;
  sa.place(wm * TM * 32);
  sb.place(wn * TN * 32);
  // the first two tiles' loads
  auto start = [&] {
    const int left = p.k_end - p.k0;
    if (left == 0) return;
    sa.plan(static_cast<const __bf16*>(a.a) + p.m0 * a.a_m + p.k0 * a.a_k, A_DENSE ? a.a_m : a.a_k, p.m_end - p.m0);
    sb.plan(static_cast<const __bf16*>(a.b) + (OVER_ROWS ? 0 : p.g * a.b_g) + p.k0 * a.b_k + p.n0 * a.b_n, B_DENSE ? a.b_n : a.b_k, a.n - p.n0);
    sa.load_all(0, to_a(0), left);
    sb.load_all(0, to_b(0), left);
    sb.load_all(1, to_b(1), left - kGroupK);  // of k that do not exist: zeros, so that the loads can be counted
    sa.load_all(1, to_a(1), left - kGroupK);
  };

  start();
  bool stored = false;  // stores of the block before are on their way behind the loads
  while (true) {
    f32x16 acc[TN][TM];
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int m = 0; m < TM; ++m) acc[n][m] = (f32x16)0.0f;
    bf16x8 fa[2][TM], fb[2][TN];
    auto read = [&](int which, int ba, int bb, int s, int i) {
      if (i < TN)
        fb[which][i] = sb.read(lds + 2 * SideA::kBytes + bb * SideB::kBytes, i, s);
      else
        fa[which][i - TN] = sa.read(lds + ba * SideA::kBytes, i - TN, s);
    };
    // 16 k, and what goes between the products: part i of kMma
    auto multiply = [&](int which, auto&& between) {
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[which][n], fa[which][m], acc[n][m], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          between(m * TN + n);
          __builtin_amdgcn_sched_barrier(0);
        }
    };

    // the sums stay where the matrix unit adds to them, past the branches too
    auto keep = [&] {
      if constexpr (kMma == 16) {
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int m = 0; m < TM; ++m) asm volatile("" : "+a"(acc[n][m]));
      }
    };
    keep();

    const int all = p.k_end - p.k0;
    if (all) {
      // loads and stores are counted together and in order
      if (stored)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kStores + SideA::kLoads + SideB::kLoads < 63 ? kStores + SideA::kLoads + SideB::kLoads : 63) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(SideA::kLoads + SideB::kLoads) : "memory");
      group_barrier();
#pragma unroll
      for (int i = 0; i < kReads; ++i) read(0, 0, 0, 0, i);
      int ba = 0, bb = 0;
      const char *pa = sa.base + 2 * sa.step, *pb = sb.base + 2 * sb.step;  // of tile t + 2
      auto tile = [&](auto whole, int left) {  // left: k of tile t + 2 and behind
        constexpr bool kWhole = decltype(whole)::value;
        const int next_a = ba ^ 1, next_b = bb == 2 ? 0 : bb + 1;
        const uint32_t ta = to_a(ba), tb = to_b(bb == 0 ? 2 : bb - 1);
#pragma unroll
        for (int s = 0; s + 1 < kGroupSteps; ++s)
          multiply(s & 1, [&](int i) {
#pragma unroll
            for (int r = 0; r < kReads; ++r)
              if (r * kMma / kReads == i) read((s + 1) & 1, ba, bb, s + 1, r);
#pragma unroll
            for (int r = 0; r < SideB::kLoads; ++r)
              if (s == 0 && (2 * r + 1) * kMma / (2 * SideB::kLoads) == i) sb.template load<kWhole>(pb, tb, left, r);
          });
        asm volatile("s_waitcnt lgkmcnt(0) vmcnt(%0)" ::"n"(SideB::kLoads) : "memory");
        group_barrier();
        multiply((kGroupSteps - 1) & 1, [&](int i) {
#pragma unroll
          for (int r = 0; r < kReads; ++r)
            if (r * kMma / kReads == i) read(0, next_a, next_b, 0, r);
#pragma unroll
          for (int r = 0; r < SideA::kLoads; ++r)
            if ((2 * r + 1) * kMma / (2 * SideA::kLoads) == i) sa.template load<kWhole>(pa, ta, left, r);
        });
        pa += sa.step;
        pb += sb.step;
        ba = next_a;
        bb = next_b;
      };
      int left = all - 2 * kGroupK;
      for (; left >= kGroupK; left -= kGroupK) tile(std::true_type(), left);
      keep();
      for (; left > -2 * kGroupK; left -= kGroupK) tile(std::false_type(), left);
      keep();
      // no wavefront reads LDS any more that counts, and this one's last loads (zeros) are in
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    keep();
    const GroupPlace done = p;
    id += OVER_ROWS ? gridDim.x : gridDim.x / 8;
    const bool more = id < end;
    if (more) {
      p = find(id);
      start();
    }
    keep();

    const int width = group_part_width(a.n);
    const int64_t c_m = PARTS ? width : a.c_m;
    char* C = PARTS ? reinterpret_cast<char*>(a.part + ((done.split * (OVER_ROWS ? a.groups : 1) + (OVER_ROWS ? done.g : 0)) * (int64_t)a.m + done.m0) * width + done.n0)
                    : reinterpret_cast<char*>(static_cast<__bf16*>(a.c) + (OVER_ROWS ? done.g * a.c_g : 0) + done.m0 * c_m + done.n0);
    constexpr int kSize = PARTS ? 4 : 2;
    const auto out = __builtin_amdgcn_make_buffer_rsrc(C, 0, 0x7fffffff, 0x00020000);
    const int l = __lane_id(), h = l >> 5;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const int row = (wm * TM + m) * 32 + (l & 31);
      const uint32_t row_at = row < done.m_end - done.m0 ? (uint32_t)(row * c_m) * kSize : 0x80000000u;
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
          union {
            __bf16 x[8];
            uint32_t u[8];
            u32x4 v[2];
          } r;
          constexpr int kWords = PARTS ? 4 : 2;
          if constexpr (PARTS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.u[e] = __float_as_uint(acc[n][m][8 * q + e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.x[e] = (__bf16)acc[n][m][8 * q + e];
          }
          // a lane and the one 32 on hold fours of columns in turn: now eight in a row each
#pragma unroll
          for (int e = 0; e < kWords; ++e) {
            const auto w = __builtin_amdgcn_permlane32_swap(r.u[e], r.u[kWords + e], false, false);
            r.u[e] = w[0];
            r.u[kWords + e] = w[1];
          }
          const int col = (wn * TN + n) * 32 + 16 * q + 8 * h;
          // past the last row or column: past the buffer's end, where nothing is written.  So every store is made, and counted.
          const uint32_t to_at = done.n0 + col < a.n ? row_at + col * kSize : 0x80000000u;
          __builtin_amdgcn_raw_buffer_store_b128(r.v[0], out, to_at, 0, 0);
          if constexpr (PARTS) __builtin_amdgcn_raw_buffer_store_b128(r.v[1], out, to_at + 16, 0, 0);
          __builtin_amdgcn_sched_barrier(0);  // a few registers at a time
        }
    }
    if (!more) return;
    stored = true;
  }
}

namespace {

template <bool PARTS, int BM, int BN, int WM, int WN>
void group_launch(bool over_rows, const GroupArgs& a, hipStream_t s) {
  constexpr int64_t kSlots = 256 * group_places(BM, BN);  // workgroups at a time
  const int64_t columns = tiles(a.n, BN) * a.splits;
  if (over_rows) {
    // Short sums go from block to block as well; long ones, of different lengths, are left to whichever place is free.  us, left and from block
    // to block, groups of one length and of lengths between 0 and 4 times that: 16 groups, 2048 x 4096, of 4 rows: 93.5, 81.0 and 86.8, 75.4; 128:
    // 113, 107 and 114, 104; 256: 136, 130 and 134, 132; 384: 162, 158 and 158, 157; 1024: 266, 275 and 271, 282.  40 groups, 1024 x 1024, of 64:
    // 38.1, 36.0 and 35.8, 35.4; 128: 43.3, 41.1 and 38.4, 40.8; 256: 50.7, 49.5 and 44.7, 51.0; 1024: 101, 104 and 89, 117.  64 groups, 512 x 2048, of
    // 128: 62.1, 61.3 and 59.1, 56.7; 256: 76.8, 69.7 and 71.0, 70.3; 512: 107, 104 and 102, 115.
    const int64_t all = a.groups * tiles(a.m, BM) * columns;
    const unsigned blocks = (unsigned)(a.rows / a.groups < 256 ? std::min(kSlots, all) : all);
    if constexpr (BM >= 128) k_group_mfma<false, false, true, PARTS, BM, BN, WM, WN><<<blocks, 256, 0, s>>>(a);
    return;
  }
  const int64_t most = (tiles(a.rows, BM) + std::min<int64_t>(a.groups + 2, a.rows)) * columns;
  const unsigned blocks = (unsigned)std::min(kSlots, tiles(most, 8) * 8);
  if (a.b_k == 1)
    k_group_mfma<true, true, false, PARTS, BM, BN, WM, WN><<<blocks, 256, 0, s>>>(a);
  else
    k_group_mfma<true, false, false, PARTS, BM, BN, WM, WN><<<blocks, 256, 0, s>>>(a);
}
template <int BM, int BN, int WM, int WN>
void group_launch(bool over_rows, const GroupArgs& a, hipStream_t s) {
  if (a.splits > 1)
    group_launch<true, BM, BN, WM, WN>(over_rows, a, s);
  else
    group_launch<false, BM, BN, WM, WN>(over_rows, a, s);
}

}  // namespace

// C's rows dense, A's and B's k dense or not.  The caller has checked alignment, sizes and the grid.
hipError_t launch_group_mfma(bool over_rows, int tile, const GroupArgs& a, hipStream_t s) {
  switch (tile) {
    case kGroup256x256: group_launch<256, 256, 2, 2>(over_rows, a, s); break;
    case kGroup128x256: group_launch<128, 256, 2, 2>(over_rows, a, s); break;
    case kGroup128x128: group_launch<128, 128, 2, 2>(over_rows, a, s); break;
    case kGroup32x256: group_launch<32, 256, 1, 4>(over_rows, a, s); break;
    default: group_launch<32, 128, 1, 4>(over_rows, a, s); break;
  }
  return hipGetLastError();
}

}  // namespace gs
