// gs_group.hip -- products of rows with their group's weights (experts, or heads of a kind), and their
// gradients, for gfx950: float32, and bfloat16 matrices whose rows do not all start on 16 bytes
// (gs_group_mfma.hip has the others).
//
//   y[r] = x[r] W[g(r)],  dx[r] = dy[r] W[g(r)]^T,  dW[g] = sum over the group's rows of x[r]^T dy[r].
//
// A workgroup of eight wavefronts makes 128 x 128 results (or 128 x 64) over tiles of 32 k, in two halves of LDS.  Tiles pass through
// registers, loaded two ahead at any alignment, and enter LDS in the matrix unit's terms: float32 as three bfloat16 that hold
// all of its bits, split once for the workgroup while the tile before is multiplied (gs_mfma.h).  A sum's last tile ends with
// the last k: its eights are loaded whole, and what the ones before had is cut (1955 rows of 5 groups, 363 x 250 in bfloat16, the three
// products: 31.9 us with element loads for what 64 does not divide, 27.8 so).
//
// float32 is bound by the matrix units at the power they get: 7814 rows of 8, 2048 x 4096: 800 us, 164 TFLOP/s, 980 TFLOP/s of
// bfloat16 products.  bfloat16: 18583 rows of 10, 4797 x 777, 352, 380 and 270 us, 365 to 515 TFLOP/s, by loads that start off 16 bytes
// (this kernel is 10 to 30% faster on rows on 16 bytes, the other takes 214, 199 and 194 us for 4800 x 776) and their way through registers; blocks of 256 x 128
// were no faster.
//
// Where a sum is long and the results are few, several workgroups share it: their parts go to a workspace in
// float32, and a second kernel adds them in a fixed order.
#include <algorithm>
#include <cmath>

#include "gs_group.h"
#include "gs_mfma.h"

namespace gs {

hipError_t launch_group_mfma(bool over_rows, int tile, const GroupArgs& a, hipStream_t s);

constexpr int kStagedTile = 128, kStagedK = 32, kStagedThreads = 512;
constexpr int kStagedAhead = 2;  // tiles on their way

// x as a sum of three bfloat16, two elements at a time: 88 operations for a thread's sixteen where frag_split, which keeps an infinity apart
// (here it makes NaNs), takes 156; splitting, not the products, is what a tile waits for.
__device__ __forceinline__ Frag<float> group_split(f32x8 x) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  union {
    Frag<float> f;
    uint32_t u[3][4];
  } r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f32x2 y = {x[2 * j], x[2 * j + 1]};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      r.u[k][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
      y[0] -= __uint_as_float(r.u[k][j] << 16);
      y[1] -= __uint_as_float(r.u[k][j] & 0xffff0000u);
    }
  }
  return r.f;
}

// Eight elements of memory on their way to LDS: all of them, at any alignment, or the first n and zeros behind.
template <typename T>
struct Eight;
template <>
struct Eight<__bf16> {
  bf16x8 v;
  __device__ __forceinline__ void load(const __bf16* p) {
    typedef __bf16 V __attribute__((ext_vector_type(8), aligned(2)));
    v = *reinterpret_cast<const V*>(p);
  }
  __device__ __forceinline__ void load(const __bf16* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : (__bf16)0.0f;
  }
  __device__ __forceinline__ Frag<__bf16> parts() const { return {v}; }
};
template <>
struct Eight<float> {
  f32x8 v;
  __device__ __forceinline__ void load(const float* p) {
    typedef float V __attribute__((ext_vector_type(4), aligned(4)));
    const V a = *reinterpret_cast<const V*>(p), b = *reinterpret_cast<const V*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
  __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
  __device__ __forceinline__ Frag<float> parts() const { return group_split(v); }
};

// Where eight rows (or columns) are that the tile counts from `at` on (a multiple of 8), of `rows`: the last eight in the place of a few.
template <bool NARROW>
__device__ __forceinline__ int eight_at(int at, int rows) {
  return NARROW ? at : min(at, rows - 8);
}

// One operand's tile of 128 rows (or columns) by 32 k, in LDS as gs_group_mfma.hip's but for rows of 64 bytes where k is
// dense (chunk c of row r at c ^ (r / 4 % 4)); float32's three parts one after another.
template <typename T, bool K_DENSE, bool OVER_ROWS, bool NARROW, int R>
struct StagedSide {
  static constexpr int kChunks = (K_DENSE ? kStagedK : R) / 8, kPart = R * kStagedK * 2;
  static_assert(R == 64 || R == 128, "an eight a thread, of the first threads where there are fewer");
  static constexpr int kParts = sizeof(Frag<T>) / sizeof(bf16x8), kBytes = kParts * kPart;

  const T* base;    // of the tile at k0
  int64_t step;     // elements of 32 k
  int64_t stride;   // of the axis that is not dense
  int64_t off, off_last;
  int cut;          // of the last tile's eight: the first elements, which do not count
  int rows;
  int at;
  Eight<T> x[kStagedAhead];  // tiles on their way

  static __device__ __forceinline__ int mix(int r) {
    if (K_DENSE) return (r >> 2) & 3;
    return R == 64 ? ((r & 2) << 1) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
  }
  static __device__ __forceinline__ int item() { return (int)threadIdx.x % (R * kStagedK / 8); }
  static __device__ __forceinline__ int row() { return item() / kChunks; }
  static __device__ __forceinline__ int chunk() { return item() % kChunks; }

  // The last tile, of which k < left exist (of 1 to 32): its eights end with the last k, and count from where the one before ended.
  __device__ __forceinline__ void plan(const T* p, int64_t s, int n, int left, int first) {
    base = p;
    stride = s;
    rows = n;
    step = K_DENSE ? kStagedK : kStagedK * s;
    const int r = row(), c = chunk() * 8;
    if constexpr (K_DENSE) {
      const int k = min(c, left - 8);
      off = min(r, rows - 1) * stride;
      off_last = off + k;
      off += c;
      cut = c - k;
    } else {  // rows of k: a sum over rows may have fewer than eight
      const int r8 = r & ~7, k = OVER_ROWS ? min(r, left - 1) : min(r8, left - 8) + r - r8, col = eight_at<NARROW>(c, rows);
      off = r * stride + col;
      off_last = k * stride + col;
      cut = k < (OVER_ROWS ? r : r8) ? 8 : 0;
    }
    const int l = __lane_id(), h = l >> 5, i = l & 15;
    if constexpr (K_DENSE) {
      at = (first + (l & 31)) * (kChunks * 16) + ((h ^ mix(l & 31)) << 4);
    } else {
      const int from = 8 * h + (i >> 2), chunk_at = first / 8 + (2 * ((l >> 4) & 1) + ((i & 3) >> 1));
      at = from * (kChunks * 16) + ((chunk_at ^ mix(from)) << 4) + 8 * (i & 1);
    }
  }
  // A tile.  Rows (or columns) that do not exist are read as others: what comes of them is not stored.
  __device__ __forceinline__ void load(int to, int tile, bool last) {
    x[to].load(base + tile * step + (last ? off_last : off));
  }
  __device__ __forceinline__ void cut_last(int from) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[from].v[e] = e < cut ? (T)0.0f : x[from].v[e];
  }
  // NARROW: any tile, of which k < left exist; the others are 0.
  __device__ __forceinline__ void load_part(int to, int tile, int left) {
    const int c = chunk() * 8;
    x[to].load(base + tile * step + off, K_DENSE ? left - c : row() >= left ? 0 : rows - c);
  }
  __device__ __forceinline__ void store(int from, char* tile) const {
    if (R * kStagedK / 8 < kStagedThreads && threadIdx.x >= R * kStagedK / 8) return;  // (whole wavefronts)
    const int r = row(), c = chunk();
    union {
      Frag<T> f;
      bf16x8 v[kParts];
    } u;
    u.f = x[from].parts();
#pragma unroll
    for (int k = 0; k < kParts; ++k) *reinterpret_cast<bf16x8*>(tile + k * kPart + r * (kChunks * 16) + ((c ^ mix(r)) << 4)) = u.v[k];
  }
  __device__ __forceinline__ Frag<T> read(const char* tile, int m, int s) const {
    union {
      Frag<T> f;
      bf16x8 v[kParts];
    } u;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const char* p = tile + k * kPart;
      if constexpr (K_DENSE) {
        u.v[k] = *reinterpret_cast<const bf16x8*>(p + (at ^ (s << 5)) + m * 32 * (kChunks * 16));
      } else {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
        const int o = at ^ (m << 6);
        union {
          s16x4 q[2];
          bf16x8 v;
        } w;
        p += 16 * s * (kChunks * 16);
        w.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + o));
        w.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * (kChunks * 16) + (o ^ 16)));
        u.v[k] = w.v;
      }
    }
    return u.f;
  }
};

// The running sums of a block.  float32: the products of the leading parts apart from the five smaller ones, whose sum is
// 2^-8 of theirs, so that a sum over k is rounded once for 16 k and not six times (over 3648 k, against 64 bits: 9e-7 -> 3.7e-7 of the
// result's norm).
template <typename T>
struct Sums;
template <>
struct Sums<__bf16> {
  f32x16 c = (f32x16)0.0f;
  __device__ __forceinline__ void add(const Frag<__bf16>& a, const Frag<__bf16>& b) { c = mma(a, b, c); }
  __device__ __forceinline__ float get(int i) const { return c[i]; }
};
template <>
struct Sums<float> {
  f32x16 c = (f32x16)0.0f, rest = (f32x16)0.0f;
  __device__ __forceinline__ void add(const Frag<float>& a, const Frag<float>& b) {
    rest = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2], b.p[0], rest, 0, 0, 0);
    rest = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[2], rest, 0, 0, 0);
    rest = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], rest, 0, 0, 0);
    rest = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[0], rest, 0, 0, 0);
    rest = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[1], rest, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int i) const { return c[i] + rest[i]; }
};

// The place in a row of `all` that a workgroup takes, which is the `i`-th to start: an eighth of the row to each XCD, whose workgroups are
// every eighth.
__device__ __forceinline__ uint32_t group_dealt(uint32_t i, uint32_t all) {
  const uint32_t q = all / 8, more = all % 8, xcd = i % 8;
  return xcd * q + min(xcd, more) + i / 8;
}

// NARROW: a matrix with rows of fewer than eight elements.
template <typename T, bool A_DENSE, bool B_DENSE, bool OVER_ROWS, bool NARROW, int BN>
__global__ __launch_bounds__(kStagedThreads, BN == 64 ? 4 : 2) void k_group_staged(GroupArgs a) {
  constexpr int TM = 1, TN = BN / 64;  // a wavefront's 32 x 64 (or 32) of the block
  using SideA = StagedSide<T, A_DENSE, OVER_ROWS, NARROW, kStagedTile>;
  using SideB = StagedSide<T, B_DENSE, OVER_ROWS, NARROW, BN>;
  constexpr int kTile = SideA::kBytes + SideB::kBytes;
  __shared__ __align__(1024) char lds[2 * kTile];
  const int n_tiles = (a.n + BN - 1) / BN;
  int m0, n0, m_end, k0, k_end, g, split;
  if constexpr (OVER_ROWS) {
    const uint32_t m_tiles = (a.m + kStagedTile - 1) / kStagedTile, each = m_tiles * n_tiles * a.splits;
    const uint32_t rank = blockIdx.x / each, in = blockIdx.x - rank * each;
    g = group_by_length(a, rank);
    const uint32_t i = group_dealt(in, each), rest = i % (m_tiles * n_tiles);
    split = i / (m_tiles * n_tiles);
    m0 = rest / n_tiles * kStagedTile;
    n0 = rest % n_tiles * BN;
    m_end = a.m;
    k0 = group_bound(a, g + 1);
    k_end = max(group_bound(a, g + 2), k0);
  } else {
    GroupTiles<kStagedTile> spans;
    const uint32_t columns = n_tiles * a.splits;
    uint32_t m_tiles = 0;
    spans.look(a, 0);
    if (a.groups + 2 <= kWave) {  // (else counting them would take as long again as finding one)
      m_tiles = min(spans.last(), (uint32_t)((a.rows + kStagedTile - 1) / kStagedTile + min(a.groups + 2, a.rows)));
      if (blockIdx.x >= m_tiles * columns) return;
    }
    // many blocks of rows: an eighth of them to each XCD, there in patches of sixteen by some columns, so that its cache holds what they share
    // (bfloat16, 5101 rows of 18, 2625 x 513: 52 -> 39 us; 4001 rows of 2, 4097 x 1025: 130 -> 109); few (float32, 800 rows of 4, 512 x 1024,
    // back: 20.0, so 22.6): one after another
    uint32_t mt = blockIdx.x / columns, column = blockIdx.x - mt * columns;
    constexpr uint32_t kHigh = 16;
    if (m_tiles > kHigh) {
      const uint32_t i = group_dealt(blockIdx.x, m_tiles * columns);
      const uint32_t patch = i / (kHigh * columns), rest = i - patch * kHigh * columns, high = min(kHigh, m_tiles - patch * kHigh);
      mt = patch * kHigh + rest % high;
      column = rest / high;
    }
    const GroupSpan s = spans.find(a, mt);
    if (s.first >= s.last) return;
    g = s.group;
    m0 = s.first;
    m_end = s.last;
    split = column / n_tiles;
    n0 = (column - split * n_tiles) * BN;
    k0 = 0;
    k_end = g < 0 ? 0 : a.k;
  }
  group_part(a, split, kStagedK, &k0, &k_end);
  const int wave = threadIdx.x / kWave, wm = wave % 4, wn = wave / 4;

  Sums<T> acc[TN][TM];
  if (k0 < k_end) {
    SideA sa;
    SideB sb;
    const int all = k_end - k0, tiles = (all + kStagedK - 1) / kStagedK, left = all - (tiles - 1) * kStagedK;
    sa.plan(static_cast<const T*>(a.a) + m0 * a.a_m + k0 * a.a_k, A_DENSE ? a.a_m : a.a_k, m_end - m0, left, wm * TM * 32);
    sb.plan(static_cast<const T*>(a.b) + (OVER_ROWS ? 0 : g * a.b_g) + k0 * a.b_k + n0 * a.b_n, B_DENSE ? a.b_n : a.b_k, a.n - n0, left, wn * TN * 32);
    auto load = [&](int to, int t) {  // past the last: that one again, for nothing
      t = min(t, tiles - 1);
      sa.load(to, t, t == tiles - 1);
      sb.load(to, t, t == tiles - 1);
    };
    auto store = [&](int from, int buffer, int t) {
      if (t == tiles - 1 && left < kStagedK) {
        sa.cut_last(from);
        sb.cut_last(from);
      }
      sa.store(from, lds + buffer * kTile);
      sb.store(from, lds + buffer * kTile + SideA::kBytes);
    };
    auto multiply = [&](int buffer) {
      const char* tile = lds + buffer * kTile;
#pragma unroll
      for (int s = 0; s < kStagedK / 16; ++s) {
        Frag<T> fa[TM], fb[TN];
#pragma unroll
        for (int n = 0; n < TN; ++n) fb[n] = sb.read(tile + SideA::kBytes, n, s);
#pragma unroll
        for (int m = 0; m < TM; ++m) fa[m] = sa.read(tile, m, s);
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int n = 0; n < TN; ++n) acc[n][m].add(fb[n], fa[m]);
      }
    };
    if constexpr (NARROW) {
      for (int t = 0; t < tiles; ++t) {
        sa.load_part(0, t, all - t * kStagedK);
        sb.load_part(0, t, all - t * kStagedK);
        store(0, 0, -1);
        __syncthreads();
        multiply(0);
        __syncthreads();
      }
    } else {
      // while a tile is multiplied, the next goes to the other half of LDS and the two behind it are on their way, with no branch
      // between a load and its use
      load(0, 0);
      if (tiles > 1) {
        load(1, 1);
        store(0, 0, 0);
        load(0, 2);
        __syncthreads();
        for (int t = 0; t + 1 < tiles; t += 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            store(i ^ 1, i ^ 1, t + i + 1);
            load(i ^ 1, t + i + 3);
            multiply(i);
            __syncthreads();
          }
        }
      } else {
        store(0, 0, 0);
        __syncthreads();
      }
      if (tiles & 1) multiply(0);
    }
  }

  T* C = static_cast<T*>(a.c) + (OVER_ROWS ? g * a.c_g : 0);
  const int width = group_part_width(a.n);
  float* part = a.part + ((int64_t)split * (OVER_ROWS ? (int64_t)a.groups * a.m : a.rows) + (OVER_ROWS ? (int64_t)g * a.m : 0)) * width;
  const int l = __lane_id(), h = l >> 5;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    int row = m0 + (wm * TM + m) * 32 + (l & 31);
    const bool there = A_DENSE || NARROW ? row < m_end : (row & ~7) < m_end;
    if constexpr (!A_DENSE) row = eight_at<NARROW>(row & ~7, m_end) + (row & 7);
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        // a lane and the one 32 on hold fours of columns in turn: now eight in a row each
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[n][m].get(8 * q + e)), __float_as_uint(acc[n][m].get(8 * q + 4 + e)), false, false);
          x[e] = __uint_as_float(w[0]);
          x[4 + e] = __uint_as_float(w[1]);
        }
        int col = n0 + (wn * TN + n) * 32 + 16 * q + 8 * h;
        if (!there || col >= a.n) continue;
        if constexpr (!B_DENSE) col = eight_at<NARROW>(col, a.n);
        const int some = min(a.n - col, 8);
        if (a.splits > 1)
          store_units(part + (int64_t)row * width + col, some, x);
        else
          store_units(C + row * a.c_m + col, some, x);
      }
  }
}

// C from the parts, in a fixed order: eight results a thread, which adds every LANES-th part where there are many, and then the threads'
// sums in turn.
template <typename T, int LANES>
__global__ __launch_bounds__(256) void k_group_join(GroupArgs a, int64_t rows, int outer_rows, int64_t outer_stride) {
  constexpr int kResults = 256 / LANES;
  const int width = group_part_width(a.n), chunks = width / 8;
  const int at = threadIdx.x % kResults, lane = threadIdx.x / kResults;
  const int64_t i = (int64_t)blockIdx.x * kResults + at, row = i / chunks;
  const int col = (int)(i - row * chunks) * 8;
  float x[8] = {};
  if (row < rows) {
    const float* p = a.part + row * width + col;
#pragma unroll 4
    for (int s = lane; s < a.splits; s += LANES) {
      float y[8];
      load_elems<8>(p + s * rows * width, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += y[e];
    }
  }
  if constexpr (LANES > 1) {
    __shared__ float sums[LANES][kResults][8 + 1];
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[lane][at][e] = x[e];
    __syncthreads();
    if (lane > 0) return;
    for (int l = 1; l < LANES; ++l)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += sums[l][at][e];
  }
  if (row >= rows) return;
  const int64_t outer = row / outer_rows, in = row - outer * outer_rows;
  store_units(static_cast<T*>(a.c) + outer * outer_stride + in * a.c_m + col, min(a.n - col, 8), x);
}

namespace {

// Whether every row of the three matrices starts on 16 bytes and holds whole chunks of 16, at distances that
// a thread's 32-bit offsets reach.
bool group_aligned(bool over_rows, const GroupArgs& a) {
  constexpr int64_t kFar = 1 << 22;
  const int64_t as = over_rows || a.a_k != 1 ? a.a_k : a.a_m, bs = a.b_n == 1 ? a.b_k : a.b_n;
  for (const void* p : {a.a, a.b, static_cast<const void*>(a.c)})
    if ((uintptr_t)p % 16) return false;
  return as % 8 == 0 && bs % 8 == 0 && a.b_g % 8 == 0 && a.c_g % 8 == 0 && a.c_m % 8 == 0 && as <= kFar && bs <= kFar && a.c_m <= kFar &&
         a.n % 8 == 0 && (over_rows ? a.m : a.k) % 8 == 0;
}

template <typename T, bool NARROW, int BN>
void staged_launch(bool over_rows, const GroupArgs& a, hipStream_t s) {
  const int64_t m_tiles = over_rows ? a.groups * tiles(a.m, kStagedTile) : tiles(a.rows, kStagedTile) + std::min(a.groups + 2, a.rows);
  const unsigned blocks = (unsigned)(m_tiles * tiles(a.n, BN) * a.splits);
  if (over_rows)
    k_group_staged<T, false, false, true, NARROW, BN><<<blocks, kStagedThreads, 0, s>>>(a);
  else if (a.b_k == 1)
    k_group_staged<T, true, true, false, NARROW, BN><<<blocks, kStagedThreads, 0, s>>>(a);
  else
    k_group_staged<T, true, false, false, NARROW, BN><<<blocks, kStagedThreads, 0, s>>>(a);
}
template <typename T>
void staged_launch(bool over_rows, int tile, const GroupArgs& a, hipStream_t s) {
  if (a.n < 8 || (over_rows ? a.m : a.k) < 8)
    staged_launch<T, true, 128>(over_rows, a, s);
  else if (tile == kGroupStaged64)
    staged_launch<T, false, 64>(over_rows, a, s);
  else
    staged_launch<T, false, 128>(over_rows, a, s);
}

}  // namespace

// Workgroups of a launch at most, before the sums are split (which they are up to 2048 only), each of up to 512 threads: the
// caller checks that a grid takes them.
int64_t group_tiles(bool over_rows, int64_t rows, int64_t m, int64_t n, int64_t groups) {
  return over_rows ? groups * tiles(m, kStagedTile) * tiles(n, 64) : (tiles(rows, kStagedTile) + std::min(groups + 2, rows)) * tiles(n, 64);
}

namespace {

struct GroupPlan {
  int tile, splits;
};

// The block of results and the parts of the sums with the least time by a model: rounds of workgroups on the CUs' places, each a
// start and an end and a time for 64 k, and the join of the parts.  Workgroups that go from block to block end in whole rounds; the
// staged ones fill in for each other, and have their CU to themselves where they are few.  Rows of a group are not known here: the
// last block of rows of each is taken as half full.
//
// Measured, us (by rows; 256 x 256, 128 x 256, 128 x 128, 32 x 256, 32 x 128): 7814 rows of 8 groups, 2048 x 4096: 149 139 154 298
// 295; 782 rows 46 37 40 48 50; 64 rows of 16 groups 52 49 47 43 47; 3907 rows of one, 2048 x 2048: 45 35 36 66 66; 20000 rows of 8, 512 x 256:
// 18 13 15 19 17; 64 rows of 4, 4096 x 512, in the best number of parts: 19 17 14 14 13, in one 32 x 128: 33.  Over rows (the first
// three): 7814 rows of 8, 2048 x 4096: 143 169 163; 20000 rows of 8, 512 x 256: 32 26 22 in 8, 8 and 4 parts, 66 in one; 40000
// rows of one, 1024 x 512: 63 57 65 in 32, 16 and 16 parts.  Many parts: 200000 rows of one, 256 x 256: 74 in 32, 50 in 64, 46 in 128;
// float32, 30039 rows of one, 40 x 96: 39 in 32, 26 in 64, 19.5 in 128.
// Staged (128 x 128, 128 x 64): float32, 4000 rows of 2, 4096 x 1024: 221 244; 800 rows of 4, 512 x 1024: 22 17; 43816 rows of one, 40 x 528,
// back: 50 31; 158 rows of 37, 3496 x 165: 78 49; 51701 rows of 13, 82 x 82, by rows 19 23, over rows 32 28;
// bfloat16, 1955 rows of 5, 363 x 250: 9.5 9.0; 20000 rows of 8, 513 x 257: 25 39.
struct GroupShape {
  int bm, bn, places;
  double fix, by_rows, over;  // us: a block, and 64 k
  int few;                    // workgroups up to which they take `alone` of that
  double alone;
};

GroupPlan group_plan(bool over_rows, bool staged, bool f32, int64_t rows, int64_t m, int64_t n, int64_t k, int64_t groups) {
  static const GroupShape kShapes[kGroupTiles] = {
      {256, 256, 256, 6.0, 1.5, 1.6, 0, 1.0}, {128, 256, 256, 3.0, 1.0, 1.15, 0, 1.0}, {128, 128, 512, 3.0, 1.15, 1.2, 0, 1.0},
      {32, 256, 256, 2.0, 0.5, 0.0, 0, 1.0},  {32, 128, 512, 2.0, 0.5, 0.0, 0, 1.0},   {128, 128, 512, 4.0, 1.3, 1.3, 256, 0.7},
      {128, 64, 1024, 4.0, 1.6, 1.6, 256, 0.45}};
  static const GroupShape kFloat[2] = {{128, 128, 256, 6.0, 3.2, 3.2, 0, 1.0}, {128, 64, 512, 4.0, 3.8, 3.8, 256, 0.6}};
  const double used = (double)std::min(groups, over_rows ? groups : rows);
  const double length = over_rows ? (double)rows / (double)std::max<int64_t>(groups, 1) : (double)k;
  GroupPlan best{staged ? kGroupStaged128 : kGroup128x128, 1};
  double least = 1e300;
  for (int t = 0; t < kGroupTiles; ++t) {
    const GroupShape& x = f32 && t >= kGroupStaged128 ? kFloat[t - kGroupStaged128] : kShapes[t];
    if ((t >= kGroupStaged128) != staged || (over_rows && x.bm < 128)) continue;
    const double m_tiles = over_rows ? (double)(groups * tiles(m, x.bm)) : std::max(used, (double)rows / x.bm + 0.5 * used);
    const double blocks = std::max(1.0, m_tiles * (double)tiles(n, x.bn));
    for (int splits = 1; splits <= 256; splits *= 2) {
      if (splits > 1 && (length < 128.0 * splits || blocks * splits > 2.0 * x.places)) break;
      const double full = blocks * splits / x.places;
      const double rounds = full <= 1.0 ? 1.0 : staged ? full + 0.3 : 0.5 * (std::ceil(0.94 * full) + std::ceil(1.06 * full));  // (blocks are known to 6%)
      const double each = (over_rows ? x.over : x.by_rows) * (blocks * splits <= x.few ? x.alone : 1.0);
      // over rows, in one round the longest group ends last
      double time = rounds * (x.fix + std::ceil(length * (over_rows && groups > 1 && full <= 1.0 ? 1.7 : 1.0) / splits / 64.0) * each);
      if (splits > 1) time += 5.0 + (double)splits * (double)(over_rows ? groups * m : rows) * (double)n * 8.0 / 4e6;
      if (time < least) {
        least = time;
        best = {t, splits};
      }
    }
  }
  return best;
}

}  // namespace

// Bytes of the parts, whichever kernel makes them.
size_t group_part_bytes(bool over_rows, int type, int64_t rows, int64_t m, int64_t n, int64_t k, int64_t groups) {
  int splits = group_plan(over_rows, true, type == GS_F32, rows, m, n, k, groups).splits;
  if (type == GS_BF16) splits = std::max(splits, group_plan(over_rows, false, false, rows, m, n, k, groups).splits);
  return splits > 1 ? (size_t)splits * (over_rows ? groups * m : rows) * group_part_width((int)n) * sizeof(float) : 0;
}

hipError_t launch_group(bool over_rows, GroupArgs a, int type, void* ws, hipStream_t s) {
  const int64_t blocks = group_tiles(over_rows, a.rows, a.m, a.n, a.groups);
  if (blocks == 0) return hipSuccess;
  const GroupPlan plan = group_plan(over_rows, type == GS_F32 || !group_aligned(over_rows, a), type == GS_F32, a.rows, a.m, a.n, a.k, a.groups);
  a.splits = plan.splits;
  a.part = static_cast<float*>(ws);
  hipError_t e;
  if (plan.tile < kGroupStaged128) {
    e = launch_group_mfma(over_rows, plan.tile, a, s);
  } else {
    if (type == GS_BF16)
      staged_launch<__bf16>(over_rows, plan.tile, a, s);
    else
      staged_launch<float>(over_rows, plan.tile, a, s);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = over_rows ? (int64_t)a.groups * a.m : a.rows;
  const int outer = over_rows ? a.m : a.rows;
  const int64_t results = rows * (group_part_width(a.n) / 8);
  // eight threads a result where parts are many: 30039 rows, 40 x 96, dW in 128 parts 15.0 us for 24.5, 60 rows of 2, 8192 x 256, in 64 13.6 for
  // 16.4; 40000 rows, 1024 x 512, in 16 parts 56.8 for 53.6
  if (a.splits > 16) {
    const unsigned groups = (unsigned)tiles(results, 32);
    type == GS_BF16 ? k_group_join<__bf16, 8><<<groups, 256, 0, s>>>(a, rows, outer, a.c_g) : k_group_join<float, 8><<<groups, 256, 0, s>>>(a, rows, outer, a.c_g);
  } else {
    const unsigned groups = (unsigned)tiles(results, 256);
    type == GS_BF16 ? k_group_join<__bf16, 1><<<groups, 256, 0, s>>>(a, rows, outer, a.c_g) : k_group_join<float, 1><<<groups, 256, 0, s>>>(a, rows, outer, a.c_g);
  }
  return hipGetLastError();
}

}  // namespace gs
