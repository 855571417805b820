// gs_mfma.h -- operands of the 32x32 matrix instructions for the attention kernels, gfx950.
// Internal to libgsraster.
//
// One step of a product C[32][32] += A[32][16] B[16][32]: lane l gives row (A) or column (B)
// l % 32 and the eight k values 8 (l / 32) + 0..7, and holds of C column l % 32, rows
// crow(r, l / 32) for r = 0..15.  bfloat16 is one instruction.
//
// float32 is six: x = x0 + x1 + x2 with three bfloat16 holds x's 24 significant bits, and of the nine
// products of two such sums the three smallest (2^-24 and less of the whole) are left out.  The
// matrix unit does 16 bfloat16 products in the time of one float32 product, so this is 2.7 times
// its float32 rate at the same accuracy (attention against 64 bits: 6e-7 by either).
//
// A product whose result is the next one's B operand needs no exchange between lanes: C's
// registers 8 s .. 8 s + 7 of a lane are rows 16 s + {0..3, 8..11} + 4 (l / 32), and serve as the
// k values of step s when the A operand is gathered in that order (frag_cols).
//
// Tiles in LDS: rows of DP elements, dense, in chunks of 16 bytes whose place in the row is
// permuted by the row (swizzle), so that both ways of reading a tile are free of bank conflicts:
// sixteen rows at one chunk (frag_rows), and four rows at four chunks (frag_cols).
#pragma once

#include <type_traits>
#include <utility>

#include "gs_elem.h"

namespace gs {

template <typename T>
struct Frag;  // eight k values of a lane
template <>
struct Frag<__bf16> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  bf16x8 p[3];
};

// x as a sum of three bfloat16.  (What rounds to an infinity is one.)
__device__ __forceinline__ Frag<float> frag_split(f32x8 x) {
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f.p[0][j] = (__bf16)x[j];
    const float top = (float)f.p[0][j];
    x[j] = fabsf(top) == INFINITY ? 0.0f : x[j] - top;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f.p[1][j] = (__bf16)x[j];
    f.p[2][j] = (__bf16)(x[j] - (float)f.p[1][j]);
  }
  return f;
}

__device__ __forceinline__ f32x16 mma(const Frag<__bf16>& a, const Frag<__bf16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<float>& a, const Frag<float>& b, f32x16 c) {
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2], b.p[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[2], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[1], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}

// Row of C that register r of a lane in half h = l / 32 holds.
__device__ __forceinline__ constexpr int crow(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Eight float32 values as a fragment.
template <typename T>
__device__ __forceinline__ Frag<T> frag_from(const f32x8& x) {
  if constexpr (sizeof(T) == 4) {
    return frag_split(x);
  } else {
    Frag<T> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = (__bf16)x[j];
    return f;
  }
}

// Registers 8 s .. 8 s + 7 of a result as the B operand of step s.
template <typename T>
__device__ __forceinline__ Frag<T> frag_of(const f32x16& c, int s) {
  f32x8 x;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = c[8 * s + j];
  return frag_from<T>(x);
}

// What the rounding of frag_of(c, s) = f left out, as a fragment.
__device__ __forceinline__ Frag<__bf16> frag_rest(const f32x16& c, int s, const Frag<__bf16>& f) {
  Frag<__bf16> g;
#pragma unroll
  for (int j = 0; j < 8; ++j) g.v[j] = (__bf16)(c[8 * s + j] - (float)f.v[j]);
  return g;
}

template <typename T, int DP>
struct Tile;

template <int DP>
struct Tile<__bf16, DP> {
  static constexpr int kChunks = DP / 8;  // chunks of a row
  static constexpr int kRowBytes = DP * 2;
  // Chunk c of row r lies at c ^ mix(r).  The banks are 256 bytes wide: a read of 16-byte chunks
  // takes 16 rows at once, which need 16 places, and a transposing read four rows of four chunks,
  // which need the four quarters.  Rows of a multiple of 256 bytes all start at the same place: four
  // bits of the row, the low two in quarters; rows of 128 bytes alternate, rows of 64 or 192 bytes
  // start at the four quarters by themselves.
  static __device__ __forceinline__ int mix(int r) {
    if constexpr (kRowBytes % 256 == 0)
      return ((r & 3) << 2) | ((r >> 2) & 3);
    else if constexpr (kRowBytes % 256 == 128)
      return ((r & 2) << 1) | ((r >> 2) & 3);
    else
      return (r >> 2) & 3;
  }
  static __device__ __forceinline__ int at(int r, int c) { return r * kRowBytes + ((c ^ mix(r)) << 4); }

  // Where the lane reads, from the start of a tile; made once a kernel.
  struct Lane {
    int row, col;
    __device__ __forceinline__ Lane() {
      const int l = __lane_id(), h = l >> 5, i = l & 15;
      row = at(l & 31, h);
      col = at(4 * h + (i >> 2), 2 * ((l >> 4) & 1) + ((i & 3) >> 1)) + 8 * (i & 1);
    }
  };

  // A (or B) operand, row (or column) m0 + l % 32, k = 16 s + 8 (l / 32) + 0..7: k runs along the
  // tile's rows.  m0 is a multiple of 32.  The steps differ in chunk bits above the lane's own, which
  // are an exclusive-or away (or, past four chunks of a row of 192 bytes, a sum).
  static __device__ __forceinline__ Frag<__bf16> frag_rows(const char* tile, const Lane& lane, int m0, int s) {
    const int o = kChunks == 12 ? (lane.row ^ ((s & 1) << 5)) + ((s >> 1) << 6) : lane.row ^ (s << 5);
    return {*reinterpret_cast<const bf16x8*>(tile + m0 * kRowBytes + o)};
  }

  // A operand of the transposed tile: row m = column c0 + l % 32 of the tile, k = the tile's rows
  // r0 + {0..3, 8..11} + 4 (l / 32) (the order of a result's registers).  r0 is a multiple of 16, c0
  // of 32.  Each group of 16 lanes names four rows of 16 columns, eight bytes a lane, and receives
  // their transpose: lane i column i of the four rows.  Eight rows on, the swizzle differs by 2.
  static __device__ __forceinline__ Frag<__bf16> frag_cols(const char* tile, const Lane& lane, int r0, int c0) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int o = kChunks % 8 == 4 ? lane.col + 2 * c0 : lane.col ^ (2 * c0);
    union {
      s16x4 q[2];
      bf16x8 v;
    } u;
    u.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + r0 * kRowBytes + o));
    u.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + (r0 + 8) * kRowBytes + (o ^ 32)));
    return {u.v};
  }
};

// float32: three bfloat16 tiles of 64 rows, one after another, for the three parts.
template <int DP>
struct Tile<float, DP> {
  using Part = Tile<__bf16, DP>;
  using Lane = typename Part::Lane;
  static constexpr int kPart = 64 * Part::kRowBytes;  // bytes

  static __device__ __forceinline__ Frag<float> frag_rows(const char* tile, const Lane& lane, int m0, int s) {
    Frag<float> f;
#pragma unroll
    for (int k = 0; k < 3; ++k) f.p[k] = Part::frag_rows(tile + k * kPart, lane, m0, s).v;
    return f;
  }
  static __device__ __forceinline__ Frag<float> frag_cols(const char* tile, const Lane& lane, int r0, int c0) {
    Frag<float> f;
#pragma unroll
    for (int k = 0; k < 3; ++k) f.p[k] = Part::frag_cols(tile + k * kPart, lane, r0, c0).v;
    return f;
  }
};

// B operand straight from memory: the lane's row p (16-byte aligned, d elements long), k = 16 s +
// 8 (l / 32) + 0..7; zeros past d and where the row does not count.
template <typename T>
__device__ __forceinline__ Frag<T> frag_mem(const T* p, int d, int s, bool counts) {
  const int k = 16 * s + 8 * (__lane_id() >> 5);
  Frag<T> f = {};
  if (counts && k < d) {  // d is a multiple of 8
    if constexpr (sizeof(T) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(p + k);
    } else {
      float x[8];
      load_elems<8>(p + k, x);
      f = frag_split(f32x8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]});
    }
  }
  return f;
}

// N products in a row whose A operands come from LDS, P of them on the way at any time: load(i) reads
// operand i, use(i, operand) multiplies (and does what comes between).  LDS reads and products keep
// this order; vector arithmetic may move between them.  Left to itself the compiler reads an
// operand just before its product and waits out the latency each time.
// The indices are compile-time constants (every operand a register of its own).
template <int I>
using Index = std::integral_constant<int, I>;

template <typename T, int N, int P, class Load, class Use, int... I>
__device__ __forceinline__ void stream_all(Load&& load, Use&& use, std::integer_sequence<int, I...>) {
  Frag<T> f[N];
  auto ahead = [&](auto i) {
    if constexpr (decltype(i)::value < N) f[decltype(i)::value] = load(i);
  };
  auto first = [&](auto i) {
    if constexpr (decltype(i)::value < P) ahead(i);
  };
  auto step = [&](auto i) {
    constexpr int k = decltype(i)::value;
    __builtin_amdgcn_sched_barrier(0x6);  // only vector and scalar arithmetic cross
    use(i, f[k]);
    __builtin_amdgcn_sched_barrier(0x6);
    ahead(Index<k + P>());
  };
  (first(Index<I>()), ...);
  (step(Index<I>()), ...);
}
template <typename T, int N, int P, class Load, class Use>
__device__ __forceinline__ void stream(Load&& load, Use&& use) {
  stream_all<T, N, P>(load, use, std::make_integer_sequence<int, N>());
}

// The same with every sign bit flipped by `flip` (gs_attn.h).
template <typename T>
__device__ __forceinline__ Frag<T> frag_flip(Frag<T> f, uint32_t flip) {
  union {
    Frag<T> f;
    uint32_t u[sizeof(Frag<T>) / 4];
  } x;
  x.f = f;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Frag<T>) / 4); ++i) x.u[i] ^= flip;
  return x.f;
}

// The same with every element multiplied by 0: finite ones become 0, others NaN.
template <typename T>
__device__ __forceinline__ Frag<T> frag_zeros(Frag<T> f) {
  union {
    Frag<T> f;
    __bf16 x[sizeof(Frag<T>) / 2];
  } x;
  x.f = f;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Frag<T>) / 2); ++i) x.x[i] = (__bf16)((float)x.x[i] * 0.0f);
  return x.f;
}

// max and sum with the lane of the other half that holds the same column.
__device__ __forceinline__ float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

}  // namespace gs
