// gs_mfma.h -- operands of the 32x32 matrix instructions for the attention kernels, gfx950.
// Internal to libgsraster.
//
// One step of a product C[32][32] += A[32][16] B[16][32]: lane l gives row (A) or column (B)
// l % 32 and the eight k values 8 (l / 32) + 0..7, and holds of C column l % 32, rows
// crow(r, l / 32) for r = 0..15.  bfloat16 is one instruction; float32 is eight (two k values
// each: which k an element stands for is free as long as A and B agree).
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
  f32x8 v;
};

__device__ __forceinline__ f32x16 mma(const Frag<__bf16>& a, const Frag<__bf16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<float>& a, const Frag<float>& b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}

// Row of C that register r of a lane in half h = l / 32 holds.
__device__ __forceinline__ constexpr int crow(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Registers 8 s .. 8 s + 7 of a result as the B operand of step s.
template <typename T>
__device__ __forceinline__ Frag<T> frag_of(const f32x16& c, int s) {
  Frag<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = (decltype(f.v[0] + f.v[0]))c[8 * s + j];
  return f;
}
template <>
__device__ __forceinline__ Frag<__bf16> frag_of<__bf16>(const f32x16& c, int s) {
  Frag<__bf16> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = (__bf16)c[8 * s + j];
  return f;
}

// What the rounding of frag_of(c, s) = f left out, as a fragment.
template <typename T>
__device__ __forceinline__ Frag<T> frag_rest(const f32x16& c, int s, const Frag<T>& f) {
  Frag<T> g;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(T) == 2)
      g.v[j] = (__bf16)(c[8 * s + j] - (float)f.v[j]);
    else
      g.v[j] = 0;
  }
  return g;
}

// Eight float32 values as a fragment.
template <typename T>
__device__ __forceinline__ Frag<T> frag_from(const f32x8& x) {
  Frag<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(T) == 2)
      f.v[j] = (__bf16)x[j];
    else
      f.v[j] = x[j];
  }
  return f;
}
template <typename T, int DP>
struct Tile {
  static constexpr int kPer = 16 / sizeof(T);        // elements of a chunk
  static constexpr int kChunks = DP / kPer;          // chunks of a row
  static constexpr int kRowBytes = DP * sizeof(T);
  // Chunk c of row r lies at c ^ mix(r).  The banks are 256 bytes wide: a read of 16-byte chunks
  // takes 16 rows at once, which need 16 places, and a transposing read four rows of four chunks,
  // which need the four quarters.  Rows of a multiple of 256 bytes all start at the same place: four
  // bits of the row, the low two in quarters; rows of 128 bytes more alternate, rows of 64 or 192
  // bytes more start at the four quarters by themselves.
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
      row = at(l & 31, sizeof(T) == 2 ? h : 2 * h);
      col = at(4 * h + (i >> 2), 2 * ((l >> 4) & 1) + ((i & 3) >> 1)) + 8 * (i & 1);
    }
  };

  // A (or B) operand, row (or column) m0 + l % 32, k = 16 s + 8 (l / 32) + 0..7: k runs along the
  // tile's rows.  m0 is a multiple of 32.  The steps differ in chunk bits above the lane's own, which
  // are an exclusive-or away (or, past four chunks of a row of 192 bytes, a sum).
  static __device__ __forceinline__ Frag<T> frag_rows(const char* tile, const Lane& lane, int m0, int s) {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      const int o = kChunks % 8 == 4 && kChunks > 4 ? (lane.row ^ ((s & 1) << 5)) + ((s >> 1) << 6) : lane.row ^ (s << 5);
      f.v = *reinterpret_cast<const bf16x8*>(tile + m0 * kRowBytes + o);
    } else {
      const int o = kChunks == 24 ? (lane.row ^ ((s & 1) << 6)) + ((s >> 1) << 7) : lane.row ^ (s << 6);
      const f32x4 a = *reinterpret_cast<const f32x4*>(tile + m0 * kRowBytes + o);
      const f32x4 b = *reinterpret_cast<const f32x4*>(tile + m0 * kRowBytes + (o ^ 16));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.v[j] = a[j];
        f.v[4 + j] = b[j];
      }
    }
    return f;
  }

  // A operand of the transposed tile: row m = column c0 + l % 32 of the tile, k = the tile's rows
  // r0 + {0..3, 8..11} + 4 (l / 32) (the order of a result's registers).  r0 is a multiple of 16, c0
  // of 32.
  static __device__ __forceinline__ Frag<T> frag_cols(const char* tile, const Lane& lane, int r0, int c0) {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      // Each group of 16 lanes names four rows of 16 columns, eight bytes a lane, and receives
      // their transpose: lane i column i of the four rows.  Eight rows on the swizzle differs by 2.
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const int o = kChunks % 8 == 4 ? lane.col + 2 * c0 : lane.col ^ (2 * c0);
      union {
        s16x4 q[2];
        bf16x8 v;
      } u;
      u.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + r0 * kRowBytes + o));
      u.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + (r0 + 8) * kRowBytes + (o ^ 32)));
      f.v = u.v;
    } else {
      const int l = __lane_id(), h = l >> 5, c = c0 + (l & 31);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f.v[j] = *reinterpret_cast<const float*>(tile + at(r0 + 8 * (j >> 2) + 4 * h + (j & 3), c >> 2) + 4 * (c & 3));
    }
    return f;
  }
};

// B operand straight from memory: the lane's row p (16-byte aligned, d elements long), k = 16 s +
// 8 (l / 32) + 0..7; zeros past d and where the row does not count.
template <typename T>
__device__ __forceinline__ Frag<T> frag_mem(const T* p, int d, int s, bool counts) {
  const int k = 16 * s + 8 * (__lane_id() >> 5);
  Frag<T> f;
  if (counts && k < d) {  // d is a multiple of 8
    if constexpr (sizeof(T) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(p + k);
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p + k), b = *reinterpret_cast<const f32x4*>(p + k + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.v[j] = a[j];
        f.v[4 + j] = b[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = 0;
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
