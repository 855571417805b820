// gs_elem.h -- element types of the token operators: loads to float32 and stores rounded once.
// Internal to libgsraster.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gs_tokens.h"

namespace gs {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// N consecutive elements at p (aligned to N elements or 16 bytes, whichever is less) <-> float32.
template <int N>
__device__ __forceinline__ void load_elems(const __bf16* p, float (&x)[N]) {
  typedef __bf16 V __attribute__((ext_vector_type(N)));
  const V v = *reinterpret_cast<const V*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = (float)v[i];
}
template <int N>
__device__ __forceinline__ void load_elems(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i + j] = v[j];
  }
}
template <int N>
__device__ __forceinline__ void store_elems(__bf16* p, const float (&x)[N]) {
  typedef __bf16 V __attribute__((ext_vector_type(N)));
  V v;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (__bf16)x[i];
  *reinterpret_cast<V*>(p) = v;
}
template <int N>
__device__ __forceinline__ void store_elems(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = x[i + j];
    *reinterpret_cast<f32x4*>(p + i) = v;
  }
}

// The calls' tensors with a typed base.
template <typename T>
struct Heads {
  T* p;
  int64_t b, t, h;
};
template <typename T>
inline Heads<T> heads_of(const gs_heads& x) {
  return {static_cast<T*>(x.data), x.batch_stride, x.token_stride, x.head_stride};
}

}  // namespace gs
