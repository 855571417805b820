// gs_gate.hip -- gated activation that keeps its inputs for the backward pass as 8-bit codes, and
// the backward pass that reads the codes, for gfx950.
//
// "Training 10M Gaussians in 8 GB: Spirula Studio's VRAM efficiency" (mhpq.cn), quantised training
// section: fixed-point codes with a (min, max) pair per 256 units, here over the two inputs of
// y = act(gate) * up, which a feed-forward layer would otherwise hold until its backward pass
// (bfloat16: 2 + 2 bytes a unit pair, and y's 2; as codes 1 + 1, and y made again where the caller's backward pass
// asks for it).
//
// A half wavefront takes 256 consecutive units of a row, eight a lane, of gate and of up: one read,
// the extremes across 32 lanes, codes and y written.  The code is decided in float64, as the
// definition says (ties are not rare with bfloat16's few values in a block); a product and an addition of
// 1.5 * 2^52 leave rint() of the product in the sum's low word.
//
// Forward 2 inputs, y and 2 codes a unit; back 2 codes and dy, 2 gradients and y: the memory bounds both.  39063 x 2752 in
// float32: 285 us, 5.3 TB/s; back 361 us, 5.4 TB/s (a copy of 2 GiB: 4.8).  3907 x 4096 in bfloat16: 30 us, 4.3 TB/s;
// back 25 to 32 us, 6.3 to 4.9 TB/s (as much as the last cache has kept of the forward call).  4 x 1001: 5 us each.  No loop over blocks of
// units: a half wavefront has one, so that a workgroup's reads are a row's next kilobytes.
#include "gs_device.h"
#include "gs_elem.h"

namespace gs {

constexpr int kGateBlock = 256;  // units of a bounds pair
constexpr int kGateUnits = 8;    // units a lane

// act(x) and, where wanted, its derivative.
template <int ACT>
__device__ __forceinline__ float gate_act(float x) {
  if constexpr (ACT == GS_ACT_SILU) {
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
  } else {
    constexpr float k = 0.7978845608028654f;  // sqrt(2 / pi)
    const float z = k * x * fmaf(0.044715f * x, x, 1.0f);
    // (1 + tanh z) / 2 = 1 / (1 + e^(-2 z))
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-2.0f * kLog2e * z));
  }
}
template <int ACT>
__device__ __forceinline__ void gate_act_grad(float x, float* act, float* grad) {
  if constexpr (ACT == GS_ACT_SILU) {
    const float h = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
    *act = x * h;
    *grad = h * fmaf(x, 1.0f - h, 1.0f);
  } else {
    constexpr float k = 0.7978845608028654f;
    // h is exactly 0 or 1 beyond 32, where the cube would overflow in the end; a NaN passes
    const float c = x > 32.0f ? 32.0f : x < -32.0f ? -32.0f : x;
    const float z = k * c * fmaf(0.044715f * c, c, 1.0f);
    const float h = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-2.0f * kLog2e * z));
    *act = x * h;
    // h + x h (1 - h) 2 z'
    *grad = h * fmaf(c * (1.0f - h), 2.0f * k * fmaf(3.0f * 0.044715f * c, c, 1.0f), 1.0f);
  }
}

__device__ __forceinline__ float half_min(float v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) v = fminf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

// The eight units at p, of which `n` exist.
template <bool VEC, typename T>
__device__ __forceinline__ void gate_load(const T* p, int n, float (&x)[8]) {
  if (VEC && n == 8) {
    load_elems<8>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? (float)p[i] : 0.0f;
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void gate_store(T* p, int n, const float (&x)[8]) {
  if (VEC && n == 8) {
    store_elems<8>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (T)x[i];
  }
}

// Codes and bounds of the block's units x (n of them here): (lo, hi) in every lane.
template <bool VEC>
__device__ __forceinline__ void gate_encode(const float (&x)[8], int n, uint8_t* codes, float2* bounds) {
#pragma clang fp contract(off)
  float lo = INFINITY, hi = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      bad |= !(fabsf(x[i]) < INFINITY);
    }
  lo = half_min(lo);
  hi = half_max(hi);
  const uint64_t any = __ballot(bad);
  const uint32_t mine = __lane_id() < 32 ? (uint32_t)any : (uint32_t)(any >> 32);
  if (mine) lo = hi = __int_as_float(0x7fc00000);
  const double scale = hi > lo ? 255.0 * (1.0 / ((double)hi - (double)lo)) : 0.0;
  const double base = mine ? 0.0 : (double)lo;
  uint32_t q[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double t = mine ? 0.0 : ((double)x[i] - base) * scale;
    const uint32_t c = (uint32_t)__double_as_longlong(t + 6755399441055744.0) & 255u;
    q[i >> 2] |= c << (8 * (i & 3));
  }
  if (VEC && n == 8) {
    *reinterpret_cast<uint2*>(codes) = make_uint2(q[0], q[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) codes[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
  }
  if ((__lane_id() & 31) == 0) *bounds = make_float2(lo, hi);
}

// The half wavefront's block (large grids have a second axis: gate_grid).
__device__ __forceinline__ uint32_t gate_item() {
  return (blockIdx.y * gridDim.x + blockIdx.x) * 8 + threadIdx.x / 32;
}

template <typename T, int ACT, bool VEC>
__global__ __launch_bounds__(256) void k_gate8_fwd(uint32_t items, uint32_t blocks, int64_t rows, int64_t width,
                                                   const T* __restrict__ gate, int64_t gs, const T* __restrict__ up,
                                                   int64_t us, T* __restrict__ y, int64_t ys,
                                                   uint8_t* __restrict__ codes, float2* __restrict__ bounds) {
  const uint32_t item = gate_item();
  if (item >= items) return;  // uniform over half wavefronts, which do not exchange with each other
  const uint32_t row = item / blocks, blk = item - row * blocks;
  const int64_t u0 = (int64_t)blk * kGateBlock + (threadIdx.x & 31) * kGateUnits;
  const int64_t left = width - u0;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  float g[8], u[8], r[8];
  gate_load<VEC>(gate + row * gs + u0, n, g);
  gate_load<VEC>(up + row * us + u0, n, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = gate_act<ACT>(g[i]) * u[i];
  gate_store<VEC>(y + row * ys + u0, n, r);
  const int64_t at = (int64_t)row * width + u0;
  gate_encode<VEC>(g, n, codes + at, bounds + item);
  gate_encode<VEC>(u, n, codes + rows * width + at, bounds + rows * blocks + item);
}

template <bool VEC>
__device__ __forceinline__ void gate_decode(const uint8_t* codes, int n, float2 b, float (&x)[8]) {
#pragma clang fp contract(off)
  uint32_t q[2] = {0, 0};
  if (VEC && n == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(codes);
    q[0] = v.x;
    q[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i >> 2] |= (uint32_t)codes[i] << (8 * (i & 3));
  }
  const float step = (b.y - b.x) * (1.0f / 255.0f);
  const float lo = step < INFINITY ? b.x : __int_as_float(0x7fc00000);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = lo + (float)((q[i >> 2] >> (8 * (i & 3))) & 255u) * step;
}

template <typename T, int ACT, bool VEC>
__global__ __launch_bounds__(256) void k_gate8_bwd(uint32_t items, uint32_t blocks, int64_t rows, int64_t width,
                                                   const T* __restrict__ dy, int64_t dys,
                                                   const uint8_t* __restrict__ codes, const float2* __restrict__ bounds,
                                                   T* __restrict__ dgate, int64_t gs, T* __restrict__ dup, int64_t us,
                                                   T* __restrict__ y, int64_t ys) {
  const uint32_t item = gate_item();
  if (item >= items) return;
  const uint32_t row = item / blocks, blk = item - row * blocks;
  const int64_t u0 = (int64_t)blk * kGateBlock + (threadIdx.x & 31) * kGateUnits;
  const int64_t left = width - u0;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  const int64_t at = (int64_t)row * width + u0;
  float d[8], g[8], u[8], rg[8], ru[8], ry[8];
  gate_load<VEC>(dy + row * dys + u0, n, d);
  gate_decode<VEC>(codes + at, n, bounds[item], g);
  gate_decode<VEC>(codes + rows * width + at, n, bounds[rows * blocks + item], u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, da;
    gate_act_grad<ACT>(g[i], &a, &da);
    rg[i] = d[i] * u[i] * da;
    ru[i] = d[i] * a;
    ry[i] = a * u[i];
  }
  gate_store<VEC>(dgate + row * gs + u0, n, rg);
  gate_store<VEC>(dup + row * us + u0, n, ru);
  if (y) gate_store<VEC>(y + row * ys + u0, n, ry);
}

namespace {
// Workgroups of eight blocks each, as few rows of them as a grid's axis (fewer than 2^32 work items) allows.
dim3 gate_grid(uint32_t items) {
  constexpr uint32_t kMost = 1u << 23;
  const uint32_t groups = (items + 7) / 8, rows = (groups + kMost - 1) / kMost;
  return dim3((groups + rows - 1) / rows, rows);
}

template <typename T, int ACT>
void gate_fwd(bool vec, dim3 groups, uint32_t items, uint32_t blocks, int64_t rows, int64_t width,
              const void* gate, int64_t gs, const void* up, int64_t us, void* y, int64_t ys, uint8_t* codes,
              float* bounds, hipStream_t s) {
  const T *g = static_cast<const T*>(gate), *u = static_cast<const T*>(up);
  float2* b = reinterpret_cast<float2*>(bounds);
  if (vec)
    k_gate8_fwd<T, ACT, true><<<groups, 256, 0, s>>>(items, blocks, rows, width, g, gs, u, us, static_cast<T*>(y), ys, codes, b);
  else
    k_gate8_fwd<T, ACT, false><<<groups, 256, 0, s>>>(items, blocks, rows, width, g, gs, u, us, static_cast<T*>(y), ys, codes, b);
}
template <typename T, int ACT>
void gate_bwd(bool vec, dim3 groups, uint32_t items, uint32_t blocks, int64_t rows, int64_t width, const void* dy,
              int64_t dys, const uint8_t* codes, const float* bounds, void* dgate, int64_t gs, void* dup, int64_t us,
              void* y, int64_t ys, hipStream_t s) {
  const T* d = static_cast<const T*>(dy);
  const float2* b = reinterpret_cast<const float2*>(bounds);
  T *dg = static_cast<T*>(dgate), *du = static_cast<T*>(dup), *yy = static_cast<T*>(y);
  if (vec)
    k_gate8_bwd<T, ACT, true><<<groups, 256, 0, s>>>(items, blocks, rows, width, d, dys, codes, b, dg, gs, du, us, yy, ys);
  else
    k_gate8_bwd<T, ACT, false><<<groups, 256, 0, s>>>(items, blocks, rows, width, d, dys, codes, b, dg, gs, du, us, yy, ys);
}
}  // namespace

// `vec`: every row of every matrix starts at a 16-byte boundary (codes: 8 bytes).
hipError_t launch_gate8_fwd(bool vec, int64_t rows, int64_t width, int act, int type, const void* gate, int64_t gs,
                            const void* up, int64_t us, void* y, int64_t ys, uint8_t* codes, float* bounds,
                            hipStream_t s) {
  const uint32_t blocks = (uint32_t)((width + kGateBlock - 1) / kGateBlock), items = (uint32_t)(rows * blocks);
  const dim3 groups = gate_grid(items);
  auto f = type == GS_BF16 ? (act == GS_ACT_SILU ? gate_fwd<__bf16, GS_ACT_SILU> : gate_fwd<__bf16, GS_ACT_GELU>)
                           : (act == GS_ACT_SILU ? gate_fwd<float, GS_ACT_SILU> : gate_fwd<float, GS_ACT_GELU>);
  f(vec, groups, items, blocks, rows, width, gate, gs, up, us, y, ys, codes, bounds, s);
  return hipGetLastError();
}

hipError_t launch_gate8_bwd(bool vec, int64_t rows, int64_t width, int act, int type, const void* dy, int64_t dys,
                            const uint8_t* codes, const float* bounds, void* dgate, int64_t gs, void* dup, int64_t us,
                            void* y, int64_t ys, hipStream_t s) {
  const uint32_t blocks = (uint32_t)((width + kGateBlock - 1) / kGateBlock), items = (uint32_t)(rows * blocks);
  const dim3 groups = gate_grid(items);
  auto f = type == GS_BF16 ? (act == GS_ACT_SILU ? gate_bwd<__bf16, GS_ACT_SILU> : gate_bwd<__bf16, GS_ACT_GELU>)
                           : (act == GS_ACT_SILU ? gate_bwd<float, GS_ACT_SILU> : gate_bwd<float, GS_ACT_GELU>);
  f(vec, groups, items, blocks, rows, width, dy, dys, codes, bounds, dgate, gs, dup, us, y, ys, s);
  return hipGetLastError();
}

}  // namespace gs
