// gs_adamw.hip -- one step of AdamW over many tensors at once, moments in float32 or as 8-bit codes
// with bounds for each 256 units, for gfx950.
//
//   m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr decay) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
//
// Codes are spaced for what they feed: sqrt(v) divides the step, and moments of one block lie orders of
// magnitude apart, so m goes by the square of its code and v by the fourth power (sqrt(v) by the square), down
// to 1/16129 and 1/65025 of the block's largest.  v > 0 keeps a code of 1 at least: a second moment
// of 0 beside a first moment would make a step of m / eps.
//
// Memory bounds it: 48M units with moments in 32 bits take 249 us, 5.4 TB/s; 100M in 8 bits with bfloat16 gradients and copies 313 us,
// 5.1 TB/s (the vector units are busy 85% of it), and the moments that the codes stand for 5.6 TB/s.
//
// A wavefront takes a block of 256 units, four a lane.  Moments are updated, and codes decided, in
// float64 (the device's float64 rate is its float32 rate): a code is found with float32 roots and set right
// against its two borders, which are exact.  The tensors' table travels in the kernel's arguments, 64
// tensors a launch, so that nothing is copied to the device and a captured graph holds its own.
#include <algorithm>

#include "gs_device.h"
#include "gs_elem.h"
#include "gs_wave.h"

namespace gs {

constexpr int kAdamwBlock = 256, kAdamwTensors = 64;

struct AdamwTable {
  float* param[kAdamwTensors];
  const void* grad[kAdamwTensors];
  __bf16* copy[kAdamwTensors];
  int64_t n[kAdamwTensors];
  double keep[kAdamwTensors];      // 1 - lr decay
  uint32_t first[kAdamwTensors];   // the tensor's first block in this launch (past the last tensor: all ones)
  void *m, *v;                     // of the launch's first block
  float2* bounds;
  const float* grad_scale;
  double b1, b2, c1, c2;
  double rate, eps;                // -lr and epsilon with the bias corrections: m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps)
  uint32_t blocks, each;  // of the launch, of a wavefront
};

constexpr double kAdamwM = 127.0 * 127.0, kAdamwV = 255.0 * 255.0 * 255.0 * 255.0;

// What codes stand for, with q the block's bound times 1 / 127^2 or 1 / 255^4.  With decays like 0.9 a tenth of the new bounds lies, in
// exact arithmetic, halfway between two float32s, so that the last bit of float64 decides.  The order of the operations is therefore one
// that float64 code comes to of itself: q c |c|, then beta times it, each rounded, and the gradient's part added in one operation.
__device__ __forceinline__ double adamw_m_of(double q, int c) {
  const double d = (double)c;
  return q * d * fabs(d);
}
__device__ __forceinline__ double adamw_v_of(double q, uint32_t c) { return q * (double)(c * c * (c * c)); }

// rint(sqrt(t)) for t in [0, 127^2]: float32's, and a step where t lies past a border.
__device__ __forceinline__ int adamw_code_m(double t) {
  float r = rintf(__builtin_amdgcn_sqrtf((float)t));
  const float s = fmaf(r, r, 0.25f);  // exact
  if (t > (double)(s + r)) r += 1.0f;
  if (r > 0.0f && t < (double)(s - r)) r -= 1.0f;
  return min((int)r, 127);
}
// rint(sqrt(sqrt(t))) for t in [0, 255^4].
__device__ __forceinline__ int adamw_code_v(double t) {
  float r = rintf(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf((float)t)));
  const double hi = (double)(r + 0.5f), lo = (double)(r - 0.5f);
  const double hi2 = hi * hi, lo2 = lo * lo;
  if (t > hi2 * hi2) r += 1.0f;
  if (r > 0.0f && t < lo2 * lo2) r -= 1.0f;
  return min((int)r, 255);
}

// x / (sqrt(v) + eps) with the hardware's float64 estimates of a root's reciprocal and of a reciprocal, 2^-24.2 and 2^-24.4 off at most
// (measured over 2^24 values): float32's accuracy over float64's range.  v of 0 and infinity are the formula's.
__device__ __forceinline__ double adamw_quotient(double x, double v, double eps) {
  const double root = v * __builtin_amdgcn_rsq(fmin(fmax(v, 1e-300), 1e300));
  return x * __builtin_amdgcn_rcp(root + eps);
}

// 1 / x to float64's accuracy, of a float32.
__device__ __forceinline__ double adamw_inverse(float x) {
  const double d = x;
  double r = __builtin_amdgcn_rcp(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(r, fma(-d, r, 1.0), r);
  return r;
}

constexpr int kAdamwUnits = kAdamwBlock / kWave;  // units a lane

// A block's units of a lane, as they lie in memory.
template <int BITS>
struct AdamwLane {
  float p[kAdamwUnits], g[kAdamwUnits];
  float m[BITS == 32 ? kAdamwUnits : 1], v[BITS == 32 ? kAdamwUnits : 1];
  uint32_t cm, cv;
  float2 top;
};

template <typename TG, int BITS>
__global__ __launch_bounds__(256) void k_adamw(AdamwTable a) {
  constexpr int R = kAdamwUnits;
  const uint32_t from = __builtin_amdgcn_readfirstlane((blockIdx.x * 4 + threadIdx.x / kWave) * a.each), to = min(from + a.each, a.blocks);
  if (from >= to) return;  // whole wavefronts, which do not exchange with each other
  const uint32_t first = a.first[__lane_id()];
  const double scale = a.grad_scale ? (double)*a.grad_scale : 1.0;
  // the tensor of a block: a lane looks at each one's first
  auto tensor = [&](uint32_t blk) { return __popcll(__ballot(first <= blk)) - 1; };
  auto unit = [&](uint32_t blk, int t) { return (int64_t)(blk - a.first[t]) * kAdamwBlock + __lane_id() * R; };
  auto units = [&](int64_t u0, int t) {
    const int64_t left = a.n[t] - u0;
    return left >= R ? R : left > 0 ? (int)left : 0;
  };
  auto load = [&](uint32_t blk, AdamwLane<BITS>& x) {
    const int t = tensor(blk);
    const int64_t u0 = unit(blk, t), at = (int64_t)blk * kAdamwBlock + __lane_id() * R;
    const int n = units(u0, t);
    load_units(a.param[t] + u0, n, x.p);
    load_units(static_cast<const TG*>(a.grad[t]) + u0, n, x.g);
    if constexpr (BITS == 32) {
      load_elems<R>(static_cast<const float*>(a.m) + at, x.m);
      load_elems<R>(static_cast<const float*>(a.v) + at, x.v);
    } else {
      x.cm = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + at);
      x.cv = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + at);
      x.top = a.bounds[blk];
    }
  };
  auto step = [&](uint32_t blk, AdamwLane<BITS>& x) {
    const int t = tensor(blk);
    const int64_t u0 = unit(blk, t), at = (int64_t)blk * kAdamwBlock + __lane_id() * R;
    const int n = units(u0, t);
    const double keep = a.keep[t];
    double m[R], v[R];
    const double sm = BITS == 32 ? 0.0 : (double)x.top.x * (1.0 / kAdamwM), sv = BITS == 32 ? 0.0 : (double)x.top.y * (1.0 / kAdamwV);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = BITS == 32 ? (double)x.m[BITS == 32 ? i : 0] : adamw_m_of(sm, (int)(int8_t)(x.cm >> (8 * i)));
      v[i] = BITS == 32 ? (double)x.v[BITS == 32 ? i : 0] : adamw_v_of(sv, (x.cv >> (8 * i)) & 255u);
      const double g = (double)x.g[i] * scale;
      m[i] = fma(a.c1, g, a.b1 * m[i]);
      v[i] = fma(a.c2, g * g, a.b2 * v[i]);
      x.p[i] = (float)fma((double)x.p[i], keep, adamw_quotient(a.rate * m[i], v[i], a.eps));
    }
    store_units(a.param[t] + u0, n, x.p);
    if (a.copy[t]) store_units(a.copy[t] + u0, n, x.p);
    if constexpr (BITS == 32) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        x.m[i] = i < n ? (float)m[i] : 0.0f;
        x.v[i] = i < n ? (float)v[i] : 0.0f;
      }
      store_elems<R>(static_cast<float*>(a.m) + at, x.m);
      store_elems<R>(static_cast<float*>(a.v) + at, x.v);
    } else {
      if (__any(n < R)) {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i >= n) m[i] = v[i] = 0.0;
      }
      // largest as integers: float32s of one sign are ordered so, infinities and NaNs above them
      uint32_t mu = 0, vu = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        mu = max(mu, __float_as_uint((float)m[i]) & 0x7fffffffu);
        vu = max(vu, __float_as_uint((float)v[i]) & 0x7fffffffu);
      }
      mu = (uint32_t)wave_minmax<true>((int)mu);
      vu = (uint32_t)wave_minmax<true>((int)vu);
      const float mt = __uint_as_float(mu < 0x7f800000u ? mu : 0x7fc00000u), vt = __uint_as_float(vu < 0x7f800000u ? vu : 0x7fc00000u);
      // a bound of NaN or 0 makes codes of 0
      const double im = mt > 0.0f ? kAdamwM * adamw_inverse(mt) : 0.0, iv = vt > 0.0f ? kAdamwV * adamw_inverse(vt) : 0.0;
      // float32's roots decide all codes but those next to a border between two: they are off by 1.25 and 1.63 times 2^-23 at most (a
      // conversion's 2^-24 under one root and two, and 2^-23 for each root), 1.9e-5 of 127 and 5e-5 of 255
      uint32_t cm = 0, cv = 0;
      bool near = true;
      // bounds below float32's normal numbers may be a half and more below their largest moments, whose codes then need their limits
      if (mt >= 0x1p-126f && vt >= 0x1p-126f) {
        near = false;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float y = __builtin_amdgcn_sqrtf((float)(fabs(m[i]) * im)), z = __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf((float)(v[i] * iv)));
          const float ry = rintf(y), rz = rintf(z);
          near |= fabsf(y - ry) > 0.5f - 0x1p-15f || fabsf(z - rz) > 0.5f - 0x1p-14f;
          const int c = (int)ry, e = (int)rz;
          cm |= ((uint32_t)(m[i] < 0.0 ? -c : c) & 255u) << (8 * i);
          cv |= (uint32_t)(v[i] > 0.0 ? max(e, 1) : e) << (8 * i);
        }
      }
      if (__any(near)) {
        cm = cv = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          int c = im > 0.0 ? adamw_code_m(fabs(m[i]) * im) : 0;
          c = m[i] < 0.0 ? -c : c;
          int e = iv > 0.0 ? adamw_code_v(v[i] * iv) : 0;
          if (iv > 0.0 && v[i] > 0.0) e = max(e, 1);
          cm |= ((uint32_t)c & 255u) << (8 * i);
          cv |= (uint32_t)e << (8 * i);
        }
      }
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + at) = cm;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + at) = cv;
      if (__lane_id() == 0) a.bounds[blk] = make_float2(mt, vt);
    }
  };
  // a block's loads run under the one before
  AdamwLane<BITS> x, next;
  load(from, x);
  for (uint32_t blk = from; blk < to; ++blk) {
    if (blk + 1 < to) load(blk + 1, next);
    step(blk, x);
    x = next;
  }
}

// What the codes stand for, rounded once.
__global__ __launch_bounds__(256) void k_adamw_moments(uint32_t blocks, const uint8_t* __restrict__ m,
                                                       const uint8_t* __restrict__ v,
                                                       const float2* __restrict__ bounds, float* __restrict__ out_m,
                                                       float* __restrict__ out_v) {
  const uint32_t blk = blockIdx.x * 8 + threadIdx.x / 32;
  if (blk >= blocks) return;
  const int64_t at = (int64_t)blk * kAdamwBlock + (threadIdx.x & 31) * 8;
  const uint2 cm = *reinterpret_cast<const uint2*>(m + at), cv = *reinterpret_cast<const uint2*>(v + at);
  const float2 top = bounds[blk];
  const double sm = (double)top.x * (1.0 / kAdamwM), sv = (double)top.y * (1.0 / kAdamwV);
  float mf[8], vf[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t wm = i < 4 ? cm.x : cm.y, wv = i < 4 ? cv.x : cv.y;
    mf[i] = (float)adamw_m_of(sm, (int)(int8_t)(wm >> (8 * (i & 3))));
    vf[i] = (float)adamw_v_of(sv, (wv >> (8 * (i & 3))) & 255u);
  }
  store_elems<8>(out_m + at, mf);
  store_elems<8>(out_v + at, vf);
}

hipError_t launch_adamw(int count, const gs_adamw_tensor* tensors, int grad_type, int bits, void* m, void* v,
                        float* bounds, const gs_adamw_params& h, const float* grad_scale, hipStream_t s) {
  AdamwTable a{};
  a.grad_scale = grad_scale;
  a.b1 = h.beta1;
  a.b2 = h.beta2;
  a.c1 = 1.0 - h.beta1;
  a.c2 = 1.0 - h.beta2;
  const double root = sqrt(1.0 - pow(h.beta2, (double)h.step));
  a.rate = -h.lr * root / (1.0 - pow(h.beta1, (double)h.step));
  a.eps = h.eps * root;
  char *mp = static_cast<char*>(m), *vp = static_cast<char*>(v);
  const int64_t each = (int64_t)kAdamwBlock * (bits / 8);
  int64_t done = 0;  // blocks of the launches before
  for (int i = 0; i < count;) {
    int k = 0;
    uint32_t blocks = 0;
    for (; i < count && k < kAdamwTensors; ++i) {
      const gs_adamw_tensor& x = tensors[i];
      if (x.n == 0) continue;
      a.param[k] = x.param;
      a.grad[k] = x.grad;
      a.copy[k] = static_cast<__bf16*>(x.copy);
      a.n[k] = x.n;
      a.keep[k] = 1.0 - h.lr * x.decay;
      a.first[k++] = blocks;
      blocks += (uint32_t)((x.n + kAdamwBlock - 1) / kAdamwBlock);
    }
    if (!blocks) break;
    for (; k < kAdamwTensors; ++k) a.first[k] = ~0u;
    a.blocks = blocks;
    a.m = mp + done * each;
    a.v = vp + done * each;
    a.bounds = reinterpret_cast<float2*>(bounds) + (bits == 8 ? done : 0);
    // two blocks a wavefront hide the second one's loads (100M units, of 368 us then: 347); few blocks are spread out (900k units: 8.1 us,
    // two a wavefront 8.9)
    a.each = blocks >= 65536 ? 2 : 1;
    const unsigned groups = (blocks + 4 * a.each - 1) / (4 * a.each);
    if (bits == 8)
      grad_type == GS_BF16 ? k_adamw<__bf16, 8><<<groups, 256, 0, s>>>(a) : k_adamw<float, 8><<<groups, 256, 0, s>>>(a);
    else
      grad_type == GS_BF16 ? k_adamw<__bf16, 32><<<groups, 256, 0, s>>>(a) : k_adamw<float, 32><<<groups, 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    done += blocks;
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(int64_t blocks, const int8_t* m, const uint8_t* v, const float* bounds, float* out_m,
                                float* out_v, hipStream_t s) {
  k_adamw_moments<<<(unsigned)((blocks + 7) / 8), 256, 0, s>>>((uint32_t)blocks, reinterpret_cast<const uint8_t*>(m), v,
                                                               reinterpret_cast<const float2*>(bounds), out_m, out_v);
  return hipGetLastError();
}

}  // namespace gs
