// gs_layer_norm.hip -- layer norm of rows and its gradient, with the sums of the weight's and the
// bias's gradient over all rows, for gfx950.
//
//   xh = (x - mean) rstd, y = w xh + b;
//   back: g = w dy, dx = rstd (g - mean(g) - xh mean(g xh)), dw = sum dy xh, db = sum dy.
//
// A row belongs to G lanes, J chunks of eight units each, and stays in their registers: one read of
// memory, then the mean, then the sums over d = x - mean (its squares, and back also g and g d, all
// in one exchange: g xh is g d rstd).  The variance is taken about the mean, not as a difference of
// sums, so that rows far from 0 lose nothing.
//
// Memory bounds it: 39063 rows of 4096 in float32 take 227 us forward and 360 + 5 back, 5.6 and 5.3 TB/s.  Short of that, with 3907 rows of
// 2048 in bfloat16 (8.6 us, 14.7 + 4.0 back), the arithmetic of a unit (vector units busy 85% and 68%) and the sum of the parts.
//
// Chunks are loaded as vectors at any alignment (the memory takes them; a row of odd length starts
// anywhere); the row's last chunk, where it is short, goes unit by unit.
#include <algorithm>

#include "gs_device.h"
#include "gs_elem.h"
#include "gs_wave.h"

namespace gs {

struct LayerNormArgs {
  int64_t rows;
  const void *x, *dy;
  void* y;  // back: dx
  int64_t xs, ds, ys;
  const float *w, *b;
  float* part;  // [workgroups][2][padded width]
  float *dw, *db;
  int32_t width;
  float eps, inv_width;
};

// A row is summed as 2^-15 of its units, 16384 at most, so that its sum is a float32 wherever its mean is one.  A power of two changes
// no bit of the mean (but for sums below 2^-111, which no variance that float32 holds has beside it).
constexpr float kRowScale = 0x1p-15f;

constexpr int layer_norm_threads(int g) { return g > kWave ? g : 256; }  // one row of several wavefronts, or several rows

// Sums over the G lanes of a row, in each of them.
template <int G, int N>
struct RowSum {
  static constexpr int kWaves = G / kWave;
  float (*space)[kWaves > 0 ? kWaves : 1][N];  // two of them, taken in turn: one barrier an exchange
  int turn = 0;

  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] += dpp_get<0xB1, 0xF>(v[i]);
      v[i] += dpp_get<0x4E, 0xF>(v[i]);
      v[i] += dpp_get<0x141, 0xF>(v[i]);
      v[i] += dpp_get<0x140, 0xF>(v[i]);  // every lane of a row of 16 has its sum
    }
    if constexpr (G >= 32) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], 16, 64);
    }
    if constexpr (G >= kWave) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], 32, 64);
    }
    if constexpr (G > kWave) {
      if (__lane_id() == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) space[turn][threadIdx.x / kWave][i] = v[i];
      }
      __syncthreads();
      // every lane takes one wavefront's, and adds those of its neighbours
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = space[turn][__lane_id() % kWaves][i];
        v[i] += dpp_get<0xB1, 0xF>(v[i]);
        if constexpr (kWaves >= 4) v[i] += dpp_get<0x4E, 0xF>(v[i]);
        if constexpr (kWaves >= 8) v[i] += dpp_get<0x141, 0xF>(v[i]);
        if constexpr (kWaves >= 16) v[i] += dpp_get<0x140, 0xF>(v[i]);
      }
      turn ^= 1;
    }
  }
};

// Eight units of a row as they lie in memory, so that a row's loads run under the row before.
template <typename T>
struct RowUnits {
  typedef T V __attribute__((ext_vector_type(8)));
  V v;
  __device__ __forceinline__ void load(const T* p, int n) {
    if (n >= 8) {
      typedef T U __attribute__((ext_vector_type(8), aligned(sizeof(T))));
      v = *reinterpret_cast<const U*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : (T)0.0f;
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
  }
};

template <typename T, int G, int J, bool BWD>
__global__ __launch_bounds__(layer_norm_threads(G)) void k_layer_norm(LayerNormArgs a) {
  constexpr int kThreads = layer_norm_threads(G), kRows = kThreads / G;  // rows of a workgroup at once
  constexpr int kWaves = G / kWave > 0 ? G / kWave : 1;
  __shared__ float space1[2][kWaves][1], space3[2][kWaves][BWD ? 3 : 1];
  RowSum<G, 1> sum_x{space1};
  RowSum<G, BWD ? 3 : 1> sum_d{space3};
  const int lane = threadIdx.x % G, sub = threadIdx.x / G;
  int n[J];  // units of each chunk
#pragma unroll
  for (int j = 0; j < J; ++j) n[j] = min(max(a.width - (lane + G * j) * 8, 0), 8);
  float w[J][8], b[J][8], dw[J][8] = {}, db[J][8] = {};
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[j][i] = 1.0f;
      b[j][i] = 0.0f;
    }
    if (a.w) load_units(a.w + (lane + G * j) * 8, n[j], w[j]);
    if (!BWD && a.b) load_units(a.b + (lane + G * j) * 8, n[j], b[j]);
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  const bool ragged = a.width % 8 != 0;
  RowUnits<T> next_x[J], next_g[J];
  auto load = [&](int64_t row) {
    const T* xp = static_cast<const T*>(a.x) + row * a.xs + lane * 8;
#pragma unroll
    for (int j = 0; j < J; ++j) next_x[j].load(xp + G * j * 8, n[j]);
    if constexpr (BWD) {
      const T* gp = static_cast<const T*>(a.dy) + row * a.ds + lane * 8;
#pragma unroll
      for (int j = 0; j < J; ++j) next_g[j].load(gp + G * j * 8, n[j]);
    }
  };
  // Forward, a row's loads run under the row before (39063 rows of 4096 in float32: 245 -> 228 us).  Back, where the sums take the
  // registers, other workgroups' do (there 350 -> 382; bfloat16, 15000 rows of 5000: 126 -> 194), but for rows of two wavefronts in
  // bfloat16 (60000 of 1000: 95 -> 86).
  constexpr bool kAhead = !BWD || (sizeof(T) == 2 && G == 128);
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  if (kAhead && row < a.rows) load(row);
  for (; row < a.rows; row += step) {  // uniform over the row's lanes
    float x[J][8], g[J][8], s[1] = {0.0f};
    if (!kAhead) load(row);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      next_x[j].get(x[j]);
      if constexpr (BWD) next_g[j].get(g[j]);
    }
    if (kAhead && row + step < a.rows) load(row + step);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] = fmaf(x[j][i], kRowScale, s[0]);
    sum_x(s);
    const float mean = s[0] * (a.inv_width / kRowScale);
    float t[BWD ? 3 : 1] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float mu = n[j] > 0 ? mean : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] -= mu;
    }
    if (ragged) {  // (a row's last chunk may be short)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= n[j]) x[j][i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = x[j][i];
        t[0] = fmaf(d * a.inv_width, d, t[0]);  // the mean of squares: their sum overflows before it
        if constexpr (BWD) {
          const float gw = g[j][i] * w[j][i];
          t[1] += gw;
          t[2] = fmaf(gw, d, t[2]);
        }
      }
    sum_d(t);
    const float rstd = 1.0f / sqrtf(t[0] + a.eps);
    T* yp = static_cast<T*>(a.y) + row * a.ys + lane * 8;
    if constexpr (!BWD) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = fmaf(x[j][i] * rstd, w[j][i], b[j][i]);
        store_units(yp + G * j * 8, n[j], x[j]);
      }
    } else {
      const float mg = t[1] * a.inv_width, mgx = t[2] * rstd * a.inv_width;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = x[j][i] * rstd;
          dw[j][i] = fmaf(g[j][i], xh, dw[j][i]);
          db[j][i] += g[j][i];
          r[i] = rstd * (fmaf(g[j][i], w[j][i], -mg) - xh * mgx);
        }
        store_units(yp + G * j * 8, n[j], r);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.dw && !a.db) return;
    // the workgroup's sum for each unit, over its rows at once in a fixed order
    constexpr int kUnits = 8 * G * J;
    const int padded = (a.width + 7) & ~7;
    float* part = a.part + (int64_t)blockIdx.x * 2 * padded;
    if constexpr (kRows > 1) {
      __shared__ float both[2][kUnits];
#pragma unroll
      for (int d = G; d < kWave; d <<= 1)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dw[j][i] += __shfl_xor(dw[j][i], d, 64);
            db[j][i] += __shfl_xor(db[j][i], d, 64);
          }
      for (int v = 0; v < kThreads / kWave; ++v) {
        if ((int)threadIdx.x / kWave == v && (int)__lane_id() < G) {
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int u = (lane + G * j) * 8 + i;
              both[0][u] = v ? both[0][u] + dw[j][i] : dw[j][i];
              both[1][u] = v ? both[1][u] + db[j][i] : db[j][i];
            }
        }
        __syncthreads();
      }
      for (int u = threadIdx.x; u < a.width; u += kThreads) {
        if (gridDim.x > 1) {
          part[u] = both[0][u];
          part[padded + u] = both[1][u];
        } else {
          if (a.dw) a.dw[u] = both[0][u];
          if (a.db) a.db[u] = both[1][u];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int u = (lane + G * j) * 8;
        if (gridDim.x > 1) {
          if (n[j] > 0) {
            store_elems<8>(part + u, dw[j]);
            store_elems<8>(part + padded + u, db[j]);
          }
        } else {
          if (a.dw) store_units(a.dw + u, n[j], dw[j]);
          if (a.db) store_units(a.db + u, n[j], db[j]);
        }
      }
    }
  }
}

// dw and db from the workgroups' parts, in a fixed order: 32 units a workgroup, 32 threads a unit, then
// a tree.
__global__ __launch_bounds__(1024) void k_layer_norm_join(const float* __restrict__ part, int width, int padded,
                                                          int parts, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sum[16][32];
  float* const to = blockIdx.y ? db : dw;
  if (!to) return;
  const int u = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  float t = 0.0f;
  if (u < width) {
    const float* p = part + (int64_t)blockIdx.y * padded + u;
    int k = row;
    for (; k + 32 * 7 < parts; k += 32 * 8) {  // eight loads in flight
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[(int64_t)(k + 32 * i) * 2 * padded];
#pragma unroll
      for (int i = 0; i < 8; ++i) t += x[i];
    }
    for (; k < parts; k += 32) t += p[(int64_t)k * 2 * padded];
  }
  t += __shfl_xor(t, 32, 64);
  if (__lane_id() < 32) sum[threadIdx.x >> 6][threadIdx.x & 31] = t;
  __syncthreads();
  if (threadIdx.x < 32 && u < width) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][threadIdx.x];
    to[u] = t;
  }
}

__global__ void k_layer_norm_none(int width, float* __restrict__ dw, float* __restrict__ db) {
  const int u = blockIdx.x * 256 + threadIdx.x;
  if (u >= width) return;
  if (dw) dw[u] = 0.0f;
  if (db) db[u] = 0.0f;
}

namespace {

struct LayerNormPlan {
  int g, j;
};

// Lanes of a row and their chunks: as few lanes as hold it with one each, so that more than half of them work; two from 8192 units on.
// Half as many lanes with two chunks each, where a quarter of the lanes or more would be idle, us: rows of one wavefront instead of two, 60000 of
// 700: bfloat16 45 -> 32 and back 72 -> 52, float32 72 -> 75 and back 115 -> 105; of four instead of eight, 30000 of 2500: bfloat16 81 -> 77 (40000
// of 3000: 99 -> 109) and back 145 -> 122, float32 120 -> 128 and back 165 -> 184; of eight instead of sixteen, 15000 of 5000: bfloat16 87 -> 69
// and back 126 -> 149, float32 121 -> 113 and back 184 either way.  (Of two instead of four: 50000 of 1500 in bfloat16 64 -> 68, back 117 -> 107,
// 8000 of 1536 back 23 -> 25: left.)
LayerNormPlan layer_norm_plan(int width, int type, bool bwd) {
  const int chunks = (width + 7) / 8;
  int g = 16;
  while (g < chunks && g < 1024) g *= 2;
  if (chunks * 4 <= 3 * g && (g == 128 ? type == GS_BF16 || bwd : g == 512 ? type == GS_BF16 && bwd : g == 1024 && !bwd)) return {g / 2, 2};
  return {g, chunks > 1024 ? 2 : 1};
}

// Back, each workgroup leaves a part of dw and db, and few rows are not worth many parts.  Workgroups at most, us with the parts' sum:
//   16 and 8 wavefronts a row.  float32: 8192 rows of 4096: 81.5 with 512, 82.3 with 768, 85.4 with 1024; 10000 of 8192: 106 with 512, 120 with
//   1024.  bfloat16, of which half as much is on its way: 1024 of 3500: 18.7 with 512, 19.7 with 768, 24.2 with 1024; 8192: 47.4, 42.7, 50.4; 30000:
//   193, 156, 201; of 4096: 149.6, 150.4, 178.
//   Four, from 12288 rows on bfloat16 1536 but for rows of 2048, else 1024.  50000 rows, with 1024 and 1536: of 1100 138, 110; 1536 103, 98; 1900 160,
//   130; 2047 183, 156; 2048 119, 125.  12288 rows: of 1100 35.2, 32.2; 1536 29.5, 29.1; 1800 36.0, 35.6.  8192: 26.7, 25.5; 23.2, 23.9; 28.0, 29.0.
//   4096: 19.5, 20.3; 17.3, 18.5; 21.1, 22.3.  float32, 50000: of 1032 128, 136; 2048 245, 254.
//   Two, from 12288 rows on bfloat16 2048, float32 1536 but for rows of 1024, else 1024.  60000 rows, with 1024, 1536 and 2048: bfloat16 of 800 112, 91,
//   77; 1024 81, 81, 77; float32 of 800 129, 114, 120; 1000 144, 145, 153; 1024 135, 141, 147.  12288 rows: bfloat16 of 800 26.6, 24.1, 23.2; 1000 28.0,
//   26.3, 26.3; float32 of 800 28.3, 26.6, 27.3; 1000 33.0, 32.5, 34.1.  8192: 20.8, 19.7, 19.5; 22.6, 22.0, 22.8; 22.2, 21.4, 22.2; 26.0, 25.8, 27.0 (of 1024
//   in bfloat16 19.0, 20.0, 20.9).  4096: 15.4, 16.5, 17.8; 18.1, 19.7, 21.7; 15.6, 15.6, 16.7; 18.4, 19.3, 21.2.
int layer_norm_blocks(int64_t rows, int width, bool bwd, int type) {
  const LayerNormPlan p = layer_norm_plan(width, type, bwd);
  const int64_t each = layer_norm_threads(p.g) / p.g, need = (rows + each - 1) / each;
  int most = 2048;
  if (bwd) {
    most = 1024;
    if (p.g == 1024) most = 512;
    if (p.g == 512) most = type == GS_BF16 ? 768 : 512;
    if (rows >= 12288 && p.g == 256 && type == GS_BF16 && width < 2048) most = 1536;
    if (rows >= 12288 && p.g == 128 && type == GS_BF16) most = 2048;
    if (rows >= 12288 && p.g == 128 && type == GS_F32 && width < 1024) most = 1536;
  }
  return (int)std::min<int64_t>(need, most);
}

template <typename T, bool BWD>
void layer_norm_pick(LayerNormPlan p, const LayerNormArgs& a, int blocks, hipStream_t s) {
  const dim3 grid(blocks);
  const int threads = layer_norm_threads(p.g);
  switch (p.g * p.j) {
    case 16: k_layer_norm<T, 16, 1, BWD><<<grid, threads, 0, s>>>(a); return;
    case 32: k_layer_norm<T, 32, 1, BWD><<<grid, threads, 0, s>>>(a); return;
    case 64: k_layer_norm<T, 64, 1, BWD><<<grid, threads, 0, s>>>(a); return;
    case 128:
      if constexpr (BWD || sizeof(T) == 2)
        if (p.j == 2) {
          k_layer_norm<T, 64, 2, BWD><<<grid, threads, 0, s>>>(a);
          return;
        }
      k_layer_norm<T, 128, 1, BWD><<<grid, threads, 0, s>>>(a);
      return;
    case 256: k_layer_norm<T, 256, 1, BWD><<<grid, threads, 0, s>>>(a); return;
    case 512:
      if constexpr (BWD && sizeof(T) == 2)
        if (p.j == 2) {
          k_layer_norm<T, 256, 2, BWD><<<grid, threads, 0, s>>>(a);
          return;
        }
      k_layer_norm<T, 512, 1, BWD><<<grid, threads, 0, s>>>(a);
      return;
    case 1024:
      if constexpr (!BWD)
        if (p.j == 2) {
          k_layer_norm<T, 512, 2, BWD><<<grid, threads, 0, s>>>(a);
          return;
        }
      k_layer_norm<T, 1024, 1, BWD><<<grid, threads, 0, s>>>(a);
      return;
    default: k_layer_norm<T, 1024, 2, BWD><<<grid, threads, 0, s>>>(a);
  }
}

}  // namespace

size_t layer_norm_workspace_bytes(int64_t rows, int width) {
  if (rows == 0 || width == 0) return 0;
  const int blocks = std::max(layer_norm_blocks(rows, width, true, GS_BF16), layer_norm_blocks(rows, width, true, GS_F32));
  return blocks > 1 ? (size_t)blocks * 2 * ((width + 7) & ~7) * sizeof(float) : 0;
}

// dy NULL: forward.
hipError_t launch_layer_norm(int64_t rows, int width, int type, float eps, const void* dy, int64_t ds, const void* x,
                             int64_t xs, const float* w, const float* b, void* y, int64_t ys, float* dw, float* db,
                             void* ws, hipStream_t s) {
  if (rows == 0) {
    k_layer_norm_none<<<(width + 255) / 256, 256, 0, s>>>(width, dw, db);
    return hipGetLastError();
  }
  LayerNormArgs a{};
  a.rows = rows;
  a.x = x; a.xs = xs;
  a.dy = dy; a.ds = ds;
  a.y = y; a.ys = ys;
  a.w = w; a.b = b;
  a.part = static_cast<float*>(ws);
  a.dw = dw; a.db = db;
  a.width = width;
  a.eps = eps;
  a.inv_width = 1.0f / (float)width;
  const LayerNormPlan p = layer_norm_plan(width, type, dy != nullptr);
  const int blocks = layer_norm_blocks(rows, width, dy != nullptr, type);
  if (type == GS_BF16)
    dy ? layer_norm_pick<__bf16, true>(p, a, blocks, s) : layer_norm_pick<__bf16, false>(p, a, blocks, s);
  else
    dy ? layer_norm_pick<float, true>(p, a, blocks, s) : layer_norm_pick<float, false>(p, a, blocks, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1 || (!dw && !db)) return e;
  k_layer_norm_join<<<dim3((width + 31) / 32, 2), 1024, 0, s>>>(a.part, width, (width + 7) & ~7, blocks, dw, db);
  return hipGetLastError();
}

}  // namespace gs
