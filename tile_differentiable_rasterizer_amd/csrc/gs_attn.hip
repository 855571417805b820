// gs_attn.hip -- attention of query rows to the keys of another sequence, forward, for gfx950.
//
// softmax in one pass over the keys: with m the running maximum and l the running sum of
// 2^(s - m), a tile that raises m scales l and the output by 2^(m_old - m).
//
// The scores are computed transposed, S^T[key][row] = K Q^T, so that a lane holds scores of one
// row only (its column of the result): maximum and sum are in-lane but for one exchange between
// the halves, the row's statistics are one register, and the weights are at once the B operand of
// O^T[d][row] = V^T P^T.  The weights enter that product in the element type (bfloat16: an error
// of 2^-8 of each weight at most, of the order of the output's own rounding; float32: in three bfloat16
// parts that hold all of its bits); everything else is float32.
//
// A workgroup has 128 rows, 32 a wavefront (a matrix instruction's columns), and walks tiles of 64 keys, whose next
// one's loads run beside this one's products.  64 rows a wavefront halve the LDS reads, but leave one wavefront a
// SIMD: 400 TFLOP/s instead of 900 at D 128.
//
// What bounds it are the products and the vector arithmetic of the softmax (a score's multiply and add, exponential, sum,
// half a rounding), which the SIMDs do one or the other: busy 56% and 39% of the time at D 128, 42% and 60% at 64.
// Two tiles at once with one's exponentials between the other's products is no faster (D 64 711 -> 669 TFLOP/s).
// Whole calls: D 128, 2 x 3907 x 8160, 32 heads 975 us, 1.07 PFLOP/s; D 64, 3907 x 32768, 16 heads 740 us, 0.71;
// D 64, 3 x 3907 x 3600, 16 heads 262 us, 0.66; float32 D 64, 2 x 2400 x 2500, 8 heads 191 us, 0.13 (a product of
// 8192 x 8192: bfloat16 1.35, float32 0.15).  One token of 32 heads for each of 8 sequences of up to 8160
// states, 79 MB: 22 us and 4 to join, 3.1 TB/s.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gs_attn.h"

namespace gs {

// A tile's weights are taken relative to the maximum known before it, and the tile's sum tells
// whether that was too low: only then (and on a row's first tile) the maximum is looked for, the
// sums are scaled and the weights taken again.  Weights of up to this cost float32 and bfloat16
// nothing (they are relative in both).  (The maximum sought on every tile: D 64 724 TFLOP/s instead of 782, D 128
// 900 instead of 938.)
constexpr float kMostWeight = 1024.0f;

template <typename T, int DP>
__global__ __launch_bounds__(256, (kWavesOf<T, DP>)) void k_attn_fwd(AttnArgs a) {
  using Ti = Tile<T, DP>;
  using Both = Pair<T, DP, kAttnKeys>;
  __shared__ __align__(16) char lds[Both::kTiles][Both::kBytes];  // keys and values
  __shared__ int scratch[4][4];
  __shared__ uint64_t words[4];
  const RowBlock block(a);
  const int b = block.b, hk = block.hk, split = block.split;
  const int lane = __lane_id(), half = lane >> 5;
  const int row = (block.rt * 4 + (threadIdx.x >> 6)) * 32 + (lane & 31);
  const bool valid = row < a.rows;
  const int i = valid ? row / a.group : 0, h = hk * a.group + (valid ? row - i * a.group : 0);
  int2 range = row_range(a, b, i);
  const bool live = valid && range.x < range.y;
  if (!live) range = make_int2(0, 0);
  const Seen seen = block_seen(a, b, range, scratch);

  Frag<T> qf[DP / 16];
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) qf[s] = frag_flip(frag_mem<T>(head_ptr<T>(a.q, b, i, h), a.d, s, live), a.flip);
  if (a.scale == 0.0f) {
    // a slope of 0 could not tell scores from keys that are not seen (0 times -inf): the queries take it
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) qf[s] = frag_zeros(qf[s]);
  }
  f32x16 o[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) o[t] = (f32x16)0.0f;
  // m: the score that the weights are relative to (not below the row's maximum by more than
  // kMostWeight allows); base = m * slope; l: sum of the lane's weights
  float m = live ? -INFINITY : 0.0f, base = 0.0f, l = 0.0f;

  const int t_lo = seen.first / kAttnKeys, t_n = seen.last > seen.first ? (seen.last + kAttnKeys - 1) / kAttnKeys - t_lo : 0;
  Tiles tile;
  tile.t = t_lo + (int)((int64_t)t_n * split / a.splits);
  tile.end = t_lo + (int)((int64_t)t_n * (split + 1) / a.splits);
  const T* kh = head_ptr<T>(a.k, b, 0, hk);
  const T* vh = head_ptr<T>(a.v, b, 0, hk);
  Both kv;
  kv.a.plan(a.k, 1, a.d);
  kv.b.plan(a.v, 1, a.d);
  auto load = [&](int buf) {
    const T *k = kh + tile.k0 * a.k.token_stride, *v = vh + tile.k0 * a.v.token_stride;
    kv.a.load(kv.at(lds, buf, 0), a.d, tile.word, k, [&](int r) { return k + r * a.k.token_stride; });
    kv.b.load(kv.at(lds, buf, 1), a.d, tile.word, v, [&](int r) { return v + r * a.v.token_stride; });
  };
  tile.next(a, b, seen, range, words);
  if (tile.word) load(0);
  const bool idle = row - (lane & 31) >= a.rows;  // no row: such a wavefront only loads
  const typename Ti::Lane at;
  // one tile, in the buffers that the compiler knows (offsets then are immediates)
  auto one = [&](auto which) {
    constexpr int buf = decltype(which)::value;
    const uint64_t word = tile.word;
    const int k0 = tile.k0;
    const bool ragged = tile.ragged;
    kv.ready(lds);
    tile.next(a, b, seen, range, words);
    if (tile.word) load(buf ^ 1);
    const char *kt = kv.at(lds, buf, 0), *vt = kv.at(lds, buf, 1);

    if (idle) return;
    f32x16 s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j] = (f32x16)0.0f;
#pragma unroll
      for (int st = 0; st < DP / 16; ++st) s[j] = mma(Ti::frag_rows(kt, at, 32 * j, st), qf[st], s[j]);
    }
    if (ragged || word != ~0ull) {
      // a row that sees nothing takes the tile's keys as they are; its result is not used
      uint64_t mine = word;
      if (ragged && live) mine &= range_word(range.x, range.y, k0);
      const uint32_t lo = (uint32_t)mine >> (4 * half), hi = (uint32_t)(mine >> 32) >> (4 * half);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[0][r] = (lo >> crow(r, 0)) & 1 ? s[0][r] : -INFINITY;
        s[1][r] = (hi >> crow(r, 0)) & 1 ? s[1][r] : -INFINITY;
      }
    }
    Frag<T> p[4];
    float sum;
    auto weigh = [&] {
      sum = 0.0f;
#pragma unroll
      for (int step = 0; step < 4; ++step) {
        f32x8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __builtin_amdgcn_exp2f(fmaf(s[step >> 1][8 * (step & 1) + e], a.slope, -base));
        p[step] = frag_from<T>(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += w[e];  // before they are rounded: lse is float32
      }
    };
    weigh();
    if (__any(!(m > -INFINITY) || sum > kMostWeight)) {
      float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
      for (int r = 1; r < 16; ++r) top = fmaxf(fmaxf(top, s[0][r]), s[1][r]);
      top = fmaxf(m, pair_max(top));
      const float before = base;
      base = top == -INFINITY ? 0.0f : top * a.slope;
      const float keep = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(before - base);
      m = top;
      l *= keep;
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt) o[dt] *= keep;
      weigh();
    }
    l += sum;
#pragma unroll
    for (int step = 0; step < 4; ++step)
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt) o[dt] = mma(Ti::frag_cols(vt, at, 16 * step, 32 * dt), p[step], o[dt]);
  };
  while (tile.word) {
    one(std::integral_constant<int, 0>());
    if (!tile.word) break;
    one(std::integral_constant<int, 1>());
  }

  const float sum = pair_sum(l);
  if (!valid) return;
  const bool none = !live || sum == 0.0f;  // (a row of NaN is not none)
  if (a.splits == 1) {
    const float inv = none ? 0.0f : 1.0f / sum;
    T* op = head_ptr<T>(a.out, b, i, h);
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d = 32 * dt + 8 * c + 4 * half;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = none ? 0.0f : o[dt][4 * c + e] * inv;
        if (d < a.d) store_elems<4>(op + d, x);
      }
    if (a.lse && half == 0)
      a.lse[((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i] = none ? -INFINITY : (base + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
  } else {
    const int64_t place = ((int64_t)(split * a.batch + b) * a.kv_heads + hk) * a.rows + row;
    float* op = a.part + place * DP;
    if (!none) {
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = o[dt][4 * c + e];
          store_elems<4>(op + 32 * dt + 8 * c + 4 * half, x);
        }
    }
    if (half == 0) a.part_ml[place] = make_float2(none ? -INFINITY : base, none ? 0.0f : sum);
  }
}

// Key tiles that each block of 128 rows (sequence, block) may see: one wavefront each.
__global__ __launch_bounds__(256) void k_attn_lengths(AttnArgs a, int items, int32_t* __restrict__ lengths) {
  const int item = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= items) return;
  const int blocks = (a.rows + 127) / 128, b = item / blocks, rt = item - b * blocks;
  int first = INT32_MAX, last = 0;
  for (int i = rt * 128 / a.group + (int)__lane_id(); i <= min(rt * 128 + 127, a.rows - 1) / a.group; i += 64) {
    const int2 r = row_range(a, b, i);
    if (r.x < r.y) {
      first = min(first, r.x);
      last = max(last, r.y);
    }
  }
  first = wave_min_i(first);
  last = wave_max_i(last);
  if (__lane_id() == 0) lengths[item] = last > first ? (last - 1) / kAttnKeys - first / kAttnKeys + 1 : 0;
}

// order[] = the blocks, longest first (by 1024 classes of length; within a class in no certain order,
// which no result depends on).  One workgroup.
__global__ __launch_bounds__(1024) void k_attn_order(int items, int tiles, const int32_t* __restrict__ lengths,
                                                     int32_t* __restrict__ order) {
  __shared__ int count[1024];
  __shared__ int waves[16];
  const int t = threadIdx.x;
  count[t] = 0;
  __syncthreads();
  auto place = [&](int i) { return 1023 - (int)((int64_t)lengths[i] * 1023 / tiles); };
  for (int i = t; i < items; i += 1024) atomicAdd(&count[place(i)], 1);
  __syncthreads();
  const int mine = count[t], upto = wave_inclusive_scan(mine);
  if (__lane_id() == 63) waves[t >> 6] = upto;
  __syncthreads();
  int before = upto - mine;
  for (int w = 0; w < (t >> 6); ++w) before += waves[w];
  count[t] = before;
  __syncthreads();
  for (int i = t; i < items; i += 1024) order[atomicAdd(&count[place(i)], 1)] = i;
}

// Joins the splits of a row: weights 2^(m_s - max m).  One workgroup for ROWS rows; a row's splits
// are shared out over its 256 / (ROWS * DP / 4) groups of DP / 4 lanes (four elements a lane), which
// meet in LDS.  Few rows leave the splits' loads as the only parallelism.  Memory bound: 4 parts of 62512 rows
// of 64 15 us, 4.7 TB/s.
template <typename T, int DP, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int kLanes = DP / 4, kGroups = 256 / kLanes / ROWS;
  __shared__ float4 sum[ROWS][kGroups][kLanes];
  __shared__ float2 ml[ROWS][kGroups];
  const int64_t n = (int64_t)a.batch * a.kv_heads * a.rows;
  const int g = threadIdx.x / kLanes, r = g % ROWS, part = g / ROWS, d = (threadIdx.x % kLanes) * 4;
  const int64_t at = (int64_t)blockIdx.x * ROWS + r;
  const bool here = part < kGroups && at < n;
  float m = -INFINITY, l = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (here) {
    for (int s = part; s < a.splits; s += kGroups) m = fmaxf(m, a.part_ml[s * n + at].x);
#pragma unroll 4
    for (int s = part; s < a.splits; s += kGroups) {
      const float2 w = a.part_ml[s * n + at];
      const float4 v = *reinterpret_cast<const float4*>(a.part + (s * n + at) * DP + d);
      const bool seen = w.x != -INFINITY;  // else its sums are not written
      const float add = seen ? __builtin_amdgcn_exp2f(w.x - m) : 0.0f;
      l = fmaf(w.y, add, l);
      x = make_float4(fmaf(seen ? v.x : 0.0f, add, x.x), fmaf(seen ? v.y : 0.0f, add, x.y), fmaf(seen ? v.z : 0.0f, add, x.z), fmaf(seen ? v.w : 0.0f, add, x.w));
    }
    sum[r][part][d / 4] = x;
    if (d == 0) ml[r][part] = make_float2(m, l);
  }
  __syncthreads();
  if (part != 0 || at >= n) return;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) m = fmaxf(m, ml[r][i].x);
  const float base = m == -INFINITY ? 0.0f : m;
  l = 0.0f;
  float y[4] = {};
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float w = __builtin_amdgcn_exp2f(ml[r][i].x - base);
    const float4 v = sum[r][i][d / 4];
    l = fmaf(ml[r][i].y, w, l);
    y[0] = fmaf(v.x, w, y[0]);
    y[1] = fmaf(v.y, w, y[1]);
    y[2] = fmaf(v.z, w, y[2]);
    y[3] = fmaf(v.w, w, y[3]);
  }
  const bool none = m == -INFINITY;
  const float inv = none ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  const int bh = (int)(at / a.rows), row = (int)(at - (int64_t)bh * a.rows);
  const int b = bh / a.kv_heads, i = row / a.group, h = (bh - b * a.kv_heads) * a.group + row - i * a.group;
  if (d < a.d) store_elems<4>(head_ptr<T>(a.out, b, i, h) + d, y);
  if (a.lse && d == 0)
    a.lse[((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

namespace {

template <typename T, int DP>
hipError_t fwd_launch(const AttnArgs& a, hipStream_t s) {
  const int64_t nbh = (int64_t)a.batch * a.kv_heads;
  const int64_t blocks = nbh * ((a.rows + 127) / 128) * a.splits;
  k_attn_fwd<T, DP><<<(unsigned)blocks, 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  // rows a workgroup: all that its lanes hold where there are rows enough, else one (a token at a
  // time, 16 splits: 14 -> 5 us)
  constexpr int kAll = 256 / (DP / 4);
  const int64_t n = nbh * a.rows;
  if (n >= 4096)
    k_attn_join<T, DP, kAll><<<(unsigned)((n + kAll - 1) / kAll), 256, 0, s>>>(a);
  else
    k_attn_join<T, DP, 1><<<(unsigned)n, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int attn_padded(int d) { return (d + 31) / 32 * 32; }

// Parts that a long axis is split into: those for which a model of the time gives the least.
//
// blocks workgroups, each over `tiles` tiles of tile_us (another workgroup of its CU beside it), become n = blocks s
// of 1 / s the length on `slots` places: full rounds of them, then a rest.  A rest of up to half the places leaves
// every CU one workgroup at most, which alone runs 1.4 times as fast (float32 above 64 elements has one place a
// CU anyway).  Where rows see ranges of their own, workgroups fill in for each other and the longest end late.
// 3 us a round start and end it; the parts cost 4 us for the launch that joins them and part_us each, written and
// read.  At most four rounds.  heads s that is a multiple of the eight XCDs lets the workgroups of one key head
// share an L2 (2%).  Too few blocks for a quarter of the places: a part for each place.
//
// Measured: 2 x 2600 rows x 1000 keys, 8 heads of 128 (336 blocks): 1, 2, 3 parts 36, 53, 54 us; 2 x 2400 x 2500 in
// float32, 64 elements (304 blocks): 243, 229, 191, 4 parts 191; 3907 x 30000, ranges of their own, 4 heads (492
// blocks): 477, 334, 348, 335; backward over 8704 keys, 4 heads of 128 (272 blocks of keys): 1166, 1252, 1023,
// 1094; a token at a time, 32 blocks: 8 parts 29 us, 16 25, 32 28.  92 shapes of 100 to 1300 blocks, against as many
// parts as give each place a workgroup: forward 1.10, backward 1.15 times as fast.
int attn_splits(int64_t heads, int64_t each, int64_t tiles, bool uneven, int slots, double tile_us, double part_us) {
  const int64_t blocks = heads * each, most = tiles / 2;
  if (blocks <= 0 || most < 2) return 1;
  if (blocks < slots / 4) return (int)std::min(most, slots / blocks);  // nothing to weigh
  const double alone = slots > 256 ? 0.72 : 1.0;
  double least = 0.0;
  int best = 0;
  for (int s = 1; s == 1 || (s <= most && s * blocks <= 4 * slots); ++s) {
    const double n = (double)(blocks * s) / slots, full = std::floor(n), rest = n - full;
    double rounds = full + (rest == 0.0 ? 0.0 : rest <= 0.5 ? alone : 1.0 - (1.0 - alone) * (1.0 - rest) / 2.0);
    if (uneven) rounds = std::max(alone, 0.55 * n + 0.35);
    double us = rounds * (tile_us * tiles / s + 3.0) + (s > 1 ? 4.0 + s * part_us : 0.0);
    if (s > 1 && heads * s % 8) us *= 1.02;
    if (best == 0 || us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

// Workgroups that the device holds of the kernels that own rows or keys.
int attn_slots(const gs_cross_attn& p) { return p.type == GS_BF16 || attn_padded(p.head_dim) <= 64 ? 512 : 256; }

// Time of one forward tile (128 rows, 64 keys) with all places taken, as measured: bfloat16 1.3 us of 64
// elements, 2.3 of 128; float32 7.2 and 9.1.
double attn_tile_us(const gs_cross_attn& p) {
  const int d = attn_padded(p.head_dim);
  return p.type == GS_BF16 ? 0.35 + 0.015 * d : d <= 64 ? 0.112 * d : 0.071 * d;
}

// Blocks of 128 rows to be put in order of length, or 0.  Rows with ranges of their own, or sequences
// of several lengths, make workgroups of different lengths; longest first, the short ones fill the
// end.  Worth its two launches (8 us) where the kernel takes ten times that: from 2^28 (row, key) pairs.
int attn_order_items(const gs_cross_attn& p) {
  const int64_t rows = p.q_len * (p.q_heads / p.kv_heads), items = p.batch * ((rows + 127) / 128);
  if (!p.ranges || p.k_len <= 0 || items < 64 || items > 65536) return 0;
  return p.batch * p.kv_heads * rows >= ((int64_t)1 << 28) / p.k_len ? (int)items : 0;
}

// space: two int32 for each of attn_order_items().
hipError_t launch_attn_order(AttnArgs& a, int items, int32_t* space, hipStream_t s) {
  k_attn_lengths<<<(unsigned)((items + 3) / 4), 256, 0, s>>>(a, items, space);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;  // the order takes LDS addresses by the lengths
  k_attn_order<<<1, 1024, 0, s>>>(items, (a.k_len + kAttnKeys - 1) / kAttnKeys, space, space + items);
  a.order = space + items;
  return hipGetLastError();
}

int attn_row_splits(const gs_cross_attn& p, double tile_us) {
  const int64_t rows = p.q_len * (p.q_heads / p.kv_heads), heads = p.batch * p.kv_heads;
  const double part_us = 8e-6 / 4 * heads * rows * attn_padded(p.head_dim);  // 8 bytes an element at 4 TB/s
  return attn_splits(heads, (rows + 127) / 128, (p.k_len + kAttnKeys - 1) / kAttnKeys, p.ranges && p.ranges_row_stride,
                     attn_slots(p), tile_us, part_us);
}

int attn_fwd_splits(const gs_cross_attn& p) { return attn_row_splits(p, attn_tile_us(p)); }
int attn_bwd_q_splits(const gs_cross_attn& p) { return attn_row_splits(p, 1.4 * attn_tile_us(p)); }

hipError_t launch_attn_fwd(AttnArgs a, int type, hipStream_t s) {
  switch (attn_padded(a.d) + type) {
    case 32 + GS_BF16: return fwd_launch<__bf16, 32>(a, s);
    case 64 + GS_BF16: return fwd_launch<__bf16, 64>(a, s);
    case 96 + GS_BF16: return fwd_launch<__bf16, 96>(a, s);
    case 128 + GS_BF16: return fwd_launch<__bf16, 128>(a, s);
    case 32 + GS_F32: return fwd_launch<float, 32>(a, s);
    case 64 + GS_F32: return fwd_launch<float, 64>(a, s);
    case 96 + GS_F32: return fwd_launch<float, 96>(a, s);
    default: return fwd_launch<float, 128>(a, s);
  }
}

}  // namespace gs
