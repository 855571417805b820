// gs_attn_bwd.hip -- gradients of the attention, for gfx950.
//
// The weights are made again from the scores and the kept lse: p = e^(s - lse).  Two kernels, each
// with its results in registers from start to end, so that no sum goes through atomics and its
// order is fixed: k_attn_bwd_kv owns 128 keys and walks the rows (of every query head that shares
// them), k_attn_bwd_q owns 128 rows and walks the keys.  That computes the scores twice (7
// products of a tile instead of 5).
// The row kernel goes first and leaves the rows' statistics for the other: lse in base 2, delta = dout . out,
// and what each tile of 64 rows may see (a kernel of their own before it: 4 x 256 x 256, 16 heads of 64,
// 44 us instead of 40; 3907 x 8160, 32 heads of 128 +0.4%).
//
// kv: S[row][key] = Q K^T and dP[row][key] = dO V^T leave a lane with one key and 16 rows, the B
// operand of dV^T[d][key] = dO^T P and dK^T[d][key] = Q^T dS.  q: as the forward kernel, S^T and
// dP^T = V dO^T, then dQ^T[d][row] = K^T dS^T.
// p and dS enter the products in the element type (bfloat16: rounded once, 2^-8 of each at most; float32: in three
// parts that hold all of their bits).
//
// Products and vector arithmetic take turns on the SIMDs, as in the forward kernel: busy 62% + 38% (rows) and 56% + 31%
// (keys) of the time at D 128, 49% + 59% and 44% + 41% at 64; the keys' kernel also waits, for LDS, which it reads 2.0
// times a product (the rows' kernel 1.3).  2 x 3907 x 8160, 32 heads of 128: rows 1.40 ms, keys 1.94 ms (1.12 and 1.08 PFLOP/s);
// 3 x 3907 x 3600, 16 of 64, lengths 3600, 2250 and 0: 165 to 170 and 291 to 308 us; float32, 2 x 391 x 2500, 8 of 64, a
// quarter of the keys masked: 55 to 57 and 89 to 92 us.
#include "gs_attn.h"

namespace gs {

constexpr int kBwdRows = 64;  // rows of a RowTile
constexpr int kShortTiles = 4;  // key tiles up to which a row's delta is taken from its weights
// LDS operands on the way.  bfloat16: 2 is 1% slower, 6 spills at D 128 (13%).  float32, whose operands
// are three times as large and feed six products: 1 up to D 64 (2: 4-9% slower), above 2 (1: 7%).
template <typename T, int DP>
constexpr int kAhead = sizeof(T) == 2 ? 4 : DP <= 64 ? 1 : 2;

// How the kv kernel fits its registers: the results take DP of them, the fragments of its keys and
// values DP / 2 (bfloat16) or 3 DP / 2.
template <typename T, int DP>
struct KvShape {
  // bfloat16 D 128: the values' fragments stay in LDS, and tiles of 32 rows make room there, so that
  // two wavefronts share a SIMD (one, with everything in registers: both kernels of 2 x 3907 x 8160 3.98 ms
  // instead of 3.50)
  static constexpr bool kValuesInLds = sizeof(T) == 2 && DP == 128;
  static constexpr int kRows = kValuesInLds ? 32 : kBwdRows;  // of a tile
  // (three at bfloat16 D 64, with the values in LDS: the ragged training step 608 us instead of 600)
  static constexpr int kWaves = kValuesInLds || DP <= (sizeof(T) == 2 ? 96 : 64) ? 2 : 1;  // a SIMD
};

template <typename T, int DP>
__global__ __launch_bounds__(256, (KvShape<T, DP>::kWaves)) void k_attn_bwd_kv(AttnArgs a) {
  using Ti = Tile<T, DP>;
  using Sh = KvShape<T, DP>;
  using Both = Pair<T, DP, Sh::kRows>;
  constexpr int kRows = Sh::kRows, kPerInfo = kBwdRows / kRows;
  constexpr int kS = DP / 16, kD = DP / 32;  // k steps of the scores; blocks of the results' elements
  __shared__ __align__(32) char lds[Both::kTiles][Both::kBytes];  // queries and output gradients
  __shared__ __align__(32) float2 stat[2][kRows];
  __shared__ __align__(16) char vt[Sh::kValuesInLds ? 128 * DP * 2 : 16];
  const int nbh = a.batch * a.kv_heads;
  const int bh = blockIdx.x % nbh, rest = blockIdx.x / nbh;
  const int split = rest % a.splits, kb = rest / a.splits;
  const int b = bh / a.kv_heads, hk = bh - b * a.kv_heads;
  const int lane = __lane_id(), half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = kb * 128, k1 = min(k0 + 128, a.k_len);
  const int wk0 = k0 + wave * 32, key = wk0 + (lane & 31);
  const bool open = key < a.k_len && (!a.mask || a.mask[b * a.mask_b + key] != 0);

  Frag<T> kf[kS], vf[kS];
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    kf[s] = frag_flip(frag_mem<T>(head_ptr<T>(a.k, b, key, hk), a.d, s, open), a.flip);
    vf[s] = frag_mem<T>(head_ptr<T>(a.v, b, key, hk), a.d, s, open);
  }
  if constexpr (Sh::kValuesInLds) {  // each wavefront's own 32 rows
#pragma unroll
    for (int s = 0; s < kS; ++s)
      *reinterpret_cast<Frag<T>*>(vt + Ti::at(wave * 32 + (lane & 31), 2 * s + half)) = vf[s];
  }
  f32x16 dk[kD], dv[kD];
#pragma unroll
  for (int t = 0; t < kD; ++t) dk[t] = dv[t] = (f32x16)0.0f;

  const int infos = (a.rows + kBwdRows - 1) / kBwdRows, tiles = infos * kPerInfo;
  const int t_end = (int)((int64_t)tiles * (split + 1) / a.splits);
  const RowTile* info = a.row_tiles + (int64_t)bh * infos;
  const float2* row_stat = a.stat + (int64_t)bh * infos * kBwdRows;
  const T* qh = head_ptr<T>(a.q, b, 0, hk * a.group);
  const T* gh = head_ptr<T>(a.dout, b, 0, hk * a.group);
  Both qg;
  qg.a.plan(a.q, a.group, a.d);
  qg.b.plan(a.dout, a.group, a.d);
  // the next tile from t on whose rows see some of the keys (the same for every thread)
  RowTile next;
  auto find = [&](int t) {
    for (; t < t_end; ++t) {
      const RowTile x = info[t / kPerInfo];
      next.word = uniform(x.word);
      next.first = uniform(x.first);
      next.last = uniform(x.last);
      next.all_from = uniform(x.all_from);
      next.all_to = uniform(x.all_to);
      if (next.word && next.first < k1 && next.last > k0) break;
    }
    return t;
  };
  const int64_t q_step = kRows / a.group * a.q.token_stride, g_step = kRows / a.group * a.dout.token_stride;  // used where even
  auto load = [&](int t, int buf) {
    const int r0 = t * kRows;
    uint64_t word = next.word;
    if constexpr (kPerInfo == 2) word = t & 1 ? word >> 32 : word & 0xffffffffu;
    auto offset = [&](int r, const gs_heads& x) {
      const int i = r / a.group;
      return i * x.token_stride + (r - i * a.group) * x.head_stride;
    };
    qg.a.load(qg.at(lds, buf, 0), a.d, word, qh + t * q_step, [&](int r) { return qh + offset(r0 + r, a.q); });
    qg.b.load(qg.at(lds, buf, 1), a.d, word, gh + t * g_step, [&](int r) { return gh + offset(r0 + r, a.dout); });
    if (wave < kRows / 32)  // 64 words each
      load_to_lds4((const float*)(row_stat + r0) + wave * 64, lane * 4, lds_address((const float*)stat[buf] + wave * 64));
  };

  const typename Ti::Lane at;
  int t = find((int)((int64_t)tiles * split / a.splits));
  if (t < t_end) load(t, 0);
  for (int buf = 0; t < t_end; buf ^= 1) {
    qg.ready(lds);
    const int now = t;
    const bool ragged = next.all_from > k0 || next.all_to < k1;
    t = find(t + 1);
    if (t < t_end) load(t, buf ^ 1);
    const char *qt = qg.at(lds, buf, 0), *gt = qg.at(lds, buf, 1);
    const float2* st2 = stat[buf];
    if (wk0 >= k1) continue;  // no key: such a wavefront only loads
    uint32_t sees = ~0u;  // of row `lane` of the tile: the wavefront's keys that it sees
    if (ragged) {
      const int row = now * kRows + lane;
      const int2 range = row < a.rows ? row_range(a, b, row / a.group) : make_int2(0, 0);
      sees = (uint32_t)range_word(range.x, range.y, wk0);
    }
#pragma unroll 1
    for (int j = 0; j < kRows / 32; ++j) {
      f32x16 s = (f32x16)0.0f, dp = (f32x16)0.0f;
      Frag<T> pf, df, held;
      // scores and dP of 32 rows (their operands in turn), then dV and dK
      constexpr int kEach = Sh::kValuesInLds ? 3 : 2, kFirst = kEach * kS;
      stream<T, kFirst + 4 * kD, kAhead<T, DP>>(
          [&](auto index) {
            constexpr int i = decltype(index)::value, m = i - kFirst, w = i % kEach;
            if constexpr (i >= kFirst)
              return Ti::frag_cols(m & 1 ? qt : gt, at, 32 * j + 16 * (m / (2 * kD)), 32 * ((m >> 1) % kD));
            else if constexpr (w == 2)
              return Ti::frag_rows(vt, at, wave * 32, i / kEach);
            else
              return Ti::frag_rows(w ? gt : qt, at, 32 * j, i / kEach);
          },
          [&](auto index, const Frag<T>& f) {
            constexpr int i = decltype(index)::value, m = i - kFirst, w = i % kEach, dt = (m >> 1) % kD;
            if constexpr (i < kFirst) {
              if constexpr (w == 0) s = mma(f, kf[i / kEach], s);
              if constexpr (w == 1 && kEach == 2) dp = mma(f, vf[i / kEach], dp);
              if constexpr (w == 1 && kEach == 3) held = f;
              if constexpr (w == 2) dp = mma(held, f, dp);
              if constexpr (i == kFirst - 1) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const f32x8 x = *reinterpret_cast<const f32x8*>(&st2[32 * j + 8 * c + 4 * half]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[4 * c + e], a.slope, -x[2 * e]));
                    s[4 * c + e] = p;
                    dp[4 * c + e] = p * (dp[4 * c + e] - x[2 * e + 1]);
                  }
                }
                if (ragged) {
#pragma unroll
                  for (int r = 0; r < 16; ++r) {
                    const bool in = (__shfl((int)sees, 32 * j + crow(r, half), 64) >> (lane & 31)) & 1;
                    s[r] = in ? s[r] : 0.0f;
                    dp[r] = in ? dp[r] : 0.0f;
                  }
                }
              }
            } else {
              if constexpr (m % (2 * kD) == 0) {
                pf = frag_of<T>(s, m / (2 * kD));
                df = frag_of<T>(dp, m / (2 * kD));
              }
              if constexpr (m & 1)
                dk[dt] = mma(f, df, dk[dt]);
              else
                dv[dt] = mma(f, pf, dv[dt]);
            }
          });
    }
  }

  if (key >= a.k_len) return;
  const bool parts = a.splits > 1;
  const int64_t n = (int64_t)nbh * a.k_len, place = (int64_t)bh * a.k_len + key;
  T* kp = head_ptr<T>(a.dk, b, key, hk);
  T* vp = head_ptr<T>(a.dv, b, key, hk);
  float* kw = a.part + (split * 2 * n + place) * DP;
  float* vw = kw + n * DP;
#pragma unroll
  for (int dt = 0; dt < kD; ++dt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = 32 * dt + 8 * c + 4 * half;
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // a masked key's are products with its zeros' weights: not used
        x[e] = open ? dk[dt][4 * c + e] * a.scale : 0.0f;
        y[e] = open ? dv[dt][4 * c + e] : 0.0f;
      }
      if (parts) {
        store_elems<4>(kw + d, x);
        store_elems<4>(vw + d, y);
      } else if (d < a.d) {
        store_elems<4>(kp + d, x);
        store_elems<4>(vp + d, y);
      }
    }
}

template <typename T, int DP>
__global__ __launch_bounds__(256, (kWavesOf<T, DP>)) void k_attn_bwd_q(AttnArgs a) {
  using Ti = Tile<T, DP>;
  constexpr int kS = DP / 16, kD = DP / 32;
  using Both = Pair<T, DP, kAttnKeys>;
  __shared__ __align__(16) char lds[Both::kTiles][Both::kBytes];  // keys and values
  __shared__ int scratch[4][4];
  __shared__ uint64_t words[4];
  const RowBlock block(a);
  const int b = block.b, hk = block.hk, split = block.split, bh = b * a.kv_heads + hk;
  const int lane = __lane_id(), half = lane >> 5;
  const int row = block.rt * 128 + (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool valid = row < a.rows;
  const int i = valid ? row / a.group : 0, h = hk * a.group + (valid ? row - i * a.group : 0);
  int2 range = row_range(a, b, i);
  float2 stat = make_float2(INFINITY, 0.0f);  // a row without keys: every weight is 2^-inf = 0
  const float lse = valid ? a.lse[((int64_t)b * a.kv_heads * a.group + h) * a.q_len + i] : -INFINITY;
  const bool live = valid && range.x < range.y && lse != -INFINITY;
  if (live)
    stat.x = lse * kLog2e;
  else
    range = make_int2(0, 0);
  const Seen seen = block_seen(a, b, range, scratch);
  const int t_lo = seen.first / kAttnKeys, t_n = seen.last > seen.first ? (seen.last + kAttnKeys - 1) / kAttnKeys - t_lo : 0;

  Frag<T> qf[kS], gf[kS];
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    qf[s] = frag_flip(frag_mem<T>(head_ptr<T>(a.q, b, i, h), a.d, s, live), a.flip);
    gf[s] = frag_mem<T>(head_ptr<T>(a.dout, b, i, h), a.d, s, live);
  }
  if (t_n > kShortTiles) {
    const T *op = head_ptr<T>(a.out, b, i, h), *gp = head_ptr<T>(a.dout, b, i, h);
    float delta = 0.0f;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const int d = 16 * s + 8 * half;
      if (live && d < a.d) {
        float x[8], y[8];
        load_elems<8>(op + d, x);
        load_elems<8>(gp + d, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf(x[e], y[e], delta);
      }
    }
    if (live) stat.y = pair_sum(delta);
  }
  const T* kh = head_ptr<T>(a.k, b, 0, hk);
  const T* vh = head_ptr<T>(a.v, b, 0, hk);
  Both kv;
  kv.a.plan(a.k, 1, a.d);
  kv.b.plan(a.v, 1, a.d);
  const typename Ti::Lane at;
  const bool idle = row - (lane & 31) >= a.rows;  // no row: such a wavefront only loads

  // Calls body(keys' tile, values' tile, the row's keys of the tile, whether it sees less than all)
  // for each tile from `begin` to `end` that some row sees something of.
  auto walk = [&](int begin, int end, auto&& body) {
    Tiles tile;
    tile.t = begin;
    tile.end = end;
    auto load = [&](int buf) {
      const T *k = kh + tile.k0 * a.k.token_stride, *v = vh + tile.k0 * a.v.token_stride;
      kv.a.load(kv.at(lds, buf, 0), a.d, tile.word, k, [&](int r) { return k + r * a.k.token_stride; });
      kv.b.load(kv.at(lds, buf, 1), a.d, tile.word, v, [&](int r) { return v + r * a.v.token_stride; });
    };
    tile.next(a, b, seen, range, words);
    if (tile.word) load(0);
    for (int buf = 0; tile.word; buf ^= 1) {
      const uint64_t word = tile.word;
      const int k0 = tile.k0;
      const bool ragged = tile.ragged;
      kv.ready(lds);
      tile.next(a, b, seen, range, words);
      if (tile.word) load(buf ^ 1);
      if (!idle)
        body(kv.at(lds, buf, 0), kv.at(lds, buf, 1), ragged ? word & range_word(range.x, range.y, k0) : word, ragged || word != ~0ull);
    }
  };

  // Over few keys `out` is as large as the values, and its rounding shows in delta = dout . out, which
  // enters every dS of the row: there delta is taken from the weights, sum_j p_j dout . v_j (a row of
  // two keys: error of dq and dk 2.0 -> 1.4 times that of their own rounding).  From 256 keys on
  // out is an average and its rounding does not show.
  if (t_n <= kShortTiles) {
    float delta = 0.0f;
    walk(t_lo, t_lo + t_n, [&](const char* kt, const char* vt, uint64_t mine, bool part) {
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        f32x16 s = (f32x16)0.0f, dp = (f32x16)0.0f;
#pragma unroll
        for (int st = 0; st < kS; ++st) {
          s = mma(Ti::frag_rows(kt, at, 32 * j, st), qf[st], s);
          dp = mma(Ti::frag_rows(vt, at, 32 * j, st), gf[st], dp);
        }
        const uint32_t bits = (uint32_t)(mine >> (32 * j)) >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float w = __builtin_amdgcn_exp2f(fmaf(s[r], a.slope, -stat.x)) * dp[r];
          delta += !part || ((bits >> crow(r, 0)) & 1) ? w : 0.0f;
        }
      }
    });
    if (live) stat.y = pair_sum(delta);
    __syncthreads();  // the tiles are read again
  }
  if (split == 0) {  // for the kv kernel
    const int infos = (a.rows + kBwdRows - 1) / kBwdRows, wave = threadIdx.x >> 6;
    if (half == 0 && row < infos * kBwdRows) a.stat[(int64_t)bh * infos * kBwdRows + row] = stat;
    const uint32_t word = (uint32_t)__ballot(live);
    const int first = wave_min_i(live ? range.x : INT32_MAX), last = wave_max_i(live ? range.y : 0);
    const int from = wave_max_i(live ? range.x : 0), to = wave_min_i(live ? range.y : INT32_MAX);
    if (lane == 0) {
      words[wave] = word;
      scratch[wave][0] = first;
      scratch[wave][1] = last;
      scratch[wave][2] = from;
      scratch[wave][3] = to;
    }
    __syncthreads();
    const int info = block.rt * 2 + threadIdx.x;
    if (threadIdx.x < 2 && info < infos) {
      const int w = 2 * threadIdx.x;
      RowTile x;
      x.word = words[w] | words[w + 1] << 32;
      x.first = min(scratch[w][0], scratch[w + 1][0]);
      x.last = max(scratch[w][1], scratch[w + 1][1]);
      x.all_from = max(scratch[w][2], scratch[w + 1][2]);
      x.all_to = min(scratch[w][3], scratch[w + 1][3]);
      a.row_tiles[(int64_t)bh * infos + info] = x;
    }
    __syncthreads();  // the words are written again
  }

  f32x16 dq[kD];
#pragma unroll
  for (int t = 0; t < kD; ++t) dq[t] = (f32x16)0.0f;
  const int t_begin = t_lo + (int)((int64_t)t_n * split / a.splits), t_end = t_lo + (int)((int64_t)t_n * (split + 1) / a.splits);
  walk(t_begin, t_end, [&](const char* kt, const char* vt, uint64_t mine, bool part) {
#pragma unroll (sizeof(T) == 2 ? 2 : 1)
    for (int j = 0; j < 2; ++j) {
      f32x16 s = (f32x16)0.0f, dp = (f32x16)0.0f;
      Frag<T> df;
      constexpr bool kRest = sizeof(T) == 2 && DP == 32;
      constexpr int kFirst = 2 * kS;
      stream<T, kFirst + 2 * kD, kAhead<T, DP>>(
          [&](auto index) {
            constexpr int i = decltype(index)::value, m = i - kFirst;
            if constexpr (i >= kFirst)
              return Ti::frag_cols(kt, at, 32 * j + 16 * (m / kD), 32 * (m % kD));
            else
              return Ti::frag_rows(i & 1 ? vt : kt, at, 32 * j, i / 2);
          },
          [&](auto index, const Frag<T>& f) {
            constexpr int i = decltype(index)::value, m = i - kFirst;
            if constexpr (i < kFirst) {
              if constexpr (i & 1)
                dp = mma(f, gf[i / 2], dp);
              else
                s = mma(f, qf[i / 2], s);
              if constexpr (i == kFirst - 1) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                  const float p = __builtin_amdgcn_exp2f(fmaf(s[r], a.slope, -stat.x));
                  dp[r] = p * (dp[r] - stat.y);
                }
                if (part) {
                  const uint32_t bits = (uint32_t)(mine >> (32 * j)) >> (4 * half);
#pragma unroll
                  for (int r = 0; r < 16; ++r) dp[r] = (bits >> crow(r, 0)) & 1 ? dp[r] : 0.0f;
                }
              }
            } else {
              if constexpr (m % kD == 0) df = frag_of<T>(dp, m / kD);
              dq[m % kD] = mma(f, df, dq[m % kD]);
              // Short vectors: delta's own error weighs more against dq (by 1 / sqrt(D)), so what dS lost
              // to its rounding is added (bfloat16 D 32, 4000 keys: dq's error 1.52 -> 1.06 times that of
              // rounding dq alone).
              if constexpr (kRest) dq[m % kD] = mma(f, frag_rest(dp, m / kD, df), dq[m % kD]);
            }
          });
    }
  });

  if (!valid) return;
  T* op = head_ptr<T>(a.dq, b, i, h);
  float* pp = a.part + (((int64_t)split * a.batch * a.kv_heads + bh) * a.rows + row) * DP;
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = 32 * dt + 8 * c + 4 * half;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = live ? dq[dt][4 * c + e] * a.scale : 0.0f;
      if (a.splits > 1)
        store_elems<4>(pp + d, x);
      else if (d < a.d)
        store_elems<4>(op + d, x);
    }
}

// Sums of the splits, in a fixed order: dq (KV false, over rows) or dk and dv (KV true, over keys; the
// second half of the grid's y axis is dv).  One workgroup for VECS vectors; a vector's splits are shared
// out over its groups of DP / 4 lanes (four elements a lane), which meet in LDS: few vectors leave the
// splits' loads as the only parallelism (4 rows of 96, 130 splits: 35 us by one group, 5 by ten; 208 keys
// of 128, 32 splits: 11 and 6).
template <typename T, int DP, bool KV, int VECS>
__global__ __launch_bounds__(256) void k_attn_bwd_join(AttnArgs a) {
  constexpr int kLanes = DP / 4, kGroups = 256 / kLanes / VECS;
  __shared__ f32x4 sum[kGroups > 1 ? VECS : 1][kGroups][kLanes];
  const int len = KV ? a.k_len : a.rows;
  const int64_t n = (int64_t)a.batch * a.kv_heads * len, step = KV ? 2 * n : n;
  const int g = threadIdx.x / kLanes, part = g / VECS, d = (threadIdx.x % kLanes) * 4;
  const int64_t at = (int64_t)blockIdx.x * VECS + g % VECS;
  const bool here = part < kGroups && at < n;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (here) {
    const float* p = a.part + ((KV && blockIdx.y ? n : 0) + at) * DP + d;
#pragma unroll 4
    for (int s = part; s < a.splits; s += kGroups) x += *reinterpret_cast<const f32x4*>(p + s * step * DP);
  }
  if constexpr (kGroups > 1) {
    if (here) sum[g % VECS][part][d / 4] = x;
    __syncthreads();
    if (!here || part != 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) x += sum[g][i][d / 4];
  }
  if (!here || d >= a.d) return;
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = x[e];
  const int bh = (int)(at / len), j = (int)(at - (int64_t)bh * len);
  const int b = bh / a.kv_heads, hk = bh - b * a.kv_heads;
  if constexpr (KV) {
    store_elems<4>(head_ptr<T>(blockIdx.y ? a.dv : a.dk, b, j, hk) + d, y);
  } else {
    const int i = j / a.group;
    store_elems<4>(head_ptr<T>(a.dq, b, i, hk * a.group + j - i * a.group) + d, y);
  }
}

int attn_splits(int64_t heads, int64_t each, int64_t tiles, bool uneven, int slots, double tile_us, double part_us);
int attn_padded(int d);
int attn_slots(const gs_cross_attn& p);
double attn_tile_us(const gs_cross_attn& p);

// A tile of 128 keys and 64 rows takes 2.4 times the forward pass's; dk and dv have parts.
int attn_bwd_kv_splits(const gs_cross_attn& p) {
  const int64_t rows = p.q_len * (p.q_heads / p.kv_heads), heads = p.batch * p.kv_heads;
  const double part_us = 16e-6 / 4 * heads * p.k_len * attn_padded(p.head_dim);
  return attn_splits(heads, (p.k_len + 127) / 128, (rows + kBwdRows - 1) / kBwdRows, p.ranges && p.ranges_row_stride,
                     attn_slots(p), 2.4 * attn_tile_us(p), part_us);
}

namespace {

template <typename T, int DP, bool KV>
hipError_t bwd_join(const AttnArgs& a, int64_t n, hipStream_t s) {
  constexpr int kAll = 256 / (DP / 4);
  if (n >= 4096)
    k_attn_bwd_join<T, DP, KV, kAll><<<dim3((unsigned)((n + kAll - 1) / kAll), KV ? 2 : 1), 256, 0, s>>>(a);
  else
    k_attn_bwd_join<T, DP, KV, 1><<<dim3((unsigned)n, KV ? 2 : 1), 256, 0, s>>>(a);
  return hipGetLastError();
}

// Each launch is checked before the next: the keys' kernel takes addresses by what the rows' kernel leaves.
template <typename T, int DP>
hipError_t bwd_launch(AttnArgs a, int q_splits, int kv_splits, hipStream_t s) {
  const int64_t nbh = (int64_t)a.batch * a.kv_heads, vecs = nbh * a.rows;
  if (nbh == 0 || (a.rows == 0 && a.k_len == 0)) return hipSuccess;
  hipError_t e = hipSuccess;
  if (vecs) {
    a.splits = q_splits;
    k_attn_bwd_q<T, DP><<<(unsigned)(nbh * ((a.rows + 127) / 128) * q_splits), 256, 0, s>>>(a);
    e = hipGetLastError();
    if (e == hipSuccess && q_splits > 1) e = bwd_join<T, DP, false>(a, vecs, s);
    if (e != hipSuccess) return e;
  }
  if (nbh && a.k_len) {
    a.splits = kv_splits;
    k_attn_bwd_kv<T, DP><<<(unsigned)(nbh * ((a.k_len + 127) / 128) * kv_splits), 256, 0, s>>>(a);
    e = hipGetLastError();
    if (e == hipSuccess && kv_splits > 1) e = bwd_join<T, DP, true>(a, nbh * a.k_len, s);
  }
  return e;
}

}  // namespace

hipError_t launch_attn_bwd(AttnArgs a, int type, int q_splits, int kv_splits, hipStream_t s) {
  switch (attn_padded(a.d) + type) {
    case 32 + GS_BF16: return bwd_launch<__bf16, 32>(a, q_splits, kv_splits, s);
    case 64 + GS_BF16: return bwd_launch<__bf16, 64>(a, q_splits, kv_splits, s);
    case 96 + GS_BF16: return bwd_launch<__bf16, 96>(a, q_splits, kv_splits, s);
    case 128 + GS_BF16: return bwd_launch<__bf16, 128>(a, q_splits, kv_splits, s);
    case 32 + GS_F32: return bwd_launch<float, 32>(a, q_splits, kv_splits, s);
    case 64 + GS_F32: return bwd_launch<float, 64>(a, q_splits, kv_splits, s);
    case 96 + GS_F32: return bwd_launch<float, 96>(a, q_splits, kv_splits, s);
    default: return bwd_launch<float, 128>(a, q_splits, kv_splits, s);
  }
}

}  // namespace gs
