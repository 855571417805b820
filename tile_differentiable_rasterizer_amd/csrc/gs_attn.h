// gs_attn.h -- what the forward and backward attention kernels share.  Internal to libgsraster.
//
// The query heads that share a key head are rows of one problem: row r of (sequence b, key head
// hk) is query token r / G of head hk G + r % G, so a token's heads are neighbours in memory and
// in a tile, and a tile's rows see nearly the same keys.
#pragma once

#include "gs_device.h"
#include "gs_lds.h"
#include "gs_mfma.h"

namespace gs {

struct AttnArgs {
  gs_heads q, k, v, out, dout, dq, dk, dv;
  int32_t batch, q_len, k_len, kv_heads, group, d;
  int32_t rows;    // q_len * group
  int32_t splits;  // of the long axis: keys (out, dq) or rows (dk, dv)
  float scale;
  float slope;     // |scale| log2(e); forward 1 for a scale of 0, whose scores are made of zeros
  uint32_t flip;   // sign of the scale, to be put on the queries: 0 or the sign bits of a register
  const int32_t* ranges;
  int64_t ranges_b, ranges_r;
  const uint8_t* mask;
  int64_t mask_b;
  float* lse;
  float2* stat;    // [batch * kv_heads][tiles * 64]: (lse in base 2, delta) of each row, (inf, 0) where it sees nothing
  struct RowTile* row_tiles;  // [batch * kv_heads][tiles of 64 rows]
  const int32_t* order;  // blocks of 128 rows (sequence, block), longest first; NULL: by number
  float* part;     // [splits][batch * kv_heads][rows][DP] sums, where splits > 1
  float2* part_ml; // [splits][batch * kv_heads][rows]: running maximum (base 2), sum
};

// What the rows of a tile may see (backward pass).
struct RowTile {
  uint64_t word;        // rows that see something
  int first, last;      // some row sees something in here
  int all_from, all_to; // every row that sees anything sees all of this
};

template <typename T>
__device__ __forceinline__ T* head_ptr(const gs_heads& x, int b, int t, int h) {
  return static_cast<T*>(x.data) + b * x.batch_stride + t * x.token_stride + h * x.head_stride;
}

// The keys that query row i of sequence b may see, [first, last) inside [0, k_len).
__device__ __forceinline__ int2 row_range(const AttnArgs& a, int b, int i) {
  int2 r = make_int2(0, a.k_len);
  if (a.ranges) {
    const int64_t at = 2 * (b * a.ranges_b + i * a.ranges_r);
    r.x = max(a.ranges[at], 0);
    r.y = min(a.ranges[at + 1], a.k_len);
  }
  return r;
}

// Bits of the 64 keys from k0 that exist and are not masked, the same in every lane.
__device__ __forceinline__ uint64_t key_word(const AttnArgs& a, int b, int k0) {
  const int key = k0 + (int)__lane_id();
  bool ok = key < a.k_len;
  if (ok && a.mask) ok = a.mask[b * a.mask_b + key] != 0;
  return __ballot(ok);
}

// Bits of the 64 keys from k0 that lie in [first, last).
__device__ __forceinline__ uint64_t range_word(int first, int last, int k0) {
  const int lo = max(first - k0, 0), hi = min(last - k0, 64);
  if (lo >= hi) return 0;
  return (~0ull >> (64 - (hi - lo))) << lo;
}

// A value that is the same in every lane, in scalar registers: what is decided by it is decided once.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  return (uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x);
}

__device__ __forceinline__ int wave_min_i(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = min(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ int wave_max_i(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = max(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ uint64_t wave_or(uint64_t x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x |= __shfl_xor(x, d, 64);
  return x;
}

constexpr int kAttnKeys = 64;  // keys of a tile

// What a workgroup of the kernels that own rows works on.  Consecutive workgroups, which go to the
// XCDs in turn, take the (sequence, key head)s in turn, so that the workgroups that read the same keys
// share an XCD's L2 where there are eight of them; with an order the key heads in turn.
struct RowBlock {
  int b, hk, split, rt;
  __device__ __forceinline__ explicit RowBlock(const AttnArgs& a) {
    int rest;
    if (a.order) {
      const int each = a.kv_heads * a.splits, rank = blockIdx.x / each, blocks = (a.rows + 127) / 128;
      rest = blockIdx.x - rank * each;
      const int item = a.order[rank];
      b = item / blocks;
      rt = item - b * blocks;
      split = rest / a.kv_heads;
      hk = rest - split * a.kv_heads;
    } else {
      const int nbh = a.batch * a.kv_heads, bh = blockIdx.x % nbh;
      rest = blockIdx.x / nbh;
      rt = rest / a.splits;
      split = rest - rt * a.splits;
      b = bh / a.kv_heads;
      hk = bh - b * a.kv_heads;
    }
  }
};

// Wavefronts a SIMD of the kernels that own rows: two hide each other's waits; float32 operands of more
// than 64 elements (three registers for each of bfloat16's) leave room for one.
template <typename T, int DP>
constexpr int kWavesOf = sizeof(T) == 2 || DP <= 64 ? 2 : 1;

// Ends of the keys that the workgroup's rows may see.
struct Seen {
  int first, last;      // some row sees something in here
  int all_from, all_to; // every row that sees anything sees all of this
};
// `mine`: the range of the lane's row, empty for a row that does not exist.  Rows without ranges of
// their own need no exchange.
__device__ __forceinline__ Seen block_seen(const AttnArgs& a, int b, int2 mine, int (*scratch)[4]) {
  if (!a.ranges || a.ranges_r == 0) {
    const int2 r = row_range(a, b, 0);
    if (r.x >= r.y) return {INT32_MAX, 0, 0, INT32_MAX};
    return {r.x, r.y, r.x, r.y};
  }
  const int w = threadIdx.x >> 6;
  const bool live = mine.x < mine.y;
  const int first = wave_min_i(live ? mine.x : INT32_MAX), last = wave_max_i(live ? mine.y : 0);
  const int from = wave_max_i(live ? mine.x : 0), to = wave_min_i(live ? mine.y : INT32_MAX);
  if (__lane_id() == 0) {
    scratch[w][0] = first;
    scratch[w][1] = last;
    scratch[w][2] = from;
    scratch[w][3] = to;
  }
  __syncthreads();
  Seen s = {INT32_MAX, 0, 0, INT32_MAX};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s.first = min(s.first, scratch[i][0]);
    s.last = max(s.last, scratch[i][1]);
    s.all_from = max(s.all_from, scratch[i][2]);
    s.all_to = min(s.all_to, scratch[i][3]);
  }
  __syncthreads();
  s.first = uniform(s.first);
  s.last = uniform(s.last);
  s.all_from = uniform(s.all_from);
  s.all_to = uniform(s.all_to);
  return s;
}

// Bits of the tile's keys that some row of the workgroup sees (every thread calls it).
__device__ __forceinline__ uint64_t block_word(uint64_t mine, uint64_t* scratch) {
  const uint64_t w = wave_or(mine);
  if (__lane_id() == 0) scratch[threadIdx.x >> 6] = w;
  __syncthreads();
  const uint64_t r = scratch[0] | scratch[1] | scratch[2] | scratch[3];
  __syncthreads();
  return uniform(r);
}

// Staging of ROWS vectors to a tile by 256 threads, 16 bytes a lane straight to LDS: a wavefront's
// 64 chunks lie in a row there, and the swizzle is in the address that a lane reads.  The loads are
// in flight while the tile before is worked on, and cost no registers.
//
// Where every vector counts, the vectors are evenly spaced and D fills the tile's rows, a load's
// address is a uniform base and an offset that the thread keeps from start to end.  Elsewhere each
// lane's address is made for it, and lanes of vectors that do not count, or of chunks past D, read
// zeros: nothing is read from there.
template <typename T, int DP, int ROWS>
struct Stage;

template <int DP, int ROWS>
struct Stage<__bf16, DP, ROWS> {
  using T = __bf16;
  using Ti = Tile<T, DP>;
  static constexpr int kEach = ROWS * Ti::kChunks / 256;
  static constexpr int kBytes = ROWS * Ti::kRowBytes;
  static constexpr int kBuffers = 2;  // tiles held: the next one's loads go to the other
  static_assert(kEach * 256 == ROWS * Ti::kChunks, "whole chunks a thread");
  // one offset serves all of a thread's chunks where they are whole rounds of the swizzle apart
  static constexpr bool kRegular = kEach == 1 || (256 % Ti::kChunks == 0 && 256 / Ti::kChunks % 16 == 0);
  static constexpr int kRound = kRegular && kEach > 1 ? 256 / Ti::kChunks : ROWS;  // vectors between two chunks

  uint32_t off[kRegular ? 1 : kEach];  // bytes from the tile's first vector
  int64_t round;                       // bytes of kRound vectors
  bool even;

  // Row of the tile, and chunk of the vector, that the thread's i-th 16 bytes of the tile hold.
  static __device__ __forceinline__ int row_of(int i, int tid) { return (i * 256 + tid) / Ti::kChunks; }
  static __device__ __forceinline__ int chunk_of(int i, int tid) {
    const int c = i * 256 + tid, r = c / Ti::kChunks;
    return (c - r * Ti::kChunks) ^ Ti::mix(r);
  }

  // Vectors of `group` heads a token; they are even where a round holds whole tokens.
  __device__ __forceinline__ void plan(const gs_heads& x, int group, int d) {
    even = d == DP && kRound % group == 0 && (ROWS / group) * x.token_stride + group * x.head_stride < (1 << 28);
    round = even ? kRound / group * x.token_stride * 2 : 0;
#pragma unroll
    for (int i = 0; i < (kRegular ? 1 : kEach); ++i) {
      const int r = row_of(i, threadIdx.x), t = r / group;
      off[i] = even ? (uint32_t)(t * x.token_stride + (r - t * group) * x.head_stride + chunk_of(i, threadIdx.x) * 8) * 2u : 0;
    }
  }

  // Starts the loads of a tile.  first: its vector 0; at(r): vector r; bit r of `word`: it counts.
  template <class At>
  __device__ __forceinline__ void load(char* tile, int d, uint64_t word, const T* first, At&& at) const {
    const uint32_t to = lds_address(tile + (threadIdx.x >> 6) * 1024);
    if (even && word == (~0ull >> (64 - ROWS))) {
      const char* p = reinterpret_cast<const char*>(first);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        load_to_lds16(p, off[kRegular ? 0 : i], to + i * 4096);
        if (kRegular) p += round;
      }
    } else {
      int tid = threadIdx.x;
      asm volatile("" : "+v"(tid));  // made again here: kept from tile to tile these addresses cost the other path its registers
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = row_of(i, tid), ch = chunk_of(i, tid);
        const bool counts = ((word >> r) & 1) && ch * 8 < d;
        load_to_lds16(counts ? static_cast<const void*>(at(r) + ch * 8) : kZeros, to + i * 4096);
      }
    }
  }
  // What is left to do between the barriers when the loads are in: nothing.
  __device__ __forceinline__ void store(char*) const {}
};

// float32 tiles are made of parts (gs_mfma.h), so the loads pass through registers: they are started
// a tile ahead, split, and stored when the tile before is done with.  That splits an element once for
// the workgroup instead of once for each of its wavefronts, and makes one tile in LDS enough.
template <int DP, int ROWS>
struct Stage<float, DP, ROWS> {
  using T = float;
  using Ti = Tile<float, DP>;
  using Part = typename Ti::Part;
  static constexpr int kEach = ROWS * Part::kChunks / 256;  // eights of elements a thread
  static constexpr int kBytes = 3 * Ti::kPart;
  static constexpr int kBuffers = 1;
  static_assert(ROWS == 64 && kEach * 256 == ROWS * Part::kChunks, "tiles of 64 rows, whole eights a thread");

  f32x8 x[kEach];

  __device__ __forceinline__ void plan(const gs_heads&, int, int) {}

  template <class At>
  __device__ __forceinline__ void load(char*, int d, uint64_t word, const T*, At&& at) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = i * 256 + (int)threadIdx.x, r = c / Part::kChunks, e = (c - r * Part::kChunks) * 8;
      float y[8] = {};
      if (((word >> r) & 1) && e < d) load_elems<8>(at(r) + e, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = y[j];
    }
  }
  __device__ __forceinline__ void store(char* tile) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = i * 256 + (int)threadIdx.x, r = c / Part::kChunks;
      const Frag<float> f = frag_split(x[i]);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<bf16x8*>(tile + k * Ti::kPart + Part::at(r, c - r * Part::kChunks)) = f.p[k];
    }
  }
};

// Two tensors' tiles that are worked on together, in LDS that the kernel declares: tiles[kTiles][kBytes].
template <typename T, int DP, int ROWS>
struct Pair {
  using St = Stage<T, DP, ROWS>;
  static constexpr int kBytes = St::kBytes, kTiles = 2 * St::kBuffers;
  St a, b;

  // Before a tile is worked on: its loads are in (wait_loads: every load that the thread has started),
  // and nobody works on the tile before any more.
  __device__ __forceinline__ void ready(char (*tiles)[kBytes]) {
    if constexpr (St::kBuffers == 1) {
      __syncthreads();
      a.store(tiles[0]);
      b.store(tiles[1]);
    }
    wait_loads();
    __syncthreads();
  }
  // Tile `which` (0: a's, 1: b's) of buffer `buf`.
  static __device__ __forceinline__ char* at(char (*tiles)[kBytes], int buf, int which) {
    return tiles[St::kBuffers == 2 ? 2 * buf + which : which];
  }
};

// The tiles of a workgroup's keys, one after another, without those that no row sees.  Every
// thread of the workgroup calls next() (its answer is the same for all of them).
struct Tiles {
  int t, end;       // next to look at, past the last
  int k0;           // the tile's first key
  uint64_t word;    // keys that some row sees (0: no tile left)
  bool ragged;      // some row sees only a part of them by its range

  __device__ __forceinline__ void next(const AttnArgs& a, int b, const Seen& seen, int2 mine, uint64_t* scratch) {
    word = 0;
    for (; t < end && word == 0; ++t) {
      k0 = t * kAttnKeys;
      word = a.mask || k0 + kAttnKeys > a.k_len ? key_word(a, b, k0) : ~0ull;
      ragged = k0 < seen.all_from || k0 + kAttnKeys > seen.all_to;
      if (ragged) {
        if (a.ranges_r == 0)  // the same range for all rows
          word &= range_word(seen.first, seen.last, k0);
        else
          word &= block_word(range_word(mine.x, mine.y, k0), scratch);
      }
    }
  }
};

}  // namespace gs
