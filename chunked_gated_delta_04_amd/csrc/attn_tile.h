// Device helpers of the attention kernels: which rows and keys a workgroup has,
// and a tile's way from memory into LDS.
#pragma once

#include <limits.h>

#include <utility>

#include "attn.h"

namespace gdn {

constexpr float kMinusInf = -INFINITY;

// f(0), f(1), .. f(N - 1) with compile-time numbers: register arrays are then indexed by constants
// however long the body is.
template <int... I, class F>
__device__ __forceinline__ void for_each_of(std::integer_sequence<int, I...>, const F& f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void for_each(const F& f) {
  for_each_of(std::make_integer_sequence<int, N>(), f);
}

// A tile of a pack's query rows: tokens first .. first + tokens - 1 of a sequence of `len` tokens that
// begins at bos.
struct RowTile {
  int seq, bos, len, first, tokens;
};

// Tile i of sequence n has the slot cu[n] / per + n + i (per tokens a tile), so that a tile's place
// follows from cu_seqlens alone; the sequence is the last one whose first slot is at or before
// this, found by all lanes of a wave together, 64 probes a step. tokens <= 0: no tile has the slot.
// Boundaries are clamped to [0, T], so a bad one never leads out of range.
__device__ __forceinline__ RowTile find_tile(const int32_t* cu, int N, int T, int per, int slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = N;
  while (cnt > 1) {
    const int step = (cnt + 63) >> 6, at = lane * step;
    bool ok = false;
    if (at < cnt) ok = min(max(cu[lo + at], 0), T) / per + lo + at <= slot;
    const int k = max(__popcll(__ballot(ok)) - 1, 0);
    lo += k * step;
    cnt = min(step, cnt - k * step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  RowTile t;
  t.seq = lo;
  t.bos = __builtin_amdgcn_readfirstlane(min(max(cu[lo], 0), T));
  t.len = __builtin_amdgcn_readfirstlane(min(max(cu[lo + 1], t.bos), T)) - t.bos;
  const int i = slot - t.bos / per - lo;
  t.first = i >= 0 ? i * per : t.len;
  t.tokens = min(per, t.len - t.first);
  return t;
}

// The tile of number `item`, the one with the most work first: up to 64 sequences are taken in the order of their keys
// (before(n): those that sequence n had before), a wave comparing all of them, and a sequence's tiles from the last on
// (back) or from the first. More sequences are taken in the pack's order. (8 prompts of 512 tokens, four of them after 1000
// to 2000: in the pack's order 5 % more.)
template <class Before>
__device__ __forceinline__ RowTile tile_of(const int32_t* cu, int N, int T, int per, int slots, int item, bool back,
                                           const Before& before) {
  if (N > 64) return find_tile(cu, N, T, per, back ? slots - 1 - item : item);
  const int lane = threadIdx.x & 63;
  int bos = 0, len = 0, keys = INT_MIN;
  if (lane < N) {
    bos = min(max(cu[lane], 0), T);
    len = min(max(cu[lane + 1], bos), T) - bos;
    keys = len + before(lane);
  }
  const int tiles = (len + per - 1) / per;
  int first = 0;  // tiles of the sequences before this lane's
  for (int n = 0; n < N; ++n) {
    const int k = __builtin_amdgcn_readlane(keys, n), t = __builtin_amdgcn_readlane(tiles, n);
    if (k > keys || (k == keys && n < lane)) first += t;
  }
  const uint64_t mine = __ballot(lane < N && item >= first && item < first + tiles);
  RowTile t{0, 0, 0, 0, 0};
  if (mine == 0) return t;
  t.seq = __builtin_ctzll(mine);
  t.bos = __builtin_amdgcn_readlane(bos, t.seq);
  t.len = __builtin_amdgcn_readlane(len, t.seq);
  const int i = item - __builtin_amdgcn_readlane(first, t.seq);
  t.first = (back ? __builtin_amdgcn_readlane(tiles, t.seq) - 1 - i : i) * per;
  t.tokens = min(per, t.len - t.first);
  return t;
}

// The key tiles that queries at positions lo .. hi (hi the last) may see, kT keys each, of `keys` keys:
// those with sinks, then those from the first one in a window on. (lo and hi may be negative.)
struct KeyTiles {
  int sinks, first, count;
  __device__ __forceinline__ int at(int i) const { return i < sinks ? i : first + i - sinks; }
};
template <int kT>
__device__ __forceinline__ KeyTiles key_tiles(int lo, int hi, int64_t keys, int window, int sinks) {
  const int end = (int)min((int64_t)hi + 1, keys);
  const int all = end > 0 ? (int)(((int64_t)end + kT - 1) / kT) : 0;
  KeyTiles k;
  k.first = window ? min(max((int64_t)lo + 1 - window, (int64_t)0) / kT, (int64_t)all) : 0;
  k.sinks = window ? min((int)(((int64_t)sinks + kT - 1) / kT), k.first) : 0;
  k.count = k.sinks + all - k.first;
  return k;
}
// parts of the tiles: this split's first and end
__device__ __forceinline__ int2 split_of(int count, int splits, int split, int least) {
  const int per = max((count + splits - 1) / splits, least);
  const int64_t from = (int64_t)per * split;
  return make_int2((int)min(from, (int64_t)count), (int)min(from + per, (int64_t)count));
}

// Tokens that a sequence had before, so that the positions of T more, rounded up to a tile, are 32 bits
// whatever the caller's array holds.
__device__ __forceinline__ int past_of(const KvPages& c, int seq, int T) {
  return min(max(c.offsets[seq], -(1 << 30)), 0x7fffff00 - T);
}
// Element offset of the row of position j of a sequence in the cache, or -1 where it has none.
__device__ __forceinline__ int64_t row_at(const KvPages& c, int seq, int j, int64_t keys) {
  if (j < 0 || j >= keys) return -1;
  const int col = divide(j, c.page);
  if (col >= c.columns) return -1;
  const int id = c.table[seq * c.table_stride + col];
  return id > 0 && id < c.pages ? id * c.page_stride + (j - col * c.page.by) * c.token_stride : -1;
}
// what rows without a place are read from
__device__ const uint4 zeros[1] = {};
typedef __attribute__((address_space(1))) const void Global;
__device__ __forceinline__ uint4 load16(Global* p) {
  const u32x4 x = *(__attribute__((address_space(1))) const u32x4*)p;
  return make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ int64_t from_lane(int64_t x, int lane) {
  const int lo = __shfl((int)x, lane), hi = __shfl((int)(x >> 32), lane);
  return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

// kT rows of D elements from memory into LDS by kThreads threads, 16 bytes a lane, without a stop in
// registers: request i of a wave fills the 64 pieces from (i waves + wave) 64 on, each lane fetching
// the piece of its row that belongs there (see piece_of). A barrier waits for them. Buffers that are filled while
// others are read are variables of their own: the compiler waits for a request in flight before any read
// of the same variable.
template <int D, int kT, int kThreads>
struct Tile {
  static constexpr int kPieces = kT * D / 8 / kThreads, kRows = kThreads / (D / 8);  // rows a request of all threads
  static_assert(kPieces * kThreads * 8 == kT * D, "whole requests");
  typedef uint16_t Lds[kT * D];
  static __device__ __forceinline__ int row(int i, int tid) { return tid / (D / 8) + i * kRows; }
  static __device__ __forceinline__ int column(int i, int tid) {
    return (tid % (D / 8) ^ piece_of<D>(row(i, tid))) * 8;
  }
  static __device__ __forceinline__ __attribute__((address_space(3))) void* to(Lds& tile, int i, int tid) {
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    return (__attribute__((address_space(3))) void*)(tile + (i * (kThreads / 64) + wave) * 64 * 8);
  }
  static __device__ __forceinline__ void request(Lds& tile, int i, __amdgpu_buffer_rsrc_t r, int byte_off, int tid) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to(tile, i, tid), 16, byte_off, 0, 0, 0);
  }
  // Of a cache's rows at p: this lane's at an element offset, or -1 for zeros. `rows` in lane r of each wave is where row r of
  // the tile is; a request's offset is exchanged (place) some time before it goes out.
  static __device__ __forceinline__ int64_t place(int64_t rows, int i, int tid) { return from_lane(rows, row(i, tid) & 63); }
  static __device__ __forceinline__ void request_page(Lds& tile, int i, const uint16_t* p, int64_t off, int tid) {
    Global* from = off >= 0 ? (Global*)(p + off + column(i, tid)) : (Global*)zeros;
    __builtin_amdgcn_global_load_lds(from, to(tile, i, tid), 16, 0, 0);
  }
  // The same where the rows of a wave's request, at most 8, are in one page and less than 2^24 elements apart: their place is
  // uniform, and so costs no vector work. `lane` is this lane's byte offset in them, `keys` how many rows of the tile are there.
  static constexpr int kGroup = 512 / D;
  static __device__ __forceinline__ int in_group(int i, int stride, int tid) {
    return ((tid & 63) / (D / 8) * stride + column(i, tid)) * 2;
  }
  static __device__ __forceinline__ void request_group(Lds& tile, int i, const uint16_t* p, int64_t rows, int keys, int stride,
                                                       int lane, int tid) {
    const int first = (i * (kThreads / 64) + __builtin_amdgcn_readfirstlane(tid >> 6)) * kGroup;
    const int lo = __builtin_amdgcn_readlane((int)rows, first), hi = __builtin_amdgcn_readlane((int)(rows >> 32), first);
    const int64_t off = (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
    const int n = off >= 0 ? min(keys - first, kGroup) : 0;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p) + (off >= 0 ? off : 0), 0,
                                                                      n > 0 ? ((n - 1) * stride + D) * 2 : 0, kBufferWord3);
    request(tile, i, r, lane, tid);
  }
};
// whether request_group holds for a call
inline bool in_groups(const AttnArgs& a) {
  return a.pages.page.by % 8 == 0 && a.pages.token_stride < (1 << 24) && !a.pack.window;
}

// Requests for token rows at a stride: a lane's byte offsets of request 0 (and of request 1 less a step, where the
// permutation differs), the others a step of kRows rows apart each.
template <class Tile>
struct TokenRows {
  int lane[2], step;
  __device__ __forceinline__ TokenRows(int stride, int tid) {
    step = Tile::kRows * stride * 2;
    lane[0] = (Tile::row(0, tid) * stride + Tile::column(0, tid)) * 2;
    lane[1] = lane[0] + (Tile::column(1, tid) - Tile::column(0, tid)) * 2;
  }
  // rows [0, len) from p; the others are past the resource: zeros
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t from(const uint16_t* p, int stride, int len, int D) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, len > 0 ? ((len - 1) * stride + D) * 2 : 0,
                                             kBufferWord3);
  }
  __device__ __forceinline__ void request(typename Tile::Lds& tile, int i, __amdgpu_buffer_rsrc_t r, int tid) const {
    Tile::request(tile, i, r, fresh(lane[i % 2]) + i * step, tid);
  }
};
// 16 bytes for each lane from the accumulator of 32 x 32: rows 8 b + 4 (lane / 32) + r are columns of
// the output. Lanes 0-31 get the 8 columns of b = 2 u, lanes 32-63 those of b = 2 u + 1.
template <typename T>
__device__ __forceinline__ uint4 eight_columns(const f32x16& x, int u, float f) {
  uint32_t a[2], b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = pack2<T>(x[8 * u + 2 * i] * f, x[8 * u + 2 * i + 1] * f);
    b[i] = pack2<T>(x[8 * u + 4 + 2 * i] * f, x[8 * u + 5 + 2 * i] * f);
    const auto s = __builtin_amdgcn_permlane32_swap(a[i], b[i], false, false);
    a[i] = s[0];
    b[i] = s[1];
  }
  return make_uint4(a[0], a[1], b[0], b[1]);
}
// Keeps an accumulator where it is between the steps of a loop: in the accumulation registers where a wave
// has a SIMD to itself (kAcc). The compiler's own choice moved it to other registers and back every
// step, and spilled what they held.
template <bool kAcc>
__device__ __forceinline__ void keep_accumulated(f32x16& x) {
  if constexpr (kAcc) asm volatile("" : "+a"(x));
  else asm volatile("" : "+v"(x));
}
// a lane's value and the other half's
__device__ __forceinline__ float2 both_halves(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return make_float2(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const float2 y = both_halves(x);
  return y.x + y.y;
}

// Operand of a second product from the accumulator of the first: rows 16 h .. 16 h + 15 of it in the order
// that transposing reads at rows 4 (lane / 32) and 8 + 4 (lane / 32) take.
template <typename T>
__device__ __forceinline__ uint4 operand(const f32x16& x, int h) {
  return make_uint4(pack2<T>(x[8 * h], x[8 * h + 1]), pack2<T>(x[8 * h + 2], x[8 * h + 3]),
                    pack2<T>(x[8 * h + 4], x[8 * h + 5]), pack2<T>(x[8 * h + 6], x[8 * h + 7]));
}
// Values whose place among the matrix instructions the compiler keeps: it moves what no instruction of a
// block needs to the blocks behind it.
__device__ __forceinline__ void stay_here(uint4& x) { asm volatile("" : "+v"(x.x), "+v"(x.y), "+v"(x.z), "+v"(x.w)); }
__device__ __forceinline__ void stay_here(float& x, float& y) { asm volatile("" : "+v"(x), "+v"(y)); }
__device__ __forceinline__ void zero16(f32x16& x) {
#pragma unroll
  for (int r = 0; r < 16; ++r) x[r] = 0.f;
}

}  // namespace gdn
