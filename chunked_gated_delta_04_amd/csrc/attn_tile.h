// Device helpers of the attention kernels: which rows and keys a workgroup has,
// and a tile's way from memory into LDS.
#pragma once

#include "attn.h"

namespace gdn {

constexpr float kMinusInf = -INFINITY;

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

// kT rows of D elements on their way through kThreads threads' registers into LDS, 16 bytes a piece.
template <int D, int kT, int kThreads>
struct Staged {
  static constexpr int kPieces = kT * D / 8 / kThreads, kRows = kThreads / (D / 8);  // rows a piece of all threads
  uint4 x[kPieces];
  static __device__ __forceinline__ int row(int i, int tid) { return tid / (D / 8) + i * kRows; }
  static __device__ __forceinline__ int column(int tid) { return tid % (D / 8) * 8; }
  // rows [0, len) of token rows at p; the others are zeros
  __device__ __forceinline__ void load(const uint16_t* p, int stride, int len, int tid) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p), 0, len > 0 ? ((len - 1) * stride + D) * 2 : 0, kBufferWord3);
    const int at = (row(0, tid) * stride + column(tid)) * 2;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) x[i] = load_b128(r, at + i * kRows * stride * 2);
  }
  __device__ __forceinline__ void store(uint16_t* tile, int tid) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(tile + at<D>(row(i, tid), column(tid))) = x[i];
  }
};

// Tokens that a sequence had before, so that the positions of T more, rounded up to a tile, are 32 bits
// whatever the caller's array holds.
__device__ __forceinline__ int past_of(const KvPages& c, int seq, int T) {
  return __builtin_amdgcn_readfirstlane(min(max(c.offsets[seq], -(1 << 30)), 0x7fffff00 - T));
}
// the page of the key at position j, or 0 for none
__device__ __forceinline__ int page_of(const KvPages& c, int seq, int j, int keys) {
  if (j < 0 || j >= keys) return 0;
  const int col = divide(j, c.page);
  if (col >= c.columns) return 0;
  const int id = c.table[seq * c.table_stride + col];
  return id < c.pages ? max(id, 0) : 0;
}
// offset of a row of page id > 0
__device__ __forceinline__ int64_t row_of(const KvPages& c, int id, int j) {
  return id * c.page_stride + (j - divide(j, c.page) * c.page.by) * c.token_stride;
}

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
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

}  // namespace gdn
