// Host- and device-side declarations of the softmax attention and its paged
// key-value cache. Tensors are bf16 or fp16, computed in fp32.
#pragma once

#include <hip/hip_fp16.h>

#include "lds_tile.h"
#include "layer.h"

namespace gdn {

// n / divisor for 0 <= n < 2^31: magic = ceil(2^(31 + s) / divisor) with 2^s >= divisor, so the
// product is off by less than n 2^s < 2^(31 + s) and the quotient is exact.
struct Divisor {
  uint32_t magic;
  int shift, by;
};
inline Divisor divisor(int by) {
  int s = 0;
  while (((int64_t)1 << s) < by) ++s;
  return {(uint32_t)((((uint64_t)1 << (31 + s)) + by - 1) / by), 31 + s, by};
}
__device__ __forceinline__ int divide(int n, const Divisor& d) {
  return (int)(((uint64_t)(uint32_t)n * d.magic) >> d.shift);
}

// Pages of keys and values: the token at position j of sequence n is row j % page of page
// table[n * table_stride + j / page], head h at + h * head_stride. A page that is not in
// 1 .. pages - 1, or past the table's columns, is none: its tokens are not seen and not written.
struct KvPages {
  void *k, *v;
  int64_t page_stride, token_stride, head_stride, table_stride;  // elements
  const int32_t* table;
  const int32_t* offsets;  // [N] tokens that a sequence had before
  int pages, columns;
  Divisor page;
};

// Query rows of a pack. The G query heads of a key head are rows of one matrix: row r of a sequence
// is token r / G, head r % G, so that a tile of rows shares its keys between heads.
struct AttnPack {
  const int32_t* cu;
  int N, T, HQ, HK;
  Divisor G;
  int window, sinks;  // window 0: none
  float scale;
};

struct AttnArgs {
  AttnPack pack;
  KvPages pages;  // paged
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  void* o;           // [T, HQ, D]
  float* lse;        // [T, HQ] or null
  int splits;        // parts of the keys that go to workgroups of their own, joined afterwards
  float* part;       // [splits][T * HQ][D]: sums of weights times values, then [splits][T * HQ][2]: their
                     // largest score (base 2) and weight sum
  int slots;         // row tiles: T / (tokens a tile) + N
};

struct AttnGradArgs {
  AttnPack pack;
  const void *q, *k, *v, *o, *dO;
  int64_t q_stride, k_stride, v_stride;
  const float* lse;
  float* stats;  // [grad_stats][T, HQ]: of each row, lse in base 2 (infinite where it sees nothing), scale dO . o,
                 // with fp16 its largest score gradient
  void *dq, *dk, *dv;
  int slots;                 // row tiles
  int key_slots;             // key tiles
  int pieces;                // parts of a key tile's rows
  // parts of the rows that see a sequence's sinks from behind the window; its key tiles with sinks; all those tiles' places
  int far_pieces, far_tiles, far_slots;
  float *part, *far;         // partial dk and dv
};

// rows of a workgroup's tile, 32 to a wave; with 256 columns a wave has a SIMD's registers to itself
constexpr int attn_rows(int D) { return D == 256 ? 128 : 256; }
// keys of a workgroup's tile in the backward: 32 to a wave, from 128 columns on to two
constexpr int attn_keys(int D) { return D == 256 ? 64 : 128; }
constexpr int kAttnGroup = 128; // most query heads to a key head
// whether the backward's score gradients are multiplied in units of their own: where the type's range is short
template <typename T>
constexpr bool kHasUnits = std::is_same<T, Fp16>::value;
// log2 of a row's largest weight where weights are rounded: above 1 in fp16, so that those far below it are not lost
template <typename T>
constexpr float weight_lift(int fp16) { return std::is_same<T, Fp16>::value ? (float)fp16 : 0.f; }
constexpr int grad_stats(Elem type) { return type == Elem::kFp16 ? 3 : 2; }

hipError_t launch_attn_fwd(Elem type, int D, bool paged, const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_step(Elem type, int D, const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_join(Elem type, int D, const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bwd(Elem type, int D, const AttnGradArgs& a, hipStream_t s);

struct AppendArgs {
  int T, N, D, R;
  float mscale;
  const float* inv_freq;
  const int32_t* cu;  // null: token t is sequence t's
  RotaryRows q, k;    // k's results go to the cache
  const void* v;
  int64_t v_stride;
  KvPages pages;
};
hipError_t launch_kv_append(Elem type, bool interleaved, bool wide, const AppendArgs& a, hipStream_t s);

// ---------------------------------------------------------------- matrix instructions of both types
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <typename T>
__device__ __forceinline__ f32x16 mfma32_of(const uint4& a, const uint4& b, const f32x16& c) {
  if constexpr (std::is_same<T, Bf16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ f32x4 mfma16_of(const uint4& a, const uint4& b, const f32x4& c) {
  if constexpr (std::is_same<T, Bf16>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, Bf16>::value) return pk2(a, b);
  else return from_f32<T>(a).u | (uint32_t)from_f32<T>(b).u << 16;
}

}  // namespace gdn
