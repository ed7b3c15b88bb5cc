// Host- and device-side declarations of the operators around the recurrences:
// rotary positions and the root-mean-square norm. Their tensors are bf16, fp16
// or fp32, computed in fp32.
#pragma once

#include <hip/hip_fp16.h>

#include <type_traits>

#include "gdn_common.h"

namespace gdn {

// element types, numbered as gdn_dtype
enum class Elem : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

struct Bf16 {
  uint16_t u;
};
struct Fp16 {
  uint16_t u;
};

__device__ __forceinline__ float to_f32(Bf16 x) { return bf2f(x.u); }
__device__ __forceinline__ float to_f32(Fp16 x) { return (float)__builtin_bit_cast(_Float16, x.u); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float x) { return {f2bf(x)}; }
template <>
__device__ __forceinline__ Fp16 from_f32<Fp16>(float x) { return {__builtin_bit_cast(uint16_t, (_Float16)x)}; }
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

// N consecutive elements as fp32: 16 bytes at once where N elements are 16
// bytes (p 16-byte aligned), else element by element.
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float* x) {
  if constexpr (N * sizeof(T) == 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(p[i]);
  }
}
// 16 bytes of T as one vector value (a struct of words, or elements one by one, the
// compiler may store in pieces)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_in __attribute__((may_alias));              // in tensors of any type
typedef u32x4 u32x4_any __attribute__((may_alias, aligned(2)));  // at any element's address
template <typename T>
__device__ __forceinline__ u32x4 pack16(const float* x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) w[i] = __float_as_uint(x[i]);
    else if constexpr (std::is_same<T, Bf16>::value) w[i] = pk2(x[2 * i], x[2 * i + 1]);
    else w[i] = from_f32<T>(x[2 * i]).u | (uint32_t)from_f32<T>(x[2 * i + 1]).u << 16;
  }
  return w;
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float* x) {
  if constexpr (N * sizeof(T) == 16) {
    *reinterpret_cast<u32x4_in*>(p) = pack16<T>(x);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = from_f32<T>(x[i]);
  }
}

// Columns c .. c + V - 1 (16 bytes) of a row of n, of any length and alignment: the
// memory path takes 16 bytes from any address. Columns past n are zeros, and not
// stored. A row's last piece is taken from its last V columns and moved down, by a
// lane without a branch for each column, and stored column by column.
template <typename T, int V>
__device__ __forceinline__ void load_any(const T* row, int c, int n, float* x) {
  static_assert(V * sizeof(T) == 16, "16 bytes");
  if (n >= V) {
    const int from = min(c, n - V);
    u32x4 w = *reinterpret_cast<const u32x4_any*>(row + from);
    if (from != c) {
      const int by = (c - from) * (int)sizeof(T);  // bytes that the columns move down
      if (by >= 16) w = u32x4{0, 0, 0, 0};
      if (by & 8) w = u32x4{w[2], w[3], 0, 0};
      if (by & 4) w = u32x4{w[1], w[2], w[3], 0};
      if (by & 2) w = w >> 16 | u32x4{w[1], w[2], w[3], 0} << 16;
    }
    T e[V];
    __builtin_memcpy(e, &w, sizeof(e));
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = c + i < n ? to_f32(row[c + i]) : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_any(T* row, int c, int n, const float* x) {
  const u32x4 w = pack16<T>(x);
  if (c + V <= n) {
    *reinterpret_cast<u32x4_any*>(row + c) = w;
  } else {
    T e[V];
    __builtin_memcpy(e, &w, sizeof(e));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < n) row[c + i] = e[i];
  }
}

// One set of rows [T, heads, D] of the rotary operator: in and out may be the same.
struct RotaryRows {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;  // elements between tokens
  int heads;
};

struct RotaryArgs {
  int T, D, R;
  float mscale, sign;  // sign -1: the transposed turn
  const float* inv_freq;
  const int32_t* positions;  // [T], or null: by the sequences
  int N;
  const int32_t* cu;
  const int32_t* offsets;  // [N] or null
  RotaryRows q, k;
};

// wide: whole pieces of 16 bytes, aligned (the caller has checked extents and alignment)
hipError_t launch_rotary(Elem type, bool interleaved, bool wide, const RotaryArgs& a, hipStream_t s);

struct NormArgs {
  int rows, D;
  float eps, unit;  // the weight's offset
  int group;        // columns a scale: 0 none (no e4m3 output), D a row, or 128
  const void *x, *residual, *weight;
  int64_t x_stride, residual_stride;
  void *residual_out, *y;
  uint8_t* y8;
  float *scales, *rstd;
};
hipError_t launch_rmsnorm_fwd(Elem type, bool wide, const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  int rows, D;
  float unit;
  const void *s, *weight, *dy, *ds;
  const float* rstd;
  int64_t s_stride;
  void* dx;
  float *dweight, *partial;  // partial: [norm_partials, norm_pitch(D)], or null without dweight
};
// columns of a partial sum's row: whole pieces of any type
__host__ __device__ constexpr int norm_pitch(int D) { return (D + 7) / 8 * 8; }
// threads of the forward's launch
int64_t norm_threads(int rows, int D);
// row groups that each sum one partial of dweight
int norm_partials(int rows, int D);
hipError_t launch_rmsnorm_bwd(Elem type, bool wide, const NormGradArgs& a, hipStream_t s);

constexpr int kNormMaxD = 16384;

}  // namespace gdn
