// Device helpers of the kernels that turn head rows by rotary positions.
#pragma once

#include "layer.h"

namespace gdn {

// Cosine and sine of position * freq. The angle of a far position needs more than
// fp32: at position 10^6 the product's rounding alone is 0.03 radians. It is formed
// in fp64 and its whole turns are taken off before the sine and cosine.
__device__ __forceinline__ float2 turn_of(int64_t position, float freq) {
  const double turns = (double)position * (double)freq * 0.15915494309189533577;
  float s, c;
  sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
  return make_float2(c, s);
}

// Units of a head row, 16 bytes (V columns) each: those of the turning columns, or
// of their first half, whose unit takes the same columns of the second half with it,
// and those of the copied columns.
template <int V, bool kInter>
__host__ __device__ __forceinline__ int turning_units(int R) {
  return ((kInter ? R : R / 2) + V - 1) / V;
}
template <int V>
__host__ __device__ __forceinline__ int copied_units(int D, int R) {
  return (D - R + V - 1) / V;
}

template <typename T, int V, bool kWide>
__device__ __forceinline__ void load_unit(const T* row, int c, int n, float* x) {
  if constexpr (kWide) load_n<T, V>(row + c, x);
  else load_any<T, V>(row, c, n, x);
}
template <typename T, int V, bool kWide>
__device__ __forceinline__ void store_unit(T* row, int c, int n, const float* x) {
  if constexpr (kWide) store_n<T, V>(row + c, x);
  else store_any<T, V>(row, c, n, x);
}

// Unit u of a head row. (In place, load_any may read columns that another unit is
// writing; it drops those.)
template <typename T, int V, bool kInter, bool kWide>
__device__ __forceinline__ void unit(const T* in, T* out, const float2* cs, int u, int turning, int D, int R) {
  if (u >= turning) {
    const int c = (u - turning) * V;
    float x[V];
    load_unit<T, V, kWide>(in + R, c, D - R, x);
    store_unit<T, V, kWide>(out + R, c, D - R, x);
    return;
  }
  const int c = u * V;
  const auto turn = [&](int j) { return cs[kWide ? j : min(j, R / 2 - 1)]; };
  if constexpr (kInter) {
    float x[V], y[V];
    load_unit<T, V, kWide>(in, c, R, x);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 t = turn(u * (V / 2) + i / 2);
      y[i] = x[i] * t.x - x[i + 1] * t.y;
      y[i + 1] = x[i] * t.y + x[i + 1] * t.x;
    }
    store_unit<T, V, kWide>(out, c, R, y);
  } else {
    float x0[V], x1[V], y0[V], y1[V];
    load_unit<T, V, kWide>(in, c, R / 2, x0);
    load_unit<T, V, kWide>(in + R / 2, c, R / 2, x1);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 t = turn(c + i);
      y0[i] = x0[i] * t.x - x1[i] * t.y;
      y1[i] = x0[i] * t.y + x1[i] * t.x;
    }
    store_unit<T, V, kWide>(out, c, R / 2, y0);
    store_unit<T, V, kWide>(out + R / 2, c, R / 2, y1);
  }
}

}  // namespace gdn
