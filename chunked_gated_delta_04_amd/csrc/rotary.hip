// Rotary positions: the first R columns of every head row turn, in pairs, by
// position * inv_freq[j], q's and k's heads in one launch. Pair j is columns
// (j, j + R/2), or interleaved (2 j, 2 j + 1); the other columns are copied.
// The gradient is the turn back, so the backward is the same kernel with the
// sine's sign changed.
//
// The angle of a far position needs more than fp32: at position 10^6 the
// product's rounding alone is 0.03 radians. position * inv_freq is formed in
// fp64 and its whole turns are taken off before the sine and cosine, once for
// each (token, pair) and shared by all heads through LDS.
//
// Bound by HBM: every element is read and written once. q and k of 16384 tokens,
// 32 + 32 heads of 128 in bf16 (537 MB): 91 us, 5.9 TB/s.
#include <algorithm>

#include "layer.h"

namespace gdn {

namespace {

// Tokens per workgroup where one token's units would leave most of its 256 threads
// idle (at most 64 units; one wave then makes a token's angles). 16384 tokens of 4 +
// 1 heads of 64 columns, 20 units: 8.1 us, and 12.2 with one token; 32 + 32 heads
// of 128, 512 units: 113 us, and 100 with one; 256 tokens of these: 7.5 and 4.3.
constexpr int kTok = 4;

struct TokenAt {
  int64_t pos;
  bool live;
};
// Position of token t: given, or its place in its sequence plus the sequence's
// offset. Boundaries are only compared, never used as addresses.
__device__ __forceinline__ TokenAt token_at(const RotaryArgs& a, int t) {
  if (a.positions) return {a.positions[t], true};
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = a.N;
  while (cnt > 1) {  // the last sequence that begins at or before t, 64 probes a step
    const int step = (cnt + 63) >> 6, at = lane * step;
    const bool ok = at < cnt && a.cu[lo + at] <= t;
    const int k = max(__popcll(__ballot(ok)) - 1, 0);
    lo += k * step;
    cnt = min(step, cnt - k * step);
  }
  const int b = a.cu[lo];
  return {(int64_t)(t - b) + (a.offsets ? a.offsets[lo] : 0), t >= b && t < a.cu[lo + 1]};
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

}  // namespace

// Tokens first .. T - 1, as many as the grid takes.
template <typename T, int V, bool kInter, bool kWide, int kTokens>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int first) {
  extern __shared__ float2 cs[];  // [kTokens][R / 2]
  __shared__ bool live[kTokens];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int t0 = first + blockIdx.x * kTokens, pairs = a.R / 2;
  // a wave for each token, or all four for one
  const int mine = kTokens == 1 ? 0 : wave;
  if (t0 + mine < a.T) {
    const TokenAt at = token_at(a, t0 + mine);
    if (lane == 0) live[mine] = at.live;
    for (int j = kTokens == 1 ? tid : lane; j < pairs; j += kTokens == 1 ? 256 : 64) {
      const double turns = (double)at.pos * (double)a.inv_freq[j] * 0.15915494309189533577;
      float s, c;
      sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
      cs[mine * pairs + j] = make_float2(c * a.mscale, s * a.mscale * a.sign);
    }
  }
  __syncthreads();
  const int turning = turning_units<V, kInter>(a.R), units = turning + copied_units<V>(a.D, a.R);
  const int heads = a.q.heads + a.k.heads, n = units * heads;
  for (int i = tid; i < n * kTokens; i += 256) {
    const int tok = i / n, rest = i - tok * n, head = rest / units, u = rest - head * units;
    const int64_t t = t0 + tok;
    if (t >= a.T || !live[tok]) continue;
    const bool isq = head < a.q.heads;
    const RotaryRows& r = isq ? a.q : a.k;
    const int h = isq ? head : head - a.q.heads;
    const T* in = static_cast<const T*>(r.in) + t * r.in_stride + (int64_t)h * a.D;
    T* out = static_cast<T*>(r.out) + t * r.out_stride + (int64_t)h * a.D;
    if (u >= turning && in == out) continue;  // in place: nothing to copy
    unit<T, V, kInter, kWide>(in, out, cs + tok * pairs, u, turning, a.D, a.R);
  }
}

namespace {

// A launch counts its threads in 32 bits: more tokens than these workgroups of 256
// threads take go in several launches.
constexpr int kMaxBlocks = 1 << 23;

template <typename T, int V, bool kInter, bool kWide, int kTokens>
hipError_t rotary_launches(const RotaryArgs& a, hipStream_t s) {
  const size_t lds = kTokens * sizeof(float2) * (a.R / 2);
  for (int first = 0; first < a.T; first += kMaxBlocks * kTokens) {
    const int blocks = std::min((a.T - first + kTokens - 1) / kTokens, kMaxBlocks);
    hipLaunchKernelGGL((rotary_kernel<T, V, kInter, kWide, kTokens>), dim3(blocks), dim3(256), lds, s, a, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, bool kInter, bool kWide>
hipError_t rotary_of(const RotaryArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t units = turning_units<V, kInter>(a.R) + copied_units<V>(a.D, a.R);
  if (units * (a.q.heads + a.k.heads) * kTok <= 256) return rotary_launches<T, V, kInter, kWide, kTok>(a, s);
  return rotary_launches<T, V, kInter, kWide, 1>(a, s);
}

template <typename T>
hipError_t rotary_type(bool inter, bool wide, const RotaryArgs& a, hipStream_t s) {
  if (inter) return wide ? rotary_of<T, true, true>(a, s) : rotary_of<T, true, false>(a, s);
  return wide ? rotary_of<T, false, true>(a, s) : rotary_of<T, false, false>(a, s);
}

}  // namespace

hipError_t launch_rotary(Elem type, bool inter, bool wide, const RotaryArgs& a, hipStream_t s) {
  switch (type) {
    case Elem::kBf16: return rotary_type<Bf16>(inter, wide, a, s);
    case Elem::kFp16: return rotary_type<Fp16>(inter, wide, a, s);
    default: return rotary_type<float>(inter, wide, a, s);
  }
}

}  // namespace gdn
