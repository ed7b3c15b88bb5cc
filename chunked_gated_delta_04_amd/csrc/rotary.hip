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
#include "layer.h"

namespace gdn {

namespace {

// Tokens per workgroup where one token's pieces would leave most of its 256 threads
// idle (at most 64 pieces; one wave then makes a token's angles). 16384 tokens of 4 +
// 1 heads of 64 columns, 20 pieces: 8.1 us, and 12.2 with one token; 32 + 32 heads
// of 128, 512 pieces: 113 us, and 100 with one; 256 tokens of these: 7.5 and 4.3.
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

// columns of a turning unit
template <int V, bool kInter>
constexpr int columns_of = kInter ? (V > 1 ? V : 2) : 2 * V;

// Unit u of a head row: V pairs (two loads of V columns, or with interleaved
// pairs one load of V columns), or V copied columns.
template <typename T, int V, bool kInter>
__device__ __forceinline__ void unit(const T* in, T* out, const float2* cs, int u, int turning, int R) {
  if (u < turning) {
    if constexpr (kInter) {
      constexpr int W = columns_of<V, true>;
      float x[W], y[W];
      load_n<T, W>(in + u * W, x);
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        const float2 c = cs[(u * W + i) / 2];
        y[i] = x[i] * c.x - x[i + 1] * c.y;
        y[i + 1] = x[i] * c.y + x[i + 1] * c.x;
      }
      store_n<T, W>(out + u * W, y);
    } else {
      float x0[V], x1[V], y0[V], y1[V];
      load_n<T, V>(in + u * V, x0);
      load_n<T, V>(in + R / 2 + u * V, x1);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 c = cs[u * V + i];
        y0[i] = x0[i] * c.x - x1[i] * c.y;
        y1[i] = x0[i] * c.y + x1[i] * c.x;
      }
      store_n<T, V>(out + u * V, y0);
      store_n<T, V>(out + R / 2 + u * V, y1);
    }
  } else {
    float x[V];
    const int c = R + (u - turning) * V;
    load_n<T, V>(in + c, x);
    store_n<T, V>(out + c, x);
  }
}

}  // namespace

template <typename T, int V, bool kInter, int kTokens>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  extern __shared__ float2 cs[];  // [kTokens][R / 2]
  __shared__ bool live[kTokens];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int t0 = blockIdx.x * kTokens, pairs = a.R / 2;
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
  constexpr int W = columns_of<V, kInter>;
  const int turning = a.R / W, units = turning + (a.D - a.R) / V;
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
    unit<T, V, kInter>(in, out, cs + tok * pairs, u, turning, a.R);
  }
}

namespace {

template <typename T, int V, bool kInter>
hipError_t rotary_of(const RotaryArgs& a, hipStream_t s) {
  const size_t lds = sizeof(float2) * (a.R / 2);
  constexpr int W = columns_of<V, kInter>;
  const int64_t pieces = (int64_t)(a.R / W + (a.D - a.R) / V) * (a.q.heads + a.k.heads);
  if (pieces * kTok <= 256)
    hipLaunchKernelGGL((rotary_kernel<T, V, kInter, kTok>), dim3((a.T + kTok - 1) / kTok), dim3(256), kTok * lds, s, a);
  else
    hipLaunchKernelGGL((rotary_kernel<T, V, kInter, 1>), dim3(a.T), dim3(256), lds, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t rotary_type(bool inter, bool wide, const RotaryArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (inter) return wide ? rotary_of<T, V, true>(a, s) : rotary_of<T, 1, true>(a, s);
  return wide ? rotary_of<T, V, false>(a, s) : rotary_of<T, 1, false>(a, s);
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
