// Root-mean-square norm of s = x + residual over the columns of each row:
//   y = s rstd (weight + unit),  rstd = 1 / sqrt(mean(s^2) + eps),
// where s is the sum rounded to the tensor's type (what the residual stream
// holds, and what the backward reads). y goes out in the tensor's type and / or
// in e4m3 with a scale for each row or each 128 columns: scale = max(largest
// |y|, 2^-100) / 448 in fp32, and y / scale rounded to nearest even.
// Backward, with n = s rstd and dn = dy (weight + unit):
//   dx = rstd (dn - n mean(dn n)) + ds,   dweight = sum over rows of dy n.
//
// Bound by HBM. A row is read once: GROUP threads hold it in registers, E
// columns each, so the mean, the scales and the outputs need no second pass.
#include "layer.h"

namespace gdn {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kTiny = 0x1p-100f;

// larger of two, NaN if one is
__device__ __forceinline__ float nmax(float a, float b) { return a > b || a != a ? a : b; }

template <int W, bool kMax>
__device__ __forceinline__ float reduce_lanes(float x) {
#pragma unroll
  for (int m = W / 2; m >= 1; m >>= 1) {
    const float y = __shfl_xor(x, m, 64);
    x = kMax ? nmax(x, y) : x + y;
  }
  return x;
}

// Sum (or NaN-keeping maximum) over a row's GROUP threads, in a fixed order.
// `part` holds a value per wave; it may be used again after two other uses.
template <int GROUP, bool kMax>
__device__ __forceinline__ float reduce_row(float x, float* part) {
  x = reduce_lanes<(GROUP < 64 ? GROUP : 64), kMax>(x);
  if constexpr (GROUP > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int i = 1; i < GROUP / 64; ++i) x = kMax ? nmax(x, part[i]) : x + part[i];
  }
  return x;
}

// The first column of a thread's piece p of V columns. 16 bytes at a time, the
// row's threads side by side; element by element, a wave takes 128 columns at
// a time, so that a scale's 128 columns belong to one wave.
template <int V, int GROUP>
__device__ __forceinline__ int column(int p, int t) {
  if constexpr (V > 1) return (p * GROUP + t) * V;
  else if constexpr (GROUP < 64) return p * GROUP + t;
  else return ((p >> 1) * (GROUP / 64) + (t >> 6)) * 128 + (p & 1) * 64 + (t & 63);
}

template <typename T, int V>
__device__ __forceinline__ void load_at(const T* row, int c, int D, float* x) {
  if (c < D) load_n<T, V>(row + c, x);
  else
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.f;
}

// e4m3 of v, to nearest even; NaN stays
__device__ __forceinline__ float into_range(float v) {
  const float c = __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max);
  return v != v ? v : c;
}
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* x) {
  if constexpr (V == 1) {
    *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(into_range(x[0]), 0.f, 0, false);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      int u = __builtin_amdgcn_cvt_pk_fp8_f32(into_range(x[4 * i]), into_range(x[4 * i + 1]), 0, false);
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(into_range(x[4 * i + 2]), into_range(x[4 * i + 3]), u, true);
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

}  // namespace

template <typename T, int V, int GROUP, int E>
__global__ __launch_bounds__(GROUP > 256 ? GROUP : 256) void rmsnorm_fwd_kernel(NormArgs a) {
  constexpr int P = E / V, NT = GROUP > 256 ? GROUP : 256, kRows = NT / GROUP;
  __shared__ float part[2][GROUP > 64 ? GROUP / 64 : 1];
  const int t = threadIdx.x % GROUP, D = a.D;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / GROUP;
  const bool on = row < a.rows;  // rows of one workgroup meet at the shuffles
  const T* x = static_cast<const T*>(a.x) + (on ? row : 0) * a.x_stride;
  float v[P][V];
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) load_at<T, V>(x, column<V, GROUP>(p, t), D, v[p]);
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + (on ? row : 0) * a.residual_stride;
    T* so = static_cast<T*>(a.residual_out) + row * D;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = column<V, GROUP>(p, t);
      float y[V];
      load_at<T, V>(r, c, D, y);
#pragma unroll
      for (int i = 0; i < V; ++i) v[p][i] = to_f32(from_f32<T>(v[p][i] + y[i]));
      if (on && c < D) store_n<T, V>(so + c, v[p]);
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) sum += v[p][i] * v[p][i];
  sum = reduce_row<GROUP, false>(sum, part[0]);
  const float rstd = 1.f / sqrtf(sum / (float)D + a.eps);
  if (a.rstd && on && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = column<V, GROUP>(p, t);
    float w[V];
    if (a.weight) load_at<T, V>(static_cast<const T*>(a.weight), c, D, w);
#pragma unroll
    for (int i = 0; i < V; ++i) v[p][i] *= a.weight ? rstd * (w[i] + a.unit) : rstd;
    if (a.y && on && c < D) store_n<T, V>(static_cast<T*>(a.y) + row * D + c, v[p]);
  }
  if (!a.y8) return;
  float top[P];  // of each piece
#pragma unroll
  for (int p = 0; p < P; ++p) {
    top[p] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) top[p] = nmax(top[p], fabsf(v[p][i]));
  }
  if (a.group == D) {
    float m = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) m = nmax(m, top[p]);
    m = nmax(reduce_row<GROUP, true>(m, part[1]), kTiny);
    const float scale = m / kE4m3Max;
    if (on && t == 0) a.scales[row] = scale;
#pragma unroll
    for (int p = 0; p < P; ++p) top[p] = scale;
  } else {
    const int groups = (D + 127) / 128;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = column<V, GROUP>(p, t);
      float m;
      if constexpr (V > 1) {
        constexpr int L = 128 / V;  // lanes of 128 columns
        if constexpr (GROUP >= L) m = reduce_lanes<L, true>(top[p]);
        else {  // the row's threads hold 128 columns in several pieces
          m = top[0];
#pragma unroll
          for (int r = 1; r < P; ++r) m = nmax(m, top[r]);
          m = reduce_lanes<GROUP, true>(m);
        }
      } else if constexpr (GROUP < 64) {
        m = top[0];
#pragma unroll
        for (int r = 1; r < P; ++r) m = nmax(m, top[r]);
        m = reduce_lanes<GROUP, true>(m);
      } else {
        m = reduce_lanes<64, true>(nmax(top[p & ~1], top[p | 1]));
      }
      m = nmax(m, kTiny) / kE4m3Max;
      if (on && c < D && c % 128 == 0) a.scales[row * groups + c / 128] = m;
#pragma unroll
      for (int i = 0; i < V; ++i) v[p][i] /= m;
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = column<V, GROUP>(p, t);
    if (a.group == D) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[p][i] /= top[p];
    }
    if (on && c < D) store_e4m3<V>(a.y8 + row * D + c, v[p]);
  }
}

template <typename T, int V, int GROUP, int E>
__global__ __launch_bounds__(GROUP > 256 ? GROUP : 256) void rmsnorm_bwd_kernel(NormGradArgs a, int step) {
  constexpr int P = E / V, NT = GROUP > 256 ? GROUP : 256, kRows = NT / GROUP;
  __shared__ float part[2][GROUP > 64 ? GROUP / 64 : 1];
  const int t = threadIdx.x % GROUP, D = a.D;
  const int first = blockIdx.x * kRows + threadIdx.x / GROUP;  // this group's first row; it takes every step-th
  float w[P][V], acc[P][V];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (a.weight) load_at<T, V>(static_cast<const T*>(a.weight), column<V, GROUP>(p, t), D, w[p]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[p][i] = a.weight ? w[p][i] + a.unit : 1.f;
      acc[p][i] = 0.f;
    }
  }
  int odd = 0;
  for (int base = blockIdx.x * kRows; base < a.rows; base += step, odd ^= 1) {
    const int64_t row = base + threadIdx.x / GROUP;
    const bool on = row < a.rows;
    const T* s = static_cast<const T*>(a.s) + (on ? row : 0) * a.s_stride;
    const T* dy = static_cast<const T*>(a.dy) + (on ? row : 0) * D;
    const float rstd = on ? a.rstd[row] : 0.f;
    float n[P][V], g[P][V], dot = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = column<V, GROUP>(p, t);
      load_at<T, V>(s, c, D, n[p]);
      load_at<T, V>(dy, c, D, g[p]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        n[p][i] *= rstd;
        if (on) acc[p][i] += g[p][i] * n[p][i];
        g[p][i] *= w[p][i];
        dot += g[p][i] * n[p][i];
      }
    }
    dot = reduce_row<GROUP, false>(dot, part[odd]) / (float)D;
    const T* ds = static_cast<const T*>(a.ds) + (on ? row : 0) * D;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = column<V, GROUP>(p, t);
      float z[V];
      if (a.ds) load_at<T, V>(ds, c, D, z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = rstd * (g[p][i] - n[p][i] * dot);
        z[i] = a.ds ? d + z[i] : d;
      }
      if (on && c < D) store_n<T, V>(static_cast<T*>(a.dx) + row * D + c, z);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = column<V, GROUP>(p, t);
    if (c < D) store_n<float, V>(a.partial + (int64_t)first * D + c, acc[p]);
  }
}

// dweight[c] = sum of the partials' column c: 4 threads a column, in a fixed order
__global__ __launch_bounds__(256) void rmsnorm_fold_kernel(int n, int D, const float* __restrict__ partial,
                                                           float* __restrict__ dweight) {
  __shared__ float sums[16][17];
  const int l = threadIdx.x & 15, part = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
  float s = 0.f;
  if (c < D)
    for (int i = part; i < n; i += 16) s += partial[(int64_t)i * D + c];
  sums[part][l] = s;
  __syncthreads();
  if (part == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += sums[i][l];
    dweight[c] = s;
  }
}

namespace {

// The threads of a row and the columns of each, for rows of D columns.
struct Shape {
  int group, each;
};
Shape shape_of(int D) {
  if (D <= 128) return {16, 8};
  if (D <= 512) return {64, 8};
  if (D <= 1024) return {64, 16};
  if (D <= 2048) return {256, 8};
  if (D <= 4096) return {256, 16};
  if (D <= 8192) return {256, 32};
  return {512, 32};
}
int rows_at_once(int D) {
  const int g = shape_of(D).group;
  return g < 256 ? 256 / g : 1;
}

template <typename T, int V, typename F>
hipError_t with_shape(int D, F&& f) {
  switch (shape_of(D).group * shape_of(D).each) {
    case 128: return f.template operator()<T, V, 16, 8>();
    case 512: return f.template operator()<T, V, 64, 8>();
    case 1024: return f.template operator()<T, V, 64, 16>();
    case 2048: return f.template operator()<T, V, 256, 8>();
    case 4096: return f.template operator()<T, V, 256, 16>();
    case 8192: return f.template operator()<T, V, 256, 32>();
    default: return f.template operator()<T, V, 512, 32>();
  }
}
template <typename F>
hipError_t with_type(Elem type, bool wide, int D, F&& f) {
  switch (type) {
    case Elem::kBf16: return wide ? with_shape<Bf16, 8>(D, f) : with_shape<Bf16, 1>(D, f);
    case Elem::kFp16: return wide ? with_shape<Fp16, 8>(D, f) : with_shape<Fp16, 1>(D, f);
    default: return wide ? with_shape<float, 4>(D, f) : with_shape<float, 1>(D, f);
  }
}

int64_t blocks_of(int rows, int D) { return ((int64_t)rows + rows_at_once(D) - 1) / rows_at_once(D); }
constexpr int kBwdBlocks = 1024;

struct Fwd {
  const NormArgs& a;
  hipStream_t s;
  template <typename T, int V, int GROUP, int E>
  hipError_t operator()() {
    hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, V, GROUP, E>), dim3((unsigned)blocks_of(a.rows, a.D)),
                       dim3(GROUP > 256 ? GROUP : 256), 0, s, a);
    return hipGetLastError();
  }
};
struct Bwd {
  const NormGradArgs& a;
  hipStream_t s;
  template <typename T, int V, int GROUP, int E>
  hipError_t operator()() {
    const int blocks = norm_partials(a.rows, a.D) / rows_at_once(a.D);
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, V, GROUP, E>), dim3(blocks), dim3(GROUP > 256 ? GROUP : 256), 0, s,
                       a, blocks * rows_at_once(a.D));
    return hipGetLastError();
  }
};

}  // namespace

int norm_partials(int rows, int D) {
  const int64_t b = blocks_of(rows, D);
  return (int)(b < kBwdBlocks ? b : kBwdBlocks) * rows_at_once(D);
}

hipError_t launch_rmsnorm_fwd(Elem type, bool wide, const NormArgs& a, hipStream_t s) {
  return with_type(type, wide, a.D, Fwd{a, s});
}

hipError_t launch_rmsnorm_bwd(Elem type, bool wide, const NormGradArgs& a, hipStream_t s) {
  if (a.rows > 0) {
    const hipError_t e = with_type(type, wide, a.D, Bwd{a, s});
    if (e != hipSuccess) return e;
  }
  if (a.dweight) {
    hipLaunchKernelGGL(rmsnorm_fold_kernel, dim3((a.D + 15) / 16), dim3(256), 0, s, norm_partials(a.rows, a.D), a.D,
                       a.partial, a.dweight);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace gdn
