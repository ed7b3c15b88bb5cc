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
// 16384 x 4096 bf16 with a residual: 84 us forward (537 MB, 6.4 TB/s), 108 us
// backward (537 MB and the partial sums of dweight, 5.1 TB/s). 8191 x 5120 fp16 with
// a residual to e4m3: 63 us (294 MB, 4.7 TB/s).
#include "layer.h"

namespace gdn {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kTiny = 0x1p-100f;

// larger of two, NaN if one is
__device__ __forceinline__ float nmax(float a, float b) { return a > b || a != a ? a : b; }
// larger of m >= 0 and |x|, NaN if one is: magnitudes are in the order of their bits, NaN last
__device__ __forceinline__ float magnitude(float m, float x) {
  return __uint_as_float(max(__float_as_uint(m), __float_as_uint(fabsf(x))));
}

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

// The first column of a thread's piece p of V columns (16 bytes of the tensor's
// type), a row's threads side by side.
template <int V, int GROUP>
__device__ __forceinline__ int column(int p, int t) {
  return (p * GROUP + t) * V;
}

// V columns of a row from c on; those past D are zeros, and not stored. kWide: D is
// a multiple of V and everything is aligned to 16 bytes. Rows of any other length or
// alignment go 16 bytes at a time all the same (load_any). 16384 x 4095, forward and
// backward: 236 us, and 659 element by element.
template <typename T, int V, bool kWide>
__device__ __forceinline__ void load_at(const T* row, int c, int D, float* x) {
  if constexpr (kWide) {
    if (c < D) load_n<T, V>(row + c, x);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.f;
  } else {
    load_any<T, V>(row, c, D, x);
  }
}
template <typename T, int V, bool kWide>
__device__ __forceinline__ void store_at(T* row, int c, int D, const float* x) {
  if constexpr (kWide) {
    if (c < D) store_n<T, V>(row + c, x);
  } else {
    store_any<T, V>(row, c, D, x);
  }
}

// 448 a / m as a division rounds it, from r = 448 / m: the remainder of a first
// quotient, exact by fma, corrects it. bf16 and fp16 rows give quotients that lie
// exactly between two e4m3 values, which a quotient off by one fp32 step would round
// to the wrong one. At most 448 for |a| <= m.
__device__ __forceinline__ float quotient(float a, float m, float r, float rm) {
  const float q = a * r;
  const float p = q * m;
  const float rem = fmaf(a, kE4m3Max, -p) - fmaf(q, m, -p);
  const float c = fmaf(rem, rm, q);
  return c == c ? c : q;  // m infinite: the remainder is no number
}
// e4m3 of values of at most 448 in magnitude, to nearest even; NaN stays
template <int V, bool kWide>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int c, int D, const float* x) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], u, true);
  }
  if (kWide ? c < D : c + V <= D) {
    __builtin_memcpy(kWide ? __builtin_assume_aligned(row + c, V) : row + c, w, V);
  } else if (!kWide) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < D) row[c + i] = (uint8_t)(w[i / 4] >> 8 * (i % 4));
  }
}

}  // namespace

template <typename T, int V, bool kWide, int GROUP, int E>
__global__ __launch_bounds__(GROUP > 256 ? GROUP : 256) void rmsnorm_fwd_kernel(NormArgs a) {
  constexpr int P = E / V, NT = GROUP > 256 ? GROUP : 256, kRows = NT / GROUP;
  __shared__ float part[3][GROUP > 64 ? GROUP / 64 : 1];
  const int t = threadIdx.x % GROUP, D = a.D;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / GROUP;
  const bool on = row < a.rows;  // rows of one workgroup meet at the shuffles
  const T* x = static_cast<const T*>(a.x) + (on ? row : 0) * a.x_stride;
  float v[P][V];
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) load_at<T, V, kWide>(x, column<V, GROUP>(p, t), D, v[p]);
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + (on ? row : 0) * a.residual_stride;
    T* so = static_cast<T*>(a.residual_out) + row * D;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = column<V, GROUP>(p, t);
      float y[V];
      load_at<T, V, kWide>(r, c, D, y);
#pragma unroll
      for (int i = 0; i < V; ++i) v[p][i] = to_f32(from_f32<T>(v[p][i] + y[i]));
      if (on) store_at<T, V, kWide>(so, c, D, v[p]);
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) sum += v[p][i] * v[p][i];
  sum = reduce_row<GROUP, false>(sum, part[0]);
  float mean = sum / (float)D;
  if (sum == __builtin_inff()) {  // past fp32, as the mean may not be: 2^-14 of it, D being at most 2^14
    sum = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float z = v[p][i] * 0x1p-7f;
        sum += z * z;
      }
    mean = reduce_row<GROUP, false>(sum, part[2]) * (0x1p14f / (float)D);
  }
  const float rstd = 1.f / sqrtf(mean + a.eps);
  if (a.rstd && on && t == 0) a.rstd[row] = rstd;
  // rstd = lift rest, lift a power of two and 1 <= rest < 2: v <- s lift (weight + unit)
  // and y = v rest. The power takes a row to its own size before the weight does, so
  // that the product passes fp32's range where y does and not before, and costs no
  // rounding. A row without a finite rstd > 0 (infinities or NaN in it, a sum past fp32,
  // or zeros with eps = 0) takes rstd itself for it.
  const bool finite = rstd > 0.f && rstd < __builtin_inff();
  const uint32_t bits = __float_as_uint(rstd);
  const float lift = finite ? __uint_as_float(bits & 0x7f800000u) : rstd;
  const float rest = finite ? __uint_as_float((bits & 0x007fffffu) | 0x3f800000u) : 1.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = column<V, GROUP>(p, t);
#pragma unroll
    for (int i = 0; i < V; ++i) v[p][i] *= lift;
    if (a.weight) {
      float w[V];
      load_at<T, V, kWide>(static_cast<const T*>(a.weight), c, D, w);
#pragma unroll
      for (int i = 0; i < V; ++i) v[p][i] *= w[i] + a.unit;
    }
    if (a.y && on) {
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = v[p][i] * rest;
      store_at<T, V, kWide>(static_cast<T*>(a.y) + row * D, c, D, y);
    }
  }
  if (!a.y8) return;
  // Scales from the largest |v| of their columns: rest cancels in y / scale, so the
  // quotients are formed from v (products of two short numbers, exact where x has 16
  // bits) and only the scale itself takes rest.
  float top[P];  // of each piece
#pragma unroll
  for (int p = 0; p < P; ++p) {
    top[p] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) top[p] = magnitude(top[p], v[p][i]);
  }
  const float least = kTiny / rest;
  const int groups = (D + 127) / 128;
  float whole = 0.f;
  if (a.group == D) {
#pragma unroll
    for (int p = 0; p < P; ++p) whole = nmax(whole, top[p]);
    whole = nmax(reduce_row<GROUP, true>(whole, part[1]), least);
    if (on && t == 0) a.scales[row] = whole * rest / kE4m3Max;
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = column<V, GROUP>(p, t);
    float m = whole;
    if (a.group != D) {
      if constexpr (GROUP >= 128 / V) {
        m = reduce_lanes<128 / V, true>(top[p]);
      } else {  // the row's threads hold its 128 columns or fewer in several pieces
        m = top[0];
#pragma unroll
        for (int r = 1; r < P; ++r) m = nmax(m, top[r]);
        m = reduce_lanes<GROUP, true>(m);
      }
      m = nmax(m, least);
      if (on && c < D && c % 128 == 0) a.scales[row * groups + c / 128] = m * rest / kE4m3Max;
    }
    const float r = kE4m3Max / m, rm = 1.f / m;
#pragma unroll
    for (int i = 0; i < V; ++i) v[p][i] = quotient(v[p][i], m, r, rm);
    if (on) store_e4m3<V, kWide>(a.y8 + row * D, c, D, v[p]);
  }
}

template <typename T, int V, bool kWide, int GROUP, int E>
__global__ __launch_bounds__(GROUP > 256 ? GROUP : 256) void rmsnorm_bwd_kernel(NormGradArgs a, int step) {
  constexpr int P = E / V, NT = GROUP > 256 ? GROUP : 256, kRows = NT / GROUP;
  __shared__ float part[2][GROUP > 64 ? GROUP / 64 : 1];
  const int t = threadIdx.x % GROUP, D = a.D;
  const int first = blockIdx.x * kRows + threadIdx.x / GROUP;  // this group's first row; it takes every step-th
  float w[P][V], acc[P][V];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (a.weight) load_at<T, V, kWide>(static_cast<const T*>(a.weight), column<V, GROUP>(p, t), D, w[p]);
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
      load_at<T, V, kWide>(s, c, D, n[p]);
      load_at<T, V, kWide>(dy, c, D, g[p]);
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
      if (a.ds) load_at<T, V, kWide>(ds, c, D, z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = rstd * (g[p][i] - n[p][i] * dot);
        z[i] = a.ds ? d + z[i] : d;
      }
      if (on) store_at<T, V, kWide>(static_cast<T*>(a.dx) + row * D, c, D, z);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = column<V, GROUP>(p, t);
    if (c < D) store_n<float, V>(a.partial + (int64_t)first * norm_pitch(D) + c, acc[p]);
  }
}

// dweight[c] = sum of the partials' column c: 32 threads a column, each every
// 32nd partial in order, then the 32 sums in order.
__global__ __launch_bounds__(1024) void rmsnorm_fold_kernel(int n, int D, const float* __restrict__ partial,
                                                            float* __restrict__ dweight) {
  constexpr int kCols = 32, kParts = 1024 / kCols, kAhead = 8;
  __shared__ float sums[kParts][kCols + 1];
  const int l = threadIdx.x % kCols, part = threadIdx.x / kCols, c = blockIdx.x * kCols + l;
  float s = 0.f;
  if (c < D) {
    for (int i0 = part; i0 < n; i0 += kParts * kAhead) {
      float x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * kParts;
        x[j] = i < n ? partial[(int64_t)i * norm_pitch(D) + c] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) s += x[j];
    }
  }
  sums[part][l] = s;
  __syncthreads();
  if (part == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < kParts; ++i) s += sums[i][l];
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
  if (D <= 5120) return {320, 16};
  if (D <= 6144) return {384, 16};
  if (D <= 8192) return {512, 16};
  if (D <= 12288) return {768, 16};
  return {1024, 16};
}
int rows_at_once(int D) {
  const int g = shape_of(D).group;
  return g < 256 ? 256 / g : 1;
}

template <typename T, int V, bool kWide, typename F>
hipError_t with_shape(int D, F&& f) {
  switch (shape_of(D).group * shape_of(D).each) {
    case 128: return f.template operator()<T, V, kWide, 16, 8>();
    case 512: return f.template operator()<T, V, kWide, 64, 8>();
    case 1024: return f.template operator()<T, V, kWide, 64, 16>();
    case 2048: return f.template operator()<T, V, kWide, 256, 8>();
    case 4096: return f.template operator()<T, V, kWide, 256, 16>();
    case 5120: return f.template operator()<T, V, kWide, 320, 16>();
    case 6144: return f.template operator()<T, V, kWide, 384, 16>();
    case 8192: return f.template operator()<T, V, kWide, 512, 16>();
    case 12288: return f.template operator()<T, V, kWide, 768, 16>();
    default: return f.template operator()<T, V, kWide, 1024, 16>();
  }
}
template <typename F>
hipError_t with_type(Elem type, bool wide, int D, F&& f) {
  switch (type) {
    case Elem::kBf16: return wide ? with_shape<Bf16, 8, true>(D, f) : with_shape<Bf16, 8, false>(D, f);
    case Elem::kFp16: return wide ? with_shape<Fp16, 8, true>(D, f) : with_shape<Fp16, 8, false>(D, f);
    default: return wide ? with_shape<float, 4, true>(D, f) : with_shape<float, 4, false>(D, f);
  }
}

int64_t blocks_of(int rows, int D) { return ((int64_t)rows + rows_at_once(D) - 1) / rows_at_once(D); }
constexpr int kBwdBlocks = 1024;  // 16384 x 4096 rows: 109 us, and 120 with 768, 158 with 512

struct Fwd {
  const NormArgs& a;
  hipStream_t s;
  template <typename T, int V, bool kWide, int GROUP, int E>
  hipError_t operator()() {
    hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, V, kWide, GROUP, E>), dim3((unsigned)blocks_of(a.rows, a.D)),
                       dim3(GROUP > 256 ? GROUP : 256), 0, s, a);
    return hipGetLastError();
  }
};
struct Bwd {
  const NormGradArgs& a;
  hipStream_t s;
  template <typename T, int V, bool kWide, int GROUP, int E>
  hipError_t operator()() {
    const int blocks = norm_partials(a.rows, a.D) / rows_at_once(a.D);
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, V, kWide, GROUP, E>), dim3(blocks), dim3(GROUP > 256 ? GROUP : 256), 0, s,
                       a, blocks * rows_at_once(a.D));
    return hipGetLastError();
  }
};

}  // namespace

int64_t norm_threads(int rows, int D) {
  const int g = shape_of(D).group;
  return blocks_of(rows, D) * (g > 256 ? g : 256);
}

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
    hipLaunchKernelGGL(rmsnorm_fold_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, s, norm_partials(a.rows, a.D), a.D,
                       a.partial, a.dweight);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace gdn
