// One token per row of the linear attention with a decay for each head, in
// place on a state pool: S <- lam S + v k^T, o = scale S q.
//
// Bound by HBM: each active (row, value head) streams its fp32 state in and
// out once (128 KiB at D = 128 against 1 KiB of everything else). The state's rows
// do not depend on each other: a workgroup takes kPart of them, four 16-byte loads
// a thread, so that a single row's 16 heads already spread over 64 CUs: 3 us. 240
// active rows of 32 heads take 165 us: 1.01 GB, 6.1 TB/s.
#include "linear.h"

namespace gdn {

namespace {

constexpr int kEach = 4;  // state rows a thread

// Sums of kEach rows over a group of L lanes at once: half the rows go to the
// other half of the lanes at each of the first two steps, so that the four sums
// take 2 + 1 + log2(L) - 2 exchanges instead of 4 log2(L). The lane whose number in
// its group is r (L / 4) ends with row r's sum, r = 0 .. 3.
template <int L>
__device__ __forceinline__ float sum_rows(const float* x, int lane) {
  static_assert(kEach == 4 && L >= 4, "two halvings");
  const bool upper = lane & (L / 2), second = lane & (L / 4);
  float a = upper ? x[2] : x[0], b = upper ? x[3] : x[1];
  a += __shfl_xor(upper ? x[0] : x[2], L / 2, 64);
  b += __shfl_xor(upper ? x[1] : x[3], L / 2, 64);
  float s = second ? b : a;
  s += __shfl_xor(second ? a : b, L / 4, 64);
#pragma unroll
  for (int m = L / 8; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
  return s;
}

}  // namespace

template <int D>
__global__ __launch_bounds__(256) void lin_step_kernel(int HV, float scale, LinRows q, LinRows k, LinRows v,
                                                       const float* __restrict__ log_decay,
                                                       float* __restrict__ pool, int slots,
                                                       const int32_t* __restrict__ idx,
                                                       uint16_t* __restrict__ o) {
  // a state row is kLanes lanes of 4 values; a thread holds one column group of rows r0, r0 + R, ...
  constexpr int kLanes = D / 4, R = 256 / kLanes, kPart = R * kEach, kParts = D / kPart;
  const int part = blockIdx.x % kParts, item = blockIdx.x / kParts;
  const int row = item / HV, hv = item - row * HV;
  const int tid = threadIdx.x, c4 = tid % kLanes, r0 = part * kPart + tid / kLanes;
  const int slot = idx[row];
  uint16_t* orow = o + ((size_t)row * HV + hv) * D;
  if (slot <= 0 || slot >= slots) {  // no state: a zero row
    if (tid < kPart / 2) reinterpret_cast<uint32_t*>(orow + part * kPart)[tid] = 0u;
    return;
  }
  float* S = pool + ((size_t)slot * HV + hv) * (size_t)(D * D) + c4 * 4;
  f32x4 s[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (r0 + R * i) * D));
  auto four = [&](const LinRows& x) {
    const uint2 u = *reinterpret_cast<const uint2*>(x.p + row * x.stride + (int64_t)(hv / x.G) * D + c4 * 4);
    return f32x4{bf2f(u.x & 0xffffu), bf2f(u.x >> 16), bf2f(u.y & 0xffffu), bf2f(u.y >> 16)};
  };
  const f32x4 qq = four(q), kk = four(k);
  const uint16_t* vr = v.p + row * v.stride + (int64_t)(hv / v.G) * D;
  float vv[kEach], sum[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) vv[i] = bf2f(vr[r0 + R * i]);
  const float decay = expf(log_decay[hv]);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    sum[i] = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[i][r] = decay * s[i][r] + vv[i] * kk[r];
      sum[i] += s[i][r] * qq[r];
    }
    __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + (r0 + R * i) * D));
  }
  const float total = sum_rows<kLanes>(sum, tid);
  if (c4 % (kLanes / 4) == 0) orow[r0 + R * (c4 / (kLanes / 4))] = f2bf(total * scale);
}

hipError_t launch_lin_step(int D, int N, int HV, float scale, const LinRows& q, const LinRows& k,
                           const LinRows& v, const float* log_decay, float* pool, int slots,
                           const int32_t* idx, uint16_t* o, hipStream_t stream) {
  const dim3 grid((unsigned)N * (unsigned)HV * (D == 128 ? 4u : 1u));
  if (D == 128)
    hipLaunchKernelGGL((lin_step_kernel<128>), grid, dim3(256), 0, stream, HV, scale, q, k, v, log_decay, pool,
                       slots, idx, o);
  else
    hipLaunchKernelGGL((lin_step_kernel<64>), grid, dim3(256), 0, stream, HV, scale, q, k, v, log_decay, pool,
                       slots, idx, o);
  return hipGetLastError();
}

}  // namespace gdn
