// One token per row of the linear attention with a decay for each head, in
// place on a state pool: S <- lam S + v k^T, o = scale S q.
//
// Bound by HBM: each active (row, value head) streams its fp32 state in and
// out once (128 KiB at D = 128 against 1 KiB of everything else).
#include "linear.h"

namespace gdn {

template <int D>
__global__ __launch_bounds__(256) void lin_step_kernel(int HV, float scale, LinRows q, LinRows k, LinRows v,
                                                       const float* __restrict__ log_decay,
                                                       float* __restrict__ pool, int slots,
                                                       const int32_t* __restrict__ idx,
                                                       uint16_t* __restrict__ o) {
  // a state row is D / 4 lanes of 4 values; a thread holds one column group of
  // rows r0, r0 + R, ...
  constexpr int kLanes = D / 4, R = 256 / kLanes, kRows = D / R;
  const int row = blockIdx.x / HV, hv = blockIdx.x - row * HV;
  const int tid = threadIdx.x, c4 = tid % kLanes, r0 = tid / kLanes;
  const int slot = idx[row];
  uint16_t* orow = o + ((size_t)row * HV + hv) * D;
  if (slot <= 0 || slot >= slots) {  // no state: a zero row
    if (tid < D / 2) reinterpret_cast<uint32_t*>(orow)[tid] = 0u;
    return;
  }
  float* S = pool + ((size_t)slot * HV + hv) * (size_t)(D * D) + c4 * 4;
  f32x4 s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (r0 + R * i) * D));
  auto four = [&](const LinRows& x) {
    const uint2 u = *reinterpret_cast<const uint2*>(x.p + row * x.stride + (int64_t)(hv / x.G) * D + c4 * 4);
    return f32x4{bf2f(u.x & 0xffffu), bf2f(u.x >> 16), bf2f(u.y & 0xffffu), bf2f(u.y >> 16)};
  };
  const f32x4 qq = four(q), kk = four(k);
  const uint16_t* vr = v.p + row * v.stride + (int64_t)(hv / v.G) * D;
  const float g = log_decay[hv], decay = expf(g);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float vv = bf2f(vr[r0 + R * i]);
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[i][r] = decay * s[i][r] + vv * kk[r];
      sum += s[i][r] * qq[r];
    }
    sum = group_sum<kLanes>(sum);
    if (c4 == 0) orow[r0 + R * i] = f2bf(sum * scale);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + (r0 + R * i) * D));
}

hipError_t launch_lin_step(int D, int N, int HV, float scale, const LinRows& q, const LinRows& k,
                           const LinRows& v, const float* log_decay, float* pool, int slots,
                           const int32_t* idx, uint16_t* o, hipStream_t stream) {
  const dim3 grid((unsigned)N * (unsigned)HV);
  if (D == 128)
    hipLaunchKernelGGL((lin_step_kernel<128>), grid, dim3(256), 0, stream, HV, scale, q, k, v, log_decay, pool,
                       slots, idx, o);
  else
    hipLaunchKernelGGL((lin_step_kernel<64>), grid, dim3(256), 0, stream, HV, scale, q, k, v, log_decay, pool,
                       slots, idx, o);
  return hipGetLastError();
}

}  // namespace gdn
