// C ABI of the operators around the recurrences: rotary positions and the
// root-mean-square norm. Every argument error returns before anything is
// enqueued.
#include <math.h>

#include <algorithm>

#include "gdn.h"
#include "layer.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

using namespace gdn;

namespace {

constexpr int kRotaryMaxD = 1024;
constexpr int kRotaryMaxT = 1 << 25;  // tokens of at most 4 launches
constexpr int64_t kMaxStride = (int64_t)1 << 31;

int size_of(int dtype) { return dtype == GDN_FP32 ? 4 : 2; }
bool known(int dtype) { return dtype == GDN_BF16 || dtype == GDN_FP16 || dtype == GDN_FP32; }
bool aligned(const void* p, int to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0; }
bool bad_stride(int64_t s, int64_t dense) { return s != 0 && (s < dense || s >= kMaxStride); }

gdn_status check_rotary(const gdn_rotary_problem* p) {
  if (!p) return GDN_ERR_NULL;
  if (p->T < 0 || p->HQ <= 0 || p->HK < 0 || p->D <= 0 || p->N < 0) return GDN_ERR_SHAPE;
  if (p->D > kRotaryMaxD || p->R < 2 || p->R > p->D || p->R % 2 != 0 || !known(p->dtype) ||
      (p->interleaved != 0 && p->interleaved != 1))
    return GDN_ERR_UNSUPPORTED;
  const int64_t dq = (int64_t)p->HQ * p->D, dk = (int64_t)p->HK * p->D;
  if (dq + dk >= ((int64_t)1 << 28)) return GDN_ERR_SHAPE;  // a token's pieces are counted in 32 bits
  if (bad_stride(p->q_stride, dq) || bad_stride(p->q_out_stride, dq) || bad_stride(p->k_stride, dk) ||
      bad_stride(p->k_out_stride, dk))
    return GDN_ERR_SHAPE;
  if (p->T > kRotaryMaxT) return GDN_ERR_SHAPE;
  if (!p->positions) {
    if (p->N == 0 && p->T != 0) return GDN_ERR_SHAPE;
    if (p->cu_seqlens_host) {
      const int32_t* cu = p->cu_seqlens_host;
      if (cu[0] != 0 || cu[p->N] != p->T) return GDN_ERR_SEQLENS;
      for (int n = 0; n < p->N; ++n)
        if (cu[n + 1] < cu[n]) return GDN_ERR_SEQLENS;
    }
  }
  return GDN_OK;
}

int rotary(const gdn_rotary_problem* p, const float* inv_freq, const void* q, const void* k, void* q_out,
           void* k_out, int64_t qs, int64_t ks, int64_t qos, int64_t kos, float sign, void* stream) {
  const gdn_status st = check_rotary(p);
  if (st != GDN_OK) return st;
  if (p->T == 0) return GDN_OK;
  if (!q || !q_out || !inv_freq || (p->HK > 0 && (!k || !k_out)) || (!p->positions && !p->cu_seqlens))
    return GDN_ERR_NULL;
  const int size = size_of(p->dtype), V = 16 / size;
  const int64_t dq = (int64_t)p->HQ * p->D, dk = (int64_t)p->HK * p->D;
  if (p->HK == 0) k = k_out = nullptr;
  for (const void* x : {q, k, (const void*)q_out, (const void*)k_out})
    if (!aligned(x, size)) return GDN_ERR_ALIGN;
  RotaryArgs a;
  a.T = p->T;
  a.D = p->D;
  a.R = p->R;
  a.mscale = p->mscale > 0.f ? p->mscale : 1.f;
  a.sign = sign;
  a.inv_freq = inv_freq;
  a.positions = p->positions;
  a.N = p->N;
  a.cu = p->cu_seqlens;
  a.offsets = p->offsets;
  a.q = {q, q_out, qs ? qs : dq, qos ? qos : dq, p->HQ};
  a.k = {k, k_out, ks ? ks : dk, kos ? kos : dk, p->HK};
  const int piece = p->interleaved ? V : 2 * V;
  bool wide = p->R % piece == 0 && p->D % V == 0;
  for (const RotaryRows& r : {a.q, a.k})
    wide = wide && aligned(r.in, 16) && aligned(r.out, 16) && r.in_stride % V == 0 && r.out_stride % V == 0;
  return launch_rotary(static_cast<Elem>(p->dtype), p->interleaved != 0, wide, a,
                       reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? GDN_OK
             : GDN_ERR_HIP;
}

gdn_status check_norm(const gdn_rmsnorm_problem* p) {
  if (!p) return GDN_ERR_NULL;
  if (p->rows < 0 || p->D <= 0) return GDN_ERR_SHAPE;
  if (p->D > kNormMaxD || !known(p->dtype) || (p->group != 0 && p->group != 128) ||
      (p->unit_offset != 0 && p->unit_offset != 1))
    return GDN_ERR_UNSUPPORTED;
  if (bad_stride(p->x_stride, p->D) || bad_stride(p->residual_stride, p->D)) return GDN_ERR_SHAPE;
  if (norm_threads(p->rows, p->D) >= (int64_t)1 << 32) return GDN_ERR_SHAPE;  // of one launch
  return GDN_OK;
}

}  // namespace

GDN_API int gdn_rotary(const gdn_rotary_problem* p, const float* inv_freq, const void* q, const void* k,
                       void* q_out, void* k_out, void* stream) {
  if (!p) return GDN_ERR_NULL;
  return rotary(p, inv_freq, q, k, q_out, k_out, p->q_stride, p->k_stride, p->q_out_stride, p->k_out_stride, 1.f,
                stream);
}

GDN_API int gdn_rotary_bwd(const gdn_rotary_problem* p, const float* inv_freq, const void* dq_out,
                           const void* dk_out, void* dq, void* dk, void* stream) {
  if (!p) return GDN_ERR_NULL;
  return rotary(p, inv_freq, dq_out, dk_out, dq, dk, p->q_out_stride, p->k_out_stride, p->q_stride, p->k_stride,
                -1.f, stream);
}

GDN_API int gdn_rotary_inv_freq(int32_t R, double base, int32_t scaling, double factor, double original,
                                float* inv_freq, float* mscale) {
  if (!inv_freq || !mscale) return GDN_ERR_NULL;
  if (scaling < GDN_ROPE_PLAIN || scaling > GDN_ROPE_YARN) return GDN_ERR_UNSUPPORTED;
  if (R < 2 || R % 2 != 0 || R > kRotaryMaxD || !(base > 1.0) || !(base < 1e30)) return GDN_ERR_SHAPE;
  if (scaling != GDN_ROPE_PLAIN && (!(factor >= 1.0) || !(factor < 1e9))) return GDN_ERR_SHAPE;
  if (scaling == GDN_ROPE_NTK) {
    if (R == 2) return GDN_ERR_SHAPE;
    base *= pow(factor, (double)R / (R - 2));
  }
  *mscale = 1.f;
  double lo = 0.0, hi = 0.0;
  if (scaling == GDN_ROPE_YARN) {
    if (!(original >= 1.0) || !(original < 1e12)) return GDN_ERR_SHAPE;
    // the (real) pair that makes so many turns in `original` positions
    auto pair = [&](double turns) { return R * log(original / (turns * 2.0 * M_PI)) / (2.0 * log(base)); };
    lo = std::max(floor(pair(32.0)), 0.0);
    hi = std::min(ceil(pair(1.0)), (double)(R - 1));
    *mscale = (float)(0.1 * log(factor) + 1.0);
  }
  for (int j = 0; j < R / 2; ++j) {
    const double f = pow(base, -2.0 * j / R);
    double x = f;
    if (scaling == GDN_ROPE_LINEAR) x = f / factor;
    if (scaling == GDN_ROPE_YARN) {
      const double ramp = std::min(std::max((j - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      x = f / factor * ramp + f * (1.0 - ramp);
    }
    inv_freq[j] = (float)x;
  }
  return GDN_OK;
}

GDN_API int gdn_rmsnorm_fwd(const gdn_rmsnorm_problem* p, const void* x, const void* residual, const void* weight,
                            void* residual_out, void* y, uint8_t* y8, float* scales, float* rstd, void* stream) {
  const gdn_status st = check_norm(p);
  if (st != GDN_OK) return st;
  if (p->rows == 0) return GDN_OK;
  if (!x || (residual && !residual_out) || (!y && !y8) || (y8 && !scales)) return GDN_ERR_NULL;
  const int size = size_of(p->dtype), V = 16 / size;
  for (const void* t : {x, residual, weight, (const void*)residual_out, (const void*)y})
    if (!aligned(t, size)) return GDN_ERR_ALIGN;
  if (!aligned(scales, 4) || !aligned(rstd, 4)) return GDN_ERR_ALIGN;
  if (!residual) residual_out = nullptr;
  NormArgs a;
  a.rows = p->rows;
  a.D = p->D;
  a.eps = p->eps;
  a.unit = p->unit_offset ? 1.f : 0.f;
  a.group = y8 ? (p->group ? p->group : p->D) : 0;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.x_stride = p->x_stride ? p->x_stride : p->D;
  a.residual_stride = p->residual_stride ? p->residual_stride : p->D;
  a.residual_out = residual_out;
  a.y = y;
  a.y8 = y8;
  a.scales = scales;
  a.rstd = rstd;
  bool wide = p->D % V == 0 && a.x_stride % V == 0 && a.residual_stride % V == 0 && aligned(y8, V);
  for (const void* t : {x, residual, weight, (const void*)residual_out, (const void*)y}) wide = wide && aligned(t, 16);
  return launch_rmsnorm_fwd(static_cast<Elem>(p->dtype), wide, a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? GDN_OK
             : GDN_ERR_HIP;
}

GDN_API size_t gdn_rmsnorm_bwd_workspace_size(const gdn_rmsnorm_problem* p) {
  return check_norm(p) == GDN_OK ? (size_t)norm_partials(p->rows, p->D) * norm_pitch(p->D) * sizeof(float) : 0;
}

GDN_API int gdn_rmsnorm_bwd(const gdn_rmsnorm_problem* p, const void* s, const void* weight, const float* rstd,
                            const void* dy, const void* ds, void* dx, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const gdn_status st = check_norm(p);
  if (st != GDN_OK) return st;
  if (p->rows > 0 && (!s || !rstd || !dy || !dx)) return GDN_ERR_NULL;
  const int size = size_of(p->dtype), V = 16 / size;
  for (const void* t : {s, weight, dy, ds, (const void*)dx})
    if (!aligned(t, size)) return GDN_ERR_ALIGN;
  if (!aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(workspace, 16)) return GDN_ERR_ALIGN;
  const size_t need = dweight ? gdn_rmsnorm_bwd_workspace_size(p) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  NormGradArgs a;
  a.rows = p->rows;
  a.D = p->D;
  a.unit = p->unit_offset ? 1.f : 0.f;
  a.s = s;
  a.weight = weight;
  a.dy = dy;
  a.ds = ds;
  a.rstd = rstd;
  a.s_stride = p->x_stride ? p->x_stride : p->D;
  a.dx = dx;
  a.dweight = dweight;
  a.partial = dweight ? static_cast<float*>(workspace) : nullptr;
  bool wide = p->D % V == 0 && a.s_stride % V == 0;
  for (const void* t : {s, weight, dy, ds, (const void*)dx}) wide = wide && aligned(t, 16);
  return launch_rmsnorm_bwd(static_cast<Elem>(p->dtype), wide, a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? GDN_OK
             : GDN_ERR_HIP;
}
