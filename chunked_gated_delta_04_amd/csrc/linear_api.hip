// C ABI of the linear attention with a decay for each head: argument checks,
// the cut of a pack into segments, launch sequencing. Every argument error
// returns before anything is enqueued.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "gdn.h"
#include "linear.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

using namespace gdn;

namespace {

#define GDN_TRY(expr)                              \
  do {                                             \
    if ((expr) != hipSuccess) return GDN_ERR_HIP;  \
  } while (0)

constexpr int64_t kMaxStride = (int64_t)1 << 23;  // a chunk's rows span less than 2^31 bytes
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // workgroups of 256 threads in one launch

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Tokens per segment, from the extents alone, so that a `saved` buffer's layout
// is its problem's (the boundaries stay on the device). Cutting a sequence costs
// two launches, a second reading of k and v and 16 D^2 bytes a segment and head,
// and makes items that run side by side.
//   Few chains (sequences x value heads): twice as long, from 128 tokens on, while
// that leaves `fill` items, of some 256 (D = 128) or 512 that run at once. Short
// segments make more states than they save time, so fewer items are enough for
// them. One sequence, 16 heads of 128, forward and backward, us:
//     tokens    128   256   512  1024  2048 a segment
//       1024     56    65
//       3000    104    92   109
//       6000    179   148   141   184
//      12288    352   284   257   262   365
//      24576          538   470   469   506
//      65536               1192  1136  1097
// and 16 heads of 64:
//       2048     44    51    69
//      10000    120   100   106   128
//      24576          228   201   224   257
//   From 128 chains on (half the CUs), and short: no cut in sequences of the mean
// length, where that takes less time by fits of these measurements (us, forward):
//                     D = 128, uncut   cut   D = 64, uncut   cut
//     16 x 1024,  8 heads         60    73              40    33
//      4 x 2048, 32 heads        108   106              64    52
//      8 x 2048, 32 heads        155   195              78    98
//     16 x 2048, 32 heads        277   419             147   201
// Fewer chains are cut by their work alone. Sequences of 1024 tokens, D = 128, us
// forward, the best cut and none: 48 chains 38 and 53, 64 chains 51 and 52, 96 chains
// 58 (72 by this rule) and 55, 128 chains 67 and 55; D = 64: 96 chains 30 and 35, 128
// chains 34 and 36, 192 chains 43 and 36.
// Uncut, a step of 64 tokens takes 3.0 us (1.9 with D = 64) while every chain has a
// CU (half a CU) to itself, and 4.5 (2.15) with 256 chains and in proportion; cut, 15
// us and 7 passes over rows at 5 TB/s. Means over 2048 are left out: where the
// lengths differ, the longest sequence's items then end long after the others (12
// sequences of 492 to 7435 tokens, 32 heads: 361 us with 2048, 469 with 4096; but 8 x
// 4096, 32 heads, 360 and 284).
int64_t segment_tokens(const gdn_linear_problem* p) {
  const int64_t work = (int64_t)p->T * p->HV, chains = (int64_t)p->N * p->HV;
  const auto fill = [&](int64_t S) { return p->K == 128 ? (S <= 1024 ? 176 : 400) : (S <= 256 ? 208 : 448); };
  int64_t S = 128;
  while (S < 4096 && 2 * S * fill(2 * S) <= work) S *= 2;
  const int64_t mean = p->N > 0 ? ((int64_t)p->T + p->N - 1) / p->N : 0;
  if (chains >= 128 && mean <= 2048) {
    const bool full = p->K == 128;
    const double step = std::max(full ? 3.0 : 1.9, (full ? 4.5 : 2.15) * (double)chains / 256);
    const double uncut = 10. + (double)mean / kChunk * step;
    const double cut = 15. + (double)work * p->K * 2 * 7 / 5e6;
    if (uncut < cut)
      while (S < mean) S *= 2;
  }
  return S;
}

bool bad_stride(int64_t s, int64_t dense) {
  return s != 0 && (s < dense || s % 8 != 0 || s >= kMaxStride);
}

gdn_status check_linear(const gdn_linear_problem* p) {
  if (!p) return GDN_ERR_NULL;
  if (p->N < 0 || p->T < 0 || p->H <= 0 || p->HV <= 0 || p->K <= 0 || p->V <= 0) return GDN_ERR_SHAPE;
  if (p->K != p->V || (p->K != 64 && p->K != 128) || p->HV % p->H != 0) return GDN_ERR_UNSUPPORTED;
  if (p->N == 0 && p->T != 0) return GDN_ERR_SHAPE;
  const int64_t qk = (int64_t)p->H * p->K, vv = (int64_t)p->HV * p->V;
  if (vv >= kMaxStride || bad_stride(p->q_stride, qk) || bad_stride(p->k_stride, qk) ||
      bad_stride(p->v_stride, vv))
    return GDN_ERR_SHAPE;
  return GDN_OK;
}

LinCut cut_of(const gdn_linear_problem* p) {
  const int64_t S = segment_tokens(p);
  return {p->cu_seqlens, p->N, p->T, p->HV, p->HV / p->H, (int)S, (int)(p->T / S + p->N)};
}

gdn_status check_pack(const gdn_linear_problem* p) {
  const gdn_status st = check_linear(p);
  if (st != GDN_OK) return st;
  const int64_t slots = (int64_t)p->T / segment_tokens(p) + p->N;
  if (2 * (slots + 8) * p->HV > kMaxBlocks ||
      (int64_t)p->N * p->HV * (p->K * p->V / 256) > 4 * kMaxBlocks)
    return GDN_ERR_SHAPE;
  if (p->cu_seqlens_host) {
    const int32_t* cu = p->cu_seqlens_host;
    if (cu[0] != 0 || cu[p->N] != p->T) return GDN_ERR_SEQLENS;
    for (int n = 0; n < p->N; ++n)
      if (cu[n + 1] < cu[n]) return GDN_ERR_SEQLENS;
  }
  return GDN_OK;
}

// As gdn_recurrent_step: an active index is in range and used once.
gdn_status check_indices(int N, int slots, const int32_t* host) {
  if (!host) return GDN_OK;
  try {
    std::vector<int32_t> act;
    for (int n = 0; n < N; ++n) {
      if (host[n] <= 0) continue;
      if (host[n] >= slots) return GDN_ERR_INDEX;
      act.push_back(host[n]);
    }
    std::sort(act.begin(), act.end());
    return std::adjacent_find(act.begin(), act.end()) == act.end() ? GDN_OK : GDN_ERR_INDEX;
  } catch (const std::bad_alloc&) {
    return GDN_ERR_INDEX;  // not checked, so not accepted
  }
}

float scale_of(const gdn_linear_problem* p) { return p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->K); }

// whether a sequence may hold more than one segment (with the host's boundaries: does)
bool several(const gdn_linear_problem* p) {
  const int64_t S = segment_tokens(p);
  if (!p->cu_seqlens_host) return p->T > S;
  for (int n = 0; n < p->N; ++n)
    if (p->cu_seqlens_host[n + 1] - p->cu_seqlens_host[n] > S) return true;
  return false;
}

size_t states_bytes(const gdn_linear_problem* p) {
  return (size_t)cut_of(p).slots * p->HV * p->K * p->V * sizeof(float);
}
size_t wide_bytes(const gdn_linear_problem* p) {  // dq or dk of every value head
  return p->HV == p->H ? 0 : (size_t)p->T * p->HV * p->K * sizeof(float);
}
// sizes do not go by the boundaries
size_t ends_bytes(const gdn_linear_problem* p) { return p->T > segment_tokens(p) ? states_bytes(p) : 0; }
size_t fwd_bytes(const gdn_linear_problem* p) { return ends_bytes(p); }
size_t bwd_bytes(const gdn_linear_problem* p) { return ends_bytes(p) + 2 * wide_bytes(p); }

LinRows rows(const uint16_t* x, int64_t stride, int heads, int G, int D) {
  return {x, stride ? stride : (int64_t)heads * D, G};
}

gdn_status check_token_args(const gdn_linear_problem* p, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const float* log_decay, const uint16_t* o) {
  if (p->T > 0 && (!q || !k || !v || !o)) return GDN_ERR_NULL;
  if (p->N > 0 && !log_decay) return GDN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

int linear_fwd(const gdn_linear_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
               const float* log_decay, const StateRef& io, uint16_t* o, void* saved, void* workspace,
               size_t workspace_bytes, void* stream) {
  gdn_status st = check_pack(p);
  if (st != GDN_OK) return st;
  st = check_token_args(p, q, k, v, log_decay, o);
  if (st != GDN_OK) return st;
  if (p->N > 0 && !p->cu_seqlens) return GDN_ERR_NULL;
  if (!aligned16(io.h0) || !aligned16(io.hT) || !aligned16(saved) || !aligned16(workspace)) return GDN_ERR_ALIGN;
  if (!saved && fwd_bytes(p) > 0 && (!workspace || workspace_bytes < fwd_bytes(p))) return GDN_ERR_WORKSPACE;
  if (p->N == 0) return GDN_OK;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const LinCut cut = cut_of(p);
  const int D = p->K, G = p->HV / p->H;
  const float scale = scale_of(p);
  const LinRows a = rows(q, p->q_stride, p->H, G, D), b = rows(k, p->k_stride, p->H, G, D),
                c = rows(v, p->v_stride, p->HV, 1, D);
  const bool cut_up = several(p);
  float* states = nullptr;  // that the segments start from, where they are needed
  if (saved) states = static_cast<float*>(saved);
  else if (cut_up) states = static_cast<float*>(workspace);
  if (cut_up) GDN_TRY(launch_lin_gather(D, false, cut, log_decay, 1.f, b, c, io.hT != nullptr, states, s));
  if (states) GDN_TRY(launch_lin_join(D, false, cut, log_decay, io, states, s));
  const LinPass pass{a, b, c, o, states, io};
  GDN_TRY(launch_lin_out(D, cut, log_decay, scale, pass, s));
  return GDN_OK;
}

}  // namespace

GDN_API size_t gdn_linear_saved_size(const gdn_linear_problem* p) {
  return check_pack(p) == GDN_OK ? states_bytes(p) : 0;
}
GDN_API size_t gdn_linear_fwd_workspace_size(const gdn_linear_problem* p) {
  return check_pack(p) == GDN_OK ? fwd_bytes(p) : 0;
}
GDN_API size_t gdn_linear_bwd_workspace_size(const gdn_linear_problem* p) {
  return check_pack(p) == GDN_OK ? bwd_bytes(p) : 0;
}

GDN_API int gdn_linear_fwd(const gdn_linear_problem* p, const uint16_t* q, const uint16_t* k,
                           const uint16_t* v, const float* log_decay, const float* h0, uint16_t* o,
                           float* hT, void* saved, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const StateRef io{h0, hT, nullptr, nullptr, 0, nullptr};
  return linear_fwd(p, q, k, v, log_decay, io, o, saved, workspace, workspace_bytes, stream);
}

GDN_API int gdn_linear_fwd_paged(const gdn_linear_problem* p, const uint16_t* q, const uint16_t* k,
                                 const uint16_t* v, const float* log_decay, float* state_pool,
                                 int32_t slots, const int32_t* ssm_state_indices,
                                 const int32_t* has_initial_state, const int32_t* indices_host,
                                 uint16_t* o, void* saved, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const gdn_status st = check_pack(p);
  if (st != GDN_OK) return st;
  if (slots < 0) return GDN_ERR_SHAPE;
  if (p->N > 0 && (!state_pool || !ssm_state_indices)) return GDN_ERR_NULL;
  if (check_indices(p->N, slots, indices_host) != GDN_OK) return GDN_ERR_INDEX;
  const StateRef io{state_pool, state_pool, ssm_state_indices, has_initial_state, slots, nullptr};
  return linear_fwd(p, q, k, v, log_decay, io, o, saved, workspace, workspace_bytes, stream);
}

GDN_API int gdn_linear_bwd(const gdn_linear_problem* p, const uint16_t* q, const uint16_t* k,
                           const uint16_t* v, const float* log_decay, const void* saved,
                           const uint16_t* dO, const float* dhT, uint16_t* dq, uint16_t* dk,
                           uint16_t* dv, float* dh0, void* workspace, size_t workspace_bytes,
                           void* stream) {
  gdn_status st = check_pack(p);
  if (st != GDN_OK) return st;
  st = check_token_args(p, q, k, v, log_decay, dO);
  if (st != GDN_OK) return st;
  if (p->T > 0 && (!dq || !dk || !dv)) return GDN_ERR_NULL;
  if (p->N > 0 && (!p->cu_seqlens || !saved)) return GDN_ERR_NULL;
  if (!aligned16(saved) || !aligned16(dhT) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(dh0) || !aligned16(workspace))
    return GDN_ERR_ALIGN;
  if (bwd_bytes(p) > 0 && (!workspace || workspace_bytes < bwd_bytes(p))) return GDN_ERR_WORKSPACE;
  if (p->N == 0) return GDN_OK;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const LinCut cut = cut_of(p);
  const int D = p->K, G = p->HV / p->H;
  const float scale = scale_of(p);
  const LinRows rq = rows(q, p->q_stride, p->H, G, D), rk = rows(k, p->k_stride, p->H, G, D),
                rv = rows(v, p->v_stride, p->HV, 1, D), ro = rows(dO, 0, p->HV, 1, D);
  char* ws = static_cast<char*>(workspace);
  const StateRef io{dhT, dh0, nullptr, nullptr, 0, nullptr}, none{};
  const float* start = static_cast<const float*>(saved);
  float* ends = several(p) ? reinterpret_cast<float*>(ws) : nullptr;  // gradients of the segments' end states
  ws += ends_bytes(p);
  const bool wide = G > 1;
  float* wq = reinterpret_cast<float*>(ws);
  float* wk = reinterpret_cast<float*>(ws + wide_bytes(p));
  const LinPass pq{ro, rv, rk, wide ? (void*)wq : dq, start, none};
  const LinPass pv{rk, rq, ro, dv, ends, io};
  const LinPass pk{rv, ro, rq, wide ? (void*)wk : dk, ends, StateRef{dhT, nullptr, nullptr, nullptr, 0, nullptr}};
  if (ends) {
    GDN_TRY(launch_lin_gather(D, true, cut, log_decay, scale, rq, ro, dh0 != nullptr, ends, s));
    GDN_TRY(launch_lin_join(D, true, cut, log_decay, io, ends, s));
  }
  GDN_TRY(launch_lin_grad(D, wide, cut, log_decay, scale, pq, pv, pk, s));
  if (wide && p->T > 0) GDN_TRY(launch_lin_fold(D, cut, wq, wk, dq, dk, s));
  return GDN_OK;
}

GDN_API int gdn_linear_step(const gdn_linear_problem* p, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const float* log_decay, float* state_pool, int32_t slots,
                            const int32_t* ssm_state_indices, const int32_t* indices_host, uint16_t* o,
                            void* stream) {
  gdn_status st = check_linear(p);
  if (st != GDN_OK) return st;
  if (p->T != p->N || slots < 0 || (int64_t)p->N * p->HV * 4 > kMaxBlocks) return GDN_ERR_SHAPE;
  st = check_token_args(p, q, k, v, log_decay, o);
  if (st != GDN_OK) return st;
  if (p->N > 0 && (!state_pool || !ssm_state_indices)) return GDN_ERR_NULL;
  if (!aligned16(state_pool)) return GDN_ERR_ALIGN;
  if (check_indices(p->N, slots, indices_host) != GDN_OK) return GDN_ERR_INDEX;
  if (p->N == 0) return GDN_OK;
  const int D = p->K, G = p->HV / p->H;
  GDN_TRY(launch_lin_step(D, p->N, p->HV, scale_of(p), rows(q, p->q_stride, p->H, G, D),
                          rows(k, p->k_stride, p->H, G, D), rows(v, p->v_stride, p->HV, 1, D), log_decay,
                          state_pool, slots, ssm_state_indices, o, reinterpret_cast<hipStream_t>(stream)));
  return GDN_OK;
}
