// New tokens' keys and values into a paged cache, k turned by rotary positions
// on the way, and q turned beside them, in one launch.
//
// Bound by HBM, or for a batch of single tokens by the latency of one pass:
// boundaries or the token's own place, page, row. A workgroup takes one token
// (or four whose rows are short): its angles go to LDS once, its cache row is
// found once, then its threads go over the pieces of 16 bytes of q's, k's and
// v's heads. 32768 tokens of 16 + 4 heads of 128, 96 columns turning: 99 us, 4.1 TB/s (none
// turning 75); one token 3.8 us.
#include <algorithm>

#include "attn_tile.h"
#include "rotary_unit.h"

namespace gdn {

namespace {

constexpr int kTok = 4;  // tokens a workgroup where one token has at most 64 pieces

// Sequence and place in it of token t: the last sequence that begins at or before t,
// 64 probes a step. Boundaries are only compared.
struct Place {
  int seq, at;
  bool live;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t) {
  if (!a.cu) return {t, 0, true};
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = a.N;
  while (cnt > 1) {
    const int step = (cnt + 63) >> 6, at = lane * step;
    const bool ok = at < cnt && a.cu[lo + at] <= t;
    const int k = max(__popcll(__ballot(ok)) - 1, 0);
    lo += k * step;
    cnt = min(step, cnt - k * step);
  }
  const int b = a.cu[lo];
  return {lo, t - b, t >= b && t < a.cu[lo + 1]};
}

}  // namespace

template <typename T, int V, bool kInter, bool kWide, int kTokens>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a, int first) {
  extern __shared__ float2 cs[];  // [kTokens][R / 2]
  __shared__ bool live[kTokens];
  __shared__ int64_t to[kTokens];  // the token's row in the cache, or -1
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int t0 = first + blockIdx.x * kTokens, pairs = a.R / 2;
  // a wave for each token, or all four for one
  const int mine = kTokens == 1 ? 0 : wave;
  if (t0 + mine < a.T) {
    const Place at = place_of(a, t0 + mine);
    const int64_t pos = (int64_t)a.pages.offsets[at.seq] + at.at;
    if (lane == 0) {
      live[mine] = at.live;
      to[mine] = at.live && pos >= 0 && pos < 0x7fffffff ? row_at(a.pages, at.seq, (int)pos, 0x7fffffff) : -1;
    }
    for (int j = kTokens == 1 ? tid : lane; j < pairs; j += kTokens == 1 ? 256 : 64) {
      const float2 t = turn_of(pos, a.inv_freq[j]);
      cs[mine * pairs + j] = make_float2(t.x * a.mscale, t.y * a.mscale);
    }
  }
  __syncthreads();
  const int turning = turning_units<V, kInter>(a.R), units = turning + copied_units<V>(a.D, a.R);
  const int whole = copied_units<V>(a.D, 0);  // of a head of v
  const int nq = a.q.heads * units, nk = a.k.heads * units, n = nq + nk + a.k.heads * whole;
  for (int i = tid; i < n * kTokens; i += 256) {
    const int tok = i / n, rest = i - tok * n;
    const int64_t t = t0 + tok;
    if (t >= a.T || !live[tok]) continue;
    const float2* turns = cs + tok * pairs;
    if (rest < nq) {
      const int h = rest / units, u = rest - h * units;
      const T* in = static_cast<const T*>(a.q.in) + t * a.q.in_stride + (int64_t)h * a.D;
      T* out = static_cast<T*>(a.q.out) + t * a.q.out_stride + (int64_t)h * a.D;
      if (u >= turning && in == out) continue;  // in place: nothing to copy
      unit<T, V, kInter, kWide>(in, out, turns, u, turning, a.D, a.R);
    } else if (to[tok] >= 0) {
      if (rest < nq + nk) {
        const int h = (rest - nq) / units, u = rest - nq - h * units;
        const T* in = static_cast<const T*>(a.k.in) + t * a.k.in_stride + (int64_t)h * a.D;
        unit<T, V, kInter, kWide>(in, static_cast<T*>(a.pages.k) + to[tok] + h * a.pages.head_stride, turns, u, turning,
                                  a.D, a.R);
      } else {
        const int h = (rest - nq - nk) / whole, c = (rest - nq - nk - h * whole) * V;
        const T* in = static_cast<const T*>(a.v) + t * a.v_stride + (int64_t)h * a.D;
        float x[V];
        load_unit<T, V, kWide>(in, c, a.D, x);
        store_unit<T, V, kWide>(static_cast<T*>(a.pages.v) + to[tok] + h * a.pages.head_stride, c, a.D, x);
      }
    }
  }
}

namespace {

// A launch counts its threads in 32 bits: more tokens than these workgroups of 256
// threads take go in several launches.
constexpr int kMaxBlocks = 1 << 23;

template <typename T, bool kInter, bool kWide, int kTokens>
hipError_t append_launches(const AppendArgs& a, hipStream_t s) {
  const size_t lds = kTokens * sizeof(float2) * (a.R / 2);
  for (int64_t first = 0; first < a.T; first += (int64_t)kMaxBlocks * kTokens) {
    const int blocks = (int)std::min((a.T - first + kTokens - 1) / kTokens, (int64_t)kMaxBlocks);
    hipLaunchKernelGGL((kv_append_kernel<T, 8, kInter, kWide, kTokens>), dim3(blocks), dim3(256), lds, s, a, (int)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, bool kInter, bool kWide>
hipError_t append_of(const AppendArgs& a, hipStream_t s) {
  const int64_t units = turning_units<8, kInter>(a.R) + copied_units<8>(a.D, a.R);
  const int64_t n = units * (a.q.heads + a.k.heads) + (int64_t)copied_units<8>(a.D, 0) * a.k.heads;
  return n * kTok <= 256 ? append_launches<T, kInter, kWide, kTok>(a, s) : append_launches<T, kInter, kWide, 1>(a, s);
}

template <typename T>
hipError_t append_type(bool inter, bool wide, const AppendArgs& a, hipStream_t s) {
  if (inter) return wide ? append_of<T, true, true>(a, s) : append_of<T, true, false>(a, s);
  return wide ? append_of<T, false, true>(a, s) : append_of<T, false, false>(a, s);
}

}  // namespace

hipError_t launch_kv_append(Elem type, bool inter, bool wide, const AppendArgs& a, hipStream_t s) {
  return type == Elem::kBf16 ? append_type<Bf16>(inter, wide, a, s) : append_type<Fp16>(inter, wide, a, s);
}

}  // namespace gdn
