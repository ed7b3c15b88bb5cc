// Gradients of the causal softmax attention over packed sequences. With the
// forward's lse, P = e^(scale s - lse), delta = dO . o = sum P (dO V^T) for each row, and
//   dS = scale P (dO V^T - delta):   dq = dS K,   dk = dS^T q,   dv = P^T dO,
// the rows of all query heads of a key head summed in dk and dv.
//
// Two kernels, without atomics: one goes over the keys for its rows (dq, and
// the rows' statistics on the way), the other over the rows for 128 keys, 64 with
// 256 columns (dk, dv). Both form the scores and dO V^T again: seven products instead
// of the five that one kernel with atomic sums of dq would take. As in the forward,
// each operand that follows from scores is used where it stands in the accumulator.
//
// Bound by the matrix unit and the waits around it. 2 x 8192 tokens, 16 + 2 heads
// of 256 columns: dq 1.52 ms (1.09 PFLOP/s of its three products), dk and dv 2.6 to 2.7 ms
// (0.83, of four); window 1024, 16 + 4 heads of 128: 250 us, 420 us, joining 13 us.
//
// P and dS are rounded once to the inputs' type, where they are multiplied; all
// sums are fp32. fp16's range is short for dS, which falls with the number of keys
// and with the cotangent's size: it is multiplied in units of a power of two that
// follows its largest value (see refit), dq and dk are taken back at the end. 8192 keys of 128
// columns, a cotangent of size 0.001: dq is 0.0005 of its norm off, of which 0.0004 is its own rounding;
// in one unit for all it was 0.024. Weights are in one unit, 2^-14. It costs the backward in fp16 3 to 6 %.
#include <algorithm>

#include "attn_tile.h"

namespace gdn {

namespace {

constexpr int kGradKeys = 64;  // keys a step of dq's kernel
constexpr int grad_threads(int D) { return D == 128 ? 512 : 256; }
// Fewest keys of a row whose delta is formed from the rounded o. dO V^T - delta cancels most where few keys are seen, and o's
// rounding then weighs more than dS's own: sequences of 1 and 2 tokens, 8 + 2 heads of 256, bf16, dq 0.0042 of its norm off, with delta
// from the weights 0.0023; from n keys on the share is o's rounding over sqrt(n). It costs the tiles at a sequence's
// start, and all those of such a window, one more pass over their keys (16384 tokens, 16 + 4 heads of 128, backward: 256
// sequences of 64 197 us without, 193 with it; window of 32 168 and 180).
constexpr int kFewKeys = 64;
constexpr int kGradRows = 64;  // rows a step of dk's and dv's kernel, one to a lane, in parts of 32

template <typename T>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  T x[8], y[8];
  __builtin_memcpy(x, &a, 16);
  __builtin_memcpy(y, &b, 16);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(to_f32(x[i]), to_f32(y[i]), s);
  return s;
}

// fp16: the factor for score gradients whose largest is `top` (in the present unit), 1 where they are between
// 2^7 and 2^15: then none is past fp16's largest, and what is lost of one is at most 2^-32 of the largest. Else
// the largest comes to 2^10 .. 2^11, and stays for some growth. unit: at most 2^40, so that sums in it are far
// from fp32's end; zeros, infinities and NaN change nothing.
// and for weights, which are at most 1: in units of 2^-14 all down to 2^-28 have full precision
constexpr int kWeightUnit = 14;
constexpr float kUnitLeast = 128.f, kUnitMost = 32768.f, kUnitEnd = 1099511627776.f;
__device__ __forceinline__ bool ill_fit(float top, float unit) {
  return (top > kUnitMost && top < INFINITY) || (top < kUnitLeast && top > 0.f && unit < kUnitEnd);
}
__device__ __forceinline__ float refit(float top, float unit) {
  const int most = 41 - __builtin_amdgcn_frexp_expf(unit);  // unit = 2^(its exponent - 1)
  return ldexpf(1.f, min(11 - __builtin_amdgcn_frexp_expf(top), most));
}

}  // namespace

template <typename T, int D>
__global__ __launch_bounds__(2 * attn_rows(D), D == 256 ? 1 : 2) void attn_grad_q_kernel(AttnGradArgs a) {
  constexpr int kT = kGradKeys, N = D / 16, DB = D / 32, kThreads = 2 * attn_rows(D);
  constexpr bool kUnits = kHasUnits<T>;
  typedef Tile<D, kT, kThreads> KTile;
  __shared__ __attribute__((aligned(16))) typename KTile::Lds k0, k1, v0, v1;
  const AttnPack& pk = a.pack;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l32 = lane & 31, hi = lane >> 5;
  const int hk = blockIdx.x % pk.HK;
  const int G = pk.G.by, per = attn_rows(D) / G;
  const RowTile rt = tile_of(pk.cu, pk.N, pk.T, per, a.slots, blockIdx.x / pk.HK, true, [](int) { return 0; });
  if (rt.tokens <= 0) return;
  const int t0 = rt.first;
  const KeyTiles kt = key_tiles<kT>(t0, t0 + rt.tokens - 1, rt.len, pk.window, pk.sinks);

  const int row = wave * 32 + l32;
  const int token = divide(row, pk.G), head = hk * G + row - token * G;
  const bool live = token < rt.tokens;
  const int t = t0 + token;
  const int wlo = t0 + divide(wave * 32, pk.G);
  const int whi = t0 + min(divide(wave * 32 + 31, pk.G), rt.tokens - 1);
  const int64_t out = (int64_t)(rt.bos + t0 + token) * pk.HQ + head;

  // Rows past the tile's tokens read its last token, and have no weights. All requests go out before one is waited for.
  const int64_t from_token = rt.bos + t0 + min(token, rt.tokens - 1), from_row = from_token * pk.HQ + head;
  uint4 q[N], g[N], y[N];
  {
    const uint16_t* pq = static_cast<const uint16_t*>(a.q) + from_token * a.q_stride + head * D + 8 * hi;
    const uint16_t* pg = static_cast<const uint16_t*>(a.dO) + from_row * D + 8 * hi;
    const uint16_t* po = static_cast<const uint16_t*>(a.o) + from_row * D + 8 * hi;
#pragma unroll
    for (int s = 0; s < N; ++s) {
      q[s] = *reinterpret_cast<const uint4*>(pq + 16 * s);
      g[s] = *reinterpret_cast<const uint4*>(pg + 16 * s);
      y[s] = *reinterpret_cast<const uint4*>(po + 16 * s);
    }
  }
  float lse = a.lse[from_row] * kLog2e, delta = 0.f;
  if (!live || lse == kMinusInf) lse = INFINITY;  // weights of rows that see nothing are zeros

  const uint16_t* kbase = static_cast<const uint16_t*>(a.k) + rt.bos * a.k_stride + hk * D;
  const uint16_t* vbase = static_cast<const uint16_t*>(a.v) + rt.bos * a.v_stride + hk * D;
  const TokenRows<KTile> kr((int)a.k_stride, tid), vr((int)a.v_stride, tid);
  auto tokens = [&](const uint16_t* base, int64_t stride, int i) {
    const int j0 = kt.at(i) * kT;
    return TokenRows<KTile>::from(base + j0 * stride, (int)stride, i < kt.count ? min(kT, rt.len - j0) : 0, D);
  };

  f32x16 dq[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) zero16(dq[i]);
  const float c = pk.scale * kLog2e;
  float scale = pk.scale, scaled = 0.f;  // scaled: scale times delta
  float unit = 1.f, largest = 0.f;       // kUnits: of this row's dS; scale, scaled and dq are in it
  const int ka = at<D>(l32, 8 * hi);
  const int j16 = lane & 15, vrow = 4 * hi + (j16 >> 2), vcol = 16 * ((lane >> 4) & 1) + 4 * (j16 & 3);
  const int va = at<D>(vrow, vcol), vb = at<D>(vrow + 8, vcol);
  const int from = pk.window ? t - pk.window : -1;  // keys in the window are past this

  // 64 keys from j0 in LDS, in two halves. The matrix instructions go in the order S0, dO V0^T, S1, dO V1^T, dq of
  // the first half, of the second, each with its LDS operand requested kAhead before; the vector unit
  // forms the weights and the scores' gradients of a half during the products that follow it.
  auto part = [&](const uint16_t* K, const uint16_t* V, int j0, const auto& fetch) {
    constexpr int kAhead = 6;
    f32x16 s[2], dp[2];
    const int j1 = j0 + kT - 1;
    bool mask = j1 > wlo;
    if (pk.window) mask = mask || (j0 <= whi - pk.window && j1 >= pk.sinks);
    const int kf = fresh(ka), c0 = fresh(va), c1 = fresh(vb);
    uint4 op[kAhead], ds[4];
    auto read = [&](auto slot) {
      constexpr int n = slot, phase = n / N, d = n % N;
      uint4& x = op[n % kAhead];
      if constexpr (phase < 4)
        x = *reinterpret_cast<const uint4*>((phase % 2 ? V : K) + (kf ^ (16 * d)) + 32 * (phase / 2) * D);
      else
        x = column8(K + (32 * (phase - 4) + 16 * (d / DB)) * D, c0 ^ (32 * (d % DB)), c1 ^ (32 * (d % DB)));
    };
    for_each<kAhead>(read);
    auto run = [&](auto slot) {
      constexpr int n = slot, phase = n / N, d = n % N;
      const uint4& x = op[n % kAhead];
      if constexpr (phase >= 4) dq[d % DB] = mfma32_of<T>(x, ds[2 * (phase - 4) + d / DB], dq[d % DB]);
      else if constexpr (phase % 2) dp[phase / 2] = mfma32_of<T>(x, g[d], d == 0 ? f32x16{} : dp[phase / 2]);
      else s[phase / 2] = mfma32_of<T>(x, q[d], d == 0 ? f32x16{} : s[phase / 2]);
      if constexpr (n + kAhead < 6 * N) read(std::integral_constant<int, n + kAhead>());
      fetch(slot);
      if constexpr (phase >= 1 && phase <= 4) {
        constexpr int half = (phase - 1) / 2;
        // the argument or difference in one slot, the rest in the next
        for_each<16>([&](auto element) {
          constexpr int e = element, at = e * (N - 1) / 16;
          if constexpr (phase % 2) {
            if constexpr (d == at) s[half][e] = fmaf(s[half][e], c, -lse);
            if constexpr (d == at + 1) s[half][e] = exp2_fast(s[half][e]);
          } else {
            if constexpr (d == at) dp[half][e] = fmaf(dp[half][e], scale, -scaled);
            if constexpr (d == at + 1) dp[half][e] *= s[half][e];
          }
        });
        if constexpr (phase % 2 == 0 && d == N - 1) {
          if constexpr (kUnits) {
            float top = 0.f;
            for_each<16>([&](auto element) {
              constexpr int e = element;
              top = fmaxf(top, fabsf(dp[half][e]));
            });
            const float2 tops = both_halves(top);
            largest = fmaxf(largest, fmaxf(tops.x, tops.y));
            const bool ill = ill_fit(largest, unit);
            if (__any(ill)) {
              const float by = ill ? refit(largest, unit) : 1.f;
              unit *= by;
              largest *= by;
              scale *= by;
              scaled *= by;
              dp[half] *= by;
#pragma unroll
              for (int i = 0; i < DB; ++i) {
                keep_accumulated<D == 256>(dq[i]);
                dq[i] *= by;
                keep_accumulated<D == 256>(dq[i]);
              }
            }
          }
          ds[2 * half] = operand<T>(dp[half], 0);
          ds[2 * half + 1] = operand<T>(dp[half], 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto hide = [&](auto half) {
      if (!mask) return;
      // positions relative to the lane's first key
      const int first = j0 + 4 * hi, most = t - first, least = from - first, sunk = pk.sinks - first;
      for_each<16>([&](auto element) {
        constexpr int e = element, j = 32 * half + 8 * (e / 4) + e % 4;
        s[half][e] = j <= most && (j > least || j < sunk) ? s[half][e] : kMinusInf;
      });
    };
    for_each<N>(run);
    hide(std::integral_constant<int, 0>());
    for_each<2 * N>([&](auto slot) { run(std::integral_constant<int, slot + N>()); });
    hide(std::integral_constant<int, 1>());
    for_each<3 * N>([&](auto slot) { run(std::integral_constant<int, slot + 3 * N>()); });
  };
  auto keep = [&] {
#pragma unroll
    for (int d = 0; d < DB; ++d) keep_accumulated<D == 256>(dq[d]);
  };

  // one step: tile i in (k, v), the next on its way to (nk, nv), a request every second slot. (A third buffer, with requests two
  // steps ahead, gained nothing in either kernel: 2 x 8192 tokens, window 1024, 16 + 4 heads of 128, 740 us for both, 723 without.)
  constexpr int P = KTile::kPieces;
  auto step = [&](int i, auto& k, auto& v, auto& nk, auto& nv) {
    const int j0 = kt.at(i) * kT, j1 = j0 + kT - 1;
    const auto krows = tokens(kbase, a.k_stride, i + 1), vrows = tokens(vbase, a.v_stride, i + 1);
    auto fetch = [&](auto slot) {
      constexpr int n = slot, r = n / 2;
      if constexpr (n % 2 == 0 && r < P) kr.request(nk, r, krows, tid);
      if constexpr (n % 2 == 0 && r >= P && r < 2 * P) vr.request(nv, r - P, vrows, tid);
    };
    keep();
    bool some = i < kt.count && wlo <= whi && j0 <= whi;
    if (pk.window) some = some && (j1 > wlo - pk.window || j0 < pk.sinks);
    if (some) part(k, v, j0, fetch);
    else for_each<4 * P>(fetch);
    keep();
    __syncthreads();
  };
  auto fill = [&](int i, auto& k, auto& v) {
    const auto krows = tokens(kbase, a.k_stride, i), vrows = tokens(vbase, a.v_stride, i);
    for_each<P>([&](auto n) {
      kr.request(k, n, krows, tid);
      vr.request(v, n, vrows, tid);
    });
  };
  // delta from o as it was rounded, or where a row may see few keys from the weights, in a pass of its own
  if (t0 < kFewKeys || (pk.window && (int64_t)pk.window + pk.sinks < kFewKeys)) {
#pragma unroll 1
    for (int i = 0; i < kt.count; ++i) {
      fill(i, k0, v0);
      __syncthreads();
      const int j0 = kt.at(i) * kT;
      for_each<2>([&](auto half) {
        f32x16 s, dp;
#pragma unroll
        for (int d = 0; d < N; ++d) {
          const int at = (fresh(ka) ^ (16 * d)) + 32 * half * D;
          s = mfma32_of<T>(*reinterpret_cast<const uint4*>(k0 + at), q[d], d == 0 ? f32x16{} : s);
          dp = mfma32_of<T>(*reinterpret_cast<const uint4*>(v0 + at), g[d], d == 0 ? f32x16{} : dp);
        }
        const int first = j0 + 4 * hi, most = t - first, least = from - first, sunk = pk.sinks - first;
        for_each<16>([&](auto element) {
          constexpr int e = element, j = 32 * half + 8 * (e / 4) + e % 4;
          const float x = j <= most && (j > least || j < sunk) ? s[e] : kMinusInf;
          delta = fmaf(exp2_fast(fmaf(x, c, -lse)), dp[e], delta);
        });
      });
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int s = 0; s < N; ++s) delta += dot8<T>(y[s], g[s]);
  }
  fill(0, k0, v0);
  delta = sum_halves(delta);
  scaled = scale * delta;
  if (live && hi == 0) {
    a.stats[out] = kUnits ? lse - kWeightUnit : lse;  // the other kernel's weights are in their unit
    a.stats[(int64_t)pk.T * pk.HQ + out] = scaled;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < kt.count; i += 2) {  // a step past the last tile does nothing
    step(i, k0, v0, k1, v1);
    step(i + 1, k1, v1, k0, v0);
  }
  if (!live) return;
  const float back = 1.f / unit;
  if (kUnits && hi == 0) a.stats[2 * (int64_t)pk.T * pk.HQ + out] = largest * back;
  uint16_t* p = static_cast<uint16_t*>(a.dq) + out * D;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<uint4*>(p + 32 * d + 16 * u + 8 * hi) = eight_columns<T>(dq[d], u, back);
}

// The rows of a sequence that see some of its keys j0 .. j0 + keys - 1: in the window, or behind it
// (far, sinks only). In rows of the G query heads, r = token G + head.
struct RowRange {
  int from, to;
};
__device__ __forceinline__ RowRange rows_of(const AttnPack& pk, int len, int j0, int keys, bool far) {
  const int G = pk.G.by;
  const int64_t W = pk.window;
  if (far) return {(int)min(j0 + W, (int64_t)len) * G, len * G};
  return {j0 * G, (int)(W ? min(j0 + keys - 1 + W, (int64_t)len) : len) * G};
}

// Where a part of the gradients of key tokens goes: [parts][tokens][HK][dk, dv][D] fp32. The parts of
// sinks hold the first `far_tiles` tiles of every sequence, side by side, or where that is more than the
// pack's tokens, by token.
__device__ __forceinline__ int64_t far_rows(const AttnGradArgs& a, int D) {
  return min((int64_t)a.pack.N * a.far_tiles * attn_keys(D), (int64_t)a.pack.T);
}
__device__ __forceinline__ float* far_at(const AttnGradArgs& a, int part, const RowTile& kt, int token, int hk, int D) {
  const int64_t rows = far_rows(a, D), dense = (int64_t)a.far_tiles * attn_keys(D);
  const int64_t r = rows < a.pack.N * dense ? kt.bos + token : kt.seq * dense + token;
  return a.far + (((part * rows + r) * a.pack.HK + hk) * 2) * D;
}
__device__ __forceinline__ float* part_at(const AttnGradArgs& a, int part, const RowTile& kt, int token, int hk, int D) {
  return a.part + ((((int64_t)part * a.pack.T + kt.bos + token) * a.pack.HK + hk) * 2) * D;
}

// Tile i of those with sinks: of every sequence its first far_tiles, or where that is more than all tiles there may be,
// all slots in the pack's order.
__device__ __forceinline__ RowTile far_tile(const AttnGradArgs& a, int i, int keys) {
  const AttnPack& pk = a.pack;
  RowTile t;
  if ((int64_t)pk.N * a.far_tiles > a.far_slots) {
    t = find_tile(pk.cu, pk.N, pk.T, keys, i);
    if (t.first / keys >= a.far_tiles) t.tokens = 0;
    return t;
  }
  t.seq = i / a.far_tiles;
  t.bos = min(max(pk.cu[t.seq], 0), pk.T);
  t.len = min(max(pk.cu[t.seq + 1], t.bos), pk.T) - t.bos;
  t.first = i % a.far_tiles * keys;
  t.tokens = min(keys, t.len - t.first);
  return t;
}

// Workgroups from number `launched` on, as many as the grid has.
template <typename T, int D>
__global__ __launch_bounds__(grad_threads(D), D == 256 ? 1 : 2) void attn_grad_kv_kernel(AttnGradArgs a, int launched) {
  // From 128 columns on two waves share the accumulators of 32 keys: each forms the scores of half of a step's rows, they
  // exchange the weights and the scores' gradients as operands through LDS, and each adds all rows up in half of the
  // columns. 256 columns would fill all registers otherwise; with 128 a SIMD then holds two waves instead of one (2 x 8192
  // tokens, window 1024, 16 + 4 heads, backward: 727 us with a wave for 32 keys, 672 in pairs).
  constexpr bool kPair = D >= 128, kUnits = kHasUnits<T>;
  constexpr int kThreads = grad_threads(D);
  constexpr int kR = kGradRows, kKeys = attn_keys(D), N = D / 16, DB = D / 32 / (kPair ? 2 : 1), M = 2 * DB;
  typedef Tile<D, kR, kThreads> RTile;
  __shared__ __attribute__((aligned(16))) typename RTile::Lds q0, q1, g0, g1;  // q and dO
  // lse, then delta; kUnits: and the largest dS
  __shared__ __attribute__((aligned(16))) float stats0[(kUnits ? 3 : 2) * kR], stats1[(kUnits ? 3 : 2) * kR];
  __shared__ uint4 exchange[kPair ? kThreads / 64 : 1][4][64];  // [wave][two operands of weights, two of gradients][lane]
  const AttnPack& pk = a.pack;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l32 = lane & 31, hi = lane >> 5;
  const int G = pk.G.by;
  int b = launched + blockIdx.x;
  const int hk = b % pk.HK;
  b /= pk.HK;
  const int role = kPair ? wave & 1 : 0, keys0 = (kPair ? wave >> 1 : wave) * 32, col0 = role * (D / 2);
  // first the rows behind the windows of the sinks' tiles, then all tiles' rows
  const int far_items = a.far_pieces * a.far_slots;
  const bool far = b < far_items;
  int piece, pieces;
  RowTile kt;
  if (far) {
    pieces = a.far_pieces;
    piece = b % pieces;
    kt = far_tile(a, b / pieces, kKeys);
  } else {
    b -= far_items;
    pieces = a.pieces;
    piece = b % pieces;
    kt = tile_of(pk.cu, pk.N, pk.T, kKeys, a.key_slots, b / pieces, false, [](int) { return 0; });
  }
  if (kt.tokens <= 0) return;
  const RowRange all = rows_of(pk, kt.len, kt.first, kKeys, far);
  const int steps = (all.to - all.from + kR - 1) / kR, share = (steps + pieces - 1) / pieces;
  const int from = all.from + min(piece * share, steps) * kR, to = min(all.to, from + share * kR);

  const int key = keys0 + l32, j = kt.first + key;
  const bool live = key < kt.tokens;
  uint4 k[N], v[N];
  {
    // keys past the tile's tokens read its last token; no row sees them
    const int64_t token = kt.bos + kt.first + min(key, kt.tokens - 1);
    const uint16_t* pkk = static_cast<const uint16_t*>(a.k) + token * a.k_stride + hk * D + 8 * hi;
    const uint16_t* pv = static_cast<const uint16_t*>(a.v) + token * a.v_stride + hk * D + 8 * hi;
#pragma unroll
    for (int s = 0; s < N; ++s) {
      k[s] = *reinterpret_cast<const uint4*>(pkk + 16 * s);
      v[s] = *reinterpret_cast<const uint4*>(pv + 16 * s);
    }
  }
  // rows that see this lane's key, and the wave's keys
  const int W = pk.window, wlo = kt.first + keys0, whi = wlo + 31;
  const int64_t none = (int64_t)1 << 40, lim = (int64_t)kt.len * G;
  int64_t seen_from = (int64_t)j * G, seen_to = W ? min(((int64_t)j + W) * G, lim) : lim;
  if (far) {
    seen_from = j < pk.sinks ? ((int64_t)j + W) * G : none;
    seen_to = lim;
  }
  const int lo = (int)min(seen_from, lim), up = (int)seen_to;  // lim < 2^31

  const uint16_t* qbase = static_cast<const uint16_t*>(a.q) + kt.bos * a.q_stride + hk * G * D;
  const uint16_t* gbase = static_cast<const uint16_t*>(a.dO) + (int64_t)kt.bos * pk.HQ * D + hk * G * D;
  const float c = pk.scale * kLog2e;
  // kUnits: of dS, by the largest of a step's 64 rows, which all waves know; dk is in it, and scale and low, the factors
  // of what a weight, in its own unit, is multiplied by
  constexpr float kWeight = kUnits ? 1.f / (1 << kWeightUnit) : 1.f;
  float unit = 1.f, low = kWeight, scale = pk.scale * kWeight;
  const int per_token = (65535 + G) / G;  // r / G = r per_token / 2^16 for r below 2^9
  // a step's rows from r0 on: offsets from its first token, its rows are of at most kR + 1 tokens
  struct Rows {
    __amdgpu_buffer_rsrc_t q, g;
    int first, before, count;
  };
  // Without a window a sequence's tiles all see its last rows, and go from those to the first: workgroups side by side then
  // read the same rows at one time. (From the first on, each begins at its own: 2 x 8192 tokens, 16 + 2 heads of 256, 2780 us.)
  const int n_steps = from < to ? (to - from + kR - 1) / kR : 0;
  auto row_of = [&](int i) { return from + (W ? i : n_steps - 1 - i) * kR; };
  auto rows_from = [&](int i) {
    const int r0 = i < n_steps ? row_of(i) : from;
    Rows r;
    r.first = __builtin_amdgcn_readfirstlane(divide(r0, pk.G));
    r.before = r0 - r.first * G;
    r.count = i < n_steps ? to - r0 : 0;
    r.q = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(qbase) + r.first * a.q_stride, 0, 0x7ffffff0, kBufferWord3);
    r.g = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(gbase) + (int64_t)r.first * pk.HQ * D, 0, 0x7ffffff0,
                                            kBufferWord3);
    return r;
  };
  auto request = [&](auto piece, auto& qs, auto& gs, const Rows& rows) {
    constexpr int i = piece;
    const int row = RTile::row(i, fresh(tid)), r = rows.before + row;
    const int token = __umul24(r, per_token) >> 16, h = r - __umul24(token, G), col = h * D + RTile::column(i, tid);
    const bool ok = row < rows.count;  // others are past the resource: zeros
    RTile::request(qs, i, rows.q, ok ? (__umul24(token, (int)a.q_stride) + col) * 2 : -1, tid);
    RTile::request(gs, i, rows.g, ok ? (__umul24(token, pk.HQ * D) + col) * 2 : -1, tid);
  };
  // The rows' statistics as the other kernel wrote them: even waves request lse, odd ones delta, one request each in every wave
  // (kUnits: and the rows' largest dS).
  auto request_stat = [&](auto& stats, const Rows& rows, int which) {
    const int r = rows.before + lane, token = __umul24(r, per_token) >> 16, h = r - __umul24(token, G);
    const float* p = a.stats + (which * (int64_t)pk.T + kt.bos + rows.first) * pk.HQ + hk * G;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), 0, 0x7ffffff0, kBufferWord3),
        (__attribute__((address_space(3))) void*)(stats + which * kR), 4,
        lane < rows.count ? (__umul24(token, pk.HQ) + h) * 4 : -1, 0, 0, 0);
  };
  auto request_stats = [&](auto& stats, const Rows& rows) {
    request_stat(stats, rows, wave & 1);
    if constexpr (kUnits) request_stat(stats, rows, 2);
  };

  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) {
    zero16(dk[i]);
    zero16(dv[i]);
  }
  const int own = role * 32 * D, others = (1 - role) * 32 * D;  // kPair: the waves' halves of a step's rows
  const int ka = at<D>(l32, 8 * hi) + own;
  const int j16 = lane & 15, vr = 4 * hi + (j16 >> 2), vc = 16 * ((lane >> 4) & 1) + 4 * (j16 & 3);
  const int va = at<D>(vr, col0 + vc), vb = at<D>(vr + 8, col0 + vc);
  // rows that see any and all of the wave's keys
  const int64_t any_from = far ? ((int64_t)wlo + W) * G : (int64_t)wlo * G;
  const int64_t any_to = far ? (wlo < pk.sinks ? lim : 0) : W ? ((int64_t)whi + W) * G : lim;
  const int64_t all_from = far ? (whi < pk.sinks ? ((int64_t)whi + W) * G : none) : (int64_t)whi * G;
  const int64_t all_to = !far && W ? ((int64_t)wlo + W) * G : lim;

  // 32 rows at r0 with their q, dO and stats in LDS. The matrix instructions go in the order S, dO V^T, dv, dk, each
  // with its LDS operand requested kAhead before, and what the vector unit does in between: the weights
  // during dO V^T, the scores' gradients during dv. (The compiler keeps the order of the slots.) kPair: Q and O hold both
  // waves' rows, r0 is this wave's; after its own dv and dk come those of the other's rows.
  auto part = [&](const uint16_t* Q, const uint16_t* O, const float* ls, const float* de, int r0, const auto& fetch) {
    constexpr int kOwn = 2 * N + 2 * M, kSlots = kOwn + (kPair ? 2 * M : 0), kAhead = 6;
    f32x16 s, dp;
    const int kf = fresh(ka), c0 = fresh(va) + own, c1 = fresh(vb) + own;
    const int e0 = fresh(va) + others, e1 = fresh(vb) + others;
    uint4 op[kAhead], p[2], ds[2];
    auto read = [&](auto slot) {
      constexpr int n = slot;
      uint4& x = op[n % kAhead];
      if constexpr (n < 2 * N) {
        x = *reinterpret_cast<const uint4*>((n < N ? Q : O) + (kf ^ (16 * (n % N))));
      } else {
        constexpr int d = (n - 2 * N) % M;
        const uint16_t* rows = ((n - 2 * N) / M % 2 ? Q : O) + 16 * (d / DB) * D;
        x = column8(rows, (n < kOwn ? c0 : e0) ^ (32 * (d % DB)), (n < kOwn ? c1 : e1) ^ (32 * (d % DB)));
      }
    };
    f32x4 stat;
    for_each<kAhead>(read);
    auto run = [&](auto slot) {
      constexpr int n = slot;
      const uint4& x = op[n % kAhead];
      if constexpr (n < N) {
        s = mfma32_of<T>(x, k[n], n == 0 ? f32x16{} : s);
      } else if constexpr (n < 2 * N) {
        dp = mfma32_of<T>(x, v[n - N], n == N ? f32x16{} : dp);
      } else if constexpr ((n - 2 * N) / M % 2 == 0) {
        constexpr int d = (n - 2 * N) % M;
        dv[d % DB] = mfma32_of<T>(x, p[d / DB], dv[d % DB]);
      } else {
        constexpr int d = (n - 2 * N) % M;
        dk[d % DB] = mfma32_of<T>(x, ds[d / DB], dk[d % DB]);
      }
      if constexpr (n + kAhead < kSlots) read(std::integral_constant<int, n + kAhead>());
      fetch(slot);
      // the weights of 16 rows, then their gradients: the argument or difference in one slot, the rest in the next
      for_each<16>([&](auto element) {
        constexpr int e = element, weight = N + e * (N - 1) / 16, gradient = 2 * N + e * (M - 1) / 16;
        if constexpr (n == weight) {
          if constexpr (e % 4 == 0) stat = *reinterpret_cast<const f32x4*>(ls + 2 * e + 4 * hi);
          s[e] = fmaf(s[e], c, -stat[e % 4]);
        }
        if constexpr (n == weight + 1) s[e] = exp2_fast(s[e]);
        if constexpr (n == gradient) {
          if constexpr (e % 4 == 0) stat = *reinterpret_cast<const f32x4*>(de + 2 * e + 4 * hi);
          if constexpr (kUnits) stat[e % 4] *= low;
          dp[e] = fmaf(dp[e], scale, -stat[e % 4]);
        }
        if constexpr (n == gradient + 1) dp[e] *= s[e];
      });
      if constexpr (n == 2 * N - 1) {
        p[0] = operand<T>(s, 0);
        p[1] = operand<T>(s, 1);
      }
      if constexpr (n == 2 * N + M - 1) {
        ds[0] = operand<T>(dp, 0);
        ds[1] = operand<T>(dp, 1);
      }
      if constexpr (kPair && n == 2 * N + M) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          exchange[wave][i][lane] = p[i];
          exchange[wave][2 + i][lane] = ds[i];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    for_each<N>(run);
    if (r0 < all_from || r0 + 32 > all_to) {
      const int least = lo - r0 - 4 * hi, most = up - r0 - 4 * hi;  // relative to the lane's first row
      for_each<16>([&](auto element) {
        constexpr int e = element, row = 8 * (e / 4) + e % 4;
        s[e] = row >= least && row < most ? s[e] : kMinusInf;
      });
    }
    for_each<kOwn - N>([&](auto slot) { run(std::integral_constant<int, slot + N>()); });
    if constexpr (kPair) {
      lds_barrier();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p[i] = exchange[wave ^ 1][i][lane];
        ds[i] = exchange[wave ^ 1][2 + i][lane];
      }
      for_each<kSlots - kOwn>([&](auto slot) { run(std::integral_constant<int, slot + kOwn>()); });
    }
  };

  auto keep = [&] {
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      keep_accumulated<(D == 256)>(dk[d]);
      keep_accumulated<(D == 256)>(dv[d]);
    }
  };

  // one step: its rows in (q, g), the next step's on their way to (nq, ng), a request every fourth slot
  auto step = [&](int index, auto& q, auto& g, auto& stats, auto& nq, auto& ng, auto& nstats) {
    const int r0 = row_of(index);
    const Rows next = rows_from(index + 1);
    request_stats(nstats, next);
    if constexpr (kUnits) {
      // a step past the last one has old statistics, and adds nothing
      const float top = stats[2 * kR + lane] * unit;
      const uint64_t large = __ballot(top > kUnitMost), fits = __ballot(top >= kUnitLeast);
      if (large || !fits) {
        float most = top < INFINITY ? top : 0.f;
        for (int x = 1; x < 64; x *= 2) most = fmaxf(most, __shfl_xor(most, x));
        if (ill_fit(most, unit)) {
          const float by = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(refit(most, unit))));
          unit *= by;
          low *= by;
          scale *= by;
#pragma unroll
          for (int i = 0; i < DB; ++i) dk[i] *= by;
        }
      }
    }
    constexpr int kParts = kPair ? 1 : kR / 32, kEach = (RTile::kPieces + kParts - 1) / kParts;
    for_each<kParts>([&](auto half) {
      const int i = kPair ? role * 32 : half * 32, r = r0 + i;
      auto fetch = [&](auto slot) {
        constexpr int n = slot, piece = half * kEach + n / 4;
        if constexpr (n % 4 == 0 && n / 4 < kEach && piece < RTile::kPieces)
          request(std::integral_constant<int, piece>(), nq, ng, next);
      };
      keep();
      // a pair's waves meet in every step: their rows or keys may be masked, but are not left out (a branch around them
      // cost registers: 2 x 8192 tokens, 16 + 2 heads of 256 columns, backward 4090 us without, 4265 with it)
      const bool some = index < n_steps && (kPair || (r + 32 > any_from && r < any_to && r < to && wlo < kt.len));
      const int at = kPair ? 0 : i * D;
      if (some) part(q + at, g + at, stats + i, stats + kR + i, r, fetch);
      else for_each<4 * kEach>(fetch);
      keep();
    });
    __syncthreads();
  };
  auto fill = [&](int index, auto& q, auto& g, auto& stats) {
    const Rows rows = rows_from(index);
    request_stats(stats, rows);
    for_each<RTile::kPieces>([&](auto i) { request(i, q, g, rows); });
  };
  fill(0, q0, g0, stats0);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < n_steps; i += 2) {  // a step past the last one does nothing
    step(i, q0, g0, stats0, q1, g1, stats1);
    step(i + 1, q1, g1, stats1, q0, g0, stats0);
  }
  if (!live) return;
  const float back = 1.f / unit;
  if constexpr (kUnits) {
#pragma unroll
    for (int i = 0; i < DB; ++i) {
      dk[i] *= back;
      dv[i] *= kWeight;
    }
  }
  const bool sunk = j / kKeys < a.far_tiles;
  if (far || a.pieces > 1 || sunk) {
    float* p = far ? far_at(a, piece, kt, j, hk, D)
                   : a.pieces > 1 ? part_at(a, piece, kt, j, hk, D) : far_at(a, a.far_pieces, kt, j, hk, D);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int col = col0 + 32 * d + 8 * n + 4 * hi;
        *reinterpret_cast<f32x4*>(p + col) = f32x4{dk[d][4 * n], dk[d][4 * n + 1], dk[d][4 * n + 2], dk[d][4 * n + 3]};
        *reinterpret_cast<f32x4*>(p + D + col) = f32x4{dv[d][4 * n], dv[d][4 * n + 1], dv[d][4 * n + 2], dv[d][4 * n + 3]};
      }
  } else {
    const int64_t at = ((int64_t)(kt.bos + j) * pk.HK + hk) * D + col0;
    uint16_t *pd = static_cast<uint16_t*>(a.dk) + at, *pv = static_cast<uint16_t*>(a.dv) + at;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        *reinterpret_cast<uint4*>(pd + 32 * d + 16 * u + 8 * hi) = eight_columns<T>(dk[d], u, 1.f);
        *reinterpret_cast<uint4*>(pv + 32 * d + 16 * u + 8 * hi) = eight_columns<T>(dv[d], u, 1.f);
      }
  }
}

// The parts of dk and dv, in order: first those in the window, then those of the rows behind it. A
// workgroup takes eight keys of a tile; without parts of the windows, of the sinks' tiles alone.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_grad_join_kernel(AttnGradArgs a, int first) {
  constexpr int kKeys = attn_keys(D);
  const AttnPack& pk = a.pack;
  const int some = blockIdx.x % (kKeys / 8) * 8, b = blockIdx.x / (kKeys / 8) + first;
  const RowTile kt = a.pieces > 1 ? find_tile(pk.cu, pk.N, pk.T, kKeys, b) : far_tile(a, b, kKeys);
  const int keys = min(8, kt.tokens - some), unit = 2 * pk.HK * D / 4;
  const bool sunk = kt.first / kKeys < a.far_tiles;
  const int from_part = a.pieces > 1 ? a.pieces : 0;
  const int from_far = sunk ? a.far_pieces + (a.pieces > 1 ? 0 : 1) : 0;
  for (int i = threadIdx.x; i < keys * unit; i += 256) {
    const int j = kt.first + some + i / unit, at = i % unit * 4, hk = at / (2 * D), col = at % (2 * D);
    f32x4 x = zero4();
    // eight requests at once
    const auto add = [&](int parts, const float* p, int64_t pitch) {
#pragma unroll 1
      for (int n = 0; n < parts; n += 8) {
        f32x4 y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = zero4();
          if (n + e < parts) y[e] = *reinterpret_cast<const f32x4*>(p + (n + e) * pitch);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x += y[e];
      }
    };
    add(from_part, part_at(a, 0, kt, j, hk, D) + col, (int64_t)pk.T * pk.HK * 2 * D);
    add(from_far, far_at(a, 0, kt, j, hk, D) + col, far_rows(a, D) * pk.HK * 2 * D);
    uint16_t* to = static_cast<uint16_t*>(col < D ? a.dk : a.dv) + ((int64_t)(kt.bos + j) * pk.HK + hk) * D + col % D;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
  }
}

namespace {

template <typename T, int D>
hipError_t bwd_of(const AttnGradArgs& a, hipStream_t s) {
  const AttnPack& pk = a.pack;
  const dim3 block(256);
  hipLaunchKernelGGL((attn_grad_q_kernel<T, D>), dim3(a.slots * pk.HK), dim3(2 * attn_rows(D)), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a launch counts its threads in 32 bits
  const int items = (a.far_pieces * a.far_slots + a.pieces * a.key_slots) * pk.HK, launch = 1 << 22;
  for (int i = 0; i < items && e == hipSuccess; i += launch) {
    hipLaunchKernelGGL((attn_grad_kv_kernel<T, D>), dim3(std::min(items - i, launch)), dim3(grad_threads(D)), 0, s, a, i);
    e = hipGetLastError();
  }
  const int tiles = a.pieces > 1 ? a.key_slots : a.far_slots, most = 1 << 19;  // of at most 16 workgroups each
  for (int first = 0; first < tiles && e == hipSuccess; first += most) {
    const int n = std::min(tiles - first, most);
    hipLaunchKernelGGL((attn_grad_join_kernel<T, D>), dim3(n * (attn_keys(D) / 8)), block, 0, s, a, first);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

hipError_t launch_attn_bwd(Elem type, int D, const AttnGradArgs& a, hipStream_t s) {
  if (type == Elem::kBf16) return D == 64 ? bwd_of<Bf16, 64>(a, s) : D == 128 ? bwd_of<Bf16, 128>(a, s) : bwd_of<Bf16, 256>(a, s);
  return D == 64 ? bwd_of<Fp16, 64>(a, s) : D == 128 ? bwd_of<Fp16, 128>(a, s) : bwd_of<Fp16, 256>(a, s);
}

}  // namespace gdn
