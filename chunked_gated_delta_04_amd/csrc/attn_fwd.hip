// Causal softmax attention over packed sequences, forward, with a sliding
// window and first tokens that stay visible, keys and values from token rows
// or from pages of a cache.
//
// A workgroup of four waves takes 128 rows of one key head (its query heads
// side by side, see AttnPack) and goes over the key tiles that they see, with
// the running maximum m and sum l of the weights p = 2^(c s - m):
//   l <- l 2^(m' - m) + sum p,  O <- O 2^(m' - m) + p V,  o = O / l,
//   lse = (m + log2 l) ln 2.
// A wave holds 32 rows as the columns of S^T = K Q^T and O^T = V^T P^T: a lane
// then has one row, its maximum and sum need one exchange with the other half
// of the wave, and the weights are the second product's operand as they stand
// in the registers: their 8 keys a lane are those of the accumulator's rows,
// and the transposing reads of V take the same ones.
//
// Scores, maxima, sums and O are fp32; the weights are rounded once to the
// inputs' type for the second product, while their sum takes them unrounded.
#include <algorithm>

#include "attn_tile.h"

namespace gdn {

namespace {

// keys a tile
template <int D>
constexpr int kFwdKeys = 64;

}  // namespace

template <typename T, int D, bool kPaged>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_fwd_kernel(AttnArgs a) {
  constexpr int kT = kFwdKeys<D>, KB = kT / 32, DB = D / 32;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2][2][kT * D];  // [buffer][k, v]
  const AttnPack& pk = a.pack;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, hi = lane >> 5;
  // the last rows of a sequence, which see the most keys, first
  int b = blockIdx.x;
  const int hk = b % pk.HK;
  b /= pk.HK;
  const int split = b % a.splits;
  const int G = pk.G.by, per = kAttnRows / G;
  const RowTile rt = find_tile(pk.cu, pk.N, pk.T, per, a.slots - 1 - b / a.splits);
  if (rt.tokens <= 0) return;

  int past = 0;
  int64_t keys = rt.len;
  if constexpr (kPaged) {
    past = past_of(a.pages, rt.seq, pk.T);
    keys = min((int64_t)past + rt.len, (int64_t)a.pages.columns * a.pages.page.by);
  }
  const int t0 = past + rt.first;  // position of the tile's first token
  const KeyTiles kt = key_tiles<kT>(t0, t0 + rt.tokens - 1, keys, pk.window, pk.sinks);
  const int2 part = split_of(kt.count, a.splits, split, 4);

  // this lane's row
  const int row = wave * 32 + l32;
  const int token = divide(row, pk.G), head = hk * G + row - token * G;
  const bool live = token < rt.tokens;
  const int t = t0 + token;
  // the wave's positions
  const int wlo = t0 + divide(wave * 32, pk.G);
  const int whi = t0 + min(divide(wave * 32 + 31, pk.G), rt.tokens - 1);
  const int64_t out = (int64_t)(rt.bos + rt.first + token) * pk.HQ + head;  // row of o

  uint4 q[D / 16];
  {
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + (int64_t)(rt.bos + rt.first + token) * a.q_stride + head * D + 8 * hi;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      q[s] = make_uint4(0, 0, 0, 0);
      if (live) q[s] = *reinterpret_cast<const uint4*>(p + 16 * s);
    }
  }

  const uint16_t* kbase = static_cast<const uint16_t*>(kPaged ? a.pages.k : a.k);
  const uint16_t* vbase = static_cast<const uint16_t*>(kPaged ? a.pages.v : a.v);
  if constexpr (kPaged) {
    kbase += hk * a.pages.head_stride;
    vbase += hk * a.pages.head_stride;
  } else {
    kbase += rt.bos * a.k_stride + hk * D;
    vbase += rt.bos * a.v_stride + hk * D;
  }

  Staged<D, kT, 256> ks, vs;
  int id = 0;                 // page of row `lane` of the tile after the next
  uint64_t seen_next = ~0ull; // which rows of the next tile have a page
  auto look = [&](int i) {
    if constexpr (kPaged) id = i < part.y ? page_of(a.pages, rt.seq, kt.at(i) * kT + lane, (int)keys) : 0;
  };
  auto load = [&](int i) {
    const int j0 = kt.at(i) * kT;
    if constexpr (kPaged) {
      seen_next = __ballot(id > 0);
#pragma unroll
      for (int n = 0; n < ks.kPieces; ++n) {
        const int r = ks.row(n, tid), pid = __shfl(id, r);
        ks.x[n] = vs.x[n] = make_uint4(0, 0, 0, 0);
        if (pid > 0) {
          const int64_t off = row_of(a.pages, pid, j0 + r) + ks.column(tid);
          ks.x[n] = *reinterpret_cast<const uint4*>(kbase + off);
          vs.x[n] = *reinterpret_cast<const uint4*>(vbase + off);
        }
      }
      look(i + 1);
    } else {
      const int len = min(kT, rt.len - j0);
      ks.load(kbase + j0 * a.k_stride, (int)a.k_stride, len, tid);
      vs.load(vbase + j0 * a.v_stride, (int)a.v_stride, len, tid);
    }
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
  float m = kMinusInf, l = 0.f;
  const float c = pk.scale * kLog2e;
  const int ka = at<D>(l32, 8 * hi);
  const int j16 = lane & 15, vr = 4 * hi + (j16 >> 2), vc = 16 * ((lane >> 4) & 1) + 4 * (j16 & 3);
  const int va = at<D>(vr, vc), vb = at<D>(vr + 8, vc);

  if (part.x < part.y) {
    look(part.x);
    load(part.x);
    ks.store(lds[0][0], tid);
    vs.store(lds[0][1], tid);
  }
  __syncthreads();
  for (int i = part.x, buf = 0; i < part.y; ++i, buf ^= 1) {
    const uint64_t seen = seen_next;
    const int j0 = kt.at(i) * kT, j1 = j0 + kT - 1;
    if (i + 1 < part.y) load(i + 1);
    // rows of this wave that see a key of the tile
    bool some = wlo <= whi && j0 <= whi;
    if (pk.window) some = some && (j1 > wlo - pk.window || j0 < pk.sinks);
    if (some) {
      const uint16_t *K = lds[buf][0], *V = lds[buf][1];
      f32x16 s[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[kb][r] = 0.f;
      const int kf = fresh(ka);
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          s[kb] = mfma32_of<T>(*reinterpret_cast<const uint4*>(K + (kf ^ (16 * d)) + 32 * kb * D), q[d], s[kb]);
      bool mask = j1 > wlo;
      if (pk.window) mask = mask || (j0 <= whi - pk.window && j1 >= pk.sinks);
      if constexpr (kPaged) mask = mask || ~seen != 0;
      if (mask) {
        const int from = pk.window ? t - pk.window : -1;  // keys in the window are past this
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int jr = 32 * kb + 8 * (r >> 2) + 4 * hi + (r & 3), j = j0 + jr;
            bool ok = j <= t && (j > from || j < pk.sinks);
            if constexpr (kPaged) ok = ok && (seen >> jr & 1);
            s[kb][r] = ok ? s[kb][r] : kMinusInf;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
      top = fmaxf(top, other_half(top)) * c;
      const float now = fmaxf(m, top);
      const float base = now == kMinusInf ? 0.f : now;  // a row that has seen nothing yet
      if (__any(now > m)) {
        const float f = exp2_fast(m - base);
        l *= f;
#pragma unroll
        for (int i2 = 0; i2 < DB; ++i2)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[i2][r] *= f;
      }
      m = now;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[kb][r] = exp2_fast(fmaf(s[kb][r], c, -base));
          l += s[kb][r];
        }
      }
      const int v0 = fresh(va), v1 = fresh(vb);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 p = make_uint4(pack2<T>(s[kb][8 * h], s[kb][8 * h + 1]), pack2<T>(s[kb][8 * h + 2], s[kb][8 * h + 3]),
                                     pack2<T>(s[kb][8 * h + 4], s[kb][8 * h + 5]), pack2<T>(s[kb][8 * h + 6], s[kb][8 * h + 7]));
#pragma unroll
          for (int d = 0; d < DB; ++d)
            o[d] = mfma32_of<T>(column8(V + (32 * kb + 16 * h) * D, v0 ^ (32 * d), v1 ^ (32 * d)), p, o[d]);
        }
    }
    if (i + 1 < part.y) {
      ks.store(lds[buf ^ 1][0], tid);
      vs.store(lds[buf ^ 1][1], tid);
    }
    __syncthreads();
  }
  l += other_half(l);
  if (!live) return;
  if (a.splits == 1) {
    const float f = l > 0.f || l != l ? 1.f / l : 0.f;  // a row that sees nothing is zeros
    uint16_t* po = static_cast<uint16_t*>(a.o) + out * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<uint4*>(po + 32 * d + 16 * u + 8 * hi) = eight_columns<T>(o[d], u, f);
    if (a.lse && hi == 0) a.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
  } else {
    const int64_t rows = (int64_t)pk.T * pk.HQ, at = rows * split + out;
    float* ml = a.part + rows * a.splits * D + 2 * at;
    if (hi == 0) *reinterpret_cast<float2*>(ml) = make_float2(m, l);
    if (part.x >= part.y) return;  // the join reads no sums of weight 0
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(a.part + at * D + 32 * d + 8 * g + 4 * hi) =
            f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
  }
}

// o and lse of a row from its parts: sums of weights relative to their own maxima. A workgroup takes
// a row, its threads D / 4 columns each and a share of the parts.
template <typename T, int D>
__global__ __launch_bounds__(512) void attn_join_kernel(AttnArgs a) {
  constexpr int kColumns = D / 4;
  __shared__ float sums[512 * 4];
  __shared__ float ls[512 / kColumns];
  const AttnPack& pk = a.pack;
  const int64_t row = blockIdx.x, rows = (int64_t)pk.T * pk.HQ;
  if (pk.cu && row / pk.HQ >= pk.cu[pk.N]) return;  // behind the last sequence
  const float2* ml = reinterpret_cast<const float2*>(a.part + rows * a.splits * D) + row;
  const int share = threadIdx.x / kColumns, shares = blockDim.x / kColumns, col = threadIdx.x % kColumns * 4;
  float m = kMinusInf;
  for (int s = threadIdx.x & 63; s < a.splits; s += 64) m = fmaxf(m, ml[s * rows].x);
  for (int x = 1; x < 64; x *= 2) m = fmaxf(m, __shfl_xor(m, x));
  const float base = m == kMinusInf ? 0.f : m;
  float l = 0.f;
  f32x4 o = zero4();
#pragma unroll 4
  for (int s = share; s < a.splits; s += shares) {
    const float2 x = ml[s * rows];
    const float w = exp2_fast(x.x - base);
    if (x.x != kMinusInf || x.y != 0.f) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(a.part + (row + s * rows) * D + col);
      o += y * w;
      l += x.y * w;
    }
  }
  if (shares > 1) {
    *reinterpret_cast<f32x4*>(sums + 4 * threadIdx.x) = o;
    if (col == 0) ls[share] = l;
    __syncthreads();
    if (share > 0) return;
    for (int i = 1; i < shares; ++i) {
      o += *reinterpret_cast<const f32x4*>(sums + 4 * (threadIdx.x + i * kColumns));
      l += ls[i];
    }
  }
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D + col) =
      make_uint2(pack2<T>(o[0] * f, o[1] * f), pack2<T>(o[2] * f, o[3] * f));
  if (a.lse && col == 0) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

namespace {

template <typename T>
hipError_t fwd_of(int D, bool paged, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(a.slots * a.pack.HK * a.splits), block(256);
#define GDN_FWD(d)                                                                                \
  if (paged) hipLaunchKernelGGL((attn_fwd_kernel<T, d, true>), grid, block, 0, s, a);             \
  else hipLaunchKernelGGL((attn_fwd_kernel<T, d, false>), grid, block, 0, s, a)
  if (D == 64) GDN_FWD(64);
  else if (D == 128) GDN_FWD(128);
  else GDN_FWD(256);
#undef GDN_FWD
  return hipGetLastError();
}
template <typename T>
hipError_t join_of(int D, const AttnArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)a.pack.T * a.pack.HQ));
  // as many threads as parts read at once, eight of them each
  const int columns = D / 4;
  int shares = std::max(64 / columns, 1);
  while (shares * columns < 512 && shares * 4 < a.splits) shares *= 2;
  const dim3 block(shares * columns);
  if (D == 64) hipLaunchKernelGGL((attn_join_kernel<T, 64>), grid, block, 0, s, a);
  else if (D == 128) hipLaunchKernelGGL((attn_join_kernel<T, 128>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((attn_join_kernel<T, 256>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_fwd(Elem type, int D, bool paged, const AttnArgs& a, hipStream_t s) {
  return type == Elem::kBf16 ? fwd_of<Bf16>(D, paged, a, s) : fwd_of<Fp16>(D, paged, a, s);
}
hipError_t launch_attn_join(Elem type, int D, const AttnArgs& a, hipStream_t s) {
  return type == Elem::kBf16 ? join_of<Bf16>(D, a, s) : join_of<Fp16>(D, a, s);
}

}  // namespace gdn
