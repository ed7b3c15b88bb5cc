// Causal softmax attention over packed sequences, forward, with a sliding
// window and first tokens that stay visible, keys and values from token rows
// or from pages of a cache.
//
// A workgroup of eight waves (four with 256 columns) takes 256 (128) rows of one
// key head, its query heads side by side (see AttnPack), and goes over the key
// tiles that they see, with the running maximum m and sum l of the weights
// p = 2^(c s - m):
//   l <- l 2^(m' - m) + sum p,  O <- O 2^(m' - m) + p V,  o = O / l,
//   lse = (m + log2 l) ln 2.
// A wave holds 32 rows as the columns of S^T = K Q^T and O^T = V^T P^T: a lane
// then has one row, its maximum and sum need one exchange with the other half
// of the wave, and the weights are the second product's operand as they stand
// in the registers: their 8 keys a lane are those of the accumulator's rows,
// and the transposing reads of V take the same ones.
//
// Scores, maxima, sums and O are fp32; the weights are rounded once to the
// inputs' type for the second product, while their sum takes them unrounded. In
// fp16 a row's largest weight is 2^7 to 2^15 for that, so that those down to 2^-21 of it keep full precision and
// those down to 2^-31 some.
//
// Bound by the matrix unit and by what the vector unit adds to it: the slots of
// a step interleave the scores of the next tile, the weights of this one and the
// product of the one before. 2 x 8192 tokens, 16 + 2 heads of 256 columns: 1072 to 1086 us,
// 1.02 PFLOP/s (a library's product of 8192^3: 1.32). With tiles through registers, masks
// by positions and the compiler's own order it was 2365 us.
#include <algorithm>

#include "attn_tile.h"

namespace gdn {

namespace {

constexpr int kFwdKeys = 64;  // keys a tile

// where the keys are: token rows, pages whose rows come in groups of 8 (see request_group; 8 x 512 tokens, four after 1000 to
// 2000: by rows 8 % more), other pages, and a window's, whose edge may leave part of a group unread
enum { kTokens, kGroups, kPages };

}  // namespace

template <typename T, int D, int kKeys>
__global__ __launch_bounds__(2 * attn_rows(D), D == 256 ? 1 : 2) void attn_fwd_kernel(AttnArgs a) {
  constexpr int kT = kFwdKeys, N = D / 16, DB = D / 32, kThreads = 2 * attn_rows(D);
  constexpr bool kPaged = kKeys != kTokens;
  constexpr float kLift = weight_lift<T>(7);  // and 8 for a maximum that grows
  typedef Tile<D, kT, kThreads> KTile;
  __shared__ __attribute__((aligned(16))) typename KTile::Lds k0, k1, v0, v1;
  const AttnPack& pk = a.pack;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l32 = lane & 31, hi = lane >> 5;
  int b = blockIdx.x;
  const int hk = b % pk.HK;
  b /= pk.HK;
  const int split = b % a.splits;
  const int G = pk.G.by, per = attn_rows(D) / G;
  const RowTile rt = tile_of(pk.cu, pk.N, pk.T, per, a.slots, b / a.splits, true,
                             [&](int n) { return kPaged ? past_of(a.pages, n, pk.T) : 0; });
  if (rt.tokens <= 0) return;

  int past = 0;
  int64_t keys = rt.len;
  if constexpr (kPaged) {
    past = __builtin_amdgcn_readfirstlane(past_of(a.pages, rt.seq, pk.T));
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
  const int64_t all = (int64_t)pk.T * pk.HQ;

  if (part.x >= part.y) {  // nothing to see, or nothing left for this split
    if (!live || hi) return;
    if (a.splits > 1) {  // the join reads no sums of weight 0
      *reinterpret_cast<float2*>(a.part + all * a.splits * D + 2 * (all * split + out)) = make_float2(kMinusInf, 0.f);
    } else {
      uint4* po = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D);
      for (int i = 0; i < D / 8; ++i) po[i] = make_uint4(0, 0, 0, 0);
      if (a.lse) a.lse[out] = kMinusInf;
    }
    return;
  }

  uint4 q[N];
  {
    // rows past the tile's tokens read its last token, and are not stored
    const uint16_t* p = static_cast<const uint16_t*>(a.q) +
                        (int64_t)(rt.bos + rt.first + min(token, rt.tokens - 1)) * a.q_stride + head * D + 8 * hi;
#pragma unroll
    for (int s = 0; s < N; ++s) q[s] = *reinterpret_cast<const uint4*>(p + 16 * s);
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
  // paged: where row `lane` of tiles i, i + 1 and i + 2 is; rows that no token of the tile has in its window are not read
  // (a freed page may hold anything)
  int64_t rows[3] = {-1, -1, -1};
  auto look = [&](int i) -> int64_t {
    if (!kPaged || i >= part.y) return -1;
    const int j = kt.at(i) * kT + lane;
    if (kKeys == kPages && pk.window && j <= t0 - pk.window && j >= pk.sinks) return -1;
    return row_at(a.pages, rt.seq, j, keys);
  };
  const TokenRows<KTile> kr((int)a.k_stride, tid), vr((int)a.v_stride, tid);
  int64_t off = -1;  // kPages: where this lane's piece of the next request is
  const int pitch = (int)a.pages.token_stride;  // kGroups: of a page's rows, and this lane's places in a group
  const int group[2] = {KTile::in_group(0, pitch, tid), KTile::in_group(1, pitch, tid)};
  auto page_rows = [&](auto& to, auto i, const uint16_t* base, int64_t at, int tile) {
    if constexpr (kKeys == kGroups)
      KTile::request_group(to, i, base, at, (int)min(keys - (int64_t)kt.at(tile) * kT, (int64_t)kT), pitch, fresh(group[i % 2]), tid);
    else
      KTile::request_page(to, i, base, KTile::place(at, i, tid), tid);
  };
  // resource of tile i's token rows; past the last tile empty, or rows that nobody reads
  auto tokens = [&](const uint16_t* base, int64_t stride, int i) {
    const int j0 = kt.at(i) * kT;
    return TokenRows<KTile>::from(base + j0 * stride, (int)stride, min(kT, rt.len - j0), D);
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) zero16(o[i]);
  float m = kMinusInf, l = 0.f;
  const float c = pk.scale * kLog2e;
  const int ka = at<D>(l32, 8 * hi);
  const int j16 = lane & 15, vrow = 4 * hi + (j16 >> 2), vcol = 16 * ((lane >> 4) & 1) + 4 * (j16 & 3);
  const int va = at<D>(vrow, vcol), vb = at<D>(vrow + 8, vcol);
  const int from = pk.window ? t - pk.window : -1;  // keys in the window are past this

  // One step: the weights p of a tile from its scores s, while the matrix unit forms the next tile's scores `next` from K
  // and adds the tile before's weights times V, `before`, to O. A slot has one matrix instruction, of these in turn, and a
  // share of the vector unit's work and of the requests for the tiles to come (`fetch`: issued together they held the
  // matrix unit up); the LDS operands are requested kAhead instructions of their kind before.
  auto step = [&](f32x16(&s)[2], f32x16(&next)[2], uint4(&p)[4], const uint4(&before)[4], const uint16_t* K,
                  const uint16_t* V, int j0, uint64_t seen, const auto& fetch) {
    constexpr int kSlots = 4 * N, kTop = kSlots / 4, kAhead = 3;
    bool mask = j0 + kT - 1 > wlo;
    if (pk.window) mask = mask || (j0 <= whi - pk.window && j0 + kT > pk.sinks);
    if constexpr (kPaged) mask = mask || ~seen != 0;
    if (mask) {
      // against constants: positions and the pages' bits relative to the lane's first key
      const int first = j0 + 4 * hi, most = t - first, least = from - first, far = pk.sinks - first;
      const uint64_t has = seen >> (4 * hi);
      for_each<32>([&](auto element) {
        constexpr int e = element, r = e % 16, j = 32 * (e / 16) + 8 * (r / 4) + r % 4;
        bool ok = j <= most && (j > least || j < far);
        if constexpr (kPaged) ok = ok && (has >> j & 1);
        s[e / 16][r] = ok ? s[e / 16][r] : kMinusInf;
      });
    }
    const int kf = fresh(ka), c0 = fresh(va), c1 = fresh(vb);
    uint4 ko[kAhead], vo[kAhead];
    auto read = [&](auto slot) {
      constexpr int n = slot / 2;
      if constexpr (slot % 2 == 0)
        ko[n % kAhead] = *reinterpret_cast<const uint4*>(K + (kf ^ (16 * (n / 2))) + 32 * (n % 2) * D);
      else
        vo[n % kAhead] = column8(V + 16 * (n / DB) * D, c0 ^ (32 * (n % DB)), c1 ^ (32 * (n % DB)));
    };
    for_each<2 * kAhead>(read);
    float top = kMinusInf, base = 0.f, f = 1.f, sum[2] = {0.f, 0.f};
    for_each<kSlots>([&](auto slot) {
      constexpr int n = slot, i = n / 2;
      if constexpr (n % 2 == 0) next[i % 2] = mfma32_of<T>(ko[i % kAhead], q[i / 2], i < 2 ? f32x16{} : next[i % 2]);
      else o[i % DB] = mfma32_of<T>(vo[i % kAhead], before[i / DB], o[i % DB]);
      if constexpr (n + 2 * kAhead < kSlots) read(std::integral_constant<int, n + 2 * kAhead>());
      fetch(slot);
      for_each<32>([&](auto element) {
        constexpr int e = element;
        if constexpr (e * kTop / 32 == n) top = fmaxf(top, s[e / 16][e % 16]);
      });
      if constexpr (n == kTop - 1) {
        const float2 tops = both_halves(top);
        top = fmaxf(tops.x, tops.y) * c;
        // What weights are relative to follows the row's maximum only where that has grown by a factor of 2^8: weights
        // up to that are as exact. The maximum's own weight is 2^kLift then.
        const float now = top > m + (8.f + kLift) ? top - kLift : m;
        base = now == kMinusInf ? 0.f : now;  // a row that has seen nothing yet
        f = exp2_fast(m - base);
        m = now;
      }
      // a weight's argument, exponential and share of the sum in slots of their own: none waits for the one before
      for_each<32>([&](auto element) {
        constexpr int e = element, at = kTop + e * (kSlots - kTop - 2) / 32;
        float x = s[e / 16][e % 16];
        if constexpr (n == at) x = fmaf(x, c, -base);
        if constexpr (n == at + 1) x = exp2_fast(x);
        if constexpr (n == at + 2) {
          sum[e % 2] += x;
          if constexpr (e % 8 == 7) {
            p[e / 8] = operand<T>(s[e / 16], e / 8 % 2);
            stay_here(p[e / 8]);
            stay_here(sum[0], sum[1]);
          }
        }
        s[e / 16][e % 16] = x;
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    l = fmaf(l, f, sum[0] + sum[1]);
    if (__any(f != 1.f)) {
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
    }
  };
  auto keep = [&] {
#pragma unroll
    for (int d = 0; d < DB; ++d) keep_accumulated<D == 256>(o[d]);
  };

  // K of the first two tiles, scores of the first; the weights before it are zeros, and so is their V
  f32x16 s0[2], s1[2];
  uint4 p0[4], p1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p1[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int n = 0; n < 3; ++n) rows[n] = look(part.x + n);
  const auto first = tokens(kbase, a.k_stride, part.x), second = tokens(kbase, a.k_stride, part.x + 1);
  for_each<KTile::kPieces>([&](auto i) {
    if constexpr (kPaged) {
      page_rows(k0, i, kbase, rows[0], part.x);
      page_rows(k1, i, kbase, rows[1], part.x + 1);
    } else {
      kr.request(k0, i, first, tid);
      kr.request(k1, i, second, tid);
    }
  });
  for (int i = tid; i < kT * D / 8; i += kThreads) reinterpret_cast<uint4*>(v1)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
      s0[kb] = mfma32_of<T>(*reinterpret_cast<const uint4*>(k0 + (ka ^ (16 * d)) + 32 * kb * D), q[d],
                            d == 0 ? f32x16{} : s0[kb]);
  __syncthreads();
  // Step i has K of tile i + 1 and V of tile i - 1 in LDS; K of i + 2 and V of i come into the other buffers meanwhile.
  auto turn = [&](int i, auto& nk, auto& nv, const uint16_t* K, const uint16_t* V, f32x16(&s)[2], f32x16(&next)[2],
                  uint4(&p)[4], const uint4(&before)[4]) {
    uint64_t seen = ~0ull;
    if constexpr (kPaged) seen = __ballot(rows[0] >= 0);
    const auto krows = tokens(kbase, a.k_stride, i + 2), vrows = tokens(vbase, a.v_stride, i);
    const int64_t kat = rows[2], vat = rows[0];
    // request r in slot 2 r (of V after those of K), a page's offset two slots before it
    auto fetch = [&](auto slot) {
      constexpr int n = slot, P = KTile::kPieces, r = n / 2;
      if constexpr (kKeys == kGroups) {
        if constexpr (n % 2 == 0 && r < P) page_rows(nk, std::integral_constant<int, r>(), kbase, kat, i + 2);
        if constexpr (n % 2 == 0 && r >= P && r < 2 * P) page_rows(nv, std::integral_constant<int, r - P>(), vbase, vat, i);
      } else if constexpr (kPaged) {
        if constexpr (n % 2 == 0 && n > 0 && r <= P) KTile::request_page(nk, r - 1, kbase, off, tid);
        if constexpr (n % 2 == 0 && r > P && r <= 2 * P) KTile::request_page(nv, r - 1 - P, vbase, off, tid);
        if constexpr (n % 2 == 0 && r < 2 * P) off = KTile::place(r < P ? kat : vat, r % P, tid);
      } else {
        if constexpr (n % 2 == 0 && r < P) kr.request(nk, r, krows, tid);
        if constexpr (n % 2 == 0 && r >= P && r < 2 * P) vr.request(nv, r - P, vrows, tid);
      }
      if constexpr (kPaged && n == 4 * P + 2) {
        rows[0] = rows[1];
        rows[1] = rows[2];
        rows[2] = look(i + 3);
      }
    };
    keep();
    // past the last tile no row sees anything
    step(s, next, p, before, K, V, i < part.y ? kt.at(i) * kT : whi + 64, seen, fetch);
    keep();
    __syncthreads();
  };
#pragma unroll 1
  for (int i = part.x; i < part.y; i += 2) {
    turn(i, k0, v0, k1, v1, s0, s1, p0, p1);
    turn(i + 1, k1, v1, k0, v0, s1, s0, p1, p0);
  }
  if ((part.y - part.x) % 2 == 0) {  // else the step past the last tile has added it
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < DB; ++d)
        o[d] = mfma32_of<T>(column8(v1 + 16 * i * D, va ^ (32 * d), vb ^ (32 * d)), p1[i], o[d]);
  }

  l = sum_halves(l);
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
    const int64_t at = all * split + out;
    if (hi == 0) *reinterpret_cast<float2*>(a.part + all * a.splits * D + 2 * at) = make_float2(m, l);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(a.part + at * D + 32 * d + 8 * g + 4 * hi) =
            f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
  }
}

// o and lse of a row from its parts: sums of weights relative to their own maxima. 16 lanes take 64
// columns of a row, kShares such groups a share of the parts each, of which a lane requests eight at once.
template <typename T, int D, int kShares>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int kBlocks = D / 64, kUnits = 16 / kShares;  // columns blocks of a row; units of a workgroup
  const AttnPack& pk = a.pack;
  const int64_t rows = (int64_t)pk.T * pk.HQ;
  const int group = threadIdx.x >> 4, lane = threadIdx.x & 15, share = group % kShares;
  const int64_t unit = (int64_t)blockIdx.x * kUnits + group / kShares, row = unit / kBlocks;
  // behind the last sequence, or the last unit: nothing is written
  const bool live = row < (pk.cu ? min((int64_t)min(max(pk.cu[pk.N], 0), pk.T) * pk.HQ, rows) : rows);
  const int col = (int)(unit % kBlocks) * 64 + lane * 4;
  const float2* ml = reinterpret_cast<const float2*>(a.part + rows * a.splits * D) + row;
  float m = kMinusInf, l = 0.f, base = 0.f;
  f32x4 o = zero4();
  if (live) {
    for (int s = lane; s < a.splits; s += 16) m = fmaxf(m, ml[s * rows].x);
    for (int x = 1; x < 16; x *= 2) m = fmaxf(m, __shfl_xor(m, x));
    base = m == kMinusInf ? 0.f : m;
#pragma unroll 1
    for (int s0 = share; s0 < a.splits; s0 += 8 * kShares) {
      float2 x[8];
      f32x4 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int s = s0 + i * kShares;
        x[i] = make_float2(kMinusInf, 0.f);
        if (s < a.splits) x[i] = ml[s * rows];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = zero4();  // a part without weight holds no sums
        if (x[i].x != kMinusInf || x[i].y != 0.f)
          y[i] = *reinterpret_cast<const f32x4*>(a.part + (row + (s0 + i * kShares) * rows) * D + col);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = exp2_fast(x[i].x - base);
        l = fmaf(x[i].y, w, l);
        o += y[i] * w;
      }
    }
  }
  if constexpr (kShares > 1) {
    __shared__ float sums[16][16][5];
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[group][lane][i] = o[i];
    sums[group][lane][4] = l;
    __syncthreads();
    if (share > 0) return;
    for (int i = 1; i < kShares; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] += sums[group + i][lane][c];
      l += sums[group + i][lane][4];
    }
  }
  if (!live) return;
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D + col) =
      make_uint2(pack2<T>(o[0] * f, o[1] * f), pack2<T>(o[2] * f, o[3] * f));
  if (a.lse && col == 0) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

namespace {

template <typename T>
hipError_t fwd_of(int D, bool paged, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(a.slots * a.pack.HK * a.splits), block(2 * attn_rows(D));
#define GDN_FWD(d)                                                                                                 \
  if (!paged) hipLaunchKernelGGL((attn_fwd_kernel<T, d, kTokens>), grid, block, 0, s, a);                          \
  else if (in_groups(a)) hipLaunchKernelGGL((attn_fwd_kernel<T, d, kGroups>), grid, block, 0, s, a);         \
  else hipLaunchKernelGGL((attn_fwd_kernel<T, d, kPages>), grid, block, 0, s, a)
  if (D == 64) GDN_FWD(64);
  else if (D == 128) GDN_FWD(128);
  else GDN_FWD(256);
#undef GDN_FWD
  return hipGetLastError();
}
template <typename T, int D>
hipError_t join_of(const AttnArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.pack.T * a.pack.HQ * (D / 64);
  const dim3 block(256);
  // a lane's eight requests hold every part where the rows alone fill no chip (one token of 16 + 2 heads over 131072, 128
  // parts: 61.9 us, with one share 76.4)
  if (a.splits > 16 && units < 4096)
    hipLaunchKernelGGL((attn_join_kernel<T, D, 16>), dim3((uint32_t)units), block, 0, s, a);
  else
    hipLaunchKernelGGL((attn_join_kernel<T, D, 1>), dim3((uint32_t)((units + 15) / 16)), block, 0, s, a);
  return hipGetLastError();
}
template <typename T>
hipError_t join_type(int D, const AttnArgs& a, hipStream_t s) {
  return D == 64 ? join_of<T, 64>(a, s) : D == 128 ? join_of<T, 128>(a, s) : join_of<T, 256>(a, s);
}

}  // namespace

hipError_t launch_attn_fwd(Elem type, int D, bool paged, const AttnArgs& a, hipStream_t s) {
  return type == Elem::kBf16 ? fwd_of<Bf16>(D, paged, a, s) : fwd_of<Fp16>(D, paged, a, s);
}
hipError_t launch_attn_join(Elem type, int D, const AttnArgs& a, hipStream_t s) {
  return type == Elem::kBf16 ? join_type<Bf16>(D, a, s) : join_type<Fp16>(D, a, s);
}

}  // namespace gdn
