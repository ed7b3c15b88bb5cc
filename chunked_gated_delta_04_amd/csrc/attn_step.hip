// Softmax attention of one new token a sequence over its paged cache.
//
// HBM bound: every visible key and value is read once for 16 query heads of its
// key head (the rows of one matrix product), and again for each further 16. The keys of a sequence
// are split over workgroups, as many as fill the chip, and over the four waves
// of each; a wave goes over its tiles of 32 keys by itself, with its own
// maximum and sum and its own LDS, no barrier and its next tile's rows on
// their way. The waves' results are joined in LDS, the workgroups' by
// attn_join_kernel. 240 rows of up to 8192 tokens, 32 + 8 heads of 128: 756 us, 5.3
// TB/s; one row over 131072 tokens, 16 + 2 heads of 256: 54 us, 5.0 TB/s, and the join 6.
//
// As in the forward, scores are S^T = K Q^T, so that the weights are the second
// product's operand where they stand, in fp16 relative to a largest one of 2^14.
#include "attn_tile.h"

namespace gdn {

namespace {

constexpr int kStepKeys = 32;

// kT rows of keys and values of a cache on their way through a wave's registers into its LDS, 16 bytes a piece.
template <int D, int kT>
struct Staged {
  static constexpr int kPieces = kT * D / 8 / 64, kRows = 64 / (D / 8);  // rows a piece of all lanes
  uint4 k[kPieces], v[kPieces];
  static __device__ __forceinline__ int row(int i, int lane) { return lane / (D / 8) + i * kRows; }
  static __device__ __forceinline__ int column(int lane) { return lane % (D / 8) * 8; }
  // lane r has the offset of row r, or -1 for zeros
  __device__ __forceinline__ void gather(const uint16_t* pk, const uint16_t* pv, int64_t rows, int lane) {
    int64_t off[kPieces];  // all exchanged before the first is waited for
#pragma unroll
    for (int i = 0; i < kPieces; ++i) off[i] = from_lane(rows, row(i, lane));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      k[i] = load16(off[i] >= 0 ? (Global*)(pk + off[i] + column(lane)) : (Global*)zeros);
      v[i] = load16(off[i] >= 0 ? (Global*)(pv + off[i] + column(lane)) : (Global*)zeros);
    }
  }
  __device__ __forceinline__ void store(uint16_t* K, uint16_t* V, int lane) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(K + at<D>(row(i, lane), column(lane))) = k[i];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(V + at<D>(row(i, lane), column(lane))) = v[i];
  }
};

}  // namespace

template <typename T, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_step_kernel(AttnArgs a) {
  constexpr int kT = kStepKeys, DB = D / 16;
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * 2 * kT * D];  // [wave][k, v]
  const AttnPack& pk = a.pack;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i16 = lane & 15, q4 = lane >> 4;
  const int G = pk.G.by, row_tiles = (G + 15) >> 4;
  int b = blockIdx.x;
  const int hk = b % pk.HK;
  b /= pk.HK;
  const int g0 = b % row_tiles * 16;
  b /= row_tiles;
  const int split = b % a.splits, seq = b / a.splits;

  const int t = __builtin_amdgcn_readfirstlane(past_of(a.pages, seq, 1));
  const int64_t keys = min((int64_t)t + 1, (int64_t)a.pages.columns * a.pages.page.by);
  const KeyTiles kt = key_tiles<kT>(t, t, keys, pk.window, pk.sinks);
  const int2 part = split_of(kt.count, a.splits, split, 4);
  const int from = pk.window ? t - pk.window : -1;

  const int head = hk * G + g0 + i16;
  uint4 q[D / 32];
  {
    // rows past the group read its last head, and are not stored
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + seq * a.q_stride + min(head, hk * G + G - 1) * D + 8 * q4;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) q[s] = *reinterpret_cast<const uint4*>(p + 32 * s);
  }
  const uint16_t* kbase = static_cast<const uint16_t*>(a.pages.k) + hk * a.pages.head_stride;
  const uint16_t* vbase = static_cast<const uint16_t*>(a.pages.v) + hk * a.pages.head_stride;
  uint16_t *K = lds + wave * 2 * kT * D, *V = K + kT * D;

  Staged<D, kT> staged;
  int64_t at_next = -1;   // where row lane % 32 of the tile after the next is, -1 where it is not seen
  uint32_t seen_next = 0; // the rows of the next tile that are seen
  auto look = [&](int i) {
    at_next = -1;
    if (i < part.y) {
      const int j = kt.at(i) * kT + (lane & 31);
      if (j > from || j < pk.sinks) at_next = row_at(a.pages, seq, j, keys);
    }
  };
  auto load = [&](int i) {
    seen_next = (uint32_t)__ballot(at_next >= 0);
    staged.gather(kbase, vbase, at_next, lane);
    look(i + 4);
  };

  f32x4 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = zero4();
  float m = kMinusInf, l = 0.f;
  const float c = pk.scale * kLog2e;
  const int ka = at<D>(i16, 8 * q4);
  const int vr = 4 * q4 + (i16 >> 2), va = at<D>(vr, 4 * (i16 & 3));

  int i = part.x + wave;
  look(i);
  if (i < part.y) load(i);
  for (; i < part.y; i += 4) {
    const uint32_t seen = seen_next;
    staged.store(K, V, lane);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();  // a wave's LDS requests are done in order
    if (i + 4 < part.y) load(i + 4);
    f32x4 s[2] = {zero4(), zero4()};
    const int kf = fresh(ka);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        s[kb] = mfma16_of<T>(*reinterpret_cast<const uint4*>(K + (kf ^ (32 * d)) + 16 * kb * D), q[d], s[kb]);
    if (~seen) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!(seen >> (16 * kb + 4 * q4 + r) & 1)) s[kb][r] = kMinusInf;
    }
    float top = kMinusInf;
#pragma unroll
    for (int r = 0; r < 4; ++r) top = fmaxf(top, fmaxf(s[0][r], s[1][r]));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32)) * c - weight_lift<T>(14);
    const float now = fmaxf(m, top), base = now == kMinusInf ? 0.f : now;
    if (__any(now > m)) {
      const float f = exp2_fast(m - base);
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
    }
    m = now;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[kb][r] = exp2_fast(fmaf(s[kb][r], c, -base));
        l += s[kb][r];
      }
    // a lane's 8 keys: 4 q4 + r of the first 16 and of the second
    const uint4 p = make_uint4(pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]), pack2<T>(s[1][0], s[1][1]),
                               pack2<T>(s[1][2], s[1][3]));
    const int v0 = fresh(va);
#pragma unroll
    for (int d = 0; d < DB; ++d)
      o[d] = mfma16_of<T>(column8(V, v0 ^ (16 * d), (v0 ^ (16 * d)) + 16 * D), p, o[d]);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // the waves' results, each in its own LDS: sums [16][D], then maximum and sum of each row
  float* mine = reinterpret_cast<float*>(lds + wave * 2 * kT * D);
#pragma unroll
  for (int d = 0; d < DB; ++d) *reinterpret_cast<f32x4*>(mine + i16 * D + 16 * d + 4 * q4) = o[d];
  __shared__ float2 ml[4][16];
  if (q4 == 0) ml[wave][i16] = make_float2(m, l);
  __syncthreads();
  constexpr int kColumns = D / 4, kShares = 256 / kColumns;  // rows at a time
  const int col = tid % kColumns * 4;
  const int rows = min(G - g0, 16);
  const int64_t all = (int64_t)pk.T * pk.HQ;
#pragma unroll 1
  for (int r = tid / kColumns; r < rows; r += kShares) {
    float top = kMinusInf, sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w][r].x);
    const float base = top == kMinusInf ? 0.f : top;
    f32x4 x = zero4();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = exp2_fast(ml[w][r].x - base);
      sum += ml[w][r].y * f;
      x += *reinterpret_cast<const f32x4*>(reinterpret_cast<float*>(lds + w * 2 * kT * D) + r * D + col) * f;
    }
    const int64_t out = (int64_t)seq * pk.HQ + hk * G + g0 + r;
    if (a.splits == 1) {
      const float f = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + out * D + col) =
          make_uint2(pack2<T>(x[0] * f, x[1] * f), pack2<T>(x[2] * f, x[3] * f));
      if (a.lse && col == 0) a.lse[out] = (top + log2f(sum)) * 0.6931471805599453f;
    } else {
      const int64_t at = all * split + out;
      if (col == 0) *reinterpret_cast<float2*>(a.part + all * a.splits * D + 2 * at) = make_float2(top, sum);
      *reinterpret_cast<f32x4*>(a.part + at * D + col) = x;
    }
  }
}

hipError_t launch_attn_step(Elem type, int D, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(a.pack.N * a.splits * ((a.pack.G.by + 15) / 16) * a.pack.HK), block(256);
#define GDN_STEP(t)                                                                                      \
  if (D == 64) hipLaunchKernelGGL((attn_step_kernel<t, 64>), grid, block, 0, s, a);                  \
  else if (D == 128) hipLaunchKernelGGL((attn_step_kernel<t, 128>), grid, block, 0, s, a);           \
  else hipLaunchKernelGGL((attn_step_kernel<t, 256>), grid, block, 0, s, a)
  if (type == Elem::kBf16) { GDN_STEP(Bf16); } else { GDN_STEP(Fp16); }
#undef GDN_STEP
  return hipGetLastError();
}

}  // namespace gdn
