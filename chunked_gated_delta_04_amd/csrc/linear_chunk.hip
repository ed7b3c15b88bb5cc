// Linear attention with a decay for each head, over packed sequences.
//
// Per value head with lam = e^log_decay: S_t = lam S_{t-1} + v_t k_t^T and
// o_t = scale S_t q_t. A chunk of 64 tokens with the state S before it is, for
// its tokens i (0-based) and length L,
//   o_i = scale lam^(i+1) S q_i + sum_{j <= i} scale lam^(i-j) (q_i . k_j) v_j
//   S  <- lam^L S + sum_j lam^(L-1-j) v_j k_j^T.
// Each gradient has the same form: dq_i takes (dO, v, k) for (q, k, v) and the
// state's transpose; with the gradient G of the state after a token,
// G_t = lam G_{t+1} + scale dO_t q_t^T, dv_t = G_t k_t takes (k, q, dO) and
// dk_t = G_t^T v_t takes (v, dO, q), both from the last token to the first. So
// one kernel, lin_pass, computes o and all three gradients.
//
// Precision: bf16 operands with fp32 accumulation. The products (q_i . k_j)
// times their decay, and the carried state, are each rounded to bf16 once
// where they are multiplied with v and q: an error of the size of the output's
// own rounding. The state itself stays fp32, and what a chunk adds to it keeps
// fp32's precision: the decayed rows of c (fp32) enter the MFMA as three bf16
// pieces that hold all 24 bits, against b's exact bf16 rows.
#include "linear.h"

namespace gdn {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// log_decay in base 2. Everything from -128 down is decay zero between any two
// tokens (e^-128 is below fp32's range); the bound keeps -inf * 0 out.
__device__ __forceinline__ float decay2(float log_decay) {
  return (log_decay < -128.f ? -128.f : log_decay) * kLog2e;
}
__device__ __forceinline__ float power(float g2, int n) { return exp2_fast(g2 * (float)n); }

// One segment: its sequence, the sequence's bounds and the segment's.
struct Segment {
  int seq, bos, eos, t0, t1, index;
};

// The sequence of a segment slot: the last n whose first slot cu[n] / S + n is
// at or before it, by all lanes of a wave together (64 probes a step).
// Boundaries are clamped to [0, T], so a bad one never leads out of range.
__device__ __forceinline__ Segment find_segment(const LinCut& c, int slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = c.N;
  while (cnt > 1) {
    const int step = (cnt + 63) >> 6;
    const int at = lane * step;
    bool ok = false;
    if (at < cnt) ok = min(max(c.cu[lo + at], 0), c.T) / c.S + lo + at <= slot;
    const int k = max(__popcll(__ballot(ok)) - 1, 0);
    lo += k * step;
    cnt = min(step, cnt - k * step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  Segment s;
  s.seq = lo;
  s.bos = min(max(c.cu[lo], 0), c.T);
  s.eos = min(max(c.cu[lo + 1], s.bos), c.T);
  s.index = slot - (s.bos / c.S + lo);
  const int64_t t0 = s.bos + (int64_t)s.index * c.S;
  s.t0 = (int)min(t0, (int64_t)c.T);
  s.t1 = (int)min(t0 + c.S, (int64_t)s.eos);
  return s;
}
// whether the slot holds a segment: each sequence, an empty one too, has its first
__device__ __forceinline__ bool unused(const Segment& s) {
  return s.index < 0 || (s.index > 0 && s.t0 >= s.eos);
}

// Where sequence seq's state comes from (null: zero) and goes to (null: nowhere).
struct StateAt {
  const float* from;
  float* to;
};
__device__ __forceinline__ StateAt state_at(const StateRef& io, int seq, int hv, int HV, int DD) {
  size_t base = ((size_t)seq * HV + hv) * DD;
  const float* from = io.h0;
  float* to = io.hT;
  if (io.idx) {
    const int sl = io.idx[seq];
    const bool live = sl > 0 && sl < io.slots;
    base = live ? ((size_t)sl * HV + hv) * DD : 0;
    from = live && (!io.init || io.init[seq] != 0) ? io.h0 : nullptr;
    to = live ? io.hT : nullptr;
  }
  return {from ? from + base : nullptr, to ? to + base : nullptr};
}

// LDS rows of D bf16 with 8 elements of padding: 16-byte fragment reads of
// consecutive rows then start 4 banks apart.
template <int D>
constexpr int kPitch = D + 8;
constexpr int kPPitch = kChunk + 8;

// 64 rows of one operand, 16 bytes a piece, held by the NT threads.
template <int D, int NT>
struct RowRegs {
  static constexpr int kPieces = kChunk * D / 8 / NT;
  uint4 x[kPieces];
  __device__ __forceinline__ void load(const LinRows& r, int64_t t0, int len, int hv, int tid) {
    // rows past the chunk's end read as zeros
    const int bytes = len > 0 ? (int)(((len - 1) * r.stride + D) * 2) : 0;
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(r.p) + t0 * r.stride + (int64_t)(hv / r.G) * D, 0, bytes, kBufferWord3);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = tid + i * NT, row = e / (D / 8), col = e % (D / 8);
      x[i] = load_b128(rsrc, (int)(row * r.stride * 2) + col * 16);
    }
  }
  __device__ __forceinline__ void store(uint16_t* tile, int tid) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = tid + i * NT, row = e / (D / 8), col = e % (D / 8);
      *reinterpret_cast<uint4*>(tile + row * kPitch<D> + col * 8) = x[i];
    }
  }
};

// The carried state of a wave: X[k][32 w + lane % 32] for all k. Register
// 8 m + e of tile kb is k = 32 kb + 16 m + 8 (lane / 32) + e: the accumulator's
// rows, taken in an order that makes 8 consecutive k one MFMA operand, so that
// the state is multiplied from the registers that it is gathered in. (The
// operand gathered from, b^T, is read in that order: see b_col8.)
template <int D>
struct State {
  static constexpr int KB = D / 32;
  f32x16 x[KB];

  // kT: stored [k][column] instead of [column][k]
  template <bool kT>
  __device__ __forceinline__ void load(const float* p, int col, int hi) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int k = 32 * kb + 16 * m + 8 * hi;
        if (!p) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[kb][8 * m + e] = 0.f;
        } else if constexpr (kT) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[kb][8 * m + e] = p[(k + e) * D + col];
        } else {
          const f32x4 u = *reinterpret_cast<const f32x4*>(p + col * D + k);
          const f32x4 w = *reinterpret_cast<const f32x4*>(p + col * D + k + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[kb][8 * m + e] = u[e];
            x[kb][8 * m + 4 + e] = w[e];
          }
        }
      }
  }
  template <bool kT>
  __device__ __forceinline__ void store(float* p, int col, int hi) const {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int k = 32 * kb + 16 * m + 8 * hi;
        if constexpr (kT) {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[(k + e) * D + col] = x[kb][8 * m + e];
        } else {
          *reinterpret_cast<f32x4*>(p + col * D + k) =
              f32x4{x[kb][8 * m], x[kb][8 * m + 1], x[kb][8 * m + 2], x[kb][8 * m + 3]};
          *reinterpret_cast<f32x4*>(p + col * D + k + 4) =
              f32x4{x[kb][8 * m + 4], x[kb][8 * m + 5], x[kb][8 * m + 6], x[kb][8 * m + 7]};
        }
      }
  }
  __device__ __forceinline__ bf16x8 operand(int kb, int m) const {
    const f32x16& s = x[kb];
    return __builtin_bit_cast(bf16x8, make_uint4(pk2(s[8 * m], s[8 * m + 1]), pk2(s[8 * m + 2], s[8 * m + 3]),
                                                 pk2(s[8 * m + 4], s[8 * m + 5]), pk2(s[8 * m + 6], s[8 * m + 7])));
  }
};

// Column c0 + lane % 16 of rows r0 .. r0 + 7 (as lds_col8), the 16 columns'
// middle groups of four exchanged: the order of State's rows.
__device__ __forceinline__ bf16x8 b_col8(const uint16_t* tile, int pitch, int r0, int c0, int lane) {
  const int j = lane & 15, piece = ((j & 1) << 1) | ((j >> 1) & 1);
  const uint2 a = lds_tr16(tile + (r0 + (j >> 2)) * pitch + c0 + 4 * piece);
  const uint2 b = lds_tr16(tile + (r0 + 4 + (j >> 2)) * pitch + c0 + 4 * piece);
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}

// c's columns of one 16-token step times the tokens' weights, as three bf16
// operands whose sum holds the fp32 products' 24 bits.
struct Split {
  bf16x8 hi, mid, lo;
};
__device__ __forceinline__ Split split(const uint4& c, const float* w) {
  uint32_t h[4], m[4], l[4];
  const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(u[i] << 16) * w[2 * i];
    const float x1 = __uint_as_float(u[i] & 0xffff0000u) * w[2 * i + 1];
    h[i] = pk2(x0, x1);
    const float r0 = x0 - __uint_as_float(h[i] << 16), r1 = x1 - __uint_as_float(h[i] & 0xffff0000u);
    m[i] = pk2(r0, r1);
    l[i] = pk2(r0 - __uint_as_float(m[i] << 16), r1 - __uint_as_float(m[i] & 0xffff0000u));
  }
  return {__builtin_bit_cast(bf16x8, make_uint4(h[0], h[1], h[2], h[3])),
          __builtin_bit_cast(bf16x8, make_uint4(m[0], m[1], m[2], m[3])),
          __builtin_bit_cast(bf16x8, make_uint4(l[0], l[1], l[2], l[3]))};
}

// Weight of token t of a chunk of len tokens in the state: front to back
// lam^(len - 1 - t), back to front scale lam^(t + 1); zero past the end (where
// the rows are zeros, and a weight past fp32's range must not meet them).
template <bool kBack>
__device__ __forceinline__ float weight(float g2, float scale, int t, int len) {
  if (t >= len) return 0.f;
  return kBack ? scale * power(g2, t + 1) : power(g2, len - 1 - t);
}

// X <- lam^len X + b^T diag(w) c for one chunk in LDS.
template <int D>
__device__ __forceinline__ void gather_chunk(State<D>& X, float decay, const uint16_t* Bs, const uint4* cc,
                                             const float* ws, int lane) {
  const int g = lane >> 4, hi = lane >> 5;
#pragma unroll
  for (int kb = 0; kb < State<D>::KB; ++kb)
#pragma unroll
    for (int r = 0; r < 16; ++r) X.x[kb][r] *= decay;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const Split v = split(cc[s], ws + 16 * s + 8 * hi);
#pragma unroll
    for (int kb = 0; kb < State<D>::KB; ++kb) {
      const bf16x8 k = b_col8(Bs, kPitch<D>, 16 * s + 8 * (g >> 1), 32 * kb + 16 * (g & 1), lane);
      X.x[kb] = mfma32(k, v.lo, X.x[kb]);
      X.x[kb] = mfma32(k, v.mid, X.x[kb]);
      X.x[kb] = mfma32(k, v.hi, X.x[kb]);
    }
  }
}

template <int D>
__device__ __forceinline__ void load_columns(uint4* cc, const uint16_t* Cs, int wave, int lane) {
  const int g = lane >> 4;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    cc[s] = lds_col8(Cs, kPitch<D>, 16 * s + 8 * (g >> 1), 32 * wave + 16 * (g & 1), lane);
}

}  // namespace

// One workgroup per (segment, value head), one wave per 32 columns of the
// state and the output.
template <int D, bool kBack, bool kT, bool kWide>
__global__ __launch_bounds__(2 * D, 2) void lin_pass_kernel(LinCut cut, const float* __restrict__ log_decay,
                                                            float scale, LinPass p) {
  constexpr int NW = D / 32, NT = 64 * NW;
  const int hv = blockIdx.x % cut.HV, slot = blockIdx.x / cut.HV;
  const Segment sg = find_segment(cut, slot);
  if (unused(sg)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int l32 = lane & 31, hi = lane >> 5, l16 = lane & 15, q4 = lane >> 4;
  const float g2 = decay2(log_decay[hv]);

  __shared__ __align__(16) uint16_t As[kChunk * kPitch<D>];
  __shared__ __align__(16) uint16_t Bs[kChunk * kPitch<D>];
  __shared__ __align__(16) uint16_t Cs[kChunk * kPitch<D>];
  __shared__ __align__(16) uint16_t Ps[kChunk * kPPitch];
  __shared__ __align__(16) float ws[kChunk];

  // P's tiles on the far side of the diagonal stay zero
  for (int i = tid; i < kChunk * kPPitch / 8; i += NT) reinterpret_cast<uint4*>(Ps)[i] = make_uint4(0, 0, 0, 0);

  const bool first = kBack ? sg.t1 >= sg.eos : sg.index == 0;  // the first that the pass meets
  const bool last = kBack ? sg.index == 0 : sg.t1 >= sg.eos;
  const StateAt at = state_at(p.io, sg.seq, hv, cut.HV, D * D);
  const int col = 32 * wave + l32;
  State<D> X;
  (void)first;
  X.template load<kT>(p.start ? p.start + ((size_t)slot * cut.HV + hv) * (D * D) : at.from, col, hi);

  const int chunks = (sg.t1 - sg.t0 + kChunk - 1) / kChunk;
  for (int i = 0; i < chunks; ++i) {
    const int c = kBack ? chunks - 1 - i : i;
    const int64_t t0 = sg.t0 + c * kChunk;
    const int len = min(kChunk, sg.t1 - (int)t0);
    RowRegs<D, NT> ra, rb, rc;
    ra.load(p.a, t0, len, hv, tid);
    rb.load(p.b, t0, len, hv, tid);
    rc.load(p.c, t0, len, hv, tid);
    __syncthreads();  // the last chunk's readers are done
    ra.store(As, tid);
    rb.store(Bs, tid);
    rc.store(Cs, tid);
    if (tid < kChunk) ws[tid] = weight<kBack>(g2, scale, tid, len);
    __syncthreads();

    // P[i][j] = scale lam^|i - j| a_i . b_j, in 16 x 16 tiles on and beside the
    // diagonal, as P^T tiles so that a lane holds 4 consecutive j of one i
#pragma unroll
    for (int n = 0; n < 16 / NW; ++n) {
      const int tile = wave + NW * n, ti = tile >> 2, tj = tile & 3;
      if (kBack ? tj < ti : tj > ti) continue;
      f32x4 acc = zero4();
#pragma unroll
      for (int s = 0; s < D / 32; ++s)
        acc = mfma(ld8(Bs + (16 * tj + l16) * kPitch<D> + 32 * s + 8 * q4),
                   ld8(As + (16 * ti + l16) * kPitch<D> + 32 * s + 8 * q4), acc);
      const int pi = 16 * ti + l16, pj = 16 * tj + 4 * q4;
      float w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = kBack ? pj + r - pi : pi - pj - r;
        w[r] = d >= 0 ? acc[r] * (scale * power(g2, d)) : 0.f;
      }
      *reinterpret_cast<uint2*>(Ps + pi * kPPitch + pj) = pack4_bf16(w[0], w[1], w[2], w[3]);
    }

    // the state's part of the output, transposed: rows are columns of c
    f32x16 o[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[tb][r] = 0.f;
#pragma unroll
    for (int kb = 0; kb < State<D>::KB; ++kb)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const bf16x8 x = X.operand(kb, m);
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
          o[tb] = mfma32(x, ld8(As + (32 * tb + l32) * kPitch<D> + 32 * kb + 16 * m + 8 * hi), o[tb]);
      }
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const int t = 32 * tb + l32;
      const float f = kBack ? power(g2, max(len - 1 - t, 0)) : scale * power(g2, t + 1);
#pragma unroll
      for (int r = 0; r < 16; ++r) o[tb][r] *= f;
    }
    uint4 cc[4];
    load_columns<D>(cc, Cs, wave, lane);
    __syncthreads();  // P is there
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (kBack ? s < 2 * tb : s >= 2 * tb + 2) continue;
        o[tb] = mfma32(__builtin_bit_cast(bf16x8, cc[s]),
                       ld8(Ps + (32 * tb + l32) * kPPitch + 16 * s + 8 * hi), o[tb]);
      }

    // row t = 32 tb + lane % 32; register 4 j + i is column 8 j + 4 (lane / 32) + i
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const int t = 32 * tb + l32;
      const size_t row = ((size_t)(t0 + t) * cut.HV + hv) * D + 32 * wave;
      if (t < len) {
        if constexpr (kWide) {
          float* out = static_cast<float*>(p.out) + row;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4*>(out + 8 * j + 4 * hi) =
                f32x4{o[tb][4 * j], o[tb][4 * j + 1], o[tb][4 * j + 2], o[tb][4 * j + 3]};
        }
      }
      if constexpr (!kWide) {
        // the half-waves exchange 4 columns, so that a lane stores 8 in a row
        uint16_t* out = static_cast<uint16_t*>(p.out) + row;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const f32x16& v = o[tb];
          const auto x = __builtin_amdgcn_permlane32_swap(pk2(v[8 * m], v[8 * m + 1]), pk2(v[8 * m + 4], v[8 * m + 5]), false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(pk2(v[8 * m + 2], v[8 * m + 3]), pk2(v[8 * m + 6], v[8 * m + 7]), false, false);
          if (t < len) *reinterpret_cast<uint4*>(out + 16 * m + 8 * hi) = make_uint4(x[0], y[0], x[1], y[1]);
        }
      }
    }
    gather_chunk<D>(X, power(g2, len), Bs, cc, ws, lane);
  }
  if (last && at.to) X.template store<kT>(at.to, col, hi);
}

// What a segment adds to the state, from a zero start.
template <int D, bool kBack>
__global__ __launch_bounds__(2 * D, 2) void lin_gather_kernel(LinCut cut, const float* __restrict__ log_decay,
                                                              float scale, LinRows b, LinRows c,
                                                              float* __restrict__ states) {
  constexpr int NW = D / 32, NT = 64 * NW;
  const int hv = blockIdx.x % cut.HV, slot = blockIdx.x / cut.HV;
  const Segment sg = find_segment(cut, slot);
  if (unused(sg) || (kBack ? sg.index == 0 : sg.t1 >= sg.eos)) return;  // nothing follows it
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const float g2 = decay2(log_decay[hv]);
  __shared__ __align__(16) uint16_t Bs[kChunk * kPitch<D>];
  __shared__ __align__(16) uint16_t Cs[kChunk * kPitch<D>];
  __shared__ __align__(16) float ws[kChunk];
  State<D> X;
  X.template load<false>(nullptr, 0, 0);
  const int chunks = (sg.t1 - sg.t0 + kChunk - 1) / kChunk;
  for (int i = 0; i < chunks; ++i) {
    const int ch = kBack ? chunks - 1 - i : i;
    const int64_t t0 = sg.t0 + ch * kChunk;
    const int len = min(kChunk, sg.t1 - (int)t0);
    RowRegs<D, NT> rb, rc;
    rb.load(b, t0, len, hv, tid);
    rc.load(c, t0, len, hv, tid);
    __syncthreads();
    rb.store(Bs, tid);
    rc.store(Cs, tid);
    if (tid < kChunk) ws[tid] = weight<kBack>(g2, scale, tid, len);
    __syncthreads();
    uint4 cc[4];
    load_columns<D>(cc, Cs, wave, lane);
    gather_chunk<D>(X, power(g2, len), Bs, cc, ws, lane);
  }
  X.template store<false>(states + ((size_t)slot * cut.HV + hv) * (D * D), 32 * wave + (lane & 31), lane >> 5);
}

// Front to back along each sequence's segments (or back to front): a thread
// carries 4 values of one state.
template <int D, bool kBack>
__global__ __launch_bounds__(256) void lin_join_kernel(LinCut cut, bool gathered,
                                                       const float* __restrict__ log_decay, StateRef io,
                                                       float* __restrict__ states) {
  constexpr int kBlocks = D * D / 1024;
  const int piece = blockIdx.x % kBlocks, hv = blockIdx.x / kBlocks % cut.HV;
  const int seq = blockIdx.x / (kBlocks * cut.HV);
  const int bos = min(max(cut.cu[seq], 0), cut.T), eos = min(max(cut.cu[seq + 1], bos), cut.T);
  const int first = bos / cut.S + seq;
  const int n = max((eos - bos + cut.S - 1) / cut.S, 1);
  const int e = piece * 1024 + threadIdx.x * 4;
  const StateAt at = state_at(io, seq, hv, cut.HV, D * D);
  const float g2 = decay2(log_decay[hv]);
  f32x4 x = zero4();
  if (at.from) x = *reinterpret_cast<const f32x4*>(at.from + e);
  for (int i = 0; i < n; ++i) {
    const int s = kBack ? n - 1 - i : i;
    float* p = states + ((size_t)(first + s) * cut.HV + hv) * (D * D) + e;
    f32x4 add = zero4();
    if (gathered && i + 1 < n) add = *reinterpret_cast<const f32x4*>(p);
    *reinterpret_cast<f32x4*>(p) = x;
    const float d = power(g2, min(cut.S, eos - bos - s * cut.S));
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = d * x[r] + add[r];
  }
}

__global__ __launch_bounds__(256) void lin_fold_kernel(int64_t n, int DH, int G, int D,
                                                       const float* __restrict__ wide, uint16_t* __restrict__ out) {
  // n pieces of 4 outputs; DH = H * D outputs a token
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t e = i * 4, t = e / DH;
    const int rest = (int)(e - t * DH), h = rest / D, d = rest - h * D;
    const float* p = wide + (t * DH + (int64_t)h * D) * G + d;
    f32x4 s = zero4();
    for (int j = 0; j < G; ++j) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + (int64_t)j * D);
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] += x[r];
    }
    *reinterpret_cast<uint2*>(out + e) = pack4_bf16(s[0], s[1], s[2], s[3]);
  }
}

namespace {

template <int D, bool kBack, bool kT, bool kWide>
hipError_t pass(const LinCut& cut, const float* log_decay, float scale, const LinPass& p, hipStream_t s) {
  hipLaunchKernelGGL((lin_pass_kernel<D, kBack, kT, kWide>), dim3((unsigned)cut.slots * (unsigned)cut.HV),
                     dim3(2 * D), 0, s, cut, log_decay, scale, p);
  return hipGetLastError();
}

template <int D>
hipError_t pass_of(LinKind kind, bool wide, const LinCut& cut, const float* log_decay, float scale,
                   const LinPass& p, hipStream_t s) {
  switch (kind) {
    case LinKind::kOut: return pass<D, false, false, false>(cut, log_decay, scale, p, s);
    case LinKind::kDq:
      return wide ? pass<D, false, true, true>(cut, log_decay, scale, p, s)
                  : pass<D, false, true, false>(cut, log_decay, scale, p, s);
    case LinKind::kDv: return pass<D, true, false, false>(cut, log_decay, scale, p, s);
    default:
      return wide ? pass<D, true, true, true>(cut, log_decay, scale, p, s)
                  : pass<D, true, true, false>(cut, log_decay, scale, p, s);
  }
}

}  // namespace

hipError_t launch_lin_pass(LinKind kind, bool wide, int D, const LinCut& cut, const float* log_decay,
                           float scale, const LinPass& p, hipStream_t s) {
  return D == 128 ? pass_of<128>(kind, wide, cut, log_decay, scale, p, s)
                  : pass_of<64>(kind, wide, cut, log_decay, scale, p, s);
}

hipError_t launch_lin_gather(bool back, int D, const LinCut& cut, const float* log_decay, float scale,
                             const LinRows& b, const LinRows& c, float* states, hipStream_t s) {
  const dim3 grid((unsigned)cut.slots * (unsigned)cut.HV), block(2 * D);
  if (D == 128 && back)
    hipLaunchKernelGGL((lin_gather_kernel<128, true>), grid, block, 0, s, cut, log_decay, scale, b, c, states);
  else if (D == 128)
    hipLaunchKernelGGL((lin_gather_kernel<128, false>), grid, block, 0, s, cut, log_decay, scale, b, c, states);
  else if (back)
    hipLaunchKernelGGL((lin_gather_kernel<64, true>), grid, block, 0, s, cut, log_decay, scale, b, c, states);
  else
    hipLaunchKernelGGL((lin_gather_kernel<64, false>), grid, block, 0, s, cut, log_decay, scale, b, c, states);
  return hipGetLastError();
}

hipError_t launch_lin_join(bool back, bool gathered, int D, const LinCut& cut, const float* log_decay,
                           const StateRef& io, float* states, hipStream_t s) {
  const dim3 grid((unsigned)cut.N * (unsigned)cut.HV * (unsigned)(D * D / 1024)), block(256);
  if (D == 128 && back)
    hipLaunchKernelGGL((lin_join_kernel<128, true>), grid, block, 0, s, cut, gathered, log_decay, io, states);
  else if (D == 128)
    hipLaunchKernelGGL((lin_join_kernel<128, false>), grid, block, 0, s, cut, gathered, log_decay, io, states);
  else if (back)
    hipLaunchKernelGGL((lin_join_kernel<64, true>), grid, block, 0, s, cut, gathered, log_decay, io, states);
  else
    hipLaunchKernelGGL((lin_join_kernel<64, false>), grid, block, 0, s, cut, gathered, log_decay, io, states);
  return hipGetLastError();
}

hipError_t launch_lin_fold(int D, int T, int H, int G, const float* wide, uint16_t* out, hipStream_t s) {
  const int64_t n = (int64_t)T * H * D / 4;
  const unsigned blocks = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
  hipLaunchKernelGGL(lin_fold_kernel, dim3(blocks), dim3(256), 0, s, n, H * D, G, D, wide, out);
  return hipGetLastError();
}

}  // namespace gdn
