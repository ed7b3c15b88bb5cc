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
#include <type_traits>

#include "lds_tile.h"
#include "linear.h"

namespace gdn {

namespace {

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// log_decay in base 2. Everything from -128 down is decay zero between any two
// tokens (e^-128 is below fp32's range); the bound keeps -inf * 0 out.
__device__ __forceinline__ float decay2(float log_decay) {
  return (log_decay < -128.f ? -128.f : log_decay) * kLog2e;
}
__device__ __forceinline__ float power(float g2, int n) { return exp2_fast(g2 * (float)n); }

// One segment: its sequence, the sequence's bounds and its own, its number in the
// sequence and its slot.
struct Segment {
  int seq, bos, eos, t0, t1, index, slot;
};

// The segment of number i in the order of the work: first the N sequences' first
// ones, then the others by position. Segment j > 0 of sequence n has the number
// N + cu[n] / S + j - 1, so its sequence is the last n with cu[n] / S at or before
// i - N, found by all lanes of a wave together (64 probes a step). The numbers that
// no segment has are among the last, and leave no gaps between the workgroups that
// start together: 16 x 512 tokens, 8 heads of 128, forward and backward 104 us, and
// 143 in the order of the slots, where every other one is empty.
// Boundaries are clamped to [0, T], so a bad one never leads out of range.
__device__ __forceinline__ Segment find_segment(const LinCut& c, int i) {
  int lo = i;
  if (i >= c.N) {
    const int lane = threadIdx.x & 63;
    int cnt = c.N;
    lo = 0;
    while (cnt > 1) {
      const int step = (cnt + 63) >> 6;
      const int at = lane * step;
      bool ok = false;
      if (at < cnt) ok = min(max(c.cu[lo + at], 0), c.T) / c.S <= i - c.N;
      const int k = max(__popcll(__ballot(ok)) - 1, 0);
      lo += k * step;
      cnt = min(step, cnt - k * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
  }
  Segment s;
  s.seq = lo;
  s.bos = min(max(c.cu[lo], 0), c.T);
  s.eos = min(max(c.cu[lo + 1], s.bos), c.T);
  s.index = i < c.N ? 0 : i - c.N - s.bos / c.S + 1;
  if (i >= c.N && s.index < 1) s.index = -1;  // bad boundaries
  s.slot = s.bos / c.S + lo + s.index;
  const int64_t t0 = s.bos + (int64_t)s.index * c.S;
  s.t0 = (int)min(t0, (int64_t)c.T);
  s.t1 = (int)min(t0 + c.S, (int64_t)s.eos);
  return s;
}
// whether it is its whole sequence
__device__ __forceinline__ bool whole(const Segment& s) { return s.index == 0 && s.t1 >= s.eos; }
__device__ __forceinline__ int chunks_of(const Segment& s) { return (s.t1 - s.t0 + kChunk - 1) / kChunk; }
// whether the number has no segment: each sequence, an empty one too, has its first
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

constexpr int kPPitch = kChunk + 8;

// 64 rows of one operand, 16 bytes a piece, held by the NT threads.
template <int D, int NT>
struct RowRegs {
  static constexpr int kPieces = kChunk * D / 8 / NT, kRows = kChunk / kPieces;  // rows a piece of all threads
  uint4 x[kPieces];
  // Piece i of the rows that a resource of chunk_rows covers; lane_byte: this thread's row (of kRows) and piece.
  // Rows past the chunk's end lie past the resource and read as zeros.
  __device__ __forceinline__ void load(int i, __amdgpu_buffer_rsrc_t rows, int lane_byte, int step_bytes) {
    x[i] = load_b128(rows, lane_byte + i * step_bytes);
  }
  static __device__ __forceinline__ int lane_byte(int stride, int tid) {
    return tid / (D / 8) * stride * 2 + tid % (D / 8) * 16;
  }
  __device__ __forceinline__ void store(uint16_t* tile, int tid) const {
    const int off = at<D>(tid / (D / 8), tid % (D / 8) * 8);  // kRows is a multiple of 16
#pragma unroll
    for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(tile + off + i * kRows * D) = x[i];
  }
};
// the head's columns of the pack's first token
template <int D>
__device__ __forceinline__ const uint16_t* head_of(const LinRows& r, int hv) {
  return r.p + (int64_t)(hv / r.G) * D;
}

// The rows of len tokens from t0 on (none: an empty resource), of a head whose columns of token 0 are at p.
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const uint16_t* p, int stride, int t0, int len) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p) + (int64_t)t0 * stride, 0,
                                           len > 0 ? ((len - 1) * stride + D) * 2 : 0, kBufferWord3);
}

// Offsets of a wave's operand reads: one lane-dependent part each, to which a
// read's pieces add by xor (they are bits below the row's) and its 16-row tiles
// by plus.
template <int D>
struct Lane {
  int row32, row16, ka, kb, va, vb;
  __device__ __forceinline__ Lane(int lane, int wave) {
    const int l32 = lane & 31, hi = lane >> 5, l16 = lane & 15, q4 = lane >> 4, j = lane & 15;
    row32 = at<D>(l32, 8 * hi);
    row16 = at<D>(l16, 8 * q4);
    const int r = 8 * hi + (j >> 2), c = 16 * (q4 & 1);
    const int swapped = ((j & 1) << 1) | ((j >> 1) & 1);  // see State
    ka = at<D>(r, c + 4 * swapped);
    kb = at<D>(r + 4, c + 4 * swapped);
    va = at<D>(r, 32 * wave + c + 4 * (j & 3));
    vb = at<D>(r + 4, 32 * wave + c + 4 * (j & 3));
  }
};

// The carried state of a wave: X[k][32 w + lane % 32] for all k. Register
// 8 m + e of tile kb is k = 32 kb + 16 m + 8 (lane / 32) + e: the accumulator's
// rows, taken in an order that makes 8 consecutive k one MFMA operand, so that
// the state is multiplied from the registers that it is gathered in. (The
// operand gathered from, b^T, is read in that order, with the 16 columns' middle groups of
// four exchanged.)
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
  __device__ __forceinline__ void decay(float f) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) x[kb][r] *= f;
  }
  __device__ __forceinline__ bf16x8 operand(int kb, int m) const {
    const f32x16& s = x[kb];
    return __builtin_bit_cast(bf16x8, make_uint4(pk2(s[8 * m], s[8 * m + 1]), pk2(s[8 * m + 2], s[8 * m + 3]),
                                                 pk2(s[8 * m + 4], s[8 * m + 5]), pk2(s[8 * m + 6], s[8 * m + 7])));
  }
};

// c's columns of one 16-token step times the tokens' weights, as kPieces bf16
// operands: three hold the fp32 products' 24 bits, two their first 16.
template <int kPieces>
struct Split {
  bf16x8 x[kPieces];  // largest first
  __device__ __forceinline__ void of(const uint4& c, const float* w) {
    const uint32_t u[4] = {c.x, c.y, c.z, c.w};
    uint32_t h[kPieces][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float r0 = __uint_as_float(u[i] << 16) * w[2 * i];
      float r1 = __uint_as_float(u[i] & 0xffff0000u) * w[2 * i + 1];
#pragma unroll
      for (int n = 0; n < kPieces; ++n) {
        h[n][i] = pk2(r0, r1);
        r0 -= __uint_as_float(h[n][i] << 16);
        r1 -= __uint_as_float(h[n][i] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int n = 0; n < kPieces; ++n)
      x[n] = __builtin_bit_cast(bf16x8, make_uint4(h[n][0], h[n][1], h[n][2], h[n][3]));
  }
};

// Weight of token t of a chunk of len tokens in the state: front to back
// lam^(len - 1 - t), back to front scale lam^(t + 1); zero past the end (where
// the rows are zeros, and a weight past fp32's range must not meet them).
template <bool kBack>
__device__ __forceinline__ float weight(float g2, float scale, int t, int len) {
  if (t >= len) return 0.f;
  return kBack ? scale * power(g2, t + 1) : power(g2, len - 1 - t);
}

// X <- X + b^T diag(w) c for one chunk in LDS, 16 tokens a step. A step's
// operands are read and split while the step before multiplies.
template <int D, int kPieces>
__device__ __forceinline__ void gather_chunk(State<D>& X, const uint16_t* Bs, const uint4* cc, const float* ws,
                                             const Lane<D>& L, int hi) {
  constexpr int KB = State<D>::KB;
  const int ka = fresh(L.ka), kb = fresh(L.kb);
  uint4 k[2][KB];
  Split<kPieces> v[2];
  auto read = [&](int s) {
#pragma unroll
    for (int i = 0; i < KB; ++i) k[s & 1][i] = column8(Bs + 16 * s * D, ka ^ (32 * i), kb ^ (32 * i));
  };
  read(0);
  v[0].of(cc[0], ws + 8 * hi);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s < 3) {
      read(s + 1);
      v[(s + 1) & 1].of(cc[s + 1], ws + 16 * (s + 1) + 8 * hi);
    }
    // smallest pieces first; the state's tiles in turn, so that no product waits for the one before it
#pragma unroll
    for (int n = kPieces - 1; n >= 0; --n)
#pragma unroll
      for (int i = 0; i < KB; ++i) X.x[i] = mfma32(__builtin_bit_cast(bf16x8, k[s & 1][i]), v[s & 1].x[n], X.x[i]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int D>
__device__ __forceinline__ void load_columns(uint4* cc, const uint16_t* Cs, const Lane<D>& L) {
#pragma unroll
  for (int s = 0; s < 4; ++s) cc[s] = column8(Cs + 16 * s * D, L.va, L.vb);
}

// The n-th 16 x 16 tile of P of a wave, rows i, columns j: the 10 tiles on and on
// one side of the diagonal, 3 or 5 to a wave, the first of them of one row i, so
// that a's rows are read once for these. (With 4 waves, two tiles are formed twice,
// which costs less than a branch.)
struct Tile {
  int i, j;
};
template <int NW>
constexpr int kTilesOf = NW == 4 ? 3 : 5;
template <int NW, bool kBack>
__device__ __forceinline__ Tile tile_of(int wave, int n) {
  int i, j;
  if constexpr (NW == 4) {  // 33 32 31; 22 21 20; 11 10 30; 00 00 30 (its n = 0, 1 are the same tile)
    i = n < 2 ? 3 - wave : wave < 2 ? 3 - wave : 3;
    j = n < 2 ? max(3 - wave - n, 0) : wave < 2 ? 1 - wave : 0;
  } else {  // 33 32 31 11 10; 22 21 20 30 00
    i = n < 3 ? 3 - wave : wave == 0 ? 1 : n == 3 ? 3 : 0;
    j = n < 3 ? 3 - wave - n : wave == 0 ? 4 - n : 0;
  }
  if (kBack) return {3 - i, 3 - j};
  return {i, j};
}

}  // namespace

// What workgroup n works on: a segment, a value head, and one of `parts` passes
// (-1: nothing, at the grid's end).
//   Workgroups go to the 8 XCDs in turn. Those that read the same rows, the passes
// of a segment and the value heads of a key head, are 8 apart, so that they run on
// one XCD at one time and share its L2: a forward over 32768 tokens of 16 key and 32
// value heads reads 591 MB, and 852 with the value heads on XCDs of their own.
//   Key heads are side by side, so that a token's whole row is read at about one
// time, and a head's place moves by one from segment to segment. Without that, an
// XCD reads the same 256 bytes of every 2 KiB throughout, and two of the eight took
// 14 % longer than the others: gradients of 2 x 8192 tokens, 32 heads, 300 us, and
// 286 with it.
struct Item {
  int seg, hv, part;
};
__device__ __forceinline__ Item item_of(const LinCut& cut, int n, int parts) {
  const int H = cut.HV / cut.G, sharing = parts * cut.G;
  const int nth = n >> 3, r = nth % sharing, m = nth / sharing * 8 + (n & 7);
  if (m >= cut.slots * H) return {-1, 0, 0};
  const int seg = m / H;
  return {seg, (m + seg) % H * cut.G + r / parts, r % parts};
}
unsigned items_grid(const LinCut& cut, int parts) {
  return ((unsigned)cut.slots * (unsigned)(cut.HV / cut.G) + 7) / 8 * 8 * (unsigned)(parts * cut.G);
}

template <int D>
struct PassLds {
  uint16_t As[kChunk * D], Bs[kChunk * D], Cs[kChunk * D];
  uint16_t Ps[kChunk * kPPitch];
  float ws[kChunk];
};

// One segment of one value head by one workgroup, one wave per 32 columns of the
// state and the output, two workgroups to a CU. Alone on a CU a 64-token step of
// D = 128 takes 6400 clocks (7200 with kEnds): rows into LDS 730, P 960, the state's
// part of the output 900, P's 490, output and gathering the rest. Two to a CU take
// 5200 to 5600 a step, in which a SIMD's matrix unit is busy for 1920 (34 %), its
// vector unit for 1750 (31 %) and the CU's LDS for 2250 (40 %): the bound is how well
// two waves a SIMD fill each other's waits, and beside it HBM: o of 2 x 8192 tokens,
// 32 heads, takes 112 us (570 MB, 5.1 TB/s), the three gradients 267 us (1.4 GB, 5.2
// TB/s; the least of sixty calls, their medians 118 and 293). A third workgroup does
// not fit (244 VGPRs). Waves of 16 columns, four to a SIMD, read b^T and a twice as
// often: no faster (a step alone 7700 clocks, these gradients 297 us for 286).
// kEnds: the segment is a whole sequence whose end state goes to p.io: it is
// gathered to fp32's precision. Otherwise the carried state only meets a, rounded
// to bf16, and 16 bits of what it gathers are enough (a third less matrix work);
// what a sequence of several segments ends with is lin_join's.
template <int D, bool kBack, bool kT, bool kWide, bool kEnds>
__device__ __forceinline__ void lin_pass(const LinCut& cut, int hv, const Segment& sg,
                                         const float* __restrict__ log_decay, float scale, const LinPass& p,
                                         PassLds<D>& lds) {
  constexpr int NW = D / 32, NT = 64 * NW, kTiles = kTilesOf<NW>;
  uint16_t *As = lds.As, *Bs = lds.Bs, *Cs = lds.Cs, *Ps = lds.Ps;
  float* ws = lds.ws;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int l32 = lane & 31, hi = lane >> 5, l16 = lane & 15, q4 = lane >> 4;
  const float g2 = decay2(log_decay[hv]);

  // P's tiles on the far side of the diagonal stay zero
  for (int i = tid; i < kChunk * kPPitch / 8; i += NT) reinterpret_cast<uint4*>(Ps)[i] = make_uint4(0, 0, 0, 0);

  const StateAt state = state_at(p.io, sg.seq, hv, cut.HV, D * D);
  const int col = 32 * wave + l32;
  State<D> X;
  X.template load<kT>(p.start ? p.start + ((size_t)sg.slot * cut.HV + hv) * (D * D) : state.from, col, hi);

  const int chunks = chunks_of(sg);
  // the decays of this lane's elements of P do not change from chunk to chunk
  float pw[kTiles][4];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    const Tile x = tile_of<NW, kBack>(wave, n);
    const int d = 16 * (kBack ? x.j - x.i : x.i - x.j) + (kBack ? 4 * q4 - l16 : l16 - 4 * q4);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = kBack ? d + r : d - r;
      pw[n][r] = e >= 0 ? scale * power(g2, e) : 0.f;
    }
  }
  // the next chunk's rows are on their way while a chunk is computed
  const Lane<D> L(lane, wave);
  RowRegs<D, NT> ra, rb, rc;
  const uint16_t *ap = head_of<D>(p.a, hv), *bp = head_of<D>(p.b, hv), *cp = head_of<D>(p.c, hv);
  const int ga = (int)p.a.stride, gb = (int)p.b.stride, gc = (int)p.c.stride;  // checked: below 2^23
  const int la = ra.lane_byte(ga, tid), lb = rb.lane_byte(gb, tid), lc = rc.lane_byte(gc, tid);
  const int sa = ra.kRows * ga * 2, sb = rb.kRows * gb * 2, sc = rc.kRows * gc * 2;
  // one of the next chunk's 12 pieces; past the segment's end they are zeros that nothing reads
  __amdgpu_buffer_rsrc_t na, nb, nc;
  auto next = [&](int i) {
    const int n = max(min(i, chunks - 1), 0), t0 = sg.t0 + (kBack ? chunks - 1 - n : n) * kChunk;
    const int len = i < chunks ? min(kChunk, sg.t1 - t0) : 0;
    na = chunk_rows<D>(ap, ga, t0, len);
    nb = chunk_rows<D>(bp, gb, t0, len);
    nc = chunk_rows<D>(cp, gc, t0, len);
  };
  constexpr int kLoads = 3 * RowRegs<D, NT>::kPieces;
  auto request = [&](int j) {
    const int piece = j / 3;
    if (j % 3 == 0) ra.load(piece, na, la, sa);
    if (j % 3 == 1) rb.load(piece, nb, lb, sb);
    if (j % 3 == 2) rc.load(piece, nc, lc, sc);
  };
  using Out = typename std::conditional<kWide, float, uint16_t>::type;
  const int orow = cut.HV * D * (int)sizeof(Out);  // bytes of a token's output row
  const int ob = l32 * orow + (kWide ? (32 * wave + 4 * hi) * 4 : (32 * wave + 8 * hi) * 2);
  next(0);
#pragma unroll
  for (int j = 0; j < kLoads; ++j) request(j);
  for (int i = 0; i < chunks; ++i) {
    const int t0 = sg.t0 + (kBack ? chunks - 1 - i : i) * kChunk;
    const int len = min(kChunk, sg.t1 - t0);
    // Ahead of the other workgroup's wave until P is there: while it gathers, this one
    // gets to its next products (gradients of 2 x 8192 tokens, 32 heads, 287 -> 267 us).
    __builtin_amdgcn_s_setprio(1);
    lds_barrier();  // the last chunk's readers are done
    ra.store(As, tid);
    rb.store(Bs, tid);
    rc.store(Cs, tid);
    if (tid < kChunk) ws[tid] = weight<kBack>(g2, scale, tid, len);
    lds_barrier();
    next(i + 1);

    // P[i][j] = scale lam^|i - j| a_i . b_j, in 16 x 16 tiles on and beside the
    // diagonal, as P^T tiles so that a lane holds 4 consecutive j of one i. The
    // next chunk's requests go out between the tiles and the steps below: all at
    // once they would hold the wave up for longer than a tile takes.
    const int r16 = fresh(L.row16);
    f32x4 pt[kTiles];
    {
      // the tiles' rows of a: the first tiles' one i, then another for each
      constexpr int kFirst = NW == 4 ? 2 : 3;
      auto group = [](int n) { return n < kFirst ? 0 : n - kFirst + 1; };
      bf16x8 arow[kTiles - kFirst + 1][D / 32], brow[kTiles][D / 32];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const Tile x = tile_of<NW, kBack>(wave, n);
        pt[n] = zero4();
#pragma unroll
        for (int s = 0; s < D / 32; ++s) brow[n][s] = ld8(Bs + 16 * D * x.j + (r16 ^ (32 * s)));
        if (n == 0 || n >= kFirst) {
#pragma unroll
          for (int s = 0; s < D / 32; ++s) arow[group(n)][s] = ld8(As + 16 * D * x.i + (r16 ^ (32 * s)));
        }
        __builtin_amdgcn_sched_barrier(0);  // all reads are on their way before the first product waits for one
      }
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n) pt[n] = mfma(brow[n][s], arow[group(n)][s], pt[n]);
        if (s < kTiles) request(s);
      }
#pragma unroll
      for (int s = D / 32; s < kTiles; ++s) request(s);
    }
    auto put = [&](int n) {  // a finished tile times its decays, in bf16
      const Tile x = tile_of<NW, kBack>(wave, n);
      float w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) w[r] = pw[n][r] != 0.f ? pt[n][r] * pw[n][r] : 0.f;
      if (kBack && len < kChunk) {  // no tokens past the chunk's end: zeros, whose decays may be past fp32's range
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = 16 * x.j + 4 * q4 + r < len ? w[r] : 0.f;
      }
      *reinterpret_cast<uint2*>(Ps + (16 * x.i + l16) * kPPitch + 16 * x.j + 4 * q4) = pack4_bf16(w[0], w[1], w[2], w[3]);
    };

    // the state's part of the output, transposed: rows are columns of c
    f32x16 o[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[tb][r] = 0.f;
    const int r32 = fresh(L.row32);
    bf16x8 q[2][2];  // read one step ahead
    auto read = [&](int s) {
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) q[s & 1][tb] = ld8(As + 32 * D * tb + (r32 ^ (16 * s)));
    };
    constexpr int kSteps = D / 16, kLeft = kLoads - kTiles;
    read(0);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s + 1 < kSteps) read(s + 1);
      const bf16x8 x = X.operand(s >> 1, s & 1);
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) o[tb] = mfma32(x, q[s & 1][tb], o[tb]);
#pragma unroll
      for (int n = s * kTiles / kSteps; n < (s + 1) * kTiles / kSteps; ++n) put(n);
#pragma unroll
      for (int j = kTiles + s * kLeft / kSteps; j < kTiles + (s + 1) * kLeft / kSteps; ++j) request(j);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const int t = 32 * tb + l32;
      const float f = kBack ? power(g2, max(len - 1 - t, 0)) : scale * power(g2, t + 1);
#pragma unroll
      for (int r = 0; r < 16; ++r) o[tb][r] *= f;
    }
    uint4 cc[4];
    load_columns<D>(cc, Cs, L);
    __builtin_amdgcn_s_setprio(0);
    lds_barrier();  // P is there
    bf16x8 pr[2][4];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (kBack ? s >= 2 * tb : s < 2 * tb + 2) pr[tb][s] = ld8(Ps + (32 * tb + l32) * kPPitch + 16 * s + 8 * hi);
    X.decay(power(g2, len));  // beside these reads and products
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (kBack ? s >= 2 * tb : s < 2 * tb + 2) o[tb] = mfma32(__builtin_bit_cast(bf16x8, cc[s]), pr[tb][s], o[tb]);

    // row t = 32 tb + lane % 32; register 4 j + i is column 8 j + 4 (lane / 32) + i. Rows past the chunk's end are
    // past the buffer's, whose stores the hardware drops.
    Out* const out = static_cast<Out*>(p.out) + ((int64_t)t0 * cut.HV + hv) * D;
    const __amdgpu_buffer_rsrc_t ro =
        __builtin_amdgcn_make_buffer_rsrc(out, 0, (len - 1) * orow + D * (int)sizeof(Out), kBufferWord3);
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const f32x16& v = o[tb];
      const int byte = ob + 32 * tb * orow;
      if constexpr (kWide) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store_b128(__builtin_bit_cast(uint4, f32x4{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]}), ro, byte + 32 * j);
      } else {
        // the half-waves exchange 4 columns, so that a lane stores 8 in a row
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const auto x = __builtin_amdgcn_permlane32_swap(pk2(v[8 * m], v[8 * m + 1]), pk2(v[8 * m + 4], v[8 * m + 5]), false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(pk2(v[8 * m + 2], v[8 * m + 3]), pk2(v[8 * m + 6], v[8 * m + 7]), false, false);
          store_b128(make_uint4(x[0], y[0], x[1], y[1]), ro, byte + 32 * m);
        }
      }
    }
    gather_chunk<D, kEnds ? 3 : 2>(X, Bs, cc, ws, L, hi);
  }
  if (kEnds && state.to) X.template store<kT>(state.to, col, hi);
}

template <int D>
__global__ __launch_bounds__(2 * D, 2) void lin_out_kernel(LinCut cut, const float* __restrict__ log_decay,
                                                           float scale, LinPass p) {
  __shared__ __align__(16) PassLds<D> lds;
  const Item it = item_of(cut, blockIdx.x, 1);
  if (it.seg < 0) return;
  const Segment sg = find_segment(cut, it.seg);
  if (unused(sg)) return;
  if (whole(sg)) lin_pass<D, false, false, false, true>(cut, it.hv, sg, log_decay, scale, p, lds);
  else lin_pass<D, false, false, false, false>(cut, it.hv, sg, log_decay, scale, p, lds);
}

// What a segment adds to the state, from a zero start: sum over its tokens of
// w_t b_t c_t^T, w_t = lam^(tokens after t) (back to front: scale lam^(tokens
// from the segment's start through t)). The chunks of the largest weights come
// first, and the rest are not read once every further weight is zero in fp32
// (lam^n = 0 from e^-104 on), as it soon is for quickly forgetting heads. Bound by
// HBM: 16384 tokens, 32 heads, 60 to 66 us for 262 MB (4.2 TB/s; 16 steps, the first
// of which waits for its rows).
template <int D, bool kBack>
__device__ __forceinline__ void lin_gather(const LinCut& cut, int seg, int hv, const float* __restrict__ log_decay,
                                           float scale, const LinRows& b, const LinRows& c,
                                           bool ends, float* __restrict__ states, PassLds<D>& lds) {
  constexpr int NW = D / 32, NT = 64 * NW;
  uint16_t *Bs = lds.Bs, *Cs = lds.Cs;
  float* ws = lds.ws;
  const Segment sg = find_segment(cut, seg);
  if (unused(sg) || whole(sg) || (!ends && (kBack ? sg.index == 0 : sg.t1 >= sg.eos))) return;  // nothing needs it
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const float g2 = decay2(log_decay[hv]);
  State<D> X;
  X.template load<false>(nullptr, 0, 0);
  int chunks = chunks_of(sg);
  // 2^-150 is the first power that rounds to zero
  if (g2 < 0.f) chunks = min(chunks, (int)fminf(150.f / (-g2 * kChunk), 1e6f) + 2);
  const Lane<D> L(lane, wave);
  RowRegs<D, NT> rb, rc;
  const uint16_t *bp = head_of<D>(b, hv), *cp = head_of<D>(c, hv);
  const int gb = (int)b.stride, gc = (int)c.stride;
  const int lb = rb.lane_byte(gb, tid), lc = rc.lane_byte(gc, tid);
  const int all = chunks_of(sg);
  auto start = [&](int i) { return sg.t0 + (kBack ? i : all - 1 - i) * kChunk; };
  auto request = [&](int i) {
    const int t0 = start(i), len = min(kChunk, sg.t1 - t0);
    const __amdgpu_buffer_rsrc_t nb = chunk_rows<D>(bp, gb, t0, len), nc = chunk_rows<D>(cp, gc, t0, len);
#pragma unroll
    for (int j = 0; j < RowRegs<D, NT>::kPieces; ++j) {
      rb.load(j, nb, lb, rb.kRows * gb * 2);
      rc.load(j, nc, lc, rc.kRows * gc * 2);
    }
  };
  if (chunks > 0) request(0);
  for (int i = 0; i < chunks; ++i) {
    lds_barrier();
    rb.store(Bs, tid);
    rc.store(Cs, tid);
    if (tid < kChunk) {
      const int t = start(i) + tid;
      ws[tid] = t >= sg.t1 ? 0.f : kBack ? scale * power(g2, t - sg.t0 + 1) : power(g2, sg.t1 - 1 - t);
    }
    lds_barrier();
    if (i + 1 < chunks) request(i + 1);
    uint4 cc[4];
    load_columns<D>(cc, Cs, L);
    gather_chunk<D, 3>(X, Bs, cc, ws, L, lane >> 5);
  }
  X.template store<false>(states + ((size_t)sg.slot * cut.HV + hv) * (D * D), 32 * wave + (lane & 31), lane >> 5);
}

template <int D, bool kBack>
__global__ __launch_bounds__(2 * D, 2) void lin_gather_kernel(LinCut cut, const float* __restrict__ log_decay,
                                                              float scale, LinRows b, LinRows c, bool ends,
                                                              float* __restrict__ states) {
  __shared__ __align__(16) PassLds<D> lds;
  const Item it = item_of(cut, blockIdx.x, 1);
  if (it.seg >= 0) lin_gather<D, kBack>(cut, it.seg, it.hv, log_decay, scale, b, c, ends, states, lds);
}

// The three gradients' passes in one launch (see item_of): the rows that dv's and
// dk's passes both walk come from the L2 the second time.
template <int D, bool kWide>
__global__ __launch_bounds__(2 * D, 2) void lin_grad_kernel(LinCut cut, const float* __restrict__ log_decay,
                                                            float scale, LinPass dq, LinPass dv, LinPass dk) {
  __shared__ __align__(16) PassLds<D> lds;
  const Item it = item_of(cut, blockIdx.x, 3);
  if (it.seg < 0) return;
  const int hv = it.hv, part = it.part;
  const Segment sg = find_segment(cut, it.seg);
  if (unused(sg)) return;
  if (part == 1) lin_pass<D, true, true, kWide, false>(cut, hv, sg, log_decay, scale, dk, lds);
  else if (part == 2) lin_pass<D, false, true, kWide, false>(cut, hv, sg, log_decay, scale, dq, lds);
  else if (whole(sg)) lin_pass<D, true, false, false, true>(cut, hv, sg, log_decay, scale, dv, lds);
  else lin_pass<D, true, false, false, false>(cut, hv, sg, log_decay, scale, dv, lds);
}

// Front to back along each sequence's segments (or back to front): a thread
// carries 4 values of one state, and leaves the end of a sequence of several
// segments where io says. 512 segment states, read and written: 14 us, 5 TB/s. (16
// segments requested together serialised the loads: slower.)
template <int D, bool kBack>
__global__ __launch_bounds__(64) void lin_join_kernel(LinCut cut, const float* __restrict__ log_decay, StateRef io,
                                                       float* __restrict__ states) {
  constexpr int kBlocks = D * D / 256;
  const int piece = blockIdx.x % kBlocks, hv = blockIdx.x / kBlocks % cut.HV;
  const int seq = blockIdx.x / (kBlocks * cut.HV);
  const int bos = min(max(cut.cu[seq], 0), cut.T), eos = min(max(cut.cu[seq + 1], bos), cut.T);
  const int first = bos / cut.S + seq;
  const int n = max((eos - bos + cut.S - 1) / cut.S, 1);
  const int e = piece * 256 + threadIdx.x * 4;
  const StateAt state = state_at(io, seq, hv, cut.HV, D * D);
  const float g2 = decay2(log_decay[hv]);
  f32x4 x = zero4();
  if (state.from) x = *reinterpret_cast<const f32x4*>(state.from + e);
  const int m = n == 1 ? 0 : state.to ? n : n - 1;  // segments whose sums are there
  auto place = [&](int i) { return states + ((size_t)(first + (kBack ? n - 1 - i : i)) * cut.HV + hv) * (D * D) + e; };
  constexpr int kAhead = 8;  // segments requested together
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    f32x4 add[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      add[j] = zero4();
      if (i0 + j < m) add[j] = *reinterpret_cast<const f32x4*>(place(i0 + j));
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j, s = kBack ? n - 1 - i : i;
      if (i < n) {
        *reinterpret_cast<f32x4*>(place(i)) = x;
        const float d = power(g2, min(cut.S, eos - bos - s * cut.S));
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = d * x[r] + add[j][r];
      }
    }
  }
  if (n > 1 && state.to) *reinterpret_cast<f32x4*>(state.to + e) = x;
}

// out[t][h] = sum over the key head's G value heads of wide[t][h G + i], for
// dq and dk (blockIdx.y). Bound by HBM: 16384 tokens, 16 key and 32 value heads, 127
// us, 5.3 TB/s. The value heads' parts are fp32: rounding each to bf16 would add an
// error of the size of the result's own.
__global__ __launch_bounds__(256) void lin_fold_kernel(LinCut cut, int DH, int D,
                                                       const float* __restrict__ wq, const float* __restrict__ wk,
                                                       uint16_t* __restrict__ dq, uint16_t* __restrict__ dk) {
  const float* wide = blockIdx.y ? wk : wq;
  uint16_t* out = blockIdx.y ? dk : dq;
  const int G = cut.G;
  // pieces of 4 outputs; DH = H * D outputs a token. Rows of no sequence have no parts and stay as they were.
  const int64_t n = (int64_t)min(max(cut.cu[cut.N], 0), cut.T) * DH / 4;
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

// D = 128 or 64, and a flag that is a template argument
#define LIN_LAUNCH1(kernel, f, grid, ...)                                                                \
  do {                                                                                                   \
    const dim3 lin_grid(grid), lin_block(2 * D);                                                         \
    if (D == 128 && (f)) hipLaunchKernelGGL((kernel<128, true>), lin_grid, lin_block, 0, s, __VA_ARGS__);  \
    else if (D == 128) hipLaunchKernelGGL((kernel<128, false>), lin_grid, lin_block, 0, s, __VA_ARGS__);   \
    else if (f) hipLaunchKernelGGL((kernel<64, true>), lin_grid, lin_block, 0, s, __VA_ARGS__);            \
    else hipLaunchKernelGGL((kernel<64, false>), lin_grid, lin_block, 0, s, __VA_ARGS__);                  \
  } while (0)

hipError_t launch_lin_out(int D, const LinCut& cut, const float* log_decay, float scale, const LinPass& p,
                          hipStream_t s) {
  const dim3 grid(items_grid(cut, 1)), block(2 * D);
  if (D == 128)
    hipLaunchKernelGGL((lin_out_kernel<128>), grid, block, 0, s, cut, log_decay, scale, p);
  else
    hipLaunchKernelGGL((lin_out_kernel<64>), grid, block, 0, s, cut, log_decay, scale, p);
  return hipGetLastError();
}

hipError_t launch_lin_grad(int D, bool wide, const LinCut& cut, const float* log_decay, float scale,
                           const LinPass& dq, const LinPass& dv, const LinPass& dk, hipStream_t s) {
  LIN_LAUNCH1(lin_grad_kernel, wide, items_grid(cut, 3), cut, log_decay, scale,
              dq, dv, dk);
  return hipGetLastError();
}

hipError_t launch_lin_gather(int D, bool back, const LinCut& cut, const float* log_decay, float scale,
                             const LinRows& b, const LinRows& c, bool ends, float* states, hipStream_t s) {
  LIN_LAUNCH1(lin_gather_kernel, back, items_grid(cut, 1), cut, log_decay, scale, b, c, ends,
              states);
  return hipGetLastError();
}

hipError_t launch_lin_join(int D, bool back, const LinCut& cut, const float* log_decay, const StateRef& io,
                           float* states, hipStream_t s) {
  const dim3 grid((unsigned)cut.N * (unsigned)cut.HV * (unsigned)(D * D / 256)), block(64);
  if (D == 128 && back)
    hipLaunchKernelGGL((lin_join_kernel<128, true>), grid, block, 0, s, cut, log_decay, io, states);
  else if (D == 128)
    hipLaunchKernelGGL((lin_join_kernel<128, false>), grid, block, 0, s, cut, log_decay, io, states);
  else if (back)
    hipLaunchKernelGGL((lin_join_kernel<64, true>), grid, block, 0, s, cut, log_decay, io, states);
  else
    hipLaunchKernelGGL((lin_join_kernel<64, false>), grid, block, 0, s, cut, log_decay, io, states);
  return hipGetLastError();
}

hipError_t launch_lin_fold(int D, const LinCut& cut, const float* wq, const float* wk, uint16_t* dq, uint16_t* dk,
                           hipStream_t s) {
  const int DH = cut.HV / cut.G * D;
  const int64_t n = (int64_t)cut.T * DH / 4;
  const unsigned blocks = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
  hipLaunchKernelGGL(lin_fold_kernel, dim3(blocks, 2), dim3(256), 0, s, cut, DH, D, wq, wk, dq, dk);
  return hipGetLastError();
}

}  // namespace gdn
