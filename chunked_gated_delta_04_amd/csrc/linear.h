// Host-side declarations of the linear attention with a decay for each head.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Token rows of one operand: row t of head h starts at p + t * stride + h * D.
// Value head hv reads head hv / G.
struct LinRows {
  const uint16_t* p;
  int64_t stride;
  int G;
};

// How a pack is cut into segments that run side by side: segment i of
// sequence n covers tokens [i S, (i + 1) S) of it and has the slot
// cu[n] / S + n + i, so that a segment's place follows from cu_seqlens alone
// and T / S + N slots hold every pack. S is a multiple of the 64-token chunk.
struct LinCut {
  const int32_t* cu;
  int N, T, HV, G;  // G value heads to a key head
  int S;            // tokens per segment
  int slots;        // T / S + N
};

// One pass over the chunks of every segment, front to back or back to front:
//   out_t = sum over the pass's earlier tokens and t itself of
//           decay^|t - j| (a_t . b_j) c_j, plus a_t times the carried state X,
// where X [contracted with a][column of c] is carried with the decay and
// gathers b_j c_j^T. The four uses differ in the operands, the direction, and
// in whether X is the stored state [V][K] read along its rows or its columns.
struct LinPass {
  LinRows a, b, c;
  void* out;           // rows [T, HV, D]
  const float* start;  // [slots, HV, D, D] states that the segments start from, or null: from io
  StateRef io;         // where the sequences' states come from and a whole one's ends
};

// o: a = q, b = k, c = v, front to back.
hipError_t launch_lin_out(int D, const LinCut& cut, const float* log_decay, float scale, const LinPass& pass,
                          hipStream_t stream);
// dq: a = dO, b = v, c = k, front to back, the state's transpose; back to front
// dv: a = k, b = q, c = dO and dk: a = v, b = dO, c = q, the state's transpose.
// wide: dq's and dk's rows are fp32 rows of every value head.
hipError_t launch_lin_grad(int D, bool wide, const LinCut& cut, const float* log_decay, float scale,
                           const LinPass& dq, const LinPass& dv, const LinPass& dk, hipStream_t stream);
// What each segment of a sequence of several adds to the state that it carries
// on, from a zero start: front to back from b = k and c = v, back to front from
// b = q and c = dO. ends: the last one's too (back to front, the first one's).
hipError_t launch_lin_gather(int D, bool back, const LinCut& cut, const float* log_decay, float scale,
                             const LinRows& b, const LinRows& c, bool ends, float* states, hipStream_t stream);
// In place: what the segments add -> the states that the segments start from,
// each sequence's start state from io; and, to io, the end state of a sequence of
// several segments (a whole one's is its pass's). io's may be null.
hipError_t launch_lin_join(int D, bool back, const LinCut& cut, const float* log_decay, const StateRef& io,
                           float* states, hipStream_t stream);

// dq[t][h] = sum over the key head's G value heads of wq[t][h G + i], to bf16; dk likewise.
hipError_t launch_lin_fold(int D, const LinCut& cut, const float* wq, const float* wk, uint16_t* dq, uint16_t* dk,
                           hipStream_t s);

hipError_t launch_lin_step(int D, int N, int HV, float scale, const LinRows& q, const LinRows& k,
                           const LinRows& v, const float* log_decay, float* pool, int slots,
                           const int32_t* idx, uint16_t* o, hipStream_t stream);

}  // namespace gdn
