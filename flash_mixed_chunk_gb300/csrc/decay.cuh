// decay.cuh -- what the kernels of linear attention with a decay share: powers of
// a head's decay, the cut of a sequence into segments, and their workspace.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"

namespace fmca {
namespace {

// log2 of a head's decay.  Held in 64 bits: the exponent of a far position is a
// product with up to 2^31.  A log decay of -inf (nothing is kept) becomes one whose
// first power is 0 already, so that the power 0 is 1 and not a NaN.
__device__ __forceinline__ double decay_rate(float log_decay) {
  return (double)(log_decay < -1e6f ? -1e6f : log_decay) * 1.4426950408889634074;
}
// 2^(rate n) in 32 bits: the exponent's rounding goes back in as a factor.
__device__ __forceinline__ float decay_power(double rate, int64_t n) {
  const double e = rate * (double)n;
  const float hi = (float)e;
  const float p = exp2f(hi);
  return isinf(hi) ? p : p + p * ((float)(e - (double)hi) * 0.693147180559945f);
}
// The same as a sum of two floats: a state is multiplied by one power once a chunk,
// and a factor in 32 bits would be off by half a step in every one of them.
__device__ __forceinline__ float2 decay_power2(double rate, int n) {
  const double p = exp2(rate * (double)n);
  const float hi = (float)p;
  return make_float2(hi, isinf(hi) ? 0.f : (float)(p - (double)hi));
}

// A unit of work: one head of one sequence, a tile of dv, a segment of tokens.
struct DecayUnit {
  int b, h, vt, s;
  int t0, t1;  // the segment's tokens
  int len;     // of the sequence
};
// Units of `segs` segments each, the segments of a head next to each other.
__device__ __forceinline__ DecayUnit decay_unit(const DecayArgs &a, const DecaySplit &sp, int segs,
                                                int64_t u) {
  DecayUnit w;
  w.s = (int)(u % segs);
  u /= segs;
  w.vt = (int)(u % sp.nvt);
  u /= sp.nvt;
  w.h = (int)(u % a.H);
  w.b = (int)(u / a.H);
  w.t0 = w.s * sp.L;
  w.t1 = a.T - w.t0 < sp.L ? a.T : w.t0 + sp.L;
  w.len = a.T;
  if (a.lengths != nullptr) {
    const int32_t l = a.lengths[w.b];
    w.len = l < 0 ? 0 : l < a.T ? l : a.T;
  }
  return w;
}
// Whether this segment's unit has the sequence's last token, and with it the state
// that is returned (a sequence without tokens: its first segment's).
__device__ __forceinline__ bool decay_last(const DecayUnit &w, int L) {
  return w.s == (w.len == 0 ? 0 : (w.len - 1) / L);
}

}  // namespace
}  // namespace fmca
