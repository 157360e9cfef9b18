// decay.cuh -- what the kernels of linear attention with a decay share: powers of
// a head's decay, the cut of a sequence into segments, and their workspace.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"

namespace fmca {
namespace {

// log2 of a head's decay, as a sum of two floats: the exponent of a far position is a
// product with up to 2^31.  (64-bit arithmetic, whose pipe is a trickle here, costs a
// block that forms powers microseconds.)  A log decay of -inf (nothing is kept) becomes one
// whose first power is 0 already, and one of +inf one whose first power overflows, so that the
// power 0 is 1 and not a NaN.
struct DecayRate {
  float hi, lo;
};
__device__ __forceinline__ DecayRate decay_rate(float log_decay) {
  const float x = log_decay < -1e6f ? -1e6f : log_decay > 1e6f ? 1e6f : log_decay;  // (or NaN)
  constexpr float kHi = 1.44269502162933349609f, kLo = 1.92596299112661746887e-8f;  // log2(e)
  DecayRate r;
  r.hi = x * kHi;
  r.lo = fmaf(x, kLo, fmaf(x, kHi, -r.hi));
  return r;
}
// 2^(rate n), n >= 0: the exponent's rounding goes back in as a factor (not into an infinity,
// which would become a NaN; a power overflows from a finite exponent on, 128).
__device__ __forceinline__ float decay_power(const DecayRate &r, int n) {
  const float a = (float)(n & ~4095), b = (float)(n & 4095);  // exactly
  const float pa = a * r.hi, pb = b * r.hi;
  const float e = pa + pb, back = e - pa;
  const float rest = (pa - (e - back)) + (pb - back) + fmaf(a, r.hi, -pa) + fmaf(b, r.hi, -pb) +
                     (float)n * r.lo;
  const float p = exp2f(e);
  return isinf(p) ? p : fmaf(p, rest * 0.693147180559945f, p);
}
// The same as a sum of two floats, n up to 128: a state is multiplied by one power once a
// chunk, and a factor in 32 bits would be off by half a step in every one of them.  2^x = 2^k
// (1 + m), 1 + m = exp(t)^32 with |t| <= ln(2) / 64: t and m in two floats each, m = t + t^2 / 2
// + ..., and five times m = 2 m + m^2.  Off by under 2^-30 of itself times the exponent (of e),
// so that all the chunks of which a state still holds something add up to less than one
// rounding.  (A double exp2
// takes its warp a microsecond, and a block's first barrier waits for it.)
__device__ __forceinline__ float2 decay_power2(const DecayRate &r, int n) {
  const float fn = (float)n, x = fn * r.hi, x_rest = fmaf(fn, r.hi, -x) + fn * r.lo;
  if (!(x > -200.f && x < 128.f)) return make_float2(x < 0.f ? 0.f : exp2f(x), 0.f);
  const float k = rintf(x), g = x - k;  // exactly
  constexpr float kHi = 0.693147182464599609f / 32, kLo = -1.90465429995776804e-9f / 32;  // ln(2)
  const float t = g * kHi, t_rest = fmaf(g, kHi, -t) + fmaf(g, kLo, x_rest * kHi);
  const float q = fmaf(t * t, fmaf(t, fmaf(t, 1.f / 24, 1.f / 6), 0.5f), fmaf(t, t_rest, t_rest));
  float m = t + q, low = q - (m - t);
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const float sq = m * m, sq_rest = fmaf(m, m, -sq) + 2.f * m * low;
    const float h = 2.f * m + sq;
    low = (sq - (h - 2.f * m)) + (2.f * low + sq_rest);
    m = h;
  }
  const float h = 1.f + m, l = (m - (h - 1.f)) + low;
  const float hi = h + l, lo = l - (hi - h);
  return make_float2(ldexpf(hi, (int)k), ldexpf(lo, (int)k));
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

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Whether a head grows so much over a sequence that the chunked form does not hold: it
// multiplies by powers of up to the sequence's length, and one that leaves the range makes a NaN
// of a state, key or score of 0 and an infinity of a small one, where the recurrence, whose
// factors come one at a time, is finite.  Up to 2^100 the operands have 2^28 of room, and behind
// it speed is not what counts: 2 x 8192 tokens of 12 heads of 128 take 36 ms a token at a time,
// and 80 us in chunks.
__device__ __forceinline__ bool decay_grows(const DecayRate &r, int len) {
  return r.hi * (float)len > 100.f;
}
// The recurrence itself, for such a head: a whole sequence's unit by one block of NT threads, W
// columns of v, from state_in to state_out, with zeros behind the end.  The state lies in shared
// memory, sm: [dk][W], behind it the NT threads' sums of two tokens.  A thread has a column and
// every NT / W-th row, the rows' sums are joined in a fixed order.
template <typename T, int NT, int W>
__device__ __noinline__ void decay_tokens(const DecayArgs &a, int b, int h, int vt, int len,
                                          float lam, float *sm) {
  constexpr int RG = NT / W, U = NT > 256 ? 4 : 2;  // (more cost the callers registers)
  static_assert(NT % W == 0, "whole columns");
  const int tid = threadIdx.x, c = tid % W, r0 = tid / W, col = vt * W + c;
  const bool in = col < a.dv;
  float *const st = sm + c, *part = sm + a.dk * W + c, *next = part + NT;
  const size_t at = ((size_t)b * a.H + h) * a.dk * (size_t)a.dv + col;
  for (int d = r0; d < a.dk; d += RG)
    st[d * W] = in && a.state_in != nullptr ? a.state_in[at + (size_t)d * a.dv] : 0.f;
  const T *q = static_cast<const T *>(a.q) + b * a.qs[0] + (h / (a.H / a.Hq)) * a.qs[2];
  const T *k = static_cast<const T *>(a.k) + b * a.ks[0] + (h / (a.H / a.Hk)) * a.ks[2];
  const T *v = static_cast<const T *>(a.v) + b * a.vs[0] + (h / (a.H / a.Hv)) * a.vs[2] + col;
  T *o = static_cast<T *>(a.o) + ((size_t)b * a.T * a.H + h) * (size_t)a.dv + col;
  for (int t = 0; t < len; ++t, q += a.qs[1], k += a.ks[1], v += a.vs[1]) {
    const float x = in ? to_f(__ldg(v)) : 0.f;
    float sum = 0.f;
    for (int d0 = r0; d0 < a.dk; d0 += U * RG) {  // U rows' loads on their way at once
      T key[U], ask[U];
      float e[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (d0 + u * RG < a.dk) {
          key[u] = __ldg(k + d0 + u * RG), ask[u] = __ldg(q + d0 + u * RG);
          e[u] = st[(d0 + u * RG) * W];
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (d0 + u * RG < a.dk) {
          e[u] = fmaf(lam, e[u], to_f(key[u]) * x);
          st[(d0 + u * RG) * W] = e[u];
          sum = fmaf(to_f(ask[u]), e[u], sum);
        }
    }
    part[r0 * W] = sum;
    __syncthreads();
    if (r0 == 0 && in) {
      float y = 0.f;
      for (int i = 0; i < RG; ++i) y += part[i * W];
      put(o + (size_t)t * a.H * a.dv, a.scale * y);
    }
    float *const last = part;
    part = next, next = last;
  }
  if (!in) return;
  for (int t = len + r0; t < a.T; t += RG) put(o + (size_t)t * a.H * a.dv, 0.f);
  if (a.state_out != nullptr)
    for (int d = r0; d < a.dk; d += RG) a.state_out[at + (size_t)d * a.dv] = st[d * W];
}

}  // namespace
}  // namespace fmca
