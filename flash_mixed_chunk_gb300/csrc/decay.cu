// decay.cu -- linear attention with a decay for each head, on the CUDA cores:
//
//   S_t = lam S_{t-1} + k_t^T v_t,   o_t = scale q_t S_t,   lam = exp(log_decay)
//
// decay_step runs one token of every sequence (the recurrence itself); decay_prompt
// whole prompts in the chunked form, for 32-bit operands and for the sizes and
// strides that the tensor-core kernel (tc_decay.cuh) does not take:
//
//   o_i = scale (sum_{j <= i} lam^(i-j) (q_i k_j) v_j + lam^(i+1) q_i S)   rows of a chunk
//   S   = lam^n S + sum_j lam^(n-1-j) k_j^T v_j                            its n tokens
//
// Every power has an exponent >= 0, so that a strong decay underflows and never
// overflows.  A sequence is cut into segments where there are fewer heads than SMs:
// a first launch forms what each segment adds to the state, a second one starts
// every segment from the sum of those before it.
//
// All kernels are programmatic dependents of what runs ahead of them on the stream
// and wait for it before they read or write.
//
// Measured: fp32 prompts of 3 x 777 tokens, 6 heads of 37 x 75, 50 us, 8 x 1024 of 12 heads of 64
// 150 us (16 TFLOP/s, of about 70).  Bound by the chunks' chain of barriers and trips to shared
// memory (100 tokens, four chunks in two launches: 21.5 us): an SM issues in under half of its
// cycles with up to 24 warps, 40 % of them products.  32 tokens a chunk: the weights' share
// of the work stays under the state's from dk 32 on.  A step of 64 sequences of 12 heads of 128
// takes 16.5 us, 101 MB at 6.1 TB/s (91 % of a copy's rate); one sequence's 2.1 us on the
// device, a launch and three trips to memory.
#include <cuda_runtime.h>

#include <cstdint>

#include "decay.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace fmca {
namespace {

constexpr int kThreads = 256;
constexpr int C = 32;         // tokens of a chunk
constexpr int DVT = 64;       // columns of v of a unit
constexpr int VS = DVT + 4;   // row of the v tile in shared memory

// ------------------------------------------------------------------- prompts

constexpr int WS = C + 4;  // row of the weights
static_assert(C == 32 && VS == 68 && WS == 36, "decay_floats counts these");
static_assert(decay_floats(1) >= 4 * DVT + 2 * kThreads, "decay_tokens' state and sums");
__device__ __forceinline__ float4 &at4(float *p) { return *reinterpret_cast<float4 *>(p); }
__device__ __forceinline__ void fma4(float x, const float4 &y, float4 &z) {
  z.x = fmaf(x, y.x, z.x), z.y = fmaf(x, y.y, z.y);
  z.z = fmaf(x, y.z, z.z), z.w = fmaf(x, y.w, z.w);
}

// A block is one unit.  LOCAL: what segments 0 .. S-2 add to the state, into
// slots 1 .. S-1 of the workspace (segment 0 starts from the carried state, a copy
// of which goes to slot 0: the second launch may overwrite it in place).
template <typename T, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 3)
    decay_prompt(const __grid_constant__ DecayArgs a, const DecaySplit sp,
                 float *__restrict__ slots) {
  extern __shared__ float4 smem4[];
  float *sm = reinterpret_cast<float *>(smem4);
  const int dk = a.dk, dkp = decay_dk4(dk), ks = decay_row(dk);
  // q, k, k with its weights in the state, v, the state, the chunk's weights, the powers
  float *sq = sm, *sk = sq + C * ks, *kw = sk + C * ks, *sv = kw + C * ks, *st = sv + C * VS;
  float *sw = st + dkp * DVT, *pw = sw + C * WS;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;

  griddep_wait();
  griddep_launch_dependents();
  const int segs = LOCAL ? sp.S - 1 : sp.S;
  const DecayUnit w = decay_unit(a, sp, segs, blockIdx.x);
  const int v0 = w.vt * DVT, nv = a.dv - v0 < DVT ? a.dv - v0 : DVT;
  const size_t slot = (size_t)dk * DVT;
  float *own = slots + (((size_t)w.b * a.H + w.h) * sp.nvt + w.vt) * sp.S * slot;
  const DecayRate rate = decay_rate(a.log_decay[w.h]);
  if (decay_grows(rate, w.len)) {
    if (!LOCAL && w.s == 0)
      decay_tokens<T, kThreads, DVT>(a, w.b, w.h, w.vt, w.len, decay_power(rate, 1), sm);
    return;
  }
  if (tid <= C) pw[tid] = decay_power(rate, tid);
  __shared__ float2 whole;
  __shared__ float from[64];  // the segments' powers at this one's start
  if (!LOCAL && tid >= 128 && tid - 128 <= w.s)
    from[tid - 128] = decay_power(rate, w.t0 - (tid - 128) * sp.L);
  if (tid == 64) whole = decay_power2(rate, C);  // (read behind the first chunk's barriers)

  // the state at the segment's start
  const size_t at = ((size_t)w.b * a.H + w.h) * dk * (size_t)a.dv + v0;
  __syncthreads();
  const int warp = tid / 32, lane = tid % 32;
  if (sp.S == 1 || (LOCAL && w.s == 0)) {
#pragma unroll 4
    for (int i = tid; i < dkp * DVT; i += kThreads) {
      const int d = i / DVT, c = i % DVT;
      const bool in = a.state_in != nullptr && d < dk && c < nv;
      const float x = in ? a.state_in[at + (size_t)d * a.dv + c] : 0.f;
      st[i] = x;
      if (LOCAL && d < dk) own[i] = x;
    }
  } else {
    // four columns a thread, the loads of several segments on their way
    const int last = !LOCAL && w.t0 < w.len ? w.s : 0;
    const size_t slot4 = slot / 4;
    for (int i = tid; i < dkp * DVT / 4; i += kThreads) {
      const float4 *const p = reinterpret_cast<const float4 *>(own) + i;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < dk * DVT / 4) {
        if (!LOCAL && w.s == 0) x = *p;
#pragma unroll 8
        for (int s = 1; s <= last; ++s) fma4(from[s], p[s * slot4], x);
      }
      at4(st + 4 * i) = x;
    }
  }
  // a segment that nothing comes behind is nobody's start
  const int end = w.t1 < w.len ? w.t1 : w.len;
  if (LOCAL && w.t1 >= w.len) return;

  const T *q = static_cast<const T *>(a.q) + w.b * a.qs[0] + (w.h / (a.H / a.Hq)) * a.qs[2];
  const T *k = static_cast<const T *>(a.k) + w.b * a.ks[0] + (w.h / (a.H / a.Hk)) * a.ks[2];
  const T *v = static_cast<const T *>(a.v) + w.b * a.vs[0] + (w.h / (a.H / a.Hv)) * a.vs[2] + v0;
  T *o = static_cast<T *>(a.o) + ((size_t)w.b * a.T * a.H + w.h) * (size_t)a.dv + v0;
  const size_t orow = (size_t)a.H * a.dv;

  for (int t = w.t0; t < end; t += C) {
    const int n = end - t < C ? end - t : C;
    __syncthreads();  // the last chunk's reads of the tiles
    // tokens behind the end are zeros, whatever the arrays hold there
    // (a warp's four rows, loads ahead of stores: one trip to memory for all of them)
    constexpr int R = C / (kThreads / 32);
    T y[2 * R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      const int r = warp + kThreads / 32 * (i % R), c = lane + 32 * (i / R);
      if (r < n && c < nv) y[i] = __ldg(v + (int64_t)(t + r) * a.vs[1] + c);
    }
#pragma unroll 2
    for (int d = lane; d < dkp; d += 32) {
      T x[2 * R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = warp + kThreads / 32 * i;
        if (r >= n || d >= dk) continue;
        if (!LOCAL) x[i] = __ldg(q + (int64_t)(t + r) * a.qs[1] + d);
        x[R + i] = __ldg(k + (int64_t)(t + r) * a.ks[1] + d);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = warp + kThreads / 32 * i;
        const bool in = r < n && d < dk;
        const float key = in ? to_f(x[R + i]) : 0.f;
        if (!LOCAL) {
          sq[r * ks + d] = in ? to_f(x[i]) : 0.f;
          sk[r * ks + d] = key;
        }
        kw[r * ks + d] = in ? key * pw[n - 1 - r] : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      const int r = warp + kThreads / 32 * (i % R), c = lane + 32 * (i / R);
      sv[r * VS + c] = r < n && c < nv ? to_f(y[i]) : 0.f;
    }
    __syncthreads();
    if (!LOCAL) {
      // rows 2 ty and 2 ty + 1, keys tx and tx + 16
      float acc[2][2] = {};
#pragma unroll 2
      for (int d = 0; d < dkp; d += 4) {
        const float4 x[2] = {at4(sq + 2 * ty * ks + d), at4(sq + (2 * ty + 1) * ks + d)};
        const float4 y[2] = {at4(sk + tx * ks + d), at4(sk + (tx + 16) * ks + d)};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y,
                        fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int gap = 2 * ty + i - (tx + 16 * j);
          sw[(2 * ty + i) * WS + tx + 16 * j] = gap >= 0 ? acc[i][j] * pw[gap] : 0.f;
        }
      __syncthreads();
      float4 near[2] = {}, far[2] = {};
#pragma unroll 2
      for (int j = 0; j <= 2 * ty + 1; j += 4) {
        const float4 x0 = at4(sw + 2 * ty * WS + j), x1 = at4(sw + (2 * ty + 1) * WS + j);
        const float *p0 = &x0.x, *p1 = &x1.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (a weight of 0 would not keep an infinity or a NaN out)
          const float4 y = at4(sv + (j + i) * VS + 4 * tx);
          if (j + i <= 2 * ty) fma4(p0[i], y, near[0]);
          if (j + i <= 2 * ty + 1) fma4(p1[i], y, near[1]);
        }
      }
#pragma unroll 2
      for (int d = 0; d < dkp; d += 4) {
        const float4 x0 = at4(sq + 2 * ty * ks + d), x1 = at4(sq + (2 * ty + 1) * ks + d);
        const float *p0 = &x0.x, *p1 = &x1.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 y = at4(st + (d + i) * DVT + 4 * tx);
          fma4(p0[i], y, far[0]);
          fma4(p1[i], y, far[1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * ty + i;
        if (r >= n) continue;
        const float *x = &near[i].x, *y = &far[i].x;
        T *row = o + (size_t)(t + r) * orow;
        for (int c = 0; c < 4; ++c)
          if (4 * tx + c < nv) put(row + 4 * tx + c, a.scale * fmaf(pw[r + 1], y[c], x[c]));
      }
    }
    if (!LOCAL) __syncthreads();  // all have read the state
    const float2 g = n == C ? whole : make_float2(pw[n], 0.f);
    // places 4 ty .. 4 ty + 3 of dk, columns 4 tx .. 4 tx + 3
    for (int d = 4 * ty; d < dkp; d += 64) {
      float4 add[4] = {};
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float4 x = at4(kw + j * ks + d), y = at4(sv + j * VS + 4 * tx);
        fma4(x.x, y, add[0]);
        fma4(x.y, y, add[1]);
        fma4(x.z, y, add[2]);
        fma4(x.w, y, add[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4 &p = at4(st + (d + i) * DVT + 4 * tx);
        const float4 s = p;
        p = make_float4(fmaf(s.x, g.x, fmaf(s.x, g.y, add[i].x)),
                        fmaf(s.y, g.x, fmaf(s.y, g.y, add[i].y)),
                        fmaf(s.z, g.x, fmaf(s.z, g.y, add[i].z)),
                        fmaf(s.w, g.x, fmaf(s.w, g.y, add[i].w)));
      }
    }
  }
  __syncthreads();
  if (LOCAL) {
    for (int i = tid; i < dk * DVT; i += kThreads) own[(w.s + 1) * slot + i] = st[i];
    return;
  }
  // outputs behind the sequence's end
  const int z0 = w.t0 > w.len ? w.t0 : w.len;
  for (int r = z0 + warp; r < w.t1; r += kThreads / 32)
    for (int c = lane; c < nv; c += 32) put(o + (size_t)r * orow + c, 0.f);
  if (a.state_out != nullptr && decay_last(w, sp.L))
    for (int i = tid; i < dk * DVT; i += kThreads)
      if (i % DVT < nv) a.state_out[at + (size_t)(i / DVT) * a.dv + i % DVT] = st[i];
}

// -------------------------------------------------------------- single tokens

// A block is W = LR VEC columns of one head's state.  LR threads side by side have a
// row of them, 256 / LR rows at a time; a thread reads, scales, adds to and writes
// its places of the state, and adds q_d S_d to its columns' sums, which the rows'
// threads join in a fixed order.  Bound by the state, read once and written once; eight
// rows of a thread are on their way at once.
template <typename T, int VEC, int LR>
__global__ void __launch_bounds__(kThreads)
    decay_step(const __grid_constant__ DecayArgs a, float *__restrict__ state) {
  constexpr int W = LR * VEC, RP = kThreads / LR, U = 8;
  __shared__ float sq[kDecayMaxK], sk[kDecayMaxK];
  __shared__ float part[RP][W];
  const int nvt = (a.dv + W - 1) / W;
  const int vt = (int)(blockIdx.x % nvt);
  const int64_t bh = blockIdx.x / nvt;
  const int h = (int)(bh % a.H);
  const int64_t b = bh / a.H;
  const int tid = threadIdx.x, rp = tid / LR, c = vt * W + (tid % LR) * VEC;
  const bool in = c < a.dv;
  using V = typename std::conditional<VEC == 4, float4, float>::type;

  griddep_wait();
  griddep_launch_dependents();
  float *p = state + (bh * a.dk) * (int64_t)a.dv + c;
  const T *q = static_cast<const T *>(a.q) + b * a.qs[0] + (h / (a.H / a.Hq)) * a.qs[2];
  const T *k = static_cast<const T *>(a.k) + b * a.ks[0] + (h / (a.H / a.Hk)) * a.ks[2];
  const T *v = static_cast<const T *>(a.v) + b * a.vs[0] + (h / (a.H / a.Hv)) * a.vs[2] + c;
  V s[U];
  // the first rows are on their way while q and k come in
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (in && rp + u * RP < a.dk)
      s[u] = *reinterpret_cast<const V *>(p + (int64_t)(rp + u * RP) * a.dv);
  if (tid < a.dk) {
    sq[tid] = to_f(q[tid]);
    sk[tid] = to_f(k[tid]);
  }
  float x[VEC], sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    x[i] = in ? to_f(v[i]) : 0.f;
    sum[i] = 0.f;
  }
  const float lam = decay_power(decay_rate(a.log_decay[h]), 1);
  __syncthreads();
  for (int r0 = rp; r0 < a.dk; r0 += U * RP) {
    if (r0 != rp) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (in && r0 + u * RP < a.dk)
          s[u] = *reinterpret_cast<const V *>(p + (int64_t)(r0 + u * RP) * a.dv);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RP;
      if (!in || r >= a.dk) continue;
      float *e = reinterpret_cast<float *>(&s[u]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        e[i] = fmaf(lam, e[i], sk[r] * x[i]);
        sum[i] = fmaf(sq[r], e[i], sum[i]);
      }
      *reinterpret_cast<V *>(p + (int64_t)r * a.dv) = s[u];
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) part[rp][(tid % LR) * VEC + i] = sum[i];
  __syncthreads();
  if (tid < W && vt * W + tid < a.dv) {
    float y = 0.f;
#pragma unroll 8
    for (int i = 0; i < RP; ++i) y += part[i][tid];
    put(static_cast<T *>(a.o) + bh * a.dv + vt * W + tid, a.scale * y);
  }
}

template <typename T>
int step(const DecayArgs &a, float *state, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  const int64_t bh = (int64_t)a.B * a.H;
  const auto blocks = [&](int W) { return bh * ((a.dv + W - 1) / W); };
  if (a.dv % 4) {
    cfg.gridDim = dim3((unsigned)blocks(32));
    return cudaLaunchKernelEx(&cfg, decay_step<T, 1, 32>, a, state) == cudaSuccess ? 0 : 1;
  }
  // 64 columns a block, two lines of every row; 32 where fewer than an SM's worth of blocks
  // would do so.  64 sequences of 12 heads of 128: 16.5 us, with 32 columns 17.9, with 128 17.3;
  // 16 sequences 5.7, 6.5, 6.2; 2 sequences (24 blocks) 2.9, with 32 2.55, with 128 3.9.
  auto *kern = decay_step<T, 4, 16>;
  int W = 64;
  if (blocks(64) < kDecaySms) kern = decay_step<T, 4, 8>, W = 32;
  cfg.gridDim = dim3((unsigned)blocks(W));
  return cudaLaunchKernelEx(&cfg, kern, a, state) == cudaSuccess ? 0 : 1;
}

template <typename T>
int prompt(const DecayArgs &a, float *slots, cudaStream_t stream) {
  const DecaySplit sp = decay_split_simt(a.B, a.T, a.H, a.dk, a.dv);
  const size_t smem = sizeof(float) * (size_t)decay_floats(a.dk);
  static OncePerDevice attrs;
  if (!attrs.run([] {
        const int most = (int)sizeof(float) * decay_floats(kDecayMaxK);
        return cudaFuncSetAttribute(decay_prompt<T, true>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    most) == cudaSuccess &&
               cudaFuncSetAttribute(decay_prompt<T, false>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    most) == cudaSuccess;
      }))
    return 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  const int64_t heads = (int64_t)a.B * a.H * sp.nvt;
  if (sp.S > 1) {
    cfg.gridDim = dim3((unsigned)(heads * (sp.S - 1)));
    if (cudaLaunchKernelEx(&cfg, decay_prompt<T, true>, a, sp, slots) != cudaSuccess) return 1;
  }
  cfg.gridDim = dim3((unsigned)(heads * sp.S));
  return cudaLaunchKernelEx(&cfg, decay_prompt<T, false>, a, sp, slots) == cudaSuccess ? 0 : 1;
}

}  // namespace

int launch_decay_simt(const DecayArgs &a, void *workspace, cudaStream_t stream) {
  float *slots = static_cast<float *>(workspace);
  return a.bf16 ? prompt<__nv_bfloat16>(a, slots, stream) : prompt<float>(a, slots, stream);
}

int launch_decay_step(const DecayArgs &a, float *state, cudaStream_t stream) {
  return a.bf16 ? step<__nv_bfloat16>(a, state, stream) : step<float>(a, state, stream);
}

}  // namespace fmca
