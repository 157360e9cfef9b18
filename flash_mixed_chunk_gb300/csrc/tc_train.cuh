// tc_train.cuh -- the training operators on the tensor cores around the
// products of tc_tgemm: the softmax cross entropy over a vocabulary and its
// gradients, and the gradients of the GAU projections.
//
//   loss_m = log sum_v exp(z_mv) - z_m,t(m),  z = X W^T, for the rows m that
//            have a target t(m) in 0 .. V - 1
//   dX_m = g_m sum_v (p_mv - [v = t(m)]) W_v,  dW_v = sum_m g_m (p_mv - [v = t(m)]) X_m
//
// The rows with a target are copied next to each other first (vocab_gather),
// so that a row without one costs nothing in the products and whatever its X
// holds (NaN included) reaches nothing.  The number of such rows stays on the
// device; every kernel reads it there, so the calls can be captured.  Few rows
// are taken as they are (vocab_compact), a launch fewer in either direction.
//
// The forward pass keeps, per row and 128 columns (64 of a small product), the
// maximum and the sum of exp(z - maximum), 1/32 of the logits' bytes at bf16;
// vocab_reduce joins them.  The backward pass forms the logits again, a piece of the
// vocabulary at a time, as (p - onehot) g / max|g| in bf16 (the scale goes
// back in fp32 at the end, so that equal weights are not rounded), and takes
// both gradients of the piece from it in one launch.  dX adds up over the
// pieces in fp32.
#pragma once

#include "tc_tgemm.cuh"

namespace fmca {
namespace {

constexpr int kGatherThreads = 256;

__device__ __forceinline__ bool has_target(int64_t t, int V) { return t >= 0 && t < V; }

// Sum over a block of 256 threads; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int *red) {
  __syncthreads();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kGatherThreads / 32; ++i) t += red[i];
  return t;
}

struct GatherArgs {
  const __nv_bfloat16 *X;   // [M][d]
  const int64_t *target;    // [M]
  int M, V, d, per;         // rows a block
  __nv_bfloat16 *Xc;        // [M][d] compact rows
  int *idx, *tgt;           // [M] compact
  TgHeader *hdr;
  float *loss, *lse_out;    // forward: 0 for rows without a target
  const float *lse, *dloss; // backward
  float *lse_c, *g_c;       // backward, compact
  float *tops;              // backward: the blocks' largest |dloss|
  __nv_bfloat16 *dX;        // backward: rows without a target are 0
};

// Copies the rows that have a target next to each other, in order.  A block
// takes `per` rows (an even number) and counts the targets of all rows before
// its own by itself: M / 512 loads a thread from L2 instead of a pass over the
// blocks.
template <bool kBackward>
__global__ void __launch_bounds__(kGatherThreads) vocab_gather(GatherArgs a) {
  __shared__ int red[kGatherThreads / 32];
  __shared__ float redf[kGatherThreads / 32];
  __shared__ int pos_s[kGatherThreads];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t r0 = (int64_t)blockIdx.x * a.per;
  const int64_t r1 = r0 + a.per < a.M ? r0 + a.per : a.M;
  int n = 0;
  if ((reinterpret_cast<uintptr_t>(a.target) & 15u) == 0) {
#pragma unroll 8
    for (int64_t m = 2 * tid; m < r0; m += 2 * kGatherThreads) {
      const longlong2 t = *reinterpret_cast<const longlong2 *>(a.target + m);
      n += (has_target(t.x, a.V) ? 1 : 0) + (has_target(t.y, a.V) ? 1 : 0);
    }
  } else {  // labels shifted by one token
#pragma unroll 8
    for (int64_t m = tid; m < r0; m += kGatherThreads) n += has_target(a.target[m], a.V) ? 1 : 0;
  }
  int base = block_sum(n, red);
  const int nv = a.d / 8;
  float top = 0.f;
  for (int64_t m0 = r0; m0 < r1; m0 += kGatherThreads) {
    const int64_t m = m0 + tid;
    const int64_t t = m < r1 ? a.target[m] : -1;
    const bool has = has_target(t, a.V);
    const uint32_t votes = __ballot_sync(0xffffffffu, has);
    __syncthreads();
    if (lane == 0) red[warp] = __popc(votes);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kGatherThreads / 32; ++i) {
      before += i < warp ? red[i] : 0;
      all += red[i];
    }
    const int pos = base + before + __popc(votes & ((1u << lane) - 1));
    if (has) {
      a.idx[pos] = (int)m;
      a.tgt[pos] = (int)t;
      if constexpr (kBackward) {
        const float g = a.dloss[m];
        a.lse_c[pos] = a.lse[m];
        a.g_c[pos] = g;
        top = fmaxf(top, fabsf(g));
      }
    } else if (m < r1) {
      if constexpr (!kBackward) {
        a.loss[m] = 0.f;
        a.lse_out[m] = 0.f;
      }
    }
    pos_s[tid] = has ? pos : -1;
    base += all;
    __syncthreads();
    const int rows = (int)(r1 - m0 < kGatherThreads ? r1 - m0 : kGatherThreads);
    for (int r = warp; r < rows; r += kGatherThreads / 32) {
      const int p = pos_s[r];
      if (p >= 0) {
        const uint4 *src = reinterpret_cast<const uint4 *>(a.X + (m0 + r) * a.d);
        uint4 *dst = reinterpret_cast<uint4 *>(a.Xc + (int64_t)p * a.d);
        for (int v = lane; v < nv; v += 128) {  // four loads on their way at once
          uint4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (v + 32 * k < nv) x[k] = __ldg(src + v + 32 * k);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (v + 32 * k < nv) dst[v + 32 * k] = x[k];
        }
      } else if constexpr (kBackward) {
        uint4 *dst = reinterpret_cast<uint4 *>(a.dX + (m0 + r) * a.d);
        for (int v = lane; v < nv; v += 32) dst[v] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == gridDim.x - 1) {
    // the last block knows the number of rows; zero rows up to the next
    // multiple of 64 complete the products' last step over the tokens
    const int count = base;
    const int64_t end = min((int64_t)(count + 63) / 64 * 64, (int64_t)a.M);
    uint4 *dst = reinterpret_cast<uint4 *>(a.Xc);
    for (int64_t v = (int64_t)count * nv + tid; v < end * nv; v += kGatherThreads)
      dst[v] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) a.hdr->count = count;
  }
  if constexpr (kBackward) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) redf[warp] = top;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int i = 1; i < kGatherThreads / 32; ++i) top = fmaxf(top, redf[i]);
      a.tops[blockIdx.x] = top;
    }
  }
}

// loss and lse of the rows from the products' partial maxima and sums: 32
// rows a block, 32 lanes of parts each, joined in order.  The rows are compact
// (idx, hdr), or as they are (target; one without a target has loss and lse 0).
constexpr int kReduceLanes = 32;
__global__ void __launch_bounds__(32 * kReduceLanes)
    vocab_reduce(const float2 *__restrict__ part, const float *__restrict__ ztgt,
                 const int *__restrict__ idx, const TgHeader *__restrict__ hdr,
                 const int64_t *__restrict__ target, float *loss, float *lse, int parts, int M,
                 int V) {
  __shared__ float2 s[kReduceLanes][32];
  griddep_wait();
  const int count = hdr != nullptr ? hdr->count : M;
  const int r = threadIdx.x % 32, l = threadIdx.x / 32;
  const int64_t m = (int64_t)blockIdx.x * 32 + r;
  if ((int64_t)blockIdx.x * 32 >= count) return;
  // (top, sum) with sum = sum exp(z - top); (-infinity, 0) is nothing
  auto join = [](float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x), ref = top == -INFINITY ? 0.f : top;
    return make_float2(
        top, a.y * tg_exp2((a.x - ref) * kLog2e) + b.y * tg_exp2((b.x - ref) * kLog2e));
  };
  float2 t = make_float2(-INFINITY, 0.f);
  if (m < count) {
#pragma unroll 8
    for (int p = l; p < parts; p += kReduceLanes) t = join(t, __ldg(part + (int64_t)p * M + m));
  }
  s[l][r] = t;
  __syncthreads();
  if (l == 0 && m < count) {
#pragma unroll
    for (int i = 1; i < kReduceLanes; ++i) t = join(t, s[i][r]);
    const float v = t.x + logf(t.y);
    if (target == nullptr) {
      const int row = idx[m];
      lse[row] = v;
      loss[row] = v - ztgt[m];
    } else {
      const bool has = has_target(target[m], V);
      lse[m] = has ? v : 0.f;
      loss[m] = has ? v - ztgt[m] : 0.f;
    }
  }
}

// The tiles that a cut went through: the sum of their parts, rounded.  Every
// block makes the list of those tiles while the products still run (a ring of
// 6 leaves room for a block beside them), then the blocks share the tiles in
// pieces of 256 threads (a warp's loads are consecutive), the parts in order.
constexpr int kJoinThreads = 256;
static_assert(kJoinThreads > kTgMaxCtas, "a thread a cut");

// The listed tiles, COLS columns of a row a thread: list_s the first cut,
// list_a .. list_b the numbers of its parts' groups in part_s.
template <int CG, int COLS>
__device__ __forceinline__ void tg_join_tiles(const TgParams &P, const TgPlan &plan,
                                              const int *list_s, const int *list_a,
                                              const int *list_b, const int *part_s, int list_n,
                                              float alpha) {
  constexpr int kAcross = 256 / COLS, kPieces = 128 * kAcross * CG / kJoinThreads;
  const int tasks = list_n * plan.side * kPieces;
  for (int task = (int)blockIdx.x; task < tasks; task += (int)gridDim.x) {
    const int lane = task / kPieces % plan.side, item = task / (kPieces * plan.side);
    const int first = list_s[item], n1 = list_b[item];
    const TgCut f = tg_cut(plan, first, plan.groups);
    const TgShape &h = plan.s[f.pi];
    const int across = h.Nt / plan.side, panel = f.tile + h.dealt;
    const int mt = panel / across, nt = (panel - mt * across) * plan.side + lane;
    const int t = task % kPieces * kJoinThreads + (int)threadIdx.x;
    const int row = t % 128, q = t / 128 % kAcross, rank = t / (128 * kAcross);
    const int m = (mt * CG + rank) * 128 + row, col = nt * 256 + q * COLS;
    if (m >= h.M || col >= P.K) continue;
    float v[COLS];
#pragma unroll
    for (int k = 0; k < COLS; ++k) v[k] = 0.f;
#pragma unroll(COLS == 4 ? 16 : 4)
    for (int n = list_a[item]; n < n1; ++n) {
      const int x = part_s[n];
      // the tile's first part is the last one of its worker, the others first
      const float *slot =
          P.slots +
          (int64_t)tg_part(x * plan.side + lane, x >= first, CG, rank) * kTgSlotFloats;
#pragma unroll
      for (int j = 0; j < COLS / 4; ++j) {
        const float4 o = *reinterpret_cast<const float4 *>(
            slot + tg_slot_offset(row, q * (COLS / 4) + j));
        v[4 * j] += o.x, v[4 * j + 1] += o.y, v[4 * j + 2] += o.z, v[4 * j + 3] += o.w;
      }
    }
    __nv_bfloat16 *out = f.pi ? P.D1 + (int64_t)(P.idx != nullptr ? P.idx[m] : m) * P.K
                              : P.D0 + (int64_t)(plan.col0 + m) * P.K;
    uint32_t o[COLS / 2];
    const bool live = f.pi == 0 || P.keep == nullptr || P.keep[m] != 0;
#pragma unroll
    for (int k = 0; k < COLS / 2; ++k)
      o[k] = live ? pack_bf16x2(alpha * v[2 * k], alpha * v[2 * k + 1]) : 0u;
    if constexpr (COLS == 4) {
      *reinterpret_cast<uint2 *>(out + col) = make_uint2(o[0], o[1]);
    } else {
      *reinterpret_cast<uint4 *>(out + col) = make_uint4(o[0], o[1], o[2], o[3]);
      if (col + 8 < P.K)
        *reinterpret_cast<uint4 *>(out + col + 8) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <int CG>
__global__ void __launch_bounds__(kJoinThreads)
    tg_join(const __grid_constant__ TgParams P, int workers, int last) {
  __shared__ TgPlan plan;
  __shared__ int cut_s[kTgMaxCtas + 1];        // where the groups' parts begin
  __shared__ int part_s[kTgMaxCtas + 1];                // groups that have a part
  __shared__ int2 warp_s[kJoinThreads / 32];
  __shared__ int list_s[kTgMaxCtas], list_a[kTgMaxCtas], list_b[kTgMaxCtas], list_n;
  // launched by a TG_GRAD that had waited for what wrote the header
  if (P.hdr != nullptr && P.piece > 0 && last == 0 &&
      P.piece >= tg_pieces(tg_count(P.hdr), P.N, P.cap_boxes).np) {
    griddep_wait();
    return;
  }
  if (threadIdx.x == 0)
    plan = tg_plan<CG, TG_GRAD>(P, P.piece, P.hdr != nullptr ? tg_count(P.hdr) : P.M, workers);
  __syncthreads();
  const int groups = plan.groups, w = (int)threadIdx.x;
  TgCut c = {};
  if (w <= groups) {
    c = tg_cut(plan, w, groups);
    cut_s[w] = c.pos;
  }
  __syncthreads();
  // the groups that have a part, and the cuts that are a panel's first, each
  // numbered in order (the same in every block)
  const bool has = w < groups && cut_s[w + 1] > cut_s[w];
  const bool first_cut =
      w > 0 && w < groups && tg_first_cut(plan, c, cut_s[w - 1], last != 0);
  const uint32_t votes = __ballot_sync(0xffffffffu, has);
  const uint32_t votes2 = __ballot_sync(0xffffffffu, first_cut);
  const uint32_t below = (1u << (w % 32)) - 1;
  if (w % 32 == 0) warp_s[w / 32] = make_int2(__popc(votes), __popc(votes2));
  __syncthreads();
  int at = __popc(votes & below), item_at = __popc(votes2 & below);
  for (int i = 0; i < w / 32; ++i) at += warp_s[i].x, item_at += warp_s[i].y;
  if (has || w == groups) part_s[at] = w;  // (groups: the end)
  if (w == groups) list_n = item_at;
  __syncthreads();
  if (first_cut) {
    const int end = c.pos - c.off + plan.s[c.pi].len;
    int b = at;
    while (part_s[b] < groups && cut_s[part_s[b]] < end) ++b;
    list_s[item_at] = w;
    list_a[item_at] = at - 1;  // the group before the cut
    list_b[item_at] = b;
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const float alpha = P.gmax != nullptr ? *P.gmax : 1.f;
  // 16 columns a thread; of few tiles (each of many parts) 4, so that the
  // parts are read at the same time
  if (list_n * plan.side > 4)
    tg_join_tiles<CG, 16>(P, plan, list_s, list_a, list_b, part_s, list_n, alpha);
  else
    tg_join_tiles<CG, 4>(P, plan, list_s, list_a, list_b, part_s, list_n, alpha);
}

// ---------------------------------------------------------------- host side
// Launch configuration of one tc_tgemm (its attributes live in the object).
template <int CG, int KIND, int NT>
struct TgLaunch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  TgLaunch(int workers, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3(workers * CG);
    cfg.blockDim = dim3(TG_THREADS);
    cfg.dynamicSmemBytes = TgCfg<CG, KIND, NT>::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
  }
};

// CTAs (or pairs) that the current device holds at once, 0 on an error.  Pairs
// sit within a group of SMs, so there can be fewer than half the SMs: the
// units are dealt to the workers beforehand, and one that had to wait for
// another to leave would double the time.
template <int CG, int KIND, int NT>
int tg_resident() {
  static OncePerDevice once;
  static int resident[OncePerDevice::kMaxDevices];
  int dev = 0;
  if (!once.run([] {
        int d = 0, n = 0;
        if (cudaGetDevice(&d) != cudaSuccess ||
            cudaFuncSetAttribute(tc_tgemm<CG, KIND, NT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)TgCfg<CG, KIND, NT>::SMEM) != cudaSuccess)
          return false;
        n = num_sms() / CG;
        if (CG == 2) {
          TgLaunch<CG, KIND, NT> l(n, nullptr);
          l.cfg.attrs = &l.attr[1];
          l.cfg.numAttrs = 1;
          int fit = 0;
          if (cudaOccupancyMaxActiveClusters(&fit, tc_tgemm<CG, KIND, NT>, &l.cfg) != cudaSuccess)
            return false;
          if (fit < n) n = fit;
        }
        if (n * CG > kTgMaxCtas) n = kTgMaxCtas / CG;
        resident[d] = n;
        return n > 0;
      }) ||
      cudaGetDevice(&dev) != cudaSuccess)
    return 0;
  return resident[dev];
}

template <int CG, int KIND, int NT>
int launch_tgemm_kind(const TgParams &P, int workers, cudaStream_t stream) {
  TgLaunch<CG, KIND, NT> l(workers, stream);
  return cudaLaunchKernelEx(&l.cfg, tc_tgemm<CG, KIND, NT>, P) == cudaSuccess ? 0 : 1;
}

// Workers of a launch: all that are resident at once, no more than there are
// units (parts of 8 k steps) with every row taking part.
template <int CG, int KIND, int NT>
int tg_workers(const TgParams &P) {
  int w = tg_resident<CG, KIND, NT>();
  if (w > 0) {
    const TgPlan p = tg_plan<CG, KIND, NT>(P, P.piece, P.M, w);
    int64_t units = p.s[0].tiles;
    if (KIND == TG_GRAD) {
      units = 0;
      for (const TgShape &h : p.s) units += (int64_t)h.tiles * (h.ks < 16 ? 1 : h.ks / 8);
    }
    if (units < w) w = (int)units;
  }
  return w;
}
template <int CG, int KIND, int NT = 256>
int launch_tgemm(const TgParams &P, cudaStream_t stream) {
  const int w = tg_workers<CG, KIND, NT>(P);
  return w > 0 ? launch_tgemm_kind<CG, KIND, NT>(P, w, stream) : 1;
}

// Whether a product with its tokens as rows goes in 128 x 128 tiles: while those
// fit on the CTAs at once.  A tile's k steps and epilogue take half the time
// then: projection gradients of 1001 x 520, e 448, s 64 16.7 us (CTA pairs
// 21.2), the loss's gradients of 88 x 164 x 560 13.5 (19.3).
template <int KIND>
bool tg_small(int M, int N) {
  return tg_small_tiles(M, N) <= tg_resident<1, KIND, 128>();
}
template <int CG, int KIND>
int launch_nt(const TgParams &P, bool small, cudaStream_t stream) {
  return small ? launch_tgemm<1, KIND, 128>(P, stream) : launch_tgemm<CG, KIND>(P, stream);
}

// Whether the gradients of a single piece, not cut in any case (plan), go in
// 128 x 128 tiles: while those fit on the CTAs at once.  A tile's k steps and
// epilogue take half the time then.
bool tg_small_grad(const TgParams &P, const TgPlan &plan) {
  const int r = tg_resident<1, TG_GRAD, 128>();
  if (P.hdr != nullptr || r <= 0 || !plan.apart || plan.s[0].dealt + plan.s[1].dealt > 0)
    return false;
  const TgPlan p = tg_plan<1, TG_GRAD, 128>(P, 0, P.M, r);
  return (int64_t)p.s[0].tiles + p.s[1].tiles <= r;
}

// TG_GRAD on piece P.piece of np, and the sums of the tiles that were cut.
// Without a device count the cuts are known here, and there may be none.
template <int CG>
int launch_grad(const TgParams &P, int np, cudaStream_t stream) {
  const int w = tg_workers<CG, TG_GRAD, 256>(P);
  if (w <= 0) return 1;
  const TgPlan p = tg_plan<CG, TG_GRAD>(P, P.piece, P.M, w);
  if (np == 1 && tg_small_grad(P, p)) return launch_tgemm<1, TG_GRAD, 128>(P, stream);
  if (launch_tgemm_kind<CG, TG_GRAD, 256>(P, w, stream)) return 1;
  bool join = P.hdr != nullptr;  // the cuts are not known here
  for (int x = 1; x < p.groups && !join; ++x) join = tg_cut(p, x, p.groups).off != 0;
  if (!join || w < 2) return 0;
  return launch_dependent(tg_join<CG>, 3 * kTgMaxCtas, kJoinThreads, 0, stream, P, w,
                          P.piece == np - 1 ? 1 : 0) == cudaSuccess
             ? 0
             : 1;
}

// Whether the vocabulary loss makes its rows compact.  Not up to 128 rows (one
// tile in any case), nor up to 512 while all of them cost less in the products
// (8 GFLOP, 5 us) than the launch that would sort them out: 455 rows against
// 2245 x 680 take 35.4 us forward and backward as they are, 40.7 compact.
bool vocab_compact(int M, int V, int d) {
  return M > 512 || (M > 128 && 2.0 * M * V * d > 8e9);
}

// CTA pairs for more rows than one CTA's tile has; up to 128 rows (a short
// fine-tuning batch, a few tokens) half of a pair's tile would stay empty.
bool tg_pairs(int M) { return M > 128; }

// X [M][K] and W [N][K] of the products with tokens as rows
template <int CG>
bool nt_maps(TgParams &P, const void *X, const void *W, int M, int N, int K, bool small) {
  return make_map_bf16(&P.A, X, K, M, 64, 128) &&
         make_map_bf16(&P.B, W, K, N, 64, small ? 128 : 256 / CG);
}

template <int CG>
int vocab_loss_cg(const void *X, const void *W, const int64_t *target, float *loss, float *lse,
                      int M, int V, int d, void *workspace, cudaStream_t stream) {
  const VocabLossLayout L = vocab_loss_layout(M, V, d);
  char *ws = static_cast<char *>(workspace);
  GatherArgs a = {};
  a.X = static_cast<const __nv_bfloat16 *>(X);
  a.target = target;
  a.M = M, a.V = V, a.d = d;
  a.Xc = reinterpret_cast<__nv_bfloat16 *>(ws + L.Xc);
  a.idx = reinterpret_cast<int *>(ws + L.idx);
  a.tgt = reinterpret_cast<int *>(ws + L.tgt);
  a.hdr = reinterpret_cast<TgHeader *>(ws + L.hdr);
  a.loss = loss, a.lse_out = lse;
  const bool compact = vocab_compact(M, V, d);
  if (compact) {
    const int blocks = M < kTgMaxCtas * 2 ? M : kTgMaxCtas * 2;
    a.per = ((M + blocks - 1) / blocks + 1) / 2 * 2;
    if (launch_dependent(vocab_gather<false>, (M + a.per - 1) / a.per, kGatherThreads, 0, stream,
                         a) != cudaSuccess)
      return 1;
  }

  TgParams P = {};
  const bool small = tg_small<TG_LSE>(M, V);
  if (!nt_maps<CG>(P, compact ? a.Xc : a.X, W, M, V, d, small)) return 2;
  P.M = M, P.N = V, P.K = d;
  P.hdr = compact ? a.hdr : nullptr;
  P.target = compact ? nullptr : target;
  P.part = reinterpret_cast<float2 *>(ws + L.part);
  P.ztgt = reinterpret_cast<float *>(ws + L.ztgt);
  P.tgt = a.tgt;
  if (int rc = launch_nt<CG, TG_LSE>(P, small, stream)) return rc;

  return launch_dependent(vocab_reduce, (M + 31) / 32, 32 * kReduceLanes, 0, stream,
                          (const float2 *)P.part, (const float *)P.ztgt, (const int *)a.idx, P.hdr,
                          P.target, loss, lse, 2 * (small ? (V + 127) / 128 : (V + 255) / 256), M,
                          V) == cudaSuccess
             ? 0
             : 1;
}

template <int CG>
int vocab_loss_backward_cg(const void *X, const void *W, const int64_t *target,
                               const float *lse, const float *dloss, void *dX, void *dW, int M,
                               int V, int d, void *workspace, cudaStream_t stream) {
  const VocabGradLayout L = vocab_grad_layout(M, V, d);
  char *ws = static_cast<char *>(workspace);
  GatherArgs a = {};
  a.X = static_cast<const __nv_bfloat16 *>(X);
  a.target = target;
  a.M = M, a.V = V, a.d = d;
  a.Xc = reinterpret_cast<__nv_bfloat16 *>(ws + L.Xc);
  a.idx = reinterpret_cast<int *>(ws + L.idx);
  a.tgt = reinterpret_cast<int *>(ws + L.tgt);
  a.hdr = reinterpret_cast<TgHeader *>(ws + L.hdr);
  a.lse = lse, a.dloss = dloss;
  a.lse_c = reinterpret_cast<float *>(ws + L.lse);
  a.g_c = reinterpret_cast<float *>(ws + L.g);
  a.tops = reinterpret_cast<float *>(ws + L.tops);
  a.dX = static_cast<__nv_bfloat16 *>(dX);
  const bool compact = vocab_compact(M, V, d);
  if (compact) {
    const int blocks = M < kTgMaxCtas * 2 ? M : kTgMaxCtas * 2;
    a.per = ((M + blocks - 1) / blocks + 1) / 2 * 2;
    if (launch_dependent(vocab_gather<true>, (M + a.per - 1) / a.per, kGatherThreads, 0, stream,
                         a) != cudaSuccess)
      return 1;
  }

  TgParams P = {}, Q = {};
  const TgPieces pieces = tg_pieces(M, V, L.cap_boxes);  // with fewer rows no more of them
  const bool small = tg_small<TG_PROB>(M, pieces.tp * 256);
  if (!nt_maps<CG>(P, compact ? a.Xc : a.X, W, M, V, d, small)) return 2;
  P.M = M, P.N = V, P.K = d;
  P.cap_boxes = L.cap_boxes;
  P.gmax = &a.hdr->gmax;
  P.gmax_out = &a.hdr->gmax;
  P.tops = a.tops;
  P.n_tops = compact ? (M + a.per - 1) / a.per : 0;
  if (compact) {
    P.hdr = a.hdr;
    P.tgt = a.tgt;
    P.lse = a.lse_c, P.g = a.g_c;
  } else {
    P.target = target;
    P.lse = lse, P.g = dloss;
    P.X = a.X, P.Xz = a.Xc;
    P.keep = a.idx;
  }
  const uint64_t box_rows = (uint64_t)L.cap_boxes * 64;
  if (!make_map_bf16(&P.S, ws + L.boxes, 64, box_rows, 64, 32)) return 2;
  Q = P;
  Q.blocked = 1;
  if (!make_map_bf16(&Q.A, ws + L.boxes, 64, box_rows, 64, 64) ||
      !make_map_bf16(&Q.A1, ws + L.boxes, 64, box_rows, 64, 128) ||
      !make_map_bf16(&Q.B, a.Xc, d, M, 64, 64) || !make_map_bf16(&Q.B1, W, d, V, 64, 64))
    return 2;
  Q.idx = compact ? a.idx : nullptr;
  Q.D0 = static_cast<__nv_bfloat16 *>(dW);
  Q.D1 = static_cast<__nv_bfloat16 *>(dX);
  Q.sums = reinterpret_cast<float *>(ws + L.sums);
  Q.slots = reinterpret_cast<float *>(ws + L.slots);
  for (int k = 0; k < pieces.np; ++k) {
    P.piece = Q.piece = k;
    if (int rc = launch_nt<CG, TG_PROB>(P, small, stream)) return rc;
    if (int rc = launch_grad<CG>(Q, pieces.np, stream)) return rc;
  }
  return 0;
}

template <int CG>
int gau_project_backward_cg(const void *X, const void *Wt, const void *dU, const void *dV,
                                const void *dZ, void *dX, void *dWt, int M, int d, int e, int s,
                                void *workspace, cudaStream_t stream) {
  const int N = 2 * e + s;
  const ProjectGradLayout L = project_grad_layout(M, N);
  char *ws = static_cast<char *>(workspace);
  TgParams P = {}, Q = {};
  const bool small = tg_small<TG_SILU>(M, N);
  if (!nt_maps<CG>(P, X, Wt, M, N, d, small)) return 2;
  P.M = M, P.N = N, P.K = d;
  P.cap_boxes = L.cap_boxes;
  P.n0 = e, P.n1 = 2 * e;
  const uint64_t box_rows = (uint64_t)L.cap_boxes * 64;
  if (!make_map_bf16(&P.S, ws + L.boxes, 64, box_rows, 64, 32) ||
      !make_map_bf16(&P.U0, dU, e, M, 64, 32) || !make_map_bf16(&P.U1, dV, e, M, 64, 32) ||
      !make_map_bf16(&P.U2, dZ, s, M, 64, 32))
    return 2;
  Q = P;
  Q.blocked = 1;
  if (!make_map_bf16(&Q.A, ws + L.boxes, 64, box_rows, 64, 64) ||
      !make_map_bf16(&Q.A1, ws + L.boxes, 64, box_rows, 64, 128) ||
      !make_map_bf16(&Q.B, X, d, M, 64, 64) || !make_map_bf16(&Q.B1, Wt, d, N, 64, 64))
    return 2;
  Q.D0 = static_cast<__nv_bfloat16 *>(dWt);
  Q.D1 = static_cast<__nv_bfloat16 *>(dX);
  Q.slots = reinterpret_cast<float *>(ws + L.slots);
  if (int rc = launch_nt<CG, TG_SILU>(P, small, stream)) return rc;
  return launch_grad<CG>(Q, 1, stream);
}

template <int CG>
int gau_output_backward_cg(const void *Y, const void *Wo_t, const void *dOut, void *dY,
                               void *dWo_t, int M, int e, int d, void *workspace,
                               cudaStream_t stream) {
  const OutputGradLayout L = output_grad_layout();
  char *ws = static_cast<char *>(workspace);
  TgParams Q = {};
  // A = dOut [tokens][d], read by columns for dWo_t [d][e], by rows for dY
  if (!make_map_bf16(&Q.A, dOut, d, M, 64, 64) || !make_map_bf16(&Q.A1, dOut, d, M, 64, 128) ||
      !make_map_bf16(&Q.B, Y, e, M, 64, 64) ||
      !make_map_bf16(&Q.B1, Wo_t, e, d, 64, 64))
    return 2;
  Q.M = M, Q.N = d, Q.K = e;
  Q.D0 = static_cast<__nv_bfloat16 *>(dWo_t);
  Q.D1 = static_cast<__nv_bfloat16 *>(dY);
  Q.slots = reinterpret_cast<float *>(ws + L.slots);
  return launch_grad<CG>(Q, 1, stream);
}

}  // namespace

int launch_vocab_loss(const void *X, const void *W, const int64_t *target, float *loss, float *lse,
                      int M, int V, int d, void *workspace, cudaStream_t stream) {
  return (tg_pairs(M) ? vocab_loss_cg<2> : vocab_loss_cg<1>)(X, W, target, loss, lse, M, V, d,
                                                            workspace, stream);
}

int launch_vocab_loss_backward(const void *X, const void *W, const int64_t *target,
                               const float *lse, const float *dloss, void *dX, void *dW, int M,
                               int V, int d, void *workspace, cudaStream_t stream) {
  return (tg_pairs(M) ? vocab_loss_backward_cg<2> : vocab_loss_backward_cg<1>)(
      X, W, target, lse, dloss, dX, dW, M, V, d, workspace, stream);
}

int launch_gau_project_backward(const void *X, const void *Wt, const void *dU, const void *dV,
                                const void *dZ, void *dX, void *dWt, int M, int d, int e, int s,
                                void *workspace, cudaStream_t stream) {
  return (tg_pairs(M) ? gau_project_backward_cg<2> : gau_project_backward_cg<1>)(
      X, Wt, dU, dV, dZ, dX, dWt, M, d, e, s, workspace, stream);
}

int launch_gau_output_backward(const void *Y, const void *Wo_t, const void *dOut, void *dY,
                               void *dWo_t, int M, int e, int d, void *workspace,
                               cudaStream_t stream) {
  return (tg_pairs(M) ? gau_output_backward_cg<2> : gau_output_backward_cg<1>)(
      Y, Wo_t, dOut, dY, dWo_t, M, e, d, workspace, stream);
}

}  // namespace fmca
