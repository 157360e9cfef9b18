// tc_tgemm.cuh -- the matrix products of the training operators around the
// attention core, on the tensor cores: one persistent tcgen05 kernel, four
// uses (KIND).  Tokens are rows m, outputs (vocabulary entries or projection
// features) are columns v, model features are d:
//
//   TG_LSE   Z = X W^T           per row the maximum and the sum of
//                                exp(z - maximum) of every NT / 2 columns, and the
//                                target's logit; Z itself is not stored
//   TG_PROB  Z = X W^T           the piece's (softmax(z) - onehot) * g, bf16
//   TG_SILU  Z = X W^T           dpre = dOut * silu'(z), bf16
//   TG_GRAD  dW = A^T X, dX = A W   from that bf16 matrix A (or a row-major
//                                one), two problems in one launch
//
// Operands are read by TMA into 128-byte-swizzled tiles, K-major or MN-major
// by descriptor, so no operand is ever transposed in memory.  The matrix A
// that TG_PROB and TG_SILU write lies in boxes of 64 tokens x 64 columns (8
// KB, row after row): box (c, t) of column block c and token block t is number
// c * n_tok64 + t.  The same box is a K-major tile for dX and an MN-major one
// for dW, and the width of a piece can be chosen on the device.
//
// A unit is a tile of 128 CG x NT outputs: NT = 256, or 128 (with CG = 1) for
// products of so few tiles that all run at once; CG = 1 one CTA, CG = 2 a pair of
// CTAs on one tcgen05 tile of M = 256 (each holds its 128 rows of A, half of
// B's 256 rows and the accumulator of its rows).  A pair reads (128 + 128) x 64
// operands a CTA and k step instead of (128 + 256) x 64, which is what bounds
// the single-CTA form: its operand traffic from L2.  K runs in 64-deep stages
// through a ring in shared memory into one of two TMEM accumulators.  Warps: 0
// TMA producer, 1 MMA issuer (of a pair: the first CTA's), 2-9 epilogue; every
// warp works out the units by itself, so there is no queue.  Every wait is
// bounded.  Included by tc.cu (through tc_train.cuh).
#pragma once

#include "tc_common.cuh"
#include "tg_plan.h"

namespace fmca {
namespace {

constexpr int TG_EPI_WARPS = 8;
constexpr int TG_THREADS = 64 + 32 * TG_EPI_WARPS;

// Shared memory of a CTA: the ring, and for the kinds that write A (TG_PROB,
// TG_SILU) 8 KB a warp to stage its 32 rows x 128 columns.
template <int CG, int KIND, int NT>
struct TgCfg {
  static constexpr uint32_t A_BYTES = 128 * 64 * 2;              // 16 KB
  static constexpr uint32_t B_BYTES = (NT / CG) * 64 * 2;        // 32 or 16 KB
  static constexpr uint32_t SLOT = A_BYTES + B_BYTES;
  static constexpr bool STAGED = KIND == TG_PROB || KIND == TG_SILU;
  static constexpr int RING = STAGED ? (NT / CG == 128 ? 5 : 3) : (NT / CG == 128 ? 6 : 4);
  static constexpr uint32_t PIECE = 32 * 64 * 2;                 // 32 rows x 64 columns
  static constexpr uint32_t STAGE = STAGED ? TG_EPI_WARPS * 2 * PIECE : 0;
  static constexpr uint32_t SMEM = RING * SLOT + STAGE + 1024;
  static_assert(SMEM + 1024 <= 232448, "tc_tgemm exceeds 227 KB of shared memory");
};

// What stays on the device: the number of rows that take part (the rows'
// preparation) and the largest |dloss| among them (TG_PROB; 1 if not finite).
struct TgHeader {
  int count;
  float gmax;
};
// The count as it is in L2 (a kernel may look before the grid ahead is over).
__device__ __forceinline__ int tg_count(const TgHeader *h) {
  return (int)ld_acquire_gpu(reinterpret_cast<const unsigned int *>(&h->count));
}

struct TgParams : TgSizes {
  CUtensorMap A, B;    // NT kinds: X [M][K] box {64, 128}, W [N][K] box {64, 256 / CG}
                       // TG_GRAD: A of problem 0, box {64, 64}, and (A1) of
                       // problem 1, box {64, 128}; B and B1, box {64, 64}
  CUtensorMap A1, B1;
  CUtensorMap S;       // TG_PROB, TG_SILU: the boxes as rows of 64, box {64, 32}
  CUtensorMap U0, U1, U2;  // TG_SILU: the incoming gradients, box {64, 32}
  int piece;           // piece of the column axis (TG_PROB, TG_GRAD)
  const TgHeader *hdr; // device count of rows (NULL: M)
  const float *gmax;   // scale of dW and dX (NULL: 1)
  const int *idx;      // compact row -> row (NULL: the same)
  // few rows, taken as they are: their targets (TG_LSE, TG_PROB), and what
  // TG_PROB leaves for TG_GRAD: whether a row has one, X with 0 in the others
  const int64_t *target;
  const __nv_bfloat16 *X;
  __nv_bfloat16 *Xz;
  int *keep;
  // TG_PROB: the largest |dloss| of the rows' blocks, and where it goes
  const float *tops;
  int n_tops;
  float *gmax_out;
  // TG_LSE
  float2 *part;        // [2 ceil(N / NT)][M]
  float *ztgt;         // [M]
  const int *tgt;      // [M]
  // TG_PROB
  const float *lse, *g;
  // TG_SILU: gradients of the activations (U0, U1, U2), columns [0, n0), [n0,
  // n1), [n1, N), multiples of 64
  int n0, n1;
  // TG_GRAD
  __nv_bfloat16 *D0;   // dW [V][K]
  __nv_bfloat16 *D1;   // dX [tokens][K]
  float *slots;        // two fp32 tiles of 128 x 256 a worker and CTA: its cut tiles
  float *sums;         // dX's tiles between pieces, fp32
};

// ------------------------------------------------------------- CTA pairs
template <int CG>
__device__ __forceinline__ uint32_t tg_rank() {
  if constexpr (CG == 1) return 0;
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t tg_mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
template <int CG>
__device__ __forceinline__ void tg_sync_all() {
  if constexpr (CG == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  }
}
// 2-D TMA load into this CTA's shared memory, counted on the barrier at the
// shared-cluster address `bar` (a pair: the first CTA's).
template <int CG>
__device__ __forceinline__ void tg_load(void *dst, const CUtensorMap *map, uint32_t bar, int x,
                                        int y) {
  if constexpr (CG == 1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
// Brings a 2-D box into L2 (no shared memory, no barrier).
__device__ __forceinline__ void tg_prefetch_l2(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
template <int CG>
__device__ __forceinline__ void tg_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 1) {
    mma_bf16_ss(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Arrive on `bar` (a pair: in both CTAs) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void tg_commit(uint64_t *bar) {
  if constexpr (CG == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tg_tmem_alloc(uint32_t *dst, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tg_tmem_dealloc(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 1)
    tmem_dealloc(addr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}
// mbar_wait on a barrier that threads of the other CTA of a pair arrive on.
template <int CG>
__device__ __forceinline__ bool tg_wait_pair(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  if constexpr (CG == 1) return mbar_wait(bar, parity, limit_ns);
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}
// The epilogue's arrival on the MMA issuer's barrier (a pair: the first CTA's).
template <int CG>
__device__ __forceinline__ void tg_arrive_leader(uint64_t *bar) {
  if constexpr (CG == 1)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     tg_mapa(smem_u32(bar), 0))
                 : "memory");
}

// ------------------------------------------------------------- elementwise
__device__ __forceinline__ float tg_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 32 bytes to global memory (32-byte aligned).
__device__ __forceinline__ void tg_store32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 values of this thread's row rounded to bf16 into half h of its warp's
// staged piece (32 rows of 128 bytes, 128-byte swizzle).
__device__ __forceinline__ void tg_stage(uint8_t *piece, int lane, int h, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4 *>(piece + sw128_offset(lane, h * 64 + 16 * q)) =
        make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                   pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                   pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
}
// Element offset of 4-column group j of row `row` in an fp32 partial tile of
// 128 x 256: rows next to each other, so that a warp's 32 rows are 512
// consecutive bytes.
__host__ __device__ inline int64_t tg_slot_offset(int row, int j) {
  return ((int64_t)j * 128 + row) * 4;
}
constexpr int64_t kTgSlotFloats = 128 * 256;

// The scale of dW and dX from a warp's largest |dloss| (1 for an infinite one,
// which the other rows could not bear).
__device__ __forceinline__ float tg_scale(float top) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top == INFINITY ? 1.f : top;
}

// TG_PROB on rows as they are (512 at most): the largest |dloss| of those that
// have a target, the same in every warp of the launch, and, shared between the
// warps, what TG_GRAD needs: the rows' marks and X without the others' contents
// (0 times NaN would be NaN).
__device__ __forceinline__ float tg_rows_as_they_are(const TgParams &P, int count, int w, int W,
                                                     int lane) {
  float top = 0.f;
#pragma unroll 4
  for (int r = lane; r < count; r += 32) {
    const int64_t t = P.target[r];
    if (t >= 0 && t < P.N) top = fmaxf(top, fabsf(P.g[r]));
  }
  top = tg_scale(top);
  if (w == 0 && lane == 0) *P.gmax_out = top;
  for (int r = w; r < count; r += W) {
    const int64_t t = P.target[r];
    const bool has = t >= 0 && t < P.N;
    if (lane == 0) P.keep[r] = has ? 1 : 0;
    const uint4 *src = reinterpret_cast<const uint4 *>(P.X + (int64_t)r * P.K);
    uint4 *dst = reinterpret_cast<uint4 *>(P.Xz + (int64_t)r * P.K);
    for (int v = lane; v < P.K / 8; v += 32)
      dst[v] = has ? __ldg(src + v) : make_uint4(0u, 0u, 0u, 0u);
  }
  return top;
}

template <int CG, int KIND, int NT>
__global__ void __launch_bounds__(TG_THREADS, 1)
    tc_tgemm(const __grid_constant__ TgParams P) {
  using Cfg = TgCfg<CG, KIND, NT>;
  static_assert(NT == 256 || CG == 1);
  constexpr int RING = Cfg::RING;
  // With few of the rows taking part the pieces are wide and the last launches
  // have none (every kernel ahead has waited for the one that counts).
  if ((KIND == TG_PROB || KIND == TG_GRAD) && P.hdr != nullptr && P.piece > 0 &&
      P.piece >= tg_pieces(tg_count(P.hdr), P.N, P.cap_boxes).np) {
    griddep_wait();
    return;
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[RING], empty[RING];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
  __shared__ __align__(8) uint64_t up_full[2 * TG_EPI_WARPS];  // TG_SILU: gradients staged
  __shared__ uint32_t tmem_base;
  __shared__ TgPlan plan;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = tg_rank<CG>();
  const int worker = (int)blockIdx.x / CG, workers = (int)gridDim.x / CG;
  // A programmatic dependent: it may be here while the work ahead on the
  // stream is still running, and reads none of that work's results before the
  // grid wait.  TG_GRAD may look at the row count: it was launched by a TG_PROB
  // that had waited for the kernel that counts (or has none).
  const bool early = KIND == TG_GRAD || P.hdr == nullptr;
  if (threadIdx.x == 96) {
    tma_prefetch_desc(&P.A);
    tma_prefetch_desc(&P.B);
    if (KIND == TG_GRAD) {
      tma_prefetch_desc(&P.A1);
      tma_prefetch_desc(&P.B1);
    }
    if (early)
      plan = tg_plan<CG, KIND, NT>(P, P.piece, P.hdr != nullptr ? tg_count(P.hdr) : P.M, workers);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], TG_EPI_WARPS * CG);
    }
    for (int i = 0; i < 2 * TG_EPI_WARPS; ++i) mbar_init(&up_full[i], 1);
    fence_mbar_init();
  }
  if (warp == 1) tg_tmem_alloc<CG>(&tmem_base, 512);
  tc_fence_before();
  tg_sync_all<CG>();
  tc_fence_after();
  const uint32_t tbase = tmem_base;
  // every warp walks the units by itself; the first one is found ahead of the
  // grid wait where the plan was made there
  TgWalk<KIND> walk(plan);
  TgUnit ahead;
  bool more = false;
  if (early) {
    walk.start(worker, workers);
    more = walk.next(ahead);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (!early) {
    if (threadIdx.x == 96) plan = tg_plan<CG, KIND, NT>(P, P.piece, tg_count(P.hdr), workers);
    __syncthreads();
    walk.start(worker, workers);
    more = walk.next(ahead);
  }
  const int count = plan.count, col0 = plan.col0, n_tok64 = plan.pc.n_tok64;

  if (warp == 0) {
    // =========================== TMA producer
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (TgUnit u; ok && more; more = walk.next(ahead)) {
        u = ahead;
        const int m0 = u.mt * 128 * CG + (int)rank * 128;
        const int nb0 = u.nt * NT + (int)rank * 128;
        for (int ks = 0; ks < u.nks; ++ks, ++it) {
          const int slot = it % RING;
          if (it >= RING && !mbar_wait(&empty[slot], ((it / RING) - 1) & 1, kWaitLimitNs)) {
            record_timeout(1001);
            ok = false;
            break;
          }
          uint8_t *sa = smem + slot * Cfg::SLOT, *sb = sa + Cfg::A_BYTES;
          uint32_t bar = smem_u32(&full[slot]);
          if constexpr (CG == 2) bar = tg_mapa(bar, 0);
          // out-of-range rows and columns arrive as zeros; full boxes count
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], Cfg::SLOT * CG);
          const int kk = (u.ks0 + ks) * 64;
          if constexpr (KIND != TG_GRAD) {
            tg_load<CG>(sa, &P.A, bar, kk, m0);
            tg_load<CG>(sb, &P.B, bar, kk, col0 + nb0);
          } else {
            const CUtensorMap *mB = u.pi ? &P.B1 : &P.B;
            if (u.pi) {
              // rows m, columns k (in the boxes: column block kk / 64, two token
              // blocks, one behind the other)
              if (P.blocked)
                tg_load<CG>(sa, &P.A1, bar, 0, (kk / 64) * n_tok64 * 64 + m0);
              else
                tg_load<CG>(sa, &P.A1, bar, kk, m0);
            } else if (P.blocked) {
              // columns m: column blocks m0 / 64 and the next, token block kk / 64
              const int row0 = (m0 / 64) * n_tok64 * 64 + kk;
              tg_load<CG>(sa, &P.A, bar, 0, row0);
              tg_load<CG>(sa + 8192, &P.A, bar, 0, row0 + n_tok64 * 64);
            } else {  // rows k, columns m
              tg_load<CG>(sa, &P.A, bar, m0, kk);
              tg_load<CG>(sa + 8192, &P.A, bar, m0 + 64, kk);
            }
            // rows k (problem 1: from the piece's first row of W), columns n
            const int krow = kk + (u.pi ? col0 : 0);
#pragma unroll
            for (int q = 0; q < NT / 64 / CG; ++q)
              tg_load<CG>(sb + q * 8192, mB, bar, nb0 + 64 * q, krow);
          }
        }
      }
      // wait (bounded) until every slot's last use is over: its copies have
      // landed and, in a pair, no arrival is on its way to a CTA that has left
      for (int q = (it > RING ? it - RING : 0); ok && q < it; ++q)
        if (!mbar_wait(&empty[q % RING], (q / RING) & 1, kWaitLimitNs)) {
          record_timeout(1002);
          break;
        }
    }
  } else if (warp == 1) {
    // =========================== MMA issuer (of a pair: the first CTA)
    if (lane == 0 && rank == 0) {
      constexpr bool kMn = KIND == TG_GRAD;
      constexpr uint32_t id_k = idesc_bf16_f32(128 * CG, NT, false, kMn);
      constexpr uint32_t id_mn = idesc_bf16_f32(128 * CG, NT, true, kMn);
      int it = 0;
      bool ok = true;
      TgUnit u;
      int i = 0;
      for (; ok && more; ++i, more = walk.next(ahead)) {
        u = ahead;
        const int buf = i & 1, use = i >> 1;
        if (use >= 1 && !tg_wait_pair<CG>(&acc_empty[buf], (use - 1) & 1, kWaitLimitNs)) {
          record_timeout(1011);
          ok = false;
          break;
        }
        tc_fence_after();
        const bool a_mn = kMn && u.pi == 0;
        const uint32_t idesc = a_mn ? id_mn : id_k;
        const uint32_t dcol = tbase + (uint32_t)buf * 256u;
        for (int ks = 0; ks < u.nks; ++ks, ++it) {
          const int slot = it % RING;
          if (!mbar_wait(&full[slot], (it / RING) & 1, kWaitLimitNs)) {
            record_timeout(1012);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + slot * Cfg::SLOT), sb = sa + Cfg::A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // K-major: the next 16 k are 32 bytes further along each row;
            // MN-major: 16 k rows further (LBO: between 64-column boxes)
            const uint64_t ad = a_mn ? smem_desc_sw128(sa + kk * 2048, 8192, 1024)
                                     : smem_desc_sw128(sa + kk * 32, 16, 1024);
            const uint64_t bd = kMn ? smem_desc_sw128(sb + kk * 2048, 8192, 1024)
                                    : smem_desc_sw128(sb + kk * 32, 16, 1024);
            tg_mma<CG>(dcol, ad, bd, idesc, (ks | kk) != 0);
          }
          tg_commit<CG>(&empty[slot]);
        }
        if (!ok) break;
        tg_commit<CG>(&acc_full[buf]);
      }
      // the last accumulators have been read, so every MMA is over
      for (int q = (i > 2 ? i - 2 : 0); ok && q < i; ++q)
        if (!tg_wait_pair<CG>(&acc_empty[q & 1], (q >> 1) & 1, kWaitLimitNs)) {
          record_timeout(1013);
          break;
        }
    }
  } else {
    // =========================== epilogue warps
    // Warp w reads TMEM lanes 32 (w % 4) .. (its 32 rows, one a thread) of
    // columns kHalf half .. + kHalf, 64 at a time (NQ pieces).
    constexpr int kHalf = NT / 2, NQ = kHalf / 64;
    const int quad = warp & 3, half = (warp - 2) / 4;
    const int row = quad * 32 + lane;
    uint8_t *stage = smem + RING * Cfg::SLOT + (warp - 2) * 2 * Cfg::PIECE;
    TgUnit u;
    // TG_SILU: the incoming gradients of this warp's rows and 64 columns (piece
    // q) of a unit, into the piece that it then works on in place
    uint64_t *up = up_full + 2 * (warp - 2);
    auto fetch = [&](const TgUnit &f, int q, bool l2_only) {
      const int row0 = f.mt * 128 * CG + (int)rank * 128 + quad * 32;
      const int col = f.nt * NT + half * kHalf + 64 * q;
      // columns past the last array arrive as zeros
      const CUtensorMap *map = col < P.n0 ? &P.U0 : col < P.n1 ? &P.U1 : &P.U2;
      const int x = col < P.n0 ? col : col < P.n1 ? col - P.n0 : col - P.n1;
      if (l2_only) {
        tg_prefetch_l2(map, x, row0);
      } else {
        mbar_arrive_expect_tx(&up[q], Cfg::PIECE);
        tma_load_2d(stage + q * Cfg::PIECE, map, &up[q], x, row0);
      }
    };
    int fetched[2] = {0, 0}, used[2] = {0, 0};
    if constexpr (KIND == TG_SILU) {
      if (more) {
        if (lane == 0) fetch(ahead, 0, false);
        ++fetched[0];
      }
    }
    // a finished piece (32 tokens x 64 columns) to its place in the boxes
    auto store_piece = [&](const TgUnit &f, int q, uint8_t *piece) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int row0 = f.mt * 128 * CG + (int)rank * 128 + quad * 32;
        const int block = (f.nt * NT + half * kHalf) / 64 + q;
        tma_store_2d(&P.S, piece, 0, block * n_tok64 * 64 + row0);
        bulk_commit_group();
      }
      __syncwarp();
    };
    float gmax = 0.f;
    const float alpha = KIND == TG_GRAD && P.gmax != nullptr ? *P.gmax : 1.f;
    if constexpr (KIND == TG_PROB) {
      if (P.target == nullptr) {
        for (int b = lane; b < P.n_tops; b += 32) gmax = fmaxf(gmax, P.tops[b]);
        gmax = tg_scale(gmax);
        if (blockIdx.x == 0 && warp == 2 && lane == 0) *P.gmax_out = gmax;
      } else {
        gmax = tg_rows_as_they_are(P, count, (int)blockIdx.x * TG_EPI_WARPS + warp - 2,
                                   (int)gridDim.x * TG_EPI_WARPS, lane);
      }
    }
    for (int i = 0; more; ++i) {
      u = ahead;
      more = walk.next(ahead);
      const int buf = i & 1, use = i >> 1;
      const int m = u.mt * 128 * CG + (int)rank * 128 + row;  // row of the product
      const int c0 = u.nt * NT + half * kHalf;                // first column in the piece
      // TG_SILU: piece 0 was fetched as soon as the unit before had left it;
      // piece 1, stored last, follows now.  The next unit's gradients come to
      // L2 meanwhile: their pieces are free too late for a trip to DRAM.
      if constexpr (KIND == TG_SILU && NQ == 2) {
        if (lane == 0) {
          bulk_wait_group_read<0>();
          fetch(u, 1, false);
          if (more) {
            fetch(ahead, 0, true);
            fetch(ahead, 1, true);
          }
        }
        ++fetched[1];
        __syncwarp();
      }
      // TG_LSE, TG_PROB: the row's constants, before the accumulator is ready
      bool in_rows = m < count;
      float row_lse = 0.f, row_g = 0.f;
      int row_at = -1;
      if constexpr (KIND == TG_LSE || KIND == TG_PROB) {
        if (P.target == nullptr) {
          if (in_rows) row_at = P.tgt[m] - col0 - c0;
        } else {
          const int64_t t = in_rows ? P.target[m] : -1;
          in_rows = t >= 0 && t < P.N;
          if (in_rows) row_at = (int)t - col0 - c0;
        }
      }
      if constexpr (KIND == TG_PROB) {
        if (in_rows) {
          row_lse = P.lse[m] * kLog2e;
          row_g = P.g[m];
        }
      }
      // TG_GRAD: where the row goes
      bool live = true;  // dX of a row without a target is 0, whatever W holds
      __nv_bfloat16 *out = nullptr;
      if constexpr (KIND == TG_GRAD) {
        if (m < plan.s[u.pi].M) {
          if (u.pi) {
            if (P.keep != nullptr) live = P.keep[m] != 0;
            out = P.D1 + (int64_t)(P.idx != nullptr ? P.idx[m] : m) * P.K;
          } else {
            out = P.D0 + (int64_t)(col0 + m) * P.K;
          }
        }
      }
      if (!mbar_wait(&acc_full[buf], use & 1, kWaitLimitNs)) {
        if (lane == 0) record_timeout(1020);
        break;
      }
      tc_fence_after();
      const uint32_t dcol =
          tbase + (uint32_t)buf * 256u + (uint32_t)(half * kHalf) + ((uint32_t)(quad * 32) << 16);
      // this warp's last read of the accumulator
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tg_arrive_leader<CG>(&acc_empty[buf]);
      };
      if constexpr (KIND == TG_LSE) {
        constexpr int NC = kHalf / 32;
        uint32_t r[NC][32];
#pragma unroll
        for (int c = 0; c < NC; ++c) tmem_ld32(dcol + 32 * c, r[c]);
        tmem_ld_wait();
        release();
        // columns past the vocabulary count as -infinity
        if (c0 + kHalf > P.N) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c0 + 32 * c + j >= P.N) r[c][j] = 0xFF800000u;
        }
        float mx[NC], sm[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) mx[c] = -INFINITY, sm[c] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) mx[c] = fmaxf(mx[c], __uint_as_float(r[c][j]));
        float top = fmaxf(mx[0], mx[1]);
        if constexpr (NC == 4) top = fmaxf(top, fmaxf(mx[2], mx[3]));
        // a row of -infinities has the sum 0 (not exp(-inf + inf))
        const float ref = top == -INFINITY ? 0.f : top * kLog2e;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            sm[c] += tg_exp2(fmaf(__uint_as_float(r[c][j]), kLog2e, -ref));
        float sum = sm[0] + sm[1];
        if constexpr (NC == 4) sum += sm[2] + sm[3];
        if (in_rows) P.part[(int64_t)(u.nt * 2 + half) * P.M + m] = make_float2(top, sum);
        const int at = row_at;
        if (__any_sync(0xffffffffu, at >= 0 && at < kHalf)) {
          float z = 0.f;
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (at == 32 * c + j) z = __uint_as_float(r[c][j]);
          if (at >= 0 && at < kHalf) P.ztgt[m] = z;
        }
      } else {
        // 64 columns at a time, in chunks of 32
        const float g = KIND == TG_PROB && gmax > 0.f ? row_g / gmax : row_g;
        const bool any = KIND == TG_PROB && __any_sync(0xffffffffu, row_at >= 0 && row_at < kHalf);
        const int left = plan.width - c0;  // TG_PROB: columns of the piece from here on
        // TG_GRAD: problem 1 over several pieces adds to what the pieces before
        // left; a cut tile's part goes to the place of the worker's tile that
        // was begun by another (its first) or is ended by another (its last)
        const TgShape &h = plan.s[KIND == TG_GRAD ? u.pi : 0];
        const bool last = !P.blocked || u.pi == 0 || P.piece == plan.pc.np - 1;
        const bool direct = u.whole && last;
        const bool add = u.pi == 1 && P.blocked && P.piece > 0;
        float *slot = nullptr;
        bool wide = false;
        if constexpr (KIND == TG_GRAD) {
          const int cut = tg_part(worker, u.ks0 > 0, CG, (int)rank);
          slot = u.whole ? P.sums + ((int64_t)(u.mt * CG + (int)rank) * h.Nt + u.nt) * kTgSlotFloats
                         : P.slots + (int64_t)cut * kTgSlotFloats;
          wide = P.K % 16 == 0 && (reinterpret_cast<uintptr_t>(u.pi ? P.D1 : P.D0) & 31u) == 0;
        }
        bool ok = true;
#pragma unroll
        for (int q2 = 0; q2 < NQ; ++q2) {
          uint32_t r[2][32];
          tmem_ld32(dcol + 64 * q2, r[0]);
          tmem_ld32(dcol + 64 * q2 + 32, r[1]);
          uint8_t *piece = stage + q2 * Cfg::PIECE;
          if constexpr (KIND == TG_PROB) {  // the store from this piece a unit ago has read it
            if (lane == 0) bulk_wait_group_read<NQ - 1>();
            __syncwarp();
          }
          if constexpr (KIND == TG_SILU) {
            ok = mbar_wait(&up[q2], i & 1, kWaitLimitNs);
          }
          tmem_ld_wait();
          if (!ok) break;
          if constexpr (KIND == TG_SILU) ++used[q2];
          if (q2 == NQ - 1) release();
          if (KIND == TG_GRAD && u.nks == 0) {  // nothing was multiplied: the product is 0
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
              for (int j = 0; j < 32; ++j) r[c2][j] = 0u;
          }
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            const int c = 2 * q2 + c2;
            float v[32];
            if constexpr (KIND == TG_PROB) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                v[j] = tg_exp2(fmaf(__uint_as_float(r[c2][j]), kLog2e, -row_lse)) * g;
              if (any) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (row_at == 32 * c + j)  // (p - 1) g, the difference formed first
                    v[j] = (tg_exp2(fmaf(__uint_as_float(r[c2][j]), kLog2e, -row_lse)) - 1.f) * g;
              }
              if (!in_rows || left < kHalf) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!in_rows || 32 * c + j >= left) v[j] = 0.f;
              }
            } else if constexpr (KIND == TG_SILU) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint4 g4 =
                    *reinterpret_cast<const uint4 *>(piece + sw128_offset(lane, c2 * 64 + 16 * q));
                const uint32_t ww[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float z = __uint_as_float(r[c2][8 * q + k]);
                  const float sig = __fdividef(1.f, 1.f + __expf(-z));
                  const float d = (k & 1) ? bf16_hi(ww[k / 2]) : bf16_lo(ww[k / 2]);
                  v[8 * q + k] = d * sig * fmaf(z, 1.f - sig, 1.f);
                }
              }
              if (NQ == 2 && c == 2 && more) {  // the store of piece 0 has read it
                if (lane == 0) {
                  bulk_wait_group_read<0>();
                  fetch(ahead, 0, false);
                }
                ++fetched[0];
              }
              // rows past the last and columns past the last array: z and the
              // gradient both came in as zeros, so these are zeros
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[c2][j]);
              if (add) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float4 o = *reinterpret_cast<const float4 *>(
                      slot + tg_slot_offset(row, half * (kHalf / 4) + c * 8 + j));
                  v[4 * j] += o.x, v[4 * j + 1] += o.y, v[4 * j + 2] += o.z, v[4 * j + 3] += o.w;
                }
              }
              if (!direct) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  *reinterpret_cast<float4 *>(
                      slot + tg_slot_offset(row, half * (kHalf / 4) + c * 8 + j)) =
                      make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
              } else if (out != nullptr) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  uint32_t w[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    w[k] = live ? pack_bf16x2(alpha * v[16 * q + 2 * k],
                                              alpha * v[16 * q + 2 * k + 1])
                                : 0u;
                  const int cq = c0 + 32 * c + 16 * q;
                  if (wide) {
                    if (cq < P.K) tg_store32(out + cq, w);
                  } else {  // rows start on 16-byte boundaries only
                    if (cq < P.K)
                      *reinterpret_cast<uint4 *>(out + cq) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (cq + 8 < P.K)
                      *reinterpret_cast<uint4 *>(out + cq + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                  }
                }
              }
            }
            if constexpr (Cfg::STAGED) {
              tg_stage(piece, lane, c2, v);
              if (c2 == 1) store_piece(u, q2, piece);
            }
          }
        }
        if constexpr (KIND == TG_SILU && NQ == 1) {
          if (ok && more) {  // the only piece is free once its store has read it
            if (lane == 0) {
              bulk_wait_group_read<0>();
              fetch(ahead, 0, false);
            }
            ++fetched[0];
          }
        }
        if (!ok) {
          if (lane == 0) record_timeout(1021);
          break;
        }
      }
    }
    // a wait that ran out may have left gradients on their way
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (fetched[q] > used[q] && !mbar_wait(&up[q], (fetched[q] - 1) & 1, kWaitLimitNs) &&
          lane == 0)
        record_timeout(1022);
    // staged pieces have been read (and, before the kernel ends, written)
    if constexpr (Cfg::STAGED) {
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
    }
  }
  // the single-lane roles rejoin their warps before the block-wide barrier,
  // which counts converged warps
  __syncwarp();
  tc_fence_before();
  tg_sync_all<CG>();
  if (warp == 1) tg_tmem_dealloc<CG>(tbase, 512);
}

}  // namespace
}  // namespace fmca
