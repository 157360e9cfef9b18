// tc_decay.cuh -- linear attention with a decay for each head over whole prompts, on
// the tensor cores (bf16, dk and dv multiples of 8, dk <= 128).  Included by tc.cu.
//
//   o_i = scale (sum_{j <= i} lam^(i-j) (q_i k_j) v_j + lam^(i+1) q_i S)   rows of a chunk
//   S   = lam^n S + sum_j lam^(n-1-j) k_j^T v_j                            its n tokens
//
// A CTA walks one unit (a head of one sequence, 128 columns of dv, a segment of the
// tokens) in chunks of 128 tokens: q, k and v are read once, and the state stays in
// registers, fp32.  Of each chunk four products, accumulators in TMEM:
//
//   Sc = Q K^T          then P = Sc lam^(i-j), masked, bf16, back into TMEM
//   O  = Q S            S: the state before the chunk, rounded to bf16
//   O  = lam^(i+1) O + P V      (the rows scaled in place in between, P and they by scale)
//   D  = K~^T V         K~_j = lam^(n-1-j) k_j
//   o = O,   S = lam^n S + D
//
// What is rounded: P and the operand S, half a step of bf16 each, as is the output.  Outputs are
// off by 2.35e-3 of their root mean square with these, by 1.65e-3 with their own rounding alone.
// A second term of either would be a fifth product of a chunk, and for S 32 KB of shared memory,
// which has none left at 128 x 128; the state, which carries errors on, is not rounded.
// K~ is not: a product of a weight in 24 bits and a key in 8 goes in as three bf16
// terms (what is left out is under 2^-26 of it), the smallest first, as the tensor
// cores' sums may cut bits; a state with one term would be off by 2^-9 and one with two
// by 2.8e-6, where fp32 sums are off by about 1e-6.  Every power has an exponent >= 0,
// so a strong decay underflows and never overflows.
//
// Where there are fewer units than SMs a sequence is cut into S segments: a first
// launch (LOCAL) forms only the segments' states, a second starts every segment from
// the sum of those before it.
//
// Warps (768 threads): 0 TMA, 1 and 3 MMA issuers, 2 a look at v and the output stores; 4-11 P
// and the outputs; 12-15 K~'s terms, from K in place (the first term) and through two buffers
// of 32 tokens (the others); 16-23 the state, from D in TMEM, and its bf16 copy in shared
// memory.  P takes the columns of the scores that its own warp has read, of one of two
// buffers.
//
// Measured: 2 x 8192 tokens of 12 heads of 128 75 us (201 MB: 2.7 TB/s, 40 % of a copy's rate;
// under a profiler the states' launch 28 and the outputs' 59), 1 x 32768 of 16 176 us, 8 x
// 1024 of 12 heads with one q and k 40 us, 37 tokens 6.6 us; with a unit uncut on every SM, 2
// x 8192 of 75 heads, 245 us, 5.2 TB/s, 77 % of a copy's rate. Not bound by memory (the same
// from L2) nor by the products (the pipe is busy 26 % of the time): a chunk of the outputs'
// launch takes about 3.6 us on an SM, in which the state goes once around (D, the sum in
// registers, its bf16 copy, Q S) while 24 warps pass the tiles through shared memory: keys
// read, three terms written, v looked at, the weights and both accumulators through registers.
// Without the keys' terms a chunk takes 10 % less, without the weights 2 %, with one term's
// products 2 %. Around the chunks are 8 us: the start, the first copies, the last outputs. So
// the cut: whole heads of 128 columns, one unit an SM, as many segments as there are SMs,
// though k and v of all but the last are read twice. Chunks of 128: the products' tile; the
// weights' work grows with the chunk, the state's with the number of them, and at 128 x 128 x
// 128 they are equal.
#pragma once

#include "decay.cuh"
#include "tc_common.cuh"

namespace fmca {
namespace {

constexpr int DA_THREADS = 768;
constexpr int DA_SLOTS = 12;             // ring slots at most
constexpr uint32_t DA_ATOM = 16384;      // 64 columns of 128 tokens
constexpr uint32_t DA_SMEM = 229376;     // ring, state, terms
constexpr uint32_t DA_COL_SC = 0, DA_COL_O = 256, DA_COL_D = 384;  // two of Sc
constexpr int DA_OUT_WARP = 4, DA_KEY_WARP = 12, DA_STATE_WARP = 16;
// Registers of a thread: 80 at the launch of 768; the state's 64 places need more, the
// first four warps and the keys' less.
constexpr int DA_REG_ISSUE = 48, DA_REG_OUT = 80, DA_REG_KEYS = 64, DA_REG_STATE = 104;
static_assert(128 * DA_REG_ISSUE + 256 * DA_REG_OUT + 128 * DA_REG_KEYS + 256 * DA_REG_STATE <=
                  80 * DA_THREADS,
              "tc_decay's warps would wait for registers that the block has not");

// Shared memory by the 64-column blocks of dk (ka) and of the unit's dv (va).
__host__ __device__ inline uint32_t da_slot(int ka, int va) {
  return DA_ATOM * (uint32_t)(ka > va ? ka : va);
}
__host__ __device__ inline uint32_t da_state_bytes(int ka, int va) {
  return 8192u * (uint32_t)(ka * va);
}
static_assert(4 * (128 * 128 + 2 * DA_THREADS) <= DA_SMEM, "decay_tokens' state and sums");
__host__ __device__ inline uint32_t da_term_bytes(int ka) { return DA_ATOM * (uint32_t)ka; }
// The places of a ring each of q, k and v tiles (LOCAL: of k and v, and no state tile).
// One ring of all three in turn would have k wait for the place that outputs leave last.
struct DaRings {
  int q, k, v;
};
__host__ __device__ inline DaRings da_rings(bool local, int ka, int va) {
  const uint32_t room = DA_SMEM - da_term_bytes(ka) - (local ? 0 : da_state_bytes(ka, va));
  int n = (int)(room / da_slot(ka, va));
  n = n < DA_SLOTS ? n : DA_SLOTS;
  return local ? DaRings{0, n / 2, n / 2} : DaRings{n / 3, (n + 1) / 3, (n + 2) / 3};
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A wait with a limit of turns (each suspends the thread for up to a microsecond; seconds in
// all), without a look at the clock: the roles' loops of a chunk share the instruction
// caches, and what is not in a warp's nearest one costs it more than its products.
__device__ __forceinline__ bool da_wait(uint64_t *bar, int use) {
#pragma unroll 1
  for (int i = 0; !mbar_try_wait_sleep(bar, (uint32_t)use & 1u, 1000u); ++i)
    if (i > (1 << 23)) return false;
  return true;
}

// A place in a ring and how often it has been used before, kept step by step: a division
// by the ring's length takes a role longer than its products.
struct RingAt {
  int slot, use;
  __device__ __forceinline__ explicit RingAt(int first) : slot(first), use(0) {}
  __device__ __forceinline__ void step(int first, int n) {
    if (++slot == first + n) slot = first, ++use;
  }
};

// Two floats in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Two products of bf16, plus `sum`: finite only if all are.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t x, uint32_t y, uint32_t sum) {
  uint32_t z;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(z) : "r"(x), "r"(y), "r"(sum));
  return z;
}
__device__ __forceinline__ bool wild_lo(uint32_t x) { return (x & 0x7F80u) == 0x7F80u; }
__device__ __forceinline__ bool wild_hi(uint32_t x) { return (x & 0x7F800000u) == 0x7F800000u; }

// By one warp: what is not finite in a tile of n rows of 64 columns becomes 0, and
// row[0 .. 63] each column's first row with such a value (128: none).
__device__ __noinline__ void tame(uint8_t *tile, int n, uint8_t *row, int lane) {
  int at[2] = {128, 128};
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    uint32_t *const p = reinterpret_cast<uint32_t *>(tile + sw128_offset(i, 4u * lane));
    const uint32_t y = *p;
    const bool lo = wild_lo(y), hi = wild_hi(y);
    if (lo && at[0] > i) at[0] = i;
    if (hi && at[1] > i) at[1] = i;
    if (lo || hi) *p = y & (lo ? 0xFFFF0000u : ~0u) & (hi ? 0xFFFFu : ~0u);
  }
  row[2 * lane] = (uint8_t)at[0];
  row[2 * lane + 1] = (uint8_t)at[1];
}

// Two keys times w as three bf16 terms.
__device__ __forceinline__ void key_terms(uint32_t k, float2 w, uint32_t &t0, uint32_t &t1,
                                          uint32_t &t2) {
  const float2 minus = make_float2(-1.f, -1.f);
  float2 x = mul2(make_float2(bf16_lo(k), bf16_hi(k)), w);
  t0 = pack_bf16x2(x.x, x.y);
  x = fma2(make_float2(bf16_lo(t0), bf16_hi(t0)), minus, x);
  t1 = pack_bf16x2(x.x, x.y);
  x = fma2(make_float2(bf16_lo(t1), bf16_hi(t1)), minus, x);
  t2 = pack_bf16x2(x.x, x.y);
}

// first: this launch is the call's first (it waits for the work ahead; the second one
// waits for the first before it reads a state).
// ka: the 64-column blocks of dk.
template <bool LOCAL, int ka>
__global__ void __launch_bounds__(DA_THREADS, 1)
    tc_decay(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
             const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapO,
             const __grid_constant__ DecayArgs a,
             const DecaySplit sp, float *__restrict__ slots, int first) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[DA_SLOTS], empty[DA_SLOTS], x_ready[2], x_free[2];
  __shared__ __align__(8) uint64_t staged[2], stored[2];
  __shared__ __align__(8) uint64_t sc_full[2], qs_full, p_ready, o_full, o_free, s_ready, d_full[2],
      d_free[2], v_ready[2], mma_done[2], whole_ready;
  __shared__ __align__(16) float back[16];  // lam^(15 - j)
  __shared__ float power[129];              // lam^j
  __shared__ float from[64];                // the segments' powers at this one's start
  __shared__ float2 whole_s;                // lam^128
  // whether a chunk's v holds a value that is not finite, and each column's first such row
  __shared__ uint8_t wild[2], wild_row[2][128];
  __shared__ uint32_t tmem_base;

  // (the same in all of a warp's lanes, for the compiler too: the products' operands then
  // come straight from uniform registers)
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (first) griddep_wait();
  if (LOCAL || first) griddep_launch_dependents();
  const DecayUnit w = decay_unit(a, sp, LOCAL ? sp.S - 1 : sp.S, blockIdx.x);
  const int v0 = w.vt * 128, nv = a.dv - v0 < 128 ? a.dv - v0 : 128;
  const int va = nv > 64 ? 2 : 1;
  const int va_all = a.dv > 64 ? 2 : 1;  // the ring's, of every unit
  const uint32_t slot_bytes = da_slot(ka, va_all);
  const DaRings rings = da_rings(LOCAL, ka, va_all);
  const int k0 = rings.q, v0s = rings.q + rings.k, n_slots = v0s + rings.v;  // first places
  uint8_t *const terms = smem + n_slots * slot_bytes;
  uint8_t *const s_tile = terms + da_term_bytes(ka);
  const DecayRate rate = decay_rate(a.log_decay[w.h]);
  if (decay_grows(rate, w.len)) {
    if (!first) {
      griddep_wait();
      if (!LOCAL) griddep_launch_dependents();
    }
    if (!LOCAL && w.s == 0)
      decay_tokens<__nv_bfloat16, DA_THREADS, 128>(a, w.b, w.h, w.vt, w.len, decay_power(rate, 1),
                                                   reinterpret_cast<float *>(smem));
    return;
  }
  const int end = w.t1 < w.len ? w.t1 : w.len;
  // (LOCAL: a segment that nothing comes behind is nobody's start)
  const int chunks = end <= w.t0 || (LOCAL && w.t1 >= w.len)
                         ? 0
                         : (end - w.t0 + 127) / 128;
  constexpr int DBUF = LOCAL ? 2 : 1;  // of D (LOCAL: O's columns are free)
  const auto tokens = [&](int g) {
    const int n = end - w.t0 - 128 * g;
    return n < 128 ? n : 128;
  };

  // k, q and v (0, 1, 2) of chunk g into the place r
  const auto load = [&](int g, int what, RingAt &r) {
    const CUtensorMap *const map = what == 0 ? &mapK : what == 1 ? &mapQ : &mapV;
    const int atoms = what == 2 ? va : ka, x0 = what == 2 ? v0 : 0;
    const int head = w.h / (a.H / (what == 0 ? a.Hk : what == 1 ? a.Hq : a.Hv));
    mbar_arrive_expect_tx(&full[r.slot], DA_ATOM * (uint32_t)atoms);
#pragma unroll 1
    for (int x = 0; x < atoms; ++x)
      tma_load_4d(smem + r.slot * slot_bytes + x * DA_ATOM, map, &full[r.slot], x0 + 64 * x, head,
                  w.t0 + 128 * g, w.b);
    if (what == 0)
      r.step(k0, rings.k);
    else if (what == 1)
      r.step(0, rings.q);
    else
      r.step(v0s, rings.v);
  };

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < n_slots; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      fence_mbar_init();
      // the first chunk is on its way while the block gets ready
      RingAt rq(0), rk(k0), rv(v0s);
      if (chunks > 0) {
        load(0, 0, rk);
        if (!LOCAL) load(0, 1, rq);
        load(0, 2, rv);
      }
    } else if (lane < 3) {
      const int i = lane - 1;
      mbar_init(&x_ready[i], 4);
      mbar_init(&x_free[i], 1);
      mbar_init(&staged[i], 8);
      mbar_init(&stored[i], 1);
      mbar_init(&sc_full[i], 1);
      mbar_init(&d_full[i], 1);
      mbar_init(&v_ready[i], 5);
      mbar_init(&d_free[i], 8);
      mbar_init(&mma_done[i], 1);
      fence_mbar_init();
    } else if (lane == 3) {
      mbar_init(&qs_full, 1);
      mbar_init(&p_ready, 8);
      mbar_init(&o_full, 1);
      mbar_init(&o_free, 8);
      mbar_init(&s_ready, 8);
      mbar_init(&whole_ready, 1);
      fence_mbar_init();
    }
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + 129) {
    const int j = (int)threadIdx.x - 64;
    const float p = decay_power(rate, j);
    power[j] = p;
    if (j < 16) back[15 - j] = p;
  }
  if (!LOCAL && threadIdx.x >= 512 && (int)threadIdx.x - 512 <= w.s)
    from[threadIdx.x - 512] = decay_power(rate, w.t0 - ((int)threadIdx.x - 512) * sp.L);
  if (warp == 1) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base;
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  // After a wait that ran out a thread waits no more: it goes through its chunks without
  // (what it writes is no result), arrives where others wait, and ends.
  bool dead = false;
  const auto wait = [&](uint64_t *bar, int use, int code) {
    if (!dead && !da_wait(bar, use)) {
      record_timeout(code);
      dead = true;
    }
  };

  if (warp < DA_OUT_WARP) {
    regs_dec<DA_REG_ISSUE>();
    if (warp == 0 && lane == 0) {
      // =========================== TMA
      RingAt rq(0), rk(k0), rv(v0s);
      if (chunks > 0) {  // (the first chunk's are issued)
        if (!LOCAL) rq.step(0, rings.q);
        rk.step(k0, rings.k);
        rv.step(v0s, rings.v);
      }
      bool ok = true;
#pragma unroll 1
      for (int g = 1; ok && g < chunks; ++g) {
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
          if (LOCAL && i == 1) continue;
          RingAt r = i == 2 ? rv : i == 1 ? rq : rk;
          if (r.use > 0 && !da_wait(&empty[r.slot], r.use - 1)) {
            record_timeout(1101);
            ok = false;
            break;
          }
          load(g, i, r);
          if (i == 2)
            rv = r;
          else if (i == 1)
            rq = r;
          else
            rk = r;
        }
      }
      // the last copy issued into each place has landed
      for (int i = 0; i < n_slots; ++i) {
        const RingAt &r = i < k0 ? rq : i < v0s ? rk : rv;
        const int uses = r.use + (i < r.slot ? 1 : 0);
        if (uses > 0 && !da_wait(&full[i], uses - 1)) record_timeout(1102);
      }
    }
    // Two warps issue products, the state's (1) and the outputs' (3): either's waits are the
    // other's time.  All of a warp's lanes go through, one issues.
    if (warp == 1 || (!LOCAL && warp == 3)) {
      const bool lead = elect_one();
      const uint32_t nvc = 64u * (uint32_t)va;
      // descriptors: 16-byte steps in their low bits
      const auto slot_of = [&](const RingAt &r) { return smem_u32(smem + r.slot * slot_bytes); };
      const auto got = [&](uint64_t *bar, int use, int code) {
        if (__all_sync(0xFFFFFFFFu, da_wait(bar, use))) return true;
        if (lead) record_timeout(code);
        return false;
      };
      bool ok = true;
      if (warp == 1) {
        // =========================== D = K~^T V
        const uint32_t id_d = idesc_bf16_f32(128, nvc, true, true);
        const uint32_t lbo_k = ka == 2 ? DA_ATOM : 0;
        const uint64_t x_desc = smem_desc_sw128(smem_u32(terms), ka == 2 ? 4096 : 0, 1024);
        RingAt rk(k0), rv(v0s);
        int xn = 0;
        for (int g = 0; ok && g < chunks; ++g, rk.step(k0, rings.k), rv.step(v0s, rings.v)) {
          const int n = tokens(g);
          const uint64_t kd = smem_desc_sw128(slot_of(rk), lbo_k, 1024);
          const uint64_t vd = smem_desc_sw128(slot_of(rv), DA_ATOM, 1024);
          if ((g >= DBUF && !got(&d_free[g % DBUF], g / DBUF - 1, 1119)) ||
              !got(&full[rv.slot], rv.use, 1115))
            break;
          const uint32_t dcol = tbase + DA_COL_D - 128u * (uint32_t)(g % DBUF);
#pragma unroll 1
          for (int qt = 0; 32 * qt < n; ++qt, ++xn) {
            if (!got(&x_ready[xn & 1], xn >> 1, 1116)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t x1 = x_desc + (uint32_t)(xn & 1) * (uint32_t)ka * (2 * 4096 / 16);
            const uint64_t x2 = x1 + (uint32_t)ka * (4096 / 16);
            const uint64_t k1 = kd + (uint32_t)qt * (4096 / 16);
            const uint64_t v1 = vd + (uint32_t)qt * (4096 / 16);
            if (lead) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {  // 16 tokens
                mma_bf16_ss(dcol, x2 + 128u * i, v1 + 128u * i, id_d, (qt | i) > 0);
                mma_bf16_ss(dcol, x1 + 128u * i, v1 + 128u * i, id_d, 1);
                mma_bf16_ss(dcol, k1 + 128u * i, v1 + 128u * i, id_d, 1);
              }
              mma_commit(&x_free[xn & 1]);
            }
          }
          if (ok && lead) {
            mma_commit(&d_full[g & 1]);
            mma_commit(&empty[rk.slot]);
            if (LOCAL) mma_commit(&empty[rv.slot]);
          }
        }
        if (lead) mma_commit(&mma_done[0]);
        got(&mma_done[0], 0, 1118);
      } else {
        // =========================== Sc, Q S and P V
        const uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
        const uint32_t id_o = idesc_bf16_f32(128, nvc, false, true);
        const uint64_t s_desc = smem_desc_sw128(smem_u32(s_tile), 8192u * (uint32_t)ka, 1024);
        RingAt rq(0), rk(k0), rv(v0s);  // of the next scores, and the chunk's v
        RingAt cq(0);                   // of the chunk's q
        for (int g = -1; ok && g < chunks; ++g) {
          if (g >= 0) {
            if (!got(&s_ready, g, 1113) || (g > 0 && !got(&o_free, g - 1, 1114))) break;
            tc_fence_after();
            uint64_t qd = smem_desc_sw128(slot_of(cq), 0, 1024), sd = s_desc;
            if (lead) {
#pragma unroll
              for (int x = 0; x < ka; ++x, qd += DA_ATOM / 16, sd += 8192 / 16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 16 rows of the state
                  mma_bf16_ss(tbase + DA_COL_O, qd + 2u * i, sd + 128u * i, id_o, (x | i) > 0);
              }
              mma_commit(&qs_full);
              mma_commit(&empty[cq.slot]);
            }
            cq.step(0, rings.q);
            if (!got(&p_ready, g, 1117) || !got(&v_ready[g & 1], g >> 1, 1112)) break;
            tc_fence_after();
            const uint32_t pc = tbase + DA_COL_SC + 128u * (uint32_t)(g & 1);
            const uint64_t vd = smem_desc_sw128(slot_of(rv), DA_ATOM, 1024);
            const int steps = (tokens(g) + 15) / 16;
            if (lead) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < steps)
                  mma_bf16_ts(tbase + DA_COL_O, pc + (uint32_t)(i / 4) * 64 + (uint32_t)(i % 4) * 8,
                              vd + 128u * i, id_o, 1);
              mma_commit(&o_full);
            }
            rv.step(v0s, rings.v);
          }
          if (g + 1 == chunks) break;
          // the next scores, into the buffer whose weights the products of chunk g - 1 have
          // read (o_free of that chunk)
          if (!got(&full[rq.slot], rq.use, 1110) || !got(&full[rk.slot], rk.use, 1111)) break;
          tc_fence_after();
          uint64_t q = smem_desc_sw128(slot_of(rq), 0, 1024);
          uint64_t k = smem_desc_sw128(slot_of(rk), 0, 1024);
          const uint32_t sc = tbase + DA_COL_SC + 128u * (uint32_t)((g + 1) & 1);
          if (lead) {
#pragma unroll
            for (int x = 0; x < ka; ++x, q += DA_ATOM / 16, k += DA_ATOM / 16) {
#pragma unroll
              for (int i = 0; i < 4; ++i)  // 16 of dk: 32 bytes of the rows
                mma_bf16_ss(sc, q + 2u * i, k + 2u * i, id_sc, (x | i) > 0);
            }
            mma_commit(&sc_full[(g + 1) & 1]);
          }
          rq.step(0, rings.q);
          rk.step(k0, rings.k);
        }
        if (lead) mma_commit(&mma_done[1]);
        got(&mma_done[1], 0, 1118);
      }
    }
    if (warp == 2 && lane == 0) {  // (only the state's warps wait for it, and late)
      whole_s = decay_power2(rate, 128);
      mbar_arrive(&whole_ready);
    }
    if (!LOCAL && warp == 2) {
      __syncwarp();
      // =========================== a look at v a chunk ahead, and output stores
      // A weight of 0 keeps no infinity or NaN of a later token out of a row's sum.  So v is
      // looked through (1 or 2 % of the time; with a bounds check at every read it was 10, as
      // this warp's instructions hold up those of its quarter of the SM); where it holds one, it
      // is taken out once the state's product has had it, and the rows from there on become NaN.
      RingAt rv(v0s), ro(v0s);
      const auto got = [&](uint64_t *bar, int use, int code) {
        if (__all_sync(0xFFFFFFFFu, da_wait(bar, use))) return true;
        if (lane == 0) record_timeout(code);
        return false;
      };
      // whichever comes first, the next v or the next outputs (v two chunks ahead of them at
      // most: so many buffers has `wild`)
      int seen = 0, sent = 0;
#pragma unroll 1
      for (int turns = 0; sent < chunks; ++turns) {
        const bool look = seen < chunks && seen < sent + 2 &&
                          __all_sync(0xFFFFFFFFu, mbar_try_wait_sleep(&full[rv.slot],
                                                                      (uint32_t)rv.use & 1u, 100u));
        if (look) {
          uint8_t *const v = smem + rv.slot * slot_bytes;
          const int n = tokens(seen), buf = seen & 1;
          uint32_t sum[2] = {};
          // 32 rows of 64 columns at a time
          const uint8_t *p = v + 16 * lane;
          const auto add = [&](const uint4 &y) {
            sum[0] = fma_bf16x2(y.x, y.y, sum[0]);
            sum[1] = fma_bf16x2(y.z, y.w, sum[1]);
          };
          if (n == 128) {
#pragma unroll 1
            for (int i = 0; i < 4 * va; ++i, p += DA_ATOM / 4) {
#pragma unroll
              for (int j = 0; j < 8; ++j) add(*reinterpret_cast<const uint4 *>(p + 512 * j));
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < 4 * va; ++i, p += DA_ATOM / 4) {
              const int left = (n - 32 * (i & 3)) * 8 - lane;
#pragma unroll 1
              for (int j = 0; 32 * j < left && j < 8; ++j)
                add(*reinterpret_cast<const uint4 *>(p + 512 * j));
            }
          }
          // (or values whose products overflow: then there is nothing to take out)
          const bool any = __any_sync(0xFFFFFFFFu, wild_lo(sum[0]) || wild_hi(sum[0]) ||
                                                       wild_lo(sum[1]) || wild_hi(sum[1]));
          if (any) {
            if (!got(&d_full[buf], seen >> 1, 1152)) break;
#pragma unroll 1
            for (int x = 0; x < va; ++x) tame(v + x * DA_ATOM, n, &wild_row[buf][64 * x], lane);
            fence_proxy_async_smem();
          }
          if (lane == 0) wild[buf] = any;
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_ready[buf]);
          rv.step(v0s, rings.v);
          ++seen, turns = 0;
        }
        if (sent < seen &&
            __all_sync(0xFFFFFFFFu,
                       mbar_try_wait_sleep(&staged[sent & 1], (uint32_t)(sent >> 1) & 1u, 100u))) {
          if (lane == 0) {
            for (int x = 0; x < va; ++x)
              tma_store_4d(&mapO, smem + ro.slot * slot_bytes + x * DA_ATOM, v0 + 64 * x, w.h,
                           w.t0 + 128 * sent, w.b);
            bulk_commit_group();
            bulk_wait_group_read<0>();
            mbar_arrive(&empty[ro.slot]);
            mbar_arrive(&stored[sent & 1]);
          }
          __syncwarp();
          ro.step(v0s, rings.v);
          ++sent, turns = 0;
        } else if (turns > (1 << 23)) {
          if (lane == 0) record_timeout(1150);
          break;
        }
      }
      if (lane == 0) bulk_wait_group<0>();
    }
  } else if (!LOCAL && warp < DA_KEY_WARP) {
    // =========================== P and the outputs: a row and 64 columns a thread
    const int quad = warp & 3, half = (warp - DA_OUT_WARP) >> 2, row = quad * 32 + lane;
    const float ahead = a.scale * power[row + 1], rate_f = rate.hi;
    const uint32_t ocol = tbase + lane_off + DA_COL_O + 64u * (uint32_t)half;
    RingAt rv(v0s);
    for (int g = 0; g < chunks; ++g, rv.step(v0s, rings.v)) {
      wait(&sc_full[g & 1], g >> 1, 1120);
      __syncwarp();
      tc_fence_after();
      const uint32_t sc = tbase + lane_off + DA_COL_SC + 128u * (uint32_t)(g & 1) +
                          64u * (uint32_t)half;
      // opaque: their products would be kept for all chunks, in registers that are not there
      float rf = rate_f;
      int ln = lane;
      asm volatile("" : "+f"(rf), "+r"(ln));
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {  // 16 keys: all before the warp's rows, or on the diagonal
        const int at = 64 * half + 16 * c - 32 * quad;  // the first, from the warp's first row
        uint32_t r[16], p[8];
        if (at < 32) {
          tmem_ld16(sc + 16u * (uint32_t)c, r);
          tmem_ld_wait();
        }
        if (at < 0) {
          const float f = a.scale * power[ln - at - 15];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(&back[j]);
            const float2 f2 = make_float2(f, f);
            const float2 a2 = mul2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                   mul2(f2, make_float2(d.x, d.y)));
            const float2 b2 =
                mul2(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                     mul2(f2, make_float2(d.z, d.w)));
            p[j / 2] = pack_bf16x2(a2.x, a2.y);
            p[j / 2 + 1] = pack_bf16x2(b2.x, b2.y);
          }
        } else if (at < 32) {
          const int gap = ln - at;
#pragma unroll
          for (int j = 0; j < 16; j += 2) {  // (a power with an exponent below 0 is dropped)
            const float x = __uint_as_float(r[j]) * (a.scale * exp2_fast(rf * (float)(gap - j)));
            const float y =
                __uint_as_float(r[j + 1]) * (a.scale * exp2_fast(rf * (float)(gap - j - 1)));
            p[j / 2] = pack_bf16x2(j <= gap ? x : 0.f, j < gap ? y : 0.f);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = 0u;
        }
        tmem_st8(sc + 8u * (uint32_t)c, p);  // of 64 scores' columns the first 32
      }
      // Q S times each row's power, in place: the weights' products are added to it
      wait(&qs_full, g, 1121);
      __syncwarp();
      tc_fence_after();
      if (half < va) {
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          uint32_t r[16];
          tmem_ld16(ocol + (uint32_t)c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float2 y = mul2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                  make_float2(ahead, ahead));
            r[j] = __float_as_uint(y.x), r[j + 1] = __float_as_uint(y.y);
          }
          tmem_st16(ocol + (uint32_t)c, r);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready);

      wait(&v_ready[g & 1], g >> 1, 1133);
      const bool odd = wild[g & 1] != 0;
      wait(&o_full, g, 1130);
      __syncwarp();
      tc_fence_after();
      wait(&d_full[g & 1], g >> 1, 1132);  // D has read v too
      if (g > 1) wait(&stored[g & 1], (g >> 1) - 1, 1131);
      // Through v's place in the ring, which its products have left, and out by TMA: 32-byte
      // stores from the registers hold the SM's other shared memory traffic up (for 1800 of the
      // 10000 cycles that a chunk took with them).  Rows behind the end are zeros.
      const bool in = row < tokens(g);
      if (half < va) {
        uint8_t *const out = smem + rv.slot * slot_bytes + (uint32_t)half * DA_ATOM;
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t r[32];
          tmem_ld32(ocol + (uint32_t)c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t x =
                pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            r[j] = in ? x : 0u;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(out + sw128_offset((uint32_t)row, 2u * c + 16u * j)) =
                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        }
        if (odd && in) {
#pragma unroll 1
          for (int c = 0; c < 64; ++c)
            if (row >= wild_row[g & 1][64 * half + c])
              *reinterpret_cast<uint16_t *>(out + sw128_offset((uint32_t)row, 2u * c)) = 0x7FFFu;
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();  // the next chunk's products may take the columns
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_free);
        mbar_arrive(&staged[g & 1]);
      }
    }
  } else if (warp < DA_STATE_WARP) {
    // =========================== the keys' terms, 32 tokens at a time by four warps
    // (LOCAL: the warps that have no outputs are four more; they take turns)
    regs_dec<DA_REG_KEYS>();
    constexpr int GROUPS = LOCAL ? 2 : 1;
    const int kt = (int)threadIdx.x & 127, group = LOCAL ? (DA_STATE_WARP - 1 - warp) >> 2 : 0;
    const int r = kt >> 3, p16 = (kt & 7) * 16;  // of 16 tokens, of a row's 128 bytes
    int xn = 0;  // uses of the buffer ahead (of both, by one group)
    RingAt rk(k0), rv(v0s);
    for (int g = group < GROUPS ? 0 : chunks; g < chunks;
         ++g, rk.step(k0, rings.k), rv.step(v0s, rings.v)) {
      const int n = tokens(g);
      // the first term replaces K, which Sc has read by then
      if (!LOCAL) wait(&sc_full[g & 1], g >> 1, 1140);
      wait(&full[rk.slot], rk.use, 1141);
      uint8_t *const k = smem + rk.slot * slot_bytes;
      if (!LOCAL || n < 128) wait(&full[rv.slot], rv.use, 1142);
      if (n < 128) {  // rows behind the end are zeros, whatever they hold
        uint8_t *const v = smem + rv.slot * slot_bytes;
        for (int i = kt; group == 0 && i < (128 - n) * 8; i += 128)
          for (int x = 0; x < va; ++x)
            *reinterpret_cast<uint4 *>(v + x * DA_ATOM + n * 128 + i * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        // (of k this thread's own places)
        for (int j = r; j < 128; j += 16)
          for (int x = 0; j >= n && x < ka; ++x)
            *reinterpret_cast<uint4 *>(k + x * DA_ATOM + j * 128 + p16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (!LOCAL && lane == 0) mbar_arrive(&v_ready[g & 1]);
#pragma unroll 1
      for (int qt = group; 32 * qt < n; qt += GROUPS, ++xn) {
        const int buf = LOCAL ? group : xn & 1, use = LOCAL ? xn : xn >> 1;
        if (use > 0) wait(&x_free[buf], use - 1, 1143);
        uint8_t *const x = terms + (uint32_t)buf * 2 * (uint32_t)ka * 4096 + r * 128 + p16;
        uint8_t *const kp = k + (qt * 32 + r) * 128 + p16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 16 tokens
          const int j = qt * 32 + 16 * h + r;
          const float wj = j < n ? power[n - 1 - j] : 0.f;
          const float2 w2 = make_float2(wj, wj);
          uint4 raw[ka];
#pragma unroll
          for (int i = 0; i < ka; ++i) {
            raw[i] = *reinterpret_cast<const uint4 *>(kp + i * DA_ATOM + h * 2048);
          }
#pragma unroll
          for (int i = 0; i < ka; ++i) {
            uint4 t0, t1, t2;
            key_terms(raw[i].x, w2, t0.x, t1.x, t2.x);
            key_terms(raw[i].y, w2, t0.y, t1.y, t2.y);
            key_terms(raw[i].z, w2, t0.z, t1.z, t2.z);
            key_terms(raw[i].w, w2, t0.w, t1.w, t2.w);
            *reinterpret_cast<uint4 *>(kp + i * DA_ATOM + h * 2048) = t0;
            *reinterpret_cast<uint4 *>(x + i * 4096 + h * 2048) = t1;
            *reinterpret_cast<uint4 *>(x + (ka + i) * 4096 + h * 2048) = t2;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_ready[buf]);
      }
    }
  } else {
    // =========================== the state: row `row`, 64 columns a thread
    regs_inc<DA_REG_STATE>();
    const int sw = warp - DA_STATE_WARP, half = sw >> 2, row = (warp & 3) * 32 + lane;
    const int st = sw * 32 + lane;
    const bool mine = row < a.dk && half < va;
    float S[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) S[j] = 0.f;
    if (!first) {
      griddep_wait();
      if (!LOCAL) griddep_launch_dependents();
    }
    float4 *const own = reinterpret_cast<float4 *>(
        slots + (((size_t)w.b * a.H + w.h) * sp.nvt + w.vt) * sp.S * kDecaySlot);
    const size_t at = (((size_t)w.b * a.H + w.h) * a.dk + row) * (size_t)a.dv + v0 + 64 * half;
    const int cols = nv - 64 * half;
    if (sp.S == 1 || (LOCAL && w.s == 0)) {
      if (mine && a.state_in != nullptr) {
#pragma unroll
        for (int j = 0; j < 64; j += 4)
          if (j < cols) {
            const float4 x = *reinterpret_cast<const float4 *>(a.state_in + at + j);
            S[j] = x.x, S[j + 1] = x.y, S[j + 2] = x.z, S[j + 3] = x.w;
          }
      }
      if (LOCAL) {  // a copy: the second launch may write state_out over state_in
#pragma unroll
        for (int j = 0; j < 64; j += 4)
          own[(j / 4) * 256 + st] = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
      }
    } else if (!LOCAL && (w.s == 0 || chunks > 0)) {
      for (int s = w.s == 0 ? 0 : 1; s <= w.s; ++s) {
        const float f = from[s];
        const float4 *p = own + (size_t)s * (kDecaySlot / 4);
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 x = __ldcg(p + (j / 4) * 256 + st);
          S[j] = fmaf(f, x.x, S[j]);
          S[j + 1] = fmaf(f, x.y, S[j + 1]);
          S[j + 2] = fmaf(f, x.z, S[j + 2]);
          S[j + 3] = fmaf(f, x.w, S[j + 3]);
        }
      }
    }
    wait(&whole_ready, 0, 1146);
    const float2 whole = whole_s;
    const auto publish = [&]() {  // the operand of the next chunk's Q S
      if (row < 64 * ka && half < va) {
        uint8_t *p = s_tile + (uint32_t)(half * ka) * 8192u;
#pragma unroll
        for (int j = 0; j < 64; j += 8)
          *reinterpret_cast<uint4 *>(p + sw128_offset((uint32_t)row, 2u * (uint32_t)j)) =
              make_uint4(pack_bf16x2(S[j], S[j + 1]), pack_bf16x2(S[j + 2], S[j + 3]),
                         pack_bf16x2(S[j + 4], S[j + 5]), pack_bf16x2(S[j + 6], S[j + 7]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_ready);
    };
    if (!LOCAL && chunks > 0) publish();
    for (int g = 0; g < chunks; ++g) {
      const int n = tokens(g);
      wait(&d_full[g & 1], g >> 1, 1144);
      __syncwarp();
      tc_fence_after();
      const uint32_t dcol = tbase + lane_off + DA_COL_D - 128u * (uint32_t)(g % DBUF) +
                            64u * (uint32_t)half;
      const float2 f = n == 128 ? whole : make_float2(power[n], 0.f);
      if (half < va) {
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          uint32_t d[2][16];
          tmem_ld16(dcol + (uint32_t)(16 * c), d[0]);
          tmem_ld16(dcol + (uint32_t)(16 * c + 16), d[1]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float *const s = S + 16 * c + j;
            const float2 o = make_float2(s[0], s[1]);
            const float2 y = fma2(o, make_float2(f.x, f.x),
                                  fma2(o, make_float2(f.y, f.y),
                                       make_float2(__uint_as_float(d[j / 16][j % 16]),
                                                   __uint_as_float(d[j / 16][j % 16 + 1]))));
            s[0] = y.x, s[1] = y.y;
          }
        }
      }
      tc_fence_before();  // the next chunk's products may take D's columns
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_free[g % DBUF]);
      if (!LOCAL && g + 1 < chunks) {
        wait(&qs_full, g, 1145);  // Q S has read the tile
        __syncwarp();
        publish();
      }
    }
    if (LOCAL) {
      if (chunks > 0) {
        float4 *p = own + (size_t)(w.s + 1) * (kDecaySlot / 4);
#pragma unroll
        for (int j = 0; j < 64; j += 4)
          p[(j / 4) * 256 + st] = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
      }
    } else if (mine && a.state_out != nullptr && decay_last(w, sp.L)) {
#pragma unroll
      for (int j = 0; j < 64; j += 4)
        if (j < cols)
          *reinterpret_cast<float4 *>(a.state_out + at + j) =
              make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    }
  }
  if (!LOCAL) {
    // outputs behind the sequence's last chunk
    const int z0 = w.t0 + 128 * chunks;
    const int per = nv / 8;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) +
                       (((size_t)w.b * a.T + z0) * a.H + w.h) * (size_t)a.dv + v0;
#pragma unroll 1
    for (int r = warp; r < w.t1 - z0; r += DA_THREADS / 32)
#pragma unroll 1
      for (int i = lane; i < per; i += 32)
        *reinterpret_cast<uint4 *>(o + (size_t)r * a.H * a.dv + i * 8) = make_uint4(0u, 0u, 0u, 0u);
  }
  // the single-lane roles rejoin their warps before the block-wide barrier
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

// 4-D map over [B][T][heads][d]: boxes of 64 elements of one head of 128 tokens.
bool make_map_decay(CUtensorMap *m, const void *base, int d, int heads, int T, int B,
                    const int64_t *stride) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  // the stride of a dimension of one is any that the map takes
  const auto bytes = [](int64_t s) { return (cuuint64_t)(s == 0 ? 16 : 2 * s); };
  cuuint64_t strides[3] = {bytes(stride[2]), bytes(stride[1]), bytes(stride[0])};
  cuuint32_t box[4] = {64, 1, 128, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_tc_decay(const DecayArgs &a, void *workspace, cudaStream_t stream) {
  CUtensorMap mQ, mK, mV, mO;
  const int64_t os[3] = {(int64_t)a.T * a.H * a.dv, (int64_t)a.H * a.dv, a.dv};
  if (!make_map_decay(&mQ, a.q, a.dk, a.Hq, a.T, a.B, a.qs) ||
      !make_map_decay(&mK, a.k, a.dk, a.Hk, a.T, a.B, a.ks) ||
      !make_map_decay(&mV, a.v, a.dv, a.Hv, a.T, a.B, a.vs) ||
      !make_map_decay(&mO, a.o, a.dv, a.H, a.T, a.B, os))
    return 2;
  static OncePerDevice attrs;
  if (!attrs.run([] {
        const auto set = [](auto *kern) {
          return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)DA_SMEM + 1024) == cudaSuccess;
        };
        return set(tc_decay<true, 1>) && set(tc_decay<true, 2>) && set(tc_decay<false, 1>) &&
               set(tc_decay<false, 2>);
      }))
    return 1;
  const DecaySplit sp = decay_split_tc(a.B, a.T, a.H, a.dv);
  float *slots = static_cast<float *>(workspace);
  const int64_t heads = (int64_t)a.B * a.H * sp.nvt;
  PdlConfig cfg(stream, true);
  cfg.cfg.blockDim = dim3(DA_THREADS);
  cfg.cfg.dynamicSmemBytes = DA_SMEM + 1024;
  if (sp.S > 1) {
    cfg.cfg.gridDim = dim3((unsigned)(heads * (sp.S - 1)));
    if (cudaLaunchKernelEx(&cfg.cfg, a.dk > 64 ? tc_decay<true, 2> : tc_decay<true, 1>, mQ, mK, mV,
                           mO, a, sp, slots, 1) != cudaSuccess)
      return 1;
  }
  cfg.cfg.gridDim = dim3((unsigned)(heads * sp.S));
  return cudaLaunchKernelEx(&cfg.cfg, a.dk > 64 ? tc_decay<false, 2> : tc_decay<false, 1>, mQ, mK,
                            mV, mO, a, sp, slots, sp.S > 1 ? 0 : 1) == cudaSuccess
             ? 0
             : 1;
}

}  // namespace fmca
