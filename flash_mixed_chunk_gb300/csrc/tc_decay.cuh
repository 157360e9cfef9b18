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
//   O1 = P V,  O2 = Q S     S: the state before the chunk, rounded to bf16
//   D  = K~^T V         K~_j = lam^(n-1-j) k_j
//   o = scale (O1 + lam^(i+1) O2),   S = lam^n S + D
//
// What is rounded: P and the operand S, half a step of bf16 each, as is the output.
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
// Warps (576 threads): 0 TMA, 1 MMA issuer, 2-5 P, 6-9 outputs, 10-17 the state: K~'s
// terms from K in place (the first term) and through two buffers of 32 tokens (the
// others), then D from TMEM into the state and its bf16 copy in shared memory.  P
// takes Sc's columns; the issuer forms the next Sc when PV is through.
#pragma once

#include "decay.cuh"
#include "tc_common.cuh"

namespace fmca {
namespace {

constexpr int DA_THREADS = 576;
constexpr int DA_SLOTS = 12;             // ring slots at most
constexpr uint32_t DA_ATOM = 16384;      // 64 columns of 128 tokens
constexpr uint32_t DA_SMEM = 229376;     // ring, state, terms
constexpr uint32_t DA_COL_SC = 0, DA_COL_O1 = 128, DA_COL_O2 = 256, DA_COL_D = 384;
constexpr int DA_STATE_WARP = 10;

// Shared memory by the 64-column blocks of dk (ka) and of the unit's dv (va).
__host__ __device__ inline uint32_t da_slot(int ka, int va) {
  return DA_ATOM * (uint32_t)(ka > va ? ka : va);
}
__host__ __device__ inline uint32_t da_state_bytes(int ka, int va) {
  return 8192u * (uint32_t)(ka * va);
}
__host__ __device__ inline uint32_t da_term_bytes(int ka) { return DA_ATOM * (uint32_t)ka; }
__host__ __device__ inline int da_slots(int ka, int va) {
  const int n = (int)((DA_SMEM - da_state_bytes(ka, va) - da_term_bytes(ka)) / da_slot(ka, va));
  return n < DA_SLOTS ? n : DA_SLOTS;
}

// One 16-byte vector of keys times w as three bf16 terms.
__device__ __forceinline__ void key_terms(const uint4 &raw, float w, uint4 &t0, uint4 &t1,
                                          uint4 &t2) {
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t a[4], b[4], c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = bf16_lo(in[i]) * w, y = bf16_hi(in[i]) * w;
    a[i] = pack_bf16x2(x, y);
    x -= bf16_lo(a[i]), y -= bf16_hi(a[i]);
    b[i] = pack_bf16x2(x, y);
    x -= bf16_lo(b[i]), y -= bf16_hi(b[i]);
    c[i] = pack_bf16x2(x, y);
  }
  t0 = make_uint4(a[0], a[1], a[2], a[3]);
  t1 = make_uint4(b[0], b[1], b[2], b[3]);
  t2 = make_uint4(c[0], c[1], c[2], c[3]);
}

// first: this launch is the call's first (it waits for the work ahead; the second one
// waits for the first before it reads a state).
template <bool LOCAL>
__global__ void __launch_bounds__(DA_THREADS, 1)
    tc_decay(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
             const __grid_constant__ CUtensorMap mapV, const __grid_constant__ DecayArgs a,
             const DecaySplit sp, float *__restrict__ slots, int first) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[DA_SLOTS], empty[DA_SLOTS], x_ready[2], x_free[2];
  __shared__ __align__(8) uint64_t sc_full, p_ready, o_full, o_free, s_ready, d_full, mma_done;
  __shared__ __align__(16) float back[32];  // lam^(31 - j)
  __shared__ float power[129];              // lam^j
  __shared__ uint32_t tmem_base;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (first) griddep_wait();
  if (LOCAL || first) griddep_launch_dependents();
  const DecayUnit w = decay_unit(a, sp, LOCAL ? sp.S - 1 : sp.S, blockIdx.x);
  const int v0 = w.vt * 128, nv = a.dv - v0 < 128 ? a.dv - v0 : 128;
  const int ka = a.dk > 64 ? 2 : 1, va = nv > 64 ? 2 : 1;
  const int va_all = a.dv > 64 ? 2 : 1;  // the ring's, of every unit
  const uint32_t slot_bytes = da_slot(ka, va_all);
  const int n_slots = da_slots(ka, va_all);
  uint8_t *const s_tile = smem + n_slots * slot_bytes;
  uint8_t *const terms = s_tile + da_state_bytes(ka, va_all);
  const double rate = decay_rate(a.log_decay[w.h]);
  const int64_t end = w.t1 < w.len ? w.t1 : w.len;
  // (LOCAL: a segment that nothing comes behind is nobody's start)
  const int chunks = end <= w.t0 || (LOCAL && w.t1 >= w.len)
                         ? 0
                         : (int)((end - w.t0 + 127) / 128);
  const auto tokens = [&](int g) {
    const int64_t n = end - w.t0 - 128 * (int64_t)g;
    return n < 128 ? (int)n : 128;
  };
  constexpr int PER = LOCAL ? 2 : 3;  // ring items of a chunk: (Q,) K, V

  if (threadIdx.x == 0) {
    for (int i = 0; i < n_slots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x_ready[i], 8);
      mbar_init(&x_free[i], 1);
    }
    mbar_init(&sc_full, 1);
    mbar_init(&p_ready, 4);
    mbar_init(&o_full, 1);
    mbar_init(&o_free, 4);
    mbar_init(&s_ready, 8);
    mbar_init(&d_full, 1);
    mbar_init(&mma_done, 1);
    fence_mbar_init();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + 129) {
    const int j = (int)threadIdx.x - 64;
    const float p = decay_power(rate, j);
    power[j] = p;
    if (j < 32) back[31 - j] = p;
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base;
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  // all of a warp's lanes, or none
  const auto wait = [&](uint64_t *bar, int use, int code) {
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, (uint32_t)use & 1u, kWaitLimitNs));
    if (!ok && lane == 0) record_timeout(code);
    return ok;
  };

  if (warp == 0) {
    // =========================== TMA
    if (lane == 0) {
      if (!LOCAL) tma_prefetch_desc(&mapQ);
      tma_prefetch_desc(&mapK);
      tma_prefetch_desc(&mapV);
      const int hq = w.h / (a.H / a.Hq), hk = w.h / (a.H / a.Hk), hv = w.h / (a.H / a.Hv);
      int it = 0;
      for (int g = 0; g < chunks; ++g) {
        const int t = (int)(w.t0 + 128 * (int64_t)g);
        bool ok = true;
        for (int i = 3 - PER; i < 3; ++i, ++it) {
          const int slot = it % n_slots;
          if (it >= n_slots && !mbar_wait(&empty[slot], ((it / n_slots) - 1) & 1, kWaitLimitNs)) {
            record_timeout(1101);
            ok = false;
            break;
          }
          const int atoms = i == 2 ? va : ka;
          mbar_arrive_expect_tx(&full[slot], DA_ATOM * (uint32_t)atoms);
          for (int x = 0; x < atoms; ++x)
            tma_load_4d(smem + slot * slot_bytes + x * DA_ATOM,
                        i == 0 ? &mapQ : i == 1 ? &mapK : &mapV, &full[slot],
                        (i == 2 ? v0 : 0) + 64 * x, i == 0 ? hq : i == 1 ? hk : hv, t, w.b);
        }
        if (!ok) break;
      }
      // the last copy issued into each slot has landed
      for (int q = it > n_slots ? it - n_slots : 0; q < it; ++q)
        if (!mbar_wait(&full[q % n_slots], (q / n_slots) & 1, kWaitLimitNs)) record_timeout(1102);
    }
  } else if (warp == 1) {
    // =========================== MMA issuer
    if (lane == 0) {
      const uint32_t nvc = 64u * (uint32_t)va;
      const uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
      const uint32_t id_o = idesc_bf16_f32(128, nvc, false, true);
      const uint32_t id_d = idesc_bf16_f32(128, nvc, true, true);
      const uint32_t lbo_k = ka == 2 ? DA_ATOM : 0, lbo_x = ka == 2 ? 4096 : 0;
      const uint32_t st = smem_u32(s_tile), lbo_s = 8192u * (uint32_t)ka;
      const auto slot_of = [&](int it) { return smem_u32(smem + (it % n_slots) * slot_bytes); };
      const auto got = [&](uint64_t *bar, int use, int code) {
        if (mbar_wait(bar, (uint32_t)use & 1u, kWaitLimitNs)) return true;
        record_timeout(code);
        return false;
      };
      int xn = 0;
      for (int g = 0; g < chunks; ++g) {
        const int n = tokens(g), it0 = g * PER;
        const int ik = it0 + PER - 2, iv = it0 + PER - 1;
        const uint32_t k = slot_of(ik), v = slot_of(iv), q = slot_of(it0);
        if (!LOCAL) {
          if (!got(&full[it0 % n_slots], it0 / n_slots, 1110) ||
              !got(&full[ik % n_slots], ik / n_slots, 1111) ||
              (g > 0 && !got(&o_full, g - 1, 1112)))
            break;
          tc_fence_after();
          for (int i = 0; i < 4 * ka; ++i) {
            const uint32_t off = (uint32_t)(i / 4) * DA_ATOM + (uint32_t)(i % 4) * 32;
            mma_bf16_ss(tbase + DA_COL_SC, smem_desc_sw128(q + off, 0, 1024),
                        smem_desc_sw128(k + off, 0, 1024), id_sc, i > 0);
          }
          mma_commit(&sc_full);
          if (!got(&s_ready, g, 1113) || (g > 0 && !got(&o_free, g - 1, 1114))) break;
          tc_fence_after();
          for (int i = 0; i < 4 * ka; ++i) {
            const uint32_t off = (uint32_t)(i / 4) * DA_ATOM + (uint32_t)(i % 4) * 32;
            mma_bf16_ss(tbase + DA_COL_O2, smem_desc_sw128(q + off, 0, 1024),
                        smem_desc_sw128(st + (uint32_t)i * 2048, lbo_s, 1024), id_o, i > 0);
          }
          mma_commit(&empty[it0 % n_slots]);
        }
        if (!got(&full[iv % n_slots], iv / n_slots, 1115)) break;
        bool ok = true;
        for (int qt = 0; qt < (n + 31) / 32; ++qt, ++xn) {
          if (!got(&x_ready[xn & 1], xn >> 1, 1116)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t x = smem_u32(terms) + (uint32_t)(xn & 1) * 2 * (uint32_t)ka * 4096;
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // 16 tokens
            const uint32_t off = (uint32_t)qt * 4096 + (uint32_t)i * 2048;
            const uint64_t bd = smem_desc_sw128(v + off, DA_ATOM, 1024);
            mma_bf16_ss(tbase + DA_COL_D,
                        smem_desc_sw128(x + (uint32_t)ka * 4096 + (uint32_t)i * 2048, lbo_x, 1024),
                        bd, id_d, (qt | i) > 0);
            mma_bf16_ss(tbase + DA_COL_D, smem_desc_sw128(x + (uint32_t)i * 2048, lbo_x, 1024), bd,
                        id_d, 1);
            mma_bf16_ss(tbase + DA_COL_D, smem_desc_sw128(k + off, lbo_k, 1024), bd, id_d, 1);
          }
          mma_commit(&x_free[xn & 1]);
        }
        if (!ok) break;
        mma_commit(&d_full);
        mma_commit(&empty[ik % n_slots]);
        if (!LOCAL) {
          if (!got(&p_ready, g, 1117)) break;
          tc_fence_after();
          for (int i = 0; i < (n + 15) / 16; ++i)
            mma_bf16_ts(tbase + DA_COL_O1, tbase + DA_COL_SC + (uint32_t)i * 8,
                        smem_desc_sw128(v + (uint32_t)i * 2048, DA_ATOM, 1024), id_o, i > 0);
          mma_commit(&o_full);
        }
        mma_commit(&empty[iv % n_slots]);
      }
      mma_commit(&mma_done);
      if (!mbar_wait(&mma_done, 0, kWaitLimitNs)) record_timeout(1118);
    }
  } else if (warp < 6) {
    // =========================== P: a row of Sc a thread
    const int quad = warp & 3;
    for (int g = 0; !LOCAL && g < chunks; ++g) {
      if (!wait(&sc_full, g, 1120)) break;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {  // 64 keys
        uint32_t p[32];
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          const int c = 2 * h + c2;  // 32 keys: all before the warp's rows, or on the diagonal
          uint32_t r[32];
          if (c <= quad) {
            tmem_ld32(tbase + lane_off + DA_COL_SC + 32u * (uint32_t)c, r);
            tmem_ld_wait();
          }
          if (c < quad) {
            const float f = power[32 * (quad - c) + lane - 31];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 d = *reinterpret_cast<const float4 *>(&back[j]);
              p[16 * c2 + j / 2] = pack_bf16x2(__uint_as_float(r[j]) * (f * d.x),
                                               __uint_as_float(r[j + 1]) * (f * d.y));
              p[16 * c2 + j / 2 + 1] = pack_bf16x2(__uint_as_float(r[j + 2]) * (f * d.z),
                                                   __uint_as_float(r[j + 3]) * (f * d.w));
            }
          } else if (c == quad) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float x = j <= lane ? __uint_as_float(r[j]) * power[lane - j] : 0.f;
              const float y = j < lane ? __uint_as_float(r[j + 1]) * power[lane - j - 1] : 0.f;
              p[16 * c2 + j / 2] = pack_bf16x2(x, y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[16 * c2 + j] = 0u;
          }
        }
        tmem_st32(tbase + lane_off + DA_COL_SC + 32u * (uint32_t)h, p);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready);
    }
  } else if (warp < DA_STATE_WARP) {
    // =========================== outputs: a row a thread
    const int row = (warp & 3) * 32 + lane;
    const float ahead = power[row + 1];
    const size_t orow = (size_t)a.H * a.dv;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) +
                       (((size_t)w.b * a.T + w.t0 + row) * a.H + w.h) * (size_t)a.dv + v0;
    for (int g = 0; !LOCAL && g < chunks; ++g, o += 128 * orow) {
      if (!wait(&o_full, g, 1130)) break;
      tc_fence_after();
      const bool in = row < tokens(g);
#pragma unroll 1
      for (int c = 0; c < 64 * va; c += 32) {
        uint32_t x[32], y[32];
        tmem_ld32(tbase + lane_off + DA_COL_O1 + (uint32_t)c, x);
        tmem_ld32(tbase + lane_off + DA_COL_O2 + (uint32_t)c, y);
        tmem_ld_wait();
        if (c + 32 >= 64 * va) {  // the next chunk's products may take the columns
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = j + 2 * i;
            r[i] = pack_bf16x2(
                a.scale * fmaf(ahead, __uint_as_float(y[e]), __uint_as_float(x[e])),
                a.scale * fmaf(ahead, __uint_as_float(y[e + 1]), __uint_as_float(x[e + 1])));
          }
          if (in && c + j < nv)
            *reinterpret_cast<uint4 *>(o + c + j) = make_uint4(r[0], r[1], r[2], r[3]);
        }
      }
    }
  } else {
    // =========================== the state: row `row`, 64 columns a thread
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
        const float f = w.s == 0 ? 1.f : decay_power(rate, w.t0 - (int64_t)s * sp.L);
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
    const float2 whole = decay_power2(rate, 128);
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
    const int r = st >> 3, p16 = (st & 7) * 16;  // of 32 tokens, of a row's 128 bytes
    int xn = 0;
    for (int g = 0; g < chunks; ++g) {
      const int n = tokens(g), ik = g * PER + PER - 2, iv = ik + 1;
      // the first term replaces K, which Sc has read by then
      if ((!LOCAL && !wait(&sc_full, g, 1140)) || !wait(&full[ik % n_slots], ik / n_slots, 1141))
        break;
      uint8_t *const k = smem + (ik % n_slots) * slot_bytes;
      if (n < 128) {  // rows behind the end are zeros, whatever they hold
        if (!wait(&full[iv % n_slots], iv / n_slots, 1142)) break;
        uint8_t *const v = smem + (iv % n_slots) * slot_bytes;
        for (int i = st; i < (128 - n) * 8; i += 256)
          for (int x = 0; x < va; ++x)
            *reinterpret_cast<uint4 *>(v + x * DA_ATOM + n * 128 + i * 16) =
                make_uint4(0u, 0u, 0u, 0u);
      }
      bool ok = true;
      for (int qt = 0; qt < (n + 31) / 32; ++qt, ++xn) {
        if (xn >= 2 && !wait(&x_free[xn & 1], (xn >> 1) - 1, 1143)) {
          ok = false;
          break;
        }
        const int j = qt * 32 + r;
        uint8_t *const x = terms + (uint32_t)(xn & 1) * 2 * (uint32_t)ka * 4096 + r * 128 + p16;
        for (int i = 0; i < ka; ++i) {
          uint4 *const kp = reinterpret_cast<uint4 *>(k + i * DA_ATOM + j * 128 + p16);
          uint4 t0 = make_uint4(0u, 0u, 0u, 0u), t1 = t0, t2 = t0;
          if (j < n) key_terms(*kp, power[n - 1 - j], t0, t1, t2);
          *kp = t0;
          *reinterpret_cast<uint4 *>(x + i * 4096) = t1;
          *reinterpret_cast<uint4 *>(x + (ka + i) * 4096) = t2;
        }
        fence_proxy_async_smem();
        tc_fence_before();  // D's columns have been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_ready[xn & 1]);
      }
      if (!ok || !wait(&d_full, g, 1144)) break;
      tc_fence_after();
      const float2 f = n == 128 ? whole : make_float2(power[n], 0.f);
      if (half < va) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t d[32];
          tmem_ld32(tbase + lane_off + DA_COL_D + (uint32_t)(64 * half + 32 * c), d);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            S[32 * c + j] = fmaf(S[32 * c + j], f.x,
                                 fmaf(S[32 * c + j], f.y, __uint_as_float(d[j])));
        }
      }
      if (!LOCAL && g + 1 < chunks) publish();
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
    // outputs behind the sequence's end
    const int64_t z0 = w.t0 > w.len ? w.t0 : w.len;
    const int per = nv / 8;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) +
                       (((size_t)w.b * a.T + z0) * a.H + w.h) * (size_t)a.dv + v0;
    for (int64_t i = threadIdx.x; i < (w.t1 - z0) * per; i += DA_THREADS)
      *reinterpret_cast<uint4 *>(o + (size_t)(i / per) * a.H * a.dv + (i % per) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
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
  CUtensorMap mQ, mK, mV;
  if (!make_map_decay(&mQ, a.q, a.dk, a.Hq, a.T, a.B, a.qs) ||
      !make_map_decay(&mK, a.k, a.dk, a.Hk, a.T, a.B, a.ks) ||
      !make_map_decay(&mV, a.v, a.dv, a.Hv, a.T, a.B, a.vs))
    return 2;
  static OncePerDevice attrs;
  if (!attrs.run([] {
        return cudaFuncSetAttribute(tc_decay<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)DA_SMEM + 1024) == cudaSuccess &&
               cudaFuncSetAttribute(tc_decay<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)DA_SMEM + 1024) == cudaSuccess;
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
    if (cudaLaunchKernelEx(&cfg.cfg, tc_decay<true>, mQ, mK, mV, a, sp, slots, 1) != cudaSuccess)
      return 1;
  }
  cfg.cfg.gridDim = dim3((unsigned)(heads * sp.S));
  return cudaLaunchKernelEx(&cfg.cfg, tc_decay<false>, mQ, mK, mV, a, sp, slots,
                            sp.S > 1 ? 0 : 1) == cudaSuccess
             ? 0
             : 1;
}

}  // namespace fmca
