// beam.cu -- beam search over logits, and the reordering of states that follows it.
//
// beam_select: of the candidates (beam k, token v) of a batch element,
//
//   c[k, v] = score_k + z[k, v] - lse_k,   lse_k = log sum_v exp(z[k, v])
//
// the n largest, equal ones by the lowest k V + v.  A finished beam has one
// candidate, its score with the pad token.  Bound by the logits, read once: a warp
// holds 1024 of a row in registers, takes their maximum and sum, and keeps the row's
// n largest as one sorted list across its lanes (64-bit keys: the value in an order
// of unsigned numbers, then the complement of the index).  Within a beam the order
// of the logits is that of the candidates, so no candidate is formed before the
// last step, which compares the n best of every beam in 64 bits: in 32 the rounding
// of c would decide between beams.  One launch: a cluster of blocks is one batch
// element, and joins its lists through distributed shared memory, in a fixed order.
// Rows of one call are cut the same way, so that equal rows give equal sums and the
// tie goes to the lower beam.
//
// Measured: one element, 4 beams of 32000 in bf16, 9.3 us (2 of the launch, the rest a chain:
// a row's part, the lists of a block, of the cluster, of the beams); 64 x 8 of 50001 in fp32,
// 16 candidates, none finished, 31 us, 102 MB at 3.3 TB/s (49 % of a copy's rate): an SM with
// work issues in half of its cycles, about 20 instructions a logit, half of them to load,
// compare and sum it, half for the lists, which a warp of 12 parts of a row changes in most of
// them; and 256 blocks do not spread evenly over 152 SMs.  64 x 8 of 32000 in bf16 20 us.
//
// beam_reorder: rows of up to 16 arrays, t[b, k] = t[b, parent[b, k]] in place, one
// launch.  A thread holds its bytes of every beam that changes in registers before
// it writes the first: no second buffer, and beams that stay are neither read (but
// as somebody's parent) nor written.  Bound by the bytes: 64 rows of 4.7 MB, 448 MB read
// and written, in 67 us: 6.7 TB/s, a copy's rate.
//
// Both are programmatic dependents of what runs ahead of them on the stream and wait
// for it before they read or write.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fmca {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int E = 32;           // logits of a lane (in registers twice: these and the next)
constexpr int TASK = 32 * E;    // of a warp at a time
constexpr int kPool = 256;      // keys that a warp gathers before it sorts them
constexpr int kFew = 2;          // lanes that a warp goes through one by one
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kInf = __builtin_huge_valf();

// ---------------------------------------------------------- keys in a warp's lanes

__device__ __forceinline__ uint64_t key_of(float z, uint32_t index) {
  const uint32_t u = __float_as_uint(z + 0.f);  // -0 is 0
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

// 64-bit values in an order of unsigned numbers (comparisons of doubles go through a
// pipe of two a clock), larger than 0.
__device__ __forceinline__ uint64_t order_of(double c) {
  const uint64_t u = (uint64_t)__double_as_longlong(c + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double value_of(uint64_t o) {
  return __longlong_as_double((long long)(o >> 63 ? o & 0x7FFFFFFFFFFFFFFFull : ~o));
}

// One step of a bitonic network: lanes off apart, the larger to the lower lane
// (down) or to the upper.
template <typename K>
__device__ __forceinline__ K exchange(K k, int off, bool down, int lane) {
  const K o = __shfl_xor_sync(kAll, k, off);
  const bool larger = ((lane & off) == 0) == down;
  return larger == (o > k) ? o : k;
}
// Largest first.
template <typename K>
__device__ __forceinline__ K sort32(K k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int off = size / 2; off > 0; off /= 2)
      k = exchange(k, off, size == 32 || (lane & size) == 0, lane);
  return k;
}
// The 32 largest of two lists, largest first, each.
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b, int lane) {
  b = __shfl_sync(kAll, b, 31 - lane);
  a = a > b ? a : b;
#pragma unroll
  for (int off = 16; off > 0; off /= 2) a = exchange(a, off, true, lane);
  return a;
}

// Of two lists of (value, index), largest value and of equal ones the lowest index
// first, the 32 first, into the first list.
__device__ __forceinline__ void merge_pairs(uint64_t &c, uint64_t &at, uint64_t c2, uint64_t at2,
                                            int lane) {
  const auto ahead = [](uint64_t x, uint64_t i, uint64_t y, uint64_t j) {
    return x > y || (x == y && i < j);
  };
  c2 = __shfl_sync(kAll, c2, 31 - lane);
  at2 = __shfl_sync(kAll, at2, 31 - lane);
  if (ahead(c2, at2, c, at)) c = c2, at = at2;
#pragma unroll
  for (int off = 16; off > 0; off /= 2) {
    const uint64_t x = __shfl_xor_sync(kAll, c, off), i = __shfl_xor_sync(kAll, at, off);
    if (((lane & off) == 0) == ahead(x, i, c, at)) c = x, at = i;
  }
}

// exp(x), x <= 0 (what is under 2^-126 is 0)
__device__ __forceinline__ float exp_below(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}

// log(s) of a sum, s >= 1, to about 1e-9, where the sum itself is good to 1e-7: s = 2^e f, f
// within a half power of 1, and log f = 2 atanh z, z = (f - 1) / (f + 1), as a float, its rest
// and the series behind it.  (The double log took 1 us of the smallest call's 8, 4 of 34 at 64 x
// 8 of 50001.)
__device__ __forceinline__ double log_sum(float s) {
  const uint32_t u = __float_as_uint(s);
  int e = (int)(u >> 23) - 127;
  float f = __uint_as_float((u & 0x007FFFFFu) | 0x3F800000u);
  if (f > 1.41421356f) f *= 0.5f, ++e;
  const float n = f - 1.f, d = f + 1.f, rest = f - (d - 1.f);  // (n is exact)
  const float z = n / d;
  const float z_rest = (fmaf(-z, d, n) - z * rest) / d;
  const float y = z * z;
  const float series =
      y * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 2.f / 11, 2.f / 9), 2.f / 7), 2.f / 5), 2.f / 3);
  return fma((double)e, 0.693147180559945309,
             2.0 * (double)z + (double)fmaf(z, series, 2.f * z_rest));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// The 32 largest of `count` lists of n keys, largest first each, `stride` keys apart:
// short ones several at a time, as one sort of 32.
__device__ __forceinline__ uint64_t merge_lists(const uint64_t *lists, int count, int stride, int n,
                                                int lane) {
  uint64_t list = 0;
  const int per = n <= 8 ? 32 / n : 1;
  for (int w = 0; w < count; w += per) {
    const int at = w + lane / n;
    uint64_t o = 0;
    if (lane / n < per && at < count) o = lists[at * stride + lane % n];
    if (!__any_sync(kAll, o != 0)) continue;
    list = merge32(list, per > 1 ? sort32(o, lane) : o, lane);
  }
  return list;
}

// (maximum, sum of exp(z - maximum)) of two parts; a maximum that is -inf has
// nothing, one that is +inf or NaN makes the row's NaN.
struct Part {
  float m, s;
};
__device__ __forceinline__ Part join(const Part &a, const Part &b) {
  const float m = max_nan(a.m, b.m);
  if (m == -kInf) return Part{m, 0.f};
  return Part{m, a.s * expf(a.m - m) + b.s * expf(b.m - m)};
}

// ------------------------------------------------------------------- the logits

template <int BYTES>
struct Vec;
template <>
struct Vec<16> { using type = uint4; };
template <>
struct Vec<4> { using type = uint32_t; };
template <>
struct Vec<2> { using type = uint16_t; };

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// A lane's logits of one task, as they are in memory.  Vectors of BYTES bytes: those of
// a call, so that all its rows are cut the same way.
template <typename T, int BYTES>
struct Task {
  static constexpr int EV = BYTES / (int)sizeof(T), NV = E / EV;
  using raw_t = typename Vec<BYTES>::type;
  union Raw {
    raw_t raw;
    T v[EV];
    __device__ Raw() {}
  } r[NV];
  __device__ __forceinline__ void load(const T *__restrict__ row, int V, int t, int lane) {
    const int64_t first = (int64_t)t * TASK + lane * EV;
    const raw_t *const p = reinterpret_cast<const raw_t *>(row + first);
    if ((int64_t)(t + 1) * TASK <= V) {
#pragma unroll
      for (int j = 0; j < NV; ++j) r[j].raw = __ldg(p + j * 32);
      return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (first + j * 32 * EV < V) r[j].raw = __ldg(p + j * 32);
  }
  // -inf behind the row's end
  __device__ __forceinline__ void get(int V, int t, int lane, float (&z)[E]) const {
    if ((int64_t)(t + 1) * TASK <= V) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < EV; ++i) z[j * EV + i] = to_f(r[j].v[i]);
      return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (int64_t)t * TASK + (j * 32 + lane) * EV < V;
#pragma unroll
      for (int i = 0; i < EV; ++i) z[j * EV + i] = in ? to_f(r[j].v[i]) : -kInf;
    }
  }
};
// Index of a lane's logit i.
template <typename T, int BYTES>
__device__ __forceinline__ uint32_t index_of(int t, int lane, int i) {
  constexpr int EV = BYTES / (int)sizeof(T);
  return (uint32_t)t * TASK + ((i / EV) * 32 + lane) * EV + i % EV;
}

struct SelectArgs {
  const void *logits;
  int64_t row;  // elements between rows
  const float *scores;
  const uint8_t *finished;
  float *score;
  int64_t *parent, *token;
  int K, V, n, pad;
  int group;  // warps of a cluster that share a beam (a power of 2)
};

// Shared memory of a block, in words of 64 bits: the n keys and the part of every (beam,
// warp), the same of every (beam, block) in the cluster's first block, and the nth
// largest value of every (beam, warp) so far.
struct SelectSmem {
  int keys, parts, got, got_parts, tops, total;
};
__host__ __device__ inline SelectSmem select_smem(int K, int n) {
  SelectSmem s;
  s.keys = 0;
  s.parts = s.keys + K * kWarps * n;
  s.got = s.parts + K * kWarps;
  s.got_parts = s.got + K * kBeamCluster * n;
  s.tops = s.got_parts + K * kBeamCluster;
  s.total = s.tops + K * kWarps / 2;
  return s;
}
static_assert(kWarps * kPool >= 2 * (kWarps / 2) * 32, "half the warps' lists of pairs");

// The two halves of a barrier over the cluster's threads (those that have ended do not
// count); what was written before the first is there behind the second.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The next float above v (finite).
__device__ __forceinline__ float nextafter_up(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return __uint_as_float(u >> 31 ? u - 1 : u + 1);
}

template <typename T, int BYTES>
__global__ void __launch_bounds__(kThreads, 2)
    beam_select(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint64_t sm64[];
  __shared__ uint64_t pool[kWarps][kPool];
  const int K = a.K, n = a.n;
  const SelectSmem at = select_smem(K, n);
  uint64_t *keys = sm64 + at.keys;                               // [K][kWarps][n]
  Part *parts = reinterpret_cast<Part *>(sm64 + at.parts);       // [K][kWarps]
  uint64_t *keys_got = sm64 + at.got;                            // [K][kBeamCluster][n]
  Part *parts_got = reinterpret_cast<Part *>(sm64 + at.got_parts);  // [K][kBeamCluster]
  volatile uint32_t *tops = reinterpret_cast<uint32_t *>(sm64 + at.tops);  // [K][kWarps]

  cg::cluster_group cluster = cg::this_cluster();
  const int NC = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  cluster_arrive();  // this block's shared memory is there
  const int64_t b = blockIdx.x / NC;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int NT = (a.V - 1) / TASK + 1;
  // nothing yet
  for (int i = tid; i < K * kWarps * n; i += kThreads) keys[i] = 0;
  for (int i = tid; i < K * kWarps; i += kThreads) {
    parts[i] = Part{-kInf, 0.f};
    tops[i] = 0;
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  const float *scores = a.scores + b * K;
  const uint8_t *finished = a.finished == nullptr ? nullptr : a.finished + b * K;
  const int me = rank * kWarps + warp;
  const int groups = NC * kWarps / a.group, in_group = me % a.group;
  // the warps of this block that share a beam, and how many of its n a warp answers for
  const int near = a.group < kWarps ? a.group : kWarps, nth = (n + near - 1) / near;
  const int first = warp & ~(near - 1);

  for (int k = me / a.group; k < K; k += groups) {
    uint64_t list = 0;  // 0: no key
    Part sum{-kInf, 0.f};
    if (isfinite(scores[k]) && !(finished != nullptr && finished[k])) {
      const T *row = static_cast<const T *>(a.logits) + (b * K + k) * a.row;
      Task<T, BYTES> task;
      if (in_group < NT) task.load(row, a.V, in_group, lane);
      for (int t = in_group; t < NT; t += a.group) {
        float z[E];
        task.get(a.V, t, lane, z);
        // the next ones are on their way while these are gone through
        if (t + a.group < NT) task.load(row, a.V, t + a.group, lane);
        float top = max_nan(z[0], z[1]);
#pragma unroll
        for (int i = 2; i < E; i += 2) top = max_nan(top, z[i], z[i + 1]);
        float most = top;
#pragma unroll
        for (int off = 16; off > 0; off /= 2)
          most = max_nan(most, __shfl_xor_sync(kAll, most, off));
        const float m = max_nan(sum.m, most);
        if (!(m < kInf)) {  // NaN or +inf: this row has no candidates
          sum.m = m;
          break;
        }
        if (m == -kInf) continue;
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) add += exp_below(z[i] - m);
        sum.s = (sum.s == 0.f ? 0.f : sum.s * exp_below(sum.m - m)) + add;
        sum.m = m;

        // What may enter the list: with a full one whatever is above its last (an
        // equal value here has a higher index); before that whatever reaches the
        // n-th largest of the lanes' maxima, n of the values do.  And nothing below what
        // the block's warps of this beam have together: each its nth largest (as read at
        // any time; they only rise, and where they stand the answer does not depend on).
        const uint64_t last = __shfl_sync(kAll, list, n - 1);
        const uint32_t seen = lane < near ? tops[k * kWarps + first + lane] : 0xFFFFFFFFu;
        const uint32_t floor = __reduce_min_sync(kAll, seen);
        float v = floor != 0 ? key_value((uint64_t)floor << 32) : -kInf;
        if (last != 0 && !(v > key_value(last))) {
          v = key_value(last);
          if (!(most > v)) continue;
          v = nextafter_up(v);
        } else if (last == 0) {
          v = fmaxf(v, __shfl_sync(kAll, sort32(top, lane), n - 1));
        }
        if (most < v) continue;
        // one key into its place in the list
        const auto put = [&](uint64_t &mine, int from) {
          const uint64_t key = __shfl_sync(kAll, mine, from);
          const uint64_t up = __shfl_up_sync(kAll, list, 1);
          if (list < key) list = lane == 0 || up > key ? key : up;
        };
        // few lanes: the warp goes through each one's logits (read again: a register of a
        // place known at run time is none).  (64 x 8 of 50001: 34.3 us; 35.2 without, 35.7 with
        // up to 8 lanes.)
        const unsigned who = __ballot_sync(kAll, top >= v);
        if (last != 0 && __popc(who) <= kFew) {
          for (unsigned w = who; w != 0; w &= w - 1) {
            const uint32_t at = index_of<T, BYTES>(t, __ffs(w) - 1, lane);
            const float x = at < (uint32_t)a.V ? to_f(__ldg(row + at)) : -kInf;
            uint64_t mine = x >= v ? key_of(x, at) : 0;
            for (unsigned act = __ballot_sync(kAll, mine != 0); act != 0; act &= act - 1)
              put(mine, __ffs(act) - 1);
          }
          const uint64_t own = __shfl_sync(kAll, list, nth - 1);
          if (lane == 0) tops[k * kWarps + warp] = (uint32_t)(own >> 32);
          continue;
        }
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) mask |= z[i] >= v ? 1u << i : 0u;
        if (v == -kInf) {
#pragma unroll
          for (int i = 0; i < E; ++i) mask &= z[i] > -kInf ? ~0u : ~(1u << i);
        }
        // a lane's first that may, read again: a register of a place known at run time is
        // none
        const auto pop = [&]() -> uint64_t {
          if (mask == 0) return 0;
          const uint32_t at = index_of<T, BYTES>(t, lane, __ffs(mask) - 1);
          mask &= mask - 1;
          return key_of(to_f(__ldg(row + at)), at);
        };
        int before = __popc(mask);
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const int o = __shfl_up_sync(kAll, before, off);
          if (lane >= off) before += o;
        }
        const int count = __shfl_sync(kAll, before, 31);
        before -= __popc(mask);
        // one by one into their places (64 x 8 beams of 32000 took 24.6 us, and 26.4 sorting
        // them always)
        if (count <= 6) {
          uint64_t mine = pop();
          for (unsigned act; (act = __ballot_sync(kAll, mine != 0)) != 0;) {
            const int from = __ffs(act) - 1;
            put(mine, from);
            if (lane == from) mine = pop();
          }
        } else if (count <= kPool) {
          while (mask != 0) {
            const int to = before++;
            pool[warp][to] = pop();
          }
          __syncwarp();
          for (int i = 0; i < count; i += 32) {
            const uint64_t k1 = i + lane < count ? pool[warp][i + lane] : 0;
            list = merge32(list, sort32(k1, lane), lane);
          }
          __syncwarp();
        } else {  // many equal values, or few lanes with any
          while (__any_sync(kAll, mask != 0)) {
            const uint64_t k1 = pop();
            if (__any_sync(kAll, k1 > __shfl_sync(kAll, list, n - 1)))
              list = merge32(list, sort32(k1, lane), lane);
          }
        }
        const uint64_t own = __shfl_sync(kAll, list, nth - 1);
        if (lane == 0) tops[k * kWarps + warp] = (uint32_t)(own >> 32);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off /= 2) sum.s += __shfl_xor_sync(kAll, sum.s, off);
    if (lane < n) keys[(k * kWarps + warp) * n + lane] = list;
    if (lane == 0) parts[k * kWarps + warp] = sum;
  }
  __syncthreads();
  // the block's list of every beam, into the first block's memory
  cluster_wait();
  for (int k = warp; k < K; k += kWarps) {
    const uint64_t list = merge_lists(keys + (size_t)k * kWarps * n, kWarps, n, n, lane);
    Part sum{-kInf, 0.f};
    for (int w = 0; w < kWarps; ++w) {
      const Part p = parts[k * kWarps + w];
      if (p.m != -kInf) sum = join(sum, p);  // (else a warp without a part of this row)
    }
    if (lane < n)
      cluster.map_shared_rank(keys_got, 0)[(k * kBeamCluster + rank) * n + lane] = list;
    if (lane == 0) cluster.map_shared_rank(parts_got, 0)[k * kBeamCluster + rank] = sum;
  }
  __syncwarp();
  cluster_arrive();
  if (rank != 0) return;  // nobody reads this block's memory
  cluster_wait();
  {
    // a warp's beams: the n best of each as candidates, and of them the n best
    uint64_t best = 0, where = 0;  // a lane's place in the list, by value, then the lower index
    for (int k = warp; k < K; k += kWarps) {
      const uint64_t list = merge_lists(keys_got + (size_t)k * kBeamCluster * n, NC, n, n, lane);
      Part sum{-kInf, 0.f};
      for (int r = 0; r < NC; ++r) {
        const Part p = parts_got[k * kBeamCluster + r];
        if (p.m != -kInf) sum = join(sum, p);
      }
      uint64_t c = 0, flat = (uint64_t)k * a.V + key_index(list);
      if (finished != nullptr && finished[k]) {
        if (lane == 0 && isfinite(scores[k])) c = order_of((double)scores[k]);
        flat = (uint64_t)k * a.V + a.pad;
      } else if (list != 0 && isfinite(sum.m)) {
        c = order_of((double)scores[k] +
                     ((double)key_value(list) - ((double)sum.m + log_sum(sum.s))));
      }
      if (lane >= n) c = 0;
      merge_pairs(best, where, c, flat, lane);
    }
    // the warps' lists, pair by pair
    uint64_t *list_c = &pool[0][0], *list_at = list_c + kWarps / 2 * 32;
    for (int half = kWarps / 2; half > 0; half /= 2) {
      __syncthreads();
      if (warp >= half && warp < 2 * half) {
        list_c[(warp - half) * 32 + lane] = best;
        list_at[(warp - half) * 32 + lane] = where;
      }
      __syncthreads();
      if (warp < half)
        merge_pairs(best, where, list_c[warp * 32 + lane], list_at[warp * 32 + lane], lane);
    }
    if (warp == 0) {
      if (best != 0 && lane < n) {
        a.score[b * n + lane] = (float)value_of(best);
        a.parent[b * n + lane] = (int64_t)(where / (uint32_t)a.V);
        a.token[b * n + lane] = (int64_t)(where % (uint32_t)a.V);
      } else if (lane < n) {  // a place without a candidate
        a.score[b * n + lane] = -kInf;
        a.parent[b * n + lane] = lane % K;
        a.token[b * n + lane] = a.pad;
      }
    }
  }
}

// ------------------------------------------------------------------- reordering

struct ReorderArgs {
  BeamPiece p[kBeamPieces];
  int64_t first[kBeamPieces + 1];  // blocks ahead of each piece's
  const int64_t *parent;
  int n, K;
};

template <typename V, int KM>
__device__ __forceinline__ void reorder(char *p, int64_t row, const int *par, int K) {
  V v[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k)
    if (k < K && par[k] != k) v[k] = *reinterpret_cast<const V *>(p + par[k] * row);
#pragma unroll
  for (int k = 0; k < KM; ++k)
    if (k < K && par[k] != k) *reinterpret_cast<V *>(p + k * row) = v[k];
}

// A block is 256 vectors of one piece's rows, at all beams of one batch element.
template <int KM>
__global__ void __launch_bounds__(kThreads)
    beam_reorder(const __grid_constant__ ReorderArgs a) {
  __shared__ int par[KM];
  int i = 0;
  while (i + 1 < a.n && (int64_t)blockIdx.x >= a.first[i + 1]) ++i;
  const BeamPiece &p = a.p[i];
  const int64_t at = (int64_t)blockIdx.x - a.first[i];
  const int64_t per = (p.bytes / p.vec + kThreads - 1) / kThreads;
  const int64_t b = at / per, x = ((at % per) * kThreads + threadIdx.x) * p.vec;
  griddep_wait();
  griddep_launch_dependents();
  if ((int)threadIdx.x < a.K) {
    const int64_t q = a.parent[b * a.K + threadIdx.x];
    par[threadIdx.x] = q >= 0 && q < a.K ? (int)q : (int)threadIdx.x;
  }
  __syncthreads();
  if (x >= p.bytes) return;
  char *at0 = static_cast<char *>(p.base) + b * a.K * p.row + x;
  if (p.vec == 16)
    reorder<uint4, KM>(at0, p.row, par, a.K);
  else if (p.vec == 4)
    reorder<uint32_t, KM>(at0, p.row, par, a.K);
  else
    reorder<uint8_t, KM>(at0, p.row, par, a.K);
}

template <typename T, int BYTES>
int select(const SelectArgs &a, int B, int NC, cudaStream_t stream) {
  static OncePerDevice attrs;
  if (!attrs.run([] {
        return cudaFuncSetAttribute(beam_select<T, BYTES>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    8 * select_smem(kBeamMax, kBeamMax).total) == cudaSuccess;
      }))
    return 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)NC;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)((int64_t)B * NC));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 8 * (size_t)select_smem(a.K, a.n).total;
  return cudaLaunchKernelEx(&cfg, beam_select<T, BYTES>, a) == cudaSuccess ? 0 : 1;
}

}  // namespace

int launch_beam_select(const void *logits, int64_t row, const float *scores,
                       const uint8_t *finished, float *score, int64_t *parent, int64_t *token,
                       int B, int K, int V, int n, int pad, int bf16, cudaStream_t stream) {
  SelectArgs a{logits, row, scores, finished, score, parent, token, K, V, n, pad, 0};
  // a beam's row has NT warps' work; as many blocks as run at once (two an SM), no more
  // than have any.  (One element of 4 beams of 32000: 10.0 us on 8 blocks, 20.7 on one.)
  const int64_t NT = ((int64_t)V + TASK - 1) / TASK;
  int NC = 1;
  while (NC < kBeamCluster && (int64_t)B * 2 * NC <= 2 * 152 && NC * kWarps < NT * K) NC *= 2;
  // warps that share a beam: a warp's first task of a row costs about twice the others'
  // (its list begins).  64 x 8 beams of 32000: 24.6 us; 51.9 with one warp a beam, 35.7 with
  // all of a cluster's warps on every beam.  1 x 32 of 50000: 59.9; 86 and 178.
  int64_t least = INT64_MAX;
  for (int group = 1; group <= NC * kWarps; group *= 2) {
    const int64_t groups = NC * kWarps / group;
    const int64_t cost = (K + groups - 1) / groups * ((NT + group - 1) / group + 1);
    if (cost < least) least = cost, a.group = group;
  }
  const int el = bf16 ? 2 : 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(logits);
  const auto fits = [&](int bytes) {
    return at % bytes == 0 && ((int64_t)V * el) % bytes == 0 && (row * el) % bytes == 0;
  };
  if (bf16) {  // (64 x 8 beams of 32000: 24.6 us by 16 bytes, 25.4 by 4)
    if (fits(16)) return select<__nv_bfloat16, 16>(a, B, NC, stream);
    if (fits(4)) return select<__nv_bfloat16, 4>(a, B, NC, stream);
    return select<__nv_bfloat16, 2>(a, B, NC, stream);
  }
  return fits(16) ? select<float, 16>(a, B, NC, stream) : select<float, 4>(a, B, NC, stream);
}

int launch_beam_reorder(const BeamPiece *pieces, int n, const int64_t *parent, int B, int K,
                        cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  for (int i = 0; i < n;) {
    ReorderArgs a{};
    a.parent = parent;
    a.K = K;
    int64_t blocks = 0;
    for (; i < n && a.n < kBeamPieces; ++i) {
      BeamPiece p = pieces[i];
      if (p.bytes == 0) continue;
      const int64_t bits = (int64_t)reinterpret_cast<uintptr_t>(p.base) | p.row | p.bytes;
      p.vec = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
      const int64_t more = B * ((p.bytes / p.vec + kThreads - 1) / kThreads);
      if (blocks + more > 0x7FFFFFFF) {
        if (blocks == 0) return 1;
        break;
      }
      a.p[a.n] = p;
      a.first[a.n] = blocks;
      blocks += more;
      a.first[++a.n] = blocks;
    }
    if (a.n == 0) continue;
    cfg.gridDim = dim3((unsigned)blocks);
    auto *kern = K <= 4 ? beam_reorder<4> : K <= 8 ? beam_reorder<8> : K <= 16 ? beam_reorder<16>
                                                                            : beam_reorder<32>;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return 1;
  }
  return 0;
}

}  // namespace fmca
