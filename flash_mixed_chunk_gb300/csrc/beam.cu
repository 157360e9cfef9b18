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
// last step, which compares the n best of every beam in 64 bits.  lse comes from fp32
// sums first, good to some 1e-6; where candidates of two beams are closer than that, their
// rows are summed once more, to 2^-29, before it decides (lse_near).  One launch: a
// cluster of blocks is one batch element, and joins its lists through distributed shared
// memory, in a fixed order.  Rows of one call are cut the same way, so that equal rows
// give equal sums and the tie goes to the lower beam.
//
// Measured (calls replayed from a graph): one element, 4 beams of 32000 in bf16, 10.3 us (2 of
// the launch, the rest a chain: a row's part, the lists of a block, of the cluster, of the beams,
// 0.6 the look for close ones); 64 x 8 of 50001 in fp32, 16 candidates, a fifth of the beams
// finished, 30.0 us, 82 MB at 2.7 TB/s (41 % of a copy's rate), and 44 where an element has
// close candidates (4 of 60 inputs): an SM with work issues in 35 % of its cycles, 17
// instructions a logit, half of them to load, compare and sum it, half for the lists, which a
// warp of 12 parts of a row changes in most of them; and 256 blocks do not spread evenly over
// 152 SMs.  64 x 8 of 32000 in bf16 20.4 us, 1 x 4 of 150000 16, 1 x 32 of 50000 52.
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

#include <cmath>
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

// exp(x), x <= 2 (what is under 2^-126 is 0)
__device__ __forceinline__ float exp_below(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}

// log(s) of a sum, s >= 1/8, to about 1e-9: s = 2^e f, f within a half power of 1, and log f = 2
// atanh z, z = (f - 1) / (f + 1), as a float, its rest and the series behind it.  (The double log
// took 1 us of the smallest call's 8, 4 of 34 at 64 x 8 of 50001.)
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

// What a part of a row is measured from, m, and its sum of exp(z - m).  m is -inf where there is
// nothing yet, and +inf or NaN where the row has no candidates; else the largest logit so far is
// between m and m + kSlack.
struct Part {
  float m, s;
};
constexpr float kSlack = 2.f;
// Eight lanes' parts as one, in each of them: one factor for each, and the sums as a tree.
__device__ __forceinline__ Part join8(const Part &p) {
  float m = p.m;
#pragma unroll
  for (int off = 4; off > 0; off /= 2) m = max_nan(m, __shfl_xor_sync(kAll, m, off));
  float s = p.m == -kInf ? 0.f : p.s * expf(p.m - m);
#pragma unroll
  for (int off = 4; off > 0; off /= 2) s += __shfl_xor_sync(kAll, s, off);
  return Part{m, s};
}
static_assert(kWarps == 8 && kBeamCluster == 8, "parts that join8 joins");

// s + x as a sum of two floats, the rest added to `rest`.
__device__ __forceinline__ void add2(float &s, float &rest, float x) {
  const float t = s + x, y = t - s;
  rest += (s - (t - y)) + (x - y);
  s = t;
}
// exp(z - m) of N logits from AT on, as a tree (one after the other, equal terms would all be
// rounded to the same side).
template <int AT, int N>
__device__ __forceinline__ float sum_exp(const float (&z)[E], float m) {
  if constexpr (N == 1)
    return exp_below(z[AT] - m);
  else
    return sum_exp<AT, N / 2>(z, m) + sum_exp<AT + N / 2, N / 2>(z, m);
}

// How far a row's log sum of exponentials may be off, and what is done about it.  In u = 2^-24:
// of a term the difference z - m, its product with log2(e) and that constant 2.22 |z - m|, and
// ex2.approx 4; where m moves, by more than kSlack, 5 for the factor.  By its share of the sum a
// row's term lies ln V under the maximum at most, on average (the entropy is at most ln V, and
// the sum at least its largest term), so these are 2.22 (ln V + 6) + 4 + 5 (ln V / 2 + 2).  The
// tree of a task 5, the tasks as two floats 1, the lanes 6, the joins of warps and of blocks 6.4
// each.  In all under (54 + 5 ln V) u, 6.5e-6 at 50000.
// That is too much between beams: candidates of different ones may lie closer.  So where two that
// matter are within twice as much of each other, their beams' rows are summed again, to 2^-29
// (exact_sum).
inline double lse_near(int V) { return 2.0 * (54.0 + 5.0 * log((double)V)) / (1 << 24); }

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
  double near;  // candidates of different beams that are closer may be in the wrong order
};

// sum exp(z - m) to 2^-29 over the logits from `first` on, `step` apart: exp(x) = 2^(N / 64)
// exp(r), N = rint(64 x / ln 2), with x = z - m and r = x - N ln(2) / 64 as sums of two floats,
// the powers from a table of two floats, the sum in two floats.  What is off: r by 2^-31, as p =
// exp(r) - 1 and the power's product with it are.  m: within kSlack under the row's maximum.
// (About 45 instructions a logit.)
template <typename T>
__device__ __forceinline__ double exact_sum(const T *__restrict__ row, int V, int first, int step,
                                            float m, const float2 *powers) {
  constexpr float kN = 92.3324826f, kA = 1420.f / 131072, kB = -3.3155381258556e-06f;
  constexpr int U = 8;  // logits on their way while as many are gone through
  float next[U], s = 0.f, rest = 0.f;
  const auto load = [&](int64_t at) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      next[u] = at + u * step < V ? to_f(__ldg(row + at + u * step)) : -kInf;
  };
  load(first);
  for (int64_t i = first; i < V; i += U * step) {
    float z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) z[u] = next[u];
    load(i + U * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float d = z[u] - m, y = d - z[u], x = fmaxf(d, -60.f);  // 2^-86 of the sum: nothing
      const float x_rest = d > -60.f ? (z[u] - (d - y)) - (m + y) : 0.f;
      const float n = rintf(x * kN);
      const float r = fmaf(-n, kB, fmaf(-n, kA, x)) + x_rest;  // (n kA has 24 bits)
      const float p = fmaf(r * r, fmaf(r, fmaf(r, 1.f / 24, 1.f / 6), 0.5f), r);
      const int k = (int)n;
      const float2 w = powers[k & 63];
      const float up = __int_as_float(((k >> 6) + 127) << 23);
      const float hi = w.x * up, lo = fmaf(w.x, p, w.y) * up, term = hi + lo;
      add2(s, rest, term);
      rest += lo - (term - hi);
    }
  }
  return (double)s + (double)rest;
}

// The two halves of a barrier over the cluster's threads (those that have ended do not
// count); what was written before the first is there behind the second.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The log sums of the beams in `which`, again and to 2^-29, by all blocks of the cluster (behind
// a barrier of theirs): into the first one's lse.  mem: 7 kPool words of every block's shared
// memory.  Out of line: in it, the kernel's main path was 0.9 to 2.8 us longer.
template <typename T>
__device__ __noinline__ void settle(const SelectArgs &a, int64_t b, unsigned which,
                                    const float *from, double *lse, uint64_t *mem, int rank,
                                    int NC) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  double *const sums = reinterpret_cast<double *>(mem);  // [K][kBeamCluster], the first block's
  double *const part = sums + kBeamMax * kBeamCluster;   // the warps'
  float2 *const powers = reinterpret_cast<float2 *>(part + kWarps);
  static_assert(kBeamMax * kBeamCluster + kWarps + 64 <= (kWarps - 1) * kPool, "mem");
  if (tid < 64) {
    const double p = exp2((double)tid / 64);
    powers[tid] = make_float2((float)p, (float)(p - (double)(float)p));
  }
  __syncthreads();
  for (unsigned w = which; w != 0; w &= w - 1) {
    const int k = __ffs(w) - 1;
    const T *row = static_cast<const T *>(a.logits) + (b * a.K + k) * a.row;
    double sum = exact_sum<T>(row, a.V, rank * kThreads + tid, NC * kThreads, from[k], powers);
#pragma unroll
    for (int off = 16; off > 0; off /= 2) sum += __shfl_xor_sync(kAll, sum, off);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      sum = 0.0;
      for (int i = 0; i < kWarps; ++i) sum += part[i];
      cg::this_cluster().map_shared_rank(sums, 0)[k * kBeamCluster + rank] = sum;
    }
    __syncthreads();
  }
  cluster_arrive();
  if (rank != 0) return;
  cluster_wait();
  if (tid < a.K && which >> tid & 1) {
    double sum = 0.0;
    for (int r = 0; r < NC; ++r) sum += sums[tid * kBeamCluster + r];
    lse[tid] = (double)from[tid] + log(sum);
  }
  __syncthreads();
}

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
  // what the end needs of every beam: its log sum and what its row is measured from; the beams
  // whose order is not sure, the values that are as close as that to the last place's, its beam
  __shared__ double lse[kBeamMax];
  __shared__ float from[kBeamMax];
  __shared__ unsigned unsure;
  __shared__ uint64_t border[2];
  __shared__ int border_beam;
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
  if (tid == 0) unsure = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  const float *scores = a.scores + b * K;
  const unsigned finished =
      a.finished == nullptr ? 0 : __ballot_sync(kAll, lane < K && a.finished[b * K + lane]);
  const int me = rank * kWarps + warp;
  const int groups = NC * kWarps / a.group, in_group = me % a.group;
  // the warps of this block that share a beam, and how many of its n a warp answers for
  const int near = a.group < kWarps ? a.group : kWarps, nth = (n + near - 1) / near;
  const int first = warp & ~(near - 1);

  for (int k = me / a.group; k < K; k += groups) {
    uint64_t list = 0;  // 0: no key
    float m = -kInf, s = 0.f, rest = 0.f;
    if (isfinite(scores[k]) && !(finished >> k & 1)) {
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
        const float high = max_nan(m, most);
        if (!(high < kInf)) {  // NaN or +inf: this row has no candidates
          m = high;
          break;
        }
        if (high == -kInf) continue;
        if (high > m + kSlack) {
          const float f = exp_below(m - high);
          s = __fmul_rn(s, f), rest = __fmul_rn(rest, f);
          m = high;
        }
        add2(s, rest, sum_exp<0, E>(z, m));

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
        // place known at run time is none).  (64 x 8 of 50001, 16 candidates: 32.1 us; 33.1
        // without, 33.7 with up to 8 lanes.  1 x 32 of 50000: 51.2; 53.6 and 52.8.  1 x 4: alike.)
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
        // one by one into their places (64 x 8 beams of 50001 32.1 us, 32.5 sorting them
        // always; of 32000 in bf16 20.1 and 20.5; 1 x 4 alike)
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
    s += rest;
#pragma unroll
    for (int off = 16; off > 0; off /= 2) s += __shfl_xor_sync(kAll, s, off);
    if (lane < n) keys[(k * kWarps + warp) * n + lane] = list;
    if (lane == 0) parts[k * kWarps + warp] = Part{m, s};
  }
  __syncthreads();
  // the block's list of every beam, into the first block's memory
  cluster_wait();
  for (int k = warp; k < K; k += kWarps) {
    const uint64_t list = merge_lists(keys + (size_t)k * kWarps * n, kWarps, n, n, lane);
    const Part sum = join8(parts[k * kWarps + lane % kWarps]);
    if (lane < n)
      cluster.map_shared_rank(keys_got, 0)[(k * kBeamCluster + rank) * n + lane] = list;
    if (lane == 0) cluster.map_shared_rank(parts_got, 0)[k * kBeamCluster + rank] = sum;
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  // The first block joins the lists.  The others wait to hear that nothing is unsure, or help.
  uint64_t *const lists = keys, *const found = keys + K * n;  // [K][n] each: keys, candidates
  if (rank == 0) {
    for (int k = warp; k < K; k += kWarps) {
      const uint64_t list = merge_lists(keys_got + (size_t)k * kBeamCluster * n, NC, n, n, lane);
      const Part sum =
          join8(lane % 8 < NC ? parts_got[k * kBeamCluster + lane % 8] : Part{-kInf, 0.f});
      if (lane < n) lists[k * n + lane] = isfinite(sum.m) ? list : 0;
      if (lane == 0) {
        lse[k] = (double)sum.m + log_sum(sum.s);
        from[k] = sum.m;
      }
    }
    __syncwarp();
  }
  for (bool again = false;; again = true) {
    uint64_t best = 0, where = 0;  // a lane's place in the list, by value, then the lower index
    int beam = 0;                  // (of it, in the first warp)
    if (rank == 0) {
      // a warp's beams: the n best of each as candidates, and of them the n best
      for (int k = warp; k < K; k += kWarps) {
        const uint64_t list = lane < n ? lists[k * n + lane] : 0;
        uint64_t c = 0, flat = (uint64_t)k * a.V + key_index(list);
        if (finished >> k & 1) {
          if (lane == 0 && isfinite(scores[k])) c = order_of((double)scores[k]);
          flat = (uint64_t)k * a.V + a.pad;
        } else if (list != 0) {
          c = order_of((double)scores[k] + ((double)key_value(list) - lse[k]));
        }
        if (lane < n) found[k * n + lane] = c;
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
      if (warp == 0) beam = (int)(where / (uint32_t)a.V);
      if (!again && K > 1) {
        // Neighbours of different beams in the list that are too close, and candidates of other
        // beams that are too close to its last: both beams are unsure.  (Whatever else could
        // change places has such a pair between.)
        if (warp == 0) {
          const double c = value_of(best);
          const uint64_t least = order_of(c - a.near), next = __shfl_down_sync(kAll, best, 1);
          const int beam2 = __shfl_down_sync(kAll, beam, 1);
          unsigned mask = 0;
          if (lane + 1 < n && next != 0 && beam != beam2 && next >= least)
            mask = (1u << beam | 1u << beam2) & ~finished;
          mask = __reduce_or_sync(kAll, mask);
          if (lane == 0) unsure = mask;
          if (lane == n - 1) {
            border[0] = least, border[1] = order_of(c + a.near);
            border_beam = best != 0 ? beam : -1;  // an empty place: nothing is left out
          }
        }
        __syncthreads();
        unsigned mask = unsure;
        if (border_beam >= 0 && lane < n)
          for (int k = warp; k < K; k += kWarps) {
            const uint64_t c = found[k * n + lane];
            if (k != border_beam && c >= border[0] && c <= border[1])
              mask |= (1u << k | 1u << border_beam) & ~finished;
          }
        if (__syncthreads_or((int)mask)) {
          if (mask != 0) atomicOr(&unsure, mask);
          __syncthreads();
          for (int i = tid; i < NC * K; i += kThreads) {
            if (i % K == 0) *cluster.map_shared_rank(&unsure, i / K) = unsure;
            cluster.map_shared_rank(from, i / K)[i % K] = from[i % K];
          }
        }
      }
    }
    if (!again) {
      __syncwarp();
      cluster_arrive();
      if (rank != 0) cluster_wait();
      if (unsure != 0) {
        if (rank == 0) cluster_wait();
        settle<T>(a, b, unsure, from, lse, &pool[1][0], rank, NC);
        if (rank != 0) return;
        continue;
      }
      if (rank != 0) return;
    }
    if (warp == 0) {
      if (best != 0 && lane < n) {
        a.score[b * n + lane] = (float)value_of(best);
        a.parent[b * n + lane] = beam;
        a.token[b * n + lane] = (int64_t)(where - (uint64_t)beam * a.V);
      } else if (lane < n) {  // a place without a candidate
        a.score[b * n + lane] = -kInf;
        a.parent[b * n + lane] = lane % K;
        a.token[b * n + lane] = a.pad;
      }
    }
    return;
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
  SelectArgs a{logits, row, scores, finished, score, parent, token, K, V, n, pad, 0,
               lse_near(V)};
  // a beam's row has NT warps' work; as many blocks as run at once (two an SM), no more
  // than have any.  (One element of 4 beams of 32000: 10.1 us on 8 blocks, 20.0 on one; 64 x 8
  // 20.1 on 4 blocks each, 37.5 on one.)
  const int64_t NT = ((int64_t)V + TASK - 1) / TASK;
  int NC = 1;
  while (NC < kBeamCluster && (int64_t)B * 2 * NC <= 2 * 152 && NC * kWarps < NT * K) NC *= 2;
  // warps that share a beam: a warp's first task of a row costs about twice the others'
  // (its list begins).  64 x 8 beams of 32000: 20.1 us; 45.3 with one warp a beam, 30.2 with
  // all of a cluster's warps on every beam.  1 x 32 of 50000: 51.2; 77 and 172.
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
  if (bf16) {  // (64 x 8 beams of 32000: 20.1 us by 16 bytes, 20.6 by 4)
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
