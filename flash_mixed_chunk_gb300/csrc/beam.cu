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
// beam_reorder: rows of up to 16 arrays, t[b, k] = t[b, parent[b, k]] in place, one
// launch.  A thread holds its bytes of every beam that changes in registers before
// it writes the first: no second buffer, and beams that stay are neither read (but
// as somebody's parent) nor written.
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
constexpr int E = 32;           // logits of a lane
constexpr int TASK = 32 * E;    // of a warp at a time
constexpr int kPool = 128;      // keys that a warp gathers before it sorts them
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

__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
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

// A lane's logits of one task; -inf behind the row's end.  Vectors of BYTES bytes:
// those of a call, so that all its rows are cut the same way.
template <typename T, int BYTES>
__device__ __forceinline__ void load_task(const T *__restrict__ row, int V, int t, int lane,
                                          float (&z)[E]) {
  constexpr int EV = BYTES / (int)sizeof(T), NV = E / EV;
  using raw_t = typename Vec<BYTES>::type;
  union Raw {
    raw_t raw;
    T v[EV];
    __device__ Raw() {}
  } r[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t at = (int64_t)t * TASK + (j * 32 + lane) * EV;
    if (at < V) r[j].raw = __ldg(reinterpret_cast<const raw_t *>(row + at));
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = (int64_t)t * TASK + (j * 32 + lane) * EV < V;
#pragma unroll
    for (int i = 0; i < EV; ++i) z[j * EV + i] = in ? to_f(r[j].v[i]) : -kInf;
  }
}
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

// Shared memory of a block: the n keys and the part of every (beam, warp), and the
// same of every beam joined over the block's warps.
__host__ __device__ inline size_t select_smem(int K, int n) {
  return (size_t)K * (kWarps + 1) * (8 * (size_t)n + 8);
}

template <typename T, int BYTES>
__global__ void __launch_bounds__(kThreads)
    beam_select(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint64_t sm64[];
  __shared__ uint64_t pool[kWarps][kPool];
  const int K = a.K, n = a.n;
  uint64_t *keys = sm64;                                        // [K][kWarps][n]
  uint64_t *keys_all = keys + (size_t)K * kWarps * n;           // [K][n]
  Part *parts = reinterpret_cast<Part *>(keys_all + (size_t)K * n);  // [K][kWarps]
  Part *part_all = parts + K * kWarps;                          // [K]

  cg::cluster_group cluster = cg::this_cluster();
  const int NC = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / NC;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int NT = (a.V + TASK - 1) / TASK;
  griddep_wait();
  griddep_launch_dependents();

  const float *scores = a.scores + b * K;
  const uint8_t *finished = a.finished == nullptr ? nullptr : a.finished + b * K;
  const int all = NC * kWarps, me = rank * kWarps + warp;
  const int groups = all / a.group, in_group = me % a.group;

  for (int k = 0; k < K; ++k) {
    uint64_t list = 0;  // 0: no key
    Part sum{-kInf, 0.f};
    const bool on = isfinite(scores[k]) && !(finished != nullptr && finished[k]) &&
                    k % groups == me / a.group;
    if (on) {
      const T *row = static_cast<const T *>(a.logits) + (b * K + k) * a.row;
      for (int t = in_group; t < NT; t += a.group) {
        float z[E];
        load_task<T, BYTES>(row, a.V, t, lane, z);
        float top = z[0];
#pragma unroll
        for (int i = 1; i < E; ++i) top = max_nan(top, z[i]);
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
        for (int i = 0; i < E; ++i) add += __expf(z[i] - m);
        sum.s = (sum.s == 0.f ? 0.f : sum.s * __expf(sum.m - m)) + add;
        sum.m = m;

        // What may enter the list: with a full one whatever is above its last (an
        // equal value here has a higher index); before that whatever reaches the
        // n-th largest of the lanes' maxima, n of the values do.
        const uint64_t last = __shfl_sync(kAll, list, n - 1);
        uint32_t mask = 0;
        if (last != 0) {
          const float v = key_value(last);
          if (!(most > v)) continue;
#pragma unroll
          for (int i = 0; i < E; ++i) mask |= z[i] > v ? 1u << i : 0u;
        } else {
          const float v = __shfl_sync(kAll, sort32(top, lane), n - 1);
#pragma unroll
          for (int i = 0; i < E; ++i) mask |= z[i] >= v && z[i] > -kInf ? 1u << i : 0u;
        }
        int before = __popc(mask);
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const int o = __shfl_up_sync(kAll, before, off);
          if (lane >= off) before += o;
        }
        const int count = __shfl_sync(kAll, before, 31);
        before -= __popc(mask);
        if (count <= kPool) {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (mask >> i & 1) pool[warp][before++] = key_of(z[i], index_of<T, BYTES>(t, lane, i));
          __syncwarp();
          for (int i = 0; i < count; i += 32) {
            const uint64_t k1 = i + lane < count ? pool[warp][i + lane] : 0;
            list = merge32(list, sort32(k1, lane), lane);
          }
          __syncwarp();
        } else {  // many equal values, or few lanes with any
#pragma unroll 1
          for (int i = 0; i < E; ++i) {
            float v = -kInf;
#pragma unroll
            for (int j = 0; j < E; ++j) v = i == j ? z[j] : v;
            const uint64_t k1 = mask >> i & 1 ? key_of(v, index_of<T, BYTES>(t, lane, i)) : 0;
            if (__any_sync(kAll, k1 > __shfl_sync(kAll, list, n - 1)))
              list = merge32(list, sort32(k1, lane), lane);
          }
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off /= 2) sum.s += __shfl_xor_sync(kAll, sum.s, off);
    if (lane < n) keys[(k * kWarps + warp) * n + lane] = list;
    if (lane == 0) parts[k * kWarps + warp] = sum;
  }
  __syncthreads();
  for (int k = warp; k < K; k += kWarps) {
    uint64_t list = 0;
    Part sum{-kInf, 0.f};
    for (int w = 0; w < kWarps; ++w) {
      const uint64_t o = lane < n ? keys[(k * kWarps + w) * n + lane] : 0;
      if (__any_sync(kAll, o != 0)) list = merge32(list, o, lane);
      sum = join(sum, parts[k * kWarps + w]);
    }
    if (lane < n) keys_all[k * n + lane] = list;
    if (lane == 0) part_all[k] = sum;
  }
  cluster.sync();
  if (rank == 0) {
    // the n best of every beam as candidates, over the lists of the block's warps
    double *cand = reinterpret_cast<double *>(keys);  // [K][n]
    int64_t *flat = reinterpret_cast<int64_t *>(keys + (size_t)K * n);
    for (int k = warp; k < K; k += kWarps) {
      uint64_t list = 0;
      Part sum{-kInf, 0.f};
      for (int r = 0; r < NC; ++r) {
        const uint64_t *o = cluster.map_shared_rank(keys_all, r);
        const Part *p = cluster.map_shared_rank(part_all, r);
        list = merge32(list, lane < n ? o[k * n + lane] : 0, lane);
        sum = join(sum, p[k]);
      }
      const double score = (double)scores[k];
      bool some = list != 0 && isfinite(sum.m);
      double c = some ? score + ((double)key_value(list) - ((double)sum.m + log((double)sum.s)))
                      : 0.0;
      uint32_t token = key_index(list);
      if (isfinite(scores[k]) && finished != nullptr && finished[k]) {
        some = lane == 0;
        c = score;
        token = (uint32_t)a.pad;
      }
      if (lane < n) {
        cand[k * n + lane] = c;
        flat[k * n + lane] = some ? (int64_t)k * a.V + token : -1;
      }
    }
    __syncthreads();
    int some = 0;
    for (int i = tid; i < K * n; i += kThreads) {
      const int64_t f = flat[i];
      if (f < 0) continue;
      ++some;
      const double c = cand[i];
      int better = 0;
      for (int j = 0; j < K * n; ++j)
        better += flat[j] >= 0 && (cand[j] > c || (cand[j] == c && flat[j] < f)) ? 1 : 0;
      if (better < n) {
        a.score[b * n + better] = (float)c;
        a.parent[b * n + better] = f / a.V;
        a.token[b * n + better] = f % a.V;
      }
    }
    // places without a candidate
    int *count = reinterpret_cast<int *>(pool);
    if (tid == 0) *count = 0;
    __syncthreads();
    if (some > 0) atomicAdd(count, some);
    __syncthreads();
    for (int i = *count + tid; i < n; i += kThreads) {
      a.score[b * n + i] = -kInf;
      a.parent[b * n + i] = i % K;
      a.token[b * n + i] = a.pad;
    }
  }
  cluster.sync();  // the other blocks' lists stay until they are read
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
                                    (int)select_smem(kBeamMax, kBeamMax)) == cudaSuccess;
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
  cfg.dynamicSmemBytes = select_smem(a.K, a.n);
  return cudaLaunchKernelEx(&cfg, beam_select<T, BYTES>, a) == cudaSuccess ? 0 : 1;
}

}  // namespace

int launch_beam_select(const void *logits, int64_t row, const float *scores,
                       const uint8_t *finished, float *score, int64_t *parent, int64_t *token,
                       int B, int K, int V, int n, int pad, int bf16, cudaStream_t stream) {
  SelectArgs a{logits, row, scores, finished, score, parent, token, K, V, n, pad, 0};
  // a beam's row has NT warps' work; as many blocks as give about 24 warps an SM,
  // no more than have any
  const int64_t NT = ((int64_t)V + TASK - 1) / TASK;
  int NC = 1;
  while (NC < kBeamCluster && (int64_t)B * NC * kWarps < 24 * 152 && NC * kWarps < NT * K) NC *= 2;
  int group = 1;
  while (group < NC * kWarps && group < NT) group *= 2;
  a.group = group;
  const int el = bf16 ? 2 : 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(logits);
  const auto fits = [&](int bytes) {
    return at % bytes == 0 && ((int64_t)V * el) % bytes == 0 && (row * el) % bytes == 0;
  };
  if (bf16) {
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
