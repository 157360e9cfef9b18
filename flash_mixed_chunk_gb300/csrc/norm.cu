// norm.cu -- layer norm of the residual stream around a GAU layer, forward and
// backward, for rows [M][d]:
//
//   h = x + r (rounded to the I/O type and stored; without r, h = x)
//   mean = sum_j h_j / d,  var = sum_j (h_j - mean)^2 / d,  rstd = (var + eps)^-1/2
//   xhat = (h - mean) rstd,  y = xhat w + b
//
//   t = dy w,  dx = rstd (t - mean_j t - xhat mean_j (t xhat)) + dh
//   dw = sum_rows dy xhat,  db = sum_rows dy
//
// Bound by the bytes: a forward row is read once and written once (with a
// residual branch two reads, two writes), so a row lives in registers from its
// load to its store and the variance is the two-pass one (deviations from the
// mean, no difference of large squares).  All arithmetic is fp32; h is rounded
// before its statistics are taken, so that the backward pass, which reads the
// stored h, differentiates exactly what the forward pass normalised.
//
// A row belongs to one warp (d <= 1024) or to one block of 256 threads (d <=
// 8192): 8, 16, 24 or 32 elements a thread, in 16-byte vectors where d allows
// it, else 4-byte ones, else single elements.  Rows that would fill a warp's
// registers (and, backward, its shared memory) with few threads at work (fp32
// beyond 512 elements, narrow vectors beyond 256) belong to half a block or (up
// to 512) a quarter: 5001 fp32 rows of 1001 take 16.5 us backward (34.6 with a
// warp a row) and 10.9 forward (14.3), 9001 of 301 11.4 (14.2); forward the short
// ones of many rows would be better off with a warp (9001 of 301: 7.2 and 6.2,
// 300 rows 2.1 and 2.4).  Backward, bf16 rows in 16-byte vectors have three warps
// from 513 elements on and four from 769 (norm_wide), and fp32 rows and rows of
// pairs of bf16 512 threads from 2049 to 4096 (norm_long_held).
//
// Times in this file: calls in a captured loop over three sets of inputs, the
// backward pass with both its launches; rows with a residual branch (backward: its
// gradient), but for the fp32 rows of 1001 and the 9001 of 301 just above, which
// have none.
//
// Every kernel is a programmatic dependent of what runs ahead of it on the
// stream: its blocks are on their way while that ends, and read nothing before
// the grid wait (a pass forward and backward of 4096 x 768, calls queued one by
// one: 20.7 us, so 15.0; captured the same either way).
//
// The backward pass keeps dw and db of the rows it has seen in registers, one
// partial row a block in the workspace, and a second kernel adds the partial
// rows in a fixed order (no atomics: the same bits every time).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fmca {
namespace {

constexpr int kNormThreads = 256;
constexpr size_t kNormMaxSmem = 200 << 10;  // of a block of the backward pass
constexpr size_t kNormSmSmem = 220 << 10;   // of an SM's blocks

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, int VEC>
struct Pack {
  using raw_t = typename Raw<(int)sizeof(T) * VEC>::type;
  union {
    raw_t raw;
    T v[VEC];
  };
  __device__ Pack() {}
};

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *in) {
  Pack<T, VEC> k;
#pragma unroll
  for (int i = 0; i < VEC; ++i) k.v[i] = from_f<T>(in[i]);
  *reinterpret_cast<typename Pack<T, VEC>::raw_t *>(p) = k.raw;
}
// VEC fp32 weights (column offset a multiple of VEC)
template <int VEC>
__device__ __forceinline__ void load_w(const float *__restrict__ p, float *out) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + i);
      out[4 * i] = v.x, out[4 * i + 1] = v.y, out[4 * i + 2] = v.z, out[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = __ldg(p + i);
  }
}

// The sums of a.x and a.y over the threads of a row's group: a warp, some warps
// of a block or the block (two sets of shared words in turn, so that one barrier
// a sum is enough; some warps meet at a barrier of their own).
template <int GROUP, int THREADS>
__device__ __forceinline__ void group_sync() {
  if constexpr (GROUP == 32)
    __syncwarp();
  else if constexpr (GROUP == THREADS)
    __syncthreads();
  else
    named_bar_sync(1 + threadIdx.x / GROUP, GROUP);
}
template <int GROUP, int THREADS>
__device__ __forceinline__ float2 group_sum2(float2 a, float2 (*red)[THREADS / 32], int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
  }
  if constexpr (GROUP > 32) {
    float2 *r = red[turn];
    turn ^= 1;
    if (threadIdx.x % 32 == 0) r[threadIdx.x / 32] = a;
    const int grp = threadIdx.x / GROUP;
    group_sync<GROUP, THREADS>();
    a = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < GROUP / 32; ++i) {
      const float2 v = r[grp * (GROUP / 32) + i];
      a.x += v.x;
      a.y += v.y;
    }
  }
  return a;
}
template <int GROUP>
__device__ __forceinline__ float group_sum(float v, float2 (*red)[kNormThreads / 32], int &turn) {
  return group_sum2<GROUP, kNormThreads>(make_float2(v, 0.f), red, turn).x;
}

// T: I/O type; VEC elements a vector, N vectors a thread; GROUP threads a row.
template <typename T, int VEC, int N, int GROUP>
__global__ void __launch_bounds__(kNormThreads)
    norm_forward(const T *x, const T *res, const float *__restrict__ weight,
                 const float *__restrict__ bias, T *h, T *__restrict__ y,
                 float *__restrict__ mean_out, float *__restrict__ rstd_out, int M, int d,
                 float eps) {
  __shared__ float2 red[2][kNormThreads / 32];
  int turn = 0;
  const int lane = threadIdx.x % GROUP;
  const int64_t row = (int64_t)blockIdx.x * (kNormThreads / GROUP) + threadIdx.x / GROUP;
  griddep_wait();
  griddep_launch_dependents();
  if (row >= M) return;  // whole groups (a block is one row when GROUP is a block)
  const int nv = d / VEC;
  const T *xr = x + row * d;
  // the row stays in its own type: half the registers, twice the rows in flight
  using P = Pack<T, VEC>;
  P v[N], r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = lane + i * GROUP;
    if (c < nv) {
      v[i].raw = *reinterpret_cast<const typename P::raw_t *>(xr + (int64_t)c * VEC);
      if (res != nullptr)
        r[i].raw = *reinterpret_cast<const typename P::raw_t *>(res + row * d + (int64_t)c * VEC);
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = lane + i * GROUP;
    if (c < nv) {
      if (res != nullptr) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)  // the statistics are those of the stored sum
          v[i].v[k] = from_f<T>(to_f(v[i].v[k]) + to_f(r[i].v[k]));
        *reinterpret_cast<typename P::raw_t *>(h + row * d + (int64_t)c * VEC) = v[i].raw;
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) s += to_f(v[i].v[k]);
    }
  }
  const float inv_d = 1.0f / (float)d;
  const float mean = group_sum<GROUP>(s, red, turn) * inv_d;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = lane + i * GROUP;
    if (c < nv) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float t = to_f(v[i].v[k]) - mean;
        q += t * t;
      }
    }
  }
  const float rstd = 1.0f / sqrtf(group_sum<GROUP>(q, red, turn) * inv_d + eps);
  T *yr = y + row * d;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = lane + i * GROUP;
    if (c < nv) {
      float w[VEC], b[VEC], o[VEC];
      load_w<VEC>(weight + c * VEC, w);
      load_w<VEC>(bias + c * VEC, b);
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = (to_f(v[i].v[k]) - mean) * rstd * w[k] + b[k];
      store_vec<T, VEC>(yr + (int64_t)c * VEC, o);
    }
  }
  if (lane == 0) {
    if (mean_out != nullptr) mean_out[row] = mean;
    if (rstd_out != nullptr) rstd_out[row] = rstd;
  }
}

// Asynchronous copy of one vector to this thread's own place in shared memory;
// the thread that copied it is the only one to read it, so waiting for its
// copies (copies_wait) is all the synchronisation there is.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}
// 16 bytes of which the first n exist (the others are written as 0)
__device__ __forceinline__ void copy_async_n(void *dst, const void *src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How the backward pass brings its rows.  With up to 8 elements a thread it
// holds the weights and the row's dy and h in registers (N * VEC <= 8), else it
// reads them twice.
//   ring   each thread copies its own vectors asynchronously to its own places in
//          shared memory, which costs no registers and needs no barrier: the
//          row at hand and the next
//   ahead  the next row waits in registers: 4-byte vectors that are held (5001
//          fp32 rows of 1001: 18.4 us, through the ring 21.8; 16-byte vectors the
//          other way round, 16384 bf16 rows of 1024: 43.3 and 28.1)
//   rows   2-byte elements, which cannot be copied one by one: the group copies
//          whole rows, from the 16 bytes that a row's start lies in to those of
//          its end, and reads its elements there (2000 rows of 4001: 27.1 us,
//          read in place 80.6; 4-byte ones are better off as above, 20.5 and 18.4
//          for 5001 fp32 rows of 1001)
constexpr int kNormStages = 2, kNormRowStages = 3;
template <typename T, int VEC, int N>
struct NormFeed {
  static constexpr size_t kBytes = sizeof(T) * VEC;
  static constexpr bool kHold = N * VEC <= 8;
  static constexpr bool kAhead = kHold && kBytes == 4;
  static constexpr bool kRing = kBytes >= 4 && !kAhead;
  static constexpr bool kWhole = kBytes == 2;
};
template <typename T, int VEC, int N, int THREADS>
constexpr size_t norm_ring_bytes() {
  return NormFeed<T, VEC, N>::kRing ? (size_t)kNormStages * 3 * N * THREADS * sizeof(T) * VEC : 0;
}
// Room for a row from the 16 bytes that its start lies in to those of its end.
__host__ __device__ inline int norm_row_bytes(int d, int elem) {
  return (d * elem + 31) / 16 * 16;
}

// The first element of row `row` in its copy, and the copies of dy, h and dh (by
// the threads of a group) themselves, next to each other: the elements around
// the row come along, none beyond the last row.
template <typename T>
__device__ __forceinline__ int norm_row_first(int64_t row, int d) {
  return (int)(row * d % (16 / (int)sizeof(T)));
}
template <typename T, int GROUP>
__device__ __forceinline__ void norm_copy_row(uint8_t *dst, const T *dy, const T *h, const T *dh,
                                              int64_t row, int M, int d) {
  constexpr int kVec = 16 / (int)sizeof(T);
  const int first = norm_row_first<T>(row, d), n = (first + d + kVec - 1) / kVec;
  const int stride = norm_row_bytes(d, sizeof(T));
  const int64_t begin = row * d - first, end = (int64_t)M * d;
  for (int c = (int)threadIdx.x % GROUP; c < n; c += GROUP) {
    const int64_t at = begin + (int64_t)c * kVec;
    const int bytes = end - at < kVec ? (int)(end - at) * (int)sizeof(T) : 16;
    copy_async_n(dst + 16 * c, dy + at, bytes);
    copy_async_n(dst + stride + 16 * c, h + at, bytes);
    if (dh != nullptr) copy_async_n(dst + 2 * stride + 16 * c, dh + at, bytes);
  }
}

// Blocks on an SM: three where the registers allow it (held 16-byte vectors, 80 a
// thread), 8192 x 1536 24.3 us instead of 27.1 with two.
template <typename T, int VEC, int N, int GROUP, int THREADS>
constexpr int norm_backward_per_sm() {
  using Feed = NormFeed<T, VEC, N>;
  if (Feed::kAhead && THREADS > kNormThreads) return 1;  // the registers of a row ahead
  return Feed::kHold && Feed::kRing && (GROUP == 32 || GROUP == kNormThreads) ? 3 : 2;
}

// dx, and the block's sums of dw and db: part [blocks][2][d].  Rows are dealt
// to the groups round-robin.  While a row is reduced the next one is on its
// way; registers hold the running dw and db (2 x 8 at d = 768, three warps a row), and
// what is in flight sets the rate.
template <typename T, int VEC, int N, int GROUP, int THREADS>
__global__ void __launch_bounds__(THREADS, (norm_backward_per_sm<T, VEC, N, GROUP, THREADS>()))
    norm_backward(const T *__restrict__ dy, const T *__restrict__ h,
                  const float *__restrict__ weight, const float *__restrict__ mean_in,
                  const float *__restrict__ rstd_in, const T *__restrict__ dh,
                  T *__restrict__ dx, float *__restrict__ part, int M, int d) {
  __shared__ float2 red[2][THREADS / 32];
  extern __shared__ __align__(16) uint8_t ring[];
  int turn = 0;
  using Feed = NormFeed<T, VEC, N>;
  using P = Pack<T, VEC>;
  constexpr int kRows = THREADS / GROUP;
  constexpr bool kHold = Feed::kHold, kAhead = Feed::kAhead, kRing = Feed::kRing;
  constexpr bool kWhole = Feed::kWhole;
  const int lane = threadIdx.x % GROUP, grp = threadIdx.x / GROUP;
  const int nv = d / VEC;
  const float inv_d = 1.0f / (float)d;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t step = (int64_t)gridDim.x * kRows;
  auto place = [&](int stage, int op, int i) {
    return reinterpret_cast<T *>(ring) +
           (int64_t)(((stage * 3 + op) * N + i) * THREADS + threadIdx.x) * VEC;
  };
  auto source = [&](int op, int64_t row, int i) {
    return (op == 0 ? dy : op == 1 ? h : dh) + row * d + (int64_t)(lane + i * GROUP) * VEC;
  };
  // whole rows: stage, operand; and how they come
  auto copy_of = [&](int stage, int op) {
    return ring + ((grp * kNormRowStages + stage) * 3 + op) * norm_row_bytes(d, sizeof(T));
  };
  auto fetch_whole = [&](int64_t row, int stage) {
    if (row < M) norm_copy_row<T, GROUP>(copy_of(stage, 0), dy, h, dh, row, M, d);
    copies_commit();
  };
  P ahead[kAhead ? 3 : 1][kAhead ? N : 1];
  auto fetch = [&](int64_t row, int stage) {
    if (row < M) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (lane + i * GROUP < nv) {
#pragma unroll
          for (int op = 0; op < 3; ++op) {
            if (op == 2 && dh == nullptr) continue;
            if constexpr (kRing)
              copy_async<(int)Feed::kBytes>(place(stage, op, i), source(op, row, i));
            else if constexpr (kAhead)
              ahead[op][i].raw =
                  __ldg(reinterpret_cast<const typename P::raw_t *>(source(op, row, i)));
          }
        }
      }
    }
    if constexpr (kRing) copies_commit();
  };
  float dw[N * VEC], db[N * VEC], held_w[kHold ? N * VEC : 1];
#pragma unroll
  for (int i = 0; i < N * VEC; ++i) dw[i] = 0.f, db[i] = 0.f;
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + i * GROUP < nv) load_w<VEC>(weight + (lane + i * GROUP) * VEC, held_w + i * VEC);
  }
  int64_t row = (int64_t)blockIdx.x * kRows + grp;
  if constexpr (kWhole) {
    fetch_whole(row, 0);
    fetch_whole(row + step, 1);
  } else {
    fetch(row, 0);
  }
  // the row's, a row ahead like the rest of it (8192 x 1536: 24.3 us, with the row 27.8)
  float next_mean = 0.f, next_rstd = 0.f;
  if (row < M) next_mean = mean_in[row], next_rstd = rstd_in[row];
  if constexpr (kWhole) {
    copies_wait<1>();
    group_sync<GROUP, THREADS>();
  }
  // two stages (three of whole rows) in turn
  for (int stage = 0; row < M;
       row += step, stage = kWhole ? (stage == 2 ? 0 : stage + 1) : stage ^ 1) {
    P held[kHold ? 3 : 1][kHold ? N : 1];  // dy, h and, of a row fetched ahead, dh
    if constexpr (kAhead) {
#pragma unroll
      for (int op = 0; op < 3; ++op)
#pragma unroll
        for (int i = 0; i < N; ++i) held[op][i] = ahead[op][i];
    }
    if constexpr (!kWhole) fetch(row + step, stage ^ 1);
    const float mean = next_mean, rstd = next_rstd;
    if (row + step < M) next_mean = mean_in[row + step], next_rstd = rstd_in[row + step];
    const T *mine[kWhole ? 3 : 1];  // whole rows: this thread's first element
    if constexpr (kWhole) {
#pragma unroll
      for (int op = 0; op < 3; ++op)
        mine[op] = reinterpret_cast<const T *>(copy_of(stage, op)) + norm_row_first<T>(row, d) +
                   lane;
    }
    // vector i of operand op of this row
    auto take = [&](int op, int i, P &out) {
      if constexpr (kAhead) {
        out = held[op][i];
      } else if constexpr (kRing) {
        out.raw = *reinterpret_cast<const typename P::raw_t *>(place(stage, op, i));
      } else {
        out.v[0] = mine[op][i * GROUP];
      }
    };
    auto weights = [&](int i, float *w) {
      if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = held_w[i * VEC + k];
      } else {
        load_w<VEC>(weight + (lane + i * GROUP) * VEC, w);
      }
    };
    if constexpr (kRing) copies_wait<1>();
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (lane + i * GROUP < nv) {
        P g, xh;
        float w[VEC];
        take(0, i, g);
        take(1, i, xh);
        if constexpr (kHold) held[0][i] = g, held[1][i] = xh;
        weights(i, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float gk = to_f(g.v[k]), x = (to_f(xh.v[k]) - mean) * rstd, t = gk * w[k];
          dw[i * VEC + k] += gk * x;
          db[i * VEC + k] += gk;
          s1 += t;
          s2 += t * x;
        }
      }
    }
    if constexpr (kWhole) {
      // the next row has come: to the whole group, once it has met
      copies_wait<0>();
      if constexpr (GROUP == 32) __syncwarp();
    }
    const float2 sums = group_sum2<GROUP, THREADS>(make_float2(s1, s2), red, turn);
    // and it has left the row before this one
    if constexpr (kWhole) fetch_whole(row + 2 * step, stage == 0 ? 2 : stage - 1);
    const float m1 = sums.x * inv_d, m2 = sums.y * inv_d;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (lane + i * GROUP < nv) {
        P g, xh;
        float w[VEC], o[VEC];
        if constexpr (kHold) {
          g = held[0][i], xh = held[1][i];
        } else {
          take(0, i, g);
          take(1, i, xh);
        }
        weights(i, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          o[k] = rstd * (to_f(g.v[k]) * w[k] - m1 - (to_f(xh.v[k]) - mean) * rstd * m2);
        if (dh != nullptr) {
          P r;
          take(2, i, r);
#pragma unroll
          for (int k = 0; k < VEC; ++k) o[k] += to_f(r.v[k]);
        }
        store_vec<T, VEC>(dx + row * d + (int64_t)(lane + i * GROUP) * VEC, o);
      }
    }
  }
  // dw and db of a block lie element k of every vector next to each other
  // (k nv + c), so that a warp's stores are consecutive: in the rows' own order
  // eight lanes meet in each bank of shared memory (8192 x 1536: 29.0 us, so 24.3)
  float *pw = part + (int64_t)blockIdx.x * 2 * d;
  if constexpr (GROUP == THREADS) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = lane + i * GROUP;
      if (c < nv)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          pw[k * nv + c] = dw[i * VEC + k];
          pw[d + k * nv + c] = db[i * VEC + k];
        }
    }
  } else {
    // the groups' sums side by side in the ring's place, added in order
    if constexpr (kRing || kWhole) copies_wait<0>();
    __syncthreads();
    float *acc = reinterpret_cast<float *>(ring);  // [kRows][2][d]
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = lane + i * GROUP;
      if (c < nv)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          acc[grp * 2 * d + k * nv + c] = dw[i * VEC + k];
          acc[grp * 2 * d + d + k * nv + c] = db[i * VEC + k];
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * d; j += THREADS) {
      float t = acc[j];
#pragma unroll
      for (int q = 1; q < kRows; ++q) t += acc[q * 2 * d + j];
      pw[j] = t;
    }
  }
}

// dw and db from the blocks' partial rows: a block sums 32 columns, 32
// lanes of partial rows each, lanes joined in order.
constexpr int kNormSumCols = 32, kNormSumLanes = 32;
__global__ void __launch_bounds__(kNormSumCols *kNormSumLanes)
    norm_backward_sum(const float *__restrict__ part, float *__restrict__ dweight,
                      float *__restrict__ dbias, int blocks, int d, int vec) {
  __shared__ float s[kNormSumLanes][kNormSumCols + 1];
  griddep_wait();
  const int col = threadIdx.x % kNormSumCols, r = threadIdx.x / kNormSumCols;
  const int j = blockIdx.x * kNormSumCols + col;
  float v = 0.f;
  if (j < 2 * d) {
#pragma unroll 5
    for (int b = r; b < blocks; b += kNormSumLanes) v += part[(int64_t)b * 2 * d + j];
  }
  s[r][col] = v;
  __syncthreads();
  if (r == 0 && j < 2 * d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kNormSumLanes; ++i) t += s[i][col];
    const int nv = d / vec, at = j < d ? j : j - d;  // element at / nv of vector at % nv
    (j < d ? dweight : dbias)[at % nv * vec + at / nv] = t;
  }
}

struct NormArgs {
  const void *a, *b;  // forward: x, res; backward: dy, h
  const float *weight, *bias, *mean, *rstd;
  const void *dh;
  void *o0, *o1;      // forward: h, y; backward: dx, -
  float *f0, *f1;     // forward: mean, rstd; backward: part, -
  int M, d;
  float eps;
  int blocks;         // backward: as launch_bwd chose
};

template <typename T, int VEC, int N, int GROUP>
cudaError_t launch_fwd(const NormArgs &a, cudaStream_t stream) {
  return launch_dependent(norm_forward<T, VEC, N, GROUP>, a.blocks, kNormThreads, 0, stream,
                          static_cast<const T *>(a.a), static_cast<const T *>(a.b), a.weight,
                          a.bias, static_cast<T *>(a.o0), static_cast<T *>(a.o1), a.f0, a.f1, a.M,
                          a.d, a.eps);
}
static_assert(norm_ring_bytes<float, 4, 8, kNormThreads>() <= kNormMaxSmem,
              "two rows of every group fit");
template <typename T, int VEC, int N, int GROUP, int THREADS = kNormThreads>
cudaError_t launch_bwd(NormArgs &a, cudaStream_t stream) {
  constexpr int kRows = THREADS / GROUP;
  size_t smem = norm_ring_bytes<T, VEC, N, THREADS>();
  if (NormFeed<T, VEC, N>::kWhole)
    smem = (size_t)kRows * kNormRowStages * 3 * norm_row_bytes(a.d, sizeof(T));
  if (GROUP < THREADS) {
    const size_t sums = 2 * sizeof(float) * (size_t)a.d * kRows;
    if (sums > smem) smem = sums;
  }
  // groups of the grid: all that are resident at once, no more than rows
  constexpr int kPerSm = norm_backward_per_sm<T, VEC, N, GROUP, THREADS>();
  const int most = kNormSms * (kPerSm * smem > kNormSmSmem ? 1 : kPerSm);
  const int64_t blocks = ((int64_t)a.M + kRows - 1) / kRows;
  a.blocks = (int)(blocks < most ? blocks : most);
  if (a.blocks > norm_backward_blocks(a.M, a.d) || smem > kNormMaxSmem)
    return cudaErrorInvalidValue;  // more than the workspace or the attribute below holds
  static OncePerDevice attrs;
  if (!attrs.run([] {
        return cudaFuncSetAttribute(norm_backward<T, VEC, N, GROUP, THREADS>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kNormMaxSmem) == cudaSuccess;
      }))
    return cudaErrorInvalidValue;
  return launch_dependent(norm_backward<T, VEC, N, GROUP, THREADS>, a.blocks, THREADS, smem,
                          stream, static_cast<const T *>(a.a), static_cast<const T *>(a.b),
                          a.weight, a.mean, a.rstd, static_cast<const T *>(a.dh),
                          static_cast<T *>(a.o0), a.f0, a.M, a.d);
}

// Whether the backward pass takes rows of 2049 to 4096 elements with 512 threads,
// so that they can be held: fp32 (2000 x 4001: 44.1 us, held 27.5; 4000 x 4000:
// 52.1 and 45.7) and pairs of bf16 (2000 x 4002: 30.4 and 21.0), not the other
// bf16 rows (9001 x 4000: 64.6 and 69.0, 6000 x 2561: 47.9 and 49.6).
template <typename T, int VEC>
constexpr bool norm_long_held() {
  return sizeof(T) == 4 || VEC == 2;
}
// Elements a thread: the fewest of 8, 16, 24, 32 that cover the row.  A part of a
// block's rows are no longer than pick_group lets them be.
template <typename T, int VEC, int GROUP, bool kBackward>
cudaError_t pick_n(NormArgs &a, cudaStream_t stream) {
  constexpr int kNot = kBackward && GROUP == kNormThreads && norm_long_held<T, VEC>() ? 16 : 0;
  constexpr int kMost = GROUP > 32                    ? 32
                        : sizeof(T) * VEC < 16        ? 8
                        : sizeof(T) == 4 || kBackward ? 16
                                                      : 32;
  const int per = (a.d + GROUP * 8 - 1) / (GROUP * 8);  // eights of elements a thread
#define FMCA_NORM(E)                                                            \
  if constexpr ((E) <= kMost && (E) != kNot)                                    \
    if (per * 8 <= (E))                                                         \
      return kBackward ? launch_bwd<T, VEC, (E) / VEC, GROUP>(a, stream)        \
                       : launch_fwd<T, VEC, (E) / VEC, GROUP>(a, stream)
  FMCA_NORM(8);
  FMCA_NORM(16);
  FMCA_NORM(24);
  FMCA_NORM(32);
#undef FMCA_NORM
  return cudaErrorInvalidValue;
}
// Warps a row of the backward pass has where one warp would be short of
// registers: bf16 rows of more than 768 in 16-byte vectors four (16384 x 1024:
// 28.1 us, with a warp a row 34.8), of more than 512 three (4096 x 768: 8.9 and
// 9.3, 16384 x 768: 22.0 and 25.7, 32768 x 768: 37.4 and 43.8, 16384 x 520: 21.0
// and 22.0).  0: as in the forward pass.
constexpr int kNormWideRows = 4;
int norm_wide(int d, int elem) {
  if (elem != 2 || d % 8 || d > kNormWarpMaxD) return 0;
  return d > 768 ? 4 : d > 512 ? 3 : 0;
}
template <typename T, int VEC, bool kBackward>
cudaError_t pick_group(NormArgs &a, cudaStream_t stream) {
  if constexpr (kBackward && norm_long_held<T, VEC>())
    if (a.d > 2048 && a.d <= 4096)
      return launch_bwd<T, VEC, 8 / VEC, 2 * kNormThreads, 2 * kNormThreads>(a, stream);
  const int part = norm_part(a.d, sizeof(T), sizeof(T) * VEC);
  if constexpr (sizeof(T) * VEC < 16)
    if (part == 64)
      return kBackward ? launch_bwd<T, VEC, 8 / VEC, 64>(a, stream)
                       : launch_fwd<T, VEC, 8 / VEC, 64>(a, stream);
  if constexpr (sizeof(T) * VEC < 16 || sizeof(T) == 4)
    if (part == 128)
      return kBackward ? launch_bwd<T, VEC, 8 / VEC, 128>(a, stream)
                       : launch_fwd<T, VEC, 8 / VEC, 128>(a, stream);
  if constexpr (kBackward && VEC == 8) {
    const int warps = norm_wide(a.d, sizeof(T));
    if (warps == 4) return launch_bwd<T, VEC, 1, 128, 128 * kNormWideRows>(a, stream);
    if (warps == 3) return launch_bwd<T, VEC, 1, 96, 96 * kNormWideRows>(a, stream);
  }
  return a.d <= kNormWarpMaxD ? pick_n<T, VEC, 32, kBackward>(a, stream)
                              : pick_n<T, VEC, kNormThreads, kBackward>(a, stream);
}
template <bool kBackward>
cudaError_t pick(NormArgs &a, int bf16, cudaStream_t stream) {
  if (bf16) {
    if (a.d % 8 == 0) return pick_group<__nv_bfloat16, 8, kBackward>(a, stream);
    if (a.d % 2 == 0) return pick_group<__nv_bfloat16, 2, kBackward>(a, stream);
    return pick_group<__nv_bfloat16, 1, kBackward>(a, stream);
  }
  if (a.d % 4 == 0) return pick_group<float, 4, kBackward>(a, stream);
  return pick_group<float, 1, kBackward>(a, stream);
}

// Bytes of a vector, as pick takes them.
int norm_vec(int d, int elem) { return d * elem % 16 == 0 ? 16 : d * elem % 4 == 0 ? 4 : 2; }
// Rows of a block of the forward pass.
int norm_rows(int d, int elem) {
  const int part = norm_part(d, elem, norm_vec(d, elem));
  return kNormThreads / (part ? part : d <= kNormWarpMaxD ? 32 : kNormThreads);
}

}  // namespace

int launch_layer_norm(const void *x, const void *res, const float *weight, const float *bias,
                      void *h, void *y, float *mean, float *rstd, int M, int d, float eps,
                      int dtype_bf16, cudaStream_t stream) {
  NormArgs a = {};
  a.a = x, a.b = res, a.weight = weight, a.bias = bias;
  a.o0 = h, a.o1 = y, a.f0 = mean, a.f1 = rstd;
  a.M = M, a.d = d, a.eps = eps;
  const int rows = norm_rows(d, dtype_bf16 ? 2 : 4);
  a.blocks = (int)(((int64_t)M + rows - 1) / rows);
  return pick<false>(a, dtype_bf16, stream) == cudaSuccess ? 0 : 1;
}

int launch_layer_norm_backward(const void *dy, const void *h, const float *weight,
                               const float *mean, const float *rstd, const void *dh, void *dx,
                               float *dweight, float *dbias, int M, int d, int dtype_bf16,
                               void *workspace, cudaStream_t stream) {
  NormArgs a = {};
  a.a = dy, a.b = h, a.weight = weight, a.mean = mean, a.rstd = rstd, a.dh = dh;
  a.o0 = dx, a.f0 = static_cast<float *>(workspace);
  a.M = M, a.d = d;
  if (pick<true>(a, dtype_bf16, stream) != cudaSuccess) return 1;
  const int elem = dtype_bf16 ? 2 : 4;
  return launch_dependent(norm_backward_sum, (2 * d + kNormSumCols - 1) / kNormSumCols,
                          kNormSumCols * kNormSumLanes, 0, stream, (const float *)a.f0, dweight,
                          dbias, a.blocks, d, norm_vec(d, elem) / elem) == cudaSuccess
             ? 0
             : 1;
}

}  // namespace fmca
