// logprobs.cu -- log probabilities of given tokens, with the entropy and the likeliest alternatives.
//
//   logp[t] = x_t - m - log S0,   H = log S0 - S1 / S0,   S0 = sum e^(x - m),   S1 = sum (x - m) e^(x - m)
//
// A row is one CTA's, or, where the rows are too few to fill the GPU, a cluster's of up to 8 CTAs in slices. Threads read
// it in 16-byte words, several in flight, and keep their own maximum and sums relative to it; they meet once at
// the end, the slices in the first CTA's shared memory. Bound by HBM for many rows, by latency for one. (Slices staged in
// shared memory by bulk copies took 300 to 345 us for 2047 rows of 128256 fp32 logits: with 64 KiB of a row to a CTA, the
// joins at its end are most of its life. Three CTAs of 40 registers on an SM took 219 us, four of 32 take 199,
// 0.79 of the measured copy rate. One row of 128256: 7.4 us; 64 rows of 151936 bf16, 20 alternatives: 11.8.)
//
// Alternatives: a slice's values fall to 32 groups of threads, one of each lane of all warps (so that a slice of few words
// leaves none empty); the k-th largest of the groups' maxima is a floor that at least k values reach, and few others do
// (31 on average for k = 20). Only threads whose maximum reaches it
// have any: their words are dealt out and read again. Those values are listed and ranked by counting, on (value, lower id
// first) as one 64-bit key, so that the order is exact and independent of timing. A list that overflows falls back
// to k maxima one after another.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "tinfer.h"

namespace cg = cooperative_groups;

namespace tinfer {
namespace logprobs {

constexpr int NT = 512, NWARPS = NT / 32;
constexpr int MAX_K = 32, MAX_CLUSTER = 8;
constexpr int GROUPS = 32;             // of threads, whose maxima give the alternatives' floor: one of each lane
static_assert(MAX_CLUSTER * MAX_K <= NT, "a thread for every alternative of the slices");
static_assert(MAX_K <= GROUPS, "a floor for every k");
constexpr int LIST = 512;             // listed candidates of a slice, at most
constexpr int MAX_VOCAB = 1 << 18;
constexpr float LOG2E = 1.4426950408889634f;

struct Params {
  const void* logits;
  long long row_stride;  // elements
  const int* targets;
  float* logp;
  float* entropy;
  int* top_ids;
  float* top_logp;
  int rows, vocab, k, slice;  // slice: elements of one CTA's part of a row
};

struct Part {
  float m, s0, s1;
};

// 32 bits of logits of minus infinity.
__device__ __forceinline__ uint32_t minus_infinity(const float*) { return 0xFF800000u; }
__device__ __forceinline__ uint32_t minus_infinity(const __half*) { return 0xFC00FC00u; }
__device__ __forceinline__ uint32_t minus_infinity(const __nv_bfloat16*) { return 0xFF80FF80u; }

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

// The elements of one 16-byte word.
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[4], const float*) {
  x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8], const __half*) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8], const __nv_bfloat16*) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Larger value first, then lower id; 0: no token (masked tokens have none). Zeros of both signs are equal.
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
  const unsigned b = __float_as_uint(x + 0.f);
  const unsigned u = b & 0x80000000u ? ~b : b | 0x80000000u;
  return ((unsigned long long)u << 32) | (unsigned)~id;
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const unsigned u = (unsigned)(key >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int id_of(unsigned long long key) { return (int)~(unsigned)key; }

__device__ __forceinline__ Part join(const Part& a, const Part& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Part{m, a.s0 + b.s0, a.s1 + b.s1};  // nothing but masked tokens (or NaN)
  // (bounded, so that a part of weight 0 adds 0 and not 0 * infinity)
  const float da = a.m == -INFINITY ? 0.f : fmaxf(a.m - m, -1e30f), db = b.m == -INFINITY ? 0.f : fmaxf(b.m - m, -1e30f);
  const float wa = exp2_fast(da * LOG2E), wb = exp2_fast(db * LOG2E);
  return Part{m, a.s0 * wa + b.s0 * wb, (a.s1 + a.s0 * da) * wa + (b.s1 + b.s0 * db) * wb};
}

template <typename T>
__global__ void __launch_bounds__(NT, 4) logprobs_kernel(const __grid_constant__ Params q) {
  constexpr int N = 16 / sizeof(T);  // elements of a word
  constexpr int AHEAD = sizeof(T);   // words of a thread in flight: 16 elements, and 32 registers for four CTAs on an SM
  __shared__ Part red[NWARPS];
  __shared__ float lane_top[NWARPS][GROUPS], floor_s;
  __shared__ int listed, owners;
  __shared__ uint16_t owner[NT];
  __shared__ unsigned long long list[LIST];
  __shared__ unsigned long long best[MAX_K], warp_best[NWARPS];
  __shared__ Part parts[MAX_CLUSTER];
  __shared__ unsigned long long tops[MAX_CLUSTER * MAX_K];
  __shared__ float norm_s[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto started = cluster.barrier_arrive();  // the first CTA has to run before the others write to its memory
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int row = (int)(blockIdx.x / size);
  const T* x = static_cast<const T*>(q.logits) + row * q.row_stride;
  const int a = min(rank * q.slice, q.vocab), len = min(q.slice, q.vocab - a);

  // the slice as 16-byte words, from that of its first element to that of its last; of the words at its ends only the
  // slice's own elements are read, the others stand for masked tokens
  const uintptr_t from = reinterpret_cast<uintptr_t>(x + a);
  const int mis = (int)(from & 15) / (int)sizeof(T);  // elements before the slice in its first word
  const int words = len ? (mis + len + N - 1) / N : 0;
  const uint4* base = reinterpret_cast<const uint4*>(from & ~(uintptr_t)15);
  auto word = [&](int w) {
    if (w * N >= mis && (w + 1) * N <= mis + len) return __ldcs(base + w);
    union {
      uint4 u;
      T e[N];
    } y;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = w * N + i - mis;
      y.e[i] = at >= 0 && at < len ? x[a + at] : (T)(-INFINITY);
    }
    return y.u;
  };
  const uint32_t minus = minus_infinity(x);
  const uint4 none = make_uint4(minus, minus, minus, minus);
  if (tid == 0) listed = owners = 0;
  const bool scores = rank == 0 && tid == 0 && q.logp;
  const int target = scores ? q.targets[row] : -1;

  // ---- the walk: every thread's own maximum and its sums relative to it
  Part p{-INFINITY, 0.f, 0.f};
  for (int w = tid; w < words; w += AHEAD * NT) {
    uint4 y[AHEAD];
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) y[h] = w + h * NT < words ? word(w + h * NT) : none;
    float top = -INFINITY;
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) {
      float v[N];
      unpack(y[h], v, x);
#pragma unroll
      for (int i = 0; i < N; ++i) top = fmaxf(top, v[i]);
    }
    if (top > p.m) {
      const float d = p.m == -INFINITY ? 0.f : fmaxf(p.m - top, -1e30f), f = exp2_fast(d * LOG2E);
      p = Part{top, p.s0 * f, (p.s1 + p.s0 * d) * f};
    }
    const float m = p.m == -INFINITY ? 0.f : p.m;
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) {
      float v[N];
      unpack(y[h], v, x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float z = v[i] - m, e = exp2_fast(z * LOG2E);
        p.s0 += e;
        p.s1 = fmaf(e, fmaxf(z, -1e30f), p.s1);  // a masked token adds 0 * -1e30
      }
    }
  }
  const bool target_in = scores && target >= 0 && target < q.vocab;
  const float target_x = target_in ? value(x[target]) : 0.f;
  const float mine = p.m;
  auto other = [&](int o) { return Part{__shfl_xor_sync(~0u, p.m, o), __shfl_xor_sync(~0u, p.s0, o), __shfl_xor_sync(~0u, p.s1, o)}; };
  if (q.k) lane_top[warp][lane] = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) p = join(p, other(o));
  if (lane == 0) red[warp] = p;
  __syncthreads();
  if (warp == 0) {
    p = lane < NWARPS ? red[lane] : Part{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = 1; o < NWARPS; o *= 2) p = join(p, other(o));
  } else if (warp == 1 && q.k) {
    // the floor of the alternatives: the k-th largest of the groups' maxima, ties by the group
    float g = lane_top[0][lane];
#pragma unroll
    for (int w = 1; w < NWARPS; ++w) g = fmaxf(g, lane_top[w][lane]);
    int above = 0;
#pragma unroll
    for (int o = 1; o < GROUPS; ++o) {
      const float y = __shfl_xor_sync(~0u, g, o);
      above += y > g || (y == g && (lane ^ o) < lane);
    }
    if (above == q.k - 1) floor_s = g;
  }
  if (q.k) __syncthreads();
  cluster.barrier_wait(std::move(started));
  if (tid == 0) cluster.map_shared_rank(parts, 0)[rank] = p;

  // ---- the values at or above the floor, ranked
  if (q.k) {
    const float floor_x = floor_s;
    if (mine >= floor_x && mine > -INFINITY) owner[atomicAdd(&owners, 1)] = (uint16_t)tid;
    __syncthreads();
    const int turns = (words + NT - 1) / NT;  // words of a thread, at most
    for (int item = tid; item < owners * turns; item += NT) {
      const int w = owner[item / turns] + item % turns * NT;
      if (w >= words) continue;
      float v[N];
      unpack(word(w), v, x);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (v[i] >= floor_x && v[i] > -INFINITY) {
          const int n = atomicAdd(&listed, 1);
          if (n < LIST) list[n] = key_of(v[i], a + w * N + i - mis);
        }
    }
    if (tid < MAX_K) best[tid] = 0;
    __syncthreads();
    const int n = listed;
    if (n <= LIST) {
      for (int c = tid; c < n; c += NT) {
        const unsigned long long key = list[c];
        int above = 0;
#pragma unroll 8
        for (int i = 0; i < n; ++i) above += list[i] > key;
        if (above < q.k) best[above] = key;
      }
    } else {  // many equal or near values: one maximum after another
      unsigned long long last = ~0ull;
      for (int j = 0; j < q.k; ++j) {
        unsigned long long b = 0;
        for (int w = tid; w < words; w += NT) {
          float v[N];
          unpack(word(w), v, x);
          for (int i = 0; i < N; ++i) {
            const unsigned long long key = v[i] > -INFINITY ? key_of(v[i], a + w * N + i - mis) : 0;
            if (key < last && key > b) b = key;
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) b = max(b, __shfl_xor_sync(~0u, b, o));
        if (lane == 0) warp_best[warp] = b;
        __syncthreads();
        for (int w = 0; w < NWARPS; ++w) b = max(b, warp_best[w]);
        __syncthreads();
        if (tid == 0) best[j] = b;
        last = b;
        if (!b) break;
      }
    }
    __syncthreads();
    if (tid < q.k) cluster.map_shared_rank(tops, 0)[rank * q.k + tid] = best[tid];
  }
  cluster.sync();
  if (rank) return;

  // ---- the first CTA joins the slices
  if (tid == 0) {
    Part all = parts[0];
    for (int r = 1; r < size; ++r) all = join(all, parts[r]);
    const bool bad = !(all.m < INFINITY) || all.s0 != all.s0;
    const float norm = logf(all.s0), nan = __uint_as_float(0x7FC00000u);
    if (q.logp) q.logp[row] = !target_in || bad ? nan : target_x == -INFINITY ? -INFINITY : target_x - all.m - norm;
    if (q.entropy) q.entropy[row] = bad ? nan : all.s0 == 0.f ? 0.f : norm - all.s1 / all.s0;
    norm_s[0] = bad ? nan : all.m;
    norm_s[1] = norm;
  }
  if (!q.k) return;
  __syncthreads();
  const bool bad = norm_s[0] != norm_s[0];
  int* ids = q.top_ids + (size_t)row * q.k;
  float* lps = q.top_logp + (size_t)row * q.k;
  const int n = size * q.k;
  const int found = __syncthreads_count(tid < n && tops[tid] != 0);
  for (int c = tid; c < n; c += NT) {
    const unsigned long long key = tops[c];
    if (!key || bad) continue;
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) above += tops[i] > key;
    if (above < q.k) {
      ids[above] = id_of(key);
      lps[above] = value_of(key) - norm_s[0] - norm_s[1];
    }
  }
  for (int j = (bad ? 0 : found) + tid; j < q.k; j += NT) {
    ids[j] = -1;
    lps[j] = bad ? __uint_as_float(0x7FC00000u) : -INFINITY;
  }
}

template <typename T>
cudaError_t launch(const Params& q, int cluster, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(q.rows * cluster));
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, q);
}

}  // namespace logprobs
}  // namespace tinfer

using namespace tinfer;

extern "C" tinfer_status tinfer_op_logprobs(int rows, int vocab, int dtype, const void* logits_dev, long long row_stride,
                                            const int32_t* targets_dev, int top_k, float* logp_dev, float* entropy_dev,
                                            int32_t* top_ids_dev, float* top_logp_dev, void* stream) {
  if (rows < 1 || vocab < 1 || !logits_dev || row_stride < vocab || row_stride > (1LL << 40)) return TINFER_ERR_INVALID_ARG;
  const int size = dtype == TINFER_DTYPE_F32 ? 4 : dtype == TINFER_DTYPE_F16 || dtype == TINFER_DTYPE_BF16 ? 2 : 0;
  if (!size || reinterpret_cast<uintptr_t>(logits_dev) % size) return TINFER_ERR_INVALID_ARG;
  if (top_k < 0 || top_k > logprobs::MAX_K || (logp_dev && !targets_dev)) return TINFER_ERR_INVALID_ARG;
  if (top_k ? !top_ids_dev || !top_logp_dev : top_ids_dev || top_logp_dev) return TINFER_ERR_INVALID_ARG;
  if (!logp_dev && !entropy_dev && !top_k) return TINFER_ERR_INVALID_ARG;
  for (const void* p : {(const void*)targets_dev, (const void*)logp_dev, (const void*)entropy_dev, (const void*)top_ids_dev,
                        (const void*)top_logp_dev})
    if (reinterpret_cast<uintptr_t>(p) & 3) return TINFER_ERR_INVALID_ARG;
  if (vocab > logprobs::MAX_VOCAB || rows > (1 << 27)) return TINFER_ERR_UNSUPPORTED;
  // a CTA to a row, or for few rows as many more as run at once (three of the four that fit on an SM) and leave every
  // thread a word or two. 64 rows of 151936 bf16 logits: 11.8 us by four CTAs to a row, 15.5 by eight
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return TINFER_ERR_CUDA;
  const long long bytes = (long long)vocab * size;
  int cluster = 1;
  while (cluster < logprobs::MAX_CLUSTER && 2LL * rows * cluster <= 3 * sms && bytes / cluster > 16 * 1024) cluster *= 2;
  logprobs::Params q{logits_dev, row_stride, targets_dev, logp_dev, entropy_dev, top_ids_dev, top_logp_dev,
                     rows, vocab, top_k, ((vocab + cluster - 1) / cluster + 7) / 8 * 8};
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == TINFER_DTYPE_F32   ? logprobs::launch<float>(q, cluster, st)
                        : dtype == TINFER_DTYPE_F16 ? logprobs::launch<__half>(q, cluster, st)
                                                    : logprobs::launch<__nv_bfloat16>(q, cluster, st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}
