// logprobs.cu -- log probabilities of given tokens, with the entropy and the likeliest alternatives.
//
//   logp[t] = x_t - m - log S0,   H = log S0 - S1 / S0,   S0 = sum e^(x - m),   S1 = sum (x - m) e^(x - m)
//
// A row is read from memory once: a cluster of up to 8 CTAs takes it in slices, each slice lands in shared
// memory by one bulk copy, and the maximum, the two sums and the alternatives are three walks over it there.
// The slices' (m, S0, S1) and sorted alternatives meet in the first CTA's shared memory. Bound by HBM for
// many rows, by latency for one.
//
// Alternatives: the slice's values fall into 64 groups (four threads each); the k-th largest of the groups'
// maxima is a floor that at least k values reach, and for k <= 32 few others do. The values at or above it
// are listed and ranked by counting, on (value, lower id first) as one 64-bit key, so that the order is
// exact and independent of timing. A list that overflows falls back to k maxima one after another.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "ptx.cuh"
#include "tinfer.h"

namespace cg = cooperative_groups;

namespace tinfer {
namespace logprobs {

constexpr int NT = 256, NWARPS = NT / 32;
constexpr int MAX_K = 32, MAX_CLUSTER = 8, GROUPS = 64;
constexpr int LIST = 512;             // listed candidates of a slice, at most
constexpr int MAX_VOCAB = 1 << 18;    // 8 slices of 128 KiB of fp32
constexpr float LOG2E = 1.4426950408889634f;
constexpr long long WAIT_NS = 200LL * 1000 * 1000;

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
__global__ void __launch_bounds__(NT) logprobs_kernel(const __grid_constant__ Params q) {
  constexpr int N = 16 / sizeof(T);  // elements of a word
  extern __shared__ __align__(128) unsigned char buf[];
  __shared__ alignas(8) unsigned long long bar;
  __shared__ float red[3][NWARPS];
  __shared__ float group_top[GROUPS];
  __shared__ float floor_s;
  __shared__ int listed;
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

  // the slice as it lies in memory, from the 16-byte word of its first element to that of its last: whole
  // words by one bulk copy, the ends by ordinary loads, what is beside the row set to -infinity
  const uintptr_t from = reinterpret_cast<uintptr_t>(x + a);
  const int mis = (int)(from & 15) / (int)sizeof(T);  // elements before the slice in its first word
  const int words = len ? (mis + len + N - 1) / N : 0;
  T* s = reinterpret_cast<T*>(buf);                   // slice element i is s[mis + i]
  const int w0 = mis ? 1 : 0, w1 = (mis + len) / N;   // whole words
  if (tid == 0) {
    mbar_init(smem_addr(&bar), 1);
    mbar_fence_init();
    listed = 0;
    if (w1 > w0) {
      mbar_arrive_expect_tx(smem_addr(&bar), (uint32_t)(w1 - w0) * 16u);
      bulk_g2s(smem_addr(buf) + 16u * w0, reinterpret_cast<const void*>((from & ~(uintptr_t)15) + 16 * w0),
               (uint32_t)(w1 - w0) * 16u, smem_addr(&bar), policy_evict_first());
    }
  }
  const T masked = (T)(-INFINITY);
  if (tid < N && words) {
    if (w0 == 1) s[tid] = tid >= mis && tid - mis < len ? x[a + tid - mis] : masked;
    if (w1 < words && (w1 > 0 || w0 == 0)) {
      const int e = w1 * N + tid;
      s[e] = e - mis < len ? x[a + e - mis] : masked;
    }
  }
  float target_x = 0.f;
  bool target_in = false;
  if (rank == 0 && tid == 0 && q.logp) {
    const int t = q.targets[row];
    target_in = t >= 0 && t < q.vocab;
    if (target_in) target_x = value(x[t]);
  }
  __syncthreads();
  bool late = false;  // a copy that never arrived makes the row NaN
  if (w1 > w0) {
    const uint64_t t0 = globaltimer();
    while (!late && !mbar_try_wait(smem_addr(&bar), 0)) late = (long long)(globaltimer() - t0) > WAIT_NS;
  }

  // ---- first walk: maxima
  const uint4* sw = reinterpret_cast<const uint4*>(buf);
  float top = -INFINITY;
  for (int w = tid; w < words; w += NT) {
    float v[N];
    unpack(sw[w], v, x);
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, v[i]);
  }
  const float mine = top;
  float quad = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
  quad = fmaxf(quad, __shfl_xor_sync(~0u, quad, 2));
  if ((tid & 3) == 0) group_top[tid >> 2] = quad;
  top = quad;
#pragma unroll
  for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) red[0][warp] = top;
  __syncthreads();
  Part p;
  p.m = red[0][0];
#pragma unroll
  for (int w = 1; w < NWARPS; ++w) p.m = fmaxf(p.m, red[0][w]);

  // the floor of the alternatives: the k-th largest of the groups' maxima, ties by the group
  if (q.k && tid < GROUPS) {
    const float g = group_top[tid];
    int above = 0;
    for (int i = 0; i < GROUPS; ++i) {
      const float y = group_top[i];
      above += y > g || (y == g && i < tid);
    }
    if (above == q.k - 1) floor_s = g;
  }
  // ---- second walk: the sums
  float s0 = late ? __uint_as_float(0x7FC00000u) : 0.f, s1 = 0.f;
  const float m = p.m == -INFINITY ? 0.f : p.m;
  for (int w = tid; w < words; w += NT) {
    float v[N];
    unpack(sw[w], v, x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = v[i] - m, e = exp2_fast(z * LOG2E);
      s0 += e;
      s1 = fmaf(e, fmaxf(z, -1e30f), s1);  // a masked token adds 0 * -1e30
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s0 += __shfl_xor_sync(~0u, s0, o);
    s1 += __shfl_xor_sync(~0u, s1, o);
  }
  if (lane == 0) {
    red[1][warp] = s0;
    red[2][warp] = s1;
  }
  __syncthreads();
  p.s0 = p.s1 = 0.f;
#pragma unroll
  for (int w = 0; w < NWARPS; ++w) {
    p.s0 += red[1][w];
    p.s1 += red[2][w];
  }
  cluster.barrier_wait(std::move(started));
  if (tid == 0) cluster.map_shared_rank(parts, 0)[rank] = p;

  // ---- third walk: the values at or above the floor, ranked
  if (q.k) {
    const float floor_x = floor_s;
    if (mine >= floor_x && mine > -INFINITY)
      for (int w = tid; w < words; w += NT) {
        float v[N];
        unpack(sw[w], v, x);
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
        for (int i = 0; i < n; ++i) above += list[i] > key;
        if (above < q.k) best[above] = key;
      }
    } else {  // many equal or near values: one maximum after another
      unsigned long long last = ~0ull;
      for (int j = 0; j < q.k; ++j) {
        unsigned long long b = 0;
        for (int w = tid; w < words; w += NT) {
          float v[N];
          unpack(sw[w], v, x);
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
  int found = 0;
  for (int i = 0; i < n; ++i) found += tops[i] != 0;
  for (int c = tid; c < n; c += NT) {
    const unsigned long long key = tops[c];
    if (!key || bad) continue;
    int above = 0;
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
  const size_t smem = ((size_t)q.slice * sizeof(T) + 15) / 16 * 16 + 32;
  cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(q.rows * cluster));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
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
  // slices of 32 to 64 KiB keep three or more CTAs on an SM; few rows are cut finer to spread over more SMs
  const long long bytes = (long long)vocab * size;
  int cluster = 1;
  while (cluster < logprobs::MAX_CLUSTER && bytes / cluster > (rows * cluster < 128 ? 8 : 48) * 1024) cluster *= 2;
  logprobs::Params q{logits_dev, row_stride, targets_dev, logp_dev, entropy_dev, top_ids_dev, top_logp_dev,
                     rows, vocab, top_k, ((vocab + cluster - 1) / cluster + 7) / 8 * 8};
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == TINFER_DTYPE_F32   ? logprobs::launch<float>(q, cluster, st)
                        : dtype == TINFER_DTYPE_F16 ? logprobs::launch<__half>(q, cluster, st)
                                                    : logprobs::launch<__nv_bfloat16>(q, cluster, st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}
