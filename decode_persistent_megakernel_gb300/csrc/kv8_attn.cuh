// kv8_attn.cuh -- parameters of the attention kernels over the 8-bit cache.
#pragma once
#include <cuda.h>

#include "kv8.cuh"

namespace tinfer {
namespace kv8 {

struct AttnParams {
  Cache c;
  Rows q, out;
  Span sp;
  Rope rope;
  float* lse;    // [n_seqs][n_tokens][n_heads], may be null
  float* part;   // workspace: two parts of each CTA, one of each warp; a part is [rows][d] outputs, [rows] maxima, [rows] sums
  int n_heads, group, row_tiles, units;  // units: KV heads x row tiles
  int grid, warps, keep_l2;  // warps of a CTA
  int wait_us, withhold;     // limit of a wait; test hook: one arrival of each pipeline stays away
  float scale_log2;  // log2(e) / sqrt(d)
};

constexpr int WEIGHT_SHIFT = 14;    // weights are held times 2^14: fp16 keeps 11 bits of them down to 2^-28
// Exponents of V scales that enter the running maximum. Of a row whose keys all have the smallest one the
// sum of the softmax is 2^(WEIGHT_SHIFT - E_MIN) for each key: 2^24 keys stay below fp32's 2^128. A smaller
// scale's remainder makes its weights smaller than 1, a scale of 0 makes them 0 and counts in the sum.
// An append leaves scales of up to 2^123 (the largest number / 127, doubled); a mantissa beyond 2 would overflow fp16.
constexpr int E_MIN = -85, E_MAX = 126;
// The sum of the softmax takes a weight 2^(x + e - M) times 2^-e. Where e lies far below the largest exponent that M may
// come from, that weight falls below 2^-126 and is lost although its key may have the row's largest score: of keys with
// e no more than E_SPAN below, what is lost is below 2^-40 of the largest score's term. A tile with others
// sums 2^(x - M) itself, an exponential more for each key: between 2^-109 for the largest score and 2^(WEIGHT_SHIFT -
// E_MIN), computed times 2^SUM_LIFT so that terms down to 2^-37 of the former stay above 2^-146. (Its exponent may be as
// large as 2^8 and is rounded there, by 2^-17.) Sums are rescaled in two halves for the same reason: M moves by up to
// 2^208, the sum by far less.
constexpr int E_SPAN = 86, SUM_LIFT = 20;
constexpr int WAIT_US = 200 * 1000, WAIT_US_WITHHELD = 5 * 1000;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The square root of 2^(from - to): outputs take its square, sums each factor by itself (see E_SPAN).
__device__ __forceinline__ float half_shrink(float from, float to) {
  return from == to ? 1.f : exp2_fast(0.5f * (from - to));
}
// SUM_LIFT and the exponent of a power of two.
__device__ __forceinline__ float lifted(float x) { return (float)((int)(__float_as_uint(x) >> 23) - 127 + SUM_LIFT); }
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The sequence that holds place x of a list of work, of which prefix[s] places stand before sequence s.
template <typename I>
__device__ __forceinline__ int seq_of(const I* prefix, int n, I x) {
  int lo = 0, hi = n;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Waits for a phase of an mbarrier for a while: the hardware suspends the thread meanwhile, where polling
// would take issue slots from the warps that compute.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, int limit_us) {
  if (mbar_sleep(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_sleep(bar, parity))
    if ((long long)(globaltimer() - t0) > limit_us * 1000LL) return mbar_sleep(bar, parity);  // (time may have passed off the GPU)
  return true;
}

// The parts of a unit's rows that several CTAs hold (CTA c0's in its slot 1, the others' in their slot 0), joined in
// order. Called by all warps of a CTA of JOIN_WARPS; blockIdx.y takes a slice of the rows. A row with few parts is
// one warp's work; the parts of a long one are dealt out to all warps and meet in shared memory.
constexpr int JOIN_WARPS = 8;

template <int D, int ROWS, typename T>
__device__ void join_parts(const AttnParams& q, int seq, int head, int row0, int rows, int c0, int parts, int weight_shift) {
  constexpr int N = D / 32, NW = JOIN_WARPS;
  __shared__ alignas(16) float acc_s[NW][D];
  __shared__ float sum_s[NW], top_s[NW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool few = parts <= NW;
  auto part = [&](int c) { return q.part + (size_t)(2 * (c0 + c) + (c == 0 ? 1 : 0)) * ROWS * (D + 2); };
  auto finish = [&](int row, float top, float sum, const float (&y)[N]) {
    const float inv = 1.f / sum;
    const int qrow = row0 + row, tok = qrow / q.group, hq = head * q.group + qrow - tok * q.group;
    T* dst = static_cast<T*>(q.out.data) + seq * q.out.ss + tok * q.out.ts + hq * q.out.hs + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) store_one(dst + i, y[i] * inv);
    if (q.lse && lane == 0)
      q.lse[((size_t)seq * q.sp.n_tokens + tok) * q.n_heads + hq] = (log2f(sum) + top - (float)weight_shift) * 0.6931471805599453f;
  };
  auto load = [&](const float* p, int row, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(p + (size_t)row * D + lane * N + i);
      f[i] = v.x;
      f[i + 1] = v.y;
    }
  };
  if (few) {  // four rows of a warp at a time, their loads side by side
    constexpr int R = 4;
    for (int r0 = (blockIdx.y * NW + warp) * R; r0 < rows; r0 += NW * R * gridDim.y) {
      float top[R], sum[R], y[R][N];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        top[k] = -INFINITY;
        sum[k] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) y[k][i] = 0.f;
      }
#pragma unroll 2
      for (int c = 0; c < parts; ++c) {
        const float* p = part(c);
        float mc[R], lc[R], f[R][N];
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const int row = min(r0 + k, rows - 1);
          mc[k] = p[ROWS * D + row];
          lc[k] = p[ROWS * D + ROWS + row];
          load(p, row, f[k]);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
          if (lc[k] == 0.f) continue;  // no key of the row
          const float now = fmaxf(top[k], mc[k]);
          const float a = half_shrink(top[k], now), b = half_shrink(mc[k], now);
          top[k] = now;
          sum[k] = fmaf(lc[k] * b, b, sum[k] * a * a);
#pragma unroll
          for (int i = 0; i < N; ++i) y[k][i] = fmaf(f[k][i], b * b, y[k][i] * (a * a));
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (r0 + k < rows) finish(r0 + k, top[k], sum[k], y[k]);
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    float top = -INFINITY, sum = 0.f, y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = 0.f;
    auto add = [&](float mc, float lc, const float (&f)[N]) {
      if (lc == 0.f) return;  // no key of the row
      const float now = fmaxf(top, mc);
      const float a = half_shrink(top, now), b = half_shrink(mc, now);
      top = now;
      sum = fmaf(lc * b, b, sum * a * a);
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = fmaf(f[i], b * b, y[i] * (a * a));
    };
    constexpr int R = 8;  // parts of a warp whose loads go out together
    for (int c = warp; c < parts; c += R * NW) {
      float mc[R], lc[R], f[R][N];
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (c + k * NW < parts) {
          const float* p = part(c + k * NW);
          mc[k] = p[ROWS * D + row];
          lc[k] = p[ROWS * D + ROWS + row];
          load(p, row, f[k]);
        } else {
          lc[k] = 0.f;
        }
#pragma unroll
      for (int k = 0; k < R; ++k) add(mc[k], lc[k], f[k]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc_s[warp][lane * N + i] = y[i];
    if (lane == 0) {
      sum_s[warp] = sum;
      top_s[warp] = top;
    }
    __syncthreads();
    if (warp == 0) {
      top = -INFINITY;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = acc_s[w][lane * N + i];
        add(top_s[w], sum_s[w], f);
      }
      finish(row, top, sum, y);
    }
    __syncthreads();
  }
}

// Host: CTAs of the attention kernels, at most (workspaces are sized by it on every device alike).
constexpr int MAX_GRID = 160;
bool code_map(CUtensorMap* map, const void* codes, long long rows, int d, int kt);
// Prompts (kv8_prefill.cu): whether a call's rows are many enough, its workspace, and the launch.
constexpr int PREFILL_ROWS = 256;  // query rows of a unit there
bool is_prefill(int dtype, int head_dim, long long rows);
size_t prefill_workspace(int head_dim);
cudaError_t launch_prefill(AttnParams& q, int format, int head_dim, cudaStream_t st);

}  // namespace kv8
}  // namespace tinfer
