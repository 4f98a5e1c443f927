// head_norm.cu -- RMSNorm of each query and key head with its rotary position, in one pass.
//
//   y = R(pos) (x g / sqrt(mean(x^2) + eps))      mean over the head's head_dim elements, R on its first rotary_dim
//
// Bound by HBM for prompts (every element read and written once), by launch latency for a step. L lanes share a row (a
// power of two, 16 elements a lane: eight and their rotary partners, so that a pair never leaves its thread); the groups
// of L lanes of a CTA are dealt to its TT tokens, and the groups of one token to its heads. A token's angles are computed
// once for all its heads, into shared memory, while the first rows are on their way; a thread keeps those of its pairs
// in registers over its heads. Elements are read and written by the same thread, so rows may be normalised in place.
#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace tinfer {
namespace head_norm {

constexpr int NT = 256, MAX_D = 256, MAX_TT = 8;
constexpr int ROWS = 2;  // rows of a thread in flight

struct Params {
  kv8::Rows q, k, q_out, k_out;
  kv8::Span sp;
  const float* q_gain;  // may be null: ones
  const float* k_gain;
  int n_heads, heads;   // query heads, query and KV heads
  int d, rotary, lanes, tt, tiles;  // lanes of a row, tokens of a CTA, CTAs of a sequence
  float eps;
  unsigned long long freq[MAX_D / 2];  // as in kv8::Rope
};

// A row's factor 1 / sqrt(mean + eps) where the sum of squares leaves fp32's good range (values beyond 2^49 or below
// 2^-49 at most): in fp64, which holds every square of an fp32. Rows like that are rare; others pay one comparison.
__device__ __noinline__ double wide_factor(const float (&x)[16], bool here, int lanes, int d, float eps) {
  double s = 0.0;
  if (here)
    for (int e = 0; e < 16; ++e) s += (double)x[e] * (double)x[e];
  for (int o = lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return 1.0 / sqrt(s / d + (double)eps);
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(NT) head_norm_kernel(const __grid_constant__ Params p) {
  __shared__ float2 angle[MAX_TT * MAX_D / 2];
  __shared__ __align__(16) float gain[2][MAX_D];
  const int seq = (int)(blockIdx.x / p.tiles), t0 = (int)(blockIdx.x % p.tiles) * p.tt;
  const int pos = p.sp.pos[seq], count = p.sp.counts ? p.sp.counts[seq] : p.sp.n_tokens;
  if (pos < 0 || count < 0 || count > p.sp.n_tokens || (long long)pos + count > 0x7FFFFFFFLL) {
    if (threadIdx.x == 0 && p.sp.status) atomicOr(p.sp.status, kv8::STATUS_BAD_POS);
    return;
  }
  if (t0 >= count) return;
  const int lane = threadIdx.x & (p.lanes - 1), group = threadIdx.x / p.lanes, groups = NT / p.lanes / p.tt;
  const int tok = t0 + group / groups, first = group % groups;
  const bool here = lane * 16 < p.d, live = tok < count;
  // elements c and c2 of the lane, eight each: rotary partners, or, past the rotated ones, 16 in a row
  const bool turned = lane * 16 < p.rotary;
  const int c = turned ? lane * 8 : lane * 16, c2 = turned ? p.rotary / 2 + lane * 8 : lane * 16 + 8;

  float x[ROWS][16];
  auto load = [&](int i, int head) {
    if (live && here && head < p.heads) {
      const bool is_k = head >= p.n_heads;
      const kv8::Rows& r = is_k ? p.k : p.q;
      const TI* src = static_cast<const TI*>(r.data) + seq * r.ss + tok * r.ts + (is_k ? head - p.n_heads : head) * r.hs;
      kv8::load8(src + c, reinterpret_cast<float(&)[8]>(x[i][0]));
      kv8::load8(src + c2, reinterpret_cast<float(&)[8]>(x[i][8]));
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[i][e] = 0.f;
    }
  };
#pragma unroll
  for (int i = 0; i < ROWS; ++i) load(i, first + i * groups);

  const int half = p.rotary / 2;
  for (int i = threadIdx.x; i < p.tt * half; i += NT) {
    const int t = i / half, f = i - t * half;
    float cs, sn;
    const unsigned long long ph = p.freq[f] * (unsigned long long)(unsigned)(pos + t0 + t);
    sincospif((float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f, &sn, &cs);
    angle[i] = make_float2(cs, sn);
  }
  for (int i = threadIdx.x; i < p.d; i += NT) {
    gain[0][i] = p.q_gain ? p.q_gain[i] : 1.f;
    gain[1][i] = p.k_gain ? p.k_gain[i] : 1.f;
  }
  __syncthreads();
  float2 a[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = turned ? angle[(tok - t0) * half + c + e] : make_float2(1.f, 0.f);

  for (int h0 = first;; h0 += ROWS * groups) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int head = h0 + i * groups;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) s = fmaf(x[i][e], x[i][e], s);
      for (int o = p.lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
      const float mean = s / (float)p.d + p.eps;
      float r = __frsqrt_rn(mean);
      const bool odd = !(mean > 1e-30f && s < 1e30f);
      if (__any_sync(~0u, odd)) {  // (a whole warp, as the sums of its rows cross lanes)
        const double w = wide_factor(x[i], here, p.lanes, p.d, p.eps);
        if (odd) {
          r = 1.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) x[i][e] = (float)((double)x[i][e] * w);
        }
      }
      if (!live || !here || head >= p.heads) continue;
      const bool is_k = head >= p.n_heads;
      const float* g = gain[is_k];
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = x[i][e] * r * g[(e < 8 ? c : c2 - 8) + e];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = y[e], v = y[8 + e];
        if (turned) {
          y[e] = u * a[e].x - v * a[e].y;
          y[8 + e] = v * a[e].x + u * a[e].y;
        }
      }
      const kv8::Rows& o = is_k ? p.k_out : p.q_out;
      TO* dst = static_cast<TO*>(o.data) + seq * o.ss + tok * o.ts + (is_k ? head - p.n_heads : head) * o.hs;
      kv8::store8(dst + c, y);
      kv8::store8(dst + c2, y + 8);
    }
    if (h0 + ROWS * groups - first >= p.heads) break;  // (alike for the whole CTA: groups share the shuffles' warps)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) load(i, h0 + (ROWS + i) * groups);
  }
}

cudaError_t launch(const Params& p, int in, int out, unsigned grid, cudaStream_t st) {
  using H = __half;
  using B = __nv_bfloat16;
  if (in == TINFER_DTYPE_F32 && out == TINFER_DTYPE_F32) head_norm_kernel<float, float><<<grid, NT, 0, st>>>(p);
  else if (in == TINFER_DTYPE_F32 && out == TINFER_DTYPE_F16) head_norm_kernel<float, H><<<grid, NT, 0, st>>>(p);
  else if (in == TINFER_DTYPE_F32) head_norm_kernel<float, B><<<grid, NT, 0, st>>>(p);
  else if (in == TINFER_DTYPE_F16) head_norm_kernel<H, H><<<grid, NT, 0, st>>>(p);
  else head_norm_kernel<B, B><<<grid, NT, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace head_norm
}  // namespace tinfer

using namespace tinfer;

extern "C" tinfer_status tinfer_op_qk_norm_rope(int n_seqs, int n_tokens, int n_heads, int n_kv_heads, int head_dim,
                                                int rotary_dim, const tinfer_rows* q, const tinfer_rows* k,
                                                const float* q_gain_dev, const float* k_gain_dev, double eps,
                                                double rope_theta, const int32_t* pos_dev, const int32_t* counts_dev,
                                                const tinfer_rows* q_out, const tinfer_rows* k_out, int32_t* status_dev,
                                                void* stream) {
  if (n_seqs < 1 || n_tokens < 1 || n_heads < 1 || n_kv_heads < 1 || head_dim < 1 || !pos_dev) return TINFER_ERR_INVALID_ARG;
  if (!kv8::words_of({pos_dev, counts_dev, status_dev, q_gain_dev, k_gain_dev})) return TINFER_ERR_INVALID_ARG;
  if (!(eps >= 0.0) || !(eps < 1e30)) return TINFER_ERR_INVALID_ARG;
  if (rope_theta != 0.0 && (!(rope_theta >= 1.0) || !(rope_theta <= 1e30))) return TINFER_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > head_dim || (rotary_dim & 1)) return TINFER_ERR_INVALID_ARG;
  if (head_dim % 16 || head_dim > head_norm::MAX_D || rotary_dim % 16) return TINFER_ERR_UNSUPPORTED;
  if (n_heads > 1024 || n_kv_heads > 1024 || n_seqs > (1 << 24) || n_tokens > (1 << 24)) return TINFER_ERR_UNSUPPORTED;
  const kv8::Extent xq{n_seqs, n_tokens, n_heads, head_dim}, xk{n_seqs, n_tokens, n_kv_heads, head_dim};
  head_norm::Params p{};
  if (!kv8::rows_of(q, xq, false, p.q) || !kv8::rows_of(k, xk, false, p.k) || !kv8::rows_of(q_out, xq, true, p.q_out) ||
      !kv8::rows_of(k_out, xk, true, p.k_out))
    return TINFER_ERR_INVALID_ARG;
  if (q->dtype != k->dtype || q_out->dtype != k_out->dtype || q_out->data == k_out->data) return TINFER_ERR_INVALID_ARG;
  if (q->dtype != q_out->dtype && q->dtype != TINFER_DTYPE_F32) return TINFER_ERR_UNSUPPORTED;
  p.sp = kv8::Span{pos_dev, counts_dev, n_tokens, status_dev};
  p.q_gain = q_gain_dev;
  p.k_gain = k_gain_dev;
  p.n_heads = n_heads;
  p.heads = n_heads + n_kv_heads;
  p.d = head_dim;
  p.rotary = rope_theta == 0.0 ? 0 : rotary_dim;
  p.eps = (float)eps;
  for (p.lanes = 1; p.lanes * 16 < head_dim;) p.lanes *= 2;
  for (int i = 0; i < p.rotary / 2; ++i)  // turns of 2^-64; see kv8::Rope
    p.freq[i] = (unsigned long long)(std::pow(rope_theta, -2.0 * i / p.rotary) * 0.15915494309189533577 * 18446744073709551616.0);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return TINFER_ERR_CUDA;
  // a token to a CTA while the tokens are too few to fill the GPU so; else as many as leave each group of lanes three
  // heads, whose loads follow one another and share the angles
  const long long tokens = (long long)n_seqs * n_tokens;
  p.tt = 1;
  while (tokens > 4LL * sms * p.tt && p.tt < head_norm::MAX_TT && p.tt * 2 <= n_tokens && 3 * (head_norm::NT / p.lanes / p.tt) > p.heads) p.tt *= 2;
  p.tiles = (n_tokens + p.tt - 1) / p.tt;
  if ((long long)p.tiles * n_seqs > 0x7FFFFFFFLL) return TINFER_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (status_dev && cudaMemsetAsync(status_dev, 0, 4, st) != cudaSuccess) return TINFER_ERR_CUDA;
  const cudaError_t e = head_norm::launch(p, q->dtype, q_out->dtype, (unsigned)(p.tiles * n_seqs), st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}
