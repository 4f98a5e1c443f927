// kv8.cu -- the 8-bit KV cache: quantising keys and values as they are written, and reading them back.
//
// Each block of tokens of one KV head has one scale for K and one for V; a code stands for code * scale.
// A block is quantised against its largest magnitude, scale = max|x| / QMAX (448 for e4m3, 127 for int8).
// A block that earlier calls have started keeps its scale while the new values fit; otherwise the scale
// grows by the smallest power of two that makes them fit, and the held codes are rounded again in units
// of the new scale. The power of two keeps that harmless: an e4m3 code only moves its exponent (exact
// but for subnormals), and an int8 code's errors form a geometric series below one step, however often
// the block grows.
#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace tinfer {
namespace kv8 {

struct AppendParams {
  Cache c;
  Rows k, v;
  Span sp;
  Rope rope;
};

// The quotient x / s rounded to nearest, from the correctly rounded reciprocal r: with it one correction of the
// product by its exact remainder gives the rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990) in three
// instructions instead of a division's ten. Not where the remainder may underflow: see `plain` below.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// One CTA per (block of the cache, KV head, K or V, sequence). A thread's item is eight dimensions and their rotary
// partners d/2 further of one token; all items of the block stay in registers between the maximum and the rounding,
// so the rows are read once. Bound by issue and HBM alike for prompts (2 or 4 bytes read and 1 written per
// value), by launch latency for single tokens. 32 sequences of up to 2048 tokens, 8 heads of 64, bf16 to e4m3 (193 MB):
// 52 us, 45 without the rotation. Plain divisions and accurate angles took 70, two heads to a CTA to share angles 52.
template <int FMT, int D, typename T, int NT, int IPT>
__global__ void __launch_bounds__(NT) kv8_append_kernel(const __grid_constant__ AppendParams q) {
  constexpr int CPR = D / 16;  // items per row
  const int seq = blockIdx.z, head = blockIdx.y >> 1, is_v = blockIdx.y & 1;
  int pos, count;
  if (!span_of(q.sp, seq, q.c.max_ctx, pos, count)) {
    if (threadIdx.x == 0 && q.sp.status) atomicOr(q.sp.status, STATUS_BAD_POS);
    return;
  }
  const int block = 1 << q.c.lg_block;
  const int b = (pos >> q.c.lg_block) + blockIdx.x;
  const int start = b << q.c.lg_block;  // may pass the end only when there is nothing to do
  const long long end_new = (long long)pos + count;
  if (count == 0 || start >= end_new) return;
  const int t0 = max(pos, start), t1 = (int)min(end_new, (long long)start + block);
  const Rows& r = is_v ? q.v : q.k;
  const T* src = static_cast<const T*>(r.data) + seq * r.ss + head * r.hs;
  const size_t plane = (size_t)seq * q.c.n_kv + head;
  uint8_t* codes = (is_v ? q.c.v : q.c.k) + plane * q.c.max_ctx * D;
  float* scale_p = (is_v ? q.c.vs : q.c.ks) + plane * q.c.n_blocks + b;
  const float held = t0 > start ? *scale_p : 0.f;

  float x[IPT][16];
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const int item = threadIdx.x + i * NT, row = start + item / CPR, c = (item % CPR) * 8;
    if (row >= t0 && row < t1) {
      const T* p = src + (row - pos) * r.ts;
      load8(p + c, reinterpret_cast<float(&)[8]>(x[i][0]));
      load8(p + D / 2 + c, reinterpret_cast<float(&)[8]>(x[i][8]));
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[i][e] = 0.f;
    }
  }
  __shared__ unsigned long long freq[D / 2];
  __shared__ unsigned warp_top[NT / 32];
  if (!is_v && q.rope.on) {
    for (int i = threadIdx.x; i < D / 2; i += NT) freq[i] = q.rope.f[i];  // (threads index it apart)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      const int item = threadIdx.x + i * NT, row = start + item / CPR, c = (item % CPR) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float cs, sn;
        rope_cos_sin_fast(freq[c + e], row, cs, sn);
        const float a = x[i][e], z = x[i][8 + e];
        x[i][e] = a * cs - z * sn;
        x[i][8 + e] = z * cs + a * sn;
      }
    }
  }
  unsigned top = 0;  // largest magnitude as bits: infinities and NaN compare above every finite value
#pragma unroll
  for (int i = 0; i < IPT; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7FFFFFFFu);
  top = __reduce_max_sync(~0u, top);
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();  // (and every thread has read the held scale)
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) top = max(top, warp_top[w]);
  // the scale: a value that is not finite makes it NaN, so that whatever reads the block shows it
  const float amax = __uint_as_float(top);
  float scale;
  if (top >= 0x7F800000u || !(held < INFINITY)) {
    scale = __uint_as_float(0x7FC00000u);
  } else if (held > 0.f) {
    scale = held;
    while ((double)amax > (double)qmax<FMT>() * (double)scale) scale *= 2.f;
  } else {
    scale = top ? fmaxf(amax / qmax<FMT>(), 1.17549435e-38f) : 0.f;
  }
  const bool usable = scale > 0.f;
  if (held > 0.f && usable && scale != held) {  // the started block grew: its held codes in the new units
    const float shrink = held / scale;
    for (int i = threadIdx.x; i < (t0 - start) * (D / 4); i += NT) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes + (size_t)start * D) + i;
      float f[4];
      codes_to_float<FMT>(*w, f);
      *w = floats_to_codes<FMT>(f[0] * shrink, f[1] * shrink, f[2] * shrink, f[3] * shrink);
    }
  }
  const float rcp = usable ? 1.f / scale : 0.f;
  const bool plain = !(scale > 1e-30f && scale < 1e30f);  // far from the range's ends the remainder is exact
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const int item = threadIdx.x + i * NT, row = start + item / CPR, c = (item % CPR) * 8;
    if (row < t0 || row >= t1) continue;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* y = &x[i][4 * e];
      if (plain)
        w[e] = usable ? floats_to_codes<FMT>(y[0] / scale, y[1] / scale, y[2] / scale, y[3] / scale) : 0u;
      else
        w[e] = floats_to_codes<FMT>(quotient(y[0], scale, rcp), quotient(y[1], scale, rcp), quotient(y[2], scale, rcp),
                                    quotient(y[3], scale, rcp));
    }
    uint8_t* dst = codes + (size_t)row * D;
    *reinterpret_cast<uint2*>(dst + c) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(dst + D / 2 + c) = make_uint2(w[2], w[3]);
  }
  if (threadIdx.x == 0) *scale_p = scale;
}

struct ReadParams {
  Cache c;
  Rows k, v;
  Span sp;
};

// A thread takes eight codes at a time, four times: 8-byte loads and 16- or 32-byte stores whose neighbours are the
// neighbouring threads'. Consecutive threads walk one KV head's rows as they lie in the cache. Bound by HBM: 32 sequences
// of up to 2048 tokens, 8 heads of 64, e4m3 to bf16 (193 MB) in 31 us, 0.94 of the measured copy rate.
constexpr int READ_TURNS = 4;

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(256) kv8_read_kernel(const __grid_constant__ ReadParams q) {
  constexpr int CPR = D / 8;
  const int seq = blockIdx.z, head = blockIdx.y >> 1, is_v = blockIdx.y & 1;
  int pos, count;
  if (!span_of(q.sp, seq, q.c.max_ctx, pos, count)) {
    if (threadIdx.x == 0 && q.sp.status) atomicOr(q.sp.status, STATUS_BAD_POS);
    return;
  }
  const size_t plane = (size_t)seq * q.c.n_kv + head;
  const uint8_t* codes = (is_v ? q.c.v : q.c.k) + plane * q.c.max_ctx * D;
  const float* scales = (is_v ? q.c.vs : q.c.ks) + plane * q.c.n_blocks;
  const Rows& r = is_v ? q.v : q.k;
  T* dst = static_cast<T*>(r.data) + seq * r.ss + head * r.hs;
  uint2 w[READ_TURNS];
  float scale[READ_TURNS];
#pragma unroll
  for (int i = 0; i < READ_TURNS; ++i) {
    const long long item = ((long long)blockIdx.x * READ_TURNS + i) * 256 + threadIdx.x, tok = item / CPR;
    if (tok < count) {
      const int row = pos + (int)tok;
      w[i] = *reinterpret_cast<const uint2*>(codes + (size_t)row * D + item % CPR * 8);
      scale[i] = scales[row >> q.c.lg_block];
    }
  }
#pragma unroll
  for (int i = 0; i < READ_TURNS; ++i) {
    const long long item = ((long long)blockIdx.x * READ_TURNS + i) * 256 + threadIdx.x, tok = item / CPR;
    if (tok >= count) break;
    float f[8];
    codes_to_float<FMT>(w[i].x, f);
    codes_to_float<FMT>(w[i].y, f + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale[i];
    store8(dst + tok * r.ts + item % CPR * 8, f);
  }
}

// ---------------------------------------------------------------------------------------- host

bool cache_of(const tinfer_kv8* c, Cache& out, tinfer_status& st) {
  st = TINFER_ERR_INVALID_ARG;
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return false;
  if ((format_of(c) != E4M3 && format_of(c) != INT8) || c->n_seqs < 1 || c->n_kv_heads < 1 || c->max_ctx < 1) return false;
  if (c->block < 16 || c->block > 128 || (c->block & (c->block - 1))) return false;
  if ((reinterpret_cast<uintptr_t>(c->k_codes) & 15) || (reinterpret_cast<uintptr_t>(c->v_codes) & 15) ||
      (reinterpret_cast<uintptr_t>(c->k_scales) & 3) || (reinterpret_cast<uintptr_t>(c->v_scales) & 3))
    return false;
  st = TINFER_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->n_seqs > MAX_SEQS || c->n_kv_heads > 1024 || c->max_ctx > (1 << 24)) return false;
  int lg = 4;
  while ((1 << lg) < c->block) ++lg;
  out = Cache{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scales, c->v_scales,
              c->n_seqs, c->n_kv_heads, c->max_ctx, lg, (c->max_ctx + c->block - 1) / c->block};
  st = TINFER_OK;
  return true;
}

// Rows are read and written in 16-byte words: base and strides have to keep every row on one. The stride of an extent of
// one is not looked at. Rows that are only read may lie anywhere; those that are written must not share memory, which
// the strides show if each, from the smallest on, is no less than what the ones below it span.
bool rows_of(const tinfer_rows* r, const Extent& x, bool written, Rows& out) {
  if (!r || !r->data) return false;
  const int size = r->dtype == TINFER_DTYPE_F32 ? 4 : r->dtype == TINFER_DTYPE_F16 || r->dtype == TINFER_DTYPE_BF16 ? 2 : 0;
  if (!size || (reinterpret_cast<uintptr_t>(r->data) & 15)) return false;
  const int extents[3] = {x.seqs, x.tokens, x.heads};
  long long strides[3] = {r->seq_stride, r->token_stride, r->head_stride};
  for (int i = 0; i < 3; ++i) {
    if (extents[i] == 1) strides[i] = 0;
    if (strides[i] < 0 || strides[i] % (16 / size) || strides[i] > (1LL << 40)) return false;
  }
  out = Rows{r->data, strides[0], strides[1], strides[2]};
  if (!written) return true;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return strides[a] < strides[b]; });
  long long span = x.head_dim;
  for (int i : order) {
    if (extents[i] == 1) continue;
    if (strides[i] < span) return false;
    span += strides[i] * (extents[i] - 1);
  }
  return true;
}

bool words_of(std::initializer_list<const void*> pointers) {
  for (const void* p : pointers)
    if (reinterpret_cast<uintptr_t>(p) & 3) return false;
  return true;
}

bool clear_status(const tinfer_kv8* c, int32_t* status_dev, cudaStream_t st) {
  return !status_dev || (c->format & TINFER_KV8_KEEP_STATUS) || cudaMemsetAsync(status_dev, 0, 4, st) == cudaSuccess;
}

bool rope_of(double theta, int head_dim, Rope& out) {
  out.on = theta != 0.0;
  if (!out.on) return true;
  if (!(theta >= 1.0) || !(theta <= 1e30)) return false;
  for (int i = 0; i < head_dim / 2; ++i) {
    const double turns = std::pow(theta, -2.0 * i / head_dim) * 0.15915494309189533577;  // 1 / 2 pi
    out.f[i] = (unsigned long long)(turns * 18446744073709551616.0);
  }
  return true;
}

namespace {

template <int FMT, int D, typename T>
cudaError_t launch_append_t(const AppendParams& q, cudaStream_t st) {
  const int block = 1 << q.c.lg_block, n = q.sp.n_tokens;
  const dim3 grid((unsigned)((n + block - 2) / block + 1), (unsigned)(2 * q.c.n_kv), (unsigned)q.c.n_seqs);
  switch (block * (D / 16)) {  // items of one block: 64 (16 tokens of 64) to 1024 (128 tokens of 128)
    case 64: kv8_append_kernel<FMT, D, T, 64, 1><<<grid, 64, 0, st>>>(q); break;
    case 128: kv8_append_kernel<FMT, D, T, 128, 1><<<grid, 128, 0, st>>>(q); break;
    case 256: kv8_append_kernel<FMT, D, T, 256, 1><<<grid, 256, 0, st>>>(q); break;
    case 512: kv8_append_kernel<FMT, D, T, 256, 2><<<grid, 256, 0, st>>>(q); break;
    default: kv8_append_kernel<FMT, D, T, 256, 4><<<grid, 256, 0, st>>>(q); break;
  }
  return cudaGetLastError();
}

template <int FMT, int D, typename T>
cudaError_t launch_read_t(const ReadParams& q, cudaStream_t st) {
  const long long items = (long long)q.sp.n_tokens * (D / 8), per = 256 * READ_TURNS;
  const dim3 grid((unsigned)((items + per - 1) / per), (unsigned)(2 * q.c.n_kv), (unsigned)q.c.n_seqs);
  kv8_read_kernel<FMT, D, T><<<grid, 256, 0, st>>>(q);
  return cudaGetLastError();
}

template <int FMT, int D>
cudaError_t launch_append(const AppendParams& q, int dtype, cudaStream_t st) {
  if (dtype == TINFER_DTYPE_F32) return launch_append_t<FMT, D, float>(q, st);
  if (dtype == TINFER_DTYPE_F16) return launch_append_t<FMT, D, __half>(q, st);
  return launch_append_t<FMT, D, __nv_bfloat16>(q, st);
}
template <int FMT, int D>
cudaError_t launch_read(const ReadParams& q, int dtype, cudaStream_t st) {
  if (dtype == TINFER_DTYPE_F32) return launch_read_t<FMT, D, float>(q, st);
  if (dtype == TINFER_DTYPE_F16) return launch_read_t<FMT, D, __half>(q, st);
  return launch_read_t<FMT, D, __nv_bfloat16>(q, st);
}

}  // namespace
}  // namespace kv8
}  // namespace tinfer

using namespace tinfer;

extern "C" {

tinfer_status tinfer_op_kv8_append(const tinfer_kv8* cache, const tinfer_rows* k, const tinfer_rows* v, int n_tokens,
                                   const int32_t* pos_dev, const int32_t* counts_dev, double rope_theta,
                                   int32_t* status_dev, void* stream) {
  kv8::AppendParams q{};
  tinfer_status rc;
  if (!kv8::cache_of(cache, q.c, rc)) return rc;
  if (n_tokens < 1 || n_tokens > cache->max_ctx || !pos_dev || !kv8::words_of({pos_dev, counts_dev, status_dev}))
    return TINFER_ERR_INVALID_ARG;
  const kv8::Extent x{cache->n_seqs, n_tokens, cache->n_kv_heads, cache->head_dim};
  if (!kv8::rows_of(k, x, false, q.k) || !kv8::rows_of(v, x, false, q.v)) return TINFER_ERR_INVALID_ARG;
  if (k->dtype != v->dtype || !kv8::rope_of(rope_theta, cache->head_dim, q.rope)) return TINFER_ERR_INVALID_ARG;
  if (cache->k_codes == cache->v_codes || cache->k_scales == cache->v_scales) return TINFER_ERR_INVALID_ARG;
  q.sp = kv8::Span{pos_dev, counts_dev, n_tokens, status_dev};
  cudaStream_t st = (cudaStream_t)stream;
  if (!kv8::clear_status(cache, status_dev, st)) return TINFER_ERR_CUDA;
  cudaError_t e;
  if (kv8::format_of(cache) == kv8::E4M3)
    e = cache->head_dim == 64 ? kv8::launch_append<kv8::E4M3, 64>(q, k->dtype, st) : kv8::launch_append<kv8::E4M3, 128>(q, k->dtype, st);
  else
    e = cache->head_dim == 64 ? kv8::launch_append<kv8::INT8, 64>(q, k->dtype, st) : kv8::launch_append<kv8::INT8, 128>(q, k->dtype, st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}

tinfer_status tinfer_op_kv8_read(const tinfer_kv8* cache, int n_tokens, const int32_t* pos_dev, const int32_t* counts_dev,
                                 const tinfer_rows* k, const tinfer_rows* v, int32_t* status_dev, void* stream) {
  kv8::ReadParams q{};
  tinfer_status rc;
  if (!kv8::cache_of(cache, q.c, rc)) return rc;
  if (n_tokens < 1 || n_tokens > cache->max_ctx || !pos_dev || !kv8::words_of({pos_dev, counts_dev, status_dev}))
    return TINFER_ERR_INVALID_ARG;
  const kv8::Extent x{cache->n_seqs, n_tokens, cache->n_kv_heads, cache->head_dim};
  if (!kv8::rows_of(k, x, true, q.k) || !kv8::rows_of(v, x, true, q.v)) return TINFER_ERR_INVALID_ARG;
  if (k->dtype != v->dtype || k->data == v->data) return TINFER_ERR_INVALID_ARG;
  q.sp = kv8::Span{pos_dev, counts_dev, n_tokens, status_dev};
  cudaStream_t st = (cudaStream_t)stream;
  if (!kv8::clear_status(cache, status_dev, st)) return TINFER_ERR_CUDA;
  cudaError_t e;
  if (kv8::format_of(cache) == kv8::E4M3)
    e = cache->head_dim == 64 ? kv8::launch_read<kv8::E4M3, 64>(q, k->dtype, st) : kv8::launch_read<kv8::E4M3, 128>(q, k->dtype, st);
  else
    e = cache->head_dim == 64 ? kv8::launch_read<kv8::INT8, 64>(q, k->dtype, st) : kv8::launch_read<kv8::INT8, 128>(q, k->dtype, st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}

}  // extern "C"
