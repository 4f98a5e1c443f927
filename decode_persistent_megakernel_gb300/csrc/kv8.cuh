// kv8.cuh -- shared pieces of the 8-bit KV cache operators (kv8.cu, kv8_attn.cu, kv8_prefill.cu): the
// parameter blocks, the rotary angle, element types and the checks of positions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "ptx.cuh"
#include "tinfer.h"

namespace tinfer {
namespace kv8 {

constexpr int MAX_SEQS = 1024;     // sequences of one call
constexpr int HALF_D_MAX = 64;     // rotary pairs of the widest head
constexpr int STATUS_BAD_POS = 1;  // bits of *status_dev
constexpr int STATUS_TIMEOUT = 2;

// The cache as the kernels see it: codes [n_seqs][n_kv][max_ctx][d], scales [n_seqs][n_kv][n_blocks].
struct Cache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int n_seqs, n_kv, max_ctx, lg_block, n_blocks;
};

// Rows of one tensor: element (seq, token, head, 0) at data + seq*ss + token*ts + head*hs elements.
struct Rows {
  void* data;
  long long ss, ts, hs;
};

// Where each sequence's new tokens stand: tokens [pos[s], pos[s] + count(s)), count(s) = counts[s] or n_tokens.
struct Span {
  const int* pos;
  const int* counts;  // may be null
  int n_tokens;
  int* status;        // may be null
};

// Rotary frequencies in 64-bit fixed-point turns: f[i] = theta^(-2i/d) / 2 pi * 2^64. The phase pos * f
// is taken modulo one turn by the wrap of the 64-bit product, so a far position loses nothing (error
// below pos * 2^-64 turns, plus the 2^-53 of the frequency itself), without any fp64 arithmetic on the
// device, whose rate on this part is a hundredth of the fp32 rate.
struct Rope {
  unsigned long long f[HALF_D_MAX];
  int on;
};

__device__ __forceinline__ void rope_cos_sin(unsigned long long f, int pos, float& c, float& s) {
  const unsigned long long ph = f * (unsigned long long)(unsigned)pos;
  const float half_turns = (float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f;  // 2^-31: [-1, 1)
  sincospif(half_turns, &s, &c);
}

// The same in a few instructions, off by 2^-20 at most (the functions' stated 2^-21.2, the angle's rounding 2^-22.6):
// for keys that are rounded to 8 bits next, in half steps of 2^-8 of their block's largest value (int8) or of 2^-4
// of their own down to 2^-18.8 of the largest (e4m3). Accurate ones were a third of the append's instructions.
__device__ __forceinline__ void rope_cos_sin_fast(unsigned long long f, int pos, float& c, float& s) {
  const unsigned long long ph = f * (unsigned long long)(unsigned)pos;
  const float angle = (float)(int)(unsigned)(ph >> 32) * (4.656612873077393e-10f * 3.14159265358979f);  // [-pi, pi)
  s = __sinf(angle);
  c = __cosf(angle);
}

// First position and number of new tokens of a sequence; false (and status) when they are outside the cache.
__device__ __forceinline__ bool span_of(const Span& sp, int seq, int max_ctx, int& pos, int& count) {
  pos = sp.pos[seq];
  count = sp.counts ? sp.counts[seq] : sp.n_tokens;
  const bool ok = pos >= 0 && count >= 0 && count <= sp.n_tokens && (long long)pos + count <= max_ctx;
  if (!ok) {
    pos = 0;
    count = 0;
  }
  return ok;
}

// ---- element types: eight values from or to 16-byte aligned rows --------------------------------
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__half* p, const float* x) {
  __half2 h[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}

// Eight values to 16-byte aligned memory.
__device__ __forceinline__ void store8(float* p, const float* x) {
  store4(p, x);
  store4(p + 4, x + 4);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
  T h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) store_one(h + i, x[i]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}

// ---- 8-bit codes ----------------------------------------------------------------------------------
constexpr int E4M3 = TINFER_KV8_E4M3, INT8 = TINFER_KV8_INT8;

template <int FMT>
__device__ __forceinline__ constexpr float qmax() { return FMT == E4M3 ? 448.f : 127.f; }

// Four codes to fp16 (exact: an e4m3 value has 4 significant bits within fp16's range, an int8 one 7).
// int8: the byte with its sign flipped placed under the exponent of 1024 reads 1024 + (code + 128).
template <int FMT>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t bias = 0x64806480u;  // 1152
    uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 p = __hsub2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
    const __half2 q = __hsub2(*reinterpret_cast<__half2*>(&y), *reinterpret_cast<const __half2*>(&bias));
    lo = *reinterpret_cast<const uint32_t*>(&p);
    hi = *reinterpret_cast<const uint32_t*>(&q);
  }
}
template <int FMT>
__device__ __forceinline__ void codes_to_float(uint32_t w, float* x) {
  uint32_t a, b;
  codes_to_half<FMT>(w, a, b);
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&a)), g = __half22float2(*reinterpret_cast<__half2*>(&b));
  x[0] = f.x; x[1] = f.y; x[2] = g.x; x[3] = g.y;
}
// Four values in units of the scale to codes: nearest, ties to even, saturating.
template <int FMT>
__device__ __forceinline__ uint32_t floats_to_codes(float a, float b, float c, float d) {
  if (FMT == E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  // adding 1.5 * 2^23 leaves the nearest integer (ties to even) in the low bits
  auto one = [](float x) { return __float_as_uint(fminf(fmaxf(x, -127.f), 127.f) + 12582912.f); };
  return __byte_perm(__byte_perm(one(a), one(b), 0x0040), __byte_perm(one(c), one(d), 0x0040), 0x5410);
}

// ---- host side, shared by the entry points (kv8.cu) ----------------------------------------------
inline int format_of(const tinfer_kv8* c) { return c->format & ~(TINFER_KV8_KEEP_STATUS | TINFER_KV8_DEBUG_WITHHOLD); }
bool clear_status(const tinfer_kv8* c, int32_t* status_dev, cudaStream_t st);
bool cache_of(const tinfer_kv8* c, Cache& out, tinfer_status& st);
struct Extent {
  int seqs, tokens, heads, head_dim;
};
bool rows_of(const tinfer_rows* r, const Extent& x, bool written, Rows& out);
bool rope_of(double theta, int head_dim, Rope& out);
bool words_of(std::initializer_list<const void*> pointers);  // whether each is aligned to 4 bytes (or null)

}  // namespace kv8
}  // namespace tinfer
