// kv8_attn.cu -- attention of the last tokens of each sequence over its 8-bit KV cache.
//
//   o_i = sum_{j <= pos+i} softmax_j(q_i . k_j / sqrt(d)) v_j,   k_j = ck_j * sk[j / block], v_j = cv_j * sv[j / block]
//
// The n_tokens x group query rows that share a KV head are the rows of one matrix: every code is read
// and widened once for all of them. The work is a flat list of key tiles (sequence, KV head, row tile,
// tile of KT keys); each CTA takes an equal run of it, whatever the sequences' lengths, so that one long
// sequence spreads over the GPU and a ragged batch stays even. A run that covers a (sequence, head) only
// in part leaves (m, l, o) in the workspace, and kv8_merge_kernel joins the parts in order, so results
// do not depend on timing.
//
// Inside a CTA each warp streams its own tiles: a ring of bulk asynchronous copies per warp that runs on
// across the boundaries of the units, no barrier between the warps until a unit ends. Products run on the
// legacy warp-level tensor instruction (m16n8k16, fp16 in, fp32 accumulation): at 16 or 32 rows the
// kernel is bound by the cache's bytes, the tensor pipe is not the limit, and register operands let the
// codes go from shared memory to the product without being stored again in 16 bits.
//
// Precision. Codes widen to fp16 exactly. A query row is divided by the power of two above its largest
// magnitude, which keeps it in fp16's range, and multiplied back in the scores' fp32 scale. Query and
// weight are rounded to fp16 (2^-12 relative) for bf16 queries, whose own result is rounded to 2^-9; for
// fp32 and fp16 queries both enter as two fp16 parts (high and the remainder: 2^-23), with twice the
// products. Scores, maxima, sums and outputs are fp32.
//
// A key's V scale 2^e * f (1 <= f < 2) enters its weight: the running maximum M is taken over x + e (x
// the score in units of log 2), the weight of V is w * f with w = 2^(x + e - M), and the sum of the
// softmax adds w * 2^-e. So weights are near 1 where they matter whatever the scales of the blocks are.
#include <algorithm>
#include <cmath>

#include "kv8.cuh"
#include "kv8_attn.cuh"

namespace tinfer {
namespace kv8 {

constexpr int NW = 8;               // warps of a CTA
constexpr int NTHREADS_ATTN = NW * 32;
constexpr int STAGES = 3;
constexpr int WEIGHT_SHIFT = 14;    // weights are held times 2^14: fp16 keeps 11 bits of them down to 2^-28
// Exponents of V scales that enter the running maximum. Of a row whose keys all have the smallest one the
// sum of the softmax is 2^(WEIGHT_SHIFT - E_MIN) for each key: 2^24 keys stay below fp32's 2^128. A smaller
// scale's remainder makes its weights smaller than 1, a scale of 0 makes them 0 and counts in the sum.
constexpr int E_MIN = -85, E_MAX = 120;
constexpr long long WAIT_NS = 200LL * 1000 * 1000;

template <int D>
struct Shape {
  static constexpr int KT = 4096 / D;              // keys of one tile: 64 or 32, 4 KiB of K and 4 of V
  static constexpr int STAGE_BYTES = 2 * KT * D;
};

// ---- the list of work -------------------------------------------------------------------------
// Sequence s holds ceil(len / KT) tiles for each of its units (KV head, row tile). prefix[s] counts the
// tiles before it. Called by all threads of a CTA; returns the total.
template <int D, int NT>
__device__ int build_prefix(const AttnParams& q, int* prefix, int* scan) {
  constexpr int KT = Shape<D>::KT;
  int carry = 0;
  for (int base = 0; base < q.c.n_seqs; base += NT) {
    const int s = base + threadIdx.x;
    int tiles = 0;
    if (s < q.c.n_seqs) {
      int pos, count;
      if (!span_of(q.sp, s, q.c.max_ctx, pos, count) && blockIdx.x == 0 && q.sp.status)
        atomicOr(q.sp.status, STATUS_BAD_POS);
      if (count > 0) tiles = (pos + count + KT - 1) / KT * q.units;
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(~0u, incl, o);
      if ((threadIdx.x & 31) >= o) incl += y;
    }
    if ((threadIdx.x & 31) == 31) scan[threadIdx.x >> 5] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < NT / 32; ++w) {
      const int y = scan[w];
      if (w < (int)(threadIdx.x >> 5)) before += y;
      carry += y;
    }
    if (s < q.c.n_seqs) prefix[s] = before + incl - tiles;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[q.c.n_seqs] = carry;
  __syncthreads();
  return carry;
}

__device__ __forceinline__ int tiles_per_cta(const AttnParams& q, int total, int grid) {
  return max((total + grid - 1) / grid, q.min_tiles);
}

// The sequence that holds tile x of the list.
__device__ __forceinline__ int seq_of(const int* prefix, int n, int x) {
  int lo = 0, hi = n;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A place in the list.
template <int D>
struct Place {
  int x, seq, unit, tile, tiles;  // tiles: of one unit of this sequence
  int pos, count;
  __device__ void enter(const AttnParams& q) {
    pos = q.sp.pos[seq];
    count = q.sp.counts ? q.sp.counts[seq] : q.sp.n_tokens;
    tiles = (pos + count + Shape<D>::KT - 1) / Shape<D>::KT;
  }
  __device__ void seek(const AttnParams& q, const int* prefix, int at) {
    x = at;
    if (at >= prefix[q.c.n_seqs]) return;
    seq = seq_of(prefix, q.c.n_seqs, at);
    enter(q);
    const int in = at - prefix[seq];
    unit = in / tiles;
    tile = in - unit * tiles;
  }
  __device__ void advance(const AttnParams& q, const int* prefix, int by, int end) {
    x += by;
    tile += by;
    if (x >= end || tile < tiles) return;
    if (x < prefix[seq + 1]) {
      const int up = tile / tiles;
      unit += up;
      tile -= up * tiles;
    } else {
      seek(q, prefix, x);
    }
  }
  // Keys that the rows of this unit can see, counted from the first key of the tile.
  template <int ROWS>
  __device__ int keys(const AttnParams& q) const {
    const int rt = unit % q.row_tiles;
    if (rt * ROWS >= q.group * count) return 0;  // no rows here: the sequence has fewer new tokens
    const int last = min(min((rt * ROWS + ROWS - 1) / q.group, q.sp.n_tokens - 1), count - 1);
    return min(pos + last + 1 - tile * Shape<D>::KT, Shape<D>::KT);
  }
};

// ---- small wrappers ------------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The remainder of a pair after its rounding to fp16, again in fp16.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t high) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&high));
  return pack_half(a - h.x, b - h.y);
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if ((long long)(globaltimer() - t0) > WAIT_NS) return false;
  return true;
}

// ---- the kernel ----------------------------------------------------------------------------------
template <int D, int MT>
struct Smem {
  static constexpr int ROWS = 16 * MT;
  static constexpr int SCALES = Shape<D>::KT / 16;  // scales of one tile, at most (blocks of 16)
  alignas(128) uint8_t ring[NW][STAGES][Shape<D>::STAGE_BYTES];
  float ring_scale[NW][STAGES][2][SCALES];
  alignas(16) float part[NW][16][32 + 4];  // one pass of the merge of the warps: 16 rows x 32 dimensions
  float m[NW][ROWS], l[NW][ROWS];
  alignas(16) uint32_t qf[2][MT][D / 16][32][4];  // query fragments: high and remainder
  float row_scale[ROWS];
  alignas(8) unsigned long long full[NW][STAGES];
  int scan[NW];
  int failed;
};

template <int FMT, int D, int MT, int SPLIT, typename T>
__global__ void __launch_bounds__(NTHREADS_ATTN, 1) kv8_attn_kernel(const __grid_constant__ AttnParams q) {
  constexpr int KT = Shape<D>::KT, NT = KT / 8, ROWS = 16 * MT, DB = D / 8;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem<D, MT>& sm = *reinterpret_cast<Smem<D, MT>*>(smem_raw);
  int* prefix = reinterpret_cast<int*>(smem_raw + sizeof(Smem<D, MT>));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  if (lane == 0)
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_addr(&sm.full[warp][s]), 33);  // the copy and 32 lanes' scales
  if (tid == 0) sm.failed = 0;
  mbar_fence_init();
  const int total = build_prefix<D, NTHREADS_ATTN>(q, prefix, sm.scan);
  const int per = tiles_per_cta(q, total, gridDim.x);
  const int lo = (int)min((long long)per * blockIdx.x, (long long)total), hi = min(lo + per, total);
  if (lo >= hi) return;

  // this warp's tiles: those of [lo, hi) congruent to its index, so that the warps' shares stay even
  const int first = lo + ((warp - lo) & (NW - 1));
  Place<D> in, at;
  in.seek(q, prefix, first);
  int put = 0, got = 0;
  const uint64_t policy = q.keep_l2 ? policy_evict_normal() : policy_evict_first();
  auto issue = [&]() {  // the next tile that has keys to read goes into the ring
    int keys = 0;
    while (in.x < hi && (keys = in.template keys<ROWS>(q)) <= 0) in.advance(q, prefix, NW, hi);
    if (in.x >= hi) return;
    const int st = put % STAGES;
    const uint32_t bar = smem_addr(&sm.full[warp][st]);
    const size_t plane = (size_t)in.seq * q.c.n_kv + in.unit / q.row_tiles;
    const size_t off = (plane * q.c.max_ctx + (size_t)in.tile * KT) * D;
    if (lane == 0) {
      const uint32_t dst = smem_addr(sm.ring[warp][st]), bytes = (uint32_t)keys * D;
      mbar_arrive_expect_tx(bar, 2 * bytes);
      bulk_g2s(dst, q.c.k + off, bytes, bar, policy);
      bulk_g2s(dst + KT * D, q.c.v + off, bytes, bar, policy);
    }
    const int b0 = in.tile * KT >> q.c.lg_block, nb = ((in.tile * KT + keys - 1) >> q.c.lg_block) - b0 + 1;
    if (lane < nb) {
      cp_async_4(smem_addr(&sm.ring_scale[warp][st][0][lane]), q.c.ks + plane * q.c.n_blocks + b0 + lane);
      cp_async_4(smem_addr(&sm.ring_scale[warp][st][1][lane]), q.c.vs + plane * q.c.n_blocks + b0 + lane);
    }
    cp_async_arrive(bar);
    ++put;
    in.advance(q, prefix, NW, hi);
  };
  __syncwarp();
#pragma unroll
  for (int s = 0; s < STAGES; ++s) issue();
  at.seek(q, prefix, first);

  Place<D> seg;  // the unit that the CTA works on
  seg.seek(q, prefix, lo);
  while (seg.x < hi) {
    const int seg_end = min(hi, seg.x + seg.tiles - seg.tile);
    const bool whole = seg.tile == 0 && seg_end - seg.x == seg.tiles;
    const int head = seg.unit / q.row_tiles, rt = seg.unit % q.row_tiles;
    const int rows = min(q.group * seg.count - rt * ROWS, ROWS);  // rows of this unit (may be <= 0)

    // query rows: rotated, divided by a power of two, laid out as the products' left operands. Warp w
    // takes rows w, w + 8, ...; a lane the rotary pairs of D / 64 dimensions (lane and lane + 32).
    for (int r = warp; r < ROWS; r += NW) {
      float v[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[i] = 0.f;
      if (r < rows) {
        const int row = rt * ROWS + r, tok = row / q.group, hq = head * q.group + row % q.group;
        const T* p = static_cast<const T*>(q.q.data) + seg.seq * q.q.ss + tok * q.q.ts + hq * q.q.hs;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const int e = lane + 32 * i;
          float a = (float)p[e], z = (float)p[e + D / 2];
          if (q.rope.on) {
            float cs, sn;
            rope_cos_sin(q.rope.f[e], seg.pos + tok, cs, sn);
            const float a2 = a * cs - z * sn;
            z = z * cs + a * sn;
            a = a2;
          }
          v[i] = a;
          v[D / 64 + i] = z;
        }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      const int e2 = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 126, -100), 100) : 0;  // top < 2^e2
      const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
      if (lane == 0) sm.row_scale[r] = q.scale_log2 * __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // dimension e belongs to thread e / (D/4) of the quad, fragment (e % (D/4)) / 4, and to the
        // words a0/a1 (rows g, g + 8) or a2/a3, low or high half
        const int e = (i < D / 64 ? lane + 32 * i : D / 2 + lane + 32 * (i - D / 64));
        const int qt = e / (D / 4), in4 = e % (D / 4), ks = in4 / 4, w = (in4 & 2) + ((r & 8) ? 1 : 0);
        const float y = v[i] * down;
        const __half h = __float2half_rn(y);
        __half* f0 = reinterpret_cast<__half*>(&sm.qf[0][r / 16][ks][(r & 7) * 4 + qt][w]) + (in4 & 1);
        *f0 = h;
        if (SPLIT == 2)
          reinterpret_cast<__half*>(&sm.qf[1][r / 16][ks][(r & 7) * 4 + qt][w])[in4 & 1] = __float2half_rn(y - __half2float(h));
      }
    }
    __syncthreads();
    uint32_t qf[SPLIT][MT][D / 16][4];
    float rs[MT][2];
    int limit[MT][2];  // first key that a row does not see
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int h = 0; h < SPLIT; ++h)
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint4 w = *reinterpret_cast<const uint4*>(sm.qf[h][m][k][lane]);
          qf[h][m][k][0] = w.x; qf[h][m][k][1] = w.y; qf[h][m][k][2] = w.z; qf[h][m][k][3] = w.w;
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        rs[m][h] = sm.row_scale[m * 16 + h * 8 + g];
        limit[m][h] = seg.pos + min((rt * ROWS + m * 16 + h * 8 + g) / q.group, seg.count - 1) + 1;
      }
    }
    float o[MT][DB][4], mx[MT][2], l[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][j][i] = 0.f;
      mx[m][0] = mx[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
    }

    while (at.x < seg_end) {
      const int keys = at.template keys<ROWS>(q);
      if (keys <= 0) {
        at.advance(q, prefix, NW, hi);
        continue;
      }
      const int st = got % STAGES;
      const int key0 = at.tile * KT;
      if (!wait_bounded(smem_addr(&sm.full[warp][st]), (got / STAGES) & 1)) sm.failed = 1;
      uint8_t* kbuf = sm.ring[warp][st];
      uint8_t* vbuf = kbuf + KT * D;
      if (keys < KT) {  // rows past the copy: weights there are 0, so V must be finite
        for (int i = lane; i < (KT - keys) * (D / 16); i += 32)
          reinterpret_cast<uint4*>(vbuf + keys * D)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
      }
      const int rel = key0 & ((1 << q.c.lg_block) - 1);
      // ---- scores: n-tile j holds keys 8j .. 8j+7, column n of it key 8j + (n >> 1) + 4 (n & 1)
      float s[MT][NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int m = 0; m < MT; ++m) s[m][j][0] = s[m][j][1] = s[m][j][2] = s[m][j][3] = 0.f;
        const uint8_t* kr = kbuf + (8 * j + (g >> 1) + 4 * (g & 1)) * D + t * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(kr + 16 * c);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b0, b1;
            codes_to_half<FMT>(ws[k], b0, b1);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int h = 0; h < SPLIT; ++h) mma16816(s[m][j], qf[h][m][c * 4 + k], b0, b1);
          }
        }
      }
      // ---- x + e for every score, masked; the rows' maxima
      float vf[NT], vinv[NT];
      const bool edge = keys < KT || key0 + KT > limit[0][0];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int b = (rel + 8 * j) >> q.c.lg_block;
        const float ks = sm.ring_scale[warp][st][0][b], vs = sm.ring_scale[warp][st][1][b];
        const int e = min(max((int)((__float_as_uint(vs) >> 23) & 0xFF) - 127, E_MIN), E_MAX);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        // a scale that is not finite reaches its scores, so that the mask decides which rows it spoils
        const bool fine = vs < INFINITY;
        vf[j] = fine && vs > 0.f ? vs * inv : 0.f;
        vinv[j] = inv;
        const float fe = fine ? (float)e : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][j][i] = fmaf(s[m][j][i], ks * rs[m][i >> 1], fe);
      }
      if (edge) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 8 * j + t + 4 * (i & 1);
              if (key >= keys || key0 + key >= limit[m][i >> 1]) s[m][j][i] = -INFINITY;
            }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < NT; ++j) top = fmaxf(top, fmaxf(s[m][j][2 * h], s[m][j][2 * h + 1]));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          const float now = fmaxf(mx[m][h], top);
          const float ref = now == -INFINITY ? 0.f : now;
          const float shrink = exp2_fast(mx[m][h] - ref);
          mx[m][h] = now;
          l[m][h] *= shrink;
#pragma unroll
          for (int j = 0; j < DB; ++j) {
            o[m][j][2 * h] *= shrink;
            o[m][j][2 * h + 1] *= shrink;
          }
          const float from = ref - (float)WEIGHT_SHIFT;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 2 * h; i < 2 * h + 2; ++i) {
              const float w = exp2_fast(s[m][j][i] - from);
              l[m][h] = fmaf(w, vinv[j], l[m][h]);
              s[m][j][i] = w * vf[j];
            }
        }
      // ---- o += weights V, 16 keys at a time
#pragma unroll
      for (int p = 0; p < NT / 2; ++p) {
        uint32_t a[SPLIT][MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = s[m][2 * p + (i >> 1)][2 * (i & 1)], w = s[m][2 * p + (i >> 1)][2 * (i & 1) + 1];
            a[0][m][i] = pack_half(u, w);
            if (SPLIT == 2) a[SPLIT - 1][m][i] = pack_rest(u, w, a[0][m][i]);
          }
        // four keys of this thread; dimensions g * DB .. g * DB + DB - 1, n-tile j of the product
        // holding dimension g * DB + j in column g
        const uint8_t* vr = vbuf + (16 * p + t) * D + g * DB;
        uint32_t w[4][DB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* row = vr + 4 * i * D;  // keys t, t + 4 (first n-tile), t + 8, t + 12 (second)
          if (DB == 8) {
            const uint2 y = *reinterpret_cast<const uint2*>(row);
            w[i][0] = y.x; w[i][1] = y.y;
          } else {
            const uint4 y = *reinterpret_cast<const uint4*>(row);
            w[i][0] = y.x; w[i][1] = y.y; w[i][DB / 4 - 2] = y.z; w[i][DB / 4 - 1] = y.w;
          }
        }
#pragma unroll
        for (int c = 0; c < DB / 4; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // dimensions 4c + 2h and 4c + 2h + 1: interleave the two keys' bytes
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t b0[2], b1[2];
            codes_to_half<FMT>(__byte_perm(w[0][c], w[1][c], sel), b0[0], b0[1]);
            codes_to_half<FMT>(__byte_perm(w[2][c], w[3][c], sel), b1[0], b1[1]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int sp = 0; sp < SPLIT; ++sp) mma16816(o[m][4 * c + 2 * h + u], a[sp][m], b0[u], b1[u]);
          }
      }
      __syncwarp();
      ++got;
      at.advance(q, prefix, NW, hi);
      issue();
    }

    // ---- the warps' parts of this unit, joined in order of the warps
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[m][h] += __shfl_xor_sync(~0u, l[m][h], 1);
        l[m][h] += __shfl_xor_sync(~0u, l[m][h], 2);
        if (t == 0) {
          sm.m[warp][m * 16 + h * 8 + g] = mx[m][h];
          sm.l[warp][m * 16 + h * 8 + g] = l[m][h];
        }
      }
    __syncthreads();
    const int slot = 2 * blockIdx.x + (seg.tile == 0 ? 1 : 0);
    float* part = q.part + (size_t)slot * ROWS * (D + 2);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float shrink[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, sm.m[w][m * 16 + h * 8 + g]);
        shrink[h] = mx[m][h] == -INFINITY ? 0.f : exp2_fast(mx[m][h] - top);
      }
#pragma unroll
      for (int pass = 0; pass < D / 32; ++pass) {
        // dimension of o[m][j][i] is (2t + (i & 1)) * DB + j; a pass holds dimensions [32 pass, 32 pass + 32)
        if (2 * t * DB / 32 == pass) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d0 = (2 * t + (i & 1)) * DB - 32 * pass;
#pragma unroll
            for (int j = 0; j < DB; j += 4)
              *reinterpret_cast<float4*>(&sm.part[warp][(i >> 1) * 8 + g][d0 + j]) =
                  make_float4(o[m][j][i] * shrink[i >> 1], o[m][j + 1][i] * shrink[i >> 1],
                              o[m][j + 2][i] * shrink[i >> 1], o[m][j + 3][i] * shrink[i >> 1]);
          }
        }
        __syncthreads();
        const int r = tid >> 3, c = (tid & 7) * 4;  // 16 rows x 8 threads of four dimensions
        const int row = m * 16 + r;
        if (r < 16 && row < rows) {
          float top = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
          for (int w = 0; w < NW; ++w) top = fmaxf(top, sm.m[w][row]);
          for (int w = 0; w < NW; ++w) {
            const float lw = sm.l[w][row];
            if (lw == 0.f) continue;  // this warp saw no key of the row
            sum = fmaf(lw, exp2_fast(sm.m[w][row] - top), sum);
            const float4 y = *reinterpret_cast<const float4*>(&sm.part[w][r][c]);
            acc[0] += y.x; acc[1] += y.y; acc[2] += y.z; acc[3] += y.w;
          }
          if (whole) {
            const float inv = 1.f / sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] *= inv;
            const int qrow = rt * ROWS + row, tok = qrow / q.group, hq = head * q.group + qrow % q.group;
            T* dst = static_cast<T*>(q.out.data) + seg.seq * q.out.ss + tok * q.out.ts + hq * q.out.hs + 32 * pass + c;
            store4(dst, acc);
            if (q.lse && pass == 0 && c == 0)
              q.lse[((size_t)seg.seq * q.sp.n_tokens + tok) * q.n_heads + hq] =
                  (log2f(sum) + top - (float)WEIGHT_SHIFT) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float4*>(part + (size_t)row * D + 32 * pass + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (pass == 0 && c == 0) {
              part[ROWS * D + row] = top;
              part[ROWS * D + ROWS + row] = sum;
            }
          }
        }
        __syncthreads();
      }
    }
    seg.advance(q, prefix, seg_end - seg.x, hi);
  }
  if (tid == 0 && sm.failed && q.sp.status) atomicOr(q.sp.status, STATUS_TIMEOUT);
}

// Joins the parts of one unit that several CTAs hold, in order. One CTA per unit of a sequence, one warp
// per row at a time, a lane D / 32 dimensions.
template <int D, int MT, typename T>
__global__ void __launch_bounds__(NTHREADS_ATTN) kv8_merge_kernel(const __grid_constant__ AttnParams q) {
  constexpr int KT = Shape<D>::KT, ROWS = 16 * MT, N = D / 32;
  extern __shared__ int prefix[];
  __shared__ int scan[NW];
  pdl_wait();  // the parts are complete
  const int total = build_prefix<D, NTHREADS_ATTN>(q, prefix, scan);
  const int per = tiles_per_cta(q, total, q.grid);
  const int seq = blockIdx.x / q.units, unit = blockIdx.x % q.units;
  int pos, count;
  if (!span_of(q.sp, seq, q.c.max_ctx, pos, count) || count == 0) return;
  const int tiles = (pos + count + KT - 1) / KT;
  const int a = prefix[seq] + unit * tiles, c0 = a / per, c1 = (a + tiles - 1) / per;
  if (c0 == c1) return;  // one CTA had it whole
  const int head = unit / q.row_tiles, rt = unit % q.row_tiles;
  const int rows = min(q.group * count - rt * ROWS, ROWS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t stride = (size_t)ROWS * (D + 2);
  for (int row = warp; row < rows; row += NW) {
    auto part = [&](int c) { return q.part + (size_t)(2 * c + (c == c0 ? 1 : 0)) * stride; };
    float top = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, part(c)[ROWS * D + row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    float sum = 0.f, acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const float* p = part(c);
      const float m = p[ROWS * D + row];
      const float lc = p[ROWS * D + ROWS + row];
      const float w = lc == 0.f ? 0.f : exp2_fast(m - top);
      sum = fmaf(lc, w, sum);
      const float* y = p + (size_t)row * D + lane * N;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 f = *reinterpret_cast<const float2*>(y + i);
        acc[i] = fmaf(f.x, w, acc[i]);
        acc[i + 1] = fmaf(f.y, w, acc[i + 1]);
      }
    }
    const float inv = 1.f / sum;
    const int qrow = rt * ROWS + row, tok = qrow / q.group, hq = head * q.group + qrow % q.group;
    T* dst = static_cast<T*>(q.out.data) + seq * q.out.ss + tok * q.out.ts + hq * q.out.hs + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) store_one(dst + i, acc[i] * inv);
    if (q.lse && lane == 0)
      q.lse[((size_t)seq * q.sp.n_tokens + tok) * q.n_heads + hq] =
          (log2f(sum) + top - (float)WEIGHT_SHIFT) * 0.6931471805599453f;
  }
}

// ---------------------------------------------------------------------------------------- host
namespace {

// Row tiles of 16, or of 32 where 16 would read the cache more than once and the registers allow it.
int rows_per_tile(int rows, int head_dim) { return rows > 16 && head_dim == 64 ? 32 : 16; }

template <int FMT, int D, int MT, int SPLIT, typename T>
cudaError_t launch_t(const AttnParams& q, cudaStream_t st) {
  auto kernel = kv8_attn_kernel<FMT, D, MT, SPLIT, T>;
  const size_t smem = sizeof(Smem<D, MT>) + (size_t)(q.c.n_seqs + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<q.grid, NTHREADS_ATTN, smem, st>>>(q);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(q.c.n_seqs * q.units));
  cfg.blockDim = dim3(NTHREADS_ATTN);
  cfg.dynamicSmemBytes = (size_t)(q.c.n_seqs + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D, MT, T>, q);
}

template <int FMT, int D, int MT>
cudaError_t launch_m(const AttnParams& q, int dtype, cudaStream_t st) {
  if (dtype == TINFER_DTYPE_F32) return launch_t<FMT, D, MT, 2, float>(q, st);
  if (dtype == TINFER_DTYPE_F16) return launch_t<FMT, D, MT, 2, __half>(q, st);
  return launch_t<FMT, D, MT, 1, __nv_bfloat16>(q, st);
}
template <int FMT>
cudaError_t launch_f(const AttnParams& q, int head_dim, int rows, int dtype, cudaStream_t st) {
  if (head_dim == 128) return launch_m<FMT, 128, 1>(q, dtype, st);
  return rows == 32 ? launch_m<FMT, 64, 2>(q, dtype, st) : launch_m<FMT, 64, 1>(q, dtype, st);
}

// Multiprocessors of the current device.
int device_sms(int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// CTAs of the attention kernel, at most: the workspace is sized by this on every device alike.
constexpr int MAX_GRID = 256;

}  // namespace
}  // namespace kv8
}  // namespace tinfer

using namespace tinfer;

extern "C" {

size_t tinfer_kv8_attention_workspace(const tinfer_kv8* cache, int n_heads, int n_tokens) {
  kv8::Cache c;
  tinfer_status rc;
  if (!kv8::cache_of(cache, c, rc) || n_heads < 1 || n_heads % cache->n_kv_heads || n_tokens < 1) return 0;
  // one size for every number of rows, so that a program can keep one workspace for all its calls
  return (size_t)kv8::MAX_GRID * 2 * kv8::rows_per_tile(17, cache->head_dim) * (cache->head_dim + 2) * 4;
}

tinfer_status tinfer_op_kv8_attention(const tinfer_kv8* cache, int n_heads, int n_tokens, const tinfer_rows* q_rows,
                                      const int32_t* pos_dev, const int32_t* counts_dev, double rope_theta,
                                      const tinfer_rows* out_rows, float* lse_dev, void* workspace_dev,
                                      size_t workspace_bytes, int32_t* status_dev, void* stream) {
  kv8::AttnParams q{};
  tinfer_status rc;
  if (!kv8::cache_of(cache, q.c, rc)) return rc;
  if (n_heads < 1 || n_heads % cache->n_kv_heads || n_tokens < 1 || n_tokens > cache->max_ctx || !pos_dev)
    return TINFER_ERR_INVALID_ARG;
  const kv8::Extent x{cache->n_seqs, n_tokens, n_heads, cache->head_dim};
  if (!kv8::rows_of(q_rows, x, false, q.q) || !kv8::rows_of(out_rows, x, true, q.out) || q_rows->dtype != out_rows->dtype)
    return TINFER_ERR_INVALID_ARG;
  if (!kv8::rope_of(rope_theta, cache->head_dim, q.rope)) return TINFER_ERR_INVALID_ARG;
  if (!workspace_dev || (reinterpret_cast<uintptr_t>(workspace_dev) & 15) ||
      workspace_bytes < tinfer_kv8_attention_workspace(cache, n_heads, n_tokens))
    return TINFER_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(lse_dev) & 3) return TINFER_ERR_INVALID_ARG;
  q.group = n_heads / cache->n_kv_heads;
  q.n_heads = n_heads;
  const long long rows = (long long)q.group * n_tokens;
  const int per = kv8::rows_per_tile(rows > 16 ? 17 : 1, cache->head_dim);
  const long long row_tiles = (rows + per - 1) / per, units = row_tiles * cache->n_kv_heads;
  const int kt = 4096 / cache->head_dim;
  // the list of tiles is counted in 32 bits
  if (units * cache->n_seqs > (1LL << 30) / ((cache->max_ctx + kt - 1) / kt)) return TINFER_ERR_UNSUPPORTED;
  q.row_tiles = (int)row_tiles;
  q.units = (int)units;
  q.sp = kv8::Span{pos_dev, counts_dev, n_tokens, status_dev};
  q.lse = lse_dev;
  q.part = static_cast<float*>(workspace_dev);
  q.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)cache->head_dim));
  q.min_tiles = 1;
  q.keep_l2 = row_tiles > 1;
  int sms = 0;
  if (!kv8::device_sms(sms)) return TINFER_ERR_CUDA;
  q.grid = std::min(sms, kv8::MAX_GRID);
  cudaStream_t st = (cudaStream_t)stream;
  if (status_dev && cudaMemsetAsync(status_dev, 0, 4, st) != cudaSuccess) return TINFER_ERR_CUDA;
  const cudaError_t e = cache->format == kv8::E4M3 ? kv8::launch_f<kv8::E4M3>(q, cache->head_dim, per, q_rows->dtype, st)
                                                   : kv8::launch_f<kv8::INT8>(q, cache->head_dim, per, q_rows->dtype, st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}

}  // extern "C"
