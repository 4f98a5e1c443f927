// kv8_attn.cu -- attention of the last tokens of each sequence over its 8-bit KV cache.
//
//   o_i = sum_{j <= pos+i} softmax_j(q_i . k_j / sqrt(d)) v_j,   k_j = ck_j * sk[j / block], v_j = cv_j * sv[j / block]
//
// The n_tokens x group query rows that share a KV head are the rows of one matrix: every code is read and widened once
// for each tile of 8, 16 or 32 of them (16 at most at 128 dimensions). The work is a flat list of key tiles
// (sequence, KV head, row tile, tile of KT keys); each warp takes an equal run of it, whatever the sequences'
// lengths and counts, so that one long sequence spreads over the GPU and a ragged batch stays even. The warps of a
// CTA have neighbouring runs and join the parts of a unit that lie in them; a CTA whose run covers a unit only in
// part leaves (m, l, o) in the workspace, and kv8_merge_kernel joins these parts in order, so results do not depend on timing.
//
// Each warp streams its own tiles: a ring of bulk asynchronous copies per warp that runs on across the
// boundaries of the units, no barrier between the warps until their runs end. Products run on the
// legacy warp-level tensor instruction (m16n8k16, fp16 in, fp32 accumulation): with so few rows the tensor pipe
// is not the limit, and register operands let the codes go from shared memory to the product without being
// stored again in 16 bits. Keys (and dimensions of V) are the 16 rows of a product and query rows its
// 8 columns, so a group of 8 query heads or fewer wastes nothing on padding.
//
// Precision. Codes widen to fp16 exactly. A query row is divided by the power of two above its largest
// magnitude, which keeps it in fp16's range, and multiplied back in the scores' fp32 scale. Query and
// weight are rounded to fp16 (off by 2^-11 at most) for bf16 queries, whose own result is rounded by 2^-8; for
// fp32 and fp16 queries both enter as two fp16 parts (high and the remainder: 2^-22), with twice the
// products. Scores, maxima, sums and outputs are fp32. (bf16 rows leave the sums of a run of keys to the tensor instruction,
// which cuts them off: 2.6e-6 over 8000 keys; fp32 and fp16 rows add each tile's rounded, 4e-7.)
//
// A key's V scale 2^e * f (1 <= f < 2) enters its weight: the running maximum M is taken over x + e (x
// the score in units of log 2), the weight of V is w * f with w = 2^(x + e - M), and the sum of the
// softmax adds w * 2^-e. So weights are near 1 where they matter whatever the scales of the blocks are; where they
// are 2^86 and more apart, the sums take exponentials of their own (E_SPAN).
//
// Measured: 64 sequences of 16 to 8192 keys, 8 KV heads of 64 with 5 query heads each, int8, bf16 queries (270 MB): 56 us
// with the join, 0.72 of the measured copy rate; 61 with fp32 or fp16 queries. Two of four issue slots are used and no pipe is
// busy for more than half of the time: what 8 to 12 warps, all that the registers allow, leave uncovered of the latency
// of a tile's steps (widening, products, maximum, exponentials). One sequence of 131001 keys, 2 heads of 128 (67 MB): 23 us,
// bound by the chain of each warp's few tiles (1.4 a clock) and the join. 1152 keys, one token: 9 us, all latency.
// Earlier forms of the first took 116 us (queries as the products' rows), 92 (keys as rows) and 83 (runs by
// warps, without a unit's fixed cost). Kernels of 32 rows spill (190 bytes of stores at 255 registers, 680 with two-part
// operands), of two-part operands also those of 16 rows (190 to 210), and at 128 dimensions of 8 (110).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "kv8.cuh"
#include "kv8_attn.cuh"

namespace tinfer {
namespace gemm {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm.cu
}
namespace kv8 {

// Byte of 16-byte chunk c of a row in its tile as the copies' swizzle leaves it: 128-byte rows exchange chunks
// by the row's number modulo 8, 64-byte rows by half of it modulo 4.
template <int D>
__device__ __forceinline__ int swizzled(int c, int row) {
  return (D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) * 16;
}

template <int D>
struct Shape {
  static constexpr int KT = 4096 / D;              // keys of one tile: 64 or 32, 4 KiB of K and 4 of V
  static constexpr int STAGE_BYTES = 2 * KT * D;
};

// ---- the list of work -------------------------------------------------------------------------
// Sequence s has a unit for each KV head and each tile of its own query rows; each is FIXED empty places, which stand for
// what a unit costs beside its tiles (its queries, its end), and a place for each key tile that its rows may see, so
// that a prompt's first rows, which see few keys, count for little. prefix[s] counts the places before it. Called
// by all threads of a CTA; returns the total.
constexpr int FIXED = 4;

// In shared memory: prefix, then position and count of every sequence's new tokens (0, 0 for one that is passed over).
struct List {
  int* prefix;
  int2* span;
  __device__ List(void* at, int n) : prefix(static_cast<int*>(at)), span(reinterpret_cast<int2*>(static_cast<int*>(at) + ((n + 2) & ~1))) {}
};
size_t list_bytes(int n) { return (size_t)((n + 2) & ~1) * 4 + (size_t)n * 8; }

// The units of a KV head in one sequence. The last row of row tile rt sees pos + 1 + j keys, j = (rt ROWS + ROWS - 1) / group,
// and j / KT = rt / m with m = group KT / ROWS (ROWS divides KT), so base + rt / m tiles hold them, and are easily summed.
template <int D, int ROWS>
struct RowTiles {
  static_assert(Shape<D>::KT % ROWS == 0, "row tiles that see one key tile more come in groups of m");
  int n, base, m;
  __device__ __forceinline__ RowTiles(const AttnParams& q, int pos, int count) {
    constexpr int KT = Shape<D>::KT;
    n = q.row_tiles > 1 ? (q.group * count + ROWS - 1) / ROWS : 1;
    base = n > 1 ? pos / KT + 2 : (pos + count + KT - 1) / KT;
    m = q.group * (KT / ROWS);
  }
  __device__ __forceinline__ int tiles(int rt) const { return n == 1 ? base : base + rt / m; }
  __device__ __forceinline__ int before(int rt) const {  // places of the row tiles before rt
    if (n == 1) return rt * (base + FIXED);
    const int k = rt / m;
    return rt * (base + FIXED) + k * (rt - m) - m * (k * (k - 1) / 2);
  }
  // KV head, row tile, tile of keys (negative: an empty place) and tiles of the unit at place `in` of the sequence. Not
  // inlined: it runs once for a unit, and its registers would be the products'.
  __device__ __noinline__ int4 place(int in) const {
    const int per_head = before(n), head = in / per_head, off = in - head * per_head;
    int a = 0, b = n;  // before(a) <= off < before(b)
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (before(mid) <= off) a = mid;
      else b = mid;
    }
    return make_int4(head, a, off - before(a) - FIXED, tiles(a));
  }
};

template <int D, int ROWS>
__device__ __forceinline__ int places_of(const AttnParams& q, int s, const List& list) {
  int pos, count;
  if (!span_of(q.sp, s, q.c.max_ctx, pos, count) && blockIdx.x == 0 && q.sp.status) atomicOr(q.sp.status, STATUS_BAD_POS);
  list.span[s] = make_int2(pos, count);
  if (count == 0) return 0;
  const RowTiles<D, ROWS> r(q, pos, count);
  return r.before(r.n) * q.c.n_kv;
}

template <int D, int ROWS, int NT>
__device__ int build_list(const AttnParams& q, const List& list, int* scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = q.c.n_seqs;
  if (n <= 32) {  // every warp for itself: all write the same words, and no barrier stands before the first copy
    const int mine = lane < n ? places_of<D, ROWS>(q, lane, list) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    const int total = __shfl_sync(~0u, incl, 31);
    if (lane < n) list.prefix[lane] = incl - mine;
    if (lane == 0) list.prefix[n] = total;
    __syncwarp();
    return total;
  }
  int carry = 0;
  for (int base = 0; base < n; base += NT) {
    const int s = base + threadIdx.x;
    const int mine = s < n ? places_of<D, ROWS>(q, s, list) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < NT / 32; ++w) {
      const int y = scan[w];
      if (w < warp) before += y;
      carry += y;
    }
    if (s < n) list.prefix[s] = before + incl - mine;
    __syncthreads();
  }
  if (threadIdx.x == 0) list.prefix[n] = carry;
  __syncthreads();
  return carry;
}

// The list is dealt out in equal runs of places to the warps of all CTAs, neighbouring runs to the warps of one CTA.
// Short lists use fewer warps of every CTA rather than fewer CTAs.
struct Deal {
  int warps, per;  // warps of a CTA, places of a warp (one where the list is empty: it divides)
};
__device__ __forceinline__ Deal deal(int total, int grid, int max_warps) {
  const int warps = min(max((total + grid - 1) / grid, 1), max_warps);
  return Deal{warps, max((total + grid * warps - 1) / (grid * warps), 1)};
}

// A place in the list, with what the tiles of its unit share.
template <int D, int ROWS>
struct Place {
  int x, seq, tile, tiles;        // tile < 0: an empty place; tiles: of the unit
  int limit;                      // keys that some row of the unit sees
  int row0;                       // the KV head's first row among all rows of the cache
  int pos, count, head, rt;       // the sequence's new tokens; KV head and row tile of the unit
  __device__ void seek(const AttnParams& q, const List& list, int at) {
    x = at;
    limit = tile = 0;
    if (at >= list.prefix[q.c.n_seqs]) return;
    seq = seq_of(list.prefix, q.c.n_seqs, at);
    const int2 span = list.span[seq];
    pos = span.x;
    count = span.y;
    const RowTiles<D, ROWS> r(q, pos, count);
    const int in = at - list.prefix[seq];
    if (r.n == 1) {
      tiles = r.base;
      head = in / (tiles + FIXED);
      rt = 0;
      tile = in - head * (tiles + FIXED) - FIXED;
      limit = pos + count;
    } else {
      const int4 p = r.place(in);
      head = p.x;
      rt = p.y;
      tile = p.z;
      tiles = p.w;
      limit = pos + min((rt * ROWS + ROWS - 1) / q.group, count - 1) + 1;
    }
    row0 = (seq * q.c.n_kv + head) * q.c.max_ctx;
  }
  __device__ void next(const AttnParams& q, const List& list, int end) {
    ++x;
    if (++tile >= tiles && x < end) seek(q, list, x);
  }
};

// ---- small wrappers ------------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The remainder of a pair after its rounding to fp16, again in fp16.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t high) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&high));
  return pack_half(a - h.x, b - h.y);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// KT rows of codes from row y on; rows past the cache's end arrive as zeros.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// ---- the kernel ----------------------------------------------------------------------------------
// A CTA's shape: NG groups of 8 query rows, NW warps, STAGES slots of 8 KiB in each warp's ring. Two groups
// (one at 128 dimensions with two-part operands) leave registers for 12 warps; beyond that 8.
template <int D, int NG, int SPLIT>
struct Cfg {
  static constexpr int NW = D * NG * (SPLIT + 1) <= 384 ? 12 : 8;
  static constexpr int STAGES = NW == 12 ? 2 : 3;
  static constexpr int NT = NW * 32;
  static constexpr int ROWS = 8 * NG;
};

// A part of a unit that a warp leaves to be joined: the unit, by its first place in the list (-1: none), its
// tiles, whether it holds the unit's first and last, and where the unit's rows are (the first of the KV head's query
// rows, how many the head has).
struct Part {
  int unit, first, last, seq, head, row0, rows;
};

// The parts of one unit within a CTA: tails of warps w0 .. w1 - 1 and the head of head_warp (-1: none); rows counts
// the KV head's query rows, row0 the unit's first; ends: 2 if the first tile is among the parts, + 1 if the last is.
struct Group {
  int seq, head, row0, rows, w0, w1, head_warp, ends;
};

template <int D, int NG, int SPLIT>
struct Smem {
  using C = Cfg<D, NG, SPLIT>;
  static constexpr int SCALES = Shape<D>::KT / 16;  // scales of one tile, at most (blocks of 16)
  static_assert(C::ROWS * D * 4 <= Shape<D>::STAGE_BYTES, "a warp's outputs fit its first ring slot");
  alignas(1024) uint8_t ring[C::NW][C::STAGES][Shape<D>::STAGE_BYTES];
  alignas(16) float2 angle[C::NW][D / 2];  // cosine and sine of one token's rotary pairs
  unsigned long long freq[D / 2];
  int4 slot[C::NW][C::STAGES];            // of a tile in the ring: place in the list, first key, keys
  Part tail[C::NW], head[C::NW];          // a warp's last part (outputs in its ring) and its first (in the workspace)
  Group group[C::NW + 1];
  int groups;
  float m[2][C::NW][C::ROWS], l[2][C::NW][C::ROWS];  // of the tails and of the heads
  float ring_scale[C::NW][C::STAGES][2][SCALES];
  alignas(8) unsigned long long full[C::NW][C::STAGES];
  int scan[C::NW];
  int failed;
};

// A thread's outputs as rows of D floats: DB dimensions from g DB on of rows 2t and 2t + 1 of each group.
template <int D, int NG>
__device__ __forceinline__ void store_part(float* rows, const float (&o)[D / 16][NG][4], int g, int t) {
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < D / 8; j += 4)
        *reinterpret_cast<float4*>(rows + (n * 8 + 2 * t + h) * D + g * (D / 8) + j) =
            make_float4(o[j / 2][n][h], o[j / 2][n][2 + h], o[j / 2 + 1][n][h], o[j / 2 + 1][n][2 + h]);
}

template <int FMT, int D, int NG, int SPLIT, typename T>
__global__ void __launch_bounds__(Cfg<D, NG, SPLIT>::NT, 1) kv8_attn_kernel(const __grid_constant__ CUtensorMap map_k,
                                                                              const __grid_constant__ CUtensorMap map_v,
                                                                              const __grid_constant__ AttnParams q) {
  using C = Cfg<D, NG, SPLIT>;
  constexpr int KT = Shape<D>::KT, MK = KT / 16, MD = D / 16, ROWS = C::ROWS, DB = D / 8, NW = C::NW, STAGES = C::STAGES;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<D, NG, SPLIT>& sm = *reinterpret_cast<Smem<D, NG, SPLIT>*>(smem_raw);
  const List list(smem_raw + sizeof(sm), q.c.n_seqs);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  if (lane == 0)
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_addr(&sm.full[warp][s]), 33);  // the copy and 32 lanes' scales
  if (tid == 0) sm.failed = 0;
  mbar_fence_init();
  if (tid < D / 2) sm.freq[tid] = q.rope.f[tid];  // (threads index it apart, which parameters do one by one)
  const int total = build_list<D, ROWS, C::NT>(q, list, sm.scan);
  const Deal share = deal(total, gridDim.x, NW);
  if ((long long)share.per * share.warps * blockIdx.x >= total) return;
  const int lo = warp < share.warps ? (int)min((long long)share.per * (blockIdx.x * share.warps + warp), (long long)total) : total;
  const int hi = min(lo + share.per, total);

  // this warp's tiles, across the units' boundaries
  Place<D, ROWS> in;
  in.seek(q, list, lo);
  int put = 0, got = 0;
  const uint64_t policy = q.keep_l2 ? policy_evict_normal() : policy_evict_first();
  volatile int* failed = &sm.failed;
  auto issue = [&]() {  // the next tile that has keys to read goes into the ring
    if (__any_sync(~0u, *failed)) return;  // what is under way is still waited for, a ring's tiles at most
    while (in.x < hi && (in.tile < 0 || in.tile * KT >= in.limit)) in.next(q, list, hi);
    if (in.x >= hi) return;
    const int st = put % STAGES, key0 = in.tile * KT, keys = min(in.limit - key0, KT);
    const uint32_t bar = smem_addr(&sm.full[warp][st]);
    if (lane == 0) {
      const uint32_t dst = smem_addr(sm.ring[warp][st]);
      sm.slot[warp][st] = make_int4(in.x, key0, keys, 0);
      mbar_arrive_expect_tx(bar, 2 * KT * D);
      load_tile(dst, &map_k, in.row0 + key0, bar, policy);
      load_tile(dst + KT * D, &map_v, in.row0 + key0, bar, policy);
    }
    const int b0 = key0 >> q.c.lg_block, nb = ((key0 + keys - 1) >> q.c.lg_block) - b0 + 1;
    if (lane < nb) {
      const size_t at = (size_t)(in.seq * q.c.n_kv + in.head) * q.c.n_blocks + b0 + lane;
      cp_async_4(smem_addr(&sm.ring_scale[warp][st][0][lane]), q.c.ks + at);
      cp_async_4(smem_addr(&sm.ring_scale[warp][st][1][lane]), q.c.vs + at);
    }
    if (!(q.withhold && put == 0 && lane == 31)) cp_async_arrive(bar);
    ++put;
    in.next(q, list, hi);
  };
  __syncwarp();
#pragma unroll 1
  for (int s = 0; s < STAGES; ++s) issue();
  __syncthreads();  // the frequencies are there

  bool tail = false;  // this warp leaves a part in its registers
  if (lane == 0) sm.tail[warp].unit = sm.head[warp].unit = -1;
  float o[MD][NG][4], mx[NG][2], l[NG][2];
  Place<D, ROWS> seg;  // the unit that the warp works on
  seg.seek(q, list, lo);
  while (seg.x < hi) {
    if (seg.tile < 0) {  // past the empty places
      seg.x -= seg.tile;
      seg.tile = 0;
      if (seg.x >= hi) break;
    }
    const int seg_end = min(hi, seg.x + seg.tiles - seg.tile);
    const int head = seg.head, rt = seg.rt, pos = seg.pos, count = seg.count;
    const int rows = min(q.group * count - rt * ROWS, ROWS);  // rows of this unit

    // query rows: rotated, divided by a power of two, laid out as the scores' right operands, eight at a
    // time. A thread's operands are dimensions t D/4 .. of row g, four for each product, so it loads just those
    // and their rotary partners (which are thread t ^ 2's). The angles of a token are shared by its rows.
    uint32_t qf[SPLIT][NG][MD][2];
    float rs[NG][2];
    int limit[NG][2];  // first key that a row does not see
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      constexpr int E = D / 4;
      const int row = rt * ROWS + n * 8 + g, tok = row / q.group;
      const bool there = n * 8 + g < rows;
      float v[E];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = 0.f;
      const T* p = static_cast<const T*>(q.q.data) + seg.seq * q.q.ss + tok * q.q.ts + (head * q.group + row - tok * q.group) * q.q.hs;
      if (there) {
#pragma unroll
        for (int i = 0; i < E; i += 8) load8(p + t * E + i, reinterpret_cast<float(&)[8]>(v[i]));
      }
      if (q.rope.on && n * 8 < rows) {
        float z[E];
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = 0.f;
        if (there) {
#pragma unroll
          for (int i = 0; i < E; i += 8) load8(p + (t ^ 2) * E + i, reinterpret_cast<float(&)[8]>(z[i]));
        }
        const float sign = t < 2 ? -1.f : 1.f;
        const int last_tok = (rt * ROWS + min(n * 8 + 7, rows - 1)) / q.group;
        for (int x = (rt * ROWS + n * 8) / q.group; x <= last_tok; ++x) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            float c, s;
            rope_cos_sin(sm.freq[lane + 32 * i], pos + x, c, s);
            sm.angle[warp][lane + 32 * i] = make_float2(c, s);
          }
          __syncwarp();
          if (tok == x) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
              const float4 cs = *reinterpret_cast<const float4*>(&sm.angle[warp][(t & 1) * E + i]);
              v[i] = fmaf(z[i] * sign, cs.y, v[i] * cs.x);
              v[i + 1] = fmaf(z[i + 1] * sign, cs.w, v[i + 1] * cs.z);
            }
          }
        }
      }
      unsigned top = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      // (from 2^-120 on, so that the power, its inverse and the scores' factor are normal numbers: 11 bits are left at 2^-126)
      const int e2 = top ? min(max((int)(top >> 23) - 126, -120), 126) : 0;  // every magnitude below 2^e2 (below 4 2^e2 at the type's end)
      const float down = __uint_as_float((uint32_t)(127 - e2) << 23), up = q.scale_log2 * __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
      for (int k = 0; k < MD; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = v[4 * k + 2 * h] * down, b = v[4 * k + 2 * h + 1] * down;
          qf[0][n][k][h] = pack_half(a, b);
          if (SPLIT == 2) qf[SPLIT - 1][n][k][h] = pack_rest(a, b, qf[0][n][k][h]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        rs[n][h] = __shfl_sync(~0u, up, 8 * t + 4 * h);  // of rows 2t and 2t + 1
        limit[n][h] = pos + min((rt * ROWS + n * 8 + 2 * t + h) / q.group, count - 1) + 1;
      }
    }
    const int all_see = pos + min(rt * ROWS / q.group, count - 1) + 1;  // keys that every row sees
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int j = 0; j < MD; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][n][i] = 0.f;
      mx[n][0] = mx[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    int e_top = E_MIN;  // of the V scales so far

    while (got < put) {
      const int st = got % STAGES;
      const int4 slot = sm.slot[warp][st];
      if (slot.x >= seg_end) break;
      const int key0 = slot.y, keys = slot.z;
      if (!wait_bounded(smem_addr(&sm.full[warp][st]), (got / STAGES) & 1, q.wait_us)) *failed = 1;
      uint8_t* kbuf = sm.ring[warp][st];
      uint8_t* vbuf = kbuf + KT * D;
      if (keys < KT) {  // rows past the copy: weights there are 0, so V must be finite
        for (int i = lane; i < (KT - keys) * (D / 16); i += 32)
          reinterpret_cast<uint4*>(vbuf + keys * D)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
      }
      const int rel = key0 & ((1 << q.c.lg_block) - 1);
      // ---- scores, keys by rows: m-tile j holds keys 16j .. 16j + 15. The contraction's order is free, so
      // a thread takes D / 4 neighbouring dimensions of its keys g and g + 8: 16-byte loads, spread over the
      // banks by the swizzle that the copies wrote the tile in
      float s[MK][NG][4];
#pragma unroll
      for (int j = 0; j < MK; ++j) {
#pragma unroll
        for (int n = 0; n < NG; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.f;
        const uint8_t* kr = kbuf + (16 * j + g) * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int at = swizzled<D>(t * (D / 64) + c, g);
          const uint4 x = *reinterpret_cast<const uint4*>(kr + at), y = *reinterpret_cast<const uint4*>(kr + 8 * D + at);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a[4];
            codes_to_half<FMT>(xs[k], a[0], a[2]);
            codes_to_half<FMT>(ys[k], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
              for (int h = 0; h < SPLIT; ++h) mma16816(s[j][n], a, qf[h][n][c * 4 + k][0], qf[h][n][c * 4 + k][1]);
          }
        }
      }
      // ---- the rows' maxima of x + e = s kf rf + ef. The products stay as they are and the weights scale them again, so
      // that an exponent is rounded once, near 0 where its weight counts
      float vf[MK], vinv[MK], kf[MK], ef[MK];
      int e_low = E_MAX;
#pragma unroll
      for (int j = 0; j < MK; ++j) {
        const int b = (rel + 16 * j) >> q.c.lg_block;
        const float ks = sm.ring_scale[warp][st][0][b], vs = sm.ring_scale[warp][st][1][b];
        const int e = min(max((int)((__float_as_uint(vs) >> 23) & 0xFF) - 127, E_MIN), E_MAX);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        // a scale that is not finite reaches its scores, so that the mask decides which rows it spoils
        const bool fine = vs < INFINITY;
        vf[j] = fine && vs > 0.f ? vs * inv * (float)(1 << WEIGHT_SHIFT) : 0.f;
        vinv[j] = inv * (float)(1 << WEIGHT_SHIFT);
        kf[j] = ks;
        ef[j] = fine ? (float)e : __uint_as_float(0x7FC00000u);
        if (fine && 16 * j < keys) {
          e_low = min(e_low, e);
          e_top = max(e_top, e);
        }
      }
      float rf[NG][2];
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) rf[n][h] = rs[n][h];
      if (keys < KT || key0 + KT > all_see) {
#pragma unroll
        for (int j = 0; j < MK; ++j)
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 16 * j + 8 * (i >> 1) + g;
              // scaled before it is masked, whatever the scale of keys that are not seen
              s[j][n][i] = key >= keys || key0 + key >= limit[n][i & 1] ? -INFINITY : fmaf(s[j][n][i], kf[j] * rf[n][i & 1], ef[j]);
            }
#pragma unroll
        for (int j = 0; j < MK; ++j) {
          kf[j] = 1.f;
          ef[j] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) rf[n][0] = rf[n][1] = 1.f;
      }
      float now[NG][2];
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = -INFINITY;  // scales are not negative: the largest product of 16 keys is their largest score
#pragma unroll
          for (int j = 0; j < MK; ++j) top = fmaxf(top, fmaf(fmaxf(s[j][n][h], s[j][n][2 + h]), kf[j] * rf[n][h], ef[j]));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
          now[n][h] = fmaxf(mx[n][h], top);
          grew |= now[n][h] != mx[n][h];
        }
      if (__any_sync(~0u, grew)) {  // after the first tiles the maxima seldom move
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float half = half_shrink(mx[n][h], now[n][h]), shrink = half * half;
            mx[n][h] = now[n][h];
            l[n][h] = l[n][h] * half * half;
#pragma unroll
            for (int j = 0; j < MD; ++j) {
              o[j][n][h] *= shrink;
              o[j][n][2 + h] *= shrink;
            }
          }
      }
      if (e_top - e_low > E_SPAN) {  // the weights would lose keys: the sums take their own exponentials
#pragma unroll
        for (int j = 0; j < MK; ++j) {
          const float back = lifted(vinv[j]);
          vinv[j] = 0.f;
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float from = mx[n][i & 1] == -INFINITY ? 0.f : mx[n][i & 1];
              l[n][i & 1] = fmaf(exp2_fast(fmaf(s[j][n][i], kf[j] * rf[n][i & 1], ef[j] - from) + back), 1.f / (1 << SUM_LIFT), l[n][i & 1]);
            }
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float from = mx[n][h] == -INFINITY ? 0.f : mx[n][h];
#pragma unroll
          for (int j = 0; j < MK; ++j)
#pragma unroll
            for (int i = h; i < 4; i += 2) {
              const float w = exp2_fast(fmaf(s[j][n][i], kf[j] * rf[n][h], ef[j] - from));
              l[n][h] = fmaf(w, vinv[j], l[n][h]);
              s[j][n][i] = w * vf[j];
            }
        }
      // ---- o^T += V^T weights, 16 keys at a time; an 8 x 8 transpose turns the scores' layout (keys by
      // rows) into that of a right operand (keys down the columns)
      // The instruction's own sums are cut off, not rounded, which adds up over a long run of keys: two-part operands, whose
      // precision it would spoil, take a tile's products by themselves (32 sequences of 8000 keys, 40 heads of 64 over 8, fp32,
      // 262 MB: off by 4e-7 where they were off by 2.6e-6, in the same 52 us; 12 heads of 128 over 2, whose registers run
      // short, 131 MB: 37 us against 35)
      float part[SPLIT == 2 ? MD : 1][NG][4];
      if (SPLIT == 2) {
#pragma unroll
        for (int j = 0; j < MD; ++j)
#pragma unroll
          for (int n = 0; n < NG; ++n) part[j][n][0] = part[j][n][1] = part[j][n][2] = part[j][n][3] = 0.f;
      }
      auto& into = *[&] {
        if constexpr (SPLIT == 2) return &part;
        else return &o;
      }();
#pragma unroll
      for (int p = 0; p < MK; ++p) {
        uint32_t b[SPLIT][NG][2];
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float u = s[p][n][2 * h], w = s[p][n][2 * h + 1];
            const uint32_t high = pack_half(u, w);
            b[0][n][h] = transpose8(high);
            if (SPLIT == 2) b[SPLIT - 1][n][h] = transpose8(pack_rest(u, w, high));
          }
        // four keys of this thread; dimensions g DB .. g DB + DB - 1: m-tile m takes g DB + 2m as its row g
        // and g DB + 2m + 1 as its row g + 8
        uint32_t w[4][DB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // keys 2t, 2t + 1, 2t + 8, 2t + 9
          const int key = 2 * t + (i & 1) + 4 * (i & 2);
          const uint8_t* row = vbuf + (16 * p + key) * D + swizzled<D>(g * DB / 16, key) + (DB == 8 ? (g & 1) * 8 : 0);
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
            uint32_t a[4];
            codes_to_half<FMT>(__byte_perm(w[0][c], w[1][c], sel), a[0], a[1]);
            codes_to_half<FMT>(__byte_perm(w[2][c], w[3][c], sel), a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
              for (int sp = 0; sp < SPLIT; ++sp) mma16816(into[2 * c + h][n], a, b[sp][n][0], b[sp][n][1]);
          }
      }
      if (SPLIT == 2) {
#pragma unroll
        for (int j = 0; j < MD; ++j)
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][n][i] += into[j][n][i];
      }
      __syncwarp();
      ++got;
      issue();
      __syncwarp();
    }

#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[n][h] += __shfl_xor_sync(~0u, l[n][h], x);
    const bool first = seg.tile == 0, last = seg_end - seg.x + seg.tile == seg.tiles;
    if (first && last) {  // the whole unit: a thread holds DB dimensions of rows 2t and 2t + 1 of each group
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = n * 8 + 2 * t + h;
          if (row < rows) {
            const int qrow = rt * ROWS + row, tok = qrow / q.group, hq = head * q.group + qrow - tok * q.group;
            T* dst = static_cast<T*>(q.out.data) + seg.seq * q.out.ss + tok * q.out.ts + hq * q.out.hs + g * DB;
            const float inv = 1.f / l[n][h];
#pragma unroll
            for (int j = 0; j < DB; j += 4) {  // dimension j of the thread's DB: o[j / 2], rows g (even) and g + 8 (odd)
              const float y[4] = {o[j / 2][n][h] * inv, o[j / 2][n][2 + h] * inv, o[j / 2 + 1][n][h] * inv,
                                  o[j / 2 + 1][n][2 + h] * inv};
              store4(dst + j, y);
            }
            if (q.lse && g == 0)
              q.lse[((size_t)seg.seq * q.sp.n_tokens + tok) * q.n_heads + hq] =
                  (log2f(l[n][h]) + mx[n][h] - (float)WEIGHT_SHIFT) * 0.6931471805599453f;
          }
        }
    } else {
      const int which = seg_end >= hi ? 0 : 1;  // the run's last unit stays in registers, its first goes to the workspace
      if (g == 0)
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sm.m[which][warp][n * 8 + 2 * t + h] = mx[n][h];
            sm.l[which][warp][n * 8 + 2 * t + h] = l[n][h];
          }
      if (lane == 0)
        (which ? sm.head : sm.tail)[warp] = Part{seg.x - seg.tile, first, last, seg.seq, head, rt * ROWS, q.group * count};
      if (which == 0) {
        tail = true;
      } else {
        store_part<D, NG>(q.part + (size_t)(2 * gridDim.x + blockIdx.x * NW + warp) * ROWS * (D + 2), o, g, t);
      }
    }
    seg.seek(q, list, seg_end);
  }

  // ---- the parts that the warps of this CTA left, joined in order of the warps. A unit's parts are the tails of
  // neighbouring warps and perhaps the head of the next; all threads share the sums
  if (tail) store_part<D, NG>(reinterpret_cast<float*>(sm.ring[warp][0]), o, g, t);
  __syncthreads();
  // one group for the head of warp 0, begun by an earlier CTA, and one for the parts that begin with each warp's tail
  // (not with one that continues its neighbour's); they are few, and kept without gaps
  if (warp == 0) {
    Group u{0, 0, 0, 0, 0, 0, -1, 0};
    bool there = false;
    if (lane <= NW) {
      const Part p = lane ? sm.tail[lane - 1] : sm.head[0];
      there = p.unit >= 0 && !(lane > 1 && sm.tail[lane - 2].unit == p.unit);
      if (there) {
        int w1 = lane;
        while (lane && w1 < NW && sm.tail[w1].unit == p.unit) ++w1;  // tails of warps lane - 1 .. w1 - 1 (lane 0: none)
        const bool joins = !lane || (w1 < NW && sm.head[w1].unit == p.unit);  // and the head of warp w1
        const int last = joins ? sm.head[w1].last : sm.tail[w1 - 1].last;
        u = Group{p.seq, p.head, p.row0, p.rows, max(lane - 1, 0), w1, joins ? w1 : -1, 2 * (p.first != 0) + (last != 0)};
      }
    }
    const unsigned set = __ballot_sync(~0u, there);
    if (there) sm.group[__popc(set & ((1u << lane) - 1))] = u;
    if (lane == 0) sm.groups = __popc(set);
  }
  __syncthreads();
  constexpr int QUADS = D / 4;
  const int items = sm.groups * ROWS * QUADS;
  for (int item = tid; item < items; item += C::NT) {
    const Group u = sm.group[item / (ROWS * QUADS)];
    const int row = item / QUADS % ROWS, c = item % QUADS * 4, qrow = u.row0 + row;
    if (qrow >= u.rows) continue;
    const int w0 = u.w0, w1 = u.w1;
    const bool use_head = u.head_warp >= 0, first = u.ends & 2, last = u.ends & 1;
    float top = -INFINITY;
    for (int w = w0; w < w1; ++w) top = fmaxf(top, sm.m[0][w][row]);
    if (use_head) top = fmaxf(top, sm.m[1][u.head_warp][row]);
    float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](float lw, float mw, const float* y) {
      if (lw == 0.f) return;  // no key of the row
      const float half = half_shrink(mw, top), f = half * half;
      const float4 v = *reinterpret_cast<const float4*>(y + row * D + c);
      sum = fmaf(lw * half, half, sum);
      acc[0] = fmaf(v.x, f, acc[0]); acc[1] = fmaf(v.y, f, acc[1]); acc[2] = fmaf(v.z, f, acc[2]); acc[3] = fmaf(v.w, f, acc[3]);
    };
    for (int w = w0; w < w1; ++w) add(sm.l[0][w][row], sm.m[0][w][row], reinterpret_cast<const float*>(sm.ring[w][0]));
    if (use_head)
      add(sm.l[1][u.head_warp][row], sm.m[1][u.head_warp][row],
          q.part + (size_t)(2 * gridDim.x + blockIdx.x * NW + u.head_warp) * ROWS * (D + 2));
    const int tok = qrow / q.group, hq = u.head * q.group + qrow - tok * q.group;
    if (first && last) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= inv;
      store4(static_cast<T*>(q.out.data) + u.seq * q.out.ss + tok * q.out.ts + hq * q.out.hs + c, acc);
      if (q.lse && c == 0)
        q.lse[((size_t)u.seq * q.sp.n_tokens + tok) * q.n_heads + hq] =
            (log2f(sum) + top - (float)WEIGHT_SHIFT) * 0.6931471805599453f;
    } else {  // more of the unit in other CTAs: slot 1 of the CTA that begins it, slot 0 of the others
      float* part = q.part + (size_t)(2 * blockIdx.x + (first ? 1 : 0)) * ROWS * (D + 2);
      *reinterpret_cast<float4*>(part + row * D + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (c == 0) {
        part[ROWS * D + row] = top;
        part[ROWS * D + ROWS + row] = sum;
      }
    }
  }
  if (tid == 0 && *failed && q.sp.status) atomicOr(q.sp.status, STATUS_TIMEOUT);
}

// Joins the units that several CTAs hold: CTA (unit, as the sequence with the most tokens has them, slice of its rows).
// It is launched with the kernel before it and builds its list meanwhile; 2 to 4 us after it, latency of a few dependent
// loads from L2. CTAs without a unit leave at once: in a call of one 256-token chunk and 31 single tokens they are 31 of 32.
template <int D, int NG, typename T>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv8_merge_kernel(const __grid_constant__ AttnParams q) {
  constexpr int ROWS = 8 * NG;
  extern __shared__ int list_raw[];
  __shared__ int scan[JOIN_WARPS];
  const int seq = blockIdx.x / q.units, unit = blockIdx.x % q.units, head = unit / q.row_tiles, rt = unit % q.row_tiles;
  int pos, count;
  span_of(q.sp, seq, q.c.max_ctx, pos, count);
  const RowTiles<D, ROWS> r(q, pos, count);
  const bool there = count > 0 && rt < r.n;
  if (!there && (blockIdx.x || blockIdx.y)) return;  // (one CTA waits, so that the kernel never ends before the other)
  // the list depends on the call's inputs alone, so it is built while the parts are still being made
  const List list(list_raw, q.c.n_seqs);
  const int total = build_list<D, ROWS, JOIN_WARPS * 32>(q, list, scan);
  const Deal share = deal(total, q.grid, q.warps);
  const int per = share.per * share.warps;  // of a CTA
  const int a = list.prefix[seq] + head * r.before(r.n) + r.before(rt) + FIXED, c0 = a / per, parts = (a + r.tiles(rt) - 1) / per - c0 + 1;
  pdl_wait();  // the parts are complete
  if (!there || parts <= 1) return;  // no rows, or one CTA had it whole
  join_parts<D, ROWS, T>(q, seq, head, rt * ROWS, min(q.group * count - rt * ROWS, ROWS), c0, parts, WEIGHT_SHIFT);
}

// ---------------------------------------------------------------------------------------- host

// The codes of K or V as rows of D bytes, read KT at a time with the swizzle as wide as a row.
bool code_map(CUtensorMap* map, const void* codes, long long rows, int d, int kt) {
  const auto fn = gemm::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d};
  const cuuint32_t box[2] = {(cuuint32_t)d, (cuuint32_t)kt}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// Rows of a unit: 8, 16 or 32 (16 at 128 dimensions, whose accumulators are twice as wide).
int rows_per_tile(long long rows, int head_dim) { return rows <= 8 ? 8 : rows <= 16 || head_dim == 128 ? 16 : 32; }

template <int FMT, int D, int NG, int SPLIT, typename T>
cudaError_t launch_t(AttnParams& q, cudaStream_t st) {
  q.warps = Cfg<D, NG, SPLIT>::NW;
  auto kernel = kv8_attn_kernel<FMT, D, NG, SPLIT, T>;
  const size_t list = list_bytes(q.c.n_seqs), smem = sizeof(Smem<D, NG, SPLIT>) + list;
  constexpr int MOST = sizeof(Smem<D, NG, SPLIT>) + MAX_SEQS * 12 + 16;  // the same in every call: others may be under way
  static_assert(MOST <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
  if (e != cudaSuccess) return e;
  CUtensorMap maps[2];
  const long long cache_rows = (long long)q.c.n_seqs * q.c.n_kv * q.c.max_ctx;
  if (!code_map(&maps[0], q.c.k, cache_rows, D, Shape<D>::KT) || !code_map(&maps[1], q.c.v, cache_rows, D, Shape<D>::KT))
    return cudaErrorNotSupported;
  kernel<<<q.grid, Cfg<D, NG, SPLIT>::NT, smem, st>>>(maps[0], maps[1], q);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  // few units: a CTA for each row, so that long rows are joined side by side
  cfg.gridDim = dim3((unsigned)(q.c.n_seqs * q.units), q.c.n_seqs * q.units <= 16 ? 8 * NG : q.c.n_seqs * q.units <= 64 ? NG : 1);
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.dynamicSmemBytes = list;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D, NG, T>, q);
}

template <int FMT, int D, int NG>
cudaError_t launch_n(AttnParams& q, int dtype, cudaStream_t st) {
  if (dtype == TINFER_DTYPE_F32) return launch_t<FMT, D, NG, 2, float>(q, st);
  if (dtype == TINFER_DTYPE_F16) return launch_t<FMT, D, NG, 2, __half>(q, st);
  return launch_t<FMT, D, NG, 1, __nv_bfloat16>(q, st);
}
template <int FMT>
cudaError_t launch_f(AttnParams& q, int head_dim, int rows, int dtype, cudaStream_t st) {
  if (head_dim == 128) return rows == 8 ? launch_n<FMT, 128, 1>(q, dtype, st) : launch_n<FMT, 128, 2>(q, dtype, st);
  return rows == 8    ? launch_n<FMT, 64, 1>(q, dtype, st)
         : rows == 16 ? launch_n<FMT, 64, 2>(q, dtype, st)
                      : launch_n<FMT, 64, 4>(q, dtype, st);
}

// Rows of a unit of work and row tiles of a KV head; false where the counts do not fit: rows of the cache (their
// coordinates in the copies), query rows, the list of tiles (2^30 and one place for each unit) and the units are counted in 32 bits.
struct Units {
  int rows, row_tiles;
};
bool units_of(const tinfer_kv8* c, int n_heads, int n_tokens, bool prefill, Units& u) {
  const long long rows = (long long)(n_heads / c->n_kv_heads) * n_tokens;
  if ((long long)c->n_seqs * c->n_kv_heads * c->max_ctx > 0x7FFFFFFFLL || rows > (1LL << 30)) return false;
  u.rows = prefill ? PREFILL_ROWS : rows_per_tile(rows, c->head_dim);
  const long long row_tiles = (rows + u.rows - 1) / u.rows, kt = 4096 / c->head_dim;
  u.row_tiles = (int)row_tiles;
  return row_tiles * c->n_kv_heads * c->n_seqs <= (1LL << 30) / (prefill ? 1 : (c->max_ctx + kt - 1) / kt + FIXED);
}

// Multiprocessors of the current device.
int device_sms(int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

}  // namespace
}  // namespace kv8
}  // namespace tinfer

using namespace tinfer;

extern "C" {

size_t tinfer_kv8_attention_workspace(const tinfer_kv8* cache, int n_heads, int n_tokens) {
  kv8::Cache c;
  tinfer_status rc;
  if (!kv8::cache_of(cache, c, rc) || n_heads < 1 || n_heads % cache->n_kv_heads || n_tokens < 1 || n_tokens > cache->max_ctx) return 0;
  kv8::Units u;  // as bf16 rows, which are refused last
  const long long rows = (long long)(n_heads / cache->n_kv_heads) * n_tokens;
  if (!kv8::units_of(cache, n_heads, n_tokens, kv8::is_prefill(TINFER_DTYPE_BF16, cache->head_dim, rows), u)) return 0;
  // One size for every call, so that a program can keep one workspace for all: two parts of each CTA and one of each
  // of its warps (12 warps of 16 rows, or 8 of 32 at 64 dimensions), or two parts of 256 rows of each CTA.
  const size_t few = (size_t)kv8::MAX_GRID * (cache->head_dim == 128 ? (2 + 12) * 16 : (2 + 8) * 32) * (cache->head_dim + 2) * 4;
  return std::max(few, kv8::prefill_workspace(cache->head_dim));
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
  if (!kv8::words_of({pos_dev, counts_dev, status_dev, lse_dev})) return TINFER_ERR_INVALID_ARG;
  // over the queries' own memory a row may only replace itself
  if (q.q.data == q.out.data && (q.q.ss != q.out.ss || q.q.ts != q.out.ts || q.q.hs != q.out.hs)) return TINFER_ERR_INVALID_ARG;
  q.group = n_heads / cache->n_kv_heads;
  q.n_heads = n_heads;
  q.sp = kv8::Span{pos_dev, counts_dev, n_tokens, status_dev};
  q.lse = lse_dev;
  q.part = static_cast<float*>(workspace_dev);
  q.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)cache->head_dim));
  const bool prefill = kv8::is_prefill(q_rows->dtype, cache->head_dim, (long long)q.group * n_tokens);
  kv8::Units u;
  if (!kv8::units_of(cache, n_heads, n_tokens, prefill, u)) return TINFER_ERR_UNSUPPORTED;
  q.row_tiles = u.row_tiles;
  q.units = u.row_tiles * cache->n_kv_heads;
  q.keep_l2 = u.row_tiles > 1;
  q.withhold = (cache->format & TINFER_KV8_DEBUG_WITHHOLD) != 0;
  q.wait_us = q.withhold ? kv8::WAIT_US_WITHHELD : kv8::WAIT_US;
  int sms = 0;
  if (!kv8::device_sms(sms)) return TINFER_ERR_CUDA;
  q.grid = std::min(sms, kv8::MAX_GRID);
  cudaStream_t st = (cudaStream_t)stream;
  if (!kv8::clear_status(cache, status_dev, st)) return TINFER_ERR_CUDA;
  cudaError_t e;
  if (prefill)
    e = kv8::launch_prefill(q, kv8::format_of(cache), cache->head_dim, st);
  else
    e = kv8::format_of(cache) == kv8::E4M3 ? kv8::launch_f<kv8::E4M3>(q, cache->head_dim, u.rows, q_rows->dtype, st)
                                   : kv8::launch_f<kv8::INT8>(q, cache->head_dim, u.rows, q_rows->dtype, st);
  return e == cudaSuccess ? TINFER_OK : TINFER_ERR_CUDA;
}

}  // extern "C"
