// kv8_prefill.cu -- attention of many tokens (a prompt, or a chunk of one) over the 8-bit KV cache, on the
// fifth-generation tensor cores. The mathematics is kv8_attn.cu's; here both products are large, and the
// bound is shared between the tensor pipe, the exponentials (16 a clock on an SM) and shared memory.
//
// A unit is one KV head of one sequence with 256 of its token x group query rows, as two tiles of 128. Roles of
// a CTA (one on each SM):
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, a thread to a row: it rotates and scales the row's query into
//                   shared memory, then for each 128 keys takes their scores from tensor memory into registers, and
//                   writes the weights back over them in fp16, the left operand of the second product
//   warps 8-11      widen the codes of K and V to fp16 in the operands' swizzled layouts, two tiles ahead
//   warp 12         issues tcgen05.mma (one of its lanes): scores = Q K^T (both from shared memory), outputs += P V (P from
//                    tensor memory), the two tiles in turn, so that one's softmax runs under the other's products
// Tensor memory: two (three at 64 dimensions) 128-column score buffers and two D-column outputs. Products are issued
// by one warp and run in order, so new scores may follow the product that read the weights lying in their place.
// The softmax and the second product go by halves of 64 keys, so that the first half's product runs under the
// second half's exponentials. (Scores by halves as well cost a 128-row operand read twice, and gained nothing.)
//
// A row's running maximum is replaced only where one of its warp's would grow by nearly 2^2, and then all of them are: the
// outputs in tensor memory are rescaled by the rows' threads after the exponentials, when the product before is done and
// the scores have left their registers. Weights are held times 2^SHIFT, below 2^16 with the mantissa of their V scale: a
// key far below the largest is held to 2^-38 of it. The 4096-token prompt takes 102 us; 105 with rows by themselves
// and maxima that lag by 2 (2^-39), 99 with a lag of 2^8, which leaves 2^-32, and 112 rescaled before the exponentials.
//
// Work is dealt out in equal runs over all CTAs by the number of keys that the units see (a causal prompt's
// last rows see the whole prompt, its first almost nothing); a unit cut by a run's end leaves parts that
// prefill_merge_kernel joins.
//
// Measured: 4096-token prompt, 12 heads of 128 over 2, int8 (51.6 GFLOP): 102 us, 0.26 of the measured bf16 rate; 512 tokens over
// 8192 keys, 32 heads of 64 over 8, e4m3 (33.3 GFLOP): 69 us, 0.25. Bound by the chain of a row tile: scores from
// tensor memory, maximum, exponentials, weights, product (about 3800 clocks for 128 keys at 64 dimensions, 5500 at
// 128), which the other row tile's covers in part. 13 warps leave a thread 128
// registers, of which the softmax spills 80 to 200 bytes. The legacy warp products of kv8_attn.cu took 590 and 192 us.
#include <algorithm>
#include <type_traits>

#include "kv8_attn.cuh"

namespace tinfer {
namespace kv8 {
namespace prefill {

constexpr int KT = 128, HALF = KT / 2, ROWS = PREFILL_ROWS, TILE = 128;
static_assert(TILE == KT, "blocks of Q and K are alike");
constexpr int WARP_WIDEN = 8;      // first warp of the widening role; before it the softmax, after it the products
template <int D>
struct Roles {
  static constexpr int WIDEN = 4, MMA = WARP_WIDEN + WIDEN, NT = (MMA + 1) * 32;
  static constexpr int BUFFERS = D == 64 ? 3 : 2;       // of 128 x 128 scores in tensor memory, beside two outputs of D columns
  static constexpr int ANGLES = D == 64 ? 4096 : 1472;  // of a tile: all of 128 tokens, or of 23 (or 8 at a time)
};
constexpr int FETCH = 4;           // key tiles that are fetched into L2 ahead (64 rows of 32 x 4000 keys, 8 heads of 64: 114 -> 108 us)
constexpr int KV_STAGES = 2, SCALE_SLOTS = 4;
constexpr int SHIFT = 13;          // of the weights
constexpr float GROW = 1.99f;      // a maximum may lag behind by 2^GROW: 2^(SHIFT + GROW) 2 is below fp16's 65504
constexpr int FIXED_KEYS = 768;    // what a unit costs beside its keys, in keys (4096-token prompt: 102 us, 114 with 384)

template <int D>
struct Smem {
  alignas(1024) uint8_t q[2][TILE * D * 2];            // D / 64 blocks of [128 rows][128 bytes], swizzled
  alignas(1024) uint8_t k[KV_STAGES][KT * D * 2];      // the same: keys by rows
  alignas(1024) uint8_t v[KV_STAGES][KT * D * 2];
  alignas(16) float2 angle[2][Roles<D>::ANGLES];       // cosines and sines at the tile's tokens
  float4 scale[SCALE_SLOTS][KT / 16];                  // of 16 keys: K scale, V scale's exponent, mantissa, 2^-exponent
  int apart[SCALE_SLOTS];                              // whether a tile's V scales lie too far below earlier ones (E_SPAN)
  alignas(8) unsigned long long k_full[KV_STAGES], v_full[KV_STAGES], k_empty[KV_STAGES], v_empty[KV_STAGES];
  unsigned long long s_full[3], p_full[3][2], o_full[2][2], q_full[2], drained;  // of score buffers and row tiles, [half of the keys]
  uint32_t tmem;
  int failed;
};

// ---- the list: sequence s has, for each KV head, row tiles rt whose weight is FIXED_KEYS + pos + 1 + step (rt + 1),
// at least the keys that the tile sees, and easily summed
struct Span64 {
  int pos, count, n, last;  // n: row tiles; last: its last row
  long long base, step;
  __device__ void of(const AttnParams& q, int seq) {
    if (!span_of(q.sp, seq, q.c.max_ctx, pos, count) && blockIdx.x == 0 && q.sp.status) atomicOr(q.sp.status, STATUS_BAD_POS);
    last = q.group * count - 1;  // rows are counted in 31 bits
    n = (last + ROWS) / ROWS;
    base = FIXED_KEYS + pos + 1;
    step = (ROWS + q.group - 1) / q.group;
  }
  __device__ long long before(int rt) const { return rt * base + step * ((long long)rt * (rt + 1) / 2); }  // of one head
  __device__ int keys(const AttnParams& q, int rt) const { return pos + min(rt * ROWS + ROWS - 1, last) / q.group + 1; }
};

template <int NTH>
__device__ long long build_prefix(const AttnParams& q, long long* prefix) {
  for (int s = threadIdx.x; s < q.c.n_seqs; s += NTH) {
    Span64 sp;
    sp.of(q, s);
    prefix[s + 1] = sp.before(sp.n) * q.c.n_kv;
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // one warp sums, 32 sequences at a time
    long long carry = 0;
    for (int s0 = 0; s0 < q.c.n_seqs; s0 += 32) {
      const int s = s0 + threadIdx.x;
      long long x = s < q.c.n_seqs ? prefix[s + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if ((int)threadIdx.x >= o) x += y;
      }
      if (s < q.c.n_seqs) prefix[s + 1] = carry + x;
      carry += __shfl_sync(~0u, x, 31);
    }
    if (threadIdx.x == 0) prefix[0] = 0;
  }
  __syncthreads();
  return prefix[q.c.n_seqs];
}

// A run is at least one tile long, so that each run between a unit's first and last tile holds one of its tiles.
__device__ __forceinline__ long long run_length(long long total, int grid) {
  return max((total + grid - 1) / grid, (long long)KT);
}

// The units of a CTA's run [lo, hi), with the tiles of each that fall into it.
struct Walk {
  long long at, hi;  // where the next unit is looked for
  int seq, head, rt, first, last;  // tiles [first, last)
  int tiles, keys, pos, count;     // of the unit
  __device__ void init(long long lo, long long end) {
    at = lo;
    hi = end;
  }
  __device__ bool next(const AttnParams& q, const long long* prefix) {
    while (at < hi) {
      seq = seq_of(prefix, q.c.n_seqs, at);
      Span64 sp;
      sp.of(q, seq);
      const long long per_head = sp.before(sp.n), in = at - prefix[seq];
      head = (int)((float)in / (float)per_head);  // 64-bit divisions take a microsecond
      while (head * per_head > in) --head;
      while ((head + 1) * per_head <= in) ++head;
      const long long off = in - head * per_head;
      int a = 0, b = sp.n;  // before(a) <= off < before(b)
      while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (sp.before(mid) <= off) a = mid;
        else b = mid;
      }
      rt = a;
      const long long start = prefix[seq] + head * per_head + sp.before(rt);
      keys = sp.keys(q, rt);
      tiles = (keys + KT - 1) / KT;
      pos = sp.pos;
      count = sp.count;
      // tile t lies at start + FIXED_KEYS + t KT
      auto tile_at = [&](long long x) { return (int)min(max((x - start - FIXED_KEYS + KT - 1) / KT, 0LL), (long long)tiles); };
      first = at <= start + FIXED_KEYS ? 0 : tile_at(at);
      last = hi <= start + FIXED_KEYS ? 0 : tile_at(hi);
      at = start + sp.before(rt + 1) - sp.before(rt);
      if (first < last) return true;
    }
    return false;
  }
};

// ---- tensor cores ---------------------------------------------------------------------------------
// Operand tiles in shared memory: 128-byte rows, 128-byte swizzle, groups of 8 rows 1024 bytes apart. K-major (Q
// and K: a row is a query or key, its 128 bytes 64 dimensions): 32 bytes further for the next 16 dimensions, the
// next 64 in the next block. V is read across: a row is a key, its 128 bytes 64 columns of the product
// (N-major), 16 keys are 2048 bytes, and the leading byte offset leads to the next 64 columns.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, fp16 operands, fp32 accumulator, M 128; b_across: the right operand is N-major
__host__ __device__ constexpr uint32_t instr(int n, bool b_across) {
  return (1u << 4) | (b_across ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
}
// Issued by the one lane that `leader` names. The whole warp comes here with the same operands: they stay in uniform
// registers, where a single thread's would be moved there for every instruction (75 to 90 cycles a product of 64 columns).
__device__ __forceinline__ uint32_t elect() {
  uint32_t leader;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
  return leader;
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t i, int accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(i), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t i, int accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(i), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// 16, 32 or 64 columns, complete on return: load and wait are one statement, so that no register is moved or put aside
// between them, before its value is there.
__device__ __forceinline__ void tmem_load16(uint32_t a, uint32_t* u) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t a, uint32_t* u) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
        "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
        "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_load64(uint32_t a, uint32_t* u) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
        "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
        "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]),
        "=r"(u[32]), "=r"(u[33]), "=r"(u[34]), "=r"(u[35]), "=r"(u[36]), "=r"(u[37]), "=r"(u[38]), "=r"(u[39]),
        "=r"(u[40]), "=r"(u[41]), "=r"(u[42]), "=r"(u[43]), "=r"(u[44]), "=r"(u[45]), "=r"(u[46]), "=r"(u[47]),
        "=r"(u[48]), "=r"(u[49]), "=r"(u[50]), "=r"(u[51]), "=r"(u[52]), "=r"(u[53]), "=r"(u[54]), "=r"(u[55]),
        "=r"(u[56]), "=r"(u[57]), "=r"(u[58]), "=r"(u[59]), "=r"(u[60]), "=r"(u[61]), "=r"(u[62]), "=r"(u[63])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t a, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(a),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A wait that gives up at once when another role has: every role then runs through its loops without waiting.
struct Failed {
  volatile int* flag;
  int limit_us;
};
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, const Failed& failed) {
  if (mbar_sleep(bar, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!*failed.flag && !mbar_sleep(bar, parity))
    if ((long long)(globaltimer() - t0) > failed.limit_us * 1000LL) {
      if (!mbar_sleep(bar, parity)) *failed.flag = 1;  // (time may have passed off the GPU)
      return;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(Roles<D>::NT, 1) prefill_kernel(const __grid_constant__ AttnParams q) {
  static_assert(std::is_same_v<T, __nv_bfloat16>, "rows are loaded and results packed as bf16");
  constexpr int NT = Roles<D>::NT;
  constexpr int BUFFERS = Roles<D>::BUFFERS, O_AT = BUFFERS * KT;
  constexpr int WARP_MMA = Roles<D>::MMA, NT_WIDEN = Roles<D>::WIDEN * 32;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  long long* prefix = reinterpret_cast<long long*>(smem_raw + sizeof(Smem<D>));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < KV_STAGES; ++s) {
      mbar_init(smem_addr(&sm.k_full[s]), Roles<D>::WIDEN);
      mbar_init(smem_addr(&sm.v_full[s]), Roles<D>::WIDEN);
      mbar_init(smem_addr(&sm.k_empty[s]), 1);
      mbar_init(smem_addr(&sm.v_empty[s]), 1);
    }
    for (int t = 0; t < 3; ++t) {
      mbar_init(smem_addr(&sm.s_full[t]), 1);
      for (int h = 0; h < 2; ++h) mbar_init(smem_addr(&sm.p_full[t][h]), 4);
    }
    for (int t = 0; t < 2; ++t) {
      for (int h = 0; h < 2; ++h) mbar_init(smem_addr(&sm.o_full[t][h]), 1);
      mbar_init(smem_addr(&sm.q_full[t]), 4);
    }
    mbar_init(smem_addr(&sm.drained), 1);
    sm.failed = 0;
    mbar_fence_init();
  }
  if (warp == WARP_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  const long long total = build_prefix<NT>(q, prefix);  // ends with a barrier
  fence_after();
  const uint32_t tmem = sm.tmem;
  const Failed failed{&sm.failed, q.wait_us};
  const long long per = run_length(total, gridDim.x);
  Walk u;
  u.init(min(per * blockIdx.x, total), min(per * (blockIdx.x + 1), total));

  if (warp < WARP_WIDEN) {
    // ---- softmax: thread r of tile `tile`
    const int tile = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_at = tmem + lanes + O_AT + tile * D;
    constexpr int ANGLES = Roles<D>::ANGLES;
    const uint32_t q_smem = smem_addr(sm.q[tile]) + r * 128, stage = smem_addr(sm.q[tile]) + (warp & 3) * (32 * D * 2);
    int it = 0, jobs = 0, tiles_done = 0;  // key tiles of the CTA, of both its row tiles, and of this one
    while (u.next(q, prefix)) {
      const int row0 = u.rt * ROWS + tile * TILE, qrow = row0 + r, all = q.group * u.count;
      if (row0 >= all) {  // the unit ends in the first tile
        it += u.last - u.first;
        jobs += u.last - u.first;
        // a phase of a barrier can be told from the one before it only: the first tile's warps say when every score of
        // the jobs that are passed over here is complete
        named_sync(3, 2 * TILE);
        continue;
      }
      const int halves = u.rt * ROWS + TILE < all ? 2 : 1;  // row tiles of the unit
      jobs += tile;
      const bool there = qrow < all;
      const int tok = min(qrow / q.group, u.count - 1), hq = u.head * q.group + qrow - qrow / q.group * q.group;
      const int tok0 = row0 / q.group, ntok = (min(row0 + TILE, all) - 1) / q.group - tok0 + 1;
      const int sees = u.pos + tok + 1, first_sees = u.pos + tok0 + 1;
      float scale;
      {
        // the query row: rotated, divided by a power of two above its largest magnitude, in fp16. The angles are
        // worked out once for every token of the tile
        const T* p = static_cast<const T*>(q.q.data) + u.seq * q.q.ss + tok * q.q.ts + hq * q.q.hs;
        // the warp loads its rows one after another, whole lines at a time, and hands them out through shared memory
        uint4 raw[D / 8];
        {
          constexpr int LANES = D / 8;  // to a row
          const uint64_t mine = there ? reinterpret_cast<uint64_t>(p) : 0;
#pragma unroll
          for (int i = 0; i < LANES; ++i) {
            const int from = i * (32 / LANES) + lane / LANES;
            const char* src = reinterpret_cast<const char*>(__shfl_sync(~0u, mine, from));
            raw[i] = src ? *reinterpret_cast<const uint4*>(src + lane % LANES * 16) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < LANES; ++i) {
            const int from = i * (32 / LANES) + lane / LANES;
            sts128(stage + from * (D * 2) + ((lane % LANES ^ (from & (LANES - 1))) << 4), raw[i].x, raw[i].y, raw[i].z, raw[i].w);
          }
          __syncwarp();
#pragma unroll
          for (int c = 0; c < LANES; ++c) raw[c] = lds128(stage + lane * (D * 2) + ((c ^ (lane & (LANES - 1))) << 4));
          __syncwarp();
          // at 64 dimensions a warp's staging memory is its own rows of the operand; at 128 it lies over other warps', which
          // are not to be written before all have read theirs (with angles, their first barrier sees to it)
          if (D > 64 && !q.rope.on) named_sync(1 + tile, TILE);
        }
        float x[8], y[8];
        unsigned most = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          load8(reinterpret_cast<const T*>(&raw[c]), x);
#pragma unroll
          for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        }
        // a rotation makes no magnitude larger than sqrt(2) times the largest: one power of two of room
        const int e2 = most ? min(max((int)(most >> 23) - 125, -120), 126) : 0;
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        // chunks of eight dimensions whose angles are held at once: a power of two
        int lg_pairs = 3;
        while ((16 << (lg_pairs - 3)) <= D / 2 && ntok * (2 << lg_pairs) <= ANGLES) ++lg_pairs;
        const int cpp = 1 << (lg_pairs - 3);
        scale = q.scale_log2 * __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          load8(reinterpret_cast<const T*>(&raw[c]), x);
          load8(reinterpret_cast<const T*>(&raw[D / 16 + c]), y);
          if (q.rope.on) {
            if (c % cpp == 0) {
              named_sync(1 + tile, TILE);
              // [chunk][token][dimension]; a thread has one dimension of the chunks and every so many tokens
              const int pairs = 8 * cpp, pair = r & (pairs - 1);
              const unsigned long long freq = q.rope.f[8 * c + pair];
              float2* to = sm.angle[tile] + (pair >> 3) * ntok * 8 + (pair & 7);
#pragma unroll 4
              for (int i = r >> lg_pairs; i < ntok; i += TILE >> lg_pairs) {
                float cs, sn;
                rope_cos_sin(freq, u.pos + tok0 + i, cs, sn);
                to[8 * i] = make_float2(cs, sn);
              }
              named_sync(1 + tile, TILE);
            }
            const float4* at = reinterpret_cast<const float4*>(&sm.angle[tile][(c % cpp * ntok + tok - tok0) * 8]);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float4 f = at[i / 2];
              const float a0 = x[i], z0 = y[i], a1 = x[i + 1], z1 = y[i + 1];
              x[i] = a0 * f.x - z0 * f.y;
              y[i] = z0 * f.x + a0 * f.y;
              x[i + 1] = a1 * f.z - z1 * f.w;
              y[i + 1] = z1 * f.z + a1 * f.w;
            }
          }
          auto put = [&](int chunk, const float (&z)[8]) {  // a 16-byte chunk of the row: block chunk / 8, swizzled by the row
            sts128(q_smem + (chunk / 8) * (TILE * 128) + (((chunk & 7) ^ (r & 7)) << 4), pack_half(z[0] * down, z[1] * down),
                   pack_half(z[2] * down, z[3] * down), pack_half(z[4] * down, z[5] * down), pack_half(z[6] * down, z[7] * down));
          };
          put(c, x);
          put(D / 16 + c, y);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[tile]));
      }

      float ref = -INFINITY, sum = 0.f;
      for (int kt = u.first; kt < u.last; ++kt, ++it, ++tiles_done, jobs += halves) {
        const int buf = jobs % BUFFERS;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int n = (kt + 1) * KT > first_sees ? sees - kt * KT - h * HALF : HALF;  // keys of this half that the row sees
          const bool all_seen = __all_sync(~0u, n >= HALF);
          const float4* sc = sm.scale[it % SCALE_SLOTS] + h * (HALF / 16);
          const uint32_t at = tmem + lanes + buf * KT + h * HALF;
          wait(smem_addr(&sm.s_full[buf]), jobs / BUFFERS & 1, failed);
          fence_after();
          float s[2][32];
          tmem_load64(at, reinterpret_cast<uint32_t*>(s[0]));
          // the row's maximum: of each 16 keys' plain products first, whose scale is one
          float4 f[HALF / 16];
          float m[HALF / 16];
          const bool apart = sm.apart[it % SCALE_SLOTS];
#pragma unroll
          for (int j = 0; j < HALF / 16; ++j) f[j] = sc[j];
          if (all_seen) {
#pragma unroll
            for (int j = 0; j < HALF / 16; ++j) {
              const float* v = s[j / 2] + 16 * (j & 1);
              // a tree of three-way maxima
              const float a = fmaxf(fmaxf(v[0], v[1]), v[2]), b = fmaxf(fmaxf(v[3], v[4]), v[5]), c = fmaxf(fmaxf(v[6], v[7]), v[8]),
                          d = fmaxf(fmaxf(v[9], v[10]), v[11]), e = fmaxf(fmaxf(v[12], v[13]), v[14]);
              m[j] = fmaxf(fmaxf(fmaxf(a, b), c), fmaxf(fmaxf(d, e), v[15]));
            }
          } else {
#pragma unroll
            for (int j = 0; j < HALF / 16; ++j) {
              m[j] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (16 * j + i < n) m[j] = fmaxf(m[j], s[j / 2][16 * (j & 1) + i]);
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < HALF / 16; ++j) top = fmaxf(top, fmaf(m[j], f[j].x * scale, f[j].y));
          float shrink = 1.f;
          if (__any_sync(~0u, top > ref + GROW || ref == -INFINITY)) {  // (also the row's first keys); all of a warp's maxima at once
            const float now = fmaxf(ref, top), half = ref == -INFINITY ? 1.f : half_shrink(ref, now);
            shrink = half * half;
            ref = now;
            sum = sum * half * half;
          }
          // weights, over the scores, which are all in registers
          const float from = ref == -INFINITY ? 0.f : ref - (float)SHIFT;
          auto weights = [&](auto cut, auto apart) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float4 g = f[2 * c + j];
                const float fx = g.x * scale, fy = g.y - from;
                const float2 f2 = make_float2(fx, fx), g2 = make_float2(fy, fy), v2 = make_float2(g.z, g.z);
                const float back = lifted(g.w);
                float2 part = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  float2 e = fma2(make_float2(s[c][16 * j + i], s[c][16 * j + i + 1]), f2, g2);
                  if (cut.value) {  // masked after the scaling, whatever the scale of keys that are not seen
                    if (32 * c + 16 * j + i >= n) e.x = -INFINITY;
                    if (32 * c + 16 * j + i + 1 >= n) e.y = -INFINITY;
                  }
                  if (apart.value) part = add2(part, make_float2(exp2_fast(e.x + back), exp2_fast(e.y + back)));
                  e.x = exp2_fast(e.x);
                  e.y = exp2_fast(e.y);
                  if (!apart.value) part = add2(part, e);
                  e = __fmul2_rn(e, v2);
                  w[8 * j + i / 2] = pack_half(e.x, e.y);
                }
                sum = fmaf(part.x + part.y, apart.value ? 1.f / (1 << SUM_LIFT) : g.w, sum);
              }
              tmem_store16(at + 16 * c, w);
            }
          };
          // the warp's choice: tensor memory is stored to by whole warps
          if (apart) weights(std::true_type{}, std::true_type{});
          else if (all_seen) weights(std::false_type{}, std::false_type{});
          else weights(std::true_type{}, std::false_type{});
          // With scores ahead, the weights could run a key tile ahead of their products. A phase of a barrier can be
          // told from the one before it only, so every product is seen to be complete before the weights of the
          // next one of its half are given: the waits above and at the unit's end are then never more than one phase off
          wait(smem_addr(&sm.o_full[tile][h]), (tiles_done - 1) & 1, failed);
          // The outputs are rescaled last, when the product before has had the time of the exponentials to end, and the scores'
          // registers are free
          if (__any_sync(~0u, shrink != 1.f)) {
            wait(smem_addr(&sm.o_full[tile][h ^ 1]), (h ? tiles_done : tiles_done - 1) & 1, failed);
            fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              uint32_t o[64];
              tmem_load64(o_at + 64 * c, o);
#pragma unroll
              for (int i = 0; i < 64; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
#pragma unroll
              for (int i = 0; i < 64; i += 16) tmem_store16(o_at + 64 * c + i, o + i);
            }
          }
          tmem_store_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[buf][h]));
        }
      }
      jobs -= tile;  // (all jobs of the unit are counted)
      // ---- the unit's end
      wait(smem_addr(&sm.o_full[tile][1]), (tiles_done - 1) & 1, failed);
      fence_after();
      if (halves == 1) named_sync(3, 2 * TILE);
      const bool whole = u.first == 0 && u.last == u.tiles;
      float* part = q.part + (size_t)(2 * blockIdx.x + (u.first == 0 ? 1 : 0)) * ROWS * (D + 2);
      const int row = tile * TILE + r;
      const float inv = whole ? 1.f / sum : 1.f;
      T* dst = static_cast<T*>(q.out.data) + u.seq * q.out.ss + tok * q.out.ts + hq * q.out.hs;
      // rows leave by whole lines: through the query tile's memory, whose products are done, 2 D bytes of a row at a time
      constexpr int LANES = D / 8;
      const uint64_t mine = !there ? 0 : whole ? reinterpret_cast<uint64_t>(dst) : reinterpret_cast<uint64_t>(part + (size_t)row * D);
#pragma unroll 1
      for (int c32 = 0; c32 < D / 32; ++c32) {
        float o[32];
        tmem_load32(o_at + 32 * c32, reinterpret_cast<uint32_t*>(o));
        const int in_pass = c32 % (D / 64);  // a part's pass is D / 2 columns in fp32, a result's all D in 16 bits
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (whole && k >= 4) break;
          const int c = whole ? 4 * c32 + k : 8 * in_pass + k;
          const uint32_t to = stage + lane * (D * 2) + ((c ^ (lane & (LANES - 1))) << 4);
          if (whole)
            sts128(to, pack_bf16(o[8 * (k & 3)] * inv, o[8 * (k & 3) + 1] * inv), pack_bf16(o[8 * (k & 3) + 2] * inv, o[8 * (k & 3) + 3] * inv),
                   pack_bf16(o[8 * (k & 3) + 4] * inv, o[8 * (k & 3) + 5] * inv), pack_bf16(o[8 * (k & 3) + 6] * inv, o[8 * (k & 3) + 7] * inv));
          else
            sts128(to, __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
        }
        if (whole ? c32 < D / 32 - 1 : in_pass < D / 64 - 1) continue;
        __syncwarp();
        const int pass = whole ? 0 : c32 / (D / 64);
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
          const int from = i * (32 / LANES) + lane / LANES;
          char* to = reinterpret_cast<char*>(__shfl_sync(~0u, mine, from));
          const uint4 w = lds128(stage + from * (D * 2) + ((lane % LANES ^ (from & (LANES - 1))) << 4));
          if (to) *reinterpret_cast<uint4*>(to + pass * (D * 2) + lane % LANES * 16) = w;
        }
        __syncwarp();
      }
      fence_before();  // the next unit's products come after these loads
      if (there) {
        if (!whole) {
          part[ROWS * D + row] = ref;
          part[ROWS * D + ROWS + row] = sum;
        } else if (q.lse) {
          q.lse[((size_t)u.seq * q.sp.n_tokens + tok) * q.n_heads + hq] = (log2f(sum) + ref - (float)SHIFT) * 0.6931471805599453f;
        }
      }
    }
  } else if (warp < WARP_MMA) {
    // ---- widening
    const int t = tid - WARP_WIDEN * 32;
    constexpr int CPR = D / 16, ALL = KT * CPR, ITEMS = (ALL + NT_WIDEN - 1) / NT_WIDEN;  // 16-byte pieces of a row, and of a thread
    int it = 0;
    while (u.next(q, prefix)) {
      const size_t plane = (size_t)u.seq * q.c.n_kv + u.head;
      const uint8_t* kp = q.c.k + plane * q.c.max_ctx * D;
      const uint8_t* vp = q.c.v + plane * q.c.max_ctx * D;
      auto load = [&](const uint8_t* p, int kt, uint4 (&w)[ITEMS]) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int item = t + NT_WIDEN * i, key = kt * KT + item / CPR;
          w[i] = (ALL % NT_WIDEN == 0 || item < ALL) && key < u.keys ? *reinterpret_cast<const uint4*>(p + (size_t)key * D + item % CPR * 16) : make_uint4(0, 0, 0, 0);
        }
      };
      auto widen = [&](uint32_t to, const uint4 (&w)[ITEMS]) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int item = t + NT_WIDEN * i, row = item / CPR, c = item % CPR;
          if (ALL % NT_WIDEN && item >= ALL) break;
          // 128 dimensions: eight threads hold one row, whose halves lie in two blocks; the second half stores its
          // chunks in the other order, so that the eight meet in different banks
          const int swap = CPR == 8 && c >= 4;
          const uint32_t a = swap ? w[i].z : w[i].x, b = swap ? w[i].w : w[i].y, e = swap ? w[i].x : w[i].z, f = swap ? w[i].y : w[i].w;
          uint32_t h[8];
          codes_to_half<FMT>(a, h[0], h[1]);
          codes_to_half<FMT>(b, h[2], h[3]);
          codes_to_half<FMT>(e, h[4], h[5]);
          codes_to_half<FMT>(f, h[6], h[7]);
          const uint32_t base = to + (c / 4) * (KT * 128) + row * 128;
          const int c0 = 2 * (c & 3) + swap, c1 = 2 * (c & 3) + 1 - swap;
          sts128(base + ((c0 ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
          sts128(base + ((c1 ^ (row & 7)) << 4), h[4], h[5], h[6], h[7]);
        }
      };
      // the codes are on their way from HBM to L2 some tiles before they are loaded: a tile's lines, one to a thread
      constexpr int LINES = KT * D / 128;
      static_assert(LINES <= NT_WIDEN, "a line to a thread");
      auto fetch = [&](int kt) {
        const int at = kt * KT + t * (128 / D);
        if (t < LINES && kt < u.last && at < u.keys) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(kp + (size_t)at * D));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(vp + (size_t)at * D));
        }
      };
      uint4 wk[ITEMS], wv[ITEMS];
      int e_top = E_MIN;  // of the V scales so far
      load(kp, u.first, wk);
      for (int kt = u.first + 1; kt < u.first + FETCH; ++kt) fetch(kt);
      for (int kt = u.first; kt < u.last; ++kt, ++it) {
        fetch(kt + FETCH);
        const int st = it % KV_STAGES;
        const uint32_t parity = ((it / KV_STAGES) & 1) ^ 1;
        load(vp, kt, wv);
        wait(smem_addr(&sm.k_empty[st]), parity, failed);
        widen(smem_addr(sm.k[st]), wk);
        if (t < KT / 16) {
          const int key = kt * KT + 16 * t;
          float4 f = make_float4(0.f, 0.f, 0.f, 1.f);
          int e_low = E_MAX, e_high = E_MIN;
          if (key < u.keys) {
            const size_t b = plane * q.c.n_blocks + (key >> q.c.lg_block);
            const float ks = q.c.ks[b], vs = q.c.vs[b];
            const int e = min(max((int)((__float_as_uint(vs) >> 23) & 0xFF) - 127, E_MIN), E_MAX);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            const bool fine = vs < INFINITY;  // a scale that is not finite reaches its scores
            f = make_float4(ks, fine ? (float)e : __uint_as_float(0x7FC00000u), fine && vs > 0.f ? vs * inv : 0.f, inv);
            if (fine) e_low = e_high = e;
          }
          sm.scale[it % SCALE_SLOTS][t] = f;
          constexpr unsigned LANES = (1u << (KT / 16)) - 1;
          e_top = max(e_top, __reduce_max_sync(LANES, e_high));
          e_low = __reduce_min_sync(LANES, e_low);
          if (t == 0) sm.apart[it % SCALE_SLOTS] = e_top - e_low > E_SPAN;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0 && !(q.withhold && t == 0 && it == 0)) mbar_arrive(smem_addr(&sm.k_full[st]));
        if (kt + 1 < u.last) load(kp, kt + 1, wk);
        wait(smem_addr(&sm.v_empty[st]), parity, failed);
        widen(smem_addr(sm.v[st]), wv);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.v_full[st]));
      }
    }
  } else {
    if (warp == WARP_MMA) {
      // ---- products
      constexpr uint32_t i_s = instr(KT, false), i_o = instr(D, true);
      const uint64_t q_desc = desc(smem_addr(sm.q[0]), 16), k_desc = desc(smem_addr(sm.k[0]), 16), v_desc = desc(smem_addr(sm.v[0]), KT * 128);
      const uint32_t leader = elect();
      // Jobs: a row tile against a key tile, the unit's row tiles in turn for each key tile. A job's scores go into the
      // next score buffer, where its weights replace them; `ahead` jobs have their scores before the first has its
      // weights. Two cursors over the jobs, kept by counting: between a job's scores and the next one's values the
      // tensor pipe waits for this warp.
      struct Cursor {
        uint32_t buf, buf_phase, stage, stage_phase, tile;
        __device__ __forceinline__ void step(uint32_t last_tile) {
          if (++buf == BUFFERS) {
            buf = 0;
            buf_phase ^= 1;
          }
          if (tile == last_tile) {
            tile = 0;
            stage_phase ^= stage;
            stage ^= 1;
          } else {
            tile = 1;
          }
        }
      };
      static_assert(KV_STAGES == 2, "a cursor's stage is one bit");
      Cursor sc{0, 0, 0, 0, 0}, va{0, 0, 0, 0, 0};
      uint32_t q_phase[2] = {0, 0};
      const uint32_t bar_k = smem_addr(sm.k_full), bar_v = smem_addr(sm.v_full), bar_ke = smem_addr(sm.k_empty), bar_ve = smem_addr(sm.v_empty);
      const uint32_t bar_s = smem_addr(sm.s_full), bar_p = smem_addr(sm.p_full), bar_o = smem_addr(sm.o_full), bar_q = smem_addr(sm.q_full);
      while (u.next(q, prefix)) {
        const uint32_t last_tile = u.rt * ROWS + TILE < q.group * u.count ? 1 : 0;
        const int n = (u.last - u.first) << last_tile, ahead = min(last_tile ? BUFFERS : 2, n);
        auto scores = [&](bool new_query) {
          if (sc.tile == 0) wait(bar_k + 8 * sc.stage, sc.stage_phase, failed);
          if (new_query) {
            wait(bar_q + 8 * sc.tile, q_phase[0] ^ (sc.tile ? q_phase[1] ^ q_phase[0] : 0), failed);
            if (sc.tile) q_phase[1] ^= 1;
            else q_phase[0] ^= 1;
          }
          fence_after();
          const uint64_t a = q_desc + sc.tile * (uint32_t)(sizeof(sm.q[0]) >> 4), b = k_desc + sc.stage * (uint32_t)(sizeof(sm.k[0]) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {  // 32 bytes further in the block, then the next block
            constexpr int BLOCK = TILE * 128 >> 4;
            mma_ss(leader, tmem + sc.buf * KT, a + (k / 4) * BLOCK + (k % 4) * 2, b + (k / 4) * BLOCK + (k % 4) * 2, i_s, k > 0);
          }
          commit(leader, bar_s + 8 * sc.buf);
          if (sc.tile == last_tile) commit(leader, bar_ke + 8 * sc.stage);
          sc.step(last_tile);
        };
        for (int j = 0; j < ahead; ++j) scores(j <= (int)last_tile);
        for (int j = 0; j < n; ++j) {
          if (va.tile == 0) wait(bar_v + 8 * va.stage, va.stage_phase, failed);
          const uint32_t p = tmem + va.buf * KT, o = tmem + O_AT + va.tile * D;
          const uint64_t b = v_desc + va.stage * (uint32_t)(sizeof(sm.v[0]) >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wait(bar_p + 16 * va.buf + 8 * h, va.buf_phase, failed);
            fence_after();
#pragma unroll
            for (int k = 0; k < HALF / 16; ++k)
              mma_ts(leader, o, p + h * HALF + 8 * k, b + h * (HALF * 128 >> 4) + k * (2048 >> 4), i_o, k > 0 || h > 0 || j > (int)last_tile);
            // (the last barrier that a unit's end waits for comes last)
            if (h == 1 && va.tile == last_tile) commit(leader, bar_ve + 8 * va.stage);
            commit(leader, bar_o + 16 * va.tile + 8 * h);
          }
          va.step(last_tile);
          if (j + ahead < n) scores(false);
        }
      }
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (*failed.flag) {
    if (tid == 0 && q.sp.status) atomicOr(q.sp.status, STATUS_TIMEOUT);
    if (warp == WARP_MMA) {  // products that nobody waited for are not to run on in memory that is given back
      commit(elect(), smem_addr(&sm.drained));
      wait_bounded(smem_addr(&sm.drained), 0, q.wait_us);
    }
  }
  if (warp == WARP_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D, typename T>
__global__ void __launch_bounds__(JOIN_WARPS * 32) prefill_merge_kernel(const __grid_constant__ AttnParams q) {
  extern __shared__ long long prefix64[];
  const int seq = blockIdx.x / q.units, unit = blockIdx.x % q.units, head = unit / q.row_tiles, rt = unit % q.row_tiles;
  Span64 sp;
  sp.of(q, seq);
  if (rt >= sp.n && (blockIdx.x || blockIdx.y)) return;  // (one CTA waits, so that the kernel never ends before the other)
  const long long total = build_prefix<JOIN_WARPS * 32>(q, prefix64);
  const long long per = run_length(total, q.grid);
  int c0 = 0, parts = 0;
  if (rt < sp.n) {
    const long long start = prefix64[seq] + head * sp.before(sp.n) + sp.before(rt) + FIXED_KEYS;
    c0 = (int)(start / per);
    parts = (int)((start + (sp.keys(q, rt) - 1) / KT * KT) / per) - c0 + 1;
  }
  pdl_wait();
  if (parts <= 1) return;
  join_parts<D, ROWS, T>(q, seq, head, rt * ROWS, min(q.group * sp.count - rt * ROWS, ROWS), c0, parts, SHIFT);
}

template <int FMT, int D, typename T>
cudaError_t launch_t(AttnParams& q, cudaStream_t st) {
  auto kernel = prefill_kernel<FMT, D, T>;
  const size_t list = (size_t)(q.c.n_seqs + 1) * 8, smem = sizeof(Smem<D>) + list;
  constexpr int MOST = sizeof(Smem<D>) + (MAX_SEQS + 1) * 8;  // the same in every call: others may be under way
  static_assert(MOST <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
  if (e != cudaSuccess) return e;
  kernel<<<q.grid, Roles<D>::NT, smem, st>>>(q);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  // a CTA for 32 rows of few parts each, four rows of a warp; for fewer rows where units are few and have many parts
  // (72 rows of 8000 keys, two heads of 128: 42 us by 32 rows, 25 by one)
  const int units = q.c.n_seqs * q.units;
  cfg.gridDim = dim3((unsigned)units, (unsigned)std::min(std::max(512 / units, ROWS / 32), std::min(ROWS, q.group * q.sp.n_tokens)));
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.dynamicSmemBytes = list;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<D, T>, q);
}

template <int FMT>
cudaError_t launch_f(AttnParams& q, int head_dim, cudaStream_t st) {
  return head_dim == 64 ? launch_t<FMT, 64, __nv_bfloat16>(q, st) : launch_t<FMT, 128, __nv_bfloat16>(q, st);
}

}  // namespace prefill

// bf16 rows beyond one row tile of the other kernel, or four at 128 dimensions. fp32 and fp16 rows stay there: their
// two-part operands keep the precision of their type, which one fp16 operand would not. Here against there, in us, at 40
// rows of 8 heads of 64: 500 keys 18 : 22, 8000 keys 20 : 30, 32 sequences of 4000 keys 109 : 117; at 24 rows the last
// takes 108 : 70. Two heads of 128, 64 rows: 23 : 22, 24 : 20, 53 : 66; 128 rows: 27 : 21, 28 : 31, 61 : 110.
bool is_prefill(int dtype, int head_dim, long long rows) { return dtype == TINFER_DTYPE_BF16 && rows > (head_dim == 64 ? 32 : 64); }
size_t prefill_workspace(int head_dim) { return (size_t)MAX_GRID * 2 * PREFILL_ROWS * (head_dim + 2) * 4; }

cudaError_t launch_prefill(AttnParams& q, int format, int head_dim, cudaStream_t st) {
  return format == E4M3 ? prefill::launch_f<E4M3>(q, head_dim, st) : prefill::launch_f<INT8>(q, head_dim, st);
}

}  // namespace kv8
}  // namespace tinfer
