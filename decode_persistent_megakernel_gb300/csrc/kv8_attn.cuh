// kv8_attn.cuh -- parameters of the attention kernels over the 8-bit cache.
#pragma once
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
  float scale_log2;  // log2(e) / sqrt(d)
};

}  // namespace kv8
}  // namespace tinfer
