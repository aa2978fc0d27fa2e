// Attention over packed sequences: what the host and the kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// Rows of one work item of the attention kernels: query rows (forward, dQ)
// or key rows (dK, dV).
constexpr int kAttnRows = 128;
// Rows of the tiles that stream through LDS past a work item.
constexpr int kAttnStep = 64;
constexpr int kAttnMaxDim = 128;
constexpr float kAttnLog2e = 1.44269504088896340736f;

// One work item of a packing: rows first .. first + min(kAttnRows, len -
// first) - 1 of the sequence that starts at packed row `row0`.
struct AttnTile {
  int32_t row0;
  int32_t len;
  int32_t first;
  int32_t pad;
};

// A (tokens, heads, head_dim) bf16 tensor: element strides of a token and a
// head, head_dim contiguous.
struct HeadsView {
  unsigned char* p;
  int64_t ts, hs;
};

struct AttnArgs {
  HeadsView q, k, v, o;        // o: output of the forward pass
  HeadsView d_o, dq, dk, dv;   // backward only
  float* lse;                  // heads x lse_stride, natural logarithm
  int64_t lse_stride;
  float* max_logit;            // NULL, or a running maximum per logit_group heads
  int32_t logit_group;
  float* row_lse2;             // backward workspace: heads x row_stride, lse * log2(e)
  float* row_delta;            // backward workspace: heads x row_stride, sum_d dO * O
  int64_t row_stride;
  int32_t heads, kv_heads, head_dim;
  float scale;
  const AttnTile* by_query;    // tiles, most keys first
  const AttnTile* by_key;      // tiles, most queries first
  int32_t n_tiles;
  int32_t longest;             // tokens of the longest sequence
};

hipError_t launch_attention(const AttnArgs& a, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s);

}  // namespace muon
