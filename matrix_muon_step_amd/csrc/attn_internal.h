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
// Rows of a sequence that one work item of the first tokens' gradients sums
// over (a multiple of kAttnRows).
constexpr int kFarRows = 256;
// Work items from which on a windowed call leaves their largest logits in the
// workspace, for a launch of its own to join, instead of one atomic each
// (which follow one another, about 15 ns each where all items end at once).
// From -infinity, us, atomics | join: 384 items (4096 tokens, 12 heads of 64,
// window 256) 20.0 | 20.5; 516 (5500) 20.2 | 20.6; 640 (20 heads) 29 | 23.5; 950
// (4100 in ten sequences, 25 heads) 38 | 24.5; 2048 (16384, 16 heads, window
// 128) 48 | 39.5; 1024 (4096, 32/8 heads of 128, window 512) 63 | 60.
constexpr int kTopItems = 576;
// Chunks of a sequence that the dK/dV kernel adds itself; more are joined by a
// launch of their own first.
constexpr int kFarDirect = 8;
constexpr float kAttnLog2e = 1.44269504088896340736f;

// One work item of a packing: rows first .. first + min(kAttnRows, len -
// first) - 1 of the sequence that starts at packed row `row0`.
struct AttnTile {
  int32_t row0;
  int32_t len;
  int32_t first;
  int32_t chunk;  // kFarRows chunks of the sequences before it
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
  int32_t longest;             // most keys that a row's work item visits: tokens of the longest sequence, or fewer
  // windowed calls only
  int32_t window, sinks;       // row i sees key j <= i where i - j < window or j < sinks
  float* far;                  // backward workspace: sums over rows beyond their windows (NULL: there are none)
  int32_t far_joined;          // the first chunk's sums are a sequence's
  int32_t key_parts;           // backward: work-groups that share a key tile's query heads
  float* parts;                // backward workspace: their sums, where there are several
  float* tops;                 // forward workspace: heads x n_tiles, each item's largest logit, or NULL
};

hipError_t launch_attention(const AttnArgs& a, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s);
hipError_t launch_window_attention(const AttnArgs& a, hipStream_t s);
hipError_t launch_window_attention_backward(const AttnArgs& a, hipStream_t s);

}  // namespace muon
