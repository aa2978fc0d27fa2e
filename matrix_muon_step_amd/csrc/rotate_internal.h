// Norms of queries and keys with rotary positions: what the host and the
// kernels share.
#pragma once

#include "attn_internal.h"

namespace muon {

// Tokens of one work item, a piece of a packing's 128-row tile: few enough for
// many work items, enough to pay for a token's angles.  Calls among others, us,
// forward / gradient: 16384 tokens, 32/8 heads of 128, three axes 8 53 / 107, 16
// 55 / 116; 16384, 25/25 heads of 64 33 / 57 and 34 / 62; 4100 in ten sequences
// 11.6 / 24.5 and 12.4 / 22.8 (2 and 4 were slower in a first form).
constexpr int kRotateRows = 8;
constexpr int kRotatePieces = kAttnRows / kRotateRows;
// Work-groups of the backward kernel at most, for each of the two tensors, each
// with one partial sum of the weight's gradient in the workspace (gradient, us,
// of the 16384 tokens with heads of 128, of 64 and of the 4100: 512 107, 57 and
// 24.5; 1024 106, 59 and 26.4; 2048 110, 62 and 26.2).
constexpr int kRotateGroups = 512;
constexpr int kRotateLanes = 256;
// Heads of a lane's float32 sums of the weight's gradient at most: with the
// rounding of a work-group's partial sum below 64 half steps of what is added.
constexpr int kRotateRun = 60;
// A call whose tensors are more bytes than the memory-side cache holds writes
// past the caches.  Forward in us, through | past them, with the inputs in the
// cache and not: 16384 tokens, 32/8 heads of 128 (336 MB) 71 | 53 and 71 | 68; 25/25
// heads of 64 (210 MB) 33 | 38 and 47 | 45.  (Reads past them too were slower
// wherever the cache held the inputs.)
constexpr int64_t kRotateLarge = int64_t{256} << 20;

// One of the two tensors of a call.
struct RotateTensor {
  HeadsView x, out;     // forward: input and output; backward: input (norm only) and its gradient
  HeadsView up;         // backward: gradient of the output
  const float* weight;  // head_dim, or NULL for ones
  float* d_weight;      // backward: head_dim, or NULL
  int32_t heads;
  int32_t step_token, step_head;  // a lane's next head: (token, head) + these, carried over
};

struct RotateArgs {
  RotateTensor t[2];    // queries, keys
  const AttnTile* tiles;
  int32_t n_tiles;
  int32_t head_dim, rotary_dim;
  int32_t group_log2;   // lanes that share a head
  float eps;
  int32_t positions_64;
  const void* positions;  // axes x position_stride, or NULL: the index in the sequence
  int64_t position_stride;
  float* partials;      // backward: work-groups x 2 x head_dim
  uint64_t frequency[kAttnMaxDim / 2];  // turns per position times 2^64, modulo 2^64
  uint8_t axis[kAttnMaxDim / 2];
};

// Which kernel serves a call.
struct RotateForm {
  bool back;         // the gradient
  bool wide;         // eight pairs to a lane (rotary_dim and head_dim - rotary_dim multiples of 16), else four
  bool interleaved;
  bool norm;
  bool large;        // more bytes than the memory-side cache holds: writes past the caches
};
// Launches it and, where a weight's gradient is asked for, the kernel that joins its sums.
hipError_t launch_rotate(const RotateArgs& a, const RotateForm& f, hipStream_t s);

}  // namespace muon
