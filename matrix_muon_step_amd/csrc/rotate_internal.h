// Norms of queries and keys with rotary positions: what the host and the
// kernels share.
#pragma once

#include "attn_internal.h"

namespace muon {

// Tokens of one work item, a piece of a packing's 128-row tile.
constexpr int kRotateRows = 8;
constexpr int kRotatePieces = kAttnRows / kRotateRows;
// Work-groups of the backward kernel at most, for each of the two tensors, each
// with one partial sum of the weights' gradients in the workspace.
constexpr int kRotateGroups = 512;
constexpr int kRotateLanes = 256;
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
  bool large;        // more bytes than the caches hold: reads and writes past them
};
// Launches it and, where a weight's gradient is asked for, the kernel that joins its sums.
hipError_t launch_rotate(const RotateArgs& a, const RotateForm& f, hipStream_t s);

}  // namespace muon
