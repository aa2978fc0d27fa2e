// Global gradient norm and clipping: what the host and the kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// Elements of one work item: a tensor is cut into chunks of this many.
constexpr int kNormChunk = 8192;
// Work-groups of a launch at most (eight to a compute unit), each with one
// partial sum in the workspace.
constexpr int kNormGroups = 2048;
// Tensors of a launch (descriptors travel as kernel arguments).
constexpr int kNormBatch = 96;

struct NormDesc {
  const unsigned char* g;
  unsigned char* out;
  int64_t count;
  int32_t g_f32, out_f32;
};

struct NormBatch {
  NormDesc d[kNormBatch];
  int32_t chunks[kNormBatch + 1];  // exclusive prefix sums
  int32_t n;
  int32_t earlier;                 // partial sums that earlier launches of the call left
};

// Adds the batch's sums of squares to `partials` (one per work-group; the
// first `earlier` hold sums already).
hipError_t launch_grad_squares(const NormBatch& b, double* partials, hipStream_t s);
// norm = sqrt of the sum of `n` partials (0 for none).
hipError_t launch_grad_norm(const double* partials, int n, double* norm, hipStream_t s);
// out = g * min(1, max_norm / norm).  n < 0: *norm is read; else it is the
// root of the n partials' sum, and written.
hipError_t launch_grad_clip(const NormBatch& b, const double* partials, int n, double* norm, double max_norm,
                            hipStream_t s);

}  // namespace muon
