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

// What of a call's gradients may stay in the 256 MiB memory-side cache from
// the sum to the clipping.  Calls of more read all else, and write, past the
// caches.  Ten layers of 1600 (1.23 GB of float32 to 0.61 GB of bfloat16), sum
// and clipping in us, with this many MB kept: none 174 + 325, 66 177 + 318,
// 131 176 + 312, 197 177 + 304, 229 176 + 302; all accesses through the
// caches 214 + 330, the sum's alone 197 + 291.
constexpr int64_t kNormKeep = int64_t{224} << 20;

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
  int32_t stream;                  // chunks from the first that are read past the caches
  int32_t large;                   // the call's gradients are more than kNormKeep
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
