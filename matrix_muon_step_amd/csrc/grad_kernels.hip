// Global norm of many gradients and clipping by it on gfx950.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g * (norm > max_norm and finite ? max_norm / norm : 1)
//
// Squares of float32 numbers and their sums are formed in float64: a square
// is exact there (48 bits), none overflows or vanishes, and a norm over 10^9
// elements keeps its digits.  The vector unit does float64 products at the
// float32 rate, so memory stays the bound.  Every sum runs in a fixed order
// (lane, wave, work-group, partials), so results repeat bit for bit.
#include "grad_internal.h"
#include "muon_internal.h"

namespace muon {

namespace {

constexpr int kLanes = 256;

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// The work-group's sum, in every lane.
__device__ __forceinline__ double group_sum(double x) {
  __shared__ double part[kLanes / 64];
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < kLanes / 64; ++w) x += part[w];
  return x;
}

// Eight values of a tensor from element i on, as float32 (zeros past n).  A
// pointer need only be aligned to its element: the memory unit takes 16-byte
// accesses at any address.
template <bool F32>
struct Eight;
template <>
struct Eight<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const unsigned char* p) {
    a = gld<float4>(p);
    b = gld<float4>(p + 16);
  }
  __device__ __forceinline__ void load_some(const unsigned char* p, int n) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? gld<float>(p + 4 * k) : 0.f;
    a = {v[0], v[1], v[2], v[3]};
    b = {v[4], v[5], v[6], v[7]};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Eight<false> {
  uint4 a;
  __device__ __forceinline__ void load(const unsigned char* p) { a = gld<uint4>(p); }
  __device__ __forceinline__ void load_some(const unsigned char* p, int n) {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? gld<uint16_t>(p + 2 * k) : 0u;
    a = {v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf_lo(a.x), v[1] = bf_hi(a.x), v[2] = bf_lo(a.y), v[3] = bf_hi(a.y);
    v[4] = bf_lo(a.z), v[5] = bf_hi(a.z), v[6] = bf_lo(a.w), v[7] = bf_hi(a.w);
  }
};

template <bool F32>
__device__ __forceinline__ void store_eight(unsigned char* p, const float (&v)[8]) {
  if (F32) {
    gst(p, make_float4(v[0], v[1], v[2], v[3]));
    gst(p + 16, make_float4(v[4], v[5], v[6], v[7]));
  } else {
    gst(p, make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
  }
}
template <bool F32>
__device__ __forceinline__ void store_some(unsigned char* p, const float (&v)[8], int n) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= n) break;
    if (F32) gst(p + 4 * k, v[k]);
    else gst(p + 2 * k, static_cast<uint16_t>(pack_bf16(v[k], 0.f)));
  }
}

// What a lane does in a chunk: kNormChunk / 8 / kLanes groups of eight.
constexpr int kRounds = kNormChunk / 8 / kLanes;

__device__ __forceinline__ void add_squares(const float (&v)[8], double (&acc)[4]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const double d = v[k];
    acc[k & 3] = fma(d, d, acc[k & 3]);
  }
}

template <bool F32>
__device__ __forceinline__ void chunk_squares(const unsigned char* g, int64_t n, double (&acc)[4]) {
  constexpr int W = F32 ? 4 : 2;
  float v[8];
  if (n >= kNormChunk) {
    Eight<F32> x[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) x[r].load(g + static_cast<int64_t>(r * kLanes + threadIdx.x) * 8 * W);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      x[r].get(v);
      add_squares(v, acc);
    }
    return;
  }
  for (int i = threadIdx.x * 8; i < n; i += kLanes * 8) {
    Eight<F32> x;
    if (i + 8 <= n) x.load(g + static_cast<int64_t>(i) * W);
    else x.load_some(g + static_cast<int64_t>(i) * W, static_cast<int>(n - i));
    x.get(v);
    add_squares(v, acc);
  }
}

template <bool F32, bool OUT>
__device__ __forceinline__ void chunk_scale(const unsigned char* g, unsigned char* out, int64_t n, double f) {
  constexpr int W = F32 ? 4 : 2, O = OUT ? 4 : 2;
  float v[8];
  if (n >= kNormChunk) {
    Eight<F32> x[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) x[r].load(g + static_cast<int64_t>(r * kLanes + threadIdx.x) * 8 * W);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      x[r].get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(static_cast<double>(v[k]) * f);
      store_eight<OUT>(out + static_cast<int64_t>(r * kLanes + threadIdx.x) * 8 * O, v);
    }
    return;
  }
  for (int i = threadIdx.x * 8; i < n; i += kLanes * 8) {
    Eight<F32> x;
    const int left = static_cast<int>(n - i);
    if (left >= 8) x.load(g + static_cast<int64_t>(i) * W);
    else x.load_some(g + static_cast<int64_t>(i) * W, left);
    x.get(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(static_cast<double>(v[k]) * f);
    if (left >= 8) store_eight<OUT>(out + static_cast<int64_t>(i) * O, v);
    else store_some<OUT>(out + static_cast<int64_t>(i) * O, v, left);
  }
}

// Work-group w takes chunks w, w + gridDim.x, ... of the batch.
__global__ __launch_bounds__(kLanes) void grad_squares_kernel(const NormBatch b, double* partials) {
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int total = b.chunks[b.n];
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = find_mat(b.chunks, b.n, c);
    const NormDesc& d = b.d[i];
    const int64_t first = static_cast<int64_t>(c - b.chunks[i]) * kNormChunk;
    if (d.g_f32) chunk_squares<true>(d.g + first * 4, d.count - first, acc);
    else chunk_squares<false>(d.g + first * 2, d.count - first, acc);
  }
  const double sum = group_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
  if (threadIdx.x == 0) {
    const int w = blockIdx.x;
    gst(partials + w, w < b.earlier ? gld<double>(partials + w) + sum : sum);
  }
}

// Every work-group that needs the norm sums the partials itself, in one order.
__device__ __forceinline__ double norm_of(const double* partials, int n) {
  double x = 0.0;
  for (int i = threadIdx.x; i < n; i += kLanes) x += gld<double>(partials + i);
  return sqrt(group_sum(x));
}

__global__ __launch_bounds__(kLanes) void grad_norm_kernel(const double* partials, int n, double* norm) {
  const double x = norm_of(partials, n);
  if (threadIdx.x == 0) gst(norm, x);
}

// From the last chunk to the first, since the last ones that the sum read are
// the likeliest to be in the memory-side cache still.
__global__ __launch_bounds__(kLanes) void grad_clip_kernel(const NormBatch b, const double* partials, int n, double* norm,
                                                           double max_norm) {
  double x;
  if (n < 0) {
    x = gld<double>(norm);
  } else {
    x = norm_of(partials, n);
    // every launch of the call writes the same bits
    if (blockIdx.x == 0 && threadIdx.x == 0) gst(norm, x);
  }
  const bool clip = x > max_norm && x < __builtin_inf();
  const double f = clip ? max_norm / x : 1.0;
  for (int c = b.chunks[b.n] - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const int i = find_mat(b.chunks, b.n, c);
    const NormDesc& d = b.d[i];
    if (!clip && d.out == d.g) continue;  // in place, and as it is
    const int64_t first = static_cast<int64_t>(c - b.chunks[i]) * kNormChunk, left = d.count - first;
    if (d.g_f32) {
      if (d.out_f32) chunk_scale<true, true>(d.g + first * 4, d.out + first * 4, left, f);
      else chunk_scale<true, false>(d.g + first * 4, d.out + first * 2, left, f);
    } else {
      if (d.out_f32) chunk_scale<false, true>(d.g + first * 2, d.out + first * 4, left, f);
      else chunk_scale<false, false>(d.g + first * 2, d.out + first * 2, left, f);
    }
  }
}

dim3 groups(const NormBatch& b) {
  const int total = b.chunks[b.n];
  return dim3(total < kNormGroups ? total : kNormGroups);
}

}  // namespace

hipError_t launch_grad_squares(const NormBatch& b, double* partials, hipStream_t s) {
  hipLaunchKernelGGL(grad_squares_kernel, groups(b), dim3(kLanes), 0, s, b, partials);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double* partials, int n, double* norm, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kLanes), 0, s, partials, n, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const NormBatch& b, const double* partials, int n, double* norm, double max_norm,
                            hipStream_t s) {
  hipLaunchKernelGGL(grad_clip_kernel, groups(b), dim3(kLanes), 0, s, b, partials, n, norm, max_norm);
  return hipGetLastError();
}

}  // namespace muon
