// Global norm of many gradients and clipping by it on gfx950.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g * (norm > max_norm and finite ? max_norm / norm : 1)
//
// Squares of float32 numbers and their sums are formed in float64: a square
// is exact there (48 bits), none overflows or vanishes, and a norm over 10^9
// elements keeps its digits.  The vector unit does float64 products at the
// float32 rate, so memory stays the bound: 307 M float32 values 180 us for the
// sum (6.8 TB/s), 302 for clipping them into bfloat16 (6.1 TB/s).  Every sum runs in a fixed order
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

// A lane's run of elements, 16 bytes of the wider of the types that it reads
// and writes, so that a wave's accesses are contiguous.  A pointer need only be
// aligned to its element: the memory unit takes these accesses at any address.
// STREAM: past the caches (nontemporal).
template <int V, bool F32>
struct Run {
  static constexpr int WORDS = F32 ? V : V / 2;
  typedef uint32_t words_t __attribute__((ext_vector_type(WORDS), aligned(4 * V / WORDS * F32 + 2 * !F32)));
  uint32_t u[WORDS];
  template <bool STREAM>
  __device__ __forceinline__ void load(const unsigned char* p) {
    if (STREAM) {
      const words_t r = __builtin_nontemporal_load((const __attribute__((address_space(1))) words_t*)p);
      __builtin_memcpy(u, &r, sizeof(u));
    } else {
      *this = gld<Run>(p);
    }
  }
  __device__ __forceinline__ void load_some(const unsigned char* p, int n) {  // zeros past n
#pragma unroll
    for (int k = 0; k < WORDS; ++k) u[k] = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (k >= n) break;
      if (F32) u[k] = gld<uint32_t>(p + 4 * k);
      else u[k / 2] |= static_cast<uint32_t>(gld<uint16_t>(p + 2 * k)) << (16 * (k & 1));
    }
  }
  __device__ __forceinline__ float get(int k) const {
    if (F32) return __uint_as_float(u[k]);
    return k & 1 ? bf_hi(u[k / 2]) : bf_lo(u[k / 2]);
  }
  __device__ __forceinline__ void put(const float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < WORDS; ++k) u[k] = F32 ? __float_as_uint(v[k]) : pack_bf16(v[F32 ? 0 : 2 * k], v[F32 ? 0 : 2 * k + 1]);
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(unsigned char* p) const {
    if (STREAM) {
      words_t r;
      __builtin_memcpy(&r, u, sizeof(u));
      __builtin_nontemporal_store(r, (__attribute__((address_space(1))) words_t*)p);
    } else {
      gst(p, *this);
    }
  }
  __device__ __forceinline__ void store_some(unsigned char* p, int n) const {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (k >= n) break;
      if (F32) gst(p + 4 * k, u[k]);
      else gst(p + 2 * k, static_cast<uint16_t>(u[k / 2] >> (16 * (k & 1))));
    }
  }
};

// f(run, its first element, how many of its elements there are) for this
// lane's runs of a chunk of n elements; whole chunks have all loads under way
// before the first is used.
template <int V, bool F32, bool STREAM, class F>
__device__ __forceinline__ void for_runs(const unsigned char* g, int64_t n, F&& f) {
  constexpr int W = F32 ? 4 : 2, ROUNDS = kNormChunk / V / kLanes;
  if (n >= kNormChunk) {
    Run<V, F32> x[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) x[r].template load<STREAM>(g + (r * kLanes + threadIdx.x) * (V * W));
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) f(x[r], (r * kLanes + static_cast<int>(threadIdx.x)) * V, V);
    return;
  }
  for (int i = threadIdx.x * V; i < n; i += kLanes * V) {
    Run<V, F32> x;
    const int left = static_cast<int>(n) - i;
    if (left >= V) x.template load<STREAM>(g + i * W);
    else x.load_some(g + i * W, left);
    f(x, i, left);
  }
}

template <bool F32, bool STREAM>
__device__ __forceinline__ void chunk_squares(const unsigned char* g, int64_t n, double (&acc)[4]) {
  constexpr int V = F32 ? 4 : 8;
  for_runs<V, F32, STREAM>(g, n, [&](const Run<V, F32>& x, int, int) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const double d = x.get(k);
      acc[k & 3] = fma(d, d, acc[k & 3]);
    }
  });
}

template <bool F32, bool OUT, bool STREAM>
__device__ __forceinline__ void chunk_scale(const unsigned char* g, unsigned char* out, int64_t n, double f) {
  constexpr int V = F32 || OUT ? 4 : 8, O = OUT ? 4 : 2;
  for_runs<V, F32, STREAM>(g, n, [&](const Run<V, F32>& x, int first, int count) {
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = static_cast<float>(static_cast<double>(x.get(k)) * f);
    Run<V, OUT> y;
    y.put(v);
    if (count >= V) y.template store<STREAM>(out + first * O);
    else y.store_some(out + first * O, count);
  });
}

// Work-group w takes chunks w, w + gridDim.x, ... of the batch.  The first
// b.stream of them go past the caches, so that the memory-side cache is left
// to the last ones, which clipping reads first.
__global__ __launch_bounds__(kLanes) void grad_squares_kernel(const NormBatch b, double* partials) {
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int total = b.chunks[b.n];
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = find_mat(b.chunks, b.n, c);
    const NormDesc& d = b.d[i];
    const int64_t first = static_cast<int64_t>(c - b.chunks[i]) * kNormChunk, left = d.count - first;
    if (d.g_f32) {
      if (c < b.stream) chunk_squares<true, true>(d.g + first * 4, left, acc);
      else chunk_squares<true, false>(d.g + first * 4, left, acc);
    } else {
      if (c < b.stream) chunk_squares<false, true>(d.g + first * 2, left, acc);
      else chunk_squares<false, false>(d.g + first * 2, left, acc);
    }
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
// in the memory-side cache still.  STREAM: reads and writes go past the caches.
template <bool STREAM>
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
      if (d.out_f32) chunk_scale<true, true, STREAM>(d.g + first * 4, d.out + first * 4, left, f);
      else chunk_scale<true, false, STREAM>(d.g + first * 4, d.out + first * 2, left, f);
    } else {
      if (d.out_f32) chunk_scale<false, true, STREAM>(d.g + first * 2, d.out + first * 4, left, f);
      else chunk_scale<false, false, STREAM>(d.g + first * 2, d.out + first * 2, left, f);
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
  const auto kernel = b.large ? grad_clip_kernel<true> : grad_clip_kernel<false>;
  hipLaunchKernelGGL(kernel, groups(b), dim3(kLanes), 0, s, b, partials, n, norm, max_norm);
  return hipGetLastError();
}

}  // namespace muon
