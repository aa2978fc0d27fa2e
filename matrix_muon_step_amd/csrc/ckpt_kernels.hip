// 8-bit activation checkpoints on gfx950 and the weight gradient from them.
//
// A block of 32 tokens x 32 columns shares the exponent e, the smallest
// integer >= -117 with max |x| <= 448 * 2^e over its finite values; each
// value is held as the e4m3 number nearest to x * 2^-e (ties to even), so
// the error is at most 2^-4 of the value, or half of 2^-9 * 2^e for values
// below 2^-6 * 2^e.  NaN and infinities are held as NaN.  A held value has
// four significant bits, so it is exact in bfloat16 and the gradient
//   G[o][c] = sum_t dY[t][o] X[t][c]
// is a product of exact bfloat16 operands, accumulated in float32.
#include "ckpt_internal.h"
#include "muon_internal.h"

namespace muon {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2v_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

#define LAS __attribute__((address_space(3)))

__device__ __forceinline__ int find64(const int64_t* __restrict__ prefix, int n, int64_t blk) {
  int i = 0;
  while (i + 1 < n && prefix[i + 1] <= blk) ++i;
  return i;
}

// Loads 16 bytes of a row of `cols` elements of ES bytes from element `col`
// on (any alignment), zero past the row's end.
template <int ES>
__device__ __forceinline__ uint4 load_row16(const unsigned char* row, int col, int cols) {
  constexpr int N = 16 / ES;
  uint4 u = {0, 0, 0, 0};
  if (col + N <= cols) return gld<uint4>(row + static_cast<int64_t>(col) * ES);
  if constexpr (ES == 2) {
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? gld<uint16_t>(row + (static_cast<int64_t>(col) + i) * 2) : 0;
    __builtin_memcpy(&u, e, 16);
  } else {
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = col + i < cols ? gld<uint32_t>(row + (static_cast<int64_t>(col) + i) * 4) : 0;
    __builtin_memcpy(&u, e, 16);
  }
  return u;
}
template <int ES>
__device__ __forceinline__ void store_row16(unsigned char* row, int col, int cols, uint4 u) {
  constexpr int N = 16 / ES;
  if (col + N <= cols) {
    gst(row + static_cast<int64_t>(col) * ES, u);
    return;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (col + i < cols) {
      if constexpr (ES == 2) gst(row + (static_cast<int64_t>(col) + i) * 2, static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
      else gst(row + (static_cast<int64_t>(col) + i) * 4, w[i]);
    }
}

// LDS row pitch of the 32 x 256 staging tile (bytes): rows 64 bytes apart
// modulo the 256 bytes of the banks, so that four rows' transposing reads
// (or four rows' dword reads) meet no conflict.
template <int ES>
constexpr int kPitch = kCkGroupCols * ES + 64;

// ------------------------------------------------------------------ write
// One work-group: 32 tokens x 256 columns through LDS; each wave then takes
// two blocks, a lane the 16 values that it stores.  Bound by memory.
template <int ES>
__device__ __forceinline__ void write_group(const CkDesc& d, int R, int group, LAS unsigned char* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int CPR = kCkGroupCols * ES / 16;  // 16-byte chunks of a row
  const int c0 = group * kCkGroupCols;
  const int rows = min(kCkTile, d.tokens - R * kCkTile);
  uint4 u[kCkTile * CPR / 256];
#pragma unroll
  for (int i = 0; i < kCkTile * CPR / 256; ++i) {
    const int p = i * 256 + tid, row = p / CPR, col = c0 + (p % CPR) * (16 / ES);
    u[i] = (uint4){0, 0, 0, 0};
    if (row < rows && col < d.cols)
      u[i] = load_row16<ES>(d.x + (static_cast<int64_t>(R) * kCkTile + row) * d.stride * ES, col, d.cols);
  }
#pragma unroll
  for (int i = 0; i < kCkTile * CPR / 256; ++i) {
    const int p = i * 256 + tid, row = p / CPR;
    *(LAS u32x4_t*)(lds + row * kPitch<ES> + (p % CPR) * 16) = (u32x4_t){u[i].x, u[i].y, u[i].z, u[i].w};
  }
  __syncthreads();
  const int n = lane & 31, h = lane >> 5;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int S = c0 / kCkTile + wave * 2 + b;
    if (S >= d.blocks) continue;
    float x[16];
    if constexpr (ES == 2) {
      // transposing reads: 4 tokens of the lane's column each
      const int j = (lane & 15) >> 2, cb = (wave * 2 + b) * 32 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * (k >> 1) + 8 * h + 4 * (k & 1) + j;
        const bf16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)(lds + row * kPitch<ES> + cb * 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * k + i] = static_cast<float>(v[i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int row = 16 * (k >> 3) + 8 * h + (k & 7);
        x[k] = *(const LAS float*)(lds + row * kPitch<ES> + ((wave * 2 + b) * 32 + n) * 4);
      }
    }
    // Largest finite magnitude: the bits of non-negative floats order as
    // integers.
    int top = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int a = __float_as_int(x[k]) & 0x7fffffff;
      if (a >= 0x7f800000) x[k] = __builtin_nanf("");
      else top = max(top, a);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = max(top, __shfl_xor(top, off, 64));
    // 448 = 1.75 * 2^8
    const int e = max((top >> 23) - 135 + ((top & 0x7fffff) > 0x600000 ? 1 : 0), kCkMinExp);
    const float mul = __int_as_float((127 - e) << 23);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k] * mul, x[4 * k + 1] * mul, 0, false);
      w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k + 2] * mul, x[4 * k + 3] * mul, v, true);
    }
    const int64_t blk = static_cast<int64_t>(R) * d.blocks + S;
    gst(d.codes + blk * kCkBlockBytes + lane * 16, (uint4){w[0], w[1], w[2], w[3]});
    if (lane == 0) gst(d.exps + blk, static_cast<uint8_t>(e + 127));
  }
}

__global__ __launch_bounds__(256) void ckpt_write_kernel(const CkBatch b) {
  __shared__ __align__(1024) unsigned char smem[kCkTile * kPitch<4>];
  const int i = find64(b.prefix, b.n, blockIdx.x);
  const CkDesc d = b.d[i];
  const int idx = blockIdx.x - static_cast<int>(b.prefix[i]);
  if (d.f32) write_group<4>(d, idx / d.groups, idx % d.groups, (LAS unsigned char*)smem);
  else write_group<2>(d, idx / d.groups, idx % d.groups, (LAS unsigned char*)smem);
}

// ------------------------------------------------------------------- read
template <int ES>
__device__ __forceinline__ void read_group(const CkDesc& d, int R, int group, LAS unsigned char* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int CPR = kCkGroupCols * ES / 16;
  const int c0 = group * kCkGroupCols;
  const int rows = min(kCkTile, d.tokens - R * kCkTile);
  const int n = lane & 31, h = lane >> 5;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int S = c0 / kCkTile + wave * 2 + b;
    if (S >= d.blocks) continue;
    const int64_t blk = static_cast<int64_t>(R) * d.blocks + S;
    const uint4 u = gld<uint4>(d.codes + blk * kCkBlockBytes + lane * 16);
    const float mul = __int_as_float(static_cast<int>(gld<uint8_t>(d.exps + blk)) << 23);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const f32x2v_t v = k & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(w[k >> 1], true)
                               : __builtin_amdgcn_cvt_pk_f32_fp8(w[k >> 1], false);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * k + i, row = 16 * (t >> 3) + 8 * h + (t & 7);
        LAS unsigned char* p = lds + row * kPitch<ES> + ((wave * 2 + b) * 32 + n) * ES;
        const float x = v[i] * mul;
        if constexpr (ES == 2) *(LAS __bf16*)p = static_cast<__bf16>(x);
        else *(LAS float*)p = x;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCkTile * CPR / 256; ++i) {
    const int p = i * 256 + tid, row = p / CPR, col = c0 + (p % CPR) * (16 / ES);
    if (row < rows && col < d.cols) {
      const u32x4_t v = *(const LAS u32x4_t*)(lds + row * kPitch<ES> + (p % CPR) * 16);
      store_row16<ES>(d.x + (static_cast<int64_t>(R) * kCkTile + row) * d.stride * ES, col, d.cols,
                      (uint4){v.x, v.y, v.z, v.w});
    }
  }
}

__global__ __launch_bounds__(256) void ckpt_read_kernel(const CkBatch b) {
  __shared__ __align__(1024) unsigned char smem[kCkTile * kPitch<4>];
  const int i = find64(b.prefix, b.n, blockIdx.x);
  const CkDesc d = b.d[i];
  const int idx = blockIdx.x - static_cast<int>(b.prefix[i]);
  if (d.f32) read_group<4>(d, idx / d.groups, idx % d.groups, (LAS unsigned char*)smem);
  else read_group<2>(d, idx / d.groups, idx % d.groups, (LAS unsigned char*)smem);
}

// --------------------------------------------------------------- gradient
// One work-group: a 256 x 256 tile of G over one part of the tokens, 8 waves
// as 2 x 4, wave tile 128 (outs) x 64 (cols), 32x32x16 products.  A step is
// 32 tokens: dY's 32 x 256 (16 KB, rows of 512 bytes, 16-byte chunk c of row
// k at (c + 4 (k & 3)) mod 32 so that the transposing reads meet no bank
// conflict) and 8 checkpoint blocks (8 KB, as they lie).
constexpr int kGT = kGradTile;
constexpr int kGradStageA = 32 * kGT * 2;
constexpr int kGradStage = kGradStageA + 8 * kCkBlockBytes;

__device__ __forceinline__ void load_lds16(const unsigned char* base, uint32_t bytes, uint32_t off,
                                           LAS unsigned char* dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uintptr_t a = reinterpret_cast<uintptr_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  void* p = reinterpret_cast<void*>((static_cast<uintptr_t>(hi) << 32) | lo);
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(p, 0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LAS void*)dst, 16, off, 0, 0, 0);
#endif
}

template <bool ALIGNED>
__global__ __launch_bounds__(512, 1) void ckpt_grad_kernel(const GradBatch b) {
  __shared__ __align__(1024) unsigned char smem[2 * kGradStage];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring work items on one XCD (work-groups go to the 8 XCDs in turn)
  const int total = b.prefix[b.n], per = (total + 7) / 8;
  const int item = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (item >= total) return;
  const int mi = find_mat(b.prefix, b.n, item);
  const GradDesc d = b.d[mi];
  const int local = item - b.prefix[mi];
  const int split = local / (d.mt * d.nt), tile = local % (d.mt * d.nt);
  const int m0 = (tile % d.mt) * kGT, n0 = (tile / d.mt) * kGT;
  const int steps_all = (d.tokens + 31) / 32;
  const int s0 = split * d.per_split, s1 = min(steps_all, s0 + d.per_split);
  const int wm = (wave & 1) * 128, wn = (wave >> 1) * 64;

  auto issue = [&](int st, int slot) {
    LAS unsigned char* dst = lds + slot * kGradStage;
    const int64_t t0 = static_cast<int64_t>(st) * 32;
    const int rows = static_cast<int>(min<int64_t>(32, d.tokens - t0));
    const unsigned char* base = d.dy + (t0 * d.dy_stride + m0) * 2;
    const int width = min(kGT, d.outs - m0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = (wave + i * 8) * 64 + lane, k = p / 32, c = (p - 4 * (k & 3)) & 31;
      if constexpr (ALIGNED) {
        // whole 16-byte chunks: what the last one holds past `outs` meets only
        // rows of G that are not stored
        load_lds16(base, static_cast<uint32_t>((rows - 1) * d.dy_stride * 2 + (width * 2 + 15) / 16 * 16),
                   static_cast<uint32_t>(k * d.dy_stride * 2) + c * 16, dst + (wave + i * 8) * 1024);
      } else {
        uint4 u = {0, 0, 0, 0};
        if (k < rows && c * 8 < width) u = load_row16<2>(base + k * d.dy_stride * 2, c * 8, width);
        *(LAS u32x4_t*)(dst + p * 16) = (u32x4_t){u.x, u.y, u.z, u.w};
      }
    }
    // blocks past the last column are left out (their columns are not stored)
    const int S = min(n0 / kCkTile + wave, d.blocks - 1);
    load_lds16(d.codes + (static_cast<int64_t>(st) * d.blocks + S) * kCkBlockBytes, kCkBlockBytes, lane * 16,
               dst + kGradStageA + wave * 1024);
  };

  f32x16_t acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (f32x16_t)(0.f);
  // transposing reads: lane row 8 h + j (+ 4), column group of the lane
  const int j = (lane & 15) >> 2, krow = 8 * h + j;
  int aoff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (wm + 32 * i + 16 * ((lane >> 4) & 1) + 4 * (lane & 3)) >> 3;
    aoff[i] = krow * 512 + ((c + 4 * j) & 31) * 16 + (lane & 1) * 8;
  }
  const int S0 = min(n0 / kCkTile + (wn >> 5), d.blocks - 1), S1 = min(n0 / kCkTile + (wn >> 5) + 1, d.blocks - 1);
  if (s0 < s1) issue(s0, 0);
  for (int st = s0; st < s1; ++st) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (st + 1 < s1) issue(st + 1, (st + 1 - s0) & 1);
    const LAS unsigned char* src = lds + ((st - s0) & 1) * kGradStage;
    float mul[2];
    mul[0] = __int_as_float(static_cast<int>(gld<uint8_t>(d.exps + static_cast<int64_t>(st) * d.blocks + S0)) << 23);
    mul[1] = __int_as_float(static_cast<int>(gld<uint8_t>(d.exps + static_cast<int64_t>(st) * d.blocks + S1)) << 23);
    bf16x8_t x[2][2];
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
      const u32x4_t w = *(const LAS u32x4_t*)(src + kGradStageA + ((wn >> 5) + jb) * 1024 + lane * 16);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x2_t v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s], mul[jb], false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s], mul[jb], true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s + 1], mul[jb], false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s + 1], mul[jb], true)};
        __builtin_memcpy(&x[jb][s], v, 16);
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const LAS unsigned char* p = src + aoff[i] + s * 16 * 512;
        const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)p);
        const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)(p + 4 * 512));
        const bf16x8_t a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int jb = 0; jb < 2; ++jb)
          acc[i][jb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, x[jb][s], acc[i][jb], 0, 0, 0);
      }
  }
  // Results: column n0 + wn + 32 jb + (lane & 31), four runs of four rows.
  float* part = d.splits > 1 ? d.part + static_cast<int64_t>(split) * d.outs * d.cols : nullptr;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
      const int col = n0 + wn + 32 * jb + (lane & 31);
      if (col >= d.cols) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = m0 + wm + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row >= d.outs) continue;
        const int64_t at = static_cast<int64_t>(row) * d.cols + col;
        float v = acc[i][jb][r];
        if (part) {
          gst(part + at, v);
        } else if (d.g_f32) {
          if (d.accumulate) v += gld<float>(d.G + at * 4);
          gst(d.G + at * 4, v);
        } else {
          if (d.accumulate) v += static_cast<float>(gld<__bf16>(d.G + at * 2));
          gst(d.G + at * 2, static_cast<__bf16>(v));
        }
      }
    }
}

// Joins the parts of a split token range in order and rounds once.
__global__ __launch_bounds__(256) void grad_join_kernel(const GradBatch b) {
  const int mi = find_mat(b.sums, b.n, blockIdx.x);
  const GradDesc d = b.d[mi];
  const int64_t n = static_cast<int64_t>(d.outs) * d.cols;
  const int64_t base = static_cast<int64_t>(blockIdx.x - b.sums[mi]) * kGradSumElems;
#pragma unroll
  for (int i = 0; i < kGradSumElems / 256; ++i) {
    const int64_t at = base + i * 256 + threadIdx.x;
    if (at >= n) return;
    float v = 0.f;
    for (int s = 0; s < d.splits; ++s) v += gld<float>(d.part + s * n + at);
    if (d.g_f32) {
      if (d.accumulate) v += gld<float>(d.G + at * 4);
      gst(d.G + at * 4, v);
    } else {
      if (d.accumulate) v += static_cast<float>(gld<__bf16>(d.G + at * 2));
      gst(d.G + at * 2, static_cast<__bf16>(v));
    }
  }
}

}  // namespace

hipError_t launch_ckpt_write(const CkBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(ckpt_write_kernel, dim3(static_cast<uint32_t>(b.prefix[b.n])), dim3(256), 0, s, b);
  return hipGetLastError();
}
hipError_t launch_ckpt_read(const CkBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(ckpt_read_kernel, dim3(static_cast<uint32_t>(b.prefix[b.n])), dim3(256), 0, s, b);
  return hipGetLastError();
}
hipError_t launch_ckpt_grad(const GradBatch& b, bool aligned, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>((b.prefix[b.n] + 7) / 8 * 8));
  if (aligned) hipLaunchKernelGGL(ckpt_grad_kernel<true>, grid, dim3(512), 0, s, b);
  else hipLaunchKernelGGL(ckpt_grad_kernel<false>, grid, dim3(512), 0, s, b);
  return hipGetLastError();
}
hipError_t launch_grad_join(const GradBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(grad_join_kernel, dim3(static_cast<uint32_t>(b.sums[b.n])), dim3(256), 0, s, b);
  return hipGetLastError();
}

}  // namespace muon
