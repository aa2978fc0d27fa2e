// 8-bit activation checkpoints on gfx950 and the weight gradient from them.
//
// A block of 32 tokens x 32 columns shares the exponent e, the smallest
// integer >= -117 with max |x| <= 448 * 2^e over its finite values; each
// value is held as the e4m3 number nearest to x * 2^-e (ties to even), so
// the error is at most 2^-4 of the value, or half of 2^-9 * 2^e for values
// below 2^-6 * 2^e; from 1.875 * 2^127 on it is held as that, the largest one
// that float32 and bfloat16 can hold.  NaN and infinities are held as NaN.  A held
// value has four significant bits, so it is exact in bfloat16 and the gradient
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
// two blocks, a lane the 16 values that it stores, so that reads run along
// rows and a block is stored as 1 KB at once.  Bound by memory: 8192 x 6400
// bfloat16, 29 us, 5.4 TB/s of 6.2 that a plain copy reaches.
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
    // At the largest exponent the code after 240 would stand for 2^128, which
    // is no float32 number: what would round up to it keeps 240.
    if (e == kCkMaxExp) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (fabsf(x[k]) > 0x1.ep127f) x[k] = copysignf(0x1.ep127f, x[k]);
    }
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k] * mul, x[4 * k + 1] * mul, 0, false);
      w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k + 2] * mul, x[4 * k + 3] * mul, v, true);
    }
    const int64_t blk = static_cast<int64_t>(R) * d.blocks + S;
    gst(d.codes + blk * kCkBlockBytes + lane * 16, (uint4){w[0], w[1], w[2], w[3]});
    if (lane == 0) gst(d.exps + static_cast<int64_t>(S) * d.rblocks + R, static_cast<uint8_t>(e + 127));
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
// The other way round: 26 us, 6.0 TB/s at 8192 x 6400 to bfloat16.
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
    const float mul = __int_as_float(static_cast<int>(gld<uint8_t>(d.exps + static_cast<int64_t>(S) * d.rblocks + R)) << 23);
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
// One work-group: T x T tiles of G, each over its tokens or a part of them, NWM
// x NWN waves, 32x32x16 products.  A step is 32 tokens: dY's 32 x T (rows of 2 T
// bytes, 16-byte chunk c of row k at (c + 4 (k & 3)) mod T / 8, so that the
// transposing reads meet no bank conflict) and T / 32 checkpoint blocks as
// they lie.  A ring of four steps in LDS, filled by direct loads three steps
// ahead (ALIGNED) or, for a dY whose rows are not 16-byte aligned, through
// registers one step ahead.  The 8-bit operand halves what the right side
// reads of LDS and memory; its conversion (8 instructions a block and wave,
// the exponent applied by the same instruction) runs under the products.
// 1600 x 6400 from 16384 tokens: 363 to 410 us on different cards (0.82 to 0.92
// PFLOP/s; bfloat16 operands through the library 475), of which the joining
// launch takes 27; 12% of the products are padding of edge tiles (1600 is 6.25
// x 256), and the matrix cores are busy for 53% of the product kernel's cycles
// (58% of those of units with work).  4096 x 4096 from 2048 tokens: 64 us (1.07
// PFLOP/s).
template <int T_, int NWM_, int NWN_>
struct GradGeo {
  static constexpr int T = T_, NWM = NWM_, NWN = NWN_, NW = NWM * NWN;
  static constexpr int WM = T / NWM, WN = T / NWN, MB = WM / 32, NB = WN / 32;
  static constexpr int NC = T / 8;                 // chunks of a dY row
  static constexpr int A = 32 * T * 2;             // bytes of a step's dY
  static constexpr int STAGE = A + T / 32 * kCkBlockBytes;
  static constexpr int PA = A / 1024 / NW;         // direct loads of a wave and step: dY
  static constexpr int ROWS = NW * 64 / NC;        // rows between a wave's loads
};

// 16 bytes a lane from base + off to dst + 16 lane, zero from `bytes` on.
__device__ __forceinline__ void load_lds16(const unsigned char* base, uint32_t bytes, uint32_t off,
                                           LAS unsigned char* __restrict__ dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(base), 0, bytes, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LAS void*)dst, 16, off, 0, 0, 0);
#endif
}

// One column block of a step as right operands: 16 bytes a lane, to bfloat16.
__device__ __forceinline__ void block_operand(const LAS unsigned char* __restrict__ p, float mul, bf16x8_t (&x)[2]) {
  const u32x4_t w = *(const LAS u32x4_t*)p;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const bf16x2_t v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s], mul, false),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s], mul, true),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s + 1], mul, false),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * s + 1], mul, true)};
    __builtin_memcpy(&x[s], v, 16);
  }
}

// Left operand: 32 columns of dY (lane address at), 16 tokens.
template <int PITCH>
__device__ __forceinline__ bf16x8_t dy_operand(const LAS unsigned char* __restrict__ p) {
  const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)p);
  const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)(p + 4 * PITCH));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A wave's loads of the next step: dY rows from `ap` on, one checkpoint block.
template <class C>
struct GradLoad {
  static_assert(C::T / 32 == C::NW, "one block per wave and step");
  const unsigned char *ap, *xp;
  int ld2, xstep;        // bytes of a dY row; of a row of blocks
  int left;              // tokens from the step's first on
  int tail;              // bytes of a dY row that are read
  uint32_t off[C::PA];
  // dst: the step's place in LDS
  __device__ __forceinline__ void blocks(LAS unsigned char* __restrict__ dst, int wave, int lane) {
    load_lds16(xp, kCkBlockBytes, lane * 16, dst + C::A + wave * 1024);
    xp += xstep;
  }
  __device__ __forceinline__ void advance() {
    ap += static_cast<int64_t>(ld2) * 32;
    left -= 32;
  }
  __device__ __forceinline__ void direct(LAS unsigned char* __restrict__ dst, int wave, int lane) {
    const uint32_t bytes = static_cast<uint32_t>((min(left, 32) - 1) * ld2 + tail);
#pragma unroll
    for (int i = 0; i < C::PA; ++i) load_lds16(ap, bytes, off[i], dst + (wave + i * C::NW) * 1024);
    blocks(dst, wave, lane);
    advance();
  }
};

// One step: the loads of a later one into dst (MORE) and this one's products
// from src.  One function, so that the compiler knows that its reads do not
// depend on the loads under way.
template <class C, bool DIRECT>
__device__ __forceinline__ void grad_step(const LAS unsigned char* __restrict__ src, LAS unsigned char* __restrict__ dst,
                                          bool more, GradLoad<C>& ld, int wave, int lane, const int (&aoff)[C::MB], int boff,
                                          const float (&mul)[C::NB], f32x16_t (&acc)[C::MB][C::NB]) {
  if (more) {
    if constexpr (DIRECT) ld.direct(dst, wave, lane);
    else ld.blocks(dst, wave, lane);
  }
  bf16x8_t x[C::NB][2];
#pragma unroll
  for (int jb = 0; jb < C::NB; ++jb) block_operand(src + boff + jb * 1024, mul[jb], x[jb]);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < C::MB; ++i) {
      const bf16x8_t av = dy_operand<2 * C::T>(src + aoff[i] + s * 16 * 2 * C::T);
#pragma unroll
      for (int jb = 0; jb < C::NB; ++jb)
        acc[i][jb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, x[jb][s], acc[i][jb], 0, 0, 0);
    }
}

// Stores a wave's results: column col0 + 32 jb, rows row0 + 32 i + 8 g + r
// (g, r = 0..3).  WHOLE: every element lies in G.
template <class C, class E, bool ADD, bool WHOLE>
__device__ __forceinline__ void grad_store(const GradDesc& d, int row0, int col0, const f32x16_t (&acc)[C::MB][C::NB]) {
#pragma unroll
  for (int i = 0; i < C::MB; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = row0 + 32 * i + 8 * (r >> 2) + (r & 3);
      if (!WHOLE && row >= d.outs) continue;
      unsigned char* p = d.G + (static_cast<int64_t>(row) * d.cols + col0) * sizeof(E);
#pragma unroll
      for (int jb = 0; jb < C::NB; ++jb) {
        if (!WHOLE && col0 + 32 * jb >= d.cols) continue;
        float v = acc[i][jb][r];
        if (ADD) v += static_cast<float>(gld<E>(p + 32 * jb * sizeof(E)));
        gst(p + 32 * jb * sizeof(E), static_cast<E>(v));
      }
    }
}

// Steps s0 .. s1 - 1 (one at least) of the tile at (m0, n0) of G.
template <class C, bool ALIGNED>
__device__ __forceinline__ void grad_tile(const GradDesc& d, int m0, int n0, int s0, int s1, LAS unsigned char* lds, int wave,
                                          int lane, f32x16_t (&acc)[C::MB][C::NB]) {
  const int h = lane >> 5;
  const int wm = (wave % C::NWM) * C::WM, wn = (wave / C::NWM) * C::WN;
  const int p0 = wave * 64 + lane, k0 = p0 / C::NC, ch = (p0 - 4 * (k0 & 3)) & (C::NC - 1);
  const int width = min(C::T, d.outs - m0);
  GradLoad<C> ld;
  ld.ld2 = static_cast<int>(d.dy_stride * 2);
  ld.xstep = d.blocks * kCkBlockBytes;
  ld.ap = d.dy + (static_cast<int64_t>(s0) * 32 * d.dy_stride + m0) * 2;
  // (the last block again past the last column: those columns of G are not stored)
  ld.xp = d.codes + (static_cast<int64_t>(s0) * d.blocks + min(n0 / kCkTile + wave, d.blocks - 1)) * kCkBlockBytes;
  ld.left = d.tokens - s0 * 32;
  // The loads' range is checked for each of a chunk's four words: in the last
  // row they end with the word that holds the last element, the rest is zero.
  // In other rows a chunk goes on past `outs`: those values meet only rows of G that
  // are not stored.
  ld.tail = (width * 2 + 3) / 4 * 4;
#pragma unroll
  for (int i = 0; i < C::PA; ++i) ld.off[i] = static_cast<uint32_t>((k0 + i * C::ROWS) * ld.ld2 + ch * 16);
  // dY through registers: rows of any alignment.
  uint4 held[C::PA];
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < C::PA; ++i) {
      const int k = k0 + i * C::ROWS;
      held[i] = (uint4){0, 0, 0, 0};
      if (k < ld.left && ch * 8 < width) {
        // A chunk may run on into the rows behind (of narrow matrices, into
        // several), not past dY's last element.
        const unsigned char* p = ld.ap + static_cast<int64_t>(k) * ld.ld2;
        if (min(ld.left - 1 - k, 8) * (ld.ld2 >> 1) + d.outs - m0 >= ch * 8 + 8) held[i] = gld<uint4>(p + ch * 16);
        else held[i] = load_row16<2>(p, ch * 8, d.outs - m0);
      }
    }
  };
  auto put = [&](int at) {
#pragma unroll
    for (int i = 0; i < C::PA; ++i)
      *(LAS u32x4_t*)(lds + at + (wave + i * C::NW) * 1024 + lane * 16) =
          (u32x4_t){held[i].x, held[i].y, held[i].z, held[i].w};
    ld.advance();
  };

  // transposing reads: lane row 8 h + j (+ 4), column group of the lane
  const int j = (lane & 15) >> 2, krow = 8 * h + j;
  int aoff[C::MB];
#pragma unroll
  for (int i = 0; i < C::MB; ++i) {
    const int c = (wm + 32 * i + 16 * ((lane >> 4) & 1) + 4 * (lane & 3)) >> 3;
    aoff[i] = krow * 2 * C::T + ((c + 4 * j) & (C::NC - 1)) * 16 + (lane & 1) * 8;
  }
  const int boff = C::A + (wn >> 5) * 1024 + lane * 16;
  // Exponents of the wave's column blocks: 64 steps at a time, one a lane.
  const unsigned char* ep[C::NB];
  int exps[C::NB];
#pragma unroll
  for (int jb = 0; jb < C::NB; ++jb) {
    ep[jb] = d.exps + static_cast<int64_t>(min(n0 / kCkTile + (wn >> 5) + jb, d.blocks - 1)) * d.steps;
    exps[jb] = 0;
  }
#pragma unroll
  for (int i = 0; i < C::MB; ++i)
#pragma unroll
    for (int jb = 0; jb < C::NB; ++jb) acc[i][jb] = (f32x16_t)(0.f);

  const int n = s1 - s0;
  int cur = 0, fill = 0;  // places of this step and of the next to load
  auto next = [](int at) { return at == 3 * C::STAGE ? 0 : at + C::STAGE; };
  if constexpr (ALIGNED) {
    for (int i = 0; i < 3; ++i)
      if (i < n) {
        ld.direct(lds + fill, wave, lane);
        fill = next(fill);
      }
  } else {
    fetch();
    ld.blocks(lds, wave, lane);
    put(0);
    fill = C::STAGE;
    if (n > 1) {
      fetch();
      ld.blocks(lds + C::STAGE, wave, lane);
    }
  }
  for (int st = 0; st < n; ++st) {
    if (st % 64 == 0) {
#pragma unroll
      for (int jb = 0; jb < C::NB; ++jb) exps[jb] = gld<uint8_t>(ep[jb] + min(s0 + st + lane, d.steps - 1));
      // waited for here, not at every step's use
#pragma unroll
      for (int jb = 0; jb < C::NB; ++jb) asm volatile("" : "+v"(exps[jb]));
    }
    float mul[C::NB];
#pragma unroll
    for (int jb = 0; jb < C::NB; ++jb) mul[jb] = __int_as_float(__builtin_amdgcn_readlane(exps[jb], st & 63) << 23);
    // step st of this wave's loads has landed (of later ones, two steps' may
    // be under way, or one's registers and blocks), its reads of step st - 1
    // are behind it; past the barrier that holds for all waves
    asm volatile("" ::: "memory");
    if (st + 2 >= n) __builtin_amdgcn_s_waitcnt(0x0070);
    else __builtin_amdgcn_s_waitcnt(0x0070 + (ALIGNED ? 2 : 1) * (C::PA + 1));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int after = next(fill);
    grad_step<C, ALIGNED>(lds + cur, lds + (ALIGNED ? fill : after), st + (ALIGNED ? 3 : 2) < n, ld, wave, lane, aoff, boff,
                          mul, acc);
    if constexpr (!ALIGNED) {
      if (st + 1 < n) put(fill);
      if (st + 2 < n) fetch();
    }
    cur = next(cur);
    fill = after;
  }
}

// A wave's results into G.
template <class C>
__device__ __forceinline__ void grad_out(const GradDesc& d, int m0, int n0, int wave, int lane,
                                         const f32x16_t (&acc)[C::MB][C::NB]) {
  const bool whole = m0 + C::WM * C::NWM <= d.outs && n0 + C::WN * C::NWN <= d.cols;
  const int row0 = m0 + (wave % C::NWM) * C::WM + 4 * (lane >> 5), col0 = n0 + (wave / C::NWM) * C::WN + (lane & 31);
  if (d.g_f32) {
    if (d.accumulate) grad_store<C, float, true, false>(d, row0, col0, acc);
    else if (whole) grad_store<C, float, false, true>(d, row0, col0, acc);
    else grad_store<C, float, false, false>(d, row0, col0, acc);
  } else {
    if (d.accumulate) grad_store<C, __bf16, true, false>(d, row0, col0, acc);
    else if (whole) grad_store<C, __bf16, false, true>(d, row0, col0, acc);
    else grad_store<C, __bf16, false, false>(d, row0, col0, acc);
  }
}

// A lane's 16 bytes x of a piece, x = 0 .. 4 MB NB - 1: a wave's are 1 KB apart.
template <class C>
__device__ __forceinline__ float* piece_at(float* pieces, int64_t piece, int wave, int lane) {
  return pieces + (piece * C::NW + wave) * (C::MB * C::NB * 1024) + lane * 4;
}

// The matrix whose tiles or steps hold position pos: the last whose range
// begins at or before it (matrices without any are passed over).
template <class T>
__device__ __forceinline__ int grad_find(const T* __restrict__ prefix, int n, int64_t pos) {
  int i = 0;
  for (int k = 1; k < n; ++k)
    if (prefix[k] <= pos) i = k;
  return i;
}

// Zeros for bytes kGradZeros * piece on of a matrix without tokens (G is dense
// and 16-byte aligned), by LANES lanes.  Behind all tiles, since work items in
// between would leave some XCDs with zeros only: 2048 x 7168 in bfloat16 from
// 777 tokens 27 us, with one such empty matrix 28, as tiles among tiles 47.
template <int LANES>
__device__ __forceinline__ void grad_zeros(const GradDesc& d, int64_t piece, int lane) {
  const int64_t total = static_cast<int64_t>(d.outs) * d.cols * (d.g_f32 ? 4 : 2);
  const int64_t end = min(total, (piece + 1) * kGradZeros);
  for (int64_t at = piece * kGradZeros + lane * 16; at < end; at += LANES * 16) {
    if (at + 16 <= end) gst(d.G + at, (uint4){0, 0, 0, 0});
    else
      for (int64_t e = at; e < end; e += 2) gst(d.G + e, static_cast<uint16_t>(0));
  }
}

template <class C, bool ALIGNED>
__global__ __launch_bounds__(C::NW * 64, 2) void ckpt_grad_kernel(const GradBatch b) {
  __shared__ __align__(1024) unsigned char smem[4 * C::STAGE];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring work items on one XCD (work-groups go to the 8 XCDs in turn)
  const int items = b.parts ? b.parts : b.tiles[b.n], per = (items + 7) / 8;
  if (static_cast<int>(blockIdx.x) >= 8 * per) {
    const int zero = b.tiles[b.n] + static_cast<int>(blockIdx.x) - 8 * per, mi = grad_find(b.tiles, b.all, zero);
    grad_zeros<C::NW * 64>(b.d[mi], zero - b.tiles[mi], threadIdx.x);
    return;
  }
  const int item = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (item >= items) return;
  f32x16_t acc[C::MB][C::NB];
  if (!b.parts) {
    const int mi = grad_find(b.tiles, b.n, item);
    const GradDesc d = b.d[mi];
    const int tile = item - b.tiles[mi], m0 = tile % d.mt * C::T, n0 = tile / d.mt * C::T;
    grad_tile<C, ALIGNED>(d, m0, n0, 0, d.steps, lds, wave, lane, acc);
    grad_out<C>(d, m0, n0, wave, lane, acc);
    return;
  }
  int64_t pos = item * b.share;
  const int64_t end = min(pos + b.share, b.steps[b.n]);
  while (pos < end) {
    const int mi = grad_find(b.steps, b.n, pos);
    const GradDesc d = b.d[mi];
    const int64_t in = pos - b.steps[mi];
    const int tile = static_cast<int>(in / d.steps), s0 = static_cast<int>(in % d.steps);
    const int s1 = static_cast<int>(min<int64_t>(d.steps, s0 + (end - pos)));
    const int m0 = tile % d.mt * C::T, n0 = tile / d.mt * C::T;
    // every wave is done with the last tile's steps
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    grad_tile<C, ALIGNED>(d, m0, n0, s0, s1, lds, wave, lane, acc);
    if (s0 == 0 && s1 == d.steps) {
      grad_out<C>(d, m0, n0, wave, lane, acc);
    } else {
      float* p = piece_at<C>(b.pieces, 2 * static_cast<int64_t>(item) + (s0 == 0 ? 1 : 0), wave, lane);
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int jb = 0; jb < C::NB; ++jb)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            gst(p + ((i * C::NB + jb) * 4 + g) * 256, make_float4(acc[i][jb][4 * g], acc[i][jb][4 * g + 1],
                                                                   acc[i][jb][4 * g + 2], acc[i][jb][4 * g + 3]));
    }
    pos += s1 - s0;
  }
}

// The tiles that a border cut: their pieces summed in
// order, rounded once.  A work-group is one wave: 32 rows of what a wave of
// the product kernel holds, so that even one tile's many pieces are read by
// 32 of them.
template <class C>
__global__ __launch_bounds__(64) void grad_join_kernel(const GradBatch b) {
  using S = GradGeo<C::T, C::T / 32, C::NWN>;  // the same with one 32-row block a wave
  const int lane = threadIdx.x;
  const int strip = blockIdx.x % (C::NW * C::MB), wave = strip / C::MB, i = strip % C::MB;
  const int item = blockIdx.x / (C::NW * C::MB);
  const int mi = grad_find(b.tiles, b.n, item);
  const GradDesc d = b.d[mi];
  const int tile = item - b.tiles[mi];
  const int64_t first = b.steps[mi] + static_cast<int64_t>(tile) * d.steps, last = first + d.steps - 1;
  const int64_t w0 = first / b.share, w1 = last / b.share;
  if (w0 == w1) return;  // in one piece: stored already
  f32x16_t acc[1][C::NB];
#pragma unroll
  for (int jb = 0; jb < C::NB; ++jb) acc[0][jb] = (f32x16_t)(0.f);
#pragma unroll 4
  for (int64_t w = w0; w <= w1; ++w) {
    const float* p = piece_at<C>(b.pieces, 2 * w + (w * b.share <= first ? 1 : 0), wave, lane) + i * C::NB * 1024;
#pragma unroll
    for (int jb = 0; jb < C::NB; ++jb)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 v = gld<float4>(p + (jb * 4 + g) * 256);
        acc[0][jb][4 * g] += v.x;
        acc[0][jb][4 * g + 1] += v.y;
        acc[0][jb][4 * g + 2] += v.z;
        acc[0][jb][4 * g + 3] += v.w;
      }
  }
  const int row0 = tile % d.mt * C::T + (wave % C::NWM) * C::WM + 32 * i;
  grad_out<S>(d, row0, tile / d.mt * C::T + (wave / C::NWM) * C::WN, 0, lane, acc);
}

using Grad256 = GradGeo<256, 2, 4>;
using Grad128 = GradGeo<128, 2, 2>;

}  // namespace

hipError_t launch_ckpt_write(const CkBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(ckpt_write_kernel, dim3(static_cast<uint32_t>(b.prefix[b.n])), dim3(256), 0, s, b);
  return hipGetLastError();
}
hipError_t launch_ckpt_read(const CkBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(ckpt_read_kernel, dim3(static_cast<uint32_t>(b.prefix[b.n])), dim3(256), 0, s, b);
  return hipGetLastError();
}
template <class C>
static void launch_grad(const GradBatch& b, bool aligned, hipStream_t s) {
  const int items = b.parts ? b.parts : b.tiles[b.n];
  const dim3 grid(static_cast<uint32_t>((items + 7) / 8 * 8 + b.tiles[b.all] - b.tiles[b.n]));
  if (aligned) hipLaunchKernelGGL((ckpt_grad_kernel<C, true>), grid, dim3(C::NW * 64), 0, s, b);
  else hipLaunchKernelGGL((ckpt_grad_kernel<C, false>), grid, dim3(C::NW * 64), 0, s, b);
}
hipError_t launch_ckpt_grad(const GradBatch& b, int cfg, bool aligned, hipStream_t s) {
  if (cfg == kGrad256) launch_grad<Grad256>(b, aligned, s);
  else launch_grad<Grad128>(b, aligned, s);
  return hipGetLastError();
}
hipError_t launch_grad_join(const GradBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(grad_join_kernel<Grad256>, dim3(static_cast<uint32_t>(b.tiles[b.n]) * Grad256::NW * Grad256::MB), dim3(64), 0, s, b);
  return hipGetLastError();
}

}  // namespace muon
