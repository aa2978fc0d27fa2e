// Causal self-attention over packed sequences on gfx950, with the largest
// logit of each head (what QK-Clip needs), and its backward pass.
//
// Per sequence and head, with key head g = h / (heads / kv_heads):
//   s_ij = scale * q_i . k_j for j <= i
//   lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   delta_i = dO_i . o_i
//   dv_j = sum_i p_ij dO_i
//   ds_ij = p_ij (dO_i . v_j - delta_i)
//   dq_i = scale * sum_j ds_ij k_j,  dk_j = scale * sum_i ds_ij q_i
// dk and dv sum over the query heads that share a key head.  With a window
// (WIN) row i sees key j <= i where i - j < window or j < sinks.
//
// Every product runs on v_mfma_f32_32x32x16_bf16 with float32 accumulation.
// The score product is formed so that its result already lies as the next
// product's right operand: a 32x32 result holds, per lane (n = lane & 31,
// h = lane >> 5), column n and rows 8g + 4h + i (g, i = 0..3), and the
// operand of a 16-deep product wants, per lane, 8 values of the summed index
// for column n.  Summed indices may be taken in any order as long as both
// operands agree, so registers 8s .. 8s+7 serve product s as they are, with
// the left operand read in the same order: rows 16s + 4h + 0..3 and
// 16s + 8 + 4h + 0..3 of a row-major LDS tile, by two transposing reads.
// Softmax statistics stay in the lane that owns the row (or, in the dK/dV
// kernel, the column).
//
// Probabilities and ds are rounded to bfloat16 as operands of the second
// products (matrix cores take no wider ones at this rate); everything else
// is float32.
#pragma once

#include "attn_internal.h"
#include "muon_internal.h"

namespace muon {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

#define LAS __attribute__((address_space(3)))

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
// The rows' reference maximum moves only when a row outgrows it by 2^8:
// exponentials stay below 2^8, far inside float32 and bfloat16 range, and
// most tiles need no rescaling of the accumulators.
constexpr float kSlackLog2 = 8.f;

template <int DP>
struct Geo {
  static constexpr int KS = DP / 16;          // 16-deep steps over the head dimension
  static constexpr int DB = DP / 32;          // 32-wide blocks of the head dimension
  static constexpr int SUBB = kAttnStep * 64; // bytes of one 32-wide block of a streamed tile
  static constexpr int TILEB = DB * SUBB;     // bytes of a streamed tile
};

// A streamed tile of 64 rows lies in LDS as its 32-wide blocks one after
// another, each 64 rows of 64 bytes, with the row's four 16-byte chunks
// exclusive-or'ed by swz (muon_internal.h).  Both readers are free of bank
// conflicts with it (ordinary 16-byte reads of 32 rows; transposing reads of
// four whole rows), and since the pattern repeats every 16 rows, every
// fragment is one of four lane addresses plus a constant.

constexpr uint32_t kOutside = 0xC0000000u;  // an offset past every buffer's size (those stay below 2^31)

// Direct-to-LDS loads, 16 (WORD: 4) bytes a lane, lane i to dst + 16 i (4 i),
// from base + off + IMM, zero from byte `bytes` on.  base, bytes and dst are
// the same in every lane.  The instruction adds IMM to both of its addresses.
template <bool WORD, int IMM>
__device__ __forceinline__ void load_lds(const unsigned char* base, uint32_t bytes, uint32_t off,
                                         LAS unsigned char* __restrict__ dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  // untyped, no stride: offsets are compared with the size in bytes
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(base), 0, bytes, 0x00020000);
  if (WORD) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LAS void*)(dst - IMM), 4, off, 0, IMM, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LAS void*)(dst - IMM), 16, off, 0, IMM, 0);
#endif
}

// A wave's share of the loads of a tensor's 64-row tiles: 16 rows (16 (wave &
// 3) on) x 64 bytes per load, lane i row i / 4 and the chunk that the swizzle
// puts at place i % 4.  NW waves: loads for blocks (wave >> 2) + NW / 4 * i.
// EXACT: the head dimension is DP, else elements past it read as zero.  So do
// rows past the sequence.
template <int DP, bool EXACT, int NW>
struct TileLoad {
  static constexpr int N = DP / 8 / NW;  // loads per tile
  const unsigned char* p;                // the wave's first row of the next tile
  uint32_t off;
  int ts2, tail, dim, chunk;             // bytes of a token; valid bytes of a row from p on; EXACT only: -

  __device__ __forceinline__ TileLoad(const HeadsView& v, int64_t row, int head, int head_dim, int wave, int lane) {
    const int r = lane >> 2, c = swz(r, lane & 3), db0 = wave >> 2;
    ts2 = static_cast<int>(v.ts * 2);
    p = v.p + ((row + 16 * (wave & 3)) * v.ts + head * v.hs) * 2 + 64 * db0;
    off = static_cast<uint32_t>(r) * static_cast<uint32_t>(ts2) + c * 16;
    tail = 2 * (head_dim - 32 * db0);
    dim = head_dim - 32 * db0;
    chunk = c * 8;
  }
  __device__ __forceinline__ void move(int64_t bytes) { p += bytes; }
  template <int I>
  __device__ __forceinline__ void one(uint32_t bytes, LAS unsigned char* __restrict__ dst, int wave) const {
    uint32_t at = off;
    if (!EXACT && chunk >= dim - 8 * NW * I) at = kOutside;
    load_lds<false, 16 * NW * I>(p, bytes, at, dst + (wave + I * NW) * 1024);
  }
  // rows: what the sequence has from the tile's first row on.
  __device__ __forceinline__ void load(int rows, LAS unsigned char* __restrict__ dst, int wave) const {
    const int n = min(rows - 16 * (wave & 3), 16);
    const uint32_t bytes = n <= 0 || (!EXACT && tail <= 0) ? 0u : static_cast<uint32_t>((n - 1) * ts2 + tail);
    one<0>(bytes, dst, wave);
    if constexpr (N > 1) one<1>(bytes, dst, wave);
    if constexpr (N > 2) {
      one<2>(bytes, dst, wave);
      one<3>(bytes, dst, wave);
    }
  }
};

__device__ __forceinline__ bf16x8_t join4(bf16x4_t lo, bf16x4_t hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Lane addresses of the two fragment readers, in bytes within a tile.
//   row[e]: 16-byte read of row (lane & 31), chunk 2 e + (lane >> 5) of a block
//   tr[e]:  transposing read of rows 8 e + 4 (lane >> 5) + 0..3 of a block
struct FragOff {
  int row[2];
  int tr[2];
};
__device__ __forceinline__ FragOff frag_offsets(int lane) {
  FragOff f;
  const int r = lane & 31, h = lane >> 5;
  f.row[0] = r * 64 + swz(r, h) * 16;
  f.row[1] = r * 64 + swz(r, 2 + h) * 16;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int tr = 8 * e + 4 * h + ((lane & 15) >> 2);
    f.tr[e] = tr * 64 + swz(tr, 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) * 16 + (lane & 1) * 8;
  }
  return f;
}

// Left operand of a product over the head dimension: rows 32 b + 0..31 of a
// tile, k-step s.
template <int DP>
__device__ __forceinline__ bf16x8_t row_frag(const LAS unsigned char* __restrict__ t, const FragOff& f, int b, int s) {
  return *(const LAS bf16x8_t*)(t + f.row[s & 1] + (s >> 1) * Geo<DP>::SUBB + b * 2048);
}
// Left operand of a product over rows: columns 32 db + 0..31 of a tile,
// rows 16 t16 + 0..15 in the order of the results' registers.
template <int DP>
__device__ __forceinline__ bf16x8_t col_frag(const LAS unsigned char* __restrict__ t, const FragOff& f, int db,
                                             int t16) {
  const LAS unsigned char* p = t + db * Geo<DP>::SUBB + t16 * 1024;
  return join4(__builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)(p + f.tr[0])),
               __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)(p + f.tr[1])));
}

// Registers 8 s .. 8 s + 7 of a float32 result as a bf16 operand.
__device__ __forceinline__ bf16x8_t to_operand(const f32x16_t& x, int s) {
  uint4 u;
  u.x = pack_bf16(x[8 * s + 0], x[8 * s + 1]);
  u.y = pack_bf16(x[8 * s + 2], x[8 * s + 3]);
  u.z = pack_bf16(x[8 * s + 4], x[8 * s + 5]);
  u.w = pack_bf16(x[8 * s + 6], x[8 * s + 7]);
  bf16x8_t r;
  __builtin_memcpy(&r, &u, 16);
  return r;
}

__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Row index, within a 32-row block, of register r of a result.
__device__ __forceinline__ constexpr int res_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Between two tiles: this wave's loads have landed and its reads of the
// other buffer are behind it; past the barrier that holds for all waves.
__device__ __forceinline__ void next_tile() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) and lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// This wave's LDS accesses are behind it; past the barrier that holds for all
// waves.  Stores to memory go on.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// x of lane l and of lane l ^ 32, the lower lane's first.
__device__ __forceinline__ void halves(float x, float& lo, float& hi) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  lo = __uint_as_float(r[0]);
  hi = __uint_as_float(r[1]);
}
__device__ __forceinline__ float half_max(float x) {
  float a, b;
  halves(x, a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float half_sum(float x) {
  float a, b;
  halves(x, a, b);
  return a + b;
}

// Right operands of the rows that a wave owns, straight from global memory:
// row (lane & 31) of the wave's 32, all k-steps.  Rows at or past `rows` and
// chunks past the head dimension are zero.
template <int DP>
__device__ __forceinline__ void own_rows(const unsigned char* base, int64_t ts, int head_dim, int rows, int lane,
                                         bf16x8_t (&f)[Geo<DP>::KS]) {
  const int r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int s = 0; s < Geo<DP>::KS; ++s) {
    const int c = 2 * s + h;
    uint4 u = {0, 0, 0, 0};
    if (r < rows && c * 8 < head_dim) u = gld<uint4>(base + r * (ts * 2) + c * 16);
    __builtin_memcpy(&f[s], &u, 16);
  }
}

// Stores a transposed result (head dimension x rows) as bf16 rows: lane's
// row (lane & 31), four runs of four elements per block.
template <int DP>
__device__ __forceinline__ void store_rows(const HeadsView& v, int64_t row, int head, int head_dim, bool live, int lane,
                                           const f32x16_t (&acc)[Geo<DP>::DB], float mul) {
  if (!live) return;
  unsigned char* p = v.p + (row * v.ts + head * v.hs) * 2;
  const int h = lane >> 5;
#pragma unroll
  for (int db = 0; db < Geo<DP>::DB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * db + 8 * g + 4 * h;
      if (d < head_dim) {
        uint2 u;
        u.x = pack_bf16(acc[db][4 * g + 0] * mul, acc[db][4 * g + 1] * mul);
        u.y = pack_bf16(acc[db][4 * g + 2] * mul, acc[db][4 * g + 3] * mul);
        gst(p + d * 2, u);
      }
    }
}

// The same with 16 bytes a store: lanes l and l + 32, which hold the two halves
// of every 8 elements of a row, trade them, so that each has all of every other
// 8.  Half as many requests, which is what short work items wait for (16384
// tokens, window 64, 32/8 heads of 128: forward 127 us, with this 115).
template <int DP>
__device__ __forceinline__ void store_rows_wide(const HeadsView& v, int64_t row, int head, int head_dim, bool live, int lane,
                                                const f32x16_t (&acc)[Geo<DP>::DB], float mul) {
  unsigned char* p = v.p + (row * v.ts + head * v.hs) * 2;
  const int h = lane >> 5;
#pragma unroll
  for (int db = 0; db < Geo<DP>::DB; ++db)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      const f32x16_t& x = acc[db];
      const int i = 4 * g;
      const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(x[i] * mul, x[i + 1] * mul),
                                                      pack_bf16(x[i + 4] * mul, x[i + 5] * mul), false, false);
      const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(x[i + 2] * mul, x[i + 3] * mul),
                                                      pack_bf16(x[i + 6] * mul, x[i + 7] * mul), false, false);
      const int d = 32 * db + 8 * (g + h);
      if (live && d < head_dim) gst(p + d * 2, make_uint4(a[0], b[0], a[1], b[1]));
    }
}

// Running maximum of a float in memory, in any order of arrival with the
// same result: for values >= 0 the integer order of the bits is the float
// order, for negative ones the reverse.  NaN is passed as 0x7fffffff, which
// both orders keep; a NaN that the caller's array holds (of either sign) stays.
// The value only grows, so one that is seen to have it already (even an old
// one) needs no atomic.  Atomics on neighbouring floats follow one another, about
// 5 ns each: 4100 tokens in ten sequences, 25 heads of 64, from -infinity 43 us
// with one a wave and 33 with one a work-group, 26 where the maxima are there
// already or none are asked for; 64 x 64 tokens 44, 32 and 13.
__device__ __forceinline__ void atomic_max_float(float* p, float x) {
  const float old = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (x <= old || old != old) return;
  const int b = x != x ? 0x7fffffff : __float_as_int(x);
  if (b >= 0) atomicMax(reinterpret_cast<int*>(p), b);
  else atomicMin(reinterpret_cast<unsigned int*>(p), static_cast<unsigned int>(b));
}

// Work-groups of the kernels that own query rows (forward, dQ): 128 query rows
// of one head; key and value tiles of 64 rows stream through a double buffer
// in LDS.  4 waves of 32 rows, or (SPLIT = 2) 8 of them, wave w and w + 4 with
// the same rows and every other key tile, joined at the end: half the turns
// for the longest rows (see split_keys).
//
// With a window the tiles are those of the first tokens and, from the lowest
// key that a row of the work item sees through its window, those up to the
// diagonal; `jump` tiles between the two are passed over.
template <int DP, bool EXACT, int SPLIT, bool WIN>
struct KeyStream {
  using G = Geo<DP>;
  static constexpr int TURN = SPLIT * 2 * G::TILEB;  // bytes of a turn's tiles
  TileLoad<DP, EXACT, 4> kl, vl;
  int64_t kstep, vstep;
  int rows;    // what the sequence has from the next tile's first row on
  int fill;    // place of the next tile in LDS
  int tiles;             // of the work item
  int next_i, first_tiles, jump;  // WIN only: the next tile's number among them; see above
  __device__ __forceinline__ KeyStream(const AttnArgs& a, const AttnTile& t, int kv, int wave, int lane)
      : kl(a.k, t.row0 + static_cast<int64_t>(wave >> 2) * kAttnStep, kv, a.head_dim, wave & 3, lane),
        vl(a.v, t.row0 + static_cast<int64_t>(wave >> 2) * kAttnStep, kv, a.head_dim, wave & 3, lane) {
    kstep = static_cast<int64_t>(kl.ts2) * (SPLIT * kAttnStep);
    vstep = static_cast<int64_t>(vl.ts2) * (SPLIT * kAttnStep);
    rows = t.len - (wave >> 2) * kAttnStep;
    fill = (wave >> 2) * 2 * G::TILEB;
    tiles = (min(t.len, t.first + kAttnRows) + kAttnStep - 1) / kAttnStep;
    if (WIN) {
      next_i = wave >> 2;
      first_tiles = (a.sinks + kAttnStep - 1) / kAttnStep;
      jump = max(max(t.first - a.window + 1, 0) / kAttnStep - first_tiles, 0);
      tiles -= jump;
      if (next_i >= first_tiles) pass_over();
    }
  }
  __device__ __forceinline__ void pass_over() {
    kl.move(static_cast<int64_t>(kl.ts2) * (jump * kAttnStep));
    vl.move(static_cast<int64_t>(vl.ts2) * (jump * kAttnStep));
    rows -= jump * kAttnStep;
  }
  __device__ __forceinline__ int turns() const { return (tiles + SPLIT - 1) / SPLIT; }
  // First key of tile i of the work item's.
  __device__ __forceinline__ int key_of(int i) const { return (WIN && i >= first_tiles ? i + jump : i) * kAttnStep; }
  // Starts the loads of this wave's share of the next turn's tiles.
  __device__ __forceinline__ void next(LAS unsigned char* lds, int wave) {
    kl.load(rows, lds + fill, wave & 3);
    vl.load(rows, lds + fill + G::TILEB, wave & 3);
    kl.move(kstep);
    vl.move(vstep);
    rows -= SPLIT * kAttnStep;
    if (WIN) {
      next_i += SPLIT;
      if (next_i >= first_tiles && next_i - SPLIT < first_tiles) pass_over();
    }
    fill ^= TURN;
  }
};

// Whether no row of a wave's 32 from wq0 on sees one of the n keys from k0 on.
template <bool WIN>
__device__ __forceinline__ bool keys_hidden(const AttnArgs& a, int wq0, int k0, int n) {
  return k0 > wq0 + 31 || (WIN && wq0 - (k0 + n - 1) >= a.window && k0 >= a.sinks);
}
// -infinity in place of the scores of keys k0 + res_row(r), of 32 from k0 on,
// that row q of a wave's 32 from wq0 on does not see (windowed calls): each
// border that the block holds costs a comparison an element.
__device__ __forceinline__ void hide_keys(const AttnArgs& a, int wq0, int q, int k0, int h, f32x16_t& s) {
  const int at = q - k0 - 4 * h;  // the row itself, as res_row(r, 0) counts keys
  if (k0 + 31 > wq0) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (res_row(r, 0) > at) s[r] = -kInf;
  }
  if (wq0 + 31 - k0 >= a.window) {
    const int low = at - a.window;  // the last key behind its window
    if (k0 >= a.sinks) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (res_row(r, 0) <= low) s[r] = -kInf;
    } else {
      const int first = a.sinks - k0 - 4 * h;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (res_row(r, 0) <= low && res_row(r, 0) >= first) s[r] = -kInf;
    }
  }
}

// Hands a wave's accumulators over through LDS, 1 KB per four registers.
template <int DP>
__device__ __forceinline__ void put_acc(LAS unsigned char* __restrict__ p, const f32x16_t (&acc)[Geo<DP>::DB]) {
#pragma unroll
  for (int i = 0; i < Geo<DP>::DB * 4; ++i) {
    const f32x16_t& x = acc[i >> 2];
    const int g = 4 * (i & 3);
    *(LAS f32x4_t*)(p + i * 1024) = (f32x4_t){x[g], x[g + 1], x[g + 2], x[g + 3]};
  }
}
// acc = acc * mine + theirs * other
template <int DP>
__device__ __forceinline__ void join_acc(const LAS unsigned char* __restrict__ p, f32x16_t (&acc)[Geo<DP>::DB], float mine,
                                         float other) {
#pragma unroll
  for (int i = 0; i < Geo<DP>::DB * 4; ++i) {
    const f32x4_t o = *(const LAS f32x4_t*)(p + i * 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i >> 2][4 * (i & 3) + k] = fmaf(o[k], other, acc[i >> 2][4 * (i & 3) + k] * mine);
  }
}

// ------------------------------------------------------------------ forward
// A wave reads every fragment of a tile for its 32 rows, so with heads of 128
// the LDS (at 128 bytes a cycle) works as long as the matrix cores; 32 rows leave
// room for two work-groups to a unit (four with heads of 64), whose waves
// share a SIMD without a common barrier: one's exponentials run under the
// other's products.
// 8192 tokens, 32 heads of 128 over 8 key heads: 522 us, 1.05 PFLOP/s, the
// matrix cores 55% busy at the 1.9 GHz that the card holds under this load.
// 4100 tokens in ten sequences, 25 heads of 64: 26 us, the matrix cores 29%
// busy (with heads of 64 the exponentials and what goes with them take about
// twice the products' cycles); the longest sequence's 21 turns, about 1 us
// each among the others', end last.  With max_logit from -infinity 33 us (see
// atomic_max_float).
// With a window of 1024 and 4 first tokens: 16384 tokens, 32 heads of 128 over 8,
// 350 us (traced, once the card's clocks have settled; 8192^3 products ran at 1.19
// PFLOP/s on it), the matrix cores 44% busy (19 tiles visited for 16 that are seen, and an
// item's start and end come every 19 turns); the 4100 tokens, window 256, 22 us.
template <int DP, bool EXACT, int SPLIT, bool WIN>
__global__ __launch_bounds__(256 * SPLIT, DP == 64 ? 4 : 2) void attention_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  using KS = KeyStream<DP, EXACT, SPLIT, WIN>;
  static_assert(SPLIT == 1 || 2 * KS::TURN >= 4 * (G::DB * 4096 + 1024), "the join fits the buffer");
  __shared__ __align__(1024) unsigned char smem[2 * KS::TURN];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave >> 2;
  const int hx = blockIdx.x % a.heads;
  const AttnTile t = a.by_query[blockIdx.x / a.heads];
  const int kv = hx % a.kv_heads;
  const int head = kv * (a.heads / a.kv_heads) + hx / a.kv_heads;
  const int wq0 = t.first + 32 * (wave & 3);   // the wave's first query row in its sequence
  const int q = wq0 + (lane & 31);
  const float c = a.scale * kAttnLog2e;
  const float slack = kSlackLog2 / c;

  KS stream(a, t, kv, wave, lane);
  const int turns = stream.turns();
  const FragOff fo = frag_offsets(lane);
  stream.next(lds, wave);
  bf16x8_t qf[G::KS];
  own_rows<DP>(a.q.p + ((static_cast<int64_t>(t.row0) + wq0) * a.q.ts + head * a.q.hs) * 2, a.q.ts, a.head_dim, t.len - wq0,
               lane, qf);

  f32x16_t o[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) o[db] = (f32x16_t)(0.f);
  float m_top = -kInf, m_ref = -kInf, l = 0.f;  // l: this lane's half of the keys
  for (int it = 0; it < turns; ++it) {
    const int k0 = stream.key_of(it * SPLIT + part), cur = stream.fill ^ KS::TURN;
    next_tile();
    if (it + 1 < turns) stream.next(lds, wave);
    if (keys_hidden<WIN>(a, wq0, k0, kAttnStep) || wq0 >= t.len) continue;  // no key for the wave's rows, or it has none
    const LAS unsigned char* kt_lds = lds + cur;
    const LAS unsigned char* vt_lds = kt_lds + G::TILEB;
    f32x16_t s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      s[b] = (f32x16_t)(0.f);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) s[b] = mfma(row_frag<DP>(kt_lds, fo, b, st), qf[st], s[b]);
    }
    if constexpr (WIN) {
#pragma unroll
      for (int b = 0; b < 2; ++b) hide_keys(a, wq0, q, k0 + 32 * b, h, s[b]);
    } else if (k0 + kAttnStep - 1 > wq0) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (k0 + 32 * b + res_row(r, h) > q) s[b][r] = -kInf;
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
    m_top = fmaxf(m_top, half_max(top));
    if (__any(m_top > m_ref + slack)) {
      const float alpha = m_top == m_ref ? 1.f : __builtin_amdgcn_exp2f((m_ref - m_top) * c);
      m_ref = m_top;
      l *= alpha;
#pragma unroll
      for (int db = 0; db < G::DB; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[db][r] *= alpha;
    }
    const float ref = m_ref == -kInf ? 0.f : m_ref * c;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], c, -ref));
        l += s[b][r];
      }
#pragma unroll
    for (int t16 = 0; t16 < 4; ++t16) {
      const bf16x8_t p = to_operand(s[t16 >> 1], t16 & 1);
#pragma unroll
      for (int db = 0; db < G::DB; ++db) o[db] = mfma(col_frag<DP>(vt_lds, fo, db, t16), p, o[db]);
    }
  }
  l = half_sum(l);
  float ref = m_ref == -kInf ? 0.f : m_ref * c;  // as the exponentials had it
  if constexpr (SPLIT == 2) {
    // The second half's sums, reference and largest logit, brought to a
    // common reference.
    LAS unsigned char* at = lds + (wave & 3) * (G::DB * 4096 + 1024) + lane * 16;
    next_tile();
    if (part == 1) {
      put_acc<DP>(at, o);
      *(LAS f32x4_t*)(at + G::DB * 4096) = (f32x4_t){m_ref, m_top, l, 0.f};
    }
    next_tile();
    if (part == 1) {
      if (a.max_logit) {  // the barriers that the other waves come to below
        lds_barrier();
        lds_barrier();
      }
      return;
    }
    const f32x4_t x = *(const LAS f32x4_t*)(at + G::DB * 4096);
    const float m = fmaxf(m_ref, x[0]), common = m == -kInf ? 0.f : m * c;
    // without a reference the sums are zero (or NaN): as they are
    const float mine = m_ref == -kInf ? 1.f : __builtin_amdgcn_exp2f(ref - common);
    const float other = x[0] == -kInf ? 1.f : __builtin_amdgcn_exp2f(x[0] * c - common);
    join_acc<DP>(at, o, mine, other);
    l = fmaf(x[2], other, l * mine);
    m_top = fmaxf(m_top, x[1]);
    ref = common;
  }
  const bool live = q < t.len;
  if constexpr (WIN) store_rows_wide<DP>(a.o, static_cast<int64_t>(t.row0) + q, head, a.head_dim, live, lane, o, 1.f / l);
  else store_rows<DP>(a.o, static_cast<int64_t>(t.row0) + q, head, a.head_dim, live, lane, o, 1.f / l);
  if (live && h == 0) gst(a.lse + head * a.lse_stride + t.row0 + q, (ref + __builtin_amdgcn_logf(l)) * kLn2);
  if (a.max_logit) {
    // A row whose sum is NaN has an infinite logit, or else a NaN.
    float top = !live ? -kInf : l != l && m_top < kInf ? __builtin_nanf("") : m_top * a.scale;
#pragma unroll
    for (int off = 1; off <= 16; off <<= 1) {
      const float other = __shfl_xor(top, off, 64);
      top = top != top || other != other ? __builtin_nanf("") : fmaxf(top, other);
    }
    // one atomic for the work-group (rows past the sequence hold -infinity)
    lds_barrier();
    if (lane == 0) *(LAS float*)(lds + 4 * wave) = top;
    lds_barrier();
    if (threadIdx.x == 0) {
      const f32x4_t x = *(const LAS f32x4_t*)lds;
#pragma unroll
      for (int w = 1; w < 4; ++w) top = top != top || x[w] != x[w] ? __builtin_nanf("") : fmaxf(top, x[w]);
      if (WIN && a.tops) gst(a.tops + static_cast<int64_t>(head) * a.n_tiles + blockIdx.x / a.heads, top);
      else atomic_max_float(a.max_logit + head / a.logit_group, top);
    }
  }
}

// ------------------------------------------------------------ backward: dQ
// As in the forward pass, and bound by the same.  Also forms delta and leaves
// it, with lse in base 2, for the dK/dV kernel that follows.  Scores and their gradients are formed again here rather than
// passed on: dQ summed by atomics from the dK/dV kernel would save 2 of the 7
// products of the two kernels, but with an order that changes from run to
// run.  8192 tokens, 32 heads of 128: 680 us, 1.21 PFLOP/s, matrix cores 65%
// busy (with one wave a SIMD, 1240 us).  With the window above 451 us, 49% busy.
template <int DP, bool EXACT, int SPLIT, bool WIN>
__global__ __launch_bounds__(256 * SPLIT, DP == 64 && SPLIT == 1 ? 4 : 2) void attention_dq_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  using KS = KeyStream<DP, EXACT, SPLIT, WIN>;
  __shared__ __align__(1024) unsigned char smem[2 * KS::TURN];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave >> 2;
  const int hx = blockIdx.x % a.heads;
  const AttnTile t = a.by_query[blockIdx.x / a.heads];
  const int kv = hx % a.kv_heads;
  const int head = kv * (a.heads / a.kv_heads) + hx / a.kv_heads;
  const int wq0 = t.first + 32 * (wave & 3);
  const int q = wq0 + (lane & 31);
  const bool live = q < t.len;
  const int64_t row = static_cast<int64_t>(t.row0) + q;
  const float c = a.scale * kAttnLog2e;

  KS stream(a, t, kv, wave, lane);
  const int turns = stream.turns();
  const FragOff fo = frag_offsets(lane);
  stream.next(lds, wave);
  const int64_t row0 = static_cast<int64_t>(t.row0) + wq0;
  bf16x8_t qf[G::KS], gf[G::KS];
  own_rows<DP>(a.q.p + (row0 * a.q.ts + head * a.q.hs) * 2, a.q.ts, a.head_dim, t.len - wq0, lane, qf);
  own_rows<DP>(a.d_o.p + (row0 * a.d_o.ts + head * a.d_o.hs) * 2, a.d_o.ts, a.head_dim, t.len - wq0, lane, gf);
  float delta = 0.f;
  {
    bf16x8_t of[G::KS];
    own_rows<DP>(a.o.p + (row0 * a.o.ts + head * a.o.hs) * 2, a.o.ts, a.head_dim, t.len - wq0, lane, of);
#pragma unroll
    for (int s = 0; s < G::KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = fmaf(static_cast<float>(gf[s][e]), static_cast<float>(of[s][e]), delta);
    delta = half_sum(delta);
  }
  const float lse2 = live ? gld<float>(a.lse + head * a.lse_stride + row) * kAttnLog2e : 0.f;
  if (live && h == 0 && part == 0) {
    gst(a.row_lse2 + head * a.row_stride + row, lse2);
    gst(a.row_delta + head * a.row_stride + row, delta);
  }

  f32x16_t dq[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) dq[db] = (f32x16_t)(0.f);
  for (int it = 0; it < turns; ++it) {
    const int k0 = stream.key_of(it * SPLIT + part), cur = stream.fill ^ KS::TURN;
    next_tile();
    if (it + 1 < turns) stream.next(lds, wave);
    if (keys_hidden<WIN>(a, wq0, k0, kAttnStep) || wq0 >= t.len) continue;
    const LAS unsigned char* kt_lds = lds + cur;
    const LAS unsigned char* vt_lds = kt_lds + G::TILEB;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (WIN && keys_hidden<WIN>(a, wq0, k0 + 32 * b, 32)) continue;
      f32x16_t s = (f32x16_t)(0.f), dp = (f32x16_t)(0.f);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) s = mfma(row_frag<DP>(kt_lds, fo, b, st), qf[st], s);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) dp = mfma(row_frag<DP>(vt_lds, fo, b, st), gf[st], dp);
      if constexpr (WIN) {
        hide_keys(a, wq0, q, k0 + 32 * b, h, s);
      } else if (k0 + 32 * b + 31 > wq0) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (k0 + 32 * b + res_row(r, h) > q) s[r] = -kInf;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
#pragma unroll
      for (int s16 = 0; s16 < 2; ++s16) {
        const bf16x8_t ds = to_operand(s, s16);
#pragma unroll
        for (int db = 0; db < G::DB; ++db) dq[db] = mfma(col_frag<DP>(kt_lds, fo, db, 2 * b + s16), ds, dq[db]);
      }
    }
  }
  if constexpr (SPLIT == 2) {
    LAS unsigned char* at = lds + (wave & 3) * (G::DB * 4096) + lane * 16;
    next_tile();
    if (part == 1) put_acc<DP>(at, dq);
    next_tile();
    if (part == 1) return;
    join_acc<DP>(at, dq, 1.f, 1.f);
  }
  if constexpr (WIN) store_rows_wide<DP>(a.dq, row, head, a.head_dim, live, lane, dq, a.scale);
  else store_rows<DP>(a.dq, row, head, a.head_dim, live, lane, dq, a.scale);
}

// -------------------------------------------------------- backward: dK, dV
// One work-group: 128 key rows of one key head; the query and
// upstream-gradient tiles of every query head of the group stream past, so
// that the sums over rows and heads stay in registers, in a fixed order.
//
// 8 waves, two per SIMD.  Waves w and w + 4 hold the same 32 keys: each forms
// p and ds of one half of a 64-row tile, then wave w sums dV over both halves
// and wave w + 4 sums dK; what the other needs (ds of the first half, p of
// the second) goes through LDS, 2 KB each way.  With half of the sums a wave
// has registers to run ahead: in turn k it forms the scores of tile k, and
// its exponentials run under the products of tile k - 1.  Three tiles in LDS:
// k - 1 and k in use, k + 1 on its way.  8192 tokens, 32 heads of 128 over 8
// key heads: 980 us, 1.12 PFLOP/s, matrix cores 54% busy, the LDS (at 128
// bytes a cycle) about as long.  (4 waves of 512 registers that keep both sums 1300 us; 8 waves that
// each keep both sums, starved of registers for reads ahead, 1180 us.)
template <int DP>
struct DkvLds {
  static constexpr int ROWS = 2 * Geo<DP>::TILEB;    // q and dO tiles, then lse and delta
  static constexpr int STAGE = ROWS + 2 * kAttnStep * 4;
  static constexpr int MSG = 3 * STAGE;              // two turns of 8 waves' messages
  static constexpr int BYTES = MSG + 2 * 8 * 2048;
};

// Where the far kernel's sums of chunk `slot` and key head kv lie: dK and dV
// of the first tokens, 2 x sinks x head_dim.
__device__ __forceinline__ float* far_sum(const AttnArgs& a, int slot, int kv) {
  return a.far + (static_cast<int64_t>(slot) * a.kv_heads + kv) * (2 * a.sinks * a.head_dim);
}

// Where a share of a key tile's sums lies: dK (which = 0) or dV (1), kAttnRows x head_dim.
__device__ __forceinline__ float* part_sum(const AttnArgs& a, int tile, int kv, int part, int which) {
  const int64_t i = ((static_cast<int64_t>(tile) * a.kv_heads + kv) * a.key_parts + part) * 2 + which;
  return a.parts + i * (kAttnRows * a.head_dim);
}

// Four consecutive per-row values of a tile.
__device__ __forceinline__ f32x4_t row_values(const LAS unsigned char* __restrict__ p) { return *(const LAS f32x4_t*)p; }

// s = Q K^T and dp = dO V^T of row block b of a tile with the wave's keys.
template <int DP>
__device__ __forceinline__ void dkv_scores(const LAS unsigned char* __restrict__ tile, const FragOff& fo, int b,
                                           const bf16x8_t (&kf)[Geo<DP>::KS], const bf16x8_t (&vf)[Geo<DP>::KS],
                                           f32x16_t& s, f32x16_t& dp) {
  s = dp = (f32x16_t)(0.f);
#pragma unroll
  for (int st = 0; st < Geo<DP>::KS; ++st) s = mfma(row_frag<DP>(tile, fo, b, st), kf[st], s);
#pragma unroll
  for (int st = 0; st < Geo<DP>::KS; ++st) dp = mfma(row_frag<DP>(tile + Geo<DP>::TILEB, fo, b, st), vf[st], dp);
}

// p in place of s and ds in place of dp.
template <int DP>
__device__ __forceinline__ void dkv_softmax(const LAS unsigned char* __restrict__ tile, int b, int h, float c,
                                            f32x16_t& s, f32x16_t& dp) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const f32x4_t lse2 = row_values(tile + DkvLds<DP>::ROWS + (32 * b + 8 * g + 4 * h) * 4);
    const f32x4_t delta = row_values(tile + DkvLds<DP>::ROWS + (kAttnStep + 32 * b + 8 * g + 4 * h) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * g + i;
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2[i]));
      dp[r] = s[r] * (dp[r] - delta[i]);
    }
  }
}

// acc += (rows of block b of a tile)^T x, x two operands of 16 rows.
template <int DP>
__device__ __forceinline__ void dkv_sums(const LAS unsigned char* __restrict__ tile, const FragOff& fo, int b,
                                         const bf16x8_t (&x)[2], f32x16_t (&acc)[Geo<DP>::DB]) {
#pragma unroll
  for (int s16 = 0; s16 < 2; ++s16)
#pragma unroll
    for (int db = 0; db < Geo<DP>::DB; ++db) acc[db] = mfma(col_frag<DP>(tile, fo, db, 2 * b + s16), x[s16], acc[db]);
}

__device__ __forceinline__ void read_msg(const LAS unsigned char* __restrict__ p, bf16x8_t (&x)[2]) {
  x[0] = *(const LAS bf16x8_t*)p;
  x[1] = *(const LAS bf16x8_t*)(p + 1024);
}
__device__ __forceinline__ void write_msg(LAS unsigned char* __restrict__ p, const bf16x8_t (&x)[2]) {
  *(LAS bf16x8_t*)p = x[0];
  *(LAS bf16x8_t*)(p + 1024) = x[1];
}

// The lane number, computed where it is written (two instructions) instead of
// kept in a register: a kernel without one to spare would reload what depends
// on it from scratch memory, and wait there for the tile loads under way too
// (4100 tokens, 25 heads of 64: dK/dV 53 us, 46 without that).
__device__ __forceinline__ int fresh_lane() {
  int l = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
#endif
  return l;
}

// Query tiles of a key tile: from the diagonal to the last row that sees one of its keys (through its window).
template <bool WIN>
__device__ __forceinline__ int query_tiles(const AttnArgs& a, const AttnTile& t) {
  const int rows = t.len - t.first;
  return ((WIN ? min(rows, kAttnRows - 1 + a.window) : rows) + kAttnStep - 1) / kAttnStep;
}
// -infinity in place of the scores of rows q0 + res_row(r) whose windows begin behind the key.
__device__ __forceinline__ void hide_rows(const AttnArgs& a, int q0, int key, int h, f32x16_t& s) {
  const int last = key + a.window - 1 - q0 - 4 * h;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (res_row(r, 0) > last) s[r] = -kInf;
}

// The tiles that stream past a key tile: from the sequence's last rows back to
// the diagonal, every query head of the group in turn, so that work-groups of
// one key head read the same tiles at about the same time.
//
// With a window, key tiles next to each other want overlapping ranges of
// rows.  They all start where the row tile's number is the same modulo the
// range's tiles and wrap round at its end, so that work-groups that run
// together read the same tiles at about the same time (16384 tokens, window
// 1024, 32 heads of 128 over 8 key heads: dK/dV 622 us, 642 without, and dQ
// in front of it 451 and 460).
template <int DP, bool EXACT, int NW, bool WIN>
struct QueryStream {
  using L = DkvLds<DP>;
  TileLoad<DP, EXACT, NW> ql, gl;
  const float* stat;           // this wave's statistic: lse (wave 0) or delta (wave 1)
  int64_t stat_stride;
  int64_t q_head, q_back, g_head, g_back;  // bytes to the next head; from the last head to the first, a tile back
  int row, head, group;        // first row and head of the next tile
  int wrap;                    // WIN only: rows from the range's first tile to behind its last
  int fill;                    // its place in LDS
  // Number, in the range, of the tile to start with.
  static __device__ __forceinline__ int start(const AttnArgs& a, const AttnTile& t, int nq) {
    if (!WIN) return nq - 1;
    const int range = (kAttnRows - 1 + a.window + kAttnStep - 1) / kAttnStep;
    return min(range - 1 - t.first / kAttnStep % range, nq - 1);
  }
  // `count` query heads from head0 on.
  __device__ __forceinline__ QueryStream(const AttnArgs& a, const AttnTile& t, int head0, int count, int nq, int wave, int lane)
      : ql(a.q, t.row0 + static_cast<int64_t>(t.first) + start(a, t, nq) * kAttnStep, head0, a.head_dim, wave, lane),
        gl(a.d_o, t.row0 + static_cast<int64_t>(t.first) + start(a, t, nq) * kAttnStep, head0, a.head_dim, wave, lane) {
    group = count;
    row = t.first + start(a, t, nq) * kAttnStep;
    if (WIN) wrap = nq * kAttnStep;
    head = fill = 0;
    stat = (wave == 0 ? a.row_lse2 : a.row_delta) + head0 * a.row_stride + t.row0 + row;
    stat_stride = a.row_stride;
    q_head = a.q.hs * 2;
    g_head = a.d_o.hs * 2;
    q_back = -((group - 1) * a.q.hs + kAttnStep * a.q.ts) * 2;
    g_back = -((group - 1) * a.d_o.hs + kAttnStep * a.d_o.ts) * 2;
  }
  // Starts this wave's loads of the next of RING tiles; `first`: the range's first row.
  template <int RING>
  __device__ __forceinline__ void next(int len, int first, LAS unsigned char* lds, int wave) {
    LAS unsigned char* dst = lds + fill;
    ql.load(len - row, dst, wave);
    gl.load(len - row, dst + Geo<DP>::TILEB, wave);
    if (wave < 2)
      load_lds<true, 0>(reinterpret_cast<const unsigned char*>(stat), 4u * min(len - row, kAttnStep), fresh_lane() * 4,
                        dst + L::ROWS + wave * kAttnStep * 4);
    fill = fill == (RING - 1) * L::STAGE ? 0 : fill + L::STAGE;
    if (++head == group) {
      head = 0;
      row -= kAttnStep;
      ql.move(q_back);
      gl.move(g_back);
      stat -= (group - 1) * stat_stride + kAttnStep;
      if (WIN && row < first) {
        row += wrap;
        ql.move(static_cast<int64_t>(ql.ts2) * wrap);
        gl.move(static_cast<int64_t>(gl.ts2) * wrap);
        stat += wrap;
      }
    } else {
      ql.move(q_head);
      gl.move(g_head);
      stat += stat_stride;
    }
  }
};

// What rows beyond their windows give the first tokens' dK (which = 0) or dV
// (1): the far kernel's sums of the sequence's chunks, in order (or in the
// first of them, joined).
template <int DP>
__device__ __forceinline__ void add_far(const AttnArgs& a, const AttnTile& t, int kv, int key, int which, int h,
                                        f32x16_t (&acc)[Geo<DP>::DB]) {
  if (!a.far || key >= a.sinks || t.len <= a.window) return;
  const int first = a.window / kFarRows, end = a.far_joined ? first + 1 : (t.len + kFarRows - 1) / kFarRows;
  for (int c = first; c < end; ++c) {
    const float* p = far_sum(a, t.chunk + c, kv) + (which * a.sinks + key) * a.head_dim;
#pragma unroll
    for (int db = 0; db < Geo<DP>::DB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = 32 * db + 8 * g + 4 * h;
        if (d >= a.head_dim) continue;
        const f32x4_t x = gld<f32x4_t>(p + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[db][4 * g + i] += x[i];
      }
  }
}

template <int DP, bool EXACT, bool WIN>
__global__ __launch_bounds__(512, 2) void attention_dkv_pair_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  using L = DkvLds<DP>;
  __shared__ __align__(1024) unsigned char smem[L::BYTES];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // With a window a key tile's query heads may be shared out over several work-groups.
  const int items = WIN ? a.kv_heads * a.key_parts : a.kv_heads, item = blockIdx.x % items;
  const int kv = WIN ? item % a.kv_heads : item, part = WIN ? item / a.kv_heads : 0;
  const AttnTile t = a.by_key[blockIdx.x / items];
  int head0 = kv * (a.heads / a.kv_heads), group = a.heads / a.kv_heads;
  if (WIN) {
    const int from = part * group / a.key_parts, to = (part + 1) * group / a.key_parts;
    head0 += from;
    group = to - from;
  }
  const int nq = query_tiles<WIN>(a, t);
  const int total = nq * group;
  const int wk0 = t.first + 32 * (wave & 3), half = wave >> 2;
  const int key = wk0 + (lane & 31);
  const float c = a.scale * kAttnLog2e;

  const FragOff fo = frag_offsets(lane);
  QueryStream<DP, EXACT, 8, WIN> stream(a, t, head0, group, nq, wave, lane);
  const int64_t krow0 = static_cast<int64_t>(t.row0) + wk0;
  bf16x8_t kf[G::KS], vf[G::KS];
  own_rows<DP>(a.k.p + (krow0 * a.k.ts + kv * a.k.hs) * 2, a.k.ts, a.head_dim, t.len - wk0, lane, kf);
  own_rows<DP>(a.v.p + (krow0 * a.v.ts + kv * a.v.hs) * 2, a.v.ts, a.head_dim, t.len - wk0, lane, vf);
  f32x16_t acc[G::DB];  // dV (first half of the waves) or dK
#pragma unroll
  for (int db = 0; db < G::DB; ++db) acc[db] = (f32x16_t)(0.f);
  bf16x8_t own[2];
  f32x16_t s, dp;
  const int sum_of = half == 0 ? G::TILEB : 0;  // what the wave sums of a tile: dO or q
  int cur = 0, turn = 0;  // the tile's place; 0 or 8 * 2048, where this turn's messages go
  const int out = L::MSG + wave * 2048 + lane * 16, in = L::MSG + (wave ^ 4) * 2048 + lane * 16;
  int qs = stream.row + 32 * half, head = 0;  // the wave's first row of the tile
  auto mask = [&]() {
    if (qs < wk0 + 31 || qs + 31 >= t.len) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (key > qs + res_row(r, h) || qs + res_row(r, h) >= t.len) s[r] = -kInf;
    }
    if (WIN && qs + 31 - wk0 >= a.window) hide_rows(a, qs, key, h, s);
    if (++head == group) {
      head = 0;
      qs -= kAttnStep;
      if (WIN && qs < t.first) qs += stream.wrap;
    }
  };
  auto pass_on = [&]() {
    const bf16x8_t p[2] = {to_operand(s, 0), to_operand(s, 1)}, ds[2] = {to_operand(dp, 0), to_operand(dp, 1)};
#pragma unroll
    for (int i = 0; i < 2; ++i) own[i] = half == 0 ? p[i] : ds[i];
    const bf16x8_t other[2] = {half == 0 ? ds[0] : p[0], half == 0 ? ds[1] : p[1]};
    write_msg(lds + out + turn, other);
  };
  stream.template next<3>(t.len, t.first, lds, wave);
  next_tile();
  if (total > 1) stream.template next<3>(t.len, t.first, lds, wave);
  dkv_scores<DP>(lds + cur, fo, half, kf, vf, s, dp);
  mask();
  dkv_softmax<DP>(lds + cur, half, h, c, s, dp);
  pass_on();
  for (int it = 1; it < total; ++it) {
    next_tile();  // tile `it` and the messages of turn it - 1 are there, tile it - 2 is done with
    if (it + 1 < total) stream.template next<3>(t.len, t.first, lds, wave);
    const int prev = cur + sum_of;
    cur = cur == 2 * L::STAGE ? 0 : cur + L::STAGE;
    turn ^= 8 * 2048;
    dkv_scores<DP>(lds + cur, fo, half, kf, vf, s, dp);
    mask();
    bf16x8_t other[2];
    read_msg(lds + in + (turn ^ (8 * 2048)), other);
    dkv_sums<DP>(lds + prev, fo, half, own, acc);
    dkv_softmax<DP>(lds + cur, half, h, c, s, dp);
    dkv_sums<DP>(lds + prev, fo, half ^ 1, other, acc);
    pass_on();
  }
  next_tile();
  {
    bf16x8_t other[2];
    read_msg(lds + in + turn, other);
    dkv_sums<DP>(lds + cur + sum_of, fo, half, own, acc);
    dkv_sums<DP>(lds + cur + sum_of, fo, half ^ 1, other, acc);
  }
  if (WIN && a.key_parts > 1) {
    if (key >= t.len) return;
    float* p = part_sum(a, blockIdx.x / items, kv, part, half == 0 ? 1 : 0) + (key - t.first) * a.head_dim;
#pragma unroll
    for (int db = 0; db < G::DB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = 32 * db + 8 * g + 4 * h;
        const f32x16_t& x = acc[db];
        if (d < a.head_dim) gst(p + d, (f32x4_t){x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]});
      }
    return;
  }
  if (WIN) add_far<DP>(a, t, kv, key, half == 0 ? 1 : 0, h, acc);
  const int64_t row = static_cast<int64_t>(t.row0) + key;
  store_rows<DP>(half == 0 ? a.dv : a.dk, row, kv, a.head_dim, key < t.len, lane, acc, half == 0 ? 1.f : a.scale);
}

// The same for head dimensions up to 64 and many key tiles: 4 waves of 32 keys
// that each take all rows of a tile and both sums, in 168 registers (one value
// that only the stores need waits in scratch memory over the loop), and two tiles in LDS, so that three work-groups share a unit (the pair
// kernel's 83 KB leave room for one, whose start and end, about 6 us, lie
// open).
template <int DP, bool EXACT, bool WIN>
__global__ __launch_bounds__(256, 3) void attention_dkv_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  using L = DkvLds<DP>;
  __shared__ __align__(1024) unsigned char smem[2 * L::STAGE];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kv = blockIdx.x % a.kv_heads;
  const AttnTile t = a.by_key[blockIdx.x / a.kv_heads];
  const int nq = query_tiles<WIN>(a, t);
  const int total = nq * (a.heads / a.kv_heads);
  const int wk0 = t.first + 32 * wave;
  const int key = wk0 + (lane & 31);
  const float c = a.scale * kAttnLog2e;
  const FragOff fo = frag_offsets(lane);
  QueryStream<DP, EXACT, 4, WIN> stream(a, t, kv * (a.heads / a.kv_heads), a.heads / a.kv_heads, nq, wave, lane);
  int q0 = stream.row, head = 0, cur = 0;
  stream.template next<2>(t.len, t.first, lds, wave);
  const int64_t krow0 = static_cast<int64_t>(t.row0) + wk0;
  bf16x8_t kf[G::KS], vf[G::KS];
  own_rows<DP>(a.k.p + (krow0 * a.k.ts + kv * a.k.hs) * 2, a.k.ts, a.head_dim, t.len - wk0, lane, kf);
  own_rows<DP>(a.v.p + (krow0 * a.v.ts + kv * a.v.hs) * 2, a.v.ts, a.head_dim, t.len - wk0, lane, vf);
  f32x16_t dk[G::DB], dv[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) dk[db] = dv[db] = (f32x16_t)(0.f);
  for (int it = 0; it < total; ++it) {
    next_tile();
    if (it + 1 < total) stream.template next<2>(t.len, t.first, lds, wave);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int qs = q0 + 32 * b;
      // no query of the block sees a key of the wave
      if (qs + 31 < wk0 || qs >= t.len || wk0 >= t.len || (WIN && qs - (wk0 + 31) >= a.window)) continue;
      f32x16_t s, dp;
      dkv_scores<DP>(lds + cur, fo, b, kf, vf, s, dp);
      if (qs < wk0 + 31 || qs + 31 >= t.len) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (key > qs + res_row(r, h) || qs + res_row(r, h) >= t.len) s[r] = -kInf;
      }
      if (WIN && qs + 31 - wk0 >= a.window) hide_rows(a, qs, key, h, s);
      dkv_softmax<DP>(lds + cur, b, h, c, s, dp);
      const bf16x8_t p[2] = {to_operand(s, 0), to_operand(s, 1)}, ds[2] = {to_operand(dp, 0), to_operand(dp, 1)};
      dkv_sums<DP>(lds + cur + G::TILEB, fo, b, p, dv);
      dkv_sums<DP>(lds + cur, fo, b, ds, dk);
    }
    cur = L::STAGE - cur;
    if (++head == stream.group) {
      head = 0;
      q0 -= kAttnStep;
      if (WIN && q0 < t.first) q0 += stream.wrap;
    }
  }
  if (WIN) {
    add_far<DP>(a, t, kv, key, 0, h, dk);
    add_far<DP>(a, t, kv, key, 1, h, dv);
  }
  const int64_t row = static_cast<int64_t>(t.row0) + key;
  store_rows<DP>(a.dk, row, kv, a.head_dim, key < t.len, lane, dk, a.scale);
  store_rows<DP>(a.dv, row, kv, a.head_dim, key < t.len, lane, dv, 1.f);
}

}  // namespace

namespace {

// Whether rows are split over two wave groups: with up to two work-groups of
// either kind to a unit, the longest sequence's turns are the call's time and
// half of them pay for the join; shorter sequences and fuller cards lose by
// it.  Forward / whole backward pass in us, whole | split: 4096 tokens, 12
// heads of 64 (384 work-groups) 56 / 155 | 46 / 132, 16 of 128 (512) 92 / 272
// | 85 / 269; 1290 tokens, 25 of 64 (275) 20.8 / 59 | 19.3 / 55; 4 x 1024
// tokens, 16 of 128 (512) 30 / 94 | 34 / 102; 4096 tokens, 25 of 64 (800)
// 75 / 241 | 72 / 251.
// Windowed calls have as few turns as the window (a.longest) and end more
// evenly: the forward pass gains up to 512 work-groups with heads of 64 (4096
// tokens, 12 heads, window 1024: 28.5 | 25.9; window 512: 21.3 | 22.3; 8192, 8
// heads, window 1024: 28.2 | 26.8) and 256 with heads of 128 (2048, 16 heads,
// window 1024: 28.2 | 23.1; 4096, 16/4 heads, 512 of them: 42.7 | 47.6), the
// backward pass up to about 300 (1290, 25 of 64: 51.9 | 48.9; 4096, 12 of 64:
// 89 | 92).
template <int DP, bool WIN>
bool split_keys(const AttnArgs& a, bool back) {
  const int64_t most = !WIN ? 512 : back ? 320 : DP == 64 ? 512 : 256;
  return int64_t{a.n_tiles} * a.heads <= most && a.longest > 1024;
}

// The largest logits that a windowed call's work items left in the workspace.
hipError_t join_tops(const AttnArgs& a, hipStream_t s);

template <int DP, bool EXACT, bool WIN>
hipError_t forward(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.n_tiles) * a.heads);
  if (split_keys<DP, WIN>(a, false)) hipLaunchKernelGGL((attention_kernel<DP, EXACT, 2, WIN>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((attention_kernel<DP, EXACT, 1, WIN>), grid, dim3(256), 0, s, a);
  if constexpr (WIN) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? join_tops(a, s) : e;
  }
  return hipGetLastError();
}

// The sums that rows beyond their windows give the first tokens (windowed calls only).
template <int DP, bool EXACT>
hipError_t far_rows(const AttnArgs& a, hipStream_t s);
// The sums of key tiles whose query heads were shared out.
hipError_t join_parts(const AttnArgs& a, hipStream_t s);

template <int DP, bool EXACT, bool WIN>
hipError_t backward(const AttnArgs& a, hipStream_t s) {
  const dim3 rows(static_cast<uint32_t>(a.n_tiles) * a.heads);
  if (split_keys<DP, WIN>(a, true)) hipLaunchKernelGGL((attention_dq_kernel<DP, EXACT, 2, WIN>), rows, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((attention_dq_kernel<DP, EXACT, 1, WIN>), rows, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if constexpr (WIN) {
    if (e == hipSuccess) e = far_rows<DP, EXACT>(a, s);
  }
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<uint32_t>(a.n_tiles) * a.kv_heads * (WIN ? a.key_parts : 1));
  // Up to two key tiles for each of the 256 compute units, the longest one's
  // turns are what takes the time, and the pair kernel's are half as long;
  // with more the three-to-a-unit kernel wins.  dQ, dK and dV with heads of 64,
  // us, pair | three: 1290 tokens, 25 heads (275 tiles) 53 | 60; 4096 tokens,
  // 12 heads (384) 131 | 159; 8 x 512, 16 heads (512) 41 | 37; 25 heads: 2500
  // (500) 116 | 119, 8 x 512 (800) 70 | 50, 4096 (800) 272 | 228, 64 x 64
  // (1600) 52 | 37.  With windows up to about 1100 the three-to-a-unit kernel
  // wins from fewer on: window 512, 1290 tokens, 25 heads (275) 51.7 | 58.8; 4096,
  // 12 heads (384) 75 | 67; window 1024, 2500, 25 heads (500) 94 | 82; window
  // 2048, 4096, 12 heads 120 | 134.
  if (DP == 64 && (!WIN || a.key_parts == 1) && grid.x > (WIN && a.longest <= 1280 ? 320 : 512)) hipLaunchKernelGGL((attention_dkv_kernel<64, EXACT, WIN>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((attention_dkv_pair_kernel<DP, EXACT, WIN>), grid, dim3(512), 0, s, a);
  if constexpr (WIN) {
    e = hipGetLastError();
    return e == hipSuccess ? join_parts(a, s) : e;
  }
  return hipGetLastError();
}

}  // namespace

}  // namespace muon
