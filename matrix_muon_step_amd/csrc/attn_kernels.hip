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
// dk and dv sum over the query heads that share a key head.
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
#include "attn_internal.h"
#include "muon_internal.h"

namespace muon {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

#define LAS __attribute__((address_space(3)))

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
// The rows' reference maximum moves only when a row outgrows it by 2^8:
// exponentials stay below 2^8, far inside float32 and bfloat16 range, and
// most tiles need no rescaling of the accumulators.
constexpr float kSlackLog2 = 8.f;

template <int DP>
struct Geo {
  static constexpr int NC = DP / 8;           // 16-byte chunks of a row
  static constexpr int PITCH = DP * 2;        // bytes of a row
  static constexpr int KS = DP / 16;          // 16-deep steps over the head dimension
  static constexpr int DB = DP / 32;          // 32-wide blocks of the head dimension
  static constexpr int TILEB = kAttnStep * PITCH;  // bytes of a streamed tile
  static constexpr int NI = kAttnStep * NC / 256;  // 16-byte loads per lane and tile (4 waves)
};

// Position of chunk c in row r of an LDS tile: c ^ swz.  Both readers are
// free of bank conflicts with it: 16 rows at one chunk (ordinary 16-byte
// fragment reads) and 4 rows at 4 chunks (transposing reads) each touch all
// 64 banks once.  Repeats every 16 rows; only its upper bits depend on the
// 64-byte group, so a fragment's address moves to another k-step or 32-wide
// block by an exclusive or.
template <int DP>
__device__ __forceinline__ int tile_swz(int r) {
  return DP == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// Direct-to-LDS load of 16 (WORD: 4) bytes a lane, lane i to dst + 16 i (4 i),
// from base + off, zero from byte `bytes` on.  base, bytes and dst are the
// same in every lane.
template <bool WORD>
__device__ __forceinline__ void load_lds(const unsigned char* base, uint32_t bytes, uint32_t off,
                                         LAS unsigned char* dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uintptr_t a = reinterpret_cast<uintptr_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  void* p = reinterpret_cast<void*>((static_cast<uintptr_t>(hi) << 32) | lo);
  // untyped, no stride: offsets are compared with the size in bytes
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(p, 0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
  if (WORD) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LAS void*)dst, 4, off, 0, 0, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LAS void*)dst, 16, off, 0, 0, 0);
#endif
}

constexpr uint32_t kOutside = 0xC0000000u;  // an offset past every descriptor (their sizes stay below 2^31)

// Offsets of a lane's 16-byte loads of a 64-row tile, relative to the tile's
// first row; chunks beyond the head dimension read as zero.
template <int DP>
struct LoadOff {
  uint32_t off[Geo<DP>::NI];
};
template <int DP>
__device__ __forceinline__ LoadOff<DP> load_offsets(int wave, int lane, int64_t ts, int head_dim) {
  using G = Geo<DP>;
  LoadOff<DP> r;
#pragma unroll
  for (int i = 0; i < G::NI; ++i) {
    const int p = (wave + i * 4) * 64 + lane;
    const int row = p / G::NC;
    const int c = (p % G::NC) ^ tile_swz<DP>(row);
    r.off[i] = c * 8 < head_dim ? static_cast<uint32_t>(row) * static_cast<uint32_t>(ts * 2) + c * 16 : kOutside;
  }
  return r;
}

// Bytes that rows first .. of a sequence of `len` rows hold behind the
// address of row `first` (rows beyond the tile are never addressed).
__device__ __forceinline__ uint32_t rows_bytes(int len, int first, int64_t ts, int head_dim, int most) {
  const int rows = min(len - first, most);
  return rows <= 0 ? 0u : static_cast<uint32_t>((rows - 1) * (ts * 2) + head_dim * 2);
}

// Starts the loads of one 64-row tile into LDS (direct, 16 bytes a lane).
template <int DP>
__device__ __forceinline__ void load_tile(const unsigned char* base, uint32_t bytes, const LoadOff<DP>& lo,
                                          LAS unsigned char* __restrict__ dst, int wave) {
#pragma unroll
  for (int i = 0; i < Geo<DP>::NI; ++i) load_lds<false>(base, bytes, lo.off[i], dst + (wave + i * 4) * 1024);
}

__device__ __forceinline__ bf16x8_t join4(bf16x4_t lo, bf16x4_t hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Lane addresses of the two fragment readers, in bytes within a tile.
//   row: 16-byte read of row (lane & 31), chunk 2 s + (lane >> 5): row ^ (32 s)
//   tr[e]: transposing read of rows 8e + 4h + 0..3, 32-wide block db:
//          tr[e] ^ (64 db); 16 rows further: + 16 PITCH
template <int DP>
struct FragOff {
  int row;
  int tr[2];
};
template <int DP>
__device__ __forceinline__ FragOff<DP> frag_offsets(int lane) {
  using G = Geo<DP>;
  FragOff<DP> f;
  const int r = lane & 31, h = lane >> 5;
  f.row = r * G::PITCH + ((h ^ tile_swz<DP>(r)) << 4);
  const int cl = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int tr = 8 * e + 4 * h + ((lane & 15) >> 2);
    f.tr[e] = tr * G::PITCH + ((cl ^ tile_swz<DP>(tr)) << 4) + (lane & 1) * 8;
  }
  return f;
}

// Left operand of a product over the head dimension: rows 32 b + 0..31 of a
// tile, k-step s.
template <int DP>
__device__ __forceinline__ bf16x8_t row_frag(const LAS unsigned char* __restrict__ t, const FragOff<DP>& f, int b,
                                             int s) {
  return *(const LAS bf16x8_t*)(t + (f.row ^ (s * 32)) + b * 32 * Geo<DP>::PITCH);
}
// Left operand of a product over rows: columns 32 db + 0..31 of a tile,
// rows 16 t16 + 0..15 in the order of the results' registers.
template <int DP>
__device__ __forceinline__ bf16x8_t col_frag(const LAS unsigned char* __restrict__ t, const FragOff<DP>& f, int db,
                                             int t16) {
  const LAS unsigned char* p0 = t + (f.tr[0] ^ (db * 64)) + t16 * 16 * Geo<DP>::PITCH;
  const LAS unsigned char* p1 = t + (f.tr[1] ^ (db * 64)) + t16 * 16 * Geo<DP>::PITCH;
  return join4(__builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)p0),
               __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LAS bf16x4_t*)p1));
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

__device__ __forceinline__ float half_max(float x) { return fmaxf(x, __shfl_xor(x, 32, 64)); }
__device__ __forceinline__ float half_sum(float x) { return x + __shfl_xor(x, 32, 64); }

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

// Running maximum of a float in memory, in any order of arrival with the
// same result: for values >= 0 the integer order of the bits is the float
// order, for negative ones the reverse.  NaN is passed as 0x7fffffff, which
// both orders keep.
__device__ __forceinline__ void atomic_max_float(float* p, float x) {
  const int b = x != x ? 0x7fffffff : __float_as_int(x);
  if (b >= 0) atomicMax(reinterpret_cast<int*>(p), b);
  else atomicMin(reinterpret_cast<unsigned int*>(p), static_cast<unsigned int>(b));
}

// ------------------------------------------------------------------ forward
// One work-group: 128 query rows of one head, 4 waves of 32 rows; key and
// value tiles of 64 rows stream through a double buffer in LDS.
template <int DP>
__global__ __launch_bounds__(256, 2) void attention_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  __shared__ __align__(1024) unsigned char smem[4 * G::TILEB];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hx = blockIdx.x % a.heads;
  const AttnTile t = a.by_query[blockIdx.x / a.heads];
  const int kv = hx % a.kv_heads;
  const int head = kv * (a.heads / a.kv_heads) + hx / a.kv_heads;
  const int nk = (min(t.len, t.first + kAttnRows) + kAttnStep - 1) / kAttnStep;
  const int wq0 = t.first + 32 * wave;   // the wave's first query row in its sequence
  const int q = wq0 + (lane & 31);
  const float c = a.scale * kLog2e;
  const float slack = kSlackLog2 / c;

  const unsigned char* kbase = a.k.p + (t.row0 * a.k.ts + kv * a.k.hs) * 2;
  const unsigned char* vbase = a.v.p + (t.row0 * a.v.ts + kv * a.v.hs) * 2;
  const LoadOff<DP> ko = load_offsets<DP>(wave, lane, a.k.ts, a.head_dim);
  const LoadOff<DP> vo = load_offsets<DP>(wave, lane, a.v.ts, a.head_dim);
  const FragOff<DP> fo = frag_offsets<DP>(lane);
  auto issue = [&](int kt) {
    LAS unsigned char* dst = lds + (kt & 1) * 2 * G::TILEB;
    const int k0 = kt * kAttnStep;
    load_tile<DP>(kbase + static_cast<int64_t>(k0) * a.k.ts * 2, rows_bytes(t.len, k0, a.k.ts, a.head_dim, kAttnStep), ko, dst,
                  wave);
    load_tile<DP>(vbase + static_cast<int64_t>(k0) * a.v.ts * 2, rows_bytes(t.len, k0, a.v.ts, a.head_dim, kAttnStep), vo,
                  dst + G::TILEB, wave);
  };
  issue(0);
  bf16x8_t qf[G::KS];
  own_rows<DP>(a.q.p + ((static_cast<int64_t>(t.row0) + wq0) * a.q.ts + head * a.q.hs) * 2, a.q.ts, a.head_dim, t.len - wq0,
               lane, qf);

  f32x16_t o[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) o[db] = (f32x16_t)(0.f);
  float m_top = -kInf, m_ref = -kInf, l = 0.f;  // l: this lane's half of the keys
  for (int kt = 0; kt < nk; ++kt) {
    const int k0 = kt * kAttnStep;
    next_tile();
    if (kt + 1 < nk) issue(kt + 1);
    if (k0 > wq0 + 31) continue;  // every key lies behind the wave's rows
    const LAS unsigned char* kt_lds = lds + (kt & 1) * 2 * G::TILEB;
    const LAS unsigned char* vt_lds = kt_lds + G::TILEB;
    f32x16_t s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      s[b] = (f32x16_t)(0.f);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) s[b] = mfma(row_frag<DP>(kt_lds, fo, b, st), qf[st], s[b]);
    }
    if (k0 + kAttnStep - 1 > wq0) {
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
  const bool live = q < t.len;
  l = half_sum(l);
  store_rows<DP>(a.o, static_cast<int64_t>(t.row0) + q, head, a.head_dim, live, lane, o, 1.f / l);
  if (live && h == 0)
    gst(a.lse + head * a.lse_stride + t.row0 + q, fmaf(m_ref, a.scale, kLn2 * __builtin_amdgcn_logf(l)));
  if (a.max_logit) {
    // A row whose sum is NaN has a NaN logit (or only infinite ones).
    float top = !live ? -kInf : l != l ? __builtin_nanf("") : m_top * a.scale;
#pragma unroll
    for (int off = 1; off <= 16; off <<= 1) {
      const float other = __shfl_xor(top, off, 64);
      top = top != top || other != other ? __builtin_nanf("") : fmaxf(top, other);
    }
    if (lane == 0 && wq0 < t.len) atomic_max_float(a.max_logit + head / a.logit_group, top);
  }
}

// ------------------------------------------------------------ backward: dQ
// One work-group: 128 query rows of one head, 4 waves of 32 rows; key and
// value tiles stream past.  Also forms delta and leaves it, with lse in
// base 2, for the dK/dV kernel that follows.
template <int DP>
__global__ __launch_bounds__(256, 1) void attention_dq_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  __shared__ __align__(1024) unsigned char smem[4 * G::TILEB];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hx = blockIdx.x % a.heads;
  const AttnTile t = a.by_query[blockIdx.x / a.heads];
  const int kv = hx % a.kv_heads;
  const int head = kv * (a.heads / a.kv_heads) + hx / a.kv_heads;
  const int nk = (min(t.len, t.first + kAttnRows) + kAttnStep - 1) / kAttnStep;
  const int wq0 = t.first + 32 * wave;
  const int q = wq0 + (lane & 31);
  const bool live = q < t.len;
  const int64_t row = static_cast<int64_t>(t.row0) + q;
  const float c = a.scale * kLog2e;

  const unsigned char* kbase = a.k.p + (t.row0 * a.k.ts + kv * a.k.hs) * 2;
  const unsigned char* vbase = a.v.p + (t.row0 * a.v.ts + kv * a.v.hs) * 2;
  const LoadOff<DP> ko = load_offsets<DP>(wave, lane, a.k.ts, a.head_dim);
  const LoadOff<DP> vo = load_offsets<DP>(wave, lane, a.v.ts, a.head_dim);
  const FragOff<DP> fo = frag_offsets<DP>(lane);
  auto issue = [&](int kt) {
    LAS unsigned char* dst = lds + (kt & 1) * 2 * G::TILEB;
    const int k0 = kt * kAttnStep;
    load_tile<DP>(kbase + static_cast<int64_t>(k0) * a.k.ts * 2, rows_bytes(t.len, k0, a.k.ts, a.head_dim, kAttnStep), ko, dst,
                  wave);
    load_tile<DP>(vbase + static_cast<int64_t>(k0) * a.v.ts * 2, rows_bytes(t.len, k0, a.v.ts, a.head_dim, kAttnStep), vo,
                  dst + G::TILEB, wave);
  };
  issue(0);
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
  const float lse2 = live ? gld<float>(a.lse + head * a.lse_stride + row) * kLog2e : 0.f;
  if (live && h == 0) {
    gst(a.row_lse2 + head * a.row_stride + row, lse2);
    gst(a.row_delta + head * a.row_stride + row, delta);
  }

  f32x16_t dq[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) dq[db] = (f32x16_t)(0.f);
  for (int kt = 0; kt < nk; ++kt) {
    const int k0 = kt * kAttnStep;
    next_tile();
    if (kt + 1 < nk) issue(kt + 1);
    if (k0 > wq0 + 31) continue;
    const LAS unsigned char* kt_lds = lds + (kt & 1) * 2 * G::TILEB;
    const LAS unsigned char* vt_lds = kt_lds + G::TILEB;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x16_t s = (f32x16_t)(0.f), dp = (f32x16_t)(0.f);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) s = mfma(row_frag<DP>(kt_lds, fo, b, st), qf[st], s);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) dp = mfma(row_frag<DP>(vt_lds, fo, b, st), gf[st], dp);
      const bool edge = k0 + 32 * b + 31 > wq0;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2));
        s[r] = p * (dp[r] - delta);
        if (edge && k0 + 32 * b + res_row(r, h) > q) s[r] = 0.f;
      }
#pragma unroll
      for (int s16 = 0; s16 < 2; ++s16) {
        const bf16x8_t ds = to_operand(s, s16);
#pragma unroll
        for (int db = 0; db < G::DB; ++db) dq[db] = mfma(col_frag<DP>(kt_lds, fo, db, 2 * b + s16), ds, dq[db]);
      }
    }
  }
  store_rows<DP>(a.dq, row, head, a.head_dim, live, lane, dq, a.scale);
}

// -------------------------------------------------------- backward: dK, dV
// One work-group: 128 key rows of one key head, 4 waves of 32 keys; the
// query and upstream-gradient tiles of every query head of the group stream
// past, so that the sums over rows and heads stay in registers, in a fixed
// order.
template <int DP>
__global__ __launch_bounds__(256, 1) void attention_dkv_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  constexpr int STAGE = 2 * G::TILEB + 2 * kAttnStep * 4;
  __shared__ __align__(1024) unsigned char smem[2 * STAGE];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kv = blockIdx.x % a.kv_heads;
  const AttnTile t = a.by_key[blockIdx.x / a.kv_heads];
  const int group = a.heads / a.kv_heads;
  const int nq = (t.len - t.first + kAttnStep - 1) / kAttnStep;  // query tiles from the diagonal on
  const int total = nq * group;
  const int wk0 = t.first + 32 * wave;
  const int key = wk0 + (lane & 31);
  const float c = a.scale * kLog2e;

  const LoadOff<DP> qo = load_offsets<DP>(wave, lane, a.q.ts, a.head_dim);
  const LoadOff<DP> go = load_offsets<DP>(wave, lane, a.d_o.ts, a.head_dim);
  const FragOff<DP> fo = frag_offsets<DP>(lane);
  auto issue = [&](int it) {
    LAS unsigned char* dst = lds + (it & 1) * STAGE;
    const int head = kv * group + it / nq;
    const int q0 = t.first + (it % nq) * kAttnStep;
    const int64_t row = static_cast<int64_t>(t.row0) + q0;
    load_tile<DP>(a.q.p + (row * a.q.ts + head * a.q.hs) * 2, rows_bytes(t.len, q0, a.q.ts, a.head_dim, kAttnStep), qo, dst,
                  wave);
    load_tile<DP>(a.d_o.p + (row * a.d_o.ts + head * a.d_o.hs) * 2,
                  rows_bytes(t.len, q0, a.d_o.ts, a.head_dim, kAttnStep), go, dst + G::TILEB, wave);
    if (wave < 2) {
      const float* src = (wave == 0 ? a.row_lse2 : a.row_delta) + head * a.row_stride + row;
      load_lds<true>(reinterpret_cast<const unsigned char*>(src), 4u * min(t.len - q0, kAttnStep), lane * 4,
                  dst + 2 * G::TILEB + wave * kAttnStep * 4);
    }
  };
  issue(0);
  const int64_t krow0 = static_cast<int64_t>(t.row0) + wk0;
  bf16x8_t kf[G::KS], vf[G::KS];
  own_rows<DP>(a.k.p + (krow0 * a.k.ts + kv * a.k.hs) * 2, a.k.ts, a.head_dim, t.len - wk0, lane, kf);
  own_rows<DP>(a.v.p + (krow0 * a.v.ts + kv * a.v.hs) * 2, a.v.ts, a.head_dim, t.len - wk0, lane, vf);
  f32x16_t dk[G::DB], dv[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) dk[db] = dv[db] = (f32x16_t)(0.f);

  for (int it = 0; it < total; ++it) {
    next_tile();
    if (it + 1 < total) issue(it + 1);
    if (wk0 >= t.len) continue;
    const int q0 = t.first + (it % nq) * kAttnStep;
    const LAS unsigned char* qt = lds + (it & 1) * STAGE;
    const LAS unsigned char* gt = qt + G::TILEB;
    const LAS float* rows_lse = (const LAS float*)(qt + 2 * G::TILEB);
    const LAS float* rows_delta = rows_lse + kAttnStep;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int qs = q0 + 32 * b;
      if (qs + 31 < wk0 || qs >= t.len) continue;  // no query of the block sees a key of the wave
      f32x16_t s = (f32x16_t)(0.f), dp = (f32x16_t)(0.f);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) s = mfma(row_frag<DP>(qt, fo, b, st), kf[st], s);
#pragma unroll
      for (int st = 0; st < G::KS; ++st) dp = mfma(row_frag<DP>(gt, fo, b, st), vf[st], dp);
      const bool edge = qs < wk0 + 31 || qs + 31 >= t.len;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t lse2 = *(const LAS f32x4_t*)(rows_lse + 32 * b + 8 * g + 4 * h);
        const f32x4_t delta = *(const LAS f32x4_t*)(rows_delta + 32 * b + 8 * g + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * g + i, q = qs + 8 * g + 4 * h + i;
          float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2[i]));
          float ds = p * (dp[r] - delta[i]);
          if (edge && (key > q || q >= t.len)) p = ds = 0.f;
          s[r] = p;
          dp[r] = ds;
        }
      }
#pragma unroll
      for (int s16 = 0; s16 < 2; ++s16) {
        const bf16x8_t p = to_operand(s, s16), ds = to_operand(dp, s16);
#pragma unroll
        for (int db = 0; db < G::DB; ++db) dv[db] = mfma(col_frag<DP>(gt, fo, db, 2 * b + s16), p, dv[db]);
#pragma unroll
        for (int db = 0; db < G::DB; ++db) dk[db] = mfma(col_frag<DP>(qt, fo, db, 2 * b + s16), ds, dk[db]);
      }
    }
  }
  const bool live = key < t.len;
  const int64_t row = static_cast<int64_t>(t.row0) + key;
  store_rows<DP>(a.dk, row, kv, a.head_dim, live, lane, dk, a.scale);
  store_rows<DP>(a.dv, row, kv, a.head_dim, live, lane, dv, 1.f);
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.n_tiles) * a.heads);
  if (a.head_dim <= 64) hipLaunchKernelGGL(attention_kernel<64>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(attention_kernel<128>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s) {
  const dim3 gq(static_cast<uint32_t>(a.n_tiles) * a.heads), gk(static_cast<uint32_t>(a.n_tiles) * a.kv_heads);
  if (a.head_dim <= 64) {
    hipLaunchKernelGGL(attention_dq_kernel<64>, gq, dim3(256), 0, s, a);
    hipLaunchKernelGGL(attention_dkv_kernel<64>, gk, dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL(attention_dq_kernel<128>, gq, dim3(256), 0, s, a);
    hipLaunchKernelGGL(attention_dkv_kernel<128>, gk, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace muon
