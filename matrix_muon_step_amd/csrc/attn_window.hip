// Windowed attention: the kernels' instances (attn_kernels.h), and what rows
// beyond their windows give the gradients of the first tokens.
#include "attn_kernels.h"

namespace muon {

namespace {

// The first tokens are seen by every row, so their dK and dV are sums over
// the whole sequence, where other key tiles' are over a window's rows.  The
// pairs (row, first token) beyond the window are summed here, a work-group for
// kFarRows rows of a sequence and a key head, into float32 sums of their own
// that the dK/dV kernel adds in order: no work-group walks the whole sequence,
// and no atomics.  Rows stream past as in the dK/dV kernels.  The 4 waves
// share out 32-key blocks of the first tokens, and what is left over, the rows:
// with up to 32 of them each wave takes a 32-row half of every other tile, with
// up to 64 one half of every tile.  Bound by the reads of q and dO.
template <int DP, bool EXACT>
__global__ __launch_bounds__(256, 2) void attention_far_kernel(const AttnArgs a) {
  using G = Geo<DP>;
  using L = DkvLds<DP>;
  static_assert(2 * L::STAGE >= 4 * 32 * DP * 4, "the waves' sums fit the buffer");
  __shared__ __align__(1024) unsigned char smem[2 * L::STAGE];
  LAS unsigned char* lds = (LAS unsigned char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kv = blockIdx.x % a.kv_heads;
  // Every other tile begins a chunk (kFarRows is two tiles): first those at even
  // places of the list, then the others, since work-groups that exit at once
  // between ones that stay leave units without any (16384 tokens, 4 first
  // tokens, 32/8 heads of 128: 63 us for 100).
  const int place = blockIdx.x / a.kv_heads, evens = (a.n_tiles + 1) / 2;
  const AttnTile t = a.by_query[place < evens ? 2 * place : 2 * (place - evens) + 1];
  const int end = min(t.len, t.first + kFarRows);
  if (t.first % kFarRows != 0 || end <= a.window) return;  // no chunk's first tile, or all within their windows
  AttnTile rows = t;
  rows.first = max(t.first, a.window / kAttnStep * kAttnStep);
  const int nq = (end - rows.first + kAttnStep - 1) / kAttnStep;
  const int total = nq * (a.heads / a.kv_heads);
  const int parts = a.sinks <= 32 ? 4 : a.sinks <= 64 ? 2 : 1;  // waves that share a key block
  const int part = wave % parts, wk0 = wave / parts * 32;
  const int key = wk0 + (lane & 31);
  const float c = a.scale * kAttnLog2e;
  const FragOff fo = frag_offsets(lane);
  QueryStream<DP, EXACT, 4, false> stream(a, rows, kv * (a.heads / a.kv_heads), a.heads / a.kv_heads, nq, wave, lane);
  int q0 = stream.row, head = 0, cur = 0;
  stream.template next<2>(t.len, 0, lds, wave);
  const int64_t krow0 = static_cast<int64_t>(t.row0) + wk0;
  const int keys = min(t.len, a.sinks) - wk0;
  bf16x8_t kf[G::KS], vf[G::KS];
  own_rows<DP>(a.k.p + (krow0 * a.k.ts + kv * a.k.hs) * 2, a.k.ts, a.head_dim, keys, lane, kf);
  own_rows<DP>(a.v.p + (krow0 * a.v.ts + kv * a.v.hs) * 2, a.v.ts, a.head_dim, keys, lane, vf);
  f32x16_t dk[G::DB], dv[G::DB];
#pragma unroll
  for (int db = 0; db < G::DB; ++db) dk[db] = dv[db] = (f32x16_t)(0.f);
  for (int it = 0; it < total; ++it) {
    next_tile();
    if (it + 1 < total) stream.template next<2>(t.len, 0, lds, wave);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int qs = q0 + 32 * b;
      if (parts > 1 && b != (part & 1)) continue;             // another wave's half
      if (parts > 2 && (it & 1) != (part >> 1)) continue;     // or tile
      if (keys <= 0 || qs + 31 < a.window || qs >= t.len) continue;
      f32x16_t s, dp;
      dkv_scores<DP>(lds + cur, fo, b, kf, vf, s, dp);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int q = qs + res_row(r, h);
        if (q - key < a.window || q >= t.len || key >= a.sinks) s[r] = -kInf;
      }
      dkv_softmax<DP>(lds + cur, b, h, c, s, dp);
      const bf16x8_t p[2] = {to_operand(s, 0), to_operand(s, 1)}, ds[2] = {to_operand(dp, 0), to_operand(dp, 1)};
      dkv_sums<DP>(lds + cur + G::TILEB, fo, b, p, dv);
      dkv_sums<DP>(lds + cur, fo, b, ds, dk);
    }
    cur = L::STAGE - cur;
    if (++head == stream.group) {
      head = 0;
      q0 -= kAttnStep;
    }
  }
  // The waves' sums, dK's and then dV's, through LDS: 32 keys x DP a wave.
  float* out = far_sum(a, t.chunk + t.first / kFarRows, kv);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    lds_barrier();  // the last tile, or dK's sums, are read
    LAS unsigned char* mine = lds + (wave * 32 + (lane & 31)) * (DP * 4) + 16 * h;
#pragma unroll
    for (int db = 0; db < G::DB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x16_t& x = which ? dv[db] : dk[db];
        *(LAS f32x4_t*)(mine + 128 * db + 32 * g) = (f32x4_t){x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
      }
    lds_barrier();
    const int per_key = a.head_dim / 4;
    for (int i = threadIdx.x; i < a.sinks * per_key; i += 256) {
      const int row = i / per_key, d = (i - row * per_key) * 4;
      f32x4_t sum = (f32x4_t)(0.f);
      for (int w = 0; w < parts; ++w)
        sum += *(const LAS f32x4_t*)(lds + (((row >> 5) * parts + w) * 32 + (row & 31)) * (DP * 4) + d * 4);
      gst(out + (which * a.sinks + row) * a.head_dim + d, sum);
    }
  }
}

// Joins the sums of a sequence's chunks into its first: 64 runs of four to a
// work-group, a quarter of the chunks to each of its waves.
__global__ __launch_bounds__(256) void attention_far_join_kernel(const AttnArgs a) {
  __shared__ __align__(16) f32x4_t part[256];
  const int kv = blockIdx.x % a.kv_heads;
  const AttnTile t = a.by_query[blockIdx.x / a.kv_heads];
  if (t.first != 0 || t.len <= a.window) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.y * 64 + lane;
  const int first = a.window / kFarRows, n = (t.len + kFarRows - 1) / kFarRows - first;
  const int share = (n + 3) / 4, end = min(n, (wave + 1) * share);
  const int64_t step = far_sum(a, 1, 0) - far_sum(a, 0, 0);
  float* p = far_sum(a, t.chunk + first, kv) + 4 * i;
  const bool there = i < a.sinks * a.head_dim / 2;
  f32x4_t sum = (f32x4_t)(0.f);
  if (there) {
#pragma unroll 8
    for (int c = wave * share; c < end; ++c) sum += gld<f32x4_t>(p + c * step);
  }
  part[threadIdx.x] = sum;
  __syncthreads();
  if (wave > 0 || !there) return;
  gst(p, ((sum + part[64 + lane]) + part[128 + lane]) + part[192 + lane]);
}

// dK (blockIdx.y even) or dV of 32 keys of a tile from the shares of its query
// heads, in order, and then the sums over rows beyond their windows.
__global__ __launch_bounds__(256) void attention_part_join_kernel(const AttnArgs a) {
  const int tile = blockIdx.x / a.kv_heads, kv = blockIdx.x % a.kv_heads;
  const AttnTile t = a.by_key[tile];
  const int which = blockIdx.y & 1, row0 = 32 * (blockIdx.y >> 1), per_key = a.head_dim / 4;
  const HeadsView& v = which ? a.dv : a.dk;
  const float mul = which ? 1.f : a.scale;
  const int64_t step = part_sum(a, 0, 0, 1, 0) - part_sum(a, 0, 0, 0, 0);
  const int first = a.window / kFarRows, end = a.far_joined ? first + 1 : (t.len + kFarRows - 1) / kFarRows;
  for (int i = threadIdx.x; i < 32 * per_key; i += 256) {
    const int row = row0 + i / per_key, d = i % per_key * 4, key = t.first + row;
    if (key >= t.len) continue;
    const float* p = part_sum(a, tile, kv, 0, which) + row * a.head_dim + d;
    f32x4_t sum = gld<f32x4_t>(p);
    for (int j = 1; j < a.key_parts; ++j) sum += gld<f32x4_t>(p + j * step);
    if (a.far && key < a.sinks && t.len > a.window)
      for (int c = first; c < end; ++c)
        sum += gld<f32x4_t>(far_sum(a, t.chunk + c, kv) + (which * a.sinks + key) * a.head_dim + d);
    uint2 u;
    u.x = pack_bf16(sum[0] * mul, sum[1] * mul);
    u.y = pack_bf16(sum[2] * mul, sum[3] * mul);
    gst(v.p + ((static_cast<int64_t>(t.row0) + key) * v.ts + kv * v.hs + d) * 2, u);
  }
}

hipError_t join_parts(const AttnArgs& a, hipStream_t s) {
  if (a.key_parts == 1) return hipSuccess;
  hipLaunchKernelGGL(attention_part_join_kernel, dim3(static_cast<uint32_t>(a.n_tiles) * a.kv_heads, 2 * kAttnRows / 32),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

// An entry's largest logit over the items of its heads, which lie together.
__global__ __launch_bounds__(256) void attention_tops_kernel(const AttnArgs a) {
  __shared__ float part[4];
  const int n = a.logit_group * a.n_tiles;
  const float* p = a.tops + static_cast<int64_t>(blockIdx.x) * n;
  float top = -kInf;
  auto take = [&](float x) { top = top != top || x != x ? __builtin_nanf("") : fmaxf(top, x); };
  for (int i = threadIdx.x; i < n; i += 256) take(gld<float>(p + i));
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) take(__shfl_xor(top, off, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) take(part[w]);
  atomic_max_float(a.max_logit + blockIdx.x, top);
}

hipError_t join_tops(const AttnArgs& a, hipStream_t s) {
  if (!a.tops) return hipSuccess;
  hipLaunchKernelGGL(attention_tops_kernel, dim3(a.heads / a.logit_group), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DP, bool EXACT>
hipError_t far_rows(const AttnArgs& a, hipStream_t s) {
  if (!a.far) return hipSuccess;
  const uint32_t grid = static_cast<uint32_t>(a.n_tiles) * a.kv_heads;
  hipLaunchKernelGGL((attention_far_kernel<DP, EXACT>), dim3(grid), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.far_joined) return e;
  hipLaunchKernelGGL(attention_far_join_kernel, dim3(grid, (a.sinks * a.head_dim / 2 + 63) / 64), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_window_attention(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return a.head_dim == 64 ? forward<64, true, true>(a, s) : forward<64, false, true>(a, s);
  return a.head_dim == 128 ? forward<128, true, true>(a, s) : forward<128, false, true>(a, s);
}

hipError_t launch_window_attention_backward(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return a.head_dim == 64 ? backward<64, true, true>(a, s) : backward<64, false, true>(a, s);
  return a.head_dim == 128 ? backward<128, true, true>(a, s) : backward<128, false, true>(a, s);
}

}  // namespace muon
