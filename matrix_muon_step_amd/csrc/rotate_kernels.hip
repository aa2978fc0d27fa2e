// Norms of queries and keys per head with rotary positions in the same pass,
// and their gradient, on gfx950.
//
// Per token and head, over the head's D elements:
//   y_d = x_d r w_d,  r = 1 / sqrt(mean x^2 + eps)     (without a norm y = x)
//   pair (l, h) = (i, R/2 + i), or (2i, 2i + 1), i < R/2, at the angle
//   u = position[axis_i] f_i:  z_l = y_l cos u - y_h sin u,  z_h = y_h cos u + y_l sin u
//   z_d = y_d for d >= R
// Gradient: g = dz turned back by u, n = x r,
//   dw_d = sum over tokens and heads of g_d n_d
//   dx_d = r (w_d g_d - n_d mean(w g n))
//
// Angles: a frequency is held as turns per position times 2^64; its product
// with the position modulo 2^64 is the angle modulo one turn, exact but for the
// frequency's own rounding (2^-65 turns a position), however far the position.
// Sine and cosine of what is left of it next to a quarter turn by their power series.
//
// Bound by memory: each element is read and written once.  A lane holds 8 (or
// 4) pairs of a head, both halves of which it loads itself, so that only the
// sum of squares crosses lanes; the lanes of a head are neighbours.  The
// angles of a token serve all its heads from LDS.
#include "muon_internal.h"
#include "rotate_internal.h"

namespace muon {

namespace {

constexpr float kInf = __builtin_inff();

// cos and sin of a 2^64th of a turn times `phase`.
__device__ __forceinline__ void cos_sin(uint64_t phase, float& c, float& s) {
  phase += uint64_t{1} << 61;  // to the nearest quarter turn: what is left is within an eighth
  const uint32_t quarter = static_cast<uint32_t>(phase >> 62);
  const int32_t left = static_cast<int32_t>(static_cast<uint32_t>(phase >> 30) ^ 0x80000000u);
  // 2^-32 of a quarter turn; |u| <= pi / 4
  const float u = static_cast<float>(left) * (1.57079632679489661923f * 0x1p-32f), v = u * u;
  // sum (-1)^k u^(2k+1) / (2k+1)! and (-1)^k u^(2k) / (2k)!; the terms left out are below 2^-29
  const float sn = fmaf(u * v, fmaf(v, fmaf(v, fmaf(v, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), u);
  const float cs = fmaf(v, fmaf(v, fmaf(v, fmaf(v, fmaf(v, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -.5f), 1.f);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if (((quarter + 1) >> 1) & 1) c = -c;  // quarters 1 and 2
  if (quarter >> 1) s = -s;              // 2 and 3
}

// cos (first) and sin of every pair of a piece's tokens, token by token.
struct Angles {
  float cos[kRotateRows * kAttnMaxDim / 2];
  float sin[kRotateRows * kAttnMaxDim / 2];
};

__device__ __forceinline__ void fill_angles(const RotateArgs& a, int64_t row, int index, int n, Angles& to) {
  const int half = a.rotary_dim >> 1;
  for (int i = threadIdx.x; i < n * half; i += kRotateLanes) {
    const int token = i / half, pair = i - token * half;
    int64_t place = index + token;
    if (a.positions) {
      const int64_t at = a.axis[pair] * a.position_stride + row + token;
      place = a.positions_64 ? gld<int64_t>(static_cast<const int64_t*>(a.positions) + at)
                             : gld<int32_t>(static_cast<const int32_t*>(a.positions) + at);
    }
    cos_sin(static_cast<uint64_t>(place) * a.frequency[pair], to.cos[i], to.sin[i]);
  }
}

// x summed over the 1 << log2 (<= 16) neighbouring lanes that share a head.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float head_sum(float x, int log2) {
  if (log2 > 0) x += dpp<0xB1>(x);   // lane ^ 1
  if (log2 > 1) x += dpp<0x4E>(x);   // lane ^ 2
  if (log2 > 2) x += dpp<0x141>(x);  // lanes 0-7 mirrored: the other four's sum
  if (log2 > 3) x += dpp<0x140>(x);  // lanes 0-15 mirrored
  return x;
}

// P elements of bfloat16 as they lie in memory.
template <int P>
struct Raw;
template <>
struct Raw<8> {
  uint4 u;
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf_lo(u.x), v[1] = bf_hi(u.x), v[2] = bf_lo(u.y), v[3] = bf_hi(u.y);
    v[4] = bf_lo(u.z), v[5] = bf_hi(u.z), v[6] = bf_lo(u.w), v[7] = bf_hi(u.w);
  }
  __device__ __forceinline__ void put(const float* v) {
    u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  }
};
template <>
struct Raw<4> {
  uint2 u;
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf_lo(u.x), v[1] = bf_hi(u.x), v[2] = bf_lo(u.y), v[3] = bf_hi(u.y);
  }
  __device__ __forceinline__ void put(const float* v) { u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}; }
};

// A lane's place in a head: its pairs' two runs of P elements.  Past
// rotary_dim the rest is dealt out in halves too, and not turned.
template <int P, bool INTER>
struct Place {
  int lo, hi;     // first elements of the runs
  int pair;       // its first pair in a token's angles
  bool live, turned;
  __device__ __forceinline__ Place(const RotateArgs& a, int c) {
    const int R = a.rotary_dim, D = a.head_dim;
    live = c * 2 * P < D;
    turned = c * 2 * P < R;
    pair = c * P;
    if (INTER) {
      lo = c * 2 * P;
      hi = lo + P;
    } else if (turned) {
      lo = c * P;
      hi = lo + R / 2;
    } else {
      lo = R / 2 + c * P;  // R + (c - R / 2P) P
      hi = lo + (D - R) / 2;
    }
  }
  // x turned by the angles (BACK: against them), in place.
  template <bool BACK>
  __device__ __forceinline__ void turn(const Angles& angles, int first, float (&x)[2 * P]) const {
    if (!turned) return;
    float c[P], s[P];
#pragma unroll
    for (int i = 0; i < P; i += 4) {  // a token's angles start at a multiple of P
      const float4 cv = *static_cast<const float4*>(__builtin_assume_aligned(angles.cos + first + pair + i, 16));
      const float4 sv = *static_cast<const float4*>(__builtin_assume_aligned(angles.sin + first + pair + i, 16));
      c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
      s[i] = sv.x, s[i + 1] = sv.y, s[i + 2] = sv.z, s[i + 3] = sv.w;
    }
    if (BACK)
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] = -s[i];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float& l = x[INTER ? 2 * i : i];
      float& h = x[INTER ? 2 * i + 1 : P + i];
      const float t = fmaf(l, c[i], -h * s[i]);
      h = fmaf(h, c[i], l * s[i]);
      l = t;
    }
  }
};

// A lane's way through the (token, head) pairs of a piece.
struct Walk {
  int token, head, left;  // left: heads from here to the piece's end
  __device__ __forceinline__ Walk(int slot, int heads, int n) {
    token = slot / heads;
    head = slot - token * heads;
    left = n * heads - slot;
  }
  __device__ __forceinline__ void next(const RotateTensor& t, int slots) {
    token += t.step_token;
    head += t.step_head;
    if (head >= t.heads) {
      head -= t.heads;
      ++token;
    }
    left -= slots;
  }
};

__device__ __forceinline__ unsigned char* at(const HeadsView& v, int64_t row, int token, int head) {
  return v.p + ((row + token) * v.ts + head * v.hs) * 2;
}

// 1 / sqrt(mean x^2 + eps) of the head that x is a lane's part of.  Where the
// squares of finite values overflow, x is scaled by 2^-72 and the result
// belongs to the scaled x (eps is nothing beside it); `back` is that scale, or 1.
template <int N>
__device__ __forceinline__ float inverse_size(const RotateArgs& a, float (&x)[N], float& back) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) sum = fmaf(x[i], x[i], sum);
  sum = head_sum(sum, a.group_log2);
  back = 1.f;
  const float share = 1.f / static_cast<float>(a.head_dim);
  if (__builtin_expect(sum == kInf, 0)) {
    back = 0x1p-72f;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] *= back;
      sum = fmaf(x[i], x[i], sum);
    }
    sum = head_sum(sum, a.group_log2);
    return __builtin_amdgcn_rsqf(sum * share);
  }
  return __builtin_amdgcn_rsqf(fmaf(sum, share, a.eps));
}

template <int P>
__device__ __forceinline__ void load_weight(const float* w, int lo, int hi, bool live, float (&v)[2 * P]) {
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) v[i] = w && live ? gld<float>(w + (i < P ? lo + i : hi + i - P)) : 1.f;
}

// ------------------------------------------------------------------ forward
template <int P, bool INTER, bool NORM>
__global__ __launch_bounds__(kRotateLanes) void rotate_kernel(const RotateArgs a) {
  constexpr int U = 2;  // heads a lane has under way
  __shared__ __align__(16) Angles angles;
  const int slots = kRotateLanes >> a.group_log2, slot = threadIdx.x >> a.group_log2;
  const Place<P, INTER> place(a, threadIdx.x & ((1 << a.group_log2) - 1));
  const int half = a.rotary_dim >> 1;
  for (int64_t piece = blockIdx.x; piece < int64_t{a.n_tiles} * kRotatePieces; piece += gridDim.x) {
    const AttnTile t = a.tiles[piece / kRotatePieces];
    const int index = t.first + static_cast<int>(piece % kRotatePieces) * kRotateRows;
    const int n = min(t.len - index, kRotateRows);
    if (n <= 0) continue;
    const int64_t row = static_cast<int64_t>(t.row0) + index;
    __syncthreads();  // the last piece's angles are done with
    fill_angles(a, row, index, n, angles);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const RotateTensor& x = a.t[which];
      float w[2 * P];
      if (NORM) load_weight<P>(x.weight, place.lo, place.hi, place.live, w);
      Walk walk(slot, x.heads, n);
      while (walk.left > 0) {
        Raw<P> lo[U], hi[U];
        int token[U], head[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          token[u] = walk.token, head[u] = walk.head;
          on[u] = walk.left > 0 && place.live;
          if (on[u]) {
            const unsigned char* p = at(x.x, row, token[u], head[u]);
            lo[u] = gld<Raw<P>>(p + place.lo * 2);
            hi[u] = gld<Raw<P>>(p + place.hi * 2);
          } else {
            lo[u] = hi[u] = Raw<P>{};
          }
          walk.next(x, slots);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[2 * P];
          lo[u].get(v);
          hi[u].get(v + P);
          if (NORM) {
            float back;
            const float r = inverse_size<2 * P>(a, v, back);
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) v[i] = v[i] * r * w[i];
          }
          if (!on[u]) continue;
          place.template turn<false>(angles, token[u] * half, v);
          lo[u].put(v);
          hi[u].put(v + P);
          unsigned char* p = at(x.out, row, token[u], head[u]);
          gst(p + place.lo * 2, lo[u]);
          gst(p + place.hi * 2, hi[u]);
        }
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// Without a norm the gradient is dz turned back.
template <int P, bool INTER, bool NORM>
__global__ __launch_bounds__(kRotateLanes) void rotate_backward_kernel(const RotateArgs a) {
  constexpr int U = 2;
  __shared__ __align__(16) Angles angles;
  const int slots = kRotateLanes >> a.group_log2, slot = threadIdx.x >> a.group_log2;
  const Place<P, INTER> place(a, threadIdx.x & ((1 << a.group_log2) - 1));
  const int half = a.rotary_dim >> 1;
  const float share = 1.f / static_cast<float>(a.head_dim);
  float dw[2][2 * P];
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) dw[0][i] = dw[1][i] = 0.f;
  for (int64_t piece = blockIdx.x; piece < int64_t{a.n_tiles} * kRotatePieces; piece += gridDim.x) {
    const AttnTile t = a.tiles[piece / kRotatePieces];
    const int index = t.first + static_cast<int>(piece % kRotatePieces) * kRotateRows;
    const int n = min(t.len - index, kRotateRows);
    if (n <= 0) continue;
    const int64_t row = static_cast<int64_t>(t.row0) + index;
    __syncthreads();
    fill_angles(a, row, index, n, angles);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const RotateTensor& x = a.t[which];
      float w[2 * P];
      if (NORM) load_weight<P>(x.weight, place.lo, place.hi, place.live, w);
      Walk walk(slot, x.heads, n);
      while (walk.left > 0) {
        Raw<P> lo[U], hi[U], glo[U], ghi[U];
        int token[U], head[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          token[u] = walk.token, head[u] = walk.head;
          on[u] = walk.left > 0 && place.live;
          lo[u] = hi[u] = glo[u] = ghi[u] = Raw<P>{};
          if (on[u]) {
            const unsigned char* p = at(x.up, row, token[u], head[u]);
            glo[u] = gld<Raw<P>>(p + place.lo * 2);
            ghi[u] = gld<Raw<P>>(p + place.hi * 2);
            if (NORM) {
              const unsigned char* px = at(x.x, row, token[u], head[u]);
              lo[u] = gld<Raw<P>>(px + place.lo * 2);
              hi[u] = gld<Raw<P>>(px + place.hi * 2);
            }
          }
          walk.next(x, slots);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float g[2 * P];
          glo[u].get(g);
          ghi[u].get(g + P);
          // lanes that hold nothing (zeros) go along up to the sums over lanes
          if (on[u]) place.template turn<true>(angles, token[u] * half, g);
          if (NORM) {
            float v[2 * P], back;
            lo[u].get(v);
            hi[u].get(v + P);
            const float r = inverse_size<2 * P>(a, v, back);
            float along = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
              v[i] *= r;
              if (on[u]) dw[which][i] = fmaf(g[i], v[i], dw[which][i]);
              g[i] *= w[i];
              along = fmaf(g[i], v[i], along);
            }
            along = head_sum(along, a.group_log2) * share;
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) g[i] = r * back * fmaf(-along, v[i], g[i]);
          }
          if (!on[u]) continue;
          glo[u].put(g);
          ghi[u].put(g + P);
          unsigned char* p = at(x.out, row, token[u], head[u]);
          gst(p + place.lo * 2, glo[u]);
          gst(p + place.hi * 2, ghi[u]);
        }
      }
    }
  }
  if (!NORM || (!a.t[0].d_weight && !a.t[1].d_weight)) return;
  // This work-group's sums over its lanes, in a fixed order.
  __shared__ float part[kRotateLanes / 64][2][kAttnMaxDim];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
      float x = dw[which][i];
      for (int off = 32; off >= 1 << a.group_log2; off >>= 1) x += __shfl_xor(x, off, 64);
      if (lane < 1 << a.group_log2 && place.live) part[wave][which][i < P ? place.lo + i : place.hi + i - P] = x;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.head_dim; i += kRotateLanes) {
    const int which = i >= a.head_dim, d = i - which * a.head_dim;
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < kRotateLanes / 64; ++v) x += part[v][which][d];
    gst(a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.head_dim + i, x);
  }
}

// The weights' gradients from the work-groups' sums, in float64: 16 elements
// of one tensor to a work-group, 16 lanes to an element.
__global__ __launch_bounds__(256) void rotate_weights_kernel(const RotateArgs a, int groups) {
  __shared__ double part[16][16];
  float* out = a.t[blockIdx.y].d_weight;
  const int e = threadIdx.x & 15, r = threadIdx.x >> 4, d = blockIdx.x * 16 + e;
  double x = 0.0;
  if (d < a.head_dim && out)
    for (int i = r; i < groups; i += 16)
      x += gld<float>(a.partials + (static_cast<int64_t>(i) * 2 + blockIdx.y) * a.head_dim + d);
  part[r][e] = x;
  __syncthreads();
  if (r > 0 || d >= a.head_dim || !out) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) x += part[i][e];
  gst(out + d, static_cast<float>(x));
}

uint32_t groups_of(const RotateArgs& a, int64_t most) {
  const int64_t pieces = int64_t{a.n_tiles} * kRotatePieces;
  return static_cast<uint32_t>(pieces < most ? pieces : most);
}

template <int P, bool INTER, bool NORM>
void forward(const RotateArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((rotate_kernel<P, INTER, NORM>), dim3(groups_of(a, 1 << 20)), dim3(kRotateLanes), 0, s, a);
}
template <int P, bool INTER, bool NORM>
void backward(const RotateArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((rotate_backward_kernel<P, INTER, NORM>), dim3(groups_of(a, kRotateGroups)), dim3(kRotateLanes), 0, s,
                     a);
}

}  // namespace

hipError_t launch_rotate(const RotateArgs& a, bool wide, bool interleaved, bool norm, hipStream_t s) {
  if (wide) {
    if (interleaved) norm ? forward<8, true, true>(a, s) : forward<8, true, false>(a, s);
    else norm ? forward<8, false, true>(a, s) : forward<8, false, false>(a, s);
  } else {
    if (interleaved) norm ? forward<4, true, true>(a, s) : forward<4, true, false>(a, s);
    else norm ? forward<4, false, true>(a, s) : forward<4, false, false>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_rotate_backward(const RotateArgs& a, bool wide, bool interleaved, bool norm, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.n_tiles > 0) {
    if (wide) {
      if (interleaved) norm ? backward<8, true, true>(a, s) : backward<8, true, false>(a, s);
      else norm ? backward<8, false, true>(a, s) : backward<8, false, false>(a, s);
    } else {
      if (interleaved) norm ? backward<4, true, true>(a, s) : backward<4, true, false>(a, s);
      else norm ? backward<4, false, true>(a, s) : backward<4, false, false>(a, s);
    }
    e = hipGetLastError();
  }
  if (e != hipSuccess || (!a.t[0].d_weight && !a.t[1].d_weight)) return e;
  hipLaunchKernelGGL(rotate_weights_kernel, dim3((a.head_dim + 15) / 16, 2), dim3(256), 0, s, a,
                     static_cast<int>(groups_of(a, kRotateGroups)));
  return hipGetLastError();
}

}  // namespace muon
