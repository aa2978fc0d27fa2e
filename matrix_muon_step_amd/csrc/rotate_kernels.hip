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
// frequency's own rounding (2^-64 turns a position), however far the position.
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
    if (!live) c = 0;
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
  // Which lane of a head holds element d, and at which of its 2 P places.
  static __device__ __forceinline__ void of_element(const RotateArgs& a, int d, int& lane, int& k) {
    if (INTER) {
      lane = d / (2 * P);
      k = d % (2 * P);
      return;
    }
    const int R = a.rotary_dim;
    const bool rest = d >= R;
    const int half = (rest ? a.head_dim - R : R) / 2;
    if (rest) d -= R;
    const bool high = d >= half;
    if (high) d -= half;
    lane = (rest ? R / (2 * P) : 0) + d / P;
    k = (high ? P : 0) + d % P;
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

// A lane's way through the (token, head) pairs of a piece, with its place in
// each of N tensors.  Past its last head it stays there, where loads are
// harmless; so do the loads of lanes that hold no part of a head (as lane 0's).
template <int N>
struct Walk {
  unsigned char* p[N];
  int64_t step[N], wrap[N];  // bytes to the next head; from behind a token's last head to the next token
  int token, head, left;     // left: heads from here to the piece's end
  int heads, step_token, step_head, slots;
  __device__ __forceinline__ Walk(const RotateTensor& t, const HeadsView (&v)[N], int64_t row, int slot, int slots_, int n) {
    heads = t.heads, step_token = t.step_token, step_head = t.step_head, slots = slots_;
    left = n * heads - slot;
    if (left <= 0) slot = 0;
    token = slot / heads;
    head = slot - token * heads;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = v[i].p + ((row + token) * v[i].ts + head * v[i].hs) * 2;
      step[i] = (step_token * v[i].ts + step_head * v[i].hs) * 2;
      wrap[i] = (v[i].ts - heads * v[i].hs) * 2;
    }
  }
  __device__ __forceinline__ void next() {
    left -= slots;
    if (left <= 0) return;
    token += step_token;
    head += step_head;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] += step[i];
    if (head >= heads) {
      head -= heads;
      ++token;
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] += wrap[i];
    }
  }
};

// 1 / sqrt(mean x^2 + eps) of the head that x is a lane's part of.  Where the
// squares of finite values overflow, x is scaled by 2^-72 and the result
// belongs to the scaled x (eps is nothing beside it); `back` is that scale, or 1.
template <int N>
__device__ __forceinline__ float inverse_size(const RotateArgs& a, bool live, float (&x)[N], float& back) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) sum = fmaf(x[i], x[i], sum);
  sum = head_sum(live ? sum : 0.f, a.group_log2);
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
    sum = head_sum(live ? sum : 0.f, a.group_log2);
    return __builtin_amdgcn_rsqf(sum * share);
  }
  return __builtin_amdgcn_rsqf(fmaf(sum, share, a.eps));
}

template <int P>
__device__ __forceinline__ void load_weight(const float* w, int lo, int hi, float (&v)[2 * P]) {
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) v[i] = w ? gld<float>(w + (i < P ? lo + i : hi + i - P)) : 1.f;
}

// A work item's rows, and none for pieces past a sequence's end.
struct Piece {
  int64_t row;   // packed row of its first token
  int index, n;  // that token's index in its sequence; tokens
  __device__ __forceinline__ Piece(const RotateArgs& a, int64_t i) {
    const AttnTile t = a.tiles[i / kRotatePieces];
    index = t.first + static_cast<int>(i % kRotatePieces) * kRotateRows;
    n = min(t.len - index, kRotateRows);
    row = static_cast<int64_t>(t.row0) + index;
  }
};

// A lane's part of one head of one token.  STREAM: past the caches (see is_large).
template <int P>
struct Part {
  typedef uint32_t words_t __attribute__((ext_vector_type(P / 2)));
  Raw<P> lo, hi;
  __device__ __forceinline__ void load(const unsigned char* p, int at_lo, int at_hi) {
    lo = gld<Raw<P>>(p + at_lo);
    hi = gld<Raw<P>>(p + at_hi);
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(unsigned char* p, int at_lo, int at_hi) const {
    if (STREAM) {
      words_t l, h;
      __builtin_memcpy(&l, &lo, sizeof(lo));
      __builtin_memcpy(&h, &hi, sizeof(hi));
      __builtin_nontemporal_store(l, (__attribute__((address_space(1))) words_t*)(p + at_lo));
      __builtin_nontemporal_store(h, (__attribute__((address_space(1))) words_t*)(p + at_hi));
    } else {
      gst(p + at_lo, lo);
      gst(p + at_hi, hi);
    }
  }
  __device__ __forceinline__ void get(float (&v)[2 * P]) const {
    lo.get(v);
    hi.get(v + P);
  }
  __device__ __forceinline__ void put(const float (&v)[2 * P]) {
    lo.put(v);
    hi.put(v + P);
  }
};

// ------------------------------------------------------------------ forward
// Queries and keys in work-groups of their own (blockIdx.y), here and in the
// backward pass: twice as many for short calls, one weight (and its gradient)
// in registers at a time.  Bound by memory: 16384 tokens, 32/8 heads of 128, three
// axes 66 us (5.1 TB/s) from memory, 52 where the inputs are in the cache; a
// short call is one round of start, load, store: 8 tokens 5 us.
template <int P, bool INTER, bool NORM, bool STREAM>
__global__ __launch_bounds__(kRotateLanes) void rotate_kernel(const RotateArgs a) {
  __shared__ __align__(16) Angles angles;
  const RotateTensor& t = a.t[blockIdx.y];
  const int slots = kRotateLanes >> a.group_log2, slot = threadIdx.x >> a.group_log2;
  const Place<P, INTER> place(a, threadIdx.x & ((1 << a.group_log2) - 1));
  const int half = a.rotary_dim >> 1, lo = 2 * place.lo, hi = 2 * place.hi;
  const int64_t pieces = int64_t{a.n_tiles} * kRotatePieces;
  float w[2 * P];
  if (NORM) load_weight<P>(t.weight, place.lo, place.hi, w);
  for (int64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const Piece piece(a, i);
    if (piece.n <= 0) continue;
    Walk<2> walk(t, {t.x, t.out}, piece.row, slot, slots, piece.n);
    Part<P> now, next;
    now.load(walk.p[0], lo, hi);
    __syncthreads();  // the last piece's angles are done with
    fill_angles(a, piece.row, piece.index, piece.n, angles);
    __syncthreads();
    while (walk.left > 0) {
      unsigned char* out = walk.p[1];
      const int token = walk.token;
      walk.next();
      next.load(walk.p[0], lo, hi);
      float v[2 * P];
      now.get(v);
      if (NORM) {
        float back;
        const float r = inverse_size<2 * P>(a, place.live, v, back);
#pragma unroll
        for (int k = 0; k < 2 * P; ++k) v[k] = v[k] * r * w[k];
      }
      place.template turn<false>(angles, token * half, v);
      now.put(v);
      if (place.live) now.template store<STREAM>(out, lo, hi);
      now = next;
    }
  }
}

// ----------------------------------------------------------------- backward
// Without a norm the gradient is dz turned back.  The same tokens 101 us (5.0
// TB/s), half of it also in the vector unit: about 250 instructions for a
// lane's 16 elements.  The next head's loads are under way while one is worked
// on (without that 118 us), in 128 registers for four waves to a SIMD.
//
// A lane adds a weight's gradient up in float32 over runs of at most
// kRotateRun heads, and the runs in float64 in LDS (each lane for itself), so
// that the error does not grow with the tokens.
//
// Pieces are dealt out by number, those past a sequence's end among them, so
// sequences much shorter than a tile leave work-groups without work: 16384
// tokens, 8/8 heads of 64, 29 us in sequences of 128 or more, 207 in ones of 8.
template <int P, bool INTER, bool NORM, bool STREAM>
__global__ __launch_bounds__(kRotateLanes, 4) void rotate_backward_kernel(const RotateArgs a) {
  __shared__ __align__(16) Angles angles;
  const RotateTensor& t = a.t[blockIdx.y];
  const int slots = kRotateLanes >> a.group_log2, slot = threadIdx.x >> a.group_log2;
  const Place<P, INTER> place(a, threadIdx.x & ((1 << a.group_log2) - 1));
  const int half = a.rotary_dim >> 1, lo = 2 * place.lo, hi = 2 * place.hi, D = a.head_dim;
  const float share = 1.f / static_cast<float>(D);
  const int64_t pieces = int64_t{a.n_tiles} * kRotatePieces;
  // The lanes' sums of ended runs: all lanes' first places, then the second, ...
  constexpr int LINE = kRotateLanes + 1;
  __shared__ double part[LINE * 2 * P], sums[kRotateLanes];
  float w[2 * P], dw[2 * P];
  if (NORM) load_weight<P>(t.weight, place.lo, place.hi, w);
#pragma unroll
  for (int k = 0; k < 2 * P; ++k) dw[k] = 0.f;
  bool ended = false;
  auto end_run = [&]() {
#pragma unroll
    for (int k = 0; k < 2 * P; ++k) {
      part[k * LINE + threadIdx.x] += dw[k];
      dw[k] = 0.f;
    }
  };
  int run = 0;  // heads of the run so far, at most
  for (int64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const Piece piece(a, i);
    if (piece.n <= 0) continue;
    Walk<3> walk(t, {t.up, t.out, NORM ? t.x : t.up}, piece.row, slot, slots, piece.n);
    Part<P> up, up_next, x, x_next;
    up.load(walk.p[0], lo, hi);
    if (NORM) x.load(walk.p[2], lo, hi);
    if (NORM) {
      const int most = (piece.n * t.heads + slots - 1) / slots;  // heads of the piece to a lane
      if (run + most > kRotateRun) {
        if (!ended) {
          for (int k = 0; k < 2 * P; ++k) part[k * LINE + threadIdx.x] = 0.0;
        }
        ended = true;
        end_run();
        run = 0;
      }
      run = min(run + most, kRotateRun);
    }
    __syncthreads();
    fill_angles(a, piece.row, piece.index, piece.n, angles);
    __syncthreads();
    for (int of_run = 0; walk.left > 0; ++of_run) {
      if (NORM && of_run == kRotateRun) {
        end_run();
        of_run = 0;
      }
      unsigned char* out = walk.p[1];
      const int token = walk.token;
      walk.next();
      up_next.load(walk.p[0], lo, hi);
      if (NORM) x_next.load(walk.p[2], lo, hi);
      float g[2 * P];
      up.get(g);
      place.template turn<true>(angles, token * half, g);
      if (NORM) {
        float v[2 * P], back;
        x.get(v);
        const float r = inverse_size<2 * P>(a, place.live, v, back);
        float along = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * P; ++k) {
          v[k] *= r;
          dw[k] = fmaf(g[k], v[k], dw[k]);
          g[k] *= w[k];
          along = fmaf(g[k], v[k], along);
        }
        along = head_sum(place.live ? along : 0.f, a.group_log2) * share;
        const float scale = r * back;
#pragma unroll
        for (int k = 0; k < 2 * P; ++k) g[k] = scale * fmaf(-along, v[k], g[k]);
        x = x_next;
      }
      up.put(g);
      if (place.live) up.template store<STREAM>(out, lo, hi);
      up = up_next;
    }
  }
  if (!NORM || !t.d_weight) return;
  // This work-group's sums over its lanes, in a fixed order: an element's from
  // every slot, by as many lanes as there are for it.
#pragma unroll
  for (int k = 0; k < 2 * P; ++k) part[k * LINE + threadIdx.x] = (ended ? part[k * LINE + threadIdx.x] : 0.0) + dw[k];
  __syncthreads();
  const int shares = kRotateLanes / D, mine = threadIdx.x / D, d = threadIdx.x - mine * D;
  if (mine < shares) {
    int lane, k;
    Place<P, INTER>::of_element(a, d, lane, k);
    const double* p = part + k * LINE + lane;
    double x = 0.0;
#pragma unroll 8
    for (int v = mine; v < slots; v += shares) x += p[v << a.group_log2];
    sums[threadIdx.x] = x;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    double x = sums[d];
    for (int v = 1; v < shares; ++v) x += sums[v * D + d];
    gst(a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + blockIdx.y) * D + d, static_cast<float>(x));
  }
}

// The weights' gradients from the work-groups' sums, in float64: 8 elements
// of one tensor to a work-group, 128 lanes to four of them.
constexpr int kJoinLanes = 256, kJoinElements = 8;
__global__ __launch_bounds__(kJoinLanes) void rotate_weights_kernel(const RotateArgs a, int groups) {
  constexpr int R = kJoinLanes / (kJoinElements / 4);
  __shared__ double part[R][kJoinElements + 1];
  float* out = a.t[blockIdx.y].d_weight;
  const int e = threadIdx.x % (kJoinElements / 4) * 4, r = threadIdx.x / (kJoinElements / 4), d = blockIdx.x * kJoinElements + e;
  double x[4] = {0.0, 0.0, 0.0, 0.0};
  if (d < a.head_dim && out) {
    const float* p = a.partials + blockIdx.y * a.head_dim + d;
#pragma unroll 8
    for (int i = r; i < groups; i += R) {
      const float4 v = gld<float4>(p + static_cast<int64_t>(i) * 2 * a.head_dim);
      x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) part[r][e + k] = x[k];
  __syncthreads();
  const int o = blockIdx.x * kJoinElements + threadIdx.x;
  if (threadIdx.x >= kJoinElements || o >= a.head_dim || !out) return;
  double sum = 0.0;
#pragma unroll 8
  for (int i = 0; i < R; ++i) sum += part[i][threadIdx.x];
  gst(out + o, static_cast<float>(sum));
}

uint32_t groups_of(const RotateArgs& a, int64_t most) {
  const int64_t pieces = int64_t{a.n_tiles} * kRotatePieces;
  return static_cast<uint32_t>(pieces < most ? pieces : most);
}

template <int P, bool INTER, bool NORM, bool STREAM>
void launch(const RotateArgs& a, bool back, hipStream_t s) {
  if (back)
    hipLaunchKernelGGL((rotate_backward_kernel<P, INTER, NORM, STREAM>), dim3(groups_of(a, kRotateGroups), 2),
                       dim3(kRotateLanes), 0, s, a);
  else
    hipLaunchKernelGGL((rotate_kernel<P, INTER, NORM, STREAM>), dim3(groups_of(a, 1 << 20), 2), dim3(kRotateLanes), 0, s, a);
}
template <int P, bool INTER>
void launch(const RotateArgs& a, bool norm, bool large, bool back, hipStream_t s) {
  if (norm) large ? launch<P, INTER, true, true>(a, back, s) : launch<P, INTER, true, false>(a, back, s);
  else large ? launch<P, INTER, false, true>(a, back, s) : launch<P, INTER, false, false>(a, back, s);
}

}  // namespace

hipError_t launch_rotate(const RotateArgs& a, const RotateForm& f, hipStream_t s) {
  if (a.n_tiles > 0) {
    if (f.wide) f.interleaved ? launch<8, true>(a, f.norm, f.large, f.back, s) : launch<8, false>(a, f.norm, f.large, f.back, s);
    else f.interleaved ? launch<4, true>(a, f.norm, f.large, f.back, s) : launch<4, false>(a, f.norm, f.large, f.back, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.t[0].d_weight && !a.t[1].d_weight) return hipSuccess;
  hipLaunchKernelGGL(rotate_weights_kernel, dim3((a.head_dim + kJoinElements - 1) / kJoinElements, 2), dim3(kJoinLanes), 0, s,
                     a, static_cast<int>(groups_of(a, kRotateGroups)));
  return hipGetLastError();
}

}  // namespace muon
