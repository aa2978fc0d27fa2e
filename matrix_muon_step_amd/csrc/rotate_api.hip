// C ABI of the norms of queries and keys with rotary positions: validation, launches.
#include <string.h>

#include "packing.h"
#include "rotate_internal.h"

using namespace muon;

namespace {

struct Call {
  const muon_qk_rotate_t* a;
  const muon_heads_t *up[2];  // backward: gradients of the outputs
  float* d_weight[2];
  bool backward;
  const muon_heads_t& x(int i) const { return i ? a->k : a->q; }
  const muon_heads_t& out(int i) const { return i ? a->k_out : a->q_out; }
  const float* weight(int i) const { return i ? a->k_weight : a->q_weight; }
  int32_t heads(int i) const { return i ? a->kv_heads : a->heads; }
};

muon_status_t check_rotary(const muon_rotary_t& r, int32_t head_dim) {
  if (r.rotary_dim < 0 || r.rotary_dim > head_dim || r.rotary_dim % 8 != 0)
    return fail(MUON_ERR_UNSUPPORTED, "muon: rotary_dim must be a multiple of 8 from 0 to head_dim");
  if (r.axes < 1 || r.axes > MUON_MAX_AXES)
    return fail(MUON_ERR_INVALID_ARG, "muon: axes must be 1 to MUON_MAX_AXES");
  if (r.rotary_dim > 0 && !r.frequency) return fail(MUON_ERR_INVALID_ARG, "muon: rotary frequencies are NULL");
  for (int i = 0; i < r.rotary_dim / 2; ++i) {
    if (!isfinite(r.frequency[i]) || fabs(r.frequency[i]) > MUON_MAX_FREQUENCY)
      return fail(MUON_ERR_INVALID_ARG, "muon: rotary frequency " + std::to_string(i) +
                                            " is not finite or beyond MUON_MAX_FREQUENCY");
    if (r.axis && (r.axis[i] < 0 || r.axis[i] >= r.axes))
      return fail(MUON_ERR_INVALID_ARG, "muon: the axis of rotary pair " + std::to_string(i) + " is not below axes");
  }
  return MUON_OK;
}

bool same_view(const muon_heads_t& a, const muon_heads_t& b) {
  return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

// Turns per position times 2^64, modulo 2^64: whole turns fall out.  In 80
// bits (64 of them significant): off by at most 2^-64 turns where |f| < 1.
uint64_t turns_of(double frequency) {
  long double t = static_cast<long double>(fabs(frequency)) * 0.159154943091895335768883763372514362L;  // 1 / 2 pi
  t -= static_cast<long double>(static_cast<int64_t>(t));
  t *= 0x1p64L;
  const uint64_t u = t + 0.5L < 0x1p64L ? static_cast<uint64_t>(t + 0.5L) : 0;
  return frequency < 0 ? 0 - u : u;
}

muon_status_t check(const Call& c, muon_packing_t packing, const std::vector<Range>& more) {
  const muon_qk_rotate_t& a = *c.a;
  if (!packing) return fail(MUON_ERR_INVALID_ARG, "muon: packing is NULL");
  if (a.heads < 1 || a.kv_heads < 1) return fail(MUON_ERR_INVALID_ARG, "muon: heads and kv_heads must be >= 1");
  if (a.heads > MUON_MAX_HEADS || a.kv_heads > MUON_MAX_HEADS)
    return fail(MUON_ERR_UNSUPPORTED, "muon: more than MUON_MAX_HEADS heads");
  if (a.head_dim < 8 || a.head_dim > kAttnMaxDim || a.head_dim % 8 != 0)
    return fail(MUON_ERR_UNSUPPORTED, "muon: head_dim must be a multiple of 8 from 8 to 128");
  muon_status_t st = check_rotary(a.rotary, a.head_dim);
  if (st != MUON_OK) return st;
  if (a.norm) {
    if (!finite(a.eps) || !(a.eps >= 0x1p-126f))
      return fail(MUON_ERR_INVALID_ARG, "muon: eps must be finite and at least 2^-126");
  } else if (a.q_weight || a.k_weight) {
    return fail(MUON_ERR_INVALID_ARG, "muon: weights without a norm");
  }
  for (int i = 0; i < 2; ++i)
    if (c.d_weight[i] && !c.weight(i))
      return fail(MUON_ERR_INVALID_ARG, "muon: a gradient of weights that are NULL");
  std::vector<Range> others = more;
  auto add = [&](const void* p, int64_t bytes, uintptr_t align, bool writable, const char* what) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo % align) return fail(MUON_ERR_ALIGN, std::string("muon: ") + what + " is misaligned");
    others.push_back({lo, lo + static_cast<uintptr_t>(bytes), writable, what, 0});
    return MUON_OK;
  };
  for (int i = 0; i < 2; ++i) {
    // one weight may serve both
    if (c.weight(i) && (i == 0 || c.weight(1) != c.weight(0))) {
      st = add(c.weight(i), 4 * a.head_dim, 4, false, i ? "k_weight" : "q_weight");
      if (st != MUON_OK) return st;
    }
    if (c.d_weight[i]) {
      st = add(c.d_weight[i], 4 * a.head_dim, 4, true, i ? "d_k_weight" : "d_q_weight");
      if (st != MUON_OK) return st;
    }
  }
  const int64_t tokens = packing->tokens;
  if (a.positions && tokens > 0 && a.rotary.rotary_dim > 0) {
    if (a.position_bits != 32 && a.position_bits != 64)
      return fail(MUON_ERR_INVALID_ARG, "muon: position_bits must be 32 or 64");
    if (a.position_stride != 0 && (a.position_stride < tokens || a.position_stride > (int64_t{1} << 40)))
      return fail(MUON_ERR_INVALID_ARG, "muon: position_stride must be 0 or the packing's tokens to 2^40");
    const int width = a.position_bits / 8;
    st = add(a.positions, ((a.rotary.axes - 1) * a.position_stride + tokens) * width, width, false, "positions");
    if (st != MUON_OK) return st;
  }
  others.push_back({packing->lo, packing->hi, false, "the packing's table", 0});
  std::vector<Tensor> ts;
  static const char* const names[2][3] = {{"q", "q_out", "d_q"}, {"k", "k_out", "d_k"}};
  static const char* const back_names[2][3] = {{"q", "dq", "d_q_out"}, {"k", "dk", "d_k_out"}};
  const auto& name = c.backward ? back_names : names;
  for (int i = 0; i < 2; ++i) {
    // an output may be its own input: every element is read before it is written
    const bool reads_x = !c.backward || a.norm;
    if (reads_x && !same_view(c.x(i), c.out(i))) ts.push_back({&c.x(i), c.heads(i), false, name[i][0]});
    if (c.backward && !same_view(*c.up[i], c.out(i))) ts.push_back({c.up[i], c.heads(i), false, name[i][2]});
    ts.push_back({&c.out(i), c.heads(i), true, name[i][1]});
  }
  if (tokens > 0) return check_tensors(ts, tokens, a.head_dim, others);
  // no tensor is looked at, but the weights' gradients are written
  return check_aliasing(others);
}

// Whether a lane can hold eight pairs (16-byte accesses) rather than four: 16384
// tokens, 32/8 heads of 128, forward / gradient 53 / 107 us with eight, 55 / 125 with
// four; 8192 tokens, 16/2 heads of 80, 12.9 / 23.2 and 12.4 / 26.5.
bool is_wide(const muon_qk_rotate_t& a) {
  return a.rotary.rotary_dim % 16 == 0 && (a.head_dim - a.rotary.rotary_dim) % 16 == 0;
}

RotateArgs arguments(const Call& c, muon_packing_t packing) {
  const muon_qk_rotate_t& a = *c.a;
  RotateArgs r;
  memset(&r, 0, sizeof(r));
  const int lanes = a.head_dim / (is_wide(a) ? 16 : 8);
  while ((1 << r.group_log2) < lanes) ++r.group_log2;
  const int slots = kRotateLanes >> r.group_log2;
  for (int i = 0; i < 2; ++i) {
    RotateTensor& t = r.t[i];
    t.x = view(c.x(i));
    t.out = view(c.out(i));
    if (c.backward) t.up = view(*c.up[i]);
    t.weight = c.weight(i);
    t.d_weight = c.d_weight[i];
    t.heads = c.heads(i);
    t.step_token = slots / t.heads;
    t.step_head = slots % t.heads;
  }
  r.tiles = packing->by_query;
  r.n_tiles = static_cast<int32_t>(packing->n_tiles);
  r.head_dim = a.head_dim;
  r.rotary_dim = a.rotary.rotary_dim;
  r.eps = a.eps;
  r.positions = a.positions;
  r.positions_64 = a.position_bits == 64;
  r.position_stride = a.position_stride;
  for (int i = 0; i < a.rotary.rotary_dim / 2; ++i) {
    r.frequency[i] = turns_of(a.rotary.frequency[i]);
    r.axis[i] = static_cast<uint8_t>(a.rotary.axis ? a.rotary.axis[i] : 0);
  }
  return r;
}

// Whether the tensors of a call are more than the memory-side cache holds.
bool is_large(const Call& c, int64_t tokens) {
  const int64_t tensors = c.backward && c.a->norm ? 3 : 2;
  return tensors * tokens * (c.a->heads + c.a->kv_heads) * c.a->head_dim * 2 > kRotateLarge;
}

hipError_t launch(const Call& c, muon_packing_t packing, float* partials, void* stream) {
  RotateArgs r = arguments(c, packing);
  r.partials = partials;
  return launch_rotate(r, {c.backward, is_wide(*c.a), c.a->rotary.interleaved != 0, c.a->norm != 0, is_large(c, packing->tokens)},
                       static_cast<hipStream_t>(stream));
}

size_t partial_bytes(int32_t head_dim) { return align_up(static_cast<size_t>(kRotateGroups) * 2 * head_dim * sizeof(float)); }

}  // namespace

extern "C" {

muon_status_t muon_qk_norm_rotate(const muon_qk_rotate_t* args, muon_packing_t packing, void* stream) {
  return guarded([&] {
    if (!args) return fail(MUON_ERR_INVALID_ARG, "muon: args is NULL");
    const Call c = {args, {nullptr, nullptr}, {nullptr, nullptr}, false};
    muon_status_t st = check(c, packing, {});
    if (st == MUON_OK) st = check_device(packing);
    if (st != MUON_OK || packing->n_tiles == 0) return st;
    const hipError_t e = launch(c, packing, nullptr, stream);
    return e == hipSuccess ? MUON_OK : hip_fail(e, "norm and rotation launch");
  });
}

size_t muon_qk_norm_rotate_backward_workspace_bytes(int32_t head_dim) {
  size_t bytes = 0;
  guarded([&] {
    if (head_dim < 8 || head_dim > kAttnMaxDim || head_dim % 8 != 0)
      return fail(MUON_ERR_UNSUPPORTED, "muon: head_dim must be a multiple of 8 from 8 to 128");
    bytes = partial_bytes(head_dim);
    return MUON_OK;
  });
  return bytes;
}

muon_status_t muon_qk_norm_rotate_backward(const muon_qk_rotate_t* args, const muon_heads_t* d_q_out,
                                           const muon_heads_t* d_k_out, float* d_q_weight, float* d_k_weight,
                                           muon_packing_t packing, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!args || !d_q_out || !d_k_out) return fail(MUON_ERR_INVALID_ARG, "muon: args or an upstream gradient is NULL");
    const Call c = {args, {d_q_out, d_k_out}, {d_q_weight, d_k_weight}, true};
    std::vector<Range> more;
    const bool sums = d_q_weight || d_k_weight;
    if (sums && args->head_dim >= 8 && args->head_dim <= kAttnMaxDim) {
      const size_t need = partial_bytes(args->head_dim);
      if (!workspace || workspace_bytes < need)
        return fail(MUON_ERR_WORKSPACE, "muon: the weights' gradients need " + std::to_string(need) +
                                            " bytes of workspace");
      const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
      if (ws % kAlign) return fail(MUON_ERR_WORKSPACE, "muon: workspace must be 256-byte aligned");
      more.push_back({ws, ws + need, true, "the workspace", 0});
    }
    muon_status_t st = check(c, packing, more);
    if (st == MUON_OK) st = check_device(packing);
    if (st != MUON_OK || (packing->n_tiles == 0 && !sums)) return st;
    const hipError_t e = launch(c, packing, static_cast<float*>(workspace), stream);
    return e == hipSuccess ? MUON_OK : hip_fail(e, "norm and rotation backward launch");
  });
}

}  // extern "C"
