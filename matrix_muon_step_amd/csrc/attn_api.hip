// C ABI of the attention operators: packings, argument validation, launches.
#include <string.h>

#include <algorithm>
#include <memory>

#include "packing.h"

using namespace muon;

namespace {

muon_status_t count_tiles(const int64_t* lengths, int64_t n, int64_t* tokens, int64_t* tiles) {
  if (n < 0 || (n > 0 && !lengths)) return fail(MUON_ERR_INVALID_ARG, "muon: packing lengths missing or n < 0");
  int64_t sum = 0, count = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (lengths[i] < 0) return fail(MUON_ERR_INVALID_ARG, "muon: packing length " + std::to_string(i) + " is negative");
    if (lengths[i] > MUON_MAX_SEQUENCE)
      return fail(MUON_ERR_UNSUPPORTED, "muon: packing length " + std::to_string(i) + " exceeds MUON_MAX_SEQUENCE");
    if (lengths[i] > MUON_MAX_TOKENS - sum)
      return fail(MUON_ERR_UNSUPPORTED, "muon: a packing holds at most MUON_MAX_TOKENS tokens");
    sum += lengths[i];
    count += (lengths[i] + kAttnRows - 1) / kAttnRows;
  }
  *tokens = sum;
  *tiles = count;
  return MUON_OK;
}

size_t table_bytes_of(int64_t tiles) { return align_up(std::max<size_t>(1, 2 * sizeof(AttnTile) * tiles)); }

muon_status_t check_shape(int32_t heads, int32_t kv_heads, int32_t head_dim, float scale, muon_packing_t packing) {
  if (!packing) return fail(MUON_ERR_INVALID_ARG, "muon: packing is NULL");
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    return fail(MUON_ERR_INVALID_ARG, "muon: heads must be a positive multiple of kv_heads");
  if (heads > MUON_MAX_HEADS) return fail(MUON_ERR_UNSUPPORTED, "muon: more than MUON_MAX_HEADS heads");
  if (head_dim < 8 || head_dim > kAttnMaxDim || head_dim % 8 != 0)
    return fail(MUON_ERR_UNSUPPORTED, "muon: head_dim must be a multiple of 8 from 8 to 128");
  if (!finite(scale) || !(scale > 0.f)) return fail(MUON_ERR_INVALID_ARG, "muon: scale must be finite and > 0");
  // the kernels' exponentials are of base 2
  if (!finite(scale * kAttnLog2e)) return fail(MUON_ERR_UNSUPPORTED, "muon: scale * log2(e) is no float32 number");
  // a launch takes fewer than 2^32 lanes, a work-group up to 512
  if (packing->n_tiles * heads >= MUON_MAX_ATTENTION_ITEMS)
    return fail(MUON_ERR_UNSUPPORTED, "muon: too many work items (128-row pieces of the sequences x heads)");
  return MUON_OK;
}

// Elements from a tensor's first to one past its last.
int64_t extent(const Tensor& t, int64_t tokens, int64_t dim) {
  return (tokens - 1) * t.v->token_stride + (t.heads - 1) * t.v->head_stride + dim;
}

// True when no element of a is one of b although their extents overlap: both
// repeat with period m (elements), and within it their spans are apart.
bool apart_modulo(const Tensor& a, const Tensor& b, int64_t m, int64_t tokens, int64_t dim) {
  if (m <= 0) return false;
  int64_t span[2];
  const Tensor* t[2] = {&a, &b};
  for (int i = 0; i < 2; ++i) {
    if (tokens > 1 && t[i]->v->token_stride % m != 0) return false;
    const bool repeats = t[i]->heads == 1 || t[i]->v->head_stride % m == 0;
    span[i] = repeats ? dim : (t[i]->heads - 1) * t[i]->v->head_stride + dim;
    if (span[i] > m) return false;
  }
  const int64_t ea = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.v->data) / 2);
  const int64_t eb = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.v->data) / 2);
  const int64_t d = ((eb - ea) % m + m) % m;
  return d >= span[0] && d + span[1] <= m;
}

muon_status_t check_lse(const float* lse, int64_t stride, int64_t tokens, int64_t heads, bool writable,
                        std::vector<Range>& out) {
  if (tokens == 0) return MUON_OK;
  if (!lse) return fail(MUON_ERR_INVALID_ARG, "muon: attention lse is NULL");
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(MUON_ERR_ALIGN, "muon: attention lse is not 4-byte aligned");
  if (stride < tokens) return fail(MUON_ERR_INVALID_ARG, "muon: lse_stride is smaller than the packing's tokens");
  if (stride > (int64_t{1} << 40)) return fail(MUON_ERR_UNSUPPORTED, "muon: lse_stride too large");
  const uintptr_t p = reinterpret_cast<uintptr_t>(lse);
  out.push_back({p, p + 4 * static_cast<uintptr_t>((heads - 1) * stride + tokens), writable, "lse", 0});
  return MUON_OK;
}

// What rows see: every key before them, or a window and the first tokens.
struct Window {
  int64_t window;  // 0: none
  int64_t sinks;
};

muon_status_t check_window(const Window* w) {
  if (!w) return MUON_OK;
  if (w->window < 1) return fail(MUON_ERR_INVALID_ARG, "muon: window must be >= 1");
  if (w->sinks < 0) return fail(MUON_ERR_INVALID_ARG, "muon: sinks must be >= 0");
  if (w->sinks > MUON_MAX_SINKS) return fail(MUON_ERR_UNSUPPORTED, "muon: more than MUON_MAX_SINKS sinks");
  return MUON_OK;
}

// Whether the window hides any key of the packing's sequences.
bool hides(const Window* w, muon_packing_t p) { return w && w->window < p->longest; }

// Sets what the kernels need of the window; false where the causal kernels serve.
bool set_window(AttnArgs& a, const Window* w, muon_packing_t p) {
  a.longest = static_cast<int32_t>(p->longest);
  if (!hides(w, p)) return false;
  a.window = static_cast<int32_t>(w->window);
  a.sinks = static_cast<int32_t>(w->sinks);
  a.longest = static_cast<int32_t>(std::min<int64_t>(p->longest, w->window + w->sinks + kAttnRows));
  return true;
}

int64_t row_stride(muon_packing_t p) { return round_up(std::max<int64_t>(p->tokens, 1), 64); }

// Whether the backward pass sums over rows beyond their windows.
bool has_far(const Window* w, muon_packing_t p) { return hides(w, p) && w->sinks > 0; }

size_t row_bytes(int32_t heads, muon_packing_t p) {
  return align_up(static_cast<size_t>(row_stride(p)) * heads * 2 * sizeof(float));
}

size_t far_bytes(const muon_attention_grad_t& g, const Window* w, muon_packing_t p) {
  if (!has_far(w, p)) return 0;
  return align_up(static_cast<size_t>(p->chunks) * g.kv_heads * 2 * static_cast<size_t>(w->sinks) * g.head_dim * sizeof(float));
}

size_t part_bytes(const muon_attention_grad_t& g, muon_packing_t p, int32_t parts) {
  return parts == 1 ? 0 : static_cast<size_t>(p->n_tiles) * g.kv_heads * parts * 2 * kAttnRows * g.head_dim * sizeof(float);
}

// Work-groups that share a key tile's query heads in dK/dV, where key tiles
// are few.  One holds a compute unit (of 256) for about 6 us and, for each tile
// of rows and head, 2.4 us (heads of up to 64: 1.3); shares cost a launch and
// their float32 sums, written and read again.  Backward pass in us, one
// work-group | this many: 8/1 heads of 128, 4096 tokens, window 1024 265 | 88
// (8); 8192, window 4096 1027 | 464 (4); 16/4 of 128, 4096, window 1024 180 | 139
// (2), window 256 119 | 112 (2); 32/8 of 128, 2048, window 64 107 | 90 (2); 8192
// tokens of 32/4 (256 key tiles), window 256 270 | 297 (2).
int32_t key_parts(const muon_attention_grad_t& g, const Window* w, muon_packing_t p) {
  if (!hides(w, p)) return 1;
  const int32_t group = g.heads / g.kv_heads;
  const int64_t items = p->n_tiles * g.kv_heads;
  const double turns =
      static_cast<double>((std::min<int64_t>(p->longest, kAttnRows - 1 + w->window) + kAttnStep - 1) / kAttnStep);
  auto time = [&](int32_t parts) {
    const double rounds = static_cast<double>((items * parts + 255) / 256);
    const double turn = g.head_dim > 64 ? 2.4 : 1.3, share = (group + parts - 1) / parts;
    const double join = parts > 1 ? 4.0 + 2e-6 * static_cast<double>(part_bytes(g, p, parts)) / 12 : 0.0;
    return rounds * (6.0 + turns * share * turn) + join;
  };
  int32_t best = 1;
  for (int32_t parts = 2; parts <= std::min(group, 8); ++parts)
    if (time(parts) < 0.9 * time(best)) best = parts;
  return best;
}

size_t backward_bytes(const muon_attention_grad_t& g, const Window* w, muon_packing_t p) {
  return row_bytes(g.heads, p) + far_bytes(g, w, p) + part_bytes(g, p, key_parts(g, w, p));
}

}  // namespace

namespace muon {

muon_status_t check_tensors(const std::vector<Tensor>& ts, int64_t tokens, int64_t dim,
                            const std::vector<Range>& others) {
  if (tokens == 0) return MUON_OK;  // nothing is read or written
  for (const Tensor& t : ts) {
    const muon_heads_t& v = *t.v;
    auto refuse = [&](muon_status_t st, const char* why) {
      return fail(st, std::string("muon: tensor ") + t.name + why);
    };
    if (!v.data) return refuse(MUON_ERR_INVALID_ARG, " is NULL");
    if (v.token_stride < 0 || v.head_stride < 0) return refuse(MUON_ERR_INVALID_ARG, " has a negative stride");
    if ((reinterpret_cast<uintptr_t>(v.data) & 15u) || v.token_stride % 8 != 0 || v.head_stride % 8 != 0)
      return refuse(MUON_ERR_ALIGN, ": data must be 16-byte aligned and strides multiples of 8");
    if (v.token_stride > MUON_MAX_TOKEN_STRIDE)
      return refuse(MUON_ERR_UNSUPPORTED, ": token_stride exceeds MUON_MAX_TOKEN_STRIDE");
    if (v.head_stride > (int64_t{1} << 48)) return refuse(MUON_ERR_UNSUPPORTED, ": head_stride too large");
  }
  for (const Tensor& t : ts) {
    if (!t.writable) continue;
    const int64_t a = t.v->token_stride, b = t.v->head_stride;
    const bool tok_major = (t.heads == 1 || b >= dim) && (tokens == 1 || a >= (t.heads - 1) * b + dim);
    const bool head_major = (tokens == 1 || a >= dim) && (t.heads == 1 || b >= (tokens - 1) * a + dim);
    if (!tok_major && !head_major)
      return fail(MUON_ERR_ALIAS, std::string("muon: output ") + t.name + " overlaps itself");
  }
  auto lo = [](const Tensor& t) { return reinterpret_cast<uintptr_t>(t.v->data); };
  auto hi = [&](const Tensor& t) { return lo(t) + 2 * static_cast<uintptr_t>(extent(t, tokens, dim)); };
  auto clash = [&](const char* x, const char* y) {
    return fail(MUON_ERR_ALIAS, std::string("muon: ") + x + " overlaps " + y);
  };
  for (size_t i = 0; i < ts.size(); ++i) {
    for (size_t j = i + 1; j < ts.size(); ++j) {
      const Tensor &a = ts[i], &b = ts[j];
      if (!a.writable && !b.writable) continue;
      if (hi(a) <= lo(b) || hi(b) <= lo(a)) continue;
      const bool tok = a.v->token_stride == b.v->token_stride && apart_modulo(a, b, a.v->token_stride, tokens, dim);
      const bool head = a.v->head_stride == b.v->head_stride && apart_modulo(a, b, a.v->head_stride, tokens, dim);
      if (!tok && !head) return clash(a.name, b.name);
    }
    for (const Range& r : others)
      if ((r.writable || ts[i].writable) && r.lo < hi(ts[i]) && lo(ts[i]) < r.hi) return clash(ts[i].name, r.what);
  }
  for (size_t i = 0; i < others.size(); ++i)
    for (size_t j = i + 1; j < others.size(); ++j)
      if ((others[i].writable || others[j].writable) && others[i].lo < others[j].hi && others[j].lo < others[i].hi)
        return clash(others[i].what, others[j].what);
  return MUON_OK;
}

muon_status_t check_device(muon_packing_t packing) {
  if (packing->n_tiles == 0) return MUON_OK;
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev != packing->device)
    return fail(MUON_ERR_INVALID_ARG, "muon: the packing belongs to device " + std::to_string(packing->device) +
                                          ", the current device is " + std::to_string(dev));
  return MUON_OK;
}

}  // namespace muon

namespace {

// Workspace that a forward pass can use: its items' largest logits.
size_t forward_bytes(const muon_attention_t& g, const Window* w, muon_packing_t p) {
  const int64_t items = p->n_tiles * g.heads;
  return g.max_logit && hides(w, p) && items >= kTopItems ? align_up(static_cast<size_t>(items) * sizeof(float)) : 0;
}

muon_status_t attention(const muon_attention_t* args, const Window* w, muon_packing_t packing, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!args) return fail(MUON_ERR_INVALID_ARG, "muon: args is NULL");
  const muon_attention_t& g = *args;
  muon_status_t st = check_shape(g.heads, g.kv_heads, g.head_dim, g.scale, packing);
  if (st != MUON_OK) return st;
  st = check_window(w);
  if (st != MUON_OK) return st;
  std::vector<Range> others;
  if (workspace) {
    const size_t need = forward_bytes(g, w, packing);
    const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
    if (workspace_bytes < need)
      return fail(MUON_ERR_WORKSPACE, "muon: the attention needs " + std::to_string(need) + " bytes of workspace, or none");
    if (ws % kAlign) return fail(MUON_ERR_WORKSPACE, "muon: workspace must be 256-byte aligned");
    if (need > 0) others.push_back({ws, ws + need, true, "the workspace", 0});
    else workspace = nullptr;
  }
  st = check_lse(g.lse, g.lse_stride, packing->tokens, g.heads, true, others);
  if (st != MUON_OK) return st;
  if (g.max_logit) {
    if (reinterpret_cast<uintptr_t>(g.max_logit) & 3u)
      return fail(MUON_ERR_ALIGN, "muon: attention max_logit is not 4-byte aligned");
    if (g.logit_heads != g.heads && g.logit_heads != g.kv_heads)
      return fail(MUON_ERR_INVALID_ARG, "muon: logit_heads must be heads or kv_heads");
    const uintptr_t p = reinterpret_cast<uintptr_t>(g.max_logit);
    others.push_back({p, p + 4 * static_cast<uintptr_t>(g.logit_heads), true, "max_logit", 0});
  }
  others.push_back({packing->lo, packing->hi, false, "the packing's table", 0});
  st = check_tensors({{&g.q, g.heads, false, "q"}, {&g.k, g.kv_heads, false, "k"}, {&g.v, g.kv_heads, false, "v"},
                      {&g.o, g.heads, true, "o"}},
                     packing->tokens, g.head_dim, others);
  if (st != MUON_OK) return st;
  st = check_device(packing);
  if (st != MUON_OK || packing->n_tiles == 0) return st;
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = view(g.q);
  a.k = view(g.k);
  a.v = view(g.v);
  a.o = view(g.o);
  a.lse = g.lse;
  a.lse_stride = g.lse_stride;
  a.max_logit = g.max_logit;
  a.logit_group = g.max_logit ? g.heads / g.logit_heads : 1;
  a.heads = g.heads;
  a.kv_heads = g.kv_heads;
  a.head_dim = g.head_dim;
  a.scale = g.scale;
  a.by_query = packing->by_query;
  a.by_key = packing->by_key;
  a.n_tiles = static_cast<int32_t>(packing->n_tiles);
  const bool windowed = set_window(a, w, packing);
  a.tops = static_cast<float*>(workspace);
  const hipError_t e = (windowed ? launch_window_attention : launch_attention)(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MUON_OK : hip_fail(e, "attention launch");
}

size_t attention_backward_bytes(const muon_attention_grad_t* args, const Window* w, muon_packing_t packing) {
  size_t bytes = 0;
  guarded([&] {
    if (!args) return fail(MUON_ERR_INVALID_ARG, "muon: args is NULL");
    muon_status_t st = check_shape(args->heads, args->kv_heads, args->head_dim, args->scale, packing);
    if (st == MUON_OK) st = check_window(w);
    if (st == MUON_OK) bytes = backward_bytes(*args, w, packing);
    return st;
  });
  return bytes;
}

muon_status_t attention_backward(const muon_attention_grad_t* args, const Window* w, muon_packing_t packing,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!args) return fail(MUON_ERR_INVALID_ARG, "muon: args is NULL");
  const muon_attention_grad_t& g = *args;
  muon_status_t st = check_shape(g.heads, g.kv_heads, g.head_dim, g.scale, packing);
  if (st != MUON_OK) return st;
  st = check_window(w);
  if (st != MUON_OK) return st;
  const size_t need = backward_bytes(g, w, packing);
  if (!workspace || workspace_bytes < need)
    return fail(MUON_ERR_WORKSPACE, "muon: the attention backward needs " + std::to_string(need) +
                                        " bytes of workspace");
  const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
  if (ws % kAlign) return fail(MUON_ERR_WORKSPACE, "muon: workspace must be 256-byte aligned");
  std::vector<Range> others;
  st = check_lse(g.lse, g.lse_stride, packing->tokens, g.heads, false, others);
  if (st != MUON_OK) return st;
  others.push_back({ws, ws + need, true, "the workspace", 0});
  others.push_back({packing->lo, packing->hi, false, "the packing's table", 0});
  st = check_tensors({{&g.q, g.heads, false, "q"}, {&g.k, g.kv_heads, false, "k"}, {&g.v, g.kv_heads, false, "v"},
                      {&g.o, g.heads, false, "o"}, {&g.d_o, g.heads, false, "d_o"}, {&g.dq, g.heads, true, "dq"},
                      {&g.dk, g.kv_heads, true, "dk"}, {&g.dv, g.kv_heads, true, "dv"}},
                     packing->tokens, g.head_dim, others);
  if (st != MUON_OK) return st;
  st = check_device(packing);
  if (st != MUON_OK || packing->n_tiles == 0) return st;
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = view(g.q);
  a.k = view(g.k);
  a.v = view(g.v);
  a.o = view(g.o);
  a.d_o = view(g.d_o);
  a.dq = view(g.dq);
  a.dk = view(g.dk);
  a.dv = view(g.dv);
  a.lse = const_cast<float*>(g.lse);  // read only by the backward kernels
  a.lse_stride = g.lse_stride;
  a.row_stride = row_stride(packing);
  a.row_lse2 = static_cast<float*>(workspace);
  a.row_delta = a.row_lse2 + a.row_stride * g.heads;
  a.heads = g.heads;
  a.kv_heads = g.kv_heads;
  a.head_dim = g.head_dim;
  a.scale = g.scale;
  a.by_query = packing->by_query;
  a.by_key = packing->by_key;
  a.n_tiles = static_cast<int32_t>(packing->n_tiles);
  const bool windowed = set_window(a, w, packing);
  if (has_far(w, packing)) {
    a.far = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + row_bytes(g.heads, packing));
    a.far_joined = (packing->longest + kFarRows - 1) / kFarRows - w->window / kFarRows > kFarDirect;
  }
  a.key_parts = key_parts(g, w, packing);
  if (a.key_parts > 1)
    a.parts = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + row_bytes(g.heads, packing) +
                                       far_bytes(g, w, packing));
  const hipError_t e =
      (windowed ? launch_window_attention_backward : launch_attention_backward)(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MUON_OK : hip_fail(e, "attention backward launch");
}

}  // namespace

extern "C" {

size_t muon_packing_bytes(const int64_t* lengths, int64_t n) {
  size_t bytes = 0;
  guarded([&] {
    int64_t tokens = 0, tiles = 0;
    const muon_status_t st = count_tiles(lengths, n, &tokens, &tiles);
    if (st == MUON_OK) bytes = table_bytes_of(tiles);
    return st;
  });
  return bytes;
}

muon_status_t muon_packing_create(const int64_t* lengths, int64_t n, void* table, size_t table_bytes, void* stream,
                                  muon_packing_t* out) {
  return guarded([&] {
    if (!out) return fail(MUON_ERR_INVALID_ARG, "muon: out is NULL");
    *out = nullptr;
    int64_t tokens = 0, tiles = 0;
    const muon_status_t st = count_tiles(lengths, n, &tokens, &tiles);
    if (st != MUON_OK) return st;
    const size_t need = table_bytes_of(tiles);
    if (!table || table_bytes < need)
      return fail(MUON_ERR_WORKSPACE, "muon: the packing table needs " + std::to_string(need) + " bytes");
    if (reinterpret_cast<uintptr_t>(table) % kAlign)
      return fail(MUON_ERR_WORKSPACE, "muon: the packing table must be 256-byte aligned");
    std::vector<AttnTile> all(2 * tiles);
    int64_t k = 0, row0 = 0, chunks = 0;
    for (int64_t i = 0; i < n; ++i) {
      for (int64_t first = 0; first < lengths[i]; first += kAttnRows)
        all[k++] = {static_cast<int32_t>(row0), static_cast<int32_t>(lengths[i]), static_cast<int32_t>(first),
                    static_cast<int32_t>(chunks)};
      row0 += lengths[i];
      chunks += (lengths[i] + kFarRows - 1) / kFarRows;
    }
    std::copy(all.begin(), all.begin() + tiles, all.begin() + tiles);
    std::stable_sort(all.begin(), all.begin() + tiles,
                     [](const AttnTile& a, const AttnTile& b) { return a.first > b.first; });
    std::stable_sort(all.begin() + tiles, all.end(),
                     [](const AttnTile& a, const AttnTile& b) { return a.len - a.first > b.len - b.first; });
    std::unique_ptr<muon_packing_s> p(new muon_packing_s);
    p->device = -1;  // an empty packing needs none
    if (tiles > 0) {
      hipError_t e = hipGetDevice(&p->device);
      if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
      const hipStream_t s = static_cast<hipStream_t>(stream);
      hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
      e = hipStreamIsCapturing(s, &cap);
      if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
      if (cap != hipStreamCaptureStatusNone)
        return fail(MUON_ERR_INVALID_ARG, "muon: a packing cannot be created on a capturing stream");
      e = hipMemcpyAsync(table, all.data(), sizeof(AttnTile) * all.size(), hipMemcpyHostToDevice, s);
      if (e == hipSuccess) e = hipStreamSynchronize(s);
      if (e != hipSuccess) return hip_fail(e, "packing upload");
    }
    p->tokens = tokens;
    p->n_tiles = tiles;
    p->by_query = static_cast<const AttnTile*>(table);
    p->by_key = p->by_query + tiles;
    p->lo = reinterpret_cast<uintptr_t>(table);
    p->hi = p->lo + need;
    p->chunks = chunks;
    p->longest = n > 0 ? *std::max_element(lengths, lengths + n) : 0;
    *out = p.release();
    return MUON_OK;
  });
}

muon_status_t muon_packing_destroy(muon_packing_t packing) {
  g_last_error.clear();
  delete packing;
  return MUON_OK;
}

muon_status_t muon_attention(const muon_attention_t* args, muon_packing_t packing, void* stream) {
  return guarded([&] { return attention(args, nullptr, packing, nullptr, 0, stream); });
}

size_t muon_window_attention_workspace_bytes(const muon_attention_t* args, int64_t window, int64_t sinks,
                                             muon_packing_t packing) {
  const Window w = {window, sinks};
  size_t bytes = 0;
  guarded([&] {
    if (!args) return fail(MUON_ERR_INVALID_ARG, "muon: args is NULL");
    muon_status_t st = check_shape(args->heads, args->kv_heads, args->head_dim, args->scale, packing);
    if (st == MUON_OK) st = check_window(&w);
    if (st == MUON_OK) bytes = forward_bytes(*args, &w, packing);
    return st;
  });
  return bytes;
}

muon_status_t muon_window_attention(const muon_attention_t* args, int64_t window, int64_t sinks, muon_packing_t packing,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const Window w = {window, sinks};
  return guarded([&] { return attention(args, &w, packing, workspace, workspace_bytes, stream); });
}

size_t muon_attention_backward_workspace_bytes(const muon_attention_grad_t* args, muon_packing_t packing) {
  return attention_backward_bytes(args, nullptr, packing);
}

size_t muon_window_attention_backward_workspace_bytes(const muon_attention_grad_t* args, int64_t window, int64_t sinks,
                                                      muon_packing_t packing) {
  const Window w = {window, sinks};
  return attention_backward_bytes(args, &w, packing);
}

muon_status_t muon_attention_backward(const muon_attention_grad_t* args, muon_packing_t packing, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return guarded([&] { return attention_backward(args, nullptr, packing, workspace, workspace_bytes, stream); });
}

muon_status_t muon_window_attention_backward(const muon_attention_grad_t* args, int64_t window, int64_t sinks,
                                             muon_packing_t packing, void* workspace, size_t workspace_bytes,
                                             void* stream) {
  const Window w = {window, sinks};
  return guarded([&] { return attention_backward(args, &w, packing, workspace, workspace_bytes, stream); });
}

}  // extern "C"
