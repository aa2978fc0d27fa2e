// C ABI of the 8-bit activation checkpoints: validation, launch plan.
#include <string.h>

#include <algorithm>

#include "api_common.h"
#include "ckpt_internal.h"

using namespace muon;

namespace {

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
int64_t blocks_of(int64_t tokens, int64_t cols) { return tiles(tokens, kCkTile) * tiles(cols, kCkTile); }
size_t checkpoint_bytes(int64_t tokens, int64_t cols) {
  return align_up(std::max<size_t>(1, static_cast<size_t>(blocks_of(tokens, cols)) * (kCkBlockBytes + 1)));
}

muon_status_t check_size(int64_t tokens, int64_t cols, const std::string& id) {
  if (tokens < 0 || cols < 1) return fail(MUON_ERR_INVALID_ARG, id + " has tokens < 0 or cols < 1");
  if (tokens > MUON_MAX_TOKENS) return fail(MUON_ERR_UNSUPPORTED, id + ": tokens exceed MUON_MAX_TOKENS");
  if (cols > MUON_MAX_DIM) return fail(MUON_ERR_UNSUPPORTED, id + ": cols exceed MUON_MAX_DIM");
  return MUON_OK;
}

muon_status_t check_count(const void* items, int64_t n) {
  if (n < 0) return fail(MUON_ERR_INVALID_ARG, "muon: n < 0");
  if (n > 0 && !items) return fail(MUON_ERR_INVALID_ARG, "muon: the item array is NULL");
  if (n > (1 << 20)) return fail(MUON_ERR_UNSUPPORTED, "muon: more than 2^20 items");
  return MUON_OK;
}

muon_status_t move_all(const muon_checkpoint_t* items, int64_t n, bool write, void* stream) {
  muon_status_t st = check_count(items, n);
  if (st != MUON_OK) return st;
  std::vector<Range> rs;
  for (int64_t i = 0; i < n; ++i) {
    const muon_checkpoint_t& m = items[i];
    const std::string id = "muon: checkpoint " + std::to_string(i);
    st = check_size(m.tokens, m.cols, id);
    if (st != MUON_OK) return st;
    if (m.x_dtype != MUON_F32 && m.x_dtype != MUON_BF16)
      return fail(MUON_ERR_INVALID_ARG, id + ": x_dtype must be MUON_F32 or MUON_BF16");
    if (m.x_stride < m.cols) return fail(MUON_ERR_INVALID_ARG, id + ": x_stride is smaller than cols");
    if (m.x_stride > (int64_t{1} << 40)) return fail(MUON_ERR_UNSUPPORTED, id + ": x_stride too large");
    if (m.tokens == 0) continue;
    if (!m.x || !m.data) return fail(MUON_ERR_INVALID_ARG, id + " has a NULL x or data");
    const uintptr_t es = m.x_dtype == MUON_F32 ? 4 : 2;
    const uintptr_t x = reinterpret_cast<uintptr_t>(m.x), p = reinterpret_cast<uintptr_t>(m.data);
    if (x % es || p % kAlign) return fail(MUON_ERR_ALIGN, id + ": x or data is misaligned");
    rs.push_back({x, x + es * static_cast<uintptr_t>((m.tokens - 1) * m.x_stride + m.cols), !write, "x", i});
    rs.push_back({p, p + checkpoint_bytes(m.tokens, m.cols), write, "data", i});
  }
  st = check_aliasing(rs);
  if (st != MUON_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  CkBatch b;
  memset(&b, 0, sizeof(b));
  auto flush = [&]() -> muon_status_t {
    if (b.n == 0) return MUON_OK;
    const hipError_t e = write ? launch_ckpt_write(b, s) : launch_ckpt_read(b, s);
    memset(&b, 0, sizeof(b));
    return e == hipSuccess ? MUON_OK : hip_fail(e, "checkpoint launch");
  };
  for (int64_t i = 0; i < n; ++i) {
    const muon_checkpoint_t& m = items[i];
    if (m.tokens == 0) continue;
    const int64_t nS = tiles(m.cols, kCkTile), groups = tiles(m.cols, kCkGroupCols);
    const int64_t work = tiles(m.tokens, kCkTile) * groups;
    if (work > (int64_t{1} << 31) - 1) return fail(MUON_ERR_UNSUPPORTED, "muon: checkpoint too large for one launch");
    if (b.n == kCkBatch || b.prefix[b.n] + work > (int64_t{1} << 31) - 1) {
      st = flush();
      if (st != MUON_OK) return st;
    }
    CkDesc& d = b.d[b.n];
    d.x = static_cast<unsigned char*>(m.x);
    d.stride = m.x_stride;
    d.codes = static_cast<unsigned char*>(m.data);
    d.exps = d.codes + blocks_of(m.tokens, m.cols) * kCkBlockBytes;
    d.tokens = static_cast<int32_t>(m.tokens);
    d.cols = static_cast<int32_t>(m.cols);
    d.blocks = static_cast<int32_t>(nS);
    d.groups = static_cast<int32_t>(groups);
    d.f32 = m.x_dtype == MUON_F32;
    b.prefix[b.n + 1] = b.prefix[b.n] + work;
    ++b.n;
  }
  return flush();
}

// How a matrix's product is laid out: tiles of G, parts of the token range.
struct GradPlan {
  int64_t mt, nt, splits, per_split;
  size_t part_bytes;
};

GradPlan plan_grad(const muon_checkpoint_grad_t& m, int64_t call_tiles) {
  GradPlan p;
  p.mt = tiles(m.outs, kGradTile);
  p.nt = tiles(m.cols, kGradTile);
  const int64_t steps = tiles(m.tokens, 32);
  // Calls with fewer tiles than the 256 compute units split the token range
  // so that every unit has one, in parts of at least 16 steps.
  int64_t want = std::max<int64_t>(1, 256 / std::max<int64_t>(1, call_tiles));
  want = std::min(want, std::max<int64_t>(1, steps / 16));
  p.per_split = std::max<int64_t>(1, tiles(steps, want));
  p.splits = std::max<int64_t>(1, tiles(steps, p.per_split));
  p.part_bytes = p.splits > 1 ? align_up(static_cast<size_t>(p.splits) * m.outs * m.cols * sizeof(float)) : 0;
  return p;
}

int64_t total_tiles(const muon_checkpoint_grad_t* mats, int64_t n) {
  int64_t t = 0;
  for (int64_t i = 0; i < n; ++i) t += tiles(mats[i].outs, kGradTile) * tiles(mats[i].cols, kGradTile);
  return t;
}

muon_status_t check_grads(const muon_checkpoint_grad_t* mats, int64_t n) {
  muon_status_t st = check_count(mats, n);
  if (st != MUON_OK) return st;
  for (int64_t i = 0; i < n; ++i) {
    const muon_checkpoint_grad_t& m = mats[i];
    const std::string id = "muon: gradient " + std::to_string(i);
    st = check_size(m.tokens, m.cols, id);
    if (st != MUON_OK) return st;
    if (m.outs < 1) return fail(MUON_ERR_INVALID_ARG, id + " has outs < 1");
    if (m.outs > MUON_MAX_DIM) return fail(MUON_ERR_UNSUPPORTED, id + ": outs exceed MUON_MAX_DIM");
    if (m.g_dtype != MUON_F32 && m.g_dtype != MUON_BF16)
      return fail(MUON_ERR_INVALID_ARG, id + ": g_dtype must be MUON_F32 or MUON_BF16");
    if (m.accumulate != 0 && m.accumulate != 1) return fail(MUON_ERR_INVALID_ARG, id + ": accumulate must be 0 or 1");
    if (m.dy_stride < m.outs) return fail(MUON_ERR_INVALID_ARG, id + ": dy_stride is smaller than outs");
    if (m.dy_stride > MUON_MAX_TOKEN_STRIDE)
      return fail(MUON_ERR_UNSUPPORTED, id + ": dy_stride exceeds MUON_MAX_TOKEN_STRIDE");
  }
  return MUON_OK;
}

}  // namespace

extern "C" {

size_t muon_checkpoint_bytes(int64_t tokens, int64_t cols) {
  size_t bytes = 0;
  guarded([&] {
    const muon_status_t st = check_size(tokens, cols, "muon: checkpoint");
    if (st == MUON_OK) bytes = checkpoint_bytes(tokens, cols);
    return st;
  });
  return bytes;
}

muon_status_t muon_checkpoint_write(const muon_checkpoint_t* items, int64_t n, void* stream) {
  return guarded([&] { return move_all(items, n, true, stream); });
}

muon_status_t muon_checkpoint_read(const muon_checkpoint_t* items, int64_t n, void* stream) {
  return guarded([&] { return move_all(items, n, false, stream); });
}

size_t muon_checkpoint_grad_workspace_bytes(const muon_checkpoint_grad_t* mats, int64_t n) {
  size_t bytes = 0;
  guarded([&] {
    const muon_status_t st = check_grads(mats, n);
    if (st != MUON_OK) return st;
    const int64_t all = total_tiles(mats, n);
    for (int64_t i = 0; i < n; ++i) bytes += plan_grad(mats[i], all).part_bytes;
    return MUON_OK;
  });
  return bytes;
}

muon_status_t muon_checkpoint_grad(const muon_checkpoint_grad_t* mats, int64_t n, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    muon_status_t st = check_grads(mats, n);
    if (st != MUON_OK) return st;
    const int64_t all = total_tiles(mats, n);
    std::vector<GradPlan> plans;
    std::vector<Range> rs;
    size_t need = 0;
    for (int64_t i = 0; i < n; ++i) {
      const muon_checkpoint_grad_t& m = mats[i];
      const std::string id = "muon: gradient " + std::to_string(i);
      plans.push_back(plan_grad(m, all));
      need += plans.back().part_bytes;
      if (!m.G || (m.tokens > 0 && (!m.dy || !m.data)))
        return fail(MUON_ERR_INVALID_ARG, id + " has a NULL dy, data or G");
      const uintptr_t dy = reinterpret_cast<uintptr_t>(m.dy), p = reinterpret_cast<uintptr_t>(m.data);
      const uintptr_t g = reinterpret_cast<uintptr_t>(m.G);
      if (g % 16 || (m.tokens > 0 && (dy % 2 || p % kAlign)))
        return fail(MUON_ERR_ALIGN, id + ": dy, data or G is misaligned");
      const uintptr_t es = m.g_dtype == MUON_F32 ? 4 : 2;
      rs.push_back({g, g + es * static_cast<uintptr_t>(m.outs * m.cols), true, "G", i});
      if (m.tokens > 0) {
        rs.push_back({dy, dy + 2 * static_cast<uintptr_t>((m.tokens - 1) * m.dy_stride + m.outs), false, "dy", i});
        rs.push_back({p, p + checkpoint_bytes(m.tokens, m.cols), false, "data", i});
      }
    }
    const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
    if (need > 0) {
      if (!workspace || workspace_bytes < need)
        return fail(MUON_ERR_WORKSPACE, "muon: the gradients need " + std::to_string(need) + " bytes of workspace");
      if (ws % kAlign) return fail(MUON_ERR_WORKSPACE, "muon: workspace must be 256-byte aligned");
      rs.push_back({ws, ws + need, true, "workspace", 0});
    }
    st = check_aliasing(rs);
    if (st != MUON_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    unsigned char* part = static_cast<unsigned char*>(workspace);
    // Two kinds of launches: dY read in 16-byte direct loads, or any way.
    std::vector<unsigned char*> parts(n);
    for (int64_t i = 0; i < n; ++i) {
      parts[i] = part;
      part += plans[i].part_bytes;
    }
    for (int kind = 0; kind < 2; ++kind) {
      GradBatch b;
      memset(&b, 0, sizeof(b));
      auto flush = [&]() -> muon_status_t {
        if (b.n == 0) return MUON_OK;
        hipError_t e = launch_ckpt_grad(b, kind == 0, s);
        if (e == hipSuccess && b.sums[b.n] > 0) e = launch_grad_join(b, s);
        memset(&b, 0, sizeof(b));
        return e == hipSuccess ? MUON_OK : hip_fail(e, "gradient launch");
      };
      for (int64_t i = 0; i < n; ++i) {
        const muon_checkpoint_grad_t& m = mats[i];
        const bool aligned = reinterpret_cast<uintptr_t>(m.dy) % 16 == 0 && m.dy_stride % 8 == 0;
        if (aligned != (kind == 0)) continue;
        if (m.tokens == 0 && m.accumulate) continue;
        const GradPlan& p = plans[i];
        GradDesc& d = b.d[b.n];
        d.dy = static_cast<const unsigned char*>(m.dy);
        d.dy_stride = m.dy_stride;
        d.codes = static_cast<const unsigned char*>(m.data);
        d.exps = d.codes + blocks_of(m.tokens, m.cols) * kCkBlockBytes;
        d.G = static_cast<unsigned char*>(m.G);
        d.part = reinterpret_cast<float*>(parts[i]);
        d.tokens = static_cast<int32_t>(m.tokens);
        d.outs = static_cast<int32_t>(m.outs);
        d.cols = static_cast<int32_t>(m.cols);
        d.blocks = static_cast<int32_t>(tiles(m.cols, kCkTile));
        d.mt = static_cast<int32_t>(p.mt);
        d.nt = static_cast<int32_t>(p.nt);
        d.splits = static_cast<int32_t>(p.splits);
        d.per_split = static_cast<int32_t>(p.per_split);
        d.g_f32 = m.g_dtype == MUON_F32;
        d.accumulate = m.accumulate;
        b.prefix[b.n + 1] = b.prefix[b.n] + static_cast<int32_t>(p.mt * p.nt * p.splits);
        b.sums[b.n + 1] =
            b.sums[b.n] + (p.splits > 1 ? static_cast<int32_t>(tiles(m.outs * m.cols, kGradSumElems)) : 0);
        if (++b.n == kGradBatch) {
          st = flush();
          if (st != MUON_OK) return st;
        }
      }
      st = flush();
      if (st != MUON_OK) return st;
    }
    return MUON_OK;
  });
}

}  // extern "C"
