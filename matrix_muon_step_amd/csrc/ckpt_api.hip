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

// Work-groups of 256 lanes that a launch takes: fewer than 2^32 lanes.
constexpr int64_t kMaxGroups = int64_t{1} << 24;

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
    // (the extent in bytes stays far below 2^63)
    if (m.x_stride > (int64_t{1} << 40) || m.x_stride > (int64_t{1} << 56) / std::max<int64_t>(1, m.tokens))
      return fail(MUON_ERR_UNSUPPORTED, id + ": x_stride too large");
    if (m.tokens == 0) continue;
    if (tiles(m.tokens, kCkTile) * tiles(m.cols, kCkGroupCols) >= kMaxGroups)
      return fail(MUON_ERR_UNSUPPORTED, id + " is too large for one launch");
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
    if (b.n == kCkBatch || b.prefix[b.n] + work >= kMaxGroups) {
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
    d.rblocks = static_cast<int32_t>(tiles(m.tokens, kCkTile));
    d.groups = static_cast<int32_t>(groups);
    d.f32 = m.x_dtype == MUON_F32;
    b.prefix[b.n + 1] = b.prefix[b.n] + work;
    ++b.n;
  }
  return flush();
}

// How a launch of gradients is laid out.
struct GradPlan {
  int cfg;
  int64_t parts;   // 0: a work-group per tile
  int64_t share;   // steps of a part
  size_t bytes;    // of its pieces
};

constexpr int64_t kUnits = 256;  // compute units

// The cheapest of three layouts, by what they measured (us; a step is 32
// tokens of a tile):
//   256-tiles, one work-group of 8 waves to a unit: 6 + 0.85 a step
//     (1600 x 6400 from 16384 tokens, 175 tiles: 438)
//   128-tiles, up to three work-groups of 4 waves to a unit, which together
//     take 0.27 a step each: 8 + that (the same matrix, 650 tiles: 403; three
//     1600 x 1600 from 8192 tokens, 507 tiles: 154 against 217 with 147
//     256-tiles; but 2048 x 7168 from 777 tokens 40 against 30)
//   the work in 256-tiles cut into equal shares, one to a unit: 1.0 a step
//     with every unit busy, the pieces (256 KB each, written and read, at 4.5
//     TB/s) and a second launch (1600 x 6400: 404)
// What the model chooses against each layout forced, us (256 | 128 | shares):
//   8192 tokens, 768 x 768 34 (188 | 95 | 43 with all 256 units), three 52 (191 |
//     94 | 52), 1600 x 1600 95 (194 | 95 | 71: it overrates the shares here)
//   4096, 256 x 256 24 (96 | 48 | 77 with all units); 4096 x 1024 51 (100 | 51 | 57)
//   2048, three 768 x 768 27 (53 | 27 | 35); 4096 x 4096 64 (64 | 80 | 66)
//   512, 1600 x 1600 12 (19 | 12 | 30); 300, 768 x 768 9 (13 | 9 | 23)
//   777, four 2048 x 7168 111 (111 | 101 | 147)
//   16384, 768 x 2304 74 (377 | 184 | 74); 65536, 512 x 512 73 (1464 | 732 | 74)
// Matrices without tokens (experts that none was routed to) do not count: a
// launch of either kind stores their zeros.
GradPlan plan_grad(const muon_checkpoint_grad_t* mats, int64_t n) {
  int64_t tiles_of[kNumGradCfg] = {0, 0}, work[kNumGradCfg] = {0, 0}, longest = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t steps = tiles(mats[i].tokens, kCkTile);
    if (steps == 0) continue;
    longest = std::max(longest, steps);
    for (int c = 0; c < kNumGradCfg; ++c) {
      const int64_t t = tiles(mats[i].outs, kGradTile[c]) * tiles(mats[i].cols, kGradTile[c]);
      tiles_of[c] += t;
      work[c] += t * steps;
    }
  }
  // Rounds of items over the units, of items of average length or one of the longest.
  auto whole = [&](int c, double start, int64_t together, double step) {
    const int64_t count = std::max<int64_t>(1, tiles_of[c]);
    const double steps = static_cast<double>(tiles(tiles_of[c], kUnits)) * work[c] / count;
    return start * tiles(count, together * kUnits) + step * std::max(static_cast<double>(longest), steps);
  };
  const double t256 = whole(kGrad256, 6, 1, 0.85), t128 = whole(kGrad128, 8, 3, 0.27);
  const int64_t parts = std::min(kUnits, work[kGrad256] / 16);
  GradPlan p = {t256 <= t128 ? kGrad256 : kGrad128, 0, 0, 0};
  if (parts > 1) {
    const double pieces = static_cast<double>(parts + std::min<int64_t>(parts, tiles_of[kGrad256]));
    const double cut = 6 + 1.0 * tiles(work[kGrad256], parts) + pieces * 0.524 / 4.5 + 5.0;
    if (cut < std::min(t256, t128)) {
      p.cfg = kGrad256;
      p.share = tiles(work[kGrad256], parts);
      p.parts = tiles(work[kGrad256], p.share);
    }
  }
  if (p.parts) p.bytes = align_up(static_cast<size_t>(p.parts) * 2 * kGradTile[p.cfg] * kGradTile[p.cfg] * sizeof(float));
  return p;
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
    for (int64_t i = 0; i < n; i += kGradBatch)
      bytes = std::max(bytes, plan_grad(mats + i, std::min<int64_t>(kGradBatch, n - i)).bytes);
    return MUON_OK;
  });
  return bytes;
}

muon_status_t muon_checkpoint_grad(const muon_checkpoint_grad_t* mats, int64_t n, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    muon_status_t st = check_grads(mats, n);
    if (st != MUON_OK) return st;
    std::vector<Range> rs;
    size_t need = 0;
    for (int64_t i = 0; i < n; i += kGradBatch)
      need = std::max(need, plan_grad(mats + i, std::min<int64_t>(kGradBatch, n - i)).bytes);
    for (int64_t i = 0; i < n; ++i) {
      const muon_checkpoint_grad_t& m = mats[i];
      const std::string id = "muon: gradient " + std::to_string(i);
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
    // Launches follow one another on the stream and share the workspace.
    for (int64_t i0 = 0; i0 < n; i0 += kGradBatch) {
      const int64_t count = std::min<int64_t>(kGradBatch, n - i0);
      const GradPlan plan = plan_grad(mats + i0, count);
      GradBatch b;
      memset(&b, 0, sizeof(b));
      b.parts = static_cast<int32_t>(plan.parts);
      b.share = plan.share;
      b.pieces = static_cast<float*>(workspace);
      bool aligned = true;
      auto add = [&](const muon_checkpoint_grad_t& m) -> GradDesc& {
        GradDesc& d = b.d[b.all];
        d.dy = static_cast<const unsigned char*>(m.dy);
        d.dy_stride = m.dy_stride;
        d.codes = static_cast<const unsigned char*>(m.data);
        d.exps = d.codes + blocks_of(m.tokens, m.cols) * kCkBlockBytes;
        d.G = static_cast<unsigned char*>(m.G);
        d.tokens = static_cast<int32_t>(m.tokens);
        d.outs = static_cast<int32_t>(m.outs);
        d.cols = static_cast<int32_t>(m.cols);
        d.blocks = static_cast<int32_t>(tiles(m.cols, kCkTile));
        d.mt = static_cast<int32_t>(tiles(m.outs, kGradTile[plan.cfg]));
        d.steps = static_cast<int32_t>(tiles(m.tokens, kCkTile));
        d.g_f32 = m.g_dtype == MUON_F32;
        d.accumulate = m.accumulate;
        return d;
      };
      for (int64_t i = i0; i < i0 + count; ++i) {
        const muon_checkpoint_grad_t& m = mats[i];
        if (m.tokens == 0) continue;
        aligned = aligned && reinterpret_cast<uintptr_t>(m.dy) % 16 == 0 && m.dy_stride % 8 == 0;
        const GradDesc& d = add(m);
        const int64_t t = d.mt * tiles(m.cols, kGradTile[plan.cfg]);
        b.tiles[b.n + 1] = b.tiles[b.n] + static_cast<int32_t>(t);
        b.steps[b.n + 1] = b.steps[b.n] + t * d.steps;
        b.all = ++b.n;
      }
      for (int64_t i = i0; i < i0 + count; ++i) {
        const muon_checkpoint_grad_t& m = mats[i];
        if (m.tokens > 0 || m.accumulate) continue;
        add(m);
        const int64_t bytes = m.outs * m.cols * (m.g_dtype == MUON_F32 ? 4 : 2);
        b.tiles[b.all + 1] = b.tiles[b.all] + static_cast<int32_t>(tiles(bytes, kGradZeros));
        ++b.all;
      }
      if (b.all == 0) continue;
      hipError_t e = launch_ckpt_grad(b, plan.cfg, aligned, s);
      if (e == hipSuccess && b.parts) e = launch_grad_join(b, s);
      if (e != hipSuccess) return hip_fail(e, "gradient launch");
    }
    return MUON_OK;
  });
}

}  // extern "C"
