// C ABI of the global gradient norm and of clipping: validation, batches, launches.
#include <string.h>

#include <algorithm>
#include <utility>

#include "api_common.h"
#include "grad_internal.h"

using namespace muon;

namespace {

constexpr size_t kBytes = kNormGroups * sizeof(double);
// Chunks of a launch stay far inside 32 bits.
constexpr int64_t kMaxChunks = int64_t{1} << 30;

size_t width(int32_t dtype) { return dtype == MUON_F32 ? 4 : 2; }

int64_t chunks_of(int64_t count) { return (count + kNormChunk - 1) / kNormChunk; }

// Checks the tensors and collects their ranges; `clip`: their outputs too.
muon_status_t check_items(const muon_gradient_t* items, int64_t n, bool clip, std::vector<Range>& rs) {
  if (n < 0 || (n > 0 && !items)) return fail(MUON_ERR_INVALID_ARG, "muon: gradients missing or n < 0");
  for (int64_t i = 0; i < n; ++i) {
    const muon_gradient_t& t = items[i];
    const std::string id = "muon: gradient " + std::to_string(i);
    if (t.count < 0) return fail(MUON_ERR_INVALID_ARG, id + " has a negative count");
    if (t.count > MUON_MAX_GRADIENT) return fail(MUON_ERR_UNSUPPORTED, id + " has more than MUON_MAX_GRADIENT elements");
    if ((t.g_dtype != MUON_F32 && t.g_dtype != MUON_BF16) ||
        (clip && t.out_dtype != MUON_F32 && t.out_dtype != MUON_BF16))
      return fail(MUON_ERR_INVALID_ARG, id + ": unknown dtype");
    if (t.count == 0) continue;
    if (!t.g || (clip && !t.out)) return fail(MUON_ERR_INVALID_ARG, id + " has a NULL g or out");
    const uintptr_t g = reinterpret_cast<uintptr_t>(t.g), o = reinterpret_cast<uintptr_t>(t.out);
    if (g % width(t.g_dtype) || (clip && o % width(t.out_dtype)))
      return fail(MUON_ERR_ALIGN, id + ": g or out is not aligned to its element");
    const bool in_place = clip && g == o && t.g_dtype == t.out_dtype;
    if (!in_place) rs.push_back({g, g + width(t.g_dtype) * static_cast<uintptr_t>(t.count), false, "g", i});
    if (clip) rs.push_back({o, o + width(t.out_dtype) * static_cast<uintptr_t>(t.count), true, "out", i});
  }
  return MUON_OK;
}

muon_status_t check_workspace(void* workspace, size_t bytes, std::vector<Range>& rs) {
  if (!workspace || bytes < kBytes)
    return fail(MUON_ERR_WORKSPACE, "muon: the gradient norm needs " + std::to_string(kBytes) + " bytes of workspace");
  const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
  if (ws % kAlign) return fail(MUON_ERR_WORKSPACE, "muon: workspace must be 256-byte aligned");
  rs.push_back({ws, ws + kBytes, true, "workspace", -1});
  return MUON_OK;
}

muon_status_t check_norm(const double* norm, bool written, std::vector<Range>& rs) {
  if (!norm) return fail(MUON_ERR_INVALID_ARG, "muon: norm is NULL");
  const uintptr_t p = reinterpret_cast<uintptr_t>(norm);
  if (p % 8) return fail(MUON_ERR_ALIGN, "muon: norm is not 8-byte aligned");
  rs.push_back({p, p + 8, written, "norm", -1});
  return MUON_OK;
}

// A call's tensors in launches.
class Batches {
 public:
  Batches(const muon_gradient_t* items, int64_t n) : items_(items), n_(n) {
    for (int64_t i = 0; i < n; ++i) bytes_ += items[i].count * static_cast<int64_t>(width(items[i].g_dtype));
  }
  // The next launch's tensors, from item i on with `before` bytes in front of
  // it (both moved past them); false at the end.
  bool next(int64_t& i, int64_t& before, NormBatch& b) const {
    b.n = b.stream = 0;
    b.large = bytes_ > kNormKeep;
    b.chunks[0] = 0;
    for (; i < n_ && b.n < kNormBatch; ++i) {
      const muon_gradient_t& t = items_[i];
      if (t.count == 0) continue;
      const int64_t chunks = chunks_of(t.count), end = b.chunks[b.n] + chunks;
      if (end > kMaxChunks) break;  // the first of a launch fits: MUON_MAX_GRADIENT
      const int64_t w = static_cast<int64_t>(width(t.g_dtype));
      // whole chunks of this tensor that lie in front of the last kNormKeep bytes
      const int64_t stream = (bytes_ - kNormKeep - before) / (kNormChunk * w);
      if (stream > 0) b.stream = static_cast<int32_t>(b.chunks[b.n] + std::min(stream, chunks));
      before += t.count * w;
      b.d[b.n] = {static_cast<const unsigned char*>(t.g), static_cast<unsigned char*>(t.out), t.count,
                  t.g_dtype == MUON_F32, t.out_dtype == MUON_F32};
      b.chunks[++b.n] = static_cast<int32_t>(end);
    }
    return b.n > 0;
  }

 private:
  const muon_gradient_t* items_;
  int64_t n_, bytes_ = 0;
};

// Sums of squares into the workspace; how many partials there are.
hipError_t squares(const Batches& all, double* partials, hipStream_t s, int* count) {
  NormBatch b;
  *count = 0;
  for (int64_t i = 0, before = 0; all.next(i, before, b);) {
    b.earlier = *count;
    const hipError_t e = launch_grad_squares(b, partials, s);
    if (e != hipSuccess) return e;
    *count = std::max(*count, std::min(b.chunks[b.n], kNormGroups));
  }
  return hipSuccess;
}

}  // namespace

extern "C" {

size_t muon_grad_norm_workspace_bytes(void) { return kBytes; }

muon_status_t muon_grad_norm(const muon_gradient_t* items, int64_t n, double* norm, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return guarded([&] {
    std::vector<Range> rs;
    muon_status_t st = check_items(items, n, false, rs);
    if (st == MUON_OK) st = check_norm(norm, true, rs);
    if (st == MUON_OK) st = check_workspace(workspace, workspace_bytes, rs);
    if (st == MUON_OK) st = check_aliasing(rs);
    if (st != MUON_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    double* partials = static_cast<double*>(workspace);
    int count = 0;
    hipError_t e = squares(Batches(items, n), partials, s, &count);
    if (e == hipSuccess) e = launch_grad_norm(partials, count, norm, s);
    return e == hipSuccess ? MUON_OK : hip_fail(e, "gradient norm launch");
  });
}

muon_status_t muon_grad_clip(const muon_gradient_t* items, int64_t n, double max_norm, double* norm, int32_t norm_given,
                             void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!isfinite(max_norm) || !(max_norm > 0.0))
      return fail(MUON_ERR_INVALID_ARG, "muon: max_norm must be finite and > 0");
    std::vector<Range> rs;
    muon_status_t st = check_items(items, n, true, rs);
    if (st == MUON_OK) st = check_norm(norm, !norm_given, rs);
    if (st == MUON_OK && !norm_given) st = check_workspace(workspace, workspace_bytes, rs);
    if (st == MUON_OK) st = check_aliasing(rs);
    if (st != MUON_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    double* partials = static_cast<double*>(workspace);
    int count = -1;
    hipError_t e = hipSuccess;
    const Batches all(items, n);
    if (!norm_given) e = squares(all, partials, s, &count);
    if (e == hipSuccess && count == 0) e = launch_grad_norm(partials, 0, norm, s);
    // the last launch's tensors first: they were read last
    std::vector<std::pair<int64_t, int64_t>> starts;
    NormBatch b;
    std::pair<int64_t, int64_t> at = {0, 0};
    for (auto end = at; all.next(end.first, end.second, b); at = end) starts.push_back(at);
    for (auto it = starts.rbegin(); it != starts.rend() && e == hipSuccess; ++it) {
      all.next(it->first, it->second, b);
      e = launch_grad_clip(b, partials, count, norm, max_norm, s);
    }
    return e == hipSuccess ? MUON_OK : hip_fail(e, "gradient clip launch");
  });
}

}  // extern "C"
