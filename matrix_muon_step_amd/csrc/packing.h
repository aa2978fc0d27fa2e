// A packing's host side and the checks of the calls that take one.
#pragma once

#include "api_common.h"
#include "attn_internal.h"

// The device table holds two orders of the same work items: by falling number
// of keys (a query tile sees the keys before it) and by falling number of
// queries (a key tile is seen by the queries after it), so that the longest
// items start first.
struct muon_packing_s {
  int device;
  int64_t tokens;
  int64_t n_tiles;
  const muon::AttnTile* by_query;
  const muon::AttnTile* by_key;
  uintptr_t lo, hi;  // the table's bytes
  int64_t longest;   // tokens of the longest sequence
  int64_t chunks;    // kFarRows chunks of all sequences
};

namespace muon {

// The tensors of a call with what the checks need of them.
struct Tensor {
  const muon_heads_t* v;
  int64_t heads;
  bool writable;
  const char* name;
};

// Pointers, strides and overlaps of a call's tensors and other buffers.
muon_status_t check_tensors(const std::vector<Tensor>& ts, int64_t tokens, int64_t dim, const std::vector<Range>& others);
// Whether the packing's table is on the current device.
muon_status_t check_device(muon_packing_t packing);

inline HeadsView view(const muon_heads_t& t) {
  return {static_cast<unsigned char*>(t.data), t.token_stride, t.head_stride};
}

}  // namespace muon
