// The causal attention kernels' instances (attn_kernels.h).
#include "attn_kernels.h"

namespace muon {

hipError_t launch_attention(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return a.head_dim == 64 ? forward<64, true, false>(a, s) : forward<64, false, false>(a, s);
  return a.head_dim == 128 ? forward<128, true, false>(a, s) : forward<128, false, false>(a, s);
}

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return a.head_dim == 64 ? backward<64, true, false>(a, s) : backward<64, false, false>(a, s);
  return a.head_dim == 128 ? backward<128, true, false>(a, s) : backward<128, false, false>(a, s);
}

}  // namespace muon
