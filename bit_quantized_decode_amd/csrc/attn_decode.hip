// Attention of one new token per sequence over the paged cache (nvfp4_attn_decode).
#include "attn_kernel.h"

namespace nvfp4 {

bool attn_fits(const AttnLaunch& a) { return places_of(a) < (int64_t(1) << 31); }

size_t attn_workspace_bytes(const AttnLaunch& a) { return kCounterBytes + part_bytes_of(a); }

hipError_t launch_attn_decode(const AttnLaunch& a, hipStream_t s) {
  ModeParams<kPlain> p;
  fill_params(a, p);
  return attn_launch(a, p, s);
}

}  // namespace nvfp4
