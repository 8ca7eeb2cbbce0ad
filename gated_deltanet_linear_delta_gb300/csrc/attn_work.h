// attn_work.h -- host side of the attention's work division (attn_join.cu)
#pragma once

#include "gdn_internal.h"

namespace gdn {

struct AttnWork;
AttnWork attn_work(const AttnArgs &a, int tokens_per_tile, int min_shift);
int attn_ctas(const AttnArgs &a, const AttnWork &w, int BN);
cudaError_t launch_attn_join(const AttnArgs &a, const AttnWork &w, int ctas, cudaStream_t s);

}  // namespace gdn
