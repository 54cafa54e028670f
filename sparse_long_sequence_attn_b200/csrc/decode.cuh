// Host entry of the few-token paged attention (decode.cu).
#pragma once

#include "attn_args.cuh"

namespace longnet {
bool decode_supports(const AttnArgs& a);
int64_t decode_workspace_floats(const AttnArgs& a, bool weights);
int launch_decode(const AttnArgs& a, float* workspace, float* weights, cudaStream_t stream);
}  // namespace longnet
