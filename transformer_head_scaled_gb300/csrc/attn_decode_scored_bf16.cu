// attn_decode_scored_bf16.cu -- the decoding step with changed scores
// (attn_decode_scored.cuh) for a cache of bf16 rows.
#include "attn_decode_scored.cuh"

namespace attn {

cudaError_t launch_decode_scored_bf16(const ScoredDecodeProblem& pb, const ScoredDecodePlan& plan,
                                    float* workspace, const LaunchCtx& ctx) {
  return launch_scored_decode_fmt<kCacheBf16>(pb, plan, workspace, ctx);
}

}  // namespace attn
