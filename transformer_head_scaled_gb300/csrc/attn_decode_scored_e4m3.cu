// attn_decode_scored_e4m3.cu -- the decoding step with changed scores
// (attn_decode_scored.cuh) for a cache of e4m3 rows.
#include "attn_decode_scored.cuh"

namespace attn {

cudaError_t launch_decode_scored_e4m3(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                    const ScoredDecodePlan& plan, float* workspace,
                                    const LaunchCtx& ctx) {
  return launch_scored_decode_fmt<kCacheE4M3>(pb, maps, plan, workspace, ctx);
}

}  // namespace attn
