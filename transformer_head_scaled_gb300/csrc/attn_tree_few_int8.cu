// attn_tree_few_int8.cu -- the decoding step (attn_decode_scored.cuh) for trees of
// drafted tokens with few query rows to a key head, over a cache of int8 rows.
#include "attn_decode_scored.cuh"

namespace attn {

cudaError_t launch_tree_few_int8(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                 const ScoredDecodePlan& plan, float* workspace,
                                 const LaunchCtx& ctx, const TreeOwn& tree) {
  return launch_scored_decode_fmt<kCacheInt8, true>(pb, maps, plan, workspace, ctx, &tree);
}

}  // namespace attn
