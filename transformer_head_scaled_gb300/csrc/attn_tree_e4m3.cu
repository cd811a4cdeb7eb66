// attn_tree_e4m3.cu -- attention of a tree of drafted tokens (attn_tree.cuh) over a
// cache of e4m3 rows.
#include "attn_tree.cuh"

namespace attn {

cudaError_t launch_decode_tree_e4m3(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                                    const TreePlan& plan, void* workspace, const LaunchCtx& ctx) {
  return launch_tree_fmt<kCacheE4M3>(pb, maps, plan, workspace, ctx);
}

}  // namespace attn
