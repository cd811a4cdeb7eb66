// attn_tree_int8.cu -- attention of a tree of drafted tokens (attn_tree.cuh) over a
// cache of int8 rows.
#include "attn_tree.cuh"

namespace attn {

cudaError_t launch_decode_tree_int8(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                                    const TreePlan& plan, void* workspace, const LaunchCtx& ctx) {
  return launch_tree_fmt<kCacheInt8>(pb, maps, plan, workspace, ctx);
}

}  // namespace attn
