// attn_tree_bf16.cu -- attention of a tree of drafted tokens (attn_tree.cuh) over a
// cache of bf16 rows.
#include "attn_tree.cuh"

namespace attn {

cudaError_t launch_decode_tree_bf16(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                                    const TreePlan& plan, void* workspace, const LaunchCtx& ctx) {
  return launch_tree_fmt<kCacheBf16>(pb, maps, plan, workspace, ctx);
}

int tree_tile_keys(int d) { return d == 128 ? TCfg<kCacheBf16, 128>::BN : TCfg<kCacheBf16, 64>::BN; }
int tree_min_tiles() { return kMinTreeTiles; }

}  // namespace attn
