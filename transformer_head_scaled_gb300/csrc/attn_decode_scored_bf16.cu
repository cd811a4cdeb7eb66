// attn_decode_scored_bf16.cu -- the decoding step with changed scores
// (attn_decode_scored.cuh) for a cache of bf16 rows.
#include "attn_decode_scored.cuh"

namespace attn {

cudaError_t launch_decode_scored_bf16(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                    const ScoredDecodePlan& plan, float* workspace,
                                    const LaunchCtx& ctx) {
  return launch_scored_decode_fmt<kCacheBf16>(pb, maps, plan, workspace, ctx);
}

bool scored_decode_big(int row_bytes, int row_tile, bool whole) {
  return scored_big_tiles(row_bytes, row_tile / 8, whole);
}
int scored_decode_tile_keys(int row_bytes, bool big) { return scored_tile_keys(row_bytes, big); }
int scored_decode_warps(int row_bytes, int row_tile, bool big) {
  return DW * scored_ctas(row_bytes, row_tile / 8, big);
}
int scored_decode_min_tiles() { return kMinTiles; }

}  // namespace attn
