// attn_internal.cuh -- declarations shared by the library's translation
// units (host launchers and the status codes the kernels record).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace attn {

enum MaskKind : int { kMaskNone = 0, kMaskCausal = 1, kMaskKeyPadding = 2, kMaskBand = 3 };

// Written (first error wins) into the library's device status word.
enum DeviceStatus : int { kDevOk = 0, kDevTimeout = 1, kDevWrongPlan = 2 };

// The plan of a mask under which every query sees one run of keys: device
// arrays inside the caller's plan buffer (attn_mask_plan).  Intervals are [x, y).
constexpr int kMaskTile = 128;
// A work item of the forward: 256 queries of a batch entry, the first key that
// any of them sees and the end of those that each half sees (0: none).
struct __align__(16) QueryItem {
  int b, block, first, end[2];
  int work;  // 128-key tiles
  int pad[2];
};
// A work item of the backward: 128 keys, the first 128-query tile that sees any
// of them, and how many tiles do.
struct __align__(16) KeyItem {
  int b, tile, first, count;
};
struct MaskPlan {
  const int4* header;    // n_q, n_k, B, are the items ordered by their work?
  const int2* row_keys;  // [B][n_q] keys of a query
  const int2* key_rows;  // [B][n_k] queries of a key
  // in the order in which they are dealt out, for every head alike
  const QueryItem* query_items;  // [B * ceil(n_q / 256)]
  const KeyItem* key_items;      // [B * ceil(n_k / 128)]
};
constexpr int kMostOrdered = 2048;  // items that a plan orders by their work

// A persistent kernel deals planned items out back and forth: in every second
// round the CTAs take them in reverse, so that who got the heaviest of one round
// gets the lightest of the next.  The step from a CTA's item of an even round to
// its next one; from an odd round it is 2 * gridDim.x less this.
__device__ __forceinline__ int first_step() { return 2 * (gridDim.x - 1 - blockIdx.x) + 1; }
struct MaskLayout {
  size_t row_keys, key_rows, query_items, key_items, query_items_in, key_items_in, runs, bytes;
};
MaskLayout mask_layout(int B, int n_q, int n_k);
MaskPlan mask_plan_at(const void* plan, int B, int n_q, int n_k);

struct MaskProblem {
  int B, n_q, n_k;
  int left, right;  // -1: no bound on that side
  const int* key_lens;
  const int* doc_ids;  // [B][n_q], n_q == n_k
  const int* prefix_lens;
};

// Element strides of a [B, H, n, d] view across batch entries, heads and rows
// (d contiguous).
struct RowStrides {
  long long b, h, n;
};

// Changed scores (attn_fwd_scored, attn_bwd_scored).
struct ScoreMod {
  float softcap;        // 0: none
  const float* slopes;  // device [H] or null
  int group;            // query heads per key head
  MaskPlan plan;
  bool masked;          // whether there is a plan
  // the backward: of q, k, v (a few rows are read with plain loads), dk and dv, and
  // the parts that a key head's query heads are worked on in
  RowStrides sq, sk, sv, sdk, sdv;
  int parts;
};

// Instantiations of the tensor-core kernels: the masks given by lengths (none,
// causal, key padding), the restricted window, and changed scores under a mask
// plan, with a cap (kWide: the backward's for caps above kWideCap) and a distance
// bias or without; each keeps its code out of the others'.
enum Mode : int { kPlain = 0, kBand = 1, kScored = 2, kCap = 4, kBias = 8, kWide = 16 };

// One forward problem, device pointers, [B, H, n, d] contiguous.
struct Problem {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int B, H, n_q, n_k, d;
  float scale;
  int mask;
  const int* key_lens;
  int win_left, win_right;  // kMaskBand: query i sees keys i - win_left .. i + win_right
};

bool mask_plan_ordered(const MaskProblem& pb);
struct LaunchCtx;
cudaError_t launch_mask_plan(const MaskProblem& pb, void* plan, const LaunchCtx& ctx);

// tanh for small arguments: y (kTanh0 + kTanh1 y^2 + kTanh2 y^4), within
// 1.8e-7 of it for |y| <= kTanhSmall, and its derivative kSech0 + kSech1 y^2 +
// kSech2 y^4, within 8e-6 (least-maximum fits over that interval, made for
// this library).  Scores seldom reach 0.3 of a cap, and then need no second
// exponential and no reciprocal.
constexpr double kTanhSmall = 0.3;
constexpr double kTanh0 = 0.99999601, kTanh1 = -0.3329748, kTanh2 = 0.12522591;
constexpr double kSech0 = 0.99999215, kSech1 = -0.99840603, kSech2 = 0.61841958;
// The general form, cap - 2 cap / (1 + e^2y), errs by up to 3e-7 of the cap: above
// this cap that is more than 1e-4 of a score, and small arguments have to take
// the polynomial.
constexpr float kWideCap = 256.f;

// The cap in units of q.k (x) and log2: softcap * log2(e) * tanh(scale * x /
// softcap) = x (poly[0] + poly[1] x^2 + poly[2] x^4) for |x| <= small, and the
// derivative of tanh likewise.
struct CapPoly {
  float small, poly[3], slope[3];
};
inline CapPoly cap_poly(float scale, float softcap) {
  CapPoly c{};
  c.small = -1.f;
  if (!(softcap > 0.f)) return c;
  const double k = static_cast<double>(scale) / softcap;
  const double tanh_of[3] = {kTanh0, kTanh1, kTanh2}, sech_of[3] = {kSech0, kSech1, kSech2};
  double f = 1.0;
  for (int i = 0; i < 3; ++i, f *= k * k) {
    c.poly[i] = static_cast<float>(tanh_of[i] * f * scale * 1.4426950408889634);
    c.slope[i] = static_cast<float>(sech_of[i] * f);
  }
  // (a cap so small that the coefficients overflow is left to the general form)
  if (f < 1e30) c.small = static_cast<float>(kTanhSmall / k);
  return c;
}

// Launch context shared by every launcher.
struct LaunchCtx {
  int num_sms;
  uint64_t limit_ns;  // bounded-wait limit inside kernels
  int* status;        // device address of the status word
  cudaStream_t stream;
};

// Programmatic dependent launch (PTX griddepcontrol): a kernel launched with
// the programmatic stream serialization attribute may start while the kernel
// before it on the stream is still running.  It must pass this wait before it
// touches anything that kernel writes: the wait returns once that grid has
// completed and its memory operations are visible (at once for a kernel
// launched without the attribute).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next kernel on the stream start launching before this grid ends
// (its CTAs still wait in grid_dependency_wait for this grid to complete).
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kernel` with programmatic stream serialization: it may start (and
// run its prologue) while the previous kernel on the stream drains, so the
// kernel must call grid_dependency_wait() before it reads anything the
// previous kernel writes.  Used only for the second and later kernels of one
// library call, whose predecessor on the stream is always that call's own.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                   cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// tcgen05 bf16 path, d in {16, 32, 64, 128}.  The tensor maps describe Q, K,
// V and O as 3-D (d, n, B*H) bf16 tensors with a (min(d, 64), rows, 1) box
// in the widest swizzle a box row fits (128, 64 or 32 bytes); rows = 128 for
// Q and O, fwd_tc_kv_rows(d) for K and V.
// With `mod`: changed scores, under its plan instead of pb's mask; K and V then
// have H / mod->group heads.
cudaError_t launch_fwd_tc(const Problem& pb, const CUtensorMap& tmq, const CUtensorMap& tmk,
                          const CUtensorMap& tmv, const CUtensorMap& tmo, const LaunchCtx& ctx,
                          const ScoreMod* mod = nullptr);
int fwd_tc_kv_rows(int d);

// fp32 SIMT path (d in {16, 32, 64, 128}).
cudaError_t launch_fwd_f32(const Problem& pb, const LaunchCtx& ctx);


// Decode path (n_q <= kDecodeMaxQueries new queries against a cache).
constexpr int kDecodeMaxQueries = 8;

struct DecodeProblem {
  const void* q;        // bf16 [B, H, n_q, d]
  const void* k_cache;  // bf16 [B, H, L_max, d]
  const void* v_cache;
  void* o;              // bf16 [B, H, n_q, d]
  float* lse;           // [B, H, n_q] or null
  int B, H, n_q, L_max, d;  // d in {16, 32, 64, 128}
  float scale;
  const int* cache_lens;  // device int32[B] or null (all L_max valid)
  RowStrides sq, sk, sv, so;  // element strides (batch entry, head, row) of q, k, v, o
  int window = -1;  // restricted self-attention: keys [len - 1 - window, len); -1: all keys
};

// How the cache of each head is split across CTAs; workspace_bytes = 0 when
// one CTA per head suffices.
struct DecodePlan {
  int splits;
  int chunk;  // keys per split, a multiple of the 128-key tile
  size_t workspace_bytes;
};
// L_max: the most keys one query sees (the cache length, or the window's).
DecodePlan decode_plan(int B, int H, int n_q, int L_max, int d, int num_sms);
// maps[0..3] (d = 64; unused for the other head sizes, whose kernel reads the
// cache with plain loads): K cache, V cache as 4-D (64, L_max, H, B) bf16 with
// a (64, 128, 1, 1) box, then the same with a (64, 32, 1, 1) box for partial
// last tiles; all with 128-byte swizzle.  workspace holds plan.workspace_bytes.
cudaError_t launch_decode(const DecodeProblem& pb, const CUtensorMap* maps, const DecodePlan& plan,
                          float* workspace, const LaunchCtx& ctx);

// Backward (d = 16, 32 or 64; bf16): gradients of the forward above.
struct BwdProblem {
  const void* q;     // bf16 [B, H, n_q, d]
  const void* k;     // bf16 [B, H, n_k, d]
  const void* v;
  const void* o;     // the forward's output, bf16 [B, H, n_q, d]
  const void* dout;  // dLoss/dO, bf16 [B, H, n_q, d]
  const float* lse;  // the forward's log-sum-exp [B, H, n_q]
  void* dq;          // bf16 outputs, shaped like q, k, v
  void* dk;
  void* dv;
  int B, H, n_q, n_k, d;
  float scale;
  int mask;
  const int* key_lens;
  int win_left, win_right;  // kMaskBand: query i sees keys i - win_left .. i + win_right
  RowStrides so, sdo, sdq;  // strides of o, dout (read with plain loads) and dq (written so)
};

// Workspace of the backward: the per-query constant tiles (one [128 x 16]
// bf16 tile of 4 KB per 128-query tile and head), then the fp32 dQ
// accumulator [B, H, n_q, d].
struct BwdLayout {
  size_t num_qt, cst_off, dq_acc_off, bytes;
  // with changed scores: LSE * log2(e), padded to whole query tiles, behind them,
  // and who works on which item
  size_t lse_off, deal_off, scored_bytes;
  // and, where key heads' query heads are worked on in parts, those parts' dV and
  // dK in fp32, [dV, dK][part][B, HK, n_k, d]
  size_t part_off;
  int parts = 1;
};
BwdLayout bwd_layout(int B, int H, int n_q, int d);
BwdLayout bwd_scored_layout(int B, int H, int HK, int n_q, int n_k, int d);
bool bwd_head_size_ok(int d);
// With changed scores, D of queries that see at most this many keys comes from P
// and dP, in a kernel of its own, which runs where there may be such queries.
constexpr int kFewKeys = 16;
inline bool bwd_few_possible(bool masked, int n_k) { return masked || n_k <= kFewKeys; }
// maps: Q, K, V, dO as 4-D (d, n, H, B) bf16 with a (d, 128, 1, 1) box; dK,
// dV the same with a (d, 64, 1, 1) box (any strides); the dQ accumulator as 3-D (d, n_q, B*H)
// fp32 with a (min(d, 32), 64, 1) box; each in the swizzle of its box's row
// bytes; with `mod`, the parts of dV and dK the same as 3-D (d, n_k, 2 * parts *
// B*HK).  Three launches (preprocess, main, dQ convert), four with parts.
// With `mod`: changed scores, under its plan instead of pb's mask; the K, V, dK
// and dV maps then have H / mod->group heads.
cudaError_t launch_bwd(const BwdProblem& pb, const CUtensorMap* maps, void* workspace,
                       const LaunchCtx& ctx, const ScoreMod* mod = nullptr);

// New keys and values into an 8-bit cache with a scale per block of tokens.
struct CacheAppendProblem {
  const void* k_new;  // bf16 [B, H, n_new, d]
  const void* v_new;
  void* k_cache;  // 8-bit codes [B, H, L_max, d]
  void* v_cache;
  float* k_scale;  // [B, H, ceil(L_max / block_tokens)]
  float* v_scale;
  int B, H, n_new, L_max, d;
  bool e4m3;  // else int8
  int block_tokens;
  const int* cache_lens;  // device int32[B] or null (empty caches)
  const int* new_lens;    // device int32[B] or null (n_new each)
  RowStrides skn, svn, skc, svc;
};
cudaError_t launch_cache_append(const CacheAppendProblem& pb, const LaunchCtx& ctx);
// Blocks that the new tokens of one sequence can fall into.
int cache_blocks_touched(int n_new, int L_max, int block_tokens);

// The accepted path of a tree of drafted tokens into the caches of all layers.
struct LayerStrides {
  long long layer;
  RowStrides row;
};
struct CacheTreeProblem {
  const void* k_tree;  // bf16 [layers, B, H, n, d]
  const void* v_tree;
  void* k_cache;  // [layers, B, H, L_max, d]: bf16 rows or 8-bit codes
  void* v_cache;
  float* k_scale;  // [layers, B, H, ceil(L_max / block_tokens)]; unused for bf16
  float* v_scale;
  int layers, B, H, n, L_max, d;
  bool bf16, e4m3;
  int block_tokens;
  const int* path;        // [B, n] nodes
  const int* path_lens;   // [B]
  const int* cache_lens;  // device int32[B] or null (empty caches)
  LayerStrides src[2], dst[2];  // of keys and values
};
cudaError_t launch_cache_append_tree(const CacheTreeProblem& pb, const LaunchCtx& ctx);

// A tree of drafted tokens: nodes at most.
constexpr int kMostNodes = 128;

// Which drafted tokens stand, and the token after them.
struct TreeVerifyProblem {
  const void* target;  // probabilities [B, n, V], f32 or bf16
  const void* draft;   // likewise, or null
  const int* tokens;   // [B, n]
  const int* parents;
  const float* uniforms;
  int* path;  // [B, n]
  int* path_lens;
  int* next_tokens;
  int B, n, V;
  long long tb, tn, db, dn;  // element strides of batch entries and nodes
  bool bf16;
};
cudaError_t launch_tree_verify(const TreeVerifyProblem& pb, const LaunchCtx& ctx);

// Attention of a tree's nodes over a cache and their ancestors.
struct TreeDecodeProblem {
  const void* q;  // bf16 [B, H, n, d]
  const void* k_tree;  // bf16 [B, HK, n, d]
  const void* v_tree;
  const void* k_cache;  // [B, HK, L_max, d]
  const void* v_cache;
  const float* k_scale;  // [B, HK, ceil(L_max / block_tokens)]; unused for bf16
  const float* v_scale;
  const int* parents;  // [B, n]
  void* o;
  float* lse;  // or null
  int B, H, HK, n, L_max, d, format, block_tokens;
  float scale, softcap;  // softcap <= 0: none
  const float* slopes;   // device float[H] or null
  const int* cache_lens;  // device int32[B] or null
  int window;  // -1: none
  RowStrides sq, skt, svt, sk, sv, so;
};
struct TreePlan {
  int ctas;
  bool whole;      // a CTA takes whole units (sequence, key head, block of query rows)
  int blocks;      // of query rows of a key head
  int block_rows;  // rows of a part in the workspace
  int tree_tiles;  // tiles of the tree's own keys
  size_t part_off;  // floats before the parts in the workspace
  size_t workspace_bytes;
};
TreePlan tree_plan(int B, int HK, int rows, int n, int L_max, int d, int window, int num_sms);
int tree_tile_keys(int d);
int tree_min_tiles();
// maps: the key and the value cache with a box of a tile's rows (bf16: swizzled as
// the operand of a product; 8 bits: as bytes), then the tree's keys and values.
cudaError_t launch_decode_tree_bf16(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                                    const TreePlan& plan, void* workspace, const LaunchCtx& ctx);
cudaError_t launch_decode_tree_e4m3(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                                    const TreePlan& plan, void* workspace, const LaunchCtx& ctx);
cudaError_t launch_decode_tree_int8(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                                    const TreePlan& plan, void* workspace, const LaunchCtx& ctx);

// Decoding with changed scores against a bf16, e4m3 or int8 cache.
struct ScoredDecodeProblem {
  const void* q;  // bf16 [B, H, n_q, d]
  const void* k_cache;  // [B, HK, L_max, d]
  const void* v_cache;
  const float* k_scale;  // [B, HK, ceil(L_max / block_tokens)]; unused for bf16
  const float* v_scale;
  void* o;
  float* lse;  // or null
  int B, H, HK, n_q, L_max, d, block_tokens;
  float scale, softcap;  // softcap <= 0: none
  const float* slopes;   // device float[H] or null
  const int* cache_lens;  // device int32[B] or null
  int window;  // -1: every key up to the query
  RowStrides sq, sk, sv, so;
};
// Behind the d values of a row's part in the workspace: the scores' maximum, the
// row sum relative to it, what the values are relative to, and one to make them a
// 16-byte load.
constexpr int kPartTail = 4;
struct ScoredDecodePlan {
  int row_tile, row_tiles;  // query rows of one key head per CTA, and how many such tiles
  bool whole;  // a warp takes whole units (sequence, key head, row tile)
  int tile_keys;
  int warps;   // that share the units, or the list of their tiles
  size_t part_off;  // floats before the partial results in the workspace
  size_t workspace_bytes;
  size_t done_off = 0;  // of a tree's nodes: floats before the results of whole units
};
// The kernel's shapes, for cache rows of `row_bytes` and `row_tile` query rows:
// whether it uses big tiles, keys of one tile, resident warps per SM, least
// tiles per warp.
bool scored_decode_big(int row_bytes, int row_tile, bool whole);
int scored_decode_tile_keys(int row_bytes, bool big);
int scored_decode_warps(int row_bytes, int row_tile, bool big);
int scored_decode_min_tiles();
// maps[0..1]: the key and the value cache as 4-D (row bytes, L_max, HK, B) byte
// tensors with a (min(row bytes, 128), tile keys, 1, 1) box, with the 128-byte
// swizzle where box rows are 128 bytes.
// seen: the most keys one call can read per sequence.
ScoredDecodePlan scored_decode_plan(int B, int H, int HK, int n_q, int seen, int d, int elem_bytes,
                                    int num_sms);
// The same for few nodes of a tree of drafted tokens (n_q of them, 32 query rows of
// a key head at most: a node to a lane), with what they see of the tree.
struct TreeOwn {
  const int* parents;  // [B, n_q]
  const void* k;       // bf16 [B, HK, n_q, d]
  const void* v;
  RowStrides sk, sv;
};
// Whether it is taken.  Measured against the tensor-memory kernel below (us, this one
// first).  16 sequences of 4096-8192 tokens, 8 key heads: d = 64, bf16, 8 rows of a key
// head 45 and 62, 16 rows 51 and 62, 32 rows 70 and 65, e4m3 31 and 78, 44 and 78, 70 and
// 79; d = 128, 16 rows 84 and 84, e4m3 58 and 109, 32 rows 114 and 86, 107 and 110.  With
// few units it starts sooner: one of 4096 tokens, 8 key heads, d = 128, 32 rows 29 and 34
// (64 rows 29 and 36, but 72 and 58 at 32768 tokens).  d = 32, 32 rows 41 and 54, 64 rows
// 73 and 55, e4m3 68 and 72.  Neither the format nor the length is an argument, so the
// slower one is taken where these change the order: 17 to 32 rows of bf16 with d = 64, and
// with d = 128 few key heads of long caches.
inline bool tree_few(int B, int HK, int rows, int d) {
  return rows <= 16 || (rows <= 32 && (d < 128 || static_cast<long long>(B) * HK <= 32));
}
ScoredDecodePlan tree_few_plan(int B, int H, int HK, int n, int seen, int d, int elem_bytes,
                               int num_sms);
cudaError_t launch_tree_few_bf16(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                 const ScoredDecodePlan& plan, float* workspace,
                                 const LaunchCtx& ctx, const TreeOwn& tree);
cudaError_t launch_tree_few_e4m3(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                 const ScoredDecodePlan& plan, float* workspace,
                                 const LaunchCtx& ctx, const TreeOwn& tree);
cudaError_t launch_tree_few_int8(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                 const ScoredDecodePlan& plan, float* workspace,
                                 const LaunchCtx& ctx, const TreeOwn& tree);
cudaError_t launch_decode_scored_bf16(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                      const ScoredDecodePlan& plan, float* workspace,
                                      const LaunchCtx& ctx);
cudaError_t launch_decode_scored_e4m3(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                      const ScoredDecodePlan& plan, float* workspace,
                                      const LaunchCtx& ctx);
cudaError_t launch_decode_scored_int8(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                      const ScoredDecodePlan& plan, float* workspace,
                                      const LaunchCtx& ctx);

// Diagnostics.  The tensor maps are 2-D (64, 128) bf16, one box each.
cudaError_t launch_diag_tile(const CUtensorMap& tmq, const CUtensorMap& tmk,
                             const CUtensorMap& tmv, const void* p, float* s, float* o,
                             const LaunchCtx& ctx);
cudaError_t launch_diag_wait_timeout(uint64_t limit_ns, const LaunchCtx& ctx);

}  // namespace attn
