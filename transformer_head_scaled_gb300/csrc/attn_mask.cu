// attn_mask.cu -- the plan of a mask that leaves every query one run of keys.
//
// Query i of a batch entry sees key j iff
//   * j >= i - left and j <= i + right (either side may be absent), or
//     j < prefix (a prefix all may see; then there is no left side), and
//   * j < key_len, and
//   * i and j lie in the same document: the same maximal run of equal ids, not
//     negative.
// Each of these leaves query i an interval of keys and key j an interval of
// queries, so the attention kernels need nothing but intervals: per query and
// per key for the elements of a tile, and per 128 queries and per 128 keys (the
// union, which tiles to visit, and the intersection, which tiles need no
// test).  The plan is these four arrays; one plan serves the forward and the
// backward of every layer that shares the mask.
//
// Two kernels, both bound by launch and latency (16 bytes written per token):
//   1. with documents: per 128 tokens, the first and the last token that
//      begins a run;
//   2. per 128 queries and 128 keys: the runs around them from those, the
//      intervals and their unions and intersections.
#include "attn_internal.cuh"

namespace attn {
namespace {

constexpr int TILE = kMaskTile;

struct MaskParams {
  int4* header;
  int2* row_keys;
  int2* key_rows;
  int4* block_keys;
  int4* tile_rows;
  int2* runs;  // scratch: per tile {first, last} token that begins a run, or {n, -1}
  const int* key_lens;
  const int* doc_ids;
  const int* prefix_lens;
  int B, n_q, n_k, left, right, qt, kt;
};

__device__ __forceinline__ bool begins_run(const int* ids, int i) {
  return i == 0 || __ldg(ids + i) != __ldg(ids + i - 1);
}

__global__ void __launch_bounds__(TILE) attn_mask_runs_kernel(const MaskParams p) {
  grid_launch_dependents();
  __shared__ unsigned bits[TILE / 32];
  const int b = blockIdx.x / p.qt, tile = blockIdx.x - b * p.qt;
  const int i = tile * TILE + threadIdx.x;
  const int* ids = p.doc_ids + static_cast<size_t>(b) * p.n_q;
  const unsigned vote = __ballot_sync(0xffffffffu, i < p.n_q && begins_run(ids, i));
  if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = vote;
  __syncthreads();
  if (threadIdx.x == 0) {
    int first = p.n_q, last = -1;
    for (int w = 0; w < TILE / 32; ++w) {
      if (bits[w] == 0) continue;
      const int at = tile * TILE + 32 * w;
      if (last < 0) first = at + __ffs(bits[w]) - 1;
      last = at + 31 - __clz(bits[w]);
    }
    p.runs[blockIdx.x] = make_int2(first, last);
  }
}

// Smallest of lo and largest of hi over the CTA, for two pairs at once; every
// thread gets the result.
__device__ __forceinline__ int4 reduce_bounds(int min_a, int max_b, int max_c, int min_d,
                                              int4* scratch) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    min_a = min(min_a, __shfl_xor_sync(0xffffffffu, min_a, m));
    max_b = max(max_b, __shfl_xor_sync(0xffffffffu, max_b, m));
    max_c = max(max_c, __shfl_xor_sync(0xffffffffu, max_c, m));
    min_d = min(min_d, __shfl_xor_sync(0xffffffffu, min_d, m));
  }
  __syncthreads();  // the scratch may still be read for the previous reduction
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = make_int4(min_a, max_b, max_c, min_d);
  __syncthreads();
  int4 r = scratch[0];
#pragma unroll
  for (int w = 1; w < TILE / 32; ++w) {
    const int4 x = scratch[w];
    r = make_int4(min(r.x, x.x), max(r.y, x.y), max(r.z, x.z), min(r.w, x.w));
  }
  return r;
}

// {first, end} of the union of the CTA's intervals and of their intersection;
// an empty interval adds nothing to the union and empties the intersection.
// `in`: this thread has an interval at all.
__device__ __forceinline__ int4 summary(int2 v, bool in, int4* scratch) {
  const bool some = in && v.x < v.y;
  const int4 r = reduce_bounds(some ? v.x : 0x7fffffff, some ? v.y : 0,
                               in ? (some ? v.x : 0x7fffffff) : 0,
                               in ? (some ? v.y : 0) : 0x7fffffff, scratch);
  return r.y > 0 ? make_int4(r.x, r.y, r.z, r.w) : make_int4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(TILE) attn_mask_plan_kernel(const MaskParams p) {
  __shared__ int4 scratch[TILE / 32];
  __shared__ unsigned bits[TILE / 32];
  const int tiles = max(p.qt, p.kt);
  const int b = blockIdx.x / tiles, tile = blockIdx.x - b * tiles;
  const int i = tile * TILE + threadIdx.x;  // as a query and as a key
  if (blockIdx.x == 0 && threadIdx.x == 0)
    *p.header = make_int4(p.n_q, p.n_k, p.B, p.right >= 0 ? 1 : 0);
  int run0 = 0, run1 = 0x7fffffff;  // this token's document
  if (p.doc_ids != nullptr) {
    const int* ids = p.doc_ids + static_cast<size_t>(b) * p.n_q;
    const unsigned vote = __ballot_sync(0xffffffffu, i < p.n_q && begins_run(ids, i));
    if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = vote;
    grid_dependency_wait();  // the tiles' runs
    // the last run that begins before this tile, and the first one after it
    int before = 0, after = p.n_q;
    const int2* runs = p.runs + static_cast<size_t>(b) * p.qt;
    for (int t = threadIdx.x; t < p.qt; t += TILE) {
      const int2 r = runs[t];
      if (t < tile) before = max(before, r.y);
      if (t > tile) after = min(after, r.x);
    }
    const int4 near = reduce_bounds(after, before, 0, 0, scratch);
    run0 = near.y;
    run1 = near.x;
    // the nearest beginnings inside the tile
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
#pragma unroll
    for (int x = 0; x < TILE / 32; ++x) {
      const unsigned low = x < w ? bits[x] : (x == w ? bits[x] & (0xffffffffu >> (31 - l)) : 0u);
      if (low != 0) run0 = max(run0, tile * TILE + 32 * x + 31 - __clz(low));
    }
#pragma unroll
    for (int x = TILE / 32 - 1; x >= 0; --x) {
      const unsigned high = x > w ? bits[x] : (x == w && l < 31 ? bits[x] & (0xfffffffeu << l) : 0u);
      if (high != 0) run1 = min(run1, tile * TILE + 32 * x + __ffs(high) - 1);
    }
    if (i < p.n_q && __ldg(ids + i) < 0) run0 = run1 = 0;  // no document
  }
  const int limit = p.key_lens != nullptr ? min(max(__ldg(p.key_lens + b), 0), p.n_k) : p.n_k;
  const int prefix = p.prefix_lens != nullptr ? min(max(__ldg(p.prefix_lens + b), 0), p.n_k) : 0;
  // (left and right are at most n_q + n_k, so nothing here leaves int)
  if (tile < p.qt) {
    int2 v = make_int2(0, 0);
    if (i < p.n_q) {
      const int lo = max(run0, p.left >= 0 ? i - p.left : 0);
      const int near = p.right >= 0 ? i + p.right + 1 : p.n_k;
      const int hi = min(min(max(near, prefix), run1), limit);
      if (lo < hi) v = make_int2(lo, hi);
      p.row_keys[static_cast<size_t>(b) * p.n_q + i] = v;
    }
    const int4 s = summary(v, i < p.n_q, scratch);
    if (threadIdx.x == 0) p.block_keys[static_cast<size_t>(b) * p.qt + tile] = s;
  }
  if (tile < p.kt) {
    int2 v = make_int2(0, 0);
    if (i < p.n_k) {
      const int lo = max(run0, i < prefix || p.right < 0 ? 0 : max(i - p.right, 0));
      const int hi = min(min(p.left >= 0 ? i + p.left + 1 : p.n_q, run1), p.n_q);
      if (lo < hi && i < limit) v = make_int2(lo, hi);
      p.key_rows[static_cast<size_t>(b) * p.n_k + i] = v;
    }
    const int4 s = summary(v, i < p.n_k, scratch);
    if (threadIdx.x == 0) p.tile_rows[static_cast<size_t>(b) * p.kt + tile] = s;
  }
}

}  // namespace

MaskLayout mask_layout(int B, int n_q, int n_k) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  MaskLayout l;
  const size_t qt = (static_cast<size_t>(n_q) + TILE - 1) / TILE,
               kt = (static_cast<size_t>(n_k) + TILE - 1) / TILE;
  size_t off = 256;  // the header
  l.row_keys = off;
  off += up(static_cast<size_t>(B) * n_q * sizeof(int2));
  l.key_rows = off;
  off += up(static_cast<size_t>(B) * n_k * sizeof(int2));
  l.block_keys = off;
  off += up(B * qt * sizeof(int4));
  l.tile_rows = off;
  off += up(B * kt * sizeof(int4));
  l.runs = off;
  off += up(B * qt * sizeof(int2));
  l.bytes = off;
  return l;
}

MaskPlan mask_plan_at(const void* plan, int B, int n_q, int n_k) {
  const MaskLayout l = mask_layout(B, n_q, n_k);
  const uint8_t* base = static_cast<const uint8_t*>(plan);
  MaskPlan m;
  m.header = reinterpret_cast<const int4*>(base);
  m.row_keys = reinterpret_cast<const int2*>(base + l.row_keys);
  m.key_rows = reinterpret_cast<const int2*>(base + l.key_rows);
  m.block_keys = reinterpret_cast<const int4*>(base + l.block_keys);
  m.tile_rows = reinterpret_cast<const int4*>(base + l.tile_rows);
  return m;
}

cudaError_t launch_mask_plan(const MaskProblem& pb, void* plan, const LaunchCtx& ctx) {
  const MaskLayout l = mask_layout(pb.B, pb.n_q, pb.n_k);
  uint8_t* base = static_cast<uint8_t*>(plan);
  MaskParams p;
  p.header = reinterpret_cast<int4*>(base);
  p.row_keys = reinterpret_cast<int2*>(base + l.row_keys);
  p.key_rows = reinterpret_cast<int2*>(base + l.key_rows);
  p.block_keys = reinterpret_cast<int4*>(base + l.block_keys);
  p.tile_rows = reinterpret_cast<int4*>(base + l.tile_rows);
  p.runs = reinterpret_cast<int2*>(base + l.runs);
  p.key_lens = pb.key_lens;
  p.doc_ids = pb.doc_ids;
  p.prefix_lens = pb.prefix_lens;
  p.B = pb.B;
  p.n_q = pb.n_q;
  p.n_k = pb.n_k;
  p.left = pb.left;
  p.right = pb.right;
  p.qt = (pb.n_q + TILE - 1) / TILE;
  p.kt = (pb.n_k + TILE - 1) / TILE;
  const unsigned grid = static_cast<unsigned>(pb.B) * (p.qt > p.kt ? p.qt : p.kt);
  if (pb.doc_ids == nullptr) {
    attn_mask_plan_kernel<<<grid, TILE, 0, ctx.stream>>>(p);
    return cudaGetLastError();
  }
  attn_mask_runs_kernel<<<static_cast<unsigned>(pb.B) * p.qt, TILE, 0, ctx.stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(attn_mask_plan_kernel, dim3(grid), dim3(TILE), 0, ctx.stream, p);
}

}  // namespace attn
