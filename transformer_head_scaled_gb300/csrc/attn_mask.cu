// attn_mask.cu -- the plan of a mask that leaves every query one run of keys.
//
// Query i of a batch entry sees key j iff
//   * j >= i - left and j <= i + right (either side may be absent), or
//     j < prefix (a prefix all may see; then there is no left side), and
//   * j < key_len, and
//   * i and j lie in the same document: the same maximal run of equal ids, not
//     negative.
// Each of these leaves query i an interval of keys and key j an interval of
// queries, so the attention kernels need nothing but intervals, and, per work
// item, the tiles that it has to visit: the forward's items are 256 queries with
// the keys that each half sees, the backward's 128 keys with the queries that see
// them.  The items stand in the order in which they are to be dealt out, the
// heaviest first where that is known: under a causal mask the last queries (the
// first keys); with documents, whose work has no simple order, by counting.  One
// plan serves the forward and the backward of every layer that shares the mask.
//
// Kernels, all bound by launch and latency (16 bytes written per token):
//   1. with documents: per 256 tokens, the first and the last token that begins
//      a run;
//   2. per 256 queries and 256 keys: the runs around them from those, the
//      intervals, and the items;
//   3. with documents: the items by falling work, each one's rank the number of
//      items with more (kMostOrdered of them at most; more even out anyway).
// Measured in a graph: 2 us for 8 x 4096 tokens without documents (one kernel),
// 6 us for 4 x 4096 with documents, 26 us for one row of 131072.
#include "attn_internal.cuh"

namespace attn {
namespace {

constexpr int BLOCK = 256;  // tokens per CTA: an item of the forward, two of the backward
constexpr int WARPS = BLOCK / 32;

struct MaskParams {
  int4* header;
  int2* row_keys;
  int2* key_rows;
  QueryItem* query_items;
  KeyItem* key_items;
  // with ordering: the items before it
  QueryItem* query_items_in;
  KeyItem* key_items_in;
  int2* runs;  // per block {first, last} token that begins a run, or {n, -1}
  const int* key_lens;
  const int* doc_ids;
  const int* prefix_lens;
  int B, n_q, n_k, left, right, qb, kb, ordered;
};

__device__ __forceinline__ bool begins_run(const int* ids, int i) {
  return i == 0 || __ldg(ids + i) != __ldg(ids + i - 1);
}

__global__ void __launch_bounds__(BLOCK) attn_mask_runs_kernel(const MaskParams p) {
  grid_launch_dependents();
  __shared__ unsigned bits[WARPS];
  const int b = blockIdx.x / p.qb, block = blockIdx.x - b * p.qb;
  const int i = block * BLOCK + threadIdx.x;
  const int* ids = p.doc_ids + static_cast<size_t>(b) * p.n_q;
  const unsigned vote = __ballot_sync(0xffffffffu, i < p.n_q && begins_run(ids, i));
  if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = vote;
  __syncthreads();
  if (threadIdx.x == 0) {
    int first = p.n_q, last = -1;
    for (int w = 0; w < WARPS; ++w) {
      if (bits[w] == 0) continue;
      const int at = block * BLOCK + 32 * w;
      if (last < 0) first = at + __ffs(bits[w]) - 1;
      last = at + 31 - __clz(bits[w]);
    }
    p.runs[blockIdx.x] = make_int2(first, last);
  }
}

// Smallest lo and largest hi of each half of the CTA (threads 0-127, 128-255);
// every thread gets both: {lo, hi, lo, hi}.
__device__ __forceinline__ int4 reduce_halves(int lo, int hi, int2* scratch) {
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();  // the scratch may still be read for the previous reduction
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = make_int2(lo, hi);
  __syncthreads();
  int4 r = make_int4(0x7fffffff, 0, 0x7fffffff, 0);
#pragma unroll
  for (int w = 0; w < WARPS / 2; ++w) {
    const int2 x = scratch[w], y = scratch[w + WARPS / 2];
    r = make_int4(min(r.x, x.x), max(r.y, x.y), min(r.z, y.x), max(r.w, y.y));
  }
  return r;
}

__device__ __forceinline__ int tiles_of(int first, int end) {
  return end > 0 ? (end + kMaskTile - 1) / kMaskTile - first / kMaskTile : 0;
}

__global__ void __launch_bounds__(BLOCK) attn_mask_plan_kernel(const MaskParams p) {
  grid_launch_dependents();
  __shared__ int2 scratch[WARPS];
  __shared__ unsigned bits[WARPS];
  const int blocks = max(p.qb, p.kb);
  const int b = blockIdx.x / blocks, block = blockIdx.x - b * blocks;
  const int i = block * BLOCK + threadIdx.x;  // as a query and as a key
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.header = make_int4(p.n_q, p.n_k, p.B, p.ordered);
  int run0 = 0, run1 = 0x7fffffff;  // this token's document
  if (p.doc_ids != nullptr) {
    const int* ids = p.doc_ids + static_cast<size_t>(b) * p.n_q;
    const unsigned vote = __ballot_sync(0xffffffffu, i < p.n_q && begins_run(ids, i));
    if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = vote;
    grid_dependency_wait();  // the blocks' runs
    // the last run that begins before this block, and the first one after it
    int before = 0, after = p.n_q;
    const int2* runs = p.runs + static_cast<size_t>(b) * p.qb;
    for (int t = threadIdx.x; t < p.qb; t += BLOCK) {
      const int2 r = runs[t];
      if (t < block) before = max(before, r.y);
      if (t > block) after = min(after, r.x);
    }
    const int4 near = reduce_halves(after, before, scratch);
    run0 = max(near.y, near.w);
    run1 = min(near.x, near.z);
    // the nearest beginnings inside the block
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
#pragma unroll
    for (int x = 0; x < WARPS; ++x) {
      const unsigned low = x < w ? bits[x] : (x == w ? bits[x] & (0xffffffffu >> (31 - l)) : 0u);
      if (low != 0) run0 = max(run0, block * BLOCK + 32 * x + 31 - __clz(low));
    }
#pragma unroll
    for (int x = WARPS - 1; x >= 0; --x) {
      const unsigned high = x > w ? bits[x] : (x == w && l < 31 ? bits[x] & (0xfffffffeu << l) : 0u);
      if (high != 0) run1 = min(run1, block * BLOCK + 32 * x + __ffs(high) - 1);
    }
    if (i < p.n_q && __ldg(ids + i) < 0) run0 = run1 = 0;  // no document
  }
  const int limit = p.key_lens != nullptr ? min(max(__ldg(p.key_lens + b), 0), p.n_k) : p.n_k;
  const int prefix = p.prefix_lens != nullptr ? min(max(__ldg(p.prefix_lens + b), 0), p.n_k) : 0;
  const bool later_heavier = p.right >= 0;
  // (left < n_q and right < n_k, 2^30 tokens at most, so nothing here leaves int)
  if (block < p.qb) {
    int2 v = make_int2(0, 0);
    if (i < p.n_q) {
      const int lo = max(run0, p.left >= 0 ? i - p.left : 0);
      const int near = p.right >= 0 ? i + p.right + 1 : p.n_k;
      const int hi = min(min(max(near, prefix), run1), limit);
      if (lo < hi) v = make_int2(lo, hi);
      p.row_keys[static_cast<size_t>(b) * p.n_q + i] = v;
    }
    const int4 r = reduce_halves(v.x < v.y ? v.x : 0x7fffffff, v.y, scratch);
    if (threadIdx.x == 0) {
      QueryItem item;
      item.b = b;
      item.block = block;
      item.first = max(r.y, r.w) > 0 ? min(r.x, r.z) : 0;
      item.end[0] = r.y;
      item.end[1] = r.w;
      item.work = tiles_of(item.first, r.y) + tiles_of(item.first, r.w);
      item.pad[0] = item.pad[1] = 0;
      if (p.ordered)
        p.query_items_in[blockIdx.x / blocks * p.qb + block] = item;
      else
        p.query_items[later_heavier ? (p.qb - 1 - block) * p.B + b : b * p.qb + block] = item;
    }
  }
  if (block < p.kb) {
    int2 v = make_int2(0, 0);
    if (i < p.n_k) {
      const int lo = max(run0, i < prefix || p.right < 0 ? 0 : max(i - p.right, 0));
      const int hi = min(min(p.left >= 0 ? i + p.left + 1 : p.n_q, run1), p.n_q);
      if (lo < hi && i < limit) v = make_int2(lo, hi);
      p.key_rows[static_cast<size_t>(b) * p.n_k + i] = v;
    }
    const int4 r = reduce_halves(v.x < v.y ? v.x : 0x7fffffff, v.y, scratch);
    const int kt = (p.n_k + kMaskTile - 1) / kMaskTile, tile = 2 * block + threadIdx.x;
    if (threadIdx.x < 2 && tile < kt) {
      const int first = threadIdx.x == 0 ? r.x : r.z, end = threadIdx.x == 0 ? r.y : r.w;
      KeyItem item;
      item.b = b;
      item.tile = tile;
      item.first = end > 0 ? first / kMaskTile : 0;
      item.count = tiles_of(first, end);
      if (p.ordered)
        p.key_items_in[b * kt + tile] = item;
      else
        p.key_items[later_heavier ? tile * p.B + b : b * kt + tile] = item;
    }
  }
}

// The items by falling work, ties in index order.  grid.y: 0 the forward's, 1 the
// backward's.
__global__ void __launch_bounds__(BLOCK) attn_mask_order_kernel(const MaskParams p) {
  // work << 11 | how far from the last item: one comparison
  __shared__ __align__(16) uint32_t place[kMostOrdered];
  static_assert(kMostOrdered == 1 << 11, "the bits of an item's index");
  const bool keys = blockIdx.y == 1;
  const int n = p.B * (keys ? (p.n_k + kMaskTile - 1) / kMaskTile : p.qb);
  if (static_cast<int>(blockIdx.x) * BLOCK >= n) return;
  grid_dependency_wait();  // the items
  const int n4 = (n + 3) & ~3;
  for (int e = threadIdx.x; e < n4; e += BLOCK) {
    const int work = e >= n ? 0 : (keys ? p.key_items_in[e].count : p.query_items_in[e].work);
    place[e] = e >= n ? 0u : static_cast<uint32_t>(min(work, (1 << 21) - 1)) << 11 | (kMostOrdered - 1 - e);
  }
  __syncthreads();
  const int e = blockIdx.x * BLOCK + threadIdx.x;
  if (e >= n) return;
  const uint32_t mine = place[e];
  int rank = 0;
  for (int x = 0; x < n4; x += 4) {
    const uint4 other = *reinterpret_cast<const uint4*>(place + x);
    rank += (other.x > mine) + (other.y > mine) + (other.z > mine) + (other.w > mine);
  }
  if (keys)
    p.key_items[rank] = p.key_items_in[e];
  else
    p.query_items[rank] = p.query_items_in[e];
}

}  // namespace

MaskLayout mask_layout(int B, int n_q, int n_k) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  MaskLayout l;
  const size_t qb = (static_cast<size_t>(n_q) + BLOCK - 1) / BLOCK,
               kt = (static_cast<size_t>(n_k) + kMaskTile - 1) / kMaskTile;
  const size_t queries = up(B * qb * sizeof(QueryItem)), keys = up(B * kt * sizeof(KeyItem));
  // (the copy before ordering; larger plans are not ordered)
  const bool room = B * qb <= kMostOrdered && B * kt <= kMostOrdered;
  size_t off = 256;  // the header
  l.row_keys = off;
  off += up(static_cast<size_t>(B) * n_q * sizeof(int2));
  l.key_rows = off;
  off += up(static_cast<size_t>(B) * n_k * sizeof(int2));
  l.query_items = off;
  off += queries;
  l.key_items = off;
  off += keys;
  l.query_items_in = off;
  off += room ? queries : 0;
  l.key_items_in = off;
  off += room ? keys : 0;
  l.runs = off;
  off += up(B * qb * sizeof(int2));
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
  m.query_items = reinterpret_cast<const QueryItem*>(base + l.query_items);
  m.key_items = reinterpret_cast<const KeyItem*>(base + l.key_items);
  return m;
}

bool mask_plan_ordered(const MaskProblem& pb) {
  const long long qb = (static_cast<long long>(pb.n_q) + BLOCK - 1) / BLOCK,
                  kt = (static_cast<long long>(pb.n_k) + kMaskTile - 1) / kMaskTile;
  return pb.doc_ids != nullptr && pb.B * kt > 1 && pb.B * qb <= kMostOrdered &&
         pb.B * kt <= kMostOrdered;
}

cudaError_t launch_mask_plan(const MaskProblem& pb, void* plan, const LaunchCtx& ctx) {
  const MaskLayout l = mask_layout(pb.B, pb.n_q, pb.n_k);
  uint8_t* base = static_cast<uint8_t*>(plan);
  MaskParams p;
  p.header = reinterpret_cast<int4*>(base);
  p.row_keys = reinterpret_cast<int2*>(base + l.row_keys);
  p.key_rows = reinterpret_cast<int2*>(base + l.key_rows);
  p.query_items = reinterpret_cast<QueryItem*>(base + l.query_items);
  p.key_items = reinterpret_cast<KeyItem*>(base + l.key_items);
  p.query_items_in = reinterpret_cast<QueryItem*>(base + l.query_items_in);
  p.key_items_in = reinterpret_cast<KeyItem*>(base + l.key_items_in);
  p.runs = reinterpret_cast<int2*>(base + l.runs);
  p.key_lens = pb.key_lens;
  p.doc_ids = pb.doc_ids;
  p.prefix_lens = pb.prefix_lens;
  p.B = pb.B;
  p.n_q = pb.n_q;
  p.n_k = pb.n_k;
  p.left = pb.left;
  p.right = pb.right;
  p.qb = (pb.n_q + BLOCK - 1) / BLOCK;
  p.kb = (pb.n_k + BLOCK - 1) / BLOCK;
  p.ordered = mask_plan_ordered(pb) ? 1 : 0;
  const unsigned grid = static_cast<unsigned>(pb.B) * (p.qb > p.kb ? p.qb : p.kb);
  if (pb.doc_ids == nullptr) {
    attn_mask_plan_kernel<<<grid, BLOCK, 0, ctx.stream>>>(p);
    return cudaGetLastError();
  }
  attn_mask_runs_kernel<<<static_cast<unsigned>(pb.B) * p.qb, BLOCK, 0, ctx.stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(attn_mask_plan_kernel, dim3(grid), dim3(BLOCK), 0, ctx.stream, p);
  if (e != cudaSuccess || !p.ordered) return e;
  const int kt = (pb.n_k + kMaskTile - 1) / kMaskTile;
  return launch_dependent(attn_mask_order_kernel, dim3((pb.B * kt + BLOCK - 1) / BLOCK, 2),
                          dim3(BLOCK), 0, ctx.stream, p);
}

}  // namespace attn
