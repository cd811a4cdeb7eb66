// attn_tree_verify.cu -- which of a tree's drafted tokens stand, given the
// target's probabilities, and the token that follows them.
//
// The walk begins at the root (node 0).  At a node with the target's row p and,
// if the draft drew the node's children by chance, the draft's row q, children
// are tried in order.  With C_0 = 0 and Z_0 = 1, child k of token x and random
// number u stands if
//     u Z_k q(x) < r_k(x),    r_k(v) = max(p(v) - C_k q(v), 0),
//     C_k+1 = C_k + Z_k,      Z_k+1 = sum_v r_k+1(v)
// which is drawing with rejections from the same q again and again: what is left
// of the target's probability after one rejection is max(r_k - Z_k q, 0), and
// max(max(p - C q, 0) - Z q, 0) = max(p - (C + Z) q, 0) because q is not
// negative.  Without a q the children were chosen without chance: q(x) = 1, r is
// p without the tokens that did not stand, Z = 1 less their probabilities.  The
// next token is drawn from the r of the node where the walk ends.
//
// Bound by memory: the rows of p and q where a child was rejected or the walk
// ends.  What the walk needs of the other rows, p and q at each node's own
// token, is gathered in one round of loads for all nodes before it begins.  A
// row is read by a cluster of CTAs, each a run of it, in segments of 512 values
// or more by one warp; a segment's sum stays in shared memory, so that finding
// the next token reads one segment again and not the row.
//
// The sums are of integers, floor(2^60 r): exact, so that neither the order of
// the additions nor the number of CTAs changes an answer; rows that sum to 15 at
// most fit 64 bits.  r itself is rounded to fp32 once (C as a high and a low
// part, two fused multiply-adds); the tests of single nodes are in fp64, a few
// instructions on a unit that is too slow here for whole rows.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "attn_internal.cuh"

namespace attn {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 512;   // values of a segment, times a whole number for the largest rows
constexpr int kMostSegments = 1024;  // of one CTA
constexpr int kMostCluster = 8;
constexpr float kOne = 0x1p60f;  // a probability of 1 in the sums

struct VerifyParams {
  TreeVerifyProblem pb;
  int cluster, seg, segs;  // CTAs per sequence, values per segment, segments per CTA
};

struct Shared {
  int parent[kMostNodes], token[kMostNodes];
  float p[kMostNodes], q[kMostNodes], u[kMostNodes];  // at each node's token in its parent's rows
  u64 seg[kMostSegments];
  u64 warp_sum[kWarps];
  u64 total[2][kMostCluster];  // of each CTA's run; alternate scans take alternate ones
};

// A row to draw from: max(p - C q, 0), q null: p.
template <class T>
struct Row {
  const T* p;
  const T* q;
  float c_hi, c_lo;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// What is left of one probability, as an integer; NaN counts as 0.
__device__ __forceinline__ u64 left_of(float p, float q, float c_hi, float c_lo) {
  const float r = __fmaf_rn(-c_lo, q, __fmaf_rn(-c_hi, q, p));
  return __float2ull_rz(__saturatef(r) * kOne);
}

template <class T>
__device__ __forceinline__ u64 left_at(const Row<T>& row, int v) {
  return left_of(widen(__ldg(row.p + v)), row.q ? widen(__ldg(row.q + v)) : 0.f, row.c_hi,
                 row.c_lo);
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Sums of the 16 bytes of values that each of `LOADS` loads gives a lane.
template <class T, bool VEC>
__device__ __forceinline__ u64 block_sum(const Row<T>& row, int at, int end, int lane) {
  u64 sum = 0;
  if constexpr (VEC) {
    constexpr int E = 16 / sizeof(T), N = kSegment / (32 * E);
    if (at + kSegment <= end) {
      uint4 p[N], q[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = __ldg(reinterpret_cast<const uint4*>(row.p + at) + i * 32 + lane);
        q[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row.q) q[i] = __ldg(reinterpret_cast<const uint4*>(row.q + at) + i * 32 + lane);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const T* x = reinterpret_cast<const T*>(&p[i]);
        const T* y = reinterpret_cast<const T*>(&q[i]);
#pragma unroll
        for (int e = 0; e < E; ++e) sum += left_of(widen(x[e]), widen(y[e]), row.c_hi, row.c_lo);
      }
      return sum;
    }
  }
#pragma unroll
  for (int i = 0; i < kSegment / 32; ++i) {
    const int v = at + i * 32 + lane;
    if (v < end) sum += left_at(row, v);
  }
  return sum;
}

// floor(u * total) for u in [0, 1)
__device__ __forceinline__ u64 part_of(float u, u64 total) {
  if (!(u > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(fminf(u, 0x1.fffffep-1f));
  const int exp = bits >> 23;
  if (exp == 0) return 0;  // below 2^-126: total is below 2^64
  const u64 m = (bits & 0x7fffffu) | 0x800000u;
  const int s = 150 - exp;  // u = m 2^-s, s >= 24
  const u64 lo = m * total, hi = __umul64hi(m, total);
  if (s >= 128) return 0;
  return s < 64 ? (hi << (64 - s)) | (lo >> s) : hi >> (s - 64);
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) attn_tree_verify_kernel(const VerifyParams par) {
  __shared__ Shared sm;
  const TreeVerifyProblem& pb = par.pb;
  const int rank = blockIdx.x % par.cluster, b = blockIdx.x / par.cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* target = static_cast<const T*>(pb.target) + b * pb.tb;
  const T* draft = pb.draft ? static_cast<const T*>(pb.draft) + b * pb.db : nullptr;
  const int begin = min(static_cast<long long>(rank) * par.segs * par.seg, static_cast<long long>(pb.V));
  const int end = min(begin + static_cast<long long>(par.segs) * par.seg,
                      static_cast<long long>(pb.V));

  if (tid < kMostNodes) {
    int parent = -1, token = -1;
    float p = 0.f, q = 1.f, u = 0.f;
    if (tid < pb.n) {
      const long long at = static_cast<long long>(b) * pb.n + tid;
      parent = __ldg(pb.parents + at);
      token = __ldg(pb.tokens + at);
      u = __ldg(pb.uniforms + at);
      if (tid == 0 || parent < 0 || parent >= tid) parent = -1;
      if (parent >= 0 && token >= 0 && token < pb.V) {
        p = widen(__ldg(target + parent * pb.tn + token));
        if (draft) q = widen(__ldg(draft + parent * pb.dn + token));
      } else {
        token = -1;
      }
    }
    sm.parent[tid] = parent;
    sm.token[tid] = token;
    sm.p[tid] = p > 0.f ? p : 0.f;
    sm.q[tid] = q > 0.f ? q : 0.f;
    sm.u[tid] = u;
  }
  __syncthreads();

  int scans = 0;
  // The sum of a row over the whole cluster, and the segments' in shared memory.
  // `without`: less the tokens of that node's children (all of them rejected).
  auto scan = [&](const Row<T>& row, int without) -> u64 {
    for (int s = warp; s < par.segs; s += kWarps) {
      u64 sum = 0;
      const int at = begin + s * par.seg, to = min(at + par.seg, end);
      for (int v = at; v < to; v += kSegment) sum += block_sum<T, VEC>(row, v, to, lane);
      sum = warp_sum(sum);
      if (lane == 0) sm.seg[s] = sum;
    }
    __syncthreads();
    if (without >= 0 && tid < pb.n && sm.parent[tid] == without) {
      const int x = sm.token[tid];
      bool first = x >= begin && x < end;  // (-1 is in nobody's run)
      for (int e = without + 1; e < tid && first; ++e)
        first = !(sm.parent[e] == without && sm.token[e] == x);
      if (first) atomicAdd(&sm.seg[(x - begin) / par.seg], 0ull - left_at(row, x));
    }
    __syncthreads();
    u64 sum = 0;
    for (int s = tid; s < par.segs; s += kThreads) sum += sm.seg[s];
    sum = warp_sum(sum);
    if (lane == 0) sm.warp_sum[warp] = sum;
    __syncthreads();
    u64* total = sm.total[scans++ & 1];
    if (tid < par.cluster) {
      sum = 0;
      for (int i = 0; i < kWarps; ++i) sum += sm.warp_sum[i];
      if (par.cluster > 1)
        *cg::this_cluster().map_shared_rank(total + rank, tid) = sum;
      else
        total[0] = sum;
    }
    if (par.cluster > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
    sum = 0;
    for (int i = 0; i < par.cluster; ++i) sum += total[i];
    return sum;
  };

  // ---- the walk, by every thread alike
  int cur = 0, len = 1;
  double C = 0.0, Z = 1.0;
  u64 sum = 0;
  bool scanned = false;  // whether the segments hold the row to draw from
  int* path = pb.path + static_cast<long long>(b) * pb.n;
  auto row_at = [&](bool rejected) {
    Row<T> row;
    row.p = target + cur * pb.tn;
    row.q = draft && rejected ? draft + cur * pb.dn : nullptr;
    row.c_hi = static_cast<float>(C);
    row.c_lo = static_cast<float>(C - row.c_hi);
    return row;
  };
  if (rank == 0 && tid == 0) path[0] = 0;
  bool went = true, rejected = false;
  while (went) {
    went = false;
    for (int w = cur >> 5; w < kMostNodes / 32 && !went; ++w) {
      unsigned kids = __ballot_sync(0xffffffffu, sm.parent[32 * w + lane] == cur);
      while (kids != 0 && !went) {
        const int c = 32 * w + __ffs(kids) - 1;
        kids &= kids - 1;
        const double q = sm.q[c];
        double r = sm.p[c];
        if (draft) {
          r = fmax(r - C * q, 0.0);
        } else {
          // an earlier child of the same token did not stand: nothing is left of it
          for (int v = cur >> 5; v <= w; ++v) {
            const int e = 32 * v + lane;
            if (__any_sync(0xffffffffu, e < c && sm.parent[e] == cur && sm.token[e] == sm.token[c]))
              r = 0.0;
          }
        }
        if (static_cast<double>(sm.u[c]) * Z * q < r) {
          went = true;
          cur = c;
          if (rank == 0 && tid == 0) path[len] = c;
          ++len;
          C = 0.0;
          Z = 1.0;
          scanned = rejected = false;
        } else {
          rejected = true;
          if (draft) {
            C += Z;
            sum = scan(row_at(true), -1);
            scanned = true;
            Z = static_cast<double>(sum) * 0x1p-60;
          } else {
            Z -= r;
          }
        }
      }
    }
  }
  if (rank == 0) {
    for (int i = len + tid; i < pb.n; i += kThreads) path[i] = -1;
    if (tid == 0) pb.path_lens[b] = len;
  }

  // ---- the next token
  Row<T> row = row_at(rejected);
  int without = !draft && rejected ? cur : -1;
  if (!scanned) sum = scan(row, without);
  if (sum == 0) {  // nothing is left (the draft's row covers the target's): the target's own
    row = row_at(false);
    without = -1;
    if (rejected) sum = scan(row, -1);
  }
  if (sum == 0) {
    if (rank == 0 && tid == 0) pb.next_tokens[b] = -1;
    return;
  }
  u64 t = part_of(sm.u[0], sum);  // the first token whose running sum exceeds it
  const u64* total = sm.total[(scans - 1) & 1];
  int owner = 0;
  while (owner + 1 < par.cluster && t >= total[owner]) t -= total[owner++];
  if (owner != rank || warp != 0) return;
  auto find = [&](u64 mine) {  // the lane that it falls to, and what is left of t there
    u64 upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += x;
    }
    const unsigned over = __ballot_sync(0xffffffffu, upto > t);
    const int at = over ? __ffs(over) - 1 : 32;
    t -= __shfl_sync(0xffffffffu, at < 32 ? upto - mine : upto, at < 32 ? at : 31);
    return at;
  };
  const int each = (par.segs + 31) / 32;
  u64 mine = 0;
  for (int i = lane * each; i < min((lane + 1) * each, par.segs); ++i) mine += sm.seg[i];
  int s = min(find(mine), 31) * each;
  while (s + 1 < par.segs && t >= sm.seg[s]) t -= sm.seg[s++];
  auto value = [&](int v) {
    if (v >= end) return 0ull;
    if (without >= 0)
      for (int e = without + 1; e < pb.n; ++e)
        if (sm.parent[e] == without && sm.token[e] == v) return 0ull;
    return left_at(row, v);
  };
  constexpr int kEach = kSegment / 32;
  const int stop = min(begin + (s + 1) * par.seg, end);
  for (int v = begin + s * par.seg; v < stop; v += kSegment) {
    mine = 0;
    for (int i = 0; i < kEach; ++i) mine += value(v + lane * kEach + i);
    const int at = find(mine);
    if (at == 32) continue;
    if (lane == at) {
      int x = v + lane * kEach;
      u64 w = value(x);
      while (t >= w && x + 1 < end) {
        t -= w;
        w = value(++x);
      }
      pb.next_tokens[b] = x;
    }
    return;
  }
}

template <class T, bool VEC>
cudaError_t launch(const VerifyParams& par, const LaunchCtx& ctx) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(par.pb.B * par.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = par.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tree_verify_kernel<T, VEC>, par);
}

}  // namespace

cudaError_t launch_tree_verify(const TreeVerifyProblem& pb, const LaunchCtx& ctx) {
  VerifyParams par;
  par.pb = pb;
  // CTAs per sequence: as many as keep every CTA resident, with a segment for
  // each of a CTA's warps
  int cluster = 1;
  while (cluster < kMostCluster && 2LL * cluster * pb.B <= 2LL * ctx.num_sms &&
         2LL * cluster * kWarps * kSegment <= pb.V)
    cluster *= 2;
  par.cluster = cluster;
  const long long most = static_cast<long long>(cluster) * kMostSegments * kSegment;
  par.seg = static_cast<int>(kSegment * ((pb.V + most - 1) / most));
  const int segs = (pb.V + par.seg - 1) / par.seg;
  par.segs = (segs + cluster - 1) / cluster;
  const int es = pb.bf16 ? 2 : 4;
  auto whole = [&](const void* base, long long sb, long long sn) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && sb * es % 16 == 0 && sn * es % 16 == 0;
  };
  const bool vec = whole(pb.target, pb.tb, pb.tn) && (!pb.draft || whole(pb.draft, pb.db, pb.dn));
  if (pb.bf16)
    return vec ? launch<__nv_bfloat16, true>(par, ctx) : launch<__nv_bfloat16, false>(par, ctx);
  return vec ? launch<float, true>(par, ctx) : launch<float, false>(par, ctx);
}

}  // namespace attn
