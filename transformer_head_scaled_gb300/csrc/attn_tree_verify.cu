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
// Bound by memory for many sequences, the rows of p and q where a child was rejected
// or the walk ends; else by the chain of a sequence's scans, one after the other,
// since each C needs the sum before it (1.5 to 2 us a scan: the loads 0.7, the
// exchange in the cluster 0.4, the walk 0.5).  128 sequences of 32 nodes over 131072
// fp32 values take 63 us (read once: 20), 64 of 64 nodes over 131072 bf16 values
// without a draft's row 19 us (2.5), one of 6 nodes over 32000 fp32 values 9 us.
// What the walk needs of the other rows, p and q at each node's own
// token, is gathered in one round of loads for all nodes before it begins.  A
// row is read by a cluster of CTAs, each a run of it, in segments of 512 values
// or more by one warp; a segment's sum stays in shared memory, so that finding
// the next token reads one segment again and not the row.
//
// The sums are of integers, floor(2^60 r): exact, so that neither the order of
// the additions nor the number of CTAs changes an answer; rows that sum to 15 at
// most fit 64 bits.  r itself is rounded to fp32 once (C as a high and a low
// part, two fused multiply-adds); the tests of single nodes are in pairs of fp32
// numbers.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "attn_internal.cuh"

namespace attn {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 512;   // values of a segment, times a whole number for the largest rows
constexpr int kMostSegments = 512;  // of one CTA
constexpr int kMostCluster = 16;

struct VerifyParams {
  TreeVerifyProblem pb;
  int cluster, seg, segs;  // CTAs per sequence, values per segment, segments per CTA
};

// A number as the sum of two fp32 ones, lo at most half a step of hi: 48 bits, for
// what the walk compares (fp64 is slower here by far: a test took 1700 cycles).
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

// p - c q
__device__ __forceinline__ Pair less(float p, Pair c, float q) {
  const float m = __fmul_rn(c.hi, q);
  const Pair s = two_sum(p, -m);
  return two_sum(s.hi, __fmaf_rn(-c.lo, q, __fsub_rn(s.lo, __fmaf_rn(c.hi, q, -m))));
}

// 2^-60 x
__device__ __forceinline__ Pair pair_of(u64 x) {
  const Pair s = two_sum(static_cast<float>(static_cast<uint32_t>(x >> 40)) * 0x1p-20f,
                         static_cast<float>(static_cast<uint32_t>(x >> 16) & 0xffffffu) * 0x1p-44f);
  return two_sum(s.hi, s.lo + static_cast<float>(static_cast<uint32_t>(x) & 0xffffu) * 0x1p-60f);
}

// How far the walk is (shared memory keeps it while a row is summed).
struct Walk {
  Pair C, Z;
  int cur, len, next;  // the node, its depth, the child to test next
  bool rejected;       // a child of the node
  bool at_end;
};

struct Shared {
  int parent[kMostNodes], token[kMostNodes];
  float p[kMostNodes], q[kMostNodes], u[kMostNodes];  // at each node's token in its parent's rows
  Walk walk;
  u64 seg[kMostSegments];
  u64 sums[2][kMostCluster][kWarps];  // of each CTA's warps; alternate scans take alternate ones
};

// A row to draw from: max(p - C q, 0), q null: p.
template <class T>
struct Row {
  const T* p;
  const T* q;
  Pair c;
};

// The cluster's barrier in its two halves.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// What is left of one probability; a NaN of p counts as 0, one of q has to be 0 already.
__device__ __forceinline__ float left_of(float p, float q, Pair c) {
  return __saturatef(__fmaf_rn(-c.lo, q, __fmaf_rn(-c.hi, q, p)));
}

// floor(2^60 r), r in [0, 1].  By shifts of the significand: the conversion instruction
// to 64 bits is one of the fp64 unit's, which bound the kernel (128 sequences of 131072
// fp32 values 162 us).
__device__ __forceinline__ u64 fixed(float r) {
  const uint32_t bits = __float_as_uint(r);
  // r = m 2^(e - 150) and r 2^60 = (m 2^40) 2^(e - 130); shifts by 64 and more give 0
  u64 x = static_cast<u64>((bits << 8) | 0x80000000u) << 32;
  asm("shr.u64 %0, %0, %1;" : "+l"(x) : "r"(130u - (bits >> 23)));
  return x;
}

template <class T>
__device__ __forceinline__ float left_at(const Row<T>& row, int v) {
  return left_of(widen(__ldg(row.p + v)), row.q ? fmaxf(widen(__ldg(row.q + v)), 0.f) : 0.f,
                 row.c);
}

// The warp's sum: of three parts that 32 bits hold 32 times.
__device__ __forceinline__ u64 warp_sum(u64 x) {
  const u64 a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x) & 0x3fffffu);
  const u64 b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 22) & 0x3fffffu);
  const u64 c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 44));
  return a + (b << 22) + (c << 44);
}

// A lane's part of a block of a row: the bytes of kPart loads.
constexpr int kEach = kSegment / 32;
template <class T>
constexpr int kPart = kEach * static_cast<int>(sizeof(T)) / 16;

template <class T, bool VEC>
__device__ __forceinline__ void load_part(const T* row, int at, int end, int lane,
                                          uint4 (&x)[kPart<T>]) {
  if (VEC && at + kSegment <= end) {
#pragma unroll
    for (int i = 0; i < kPart<T>; ++i)
      x[i] = __ldg(reinterpret_cast<const uint4*>(row + at) + i * 32 + lane);
  } else {
    T* v = reinterpret_cast<T*>(x);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = at + i * 32 + lane;
      v[i] = k < end ? __ldg(row + k) : T(0.f);
    }
  }
}

// 0 in the place of NaN in a lane's part of the draft's row.
__device__ __forceinline__ void no_nan(uint4 (&x)[kPart<float>]) {
  float* v = reinterpret_cast<float*>(x);
#pragma unroll
  for (int i = 0; i < kEach; ++i) v[i] = fmaxf(v[i], 0.f);
}
__device__ __forceinline__ void no_nan(uint4 (&x)[kPart<__nv_bfloat16>]) {
  __nv_bfloat162* v = reinterpret_cast<__nv_bfloat162*>(x);
  const __nv_bfloat162 zero = __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
#pragma unroll
  for (int i = 0; i < kEach / 2; ++i) v[i] = __hmax2(v[i], zero);
}

template <class T>
__device__ __forceinline__ u64 part_sum(const uint4 (&p)[kPart<T>], const uint4 (&q)[kPart<T>],
                                        const Row<T>& row) {
  const T* x = reinterpret_cast<const T*>(p);
  const T* y = reinterpret_cast<const T*>(q);
  u64 sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += fixed(left_of(widen(x[i]), widen(y[i]), row.c));
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
__global__ void __launch_bounds__(kThreads, 4) attn_tree_verify_kernel(const VerifyParams par) {
  __shared__ Shared sm;
  const TreeVerifyProblem& pb = par.pb;
  // (all CTAs of a cluster have started before one writes to another's shared memory)
  if (par.cluster > 1) cluster_arrive();
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
    sm.p[tid] = p > 0.f ? fminf(p, 0x1p99f) : 0.f;  // (infinity has no difference)
    sm.q[tid] = q > 0.f ? fminf(q, 0x1p99f) : 0.f;
    sm.u[tid] = u;
  }
  __syncthreads();

  int scans = 0;
  // The sum of a row over the whole cluster, and the segments' in shared memory.
  // `without`: less the tokens of that node's children (all of them rejected).
  auto scan = [&](const Row<T>& row, int without) -> u64 {
    u64 mine = 0;
    for (int s = warp; s < par.segs; s += kWarps) {
      const int at = begin + s * par.seg, to = min(at + par.seg, end);
      u64 part = 0;
      for (int v = at; v < to; v += kSegment) {
        uint4 p[kPart<T>], q[kPart<T>];
#pragma unroll
        for (int i = 0; i < kPart<T>; ++i) q[i] = make_uint4(0u, 0u, 0u, 0u);
        load_part<T, VEC>(row.p, v, to, lane, p);
        if (row.q) {
          load_part<T, VEC>(row.q, v, to, lane, q);
          no_nan(q);
        }
        part += part_sum(p, q, row);
      }
      if (without >= 0) {
        for (int e = without + 1 + lane; e < pb.n; e += 32) {
          const int x = sm.token[e];
          bool first = sm.parent[e] == without && x >= at && x < to;  // (-1 is in no segment)
          for (int c = without + 1; c < e && first; ++c)
            first = !(sm.parent[c] == without && sm.token[c] == x);
          if (first) part -= fixed(left_at(row, x));
        }
      }
      part = warp_sum(part);
      if (lane == 0) sm.seg[s] = part;
      mine += part;
    }
    // every warp's sum to every CTA, and all of them again there
    u64(&sums)[kMostCluster][kWarps] = sm.sums[scans & 1];
    if (par.cluster > 1) {
      if (scans == 0) cluster_wait();
      if (lane < par.cluster) *cg::this_cluster().map_shared_rank(&sums[rank][warp], lane) = mine;
      cluster_arrive();
      cluster_wait();
    } else {
      if (lane == 0) sums[0][warp] = mine;
      __syncthreads();
    }
    ++scans;
    u64 sum = 0;
    for (int i = lane; i < par.cluster * kWarps; i += 32) sum += (&sums[0][0])[i];
    return warp_sum(sum);
  };

  // ---- the walk: by the first warp, up to where a row has to be summed; all warps
  // sum it
  const bool writes = rank == 0 && tid == 0;
  if (tid == 0) sm.walk = {{0.f, 0.f}, {1.f, 0.f}, 0, 1, 0, false, false};
  if (writes) pb.path[static_cast<long long>(b) * pb.n] = 0;
  u64 sum = 0;
  Row<T> row;
  int without = -1;
  bool at_end = false, own = false;
  while (true) {
    if (!at_end) {
      if (warp == 0) {
        __syncwarp();
        Walk w = sm.walk;
        if (w.rejected) w.Z = draft ? pair_of(sum) : w.Z;
        while (true) {
          int c = pb.n;  // the first child from `next` on
#pragma unroll
          for (int i = kMostNodes / 32 - 1; i >= 0; --i) {
            const int e = 32 * i + lane;
            const unsigned kids = __ballot_sync(0xffffffffu, e >= w.next && sm.parent[e] == w.cur);
            if (kids != 0) c = 32 * i + __ffs(kids) - 1;
          }
          w.at_end = c == pb.n;
          if (w.at_end) break;
          const float q = sm.q[c], u = sm.u[c];
          Pair r{sm.p[c], 0.f};
          if (draft) {
            r = less(r.hi, w.C, q);
            if (!(r.hi > 0.f)) r = {0.f, 0.f};
          } else if (w.rejected) {
            // an earlier child of the same token did not stand: nothing is left of it
            for (int v = w.cur >> 5; v <= c >> 5; ++v) {
              const int e = 32 * v + lane;
              if (__any_sync(0xffffffffu,
                             e < c && sm.parent[e] == w.cur && sm.token[e] == sm.token[c]))
                r = {0.f, 0.f};
            }
          }
          w.next = c + 1;
          const float uz = __fmul_rn(u, w.Z.hi);  // u Z q - r, with what its parts round off
          const float rest = __fmaf_rn(u, w.Z.lo, __fmaf_rn(u, w.Z.hi, -uz));
          if (__fmaf_rn(uz, q, -r.hi) + __fmaf_rn(rest, q, -r.lo) < 0.f) {
            if (writes) pb.path[static_cast<long long>(b) * pb.n + w.len] = c;
            w = {{0.f, 0.f}, {1.f, 0.f}, c, w.len + 1, c + 1, false, false};
          } else {
            w.rejected = true;
            if (draft) {
              w.C = plus(w.C, w.Z);
              break;
            }
            w.Z = plus(w.Z, {-r.hi, -r.lo});
          }
        }
        if (lane == 0) sm.walk = w;
      }
      __syncthreads();  // (the next write of it is behind a barrier of the scan)
      at_end = sm.walk.at_end;
      row = {target + sm.walk.cur * pb.tn,
             draft && sm.walk.rejected ? draft + sm.walk.cur * pb.dn : nullptr, sm.walk.C};
      if (at_end && !draft && sm.walk.rejected) without = sm.walk.cur;
    }
    // (at the end after a rejection the segments hold the row to draw from)
    if (!at_end || own || !sm.walk.rejected || !draft) sum = scan(row, without);
    if (!at_end) continue;
    if (sum != 0 || !sm.walk.rejected || own) break;
    // nothing is left (the draft's row covers the target's): the target's own
    own = true;
    row.q = nullptr;
    without = -1;
  }
  if (rank == 0 && warp == 0) {
    for (int i = sm.walk.len + lane; i < pb.n; i += 32)
      pb.path[static_cast<long long>(b) * pb.n + i] = -1;
    if (lane == 0) pb.path_lens[b] = sm.walk.len;
  }

  // ---- the next token
  if (sum == 0) {
    if (writes) pb.next_tokens[b] = -1;
    return;
  }
  u64 t = part_of(sm.u[0], sum);  // the first token whose running sum exceeds it
  int owner = 0;  // the CTA that it falls to
  for (; owner + 1 < par.cluster; ++owner) {
    u64 run = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) run += sm.sums[(scans - 1) & 1][owner][i];
    if (t < run) break;
    t -= run;
  }
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
  const int stop = min(begin + (s + 1) * par.seg, end);
  for (int v = begin + s * par.seg; v < stop; v += kSegment) {
    const int first = v + lane * kEach;  // of a lane's values, one after the other
    unsigned gone = 0;  // those that are no more there
    if (without >= 0) {
      for (int w = 0; w < kMostNodes / 32; ++w) {
        const int x = sm.parent[32 * w + lane] == without ? sm.token[32 * w + lane] - v : -1;
        unsigned in = __ballot_sync(0xffffffffu, x >= 0 && x < kSegment);
        for (; in != 0; in &= in - 1) {
          const int y = __shfl_sync(0xffffffffu, x, __ffs(in) - 1);
          if (y / kEach == lane) gone |= 1u << (y % kEach);
        }
      }
    }
    float left[kEach];
    mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) left[i] = first + i < stop ? left_at(row, first + i) : 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (gone >> i & 1u) left[i] = 0.f;
      mine += fixed(left[i]);
    }
    const int at = find(mine);
    if (at == 32) continue;
    if (lane == at) {
      int x = 0;
      bool found = false;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        found = found || t < fixed(left[i]);
        if (!found) {
          t -= fixed(left[i]);
          ++x;
        }
      }
      pb.next_tokens[b] = first + min(x, kEach - 1);
    }
    return;
  }
}

template <class T, bool VEC>
cudaError_t launch(const VerifyParams& par, const LaunchCtx& ctx) {
  if (par.cluster > 8) {  // (of the current device: set for each call)
    const cudaError_t e = cudaFuncSetAttribute(
        attn_tree_verify_kernel<T, VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
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
  const int es = pb.bf16 ? 2 : 4;
  // CTAs per sequence: as many as are all resident, four per SM, with at least a
  // segment for each of two warps of each; and up to twice as many where a chain of scans
  // is over runs of 16384 values and more.  Measured (us, with 2, 4, 8, 16 of them):
  // 1 sequence of 131072 fp32 values 21, 14, 11, 9; 32 sequences 53, 33, 24, 21; 64 of
  // 32000 28, 21, 20, 29; 128 of 8000 17, 17, 26, 46; 128 of 131072 97, 69, 63, 74; 100 of
  // 150000 -, 70, 56, 60; without a draft's row 128 of 150000 bf16 values 31, 26, 31, 48.
  int cluster = 1;
  while (cluster < kMostCluster && 2048LL * cluster <= pb.V &&
         2LL * cluster * pb.B <=
             (pb.draft && 32768LL * cluster <= pb.V ? 8LL : 4LL) * ctx.num_sms)
    cluster *= 2;
  par.cluster = cluster;
  const long long most = static_cast<long long>(cluster) * kMostSegments * kSegment;
  par.seg = static_cast<int>(kSegment * ((pb.V + most - 1) / most));
  const int segs = (pb.V + par.seg - 1) / par.seg;
  par.segs = (segs + cluster - 1) / cluster;
  auto whole = [&](const void* base, long long sb, long long sn) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && sb * es % 16 == 0 && sn * es % 16 == 0;
  };
  const bool vec = whole(pb.target, pb.tb, pb.tn) && (!pb.draft || whole(pb.draft, pb.db, pb.dn));
  if (pb.bf16)
    return vec ? launch<__nv_bfloat16, true>(par, ctx) : launch<__nv_bfloat16, false>(par, ctx);
  return vec ? launch<float, true>(par, ctx) : launch<float, false>(par, ctx);
}

}  // namespace attn
