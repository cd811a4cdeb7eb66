// attn_decode_scored.cuh -- a decoding step with changed scores against a
// key/value cache in bf16 or in 8 bits (e4m3 or int8 codes with one scale for
// each block of T tokens and head).  Included by one source file per cache
// format.
//
// For query head h (key head h / G, G query heads share one), new query i of
// n_q, standing at position p_i = L - n_q + i of its sequence of L tokens:
//
//   x_j = cap * tanh(scale * q_i . k_j / cap) - slope_h * (p_i - j)
//   O_i = sum_j softmax_j(x) v_j,   LSE_i = ln sum_j exp(x_j)
//
// over the keys j <= p_i (and j >= p_i - window).  Without a cap the first
// term is the plain score.
//
// Bound by HBM: every visible cache byte is read once for each 32 query rows of a
// key head (G * n_q of them; with more, the tiles of rows each copy the cache in, a
// part of it from L2: 4 x 65536 tokens, d = 128, e4m3, group of 8, 4 queries 93 us, 8
// queries 162).  An 8-bit cache leaves
// 4 FLOPs per byte and query row, so with G * n_q rows per key head the CUDA
// cores would be the bound from about 5 rows on; the products run on the
// tensor cores instead, in the warp-level m16n8k16 form: the tile of queries
// (at most 32 rows) is far too small for a tcgen05 tile, and this form takes
// its operands from registers, where codes are widened on their way from a
// warp's ring of tiles in shared memory:
//   S = Q K^T  queries are the 16 rows, 8 keys the columns;
//   O^T = V^T P^T  16 values of d are the rows, 8 queries the columns: the
//       accumulator layout of S is the operand layout of P^T as it stands.
// The k index of a product may be permuted freely when both operands agree,
// so a lane's 16 consecutive bytes of a key row are whole operands, and the
// rows of O^T likewise, so a lane's 16 consecutive bytes of a value row are.
//
// 8-bit codes are widened to f16, which holds both kinds exactly; q is
// brought to f16 by a power of two per row (within 2^-25 of the row's
// largest entry), and P times the value scale is rounded to f16 as the operand of
// the second product:
//   2^(x_j + log2 v_j - m' + 7),  m' a running maximum of x_j + log2 v_j of its own,
// so that its precision follows what a key adds to the output, whatever the scales
// of keys without weight are, and 2^-21 of the largest of them is still a normal
// f16 number.  The row sum takes exponentials relative to the scores' maximum,
// in fp32.  (With one exponential for both, relative to the largest scale so far, a
// block of large values and no weight took the others' P out of f16's range: O off
// by 1 % at 2^14 times their scale, by 20 % at 2^18.)  A bf16 cache multiplies in
// bf16, P rounded to bf16 as in the forward.  Softmax statistics, scores and
// accumulators are fp32.
//
// Work split, two ways (scored_decode_plan chooses):
//  * whole: every warp takes whole units (a unit is one sequence, key head and
//    tile of query rows), the w-th, the (w + W)-th and so on, and writes them
//    out.  For caches short enough that the longest one is a short job for one
//    warp, and enough of them to occupy the SMs.
//  * split: the visible cache is one list of tiles of KT keys, unit by unit, and
//    every resident warp takes an equal run of it, whatever the lengths are; a
//    run may end one unit and begin another.  Units that several warps share go
//    through the workspace to a second kernel.
// Either way a warp keeps its own running softmax and its own ring of STAGES
// tiles in shared memory, filled by TMA across unit boundaries: it waits for
// its own copies only, never for another warp, and memory stays busy while it
// computes.
//
// TREE: the queries are the nodes of trees of drafted tokens (attn_decode_tree) with
// at most 32 rows to a key head.  Node i stands at L + depth_i and sees the whole cache; what
// it sees of its tree, its ancestors' own keys, is taken by the second kernel, which
// needs nothing of the first for that and does it while the first still runs.  Every
// unit's result therefore goes through the workspace.  Measured: 64 sequences of 64 to
// 512 tokens, 8 heads of d = 64, int8, 16 nodes 21 us (floor 3.4); 32 of 2 to 4 thousand,
// 16 heads, e4m3, caps, 25 nodes 112 us (31), the first kernel 95 of them (four
// special-function operations a score, two of the cap and one for each running maximum, at
// two warps per scheduler); one of 512 tokens, 5 nodes 7.7 us, launches and latencies.
//
// Measured (the floor is the visible cache at the rate of a plain copy, 6.7 TB/s):
// 4 sequences of 65 to 131 thousand tokens, 32 query heads on 8, d = 128, e4m3,
// distance bias: 132 us (floor 121); the same with a bf16 cache at its floor, 235
// us.  32 of 2 to 4 thousand, 16 heads of d = 64, e4m3, caps: 45 us (30), of which
// 7 are the join.  256 of 64 to 512, 8 heads, int8, whole units: 27 us (11); one
// warp's chain of tiles is what it takes, 1.2 us each with 13 warps on an SM (128
// registers a thread leave room for 16).  Copies alone, 32 x 4096 at full length:
// 47 us against the kernel's 55.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_internal.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

using namespace ptx;

enum CacheFormat : int { kCacheBf16 = 0, kCacheE4M3 = 1, kCacheInt8 = 2 };

constexpr int DW = 4;  // warps per CTA
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.4426950408889634f;
// A running maximum is kept until a score exceeds it by more than this (log2
// units): P stays below 2^8, harmless for f16 and the fp32 accumulators.
constexpr float kRescale = 8.0f;
// 8-bit caches: the operand of the second product is 2^7 at its running maximum,
// below 2^15 with the above, inside f16's range.
constexpr float kLift = 7.0f;

struct ScoredDecParams {
  const __nv_bfloat16* q;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* o;
  float* lse;
  float* part;        // [warp][2][query rows][D + kPartTail]: a part of a row's result
  unsigned* first;  // split: [B + 1], the list index of each sequence's first tile, and the total
  const int* cache_lens;
  const float* slopes;
  RowStrides sq, so;
  const uint8_t* k;  // the caches and their byte strides, for copies of runs of rows
  const uint8_t* v;
  RowStrides sk, sv;
  bool run_k, run_v;  // the rows of a head lie side by side
  uint64_t limit_ns;
  int* status;
  int B, HK, G, n_q, L_max, T_log2, num_blocks, window, row_tiles;
  int warps, units;
  bool whole;
  float scale, softcap;
  // TREE
  const int* parents;  // [B][n_q]
  const __nv_bfloat16* k_tree;
  const __nv_bfloat16* v_tree;
  RowStrides skt, svt;
  float* done;  // [unit][query rows][D + kPartTail]: results of units that one warp took
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes of one word to two f16 pairs (codes 0, 1 and codes 2, 3).
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kCacheE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // c + 128 as the low byte of the f16 number 1024 + (c + 128), minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// BYTES (2, 4, 8 or 16) from shared memory into the first words of w.
template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* at, uint32_t* w) {
  if (BYTES == 16) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if (BYTES == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    w[0] = x.x, w[1] = x.y;
  } else if (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  } else {
    w[0] = *reinterpret_cast<const uint16_t*>(at);
  }
}

// Keys per warp and tile for rows of `row_bytes`: 2 KB of keys, 16 to 64 of
// them; 4 KB where the work is split and one tile of query rows leaves the
// registers for it (131072-token contexts 139 -> 132 us; whole short caches are
// faster in small tiles, 27 against 31 us).
constexpr bool scored_big_tiles(int row_bytes, int row_tiles, bool whole) {
  return !whole && row_tiles == 1 && (row_bytes == 64 || row_bytes == 128);
}
constexpr int scored_tile_keys(int row_bytes, bool big) {
  return (row_bytes >= 128 ? 16 : (row_bytes >= 64 ? 32 : 64)) * (big ? 2 : 1);
}
constexpr int scored_stages(bool big) { return big ? 2 : 3; }
// Bytes of a warp's ring: keys and values of its stages.
constexpr int scored_ring(int row_bytes, bool big) {
  return scored_stages(big) * 2 * scored_tile_keys(row_bytes, big) * row_bytes;
}
// Resident CTAs per SM: what the registers allow, by row tiles, and what 228 KB of
// shared memory do (a CTA's rings, 1 KB to align them, 1 KB of its own and 1 KB that
// the system takes): two for the 256-byte rows of a bf16 cache at d = 128.
constexpr int scored_ctas(int row_bytes, int row_tiles, bool big) {
  const int regs = row_tiles > 1 ? 2 : (big ? 3 : 4);
  const int smem = 228 * 1024 / (DW * scored_ring(row_bytes, big) + 3 * 1024);
  return regs < smem ? regs : smem;
}
// A warp's run is at least this many tiles: below it the start of a run and the
// join of its result cost more than the tiles.
constexpr int kMinTiles = 2;

// Shapes per cache format, head size D and row tiles (8 queries each).
template <int FMT_, int D_, int NR_, bool BIG_>
struct DCfg {
  static constexpr int FMT = FMT_, D = D_, NR = NR_;
  static constexpr int ES = FMT_ == kCacheBf16 ? 2 : 1;
  static constexpr int RB = D_ * ES;               // bytes of a cache row
  static constexpr int BB = RB < 128 ? RB : 128;   // bytes of a row in one TMA box
  static constexpr int NB = RB / BB;               // boxes per tile
  static constexpr int KT = scored_tile_keys(RB, BIG_);
  static constexpr uint32_t TILE = KT * RB;        // a tile of keys (or of values)
  static constexpr uint32_t BOX = KT * BB;
  static constexpr int STAGES = scored_stages(BIG_);
  static constexpr int NT = KT / 8;   // 8-key column tiles of S
  static constexpr int NG = KT / 16;  // 16-key groups (one k step of O^T)
  // K: a lane's quarter of a row, in loads of KV bytes
  static constexpr int KV = RB / 4 < 16 ? RB / 4 : 16;
  static constexpr int KW = KV / 4;          // words per load
  static constexpr int KE = KV / ES;         // elements per load
  static constexpr int KB = BB / 4 / KV;     // loads per box
  static constexpr int KL = NB * KB;         // loads per row
  static constexpr int KS = D_ / 16;         // k steps of S
  // V: a lane's eighth of a row, in loads of VV bytes, one per box
  static constexpr int VV = BB / 8;
  static constexpr int VW = VV < 4 ? 1 : VV / 4;
  static constexpr int VE = VV / ES;
  static constexpr int MT = D_ / 16;                // 16-row tiles of O^T
  static constexpr int MQ = NR_ > 1 ? NR_ / 2 : 1;  // 16-query tiles of S
  static constexpr uint32_t RING = scored_ring(RB, BIG_);  // shared memory of a warp
  static constexpr int CTAS = scored_ctas(RB, NR_, BIG_);
  // Rows shorter than 128 bytes whose cache rows lie side by side are copied as
  // one run of bytes: a tiled copy takes about four cycles of the SM's copy
  // engine per box row, which for 64-byte rows is the time of 16 bytes a cycle,
  // less than an SM's share of the memory rate.
  static constexpr bool RUNS = RB < 128;
  // Which key of an 8-key tile is column c: for 32-byte rows an order in which
  // the rows that a value load touches do not share banks.
  static constexpr uint32_t ORDER = RB == 32 ? 0x57463120u : 0x76543210u;
  __device__ static constexpr int key_of(int c) { return (ORDER >> (4 * c)) & 7; }
  // the 16-byte chunk position XOR of row r: 128-byte rows are swizzled
  __device__ static constexpr uint32_t swz(uint32_t r) { return BB == 128 ? r & 7 : 0u; }
  static_assert(RB >= 128 || NB == 1, "one box");
};

// The d index of the first element that lane t holds for k step s of S: the
// lane's words in load order, four elements per step.
template <class C>
__device__ __forceinline__ int key_elem(int step, int t) {
  constexpr int per = C::KE / 4;  // steps per load
  const int load = step / per, box = load / C::KB, i = load % C::KB;
  return box * (C::BB / C::ES) + (t * C::KB + i) * C::KE + 4 * (step % per);
}
// The d index of a lane's e-th value element (group g).
template <class C>
__device__ __forceinline__ int val_elem(int e, int g) {
  return (e / C::VE) * 8 * C::VE + g * C::VE + e % C::VE;
}

// The visible keys of a sequence, in tiles.
struct SeqTiles {
  int L;      // tokens in the cache
  int key0;   // first key that any of the queries sees
  int base0;  // where its tiles begin: a tile boundary, so that no tile (or no 16-key
              // group of it) crosses a scale block
  int tiles;
};
template <int KT, bool TREE>
__device__ __forceinline__ SeqTiles seq_tiles(const ScoredDecParams& p, int b) {
  SeqTiles s;
  s.L = p.L_max;
  if (p.cache_lens != nullptr) s.L = min(max(__ldg(p.cache_lens + b), 0), p.L_max);
  s.key0 = p.window >= 0 ? max(s.L - (TREE ? 0 : p.n_q) - p.window, 0) : 0;
  s.base0 = s.key0 & ~(KT - 1);
  s.tiles = (s.L - s.base0 + KT - 1) / KT;
  if (TREE && s.key0 >= s.L) s.tiles = 0;  // (a window of no key before the tree)
  return s;
}

// A place in a warp's work: a tile of a unit = b * subs + sub, sub = key head *
// row_tiles + row tile.
template <int KT, bool TREE>
struct Cursor {
  SeqTiles s;
  int unit, b, sub, tile;
  __device__ __forceinline__ void at_unit(const ScoredDecParams& p, int subs, int u) {
    unit = u;
    tile = 0;
    const int nb = u / static_cast<unsigned>(subs);
    sub = u - nb * subs;
    if (nb != b) {
      b = nb;
      s = seq_tiles<KT, TREE>(p, b);
    }
  }
  // the next unit of this warp; with skip, the next one that has tiles
  __device__ __forceinline__ bool next(const ScoredDecParams& p, int subs, bool skip) {
    const int step = p.whole ? p.warps : 1;
    int u = unit;
    do {
      if (p.units - u <= step) return false;
      u += step;
      at_unit(p, subs, u);
    } while (skip && s.tiles == 0);
    return true;
  }
};

// Accumulators relative to 2^from, over a row sum relative to 2^m: times this
// factor twice (its square may leave fp32 where the result does not).
__device__ __forceinline__ float value_factor(float from, float m) {
  return from == -INFINITY ? 0.f : ex2(0.5f * (from - m));
}

// Tiles per warp: an equal share, kMinTiles at least.
__device__ __forceinline__ unsigned share_of(unsigned total, int warps) {
  const unsigned each = total / static_cast<unsigned>(warps) + 1;
  return each < kMinTiles ? kMinTiles : each;
}

// The depth of a tree's node `lane` (0 where there is no node), n <= 32, by a warp: after
// round k of pointer doubling a node knows how far its 2^k-th ancestor is.
__device__ __forceinline__ int node_depth(const int* parents, int n, int lane) {
  int up = lane < n ? __ldg(parents + lane) : -2;
  if (up < -1 || up >= lane) up = -2;
  int depth = up >= 0 ? 1 : 0;
  for (int r = 1; r < n; r *= 2) {
    const int from = max(up, 0), far = __shfl_sync(0xffffffffu, depth, from),
              further = __shfl_sync(0xffffffffu, up, from);
    if (up >= 0) {
      depth += far;
      up = further;
    }
  }
  return up == -1 ? depth : 0;
}

template <int FMT, int D, int NR, bool BIG, bool TREE>
__global__ void __launch_bounds__(DW * 32, DCfg<FMT, D, NR, BIG>::CTAS)
    attn_decode_scored_kernel(const __grid_constant__ CUtensorMap tmk,
                              const __grid_constant__ CUtensorMap tmv, const ScoredDecParams p) {
  using C = DCfg<FMT, D, NR, BIG>;
  constexpr int KT = C::KT, NT = C::NT, NG = C::NG, MQ = C::MQ;
  constexpr bool Q8 = FMT != kCacheBf16;
  constexpr int ROWS = NR * 8;
  constexpr int RS = NR > 1 ? 2 : 1;  // used 8-row halves of a 16-query tile
  extern __shared__ uint8_t smem_raw[];
  // the rings at a 1024-byte boundary (an offset, so that the compiler still
  // knows the address space)
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[DW][C::STAGES];
  grid_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int subs = p.HK * p.row_tiles;
  const int w = blockIdx.x * DW + warp;

  // ---- where this warp's work begins, and how many tiles it is
  Cursor<KT, TREE> cur;
  cur.b = -1;
  int count = 0;
  if (p.whole) {
    if (w >= p.warps) return;
    cur.at_unit(p, subs, w);
    Cursor<KT, TREE> c = cur;
    do count += c.s.tiles;
    while (c.next(p, subs, false));
  } else {
    __shared__ unsigned upto[DW * 32];  // tiles of the list up to each thread's sequences
    __shared__ unsigned warp_sum[DW];
    // thread i sums the sequences [i, i + 1) * per
    const int per = (p.B + DW * 32 - 1) / (DW * 32);
    const int seq0 = min(static_cast<int>(threadIdx.x) * per, p.B), seq1 = min(seq0 + per, p.B);
    unsigned sum = 0;
    for (int b = seq0; b < seq1; ++b) sum += seq_tiles<KT, TREE>(p, b).tiles;
    sum *= subs;
    unsigned run = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, run, m);
      if (lane >= m) run += x;
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    unsigned total = 0;
#pragma unroll
    for (int i = 0; i < DW; ++i) {
      if (i < warp) run += warp_sum[i];
      total += warp_sum[i];
    }
    upto[threadIdx.x] = run;
    if (blockIdx.x == 0) {  // for the second kernel
      unsigned at = run - sum;
      for (int b = seq0; b < seq1; ++b) {
        p.first[b] = at;
        at += seq_tiles<KT, TREE>(p, b).tiles * subs;
      }
      if (threadIdx.x == 0) p.first[p.B] = total;
    }
    __syncthreads();
    const unsigned share = share_of(total, p.warps);
    // (share * warps stays below 2^32: total < 2^31, and warps * kMinTiles is small)
    const unsigned begin = share * w;
    if (w >= p.warps || begin >= total) return;  // a whole warp; no barrier of the CTA follows
    count = min(share, total - begin);
    int chunk = 0;
#pragma unroll
    for (int i = 0; i < DW; ++i)
      chunk += __popc(__ballot_sync(0xffffffffu, upto[i * 32 + lane] <= begin));
    unsigned at = chunk > 0 ? upto[chunk - 1] : 0u;
    int b = chunk * per;
    for (;; ++b) {
      cur.s = seq_tiles<KT, TREE>(p, b);
      const unsigned here = static_cast<unsigned>(cur.s.tiles) * subs;
      if (begin - at < here || b + 1 >= p.B) break;
      at += here;
    }
    cur.b = b;
    cur.sub = (begin - at) / static_cast<unsigned>(cur.s.tiles);
    cur.tile = (begin - at) - static_cast<unsigned>(cur.sub) * cur.s.tiles;
    cur.unit = b * subs + cur.sub;
  }

  // ---- this warp's ring
  uint8_t* const ring_at = sm + warp * C::RING;
  const uint32_t ring = smem_u32(ring_at);
  const uint32_t bars = smem_u32(&full[warp][0]);
  const int never = 0;
  Cursor<KT, TREE> ahead = cur;  // where the next copy is from (lane 0)
  if (ahead.s.tiles == 0) ahead.next(p, subs, true);
  auto fill = [&](uint32_t slot) {  // the next tile into a slot (one lane)
    const uint32_t bar = bars + 8 * slot;
    const int row = ahead.s.base0 + ahead.tile * KT;
    const int hk = p.row_tiles == 1 ? ahead.sub : ahead.sub / p.row_tiles;
    const uint32_t dst = ring + slot * 2 * C::TILE;
    if (C::RUNS) {
      // (rows past L_max are not copied: what the slot held there is masked)
      const uint32_t bytes = min(KT, p.L_max - row) * C::RB;
      mbar_arrive_expect_tx(bar, (p.run_k ? bytes : C::TILE) + (p.run_v ? bytes : C::TILE));
      if (p.run_k)
        bulk_copy_in(dst, p.k + ahead.b * p.sk.b + hk * p.sk.h + static_cast<long long>(row) * C::RB,
                     bytes, bar);
      else
        tma_load_4d(dst, &tmk, bar, 0, row, hk, ahead.b);
      if (p.run_v)
        bulk_copy_in(dst + C::TILE,
                     p.v + ahead.b * p.sv.b + hk * p.sv.h + static_cast<long long>(row) * C::RB,
                     bytes, bar);
      else
        tma_load_4d(dst + C::TILE, &tmv, bar, 0, row, hk, ahead.b);
    } else {
      mbar_arrive_expect_tx(bar, 2 * C::TILE);
#pragma unroll
      for (int x = 0; x < C::NB; ++x) {
        tma_load_4d(dst + x * C::BOX, &tmk, bar, x * C::BB, row, hk, ahead.b);
        tma_load_4d(dst + C::TILE + x * C::BOX, &tmv, bar, x * C::BB, row, hk, ahead.b);
      }
    }
    if (++ahead.tile == ahead.s.tiles) ahead.next(p, subs, true);
  };
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
    for (int n = 0; n < min(count, C::STAGES); ++n) fill(n);
  }
  __syncwarp();

  // this lane's rows of an 8-key tile: one as a key, two (a column pair) as values
  const int krow = C::key_of(g), vrow0 = C::key_of(2 * t), vrow1 = C::key_of(2 * t + 1);
  const bool capped = p.softcap > 0.f, biased = p.slopes != nullptr;
  const bool wide_cap = p.softcap > kWideCap;
  const float cap2 = p.softcap * kLog2e;
  // a product times this is the score in log2 units, or the cap's exponent
  const float unit_scale = p.scale * kLog2e * (capped ? 2.f / p.softcap : 1.f);

  bool ok = true;
  int it = 0;
  uint32_t slot = 0, phase = 0;  // of tile `it`
  do {
  // ---- one unit of the work: `seg` of its tiles
  const int seg = min(cur.s.tiles - cur.tile, count - it);
  const int seg_it = it;
  const bool leads = it == 0;
  const int b = cur.b, hk = p.row_tiles == 1 ? cur.sub : cur.sub / p.row_tiles, rt = cur.sub - hk * p.row_tiles;
  const int rows = min(p.G * p.n_q - rt * ROWS, ROWS);  // query rows of this unit
  const int L = cur.s.L, key0 = cur.s.key0, base0 = cur.s.base0 + cur.tile * KT;
  // first key that the last query sees
  const int last_lo = p.window >= 0 ? max(L - 1 + (TREE ? p.n_q : 0) - p.window, 0) : 0;
  const long long bk = static_cast<long long>(b) * p.HK + hk;
  const float* ksp = Q8 ? p.k_scale + bk * p.num_blocks : nullptr;
  const float* vsp = Q8 ? p.v_scale + bk * p.num_blocks : nullptr;
  // one scale per 16-key group; where blocks are no smaller than tiles, one per tile
  const bool one_block = (1 << p.T_log2) >= KT;
  auto load_scales = [&](const float* from, int base, float (&to)[NG]) {
    // (never a block outside the visible keys: its scale may be anything)
    to[0] = __ldg(from + (max(base, key0) >> p.T_log2));
    if (one_block) {
#pragma unroll
      for (int n = 1; n < NG; ++n) to[n] = to[0];
    } else {
#pragma unroll
      for (int n = 1; n < NG; ++n)
        to[n] = __ldg(from + (max(min(base + 16 * n, L - 1), key0) >> p.T_log2));
    }
  };
  float ks[NG], vs[NG];
  if (Q8 && seg > 0) {
    load_scales(ksp, base0, ks);
    load_scales(vsp, base0, vs);
  }

  // Queries in operand form: rows g and g + 8 of each 16-query tile.
  uint32_t qa[MQ][C::KS][4];
  float qscale[MQ][2], nslope[MQ][2];
  int pos[MQ][2];
  int depth = 0;  // TREE: of node `lane`
  if (TREE && (biased || p.window >= 0))
    depth = node_depth(p.parents + static_cast<long long>(b) * p.n_q, p.n_q, lane);
#pragma unroll
  for (int m = 0; m < MQ; ++m) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = m * 16 + r * 8 + g;
      const bool in = row < rows && (NR > 1 || r == 0);
      const int gr = rt * ROWS + (in ? row : 0);
      const int in_group = p.n_q == 1 ? gr : gr / p.n_q, qi = gr - in_group * p.n_q;
      const int head = hk * p.G + in_group;
      const __nv_bfloat16* src = p.q + b * p.sq.b + head * p.sq.h + qi * p.sq.n;
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        const uint2 w = in ? __ldg(reinterpret_cast<const uint2*>(src + key_elem<C>(s, t)))
                           : make_uint2(0u, 0u);
        qa[m][s][r] = w.x;
        qa[m][s][r + 2] = w.y;
        if (Q8) {
          const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
          const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
          top = fmaxf(fmaxf(fmaxf(top, fabsf(x.x)), fmaxf(fabsf(x.y), fabsf(y.x))), fabsf(y.y));
        }
      }
      qscale[m][r] = unit_scale;
      if (Q8) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(min(static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127, 126), -126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        qscale[m][r] = unit_scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t& w = qa[m][s][r + 2 * hf];
            const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
            const __half2 y = __floats2half2_rn(x.x * down, x.y * down);
            w = *reinterpret_cast<const uint32_t*>(&y);
          }
        }
      }
      if (TREE) {
        pos[m][r] = L + __shfl_sync(0xffffffffu, depth, qi);
      } else {
        pos[m][r] = in ? L - p.n_q + qi : -1;
      }
      nslope[m][r] = p.slopes != nullptr && in ? -__ldg(p.slopes + head) * kLog2e : 0.f;
    }
  }
  // maximum and sum of a row; mv_run: maximum of the scores times their value scales
  float m_run[MQ][2], l_run[MQ][2], mv_run[MQ][2];
  float acc[C::MT][NR][4];
#pragma unroll
  for (int m = 0; m < MQ; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) m_run[m][r] = mv_run[m][r] = -INFINITY, l_run[m][r] = 0.f;
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;

  for (int k = 0; k < seg; ++k, ++it) {
    const int base = base0 + k * KT;
    ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * slot, phase, p.limit_ns, &never));
    if (!ok) break;
    const uint8_t* kt = ring_at + slot * 2 * C::TILE;
    const uint8_t* vt = kt + C::TILE;
    // ---- S = Q K^T
    float s[MQ][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int m = 0; m < MQ; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
      const uint32_t r = 8 * n + krow;
      uint32_t kr[C::KL * C::KW];
#pragma unroll
      for (int i = 0; i < C::KL; ++i) {
        // byte t * KV * KB + i * KV of the row's box
        const uint32_t byte = (t * C::KB + i % C::KB) * C::KV;
        load_bytes<C::KV>(kt + (i / C::KB) * C::BOX + r * C::BB +
                              ((byte & ~15u) ^ (C::swz(r) << 4)) + (byte & 15u),
                          &kr[i * C::KW]);
      }
#pragma unroll
      for (int st = 0; st < C::KS; ++st) {
        uint32_t b0, b1;
        if (Q8) {
          widen4<FMT>(kr[st], b0, b1);  // word st: elements 4 st .. 4 st + 3 of the lane
        } else {
          b0 = kr[2 * st];
          b1 = kr[2 * st + 1];
        }
#pragma unroll
        for (int m = 0; m < MQ; ++m) {
          if (Q8)
            mma_f16(s[m][n], qa[m][st][0], qa[m][st][1], qa[m][st][2], qa[m][st][3], b0, b1);
          else
            mma_bf16(s[m][n], qa[m][st][0], qa[m][st][1], qa[m][st][2], qa[m][st][3], b0, b1);
        }
      }
    }

    // every row sees every key of the tile, unless it is an edge of the cache
    // or of the window
    const bool edge = base + KT > L - (TREE ? 0 : p.n_q - 1) || base < last_lo;

    float lv[NG];  // the groups' value scales in log2 units (a scale of 0: -inf)
#pragma unroll
    for (int n = 0; n < NG; ++n) lv[n] = Q8 ? __log2f(vs[n]) : 0.f;

    // ---- scores in log2 units are s * f (f = 1 once the cap or the bias is
    // in), masked; mx: this lane's largest of a row, mxv: with their value scales
    float mx[MQ][2], mxv[MQ][2], f[MQ][2][NG];
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        // (never 0, so that a masked score stays -inf)
#pragma unroll
        for (int n = 0; n < NG; ++n)
          f[m][r][n] = Q8 ? fmaxf(qscale[m][r] * ks[n], 1e-37f) : qscale[m][r];
        if (capped || biased) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[m][n][2 * r] *= f[m][r][n / 2];
            s[m][n][2 * r + 1] *= f[m][r][n / 2];
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) f[m][r][n] = 1.f;
          if (capped) {
            // tanh(y) = 1 - 2 / (1 + 2^(2 y log2(e))); the exponent is in place
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                // (a in exponent units: y = a / (2 log2(e)))
                const float a = s[m][n][2 * r + c];
                float x = fmaf(-2.f * cap2, rcp(1.f + ex2(a)), cap2);
                if (wide_cap && fabsf(a) <= 2.f * kLog2e * static_cast<float>(kTanhSmall)) {
                  const float y = a * (0.5f / kLog2e), z = y * y;
                  x = cap2 * y * fmaf(z, fmaf(z, static_cast<float>(kTanh2), static_cast<float>(kTanh1)),
                                      static_cast<float>(kTanh0));
                }
                s[m][n][2 * r + c] = x;
              }
          }
          if (biased) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // distance to this lane's key of the first 8-key tile
              const float far = static_cast<float>(pos[m][r] - base - (c ? vrow1 : vrow0));
#pragma unroll
              for (int n = 0; n < NT; ++n)
                s[m][n][2 * r + c] = fmaf(nslope[m][r], far - static_cast<float>(8 * n),
                                          s[m][n][2 * r + c]);
            }
          }
        }
        if (edge) {
          // keys [lo, hi) of the tile are visible
          const int hi = (TREE ? L : pos[m][r] + 1) - base;
          const int lo = p.window >= 0 ? max(pos[m][r] - p.window, key0) - base : -base;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = 8 * n + (c ? vrow1 : vrow0);
              if (col >= hi || col < lo) s[m][n][2 * r + c] = -INFINITY;
            }
        }
        mx[m][r] = mxv[m][r] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const float top = f[m][r][n] * fmaxf(fmaxf(s[m][2 * n][2 * r], s[m][2 * n][2 * r + 1]),
                                               fmaxf(s[m][2 * n + 1][2 * r],
                                                     s[m][2 * n + 1][2 * r + 1]));
          mx[m][r] = fmaxf(mx[m][r], top);
          if (Q8) mxv[m][r] = fmaxf(mxv[m][r], top + lv[n]);
        }
      }
    }
    bool grow = false;
#pragma unroll
    for (int m = 0; m < MQ; ++m)
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        grow |= mx[m][r] > m_run[m][r] + kRescale;
        if (Q8) grow |= mxv[m][r] > mv_run[m][r] + kRescale;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int m = 0; m < MQ; ++m) {
#pragma unroll
        for (int r = 0; r < RS; ++r) {
          float top = mx[m][r], alpha = 1.f;
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if (top > m_run[m][r] + kRescale) {
            alpha = ex2(m_run[m][r] - top);  // 0 when nothing was seen before
            m_run[m][r] = top;
            l_run[m][r] *= alpha;
          }
          if (Q8) {  // the accumulators follow the other maximum
            alpha = 1.f;
            top = mxv[m][r];
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > mv_run[m][r] + kRescale) {
              alpha = ex2(mv_run[m][r] - top);
              mv_run[m][r] = top;
            }
          }
          // this lane's accumulator columns are queries 2t and 2t + 1
          const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t);
          const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
#pragma unroll
          for (int i = 0; i < C::MT; ++i) {
            acc[i][2 * m + r][0] *= a0;
            acc[i][2 * m + r][1] *= a1;
            acc[i][2 * m + r][2] *= a0;
            acc[i][2 * m + r][3] *= a1;
          }
        }
      }
    }
    // ---- P, its row sums, and P^T (times the value scales) as the operand of O^T
    uint32_t pb[NG][NR][2];
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        const float neg_m = m_run[m][r] == -INFINITY ? 0.f : -m_run[m][r];
        const float neg_mv = mv_run[m][r] == -INFINITY ? 0.f : kLift - mv_run[m][r];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const float fn = f[m][r][n];
          const float s0 = s[m][2 * n][2 * r], s1 = s[m][2 * n][2 * r + 1],
                      s2 = s[m][2 * n + 1][2 * r], s3 = s[m][2 * n + 1][2 * r + 1];
          const float p0 = ex2(fmaf(s0, fn, neg_m)), p1 = ex2(fmaf(s1, fn, neg_m)),
                      p2 = ex2(fmaf(s2, fn, neg_m)), p3 = ex2(fmaf(s3, fn, neg_m));
          l_run[m][r] += (p0 + p1) + (p2 + p3);
          if (Q8) {
            const float off = neg_mv + lv[n];
            const __half2 y = __floats2half2_rn(ex2(fmaf(s0, fn, off)), ex2(fmaf(s1, fn, off))),
                          z = __floats2half2_rn(ex2(fmaf(s2, fn, off)), ex2(fmaf(s3, fn, off)));
            pb[n][2 * m + r][0] = *reinterpret_cast<const uint32_t*>(&y);
            pb[n][2 * m + r][1] = *reinterpret_cast<const uint32_t*>(&z);
          } else {
            pb[n][2 * m + r][0] = pack_bf16x2(p0, p1);
            pb[n][2 * m + r][1] = pack_bf16x2(p2, p3);
          }
        }
      }
    }
    if (Q8 && k + 1 < seg) {  // the next tile's scales
      load_scales(ksp, base + KT, ks);
      load_scales(vsp, base + KT, vs);
    }
    // ---- O^T += V^T P^T
    if (base < key0 || base + KT > L) {
      // rows that are no keys of this sequence may hold anything (NaN): zero
      // them in the ring
#pragma unroll 1
      for (int i = lane; i < KT * C::RB / 16; i += 32) {
        const int r = i % KT, j = base + r;  // chunk i / KT of the row's boxes
        if (j < key0 || j >= L)
          *reinterpret_cast<uint4*>(ring_at + slot * 2 * C::TILE + C::TILE +
                                    (i / KT) / (C::BB / 16) * C::BOX + r * C::BB +
                                    (i / KT) % (C::BB / 16) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      // rows of keys 2t, 2t + 1, 2t + 8 and 2t + 9 (columns of S) of the group
      uint32_t vr[4][C::NB * C::VW];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t r = 16 * n + ((e & 1) ? vrow1 : vrow0) + (e >> 1) * 8;
        const uint32_t byte = g * C::VV;
#pragma unroll
        for (int i = 0; i < C::NB; ++i)
          load_bytes<C::VV>(vt + i * C::BOX + r * C::BB +
                                ((byte & ~15u) ^ (C::swz(r) << 4)) + (byte & 15u),
                            &vr[e][i * C::VW]);
      }
      // pairs (key 2t, 2t+1) and (2t+8, 2t+9) of one d each
      auto product = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
          if (Q8)
            mma_f16(acc[i][x], a0, a1, a2, a3, pb[n][x][0], pb[n][x][1]);
          else
            mma_bf16(acc[i][x], a0, a1, a2, a3, pb[n][x][0], pb[n][x][1]);
        }
      };
      if (Q8) {
#pragma unroll
        for (int w = 0; w < C::NB * C::VW; ++w) {
          // elements 4w .. 4w+3 of the lane: two 16-row tiles (one when D = 16)
          uint32_t a[2][2], c[2][2];
          widen4<FMT>(__byte_perm(vr[0][w], vr[1][w], 0x5140), a[0][0], a[0][1]);
          widen4<FMT>(__byte_perm(vr[2][w], vr[3][w], 0x5140), c[0][0], c[0][1]);
          product(2 * w, a[0][0], a[0][1], c[0][0], c[0][1]);
          if (C::MT > 1) {
            widen4<FMT>(__byte_perm(vr[0][w], vr[1][w], 0x7362), a[1][0], a[1][1]);
            widen4<FMT>(__byte_perm(vr[2][w], vr[3][w], 0x7362), c[1][0], c[1][1]);
            product((2 * w + 1) % C::MT, a[1][0], a[1][1], c[1][0], c[1][1]);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < C::MT; ++w) {
          product(w, __byte_perm(vr[0][w], vr[1][w], 0x5410),
                  __byte_perm(vr[0][w], vr[1][w], 0x7632),
                  __byte_perm(vr[2][w], vr[3][w], 0x5410),
                  __byte_perm(vr[2][w], vr[3][w], 0x7632));
        }
      }
    }
    // every lane has read (and perhaps written) the slot: its next tile may
    // land in it
    if (base < key0 || base + KT > L) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && it + C::STAGES < count) fill(slot);
    if (++slot == C::STAGES) slot = 0, phase ^= 1;
  }
  if (!ok) break;

  // ---- this warp's result of the unit: whole, or a part of it
#pragma unroll
  for (int m = 0; m < MQ; ++m)
#pragma unroll
    for (int r = 0; r < RS; ++r) {
      l_run[m][r] += __shfl_xor_sync(0xffffffffu, l_run[m][r], 1);
      l_run[m][r] += __shfl_xor_sync(0xffffffffu, l_run[m][r], 2);
    }
  const bool whole_unit = it - seg_it == cur.s.tiles;
  float* part = p.part + (static_cast<long long>(w) * 2 + (leads ? 0 : 1)) * ROWS * (D + kPartTail);
  if (TREE && whole_unit) part = p.done + static_cast<long long>(cur.unit) * ROWS * (D + kPartTail);
#pragma unroll
  for (int x = 0; x < NR; ++x) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // this lane's accumulators hold query rows 2t + c of the 8-row tile x
      const float mm = __shfl_sync(0xffffffffu, m_run[x / 2][x & 1], 8 * t + 4 * c);
      const float ll = __shfl_sync(0xffffffffu, l_run[x / 2][x & 1], 8 * t + 4 * c);
      // what the accumulators are relative to
      const float from = Q8 ? __shfl_sync(0xffffffffu, mv_run[x / 2][x & 1], 8 * t + 4 * c) - kLift : mm;
      const int row = x * 8 + 2 * t + c;
      if (row >= rows) continue;
      if (!TREE && whole_unit) {
        const int gr = rt * ROWS + row;
        const int in_group = p.n_q == 1 ? gr : gr / p.n_q, qi = gr - in_group * p.n_q;
        const int head = hk * p.G + in_group;
        const float fac = Q8 ? value_factor(from, mm) : 1.f;
        const float inv = (ll > 0.f ? 1.f / ll : 0.f) * fac;
        __nv_bfloat16* out = p.o + b * p.so.b + head * p.so.h + qi * p.so.n;
        uint32_t word[C::MT];
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
          word[i] = pack_bf16x2(acc[i][x][c] * fac * inv, acc[i][x][2 + c] * fac * inv);
        constexpr int V = C::VE / 2 < 4 ? C::VE / 2 : 4;  // words side by side
#pragma unroll
        for (int i = 0; i < C::MT; i += V) {
          __nv_bfloat16* at = out + val_elem<C>(2 * i, g);
          if (V == 4)
            *reinterpret_cast<uint4*>(at) = make_uint4(word[i], word[i + 1], word[i + 2], word[i + 3]);
          else if (V == 2)
            *reinterpret_cast<uint2*>(at) = make_uint2(word[i], word[i + 1]);
          else
            *reinterpret_cast<uint32_t*>(at) = word[i];
        }
        if (g == 0 && p.lse != nullptr)
          p.lse[(static_cast<long long>(b) * p.HK * p.G + head) * p.n_q + qi] =
              ll > 0.f ? (mm + __log2f(ll)) * kLn2 : -INFINITY;
      } else {
        float* at = part + row * (D + kPartTail);
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
          *reinterpret_cast<float2*>(at + val_elem<C>(2 * i, g)) =
              make_float2(acc[i][x][c], acc[i][x][2 + c]);
        if (g == 0) *reinterpret_cast<float4*>(at + D) = make_float4(mm, ll, from, 0.f);
      }
    }
  }
  } while ((p.whole || it < count) && cur.next(p, subs, !p.whole));
  if (!ok && lane == 0) {
    atomicCAS(p.status, kDevOk, kDevTimeout);
    // copies still in flight land before the shared memory goes away
    for (int n = it; n < min(count, it + C::STAGES); ++n)
      mbar_wait(bars + 8 * (n % C::STAGES), (n / C::STAGES) & 1, p.limit_ns, &never);
  }
}

// What a node sees of its tree: O relative to 2^m, a lane's values side by side.
template <int E>
struct OwnPart {
  float a[E], m, l;
  bool node;
};

// E values of a bf16 row, one load.
template <int E>
__device__ __forceinline__ void load_values(const __nv_bfloat16* at, float (&x)[E]) {
  if constexpr (E == 1) {
    x[0] = __bfloat162float(*at);
  } else if constexpr (E == 2) {
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(at));
    x[0] = y.x;
    x[1] = y.y;
  } else {
    static_assert(E == 4, "head sizes up to 128");
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    const float2 y = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w.x)),
                 z = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w.y));
    x[0] = y.x;
    x[1] = y.y;
    x[2] = z.x;
    x[3] = z.y;
  }
}

// By a warp: the node's lineage in the lanes first, then N ancestors at a time (the
// node itself first): their products by N-fold sums across the warp, after which lane
// l has the score of ancestor l / (32 / N), so that cap, bias and exponential are
// computed once for each.
template <int D>
__device__ __forceinline__ OwnPart<(D + 31) / 32> tree_part(const ScoredDecParams& p, int b, int hk,
                                                            int in_group, int node, int lane) {
  constexpr int E = (D + 31) / 32, N = E == 1 ? 8 : 4, W = 32 / N;
  OwnPart<E> own;
  const int* parents = p.parents + static_cast<long long>(b) * p.n_q;
  int up = lane < p.n_q ? __ldg(parents + lane) : -2;
  if (up < -1 || up >= lane) up = -2;
  // ancestor i (0: the node) in lane i
  int line = node, at = node, length = 0;
  for (; at >= 0; ++length) {
    if (lane == length) line = at;
    at = __shfl_sync(0xffffffffu, up, at);
  }
  own.node = at == -1;
  own.m = -INFINITY;
  own.l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) own.a[e] = 0.f;
  if (!own.node) return own;
  if (p.window >= 0) length = min(length, p.window + 1);
  const int head = hk * p.G + in_group;
  const int el = min(lane * E, D - E);  // (d = 16: the upper lanes have no part)
  const __nv_bfloat16* q = p.q + b * p.sq.b + head * p.sq.h + node * p.sq.n + el;
  const __nv_bfloat16* k = p.k_tree + b * p.skt.b + hk * p.skt.h + el;
  const __nv_bfloat16* v = p.v_tree + b * p.svt.b + hk * p.svt.h + el;
  const float slope = p.slopes != nullptr ? __ldg(p.slopes + head) * kLog2e : 0.f;
  float x[E];
  load_values<E>(q, x);
  float l = 0.f;  // of this lane's ancestors
  for (int back = 0; back < length; back += N) {
    float s[N], val[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // (past the last: the node itself, at weight 0)
      const int far = back + i, who = __shfl_sync(0xffffffffu, line, far & 31);
      float key[E];
      load_values<E>(k + who * p.skt.n, key);
      load_values<E>(v + who * p.svt.n, val[i]);
      s[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (D >= 32 || lane < D) s[i] = fmaf(x[e], key[e], s[i]);
        if (far >= length) val[i][e] = 0.f;
      }
    }
    // each step halves the ancestors that a lane sums, by exchange with lane ^ w
#pragma unroll
    for (int w = 16, have = N; w > 0; w >>= 1) {
      if (have > 1) {
        have >>= 1;
#pragma unroll
        for (int i = 0; i < have; ++i) {
          const bool upper = lane & w;
          const float keep = upper ? s[i + have] : s[i], give = upper ? s[i] : s[i + have];
          s[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
      } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], w);
      }
    }
    const int far = back + lane / W;
    float y = s[0] * p.scale;
    if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
    y = far < length ? fmaf(-slope, static_cast<float>(far), y * kLog2e) : -INFINITY;
    float top = y;
#pragma unroll
    for (int w = 16; w >= W; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    top = fmaxf(top, own.m);
    const float base = top == -INFINITY ? 0.f : top;  // (scores of -inf weigh nothing)
    const float alpha = ex2(own.m - base);  // 0 at first
    own.m = top;
    const float share = ex2(y - base);
    l = fmaf(l, alpha, share);
#pragma unroll
    for (int e = 0; e < E; ++e) own.a[e] *= alpha;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = __shfl_sync(0xffffffffu, share, i * W);
#pragma unroll
      for (int e = 0; e < E; ++e) own.a[e] = fmaf(w, val[i][e], own.a[e]);
    }
  }
#pragma unroll
  for (int w = 16; w >= W; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  own.l = l;
  return own;
}

// Joins the parts of a query row.  ONE_WARP: a warp per row, eight rows to a
// CTA, for the few parts that a unit has when there are many units; else a CTA
// of eight warps per row, each warp every eighth part.  Units that one warp of
// the first kernel covered are complete; units without keys get O = 0 and LSE
// = -inf here.
// (0: no bound.  One CTA per SM for a bound takes 40 to 53 registers where none takes 32 to
// 46, and 8 sequences of 8 thousand tokens, 32 heads on 8, d = 128, 8 new queries 60.2 us
// instead of 59.0, 32 of 4 thousand, d = 16 11.7 instead of 11.3)
template <int D, int ROWS, bool ONE_WARP, bool TREE>
__global__ void __launch_bounds__(256, TREE ? 5 : 0)
    attn_decode_scored_merge_kernel(const ScoredDecParams p, unsigned total_rows) {
  constexpr int E = (D + 31) / 32;
  __shared__ float joined[ONE_WARP ? 1 : 8][D + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a lane's values: side by side for a tree's, as its loads are
  using Values = typename std::conditional<E == 4, float4, float2>::type;
  auto elem = [lane](int e) { return TREE ? lane * E + e : lane + 32 * e; };
  const unsigned id = ONE_WARP ? blockIdx.x * 8 + warp : blockIdx.x;
  const unsigned R = p.G * p.n_q;  // rows of one key head
  const unsigned bk = id / R;
  const int gr = id - bk * R, b = bk / static_cast<unsigned>(p.HK), hk = bk - b * p.HK;
  const int rt = gr / ROWS, row = gr - rt * ROWS;
  const unsigned subs = p.HK * p.row_tiles, sub = hk * p.row_tiles + rt;
  OwnPart<E> own_part;  // TREE: of the row's ancestors
  if (TREE && id < total_rows && (ONE_WARP || warp == 0))
    own_part = tree_part<D>(p, b, hk, gr / p.n_q, gr % p.n_q, lane);
  int cached_len = 0;
  if (TREE && p.whole && id < total_rows) {
    cached_len = p.L_max;
    if (p.cache_lens != nullptr) cached_len = min(max(__ldg(p.cache_lens + b), 0), p.L_max);
  }
  grid_dependency_wait();  // the parts are complete
  if (id >= total_rows) return;
  unsigned w0 = 0, u0 = 0, share = 1;
  int n;
  if (TREE && p.whole) {
    n = cached_len > 0 && p.window != 0 ? 1 : 0;
  } else {
    const unsigned here = p.first[b], next = p.first[b + 1];
    share = share_of(p.first[p.B], p.warps);
    const unsigned tiles = (next - here) / subs;
    u0 = here + tiles * sub;
    w0 = u0 / share;
    n = tiles > 0 ? static_cast<int>((u0 + tiles - 1) / share - w0) + 1 : 0;
  }
  if (!TREE && n == 1) return;
  // part i: the first warp's run may have begun before the unit
  const float* part = p.part + (static_cast<long long>(w0) * 2 * ROWS + row) * (D + kPartTail);
  constexpr int NEXT = 2 * ROWS * (D + kPartTail);
  const int late = share * w0 < u0 && !(TREE && n == 1) ? ROWS * (D + kPartTail) : 0;
  if (TREE && n == 1) {
    const long long unit = static_cast<long long>(b) * subs + sub;
    part = p.done + (unit * ROWS + row) * (D + kPartTail);
  }
  auto part_at = [&](int i) { return part + static_cast<long long>(i) * NEXT + (i == 0 ? late : 0); };
  const int first = ONE_WARP ? 0 : warp;
  constexpr int STEP = ONE_WARP ? 1 : 8;
  float mm = -INFINITY, from = -INFINITY, ll = 0.f, a[E] = {};
  // {maximum, sum, what the values are relative to}
  auto tail_of = [](const float* at) { return *reinterpret_cast<const float4*>(at + D); };
  float mb = 0.f;
  if (TREE && ONE_WARP && n == 1) {  // one round of loads
    const float4 x = tail_of(part);
    mm = x.x;
    from = x.z;
    ll = x.y;
    mb = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (elem(e) < D) a[e] = part[elem(e)];
  } else {
    for (int i = lane; i < n; i += 32) {
      const float4 x = tail_of(part_at(i));
      mm = fmaxf(mm, x.x);
      from = fmaxf(from, x.z);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
      from = fmaxf(from, __shfl_xor_sync(0xffffffffu, from, x));
    }
    mb = mm == -INFINITY ? 0.f : mm;
    const float fb = from == -INFINITY ? 0.f : from;
    // 32 of this warp's parts at a time: their weights in the lanes, then their values
    for (int c = first; c < n; c += 32 * STEP) {
      const int own = c + lane * STEP;
      float f = 0.f;
      if (own < n) {
        const float4 x = tail_of(part_at(own));
        f = ex2(x.z - fb);
        ll += ex2(x.x - mb) * x.y;
      }
      const int here_n = min((n - c + STEP - 1) / STEP, 32);
      for (int y0 = 0; y0 < here_n; y0 += 4) {  // four parts' loads in flight
        float x[4][E];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          // (past the last part: the last one again, at weight 0)
          const float* at = part_at(c + min(y0 + y, here_n - 1) * STEP);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (TREE && E > 1) {
              *reinterpret_cast<Values*>(x[y]) = *reinterpret_cast<const Values*>(at + lane * E);
              break;
            }
            x[y][e] = elem(e) < D ? at[elem(e)] : 0.f;
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float fy = __shfl_sync(0xffffffffu, f, y0 + y);
#pragma unroll
          for (int e = 0; e < E; ++e) a[e] = fmaf(fy, x[y][e], a[e]);
        }
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, x);
    if (!ONE_WARP) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (elem(e) < D) joined[warp][elem(e)] = a[e];
      if (lane == 0) joined[warp][D] = ll;
      __syncthreads();
      if (warp != 0) return;
#pragma unroll
      for (int o = 1; o < 8; ++o) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (elem(e) < D) a[e] += joined[o][elem(e)];
        ll += joined[o][D];
      }
    }
  }
  const int head = hk * p.G + gr / p.n_q, qi = gr % p.n_q;
  __nv_bfloat16* out = p.o + b * p.so.b + head * p.so.h + qi * p.so.n;
  const float fac = value_factor(from, mb);
  if (TREE) {
    // the ancestors' part joins the cache's; a place that is no node sees neither.  (Sums
    // of NaN are not 0: they go on to O and LSE)
    const bool cached = ll != 0.f && own_part.node;
    float most = fmaxf(cached ? mm : -INFINITY, own_part.node ? own_part.m : -INFINITY);
    most = most == -INFINITY ? 0.f : most;
    const float w1 = cached ? ex2(mm - most) : 0.f, w2 = own_part.node ? ex2(own_part.m - most) : 0.f;
    const float sum = fmaf(w1, ll, w2 * own_part.l), inv = sum != 0.f ? 1.f / sum : 0.f;
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      y[e] = own_part.node ? w2 * own_part.a[e] : 0.f;
      if (cached) y[e] = fmaf(w1, a[e] * fac * fac, y[e]);
      if (E == 1 && lane < D) out[lane] = __float2bfloat16_rn(y[e] * inv);
    }
#pragma unroll
    for (int e = 0; e + 1 < E; e += 2)
      reinterpret_cast<__nv_bfloat162*>(out + lane * E)[e / 2] =
          __floats2bfloat162_rn(y[e] * inv, y[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[(static_cast<long long>(b) * p.HK * p.G + head) * p.n_q + qi] =
          sum != 0.f ? (most + __log2f(sum)) * kLn2 : -INFINITY;
    return;
  }
  const float inv = (ll > 0.f ? 1.f / ll : 0.f) * fac;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (elem(e) < D) out[elem(e)] = __float2bfloat16_rn(a[e] * fac * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[(static_cast<long long>(b) * p.HK * p.G + head) * p.n_q + qi] =
        ll > 0.f ? (mm + __log2f(ll)) * kLn2 : -INFINITY;
}

template <int FMT, int D, int NR, bool BIG, bool TREE>
cudaError_t launch_scored_decode_rows(const ScoredDecParams& p, const CUtensorMap* maps,
                                      const LaunchCtx& ctx) {
  const size_t smem = DW * DCfg<FMT, D, NR, BIG>::RING + 1024;
  auto* kernel = attn_decode_scored_kernel<FMT, D, NR, BIG, TREE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kernel<<<(p.warps + DW - 1) / DW, DW * 32, smem, ctx.stream>>>(maps[0], maps[1], p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (!TREE && p.whole) return cudaSuccess;
  const unsigned rows = static_cast<unsigned>(p.B) * p.HK * p.G * p.n_q;
  // parts of a unit, on average
  if (p.whole || p.warps / p.units < 8)
    return launch_dependent(attn_decode_scored_merge_kernel<D, NR * 8, true, TREE>, dim3((rows + 7) / 8),
                            dim3(256), 0, ctx.stream, p, rows);
  return launch_dependent(attn_decode_scored_merge_kernel<D, NR * 8, false, TREE>, dim3(rows), dim3(256),
                          0, ctx.stream, p, rows);
}

template <int FMT, int D, bool TREE>
cudaError_t launch_scored_decode_d(const ScoredDecParams& p, const CUtensorMap* maps, int row_tile,
                                   const LaunchCtx& ctx) {
  constexpr int rb = D * (FMT == kCacheBf16 ? 2 : 1);
  switch (row_tile) {
    case 8:
      if constexpr (scored_big_tiles(rb, 1, false)) {
        if (!p.whole) return launch_scored_decode_rows<FMT, D, 1, true, TREE>(p, maps, ctx);
      }
      return launch_scored_decode_rows<FMT, D, 1, false, TREE>(p, maps, ctx);
    case 16: return launch_scored_decode_rows<FMT, D, 2, false, TREE>(p, maps, ctx);
    default: return launch_scored_decode_rows<FMT, D, 4, false, TREE>(p, maps, ctx);
  }
}

template <int FMT, bool TREE = false>
cudaError_t launch_scored_decode_fmt(const ScoredDecodeProblem& pb, const CUtensorMap* maps,
                                     const ScoredDecodePlan& plan, float* workspace,
                                     const LaunchCtx& ctx, const TreeOwn* tree = nullptr) {
  // (a node to a lane, a lineage's nodes to the lanes)
  if (TREE && pb.n_q > 32) return cudaErrorInvalidValue;
  ScoredDecParams p;
  p.q = static_cast<const __nv_bfloat16*>(pb.q);
  p.k_scale = pb.k_scale;
  p.v_scale = pb.v_scale;
  p.o = static_cast<__nv_bfloat16*>(pb.o);
  p.lse = pb.lse;
  p.first = reinterpret_cast<unsigned*>(workspace);
  p.part = workspace + plan.part_off;
  p.cache_lens = pb.cache_lens;
  p.slopes = pb.slopes;
  p.sq = pb.sq;
  constexpr int es = FMT == kCacheBf16 ? 2 : 1;
  p.k = static_cast<const uint8_t*>(pb.k_cache);
  p.v = static_cast<const uint8_t*>(pb.v_cache);
  p.sk = RowStrides{pb.sk.b * es, pb.sk.h * es, pb.sk.n * es};
  p.sv = RowStrides{pb.sv.b * es, pb.sv.h * es, pb.sv.n * es};
  p.run_k = pb.sk.n == pb.d;
  p.run_v = pb.sv.n == pb.d;
  p.so = pb.so;
  p.HK = pb.HK;
  p.G = pb.H / pb.HK;
  p.n_q = pb.n_q;
  p.L_max = pb.L_max;
  p.T_log2 = 0;
  while ((1 << p.T_log2) < pb.block_tokens) ++p.T_log2;
  p.num_blocks = (pb.L_max + pb.block_tokens - 1) / pb.block_tokens;
  p.window = pb.window;
  p.row_tiles = plan.row_tiles;
  p.warps = plan.warps;
  p.B = pb.B;
  p.scale = pb.scale;
  p.softcap = pb.softcap;
  p.limit_ns = ctx.limit_ns;
  p.status = ctx.status;
  p.units = pb.B * pb.HK * plan.row_tiles;
  p.whole = plan.whole;
  if (TREE) {
    p.parents = tree->parents;
    p.k_tree = static_cast<const __nv_bfloat16*>(tree->k);
    p.v_tree = static_cast<const __nv_bfloat16*>(tree->v);
    p.skt = tree->sk;
    p.svt = tree->sv;
    p.done = workspace + plan.done_off;
  }
  switch (pb.d) {
    case 16: return launch_scored_decode_d<FMT, 16, TREE>(p, maps, plan.row_tile, ctx);
    case 32: return launch_scored_decode_d<FMT, 32, TREE>(p, maps, plan.row_tile, ctx);
    case 64: return launch_scored_decode_d<FMT, 64, TREE>(p, maps, plan.row_tile, ctx);
    case 128: return launch_scored_decode_d<FMT, 128, TREE>(p, maps, plan.row_tile, ctx);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace attn
