// attn_tree.cuh -- attention of a tree of drafted tokens over a key/value cache
// in bf16 or in 8 bits.  Included by one source file per cache format.
//
// Node i of sequence b stands at position p_i = L + depth_i behind the L tokens
// of its cache and sees them and its own ancestors (itself among them):
//   x_j = cap * tanh(scale * q_i . k_j / cap) - slope_h * (p_i - p_j)
//   O_i = sum_j softmax_j(x) v_j,   LSE_i = ln sum_j exp(x_j)
// over the cached keys j (p_j = j >= p_i - window) from the cache and the
// ancestors a (p_a = L + depth_a >= p_i - window) from the tree's own keys.
//
// The kernel for more than 32 query rows of a key head (16 where the heads are large
// and many; fewer: attn_decode_scored.cuh).  Bound by HBM (the visible cache, read once
// for each 256 query rows) while the rows are few, from about 200 rows on by a tile's chain
// of scores, softmax and product.  The G * n query rows of a key head (G query heads share
// it) are the rows of tcgen05 tiles of 128, so that a cache tile is multiplied
// for all of them while it is in shared memory.
//
// Measured: 4 sequences of 65 to 131 thousand tokens, 32 heads on 8, d = 128, bf16, 64
// nodes 331 us (floor 238: the cache at the rate of a plain copy, 6.8 TB/s; 1900 cycles
// for 64 keys of 256 rows, where the products take 1024 and the exponentials 512).
// 8 of 8 to 16 thousand, 32 heads on 4, d = 128, e4m3, 61 nodes, bias and a window of
// 2047 keys 54 us (9): 6 us to the first scores, 15 tiles of 3400 cycles, 3 us to write
// parts and 5 to join them.  Every instance stands at the 128 registers that 512 threads
// leave, and spills 16 to 128 bytes.
//
// Work split: the visible cache of all sequences and key heads, and behind each
// its tree's own keys, are one list of tiles of BN keys; a unit is a sequence,
// key head and block of 256 query rows.  Every CTA (one per SM) takes an equal
// run of the list, whatever the lengths are; units that several CTAs share go
// through the workspace to a second kernel.  Where units are short every CTA
// takes whole ones instead, and there is no second kernel.
//
// Inside a CTA two streams (a softmax warpgroup and an MMA warp each) overlap
// one's exponentials with the other's products.  With more than 128 rows a stream
// takes one tile of rows and both see every key tile; with at most 128 they take
// every second 64 keys with the same rows.  With at most 64 rows the tile of 128
// holds them twice, and each copy takes 32 of the 64 keys: its probabilities of
// the others are zero.  Exponentials cost a warp the same for one row as for 32,
// and so its four warps share them.  The parts of a row are joined at its end.
// Scores go to one of two buffers of a stream in tensor memory, so that those of
// the next 64 keys are there when a softmax is done; P takes its scores' place.
//
// Warps 0-3, 4-7: softmax of stream 0 and 1; 8-11: the query rows, the nodes'
// ancestors, and for 8-bit caches the widening of codes to bf16 (exact, both
// kinds); 12, 13: copies of keys and of values; 14, 15: MMA of stream 0 and 1.
// Every wait is bounded; on timeout the kernel records kDevTimeout, all roles
// drain and the CTA returns.
#pragma once

#include <cuda_bf16.h>

#include "attn_internal.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

using namespace ptx;

enum CacheFormat : int { kCacheBf16 = 0, kCacheE4M3 = 1, kCacheInt8 = 2 };

constexpr int BM = 128;        // query rows per tile (= tensor-memory lanes)
constexpr int kTreeCapped = 1, kTreeSlopes = 2;  // what a kernel does to the scores
constexpr int kBlockRows = 2 * BM;
constexpr int AUX_WARP = 8;
constexpr int KLOAD_WARP = 12;
constexpr int VLOAD_WARP = 13;
constexpr int MMA_WARP = 14;   // and 15
constexpr int NUM_THREADS = 512;
constexpr uint32_t TMEM_COLS = 512;
constexpr int SN = 64;  // keys of one score product
constexpr float kRescale = 8.0f;  // a running maximum is kept until a score exceeds it by 2^8
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMergeStride = 20;  // floats: 16 columns of a part's row, four apart in the banks

template <int FMT_, int D_>
struct TCfg {
  static constexpr int FMT = FMT_, D = D_;
  static constexpr bool Q8 = FMT_ != kCacheBf16;
  static constexpr int BN = D_ == 128 ? 64 : 128;  // keys per tile
  static constexpr uint32_t RB = (D_ < 64 ? D_ : 64) * 2;   // bytes of a row in one block
  static constexpr int NB = D_ > 64 ? D_ / 64 : 1;
  static constexpr uint32_t SWZ = RB == 128 ? 2u : (RB == 64 ? 4u : 6u);
  static constexpr int KPB = RB / 32;
  static constexpr int CPB = RB / 16;  // 16-byte chunks of a block row
  static constexpr int QSLOTS = D_ == 128 ? 1 : 2;
  static constexpr uint32_t Q_TILE = BM * D_ * 2, Q_BLOCK = BM * RB;
  static constexpr uint32_t KV_TILE = BN * D_ * 2, KV_BLOCK = BN * RB;
  static constexpr uint32_t RAW_TILE = BN * D_;  // codes
  // ring stages: of bf16 tiles, and of tiles of codes
  static constexpr int KSTAGES = D_ >= 64 ? (Q8 ? 2 : 4) : (Q8 ? 4 : 6);
  static constexpr int VSTAGES = D_ >= 64 && Q8 ? 3 : KSTAGES;
  static constexpr int RAWS = Q8 ? (D_ >= 64 ? 3 : 6) : 1;
  static constexpr uint32_t OW = D_ < 32 ? 32 : D_;
  static constexpr int NSUB = BN / SN;
  __host__ __device__ static constexpr uint32_t col_s(int s, int b) { return SN * (2 * s + b); }
  __host__ __device__ static constexpr uint32_t col_o(int s) { return 4 * SN + OW * s; }
  __host__ __device__ static constexpr uint32_t swz(uint32_t r) {
    return ((r * RB) >> 7) & (RB / 16 - 1);
  }
  static_assert(col_o(2) <= TMEM_COLS, "tensor memory");
};

// A run of a unit's tiles.
struct TreeItem {
  int more;        // 0: the CTA's work has ended
  int b, hk;
  int row0, rows;  // of the key head's query rows
  int split;       // copies of each row in a tile (1 or 2); 0: two tiles of rows
  int L, key0;     // cached tokens, and the first one that any node sees
  int base0, ctx;  // key of the unit's first cache tile, and how many there are
  int t0, n;       // this run of its tiles
  int whole, slot;
};

struct TreeParams {
  const __nv_bfloat16* q;
  const int* parents;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* o;
  float* lse;
  float* part;      // [CTA][2]: [D / 4][block rows] four values, then [block rows] {maximum, sum, -, -}
  unsigned* first;  // [B + 1], the list index of each sequence's first tile, and the total
  const int* cache_lens;
  const float* slopes;
  RowStrides sq, so;
  const uint8_t* k;  // 8-bit caches whose rows lie side by side are copied in runs
  const uint8_t* v;
  RowStrides sk, sv;
  bool run_k, run_v, whole;
  uint64_t limit_ns;
  int* status;
  int B, H, HK, G, n, L_max, T_log2, num_blocks, window;
  int rows, blocks, block_rows;  // query rows of a key head, their blocks, rows of a part
  int tree_tiles, rounds;
  float scale_log2, cap_log2, cap_in;
  unsigned div_n;  // floor(2^31 / n) + 1
  CapPoly cap;
  bool capped, wide;
};

template <class C>
struct __align__(1024) TreeSmem {
  uint8_t q[2 * C::QSLOTS][C::Q_TILE];
  uint8_t k[C::KSTAGES][C::KV_TILE];
  uint8_t v[C::VSTAGES][C::KV_TILE];
  uint8_t raw_k[C::RAWS][C::Q8 ? C::RAW_TILE : 16];
  uint8_t raw_v[C::RAWS][C::Q8 ? C::RAW_TILE : 16];
  float merge[3 * BM / 2][kMergeStride];  // the parts of rows but the first
  float2 stat[2 * BM];
  uint32_t line[2][kMostNodes][4];  // what a node sees of the tree
  int depth[2][kMostNodes];         // -1: no node
  int up[2][kMostNodes];            // scratch: parents, and 2^k-th ancestors
  TreeItem item[2];
  uint64_t item_full[2], item_empty[2], q_empty[2];
  uint64_t k_full[C::KSTAGES], k_empty[C::KSTAGES], v_full[C::VSTAGES], v_empty[C::VSTAGES];
  uint64_t raw_full[2][C::RAWS], raw_empty[2][C::RAWS];  // keys, values
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // stream, buffer
  uint64_t drain[2];
  uint64_t q_there;  // the first item's query rows
  uint64_t aux_sync, join_sync;  // barriers of the auxiliary and of the softmax warps
  unsigned warp_sum[NUM_THREADS / 32];
  // (in this order: with `abort` last the kernel for biased scores and e4m3 codes of d = 128
  // reloads 136 spilled bytes for 116, and a window of 2048 takes 55.8 us for 54.5)
  int abort;
  int start_b;
  unsigned start_off;
  uint32_t tmem_base;
  // tile s of an item's query rows; both: an item with two of them
  __device__ __forceinline__ uint8_t* q_tile(uint32_t items, bool both, int s) {
    if (C::QSLOTS == 2) return q[2 * (items & 1) + s];
    return q[both ? s : items & 1];
  }
};

// The tiles of a sequence's visible cache and of its tree.
struct TreeSeq {
  int L, key0, base0, ctx, tiles;
};
template <int BN>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  s.L = p.L_max;
  if (p.cache_lens != nullptr) s.L = min(max(__ldg(p.cache_lens + b), 0), p.L_max);
  // (a root, at position L, sees furthest back)
  s.key0 = p.window >= 0 ? max(s.L - p.window, 0) : 0;
  s.base0 = s.key0 & ~(BN - 1);
  s.ctx = s.key0 < s.L ? (s.L - s.base0 + BN - 1) / BN : 0;
  s.tiles = s.ctx + p.tree_tiles;
  return s;
}

// How many of a tile's parts of SN keys hold any (the unit's tile `t`).
template <class C>
__device__ __forceinline__ int parts_of(const TreeItem& it, int t, int n) {
  if (C::NSUB == 1) return 1;
  const int keys = t < it.ctx ? it.L - (it.base0 + t * C::BN) : n - (t - it.ctx) * C::BN;
  return keys > SN ? 2 : 1;
}

// The tile of an item's j-th turn: with a bias the cached ones from the newest on, whose
// scores are the largest, so that O is not rescaled for each (measured: 850 of 4900 cycles
// of a tile).
template <int MODE>
__device__ __forceinline__ int tile_of(const TreeItem& it, int j) {
  if (MODE & kTreeSlopes) {
    const int cached = min(it.t0 + it.n, it.ctx) - it.t0;
    if (j < cached) return it.t0 + cached - 1 - j;
  }
  return it.t0 + j;
}

constexpr int kMinTreeTiles = 2;  // of a CTA's run
__host__ __device__ __forceinline__ unsigned tree_share(unsigned total, int ctas) {
  const unsigned each = total / static_cast<unsigned>(ctas) + 1;
  return each < kMinTreeTiles ? kMinTreeTiles : each;
}

// A CTA's place in its work.
template <int BN>
struct TreeCursor {
  TreeSeq s;
  int b, sub, tile;
  unsigned left;  // tiles (split), units (whole)
  __device__ __forceinline__ void begin(const TreeParams& p, int start_b, unsigned off,
                                        unsigned count) {
    const int subs = p.HK * p.blocks;
    left = count;
    if (p.whole) {
      b = blockIdx.x / subs;
      sub = blockIdx.x - b * subs;
      tile = 0;
      if (left > 0) s = tree_seq<BN>(p, b);
      return;
    }
    b = start_b;
    if (left == 0) return;
    s = tree_seq<BN>(p, b);
    sub = off / static_cast<unsigned>(s.tiles);
    tile = off - static_cast<unsigned>(sub) * s.tiles;
  }
  // the next run, or false at the end
  __device__ __forceinline__ bool next(const TreeParams& p, TreeItem& it) {
    if (left == 0) {
      it.more = 0;
      return false;
    }
    const int rb = sub % p.blocks;
    it.more = 1;
    it.b = b;
    it.hk = sub / p.blocks;
    it.row0 = rb * kBlockRows;
    it.rows = min(p.rows - it.row0, kBlockRows);
    it.split = it.rows > BM ? 0 : (it.rows > BM / 2 ? 1 : 2);
    it.L = s.L;
    it.key0 = s.key0;
    it.base0 = s.base0;
    it.ctx = s.ctx;
    it.t0 = tile;
    const int subs = p.HK * p.blocks;
    if (p.whole) {
      it.n = s.tiles;
      it.whole = 1;
      it.slot = 0;
      --left;
      const int was = b;
      const int u = b * subs + sub + gridDim.x;
      if (left > 0) {
        b = u / subs;
        sub = u - b * subs;
        if (b != was) s = tree_seq<BN>(p, b);
      }
      return true;
    }
    it.n = min(static_cast<unsigned>(s.tiles - tile), left);
    it.whole = it.n == s.tiles;
    // a CTA's run begins in its first unit and ends in its last
    it.slot = 0;
    left -= it.n;
    tile = 0;
    if (left > 0 && ++sub == subs) {
      sub = 0;
      s = tree_seq<BN>(p, ++b);
    }
    return true;
  }
};

// mbar_wait with all but the first test in one place of the code: with many waits it
// would not fit the instruction cache otherwise.
__device__ __noinline__ bool mbar_wait_on(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                          const volatile int* abort) {
  return mbar_wait(bar, parity, limit_ns, abort);
}
__device__ __forceinline__ bool mbar_wait_small(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                                const volatile int* abort) {
  return mbar_try_wait(bar, parity) || mbar_wait_on(bar, parity, limit_ns, abort);
}

// 16 bytes to shared memory, asynchronously; zeros where there are none.
__device__ __forceinline__ void copy_chunk(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(there ? 16u : 0u)
               : "memory");
}
__device__ __forceinline__ void copy_chunks_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One arrival for a whole warp, behind what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint64_t tree_sdesc(uint32_t smem_addr, uint32_t lbo_bytes,
                                               uint32_t sbo_bytes, uint32_t swz) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  d |= static_cast<uint64_t>(swz) << 61;
  return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Two of a word's four codes (bytes 2 * HI and 2 * HI + 1) as a bf16 pair, exactly (but
// e4m3's codes of NaN, which become +-480: see no_number).
template <int FMT, int HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  uint32_t t, y;
  if (FMT == kCacheE4M3) {
    // sign, four exponent and three mantissa bits to their places in a bf16, whose
    // exponent is then 120 too small (the smallest codes are subnormal numbers in both);
    // bytes are spread with their sign in the byte above
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(t) : "r"(w), "n"(HI ? 0xb3a2 : 0x9180));
    y = (t << 4) & 0x87f087f0u;
    const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7b80));  // 2^120
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), up);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  // the low seven bits c as 128 + c, less 128, or 256 for a negative code
  t = __byte_perm(w, 0x43434343u, HI ? 0x4342 : 0x4140);
  const uint32_t a = t & 0xff7fff7fu, b = t & 0xff80ff80u;
  const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&x);
}

// NaN in the place of the +-480 among a lane's widened codes of half a tile (no code is
// that number: 448 is the largest).  Out of the way of what widens them.
template <class C>
__device__ __noinline__ void no_number(uint8_t* out, int half, int lane) {
  for (int e = lane; e < C::BN / 2 * C::CPB * C::NB; e += 32) {
    const int nb = e / (C::BN / 2 * C::CPB);
    uint4& w = *reinterpret_cast<uint4*>(out + nb * C::KV_BLOCK + half * (C::KV_BLOCK / 2) +
                                         (e - nb * (C::BN / 2 * C::CPB)) * 16);
    auto nan = [](uint32_t x) {
      return x | (__vcmpeq2(x & 0x7fff7fffu, 0x43f043f0u) & 0x7fff7fffu);
    };
    w = make_uint4(nan(w.x), nan(w.y), nan(w.z), nan(w.w));
  }
}

// Half (0 or 1) of a tile of codes to bf16 in the layout of a swizzled copy, by a warp;
// rows outside [lo, hi) become zeros.  Four chunks of codes are in flight at a time, in a loop:
// all of them side by side would crowd the instruction cache.
template <class C>
__device__ __forceinline__ void widen_tile(const uint8_t* raw, uint8_t* out, int half, int lane,
                                           int lo, int hi) {
  constexpr int CPR = C::D / 16;  // 16-code chunks of a row
  constexpr int N = C::BN / 2 * CPR / 32, M = N < 4 ? N : 4;
  constexpr int STEP = 32 / CPR;  // rows from one of a lane's chunks to the next
  const int c = lane % CPR;
  uint8_t* to = out + (2 * c / C::CPB) * C::KV_BLOCK;
  const int c0 = 2 * c % C::CPB;
  // (the two halves of a 256-byte row would meet in the same banks)
  const bool turn = C::D == 128 && (c & 4);
  int row = half * (C::BN / 2) + lane / CPR;
  // (bit 7 of a byte whose seven low bits are all set: e4m3's two codes of NaN)
  uint32_t nans = 0;
  auto seven = [](uint32_t x) { return (x & 0x7f7f7f7fu) + 0x01010101u; };
#pragma unroll 1
  for (int e = 0; e < N; e += M) {
    uint4 w[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int r = row + i * STEP, at = C::D == 128 ? c ^ (r & 7) : c;
      w[i] = *reinterpret_cast<const uint4*>(raw + r * C::D + at * 16);
    }
#pragma unroll
    for (int i = 0; i < M; ++i, row += STEP) {
      if (row < lo || row >= hi) w[i] = make_uint4(0u, 0u, 0u, 0u);  // (a code of 0 is the number 0)
      if (C::FMT == kCacheE4M3)
        nans |= seven(w[i].x) | seven(w[i].y) | seven(w[i].z) | seven(w[i].w);
      const uint4 a = make_uint4(widen2<C::FMT, 0>(w[i].x), widen2<C::FMT, 1>(w[i].x),
                                 widen2<C::FMT, 0>(w[i].y), widen2<C::FMT, 1>(w[i].y));
      const uint4 b = make_uint4(widen2<C::FMT, 0>(w[i].z), widen2<C::FMT, 1>(w[i].z),
                                 widen2<C::FMT, 0>(w[i].w), widen2<C::FMT, 1>(w[i].w));
      uint8_t* dst = to + row * C::RB;
      const int x = C::swz(row);
      *reinterpret_cast<uint4*>(dst + (((turn ? c0 + 1 : c0) ^ x) << 4)) = turn ? b : a;
      *reinterpret_cast<uint4*>(dst + (((turn ? c0 : c0 + 1) ^ x) << 4)) = turn ? a : b;
    }
  }
  if (C::FMT == kCacheE4M3 && __any_sync(0xffffffffu, nans & 0x80808080u)) {
    __syncwarp();  // (its chunks are other lanes')
    no_number<C>(out, half, lane);
  }
}

// Zeros in the rows of a value tile that nobody sees, whatever they hold, by a warp:
// of rows [r0, r1) those outside [lo, hi), or where `node` >= 0 (the tree's node of
// row 0) the places that are no node.
template <class C>
__device__ __forceinline__ void clear_rows(const TreeParams& p, TreeSmem<C>& sm, uint8_t* v, int r0,
                                           int r1, int lo, int hi, int node, int slot, int lane) {
  auto clear = [&](int from, int to) {
    for (int e = from * C::CPB + lane; e < to * C::CPB; e += 32)
#pragma unroll
      for (int nb = 0; nb < C::NB; ++nb)
        *reinterpret_cast<uint4*>(v + nb * C::KV_BLOCK + e * 16) = make_uint4(0u, 0u, 0u, 0u);
  };
  bool any = false;
  if (node < 0) {
    if (C::Q8) return;  // done where codes are widened
    any = lo > r0 || hi < r1;
    if (any) {
      clear(r0, min(lo, r1));
      clear(max(hi, r0), r1);
    }
  } else {
    for (int r = r0; r < r1; r += 32) {
      const int at = node + r + lane;
      unsigned gone = __ballot_sync(0xffffffffu, at < p.n && sm.depth[slot][at] < 0);
      any = any || gone != 0;
      for (; gone != 0; gone &= gone - 1) {
        const int row = r + __ffs(gone) - 1;
        clear(row, row + 1);
      }
    }
  }
  if (any) {
    fence_proxy_async_smem();
    __syncwarp();
  }
}

}  // namespace
}  // namespace attn

#include "attn_tree_many.cuh"

namespace attn {
namespace {

template <class C, int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ CUtensorMap tmkt,
                     const __grid_constant__ CUtensorMap tmvt, const TreeParams p) {
  using S = TreeSmem<C>;
  constexpr int D = C::D, BN = C::BN, KSTAGES = C::KSTAGES, VSTAGES = C::VSTAGES, RAWS = C::RAWS;
  constexpr bool Q8 = C::Q8;
  extern __shared__ uint8_t smem_raw[];
  // at a 1024-byte boundary (an offset, so that the compiler still knows the address
  // space: generic accesses and their 64-bit addresses cost more than the arithmetic)
  S& sm = *reinterpret_cast<S*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const volatile int* abort = &sm.abort;
  grid_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.item_full[i]), 4);  // one arrival per warp, here and below
      mbar_init(smem_u32(&sm.item_empty[i]), 8 + 2);  // softmax threads, MMA warps
      for (int e = 0; e < 2; ++e) {
        mbar_init(smem_u32(&sm.s_full[i][e]), 1);
        mbar_init(smem_u32(&sm.p_full[i][e]), 4);
        mbar_init(smem_u32(&sm.pv_done[i][e]), 1);
      }
      mbar_init(smem_u32(&sm.drain[i]), 1);
      for (int r = 0; r < RAWS; ++r) {
        mbar_init(smem_u32(&sm.raw_full[i][r]), 1);
        mbar_init(smem_u32(&sm.raw_empty[i][r]), 2);
      }
    }
    mbar_init(smem_u32(&sm.q_there), 4);
    mbar_init(smem_u32(&sm.aux_sync), 4);
    mbar_init(smem_u32(&sm.join_sync), 8);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sm.q_empty[i]), 2);
    for (int i = 0; i < KSTAGES; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), Q8 ? 2 : 1);
      mbar_init(smem_u32(&sm.k_empty[i]), 2);  // both streams
    }
    for (int i = 0; i < VSTAGES; ++i) {
      mbar_init(smem_u32(&sm.v_full[i]), Q8 ? 2 : 1);
      mbar_init(smem_u32(&sm.v_empty[i]), 2);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == KLOAD_WARP && lane == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmkt);
  }
  if (warp == VLOAD_WARP && lane == 0) {
    prefetch_tmap(&tmv);
    prefetch_tmap(&tmvt);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
    tmem_relinquish();
  }

  // ---- where this CTA's work begins, and how much it is
  unsigned count = 0;
  const int subs = p.HK * p.blocks;
  if (p.whole) {
    const int units = p.B * subs;  // (the caller keeps it below 2^24)
    if (static_cast<int>(blockIdx.x) < units) count = (units - 1 - blockIdx.x) / gridDim.x + 1;
  } else {
    const int per = (p.B + NUM_THREADS - 1) / NUM_THREADS;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    unsigned sum = 0;
    for (int b = b0; b < b1; ++b) sum += tree_seq<BN>(p, b).tiles;
    sum *= subs;
    unsigned run = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, run, m);
      if (lane >= m) run += x;
    }
    if (lane == 31) sm.warp_sum[warp] = run;
    __syncthreads();
    unsigned total = 0;
#pragma unroll
    for (int i = 0; i < NUM_THREADS / 32; ++i) {
      const unsigned x = sm.warp_sum[i];
      if (i < warp) run += x;
      total += x;
    }
    const unsigned share = tree_share(total, gridDim.x);
    // (share * CTAs stays below 2^32: total < 2^31)
    const unsigned begin = share * blockIdx.x;
    count = begin < total ? min(share, total - begin) : 0;
    unsigned at = run - sum;
    if (blockIdx.x == 0) {  // for the second kernel
      unsigned a = at;
      for (int b = b0; b < b1; ++b) {
        p.first[b] = a;
        a += tree_seq<BN>(p, b).tiles * subs;
      }
      if (threadIdx.x == 0) p.first[p.B] = total;
    }
    if (count > 0 && begin >= at && begin < run) {
      for (int b = b0; b < b1; ++b) {
        const unsigned t = tree_seq<BN>(p, b).tiles * subs;
        if (begin - at < t) {
          sm.start_b = b;
          sm.start_off = begin - at;
          break;
        }
        at += t;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int start_b = sm.start_b;
  const unsigned start_off = sm.start_off;

  bool ok = true;
  auto fail = [&]() {
    atomicCAS(p.status, kDevOk, kDevTimeout);
    *reinterpret_cast<volatile int*>(&sm.abort) = 1;
  };

  if (warp >= MMA_WARP) {
    const int s = warp - MMA_WARP;
    ok = mma_many<C, MODE>(p, sm, tmem, s, lane);
    if (!ok && lane == 0) fail();
    // every product issued by this warp completes before tensor memory is freed
    if (elect_one()) tc_commit(smem_u32(&sm.drain[s]));
    __syncwarp();
    const int never = 0;
    mbar_wait_small(smem_u32(&sm.drain[s]), 0, p.limit_ns, &never);
  } else if (warp >= KLOAD_WARP) {
    // ---------------------------------------------------------------- copies
    if (lane == 0 && count > 0) {
      const bool is_v = warp == VLOAD_WARP;
      const uint32_t ST = Q8 ? RAWS : (is_v ? VSTAGES : KSTAGES);
      uint64_t* full = Q8 ? sm.raw_full[is_v] : (is_v ? sm.v_full : sm.k_full);
      uint64_t* empty = Q8 ? sm.raw_empty[is_v] : (is_v ? sm.v_empty : sm.k_empty);
      uint8_t* ring = Q8 ? (is_v ? &sm.raw_v[0][0] : &sm.raw_k[0][0])
                         : (is_v ? &sm.v[0][0] : &sm.k[0][0]);
      const CUtensorMap* map = is_v ? &tmv : &tmk;
      const CUtensorMap* tree_map = is_v ? &tmvt : &tmkt;
      const bool runs = is_v ? p.run_v : p.run_k;
      TreeCursor<BN> cur;
      cur.begin(p, start_b, start_off, count);
      TreeItem it;
      uint32_t cnt = 0;
      // the first query rows come before the first tiles: behind those of all CTAs at
      // once they would take 6 us and more
      ok = mbar_wait_small(smem_u32(&sm.q_there), 0, p.limit_ns, abort);
      while (ok && cur.next(p, it)) {
        const int stop = Q8 ? min(it.t0 + it.n, it.ctx) : it.t0 + it.n;
        for (int j = 0; j < stop - it.t0; ++j) {
          const int t = tile_of<MODE>(it, j);
          const uint32_t at = cnt % ST;
          ok = mbar_wait_small(smem_u32(&empty[at]), ((cnt / ST) & 1) ^ 1, p.limit_ns, abort);
          if (!ok) break;
          const uint32_t bar = smem_u32(&full[at]);
          if constexpr (Q8) {
            const uint32_t to = smem_u32(ring + at * C::RAW_TILE);
            const int key = it.base0 + t * BN;
            if (D < 128 && runs) {
              const uint32_t bytes = min(BN, p.L_max - key) * D;
              const RowStrides& st = is_v ? p.sv : p.sk;
              mbar_arrive_expect_tx(bar, bytes);
              bulk_copy_in(to, (is_v ? p.v : p.k) + it.b * st.b + it.hk * st.h +
                                   static_cast<long long>(key) * D, bytes, bar);
            } else {
              mbar_arrive_expect_tx(bar, C::RAW_TILE);
              tma_load_4d(to, map, bar, 0, key, it.hk, it.b);
            }
          } else {
            const uint32_t to = smem_u32(ring + at * C::KV_TILE);
            const bool tree = t >= it.ctx;
            mbar_arrive_expect_tx(bar, C::KV_TILE);
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb)
              tma_load_4d(to + nb * C::KV_BLOCK, tree ? tree_map : map, bar, 64 * nb,
                          tree ? (t - it.ctx) * BN : it.base0 + t * BN, it.hk, it.b);
          }
          ++cnt;
        }
      }
      if (!ok) {
        fail();
        const int never = 0;  // the copies under way land before shared memory goes away
        for (uint32_t i = 0; i < ST; ++i) {
          const uint32_t uses = cnt / ST + (i < cnt % ST ? 1u : 0u);
          if (uses > 0) mbar_wait_small(smem_u32(&full[i]), (uses - 1) & 1, p.limit_ns, &never);
        }
      }
    }
  } else if (warp >= AUX_WARP) {
    // ---------------------------------------------------------------- rows, trees, codes
    const int aw = warp - AUX_WARP, tid = aw * 32 + lane;
    TreeCursor<BN> cur;
    cur.begin(p, start_b, start_off, count);
    int has[2] = {-1, -1};  // whose tree a slot's tables hold
    uint32_t cnt = 0, raws = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait_small(smem_u32(bar), parity, p.limit_ns, abort));
      return ok;
    };
    uint32_t syncs = 0;
    auto sync = [&]() {
      warp_arrive(smem_u32(&sm.aux_sync));
      return wait(&sm.aux_sync, syncs++ & 1);
    };
    uint32_t copied = 0, phase = 0;  // ring slots that this warp copied to last, and when
    bool was_wide = false;         // the item before
    const bool small = p.n <= 32;  // every warp has all the nodes
    for (uint32_t items = 0;; ++items) {
      const int slot = items & 1;
      const int me = small ? lane : tid;  // this thread's node
      int up = -2;
      if (cur.left > 0 && has[slot] != cur.b && me < p.n)
        up = __ldg(p.parents + static_cast<long long>(cur.b) * p.n + me);
      if (!wait(&sm.item_empty[slot], ((items >> 1) & 1) ^ 1)) break;
      TreeItem it;
      const bool more = cur.next(p, it);
      if (more && !it.whole) it.slot = items == 0 ? 0 : 1;
      if (tid == 0) sm.item[slot] = it;
      if (!more) {
        warp_arrive(smem_u32(&sm.item_full[slot]));
        break;
      }
      // the query rows, each `split` times
      if (!wait(&sm.q_empty[slot], ((items >> 1) & 1) ^ 1)) break;
      // (d = 128: two tiles in all, which one item takes with both streams' rows)
      const bool wide = it.split == 0;
      if (C::QSLOTS == 1 && items > 0 && (wide || was_wide) &&
          !wait(&sm.q_empty[slot ^ 1], ((items - 1) >> 1) & 1))
        break;
      was_wide = wide;
      // (a row's head by a product with (2^31 + e) / n, 1 <= e <= n: row e < 2^31 for all 2^24
      // rows and 128 nodes, so that the quotient's whole part is exact.  All copies are
      // under way at once: in batches of 8 loads the first tile's scores came 3 us later)
      constexpr int CPR = D / 8;  // 16-byte chunks of a row
      const int tiles = it.split == 0 ? 2 : 1;
      const int lanes = it.split == 0 ? BM : BM / it.split;
      const __nv_bfloat16* q = p.q + it.b * p.sq.b + static_cast<long long>(it.hk) * p.G * p.sq.h;
      for (int s = 0; s < tiles; ++s) {
        const uint32_t to = smem_u32(sm.q_tile(items, wide, s));
#pragma unroll 4
        for (int e = tid; e < BM * CPR; e += 128) {
          const int at = e / CPR, c = e % CPR;
          const int r = s * BM + (at & (lanes - 1));
          const bool there = r < it.rows;
          const int row = it.row0 + (there ? r : 0), g = __umulhi(2u * row, p.div_n);
          copy_chunk(to + (c / C::CPB) * C::Q_BLOCK + at * C::RB + (((c % C::CPB) ^ C::swz(at)) << 4),
                     q + g * p.sq.h + (row - g * p.n) * p.sq.n + c * 8, there);
        }
      }
      copy_chunks_done();
      fence_proxy_async_smem();
      if (items == 0) warp_arrive(smem_u32(&sm.q_there));
      if (has[slot] != it.b) {
        // ancestors by pointer doubling: after round k a node knows 2^k of them
        has[slot] = it.b;
        if (up < -1 || up >= me) up = -2;
        const int parent = up;
        if (small) {
          uint32_t line = me < p.n ? 1u << lane : 0u;
          for (int r = 0; r < p.rounds; ++r) {
            const int from = max(up, 0);
            const uint32_t above = __shfl_sync(0xffffffffu, line, from);
            const int next = __shfl_sync(0xffffffffu, up, from);
            if (up >= 0) {
              line |= above;
              up = next;
            }
          }
          const bool node = up == -1;
          const int depth = node ? __popc(line) - 1 : -1;
          if (p.window >= 0 && p.window < 31) {
            // only the nearest ancestors
            uint32_t near = 0u;
            for (int k = 0, at = lane; k <= p.window; ++k) {
              if (at >= 0) near |= 1u << at;
              const int next = __shfl_sync(0xffffffffu, parent, max(at, 0));
              at = at >= 0 ? next : at;
            }
            line &= near;
          }
          if (!node) line = 0u;
          if (aw == 0) {
            sm.depth[slot][lane] = depth;
            sm.line[slot][lane][0] = line;
          } else {
            sm.depth[slot][tid] = -1;
            sm.line[slot][lane][aw] = 0u;
          }
        } else {
          uint32_t line[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) line[w] = aw == w ? 1u << lane : 0u;
          for (int r = 0; r < p.rounds && ok; ++r) {
            sm.up[0][tid] = up;
#pragma unroll
            for (int w = 0; w < 4; ++w) sm.line[slot][tid][w] = line[w];
            if (!sync()) break;
            if (up >= 0) {
#pragma unroll
              for (int w = 0; w < 4; ++w) line[w] |= sm.line[slot][up][w];
              up = sm.up[0][up];
            }
            sync();
          }
          const bool node = up == -1;
          const int depth =
              __popc(line[0]) + __popc(line[1]) + __popc(line[2]) + __popc(line[3]) - 1;
          sm.up[1][tid] = parent;
          if (!sync()) break;
          if (node && p.window >= 0 && p.window < depth) {
            // only the nearest ancestors
#pragma unroll
            for (int w = 0; w < 4; ++w) line[w] = 0u;
            int a = tid;
            for (int k = 0; k <= p.window; ++k) {
#pragma unroll
              for (int w = 0; w < 4; ++w)
                if (a >> 5 == w) line[w] |= 1u << (a & 31);
              a = sm.up[1][a];
            }
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) sm.line[slot][tid][w] = node ? line[w] : 0u;
          sm.depth[slot][tid] = node ? depth : -1;
        }
      }
      warp_arrive(smem_u32(&sm.item_full[slot]));
      if constexpr (Q8) {
        // two warps take the keys, two the values, half a tile each
        const int kv = aw & 1, half = aw >> 1;
        const uint32_t stages = kv ? VSTAGES : KSTAGES;
        uint64_t* full = kv ? sm.v_full : sm.k_full;
        uint64_t* empty = kv ? sm.v_empty : sm.k_empty;
        for (int j = 0; j < it.n; ++j, ++cnt) {
          const int t = tile_of<MODE>(it, j);
          const uint32_t at = cnt % stages, ph = (cnt / stages) & 1;
          uint8_t* to = kv ? sm.v[at] : sm.k[at];
          if (!wait(&empty[at], ph ^ 1)) break;
          if (t < it.ctx) {
            const uint32_t from = raws % RAWS;
            if (!wait(&sm.raw_full[kv][from], (raws / RAWS) & 1)) break;
            ++raws;
            const int key = it.base0 + t * BN;
            widen_tile<C>(kv ? sm.raw_v[from] : sm.raw_k[from], to, half, lane,
                          kv ? it.key0 - key : 0, kv ? it.L - key : BN);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_u32(&sm.raw_empty[kv][from]));
              mbar_arrive(smem_u32(&full[at]));
            }
            copied &= ~(1u << at);
          } else {
            // the tree's own keys are bf16 already
            if (lane == 0) {
              const uint32_t bar = smem_u32(&full[at]);
              if (half == 0) {
                mbar_arrive_expect_tx(bar, C::KV_TILE);
#pragma unroll
                for (int nb = 0; nb < C::NB; ++nb)
                  tma_load_4d(smem_u32(to) + nb * C::KV_BLOCK, kv ? &tmvt : &tmkt, bar, 64 * nb,
                              (t - it.ctx) * BN, it.hk, it.b);
              } else {
                mbar_arrive(bar);
              }
            }
            if (half == 0) {
              copied |= 1u << at;
              phase = (phase & ~(1u << at)) | (ph << at);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) {
      fail();
      const int never = 0;  // the copies under way land before shared memory goes away
      for (uint32_t i = 0; copied >> i != 0; ++i)
        if ((copied >> i) & 1u)
          mbar_wait_small(smem_u32(aw & 1 ? &sm.v_full[i] : &sm.k_full[i]), (phase >> i) & 1u,
                          p.limit_ns, &never);
    }
  } else {
    ok = softmax_many<C, MODE>(p, sm, tmem, warp >> 2, warp & 3, lane);
    if (!ok) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the parts of the units that several CTAs shared: 32 query rows of a key head, a
// row per lane, its values shared out to kJoinWarps warps, two to a CTA so that few rows
// use many SMs (2 sequences of 8 key heads of 128 rows, d = 128: 20.5 us in all, with 8
// warps 22.4, 32 19.1; 8 of 8 key heads of 256 rows 41.3, 40.5, 41.9).
template <int D>
constexpr int kJoinWarps = D < 32 ? 4 : D < 128 ? 8 : 16;
template <int D>
__global__ void __launch_bounds__(64) attn_tree_join_kernel(const TreeParams p, int ctas) {
  constexpr int K = D / 4 / kJoinWarps<D>;  // fours of a row's values that a thread joins
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * 2 + (threadIdx.x >> 5), all = w / kJoinWarps<D>;
  const int warp = w - all * kJoinWarps<D>;
  const unsigned groups = (p.rows + 31u) / 32u, bk = all / groups;
  const int b = bk / static_cast<unsigned>(p.HK), hk = bk - b * p.HK;
  const int row0 = (all - bk * groups) * 32, row = row0 + lane;
  if (row >= p.rows) return;
  const int subs = p.HK * p.blocks;
  const unsigned f0 = p.first[b], f1 = p.first[b + 1];
  const unsigned tiles = (f1 - f0) / subs;
  const unsigned begin = f0 + (hk * p.blocks + row0 / kBlockRows) * tiles;
  const unsigned share = tree_share(p.first[p.B], ctas);
  const unsigned c0 = begin / share, c1 = (begin + tiles - 1) / share;
  if (c0 == c1) return;
  const int column = 4 * p.block_rows;
  const float* at = p.part + 4 * (row % kBlockRows);
  auto part = [&](unsigned c) {
    const int slot = share * c >= begin ? 0 : 1;
    return at + (static_cast<size_t>(c) * 2 + slot) * p.block_rows * (D + kPartTail);
  };
  // four parts' loads in flight
  float most = -INFINITY, y[K][4] = {}, sum = 0.f;
  for (unsigned c = c0; c <= c1; c += 4) {
    float2 tail[4];
    float4 v[4][K];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* x = part(min(c + i, c1));
      tail[i] = *reinterpret_cast<const float2*>(x + (D / 4) * column);
#pragma unroll
      for (int k = 0; k < K; ++k)
        v[i][k] = *reinterpret_cast<const float4*>(x + (warp * K + k) * column);
    }
    const float was = most;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i > c1) tail[i].y = 0.f;
      if (tail[i].y != 0.f) most = fmaxf(most, tail[i].x);
    }
    const float old = was == -INFINITY ? 0.f : ex2(was - most);
    sum *= old;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[k][e] *= old;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = tail[i].y != 0.f ? ex2(tail[i].x - most) : 0.f;
      sum = fmaf(w, tail[i].y, sum);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        y[k][0] = fmaf(w, v[i][k].x, y[k][0]);
        y[k][1] = fmaf(w, v[i][k].y, y[k][1]);
        y[k][2] = fmaf(w, v[i][k].z, y[k][2]);
        y[k][3] = fmaf(w, v[i][k].w, y[k][3]);
      }
    }
  }
  const int g = row / p.n, node = row - g * p.n;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;  // (a sum of NaN goes on)
  __nv_bfloat16* out = p.o + b * p.so.b + (hk * p.G + g) * p.so.h + node * p.so.n + warp * K * 4;
#pragma unroll
  for (int k = 0; k < K; ++k)
    *reinterpret_cast<uint2*>(out + 4 * k) =
        make_uint2(pack_bf16x2(y[k][0] * inv, y[k][1] * inv), pack_bf16x2(y[k][2] * inv, y[k][3] * inv));
  if (warp == 0 && p.lse != nullptr)
    p.lse[(static_cast<size_t>(b) * p.H + hk * p.G + g) * p.n + node] =
        sum != 0.f ? (most + __log2f(sum)) * kLn2 : -INFINITY;
}

template <class C, int MODE>
cudaError_t launch_tree_d(const TreeParams& p, const CUtensorMap* maps, const TreePlan& plan,
                          const LaunchCtx& ctx) {
  static_assert(sizeof(TreeSmem<C>) + 1024 <= 232448, "dynamic shared memory per CTA");
  const size_t smem = sizeof(TreeSmem<C>) + 1024;
  cudaError_t err = cudaFuncSetAttribute(attn_tree_kernel<C, MODE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  attn_tree_kernel<C, MODE>
      <<<plan.ctas, NUM_THREADS, smem, ctx.stream>>>(maps[0], maps[1], maps[2], maps[3], p);
  if ((err = cudaGetLastError()) != cudaSuccess || plan.whole) return err;
  return launch_dependent(attn_tree_join_kernel<C::D>,
                          dim3(static_cast<unsigned>(p.B) * p.HK * ((p.rows + 31) / 32) *
                               (kJoinWarps<C::D> / 2)),
                          dim3(64), 0,
                          ctx.stream, p, plan.ctas);
}

template <int FMT, int D>
cudaError_t launch_tree_mode(const TreeParams& p, const CUtensorMap* maps, const TreePlan& plan,
                             const LaunchCtx& ctx) {
  using C = TCfg<FMT, D>;
  // (a kernel for each: code that is not there costs no instruction fetches)
  if (p.capped)
    return p.slopes ? launch_tree_d<C, kTreeCapped | kTreeSlopes>(p, maps, plan, ctx)
                    : launch_tree_d<C, kTreeCapped>(p, maps, plan, ctx);
  return p.slopes ? launch_tree_d<C, kTreeSlopes>(p, maps, plan, ctx)
                  : launch_tree_d<C, 0>(p, maps, plan, ctx);
}

template <int FMT>
cudaError_t launch_tree_fmt(const TreeDecodeProblem& pb, const CUtensorMap* maps,
                            const TreePlan& plan, void* workspace, const LaunchCtx& ctx) {
  TreeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(pb.q);
  p.parents = pb.parents;
  p.k_scale = pb.k_scale;
  p.v_scale = pb.v_scale;
  p.o = static_cast<__nv_bfloat16*>(pb.o);
  p.lse = pb.lse;
  p.first = static_cast<unsigned*>(workspace);
  p.part = static_cast<float*>(workspace) + plan.part_off;
  p.cache_lens = pb.cache_lens;
  p.slopes = pb.slopes;
  p.sq = pb.sq;
  p.so = pb.so;
  p.k = static_cast<const uint8_t*>(pb.k_cache);
  p.v = static_cast<const uint8_t*>(pb.v_cache);
  p.sk = pb.sk;
  p.sv = pb.sv;
  p.run_k = pb.sk.n == pb.d;
  p.run_v = pb.sv.n == pb.d;
  p.whole = plan.whole;
  p.limit_ns = ctx.limit_ns;
  p.status = ctx.status;
  p.B = pb.B;
  p.H = pb.H;
  p.HK = pb.HK;
  p.G = pb.H / pb.HK;
  p.n = pb.n;
  p.div_n = (1u << 31) / static_cast<unsigned>(pb.n) + 1u;
  p.L_max = pb.L_max;
  while ((1 << p.T_log2) < pb.block_tokens) ++p.T_log2;
  p.num_blocks = (pb.L_max + pb.block_tokens - 1) / pb.block_tokens;
  p.window = pb.window;
  p.rows = p.G * pb.n;
  p.blocks = plan.blocks;
  p.block_rows = plan.block_rows;
  p.tree_tiles = plan.tree_tiles;
  while ((1 << p.rounds) < pb.n) ++p.rounds;
  p.scale_log2 = pb.scale * kLog2e;
  p.capped = pb.softcap > 0.f;
  p.cap_log2 = pb.softcap * kLog2e;
  p.cap_in = p.capped ? 2.f * p.scale_log2 / pb.softcap : 0.f;
  p.cap = cap_poly(pb.scale, pb.softcap);
  p.wide = pb.softcap > kWideCap;
  switch (pb.d) {
    case 16: return launch_tree_mode<FMT, 16>(p, maps, plan, ctx);
    case 32: return launch_tree_mode<FMT, 32>(p, maps, plan, ctx);
    case 64: return launch_tree_mode<FMT, 64>(p, maps, plan, ctx);
    case 128: return launch_tree_mode<FMT, 128>(p, maps, plan, ctx);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace attn
