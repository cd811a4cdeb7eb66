// attn_bwd.cu -- backward of the fused attention forward for sm_103a: the
// gradients dQ, dK, dV of a loss whose gradient with respect to the output
// O = softmax(scale * Q K^T + M) V is dO.
//
// The forward is eq. (1) of "Attention Is All You Need" (section 3.2.1) with
// the masks of section 3.2.3; its gradient is what training the model of
// section 5 back-propagates through every attention layer.  Per (b, h), with
// P the row softmax recomputed from Q, K and the forward's log-sum-exp:
//
//   dV = P^T dO,   dP = dO V^T,   D_i = sum_c dO_ic O_ic,
//   dS = P * (dP - D_i)  (elementwise),   dQ = scale dS K,   dK = scale dS^T Q.
//
// Three launches (changed scores add attn_bwd_few_kernel beside the first and, for
// shared key heads worked on in parts, attn_bwd_dkv_kernel after the last):
//   1. attn_bwd_pre_kernel: per query row, the two per-query constants the
//      elementwise steps need, b_i = -LSE_i / scale and -D_i, each split into
//      three bf16 parts (hi + mid + lo) and written as [128 x 16] bf16 tiles;
//      and the row of the fp32 dQ accumulator set to zero.
//   2. attn_bwd_tc_kernel: one persistent CTA per SM walks work items = one
//      128-key tile of one (b, h); for each 128-query tile that the mask lets
//      see those keys it runs the tensor-core products of that tile pair and
//      accumulates dK and dV in tensor memory; dQ of the tile pair is added
//      into the fp32 accumulator in global memory with TMA reduces.
//   3. attn_bwd_dq_kernel: dQ = scale * accumulator, rounded to bf16.
//
// The per-query constants ride on the tensor cores: one extra K=16 step
// against an all-ones operand adds b_i to every score of column i and -D_i to
// every dP of column i,
//   S'^T = K Q^T + 1 b^T,   dP'^T = V dO^T + 1 (-D)^T,
// so that the elementwise work per element is P = 2^(scale*log2(e) * S') and
// dS = P * dP' (the three bf16 parts keep b and D to about 2^-24 relative).
//
// Kernel 2 (448 threads):
//   warps 0-7   elementwise: warp w owns tensor-memory lanes 32*(w%4).. (=
//               keys) and query columns 64*(w/4)..+63; it turns S'^T into P^T
//               (bf16, written to tensor memory) and dP'^T into dS^T (bf16,
//               written to shared memory in the 128-byte swizzled layout, two
//               buffers so that tile t+1's dS^T is written while dK(t) and
//               dQ(t) still read tile t's);
//   warps 8-11  epilogue, two groups of two warps (query or key rows 0-63 and
//               64-127), each with its own 8 KB staging buffer: dQ of each tile
//               pair (tensor memory -> swizzled fp32 staging -> TMA reduce-add
//               into the fp32 accumulator in global memory), dK and dV of each
//               item (-> bf16 -> TMA store);
//   warp  12    TMA producer: K per item (2 slots), V per item (1 slot: its
//               only reader, dP, is done with it a tile pair before the next
//               item needs it); Q and its constant tile (3 stages) and dO (2
//               stages) per query tile;
//   warp  13    tensor-memory owner and MMA issuer.
// Tensor memory (512 columns, w = max(d, 32) for head size d in {16, 32,
// 64}): S'^T [0,128)  dP'^T [128,256)  dV, dK, dQ w columns each from 256,
// then P^T (64 columns of bf16 pairs); at d = 64 dV [256,320) dK [320,384)
// dQ [384,448) P^T [448,512).  Keys are the 128 lanes of all but dQ, whose
// lanes are queries.  Q, K, V, dO tiles are [128 x d] in the swizzle of their
// 2d-byte rows; dS^T is [128 x 128] at every d.
// Products per tile pair t (all 128-row M; * = from tensor memory):
//   S'^T = K Q^T (+1 b^T)    dP'^T = V dO^T (+1 (-D)^T)    dV += P^T* dO
//   dK += dS^T Q             dQ = dS K
// issued in the order S'(t+1), dV(t), dP'(t+1), dK(t), dQ(t), so that the
// elementwise warps start on tile t+1 while the tensor pipe finishes the
// gradient products of tile t.  Every wait is bounded; on timeout the kernel
// records kDevTimeout, all roles drain and the CTA returns.
//
// Changed scores (MODE kScored, with kCap, kBias and kWide; attn_bwd_scored): dS
// gets the cap's derivative as a factor, items are a key tile of a key head with
// the query tiles of its whole group (or of a part of it), so that dK and dV of
// shared heads are sums in tensor memory.  Bound by the chain of a tile pair, as
// the plain kernel; with caps by registers.  8 x 16 x 4096, d = 64, causal, on one
// GPU: plain 919 us, by plan 912, with bias 930, with cap 1081, with both 1190.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_internal.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int BM = 128;  // queries per query tile
constexpr int BN = 128;  // keys per key tile (= tensor-memory lanes)
constexpr uint32_t DS_BLOCK = 128 * 64 * 2;  // a [128 x 64] bf16 block of dS^T: 16 KB
// Q (and its constant tile) ring: Q is last read by dK, late in a tile pair,
// so three stages let the next tile's loads start two tile pairs ahead.  dO
// is last read by dV, early in a tile pair: two stages suffice.
constexpr int QSTAGES = 3;
constexpr int OSTAGES = 2;
constexpr int NUM_THREADS = 448;
constexpr int EPI_WARP0 = 8;
constexpr int LOAD_WARP = 12;
constexpr int MMA_WARP = 13;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_S = 0, COL_DP = 128;
// The [128 x 16] bf16 constant tile of a query tile (K-major, no swizzle:
// 8-row x 16-byte core matrices, the second 8 columns 128 B after the first,
// 8-row groups 256 B apart).  Row i holds b_i in columns 0-2 (hi, mid, lo)
// and -D_i in columns 3-5; columns 6-15 are zero.
constexpr uint32_t CONST_TILE_BYTES = 128 * 16 * 2;
constexpr float LOG2E = 1.4426950408889634f;

static_assert(BM == BN, "the causal tile range assumes square tiles");

constexpr uint32_t STAGE_BYTES = 64 * 128;  // an epilogue staging buffer: 64 rows x 128 bytes
constexpr int EPI_BAR0 = 1;  // named barriers 1, 2: the two epilogue groups

// Shapes per head size d (16, 32, 64; d_k = d_v): Q, K, V and dO tiles of
// [128 x d] bf16 with rows of 2d bytes in the widest swizzle they fit; dV,
// dK and dQ accumulators of max(d, 32) tensor-memory columns (32-column
// loads never touch a neighbour); dQ added into the fp32 accumulator in boxes
// of min(d, 32) columns.  (d = 128 would need 704 tensor-memory columns.)
template <int D_>
struct BCfg {
  static constexpr uint32_t RB = D_ * 2;
  static constexpr uint32_t SWZ = RB == 128 ? 2u : (RB == 64 ? 4u : 6u);
  static constexpr uint32_t TILE = 128 * D_ * 2;
  static constexpr uint32_t OW = D_ < 32 ? 32 : D_;
  static constexpr uint32_t COL_DV = 256, COL_DK = 256 + OW, COL_DQ = 256 + 2 * OW,
                            COL_PT = 256 + 3 * OW;
  static constexpr uint32_t QRB = (D_ < 32 ? D_ : 32) * 4;  // row bytes of a dQ box
  static_assert(COL_PT + 64 <= 512, "tensor memory");
};

template <int D_, int MODE>
struct __align__(1024) Smem {
  using C = BCfg<D_>;
  uint8_t k[2][C::TILE];
  uint8_t v[C::TILE];
  uint8_t q[QSTAGES][C::TILE];
  uint8_t dout[OSTAGES][C::TILE];
  // dS^T as [128 keys x 128 queries] bf16, two buffers (tile pairs t even /
  // odd), each two 64-query column blocks of [128 x 64] in the 128-byte
  // swizzled layout.
  uint8_t dst[2][2][DS_BLOCK];
  // epilogue staging, one 64-row buffer per epilogue group: a fp32 box of
  // dQ, or dV / dK in bf16, swizzled as the tensor map it is copied with
  uint8_t stage[2][STAGE_BYTES];
  uint8_t cst[QSTAGES][CONST_TILE_BYTES];  // the constant tile of each Q stage
  // with a cap: the constants of each Q stage's queries in log2 units (LSE and,
  // with a distance bias, the query's share of it)
  float lse[MODE & kCap ? QSTAGES : 1][MODE & kCap ? BM : 4];
  // Two 8 x 8 bf16 core matrices that select columns of the constant tile:
  // [0] rows (1,1,1,0,0,0,0,0) picks b, [1] rows (0,0,0,1,1,1,0,0) picks -D.
  uint8_t sel[2][512];
  uint64_t k_full[2], k_empty[2], v_full, v_empty;
  uint64_t q_full[QSTAGES], q_empty[QSTAGES];
  uint64_t o_full[OSTAGES], o_empty[OSTAGES];
  uint64_t s_full, s_free, dp_full, dp_free;
  uint64_t p_full, p_free, ds_full, ds_free[2];
  uint64_t dq_full, dq_free, dkv_full, dkv_free;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

struct Params {
  const uint8_t* cst;  // constant tiles [BH][num_qt][CONST_TILE_BYTES]
  const int* key_lens;
  int H, n_q, n_k, BH;
  int mask;
  int win_left, win_right;  // restricted attention: query i sees keys i - left .. i + right
  int num_qt, num_kt, num_items;
  float scale_log2;  // scale * log2(e)
  float scale;
  // changed scores (kScored): BH counts key heads then
  int group;              // query heads per key head
  int parts;              // items that share a key tile, group / parts query heads each
  float cap_log2;         // softcap * log2(e); 0: no cap
  float cap_in;           // 2 log2(e) scale / softcap: tanh's exponent per unit of q.k
  const float* slopes;    // distance bias per query head, or null
  CapPoly cap;            // kWide
  const float* lse_log2;  // with a cap: [B * H][num_qt * 128]
  bool masked;
  MaskPlan plan;
  const int* next;  // the items dealt out by load: after each the next one of its CTA,
                    // then every CTA's first; or null
  uint64_t limit_ns;
  int* status;
};

// A work item: key tile kt of head bh and the query tiles qt0 .. qt0+n-1
// that see at least one of its keys.
// (kScored: bh is a key head's, and the n tiles are nq query tiles of each of
// its query heads in turn.)
struct Item {
  int bh, kt, qt0, n, key_limit;
  int nq;
  int part;  // kScored: which of the parts of the query heads
};

// An item of changed scores: the plan's, for every key head and part in turn.
__device__ __forceinline__ Item bwd_item_planned(const Params& p, int t) {
  Item it;
  const int heads = p.H / p.group;
  const int whole = p.parts == 1 ? t : t / p.parts;
  it.part = t - whole * p.parts;
  const int e = whole / heads, hk = whole - e * heads;
  it.key_limit = p.n_k;
  if (p.masked) {
    const int4 k = __ldg(reinterpret_cast<const int4*>(p.plan.key_items + e));
    it.bh = k.x * heads + hk;
    it.kt = k.y;
    it.qt0 = k.z;
    it.nq = k.w;
  } else {
    it.kt = e % p.num_kt;
    it.bh = e / p.num_kt * heads + hk;
    it.qt0 = 0;
    it.nq = p.num_qt;
  }
  it.n = it.nq * (p.group / p.parts);
  return it;
}

template <int MODE>
__device__ __forceinline__ Item bwd_item(const Params& p, int t) {
  if constexpr ((MODE & kScored) != 0) return bwd_item_planned(p, t);
  Item it;
  if (p.mask == kMaskCausal) {
    // key tiles with the most query tiles first (longest-processing-time order)
    it.kt = t / p.BH;
    it.bh = t % p.BH;
  } else {
    // the key tiles of one head back to back, so Q and dO stay hot in L2
    it.bh = t / p.num_kt;
    it.kt = t % p.num_kt;
  }
  int limit = p.n_k;
  if (p.mask == kMaskKeyPadding) {
    const int L = __ldg(p.key_lens + it.bh / p.H);
    limit = min(max(L, 0), p.n_k);
  }
  it.key_limit = limit;
  it.qt0 = 0;
  it.n = 0;
  if (it.kt * BN < limit) {
    if (p.mask == kMaskCausal) {
      // query i sees key j iff j <= i: tiles before kt see none of these keys
      it.qt0 = it.kt;
      it.n = max(p.num_qt - it.kt, 0);
    } else if (p.mask == kMaskBand) {
      // key j is seen by the queries j - right .. j + left
      const int j_lo = it.kt * BN, j_hi = min(j_lo + BN - 1, limit - 1);
      const int q_lo = max(j_lo - p.win_right, 0), q_hi = min(j_hi + p.win_left, p.n_q - 1);
      if (q_lo <= q_hi) {
        it.qt0 = q_lo / BM;
        it.n = q_hi / BM - it.qt0 + 1;
      }
    } else {
      it.n = p.num_qt;
    }
  }
  it.nq = it.n;
  it.part = 0;
  return it;
}

// The items of this CTA, one after the other: every gridDim.x-th, or, of planned
// ones, those that attn_bwd_few_kernel dealt it, else back and forth.
template <int MODE>
struct Walk {
  int x, step;  // step 0: the dealt ones
  __device__ __forceinline__ explicit Walk(const Params& p)
      : x(blockIdx.x), step((MODE & kScored) ? first_step() : static_cast<int>(gridDim.x)) {
    if constexpr ((MODE & kScored) != 0) {
      if (p.next != nullptr) {
        const int first = p.next[p.num_items + blockIdx.x];
        if (first >= 0) {
          x = first;
          step = 0;
        }
      }
    }
  }
  __device__ __forceinline__ void next(const Params& p) {
    if constexpr ((MODE & kScored) != 0) {
      if (step == 0) {
        x = max(p.next[x], x + 1);  // (always larger; so that every walk ends)
        return;
      }
    }
    x += step;
    if (MODE & kScored) step = 2 * gridDim.x - step;
  }
};

// Moves on to the next item with work, this one included; false: there is none.
template <int MODE>
__device__ __forceinline__ bool find_item(const Params& p, int num_items, Walk<MODE>& at,
                                          Item& out) {
  for (; at.x < num_items; at.next(p)) {
    out = bwd_item<MODE>(p, at.x);
    if (out.n > 0) return true;
  }
  return false;
}

template <class SmemT>
__device__ __forceinline__ void record_timeout(const Params& p, SmemT& sm) {
  atomicCAS(p.status, kDevOk, kDevTimeout);
  *reinterpret_cast<volatile int*>(&sm.abort) = 1;
}

// 3-D tiled reduce-add shared -> global (fp32 add, element type from the
// tensor map), tracked by the issuing thread's bulk groups.  Parts of the box
// outside the tensor are not touched.
__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* map, uint32_t src, int x,
                                                  int y, int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
      " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Contiguous global -> shared copy (size a multiple of 16, both addresses
// 16-byte aligned), completion counted on `bar` in bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Shared-memory matrix descriptor without swizzle (K-major: 8-row x 16-byte
// core matrices; LBO = byte step between the two 8-column halves of K = 16,
// SBO = byte step between 8-row groups).  Same fields as the 128-byte swizzle
// descriptor with layout bits 61-63 = 0.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t smem_addr, uint32_t lbo_bytes,
                                                uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  return d;
}

// One row of RBYTES (128, 64 or 32) into a tile swizzled at that width:
// 16-byte chunk g of row r lands at chunk position g ^ ((r * RBYTES / 128) %
// (RBYTES / 16)), the layout a TMA copy with that swizzle reads and writes.
template <uint32_t RBYTES>
__device__ __forceinline__ void st_row_swz(uint32_t tile, int r, const uint32_t (&w)[32]) {
  const uint32_t base = tile + r * RBYTES;
  const uint32_t x = ((static_cast<uint32_t>(r) * RBYTES) >> 7) & (RBYTES / 16 - 1);
#pragma unroll
  for (uint32_t g = 0; g < RBYTES / 16; ++g)
    st_shared_v4(base + ((g ^ x) << 4), w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
}

// Shared-memory matrix descriptor (same fields as sdesc_sw128) with the
// layout code `swz` at bits 61-63.
__device__ __forceinline__ uint64_t sdesc_swz(uint32_t smem_addr, uint32_t lbo_bytes,
                                              uint32_t sbo_bytes, uint32_t swz) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  d |= static_cast<uint64_t>(swz) << 61;
  return d;
}

// P of one thread's key and 64 queries with changed scores: emit(i, a, b, c, d)
// gets it in bf16 pairs of columns 2i .. 2i + 7 for dV, pf what multiplies dP -
// D: P times the cap's derivative.
//
// The distance bias -slope |i - j| is slope (j - i0) - slope (i - i0), i0 the
// query tile's first query: the second term is in the per-query constants
// already (attn_bwd_pre_kernel), the first, `bias` in log2 units, is this
// thread's.  Keys after their query get 2 slope (j - i) less; SLOW: some visible
// key is, or some query of the warp's tile does not see some key (two loops
// instead of branches in one, which would keep its instructions from being
// interleaved).  LINE: every key of the warp's is visible and at or after all of its
// queries, so that the correction is linear too (f * ahead is in `bias` then).
// `ahead` = j - the first of the 64 queries, f = -2 slope in log2
// units; columns outside [lim, hi) are forbidden for this key.
//
// With a cap, from r = 1 / (1 + 2^(2 y log2(e))): tanh(y) = 1 - 2 r, 1 -
// tanh^2(y) = 4 r (1 - r).  LSE comes off after the tanh, from shared memory (it
// is a constant of the column, not of the thread).  POLY: small arguments under a
// wide cap, by the polynomials of CapPoly.  (Under the usual caps these are slower
// here, 487 against 403 us on packed documents of 4 x 4096 tokens: registers bound
// this loop, not the special-function unit.)
template <int MODE, bool SLOW, bool POLY, bool LINE, class Emit>
__device__ __forceinline__ void scored_probabilities(const Params& p, const uint32_t (&s0)[32],
                                                     const uint32_t (&s1)[32], float (&pf)[64],
                                                     int lim, int hi, float bias, float ahead,
                                                     float f, const float* lse, Emit emit) {
  constexpr bool CAP = (MODE & kCap) != 0, BIAS = (MODE & kBias) != 0;
  const float c = p.scale_log2;
  const float top = p.cap_log2 + bias, m2 = -2.f * p.cap_log2;
  // The visible columns as bits, which are tested several at a time, where
  // comparisons take two instructions a score (packed documents with caps 308 ->
  // 272 us); not with caps and bias, where registers are short (big causal 1164
  // us by comparisons, 1200 by bits, without LINE).
  constexpr bool BITS = !(CAP && BIAS);
  const uint32_t see[2] = {below(hi) & ~below(lim), below(hi - 32) & ~below(lim - 32)};
#pragma unroll
  for (int c0 = 0; c0 < 64; c0 += 8) {
    const uint32_t* src = c0 < 32 ? s0 + c0 : s1 + (c0 - 32);
    float x[8];
    if constexpr (CAP && POLY) {
      const float4 l0 = *reinterpret_cast<const float4*>(lse + c0),
                   l1 = *reinterpret_cast<const float4*>(lse + c0 + 4);
      const float ln[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = __uint_as_float(src[e]), z = a * a;
        x[e] = fmaf(a, fmaf(z, fmaf(z, p.cap.poly[2], p.cap.poly[1]), p.cap.poly[0]), bias - ln[e]);
        pf[c0 + e] = fmaf(z, fmaf(z, p.cap.slope[2], p.cap.slope[1]), p.cap.slope[0]);
      }
    } else if constexpr (CAP) {
      float r[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        fma2(r[e], r[e + 1], __uint_as_float(src[e]), __uint_as_float(src[e + 1]), p.cap_in,
             p.cap_in, 0.f, 0.f);
        add2(r[e], r[e + 1], ex2(r[e]), ex2(r[e + 1]), 1.f, 1.f);
        r[e] = rcp(r[e]);
        r[e + 1] = rcp(r[e + 1]);
      }
      const float4 l0 = *reinterpret_cast<const float4*>(lse + c0),
                   l1 = *reinterpret_cast<const float4*>(lse + c0 + 4);
      fma2(x[0], x[1], r[0], r[1], m2, m2, top - l0.x, top - l0.y);
      fma2(x[2], x[3], r[2], r[3], m2, m2, top - l0.z, top - l0.w);
      fma2(x[4], x[5], r[4], r[5], m2, m2, top - l1.x, top - l1.y);
      fma2(x[6], x[7], r[6], r[7], m2, m2, top - l1.z, top - l1.w);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float q0, q1;
        fma2(q0, q1, r[e], r[e + 1], -4.f, -4.f, 4.f, 4.f);
        fma2(pf[c0 + e], pf[c0 + e + 1], r[e], r[e + 1], q0, q1, 0.f, 0.f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        fma2(x[e], x[e + 1], __uint_as_float(src[e]), __uint_as_float(src[e + 1]), c, c, bias,
             bias);
    }
    if constexpr (LINE) {
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        fma2(x[e], x[e + 1], static_cast<float>(c0 + e), static_cast<float>(c0 + e + 1), -f, -f,
             x[e], x[e + 1]);
    }
    if constexpr (SLOW) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (BIAS) x[e] = fmaf(f, fmaxf(ahead - static_cast<float>(c0 + e), 0.f), x[e]);
        if (BITS ? !(see[c0 / 32] & (1u << (c0 + e) % 32)) : c0 + e < lim || c0 + e >= hi)
          x[e] = -INFINITY;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = ex2(x[e]);
    emit(c0 / 2, pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
         pack_bf16x2(x[6], x[7]));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      if constexpr (CAP)
        fma2(pf[c0 + e], pf[c0 + e + 1], pf[c0 + e], pf[c0 + e + 1], x[e], x[e + 1], 0.f, 0.f);
      else
        pf[c0 + e] = x[e], pf[c0 + e + 1] = x[e + 1];
    }
  }
}

template <int MODE, int D_>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmq,
                       const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv,
                       const __grid_constant__ CUtensorMap tmdo,
                       const __grid_constant__ CUtensorMap tmdk,
                       const __grid_constant__ CUtensorMap tmdv,
                       const __grid_constant__ CUtensorMap tmdq,
                       const __grid_constant__ CUtensorMap tmpart, const Params p) {
  using C = BCfg<D_>;
  using S = Smem<D_, MODE>;
  constexpr int D = D_;
  constexpr bool BAND = MODE == kBand, SCORED = (MODE & kScored) != 0, CAP = (MODE & kCap) != 0;
  extern __shared__ uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &sm.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 1);
      mbar_init(smem_u32(&sm.k_empty[i]), 1);
    }
    mbar_init(smem_u32(&sm.v_full), 1);
    mbar_init(smem_u32(&sm.v_empty), 1);
    for (int i = 0; i < QSTAGES; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 1);
      mbar_init(smem_u32(&sm.q_empty[i]), 1);
    }
    for (int i = 0; i < OSTAGES; ++i) {
      mbar_init(smem_u32(&sm.o_full[i]), 1);
      mbar_init(smem_u32(&sm.o_empty[i]), 1);
    }
    mbar_init(smem_u32(&sm.s_full), 1);
    mbar_init(smem_u32(&sm.s_free), 256);
    mbar_init(smem_u32(&sm.dp_full), 1);
    mbar_init(smem_u32(&sm.dp_free), 256);
    mbar_init(smem_u32(&sm.p_full), 256);
    mbar_init(smem_u32(&sm.p_free), 1);
    mbar_init(smem_u32(&sm.ds_full), 256);
    mbar_init(smem_u32(&sm.ds_free[0]), 1);
    mbar_init(smem_u32(&sm.ds_free[1]), 1);
    mbar_init(smem_u32(&sm.dq_full), 1);
    mbar_init(smem_u32(&sm.dq_free), 128);
    mbar_init(smem_u32(&sm.dkv_full), 1);
    mbar_init(smem_u32(&sm.dkv_free), 128);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == LOAD_WARP && lane == 0) {
    prefetch_tmap(&tmq);
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    prefetch_tmap(&tmdo);
    prefetch_tmap(&tmdk);
    prefetch_tmap(&tmdv);
    prefetch_tmap(&tmdq);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0) {
    // the selector operands of the constant products (bf16 1.0 = 0x3F80):
    // word w of a 16-byte row holds columns 2w, 2w+1
    const uint32_t wi = lane & 3;
    const uint32_t sb = wi == 0 ? 0x3F803F80u : (wi == 1 ? 0x00003F80u : 0u);
    const uint32_t sd = wi == 1 ? 0x3F800000u : (wi == 2 ? 0x3F803F80u : 0u);
    reinterpret_cast<uint32_t*>(sm.sel[0])[lane] = sb;
    reinterpret_cast<uint32_t*>(sm.sel[1])[lane] = sd;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // Launched as a dependent of the preprocess kernel (which writes the
  // constant tiles and zeroes the dQ accumulator): everything above overlaps
  // its tail, nothing below runs before it has completed.
  grid_dependency_wait();

  int num_items = p.num_items;
  if constexpr (SCORED) {
    if (p.masked) {
      const int4 h = __ldg(p.plan.header);
      if (h.x != p.n_q || h.y != p.n_k || h.z * (p.H / p.group) != p.BH) {
        // a plan of other sizes: report it and do nothing
        num_items = 0;
        if (threadIdx.x == 0) atomicCAS(p.status, kDevOk, kDevWrongPlan);
      }
    }
  }
  // heads of K, V, dK and dV, and the query head of an item's g-th group member
  const int kv_heads = SCORED ? p.H / p.group : p.H;
  auto q_head = [&](const Item& item, int g) {
    return SCORED ? item.bh % kv_heads * p.group + item.part * (p.group / p.parts) + g
                  : item.bh % p.H;
  };
  // the item's next tile pair: the next query tile, then the next query head
  auto step = [](const Item& item, int& qt, int& g) {
    ++qt;
    if (SCORED && qt == item.qt0 + item.nq) {
      qt = item.qt0;
      ++g;
    }
  };

  if (warp == LOAD_WARP) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t it = 0, nv = 0, nq = 0, no = 0;  // K, V, Q and dO loads issued
      bool ok = true;
      Item item;
      for (Walk<MODE> at(p); ok && find_item(p, num_items, at, item); at.next(p)) {
        const uint32_t slot = it & 1;
        ok = mbar_wait(smem_u32(&sm.k_empty[slot]), ((it >> 1) & 1) ^ 1, p.limit_ns, abort);
        if (!ok) break;
        mbar_arrive_expect_tx(smem_u32(&sm.k_full[slot]), C::TILE);
        const int b = item.bh / kv_heads, hk = item.bh % kv_heads;
        tma_load_4d(smem_u32(sm.k[slot]), &tmk, smem_u32(&sm.k_full[slot]), 0, item.kt * BN, hk, b);
        ++it;
        int qt = item.qt0, g = 0;
        for (int i = 0; i < item.n && ok; ++i, step(item, qt, g)) {
          const int hq = q_head(item, g);
          const uint32_t st = nq % QSTAGES;
          ok = mbar_wait(smem_u32(&sm.q_empty[st]), ((nq / QSTAGES) & 1) ^ 1, p.limit_ns, abort);
          if (!ok) break;
          const uint32_t qb = smem_u32(&sm.q_full[st]);
          mbar_arrive_expect_tx(qb, C::TILE + CONST_TILE_BYTES + (CAP ? BM * 4 : 0));
          tma_load_4d(smem_u32(sm.q[st]), &tmq, qb, 0, qt * BM, hq, b);
          const size_t tile =
              (SCORED ? static_cast<size_t>(b) * p.H + hq : static_cast<size_t>(item.bh)) * p.num_qt + qt;
          bulk_load(smem_u32(sm.cst[st]), p.cst + tile * CONST_TILE_BYTES, CONST_TILE_BYTES, qb);
          if constexpr (CAP)
            bulk_load(smem_u32(sm.lse[st]), p.lse_log2 + tile * BM, BM * 4, qb);
          ++nq;
          if (i == 0) {
            // V of this item, once the previous item's last dP has read the slot
            ok = mbar_wait(smem_u32(&sm.v_empty), (nv & 1) ^ 1, p.limit_ns, abort);
            if (!ok) break;
            mbar_arrive_expect_tx(smem_u32(&sm.v_full), C::TILE);
            tma_load_4d(smem_u32(sm.v), &tmv, smem_u32(&sm.v_full), 0, item.kt * BN, hk, b);
            ++nv;
          }
          const uint32_t os = no % OSTAGES;
          ok = mbar_wait(smem_u32(&sm.o_empty[os]), ((no / OSTAGES) & 1) ^ 1, p.limit_ns, abort);
          if (!ok) break;
          const uint32_t ob = smem_u32(&sm.o_full[os]);
          mbar_arrive_expect_tx(ob, C::TILE);
          tma_load_4d(smem_u32(sm.dout[os]), &tmdo, ob, 0, qt * BM, hq, b);
          ++no;
        }
      }
      if (!ok) {
        record_timeout(p, sm);
        // the copies already issued land before the shared memory goes away:
        // wait (bounded, ignoring the abort flag) for the last phase armed on
        // every full barrier
        const int never = 0;
        auto drain = [&](uint64_t* full, uint32_t stages, uint32_t issued) {
          for (uint32_t i = 0; i < stages; ++i) {
            const uint32_t uses = issued / stages + (i < issued % stages ? 1u : 0u);
            if (uses > 0) mbar_wait(smem_u32(&full[i]), (uses - 1) & 1, p.limit_ns, &never);
          }
        };
        drain(sm.k_full, 2, it);
        drain(&sm.v_full, 1, nv);
        drain(sm.q_full, QSTAGES, nq);
        drain(sm.o_full, OSTAGES, no);
      }
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the control flow; one elected lane issues.
    constexpr uint32_t IDESC_SQ = idesc_bf16_f32(BN, BM, false, false);  // S^T, dP^T
    constexpr uint32_t IDESC_KV = idesc_bf16_f32(BN, D, false, true);    // dV (A in tensor memory), dK
    constexpr uint32_t IDESC_DQ = idesc_bf16_f32(BM, D, true, true);     // dQ
    constexpr uint32_t T16 = C::TILE >> 4;     // a [128 x d] tile in desc units
    constexpr uint32_t DS16 = DS_BLOCK >> 4;   // a dS^T column block in desc units
    constexpr uint32_t RB16 = C::RB;           // 16 rows of RB bytes in desc units
    // K-major operands (rows x d bf16, 8-row groups 8*RB bytes apart; a K
    // step of 16 elements is +32 B = +2 inside the swizzle row).
    const uint64_t kK = sdesc_swz(smem_u32(sm.k[0]), 16, 8 * C::RB, C::SWZ);
    const uint64_t kV = sdesc_swz(smem_u32(sm.v), 16, 8 * C::RB, C::SWZ);
    const uint64_t kQ = sdesc_swz(smem_u32(sm.q[0]), 16, 8 * C::RB, C::SWZ);
    const uint64_t kDO = sdesc_swz(smem_u32(sm.dout[0]), 16, 8 * C::RB, C::SWZ);
    // dS^T as the K-major A operand of dK (M = keys, K = queries): a K step
    // inside a 64-query column block is +2, the second block is +16 KB.
    const uint64_t kDST = sdesc_sw128(smem_u32(sm.dst[0][0]), 16, 1024);
    // MN-major B operands (K = the rows of the tile, N = the d columns): a K
    // step of 16 rows is 16*RB bytes (+RB16); 8-row groups 8*RB bytes apart
    // (SBO); N is one swizzle atom, LBO unused (set to 1024).
    const uint64_t nQ = sdesc_swz(smem_u32(sm.q[0]), 1024, 8 * C::RB, C::SWZ);
    const uint64_t nDO = sdesc_swz(smem_u32(sm.dout[0]), 1024, 8 * C::RB, C::SWZ);
    const uint64_t nK = sdesc_swz(smem_u32(sm.k[0]), 1024, 8 * C::RB, C::SWZ);
    // dS as the MN-major A operand of dQ (M = queries across the two column
    // blocks, 16 KB apart = LBO; K = keys, 16 rows per step = +128).
    const uint64_t nDS = sdesc_sw128(smem_u32(sm.dst[0][0]), DS_BLOCK, 1024);
    // The constant products: A = a selector (every core matrix of the 128 x 16
    // operand aliases the same 128 bytes: LBO = SBO = 0), B = the Q stage's
    // [128 queries x 16] constant tile.
    const uint64_t kSelB = sdesc_plain(smem_u32(sm.sel[0]), 0, 0);
    const uint64_t kSelD = sdesc_plain(smem_u32(sm.sel[1]), 0, 0);
    const uint64_t kCst = sdesc_plain(smem_u32(sm.cst[0]), 128, 256);
    constexpr uint32_t C16 = CONST_TILE_BYTES >> 4;

    const bool leader = elect_one();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.limit_ns, abort));
      return ok;
    };
    auto issue_s = [&](uint32_t slot, uint32_t st) {  // S^T = K Q^T
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + COL_S, kK + slot * T16 + 2 * kk, kQ + st * T16 + 2 * kk, IDESC_SQ,
                 kk > 0 ? 1u : 0u);
        mma_ss(tmem + COL_S, kSelB, kCst + st * C16, IDESC_SQ, 1u);  // + b_i
        tc_commit(smem_u32(&sm.s_full));
      }
      __syncwarp();
    };
    // dP^T = V dO^T; the last tile pair of an item releases the V slot
    auto issue_dp = [&](uint32_t qs, uint32_t os, bool last_of_item) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + COL_DP, kV + 2 * kk, kDO + os * T16 + 2 * kk, IDESC_SQ, kk > 0 ? 1u : 0u);
        mma_ss(tmem + COL_DP, kSelD, kCst + qs * C16, IDESC_SQ, 1u);  // - D_i
        tc_commit(smem_u32(&sm.dp_full));
        if (last_of_item) tc_commit(smem_u32(&sm.v_empty));
      }
      __syncwarp();
    };

    uint32_t it = 0, t = 0;
    Item cur;
    Walk<MODE> at(p);
    const bool any = find_item(p, num_items, at, cur);
    int ci = 0;  // index of tile t inside its item
    if (any && wait(&sm.k_full[0], 0) && wait(&sm.q_full[0], 0) && wait(&sm.v_full, 0) &&
        wait(&sm.o_full[0], 0)) {
      tc_fence_after();
      issue_s(0, 0);
      issue_dp(0, 0, cur.n == 1);
      while (ok) {
        const uint32_t slot = it & 1, st = t % QSTAGES, os = t % OSTAGES;
        // the next tile pair (possibly of the next item)
        Item nx = cur;
        int ni = ci + 1;
        uint32_t nit = it;
        bool has_next = true;
        if (ni >= cur.n) {
          at.next(p);
          has_next = find_item(p, num_items, at, nx);
          ni = 0;
          nit = it + 1;
        }
        const uint32_t nslot = nit & 1, nst = (t + 1) % QSTAGES, nos = (t + 1) % OSTAGES;
        // its score product goes first, as soon as S'^T of this one is in the
        // elementwise warps' registers
        if (has_next) {
          if (ni == 0 && !wait(&sm.k_full[nslot], (nit >> 1) & 1)) break;
          if (!wait(&sm.q_full[nst], ((t + 1) / QSTAGES) & 1)) break;
          if (!wait(&sm.s_free, t & 1)) break;
          tc_fence_after();
          issue_s(nslot, nst);
        }
        // dV += P^T dO (an item's first product overwrites dV, so the
        // epilogue must have read the previous item's dK and dV)
        if (ci == 0 && !wait(&sm.dkv_free, (it & 1) ^ 1)) break;
        if (!wait(&sm.p_full, t & 1)) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BM / 16; ++kk)
            mma_ts(tmem + C::COL_DV, tmem + C::COL_PT + 8 * kk, nDO + os * T16 + RB16 * kk, IDESC_KV,
                   (ci > 0 || kk > 0) ? 1u : 0u);
          tc_commit(smem_u32(&sm.p_free));
          tc_commit(smem_u32(&sm.o_empty[os]));  // the last product that reads this dO
        }
        __syncwarp();
        if (!wait(&sm.ds_full, t & 1)) break;
        tc_fence_after();
        if (has_next) {
          if (!wait(&sm.dp_free, t & 1)) break;
          if (ni == 0 && !wait(&sm.v_full, nit & 1)) break;
          if (!wait(&sm.o_full[nos], ((t + 1) / OSTAGES) & 1)) break;
          tc_fence_after();
          issue_dp(nst, nos, ni == nx.n - 1);
        }
        // dK += dS^T Q (the last product that reads this stage's Q)
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BM / 16; ++kk)
            mma_ss(tmem + C::COL_DK, kDST + (2 * (t & 1) + (kk >> 2)) * DS16 + 2 * (kk & 3),
                   nQ + st * T16 + RB16 * kk, IDESC_KV, (ci > 0 || kk > 0) ? 1u : 0u);
          tc_commit(smem_u32(&sm.q_empty[st]));
        }
        __syncwarp();
        // dQ = dS K (the epilogue must have read the previous tile's dQ)
        if (!wait(&sm.dq_free, (t & 1) ^ 1)) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ss(tmem + C::COL_DQ, nDS + 2 * (t & 1) * DS16 + 128 * kk,
                   nK + slot * T16 + RB16 * kk, IDESC_DQ, kk > 0 ? 1u : 0u);
          tc_commit(smem_u32(&sm.dq_full));
          tc_commit(smem_u32(&sm.ds_free[t & 1]));
          if (ci == cur.n - 1) {
            tc_commit(smem_u32(&sm.k_empty[slot]));
            tc_commit(smem_u32(&sm.dkv_full));
          }
        }
        __syncwarp();
        if (!has_next) break;
        cur = nx;
        ci = ni;
        it = nit;
        ++t;
      }
    }
    if (!ok && leader) record_timeout(p, sm);
    // every MMA issued completes before tensor memory is freed
    if (leader) tc_commit(smem_u32(&sm.drain));
    __syncwarp();
    const int never = 0;
    mbar_wait(smem_u32(&sm.drain), 0, p.limit_ns, &never);
  } else if (warp >= EPI_WARP0) {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // tensor-memory lane = row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // group g = rows 64g .. 64g+63 (warps 8+2g, 9+2g), staging buffer g
    const int g = quarter >> 1;
    const int rg = r & 63;  // row inside the group's 64-row box
    const bool leader = (quarter & 1) == 0 && lane == 0;
    const uint32_t stage = smem_u32(sm.stage[g]);
    const uint32_t bar_id = EPI_BAR0 + g;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.limit_ns, abort));
      return ok;
    };
    // The group's buffer is free once its previous bulk copy has read it;
    // after the rows are written, the copy may start.
    auto stage_acquire = [&]() {
      if (leader) bulk_wait_read_all();
      named_bar_sync(bar_id, 64);
    };
    auto stage_release = [&]() {
      fence_proxy_async_smem();
      named_bar_sync(bar_id, 64);
    };
    // kScored with parts: this part's dV (which = 0) or dK as fp32 rows into the
    // workspace, [dV, dK][part][B * key heads]; attn_bwd_dkv_kernel adds the parts up
    auto store_part = [&](const Item& item, int which, uint32_t (&lo)[32], uint32_t (&hi)[32],
                          float sc) {
      const int z = (which * p.parts + item.part) * p.BH + item.bh;
      const int key_row0 = item.kt * BN + 64 * g;
#pragma unroll
      for (int half = 0; half < (D > 32 ? 2 : 1); ++half) {
        uint32_t(&w)[32] = half == 0 ? lo : hi;
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * sc);
        stage_acquire();
        st_row_swz<C::QRB>(stage, rg, w);
        stage_release();
        if (leader && key_row0 < p.n_k) {
          tma_store_3d(&tmpart, stage, 32 * half, key_row0, z);
          bulk_commit_group();
        }
      }
    };
    uint32_t it = 0, t = 0;
    for (Walk<MODE> at(p); at.x < num_items && ok; at.next(p)) {
      const Item item = bwd_item<MODE>(p, at.x);
      const int key_row0 = item.kt * BN + 64 * g;
      const int b = item.bh / kv_heads, hk = item.bh % kv_heads;
      if (item.n == 0) {
        // no query sees these keys: dK = dV = 0
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = 0u;
        if (SCORED && p.parts > 1) {
          store_part(item, 0, w, w, 1.f);
          store_part(item, 1, w, w, 1.f);
          continue;
        }
        stage_acquire();
        st_row_swz<C::RB>(stage, rg, w);
        stage_release();
        if (leader && key_row0 < p.n_k) {
          tma_store_4d(&tmdk, stage, 0, key_row0, hk, b);
          tma_store_4d(&tmdv, stage, 0, key_row0, hk, b);
          bulk_commit_group();
        }
        continue;
      }
      int qt = item.qt0, member = 0;
      for (int i = 0; i < item.n; ++i, ++t, step(item, qt, member)) {
        if (!wait(&sm.dq_full, t & 1)) break;
        tc_fence_after();
        uint32_t a[32], a2[32];
        tmem_ld32(tmem + lane_off + C::COL_DQ, a);
        if constexpr (D > 32) tmem_ld32(tmem + lane_off + C::COL_DQ + 32, a2);
        tmem_ld_wait(a);
        if constexpr (D > 32) reg_fence(a2);
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.dq_free));
        // fp32 boxes of min(d, 32) columns x 64 rows per group, each added
        // into the accumulator by one TMA reduce; rows past n_q are not touched
        const int q_row0 = qt * BM + 64 * g;
        const int qbh = SCORED ? b * p.H + q_head(item, member) : item.bh;
        stage_acquire();
        st_row_swz<C::QRB>(stage, rg, a);
        stage_release();
        if (leader && q_row0 < p.n_q) {
          tma_reduce_add_3d(&tmdq, stage, 0, q_row0, qbh);
          bulk_commit_group();
        }
        if constexpr (D > 32) {
          stage_acquire();
          st_row_swz<C::QRB>(stage, rg, a2);
          stage_release();
          if (leader && q_row0 < p.n_q) {
            tma_reduce_add_3d(&tmdq, stage, 32, q_row0, qbh);
            bulk_commit_group();
          }
        }
      }
      if (!ok || !wait(&sm.dkv_full, it & 1)) break;
      tc_fence_after();
      // dV, then dK (times the scale); the accumulators are released once
      // both are in registers
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        uint32_t a[32], a2[32], w[32];
        const uint32_t col = which == 0 ? C::COL_DV : C::COL_DK;
        const float sc = which == 0 ? 1.f : p.scale;
        tmem_ld32(tmem + lane_off + col, a);
        if constexpr (D > 32) tmem_ld32(tmem + lane_off + col + 32, a2);
        tmem_ld_wait(a);
        if constexpr (D > 32) reg_fence(a2);
        if (which == 1) {
          tc_fence_before();
          mbar_arrive(smem_u32(&sm.dkv_free));
        }
        if constexpr (SCORED) {
          if (p.parts > 1) {
            store_part(item, which, a, a2, sc);
            continue;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i < D / 2)
            w[i] = pack_bf16x2(__uint_as_float(a[2 * i]) * sc, __uint_as_float(a[2 * i + 1]) * sc);
          if constexpr (D > 32)
            w[16 + i] =
                pack_bf16x2(__uint_as_float(a2[2 * i]) * sc, __uint_as_float(a2[2 * i + 1]) * sc);
        }
        stage_acquire();
        st_row_swz<C::RB>(stage, rg, w);
        stage_release();
        if (leader && key_row0 < p.n_k) {
          tma_store_4d(which == 0 ? &tmdv : &tmdk, stage, 0, key_row0, hk, b);
          bulk_commit_group();
        }
      }
      ++it;
    }
    if (leader) bulk_wait_all();
    if (!ok) record_timeout(p, sm);
  } else {
    // ------------------------------------------------------- elementwise part
    const int quarter = warp & 3;
    const int half = warp >> 2;            // query columns 64*half .. 64*half+63
    const int r = quarter * 32 + lane;      // key row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + COL_S + 64 * half;
    const uint32_t tDP = tmem + lane_off + COL_DP + 64 * half;
    const uint32_t tPT = tmem + lane_off + C::COL_PT + 32 * half;
    const float c = p.scale_log2;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.limit_ns, abort));
      return ok;
    };
    uint32_t t = 0;
    Item item;
    for (Walk<MODE> at(p); ok && find_item(p, num_items, at, item); at.next(p)) {
      const int j = item.kt * BN + r;  // this thread's key
      const bool row_valid = j < item.key_limit;
      int2 rows = make_int2(0, row_valid ? p.n_q : 0);  // kScored: this key's queries
      if constexpr (SCORED) {
        if (p.masked && row_valid)
          rows = __ldg(p.plan.key_rows + static_cast<size_t>(item.bh / kv_heads) * p.n_k + j);
      }
      int qt = item.qt0, member = 0;
      for (int i = 0; i < item.n; ++i, ++t, step(item, qt, member)) {
        // leading columns whose query precedes this key (causal diagonal
        // tile), or all of them for a key past the sequence; with the window,
        // the columns outside [lim, hi) (queries i with j < i - left or
        // j > i + right)
        int lim = 0, hi = 64;
        if (!row_valid) {
          lim = 64;
        } else if (SCORED) {
          const int qbase = qt * BM + 64 * half;
          lim = min(max(rows.x - qbase, 0), 64);
          hi = min(max(rows.y - qbase, 0), 64);
        } else if (p.mask == kMaskCausal && qt == item.kt) {
          lim = min(max(r - 64 * half, 0), 64);
        } else if (BAND) {
          const int qbase = qt * BM + 64 * half;
          lim = min(max(j - p.win_right - qbase, 0), 64);
          hi = min(max(j + p.win_left - qbase + 1, 0), 64);
        }
        if (!wait(&sm.s_full, t & 1)) break;
        // (the stage's lse was copied with its Q; the stage is held until dK of
        // this tile pair, which waits for dS)
        if (CAP && !wait(&sm.q_full[t % QSTAGES], (t / QSTAGES) & 1)) break;
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32(tS, s0);
        tmem_ld32(tS + 32, s1);
        tmem_ld_wait(s0);
        reg_fence(s1);
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.s_free));

        // P = 2^(scale * log2(e) * S') (S' already holds -LSE/scale), zero
        // where forbidden
        float pf[64];
        if constexpr (SCORED) {
          float bias = 0.f, f = 0.f;
          const int ahead = j - qt * BM - 64 * half;
          bool slow = __any_sync(0xffffffffu, lim > 0 || hi < 64);
          bool line = false;
          if constexpr ((MODE & kBias) != 0) {
            const float slope2 = LOG2E * __ldg(p.slopes + q_head(item, member));
            bias = slope2 * static_cast<float>(j - qt * BM);
            f = -2.f * slope2;
            // (with caps only: no mask 2767 -> 2211 us for 8 x 16 x 4096, causal 1155 ->
            // 1190, a third loop; without caps 1620 -> 1587, short causal 152 -> 156)
            line = CAP && !slow && __all_sync(0xffffffffu, ahead >= 63);
            // a query of this half that sees this key and comes before it
            slow = slow || __any_sync(0xffffffffu, lim < hi && lim < ahead);
          }
          const float* lse = sm.lse[CAP ? t % QSTAGES : 0] + (CAP ? 64 * half : 0);
          // P^T goes to tensor memory eight columns at a time, so that it takes
          // no registers, once its previous tile has been read by dV
          auto emit = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            if (i == 0) {
              wait(&sm.p_free, (t & 1) ^ 1);
              tc_fence_after();
            }
            tmem_st4(tPT + i, a0, a1, a2, a3);
          };
          const float fahead = static_cast<float>(ahead);
          bool poly = false;
          if constexpr ((MODE & kWide) != 0) {
            float big = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              big = max3(big, fabsf(__uint_as_float(s0[e])), fabsf(__uint_as_float(s1[e])));
            poly = __all_sync(0xffffffffu, big <= p.cap.small);
            if (poly)
              scored_probabilities<MODE, true, true, false>(p, s0, s1, pf, lim, hi, bias, fahead, f,
                                                            lse, emit);
          }
          if ((MODE & kWide) == 0 || !poly) {
            if (CAP && (MODE & kBias) != 0 && line)
              scored_probabilities<MODE, false, false, CAP && (MODE & kBias) != 0>(
                  p, s0, s1, pf, lim, hi, fmaf(f, fahead, bias), fahead, f, lse, emit);
            else if (slow)
              scored_probabilities<MODE, true, false, false>(p, s0, s1, pf, lim, hi, bias, fahead,
                                                             f, lse, emit);
            else
              scored_probabilities<MODE, false, false, false>(p, s0, s1, pf, lim, hi, bias, fahead,
                                                              f, lse, emit);
          }
          if (!ok) break;
        } else {
#pragma unroll
          for (int i2 = 0; i2 < 32; i2 += 2) {
            const uint32_t* src = i2 < 16 ? s0 + 2 * i2 : s1 + 2 * (i2 - 16);
            float x0, x1, x2, x3;
            fma2(x0, x1, __uint_as_float(src[0]), __uint_as_float(src[1]), c, c, 0.f, 0.f);
            fma2(x2, x3, __uint_as_float(src[2]), __uint_as_float(src[3]), c, c, 0.f, 0.f);
            const int c0 = 2 * i2;
            pf[c0 + 0] = (c0 + 0 < lim || (BAND && c0 + 0 >= hi)) ? 0.f : ex2(x0);
            pf[c0 + 1] = (c0 + 1 < lim || (BAND && c0 + 1 >= hi)) ? 0.f : ex2(x1);
            pf[c0 + 2] = (c0 + 2 < lim || (BAND && c0 + 2 >= hi)) ? 0.f : ex2(x2);
            pf[c0 + 3] = (c0 + 3 < lim || (BAND && c0 + 3 >= hi)) ? 0.f : ex2(x3);
          }
          uint32_t w[32];
#pragma unroll
          for (int i2 = 0; i2 < 32; ++i2) w[i2] = pack_bf16x2(pf[2 * i2], pf[2 * i2 + 1]);
          // P^T of the previous tile pair has been read by its dV product
          if (!wait(&sm.p_free, (t & 1) ^ 1)) break;
          tc_fence_after();
          tmem_st32(tPT, w);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.p_full));

        // dS = P * dP' (dP' already holds -D), computed into registers while
        // the previous tile pair's dK and dQ products still read dS^T
        if (!wait(&sm.dp_full, t & 1)) break;
        tc_fence_after();
        uint32_t e[32];  // dS as bf16 pairs, columns 2i, 2i+1
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t dp[32];
          tmem_ld32(tDP + 32 * h2, dp);
          tmem_ld_wait(dp);
          if (h2 == 1) {
            tc_fence_before();
            mbar_arrive(smem_u32(&sm.dp_free));
          }
#pragma unroll
          for (int cc = 0; cc < 32; cc += 4) {
            const int c0 = 32 * h2 + cc;
            float e0, e1, e2, e3;
            fma2(e0, e1, pf[c0], pf[c0 + 1], __uint_as_float(dp[cc]), __uint_as_float(dp[cc + 1]),
                 0.f, 0.f);
            fma2(e2, e3, pf[c0 + 2], pf[c0 + 3], __uint_as_float(dp[cc + 2]),
                 __uint_as_float(dp[cc + 3]), 0.f, 0.f);
            e[c0 / 2] = pack_bf16x2(e0, e1);
            e[c0 / 2 + 1] = pack_bf16x2(e2, e3);
          }
        }
        // dS^T buffer t % 2 was last read by the products of tile pair t - 2
        if (!wait(&sm.ds_free[t & 1], ((t >> 1) & 1) ^ 1)) break;
        st_row_swz<128>(smem_u32(sm.dst[t & 1][half]), r, e);
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&sm.ds_full));
      }
    }
    if (!ok) record_timeout(p, sm);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// x as hi + mid + lo, three bf16 values (each the rounding of what the
// previous ones leave; together within about 2^-24 of x).
__device__ __forceinline__ uint2 split3_bf16(float x) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(x);
  const float r1 = x - __bfloat162float(hi);
  const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
  const float r2 = r1 - __bfloat162float(mid);
  const __nv_bfloat16 lo = __float2bfloat16_rn(r2);
  uint2 w;
  w.x = static_cast<uint32_t>(__bfloat16_as_ushort(hi)) |
        (static_cast<uint32_t>(__bfloat16_as_ushort(mid)) << 16);
  w.y = static_cast<uint32_t>(__bfloat16_as_ushort(lo));
  return w;
}

struct PreMod {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  RowStrides sq, sk, sv;
  const int2* row_keys;  // [B][n_q], or null: every key
  const int4* header;    // the plan's sizes, or null
  const KeyItem* key_items;
  const float* slopes;
  float scale, softcap;
  int group, n_k, B;
  float* lse_log2;  // with a cap (else null)
};

// x.y over 8 bf16 pairs of lanes' values
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&b);
  float acc = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = __bfloat1622float2(a2[e]), y = __bfloat1622float2(b2[e]);
    acc = fmaf(x.x, y.x, acc);
    acc = fmaf(x.y, y.y, acc);
  }
  return acc;
}

// The items dealt out by load: each, heaviest first, to the CTA with the least
// work so far.  Run by one CTA more of attn_bwd_few_kernel, in the time of the
// pre-kernel, for a plan with documents.  Back and forth is as even where a CTA
// gets many items, or items whose weights fall steadily; with few uneven ones, the
// heaviest nearly a CTA's share, it gives every CTA as many.  Measured on 4 x 4096
// tokens, 16 query heads on 4, d = 64, caps, by the documents in a row, 512 items:
// three 416 -> 381 us, six 337 -> 297, twelve 272 -> 249 (with the masks as bits
// 338, 252 and 219); on 1 x 8192, 16 heads on one, 512 items: 339 -> 306, 285 ->
// 262, 212 -> 201; with 1024 items and more no difference.  It takes 8 us for 512 items, which the pre-kernel hides where it has
// kDealBytes to move: below, 8 x 1000 tokens, d = 32, 59 us became 67.
struct Deal {
  int* next;  // [items], then [ctas] the first ones; null: nothing to do
  int items, ctas, shares, heads;  // shares: items of one key tile; heads: query heads of each
};
constexpr int kMostDealt = 1024, kMostCtas = 256;
constexpr long long kDealPerCta = 4, kDealBytes = 1ll << 26;

__device__ __forceinline__ void deal_items(const Deal& d, const KeyItem* key_items, bool uneven) {
  if (!uneven) {
    for (int c = threadIdx.x; c < d.ctas; c += 256) d.next[d.items + c] = -1;
    return;
  }
  // load << 8 | CTA in 32 bits: a sum of kMostDealt weights stays below 2^24
  constexpr int MOST = (1 << 24) / kMostDealt - 1;
  const int most = max(MOST / d.heads - 1, 0);
  __shared__ uint32_t work[kMostDealt];
  __shared__ uint8_t owner[kMostDealt];
  for (int x = threadIdx.x; x < d.items; x += 256)
    work[x] = static_cast<uint32_t>(min(key_items[x / d.shares].count, most) * d.heads + 1) << 8;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;  // has the CTAs lane, lane + 32, ..
    uint32_t load[kMostCtas / 32];
#pragma unroll
    for (int k = 0; k < kMostCtas / 32; ++k) {
      const int c = lane + 32 * k;  // one each to begin with
      load[k] = c < d.ctas ? work[c] | c : 0xffffffffu;
    }
#pragma unroll 4
    for (int x = d.ctas; x < d.items; ++x) {
      const uint32_t w = work[x];
      uint32_t least = load[0];
#pragma unroll
      for (int k = 1; k < kMostCtas / 32; ++k) least = min(least, load[k]);
      least = __reduce_min_sync(0xffffffffu, least);
#pragma unroll
      for (int k = 0; k < kMostCtas / 32; ++k)
        if (load[k] == least) load[k] = least + w;
      if (lane == 0) owner[x] = static_cast<uint8_t>(least);
    }
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < d.ctas) {
    int last = c;
    for (int x = d.ctas; x < d.items; ++x) {
      if (owner[x] == c) {
        d.next[last] = x;
        last = x;
      }
    }
    d.next[last] = d.items;
    d.next[d.items + c] = c;
  }
}
static_assert(kMostCtas == 256, "a thread a CTA; a CTA's number in a byte");

// D of the queries that see 2 to kFewKeys keys, summed from P and dP in fp32,
// put in the place of the one from O.  That O is rounded to bf16, which errs by
// up to 2^-8 |dO| |O|; with few keys |O| is as large as a value and dP - D
// cancels, so that this rounding alone took the gradients of short documents (2
// to 9 in 17 to 48 tokens) to 6e-3 relative error in an emulation with the
// kernels' roundings; with up to 16 keys summed so they stay below 3.1e-3, with
// up to 32 below 3.0e-3, at any length.  (With one key O is that value exactly.)
//
// A CTA looks at 256 queries, lists those it has work for, and gives each of them,
// head by head, d / 8 threads.  A kernel of its own: the sums want 64 registers, which as
// part of the pre-kernel halved the warps in flight there (4 x 4096 tokens, 16
// heads, d = 64, causal: 45 us in one kernel; 26 us, with these 17 us beside it, in
// two).  Where every query sees few keys it has every row to sum: a window of 16 keys
// takes 510 us in all on 8 x 16 x 4096 tokens, d = 64, where attn_bwd_window, whose D
// is from the rounded O, takes 212.
template <int D>
__global__ void __launch_bounds__(256)
    attn_bwd_few_kernel(const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse,
                        uint8_t* __restrict__ cst, int H, int n_q, int num_qt, RowStrides sdo,
                        const PreMod mod, int heads, const Deal deal) {
  grid_launch_dependents();
  if (deal.next != nullptr && blockIdx.x == 0) {
    const int4 h = __ldg(mod.header);
    deal_items(deal, mod.key_items, h.x == n_q && h.y == mod.n_k && h.z == mod.B && h.w != 0);
    return;
  }
  const int block = blockIdx.x - (deal.next != nullptr);
  constexpr int TPR = D / 8;  // threads a row
  __shared__ int s_row[256], s_first[256], s_seen[256], s_n;
  // the CTA's 256 rows, of one batch entry, and its heads
  const int rows = (n_q + 255) / 256, groups = (H + heads - 1) / heads;
  const unsigned rest = static_cast<unsigned>(block) / groups;
  const int h0 = (block - rest * groups) * heads, hn = min(heads, H - h0);
  const unsigned b32 = rest / rows;
  const int i0 = (rest - b32 * rows) * 256;
  const long long bb = b32;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  {
    const int i = i0 + threadIdx.x;
    int2 keys = make_int2(0, mod.n_k);
    if (mod.row_keys != nullptr) {
      const int4 h = __ldg(mod.header);
      const bool fits = h.x == n_q && h.y == mod.n_k && h.z == mod.B;  // else the main kernel reports it
      keys = i < n_q && fits ? __ldg(mod.row_keys + bb * n_q + i) : make_int2(0, 0);
    }
    const int seen = keys.y - keys.x;
    if (i < n_q && seen > 1 && seen <= kFewKeys) {
      const int at = atomicAdd(&s_n, 1);  // in any order: the rows are apart
      s_row[at] = i;
      s_first[at] = keys.x;
      s_seen[at] = seen;
    }
  }
  __syncthreads();
  // the rows found, of every head
  const int n = s_n * hn, sub = threadIdx.x % TPR;
  for (int w0 = 0; w0 < n; w0 += 256 / TPR) {
    const int item = w0 + threadIdx.x / TPR;
    const bool own = item < n;
    const int at = own ? item / hn : 0, hh = h0 + (own ? item - at * hn : 0);
    const int i = own ? s_row[at] : 0, j0 = own ? s_first[at] : 0;
    const int seen = own ? s_seen[at] : 0;
    const long long bh = bb * H + hh, hk = hh / mod.group;
    const float slope = mod.slopes != nullptr ? __ldg(mod.slopes + hh) : 0.f;
    const __nv_bfloat16* kp = mod.k + bb * mod.sk.b + hk * mod.sk.h + sub * 8;
    const __nv_bfloat16* vp = mod.v + bb * mod.sv.b + hk * mod.sv.h + sub * 8;
    uint4 qv = make_uint4(0u, 0u, 0u, 0u), a = qv;
    float l = 0.f;
    if (own) {
      qv = *reinterpret_cast<const uint4*>(mod.q + bb * mod.sq.b + hh * mod.sq.h +
                                           i * mod.sq.n + sub * 8);
      a = *reinterpret_cast<const uint4*>(dout + bb * sdo.b + hh * sdo.h + i * sdo.n + sub * 8);
      l = lse[static_cast<size_t>(bh) * n_q + i];
    }
    const int most = __reduce_max_sync(0xffffffffu, seen);
    float exact = 0.f, total = 0.f;
    // four keys' loads in flight at a time
    for (int x0 = 0; x0 < most; x0 += 4) {
      uint4 kk[4], vv[4];
      float s[4], dp[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        // (past the last key: the last one again, not counted below)
        const long long j = j0 + max(min(x0 + y, seen - 1), 0);
        kk[y] = *reinterpret_cast<const uint4*>(kp + j * mod.sk.n);
        vv[y] = *reinterpret_cast<const uint4*>(vp + j * mod.sv.n);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        s[y] = dot8(qv, kk[y]);
        dp[y] = dot8(a, vv[y]);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
#pragma unroll
        for (int m = TPR / 2; m > 0; m >>= 1) {
          s[y] += __shfl_xor_sync(0xffffffffu, s[y], m);
          dp[y] += __shfl_xor_sync(0xffffffffu, dp[y], m);
        }
        s[y] *= mod.scale;
        if (mod.softcap > 0.f) s[y] = mod.softcap * tanhf(s[y] / mod.softcap);
        s[y] -= slope * fabsf(static_cast<float>(i - (j0 + x0 + y)));
        if (x0 + y < seen) {
          const float e = expf(s[y] - l);
          total += e;
          exact = fmaf(e, dp[y], exact);
        }
      }
    }
    if (own && sub == 0) {
      const int qt = i / BM, r = i % BM;
      uint8_t* row = cst +
                     (static_cast<size_t>(bh) * num_qt + qt) * static_cast<size_t>(CONST_TILE_BYTES) +
                     (r & 7) * 16 + (r >> 3) * 256;
      // Over the sum of these P, which LSE's error keeps from 1 (by 4e-6 of a score of
      // 20 under a wide cap): where one key has nearly all the weight, dP - D is next to
      // nothing and would be that error (30 % off with a second key at e^-9).
      // (without a finite LSE D is 0, not what the workspace held)
      const uint2 pd = split3_bf16(isfinite(l) && total > 0.f ? -exact / total : 0.f);
      *reinterpret_cast<uint16_t*>(row + 6) = static_cast<uint16_t>(pd.x);
      *reinterpret_cast<uint32_t*>(row + 8) = (pd.x >> 16) | (pd.y << 16);
    }
  }
}

// Per query row (d/8 threads a row, 8 elements each): D = sum_c dO_c O_c, the constant tile's
// row for this query (b = -LSE/scale and -D, three bf16 parts each), and the
// dQ accumulator row set to zero.  Rows n_q .. of the last query tile get zero
// constants (their Q and dO rows are zero-filled by the tile loads, so every
// product they enter is zero).
//
// SCORED (changed scores): the D of queries that attn_bwd_few_kernel takes is left
// to it (`few`); the two run side by side, and the last CTA here ends after it, so
// that what waits for this grid waits for both.
template <int D, bool SCORED>
__global__ void __launch_bounds__(256)
    attn_bwd_pre_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dout,
                        const float* __restrict__ lse, uint8_t* __restrict__ cst,
                        float* __restrict__ dq_acc, int H, int n_q, int num_qt, float inv_scale,
                        RowStrides so, RowStrides sdo, const PreMod mod, bool few) {
  // the main kernel may start launching now: it waits for this grid to
  // complete before it reads the constants or adds into dq_acc
  grid_launch_dependents();
  constexpr int TPR = D / 8;  // threads a row
  // a CTA's rows are of one head (whole tiles of 128 rows, 256 / TPR of them divides)
  const unsigned per_head = static_cast<unsigned>(num_qt) * (BM / (256 / TPR));
  const unsigned bh = blockIdx.x / per_head;
  const int i = static_cast<int>((blockIdx.x - bh * per_head) * (256 / TPR) + threadIdx.x / TPR);
  const int sub = threadIdx.x % TPR;
  const bool valid = i < n_q;
  const size_t src = (static_cast<size_t>(bh) * n_q + i) * D + sub * 8;  // accumulator row
  const unsigned b32 = bh / static_cast<unsigned>(H);
  const long long bb = b32, hh = bh - b32 * H;
  // does the other kernel write this query's D?
  bool skip = false;
  if (SCORED && few) {
    int seen = mod.n_k;
    if (mod.row_keys != nullptr) {
      const int4 h = __ldg(mod.header);
      const bool fits = h.x == n_q && h.y == mod.n_k && h.z == mod.B;  // else the main kernel reports it
      const int2 keys = valid && fits ? __ldg(mod.row_keys + bb * n_q + i) : make_int2(0, 0);
      seen = keys.y - keys.x;
    }
    skip = seen > 1 && seen <= kFewKeys;
  }
  float acc = 0.f;
  if (valid) {
    const uint4 a =
        *reinterpret_cast<const uint4*>(dout + bb * sdo.b + hh * sdo.h + i * sdo.n + sub * 8);
    const uint4 b = *reinterpret_cast<const uint4*>(o + bb * so.b + hh * so.h + i * so.n + sub * 8);
    acc = dot8(a, b);
    float4* z = reinterpret_cast<float4*>(dq_acc + src);
    z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int m = TPR / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
  if (sub < 2) {
    // sub 0: columns 0-7 of this query's row (b in 0-2, -D in 3-5); sub 1:
    // columns 8-15, zero
    const int qt = i / BM, n = i % BM;
    uint8_t* tile =
        cst + (static_cast<size_t>(bh) * num_qt + qt) * static_cast<size_t>(CONST_TILE_BYTES);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (sub == 0 && valid) {
      const float l = lse[static_cast<size_t>(bh) * n_q + i];
      // -inf only for a row that sees no key; a cap takes LSE off after the tanh
      float b = isfinite(l) && !(SCORED && mod.lse_log2 != nullptr) ? -l * inv_scale : 0.f;
      // the distance bias's share of the query, counted from its tile's first
      if (SCORED && mod.slopes != nullptr && mod.lse_log2 == nullptr)
        b = fmaf(-__ldg(mod.slopes + hh) * inv_scale, static_cast<float>(n), b);
      const uint2 pb = split3_bf16(b);
      const uint2 pd = split3_bf16(-acc);
      w.x = pb.x;                         // b_hi, b_mid
      w.y = pb.y | (pd.x << 16);          // b_lo, -D_hi
      w.z = (pd.x >> 16) | (pd.y << 16);  // -D_mid, -D_lo
    }
    uint8_t* dst = tile + (n & 7) * 16 + (n >> 3) * 256 + sub * 128;
    if (SCORED && skip && valid && sub == 0) {
      *reinterpret_cast<uint32_t*>(dst) = w.x;
      *reinterpret_cast<uint16_t*>(dst + 4) = static_cast<uint16_t>(w.y);
      *reinterpret_cast<uint32_t*>(dst + 12) = 0u;
    } else {
      *reinterpret_cast<uint4*>(dst) = w;
    }
    if (SCORED && mod.lse_log2 != nullptr && sub == 0) {
      const float l = valid ? lse[static_cast<size_t>(bh) * n_q + i] : 0.f;
      const float far = mod.slopes != nullptr ? __ldg(mod.slopes + hh) * static_cast<float>(n) : 0.f;
      mod.lse_log2[(static_cast<size_t>(bh) * num_qt + qt) * BM + n] =
          ((isfinite(l) ? l : 0.f) + far) * LOG2E;
    }
  }
  if (SCORED && few && blockIdx.x == gridDim.x - 1) grid_dependency_wait();
}

// The sizes that a call's plan has to be of; header null: there is no plan.  Under a
// plan of others the main kernel computes nothing and reports it, and the kernels
// after it write no gradients.
struct PlanSizes {
  const int4* header;
  int n_q, n_k, B;
  __device__ __forceinline__ bool fit() const {
    if (header == nullptr) return true;
    const int4 h = __ldg(header);
    return h.x == n_q && h.y == n_k && h.z == B;
  }
};

// dQ = scale * accumulator, rounded to bf16, written through dq's strides;
// 8 elements a thread (d8 = d / 8 threads a row).
__global__ void __launch_bounds__(256)
    attn_bwd_dq_kernel(const float* __restrict__ dq_acc, __nv_bfloat16* __restrict__ dq,
                       float scale, long long n8, int d8, int H, int n_q, RowStrides sdq,
                       const PlanSizes plan) {
  grid_dependency_wait();  // the main kernel's additions into dq_acc are complete
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n8 || !plan.fit()) return;
  const long long r = i / d8;  // row (b * H + hh) * n_q + qi of the accumulator
  const long long bh = r / n_q;
  const long long dst =
      (bh / H) * sdq.b + (bh % H) * sdq.h + (r - bh * n_q) * sdq.n + (i - r * d8) * 8;
  const float4 a = reinterpret_cast<const float4*>(dq_acc)[2 * i];
  const float4 b = reinterpret_cast<const float4*>(dq_acc)[2 * i + 1];
  uint4 out;
  out.x = pack_bf16x2(a.x * scale, a.y * scale);
  out.y = pack_bf16x2(a.z * scale, a.w * scale);
  out.z = pack_bf16x2(b.x * scale, b.y * scale);
  out.w = pack_bf16x2(b.z * scale, b.w * scale);
  *reinterpret_cast<uint4*>(dq + dst) = out;
}

// dK and dV of key heads whose query heads were worked on in parts: the parts'
// fp32 sums added up in order and rounded to bf16, 8 elements a thread.
// grid.y: 0 dV, 1 dK.
__global__ void __launch_bounds__(256)
    attn_bwd_dkv_kernel(const float* __restrict__ acc, __nv_bfloat16* __restrict__ dk,
                        __nv_bfloat16* __restrict__ dv, int parts, long long n8, int d8, int HK,
                        int n_k, RowStrides sdk, RowStrides sdv, const PlanSizes plan) {
  grid_dependency_wait();  // the parts are complete
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n8 || !plan.fit()) return;
  const long long r = i / d8;  // row (b * HK + head) * n_k + key
  const long long bh = r / n_k;
  const bool is_k = blockIdx.y == 1;
  const RowStrides st = is_k ? sdk : sdv;
  const long long dst =
      (bh / HK) * st.b + (bh % HK) * st.h + (r - bh * n_k) * st.n + (i - r * d8) * 8;
  const float4* src = reinterpret_cast<const float4*>(acc) + (is_k ? parts * n8 * 2 : 0) + 2 * i;
  float4 a = src[0], b = src[1];
  for (int x = 1; x < parts; ++x) {
    const float4 c = src[x * n8 * 2], e = src[x * n8 * 2 + 1];
    a = make_float4(a.x + c.x, a.y + c.y, a.z + c.z, a.w + c.w);
    b = make_float4(b.x + e.x, b.y + e.y, b.z + e.z, b.w + e.w);
  }
  uint4 out;
  out.x = pack_bf16x2(a.x, a.y);
  out.y = pack_bf16x2(a.z, a.w);
  out.z = pack_bf16x2(b.x, b.y);
  out.w = pack_bf16x2(b.z, b.w);
  *reinterpret_cast<uint4*>((is_k ? dk : dv) + dst) = out;
}

}  // namespace

// A key head's query heads are worked on in parts, each an item of its own, when
// there are too few (key tile, key head) items to even out over the SMs: in as
// many as make kPartItems of them.  Parts cost their dK and dV in fp32 once more
// through memory, so there are no more than that.  Packed documents in 2 x 333
// tokens, 8 query heads on 2, d = 32, 12 items: 41.6 us in one part, 28.6 us in
// four.  4 x 4096 tokens, 16 query heads on 4, d = 64, 512 items: 350 us in one
// part, 350 us in two, 375 us in four.
constexpr long long kPartItems = 512;

int bwd_parts(int B, int H, int HK, int n_k) {
  const int group = H / HK;
  const long long items = static_cast<long long>(B) * HK * ((n_k + BN - 1) / BN);
  for (int parts = 1; parts < group; ++parts)
    if (group % parts == 0 && items * parts >= kPartItems) return parts;
  return group;
}

BwdLayout bwd_layout(int B, int H, int n_q, int d) {
  BwdLayout l;
  const size_t bh = static_cast<size_t>(B) * H;
  l.num_qt = (n_q + BM - 1) / BM;
  l.cst_off = 0;
  l.dq_acc_off = bh * l.num_qt * CONST_TILE_BYTES;
  l.lse_off = l.dq_acc_off + bh * static_cast<size_t>(n_q) * d * 4;
  l.bytes = l.lse_off;
  l.deal_off = l.lse_off + bh * l.num_qt * BM * 4;
  l.part_off = l.deal_off + (kMostDealt + kMostCtas) * 4;
  l.scored_bytes = l.part_off;
  return l;
}

BwdLayout bwd_scored_layout(int B, int H, int HK, int n_q, int n_k, int d) {
  BwdLayout l = bwd_layout(B, H, n_q, d);
  l.parts = bwd_parts(B, H, HK, n_k);
  if (l.parts > 1)
    l.scored_bytes += 2 * static_cast<size_t>(l.parts) * B * HK * n_k * d * 4;
  return l;
}

namespace {

template <int MODE, int D>
cudaError_t launch_bwd_main(const Params& p, const CUtensorMap* maps, const LaunchCtx& ctx) {
  static_assert(sizeof(Smem<D, MODE>) + 1024 <= 232448, "shared memory");
  const size_t smem = sizeof(Smem<D, MODE>) + 1024;
  cudaError_t err = cudaFuncSetAttribute(attn_bwd_tc_kernel<MODE, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int grid = p.num_items < ctx.num_sms ? p.num_items : ctx.num_sms;
  return launch_dependent(attn_bwd_tc_kernel<MODE, D>, dim3(grid), dim3(NUM_THREADS), smem,
                          ctx.stream, maps[0], maps[1], maps[2], maps[3], maps[4], maps[5],
                          maps[6], maps[7], p);
}

template <int D>
cudaError_t launch_bwd_d(const BwdProblem& pb, const CUtensorMap* maps, void* workspace,
                         const LaunchCtx& ctx, const ScoreMod* mod) {
  const BwdLayout lay = bwd_layout(pb.B, pb.H, pb.n_q, D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* cst = ws + lay.cst_off;
  float* dq_acc = reinterpret_cast<float*>(ws + lay.dq_acc_off);
  float* lse_log2 = mod != nullptr && mod->softcap > 0.f
                        ? reinterpret_cast<float*>(ws + lay.lse_off)
                        : nullptr;
  const long long bh = static_cast<long long>(pb.B) * pb.H;

  const long long rows = bh * static_cast<long long>(lay.num_qt) * BM;
  constexpr int rows_per_block = 256 / (D / 8);
  const long long pre_blocks = (rows + rows_per_block - 1) / rows_per_block;
  PreMod pm{};
  if (mod != nullptr) {
    pm.q = static_cast<const __nv_bfloat16*>(pb.q);
    pm.k = static_cast<const __nv_bfloat16*>(pb.k);
    pm.v = static_cast<const __nv_bfloat16*>(pb.v);
    pm.sq = mod->sq;
    pm.sk = mod->sk;
    pm.sv = mod->sv;
    pm.row_keys = mod->masked ? mod->plan.row_keys : nullptr;
    pm.header = mod->plan.header;
    pm.key_items = mod->plan.key_items;
    pm.slopes = mod->slopes;
    pm.scale = pb.scale;
    pm.softcap = mod->softcap;
    pm.group = mod->group;
    pm.n_k = pb.n_k;
    pm.B = pb.B;
    pm.lse_log2 = lse_log2;
  }
  const auto* o = static_cast<const __nv_bfloat16*>(pb.o);
  const auto* dout = static_cast<const __nv_bfloat16*>(pb.dout);
  const int num_qt = static_cast<int>(lay.num_qt);
  const bool few = mod != nullptr && bwd_few_possible(mod->masked, pb.n_k);
  cudaError_t err = cudaSuccess;
  Deal deal{};
  if (few) {
    // four CTAs an SM are resident: heads of the same rows share one as far as it
    // takes for all to be
    const long long tiles = static_cast<long long>(pb.B) * ((pb.n_q + 255) / 256);
    const long long shares = std::min<long long>(
        pb.H, std::max<long long>(1, 4LL * ctx.num_sms / tiles));  // CTAs of the same rows
    const int heads = static_cast<int>((pb.H + shares - 1) / shares);
    long long blocks = tiles * ((pb.H + heads - 1) / heads);  // no more than pre_blocks
    const long long items = bh / mod->group * ((pb.n_k + BN - 1) / BN) * mod->parts;
    if (mod->masked && items > ctx.num_sms && items <= kDealPerCta * ctx.num_sms &&
        items <= kMostDealt && ctx.num_sms <= kMostCtas &&
        rows * (8 * D + 36) >= kDealBytes) {
      deal.next = reinterpret_cast<int*>(ws + lay.deal_off);
      deal.items = static_cast<int>(items);
      deal.ctas = ctx.num_sms;
      deal.shares = pb.H / mod->group * mod->parts;
      deal.heads = mod->group / mod->parts;
      ++blocks;
    }
    attn_bwd_few_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, ctx.stream>>>(
        dout, pb.lse, cst, pb.H, pb.n_q, num_qt, pb.sdo, pm, heads, deal);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    err = launch_dependent(attn_bwd_pre_kernel<D, true>, dim3(static_cast<unsigned>(pre_blocks)),
                           dim3(256), 0, ctx.stream, o, dout, pb.lse, cst, dq_acc, pb.H, pb.n_q,
                           num_qt, 1.f / pb.scale, pb.so, pb.sdo, pm, true);
  } else {
    auto* pre = mod != nullptr ? attn_bwd_pre_kernel<D, true> : attn_bwd_pre_kernel<D, false>;
    pre<<<static_cast<unsigned>(pre_blocks), 256, 0, ctx.stream>>>(
        o, dout, pb.lse, cst, dq_acc, pb.H, pb.n_q, num_qt, 1.f / pb.scale, pb.so, pb.sdo, pm, false);
    err = cudaGetLastError();
  }
  if (err != cudaSuccess) return err;

  Params p{};
  p.cst = cst;
  p.key_lens = pb.key_lens;
  p.H = pb.H;
  p.n_q = pb.n_q;
  p.n_k = pb.n_k;
  p.BH = static_cast<int>(bh);
  p.mask = pb.mask;
  p.win_left = pb.win_left;
  p.win_right = pb.win_right;
  p.num_qt = (pb.n_q + BM - 1) / BM;
  p.num_kt = (pb.n_k + BN - 1) / BN;
  p.num_items = p.BH * p.num_kt;
  p.scale_log2 = pb.scale * LOG2E;
  p.scale = pb.scale;
  p.limit_ns = ctx.limit_ns;
  p.status = ctx.status;
  // the main and the dQ kernels start while their predecessor drains
  // (programmatic dependent launch; each waits for it before reading its output)
  if (mod != nullptr) {
    p.mask = kMaskNone;
    p.group = mod->group;
    p.parts = mod->parts;
    p.BH = p.BH / mod->group;
    p.num_items = p.BH * p.num_kt * p.parts;
    p.cap_log2 = mod->softcap * LOG2E;
    p.cap_in = mod->softcap > 0.f ? 2.f * p.scale_log2 / mod->softcap : 0.f;
    p.slopes = mod->slopes;
    p.cap = cap_poly(pb.scale, mod->softcap);
    p.lse_log2 = lse_log2;
    p.masked = mod->masked;
    p.plan = mod->plan;
    p.next = deal.next;
    const bool cap = mod->softcap > 0.f, bias = mod->slopes != nullptr;
    const bool wide = mod->softcap > kWideCap;
    err = wide && bias  ? launch_bwd_main<kScored | kCap | kWide | kBias, D>(p, maps, ctx)
          : wide        ? launch_bwd_main<kScored | kCap | kWide, D>(p, maps, ctx)
          : cap && bias ? launch_bwd_main<kScored | kCap | kBias, D>(p, maps, ctx)
          : cap       ? launch_bwd_main<kScored | kCap, D>(p, maps, ctx)
          : bias      ? launch_bwd_main<kScored | kBias, D>(p, maps, ctx)
                      : launch_bwd_main<kScored, D>(p, maps, ctx);
  } else if (pb.mask == kMaskBand) {
    err = launch_bwd_main<kBand, D>(p, maps, ctx);
  } else {
    err = launch_bwd_main<kPlain, D>(p, maps, ctx);
  }
  if (err != cudaSuccess) return err;

  const PlanSizes sizes{mod != nullptr && mod->masked ? mod->plan.header : nullptr, pb.n_q, pb.n_k,
                        pb.B};
  const long long n8 = bh * pb.n_q * (D / 8);
  err = launch_dependent(attn_bwd_dq_kernel, dim3(static_cast<unsigned>((n8 + 255) / 256)),
                         dim3(256), 0, ctx.stream, static_cast<const float*>(dq_acc),
                         static_cast<__nv_bfloat16*>(pb.dq), pb.scale, n8, D / 8, pb.H, pb.n_q,
                         pb.sdq, sizes);
  if (err != cudaSuccess || mod == nullptr || mod->parts == 1) return err;
  const int HK = pb.H / mod->group;
  const long long k8 = static_cast<long long>(pb.B) * HK * pb.n_k * (D / 8);
  return launch_dependent(attn_bwd_dkv_kernel, dim3(static_cast<unsigned>((k8 + 255) / 256), 2),
                          dim3(256), 0, ctx.stream,
                          reinterpret_cast<const float*>(ws + lay.part_off),
                          static_cast<__nv_bfloat16*>(pb.dk), static_cast<__nv_bfloat16*>(pb.dv),
                          mod->parts, k8, D / 8, HK, pb.n_k, mod->sdk, mod->sdv, sizes);
}

}  // namespace

bool bwd_head_size_ok(int d) { return d == 16 || d == 32 || d == 64; }

cudaError_t launch_bwd(const BwdProblem& pb, const CUtensorMap* maps, void* workspace,
                       const LaunchCtx& ctx, const ScoreMod* mod) {
  switch (pb.d) {
    case 16: return launch_bwd_d<16>(pb, maps, workspace, ctx, mod);
    case 32: return launch_bwd_d<32>(pb, maps, workspace, ctx, mod);
    case 64: return launch_bwd_d<64>(pb, maps, workspace, ctx, mod);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
