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
// Bound by HBM: every visible cache byte is read once.  An 8-bit cache leaves
// 4 FLOPs per byte and query row, so with G * n_q rows per key head the CUDA
// cores would be the bound from about 5 rows on; the products run on the
// tensor cores instead, in the warp-level m16n8k16 form: the tile of queries
// (at most 32 rows) is far too small for a tcgen05 tile, and this form takes
// its operands straight from registers, so cache rows go from global memory
// to the products without a stop in shared memory:
//   S = Q K^T  queries are the 16 rows, 8 keys the columns;
//   O^T = V^T P^T  16 values of d are the rows, 8 queries the columns: the
//       accumulator layout of S is the operand layout of P^T as it stands.
// The k index of a product may be permuted freely when both operands agree,
// so a lane's 16 consecutive bytes of a key row are whole operands, and the
// rows of O^T likewise, so a lane's 16 consecutive bytes of a value row are.
//
// 8-bit codes are widened to f16, which holds both kinds exactly; q is
// brought to f16 by a power of two per row (exact down to 2^-25 of the row's
// largest entry), P and the value scales are multiplied in fp32 (relative to
// the largest value scale so far) before the rounding to f16.  A bf16 cache
// multiplies in bf16, P rounded to bf16 as in the forward.  Softmax
// statistics, scores and accumulators are fp32.
//
// One CTA of four warps works on one chunk of one key head's cache; warp w
// takes every fourth tile of KT keys with its own running softmax, the warps
// are merged in shared memory, and chunks through the workspace by a second
// kernel.  A warp asks for a tile's values before its scores and for the next
// tile's keys before its softmax, so about KT rows are in flight per warp.
#pragma once

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

struct ScoredDecParams {
  const __nv_bfloat16* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* o;
  float* lse;
  float* part;  // [unit][split][rows of the unit][D + 2]
  const int* cache_lens;
  const float* slopes;
  RowStrides sq, sk, sv, so;
  int HK, G, n_q, L_max, T_log2, num_blocks, window, splits, row_tiles;
  float scale, softcap;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
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

// BYTES (2, 4, 8 or 16) from global memory into the first words of w.
template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* src, bool in, uint32_t* w) {
  if (BYTES == 16) {
    const uint4 x = in ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if (BYTES == 8) {
    const uint2 x = in ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
    w[0] = x.x, w[1] = x.y;
  } else if (BYTES == 4) {
    w[0] = in ? __ldg(reinterpret_cast<const uint32_t*>(src)) : 0u;
  } else {
    w[0] = in ? __ldg(reinterpret_cast<const uint16_t*>(src)) : 0u;
  }
}

// Shapes per cache format, head size D and row tiles (8 queries each).
template <int FMT_, int D_, int NR_>
struct DCfg {
  static constexpr int FMT = FMT_, D = D_, NR = NR_;
  static constexpr int ES = FMT_ == kCacheBf16 ? 2 : 1;
  static constexpr int RB = D_ * ES;  // bytes of a cache row
  // keys per warp and tile: about 4 KB of keys, or 2 KB where the accumulators
  // of more query rows need the registers
  static constexpr int KT1 = RB >= 256 ? 16 : (RB >= 128 ? 32 : 64);
  static constexpr int KT = NR_ > 1 && KT1 > 16 ? KT1 / 2 : KT1;
  static constexpr int NT = KT / 8;   // 8-key column tiles of S
  static constexpr int NG = KT / 16;  // 16-key groups (one k step of O^T)
  // K: a lane's share of a row, in loads of KV bytes
  static constexpr int KV = RB / 4 < 16 ? RB / 4 : 16;
  static constexpr int KL = RB / 4 / KV;
  static constexpr int KW = KV / 4;          // words per load
  static constexpr int KE = KV / ES;         // elements per load
  static constexpr int KS = D_ / 16;         // k steps of S
  // V: a lane's share of a row, in loads of VV bytes
  static constexpr int VV = RB / 8 < 16 ? RB / 8 : 16;
  static constexpr int VL = RB / 8 / VV;
  static constexpr int VW = VV < 4 ? 1 : VV / 4;
  static constexpr int VE = VV / ES;
  static constexpr int MT = D_ / 16;         // 16-row tiles of O^T
  static constexpr int MQ = NR_ > 1 ? NR_ / 2 : 1;  // 16-query tiles of S
  // CTAs per SM that the registers allow
  static constexpr int CTAS = NR_ > 1 ? 2 : 3;
};

// One element pair per lane and m16n8k16 step s: which elements of a row
// lane t holds is  load i, elements 4 s' .. 4 s' + 3  with s = i * KE/4 + s'.
template <class C>
__device__ __forceinline__ int key_elem(int step, int t) {
  constexpr int per = C::KE / 4;
  return (step / per) * 4 * C::KE + t * C::KE + 4 * (step % per);
}
// The d index of a lane's e-th value element (group g).
template <class C>
__device__ __forceinline__ int val_elem(int e, int g) {
  return (e / C::VE) * 8 * C::VE + g * C::VE + e % C::VE;
}

template <int FMT, int D, int NR>
__global__ void __launch_bounds__(DW * 32, DCfg<FMT, D, NR>::CTAS)
    attn_decode_scored_kernel(const ScoredDecParams p) {
  using C = DCfg<FMT, D, NR>;
  constexpr int KT = C::KT, NT = C::NT, NG = C::NG, MQ = C::MQ;
  constexpr bool Q8 = FMT != kCacheBf16;
  constexpr int ROWS = NR * 8;
  extern __shared__ float sm[];  // per warp [ROWS][D + 2]: O, m, l
  grid_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // unit = ((b * HK + key head) * row_tiles + row tile) * splits + split
  const int split = static_cast<int>(blockIdx.x % p.splits);
  const long long unit = blockIdx.x / p.splits;
  const int rt = static_cast<int>(unit % p.row_tiles);
  const long long bk = unit / p.row_tiles;
  const int b = static_cast<int>(bk / p.HK), hk = static_cast<int>(bk % p.HK);
  const int rows = min(p.G * p.n_q - rt * ROWS, ROWS);  // query rows of this unit

  int L = p.L_max;
  if (p.cache_lens != nullptr) L = min(max(__ldg(p.cache_lens + b), 0), p.L_max);
  // keys any row of the unit can see, from a 16-key boundary on (so that a
  // 16-key group never crosses a scale block)
  const int key0 = p.window >= 0 ? max(L - p.n_q - p.window, 0) : 0;
  const int base0 = key0 & ~15;
  // an equal share of this sequence's tiles per split
  const int tiles = (L - base0 + KT - 1) / KT;
  const int per = (tiles + p.splits - 1) / p.splits;
  const int tile_end = min(tiles, (split + 1) * per);
  const int tile0 = split * per + warp;

  const long long krow0 = (b * p.sk.b + hk * p.sk.h) * C::ES;
  const long long vrow0 = (b * p.sv.b + hk * p.sv.h) * C::ES;
  const uint8_t* kp = p.k + krow0 + t * C::KV;
  const uint8_t* vp = p.v + vrow0 + g * C::VV;
  const long long ksn = p.sk.n * C::ES, vsn = p.sv.n * C::ES;

  uint32_t kr[NT][C::KL * C::KW];  // K: lane g's row of each 8-key tile
  uint32_t vr[NG][4][C::VL * C::VW];  // V: keys 2t, 2t+1, 2t+8, 2t+9 of each group
  float ks[NG], vs[NG];
  const float* ksp = Q8 ? p.k_scale + bk * p.num_blocks : nullptr;
  const float* vsp = Q8 ? p.v_scale + bk * p.num_blocks : nullptr;

  auto load_k = [&](int tile) {
    const int base = base0 + tile * KT;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = base + 8 * n + g;
      const bool in = j < L && j >= key0;
      const uint8_t* src = kp + j * ksn;
#pragma unroll
      for (int i = 0; i < C::KL; ++i)
        load_bytes<C::KV>(src + 4 * C::KV * i, in, &kr[n][i * C::KW]);
    }
    if (Q8) {
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const int j = base + 16 * n;
        ks[n] = j < L ? __ldg(ksp + (j >> p.T_log2)) : 0.f;
      }
    }
  };
  auto load_v = [&](int tile) {
    const int base = base0 + tile * KT;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = base + 16 * n + 2 * t + (e & 1) + (e >> 1) * 8;
        const bool in = j < L && j >= key0;
        const uint8_t* src = vp + j * vsn;
#pragma unroll
        for (int i = 0; i < C::VL; ++i)
          load_bytes<C::VV>(src + 8 * C::VV * i, in, &vr[n][e][i * C::VW]);
      }
      if (Q8) {
        const int j = base + 16 * n;
        vs[n] = j < L ? __ldg(vsp + (j >> p.T_log2)) : 0.f;
      }
    }
  };
  if (tile0 < tile_end) load_k(tile0);

  // Queries in operand form: rows g and g + 8 of each 16-query tile.
  uint32_t qa[MQ][C::KS][4];
  float qscale[MQ][2], nslope[MQ][2];
  int pos[MQ][2];
#pragma unroll
  for (int m = 0; m < MQ; ++m) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = m * 16 + r * 8 + g;
      const bool in = row < rows && (NR > 1 || r == 0);
      const int gr = rt * ROWS + (in ? row : 0);
      const int head = hk * p.G + gr / p.n_q, qi = gr % p.n_q;
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
      qscale[m][r] = p.scale;
      if (Q8) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(min(static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127, 126), -126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        qscale[m][r] = p.scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
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
      pos[m][r] = in ? L - p.n_q + qi : -1;
      nslope[m][r] = p.slopes != nullptr && in ? -__ldg(p.slopes + head) * kLog2e : 0.f;
    }
  }
  const bool capped = p.softcap > 0.f;
  const float inv_cap = capped ? 1.f / p.softcap : 0.f;
  const float cap2 = p.softcap * kLog2e;
  const bool biased = p.slopes != nullptr;

  float m_run[MQ][2], l_run[MQ][2];
  float acc[C::MT][NR][4];
#pragma unroll
  for (int m = 0; m < MQ; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) m_run[m][r] = -INFINITY, l_run[m][r] = 0.f;
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
  float vref = 0.f, inv_vref = 0.f;  // the value scale that P is held relative to

  for (int tile = tile0; tile < tile_end; tile += DW) {
    const int base = base0 + tile * KT;
    load_v(tile);
    // ---- S = Q K^T
    float s[MQ][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int m = 0; m < MQ; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
#pragma unroll
      for (int st = 0; st < C::KS; ++st) {
        uint32_t b0, b1;
        if (Q8) {
          widen4<FMT>(kr[n][st], b0, b1);  // word st: elements 4 st .. 4 st + 3 of the lane
        } else {
          b0 = kr[n][2 * st];
          b1 = kr[n][2 * st + 1];
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
    float kf[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) kf[n] = Q8 ? ks[n] : 1.f;
    if (tile + DW < tile_end) load_k(tile + DW);

    // ---- scores in log2 units, masked; their maximum per row
    float mx[MQ][2];
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
#pragma unroll
      for (int r = 0; r < (NR > 1 ? 2 : 1); ++r) {
        mx[m][r] = -INFINITY;
        const float far = static_cast<float>(pos[m][r] - base);  // distance to the tile's first key
        const bool whole =
            base + KT - 1 <= pos[m][r] && base >= key0 &&
            (p.window < 0 || base >= pos[m][r] - p.window);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f = qscale[m][r] * kf[n / 2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = s[m][n][2 * r + c] * f;
            if (capped) {
              // tanh(y) = 1 - 2 / (1 + e^2y)
              const float e2 = ex2(x * inv_cap * (2.f * kLog2e));
              x = fmaf(-2.f * cap2, rcp(1.f + e2), cap2);
            } else {
              x *= kLog2e;
            }
            const int col = 8 * n + 2 * t + c;
            if (biased) x = fmaf(nslope[m][r], far - static_cast<float>(col), x);
            if (!whole) {
              const int j = base + col;
              if (j > pos[m][r] || j < key0 || (p.window >= 0 && j < pos[m][r] - p.window))
                x = -INFINITY;
            }
            s[m][n][2 * r + c] = x;
            mx[m][r] = fmaxf(mx[m][r], x);
          }
        }
      }
    }
    bool grow = false;
#pragma unroll
    for (int m = 0; m < MQ; ++m)
#pragma unroll
      for (int r = 0; r < (NR > 1 ? 2 : 1); ++r) {
        mx[m][r] = fmaxf(mx[m][r], __shfl_xor_sync(0xffffffffu, mx[m][r], 1));
        mx[m][r] = fmaxf(mx[m][r], __shfl_xor_sync(0xffffffffu, mx[m][r], 2));
        grow |= mx[m][r] > m_run[m][r] + kRescale;
      }
    float vtop = 0.f;
    if (Q8) {
#pragma unroll
      for (int n = 0; n < NG; ++n) vtop = fmaxf(vtop, vs[n]);
    }
    if (__any_sync(0xffffffffu, grow || (Q8 && vtop > vref))) {
      float vfac = 1.f;
      if (Q8 && vtop > vref) {
        vfac = vref / (2.f * vtop);  // 0 the first time; room for the scales to come
        vref = 2.f * vtop;
        inv_vref = 1.f / vref;
      }
#pragma unroll
      for (int m = 0; m < MQ; ++m) {
#pragma unroll
        for (int r = 0; r < (NR > 1 ? 2 : 1); ++r) {
          float alpha = 1.f;
          if (mx[m][r] > m_run[m][r] + kRescale) {
            alpha = ex2(m_run[m][r] - mx[m][r]);  // 0 when nothing was seen before
            m_run[m][r] = mx[m][r];
            l_run[m][r] *= alpha;
          }
          alpha *= vfac;
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
    // ---- P, its row sums, and P^T as the operand of O^T
    uint32_t pb[NG][NR][2];
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
#pragma unroll
      for (int r = 0; r < (NR > 1 ? 2 : 1); ++r) {
        const float base_m = m_run[m][r] == -INFINITY ? 0.f : m_run[m][r];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float p0 = ex2(s[m][n][2 * r] - base_m), p1 = ex2(s[m][n][2 * r + 1] - base_m);
          sum += p0 + p1;
          if (Q8) {
            const float f = vs[n / 2] * inv_vref;
            const __half2 y = __floats2half2_rn(p0 * f, p1 * f);
            pb[n / 2][2 * m + r][n & 1] = *reinterpret_cast<const uint32_t*>(&y);
          } else {
            pb[n / 2][2 * m + r][n & 1] = pack_bf16x2(p0, p1);
          }
        }
        l_run[m][r] += sum;
      }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int n = 0; n < NG; ++n) {
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
        constexpr int WORDS = C::VL * C::VW;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          // elements 4w .. 4w+3 of the lane: two 16-row tiles (one when D = 16)
          uint32_t a[2][2], c[2][2];
          widen4<FMT>(__byte_perm(vr[n][0][w], vr[n][1][w], 0x5140), a[0][0], a[0][1]);
          widen4<FMT>(__byte_perm(vr[n][2][w], vr[n][3][w], 0x5140), c[0][0], c[0][1]);
          product(2 * w, a[0][0], a[0][1], c[0][0], c[0][1]);
          if (C::MT > 1) {
            widen4<FMT>(__byte_perm(vr[n][0][w], vr[n][1][w], 0x7362), a[1][0], a[1][1]);
            widen4<FMT>(__byte_perm(vr[n][2][w], vr[n][3][w], 0x7362), c[1][0], c[1][1]);
            product((2 * w + 1) % C::MT, a[1][0], a[1][1], c[1][0], c[1][1]);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < C::MT; ++w) {
          product(w, __byte_perm(vr[n][0][w], vr[n][1][w], 0x5410),
                  __byte_perm(vr[n][0][w], vr[n][1][w], 0x7632),
                  __byte_perm(vr[n][2][w], vr[n][3][w], 0x5410),
                  __byte_perm(vr[n][2][w], vr[n][3][w], 0x7632));
        }
      }
    }
  }

  // ---- the warps' partial results into shared memory
  float* mine = sm + static_cast<size_t>(warp) * ROWS * (D + 2);
#pragma unroll
  for (int m = 0; m < MQ; ++m)
#pragma unroll
    for (int r = 0; r < (NR > 1 ? 2 : 1); ++r) {
      float l = l_run[m][r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t == 0) {
        float* row = mine + (m * 16 + r * 8 + g) * (D + 2);
        row[D] = m_run[m][r];
        row[D + 1] = l;
      }
    }
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = x * 8 + 2 * t + (e & 1);
        const int d = val_elem<C>(2 * i + (e >> 1), g);
        mine[row * (D + 2) + d] = acc[i][x][e] * (Q8 ? vref : 1.f);
      }
  __syncthreads();
  for (int row = warp; row < rows; row += DW) {
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < DW; ++w) mm = fmaxf(mm, sm[(w * ROWS + row) * (D + 2) + D]);
    const float mb = mm == -INFINITY ? 0.f : mm;
    float f[DW], ll = 0.f;
#pragma unroll
    for (int w = 0; w < DW; ++w) {
      f[w] = ex2(sm[(w * ROWS + row) * (D + 2) + D] - mb);
      ll += f[w] * sm[(w * ROWS + row) * (D + 2) + D + 1];
    }
    const int gr = rt * ROWS + row;
    const int head = hk * p.G + gr / p.n_q, qi = gr % p.n_q;
    float* part = p.part == nullptr
                      ? nullptr
                      : p.part + ((unit * p.splits + split) * ROWS + row) * (D + 2);
    __nv_bfloat16* out = p.o + b * p.so.b + head * p.so.h + qi * p.so.n;
    const float inv = ll > 0.f ? 1.f / ll : 0.f;
    for (int d = lane; d < D; d += 32) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < DW; ++w) a += f[w] * sm[(w * ROWS + row) * (D + 2) + d];
      if (part != nullptr)
        part[d] = a;
      else
        out[d] = __float2bfloat16_rn(a * inv);
    }
    if (lane == 0) {
      if (part != nullptr) {
        part[D] = mm;
        part[D + 1] = ll;
      } else if (p.lse != nullptr) {
        p.lse[(static_cast<long long>(b) * p.HK * p.G + head) * p.n_q + qi] =
            ll > 0.f ? (mm + __log2f(ll)) * kLn2 : -INFINITY;
      }
    }
  }
}

// Joins the chunks of one query row: one warp per row.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) attn_decode_scored_merge_kernel(const ScoredDecParams p,
                                                                       long long total) {
  grid_dependency_wait();  // the chunks' results are complete
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= total) return;
  const int lane = threadIdx.x & 31;
  const int R = p.G * p.n_q;
  const long long bk = w / R;
  const int gr = static_cast<int>(w - bk * R);
  const long long unit = bk * p.row_tiles + gr / ROWS;
  const float* part = p.part + (unit * p.splits * ROWS + gr % ROWS) * (D + 2);
  const long long step = static_cast<long long>(ROWS) * (D + 2);
  float mm = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) mm = fmaxf(mm, part[s * step + D]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
  const float mb = mm == -INFINITY ? 0.f : mm;
  constexpr int E = (D + 31) / 32;
  float a[E] = {}, ll = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float f = ex2(part[s * step + D] - mb);
    ll += f * part[s * step + D + 1];
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (lane + 32 * e < D) a[e] += f * part[s * step + lane + 32 * e];
  }
  const int b = static_cast<int>(bk / p.HK), hk = static_cast<int>(bk % p.HK);
  const int head = hk * p.G + gr / p.n_q, qi = gr % p.n_q;
  __nv_bfloat16* out = p.o + b * p.so.b + head * p.so.h + qi * p.so.n;
  const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane + 32 * e < D) out[lane + 32 * e] = __float2bfloat16_rn(a[e] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[(static_cast<long long>(b) * p.HK * p.G + head) * p.n_q + qi] =
        ll > 0.f ? (mm + __log2f(ll)) * kLn2 : -INFINITY;
}

template <int FMT, int D, int NR>
cudaError_t launch_scored_decode_rows(const ScoredDecParams& p, long long bk,
                                      const LaunchCtx& ctx) {
  const size_t smem = static_cast<size_t>(DW) * NR * 8 * (D + 2) * sizeof(float);
  auto* kernel = attn_decode_scored_kernel<FMT, D, NR>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const long long units = bk * p.row_tiles * p.splits;
  kernel<<<static_cast<unsigned>(units), DW * 32, smem, ctx.stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  const long long total = bk * p.G * p.n_q;
  return launch_dependent(attn_decode_scored_merge_kernel<D, NR * 8>,
                          dim3(static_cast<unsigned>((total + 3) / 4)), dim3(128), 0, ctx.stream, p,
                          total);
}

template <int FMT, int D>
cudaError_t launch_scored_decode_d(const ScoredDecParams& p, long long bk, int row_tile,
                                   const LaunchCtx& ctx) {
  switch (row_tile) {
    case 8: return launch_scored_decode_rows<FMT, D, 1>(p, bk, ctx);
    case 16: return launch_scored_decode_rows<FMT, D, 2>(p, bk, ctx);
    default: return launch_scored_decode_rows<FMT, D, 4>(p, bk, ctx);
  }
}

template <int FMT>
cudaError_t launch_scored_decode_fmt(const ScoredDecodeProblem& pb, const ScoredDecodePlan& plan,
                                     float* workspace, const LaunchCtx& ctx) {
  ScoredDecParams p;
  p.q = static_cast<const __nv_bfloat16*>(pb.q);
  p.k = static_cast<const uint8_t*>(pb.k_cache);
  p.v = static_cast<const uint8_t*>(pb.v_cache);
  p.k_scale = pb.k_scale;
  p.v_scale = pb.v_scale;
  p.o = static_cast<__nv_bfloat16*>(pb.o);
  p.lse = pb.lse;
  p.part = plan.splits > 1 ? workspace : nullptr;
  p.cache_lens = pb.cache_lens;
  p.slopes = pb.slopes;
  p.sq = pb.sq;
  p.sk = pb.sk;
  p.sv = pb.sv;
  p.so = pb.so;
  p.HK = pb.HK;
  p.G = pb.H / pb.HK;
  p.n_q = pb.n_q;
  p.L_max = pb.L_max;
  p.T_log2 = 0;
  while ((1 << p.T_log2) < pb.block_tokens) ++p.T_log2;
  p.num_blocks = (pb.L_max + pb.block_tokens - 1) / pb.block_tokens;
  p.window = pb.window;
  p.splits = plan.splits;
  p.row_tiles = plan.row_tiles;
  p.scale = pb.scale;
  p.softcap = pb.softcap;
  const long long bk = static_cast<long long>(pb.B) * pb.HK;
  switch (pb.d) {
    case 16: return launch_scored_decode_d<FMT, 16>(p, bk, plan.row_tile, ctx);
    case 32: return launch_scored_decode_d<FMT, 32>(p, bk, plan.row_tile, ctx);
    case 64: return launch_scored_decode_d<FMT, 64>(p, bk, plan.row_tile, ctx);
    case 128: return launch_scored_decode_d<FMT, 128>(p, bk, plan.row_tile, ctx);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace attn
