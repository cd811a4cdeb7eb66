// attn_tree.cu -- attention of a tree of drafted tokens over a key/value cache.
//
// Node i of sequence b stands at position p_i = L + depth_i behind the L tokens
// of its cache and sees them and its own ancestors (itself among them):
//   x_j = cap * tanh(scale * q_i . k_j / cap) - slope_h * (p_i - p_j)
//   O_i = sum_j softmax_j(x) v_j,   LSE_i = ln sum_j exp(x_j)
// over the cached keys j (p_j = j >= p_i - window) from the cache and the
// ancestors a (p_a = L + depth_a >= p_i - window) from the tree's own keys.
//
// One warp per query row, 32 keys at a time: lane j takes the score of key j,
// then the lanes share the d values of the output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_internal.cuh"

namespace attn {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.4426950408889634f;

template <int FMT>
__device__ __forceinline__ float cache_value(const void* row, int c) {
  if (FMT == 0) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[c]);
  if (FMT == 1)
    return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(row)[c]);
  return static_cast<float>(static_cast<const int8_t*>(row)[c]);
}

template <int FMT, int D>
__global__ void __launch_bounds__(128) attn_tree_simple_kernel(const TreeDecodeProblem pb) {
  const long long row = blockIdx.x * 4LL + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(pb.B) * pb.H * pb.n) return;
  const int lane = threadIdx.x & 31;
  const int i = row % pb.n, hh = row / pb.n % pb.H, b = row / pb.n / pb.H;
  const int hk = hh / (pb.H / pb.HK);
  const int* parents = pb.parents + static_cast<long long>(b) * pb.n;
  // ancestors, and whether they lead to a root
  uint32_t line[4] = {};
  int depth = -1, at = i;
  while (at >= 0) {
    line[at >> 5] |= 1u << (at & 31);
    ++depth;
    const int up = parents[at];
    at = up < -1 || up >= at ? -2 : up;
  }
  const bool node = at == -1;
  const int L = pb.cache_lens ? min(max(pb.cache_lens[b], 0), pb.L_max) : pb.L_max;
  const int first = pb.window >= 0 ? max(L + depth - pb.window, 0) : 0;
  const float slope = pb.slopes ? pb.slopes[hh] : 0.f;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(pb.q) + b * pb.sq.b + hh * pb.sq.h +
                           i * pb.sq.n;
  constexpr int ES = FMT == 0 ? 2 : 1;
  constexpr int OC = D < 32 ? 1 : D / 32;
  float m = -INFINITY, l = 0.f, o[OC] = {};
  const int blocks = (pb.L_max + pb.block_tokens - 1) / pb.block_tokens;
  const float* ks = pb.k_scale + (FMT ? (static_cast<long long>(b) * pb.HK + hk) * blocks : 0);
  const float* vs = pb.v_scale + (FMT ? (static_cast<long long>(b) * pb.HK + hk) * blocks : 0);
  auto row_at = [&](const void* base, const RowStrides& s, int j, int es) {
    return static_cast<const uint8_t*>(base) + (b * s.b + hk * s.h + j * s.n) * es;
  };
  for (int part = 0; part < 2 && node; ++part) {
    const int end = part == 0 ? L : pb.n;
    for (int base = part == 0 ? first & ~31 : 0; base < end; base += 32) {
      const int j = base + lane;
      bool see = j < end;
      int back = 0;
      if (part == 0) {
        back = L + depth - j;
        see = see && j >= first;
      } else if (see) {
        see = (line[j >> 5] >> (j & 31)) & 1u;
        for (int a = i; a > j && see; a = parents[a]) ++back;
        see = see && (pb.window < 0 || back <= pb.window);
      }
      float x = -INFINITY;
      if (see) {
        float s = 0.f;
        if (part == 0) {
          const uint8_t* k = row_at(pb.k_cache, pb.sk, j, ES);
          for (int c = 0; c < D; ++c) s = fmaf(__bfloat162float(q[c]), cache_value<FMT>(k, c), s);
          if (FMT) s *= ks[j / pb.block_tokens];
        } else {
          const uint8_t* k = row_at(pb.k_tree, pb.skt, j, 2);
          for (int c = 0; c < D; ++c) s = fmaf(__bfloat162float(q[c]), cache_value<0>(k, c), s);
        }
        x = s * pb.scale;
        if (pb.softcap > 0.f) x = pb.softcap * tanhf(x / pb.softcap);
        x = (x - slope * back) * kLog2e;
      }
      float top = x;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      if (top == -INFINITY) continue;
      top = fmaxf(m, top);
      const float alpha = exp2f(m - top);
      const float p = exp2f(x - top);
      m = top;
      l = l * alpha + p;
#pragma unroll
      for (int c = 0; c < OC; ++c) o[c] *= alpha;
      const unsigned seen = __ballot_sync(0xffffffffu, see);
      for (int e = 0; e < 32; ++e) {
        float w = __shfl_sync(0xffffffffu, p, e);
        if (!((seen >> e) & 1u)) continue;
        const uint8_t* v = part == 0 ? row_at(pb.v_cache, pb.sv, base + e, ES)
                                     : row_at(pb.v_tree, pb.svt, base + e, 2);
        if (part == 0 && FMT) w *= vs[(base + e) / pb.block_tokens];
#pragma unroll
        for (int c = 0; c < OC; ++c)
          if (c * 32 + lane < D)
            o[c] = fmaf(w, part == 0 ? cache_value<FMT>(v, c * 32 + lane)
                                     : cache_value<0>(v, c * 32 + lane), o[c]);
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(pb.o) + b * pb.so.b + hh * pb.so.h + i * pb.so.n;
#pragma unroll
  for (int c = 0; c < OC; ++c)
    if (c * 32 + lane < D) out[c * 32 + lane] = __float2bfloat16(l > 0.f ? o[c] / l : 0.f);
  if (lane == 0 && pb.lse) pb.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int FMT>
cudaError_t launch_fmt(const TreeDecodeProblem& pb, const LaunchCtx& ctx) {
  const long long rows = static_cast<long long>(pb.B) * pb.H * pb.n;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  switch (pb.d) {
    case 16: attn_tree_simple_kernel<FMT, 16><<<grid, 128, 0, ctx.stream>>>(pb); break;
    case 32: attn_tree_simple_kernel<FMT, 32><<<grid, 128, 0, ctx.stream>>>(pb); break;
    case 64: attn_tree_simple_kernel<FMT, 64><<<grid, 128, 0, ctx.stream>>>(pb); break;
    case 128: attn_tree_simple_kernel<FMT, 128><<<grid, 128, 0, ctx.stream>>>(pb); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(const TreeDecodeProblem& pb, const LaunchCtx& ctx) {
  switch (pb.format) {
    case 0: return launch_fmt<0>(pb, ctx);
    case 1: return launch_fmt<1>(pb, ctx);
    default: return launch_fmt<2>(pb, ctx);
  }
}

}  // namespace attn
