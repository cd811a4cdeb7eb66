// attn_cache.cu -- writing new keys and values into a cache held in 8 bits,
// with one float32 scale for each block of T tokens and head.
//
// A cache row holds codes c with  value = scale[b, h, token / T] * c,  c an
// e4m3 number (|c| <= 448) or an int8 one (|c| <= 127).  For the block that a
// call's new tokens x of one (b, h) fall into, with `held` = the scale of the
// tokens the block holds already (0 when it holds none):
//
//   scale = max(held, max |x| / c_max, 2^-100),   c = round(x * (1 / scale)),
//   held codes  c <- round(c * (held * (1 / scale)))   when the scale grew,
//
// round = to the nearest code, ties to even.  The least scale keeps the
// reciprocal finite.  A scale that never shrinks while its block fills means
// a held code is rounded again only when a larger token arrives.  The codes
// are products with the correctly rounded reciprocal instead of quotients:
// one multiplication each, and the quotient differs from them by less than
// 2^-23 relative, which matters only next to a border between two codes.
//
// Bound by memory: each new element is read once (2 bytes) and written once
// (1 byte).  A block's maximum is needed before its first code, so a block's
// new tokens wait in registers between the two, up to eight 16-byte loads of a
// thread in flight; the threads that a block gets follow from the elements that
// it can get (launch_append).  Measured, 32 sequences of up to 2048 new tokens,
// 16 heads of d = 64, to e4m3: 46 us with blocks of 128, 64 or 32 tokens (6.6
// TB/s, the rate of a plain copy), 50 us with blocks of 16; to int8 48 us.  Twice
// the threads with half the loads each: 54, 50 and 79 us.  One token for 256
// sequences, 8 heads: 3 us, the launch.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "attn_internal.cuh"

namespace attn {
namespace {

struct CacheParams {
  const __nv_bfloat16* src[2];  // new keys, new values
  uint8_t* dst[2];              // their caches
  float* scale[2];
  const int* lens;      // tokens held per sequence, or null (none)
  const int* new_lens;  // new tokens per sequence, or null (n_new each)
  RowStrides ss[2], sd[2];
  int H, n_new, L_max, T, num_blocks, touched;
};

constexpr float kScaleMin = 0x1p-100f;

template <bool E4M3>
__device__ __forceinline__ float code_max() {
  return E4M3 ? 448.f : 127.f;
}

// Four values (already over their scale) to four codes, nearest, ties to even.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (E4M3) {
    // the conversion rounds to nearest even and saturates at 448
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  // (a magnitude over 127 cannot come of a product with a block's reciprocal; -128
  // times a ratio can, from a cache that something else wrote)
  auto one = [](float x) { return max(-127, __float2int_rn(x)); };
  uint32_t w;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(w) : "r"(one(d)), "r"(one(c)));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w) : "r"(one(b)), "r"(one(a)), "r"(w));
  return w;
}

template <bool E4M3>
__device__ __forceinline__ float decode1(uint32_t byte) {
  if (E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    return __half2float(__half(h));
  }
  return static_cast<float>(static_cast<int8_t>(byte));
}

// THREADS threads work on one block of one (b, head) and of keys or values;
// CHUNKS chunks of 8 elements each wait in a thread's registers.  WARP: one
// warp per block, eight blocks to a CTA and no barrier; else one CTA per block.
template <bool E4M3, bool WARP, int THREADS, int CHUNKS>
__global__ void __launch_bounds__(WARP ? 256 : THREADS)
    attn_cache_append_kernel(const CacheParams p, unsigned units, int cpr_log2) {
  __shared__ float red[WARP ? 1 : THREADS / 32];
  const unsigned unit = WARP ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && unit >= units) return;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  // unit = ((b * H + head) * touched + block) * 2 + (keys or values)
  const int kv = unit & 1u;
  const unsigned rest = unit >> 1;
  const unsigned bh = rest / static_cast<unsigned>(p.touched);
  const int b = bh / static_cast<unsigned>(p.H), hh = bh - static_cast<unsigned>(b) * p.H;
  const int len = p.lens ? min(max(__ldg(p.lens + b), 0), p.L_max) : 0;
  const int more = p.new_lens ? min(max(__ldg(p.new_lens + b), 0), p.n_new) : p.n_new;
  const int end = len + min(more, p.L_max - len);  // tokens that do not fit are dropped
  const int blk = len / p.T + static_cast<int>(rest - bh * p.touched);
  if (blk >= p.num_blocks) return;
  // (L_max is 2^30 at most, so that nothing here leaves int)
  const int row0 = blk * p.T;
  const int first = max(len, row0), last = min(end, row0 + p.T);  // new rows of this block
  if (first >= last) return;  // the same for every thread of the unit

  const __nv_bfloat16* src = p.src[kv] + b * p.ss[kv].b + hh * p.ss[kv].h +
                             static_cast<long long>(first - len) * p.ss[kv].n;
  uint8_t* dst = p.dst[kv] + b * p.sd[kv].b + hh * p.sd[kv].h;
  const int chunks = (last - first) << cpr_log2;  // 8-element chunks, a row's side by side

  // a thread's chunks stand in one column, `rows` rows apart
  const int rows = THREADS >> cpr_log2, row = tid >> cpr_log2;
  const int col = (tid - (row << cpr_log2)) * 8;
  uint4 w[CHUNKS];
  {
    const __nv_bfloat16* at = src + row * p.ss[kv].n + col;
    const long long step = rows * p.ss[kv].n;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i, at += step)
      w[i] = tid + i * THREADS < chunks ? __ldg(reinterpret_cast<const uint4*>(at))
                                        : make_uint4(0u, 0u, 0u, 0u);
  }
  float* scale_at = p.scale[kv] + static_cast<long long>(bh) * p.num_blocks + blk;
  const float held = first > row0 ? *scale_at : 0.f;
  // (the larger of two bf16 magnitudes, exactly; a NaN gives way to a number)
  __nv_bfloat162 most = __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&w[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) most = __hmax2(most, __habs2(x[e]));
  }
  float top = fmaxf(__low2float(most), __high2float(most));
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  if (!WARP) {
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) top = fmaxf(top, red[i]);
  } else {
    __syncwarp();  // every lane has read the held scale before it is replaced
  }
  const float scale = fmaxf(fmaxf(held, __fdiv_rn(top, code_max<E4M3>())), kScaleMin);
  const float inv = __frcp_rn(scale);
  {
    uint8_t* at = dst + (first + row) * p.sd[kv].n + col;
    const long long step = rows * p.sd[kv].n;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i, at += step) {
      if (tid + i * THREADS >= chunks) break;
      const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&w[i]);
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = __bfloat1622float2(x[e]);
        f[2 * e] = y.x * inv;
        f[2 * e + 1] = y.y * inv;
      }
      *reinterpret_cast<uint2*>(at) = make_uint2(encode4<E4M3>(f[0], f[1], f[2], f[3]),
                                                 encode4<E4M3>(f[4], f[5], f[6], f[7]));
    }
  }
  if (scale != held) {
    if (tid == 0) *scale_at = scale;
    // the rows the block held are rescaled; rows behind the new ones stay
    const float ratio = held * inv;
    const int old = (first - row0) << cpr_log2;
    for (int c = tid; c < old; c += THREADS) {
      const int r = c >> cpr_log2;
      uint2* at = reinterpret_cast<uint2*>(dst + static_cast<long long>(row0 + r) * p.sd[kv].n) +
                  (c - (r << cpr_log2));
      uint2 v = *at;
      uint32_t* words = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        words[e] = encode4<E4M3>(decode1<E4M3>(words[e] & 0xffu) * ratio,
                                 decode1<E4M3>((words[e] >> 8) & 0xffu) * ratio,
                                 decode1<E4M3>((words[e] >> 16) & 0xffu) * ratio,
                                 decode1<E4M3>(words[e] >> 24) * ratio);
      *at = v;
    }
  }
}

template <bool E4M3>
cudaError_t launch_append(const CacheParams& p, unsigned units, int cpr_log2, cudaStream_t stream) {
  // most 8-element chunks of new tokens that one block can get
  const int most = (p.n_new < p.T ? p.n_new : p.T) << cpr_log2;
  if (most <= 4 * 32) {
    attn_cache_append_kernel<E4M3, true, 32, 4>
        <<<(units + 7) / 8, 256, 0, stream>>>(p, units, cpr_log2);
  } else if (most <= 8 * 32) {
    attn_cache_append_kernel<E4M3, true, 32, 8>
        <<<(units + 7) / 8, 256, 0, stream>>>(p, units, cpr_log2);
  } else if (most <= 8 * 64) {
    attn_cache_append_kernel<E4M3, false, 64, 8><<<units, 64, 0, stream>>>(p, units, cpr_log2);
  } else if (most <= 8 * 128) {
    attn_cache_append_kernel<E4M3, false, 128, 8><<<units, 128, 0, stream>>>(p, units, cpr_log2);
  } else {
    attn_cache_append_kernel<E4M3, false, 256, 8><<<units, 256, 0, stream>>>(p, units, cpr_log2);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendProblem& pb, const LaunchCtx& ctx) {
  CacheParams p;
  p.src[0] = static_cast<const __nv_bfloat16*>(pb.k_new);
  p.src[1] = static_cast<const __nv_bfloat16*>(pb.v_new);
  p.dst[0] = static_cast<uint8_t*>(pb.k_cache);
  p.dst[1] = static_cast<uint8_t*>(pb.v_cache);
  p.scale[0] = pb.k_scale;
  p.scale[1] = pb.v_scale;
  p.lens = pb.cache_lens;
  p.new_lens = pb.new_lens;
  p.ss[0] = pb.skn;
  p.ss[1] = pb.svn;
  p.sd[0] = pb.skc;
  p.sd[1] = pb.svc;
  p.H = pb.H;
  p.n_new = pb.n_new;
  p.L_max = pb.L_max;
  p.T = pb.block_tokens;
  p.num_blocks = (pb.L_max + pb.block_tokens - 1) / pb.block_tokens;
  p.touched = cache_blocks_touched(pb.n_new, pb.L_max, pb.block_tokens);
  const unsigned units = 2u * pb.B * pb.H * p.touched;  // the caller keeps it below 2^31
  int cpr_log2 = 1;  // 8-element chunks of a row
  while ((8 << cpr_log2) < pb.d) ++cpr_log2;
  return pb.e4m3 ? launch_append<true>(p, units, cpr_log2, ctx.stream)
                 : launch_append<false>(p, units, cpr_log2, ctx.stream);
}

int cache_blocks_touched(int n_new, int L_max, int block_tokens) {
  // n_new tokens that start on a block's last row reach this many blocks
  const long long n = (static_cast<long long>(n_new) + block_tokens - 2) / block_tokens + 1;
  const long long all = (static_cast<long long>(L_max) + block_tokens - 1) / block_tokens;
  return static_cast<int>(n < all ? n : all);
}

}  // namespace attn
