// attn_tree_few.cuh -- attention over a tree of drafted tokens, the roles of a CTA
// for key heads with few query rows (64 at most): keys are the rows of score tiles.
// Included by attn_tree.cuh.
//
//   S^T = K Q^T   128 keys are the rows, 16 or 32 query rows the columns;
//   O^T = V^T P^T the d values are the rows, the query rows the columns (d < 128:
//         the 128 rows of the product hold the d values several times).
// A thread has one key's scores of all rows in registers, and no exponential is
// taken for rows that are not there; a key's scale and mask are the thread's own.
// What a row would have to look for over all keys of a tile, its largest score, is
// not taken: P is 2^(x - m) for a maximum m that is kept until some score exceeds it
// by 2^8, which the stream's threads tell each other by a flag at a barrier; only
// then the rows' maxima are looked for.  A thread sums the P of its own keys for
// each row; they are added up at the end.  P^T goes to shared memory as the second
// product's operand.
//
// The two streams take every second tile with the same rows, and their results are
// joined; with more than 32 rows they take 32 each of every tile.
#pragma once

namespace attn {
namespace {

template <class C>
__device__ __forceinline__ bool mma_few(const TreeParams& p, TreeSmem<C>& sm, uint32_t tmem, int s,
                                        int lane) {
  constexpr int D = C::D, BN = C::BN, KSTAGES = C::KSTAGES, VSTAGES = C::VSTAGES;
  const volatile int* abort = &sm.abort;
  bool ok = true;
  constexpr uint32_t KV16 = C::KV_TILE >> 4;
  const uint64_t dk = tree_sdesc(smem_u32(sm.k[0]), 16, 8 * C::RB, C::SWZ);
  // V^T, the values of a row side by side: with d < 128 all blocks of rows are the same one
  const uint64_t dv = tree_sdesc(smem_u32(sm.v[0]), D == 128 ? C::KV_BLOCK : 0, 8 * C::RB, C::SWZ);
  // P^T: a key's rows in 64 bytes, swizzled so
  const uint64_t dp = tree_sdesc(smem_u32(sm.prob[s]), 0, 8 * 64, 4u);
  auto qstep = [](int kk) {
    return static_cast<uint32_t>((kk / C::KPB) * (C::Q_BLOCK >> 4) + (kk % C::KPB) * 2);
  };
  auto kstep = [](int kk) {
    return static_cast<uint32_t>((kk / C::KPB) * (C::KV_BLOCK >> 4) + (kk % C::KPB) * 2);
  };
  const uint32_t t_o = tmem + C::col_o(s);
  const bool leader = elect_one();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.limit_ns, abort));
    return ok;
  };
  uint32_t u = 0;  // score products issued
  // the last one still owes its PV product, see mma_many
  bool pending = false, pfirst = false, plast = false;
  uint32_t pg = 0, pidesc = 0;
  int pslot = 0, plo = 0, phi = 0, pnode = -1;
  auto flush_pv = [&]() {
    if (!pending) return;
    const uint32_t w = u - 1;
    if (!wait(&sm.v_full[pg % VSTAGES], (pg / VSTAGES) & 1) ||
        !wait(&sm.p_full[s][w & 1], (w >> 1) & 1))
      return;
    clear_rows<C>(p, sm, sm.v[pg % VSTAGES], 0, BN, plo, phi, pnode, pslot, lane);
    tc_fence_after();
    const uint64_t a = dv + (pg % VSTAGES) * KV16;
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        mma_ss(t_o, a + C::RB * kk, dp + 64 * kk, pidesc, (!pfirst || kk > 0) ? 1u : 0u);
      tc_commit(smem_u32(&sm.pv_done[s][w & 1]));
      tc_commit(smem_u32(&sm.v_empty[pg % VSTAGES]));
      if (plast) mbar_arrive(smem_u32(&sm.item_empty[pslot]));
    }
    __syncwarp();
    pending = false;
  };
  auto next_wait = [&](uint64_t* bar, uint32_t parity) {
    if (pending && __shfl_sync(0xffffffffu, mbar_test(smem_u32(bar), parity) ? 1 : 0, 0) == 0)
      flush_pv();
    return wait(bar, parity);
  };
  uint32_t g0 = 0;
  for (uint32_t items = 0; ok; ++items) {
    const int slot = items & 1;
    if (!next_wait(&sm.item_full[slot], (items >> 1) & 1)) break;
    const TreeItem it = sm.item[slot];
    if (it.more == 0) break;
    const bool both = it.split == 0;
    const int cols = it.rows > 16 ? 32 : 16;
    const uint32_t idesc_s = idesc_bf16_f32(BM, cols, false, false);
    const uint32_t idesc_o = idesc_bf16_f32(BM, cols, true, true);
    const uint64_t dq = tree_sdesc(smem_u32(sm.q[items % C::QSLOTS][0]) + (both ? 32 * s * C::RB : 0),
                                   16, 8 * C::RB, C::SWZ);
    bool first = true;
    for (int j = 0; j < it.n && ok; ++j) {
      const uint32_t g = g0 + j;
      if (!next_wait(&sm.k_full[g % KSTAGES], (g / KSTAGES) & 1)) break;
      if (!both && (j & 1) != s) {
        if (leader) mbar_arrive(smem_u32(&sm.k_empty[g % KSTAGES]));
        if (next_wait(&sm.v_full[g % VSTAGES], (g / VSTAGES) & 1) && leader)
          mbar_arrive(smem_u32(&sm.v_empty[g % VSTAGES]));
        continue;
      }
      // (S(u) goes where S(u - 2) was, which was in registers before P(u - 2) came)
      tc_fence_after();
      const uint64_t a = dk + (g % KSTAGES) * KV16;
      const uint32_t t_s = tmem + C::col_s(s, u & 1);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(t_s, a + kstep(kk), dq + qstep(kk), idesc_s, kk > 0 ? 1u : 0u);
        tc_commit(smem_u32(&sm.s_full[s][u & 1]));
        tc_commit(smem_u32(&sm.k_empty[g % KSTAGES]));
      }
      __syncwarp();
      flush_pv();
      if (!ok) break;
      ++u;
      pending = true;
      pfirst = first;
      first = false;
      plast = false;
      pg = g;
      pidesc = idesc_o;
      pslot = slot;
      const int t = it.t0 + j, base = it.base0 + t * BN;
      plo = it.key0 - base;
      phi = it.L - base;
      pnode = t < it.ctx ? -1 : (t - it.ctx) * BN;
    }
    if (!ok) break;
    if (leader) tc_commit(smem_u32(&sm.q_empty[items % C::QSLOTS]));
    if (!first && pending) {
      plast = true;
    } else {
      // nothing of this item is owed; what one before owes does not wait for more
      if (leader) mbar_arrive(smem_u32(&sm.item_empty[slot]));
      __syncwarp();
      flush_pv();
    }
    g0 += it.n;
  }
  flush_pv();
  return ok;
}

// The largest of a warp's values (NaN left out).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <class C, bool CHANGED>
__device__ __forceinline__ bool softmax_few(const TreeParams& p, TreeSmem<C>& sm, uint32_t tmem,
                                            int s, int quarter, int lane) {
  constexpr int D = C::D, BN = C::BN;
  constexpr bool Q8 = C::Q8;
  const volatile int* abort = &sm.abort;
  bool ok = true;
  FewTables& few = sm.few[s];
  const int at = quarter * 32 + lane;  // key of the tile; tensor-memory lane
  const uint32_t lanes_at = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t tO = lanes_at + C::col_o(s);
  uint8_t* prob = sm.prob[s] + at * 64;
  const int turn = (at >> 1) & 3;  // of the 16-byte chunks of that row
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.limit_ns, abort));
    return ok;
  };
  uint32_t meets = 0, joins = 0, votes = 0;
  auto meet = [&]() {
    mbar_arrive(smem_u32(&few.meet));
    return wait(&few.meet, meets++ & 1);
  };
  auto join = [&]() {
    mbar_arrive(smem_u32(&sm.join_sync));
    return wait(&sm.join_sync, joins++ & 1);
  };
  if (at < 4) few.flag[at] = 0;
  if (at < 32) few.zero[at] = 0.f;
  uint32_t u = 0;  // tiles of this stream

  for (uint32_t items = 0; ok; ++items) {
    const int slot = items & 1;
    if (!wait(&sm.item_full[slot], (items >> 1) & 1)) break;
    const TreeItem it = sm.item[slot];
    if (it.more == 0) break;
    const bool both = it.split == 0;
    const int row_at = both ? 32 * s : 0;  // this stream's rows
    const int rows = both ? min(it.rows - row_at, 32) : it.rows;
    const bool wide = it.rows > 16;        // 32 columns
    if (at < 32) {
      const int row = it.row0 + row_at + min(at, rows - 1);
      const int g = row / p.n, node = row - g * p.n;
      const int depth = sm.depth[slot][node];
      few.node[at] = node;
      few.depth[at] = depth;
      few.first_key[at] = p.window >= 0 ? it.L + max(depth, 0) - p.window : 0;
      few.m[at] = -INFINITY;
      few.neg[at] = INFINITY;
      few.slope[at] =
          CHANGED && p.slopes ? kLog2e * __ldg(p.slopes + it.hk * p.G + g) : 0.f;
    }
    if (!meet()) break;
    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.f;
    bool first = true;

    auto tile = [&](auto nc, int t, float ks, float vs) {
      constexpr int N = decltype(nc)::value;  // columns
      const bool tree = t >= it.ctx;
      const int base = tree ? (t - it.ctx) * BN : it.base0 + t * BN;
      const uint32_t tS = lanes_at + C::col_s(s, u & 1);
      const int key = base + at;
      const bool here = tree ? key < p.n : key < it.L && key >= it.key0;
      // (a node's window begins at most n positions behind the root's)
      const bool edge = tree || base + BN > it.L || (p.window >= 0 && base < it.key0 + p.n);
      // position of the key for the bias: in the tile, or its depth
      [[maybe_unused]] const float place = CHANGED && p.slopes ? (tree ? static_cast<float>(sm.depth[slot][min(key, p.n - 1)])
                                                      : static_cast<float>(at))
                                              : 0.f;
      uint32_t y[N];  // the scores
      // scores less each row's maximum (neg) or as they are (zero), in log2 units
      auto scores = [&](const float* less) {
        if constexpr (N == 32) {
          tmem_ld32(tS, y);
          tmem_ld_wait(y);
        } else {
          tmem_ld16(tS, y);
        }
        const float* offset = less;
        if (CHANGED && p.slopes) {
          const float away = tree ? -static_cast<float>(max(few.depth[lane], 0))
                                  : static_cast<float>(base - it.L - max(few.depth[lane], 0));
          __syncwarp();
          few.offset[quarter][lane] = fmaf(few.slope[lane], away, less[lane]);
          __syncwarp();
          offset = few.offset[quarter];
        }
        if constexpr (CHANGED) {
          if (p.capped) {
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              if constexpr (Q8) y[i] = __float_as_uint(__uint_as_float(y[i]) * ks);
              big = fmaxf(big, fabsf(__uint_as_float(y[i])));
            }
            if (__all_sync(0xffffffffu, big <= p.cap.small)) {
#pragma unroll
              for (int i = 0; i < N; i += 2) {
                const float x0 = __uint_as_float(y[i]), x1 = __uint_as_float(y[i + 1]);
                float z0, z1, w0, w1;
                fma2(z0, z1, x0, x1, x0, x1, 0.f, 0.f);
                fma2(w0, w1, z0, z1, p.cap.poly[2], p.cap.poly[2], p.cap.poly[1], p.cap.poly[1]);
                fma2(w0, w1, z0, z1, w0, w1, p.cap.poly[0], p.cap.poly[0]);
                fma2(w0, w1, x0, x1, w0, w1, 0.f, 0.f);
                y[i] = __float_as_uint(w0);
                y[i + 1] = __float_as_uint(w1);
              }
            } else {
              // cap * tanh(y) = cap - 2 cap / (1 + 2^(2 y log2(e))), in log2 units
#pragma unroll
              for (int i = 0; i < N; ++i) {
                const float x0 = __uint_as_float(y[i]);
                float w = fmaf(-2.f * p.cap_log2, rcp(1.f + ex2(x0 * p.cap_in)), p.cap_log2);
                if (p.wide && fabsf(x0) <= p.cap.small) {
                  const float z = x0 * x0;
                  w = x0 * fmaf(z, fmaf(z, p.cap.poly[2], p.cap.poly[1]), p.cap.poly[0]);
                }
                y[i] = __float_as_uint(w);
              }
            }
          }
        }
        const float f = CHANGED && p.capped ? 1.f : ks * p.scale_log2;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 o = *reinterpret_cast<const float4*>(offset + i);
          float z[4];
          fma2(z[0], z[1], __uint_as_float(y[i]), __uint_as_float(y[i + 1]), f, f, o.x, o.y);
          fma2(z[2], z[3], __uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]), f, f, o.z, o.w);
          if constexpr (CHANGED) {
            if (p.slopes) {
              const float4 a = *reinterpret_cast<const float4*>(few.slope + i);
              fma2(z[0], z[1], a.x, a.y, place, place, z[0], z[1]);
              fma2(z[2], z[3], a.z, a.w, place, place, z[2], z[3]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i + e] = __float_as_uint(z[e]);
        }
        if (edge) {
          if (tree) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const uint32_t line = sm.line[slot][few.node[i]][quarter];
              if (!((line >> lane) & 1u)) y[i] = __float_as_uint(-INFINITY);
            }
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (!here || key < few.first_key[i]) y[i] = __float_as_uint(-INFINITY);
          }
        }
      };
      // 0: against the kept maxima; 1: as they are, for new ones; 2: against those
#pragma unroll 1
      for (int pass = first ? 1 : 0;; ++pass) {
        scores(pass == 1 ? few.zero : few.neg);
        if (pass == 2) break;
        if (pass == 0) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < N; i += 2)
            top = max3(top, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
          int* flag = &few.flag[votes & 3];
          if (top > kRescale) *flag = 1;
          if (!meet()) return;
          const bool settled = *reinterpret_cast<volatile int*>(flag) == 0;
          if (at == 0) few.flag[(votes + 2) & 3] = 0;
          ++votes;
          if (settled) break;
          continue;
        }
        float mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float top = warp_max(__uint_as_float(y[i]));
          if (lane == i) mine = top;
        }
        few.part[quarter][lane] = mine;
        if (!meet()) return;
        if (quarter == 0) {
          const float top = fmaxf(fmaxf(few.part[0][lane], few.part[1][lane]),
                                  fmaxf(few.part[2][lane], few.part[3][lane]));
          const float m = few.m[lane];
          float alpha = 1.f;
          if (top > m + kRescale) {
            alpha = ex2(m - top);  // 0 when m = -inf
            few.m[lane] = top;
            few.neg[lane] = -top;
          }
          few.alpha[lane] = alpha;
        }
        if (!meet()) return;
        if (!first) {
          // O is rescaled once the last product is done
          if (!wait(&sm.pv_done[s][(u - 1) & 1], ((u - 1) >> 1) & 1)) return;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < N; c += 16) {
            uint32_t o[16];
            tmem_ld16(tO + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * few.alpha[c + i]);
            tmem_st16(tO + c, o);
          }
          tmem_st_wait();
#pragma unroll
          for (int i = 0; i < N; ++i) l[i] *= few.alpha[i];
        }
      }
      uint32_t pk[N / 2];
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float a = ex2(__uint_as_float(y[i])), b = ex2(__uint_as_float(y[i + 1]));
        add2(l[i], l[i + 1], l[i], l[i + 1], a, b);
        if constexpr (Q8) fma2(a, b, a, b, vs, vs, 0.f, 0.f);
        pk[i / 2] = pack_bf16x2(a, b);
      }
      // P overwrites the last tile's once that product is done
      if (u > 0 && !wait(&sm.pv_done[s][(u - 1) & 1], ((u - 1) >> 1) & 1)) return;
#pragma unroll
      for (int c = 0; c < N / 8; ++c)
        *reinterpret_cast<uint4*>(prob + ((c ^ turn) << 4)) =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      fence_proxy_async_smem();
    };

    for (int j = both ? 0 : s; j < it.n && ok; j += both ? 1 : 2) {
      const int t = it.t0 + j;
      float ks = 1.f, vs = 1.f;
      if constexpr (Q8) {
        const int key = it.base0 + t * BN + at;
        if (t < it.ctx && key < it.L && key >= it.key0) {
          const long long blk = (static_cast<long long>(it.b) * p.HK + it.hk) * p.num_blocks +
                                (key >> p.T_log2);
          ks = __ldg(p.k_scale + blk);
          vs = __ldg(p.v_scale + blk);
        }
      }
      if (!wait(&sm.s_full[s][u & 1], (u >> 1) & 1)) break;
      tc_fence_after();
      if (wide)
        tile(std::integral_constant<int, 32>(), t, ks, vs);
      else
        tile(std::integral_constant<int, 16>(), t, ks, vs);
      if (!ok) break;
      first = false;
      tc_fence_before();
      mbar_arrive(smem_u32(&sm.p_full[s][u & 1]));
      ++u;
    }
    if (!ok) break;

    // ------------------------------------------------------------ the run's result
    if (!first) {
      if (!wait(&sm.pv_done[s][(u - 1) & 1], ((u - 1) >> 1) & 1)) break;
      tc_fence_after();
    }
    // each row's sum: over a warp's keys (lane i is left with row i's), then the warps'
#pragma unroll
    for (int w = 16; w > 0; w >>= 1)
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const bool up = lane & w;
        const float give = up ? l[i] : l[i + w], keep = up ? l[i + w] : l[i];
        l[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
      }
    few.part[quarter][lane] = l[0];
    tc_fence_before();
    if (!meet()) break;
    if (at < 32) {
      const bool alive = at < rows && few.depth[at] >= 0;
      few.sum[at] =
          alive ? (few.part[0][at] + few.part[1][at]) + (few.part[2][at] + few.part[3][at]) : 0.f;
    }
    if (!(both ? meet() : join())) break;
    // what a stream's accumulators of each row are worth in the result
    float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + it.slot) * p.block_rows *
                               (D + kPartTail);
    if (at < 32) {
      const float m0 = few.m[at], s0 = few.sum[at];
      const float m1 = both ? -INFINITY : sm.few[s ^ 1].m[at], s1 = both ? 0.f : sm.few[s ^ 1].sum[at];
      const float most = fmaxf(s0 > 0.f ? m0 : -INFINITY, s1 > 0.f ? m1 : -INFINITY);
      const float w0 = s0 > 0.f ? ex2(m0 - most) : 0.f, w1 = s1 > 0.f ? ex2(m1 - most) : 0.f;
      const float sum = fmaf(w0, s0, w1 * s1);
      few.alpha[at] = it.whole ? (sum > 0.f ? w0 / sum : 0.f) : w0;
      const int r = row_at + at, row = it.row0 + min(r, it.rows - 1), g = row / p.n;
      const int node = row - g * p.n, head = it.hk * p.G + g;
      few.out[at] = it.whole ? it.b * p.so.b + head * p.so.h + node * p.so.n
                             : static_cast<long long>(r) * (D + kPartTail);
      if (at < rows && (both || s == 0)) {
        if (!it.whole)
          *reinterpret_cast<float2*>(part + few.out[at] + D) = make_float2(most, sum);
        else if (p.lse != nullptr)
          p.lse[(static_cast<size_t>(it.b) * p.H + head) * p.n + node] =
              sum > 0.f ? (most + __log2f(sum)) * kLn2 : -INFINITY;
      }
    }
    if (!(both ? meet() : join())) break;
    tc_fence_after();
    // every lane has a value of d, of all columns; eight of them at a time go to the
    // warps that have the same value in either stream in turn
    {
      constexpr int COPIES = D == 128 ? 1 : (D == 64 ? 2 : 4);
      const int c = at % D, copy = quarter * COPIES / 4;
      const bool other = !both && it.n > (s ^ 1);  // whether the other stream had a tile
      const FewTables& far = sm.few[s ^ 1];
#pragma unroll 1
      for (int k = 0; k < (rows + 7) / 8; ++k) {
        if (!both && (k & 1) != s) continue;
        if ((both ? k : k >> 1) % COPIES != copy) continue;
        uint32_t mine[8], theirs[8];
        if (!first) tmem_ld8(tO + 8 * k, mine);
        if (other) tmem_ld8(lanes_at + C::col_o(s ^ 1) + 8 * k, theirs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 8 * k + i;
          // (columns behind the rows hold anything)
          const float w0 = first ? 0.f : few.alpha[r], w1 = other ? far.alpha[r] : 0.f;
          float o = 0.f;
          if (w0 > 0.f) o = w0 * __uint_as_float(mine[i]);
          if (w1 > 0.f) o = fmaf(w1, __uint_as_float(theirs[i]), o);
          if (r < rows && (D >= 32 || lane < D)) {
            if (it.whole)
              p.o[few.out[r] + c] = __float2bfloat16_rn(o);
            else
              part[few.out[r] + c] = o;
          }
        }
        __syncwarp();
      }
    }
    tc_fence_before();
    // the streams' tables and accumulators stay until both have read them
    if (!both && !join()) break;
    if (both && !meet()) break;
    mbar_arrive(smem_u32(&sm.item_empty[slot]));
  }
  return ok;
}

}  // namespace
}  // namespace attn
