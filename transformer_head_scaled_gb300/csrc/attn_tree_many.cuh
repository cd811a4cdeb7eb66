// attn_tree_many.cuh -- attention over a tree of drafted tokens, the roles of a CTA
// for key heads with many query rows: rows are the rows of score tiles.  Included
// by attn_tree.cuh.
#pragma once

namespace attn {
namespace {

// A stream runs through its own parts u = 0, 1, ... of 64 keys (all items) in the
// order S(0), S(1), PV(0), S(2), PV(1), ...: S(u) goes to buffer u % 2 once PV(u - 2)
// has read P there, PV(u - 1) right after it, once its P is there.  A ring slot is
// released by one arrival per stream: a commit by a stream that used the tile, a
// plain arrival by one that did not.
template <class C, int MODE>
__device__ __forceinline__ bool mma_many(const TreeParams& p, TreeSmem<C>& sm, uint32_t tmem,
                                         int s, int lane) {
  constexpr int D = C::D, BN = C::BN, KSTAGES = C::KSTAGES, VSTAGES = C::VSTAGES;
  const volatile int* abort = &sm.abort;
  bool ok = true;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(BM, SN, false, false);
  constexpr uint32_t IDESC_O = idesc_bf16_f32(BM, D, false, true);
  constexpr uint32_t KV16 = C::KV_TILE >> 4, SUB16 = SN * C::RB >> 4;
  const uint64_t dk = tree_sdesc(smem_u32(sm.k[0]), 16, 8 * C::RB, C::SWZ);
  const uint64_t dv = tree_sdesc(smem_u32(sm.v[0]), C::KV_BLOCK, 8 * C::RB, C::SWZ);
  auto qstep = [](int kk) {
    return static_cast<uint32_t>((kk / C::KPB) * (C::Q_BLOCK >> 4) + (kk % C::KPB) * 2);
  };
  auto kstep = [](int kk) {
    return static_cast<uint32_t>((kk / C::KPB) * (C::KV_BLOCK >> 4) + (kk % C::KPB) * 2);
  };
  const uint32_t t_o = tmem + C::col_o(s);
  const bool leader = elect_one();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_small(smem_u32(bar), parity, p.limit_ns, abort));
    return ok;
  };
  auto v_wait = [&](uint32_t g) { return wait(&sm.v_full[g % VSTAGES], (g / VSTAGES) & 1); };
  uint32_t u = 0;  // score products issued
  // the last one still owes its PV product: of ring tile pg, part psub; whether it is
  // its item's first, the last of its tile, the last of its item (then of pslot)
  bool pending = false, pfirst = false, prelease = false, plast = false;
  uint32_t pg = 0;
  int psub = 0, pslot = 0, plo = 0, phi = 0, pnode = -1;
  auto flush_pv = [&]() {
    if (!pending) return;
    const uint32_t w = u - 1;
    if (!v_wait(pg) || !wait(&sm.p_full[s][w & 1], (w >> 1) & 1)) return;
    clear_rows<C>(p, sm, sm.v[pg % VSTAGES], psub * SN, psub * SN + SN, plo, phi, pnode, pslot, lane);
    tc_fence_after();
    const uint64_t b = dv + (pg % VSTAGES) * KV16 + psub * SUB16;
    const uint32_t t_p = tmem + C::col_s(s, w & 1);
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < SN / 16; ++kk)
        mma_ts(t_o, t_p + kk * 8, b + C::RB * kk, IDESC_O, (!pfirst || kk > 0) ? 1u : 0u);
      tc_commit(smem_u32(&sm.pv_done[s][w & 1]));
      if (prelease) tc_commit(smem_u32(&sm.v_empty[pg % VSTAGES]));
      if (plast) mbar_arrive(smem_u32(&sm.item_empty[pslot]));
    }
    __syncwarp();
    pending = false;
  };
  // waits for a barrier, with what is pending done first where that takes time
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
    const uint64_t dq =
        tree_sdesc(smem_u32(sm.q_tile(items, both, both ? s : 0)), 16, 8 * C::RB, C::SWZ);
    bool first = true;
    for (int j = 0; j < it.n && ok; ++j) {
      const uint32_t g = g0 + j;
      const int t = tile_of<MODE>(it, j), parts = parts_of<C>(it, t, p.n);
      int sub0 = 0, sub1 = parts;  // this stream's
      if (!both) {
        sub0 = C::NSUB == 1 ? 0 : s;
        sub1 = C::NSUB == 1 ? ((j & 1) == s ? 1 : 0) : min(s + 1, parts);
      }
      if (!next_wait(&sm.k_full[g % KSTAGES], (g / KSTAGES) & 1)) break;
      if (sub0 >= sub1) {
        if (leader) mbar_arrive(smem_u32(&sm.k_empty[g % KSTAGES]));
        if (next_wait(&sm.v_full[g % VSTAGES], (g / VSTAGES) & 1) && leader)
          mbar_arrive(smem_u32(&sm.v_empty[g % VSTAGES]));
        continue;
      }
      for (int sub = sub0; sub < sub1 && ok; ++sub) {
        if (u > 1 && !wait(&sm.pv_done[s][u & 1], ((u >> 1) - 1) & 1)) break;
        tc_fence_after();
        const uint64_t b = dk + (g % KSTAGES) * KV16 + sub * SUB16;
        const uint32_t t_s = tmem + C::col_s(s, u & 1);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(t_s, dq + qstep(kk), b + kstep(kk), IDESC_S, kk > 0 ? 1u : 0u);
          tc_commit(smem_u32(&sm.s_full[s][u & 1]));
          if (sub + 1 == sub1) tc_commit(smem_u32(&sm.k_empty[g % KSTAGES]));
        }
        __syncwarp();
        // (the pending one is u - 1 until u counts this one)
        flush_pv();
        if (!ok) break;
        ++u;
        pending = true;
        pfirst = first;
        first = false;
        prelease = sub + 1 == sub1;
        plast = false;
        pg = g;
        psub = sub;
        pslot = slot;
        const int base = it.base0 + t * BN;
        plo = it.key0 - base;
        phi = it.L - base;
        pnode = t < it.ctx ? -1 : (t - it.ctx) * BN;
      }
    }
    if (!ok) break;
    if (leader) tc_commit(smem_u32(&sm.q_empty[slot]));
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

template <class C, int MODE>
__device__ __forceinline__ bool softmax_many(const TreeParams& p, TreeSmem<C>& sm, uint32_t tmem,
                                             int s, int quarter, int lane) {
  constexpr int D = C::D, BN = C::BN;
  constexpr bool Q8 = C::Q8, CAPPED = MODE & kTreeCapped, SLOPES = MODE & kTreeSlopes;
  const volatile int* abort = &sm.abort;
  bool ok = true;
  const int at = quarter * 32 + lane;  // tensor-memory lane
  const uint32_t base_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t tO = base_addr + C::col_o(s);
  uint32_t u = 0;  // parts of SN keys of this stream
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_small(smem_u32(bar), parity, p.limit_ns, abort));
    return ok;
  };
  uint32_t joins = 0;
  auto join = [&]() {
    warp_arrive(smem_u32(&sm.join_sync));
    return wait(&sm.join_sync, joins++ & 1);
  };
  for (uint32_t items = 0; ok; ++items) {
    const int slot = items & 1;
    if (!wait(&sm.item_full[slot], (items >> 1) & 1)) break;
    const TreeItem it = sm.item[slot];
    if (it.more == 0) break;
    const bool both = it.split == 0, twice = it.split == 2;
    const int copy = twice ? at >> 6 : 0;
    const int r = both ? s * BM + at : (twice ? at & 63 : at);
    const bool valid = r < it.rows;
    const bool active = __any_sync(0xffffffffu, valid);
    const int row = it.row0 + (valid ? r : 0);
    const int g = row / p.n, node = row - g * p.n, head = it.hk * p.G + g;
    const int depth = max(sm.depth[slot][node], 0);
    const bool alive = valid && sm.depth[slot][node] >= 0;
    const float slope2 = SLOPES ? kLog2e * __ldg(p.slopes + head) : 0.f;
    // position of the row's first visible key, for the window
    const int first_key = p.window >= 0 ? it.L + depth - p.window : 0;
    float m = -INFINITY, l = 0.f;
    bool first = true;

    // one part of a tile: NC of its 64 columns, from col0 on
    auto part_of_tile = [&](auto nc, int t, int sub, float sc) {
      constexpr int NC = decltype(nc)::value;
      const int col0 = NC < SN ? copy * NC : 0;
      const bool tree = t >= it.ctx;
      // the key (or node) of column 0
      const int base = (tree ? (t - it.ctx) * BN : it.base0 + t * BN) + sub * SN;
      const uint32_t tS = base_addr + C::col_s(s, u & 1);
      uint32_t x[NC / 32][32];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) tmem_ld32(tS + col0 + 32 * c, x[c]);
      // the scale of 16 columns: of the tile's block that they lie in
      auto scale_at = [&](int col, int kv) {
        return __shfl_sync(0xffffffffu, sc, kv * 8 + ((sub * SN + col0 + col) >> p.T_log2));
      };
      float factor[NC / 16];
#pragma unroll
      for (int c = 0; c < NC / 16; ++c)
        factor[c] = (Q8 ? scale_at(16 * c, 0) : 1.f) * (CAPPED ? 1.f : p.scale_log2);
      // (a factor of zero would make NaN of masked scores)
      if constexpr (Q8 && MODE == 0) {
#pragma unroll
        for (int c = 0; c < NC / 16; ++c) factor[c] = fmaxf(factor[c], 0x1p-126f);
      }
      const int hi = it.L - base, lo = first_key - base;
      const bool edge = tree || hi < SN || (p.window >= 0 && __any_sync(0xffffffffu, lo > 0));
      float off = 0.f;
      tmem_ld_wait(x[0]);
#pragma unroll
      for (int c = 1; c < NC / 32; ++c) reg_fence(x[c]);
      if constexpr (MODE != 0) {
        // finished scores in log2 units, but for `off`
        if constexpr (CAPPED) {
          float big = 0.f;
#pragma unroll
          for (int c = 0; c < NC / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              if constexpr (Q8) {
                float a, b;
                fma2(a, b, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]),
                     factor[2 * c + i / 16], factor[2 * c + i / 16], 0.f, 0.f);
                x[c][i] = __float_as_uint(a);
                x[c][i + 1] = __float_as_uint(b);
              }
              big = max3_abs(big, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
            }
          // (which form is taken follows from what nodes see alone, since the two round
          // differently: the general one where a tile holds anything else)
          const bool small = !edge && __all_sync(0xffffffffu, !alive || big <= p.cap.small);
          if (small) {
#pragma unroll
            for (int c = 0; c < NC / 32; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float x0 = __uint_as_float(x[c][i]), x1 = __uint_as_float(x[c][i + 1]);
                float z0, z1, y0, y1;
                fma2(z0, z1, x0, x1, x0, x1, 0.f, 0.f);
                fma2(y0, y1, z0, z1, p.cap.poly[2], p.cap.poly[2], p.cap.poly[1], p.cap.poly[1]);
                fma2(y0, y1, z0, z1, y0, y1, p.cap.poly[0], p.cap.poly[0]);
                fma2(y0, y1, x0, x1, y0, y1, 0.f, 0.f);
                x[c][i] = __float_as_uint(y0);
                x[c][i + 1] = __float_as_uint(y1);
              }
          } else {
            // cap * tanh(y) = cap - 2 cap / (1 + 2^(2 y log2(e))), in log2 units
#pragma unroll
            for (int c = 0; c < NC / 32; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = __uint_as_float(x[c][i]);
                float w = fmaf(-2.f * p.cap_log2, rcp(1.f + ex2(y * p.cap_in)), p.cap_log2);
                if (p.wide && fabsf(y) <= p.cap.small) {
                  const float z = y * y;
                  w = y * fmaf(z, fmaf(z, p.cap.poly[2], p.cap.poly[1]), p.cap.poly[0]);
                }
                x[c][i] = __float_as_uint(w);
              }
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a, b;
              fma2(a, b, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]),
                   factor[2 * c + i / 16], factor[2 * c + i / 16], 0.f, 0.f);
              x[c][i] = __float_as_uint(a);
              x[c][i + 1] = __float_as_uint(b);
            }
        }
        if constexpr (SLOPES) {
          if (tree) {
            off = -slope2 * depth;
#pragma unroll
            for (int c = 0; c < NC / 32; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int a = min(base + col0 + 32 * c + i, kMostNodes - 1);
                x[c][i] = __float_as_uint(fmaf(slope2, static_cast<float>(sm.depth[slot][a]),
                                               __uint_as_float(x[c][i])));
              }
          } else {
            off = -slope2 * static_cast<float>(it.L + depth - base - col0);
#pragma unroll
            for (int c = 0; c < NC / 32; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float col = static_cast<float>(32 * c + i);
                float a, b;
                fma2(a, b, col, col + 1.f, slope2, slope2, __uint_as_float(x[c][i]),
                     __uint_as_float(x[c][i + 1]));
                x[c][i] = __float_as_uint(a);
                x[c][i + 1] = __float_as_uint(b);
              }
          }
        }
      }
      if (edge) {
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) {
          const int at_col = col0 + 32 * c;
          const uint32_t see = tree ? sm.line[slot][node][(base + at_col) >> 5]
                                    : below(hi - at_col) & ~below(lo - at_col);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(see & (1u << i))) x[c][i] = __float_as_uint(-INFINITY);
        }
      }
      // the largest score, 16 columns of one scale at a time
      float mt = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC / 16; ++c) {
        float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16; i += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            m2[e] = max3(m2[e], __uint_as_float(x[c >> 1][(c & 1) * 16 + i + 2 * e]),
                         __uint_as_float(x[c >> 1][(c & 1) * 16 + i + 2 * e + 1]));
        mt = fmaxf(mt, fmaxf(m2[0], m2[1]) * (MODE != 0 ? 1.f : factor[c]));
      }
      mt += off;
      float alpha = 1.f;
      if (mt > m + kRescale) {
        alpha = ex2(m - mt);  // 0 when m = -inf
        l *= alpha;
        m = mt;
      }
      if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
        // O is rescaled once the last product is done
        if (!wait(&sm.pv_done[s][(u - 1) & 1], ((u - 1) >> 1) & 1)) return;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tmem_ld16(tO + c, o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(tO + c, o);
        }
      }
      const float neg_m = m == -INFINITY ? 0.f : off - m;
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float f = factor[2 * c + half];
          const float v = Q8 ? scale_at(32 * c + 16 * half, 1) : 1.f;
#pragma unroll
          for (int i = 16 * half; i < 16 * half + 16; i += 2) {
            float a, b;
            if constexpr (MODE != 0)
              add2(a, b, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]), neg_m, neg_m);
            else
              fma2(a, b, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]), f, f, neg_m,
                   neg_m);
            a = ex2(a);
            b = ex2(b);
            add2(l0, l1, l0, l1, a, b);
            if constexpr (Q8) fma2(a, b, a, b, v, v, 0.f, 0.f);
            pk[i >> 1] = pack_bf16x2(a, b);
          }
        }
        tmem_st16(tS + (col0 >> 1) + 16 * c, pk);
      }
      l += l0 + l1;
      if constexpr (NC < SN) {
        uint32_t z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0u;
        tmem_st16(tS + (16 - (col0 >> 1)), z);  // the other copy's columns
      }
      tmem_st_wait();
    };

    // lane i: the scale of the i-th block of keys of the j-th tile, 8 + i: of values
    auto scales_of = [&](int j) {
      float sc = 1.f;
      const int t = j < it.n ? tile_of<MODE>(it, j) : it.ctx;
      if (t < it.ctx) {
        const int base = it.base0 + t * BN, blk = (base >> p.T_log2) + (lane & 7);
        sc = 0.f;
        if (lane < 16 && (blk << p.T_log2) < min(it.L, base + BN) &&
            ((blk + 1) << p.T_log2) > it.key0)
          sc = __ldg((lane < 8 ? p.k_scale : p.v_scale) +
                     (static_cast<long long>(it.b) * p.HK + it.hk) * p.num_blocks + blk);
      }
      return sc;
    };
    float next_sc = Q8 ? scales_of(0) : 1.f;
    for (int j = 0; j < it.n && ok; ++j) {
      const int t = tile_of<MODE>(it, j), parts = parts_of<C>(it, t, p.n);
      int sub0 = 0, sub1 = parts;
      if (!both) {
        sub0 = C::NSUB == 1 ? 0 : s;
        sub1 = C::NSUB == 1 ? ((j & 1) == s ? 1 : 0) : min(s + 1, parts);
      }
      const float sc = next_sc;
      if constexpr (Q8) next_sc = scales_of(j + 1);  // (loaded a tile ahead)
      if (sub0 >= sub1) continue;
      for (int sub = sub0; sub < sub1; ++sub) {
        if (!wait(&sm.s_full[s][u & 1], (u >> 1) & 1)) break;
        tc_fence_after();
        if (active) {
          if (twice)
            part_of_tile(std::integral_constant<int, 32>(), t, sub, sc);
          else
            part_of_tile(std::integral_constant<int, 64>(), t, sub, sc);
          if (!ok) break;
        }
        first = false;
        tc_fence_before();
        warp_arrive(smem_u32(&sm.p_full[s][u & 1]));
        ++u;
      }
    }
    if (!ok) break;

    // ---------------------------------------------------------- the run's result
    if (!first) {
      if (!wait(&sm.pv_done[s][(u - 1) & 1], ((u - 1) >> 1) & 1)) break;
      tc_fence_after();
    }
    if (!alive) {
      m = -INFINITY;
      l = 0.f;
    }
    // (values of neighbouring rows side by side, four of each: a warp's stores are whole lines)
    float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + it.slot) * p.block_rows *
                               (D + kPartTail) + 4 * r;
    const int column = 4 * p.block_rows;  // from four values to the next four
    const int split = twice ? 2 : 1;
    const int pidx = s * split + copy;  // which part of the row (not both)
    // (sums of NaN are not 0: they go on to O and LSE)
    float weight = alive ? 1.f : 0.f, most = m, sum = l;
    if (!both) {
      sm.stat[threadIdx.x] = make_float2(m, l);
      if (!join()) break;
      most = -INFINITY;
      const int step = twice ? 64 : BM, at0 = twice ? r : at;
#pragma unroll 1
      for (int e = at0; e < 2 * BM; e += step) most = fmaxf(most, sm.stat[e].x);
      sum = 0.f;
#pragma unroll 1
      for (int e = at0; e < 2 * BM; e += step) {
        const float2 x = sm.stat[e];
        if (x.y != 0.f) sum = fmaf(x.y, ex2(x.x - most), sum);
      }
      weight = l != 0.f ? ex2(m - most) : 0.f;
    }
    if (it.whole) weight = sum != 0.f ? weight / sum : 0.f;
    const bool writer = valid && (both || pidx == 0);
    if (writer) {
      if (!it.whole)
        *reinterpret_cast<float2*>(part + (D / 4) * column) = make_float2(most, sum);
      else if (p.lse != nullptr)
        p.lse[(static_cast<size_t>(it.b) * p.H + head) * p.n + node] =
            sum != 0.f ? (most + __log2f(sum)) * kLn2 : -INFINITY;
    }
    __nv_bfloat16* out = p.o + it.b * p.so.b + head * p.so.h + node * p.so.n;
    const int lanes = twice ? 64 : BM;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t o[16];
      if (!first) tmem_ld16(tO + c, o);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        o[i] = weight != 0.f && !first ? __float_as_uint(__uint_as_float(o[i]) * weight) : 0u;
      if (!both) {
        if (pidx > 0) {
          uint4* to = reinterpret_cast<uint4*>(sm.merge[(pidx - 1) * lanes + r]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            to[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
        if (!join()) break;
        if (pidx == 0) {
#pragma unroll 1
          for (int w = 0; w < 2 * split - 1; ++w) {
            const float4* from = reinterpret_cast<const float4*>(sm.merge[w * lanes + r]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 y = from[e];
              o[4 * e] = __float_as_uint(__uint_as_float(o[4 * e]) + y.x);
              o[4 * e + 1] = __float_as_uint(__uint_as_float(o[4 * e + 1]) + y.y);
              o[4 * e + 2] = __float_as_uint(__uint_as_float(o[4 * e + 2]) + y.z);
              o[4 * e + 3] = __float_as_uint(__uint_as_float(o[4 * e + 3]) + y.w);
            }
          }
        }
      }
      if (writer) {
        if (it.whole) {
          uint4* to = reinterpret_cast<uint4*>(out + c);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t* y = o + 8 * e;
            to[e] = make_uint4(pack_bf16x2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                               pack_bf16x2(__uint_as_float(y[2]), __uint_as_float(y[3])),
                               pack_bf16x2(__uint_as_float(y[4]), __uint_as_float(y[5])),
                               pack_bf16x2(__uint_as_float(y[6]), __uint_as_float(y[7])));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(part + (c / 4 + e) * column) =
                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (!both && !join()) break;
      __syncwarp();
    }
    if (!ok) break;
    tc_fence_before();
    warp_arrive(smem_u32(&sm.item_empty[slot]));
  }
  return ok;
}

}  // namespace
}  // namespace attn
