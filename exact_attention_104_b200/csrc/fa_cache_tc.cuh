// Cache attention for more than 16 query rows against one run of keys (a
// prefix that a batch shares, drafted tokens, wide groups of heads), on tcgen05:
// 128-row tiles, 128-key tiles, one CTA an SM that keeps its rings and TMEM
// over its whole run of the work list (fa_cache_list.cuh).
//
//   warp 0     TMA: K and V tiles through a ring
//   warp 1     S = Q Kᵀ and O += P V; TMEM owner.  Of a unit's last key tile it
//              clears the V rows behind the last key: their weight is 0, but
//              what lies there may be NaN
//   warps 4-11 gather the unit's Q rows (the prefix's rows come from all
//              sequences) into shared memory; softmax, thread = row, the first
//              warpgroup taking keys 0-63 of a tile and the second keys 64-127
//              (the two threads of a row exchange their maxima); partial O
//
// P goes into the second product as the sum of two bf16 numbers (high part and
// remainder): with a weight good to 2^-16, O is as good as its own rounding.
// That is half more tensor work (three products a tile for two) and cost 6 % of
// the time.
//
// Measured (K and V from HBM): 8 kv heads x 8192 keys for 128 rows (d = 128), all
// SMs: 22 us, of which four tiles a CTA take 7 and the rest are start and end; 16
// units x 20001 keys for 240 rows (d = 256), the two row tiles in step: 73 us, 3.2 us a
// tile, the prefix read from HBM once.  Two things are known to stretch a tile there.
// The ring: 160 KB hold little more than one tile's K and V, so their latency shows.
// And registers: 384 threads have 168 each, and the softmax loop's 64 scores and 64
// words of P do not fit, so 324, 316 and 364 bytes a thread (d = 64, 128, 256) are
// spilled.  How much each costs has not been measured.
//
// The two warps of 32 rows meet at named barriers.  A warp whose wait gave up
// therefore goes on through the same barriers, without doing anything else.
#pragma once

#include "fa_cache_list.cuh"
#include "fa_fwd.cuh"

namespace fa {

template <int D>
struct CacheTcCfg : FwdCfg<D, 1> {
  using F = FwdCfg<D, 1>;
  static constexpr int THREADS = 384;
  static constexpr int MX_OFF = F::MISC_OFF + 16;  // fp32 [2 tiles][2 warpgroups][128]: row maxima; l at the end
  static constexpr int SMEM_BYTES = MX_OFF + 4 * 128 * 4;  // no room for slack at d = 256: the base has to be aligned
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(CacheTcCfg<D>::THREADS, 1)
    fa_cache_tc_kernel(const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const CacheParams p, const CacheList list) {
  using C = CacheTcCfg<D>;
  using Ord = KVOrder;
  grid_trigger();  // the split kernel beside this one, see launch_cache
  CacheRuns run;
  const int cta = blockIdx.x;
  if (!run.start(p, list, cta)) return;  // the same for every warp

  extern __shared__ __align__(1024) uint8_t smem_tc[];
  uint8_t* smem = smem_tc;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {  // dynamic shared memory starts on a 1024-byte boundary; the swizzle relies on it
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevCheck);
    return;
  }
  auto BAR = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_QFULL), 256);
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(BAR(C::B_KVFULL + i), 1);
      mbar_init(BAR(C::B_KVEMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::B_SFULL + i), 1);
      mbar_init(BAR(C::B_PFULL + i), 8);
      mbar_init(BAR(C::B_ODONE + i), 1);
    }
    mbar_init(BAR(C::B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  const WaitCtx wc{abort_flag, p.err, p.wait_cap};
  // tiles and chunk loads are numbered over the CTA's whole run: `tile0` and
  // `seq0` are the numbers of a run's first

  if (warp == 0) {
    if (lane == 0) {
      int seq = 0;  // chunk loads issued
      bool ok = true;
      do {
        const int n = run.t1 - run.t0;
        const CUtensorMap* mk = run.prefix ? &tmKp : &tmK;
        const CUtensorMap* mv = run.prefix ? &tmVp : &tmV;
        const int y0 = (run.prefix ? run.hkv * p.Np : (run.b * p.Hkv + run.hkv) * p.Ncap) + run.t0 * C::BN;
        for (int u = 0; u < 2 * n && ok; ++u) {
          bool is_v;
          int j;
          Ord::decode(u, n, is_v, j);
#pragma unroll
          for (int c = 0; c < C::NCH; ++c) {
            const int slot = seq % C::NSLOT;
            if (!mbar_wait(BAR(C::B_KVEMPTY + slot), ((seq / C::NSLOT) & 1) ^ 1, wc, 41)) { ok = false; break; }
            mbar_expect_tx(BAR(C::B_KVFULL + slot), C::SLOT_BYTES);
#pragma unroll
            for (int pp = 0; pp < C::CH / 64; ++pp)
              tma_load_2d(sbase + C::KV_OFF + slot * C::SLOT_BYTES + pp * C::PANEL, is_v ? mv : mk,
                          BAR(C::B_KVFULL + slot), c * C::CH + pp * 64, y0 + j * C::BN);
            ++seq;
          }
        }
      } while (ok && run.next(p, list));
      // every load issued has landed before the CTA may exit
      for (int i = max(0, seq - C::NSLOT); i < seq; ++i)
        mbar_wait_inflight(BAR(C::B_KVFULL + i % C::NSLOT), (i / C::NSLOT) & 1, wc, 42);
    }
  } else if (warp == 1) {
    const uint64_t dQ = sdesc_sw128(sbase + C::Q_OFF, 16, 1024);
    const uint64_t dK = sdesc_sw128(sbase + C::KV_OFF, 16, 1024);
    const uint64_t dV = sdesc_sw128(sbase + C::KV_OFF, C::PANEL, 1024);
    int seq0 = 0, tile0 = 0, nrun = 0;
    bool ok = true;
    do {
      const int n = run.t1 - run.t0;
      auto seq_of = [&](int u, int c) { return seq0 + u * C::NCH + c; };
      auto wait_unit = [&](int u) -> bool {
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) {
          const int s = seq_of(u, c);
          if (!mbar_wait_warp(BAR(C::B_KVFULL + s % C::NSLOT), (s / C::NSLOT) & 1, wc, 43)) return false;
        }
        tc_fence_after();
        return true;
      };
      auto release_unit = [&](int u) {
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) tc_commit_w(BAR(C::B_KVEMPTY + seq_of(u, c) % C::NSLOT));
      };
      // S(j) into its buffer, once its K tile is there
      auto issue_s = [&](int j) -> bool {
        const int u = Ord::unitK(j, n), x = (tile0 + j) & 1;
        if (!wait_unit(u)) return false;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int col = kk * 16;
          const uint32_t koff = seq_of(u, col / C::CH) % C::NSLOT * C::SLOT_BYTES;
          mma_ss_w(tbase + C::S_COL + 128 * x, sdesc_add(dQ, (kk >> 2) * C::PANEL + (kk & 3) * 32),
                   sdesc_add(dK, koff + ((col % C::CH) / 64) * C::PANEL + (kk & 3) * 32), C::IDESC_S, kk > 0 ? 1u : 0u);
        }
        tc_commit_w(BAR(C::B_SFULL + x));
        release_unit(u);
        return true;
      };
      // O (+)= P V: high parts of P in columns 0..63 of its S buffer, remainders
      // in 64..127
      auto issue_pv = [&](int j) {
        const int u = Ord::unitV(j, n), scol = C::S_COL + 128 * ((tile0 + j) & 1);
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) {
          const uint64_t db = sdesc_add(dV, seq_of(u, c) % C::NSLOT * C::SLOT_BYTES);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts_w(tbase + C::O_COL + c * C::CH, tbase + scol + part * 64 + kk * 8, sdesc_add(db, kk * 2048),
                       C::IDESC_PV, (j > 0 || part > 0 || kk > 0) ? 1u : 0u);
        }
      };
      ok = mbar_wait_warp(BAR(C::B_QFULL), nrun & 1, wc, 44);
      tc_fence_after();
      if (ok) ok = issue_s(0);
      if (ok && n > 1) ok = issue_s(1);
      for (int j = 0; j < n && ok; ++j) {
        const int T = tile0 + j, x = T & 1;
        // V of the tile; rows behind the last key are cleared
        const int u = Ord::unitV(j, n);
        ok = wait_unit(u);
        if (!ok) break;
        const int first = run.len - (run.t0 + j) * C::BN;
        if (first < C::BN) {
#pragma unroll
          for (int c = 0; c < C::NCH; ++c) {
            uint8_t* v = smem + C::KV_OFF + seq_of(u, c) % C::NSLOT * C::SLOT_BYTES;
            for (int e = lane; e < (C::BN - first) * (C::CH / 8); e += 32) {
              const int r = first + e / (C::CH / 8), col = e % (C::CH / 8);
              *reinterpret_cast<uint4*>(v + (col >> 3) * C::PANEL + r * 128 + (col & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        ok = mbar_wait_warp(BAR(C::B_PFULL + x), (T >> 1) & 1, wc, 45);
        if (!ok) break;
        tc_fence_after();
        issue_pv(j);
        tc_commit_w(BAR(C::B_ODONE + x));
        release_unit(u);
        if (j + 2 < n) ok = issue_s(j + 2);
      }
      seq0 += 2 * n * C::NCH;
      tile0 += n;
      ++nrun;
    } while (ok && run.next(p, list));
    // no MMA may still be running when TMEM is released
    tc_commit_w(BAR(C::B_DRAIN));
    mbar_wait_inflight(BAR(C::B_DRAIN), 0, wc, 47);
  } else if (warp >= 4) {
    const int quarter = warp & 3, row = quarter * 32 + lane, wg = (warp - 4) >> 2;
    const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16);
    const float sl2 = p.scale_log2;
    float* mx_s = reinterpret_cast<float*>(smem + C::MX_OFF);
    int tile0 = 0;
    bool ok = true;
    do {
      const int n = run.t1 - run.t0, rows = run.prefix ? p.M : p.R, m = run.rt * C::BM + row;
      if (threadIdx.x == 128) run.note(list, cta);
      // The Q tile: every product that read the one before has finished (its
      // scores have been read), and at the barrier all warps are done with the
      // staging of their O there.  Eight lanes copy a row's 128-byte pieces.
      named_bar_sync(5, 256);
      {
        uint4 v[4][D / 64];
        const int c = lane & 7;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int mm = run.rt * C::BM + (warp - 4) * 16 + i * 4 + (lane >> 3);
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + cache_row(p, run.prefix, run.b, run.hkv, min(mm, rows - 1)) * D);
#pragma unroll
          for (int pn = 0; pn < D / 64; ++pn) v[i][pn] = mm < rows ? src[pn * 8 + c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (warp - 4) * 16 + i * 4 + (lane >> 3);
#pragma unroll
          for (int pn = 0; pn < D / 64; ++pn)
            *reinterpret_cast<uint4*>(smem + C::Q_OFF + pn * C::PANEL + r * 128 + ((c ^ (r & 7)) << 4)) = v[i][pn];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(BAR(C::B_QFULL));

      const int row_last = cache_last(p, run.prefix, run.b, run.len, m);
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int T = tile0 + j, x = T & 1, scol = C::S_COL + 128 * x;
        ok = ok && mbar_wait_warp(BAR(C::B_SFULL + x), (T >> 1) & 1, wc, 48);
        float s[64], mx = -INFINITY;
        if (ok) {
          tc_fence_after();
          uint32_t r0[32], r1[32];
          tmem_ld32(tl + scol + wg * 64, r0);
          tmem_ld32(tl + scol + wg * 64 + 32, r1);
          tmem_ld_wait();
          reg_fence(r0);
          reg_fence(r1);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            s[c] = __uint_as_float(r0[c]);
            s[32 + c] = __uint_as_float(r1[c]);
          }
          const int key0 = (run.t0 + j) * C::BN + wg * 64;
          if (key0 + 63 > row_last) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (key0 + c > row_last) s[c] = -INFINITY;
          }
          if (p.scores && !run.prefix && m < rows) {
            float4* dst = reinterpret_cast<float4*>(
                p.scores + ((size_t)(run.b * p.Hkv + run.hkv) * p.R + m) * p.cap_pad + key0);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              dst[c] = make_float4(s[4 * c] * sl2, s[4 * c + 1] * sl2, s[4 * c + 2] * sl2, s[4 * c + 3] * sl2);
          }
          float a[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a[k] = fmaxf(s[16 * k], s[16 * k + 1]);
#pragma unroll
            for (int i = 2; i < 16; i += 2) a[k] = fmax3(a[k], s[16 * k + i], s[16 * k + i + 1]);
          }
          mx = fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
          mx_s[(x * 2 + wg) * 128 + row] = mx;
        }
        // both warps have read their scores (P overwrites them) and noted their
        // maxima; the next tile's go to the other half of mx_s
        tc_fence_before();
        named_bar_sync(1 + quarter, 64);
        tc_fence_after();
        if (!ok) continue;
        mx = fmaxf(mx, mx_s[(x * 2 + (wg ^ 1)) * 128 + row]);
        // the reference maximum moves only when a row's maximum passes it by
        // more than kRescaleTau: l and O share it, so the result is the same
        const float m_new = fmaxf(m_ref, mx * sl2);
        float alpha = 1.f;
        bool warp_rescale = false;
        if (j == 0) {
          m_ref = m_new;
        } else {
          const bool need = m_new > m_ref + kRescaleTau;
          warp_rescale = __any_sync(0xffffffffu, need);
          if (need) {
            alpha = ex2(m_ref - m_new);
            m_ref = m_new;
            l *= alpha;
          }
        }
        const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;  // no key seen yet: every P is 0
        uint64_t rs2[2] = {0, 0};
        // P = 2^(s·scale·log2e − m_ref) as high parts and remainders
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float x0, x1;
          f2_split(f2_fma(f2_make(s[2 * c], s[2 * c + 1]), f2_make(sl2, sl2), f2_make(neg_m, neg_m)), x0, x1);
          const uint64_t a = f2_make(ex2(x0), ex2(x1));
          rs2[c & 1] = f2_add(rs2[c & 1], a);
          f2_split(a, x0, x1);
          hi[c] = pack_bf16(x0, x1);
          f2_split(f2_fma(bf2_to_f2(hi[c]), f2_make(-1.f, -1.f), a), x0, x1);
          lo[c] = pack_bf16(x0, x1);
        }
        if (warp_rescale) {
          // O must hold the tile before's product before it is scaled, and be
          // scaled (half of its columns by each of the row's threads) before
          // this tile's accumulates
          ok = mbar_wait_warp(BAR(C::B_ODONE + ((T - 1) & 1)), ((T - 1) >> 1) & 1, wc, 49);
          if (!ok) continue;
          tc_fence_after();
#pragma unroll
          for (int oc = 0; oc < D / 64; ++oc) {
            uint32_t ov[32];
            const uint32_t at = tl + C::O_COL + wg * (D / 2) + oc * 32;
            tmem_ld32(at, ov);
            tmem_ld_wait();
            reg_fence(ov);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
            tmem_st32(at, ov);
          }
        }
        tmem_st32(tl + scol + wg * 32, hi);
        tmem_st32(tl + scol + 64 + wg * 32, lo);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_PFULL + x));
        float a, b2, c2, d2;
        f2_split(rs2[0], a, b2);
        f2_split(rs2[1], c2, d2);
        l += (a + b2) + (c2 + d2);
      }
      const int T = tile0 + n - 1;
      ok = ok && mbar_wait_warp(BAR(C::B_ODONE + (T & 1)), (T >> 1) & 1, wc, 50);
      // the second warpgroup's l to the first: in the half of mx_s that the last
      // tile did not use
      if (wg == 1) mx_s[(((T & 1) ^ 1) * 2 + 1) * 128 + row] = l;
      named_bar_sync(1 + quarter, 64);
      if (ok) {
        tc_fence_after();
        const size_t slot = (size_t)(run.unit + cta) * C::BM + quarter * 32;
        if (wg == 0 && m < rows)
          *reinterpret_cast<float2*>(list.part_ml + (slot + lane) * 2) =
              make_float2(m_ref, l + mx_s[(((T & 1) ^ 1) * 2 + 1) * 128 + row]);
        // O: this warp's rows, half of the columns, through its eighth of the Q
        // tile's space so that rows are written in whole lines
        constexpr int NC = D / 16;  // 16-byte pieces of a row in one pass
        float4* stage = reinterpret_cast<float4*>(smem + C::Q_OFF) + (warp - 4) * 32 * NC;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          const int col0 = wg * (D / 2) + pass * (D / 4);
#pragma unroll
          for (int cc = 0; cc < D / 64; ++cc) {
            uint32_t ov[16];
            tmem_ld16(tl + C::O_COL + col0 + cc * 16, ov);
            tmem_ld_wait();
            reg_fence(ov);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              stage[lane * NC + ((cc * 4 + i) ^ (lane & (NC - 1)))] =
                  make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]),
                              __uint_as_float(ov[4 * i + 2]), __uint_as_float(ov[4 * i + 3]));
          }
          __syncwarp();
          const int mine = min(32, rows - run.rt * C::BM - quarter * 32);  // rows of this warp (may be <= 0)
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int r = (i * 32 + lane) / NC, c = lane % NC;
            if (r < mine)
              *reinterpret_cast<float4*>(list.part_o + (slot + r) * D + col0 + 4 * c) =
                  stage[r * NC + (c ^ (r & (NC - 1)))];
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      tile0 += n;
    } while (run.next(p, list));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

}  // namespace fa
