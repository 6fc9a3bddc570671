// Cache attention for up to 16 query rows against one run of keys, and the
// joining of all partial results.
//
//   fa_cache_split_kernel    the work list of fa_cache_list.cuh, 16-row tiles
//   fa_cache_finish_kernel   O and LSE, one warp per query row; and
//                            w[j] += Σ_r 2^(S'_rj − LSE'_r) from stored scores
//
// The split kernel is bound by reading K and V.  Its rows fill one m16n8k16
// tile, so a CTA is one warp, several to an SM: TMA loads of CH keys a step
// through a ring of stages that runs ahead into the next units, S in registers,
// P handed to the second product in registers, and no barrier at all; what one
// warp does between two units the others' loads cover.  (CTAs of four warps that
// merge their results: 30 us instead of 21 for 32 x 8 caches of 64..1024 keys.)
// K and V are read once and marked to leave L2 first, where the scores and the
// partial results then stay: 202 -> 192 us for 8 x 32768 keys, d = 128.  P goes
// into the second product as the sum of two bf16 numbers (high part and
// remainder), so O has fp32-like weights; the extra instructions fit under the
// loads.  Measured, those 8 x 32768 keys, this kernel alone: 179 us for 1.07 GB, 0.91
// of the copy rate.
#pragma once

#include "fa_cache_list.cuh"

namespace fa {

// D[16x8] += A[16x16]·B[16x8], bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// log2 units by which a row maximum may pass the reference maximum before O is
// rescaled: P stays below 2^8, and no sum comes near the fp32 range
constexpr float kCacheTau = 8.0f;

template <int D>
struct CacheCfg {
  static constexpr int THREADS = 32;
  static constexpr int CH = D == 256 ? 16 : 32;  // keys of a step: the list's key tile
  static constexpr int ST = 3;                   // stages of the ring
  static constexpr int PANEL = CH * 128;         // 64 columns x CH keys (bytes)
  static constexpr int TILE = PANEL * (D / 64);  // CH keys of K or V
  static constexpr int STAGE = 2 * TILE;
  static constexpr int BAR_OFF = ST * STAGE;     // full[ST]
  static constexpr int LOAD_OFF = BAR_OFF + ST * 8;
  static constexpr int MISC_OFF = LOAD_OFF + 80;
  static constexpr int SMEM_BYTES = MISC_OFF + 16;
  static constexpr int PER_SM = D == 64 ? 8 : 4;  // CTAs an SM: 192 KB of stages
  static_assert(PER_SM * (SMEM_BYTES + 1024) <= 233472, "shared memory of an SM");
};

// How far the loads have come: they run up to ST steps ahead of the arithmetic,
// into the next units too.  Kept in shared memory by lane 0.
struct CacheLoads {
  CacheRuns run;
  int t;       // next key tile
  int more;    // whether there may be another run
  int issued;  // over all of the CTA's runs
};

template <int D>
__global__ void __launch_bounds__(CacheCfg<D>::THREADS)
    fa_cache_split_kernel(const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                          const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const CacheParams p, const CacheList list) {
  using C = CacheCfg<D>;
  CacheRuns run;
  const int cta = blockIdx.x;
  // beside the tcgen05 kernel: what comes after this kernel reads the results of
  // both, so no CTA leaves before that one has finished
  if (!run.start(p, list, cta)) {
    grid_wait();
    return;
  }

  extern __shared__ __align__(1024) uint8_t smem_split[];
  uint8_t* smem = smem_split;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {  // dynamic shared memory starts on a 1024-byte boundary; the swizzle relies on it
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevCheck);
    grid_wait();
    return;
  }
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
  const int lane = threadIdx.x;
  if (lane == 0) {
    for (int i = 0; i < C::ST; ++i) mbar_init(sbase + C::BAR_OFF + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  const uint32_t ring = sbase, bars = sbase + C::BAR_OFF;
  const WaitCtx wc{abort_flag, p.err, p.wait_cap};
  CacheLoads* ld = reinterpret_cast<CacheLoads*>(smem + C::LOAD_OFF);
  static_assert(sizeof(CacheLoads) <= 80, "space of CacheLoads");
  const uint64_t policy = policy_evict_first();
  // lane 0: the next step's loads, if there is one
  auto issue = [&] {
    if (ld->t == ld->run.t1) {
      if (!ld->more || !ld->run.next(p, list)) {
        ld->more = 0;
        return;
      }
      ld->t = ld->run.t0;
    }
    const CacheRuns& r = ld->run;
    const int st = ld->issued % C::ST;
    const int y = (r.prefix ? r.hkv * p.Np : (r.b * p.Hkv + r.hkv) * p.Ncap) + ld->t * C::CH;
    const CUtensorMap* mk = r.prefix ? &tmKp : &tmK;
    const CUtensorMap* mv = r.prefix ? &tmVp : &tmV;
    mbar_expect_tx(bars + 8 * st, C::STAGE);
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn) {
      tma_load_2d_hint(ring + st * C::STAGE + pn * C::PANEL, mk, bars + 8 * st, pn * 64, y, policy);
      tma_load_2d_hint(ring + st * C::STAGE + C::TILE + pn * C::PANEL, mv, bars + 8 * st, pn * 64, y, policy);
    }
    ++ld->t;
    ++ld->issued;
  };
  if (lane == 0) {
    ld->run = run;
    ld->t = run.t0;
    ld->more = 1;
    ld->issued = 0;
    for (int i = 0; i < C::ST; ++i) issue();
  }
  int step = 0;  // over all of the CTA's runs: numbers the ring's stages
  do {
    const int rows_total = run.prefix ? p.M : p.R;
    const int len = run.len;
    if (lane == 0) run.note(list, cta);

    // this lane's two query rows: first operand fragments and last visible key
    const int row0 = run.rt * 16 + (lane >> 2);
    uint32_t qf[D / 16][4];
    int last[2];
    size_t score_row[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int m = row0 + 8 * x;
      last[x] = cache_last(p, run.prefix, run.b, len, m);
      const uint32_t* src = nullptr;
      if (m < rows_total) {
        src = reinterpret_cast<const uint32_t*>(p.q + cache_row(p, run.prefix, run.b, run.hkv, m) * D) + (lane & 3);
        score_row[x] = ((size_t)(run.b * p.Hkv + run.hkv) * p.R + m) * p.cap_pad;
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][x] = src ? src[ks * 8] : 0u;
        qf[ks][2 + x] = src ? src[ks * 8 + 4] : 0u;
      }
    }

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool ok = true;
    for (int t = run.t0; t < run.t1; ++t, ++step) {
      const int st = step % C::ST;
      if (!mbar_wait_warp(bars + 8 * st, (step / C::ST) & 1, wc, 21)) { ok = false; break; }
      const int key0 = t * C::CH;
      const uint32_t kt = ring + st * C::STAGE, vt = kt + C::TILE;
      if (key0 + C::CH > len) {
        // what lies behind the last key may be anything, NaN too: its weight is
        // 0, its value has to be 0 as well
        const int first = len - key0;
        for (int e = lane; e < (C::CH - first) * (D / 8); e += 32) {
          const int r = first + e / (D / 8), c = e % (D / 8);
          *reinterpret_cast<uint4*>(smem + (vt - sbase) + (c >> 3) * C::PANEL + r * 128 + (c & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before later loads into the stage
        __syncwarp();
      }
      // S = Q Kᵀ
      float s[C::CH / 8][4];
#pragma unroll
      for (int nt = 0; nt < C::CH / 8; nt += 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = s[nt + 1][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int key = (nt + (lane >> 4)) * 8 + (lane & 7);
          const int c = 2 * ks + ((lane >> 3) & 1);
          uint32_t kb[4];
          ldsm_x4(kb, kt + (c >> 3) * C::PANEL + key * 128 + (((c & 7) ^ (key & 7)) << 4));
          mma16816(s[nt], qf[ks], kb[0], kb[1]);
          mma16816(s[nt + 1], qf[ks], kb[2], kb[3]);
        }
      }
      // to log2 units, masked; running maximum
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < C::CH / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + nt * 8 + 2 * (lane & 3) + (e & 1);
          s[nt][e] = key > last[e >> 1] ? -INFINITY : s[nt][e] * p.scale_log2;
          mx[e >> 1] = fmaxf(mx[e >> 1], s[nt][e]);
        }
      if (p.scores && !run.prefix) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (row0 + 8 * x < rows_total)
#pragma unroll
            for (int nt = 0; nt < C::CH / 8; ++nt)
              *reinterpret_cast<float2*>(p.scores + score_row[x] + key0 + nt * 8 + 2 * (lane & 3)) =
                  make_float2(s[nt][2 * x], s[nt][2 * x + 1]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
      }
      // the reference maximum moves only when a row's maximum passes it by more
      // than kCacheTau: l and O share it, so the result is the same
      if (__any_sync(0xffffffffu, mx[0] > m_ref[0] + kCacheTau || mx[1] > m_ref[1] + kCacheTau)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float m_new = fmaxf(m_ref[x], mx[x]);
          const float a = m_new == -INFINITY ? 1.f : ex2(m_ref[x] - m_new);
          m_ref[x] = m_new;
          l[x] *= a;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * x] *= a;
            o[n][2 * x + 1] *= a;
          }
        }
      }
      const float sub[2] = {m_ref[0] == -INFINITY ? 0.f : m_ref[0], m_ref[1] == -INFINITY ? 0.f : m_ref[1]};
#pragma unroll
      for (int nt = 0; nt < C::CH / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = ex2(s[nt][e] - sub[e >> 1]);
          l[e >> 1] += s[nt][e];
        }
      // O += P V, P as high part plus remainder
#pragma unroll
      for (int kk = 0; kk < C::CH / 16; ++kk) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const float a = s[2 * kk + (f >> 1)][2 * (f & 1)], c = s[2 * kk + (f >> 1)][2 * (f & 1) + 1];
          hi[f] = pack_bf16(a, c);
          lo[f] = pack_bf16(a - bf_lo(hi[f]), c - bf_hi(hi[f]));
        }
#pragma unroll
        for (int n = 0; n < D / 8; n += 2) {
          const int key = kk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
          const int c = n + (lane >> 4);
          uint32_t vb[4];
          ldsm_x4_t(vb, vt + (c >> 3) * C::PANEL + key * 128 + (((c & 7) ^ (key & 7)) << 4));
          mma16816(o[n], hi, vb[0], vb[1]);
          mma16816(o[n + 1], hi, vb[2], vb[3]);
          mma16816(o[n], lo, vb[0], vb[1]);
          mma16816(o[n + 1], lo, vb[2], vb[3]);
        }
      }
      __syncwarp();
      if (lane == 0) issue();
    }
    if (!ok) {  // no exit before the copies in flight have landed
      if (lane == 0)
        for (int i = step; i < ld->issued; ++i) mbar_wait_inflight(bars + 8 * (i % C::ST), (i / C::ST) & 1, wc, 22);
      grid_wait();
      return;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (row0 + 8 * x >= rows_total) continue;
      const size_t slot = (size_t)(run.unit + cta) * 16 + (lane >> 2) + 8 * x;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(list.part_o + slot * D + n * 8 + 2 * (lane & 3)) =
            make_float2(o[n][2 * x], o[n][2 * x + 1]);
      if ((lane & 3) == 0) *reinterpret_cast<float2*>(list.part_ml + slot * 2) = make_float2(m_ref[x], l[x]);
    }
  } while (run.next(p, list));
  grid_wait();
}

// Where the partial results of one query row lie, and how many there are: a
// run of consecutive slots for the prefix and one for the own keys.
struct CacheParts {
  struct Run {
    const float *o, *ml;
    size_t row;  // first row of the arrays
    int step;    // rows from one CTA's slot to the next
    __device__ __forceinline__ int set(const CacheList& l, int unit, int m) {
      const int2 ctas = l.range[unit];
      // (within bounds also after a call that gave up)
      const int c0 = min(max(ctas.x, 0), l.n_ctas - 1), c1 = min(ctas.y, l.n_ctas - 1);
      o = l.part_o;
      ml = l.part_ml;
      row = (size_t)(unit + c0) * l.rows + m % l.rows;
      step = l.rows;
      return max(0, c1 - c0 + 1);
    }
  };
  Run prefix, own;
  int n_prefix, n;
  __device__ __forceinline__ const float* o(int s, int d) const {
    return s < n_prefix ? prefix.o + (prefix.row + (size_t)s * prefix.step) * d
                        : own.o + (own.row + (size_t)(s - n_prefix) * own.step) * d;
  }
  __device__ __forceinline__ float2 ml(int s) const {
    return *reinterpret_cast<const float2*>(
        s < n_prefix ? prefix.ml + (prefix.row + (size_t)s * prefix.step) * 2
                     : own.ml + (own.row + (size_t)(s - n_prefix) * own.step) * 2);
  }
};
// Row r of the R rows of sequence b's kv head.
__device__ __forceinline__ CacheParts cache_parts(const CacheParams& p, const CacheList& lp, const CacheList& lo, int b,
                                                  int hkv, int r, int len) {
  CacheParts c;
  c.n_prefix = 0;
  if (p.Np > 0) {
    const int m = b * p.R + r;
    c.n_prefix = c.prefix.set(lp, hkv * lp.prefix_rt + m / lp.rows, m);
  }
  c.n = c.n_prefix;
  if (len > 0) c.n += c.own.set(lo, lo.prefix_units + (b * p.Hkv + hkv) * lo.own_rt + r / lo.rows, r);
  return c;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// M + log2 Σ l of a row over its partial results (+inf: it sees no key), by
// `lanes` neighbouring lanes of a warp (a power of two; all lanes call it).
__device__ __forceinline__ float cache_lse2(const CacheParts& parts, int lane, int lanes) {
  float M = -INFINITY, L = 0.f;
#pragma unroll 4
  for (int s = lane; s < parts.n; s += lanes) M = fmaxf(M, parts.ml(s).x);
  for (int off = lanes / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 4
  for (int s = lane; s < parts.n; s += lanes) {
    const float2 ml = parts.ml(s);
    if (ml.x != -INFINITY) L = fmaf(ex2(ml.x - M), ml.y, L);
  }
  for (int off = lanes / 2; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  return L > 0.f ? M + lg2(L) : INFINITY;
}

// Keys of a CTA of the weights' part of the finish kernel: many, or few with the
// rows dealt to four groups of its threads where there would be too few CTAs.
constexpr int kCacheWeightKeys = 2048, kCacheWeightKeysFew = 256;
constexpr int kCacheScoreRows = 64;  // most rows whose scores are stored

// CTAs 0 .. n_combine−1: O and LSE, one query row a warp; a row that no key is
// visible to has O = 0 and LSE = −inf.  The CTAs behind them (only with stored
// scores): weights_out[j] = weights[j] + Σ_r 2^(S'_rj − LSE'_r), one CTA for p.few ?
// kCacheWeightKeysFew : kCacheWeightKeys keys of a (sequence, kv head); keys at or
// behind the sequence's length keep their weight.  Each joins the rows' m and l by itself
// rather than wait for the others' LSE in a launch of its own.  Latency bounds it
// (lengths, range, m and l are read one after the other): 3 us and up, 18 us for
// the weights of 8 x 8 x 32768 keys with 4 rows.
template <int D>
__global__ void __launch_bounds__(256)
    fa_cache_finish_kernel(const CacheParams p, const CacheList lp, const CacheList lo, unsigned n_combine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x < n_combine) {
    const long long row = (long long)blockIdx.x * 8 + warp;
    if (row >= (long long)p.B * p.Hq * p.Nq) return;
    const int i = (int)(row % p.Nq);
    const int h = (int)(row / p.Nq % p.Hq);
    const int b = (int)(row / ((long long)p.Nq * p.Hq));
    const int len = cache_len(p, b);
    if (len < 0) {
      if (lane == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
      return;
    }
    const CacheParts parts = cache_parts(p, lp, lo, b, h / p.G, (h % p.G) * p.Nq + i, len);
    // lane s has the m and l of part s (of 32 at a time; more than 32 parts: the
    // running maximum and sum go on)
    float M = -INFINITY, L = 0.f;
    constexpr int V = D / 32;  // columns of a lane
    float acc[V];
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
    for (int s0 = 0; s0 < parts.n; s0 += 32) {
      const int cnt = min(32, parts.n - s0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < cnt) ml = parts.ml(s0 + lane);
      const float m_new = fmaxf(M, warp_max(ml.x));
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - m_new);
      const float old = M == -INFINITY ? 0.f : ex2(M - m_new);
      L = fmaf(L, old, warp_sum(f * ml.y));
      M = m_new;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] *= old;
      for (int t0 = 0; t0 < cnt; t0 += 8) {
        // eight parts' loads in flight (a part that is not there: the last one, times 0)
        float part[8][V];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float* src = parts.o(s0 + min(t0 + t, cnt - 1), D) + lane * V;
          if constexpr (V == 2) {
            const float2 v = *reinterpret_cast<const float2*>(src);
            part[t][0] = v.x, part[t][1] = v.y;
          } else {
#pragma unroll
            for (int c = 0; c < V; c += 4) {
              const float4 v = *reinterpret_cast<const float4*>(src + c);
              part[t][c] = v.x, part[t][c + 1] = v.y, part[t][c + 2] = v.z, part[t][c + 3] = v.w;
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float ft = t0 + t < cnt ? __shfl_sync(0xffffffffu, f, (t0 + t) & 31) : 0.f;
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(ft, part[t][c], acc[c]);
        }
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (size_t)row * D + lane * V);
#pragma unroll
    for (int c = 0; c < V; c += 2) dst[c / 2] = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
    if (lane == 0) p.lse[row] = L > 0.f ? (M + lg2(L)) * kLn2 : -INFINITY;
    return;
  }

  __shared__ float lse2[kCacheScoreRows];
  __shared__ float4 group_sum[4][kCacheWeightKeysFew / 4];
  const int keys = p.few ? kCacheWeightKeysFew : kCacheWeightKeys;
  const int per = (p.Ncap + keys - 1) / keys;
  const int unit = (blockIdx.x - n_combine) / per, b = unit / p.Hkv;
  // thread = four keys in a row, and with few keys one of four groups of rows
  const int group = p.few ? threadIdx.x / (kCacheWeightKeysFew / 4) : 0, n_group = p.few ? 4 : 1;
  const int quad = p.few ? threadIdx.x % (kCacheWeightKeysFew / 4) : threadIdx.x;
  const int j0 = (blockIdx.x - n_combine) % per * keys + 4 * quad;
  const int len = cache_len(p, b);
  if (len < 0) {  // this sequence's weights stay as they are
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return;
  }
  {
    const int lanes = p.R <= 16 ? 16 : 4, r = threadIdx.x / lanes;
    CacheParts parts;
    parts.n = parts.n_prefix = 0;
    if (r < p.R) parts = cache_parts(p, lp, lo, b, unit % p.Hkv, r, len);
    // a row without a visible key gives no weight (its scores are −inf)
    const float x = cache_lse2(parts, threadIdx.x % lanes, lanes);
    if (r < p.R && threadIdx.x % lanes == 0) lse2[r] = x;
  }
  __syncthreads();
  for (int c = 0; c < (p.few ? 1 : kCacheWeightKeys / 1024); ++c) {
    const int j = j0 + c * 1024;
    if (j >= p.Ncap && !p.few) break;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (j < len) {  // scores are stored up to a multiple of 16 keys at least
      const float* src = p.scores + (size_t)unit * p.R * p.cap_pad + j;
#pragma unroll 8
      for (int r = group; r < p.R; r += n_group) {
        const float4 s = *reinterpret_cast<const float4*>(src + (size_t)r * p.cap_pad);
        acc[0] += ex2(s.x - lse2[r]);
        acc[1] += ex2(s.y - lse2[r]);
        acc[2] += ex2(s.z - lse2[r]);
        acc[3] += ex2(s.w - lse2[r]);
      }
    }
    if (p.few) {
      group_sum[group][quad] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      __syncthreads();
      if (group > 0 || j >= p.Ncap) return;
#pragma unroll
      for (int g = 1; g < 4; ++g) {
        const float4 s = group_sum[g][quad];
        acc[0] += s.x;
        acc[1] += s.y;
        acc[2] += s.z;
        acc[3] += s.w;
      }
    }
    const size_t at = (size_t)unit * p.Ncap + j;
    if (p.wide && j + 4 <= p.Ncap) {
      float4 w = p.weights ? *reinterpret_cast<const float4*>(p.weights + at) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < len) w.x += acc[0];
      if (j + 1 < len) w.y += acc[1];
      if (j + 2 < len) w.z += acc[2];
      if (j + 3 < len) w.w += acc[3];
      *reinterpret_cast<float4*>(p.weights_out + at) = w;
      continue;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (j + t >= p.Ncap) continue;
      const float w = p.weights ? p.weights[at + t] : 0.f;
      p.weights_out[at + t] = j + t < len ? w + acc[t] : w;
    }
  }
}

}  // namespace fa
