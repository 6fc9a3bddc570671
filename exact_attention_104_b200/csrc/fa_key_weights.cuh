// Attention weight that every key receives, from Q, K and the rows' LSE:
//   w[j] += Σ_h Σ_i exp(s·q_hi·k_j − LSE_hi)   over the query heads h of the
// key's group and the rows i that see key j.  Query row i of Nq is position
// n − Nq + i of the sequence's n keys.
//
// Sᵀ = K Qᵀ is computed with the keys as rows, so that a thread of the
// reading warpgroups owns one key: the sum over query rows runs over the
// columns of its TMEM lane, in a register, with no exchange between threads.
// One exponential and half a packed multiply-add and addition per (row, key)
// pair bound the kernel, not the product (d multiply-adds a pair on the tensor
// cores).
//
// One CTA per (128 keys of a sequence's kv head, run of (head, 128 query rows)
// steps):
//   warp 0        TMA: the K tile once, then the Q tiles through a ring
//   warp 1        Sᵀ = K Q_tᵀ into one of four TMEM buffers; TMEM owner
//   warp 2        −LSE·log2 e of the step's rows into shared memory (−inf for
//                 rows past Nq and rows that see no key at all: weight 0)
//   warps 4-11    two warpgroups, alternate steps; thread = key
// Where the steps of a key tile are cut into several runs, each CTA writes its
// sum and fa_key_weights_reduce_kernel adds them in a fixed order.
#pragma once

#include "sm100.cuh"

namespace fa {

template <int D>
struct KeyWCfg {
  static constexpr int THREADS = 384;
  static constexpr int BM = 128;  // keys (MMA M)
  static constexpr int BN = 128;  // query rows of a step (MMA N)
  static constexpr int PANEL = 128 * 128;
  static constexpr int TILE = BM * D * 2;
  static constexpr int NST = D == 64 ? 6 : (D == 128 ? 4 : 2);
  static constexpr int NBUF = 4;  // TMEM buffers of Sᵀ, and of the rows' −LSE
  static constexpr int K_OFF = 0;
  static constexpr int Q_OFF = TILE;
  static constexpr int LSE_OFF = Q_OFF + NST * TILE;
  static constexpr int SUM_OFF = LSE_OFF + NBUF * BN * 4;
  static constexpr int BAR_OFF = SUM_OFF + BM * 4;
  static constexpr int B_KFULL = 0;
  static constexpr int B_QFULL = 1;
  static constexpr int B_QEMPTY = B_QFULL + NST;
  static constexpr int B_SFULL = B_QEMPTY + NST;
  static constexpr int B_SEMPTY = B_SFULL + NBUF;
  static constexpr int B_LFULL = B_SEMPTY + NBUF;
  static constexpr int B_DRAIN = B_LFULL + NBUF;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static constexpr uint32_t IDESC = idesc_bf16_f32(BM, BN, false, false);
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct KeyWParams {
  const float* lse;      // [B, Hq, Nq]
  const int* lengths;    // [B], or null
  const float* weights;  // [B, Hkv, Ncap], or null
  float* weights_out;
  float* part;           // [n_run][B·Hkv][key_tiles·128], or null with one run
  int B, Hq, Hkv, G, Nq, Ncap;
  int key_tiles, q_tiles, n_run, steps_per_run;
  int causal;
  float scale_log2;
  long long wait_cap;
  int* err;
};

__device__ __forceinline__ int keyw_len(const KeyWParams& p, int b) {
  const int n = p.lengths ? p.lengths[b] : p.Ncap;
  return (n < 0 || n > p.Ncap) ? -1 : n;
}

// First 128-row query tile that sees any key of tile j0 .. j0+127, and the
// number of steps (head, query tile) of that key tile.
__device__ __forceinline__ void keyw_steps(const KeyWParams& p, int len, int j0, int& qt0, int& n) {
  qt0 = 0;
  if (p.causal) {
    const int i0 = j0 - (len - p.Nq);  // row i sees key j0 when i >= i0
    qt0 = i0 > 0 ? i0 / 128 : 0;
  }
  n = j0 < len && qt0 < p.q_tiles ? p.G * (p.q_tiles - qt0) : 0;
}

template <int D>
__global__ void __launch_bounds__(KeyWCfg<D>::THREADS, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const KeyWParams p) {
  using C = KeyWCfg<D>;
  const int run = blockIdx.x % p.n_run;
  const int jt = blockIdx.x / p.n_run % p.key_tiles;
  const int unit = blockIdx.x / p.n_run / p.key_tiles;
  const int b = unit / p.Hkv, hkv = unit % p.Hkv;
  const int j0 = jt * 128;
  const int len = keyw_len(p, b);
  if (len < 0) {  // a length out of range: this sequence's weights are not written
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return;
  }
  int qt0, n_all;
  keyw_steps(p, len, j0, qt0, n_all);
  const int s0 = run * p.steps_per_run;
  const int n = min(n_all - s0, p.steps_per_run);
  const int nq = p.q_tiles - qt0;  // query tiles of a head (positive where n > 0)
  if (n <= 0) {
    // nothing visible: the weights stay as they were (one run: written here)
    const int j = j0 + threadIdx.x;
    if (p.n_run == 1 && threadIdx.x < 128 && j < p.Ncap) {
      const size_t at = (size_t)unit * p.Ncap + j;
      p.weights_out[at] = p.weights ? p.weights[at] : 0.f;
    }
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto BAR = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  float* lse_s = reinterpret_cast<float*>(smem + C::LSE_OFF);
  float* sum_s = reinterpret_cast<float*>(smem + C::SUM_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_KFULL), 1);
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(BAR(C::B_QFULL + i), 1);
      mbar_init(BAR(C::B_QEMPTY + i), 1);
    }
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(BAR(C::B_SFULL + i), 1);
      mbar_init(BAR(C::B_SEMPTY + i), 4);
      mbar_init(BAR(C::B_LFULL + i), 1);
    }
    mbar_init(BAR(C::B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  const WaitCtx wc{abort_flag, p.err, p.wait_cap};
  // step t of this CTA -> first row of its Q tile within the head, and the head
  auto step_head = [&](int t) { return hkv * p.G + (s0 + t) / nq; };
  auto step_row = [&](int t) { return (qt0 + (s0 + t) % nq) * 128; };

  float sum = 0.f;
  if (warp == 0) {
    if (lane == 0) {
      mbar_expect_tx(BAR(C::B_KFULL), C::TILE);
#pragma unroll
      for (int pn = 0; pn < D / 64; ++pn)
        tma_load_2d(sbase + C::K_OFF + pn * C::PANEL, &tmK, BAR(C::B_KFULL), pn * 64, unit * p.Ncap + j0);
      int issued = 0;
      for (int t = 0; t < n; ++t) {
        const int st = t % C::NST;
        if (!mbar_wait(BAR(C::B_QEMPTY + st), ((t / C::NST) & 1) ^ 1, wc, 31)) break;
        mbar_expect_tx(BAR(C::B_QFULL + st), C::TILE);
        const int y = (b * p.Hq + step_head(t)) * p.Nq + step_row(t);
#pragma unroll
        for (int pn = 0; pn < D / 64; ++pn)
          tma_load_2d(sbase + C::Q_OFF + st * C::TILE + pn * C::PANEL, &tmQ, BAR(C::B_QFULL + st), pn * 64, y);
        issued = t + 1;
      }
      // every load issued has landed before the CTA may exit
      mbar_wait_inflight(BAR(C::B_KFULL), 0, wc, 32);
      for (int st = 0; st < C::NST && st < issued; ++st) {
        const int last = issued - 1 - (issued - 1 - st) % C::NST;
        mbar_wait_inflight(BAR(C::B_QFULL + st), (last / C::NST) & 1, wc, 33);
      }
    }
  } else if (warp == 1) {
    bool ok = mbar_wait_warp(BAR(C::B_KFULL), 0, wc, 34);
    const uint64_t dk = sdesc_sw128(sbase + C::K_OFF, 16, 1024);
    const uint64_t dq = sdesc_sw128(sbase + C::Q_OFF, 16, 1024);
    for (int t = 0; t < n && ok; ++t) {
      const int st = t % C::NST, x = t % C::NBUF;
      if (!mbar_wait_warp(BAR(C::B_QFULL + st), (t / C::NST) & 1, wc, 35)) break;
      if (!mbar_wait_warp(BAR(C::B_SEMPTY + x), ((t / C::NBUF) & 1) ^ 1, wc, 36)) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * C::PANEL + (kk & 3) * 32;
        mma_ss_w(tbase + x * 128, sdesc_add(dk, off), sdesc_add(dq, st * C::TILE + off), C::IDESC, kk > 0 ? 1u : 0u);
      }
      tc_commit_w(BAR(C::B_SFULL + x));
      tc_commit_w(BAR(C::B_QEMPTY + st));
    }
    // no MMA may still be running when TMEM is released
    tc_commit_w(BAR(C::B_DRAIN));
    mbar_wait_inflight(BAR(C::B_DRAIN), 0, wc, 37);
  } else if (warp == 2) {
    for (int t = 0; t < n; ++t) {
      const int x = t % C::NBUF;
      if (!mbar_wait_warp(BAR(C::B_SEMPTY + x), ((t / C::NBUF) & 1) ^ 1, wc, 38)) break;
      const float* src = p.lse + ((size_t)b * p.Hq + step_head(t)) * p.Nq;
      const int i0 = step_row(t);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = i0 + c * 32 + lane;
        float v = -INFINITY;
        if (i < p.Nq) {
          v = -src[i] * kLog2e;
          if (v == INFINITY) v = -INFINITY;
        }
        lse_s[x * 128 + c * 32 + lane] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_LFULL + x));
    }
  } else if (warp >= 4) {
    const int grp = (warp - 4) >> 2, quarter = warp & 3;
    const int key = j0 + quarter * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint64_t sl2 = f2_make(p.scale_log2, p.scale_log2);
    uint64_t acc[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
    for (int t = grp; t < n; t += 2) {
      const int x = t % C::NBUF;
      const uint32_t par = (t / C::NBUF) & 1;
      if (!mbar_wait_warp(BAR(C::B_LFULL + x), par, wc, 39)) break;
      if (!mbar_wait_warp(BAR(C::B_SFULL + x), par, wc, 40)) break;
      tc_fence_after();
      // rows of the step before column c0 do not see this thread's key
      int c0 = 0;
      if (p.causal) c0 = key - (len - p.Nq) - step_row(t);
      const bool edge = __any_sync(0xffffffffu, c0 > 0);
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t r[32];
        tmem_ld32(tl + x * 128 + cc * 32, r);
        const float4* ng = reinterpret_cast<const float4*>(lse_s + x * 128 + cc * 32);
        tmem_ld_wait();
        reg_fence(r);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 g = ng[c / 4];
          float e0, e1, e2, e3;
          f2_split(f2_fma(f2_make(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sl2, f2_make(g.x, g.y)), e0, e1);
          f2_split(f2_fma(f2_make(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), sl2, f2_make(g.z, g.w)), e2,
                   e3);
          if (edge) {
            if (cc * 32 + c < c0) e0 = -INFINITY;
            if (cc * 32 + c + 1 < c0) e1 = -INFINITY;
            if (cc * 32 + c + 2 < c0) e2 = -INFINITY;
            if (cc * 32 + c + 3 < c0) e3 = -INFINITY;
          }
          acc[0] = f2_add(acc[0], f2_make(ex2(e0), ex2(e1)));
          acc[1] = f2_add(acc[1], f2_make(ex2(e2), ex2(e3)));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_SEMPTY + x));
    }
    float a, c2, d2, e2;
    f2_split(acc[0], a, c2);
    f2_split(acc[1], d2, e2);
    sum = (a + c2) + (d2 + e2);
    if (grp == 1) sum_s[quarter * 32 + lane] = sum;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (warp >= 4 && warp < 8 && !*abort_flag) {
    const int r = (warp & 3) * 32 + lane, j = j0 + r;
    sum += sum_s[r];
    if (p.n_run > 1) {
      p.part[((size_t)run * p.B * p.Hkv + unit) * (p.key_tiles * 128) + j] = sum;
    } else if (j < p.Ncap) {
      const size_t at = (size_t)unit * p.Ncap + j;
      const float w = p.weights ? p.weights[at] : 0.f;
      p.weights_out[at] = j < len ? w + sum : w;
    }
  }
}

// weights_out = weights + the runs' sums, added in order of the runs.
__global__ void __launch_bounds__(256) fa_key_weights_reduce_kernel(const KeyWParams p) {
  const int unit = blockIdx.y, b = unit / p.Hkv;
  const int j = blockIdx.x * 256 + threadIdx.x;
  const int len = keyw_len(p, b);
  if (len < 0 || j >= p.Ncap) return;
  int qt0, n;
  keyw_steps(p, len, j / 128 * 128, qt0, n);
  const int runs = (n + p.steps_per_run - 1) / p.steps_per_run;
  const size_t at = (size_t)unit * p.Ncap + j;
  float s = 0.f;
  for (int r = 0; r < runs; ++r) s += p.part[((size_t)r * p.B * p.Hkv + unit) * (p.key_tiles * 128) + j];
  const float w = p.weights ? p.weights[at] : 0.f;
  p.weights_out[at] = j < len ? w + s : w;
}

}  // namespace fa
