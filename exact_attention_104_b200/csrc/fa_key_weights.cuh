// Attention weight that every key receives, from Q, K and the rows' LSE:
//   w[j] += Σ_h Σ_i exp(s·q_hi·k_j − LSE_hi)   over the query heads h of the
// key's group and the rows i that see key j.  Query row i of Nq is position
// n − Nq + i of the sequence's n keys.
//
// Sᵀ = K Qᵀ is computed with the keys as rows, so that a thread of the
// reading warpgroups owns one key: the sum over query rows runs over the
// columns of its TMEM lane, in a register, with no exchange between threads.
// One exponential per (row, key) pair bounds the kernel, not the product (d
// multiply-adds a pair on the tensor cores): the special-function unit gives
// 16 a clock and SM, so kKeyWPoly of 8 pairs of exponentials are taken by a
// polynomial on the FMA pipe instead.
//
// The work is a list of steps, of one row tile (BN query rows) against one
// unit of keys each, in order of (sequence, kv head, unit of keys, row tile).
// Every CTA takes an equal run of that list and keeps its TMEM, its rings and
// its pipeline over the whole run.  The sums of a unit that several CTAs share
// lie in slot (CTA + unit): along the list each step changes one of the two by
// one at least, so no two pairs share a slot.  fa_key_weights_reduce_kernel
// adds the slots of a unit in a fixed order.
//
//   resident   all rows of a kv head's group fit NRES row tiles: they stay in
//              shared memory while the keys stream past, 128 to a unit
//   streaming  256 keys stay, the rows stream past; each row tile is used for
//              two products, which halves the traffic from L2
// With the causal mask a streaming unit that starts at the first query's
// position or behind it takes, of each head, the rows from the first that sees
// the unit.
//
//   warp 0        TMA: K tiles and Q tiles through two rings
//   warp 1        Sᵀ = K Qᵀ into one of NBUF TMEM buffers; TMEM owner
//   warps 2, 3    −LSE·log2 e of the step's rows into shared memory (−inf for
//                 rows past Nq and rows that see no key at all: weight 0), and
//                 what the readers have to know about the step
//   warps 4-19    four warpgroups, a 128-key part of a step each in turn;
//                 thread = key
//
// Measured (B200, 8192-token prompt, 16 heads on 4 kv heads, d = 128): 176 us a call
// on the GPU, 190 one call after the other from Python.  The three quarters of the
// exponentials that the special-function unit takes would last 92 us at 1.9 GHz, the
// product 85 us at 1.63 PFLOP/s; a warpgroup computes 70 % of the time and waits for its next
// product in most of the rest, since 512 TMEM columns hold one S buffer for
// each of the four warpgroups and no more.  (Three warpgroups with a buffer to
// spare took 181 us where four took 169.)
#pragma once

#include "sm100.cuh"

namespace fa {

// Measured on an 8192-token prompt (16 heads, d = 128): 0, 2 and 3 of 8 by the
// polynomial 172, 170 and 185 us (more than 2: the added instructions cost more
// issue slots than the special-function unit gains).
constexpr int kKeyWPoly = 2;

// 2^x of two numbers on the FMA and integer pipes.  As exp2_poly, with a
// quintic (relative error 1.7e-7 in fp32, constant term pinned to 1, c1..c5
// fitted to 2^f on [−1/2, 1/2] by iteratively reweighted least squares on the
// relative error).  Clamped at −127: the result there is exactly 0, the
// product of an exponent field of 0 and a mantissa of 0.  x must be below 128.
__device__ __forceinline__ uint64_t exp2_poly5(uint64_t x) {
  float a, b;
  f2_split(x, a, b);
  x = f2_make(fmaxf(a, -127.f), fmaxf(b, -127.f));
  const uint64_t magic = f2_make(12582912.f, 12582912.f), neg_magic = f2_make(-12582912.f, -12582912.f);
  const uint64_t r = f2_add(x, magic);
  const uint64_t f = f2_fma(f2_add(r, neg_magic), f2_make(-1.f, -1.f), x);
  uint64_t p = f2_fma(f2_make(0.001326472731307149f, 0.001326472731307149f), f,
                      f2_make(0.009671512991189957f, 0.009671512991189957f));
  p = f2_fma(p, f, f2_make(0.05550733581185341f, 0.05550733581185341f));
  p = f2_fma(p, f, f2_make(0.24022242426872253f, 0.24022242426872253f));
  p = f2_fma(p, f, f2_make(0.6931470036506653f, 0.6931470036506653f));
  p = f2_fma(p, f, f2_make(1.f, 1.f));
  float r0, r1, p0, p1;
  f2_split(r, r0, r1);
  f2_split(p, p0, p1);
  return f2_make(__int_as_float(__float_as_int(p0) + (__float_as_int(r0) << 23)),
                 __int_as_float(__float_as_int(p1) + (__float_as_int(r1) << 23)));
}

template <int D, bool RESIDENT>
struct KeyWCfg {
  static constexpr int NWG = 4;                     // reading warpgroups
  static constexpr int THREADS = 128 * (NWG + 1);
  static constexpr int BN = D == 256 ? 64 : 128;    // query rows of a step (MMA N)
  static constexpr int KU = RESIDENT ? 1 : 2;       // 128-key tiles of a unit
  static constexpr int KEYS = 128 * KU;
  static constexpr int R = KEYS / BN;               // row tiles in a unit's length
  static constexpr int KPANEL = 128 * 128, QPANEL = BN * 128;  // 64 columns (bytes)
  static constexpr int KTILE = 128 * D * 2, QTILE = BN * D * 2;
  static constexpr int NRES = D == 64 ? 4 : 2;      // row tiles that fit beside the K ring
  static constexpr int NK = RESIDENT ? (D == 64 ? 8 : (D == 128 ? 4 : 2)) : (D == 64 ? 4 : 2);
  static constexpr int NQ = RESIDENT ? NRES : (D == 64 ? 8 : (D == 128 ? 4 : 2));
  static constexpr int NBUF = 512 / BN;             // TMEM buffers of Sᵀ
  // buffers of the rows' −LSE and of the steps' KeyWStep.  A wait by parity must
  // not run a phase ahead: with a multiple of 2 and of NWG, a buffer has one
  // filling warp and the same reading warpgroups every time
  static constexpr int NL = 8;
  static constexpr int K_OFF = 0;
  static constexpr int Q_OFF = NK * KTILE;
  static constexpr int LSE_OFF = Q_OFF + NQ * QTILE;
  static constexpr int STEP_OFF = LSE_OFF + NL * BN * 4;
  static constexpr int BAR_OFF = STEP_OFF + NL * 32;
  static constexpr int B_KFULL = 0;
  static constexpr int B_KEMPTY = B_KFULL + NK;
  static constexpr int B_QFULL = B_KEMPTY + NK;
  static constexpr int B_QEMPTY = B_QFULL + NQ;
  static constexpr int B_SFULL = B_QEMPTY + NQ;
  static constexpr int B_SEMPTY = B_SFULL + NBUF;
  static constexpr int B_LFULL = B_SEMPTY + NBUF;
  static constexpr int B_LEMPTY = B_LFULL + NL;
  static constexpr int B_DRAIN = B_LEMPTY + NL;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static constexpr uint32_t IDESC = idesc_bf16_f32(128, BN, false, false);
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(NL % 2 == 0 && NL % NWG == 0, "one filling warp and fixed readers for a buffer");
};

struct KeyWParams {
  const float* lse;      // [B, Hq, Nq]
  const int* lengths;    // [B], or null
  const float* weights;  // [B, Hkv, Ncap], or null
  float* weights_out;
  float* part;           // [n_ctas + B·Hkv·units][NWG][KEYS] sums
  int2* range;           // [B·Hkv·units] first and last CTA of the unit
  uint8_t* present;      // [slots] bit g: warpgroup g has a sum there
  int B, Hq, Hkv, G, Nq, Ncap;
  int units;             // units of keys of a full cache
  int row_tiles;         // of all rows of a group: ceil(G·Nq / BN)
  int n_ctas;
  int causal;
  float scale_log2;
  long long wait_cap;
  int* err;
};

__device__ __forceinline__ int keyw_len(const KeyWParams& p, int b) {
  const int n = p.lengths ? p.lengths[b] : p.Ncap;
  return (n < 0 || n > p.Ncap) ? -1 : n;
}

// The steps of one sequence's kv head.  Units 0 .. whole−1 take all rows of
// the group, packed (row r = h·Nq + i); a later unit u takes per head the rows
// from i0 = u·KEYS − (len − Nq) on, which are len − u·KEYS.
template <class C>
struct KeyWSeq {
  int len, units, whole, kb;  // kb: row tiles in len keys
  __device__ __forceinline__ void set(const KeyWParams& p, int b) {
    len = b < p.B ? keyw_len(p, b) : 0;
    units = len > 0 && p.row_tiles > 0 ? (len + C::KEYS - 1) / C::KEYS : 0;
    kb = (len + C::BN - 1) / C::BN;
    whole = units;
    if (p.causal && C::KU == 2) whole = len > p.Nq ? min(units, (len - p.Nq + C::KEYS - 1) / C::KEYS) : 0;
  }
  __device__ __forceinline__ int head_tiles(int u) const { return kb - C::R * u; }
  __device__ __forceinline__ int steps(const KeyWParams& p, int u) const {
    return u < whole ? p.row_tiles : p.G * head_tiles(u);
  }
  // steps of units 0 .. units−1
  __device__ __forceinline__ long long total(const KeyWParams& p) const {
    const long long m = units - whole;
    return (long long)whole * p.row_tiles + p.G * (m * kb - C::R * (m * (whole + units - 1) / 2));
  }
};

// Position in the list of steps; every role of a CTA walks the same run.
template <class C>
struct KeyWIter {
  KeyWSeq<C> seq;
  int b, hkv, u, s, n;  // step s of the n of unit u
  int h, t, tiles;      // per-head units: head, row tile of the head and their number
  int left;             // steps of this CTA, this one included

  __device__ __forceinline__ void unit() {
    if (u < seq.whole) return;
    tiles = seq.head_tiles(u);
    h = s / tiles;
    t = s - h * tiles;
  }
  // This CTA's run; false if it is empty.  The whole warp calls it.
  __device__ __forceinline__ bool start(const KeyWParams& p, int cta) {
    const int lane = threadIdx.x & 31;
    long long all = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      seq.set(p, b0 + lane);
      if (seq.len < 0 && cta == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
      all += seq.total(p);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    all *= p.Hkv;
    const long long per = (all + p.n_ctas - 1) / p.n_ctas;
    long long x = per * cta;
    if (x >= all) return false;
    left = (int)(min(all, x + per) - x);
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      seq.set(p, b0 + lane);
      const long long mine = seq.total(p) * p.Hkv;
      long long sum = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, sum > x);
      if (past) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        x -= __shfl_sync(0xffffffffu, sum - mine, l);
        break;
      }
      x -= __shfl_sync(0xffffffffu, sum, 31);
    }
    seq.set(p, b);
    const long long one = seq.total(p);
    hkv = (int)(x / one);
    x -= hkv * one;
    u = 0;
    if (x < (long long)seq.whole * p.row_tiles) {
      u = (int)(x / p.row_tiles);
      x -= (long long)u * p.row_tiles;
    } else {
      x -= (long long)seq.whole * p.row_tiles;
      for (u = seq.whole; x >= seq.steps(p, u); ++u) x -= seq.steps(p, u);
    }
    s = (int)x;
    n = seq.steps(p, u);
    unit();
    return true;
  }
  // To the next step (call only while left > 1).
  __device__ __forceinline__ void next(const KeyWParams& p) {
    --left;
    if (++s < n) {
      if (++t == tiles) {
        t = 0;
        ++h;
      }
      return;
    }
    s = 0;
    if (++u == seq.units) {
      u = 0;
      if (++hkv == p.Hkv) {
        hkv = 0;
        do seq.set(p, ++b);
        while (seq.units == 0 && b < p.B);
      }
    }
    n = seq.steps(p, u);
    unit();
  }
  __device__ __forceinline__ bool packed() const { return u < seq.whole; }
  // First row of the step within the group's G·Nq rows, and how many of the
  // tile's rows count.
  __device__ __forceinline__ int row0(const KeyWParams& p) const {
    return packed() ? s * C::BN : h * p.Nq + u * C::KEYS - (seq.len - p.Nq) + t * C::BN;
  }
  __device__ __forceinline__ int rows(const KeyWParams& p) const {
    return packed() ? min(C::BN, p.G * p.Nq - s * C::BN) : min(C::BN, seq.len - u * C::KEYS - t * C::BN);
  }
  __device__ __forceinline__ bool unit_ends() const { return left == 1 || s == n - 1; }
  __device__ __forceinline__ bool head_ends() const { return left == 1 || (s == n - 1 && u == seq.units - 1); }
};

// What the reading warpgroups know of a step.
struct __align__(16) KeyWStep {
  int rows;   // rows of the tile that count
  int first;  // number within its head of the tile's first row
  int least;  // least number of a row in the tile (a packed tile may go on with row 0 of the next head)
  int need;   // number of the first row that sees the unit's first key (may be negative)
  int slot;   // where the sums go
  int keys;   // keys of the sequence from the unit's first on
  int per_head;
  int pad;
};

template <int D, bool RESIDENT>
__global__ void __launch_bounds__(KeyWCfg<D, RESIDENT>::THREADS, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const KeyWParams p) {
  using C = KeyWCfg<D, RESIDENT>;
  KeyWIter<C> it;
  const int cta = blockIdx.x;
  if (!it.start(p, cta)) return;  // the same for every warp

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto BAR = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  float* lse_s = reinterpret_cast<float*>(smem + C::LSE_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(BAR(C::B_KFULL + i), 1);
      mbar_init(BAR(C::B_KEMPTY + i), 1);
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(BAR(C::B_QFULL + i), 1);
      mbar_init(BAR(C::B_QEMPTY + i), 1);
    }
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(BAR(C::B_SFULL + i), 1);
      mbar_init(BAR(C::B_SEMPTY + i), 4);
    }
    for (int i = 0; i < C::NL; ++i) {
      mbar_init(BAR(C::B_LFULL + i), 1);
      mbar_init(BAR(C::B_LEMPTY + i), 4 * C::KU);
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

  if (warp == 0) {
    if (lane == 0) {
      int kseq = 0, qseq = 0;  // tiles issued
      bool ok = true;
      auto load_q = [&](int row) -> bool {
        const int sl = qseq % C::NQ;
        if (!mbar_wait(BAR(C::B_QEMPTY + sl), ((qseq / C::NQ) & 1) ^ 1, wc, 31)) return false;
        mbar_expect_tx(BAR(C::B_QFULL + sl), C::QTILE);
        const int y = (it.b * p.Hq + it.hkv * p.G) * p.Nq + row;
#pragma unroll
        for (int pn = 0; pn < D / 64; ++pn)
          tma_load_2d(sbase + C::Q_OFF + sl * C::QTILE + pn * C::QPANEL, &tmQ, BAR(C::B_QFULL + sl), pn * 64, y);
        ++qseq;
        return true;
      };
      bool new_unit = true, new_head = true;
      while (true) {
        if (RESIDENT && new_head)
          for (int s = 0; s < p.row_tiles && ok; ++s) ok = load_q(s * C::BN);
        if (new_unit)
          for (int k = 0; k < C::KU && ok; ++k) {
            const int sl = kseq % C::NK;
            ok = mbar_wait(BAR(C::B_KEMPTY + sl), ((kseq / C::NK) & 1) ^ 1, wc, 32);
            if (!ok) break;
            mbar_expect_tx(BAR(C::B_KFULL + sl), C::KTILE);
            const int y = (it.b * p.Hkv + it.hkv) * p.Ncap + it.u * C::KEYS + k * 128;
#pragma unroll
            for (int pn = 0; pn < D / 64; ++pn)
              tma_load_2d(sbase + C::K_OFF + sl * C::KTILE + pn * C::KPANEL, &tmK, BAR(C::B_KFULL + sl), pn * 64, y);
            ++kseq;
          }
        if (!RESIDENT && ok) ok = load_q(it.row0(p));
        if (!ok || it.left == 1) break;
        new_unit = it.unit_ends();
        new_head = it.head_ends();
        it.next(p);
      }
      // every load issued has landed before the CTA may exit
      for (int i = max(0, kseq - C::NK); i < kseq; ++i)
        mbar_wait_inflight(BAR(C::B_KFULL + i % C::NK), (i / C::NK) & 1, wc, 33);
      for (int i = max(0, qseq - C::NQ); i < qseq; ++i)
        mbar_wait_inflight(BAR(C::B_QFULL + i % C::NQ), (i / C::NQ) & 1, wc, 34);
    }
  } else if (warp == 1) {
    const uint64_t dk = sdesc_sw128(sbase + C::K_OFF, 16, 1024);
    const uint64_t dq = sdesc_sw128(sbase + C::Q_OFF, 16, 1024);
    int kseq = 0, qseq = 0, sub = 0;  // first K tile of the unit, Q tile (resident: the group's first), product
    bool new_head = true, ok = true;
    while (true) {
      // a unit at a time: what its steps have in common is off their path
      if (RESIDENT && new_head)
        for (int s = 0; s < p.row_tiles && ok; ++s)
          ok = mbar_wait_warp(BAR(C::B_QFULL + (qseq + s) % C::NQ), ((qseq + s) / C::NQ) & 1, wc, 35);
      for (int k = 0; k < C::KU && ok; ++k)
        ok = mbar_wait_warp(BAR(C::B_KFULL + (kseq + k) % C::NK), ((kseq + k) / C::NK) & 1, wc, 36);
      const int m = min(it.left, it.n - it.s);  // steps of the unit here
      for (int e = 0; e < m && ok; ++e) {
        const int qs = RESIDENT ? qseq + it.s + e : qseq;
        if (!RESIDENT) ok = mbar_wait_warp(BAR(C::B_QFULL + qs % C::NQ), (qs / C::NQ) & 1, wc, 35);
        const uint32_t qoff = qs % C::NQ * C::QTILE;
#pragma unroll
        for (int k = 0; k < C::KU; ++k) {
          const int x = sub % C::NBUF;
          ok = ok && mbar_wait_warp(BAR(C::B_SEMPTY + x), ((sub / C::NBUF) & 1) ^ 1, wc, 37);
          if (!ok) break;
          tc_fence_after();
          const uint32_t koff = (kseq + k) % C::NK * C::KTILE;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_w(tbase + x * C::BN, sdesc_add(dk, koff + (kk >> 2) * C::KPANEL + (kk & 3) * 32),
                     sdesc_add(dq, qoff + (kk >> 2) * C::QPANEL + (kk & 3) * 32), C::IDESC, kk > 0 ? 1u : 0u);
          tc_commit_w(BAR(C::B_SFULL + x));
          ++sub;
        }
        if (!RESIDENT) {
          tc_commit_w(BAR(C::B_QEMPTY + qs % C::NQ));
          ++qseq;
        }
      }
      if (!ok) break;
      it.left -= m - 1;
      it.s += m - 1;
      new_head = it.head_ends();
      for (int k = 0; k < C::KU; ++k) tc_commit_w(BAR(C::B_KEMPTY + (kseq + k) % C::NK));
      kseq += C::KU;
      if (RESIDENT && new_head) {
        for (int s = 0; s < p.row_tiles; ++s) tc_commit_w(BAR(C::B_QEMPTY + (qseq + s) % C::NQ));
        qseq += p.row_tiles;
      }
      if (it.left == 1) break;
      it.next(p);
    }
    // no MMA may still be running when TMEM is released
    tc_commit_w(BAR(C::B_DRAIN));
    mbar_wait_inflight(BAR(C::B_DRAIN), 0, wc, 38);
  } else if (warp < 4) {
    KeyWStep* steps = reinterpret_cast<KeyWStep*>(smem + C::STEP_OFF);
    int q0 = 0;       // first step of the unit here
    int filled = -1;  // this warp's step whose values are held in `st` and `v`
    KeyWStep st;
    float v[C::BN / 32];
    auto publish = [&]() -> bool {
      if (filled < 0) return true;
      const int y = filled % C::NL;
      if (!mbar_wait_warp(BAR(C::B_LEMPTY + y), ((filled / C::NL) & 1) ^ 1, wc, 39)) return false;
#pragma unroll
      for (int c = 0; c < C::BN / 32; ++c) {
        const float g = -v[c] * kLog2e;
        lse_s[y * C::BN + c * 32 + lane] = g == INFINITY ? -INFINITY : g;
      }
      if (lane == 0) steps[y] = st;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_LFULL + y));
      return true;
    };
    for (int q = 0;; ++q) {
      const size_t unit = ((size_t)it.b * p.Hkv + it.hkv) * p.units + it.u;
      if ((q & 1) == warp - 2) {
        // the loads of one step are in flight while the one before is handed over
        const int row0 = it.row0(p), rows = it.rows(p);
        const float* src = p.lse + ((size_t)it.b * p.Hq + it.hkv * p.G) * p.Nq + row0;
        float next[C::BN / 32];
#pragma unroll
        for (int c = 0; c < C::BN / 32; ++c) next[c] = c * 32 + lane < rows ? src[c * 32 + lane] : INFINITY;
        if (!publish()) {
          filled = -1;
          break;
        }
#pragma unroll
        for (int c = 0; c < C::BN / 32; ++c) v[c] = next[c];
        st.rows = rows;
        st.need = p.causal ? it.u * C::KEYS - (it.seq.len - p.Nq) : -C::KEYS;
        st.first = 0;
        if (st.need + C::KEYS > 1) st.first = it.packed() ? row0 % p.Nq : st.need + it.t * C::BN;
        st.least = it.packed() && st.first + C::BN > p.Nq ? 0 : st.first;
        st.slot = (int)unit + cta;
        st.keys = it.seq.len - it.u * C::KEYS;
        st.per_head = !it.packed();
        filled = q;
      }
      if (warp == 2 && lane == 0) {
        if (it.s == 0) p.range[unit].x = cta;
        if (it.s == it.n - 1) p.range[unit].y = cta;
        if (it.unit_ends()) {
          int g = 0;
          for (int sub = q0 * C::KU; sub < (q + 1) * C::KU && g != (1 << C::NWG) - 1; ++sub) g |= 1 << sub % C::NWG;
          p.present[unit + cta] = (uint8_t)g;
          q0 = q + 1;
        }
      }
      if (it.left == 1) break;
      it.next(p);
    }
    publish();
  } else {
    const int grp = (warp - 4) >> 2, quarter = warp & 3;
    const int mykey = quarter * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint64_t sl2 = f2_make(p.scale_log2, p.scale_log2);
    const KeyWStep* steps = reinterpret_cast<const KeyWStep*>(smem + C::STEP_OFF);
    const int n_sub = it.left * C::KU;
    float sum[C::KU];
#pragma unroll
    for (int k = 0; k < C::KU; ++k) sum[k] = 0.f;
    int slot = -1;
    auto flush = [&] {
      if (slot < 0) return;
      float* dst = p.part + ((size_t)slot * C::NWG + grp) * C::KEYS + mykey;
#pragma unroll
      for (int k = 0; k < C::KU; ++k) {
        dst[k * 128] = sum[k];
        sum[k] = 0.f;
      }
    };
    for (int sub = grp; sub < n_sub; sub += C::NWG) {
      const int q = sub / C::KU, k = sub % C::KU, x = sub % C::NBUF, y = q % C::NL;
      if (!mbar_wait_warp(BAR(C::B_LFULL + y), (q / C::NL) & 1, wc, 40)) break;
      const KeyWStep st = steps[y];
      if (st.slot != slot) {
        flush();
        slot = st.slot;
      }
      // this key is seen from row `need` of its head on; blocks of 32 columns
      // before c0 are seen from no key of the warp, those from f0 on from all
      const int need = st.need + k * 128 + mykey, need0 = need - lane;
      const bool cut = need0 - quarter * 32 + 127 > st.least;
      int rows = k * 128 < st.keys ? st.rows : 0, c0 = 0, f0 = 0, f1 = rows & ~31;
      if (cut) {
        if (st.per_head) {
          c0 = min(rows, max(0, need0 - st.first) & ~31);
          f0 = max(0, (need0 + 31 - st.first + 31) & ~31);
        } else {
          f0 = C::BN;
        }
      }
      if (!mbar_wait_warp(BAR(C::B_SFULL + x), (sub / C::NBUF) & 1, wc, 41)) break;
      tc_fence_after();
      const uint32_t base = tl + x * C::BN;
      const float4* ng = reinterpret_cast<const float4*>(lse_s + y * C::BN);
      uint64_t acc[2] = {0, 0};
      // columns [from, to) under a mask: the rest of the tile's columns are
      // another head's rows, whatever they hold
      auto masked = [&](int from, int to) {
        int i = st.first + from;
        if (!st.per_head) i %= p.Nq;
#pragma unroll 1
        for (int c0 = from; c0 < to; c0 += 16) {
          uint32_t r[16];
          tmem_ld16(base + c0, r);
          tmem_ld_wait();
          reg_fence(r);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float2 g = reinterpret_cast<const float2*>(ng)[(c0 + c) / 2];
            const bool v0 = c0 + c < to && (!cut || i >= need);
            if (++i == p.Nq) i = 0;
            const bool v1 = c0 + c + 1 < to && (!cut || i >= need);
            if (++i == p.Nq) i = 0;
            const float e0 = fmaf(__uint_as_float(r[c]), p.scale_log2, g.x);
            const float e1 = fmaf(__uint_as_float(r[c + 1]), p.scale_log2, g.y);
            acc[0] = f2_add(acc[0], f2_make(ex2(v0 ? e0 : -INFINITY), ex2(v1 ? e1 : -INFINITY)));
          }
        }
      };
      auto block = [&](const uint32_t (&r)[32], int c0) {
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 g = ng[(c0 + c) / 4];
          const uint64_t e0 = f2_fma(f2_make(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sl2,
                                     f2_make(g.x, g.y));
          const uint64_t e1 = f2_fma(f2_make(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), sl2,
                                     f2_make(g.z, g.w));
          // of the pairs 0 .. 7 of 16 columns, kKeyWPoly spread evenly
          auto exp_pair = [&](uint64_t e, int pr) -> uint64_t {
            if ((pr * kKeyWPoly) % 8 < kKeyWPoly) return exp2_poly5(e);
            float a, b2;
            f2_split(e, a, b2);
            return f2_make(ex2(a), ex2(b2));
          };
          acc[0] = f2_add(acc[0], exp_pair(e0, c / 2 % 8));
          acc[1] = f2_add(acc[1], exp_pair(e1, c / 2 % 8 + 1));
        }
      };
      if (c0 < min(f0, rows)) masked(c0, min(f0, rows));
      if (max(f0, f1) < rows) masked(max(f0, f1), rows);
      // the buffer is free for the next product as soon as its last 32 columns
      // are in registers: their arithmetic covers the product's latency
      auto release = [&](int bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(bar));
      };
      if (f0 < f1) {
#pragma unroll 1
        for (int c = f0; c < f1; c += 32) {
          uint32_t r[32];
          tmem_ld32(base + c, r);
          tmem_ld_wait();
          reg_fence(r);
          if (c + 32 >= f1) {
            tc_fence_before();
            release(C::B_SEMPTY + x);
          }
          block(r, c);
        }
      } else {
        tc_fence_before();
        release(C::B_SEMPTY + x);
      }
      release(C::B_LEMPTY + y);
      float a, b2, c2, d2;
      f2_split(acc[0], a, b2);
      f2_split(acc[1], c2, d2);
      if (C::KU == 1 || k == 0) sum[0] += (a + b2) + (c2 + d2);
      else sum[C::KU - 1] += (a + b2) + (c2 + d2);
    }
    flush();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// weights_out = weights + the sums of the key's unit, added in order of the
// CTAs and their warpgroups.
template <class C>
__global__ void __launch_bounds__(256) fa_key_weights_reduce_kernel(const KeyWParams p) {
  const int bh = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= p.Ncap) return;
  KeyWSeq<C> seq;
  seq.set(p, bh / p.Hkv);
  if (seq.len < 0) {  // this sequence's weights are not written
    if (j == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return;
  }
  const size_t at = (size_t)bh * p.Ncap + j;
  float w = p.weights ? p.weights[at] : 0.f;
  const int u = j / C::KEYS;
  if (j < seq.len && u < seq.units) {
    const size_t unit = (size_t)bh * p.units + u;
    const int2 ctas = p.range[unit];
    // (within bounds also after a call that gave up)
    const int c0 = max(ctas.x, 0), c1 = min(ctas.y, p.n_ctas - 1);
    float s = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const int present = p.present[unit + c];
#pragma unroll
      for (int g = 0; g < C::NWG; ++g)
        if (present >> g & 1) s += p.part[((unit + c) * C::NWG + g) * C::KEYS + j % C::KEYS];
    }
    w += s;
  }
  p.weights_out[at] = w;
}

}  // namespace fa
