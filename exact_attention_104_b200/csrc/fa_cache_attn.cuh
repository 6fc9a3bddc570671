// Attention of a few query rows against ragged key/value caches, with or
// without a prefix that the whole batch shares.
//
// Sequence b is the prefix (Np keys, the same for every b) followed by its own
// n_b = lengths[b] keys out of a cache with room for Ncap.  Query row i of Nq
// is position L_b − Nq + i of the L_b = Np + n_b long sequence:
//   S_j = s·q·k_j,  O = Σ_j 2^(S_j' − M) v_j / Σ_j 2^(S_j' − M)   (S' = S·log2 e)
// and the softmax over the concatenation is put together from parts: the keys
// are cut into runs ("splits"), each run gives its running maximum m, its
// normaliser l = Σ 2^(S' − m) and its unnormalised O, and
//   O = Σ_r 2^(m_r − M) O_r / Σ_r 2^(m_r − M) l_r.
// A run of the prefix serves the rows of ALL sequences (M = B·G·Nq rows of a kv
// head), a run of own keys the R = G·Nq rows of its sequence.
//
//   fa_cache_split_kernel    one CTA per (run, kv head, group of 16 rows)
//   fa_cache_combine_kernel  one warp per query row
//   fa_cache_weights_kernel  w[j] += Σ_r 2^(S'_rj − LSE'_r) from stored scores
//
// The split kernel is bound by reading K and V.  Its rows fill one m16n8k16
// tile, so each warp works alone on runs of CH keys: TMA loads of its own ring
// of stages, S in registers, P handed to the second product in registers, and
// no barrier of the CTA inside the loop.  P goes into the second product as
// the sum of two bf16 numbers (high part and remainder), so O has fp32-like
// weights; the second product's extra instructions fit under the loads.
#pragma once

#include "sm100.cuh"

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

struct CacheParams {
  const __nv_bfloat16* q;  // [B, Hq, Nq, d]
  const int* lengths;      // [B], or null: every own cache is full
  __nv_bfloat16* o;        // [B, Hq, Nq, d]
  float* lse;              // [B, Hq, Nq]
  float* part_o;           // partial results: n_split_p·Hkv·M rows of the prefix, then n_split_o·B·Hkv·R own rows
  float* part_ml;          // the same rows: m (log2 units), l
  float* scores;           // [B·Hkv][R][cap_pad] scores in log2 units, or null
  const float* weights;    // [B, Hkv, Ncap] or null
  float* weights_out;
  int B, Hq, Hkv, G, Nq, R, M;       // R = G·Nq, M = B·R
  int Np, Ncap, cap_pad;             // cap_pad: Ncap rounded up to 32
  int rg_p, n_split_p, kps_p;        // prefix: row groups, splits, keys per split
  int rg_o, n_split_o, kps_o;        // own keys
  int causal;
  float scale_log2;
  long long wait_cap;
  int* err;
};

// Number of own keys of sequence b; −1 where lengths[b] breaks its rule.
__device__ __forceinline__ int cache_len(const CacheParams& p, int b) {
  if (!p.lengths) return p.Ncap;
  const int n = p.lengths[b];
  return (n < 0 || n > p.Ncap) ? -1 : n;
}

template <int D>
struct CacheCfg {
  static constexpr int W = 4;                    // warps
  static constexpr int THREADS = W * 32;
  static constexpr int CH = D == 256 ? 16 : 32;  // keys of one warp's step
  static constexpr int ST = 3;                   // stages of each warp's ring
  static constexpr int PANEL = CH * 128;         // 64 columns x CH keys (bytes)
  static constexpr int TILE = PANEL * (D / 64);  // CH keys of K or V
  static constexpr int STAGE = 2 * TILE;
  static constexpr int RING = W * ST * STAGE;
  static constexpr int BAR_OFF = RING;           // full[W][ST]
  static constexpr int ML_OFF = BAR_OFF + W * ST * 8;  // m, l [W][16]
  static constexpr int MISC_OFF = ML_OFF + W * 16 * 2 * 4;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static_assert(W * 16 * D * 4 <= RING, "the warps' O fit over the ring");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(CacheCfg<D>::THREADS)
    fa_cache_split_kernel(const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                          const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const CacheParams p) {
  using C = CacheCfg<D>;
  // which run of keys, which rows
  const int n_prefix = p.Hkv * p.rg_p * p.n_split_p;
  const bool prefix = (int)blockIdx.x < n_prefix;
  int split, rg, hkv, b, len, rows_total, key_base;
  if (prefix) {
    int u = blockIdx.x;
    rg = u % p.rg_p;
    u /= p.rg_p;
    split = u % p.n_split_p;
    hkv = u / p.n_split_p;
    b = 0;
    len = p.Np;
    rows_total = p.M;
    key_base = hkv * p.Np;
  } else {
    int u = blockIdx.x - n_prefix;
    rg = u % p.rg_o;
    u /= p.rg_o;
    split = u % p.n_split_o;
    u /= p.n_split_o;
    hkv = u % p.Hkv;
    b = u / p.Hkv;
    len = cache_len(p, b);
    rows_total = p.R;
    key_base = (b * p.Hkv + hkv) * p.Ncap;
    if (len < 0) {  // a length out of range: nothing of this sequence is computed
      if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
      return;
    }
  }
  const int kps = prefix ? p.kps_p : p.kps_o;
  const int k0 = split * kps;
  const int k1 = min(len, k0 + kps);
  if (k0 >= k1) return;  // past the sequence's end; the combine kernel knows

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::W * C::ST; ++i) mbar_init(sbase + C::BAR_OFF + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  const CUtensorMap* mk = prefix ? &tmKp : &tmK;
  const CUtensorMap* mv = prefix ? &tmVp : &tmV;
  const int n_chunks = (k1 - k0 + C::CH - 1) / C::CH;
  const int n_mine = (n_chunks - warp + C::W - 1) / C::W;
  const uint32_t ring = sbase + warp * C::ST * C::STAGE;
  const uint32_t bars = sbase + C::BAR_OFF + warp * C::ST * 8;
  auto issue = [&](int i) {
    const int st = i % C::ST;
    const int key0 = k0 + (warp + C::W * i) * C::CH;
    mbar_expect_tx(bars + 8 * st, C::STAGE);
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn) {
      tma_load_2d(ring + st * C::STAGE + pn * C::PANEL, mk, bars + 8 * st, pn * 64, key_base + key0);
      tma_load_2d(ring + st * C::STAGE + C::TILE + pn * C::PANEL, mv, bars + 8 * st, pn * 64, key_base + key0);
    }
  };
  if (lane == 0)
    for (int i = 0; i < C::ST && i < n_mine; ++i) issue(i);

  // this lane's two query rows: first operand fragments and last visible key
  const int row0 = rg * 16 + (lane >> 2);
  uint32_t qf[D / 16][4];
  int last[2];
  size_t score_row[2] = {0, 0};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int m = row0 + 8 * x;
    last[x] = -1;
    const uint32_t* src = nullptr;
    if (m < rows_total) {
      const int bb = prefix ? m / p.R : b;
      const int r = prefix ? m - bb * p.R : m;
      const int g = r / p.Nq, i = r - g * p.Nq;
      src = reinterpret_cast<const uint32_t*>(p.q + ((size_t)(bb * p.Hq + hkv * p.G + g) * p.Nq + i) * D) + (lane & 3);
      const int nb = prefix ? cache_len(p, bb) : len;
      last[x] = len - 1;
      if (nb < 0) last[x] = -1;
      else if (p.causal) last[x] = (int)min((long long)len - 1, (long long)nb - p.Nq + i + (prefix ? p.Np : 0));
      score_row[x] = ((size_t)(b * p.Hkv + hkv) * p.R + r) * p.cap_pad;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[ks][x] = src ? src[ks * 8] : 0u;
      qf[ks][2 + x] = src ? src[ks * 8 + 4] : 0u;
    }
  }

  const WaitCtx wc{abort_flag, p.err, p.wait_cap};
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  bool ok = true;
  int done = 0;
  for (int i = 0; i < n_mine; ++i) {
    const int st = i % C::ST;
    if (!mbar_wait_warp(bars + 8 * st, (i / C::ST) & 1, wc, 21)) { ok = false; break; }
    done = i + 1;
    const int key0 = k0 + (warp + C::W * i) * C::CH;
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
    if (p.scores && !prefix) {
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
    if (lane == 0 && i + C::ST < n_mine) issue(i + C::ST);
  }
  // a warp that gave up waits for its own copies in flight
  if (!ok && lane == 0)
    for (int i = done; i < n_mine && i < done + C::ST; ++i)
      mbar_wait_inflight(bars + 8 * (i % C::ST), (i / C::ST) & 1, wc, 22);

  // merge the warps: m, l and O of every row through shared memory
  float* ml = reinterpret_cast<float*>(smem + C::ML_OFF);
  float* red = reinterpret_cast<float*>(smem);  // [W][16][D], over the ring
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    if ((lane & 3) == 0) {
      ml[(warp * 16 + (lane >> 2) + 8 * x) * 2] = m_ref[x];
      ml[(warp * 16 + (lane >> 2) + 8 * x) * 2 + 1] = l[x];
    }
  }
  __syncthreads();  // every warp has read its last stage
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x)
      *reinterpret_cast<float2*>(red + ((size_t)warp * 16 + (lane >> 2) + 8 * x) * D + n * 8 + 2 * (lane & 3)) =
          make_float2(o[n][2 * x], o[n][2 * x + 1]);
  __syncthreads();
  if (*abort_flag) return;
  const int rows = min(16, rows_total - rg * 16);
  const size_t slot0 = prefix ? ((size_t)split * p.Hkv + hkv) * p.M + rg * 16
                              : (size_t)p.n_split_p * p.Hkv * p.M +
                                    (((size_t)split * p.B + b) * p.Hkv + hkv) * p.R + rg * 16;
  for (int e = threadIdx.x; e < rows * (D / 4); e += C::THREADS) {
    const int r = e / (D / 4), c = e - r * (D / 4);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::W; ++w) M = fmaxf(M, ml[(w * 16 + r) * 2]);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < C::W; ++w) {
      const float mw = ml[(w * 16 + r) * 2];
      const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
      const float4 v = reinterpret_cast<const float4*>(red + ((size_t)w * 16 + r) * D)[c];
      L = fmaf(f, ml[(w * 16 + r) * 2 + 1], L);
      sum.x = fmaf(f, v.x, sum.x);
      sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z);
      sum.w = fmaf(f, v.w, sum.w);
    }
    reinterpret_cast<float4*>(p.part_o + (slot0 + r) * D)[c] = sum;
    if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (slot0 + r) * 2) = make_float2(M, L);
  }
}

// Where the partial results of one query row lie, and how many there are.
struct CacheParts {
  size_t prefix0, prefix_step, own0, own_step;
  int n_prefix, n;
  __device__ size_t slot(int s) const {
    return s < n_prefix ? prefix0 + s * prefix_step : own0 + (size_t)(s - n_prefix) * own_step;
  }
};
__device__ __forceinline__ CacheParts cache_parts(const CacheParams& p, int b, int hkv, int r, int len) {
  CacheParts c;
  c.prefix0 = (size_t)hkv * p.M + (size_t)b * p.R + r;
  c.prefix_step = (size_t)p.Hkv * p.M;
  c.own0 = (size_t)p.n_split_p * p.Hkv * p.M + ((size_t)b * p.Hkv + hkv) * p.R + r;
  c.own_step = (size_t)p.B * p.Hkv * p.R;
  c.n_prefix = p.n_split_p;
  c.n = p.n_split_p + (len + p.kps_o - 1) / p.kps_o;
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

// O and LSE of one query row a warp.  A row that no key is visible to has
// O = 0 and LSE = −inf.
template <int D>
__global__ void __launch_bounds__(256) fa_cache_combine_kernel(const CacheParams p) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)p.B * p.Hq * p.Nq) return;
  const int i = (int)(row % p.Nq);
  const int h = (int)(row / p.Nq % p.Hq);
  const int b = (int)(row / ((long long)p.Nq * p.Hq));
  const int len = cache_len(p, b);
  if (len < 0) {
    if (lane == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return;
  }
  const CacheParts parts = cache_parts(p, b, h / p.G, (h % p.G) * p.Nq + i, len);
  float M = -INFINITY;
  for (int s = lane; s < parts.n; s += 32) M = fmaxf(M, p.part_ml[parts.slot(s) * 2]);
  M = warp_max(M);
  constexpr int V = D / 32;  // columns of a lane
  float acc[V], L = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
  for (int s0 = 0; s0 < parts.n; s0 += 32) {
    float f = 0.f;
    if (s0 + lane < parts.n) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + parts.slot(s0 + lane) * 2);
      if (ml.x != -INFINITY) f = ex2(ml.x - M);
      L = fmaf(f, ml.y, L);
    }
    const int cnt = min(32, parts.n - s0);
#pragma unroll 4
    for (int t = 0; t < cnt; ++t) {
      const float ft = __shfl_sync(0xffffffffu, f, t);
      const float* src = p.part_o + parts.slot(s0 + t) * D + lane * V;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(ft, src[c], acc[c]);
    }
  }
  L = warp_sum(L);
  const float inv = L > 0.f ? 1.f / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (size_t)row * D + lane * V);
#pragma unroll
  for (int c = 0; c < V; c += 2) dst[c / 2] = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0) p.lse[row] = L > 0.f ? (M + lg2(L)) * kLn2 : -INFINITY;
}

// weights_out[j] = weights[j] + Σ_r 2^(S'_rj − LSE'_r); keys at or behind the
// sequence's length keep their weight.  One CTA per (sequence, kv head, 1024
// keys), rows taken 64 at a time.
__global__ void __launch_bounds__(256) fa_cache_weights_kernel(const CacheParams p) {
  __shared__ float lse2[64];
  const int unit = blockIdx.y, b = unit / p.Hkv, hkv = unit % p.Hkv;
  const int len = cache_len(p, b);
  if (len < 0) {  // this sequence's weights stay as they are
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return;
  }
  const int j0 = blockIdx.x * 1024;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < p.R && j0 < len; r0 += 64) {
    __syncthreads();
    for (int r = r0 + (threadIdx.x >> 5); r < min(p.R, r0 + 64); r += 8) {
      const int lane = threadIdx.x & 31;
      const CacheParts parts = cache_parts(p, b, hkv, r, len);
      float M = -INFINITY, L = 0.f;
      for (int s = lane; s < parts.n; s += 32) M = fmaxf(M, p.part_ml[parts.slot(s) * 2]);
      M = warp_max(M);
      for (int s = lane; s < parts.n; s += 32) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + parts.slot(s) * 2);
        if (ml.x != -INFINITY) L = fmaf(ex2(ml.x - M), ml.y, L);
      }
      L = warp_sum(L);
      // a row without a visible key gives no weight (its scores are −inf)
      if (lane == 0) lse2[r - r0] = L > 0.f ? M + lg2(L) : INFINITY;
    }
    __syncthreads();
    const float* src = p.scores + ((size_t)unit * p.R + r0) * p.cap_pad + j0 + threadIdx.x;
    for (int r = 0; r < min(64, p.R - r0); ++r)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (j0 + threadIdx.x + 256 * t < len) acc[t] += ex2(src[(size_t)r * p.cap_pad + 256 * t] - lse2[r]);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = j0 + threadIdx.x + 256 * t;
    if (j >= p.Ncap) continue;
    const size_t at = (size_t)unit * p.Ncap + j;
    const float w = p.weights ? p.weights[at] : 0.f;
    p.weights_out[at] = j < len ? w + acc[t] : w;
  }
}

}  // namespace fa
