// Eviction from a key/value cache by accumulated attention weight.
//
// Of the n keys of a sequence, count = min(n, budget) stay: where n > budget,
// the last `recent` ones and, of the others, the budget − recent of greatest
// weight (equal weights: the lower index; NaN counts as the least).  They keep
// their order.
//
//   fa_evict_select_kernel  writes the kept indices: radix select of the
//                           threshold (11, 11 and 10 bits of the weights as
//                           ordered integers), then one pass that numbers what
//                           is kept
//   fa_evict_copy_kernel    gathers K, V and the weights; bound by HBM
//   fa_evict_kernel         both, for small caches
//
// The selection of a (sequence, kv head) is one cluster of CTAs: each counts its
// share of the weights, and the counts are added up in the first CTA through
// distributed shared memory (only bins that hold something are sent).  A share
// of up to 8192 weights is read once and stays in registers; larger ones are
// read four times.
//
// Measured, 4 x 8 x 65536 weights cut to 8192 (d = 128): copy 43 us, 6.4 TB/s of kept
// rows read and written; selection 21 to 30 us.  Of that, 13 us are what a CTA does
// with its 8192 weights (16 x 8 x 8192, no cluster: 13 to 14 us, whether they are all
// equal or spread evenly over the bins, so it is not the atomic additions that
// bound it; 40 % of the issue slots are used), and the rest are the cluster's
// barriers and the bins sent: 21 us where all weights are equal, 22 where they
// spread over a few powers of two, 27 over all, 30 where they are uniform in 0 .. 1.
#pragma once

#include "sm100.cuh"

namespace fa {

struct EvictParams {
  const __nv_bfloat16 *k, *v;  // [B, Hkv, Ncap, d]
  const float* weights;        // [B, Hkv, Ncap]
  const int* lengths;          // [B], or null: every cache is full
  __nv_bfloat16 *k_out, *v_out;  // [B, Hkv, out_cap, d]
  float* weights_out;            // [B, Hkv, out_cap]
  int* index;                    // [B, Hkv, out_cap]
  int* lengths_out;              // [B]
  int B, Hkv, Ncap, out_cap, budget, recent;
  int* err;
};

// Unsigned integer with the order of the float: −0 and 0 are equal, NaN is the
// least.
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0u;
  if ((u << 1) == 0u) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.lengths ? p.lengths[b] : p.Ncap;
  return (n < 0 || n > p.Ncap) ? -1 : n;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void add_cluster(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

constexpr int kEvictThreads = 512;
constexpr int kEvictBins = 2048;
constexpr int kEvictBatch = 4 * kEvictThreads;  // weights of a batch: four in a row a thread
constexpr int kEvictHeld = 4;                   // batches that a CTA can hold in registers

// Inclusive sum over the CTA's threads in order; `tot` is shared scratch of one
// int a warp.  Ends with a barrier.
__device__ __forceinline__ int cta_scan(int x, int* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) tot[warp] = x;
  __syncthreads();
  int before = lane < kEvictThreads / 32 ? tot[lane] : 0;
#pragma unroll
  for (int off = 1; off < kEvictThreads / 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += y;
  }
  before = __shfl_sync(0xffffffffu, before, max(warp - 1, 0));
  __syncthreads();
  return (warp ? before : 0) + x;
}

struct EvictShared {
  int hist[kEvictBins];    // of this CTA
  int acc[2][kEvictBins];  // of the cluster, in its first CTA; passes alternate
  int tot[kEvictThreads / 32];
  int result[2];  // in the first CTA: the threshold's bin, how many are above it
  int both;
  int kept[2];  // of this CTA: greater than the threshold, equal to it
};

// Chooses need of the weights w[0 .. nc), of which this CTA has w[j0 .. j1), and
// writes their indices in order.  HELD: the CTA's share stays in registers.
template <bool HELD>
__device__ __forceinline__ void evict_select(EvictShared& sh, const float* w, int* index, int need, int j0, int j1,
                                             int rank, int nrank) {
  const int tid = threadIdx.x;
  const int batches = (j1 - j0 + kEvictBatch - 1) / kEvictBatch;
  uint32_t held[HELD ? kEvictHeld * 4 : 4];
  auto load = [&](int bt, uint32_t* u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + bt * kEvictBatch + 4 * tid + i;
      u[i] = j < j1 ? ordered_bits(w[j]) : 0u;
    }
  };
  if (HELD)
#pragma unroll
    for (int bt = 0; bt < kEvictHeld; ++bt) load(bt, held + 4 * bt);
  // calls f(batch, its four values) in order
  auto each = [&](auto f) {
    if (HELD) {
#pragma unroll
      for (int bt = 0; bt < kEvictHeld; ++bt)
        if (bt < batches) f(bt, held + 4 * bt);
    } else {
#pragma unroll 1
      for (int bt = 0; bt < batches; ++bt) {
        load(bt, held);
        f(bt, held);
      }
    }
  };

  // threshold T: the need-th greatest
  constexpr int PER = kEvictBins / kEvictThreads;
  uint32_t prefix = 0;
  int above = 0;          // greater than every value with this prefix
  int gt = 0, eq = 0;     // of this thread's bins: greater than the threshold, equal to it
  for (int e = tid; e < kEvictBins; e += kEvictThreads) sh.acc[0][e] = 0;
  if (nrank > 1) cluster_sync();  // every CTA has started, and the sums are clear
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    for (int e = tid; e < kEvictBins; e += kEvictThreads) {
      sh.hist[e] = 0;
      sh.acc[(pass + 1) & 1][e] = 0;  // the next pass's; cleared before its first addition by two cluster barriers
    }
    __syncthreads();
    each([&](int bt, const uint32_t* u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j0 + bt * kEvictBatch + 4 * tid + i < j1 && (pass == 0 || (u[i] >> (shift + bits)) == prefix))
          atomicAdd(&sh.hist[(u[i] >> shift) & ((1 << bits) - 1)], 1);
    });
    __syncthreads();
    // thread t has bins 2047 − 4t .. 2044 − 4t; the CTAs add theirs up in the first
    int mine[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) mine[i] = sh.hist[kEvictBins - 1 - PER * tid - i];
    if (nrank > 1) {
      const uint32_t base = mapa_shared(smem_u32(sh.acc[pass & 1]), 0);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (mine[i]) add_cluster(base + 4 * (kEvictBins - 1 - PER * tid - i), mine[i]);
      cluster_sync();
    }
    if (rank == 0) {
      const int* h = nrank > 1 ? sh.acc[pass & 1] : sh.hist;
      int c[PER], x = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) x += c[i] = h[kEvictBins - 1 - PER * tid - i];
      int before = above + cta_scan(x, sh.tot) - x;  // greater than this thread's bins
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (before < need && before + c[i] >= need) {
          sh.result[0] = kEvictBins - 1 - PER * tid - i;
          sh.result[1] = before;
        }
        before += c[i];
      }
    }
    int bin;
    if (nrank > 1) {
      cluster_sync();
      const uint32_t base = mapa_shared(smem_u32(sh.result), 0);
      bin = ld_cluster(base);
      above = ld_cluster(base + 4);
    } else {
      __syncthreads();
      bin = sh.result[0];
      above = sh.result[1];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = kEvictBins - 1 - PER * tid - i;
      if (e > bin) gt += mine[i];
      if (e == bin && pass == 2) eq = mine[i];
    }
    prefix = (prefix << bits) | (uint32_t)bin;
  }
  const uint32_t T = prefix;
  const int eq_need = need - above;  // of those equal to T, the first so many stay

  // how many of each kind lie before this CTA's share
  int gt0 = 0, eq0 = 0;
  if (nrank > 1) {
    gt = cta_scan(gt, sh.tot);
    eq = cta_scan(eq, sh.tot);
    if (tid == kEvictThreads - 1) {
      sh.kept[0] = gt;
      sh.kept[1] = eq;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      const uint32_t base = mapa_shared(smem_u32(sh.kept), r);
      gt0 += ld_cluster(base);
      eq0 += ld_cluster(base + 4);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }

  // number what is kept, in order
  each([&](int bt, const uint32_t* u) {
    const int j = j0 + bt * kEvictBatch + 4 * tid;
    int g = 0, e = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g += j + i < j1 && u[i] > T;
      e += j + i < j1 && u[i] == T;
    }
    // at most kEvictBatch of each kind: both sums in one scan
    const int both = cta_scan(g | e << 16, sh.tot);
    int gb = gt0 + (both & 0xffff) - g, eb = eq0 + (both >> 16) - e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (j + i < j1 && u[i] > T) {
        index[gb + min(eb, eq_need)] = j + i;
        ++gb;
      } else if (j + i < j1 && u[i] == T) {
        if (eb < eq_need) index[gb + eb] = j + i;
        ++eb;
      }
    }
    if (bt + 1 < batches) {
      if (tid == kEvictThreads - 1) sh.both = both;
      __syncthreads();
      gt0 += sh.both & 0xffff;
      eq0 += sh.both >> 16;
    }
  });
}

// Writes the kept indices of one (sequence, kv head), of whose candidates this
// CTA, `rank` of a cluster of `nrank`, owns its share.  False (for the whole
// cluster) where the length is out of range and nothing is written.
__device__ __forceinline__ bool evict_choose(const EvictParams& p, EvictShared& sh, int unit, int rank, int nrank) {
  const int b = unit / p.Hkv;
  const int n = evict_len(p, b);
  if (n < 0) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return false;
  }
  int* index = p.index + (size_t)unit * p.out_cap;
  const int count = min(n, p.budget);
  const int all = nrank * kEvictThreads, gid = rank * kEvictThreads + threadIdx.x;
  for (int j = count + gid; j < p.budget; j += all) index[j] = -1;
  if (unit % p.Hkv == 0 && gid == 0) p.lengths_out[b] = count;
  if (n <= p.budget) {
    for (int j = gid; j < n; j += all) index[j] = j;
    return true;
  }
  const int nc = n - p.recent, need = p.budget - p.recent;  // candidates, and how many of them stay
  for (int j = gid; j < p.recent; j += all) index[need + j] = nc + j;
  if (need == 0) return true;
  const float* w = p.weights + (size_t)unit * p.Ncap;
  const int share = (nc + nrank - 1) / nrank;
  const int j0 = min(nc, rank * share), j1 = min(nc, j0 + share);
  if (share <= kEvictHeld * kEvictBatch) evict_select<true>(sh, w, index, need, j0, j1, rank, nrank);
  else evict_select<false>(sh, w, index, need, j0, j1, rank, nrank);
  return true;
}

// Slots r0 .. r1−1 of one (sequence, kv head) by the whole CTA.  One thread moves
// 16 bytes of K and of V at a time; slots count .. budget−1 are set to zero.
template <int D>
__device__ __forceinline__ void evict_copy(const EvictParams& p, int unit, int r0, int r1) {
  constexpr int CPR = D / 8;  // 16-byte chunks of a row
  const size_t in0 = (size_t)unit * p.Ncap, out0 = (size_t)unit * p.out_cap;
  const uint4 *k = reinterpret_cast<const uint4*>(p.k), *v = reinterpret_cast<const uint4*>(p.v);
  uint4 *ko = reinterpret_cast<uint4*>(p.k_out), *vo = reinterpret_cast<uint4*>(p.v_out);
  for (int e = threadIdx.x; e < (r1 - r0) * CPR; e += blockDim.x) {
    const int r = r0 + e / CPR, c = e % CPR;
    const int src = p.index[out0 + r];
    uint4 a = make_uint4(0, 0, 0, 0), bb = a;
    if (src >= 0) {
      a = k[(in0 + src) * CPR + c];
      bb = v[(in0 + src) * CPR + c];
    }
    ko[(out0 + r) * CPR + c] = a;
    vo[(out0 + r) * CPR + c] = bb;
    if (c == 0) p.weights_out[out0 + r] = src >= 0 ? p.weights[in0 + src] : 0.f;
  }
}

// Grid: units · cluster size.
__global__ void __launch_bounds__(kEvictThreads) fa_evict_select_kernel(const EvictParams p, int nrank) {
  __shared__ EvictShared sh;
  evict_choose(p, sh, blockIdx.x / nrank, blockIdx.x % nrank, nrank);
}

constexpr int kEvictCopyRows = 32;  // slots of a CTA
template <int D>
__global__ void __launch_bounds__(256) fa_evict_copy_kernel(const EvictParams p) {
  const int unit = blockIdx.y;
  if (evict_len(p, unit / p.Hkv) < 0) return;
  const int r0 = blockIdx.x * kEvictCopyRows;
  evict_copy<D>(p, unit, r0, min(p.budget, r0 + kEvictCopyRows));
}

// Both in one launch, a CTA for each (sequence, kv head).
template <int D>
__global__ void __launch_bounds__(kEvictThreads) fa_evict_kernel(const EvictParams p) {
  __shared__ EvictShared sh;
  if (!evict_choose(p, sh, blockIdx.x, 0, 1)) return;
  __syncthreads();
  evict_copy<D>(p, blockIdx.x, 0, p.budget);
}

}  // namespace fa
