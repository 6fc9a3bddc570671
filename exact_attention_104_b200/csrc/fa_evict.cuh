// Eviction from a key/value cache by accumulated attention weight.
//
// Of the n keys of a sequence, count = min(n, budget) stay: where n > budget,
// the last `recent` ones and, of the others, the budget − recent of greatest
// weight (equal weights: the lower index; NaN counts as the least).  They keep
// their order.
//
//   fa_evict_select_kernel  writes the kept indices: radix select of the
//                           threshold (11, 11 and 10 bits of the weights as
//                           ordered integers), then one ordered pass that
//                           numbers what is kept
//   fa_evict_copy_kernel    gathers K, V and the weights; bound by HBM
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

constexpr int kEvictThreads = 1024;

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.lengths ? p.lengths[b] : p.Ncap;
  return (n < 0 || n > p.Ncap) ? -1 : n;
}

__global__ void __launch_bounds__(kEvictThreads) fa_evict_select_kernel(const EvictParams p) {
  __shared__ int hist[2048];
  __shared__ int warp_tot[32];
  __shared__ int sh_bin, sh_above;
  const int unit = blockIdx.x, b = unit / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = evict_len(p, b);
  if (n < 0) {  // nothing of this sequence is written
    if (tid == 0) atomicCAS(p.err, 0, kDevBadSeqlens);
    return;
  }
  int* index = p.index + (size_t)unit * p.out_cap;
  const int count = min(n, p.budget);
  for (int j = count + tid; j < p.budget; j += kEvictThreads) index[j] = -1;
  if (unit % p.Hkv == 0 && tid == 0) p.lengths_out[b] = count;
  if (n <= p.budget) {
    for (int j = tid; j < n; j += kEvictThreads) index[j] = j;
    return;
  }
  const int nc = n - p.recent, need = p.budget - p.recent;  // candidates, and how many of them stay
  for (int j = tid; j < p.recent; j += kEvictThreads) index[need + j] = nc + j;
  if (need == 0) return;
  const float* w = p.weights + (size_t)unit * p.Ncap;

  // threshold T: the need-th greatest of the candidates
  uint32_t prefix = 0;
  int above = 0;  // candidates greater than every value with this prefix
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    for (int e = tid; e < 2048; e += kEvictThreads) hist[e] = 0;
    __syncthreads();
    for (int j = tid; j < nc; j += kEvictThreads) {
      const uint32_t u = ordered_bits(w[j]);
      if (pass == 0 || (u >> (shift + bits)) == prefix) atomicAdd(&hist[(u >> shift) & ((1 << bits) - 1)], 1);
    }
    __syncthreads();
    // counts from the top: thread t owns bins 2047 − 2t and 2046 − 2t
    const int c0 = hist[2047 - 2 * tid], c1 = hist[2046 - 2 * tid];
    int x = c0 + c1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int t = warp_tot[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) t += y;
      }
      warp_tot[lane] = t;
    }
    __syncthreads();
    const int before = above + (warp ? warp_tot[warp - 1] : 0) + x - c0 - c1;  // greater than my two bins
    if (before < need && before + c0 >= need) {
      sh_bin = 2047 - 2 * tid;
      sh_above = before;
    } else if (before + c0 < need && before + c0 + c1 >= need) {
      sh_bin = 2046 - 2 * tid;
      sh_above = before + c0;
    }
    __syncthreads();
    prefix = (prefix << bits) | (uint32_t)sh_bin;
    above = sh_above;
    __syncthreads();
  }
  const uint32_t T = prefix;
  const int eq_need = need - above;  // of those equal to T, the first so many stay

  // one pass in order: number what is kept
  int gt0 = 0, eq0 = 0;
  for (int j0 = 0; j0 < nc; j0 += kEvictThreads) {
    const int j = j0 + tid;
    const uint32_t u = j < nc ? ordered_bits(w[j]) : 0u;
    const bool gt = j < nc && u > T, eq = j < nc && u == T;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) warp_tot[warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();
    int gt_before = gt0, eq_before = eq0, gt_all = 0, eq_all = 0;
    for (int t = 0; t < 32; ++t) {
      const int c = warp_tot[t];
      if (t < warp) {
        gt_before += c & 0xffff;
        eq_before += c >> 16;
      }
      gt_all += c & 0xffff;
      eq_all += c >> 16;
    }
    gt_before += __popc(bg & ((1u << lane) - 1));
    eq_before += __popc(be & ((1u << lane) - 1));
    if (gt || (eq && eq_before < eq_need)) index[gt_before + min(eq_before, eq_need)] = j;
    gt0 += gt_all;
    eq0 += eq_all;
    __syncthreads();
  }
}

// One thread moves 16 bytes of K and of V at a time; slots count .. budget−1
// are set to zero, those behind the budget stay as they are.
constexpr int kEvictCopyRows = 32;  // slots of a CTA
template <int D>
__global__ void __launch_bounds__(256) fa_evict_copy_kernel(const EvictParams p) {
  const int unit = blockIdx.y, b = unit / p.Hkv;
  const int n = evict_len(p, b);
  if (n < 0) return;
  constexpr int CPR = D / 8;  // 16-byte chunks of a row
  const int r0 = blockIdx.x * kEvictCopyRows, r1 = min(p.budget, r0 + kEvictCopyRows);
  const size_t in0 = (size_t)unit * p.Ncap, out0 = (size_t)unit * p.out_cap;
  const uint4 *k = reinterpret_cast<const uint4*>(p.k), *v = reinterpret_cast<const uint4*>(p.v);
  uint4 *ko = reinterpret_cast<uint4*>(p.k_out), *vo = reinterpret_cast<uint4*>(p.v_out);
  for (int e = threadIdx.x; e < (r1 - r0) * CPR; e += 256) {
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

}  // namespace fa
