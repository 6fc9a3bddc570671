// Host side of the cache operators: decoding for a batch that shares a prefix,
// decoding that accumulates the keys' attention weights, the same weights from
// a prompt's queries, and eviction by them.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_cache_attn.cuh"
#include "fa_cache_tc.cuh"
#include "fa_evict.cuh"
#include "fa_host.h"
#include "fa_key_weights.cuh"

using namespace fa_host;

cudaError_t fa_host::cache_check_word(int** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), g_fa_err);
}

namespace {

constexpr long long kIndexLimit = (1LL << 31) - 4096;  // row coordinates, with room for a box past the end

// Allows `kern` its dynamic shared memory, once per device.
template <class Kern>
fa_status allow_smem(Kern kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  const unsigned long long bit = 1ULL << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return FA_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  done.fetch_or(bit, std::memory_order_release);
  return FA_OK;
}

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Launch with leave to start before the kernel in front has finished (see
// grid_wait).
template <class... P, class... A>
fa_status launch_early(void (*kern)(P...), unsigned grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_CUDA;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// No output may overlap an input or another output.
template <int NI, int NO>
bool disjoint(const Range (&ins)[NI], const Range (&outs)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return false;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return false;
  }
  return true;
}

fa_status cache_sizes(int B, int Hq, int Hkv, int Nq, int Np, int Ncap, int d, float scale, bool* empty) {
  *empty = false;
  if (B < 0 || Nq < 0 || Np < 0 || Ncap < 0 || Hq <= 0 || Hkv <= 0 || d <= 0) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (Nq > 256) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Nq == 0) *empty = true;
  if (B > 65535 || Hq > 65535) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hq * Nq > kIndexLimit || (long long)B * Hkv * Ncap > kIndexLimit ||
      (long long)Hkv * Np > kIndexLimit || (long long)Np + Ncap > kIndexLimit)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// ------------------------------------------------------------ key weights
bool weights_sizes(int B, int Hkv, int Nk) {
  return (long long)B * Hkv <= 65535 && (long long)B * Hkv * (Nk + 255LL) <= kIndexLimit;
}
fa_status key_weights_sizes(int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale, bool* empty) {
  *empty = false;
  if (B < 0 || Nq < 0 || Nk < 0 || Hq <= 0 || Hkv <= 0 || d <= 0) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Nk == 0) {
    *empty = true;
    return FA_OK;
  }
  if (B > 65535 || Hq > 65535) return FA_ERR_UNSUPPORTED;
  if (Nq > 0 && (long long)B * Hq > kIndexLimit / Nq) return FA_ERR_UNSUPPORTED;
  if (!weights_sizes(B, Hkv, Nk)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Pure functions of the sizes, so that the workspace sizes need no device.
constexpr int kKeyWCtas = 148;
struct KeyWPlan {
  bool resident;
  int keys, units, row_tiles;  // keys of a unit
  size_t part_bytes, range_bytes, present_bytes;
  size_t total() const { return part_bytes + range_bytes + present_bytes; }
};
template <class Res, class Str>
KeyWPlan key_weights_plan_of(int B, int Hq, int Hkv, int Nq, int Nk) {
  KeyWPlan pl;
  pl.row_tiles = (int)(((long long)(Hq / Hkv) * Nq + Res::BN - 1) / Res::BN);
  pl.resident = pl.row_tiles <= Res::NRES;
  pl.keys = pl.resident ? Res::KEYS : Str::KEYS;
  pl.units = (Nk + pl.keys - 1) / pl.keys;
  const size_t units = (size_t)B * Hkv * pl.units;
  pl.part_bytes = round256((units + kKeyWCtas) * Res::NWG * pl.keys * 4);
  pl.range_bytes = round256(units * sizeof(int2));
  pl.present_bytes = round256(units + kKeyWCtas);
  return pl;
}
KeyWPlan key_weights_plan(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  switch (d) {
    case 64: return key_weights_plan_of<fa::KeyWCfg<64, true>, fa::KeyWCfg<64, false>>(B, Hq, Hkv, Nq, Nk);
    case 128: return key_weights_plan_of<fa::KeyWCfg<128, true>, fa::KeyWCfg<128, false>>(B, Hq, Hkv, Nq, Nk);
    default: return key_weights_plan_of<fa::KeyWCfg<256, true>, fa::KeyWCfg<256, false>>(B, Hq, Hkv, Nq, Nk);
  }
}

template <int D, bool RESIDENT>
fa_status launch_key_weights(const void* q, const void* k, const fa::KeyWParams& p, cudaStream_t s) {
  using C = fa::KeyWCfg<D, RESIDENT>;
  CUtensorMap tq{}, tk{};
  if (!make_map(&tk, k, (uint64_t)p.B * p.Hkv * p.Ncap, D, 128)) return FA_ERR_CUDA;
  if (p.Nq > 0 && !make_map(&tq, q, (uint64_t)p.B * p.Hq * p.Nq, D, C::BN)) return FA_ERR_CUDA;
  auto kern = fa::fa_key_weights_kernel<D, RESIDENT>;
  static std::atomic<unsigned long long> allowed{0};
  const fa_status st = allow_smem(kern, C::SMEM_BYTES, allowed);
  if (st != FA_OK) return st;
  kern<<<(unsigned)p.n_ctas, C::THREADS, C::SMEM_BYTES, s>>>(tq, tk, p);
  if (launched() != FA_OK) return FA_ERR_CUDA;
  fa::fa_key_weights_reduce_kernel<C>
      <<<dim3((unsigned)((p.Ncap + 255) / 256), (unsigned)(p.B * p.Hkv)), 256, 0, s>>>(p);
  return launched();
}
template <int D>
fa_status launch_key_weights(const void* q, const void* k, const fa::KeyWParams& p, bool resident, cudaStream_t s) {
  return resident ? launch_key_weights<D, true>(q, k, p, s) : launch_key_weights<D, false>(q, k, p, s);
}

// The arguments are checked, the workspace is large enough.
fa_status key_weights_run(const void* q, const void* k, const float* lse, const int* lengths, const float* weights,
                          float* weights_out, int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                          void* workspace, int* err, cudaStream_t s) {
  const KeyWPlan pl = key_weights_plan(B, Hq, Hkv, Nq, Nk, d);
  fa::KeyWParams p{};
  p.lse = lse;
  p.lengths = lengths;
  p.weights = weights;
  p.weights_out = weights_out;
  p.part = static_cast<float*>(workspace);
  p.range = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + pl.part_bytes);
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.Nq = Nq;
  p.Ncap = Nk;
  p.present = static_cast<uint8_t*>(workspace) + pl.part_bytes + pl.range_bytes;
  p.units = pl.units;
  p.row_tiles = pl.row_tiles;
  p.n_ctas = kKeyWCtas;
  p.causal = causal != 0;
  p.scale_log2 = scale * fa::kLog2e;
  p.wait_cap = g_wait_cap.load(std::memory_order_relaxed);
  p.err = err;
  switch (d) {
    case 64: return launch_key_weights<64>(q, k, p, pl.resident, s);
    case 128: return launch_key_weights<128>(q, k, p, pl.resident, s);
    default: return launch_key_weights<256>(q, k, p, pl.resident, s);
  }
}

// ------------------------------------------------------- decoding, weights
// Up to 16 query rows against one run of keys go to fa_cache_split_kernel, whose
// tile is 16 rows; more to fa_cache_tc_kernel.  A pure function of the sizes, so
// that the workspace sizes need no device.
constexpr int kWarpRows = 16;
constexpr int kSms = 148;
struct CachePlan {
  bool tc_p = false, tc_o = false, scores = false, key_weights = false;
  int units_w = 0, units_t = 0, ctas_w = 0;
  size_t w_o = 0, w_ml = 0, w_range = 0, t_o = 0, t_ml = 0, t_range = 0, score_off = 0, keyw_off = 0, bytes = 0;
};

CachePlan cache_plan(int B, int Hq, int Hkv, int Nq, int Np, int Ncap, int d, bool weights) {
  CachePlan pl;
  const long long R = (long long)(Hq / Hkv) * Nq, M = B * R;
  pl.tc_p = M > kWarpRows;
  pl.tc_o = R > kWarpRows;
  const long long units_p = Np > 0 ? Hkv * ((M + (pl.tc_p ? 127 : 15)) / (pl.tc_p ? 128 : 16)) : 0;
  const long long units_o = Ncap > 0 ? (long long)B * Hkv * ((R + (pl.tc_o ? 127 : 15)) / (pl.tc_o ? 128 : 16)) : 0;
  pl.units_t = (int)((pl.tc_p ? units_p : 0) + (pl.tc_o ? units_o : 0));
  pl.units_w = (int)((pl.tc_p ? 0 : units_p) + (pl.tc_o ? 0 : units_o));
  pl.ctas_w = kSms * (d == 64 ? fa::CacheCfg<64>::PER_SM : fa::CacheCfg<128>::PER_SM);  // as many as run at once
  auto take = [&](size_t bytes) {
    const size_t at = pl.bytes;
    pl.bytes += round256(bytes);
    return at;
  };
  if (pl.units_w > 0) {
    const size_t rows = ((size_t)pl.units_w + pl.ctas_w) * kWarpRows;
    pl.w_o = take(rows * d * 4);
    pl.w_ml = take(rows * 8);
    pl.w_range = take((size_t)pl.units_w * sizeof(int2));
  }
  if (pl.units_t > 0) {
    const size_t rows = ((size_t)pl.units_t + kSms) * 128;
    pl.t_o = take(rows * d * 4);
    pl.t_ml = take(rows * 8);
    pl.t_range = take((size_t)pl.units_t * sizeof(int2));
  }
  // Few rows: their scores are kept (4 bytes a row and key, written and read once)
  // and turned into weights by the kernel that joins the results.  Otherwise the keys
  // are read once more by the kernel for known LSE (2d bytes a key, and two launches).
  // With scores and with the second reading (us):
  //   up to 16 rows    205 and 307 (8 x 8 x 32768 keys, 4 rows, d 128), 248 and 307 (16
  //                    rows), 166 and 207 (16 rows, d 64): always scores
  //   17 to 64 rows    by what there is to store.  32 MB: d 64 47 to 80 and 45 to 78, d 128
  //                    55 to 88 and 57 to 90, d 256 82 to 127 and 86 to 135; 48 MB: d 64 76
  //                    and 55, d 128 78 and 68 (64 rows); 64 MB: d 256 125 and 127, 80 MB: 154
  //                    and 141
  //   96 rows          51 and 49 (4 x 2 x 10007 keys, 31 MB), but 25 and 31 with 2000 keys: the
  //                    joining kernel holds the LSE of kCacheScoreRows rows
  const size_t score_bytes = (size_t)B * Hkv * R * (((size_t)Ncap + 127) / 128 * 128) * 4;
  const size_t most = (size_t)(d == 256 ? 64 : 32) << 20;
  pl.scores = weights && (!pl.tc_o || (R <= fa::kCacheScoreRows && score_bytes <= most));
  pl.key_weights = weights && !pl.scores;
  if (pl.scores) pl.score_off = take(score_bytes);
  if (pl.key_weights) pl.keyw_off = take(key_weights_plan(B, Hq, Hkv, Nq, Ncap, d).total());
  return pl;
}

// How the two attention kernels divide the SMs when both run at once: the prefix's
// many rows take `n_ctas` of them, `split` CTAs a unit where its row tiles go in
// step (0: equal runs), the few rows of each sequence the rest.  Modelled time: the
// slower of the two, the prefix's from its key tiles and changes of unit in a CTA,
// the other's from its steps.  Measured SM time (us), kernels alone: a tile 1.3, 1.8,
// 3.2 (d = 64, 128, 256), a unit's start and end 4, 4, 6, a step 0.15, 0.28, 0.33.
// How full the caches are only the device knows: two thirds.
//
// The prefix has 28 SMs at least, which cost the other kernel nothing: 112 to 128 SMs
// read as much as HBM gives.  It leaves 16, for caches fuller than thought.  240
// sequences, 64 heads on 8, d 128, 128-key prefix, caches full to 1500 keys: 258 us
// with 8 SMs for the prefix, 246 with 28, 813 with 120.  160 such sequences, 20001
// keys, caches of 100: 244 us with 80 SMs, 178 with 132, 227 with 140.
//
// Several row tiles of a prefix read the same K and V: in step, L2 serves all but the
// first, and no CTA has more than one unit.  24 x 5 rows behind 20001 keys (d 256): 107
// us in step on 96 SMs for 133 in equal runs on 93; 48 x 5 behind 6000: 98 on 64 for
// 102 on 74.  The model has not that in it, so it may say up to a tenth more.  Beyond
// that, equal runs: 100 x 2 rows behind 4096 keys (d 128), 72 us on 76 SMs for 80 in
// step on 56 with caches two thirds full, but 90 for 80 with full ones.
struct CacheShare {
  int n_ctas, split;
};
CacheShare cache_share(int units, int unit_tiles, int row_tiles, long long steps, int d) {
  constexpr int kLeast = 28, kMost = kSms - 16;
  const double tile_us = d == 64 ? 1.3 : (d == 128 ? 1.8 : 3.2), unit_us = d == 256 ? 6 : 4;
  const double step_us = d == 64 ? 0.15 : (d == 128 ? 0.28 : 0.33);
  const long long tiles = (long long)units * unit_tiles;
  const double cost_t = tile_us * tiles + unit_us * units, cost_w = step_us * steps * 2 / 3;
  auto slower = [&](double prefix_us, int n) { return std::max(prefix_us, cost_w / (kSms - n)); };
  int n = std::min(kMost, std::max(kLeast, (int)(kSms * cost_t / (cost_t + cost_w) + 0.5)));
  n = (int)std::min<long long>(n, tiles);
  CacheShare share{n, 0};
  if (row_tiles > 1) {
    const long long run = (tiles + n - 1) / n;  // a CTA's tiles, of so many units at most:
    double best = 1.1 * slower(run * tile_us + ((run + unit_tiles - 2) / unit_tiles + 1) * unit_us, n);
    const int most = std::min(std::min(n / units + 1, unit_tiles), kMost / units);
    for (int split = std::max(1, n / units); split <= most; ++split) {
      const double us = slower((unit_tiles + split - 1) / split * tile_us + unit_us, split * units);
      if (us <= best) {
        best = us;
        share = CacheShare{split * units, split};
      }
    }
  }
  return share;
}

template <int D>
fa_status launch_cache(const CUtensorMap (&maps)[4], fa::CacheParams p, fa::CacheList lw, fa::CacheList lt,
                       bool tc_p, bool tc_o, cudaStream_t s) {
  using W = fa::CacheCfg<D>;
  using T = fa::CacheTcCfg<D>;
  lw.keys = W::CH;
  const bool have_w = lw.prefix_units + lw.own_rt > 0, have_t = lt.prefix_units + lt.own_rt > 0;
  auto tiles = [](const fa::CacheList& l, long long n) { return (n + l.keys - 1) / l.keys; };
  for (const fa::CacheList& l : {lw, lt})
    if (l.prefix_units * tiles(l, p.Np) + (long long)p.B * p.Hkv * l.own_rt * tiles(l, p.Ncap) >= (1LL << 31) - (1 << 20))
      return FA_ERR_UNSUPPORTED;
  if (have_w && have_t) {
    // The prefix's many rows and the few rows of each sequence: both kernels at
    // once, on SMs of their own, since one is bound by its softmax and the other
    // by reading keys.  The tcgen05 kernel goes first and fills its SMs' shared
    // memory; the split kernel, launched before that one ends, gets the others.
    // GPU time with caches full, two thirds and a tenth full, against one after the
    // other, each on all SMs (us): 47, 47, 41 and 59, 53, 41 (32 sequences behind 8192
    // keys, caches of 1024, d 128); 126, 109, 100 and 131, 119, 98 (24 x 5 rows behind
    // 20001, caches of 1500, d 256); 238, 174, 64 and 260, 190, 70 (240 behind 128,
    // caches of 1500, d 128).
    const CacheShare share = cache_share(lt.prefix_units, (int)tiles(lt, p.Np), lt.prefix_rt,
                                         (long long)p.B * p.Hkv * tiles(lw, p.Ncap), D);
    lt.n_ctas = share.n_ctas;
    lt.split = share.split;
    lw.n_ctas = (kSms - lt.n_ctas) * W::PER_SM;
  } else if (lt.prefix_rt > 1 && lt.own_rt == 0) {
    // the prefix alone: in step (see cache_share) where the same number of CTAs for
    // every unit uses nearly all CTAs
    const int split = lt.n_ctas / lt.prefix_units;
    if (10 * split * lt.prefix_units >= 9 * lt.n_ctas) lt.split = split;
  }
  if (have_t) {
    auto kern = fa::fa_cache_tc_kernel<D>;
    static std::atomic<unsigned long long> allowed{0};
    if (allow_smem(kern, T::SMEM_BYTES, allowed) != FA_OK) return FA_ERR_CUDA;
    kern<<<(unsigned)lt.n_ctas, T::THREADS, T::SMEM_BYTES, s>>>(maps[0], maps[1], maps[2], maps[3], p, lt);
    if (launched() != FA_OK) return FA_ERR_CUDA;
  }
  if (have_w) {
    auto kern = fa::fa_cache_split_kernel<D>;
    static std::atomic<unsigned long long> allowed{0};
    if (allow_smem(kern, W::SMEM_BYTES, allowed) != FA_OK) return FA_ERR_CUDA;
    if (have_t) {
      if (launch_early(kern, (unsigned)lw.n_ctas, W::THREADS, W::SMEM_BYTES, s, maps[0], maps[1], maps[2], maps[3], p,
                       lw) != FA_OK)
        return FA_ERR_CUDA;
    } else {
      kern<<<(unsigned)lw.n_ctas, W::THREADS, W::SMEM_BYTES, s>>>(maps[0], maps[1], maps[2], maps[3], p, lw);
      if (launched() != FA_OK) return FA_ERR_CUDA;
    }
  }
  const unsigned combine = (unsigned)(((long long)p.B * p.Hq * p.Nq + 7) / 8);
  // weights: 4 x 2 caches of 10007 keys, 64 rows: 22 us with 2048 keys a CTA, 11 with 256
  auto per_unit = [&](int keys) { return p.weights_out ? (unsigned)((p.Ncap + keys - 1) / keys) : 0u; };
  p.few = (unsigned)(p.B * p.Hkv) * per_unit(fa::kCacheWeightKeys) < 2 * kSms;
  const unsigned per = per_unit(p.few ? fa::kCacheWeightKeysFew : fa::kCacheWeightKeys);
  const unsigned ctas = combine + (unsigned)(p.B * p.Hkv) * per;
  if (ctas > 0) fa::fa_cache_finish_kernel<D><<<ctas, 256, 0, s>>>(p, tc_p ? lt : lw, tc_o ? lt : lw, combine);
  return launched();
}

// Shared by the two decoding calls; weights_out null for the prefix form.
fa_status cache_decode(const void* q, const void* kp, const void* vp, const void* k, const void* v,
                       const int* lengths, const float* weights, float* weights_out, void* o, float* lse, int B,
                       int Hq, int Hkv, int Nq, int Np, int Ncap, int d, int causal, float scale, void* workspace,
                       size_t workspace_bytes, cudaStream_t s) {
  const CachePlan pl = cache_plan(B, Hq, Hkv, Nq, Np, Ncap, d, weights_out != nullptr);
  if (!workspace || (Nq > 0 && (!q || !o || !lse || (Np > 0 && (!kp || !vp)) || (Ncap > 0 && (!k || !v)))))
    return FA_ERR_INVALID_ARG;
  for (const void* ptr : {q, kp, vp, k, v, (const void*)o, (const void*)lse})
    if (!aligned16(ptr)) return FA_ERR_INVALID_ARG;
  if (!aligned4(lengths) || !aligned4(weights) || !aligned4(weights_out)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < pl.bytes) return FA_ERR_INVALID_ARG;
  const size_t qbytes = (size_t)B * Hq * Nq * d * 2, lbytes = (size_t)B * Hq * Nq * 4;
  const size_t kvbytes = (size_t)B * Hkv * Ncap * d * 2, pbytes = (size_t)Hkv * Np * d * 2;
  const size_t wbytes = (size_t)B * Hkv * Ncap * 4;
  // weights_out may be weights itself
  const Range ins[7] = {span(q, qbytes),
                        span(kp, pbytes),
                        span(vp, pbytes),
                        span(k, kvbytes),
                        span(v, kvbytes),
                        span(lengths, lengths ? (size_t)B * 4 : 0),
                        span(weights, weights && weights != weights_out ? wbytes : 0)};
  const Range outs[4] = {span(o, qbytes), span(lse, lbytes), span(workspace, pl.bytes),
                         span(weights_out, weights_out ? wbytes : 0)};
  if (!disjoint(ins, outs)) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  const fa_status st = current_device(&di);
  if (st != FA_OK) return st;

  // boxes: the steps of the split kernel's warps, or 128 keys; the maps of an
  // absent cache are never read
  const int step = d == 256 ? fa::CacheCfg<256>::CH : fa::CacheCfg<128>::CH;
  CUtensorMap maps[4] = {};
  const uint64_t prows = (uint64_t)Hkv * Np, krows = (uint64_t)B * Hkv * Ncap;
  if (Nq > 0 && Np > 0)
    for (int i = 0; i < 2; ++i)
      if (!make_map(&maps[i], i ? vp : kp, prows, d, pl.tc_p ? 128 : step)) return FA_ERR_CUDA;
  if (Nq > 0 && Ncap > 0)
    for (int i = 0; i < 2; ++i)
      if (!make_map(&maps[2 + i], i ? v : k, krows, d, pl.tc_o ? 128 : step)) return FA_ERR_CUDA;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::CacheParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.lengths = lengths;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.scores = pl.scores ? reinterpret_cast<float*>(ws + pl.score_off) : nullptr;
  p.weights = weights;
  p.weights_out = pl.scores ? weights_out : nullptr;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.Nq = Nq;
  p.R = p.G * Nq;
  p.M = B * p.R;
  p.Np = Np;
  p.Ncap = Ncap;
  p.cap_pad = (int)pad128(Ncap);
  p.wide = Ncap % 4 == 0 && aligned16(weights) && aligned16(weights_out);
  p.causal = causal != 0;
  p.scale_log2 = scale * fa::kLog2e;
  p.wait_cap = g_wait_cap.load(std::memory_order_relaxed);
  p.err = di->err;
  fa::CacheList lw{}, lt{};
  lw.rows = kWarpRows;
  lw.n_ctas = pl.ctas_w;
  lw.part_o = reinterpret_cast<float*>(ws + pl.w_o);
  lw.part_ml = reinterpret_cast<float*>(ws + pl.w_ml);
  lw.range = reinterpret_cast<int2*>(ws + pl.w_range);
  lt.rows = lt.keys = 128;
  lt.n_ctas = kSms;
  lt.part_o = reinterpret_cast<float*>(ws + pl.t_o);
  lt.part_ml = reinterpret_cast<float*>(ws + pl.t_ml);
  lt.range = reinterpret_cast<int2*>(ws + pl.t_range);
  if (p.M > 0 && Np > 0) {
    fa::CacheList& l = pl.tc_p ? lt : lw;
    l.prefix_rt = (p.M + l.rows - 1) / l.rows;
    l.prefix_units = Hkv * l.prefix_rt;
  }
  if (p.R > 0 && Ncap > 0) {
    fa::CacheList& l = pl.tc_o ? lt : lw;
    l.own_rt = (p.R + l.rows - 1) / l.rows;
  }
  fa_status res;
  switch (d) {
    case 64: res = launch_cache<64>(maps, p, lw, lt, pl.tc_p, pl.tc_o, s); break;
    case 128: res = launch_cache<128>(maps, p, lw, lt, pl.tc_p, pl.tc_o, s); break;
    default: res = launch_cache<256>(maps, p, lw, lt, pl.tc_p, pl.tc_o, s); break;
  }
  if (res != FA_OK || !pl.key_weights || Ncap == 0) return res;
  return key_weights_run(q, k, lse, lengths, weights, weights_out, B, Hq, Hkv, Nq, Ncap, d, causal, scale,
                         ws + pl.keyw_off, di->err, s);
}

// CTAs of a cluster that selects for one (sequence, kv head): as few as can hold
// its weights in registers, 8 at most.  16 x 8 times 8192 weights: one CTA each
// 13 us, four 25 us; 4 x 8 times 65536 weights: eight 23 us, one 180 us.
fa_status evict_select(const fa::EvictParams& p, cudaStream_t s) {
  const long long units = (long long)p.B * p.Hkv;
  int nrank = 1;
  while (nrank < 8 && p.Ncap > fa::kEvictHeld * fa::kEvictBatch * nrank) nrank *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * nrank));
  cfg.blockDim = dim3(fa::kEvictThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = nrank;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fa::fa_evict_select_kernel, p, nrank) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_decode_prefix_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Np, int Ncap, int d) {
  bool empty = false;
  if (cache_sizes(B, Hq, Hkv, Nq, Np, Ncap, d, 1.f, &empty) != FA_OK) return 0;
  return empty ? 256 : std::max<size_t>(256, cache_plan(B, Hq, Hkv, Nq, Np, Ncap, d, false).bytes);
}

fa_status fa_fwd_decode_prefix(const void* q, const void* k_prefix, const void* v_prefix, const void* k,
                               const void* v, const int* lengths, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                               int Np, int Ncap, int d, int causal, float scale, void* workspace,
                               size_t workspace_bytes, void* stream) {
  bool empty = false;
  const fa_status st = cache_sizes(B, Hq, Hkv, Nq, Np, Ncap, d, scale, &empty);
  if (st != FA_OK || empty) return st;
  return cache_decode(q, k_prefix, v_prefix, k, v, lengths, nullptr, nullptr, o, lse, B, Hq, Hkv, Nq, Np, Ncap, d,
                      causal, scale, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

size_t fa_decode_weights_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  bool empty = false;
  if (cache_sizes(B, Hq, Hkv, Nq, 0, Nk, d, 1.f, &empty) != FA_OK) return 0;
  if (!weights_sizes(B, Hkv, Nk)) return 0;
  return empty ? 256 : std::max<size_t>(256, cache_plan(B, Hq, Hkv, Nq, 0, Nk, d, true).bytes);
}

fa_status fa_fwd_decode_weights(const void* q, const void* k, const void* v, const int* lengths, const float* weights,
                                float* weights_out, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                                int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty = false;
  const fa_status st = cache_sizes(B, Hq, Hkv, Nq, 0, Nk, d, scale, &empty);
  if (st != FA_OK || B == 0 || (Nq == 0 && Nk == 0)) return st;
  if (!weights_sizes(B, Hkv, Nk)) return FA_ERR_UNSUPPORTED;
  if (Nk > 0 && !weights_out) return FA_ERR_INVALID_ARG;
  return cache_decode(q, nullptr, nullptr, k, v, lengths, weights, weights_out, o, lse, B, Hq, Hkv, Nq, 0, Nk, d,
                      causal, scale, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

size_t fa_key_weights_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  bool empty = false;
  if (key_weights_sizes(B, Hq, Hkv, Nq, Nk, d, 1.f, &empty) != FA_OK) return 0;
  return empty ? 256 : key_weights_plan(B, Hq, Hkv, Nq, Nk, d).total();
}

fa_status fa_key_weights(const void* q, const void* k, const float* lse, const int* lengths, const float* weights,
                         float* weights_out, int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                         void* workspace, size_t workspace_bytes, void* stream) {
  bool empty = false;
  fa_status st = key_weights_sizes(B, Hq, Hkv, Nq, Nk, d, scale, &empty);
  if (st != FA_OK || empty) return st;
  const KeyWPlan pl = key_weights_plan(B, Hq, Hkv, Nq, Nk, d);
  if (!k || !weights_out || !workspace || (Nq > 0 && (!q || !lse))) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned4(lse) || !aligned4(lengths) || !aligned4(weights) ||
      !aligned4(weights_out))
    return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < pl.total())
    return FA_ERR_INVALID_ARG;
  const size_t wbytes = (size_t)B * Hkv * Nk * 4;
  const Range ins[5] = {span(q, (size_t)B * Hq * Nq * d * 2), span(k, (size_t)B * Hkv * Nk * d * 2),
                        span(lse, (size_t)B * Hq * Nq * 4), span(lengths, lengths ? (size_t)B * 4 : 0),
                        span(weights, weights && weights != weights_out ? wbytes : 0)};
  const Range outs[2] = {span(weights_out, wbytes), span(workspace, pl.total())};
  if (!disjoint(ins, outs)) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  st = current_device(&di);
  if (st != FA_OK) return st;
  return key_weights_run(q, k, lse, lengths, weights, weights_out, B, Hq, Hkv, Nq, Nk, d, causal, scale, workspace, di->err,
                         static_cast<cudaStream_t>(stream));
}

fa_status fa_selftest_cache_share(int B, int Hq, int Hkv, int Nq, int Np, int Ncap, int d, int* share) {
  bool empty = false;
  const fa_status st = cache_sizes(B, Hq, Hkv, Nq, Np, Ncap, d, 1.f, &empty);
  if (st != FA_OK) return st;
  if (!share) return FA_ERR_INVALID_ARG;
  share[0] = share[1] = 0;
  const CachePlan pl = cache_plan(B, Hq, Hkv, Nq, Np, Ncap, d, false);
  if (empty || pl.units_t == 0 || pl.units_w == 0) return FA_OK;
  const int rt = (int)(((long long)B * (Hq / Hkv) * Nq + 127) / 128);
  const int keys = d == 256 ? fa::CacheCfg<256>::CH : fa::CacheCfg<128>::CH;
  const CacheShare s = cache_share(Hkv * rt, (Np + 127) / 128, rt, (long long)B * Hkv * ((Ncap + keys - 1) / keys), d);
  share[0] = s.n_ctas;
  share[1] = s.split;
  return FA_OK;
}

fa_status fa_cache_evict(const void* k, const void* v, const float* weights, const int* lengths, void* k_out,
                         void* v_out, float* weights_out, int* index, int* lengths_out, int B, int Hkv, int Nk,
                         int out_cap, int budget, int recent, int d, void* stream) {
  if (B < 0 || Hkv <= 0 || Nk < 0 || d <= 0 || budget < 1 || recent < 0 || recent > budget || out_cap < budget)
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  if ((long long)B * Hkv > 65535 || (long long)B * Hkv * Nk > kIndexLimit ||
      (long long)B * Hkv * out_cap > kIndexLimit)
    return FA_ERR_UNSUPPORTED;
  if (!k_out || !v_out || !weights_out || !index || !lengths_out || (Nk > 0 && (!k || !v || !weights)))
    return FA_ERR_INVALID_ARG;
  for (const void* ptr : {k, v, (const void*)k_out, (const void*)v_out})
    if (!aligned16(ptr)) return FA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)weights, (const void*)lengths, (const void*)weights_out, (const void*)index,
                          (const void*)lengths_out})
    if (!aligned4(ptr)) return FA_ERR_INVALID_ARG;
  const size_t rows = (size_t)B * Hkv * Nk, orows = (size_t)B * Hkv * out_cap;
  const Range ins[4] = {span(k, rows * d * 2), span(v, rows * d * 2), span(weights, rows * 4),
                        span(lengths, lengths ? (size_t)B * 4 : 0)};
  const Range outs[5] = {span(k_out, orows * d * 2), span(v_out, orows * d * 2), span(weights_out, orows * 4),
                         span(index, orows * 4), span(lengths_out, (size_t)B * 4)};
  if (!disjoint(ins, outs)) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  const fa_status st = current_device(&di);
  if (st != FA_OK) return st;
  fa::EvictParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.weights = weights;
  p.lengths = lengths;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.weights_out = weights_out;
  p.index = index;
  p.lengths_out = lengths_out;
  p.B = B;
  p.Hkv = Hkv;
  p.Ncap = Nk;
  p.out_cap = out_cap;
  p.budget = budget;
  p.recent = recent;
  p.err = di->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned units = (unsigned)(B * Hkv);
  // small caches: one launch, whose one CTA a (sequence, kv head) copies too.  2 x
  // 1000 weights cut to 256 slots of 128 bytes: 23 us a call from Python for 27 with
  // two; 64 x 4000 cut to 500 of 256 bytes would take 19 us on the GPU for 14.
  if (Nk <= fa::kEvictHeld * fa::kEvictBatch && (long long)budget * d <= 1 << 15) {
    switch (d) {
      case 64: fa::fa_evict_kernel<64><<<units, fa::kEvictThreads, 0, s>>>(p); break;
      case 128: fa::fa_evict_kernel<128><<<units, fa::kEvictThreads, 0, s>>>(p); break;
      default: fa::fa_evict_kernel<256><<<units, fa::kEvictThreads, 0, s>>>(p); break;
    }
    return launched();
  }
  if (evict_select(p, s) != FA_OK) return FA_ERR_CUDA;
  const dim3 grid((unsigned)((budget + fa::kEvictCopyRows - 1) / fa::kEvictCopyRows), units);
  switch (d) {
    case 64: fa::fa_evict_copy_kernel<64><<<grid, 256, 0, s>>>(p); break;
    case 128: fa::fa_evict_copy_kernel<128><<<grid, 256, 0, s>>>(p); break;
    default: fa::fa_evict_copy_kernel<256><<<grid, 256, 0, s>>>(p); break;
  }
  return launched();
}

}  // extern "C"
