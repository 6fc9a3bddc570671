// Work lists of the cache attention kernels.
//
// Sequence b is the prefix (Np keys, the same for every b) followed by its own
// n_b = lengths[b] keys out of a cache with room for Ncap.  Query row i of Nq
// is position L_b − Nq + i of the L_b = Np + n_b long sequence:
//   S_j = s·q·k_j,  O = Σ_j 2^(S_j' − M) v_j / Σ_j 2^(S_j' − M)   (S' = S·log2 e)
// and the softmax over the concatenation is put together from parts: a run of
// keys gives its running maximum m, its normaliser l = Σ 2^(S' − m) and its
// unnormalised O, and
//   O = Σ_r 2^(m_r − M) O_r / Σ_r 2^(m_r − M) l_r.
// A run of the prefix serves the rows of ALL sequences (M = B·G·Nq rows of a kv
// head), a run of own keys the R = G·Nq rows of its sequence.
//
// A unit is a row tile against the prefix or against a sequence's own keys; the
// list holds the key tiles of all units in order, and every CTA takes an equal
// run of it: lengths that only the device knows leave no CTA idle.  Partial
// results of a unit in a CTA lie in slot (unit + CTA): from one pair to the next
// in the list one of the two grows, so every pair has a slot of its own.
#pragma once

#include "sm100.cuh"

namespace fa {

struct CacheParams {
  const __nv_bfloat16* q;  // [B, Hq, Nq, d]
  const int* lengths;      // [B], or null: every own cache is full
  __nv_bfloat16* o;        // [B, Hq, Nq, d]
  float* lse;              // [B, Hq, Nq]
  float* scores;           // [B·Hkv][R][cap_pad] scores in log2 units, or null
  const float* weights;    // [B, Hkv, Ncap] or null
  float* weights_out;
  int B, Hq, Hkv, G, Nq, R, M;  // R = G·Nq, M = B·R
  int Np, Ncap, cap_pad;        // cap_pad: Ncap rounded up to 128
  int wide;  // the weights can be moved 16 bytes at a time
  int few;   // fewer keys for each CTA that joins them
  int causal;
  float scale_log2;
  long long wait_cap;
  int* err;
};

// One kernel's list and where its partial results lie.
struct CacheList {
  int rows;          // rows of a row tile
  int keys;          // keys of a key tile
  int prefix_units;  // 0: the prefix is not in this list
  int prefix_rt;     // row tiles of the prefix's M rows
  int own_rt;        // row tiles of a sequence's R rows; 0: own keys are not in this list
  int n_ctas;
  int split;         // prefix only: CTAs a unit, so that the row tiles read the same keys at the same time; 0: equal runs
  float* part_o;     // [slots][rows][d]
  float* part_ml;    // [slots][rows][2]: m (log2 units), l
  int2* range;       // [units] first and last CTA
};

// Number of own keys of sequence b; −1 where lengths[b] breaks its rule.
__device__ __forceinline__ int cache_len(const CacheParams& p, int b) {
  if (!p.lengths) return p.Ncap;
  const int n = p.lengths[b];
  return (n < 0 || n > p.Ncap) ? -1 : n;
}

// Last key of the unit's keys that row m of its rows sees (−1: none).
__device__ __forceinline__ int cache_last(const CacheParams& p, bool prefix, int b, int len, int m) {
  if (m >= (prefix ? p.M : p.R)) return -1;
  const int bb = prefix ? m / p.R : b;
  const int nb = prefix ? cache_len(p, bb) : len;
  if (nb < 0) return -1;
  if (!p.causal) return len - 1;
  const int i = (prefix ? m - bb * p.R : m) % p.Nq;
  return (int)min((long long)len - 1, (long long)nb - p.Nq + i + (prefix ? p.Np : 0));
}
// Where row m of the unit's rows lies in q and o (in rows).
__device__ __forceinline__ size_t cache_row(const CacheParams& p, bool prefix, int b, int hkv, int m) {
  const int bb = prefix ? m / p.R : b;
  return (size_t)(bb * p.Hq + hkv * p.G) * p.Nq + (prefix ? m - bb * p.R : m);
}

// A CTA's way through the list, one unit's run of key tiles at a time.
struct CacheRuns {
  int unit, b, hkv, rt, len;  // b is 0 for the prefix
  bool prefix;
  int t0, t1;  // key tiles of the run
  int tiles;   // of the unit
  int left;    // key tiles of this CTA from t0 on

  __device__ __forceinline__ int tiles_of(const CacheList& l, int n) const { return n > 0 ? (n + l.keys - 1) / l.keys : 0; }
  __device__ __forceinline__ int own_tiles(const CacheParams& p, const CacheList& l, int bb) const {
    return bb < p.B ? p.Hkv * l.own_rt * tiles_of(l, cache_len(p, bb)) : 0;
  }
  __device__ __forceinline__ void set_prefix(const CacheParams& p, const CacheList& l) {
    prefix = true;
    b = 0;
    hkv = unit / l.prefix_rt;
    rt = unit - hkv * l.prefix_rt;
    len = p.Np;
    tiles = tiles_of(l, len);
  }
  __device__ __forceinline__ void set_unit(const CacheParams& p, const CacheList& l) {
    unit = l.prefix_units + (b * p.Hkv + hkv) * l.own_rt + rt;
  }
  __device__ __forceinline__ void set_end() { t1 = min(tiles, t0 + left); }

  // False if this CTA has nothing to do.  The whole warp calls it.  (The host
  // refuses lists of 2^31 - 2^20 key tiles and more.)
  __device__ __forceinline__ bool start(const CacheParams& p, const CacheList& l, int cta) {
    const int lane = threadIdx.x & 31;
    if (l.split > 0) {  // `split` CTAs a unit
      unit = cta / l.split;
      if (unit >= l.prefix_units) return false;
      set_prefix(p, l);
      const int per = (tiles + l.split - 1) / l.split;
      t0 = (cta - unit * l.split) * per;
      left = min(per, tiles - t0);
      set_end();
      return left > 0;
    }
    const int in_prefix = l.prefix_units > 0 ? l.prefix_units * tiles_of(l, p.Np) : 0;
    // 32 sequences at a time: their tiles and the sum up to each; the first 32
    // (mostly all) are needed twice and stay
    auto scan = [&](int b0, int& mine) {
      mine = own_tiles(p, l, b0 + lane);
      int sum = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      return sum;
    };
    int mine = 0, sum = 0, all = in_prefix;
    if (l.own_rt > 0) {
      sum = scan(0, mine);
      all += __shfl_sync(0xffffffffu, sum, 31);
      for (int b0 = 32; b0 < p.B; b0 += 32) {
        int m;
        all += __shfl_sync(0xffffffffu, scan(b0, m), 31);
      }
    }
    const unsigned per = ((unsigned)all + l.n_ctas - 1) / (unsigned)l.n_ctas;
    if ((unsigned long long)per * cta >= (unsigned)all) return false;
    int x = (int)(per * cta);
    left = min(all - x, (int)per);
    if (x < in_prefix) {
      unit = (unsigned)x / (unsigned)tiles_of(l, p.Np);
      set_prefix(p, l);
      t0 = x - unit * tiles;
      set_end();
      return true;
    }
    x -= in_prefix;
    prefix = false;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      if (b0 > 0) sum = scan(b0, mine);
      const uint32_t past = __ballot_sync(0xffffffffu, sum > x);
      if (past) {
        const int ln = __ffs(past) - 1;
        b = b0 + ln;
        x -= __shfl_sync(0xffffffffu, sum - mine, ln);
        break;
      }
      x -= __shfl_sync(0xffffffffu, sum, 31);
    }
    len = cache_len(p, b);
    tiles = tiles_of(l, len);
    const int u = (unsigned)x / (unsigned)tiles;  // within the sequence
    hkv = (unsigned)u / (unsigned)l.own_rt;
    rt = u - hkv * l.own_rt;
    t0 = x - u * tiles;
    set_unit(p, l);
    set_end();
    return true;
  }
  // To the next run; false at the end.
  __device__ __forceinline__ bool next(const CacheParams& p, const CacheList& l) {
    left -= t1 - t0;
    if (left <= 0) return false;
    t0 = 0;
    if (prefix && unit + 1 < l.prefix_units) {
      ++unit;
      set_prefix(p, l);
    } else {
      if (prefix) {
        prefix = false;
        b = -1;
        hkv = p.Hkv - 1;
        rt = l.own_rt - 1;
      }
      if (++rt == l.own_rt) {
        rt = 0;
        if (++hkv == p.Hkv) {
          hkv = 0;
          do {
            ++b;
            len = b < p.B ? cache_len(p, b) : 0;
            tiles = tiles_of(l, len);
          } while (tiles == 0 && b < p.B);
        }
      }
      set_unit(p, l);
    }
    set_end();
    return true;
  }
  // Notes which CTAs hold parts of the unit.
  __device__ __forceinline__ void note(const CacheList& l, int cta) const {
    if (t0 == 0) l.range[unit].x = cta;
    if (t1 == tiles) l.range[unit].y = cta;
  }
};

}  // namespace fa
