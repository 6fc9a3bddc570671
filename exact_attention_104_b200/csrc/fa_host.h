// Host helpers shared by the library's translation units: the device table and
// its error word, TMA descriptor encoding, argument-check primitives and the
// one-shot profiling events.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "fa.h"

namespace fa_host {

constexpr int kMaxDevices = 64;
inline std::atomic<long long> g_wait_cap{1LL << 31};  // may be set from any host thread

// pending one-shot profiling events of this host thread (fa_profile_next)
inline thread_local cudaEvent_t t_prof_start = nullptr;
inline thread_local cudaEvent_t t_prof_stop = nullptr;

struct ProfileScope {
  cudaEvent_t start, stop;
  cudaStream_t stream;
  explicit ProfileScope(cudaStream_t s) : start(t_prof_start), stop(t_prof_stop), stream(s) {
    t_prof_start = t_prof_stop = nullptr;
    if (start) cudaEventRecord(start, stream);
  }
  ~ProfileScope() {
    if (stop) cudaEventRecord(stop, stream);
  }
};

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D view [rows, d] of a bf16 tensor; boxes of 64 columns (128 bytes, the
// swizzle span) by `box_rows` rows, 128-byte swizzled in shared memory.
inline bool make_map(CUtensorMap* m, const void* ptr, uint64_t rows, int d, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D view [rows, d] of an fp32 tensor, unswizzled boxes of box_cols x box_rows
// (used as the destination of TMA reduce-adds).
inline bool make_map_f32(CUtensorMap* m, const void* ptr, uint64_t rows, int d, int box_cols, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 4};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DeviceInfo {
  bool checked = false;
  bool sm100 = false;
  int sms = 0;
  int* err = nullptr;
};
inline DeviceInfo g_dev[kMaxDevices];
inline std::mutex g_dev_mu;

// Checks for an sm_100 device and resolves the error word's device address
// (once per device, with that device current).  Defined in fa_api.cu, whose
// error word every kernel of the library records into.
fa_status current_device(DeviceInfo** out);

// Debug builds: the word of fa_cache.cu's own bulk-copy checks (each
// translation unit has its g_fa_err), which fa_device_status reads too.
cudaError_t cache_check_word(int** out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// N rounded up to a whole number of 128-row tiles.
inline long long pad128(long long n) { return (n + 127) / 128 * 128; }

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace fa_host
