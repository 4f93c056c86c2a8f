// host.cuh -- host helpers that the library's translation units share: the
// tensor-map encoder, device attributes, argument checks, workspace sizes and
// the launch of the merge.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "pagedkv.h"
#include "contract.cuh"
#include "merge.cuh"

namespace pkv {

constexpr int kMaxDevices = 64;

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

inline int sm_count(int dev) {
  static std::atomic<int> cache[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return 148;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
    v = 148;
  cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool pow2_in(int v, int lo, int hi) { return v >= lo && v <= hi && (v & (v - 1)) == 0; }

inline int log2i(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Element strides usable for 128-bit access: positive multiples of 8.
inline bool strides_ok(const int64_t *st) {
  if (!st) return false;
  for (int i = 0; i < 3; ++i)
    if (st[i] <= 0 || st[i] % 8 != 0) return false;
  return true;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t ws_acc_bytes(int64_t rows, int64_t splits, int D) {
  const size_t b = static_cast<size_t>(rows) * splits * D * sizeof(float);
  return (b + 255) & ~static_cast<size_t>(255);
}

inline size_t ws_bytes(int batch, int seqlen_q, int Hq, int D, int max_seqlen_k) {
  const int64_t rows = static_cast<int64_t>(batch) * seqlen_q * Hq;
  const int64_t splits = max_seqlen_k > 0 ? ceil_div(max_seqlen_k, pkv::kSplitTokens) : 1;
  return ws_acc_bytes(rows, splits, D) + static_cast<size_t>(rows) * splits * 2 * sizeof(float);
}

// Few rows (decode: rows x splits partials spread over one block per row)
// or many (prefill, packed batches: one warp per row).  FAR: see fold_sum.
template <int D, bool FAR = false>
int launch_merge(const pkv::MergeParams &m, int64_t rows, cudaStream_t s) {
  if (rows <= 4096) {
    pkv::merge_kernel<D, true, FAR><<<static_cast<unsigned>(rows), D, 0, s>>>(m);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  }
  // the warps stride over the rows: at most 8 blocks of 8 warps per SM
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  const int64_t need = ceil_div(rows, pkv::kMergeRowsPerBlock);
  const int64_t cap = static_cast<int64_t>(sm_count(dev)) * 8;
  const int64_t blocks = need < cap ? need : cap;
  pkv::merge_kernel<D, false, FAR><<<static_cast<unsigned>(blocks), 32 * pkv::kMergeRowsPerBlock, 0, s>>>(m);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
