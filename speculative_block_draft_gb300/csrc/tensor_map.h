// The driver's tensor-map encoder (host side), shared by abi.cu and cache_abi.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace dfl {

// The driver's tensor-map encoder, looked up once per process.
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled tensor_map_encoder() {
  static std::atomic<EncodeTiled> encode{nullptr};
  EncodeTiled e = encode.load(std::memory_order_acquire);
  if (!e) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return nullptr;
    e = reinterpret_cast<EncodeTiled>(fn);
    encode.store(e, std::memory_order_release);
  }
  return e;
}

}  // namespace dfl
