// decode_internal.h -- host helpers shared by the decode-step entry points (the expert layer, the
// paged attention and the cache pages).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../bsgemv_internal.h"

namespace bsg {

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// The current device and its SM count; BSGEMV_ERR_UNSUPPORTED without an sm_103 device.
int decode_device(int* dev, int* sms);

// BSGEMV_OK if `device` is current.
int decode_check_device(int device);

// A zeroed device allocation (BSGEMV_ERR_CUDA if it cannot be had).
int decode_alloc(void** out, size_t bytes);

// Synchronise `stream`, read and clear an error word: the status it stands for (BSGEMV_ERR_UNSUPPORTED
// for the bits of `unsupported` alone).
int decode_error_status(unsigned* err, void* stream, unsigned unsupported = 0);

// A tiled tensor map with zero fill (strides in bytes, from the second dimension on).
int decode_encode(CUtensorMap* tm, CUtensorMapDataType type, int rank, const void* base,
                  const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                  CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion);

// Allow `kernel` `smem` bytes of dynamic shared memory on the current device (`rec`: what it was
// allowed before), with the largest carveout, as for the GEMV's kernels.
template <class Kernel>
int decode_smem(Kernel kernel, AttrRecord& rec, int smem) {
  int dev = -1;
  uint64_t ctx = 0;
  if (!current_device_context(&dev, &ctx)) return BSGEMV_ERR_CUDA;
  const int d = rec.slot(dev, ctx);
  if (smem > rec.smem[d].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
      cudaGetLastError();
      return BSGEMV_ERR_CUDA;
    }
    rec.smem[d].store(smem);
  }
  return BSGEMV_OK;
}

// Launch with programmatic serialisation: the kernel may start while the one before it in the
// stream drains, and waits for it (griddepcontrol.wait) before it touches what that one writes.
template <class... Params, class... Args>
int decode_launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                  const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return BSGEMV_ERR_CUDA;
  }
  return BSGEMV_OK;
}

}  // namespace bsg
