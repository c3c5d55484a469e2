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

// Synchronise `stream`, read and clear an error word: the status it stands for.
int decode_error_status(unsigned* err, void* stream);

// cudaGetLastError as a status.
inline int decode_launched() {
  return cudaGetLastError() == cudaSuccess ? BSGEMV_OK : BSGEMV_ERR_CUDA;
}

}  // namespace bsg
