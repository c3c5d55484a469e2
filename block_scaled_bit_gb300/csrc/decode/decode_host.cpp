// decode_host.cpp -- host helpers of the decode-step entry points.
#include "decode_internal.h"

namespace bsg {

int decode_device(int* dev, int* sms) {
  int major = 0, minor = 0;
  if (cudaGetDevice(dev) != cudaSuccess) {
    cudaGetLastError();
    return BSGEMV_ERR_UNSUPPORTED;
  }
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
    cudaGetLastError();
    return BSGEMV_ERR_CUDA;
  }
  return (major == 10 && minor == 3) ? BSGEMV_OK : BSGEMV_ERR_UNSUPPORTED;
}

int decode_check_device(int device) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return BSGEMV_ERR_CUDA;
  }
  return cur == device ? BSGEMV_OK : BSGEMV_ERR_WRONG_DEVICE;
}

int decode_alloc(void** out, size_t bytes) {
  *out = nullptr;
  if (cudaMalloc(out, bytes) != cudaSuccess) {
    cudaGetLastError();
    *out = nullptr;
    return BSGEMV_ERR_CUDA;
  }
  if (cudaMemset(*out, 0, bytes) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(*out);
    *out = nullptr;
    return BSGEMV_ERR_CUDA;
  }
  return BSGEMV_OK;
}

int decode_error_status(unsigned* err, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  if (cudaMemcpyAsync(&word, err, sizeof word, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(err, 0, sizeof word, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return BSGEMV_ERR_CUDA;
  }
  return word == 0 ? BSGEMV_OK : BSGEMV_ERR_DEVICE_TIMEOUT;
}

}  // namespace bsg
