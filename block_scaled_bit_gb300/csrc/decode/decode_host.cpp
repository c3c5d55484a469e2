// decode_host.cpp -- host helpers of the decode-step entry points.
#include "decode_internal.h"

#include <cudaTypedefs.h>

#include <mutex>

namespace bsg {

int decode_encode(CUtensorMap* tm, CUtensorMapDataType type, int rank, const void* base,
                  const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                  CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (!encode) return BSGEMV_ERR_CUDA;
  cuuint64_t d[5], st[4] = {};
  cuuint32_t b[5], unit[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    unit[i] = 1;
    if (i + 1 < rank) st[i] = strides[i];
  }
  const CUresult r = encode(tm, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), d, st,
                            b, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSGEMV_OK : BSGEMV_ERR_CUDA;
}

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
  // (waited for: the first call may come on a stream that does not follow the default one)
  if (cudaMemset(*out, 0, bytes) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(*out);
    *out = nullptr;
    return BSGEMV_ERR_CUDA;
  }
  return BSGEMV_OK;
}

int decode_error_status(unsigned* err, void* stream, unsigned unsupported) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  if (cudaMemcpyAsync(&word, err, sizeof word, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(err, 0, sizeof word, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return BSGEMV_ERR_CUDA;
  }
  if (word & ~unsupported) return BSGEMV_ERR_DEVICE_TIMEOUT;
  return word == 0 ? BSGEMV_OK : BSGEMV_ERR_UNSUPPORTED;
}

}  // namespace bsg
