// moe.cu -- the mixture-of-experts layer for a few tokens (host entry points and kernels).
//
//   route     one block: top-k of each token's logits, the experts that are wanted and their
//             tokens (a 32-bit mask per expert: max_T <= 32)
//             ... and, in other blocks, x packed for the tensor cores
//   up        h[row][i] = p * silu(g) * u for every (expert, token) pair, packed likewise
//   down      y[t][n]   = sum over the token's experts, in expert order
#include <math.h>

#include <new>

#include "decode_internal.h"
#include "moe_kernel.cuh"

struct bsgemv_moe_plan_s {
  int device = -1, sms = 0;
  int fmt = 0, bf16 = 0, block_size = 0, has_zp = 0;
  int64_t H = 0, I = 0;
  int E = 0, top_k = 0, max_T = 0, flags = 0;
  int fault_skip[2] = {-1, -1};   // bsgemv_moe_set_test_fault
  uint64_t fault_wait_ns = 0;
  void* ws = nullptr;
  bsg::MoeLayout at = {};
  // tensor maps of the last few (W13, W2) pairs (a layer each: a plan serves layers in turn)
  struct MapEntry {
    const void *W13 = nullptr, *W2 = nullptr;
    CUtensorMap up, down;
  };
  static constexpr int kMaps = 64;
  MapEntry maps[kMaps];
  int next_map = 0;
};

namespace bsg {
namespace {

int maps_of(bsgemv_moe_plan_s* p, const MoeWeight& up, const MoeWeight& down, MoeParams* q) {
  for (auto& m : p->maps)
    if (m.W13 == up.W && m.W2 == down.W) {
      q->tm_up = m.up;
      q->tm_down = m.down;
      return BSGEMV_OK;
    }
  auto& m = p->maps[p->next_map];
  m.W13 = nullptr;
  int rc = moe_encode(&m.up, up, p->E, true);
  if (rc == BSGEMV_OK) rc = moe_encode(&m.down, down, p->E, false);
  if (rc != BSGEMV_OK) return rc;
  p->next_map = (p->next_map + 1) % bsgemv_moe_plan_s::kMaps;
  m.W13 = up.W;
  m.W2 = down.W;
  q->tm_up = m.up;
  q->tm_down = m.down;
  return BSGEMV_OK;
}

int run(bsgemv_moe_plan_s* p, const void* x, const void* logits, const int32_t* ids,
        const float* weights, const void* W13, const void* s13, const void* zp13, const void* W2,
        const void* s2, const void* zp2, void* y, int T, void* stream) {
  if (p == nullptr || T < 1) return BSGEMV_ERR_INVALID_ARG;
  if (T > p->max_T) return BSGEMV_ERR_M_TOO_LARGE;
  if (!x || !W13 || !s13 || !W2 || !s2 || !y || (!logits && (!ids || !weights)))
    return BSGEMV_ERR_INVALID_ARG;
  const bool third = p->has_zp || p->fmt == kNvfp4;
  if (third != (zp13 != nullptr) || third != (zp2 != nullptr)) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(W13, 16) || !aligned_to(W2, 16) || !aligned_to(y, 16) ||
      !aligned_to(s13, 4) || !aligned_to(s2, 4) || !aligned_to(zp13, 4) || !aligned_to(zp2, 4) ||
      !aligned_to(logits, (p->flags & BSGEMV_MOE_LOGITS_F32) ? 4 : 2) || !aligned_to(ids, 4) ||
      !aligned_to(weights, 4))
    return BSGEMV_ERR_MISALIGNED;
  int rc = decode_check_device(p->device);
  if (rc != BSGEMV_OK) return rc;
  MoeParams q = {};
  q.fmt = p->fmt;
  q.bf16 = p->bf16;
  q.bs = p->block_size;
  q.has_zp = p->has_zp;
  q.H = p->H;
  q.I = p->I;
  q.E = p->E;
  q.top_k = p->top_k;
  q.T = T;
  q.flags = p->flags;
  q.wait_ns = p->fault_wait_ns ? p->fault_wait_ns : kDefaultWaitNs;
  q.skip_stage[0] = p->fault_skip[0];
  q.skip_stage[1] = p->fault_skip[1];
  q.x = static_cast<const uint16_t*>(x);
  q.logits = logits;
  q.ids = ids;
  q.weights = weights;
  q.up = weight_of(p->fmt, p->block_size, p->has_zp, 2 * p->I, p->H, W13, s13, zp13);
  q.down = weight_of(p->fmt, p->block_size, p->has_zp, p->H, p->I, W2, s2, zp2);
  rc = maps_of(p, q.up, q.down, &q);
  if (rc != BSGEMV_OK) return rc;
  q.y = static_cast<uint16_t*>(y);
  char* w = static_cast<char*>(p->ws);
  q.err = reinterpret_cast<unsigned*>(w);
  q.route = reinterpret_cast<Routing*>(w + p->at.route);
  q.counters_up = reinterpret_cast<unsigned*>(w + p->at.counters_up);
  q.counters_packed = reinterpret_cast<unsigned*>(w + p->at.counters_packed);
  q.counters_down = reinterpret_cast<unsigned*>(w + p->at.counters_down);
  q.counters_group = reinterpret_cast<unsigned*>(w + p->at.counters_group);
  q.partials = reinterpret_cast<float*>(w + p->at.partials);
  q.h = reinterpret_cast<float*>(w + p->at.h);
  q.x_packed = reinterpret_cast<uint8_t*>(w + p->at.x_packed);
  q.h_packed = reinterpret_cast<uint8_t*>(w + p->at.h_packed);
  return launch_moe(q, p->sms, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace bsg

using namespace bsg;

extern "C" {

int bsgemv_moe_plan(bsgemv_moe_plan_t* out, int format, int block_size, int has_zp, int64_t H,
                    int64_t I, int E, int top_k, int max_T, int flags) {
  if (out == nullptr) return BSGEMV_ERR_INVALID_ARG;
  *out = nullptr;
  const int fmt = format & 0xFF;
  if ((format & ~(0xFF | BSGEMV_ACT_BF16)) != 0 || fmt < kInt4 || fmt > kNvfp4 ||
      (has_zp != 0 && has_zp != 1) || H < 1 || I < 1 || E < 1 || top_k < 1 || top_k > E ||
      max_T < 1 || max_T > kMoeMaxT ||
      (flags & ~(BSGEMV_MOE_RENORMALIZE | BSGEMV_MOE_LOGITS_F32)) != 0)
    return BSGEMV_ERR_INVALID_ARG;
  const bool ints = fmt == kInt4 || fmt == kInt8;
  const bool bs_ok = ints ? (block_size == 16 || block_size == 32 || block_size == 64 ||
                             block_size == 128)
                          : block_size == (fmt == kFp8 ? 128 : 16);
  if (!bs_ok || (has_zp && !ints) || E > kMoeMaxE || top_k > kMoeMaxK || H % 64 || I % 64 ||
      H % block_size || I % block_size || H >= (1 << 24) || I >= (1 << 24) ||
      2 * I * E >= (int64_t{1} << 31) || H * E >= (int64_t{1} << 31) ||
      moe_stages(fmt, H, I, E, top_k, max_T) >= (int64_t{1} << 31))
    return BSGEMV_ERR_UNSUPPORTED;
  int dev = -1, sms = 0;
  int rc = decode_device(&dev, &sms);
  if (rc != BSGEMV_OK) return rc;
  bsgemv_moe_plan_s* p = new (std::nothrow) bsgemv_moe_plan_s();
  if (!p) return BSGEMV_ERR_CUDA;
  p->device = dev;
  p->sms = sms;
  p->fmt = fmt;
  p->bf16 = (format & BSGEMV_ACT_BF16) != 0;
  p->block_size = block_size;
  p->has_zp = has_zp;
  p->H = H;
  p->I = I;
  p->E = E;
  p->top_k = top_k;
  p->max_T = max_T;
  p->flags = flags;
  p->at = moe_layout(fmt, H, I, E, top_k, max_T, sms);
  rc = decode_alloc(&p->ws, p->at.total);
  if (rc != BSGEMV_OK) {
    delete p;
    return rc;
  }
  *out = p;
  return BSGEMV_OK;
}

int bsgemv_moe_run(bsgemv_moe_plan_t plan, const void* x, const void* logits, const void* W13,
                   const void* scales13, const void* zp13, const void* W2, const void* scales2,
                   const void* zp2, void* y, int T, void* stream) {
  if (logits == nullptr) return BSGEMV_ERR_INVALID_ARG;
  return run(plan, x, logits, nullptr, nullptr, W13, scales13, zp13, W2, scales2, zp2, y, T,
             stream);
}

int bsgemv_moe_run_routed(bsgemv_moe_plan_t plan, const void* x, const int32_t* ids,
                          const float* weights, const void* W13, const void* scales13,
                          const void* zp13, const void* W2, const void* scales2, const void* zp2,
                          void* y, int T, void* stream) {
  return run(plan, x, nullptr, ids, weights, W13, scales13, zp13, W2, scales2, zp2, y, T, stream);
}

int bsgemv_moe_set_test_fault(bsgemv_moe_plan_t plan, int product, int skip_stage,
                              int64_t wait_ns) {
  if (plan == nullptr || product < 0 || product > 1 || skip_stage < -1 || wait_ns < 0)
    return BSGEMV_ERR_INVALID_ARG;
  plan->fault_skip[product] = skip_stage;
  plan->fault_skip[1 - product] = -1;
  plan->fault_wait_ns = static_cast<uint64_t>(wait_ns);
  return BSGEMV_OK;
}

int bsgemv_moe_device_status(bsgemv_moe_plan_t plan, void* stream) {
  if (plan == nullptr) return BSGEMV_ERR_INVALID_ARG;
  const int rc = decode_check_device(plan->device);
  if (rc != BSGEMV_OK) return rc;
  const int status = decode_error_status(static_cast<unsigned*>(plan->ws), stream);
  // a call whose wait ran out left arrivals in the counters: the next one starts from zero again
  if (status == BSGEMV_ERR_DEVICE_TIMEOUT &&
      (cudaMemsetAsync(static_cast<char*>(plan->ws) + plan->at.counters_up, 0,
                       plan->at.partials - plan->at.counters_up,
                       static_cast<cudaStream_t>(stream)) != cudaSuccess ||
       cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)) {
    cudaGetLastError();
    return BSGEMV_ERR_CUDA;
  }
  return status;
}

int bsgemv_moe_destroy(bsgemv_moe_plan_t plan) {
  if (plan == nullptr) return BSGEMV_OK;
  int rc = BSGEMV_OK;
  if (cudaDeviceSynchronize() != cudaSuccess) rc = BSGEMV_ERR_CUDA;
  cudaFree(plan->ws);
  delete plan;
  return rc;
}

}  // extern "C"
