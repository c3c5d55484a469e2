// moe_kernel.cuh -- kernels of the mixture-of-experts layer.
#pragma once

#include "../bsgemv_kernel.cuh"
#include "decode_internal.h"

namespace bsg {

constexpr int kMoeMaxT = 32;    // tokens per call: a token set is one 32-bit mask
constexpr int kMoeMaxE = 1024;
constexpr int kMoeMaxK = 16;
constexpr int kMoeMaxRows = kMoeMaxT * kMoeMaxK;  // (expert, token) pairs of a call

// What a call's tokens chose.  Active experts in index order; expert a's pairs are the rows
// off[a] .. off[a + 1] - 1 in token order.
struct Routing {
  int active;
  uint32_t nan_rows;               // tokens whose softmax is NaN
  int expert[kMoeMaxRows];
  uint32_t mask[kMoeMaxRows];      // tokens of the active expert
  int off[kMoeMaxRows + 1];
  int token[kMoeMaxRows];          // token of a row
  float weight[kMoeMaxRows];       // routing weight of a row
};

inline size_t routing_bytes() { return (sizeof(Routing) + 255) / 256 * 256; }

// One stacked weight: E matrices of [rows][k].
struct MoeWeight {
  const uint8_t* W;
  const uint8_t* scales;
  const uint8_t* zp;      // zero points, or nullptr
  const float* gscale;    // NVFP4: [E]
  int64_t row_bytes, scale_pitch, zp_pitch;
  int64_t rows, k;
};

struct MoeParams {
  int fmt, bf16, bs, has_zp, flags;
  int64_t H, I;
  int E, top_k, T;
  const uint16_t* x;
  const void* logits;
  const int32_t* ids;
  const float* weights;
  MoeWeight up, down;
  uint16_t* y;
  unsigned* err;
  Routing* route;
  float* h;   // [rows][I]
};

inline MoeWeight weight_of(int fmt, int bs, int has_zp, int64_t rows, int64_t k, const void* W,
                           const void* s, const void* z) {
  MoeWeight w = {};
  w.W = static_cast<const uint8_t*>(W);
  w.scales = static_cast<const uint8_t*>(s);
  w.zp = has_zp ? static_cast<const uint8_t*>(z) : nullptr;
  w.gscale = fmt == kNvfp4 ? static_cast<const float*>(z) : nullptr;
  w.rows = rows;
  w.k = k;
  const int64_t nb = k / bs;
  w.row_bytes = (fmt == kInt4 || fmt == kNvfp4) ? k / 2 : k;
  w.scale_pitch = nb * (fmt == kFp8 ? 4 : fmt == kNvfp4 ? 1 : 2);
  w.zp_pitch = fmt == kInt4 ? (nb + 1) / 2 : nb;
  return w;
}

inline size_t moe_workspace_bytes(int64_t H, int64_t I, int top_k, int max_T, int sms) {
  (void)H;
  (void)sms;
  return 256 + routing_bytes() + size_t(max_T) * top_k * I * sizeof(float);
}

int launch_moe(const MoeParams& p, int sms, cudaStream_t s);

}  // namespace bsg
