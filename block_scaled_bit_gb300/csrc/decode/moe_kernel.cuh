// moe_kernel.cuh -- kernels of the mixture-of-experts layer.
#pragma once

#include "../bsgemv_kernel.cuh"
#include "decode_internal.h"

namespace bsg {

constexpr int kMoeMaxT = 32;    // tokens per call: a token set is one 32-bit mask
constexpr int kMoeMaxE = 1024;
constexpr int kMoeMaxK = 16;
constexpr int kMoeMaxRows = kMoeMaxT * kMoeMaxK;  // (expert, token) pairs of a call

// k of a stage, and the bytes of a packed row of activations of one stage: the values in f16, then
// the fp32 factor that undoes their scale, padded so that the rows of the shared-memory ring
// start 16 banks apart (8-bit formats: 8).
__host__ __device__ constexpr int moe_stage_k(bool four) { return four ? 256 : 128; }
__host__ __device__ constexpr int moe_pitch(bool four) { return 2 * moe_stage_k(four) + (four ? 64 : 32); }

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

// A call, as the host code hands it to the kernels.
struct MoeParams {
  int fmt, bf16, bs, has_zp, flags;
  int64_t H, I;
  int E, top_k, T;
  uint64_t wait_ns;            // limit of the products' waits
  int skip_stage[2];           // test hook, UP's and DOWN's: see MoeGemmParams
  const uint16_t* x;
  const void* logits;
  const int32_t* ids;
  const float* weights;
  MoeWeight up, down;
  CUtensorMap tm_up, tm_down;  // of the weights' bytes (moe_encode)
  uint16_t* y;
  unsigned* err;
  unsigned *counters_up, *counters_down;  // arrivals per (tile, decode warp), left at zero
  unsigned* counters_group;               // ... per (block, its part opens the tile, decode warp)
  unsigned* counters_packed;              // ... per (active expert, stage of I)
  float* partials;
  Routing* route;
  float* h;                    // [rows][I]
  uint8_t *x_packed, *h_packed;  // x: see MoeGemmParams; h: [stages of I][rows][2 pitches]
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

// The workspace's parts, in bytes from its start (the error word is at 0).
struct MoeLayout {
  size_t route, counters_up, counters_packed, counters_down, counters_group, partials, h, x_packed, h_packed, total;
};
MoeLayout moe_layout(int fmt, int64_t H, int64_t I, int E, int top_k, int max_T, int sms);

// The most stages of weights that a call can have in one of its products.
inline int64_t moe_stages(int fmt, int64_t H, int64_t I, int E, int top_k, int max_T) {
  const int64_t kc = moe_stage_k(fmt == kInt4 || fmt == kNvfp4);
  const int64_t active = E < top_k * max_T ? E : top_k * max_T;
  const int64_t up = (I / 64) * ((H + kc - 1) / kc), down = (H + 127) / 128 * ((I + kc - 1) / kc);
  return active * (up > down ? up : down);
}

// Tensor map of one stacked weight (BSGEMV_ERR_CUDA if it cannot be encoded).
int moe_encode(CUtensorMap* tm, const MoeWeight& w, int E, bool up);

int launch_moe(const MoeParams& p, int sms, cudaStream_t s);

// One product's launch per weight format (a translation unit each).
struct MoeGemmParams;
int launch_moe_int4(const MoeGemmParams& p, int cpb, bool wide, bool down, int ctas, int smem,
                    cudaStream_t s);
int launch_moe_int8(const MoeGemmParams& p, int cpb, bool wide, bool down, int ctas, int smem,
                    cudaStream_t s);
int launch_moe_fp8(const MoeGemmParams& p, bool wide, bool down, int ctas, int smem,
                   cudaStream_t s);
int launch_moe_nvfp4(const MoeGemmParams& p, bool wide, bool down, int ctas, int smem,
                     cudaStream_t s);

}  // namespace bsg
