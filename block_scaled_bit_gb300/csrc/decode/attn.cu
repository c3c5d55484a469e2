// attn.cu -- single-token attention of a batch that shares a prefix, over a paged cache (host
// entry points).
#include <math.h>

#include <new>

#include "attn_kernel.cuh"
#include "decode_internal.h"

struct bsgemv_attn_plan_s {
  int device = -1, sms = 0;
  int bf16 = 0, Hq = 0, Hkv = 0, D = 0, page_size = 0, max_B = 0;
  void* ws = nullptr;
  int fault_skip[2] = {-1, -1};   // bsgemv_attn_set_test_fault
  uint64_t fault_wait_ns = 0;
  bsg::AttnLayout at = {};
  // tensor maps of the last few caches seen (a layer each)
  struct MapEntry {
    bool valid = false;
    const void *k = nullptr, *v = nullptr;
    int64_t page_stride = 0, head_stride = 0, row_stride = 0;
    int num_pages = 0;
    bsg::AttnMaps maps;
  };
  static constexpr int kMaps = 64;
  MapEntry maps[kMaps];
  int next_map = 0;
};

namespace {

// The cache's tensor maps, nullptr where its strides cannot be described.
const bsg::AttnMaps* maps_of(bsgemv_attn_plan_s* plan, const bsg::AttnParams& p) {
  for (auto& m : plan->maps)
    if (m.valid && m.k == p.k && m.v == p.v && m.page_stride == p.page_stride &&
        m.head_stride == p.head_stride && m.row_stride == p.row_stride &&
        m.num_pages == p.num_pages)
      return &m.maps;
  auto& m = plan->maps[plan->next_map];
  m.valid = false;
  if (!bsg::attn_encode(p, &m.maps)) return nullptr;
  plan->next_map = (plan->next_map + 1) % bsgemv_attn_plan_s::kMaps;
  m.valid = true;
  m.k = p.k;
  m.v = p.v;
  m.page_stride = p.page_stride;
  m.head_stride = p.head_stride;
  m.row_stride = p.row_stride;
  m.num_pages = p.num_pages;
  return &m.maps;
}

}  // namespace

using namespace bsg;

extern "C" {

int bsgemv_attn_plan(bsgemv_attn_plan_t* out, int act_bf16, int Hq, int Hkv, int D, int page_size,
                     int max_B) {
  if (out == nullptr) return BSGEMV_ERR_INVALID_ARG;
  *out = nullptr;
  if ((act_bf16 != 0 && act_bf16 != 1) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 ||
      page_size < 1 || max_B < 1 || max_B > kAttnMaxB)
    return BSGEMV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 256) || page_size < 8 || page_size > 1024 ||
      (page_size & (page_size - 1)) != 0 || Hq / Hkv > kAttnMaxGroup || Hq > 1024)
    return BSGEMV_ERR_UNSUPPORTED;
  int dev = -1, sms = 0;
  int rc = decode_device(&dev, &sms);
  if (rc != BSGEMV_OK) return rc;
  bsgemv_attn_plan_s* p = new (std::nothrow) bsgemv_attn_plan_s();
  if (!p) return BSGEMV_ERR_CUDA;
  p->device = dev;
  p->sms = sms;
  p->bf16 = act_bf16;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->D = D;
  p->page_size = page_size;
  p->max_B = max_B;
  p->at = attn_layout(Hq, Hkv, D, max_B, sms);
  rc = decode_alloc(&p->ws, p->at.total);
  if (rc != BSGEMV_OK) {
    delete p;
    return rc;
  }
  *out = p;
  return BSGEMV_OK;
}

int bsgemv_attn_run(bsgemv_attn_plan_t plan, const void* q, int64_t q_stride, const void* k,
                    const void* v, int64_t page_stride, int64_t head_stride, int64_t row_stride,
                    int num_pages, const int32_t* prefix_table, int prefix_len,
                    const int32_t* tables, int64_t table_stride, const int32_t* lens, int B,
                    float scale, void* out, float* lse, void* stream) {
  if (plan == nullptr || B < 1 || prefix_len < 0 || prefix_len >= (1 << 30) || num_pages < 1 ||
      table_stride < 0 || page_stride < 0 || head_stride < 0 || row_stride < 0 || !(scale == scale))
    return BSGEMV_ERR_INVALID_ARG;
  if (B > plan->max_B) return BSGEMV_ERR_M_TOO_LARGE;
  if (!q || !k || !v || !tables || !lens || !out || (prefix_len > 0 && !prefix_table))
    return BSGEMV_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(plan->Hq) * plan->D && B > 1) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) ||
      !aligned_to(prefix_table, 4) || !aligned_to(tables, 4) || !aligned_to(lens, 4) ||
      !aligned_to(lse, 4) || q_stride % 8 || page_stride % 8 || head_stride % 8 || row_stride % 8)
    return BSGEMV_ERR_MISALIGNED;
  const int rows = B * (plan->Hq / plan->Hkv);
  const int mode = prefix_len == 0 ? kAttnNoPrefix
                   : attn_prefix_streams(rows, plan->Hkv, plan->D, prefix_len) ? kAttnPrefixStream
                                                                               : kAttnPrefixTensor;
  // the line of tiles (attn_stream.cuh, attn_prefix.cuh) is counted in 31 bits: the prefix's part of it
  // (the sequences' own follows from lens, on the device)
  const int64_t row_tiles = (rows + kAttnRows - 1) / kAttnRows;
  if (row_tiles * plan->Hkv * (prefix_len / (4096 / plan->D) + 8) >= (int64_t{1} << 30))
    return BSGEMV_ERR_UNSUPPORTED;
  const int rc = decode_check_device(plan->device);
  if (rc != BSGEMV_OK) return rc;
  AttnParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.page_stride = page_stride;
  p.head_stride = head_stride;
  p.row_stride = row_stride;
  p.num_pages = num_pages;
  p.prefix_table = prefix_table;
  p.prefix_len = prefix_len;
  p.tables = tables;
  p.table_stride = table_stride;
  p.lens = lens;
  p.B = B;
  p.Hq = plan->Hq;
  p.Hkv = plan->Hkv;
  p.D = plan->D;
  p.page_log2 = __builtin_ctz(static_cast<unsigned>(plan->page_size));
  p.bf16 = plan->bf16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.err = static_cast<unsigned*>(plan->ws);
  p.wait_ns = plan->fault_wait_ns ? plan->fault_wait_ns : kDefaultWaitNs;
  p.skip[0] = plan->fault_skip[0];
  p.skip[1] = plan->fault_skip[1];
  p.parts = reinterpret_cast<float*>(static_cast<char*>(plan->ws) + plan->at.parts);
  p.pre_parts = reinterpret_cast<float*>(static_cast<char*>(plan->ws) + plan->at.pre_parts);
  p.cum = reinterpret_cast<int*>(static_cast<char*>(plan->ws) + plan->at.cum);
  const AttnMaps* maps = maps_of(plan, p);
  if (maps == nullptr) return BSGEMV_ERR_UNSUPPORTED;
  return launch_attn(p, mode, *maps, plan->sms, static_cast<cudaStream_t>(stream));
}

int bsgemv_attn_set_test_fault(bsgemv_attn_plan_t plan, int kernel, int skip_tile,
                               int64_t wait_ns) {
  if (plan == nullptr || kernel < 0 || kernel > 1 || skip_tile < -1 || wait_ns < 0)
    return BSGEMV_ERR_INVALID_ARG;
  plan->fault_skip[kernel] = skip_tile;
  plan->fault_skip[1 - kernel] = -1;
  plan->fault_wait_ns = static_cast<uint64_t>(wait_ns);
  return BSGEMV_OK;
}

int bsgemv_attn_device_status(bsgemv_attn_plan_t plan, void* stream) {
  if (plan == nullptr) return BSGEMV_ERR_INVALID_ARG;
  const int rc = decode_check_device(plan->device);
  if (rc != BSGEMV_OK) return rc;
  return decode_error_status(static_cast<unsigned*>(plan->ws), stream, kErrAttnLine);
}

int bsgemv_attn_destroy(bsgemv_attn_plan_t plan) {
  if (plan == nullptr) return BSGEMV_OK;
  int rc = BSGEMV_OK;
  if (cudaDeviceSynchronize() != cudaSuccess) rc = BSGEMV_ERR_CUDA;
  cudaFree(plan->ws);
  delete plan;
  return rc;
}

}  // extern "C"
