// chunk.cu -- attention of new tokens over the paged cache (host entry points).
#include <math.h>

#include <new>

#include "chunk_kernel.cuh"
#include "decode_internal.h"

struct bsgemv_chunk_plan_s {
  int device = -1, sms = 0;
  int bf16 = 0, Hq = 0, Hkv = 0, D = 0, page_size = 0, max_n = 0, max_T = 0;
  void* ws = nullptr;
  int fault_skip[2] = {-1, -1};  // bsgemv_chunk_set_test_fault
  uint64_t fault_wait_ns = 0;
  bsg::ChunkLayout at = {};
  // tensor maps of the last few caches seen (a layer each)
  struct MapEntry {
    bool valid = false;
    const void *k = nullptr, *v = nullptr;
    int64_t page_stride = 0, head_stride = 0, row_stride = 0;
    int num_pages = 0;
    bsg::ChunkMaps maps;
  };
  static constexpr int kMaps = 64;
  MapEntry maps[kMaps];
  int next_map = 0;
};

namespace {

// The cache's tensor maps, nullptr where its strides cannot be described.
const bsg::ChunkMaps* maps_of(bsgemv_chunk_plan_s* plan, const bsg::ChunkParams& p) {
  for (auto& m : plan->maps)
    if (m.valid && m.k == p.k && m.v == p.v && m.page_stride == p.page_stride &&
        m.head_stride == p.head_stride && m.row_stride == p.row_stride &&
        m.num_pages == p.num_pages)
      return &m.maps;
  auto& m = plan->maps[plan->next_map];
  m.valid = false;
  if (!bsg::chunk_encode(p, &m.maps)) return nullptr;
  plan->next_map = (plan->next_map + 1) % bsgemv_chunk_plan_s::kMaps;
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

int bsgemv_chunk_plan(bsgemv_chunk_plan_t* out, int act_bf16, int Hq, int Hkv, int D,
                      int page_size, int max_n, int max_T) {
  if (out == nullptr) return BSGEMV_ERR_INVALID_ARG;
  *out = nullptr;
  if ((act_bf16 != 0 && act_bf16 != 1) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 ||
      page_size < 1 || max_n < 1 || max_n > 65536 || max_T < 1)
    return BSGEMV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 256) || page_size < 8 || page_size > 1024 ||
      (page_size & (page_size - 1)) != 0 || Hq / Hkv > 64 || Hq > 1024 || max_T >= (1 << 24) ||
      static_cast<int64_t>(max_T) * Hq >= (int64_t{1} << 28))
    return BSGEMV_ERR_UNSUPPORTED;
  int dev = -1, sms = 0;
  int rc = decode_device(&dev, &sms);
  if (rc != BSGEMV_OK) return rc;
  bsgemv_chunk_plan_s* p = new (std::nothrow) bsgemv_chunk_plan_s();
  if (!p) return BSGEMV_ERR_CUDA;
  p->device = dev;
  p->sms = sms;
  p->bf16 = act_bf16;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->D = D;
  p->page_size = page_size;
  p->max_n = max_n;
  p->max_T = max_T;
  p->at = chunk_layout(Hq, Hkv, D, max_n, max_T, sms);
  rc = decode_alloc(&p->ws, p->at.total);
  if (rc != BSGEMV_OK) {
    delete p;
    return rc;
  }
  *out = p;
  return BSGEMV_OK;
}

int bsgemv_chunk_run(bsgemv_chunk_plan_t plan, const void* q, int64_t q_stride, const void* k,
                     const void* v, int64_t page_stride, int64_t head_stride, int64_t row_stride,
                     int num_pages, const int32_t* tables, int64_t table_stride, int num_seqs,
                     int max_pages, const int32_t* lens, const int32_t* seqs,
                     const int32_t* starts, int n, int T, float scale, float cap, int window,
                     const float* slopes, void* out, float* lse, void* stream) {
  if (plan == nullptr || n < 1 || T < 1 || num_pages < 1 || num_seqs < 1 || max_pages < 1 ||
      table_stride < max_pages || page_stride < 0 || head_stride < 0 || row_stride < 0 ||
      !isfinite(scale) || !isfinite(cap) || cap < 0.f || !isfinite(cap * 1.4426950408889634f) ||
      (cap > 0.f && !isfinite(scale / cap)) || window < 0)
    return BSGEMV_ERR_INVALID_ARG;
  if (n > plan->max_n || T > plan->max_T) return BSGEMV_ERR_M_TOO_LARGE;
  if (!q || !k || !v || !tables || !lens || !seqs || !starts || !out) return BSGEMV_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(plan->Hq) * plan->D && T > 1) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) ||
      !aligned_to(tables, 4) || !aligned_to(lens, 4) || !aligned_to(seqs, 4) ||
      !aligned_to(starts, 4) || !aligned_to(slopes, 4) || !aligned_to(lse, 4) || q_stride % 8 ||
      page_stride % 8 || head_stride % 8 || row_stride % 8)
    return BSGEMV_ERR_MISALIGNED;
  const int rc = decode_check_device(plan->device);
  if (rc != BSGEMV_OK) return rc;
  ChunkParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.page_stride = page_stride;
  p.head_stride = head_stride;
  p.row_stride = row_stride;
  p.num_pages = num_pages;
  p.tables = tables;
  p.table_stride = table_stride;
  p.num_seqs = num_seqs;
  p.max_pages = max_pages;
  p.lens = lens;
  p.seqs = seqs;
  p.starts = starts;
  p.n = n;
  p.T = T;
  p.Hq = plan->Hq;
  p.Hkv = plan->Hkv;
  p.D = plan->D;
  p.page_log2 = __builtin_ctz(static_cast<unsigned>(plan->page_size));
  p.bf16 = plan->bf16;
  p.scale = scale;
  p.cap = cap;
  p.window = window;
  p.slopes = slopes;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  char* ws = static_cast<char*>(plan->ws);
  p.head = reinterpret_cast<ChunkHead*>(ws);
  for (int i = 0; i < 2; ++i) {
    ChunkLine& line = i ? p.stream : p.tensor;
    const auto& at = i ? plan->at.stream : plan->at.tensor;
    line.blocks = reinterpret_cast<ChunkBlock*>(ws + at.blocks);
    line.cuts = reinterpret_cast<ChunkCut*>(ws + at.cuts);
    line.parts = reinterpret_cast<float*>(ws + at.parts);
    line.max_blocks = at.max_blocks;
  }
  p.fills = reinterpret_cast<int2*>(ws + plan->at.fills);
  p.wait_ns = plan->fault_wait_ns ? plan->fault_wait_ns : kDefaultWaitNs;
  p.skip[0] = plan->fault_skip[0];
  p.skip[1] = plan->fault_skip[1];
  const ChunkMaps* maps = maps_of(plan, p);
  if (maps == nullptr) return BSGEMV_ERR_UNSUPPORTED;
  return launch_chunk(p, *maps, plan->sms, static_cast<cudaStream_t>(stream));
}

int bsgemv_chunk_set_test_fault(bsgemv_chunk_plan_t plan, int kernel, int skip_tile, int64_t wait_ns) {
  if (plan == nullptr || kernel < 0 || kernel > 1 || skip_tile < -1 || wait_ns < 0)
    return BSGEMV_ERR_INVALID_ARG;
  plan->fault_skip[kernel] = skip_tile;
  plan->fault_skip[1 - kernel] = -1;
  plan->fault_wait_ns = static_cast<uint64_t>(wait_ns);
  return BSGEMV_OK;
}

int bsgemv_chunk_device_status(bsgemv_chunk_plan_t plan, void* stream) {
  if (plan == nullptr) return BSGEMV_ERR_INVALID_ARG;
  const int rc = decode_check_device(plan->device);
  if (rc != BSGEMV_OK) return rc;
  return decode_error_status(static_cast<unsigned*>(plan->ws), stream, kErrChunkLine);
}

int bsgemv_chunk_destroy(bsgemv_chunk_plan_t plan) {
  if (plan == nullptr) return BSGEMV_OK;
  int rc = BSGEMV_OK;
  if (cudaDeviceSynchronize() != cudaSuccess) rc = BSGEMV_ERR_CUDA;
  cudaFree(plan->ws);
  delete plan;
  return rc;
}

}  // extern "C"
