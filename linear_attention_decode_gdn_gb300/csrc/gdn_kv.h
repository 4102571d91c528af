// gdn_kv.h -- launch parameters of the paged-cache calls, shared by the C-ABI layer and the
// kernels. Not part of the public interface (include/gdn.h is).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "gdn.h"

namespace gdn {

constexpr int kMaxPlanBatch = 4096;  // requests of one plan (its running sums sit in shared memory)

struct KvPlanParams {
  int32_t B, max_pages, page_size, num_pages, free_capacity, slot_capacity;
  const int32_t* cached;
  const int32_t* fresh;  // new tokens, or NULL
  const int32_t* held;
  int32_t* table;
  const int32_t* free_list;
  const int32_t* free_count;
  int32_t* kv_len;
  int32_t* cu_new;
  int64_t* slot_map;
  int32_t* held_out;
  int32_t* free_count_out;
  int32_t* status;
  bool in_place;  // an output is its input's array (set by the launcher)
};

struct KvReleaseParams {
  int32_t B, max_pages, free_capacity, n;
  const int32_t* requests;
  const int32_t* table;
  int32_t* held;
  int32_t* free_list;
  int32_t* free_count;
  int32_t* status;
};

// One source of rows and where its elements go: `vecs` 8-element vectors of each of `heads`.
struct KvRows {
  const void* src;
  int64_t src_row, src_head;  // elements
  void* dst;
  int64_t dst_page, dst_pos, dst_head;  // elements
  uint32_t vecs, heads;
};

struct KvAppendParams {
  int32_t n, page_size;
  int32_t lanes;  // of a warp that share a row (set by the launcher)
  int64_t num_slots;
  bool bf16;
  KvRows a, b;  // b.vecs may be 0
  const int64_t* slot_map;
  int32_t* status;
};

constexpr int kTile = 128;        // cache positions a CTA takes at a time
constexpr int kSms = 152;         // of one GB300
constexpr int kMaxAttnCtas = 608; // workers of one attention launch (152 SMs, up to four CTAs each)

struct AttnParams {
  int32_t B, T, H, heads_kv, group;  // group = H / heads_kv
  int32_t dk, dv;
  int32_t num_pages, page_size, max_pages, window;
  int32_t cols;       // T * group: the query rows that share a kv head
  int32_t ncol;       // of these, how many one CTA takes at a time
  int32_t col_groups; // ceil(cols / ncol)
  uint32_t workers;   // CTAs, or pairs of CTAs, that share the tiles
  int32_t unit_cost;  // tiles that a unit counts for beyond its own
  int32_t starve;     // 0, or the wait that is to run out (GDN_STARVE_*)
  float scale_log2;   // scale * log2(e)
  const void* q;
  int64_t q_b, q_t, q_h;
  const void* k;
  const void* v;
  int64_t k_page, k_pos, k_head, v_page, v_pos, v_head;
  const int32_t* table;
  const int32_t* kv_len;
  void* o;
  float* lse;
  int32_t* status;
  // workspace: one record a worker, then two partial results a worker
  uint32_t* records;
  float* partials;
};

// Dynamic shared memory past 48 KB is allowed once a kernel and device; `done` is the kernel's own.
constexpr int kDevices = 64;
inline cudaError_t allow_shared(const void* kernel, int bytes, std::atomic<bool> (&done)[kDevices]) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
  return err;
}

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t stream);
cudaError_t launch_kv_release(const KvReleaseParams& p, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream);

// Columns one worker takes at a time and workers at most for a shape, on the path that runs it.
struct AttnPlan {
  bool tensor;  // the tensor-core kernel
  int ncol, max_workers, unit_cost;
};
AttnPlan attn_plan(const gdn_paged_kv& kv, int cols);
size_t attn_workspace_bytes(const AttnPlan& plan, int dv);
// records, then partials
constexpr int kRecordInts = 4;
constexpr size_t kRecordBytes = static_cast<size_t>(kMaxAttnCtas) * kRecordInts * sizeof(uint32_t);
static_assert(kRecordBytes % 16 == 0, "partials are read as vectors");

cudaError_t launch_attn(const AttnPlan& plan, AttnParams& p, cudaStream_t stream);
cudaError_t launch_attn_general(AttnParams& p, cudaStream_t stream);
cudaError_t launch_attn_tc(AttnParams& p, cudaStream_t stream);
cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t stream);

}  // namespace gdn
