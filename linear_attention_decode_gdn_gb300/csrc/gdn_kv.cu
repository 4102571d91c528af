// gdn_kv.cu -- the paged cache: pages and slots for new tokens (gdn_kv_plan), pages given
// back (gdn_kv_release) and rows written to their slots (gdn_kv_append).
#include "gdn_device.cuh"
#include "gdn_kv.h"

namespace gdn {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanCluster = 8;

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  return static_cast<int64_t>(__shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(v), d));
}

// Inclusive sum over the block's threads; every thread calls it. Returns the block's total
// in *total. 64 bits: lengths are the caller's and their sums may pass 32.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = shfl_up64(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the previous call's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return x + before;
}

// Largest b in [0, n) with sums[b] <= x (sums rise; sums[0] = 0).
__device__ __forceinline__ int find_row(const int32_t* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

// Every CTA of the (one) cluster takes the whole batch's sums for itself, in shared memory:
// that is 12 bytes read a request and spares a second launch or a grid barrier. The cluster
// barrier stands between the last read of the inputs and the first write of the outputs, so
// outputs may be the inputs' own arrays. After it the CTAs share the tokens and the pages.
__global__ void __launch_bounds__(kPlanThreads) gdn_kv_plan_kernel(const KvPlanParams p) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_sums[kPlanThreads / 32];
  __shared__ int32_t handed;            // free pages handed out
  int32_t* cu = sm;                     // [B + 1] tokens before request b
  int32_t* fresh_cu = cu + p.B + 1;     // [B] pages handed out before request b
  int32_t* start = fresh_cu + p.B;      // [B] cached length c; ~c for a request without slots
  int32_t* held = start + p.B;          // [B] pages the request had
  int32_t* held_new = held + p.B;       // [B] and has now
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();

  uint32_t bad = 0;
  int32_t avail = p.free_count[0];
  const int32_t given = avail;
  if (avail < 0 || avail > p.num_pages) {
    avail = 0;
    bad |= GDN_STATUS_BAD_LEN;
  }
  if (tid == 0) handed = 0;
  int64_t tokens = 0, pages = 0;  // of the requests before this chunk
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    int32_t c = -1, n = 0, h = 0;
    if (b < p.B) {
      c = p.cached[b];
      n = c < 0 ? 0 : (p.fresh != nullptr ? p.fresh[b] : 1);
      h = p.held[b];
    }
    bool skip = c < 0;
    if (n < 0) {
      n = 0;
      skip = true;
      bad |= GDN_STATUS_BAD_LEN;
    }
    int64_t total;
    const int64_t upto = tokens + block_scan<kPlanThreads>(n, warp_sums, &total);
    tokens += total;
    const int64_t length = static_cast<int64_t>(c) + n;
    const int64_t need = (length + p.page_size - 1) / p.page_size;
    if (!skip && (h < 0 || h > p.max_pages || need > p.max_pages || length > 0x7fffffffLL ||
                  upto > p.slot_capacity)) {
      skip = true;
      bad |= GDN_STATUS_BAD_LEN;
    }
    const int64_t want = skip || need <= h ? 0 : need - h;
    const int64_t pages_upto = pages + block_scan<kPlanThreads>(want, warp_sums, &total);
    pages += total;
    // The running sum passes `avail` at the first request that does not fit and never comes
    // back below it, so the requests that fit are a prefix of those that want a page, and
    // their sums are the pages handed out.
    const bool fits = want == 0 || pages_upto <= avail;
    if (!fits) {
      skip = true;
      bad |= GDN_STATUS_NO_PAGES;
    } else if (want > 0) {
      atomicMax(&handed, static_cast<int32_t>(pages_upto));
    }
    if (b < p.B) {
      constexpr int64_t kTop = 0x7fffffff;
      cu[b] = static_cast<int32_t>(min(upto - n, kTop));
      if (b == p.B - 1) cu[p.B] = static_cast<int32_t>(min(upto, kTop));
      fresh_cu[b] = static_cast<int32_t>(min(pages_upto - want, kTop));
      start[b] = skip ? ~max(c, 0) : c;
      held[b] = h;
      held_new[b] = fits ? h + static_cast<int32_t>(want) : h;
    }
  }
  if (bad != 0u && blockIdx.x == 0) atomic_status(p.status, bad);
  if (gridDim.x > 1) cluster_sync_all(); else __syncthreads();

  const int first = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
  for (int b = first; b <= p.B; b += step) {
    p.cu_new[b] = cu[b];
    if (b == p.B) {
      // a count outside the list is left for the caller to see
      p.free_count_out[0] = given != avail ? given : avail - handed;
      break;
    }
    const int32_t c = start[b];
    p.kv_len[b] = c < 0 ? ~c : c + (cu[b + 1] - cu[b]);
    p.held_out[b] = held_new[b];
  }
  uint32_t bad_page = 0;
  for (int f = first; f < handed; f += step) {
    const int b = find_row(fresh_cu, p.B, f);
    int32_t page = p.free_list[avail - 1 - f];
    if (page < 0 || page >= p.num_pages) {
      page = -1;
      bad_page = GDN_STATUS_BAD_PAGE;
    }
    p.table[static_cast<int64_t>(b) * p.max_pages + held[b] + (f - fresh_cu[b])] = page;
  }
  const int32_t all = cu[p.B];
  for (int i = first; i < p.slot_capacity; i += step) {
    int64_t slot = -1;
    if (i < all) {
      const int b = find_row(cu, p.B, i);
      const int32_t c = start[b];
      if (c >= 0) {
        const uint32_t pos = static_cast<uint32_t>(c) + static_cast<uint32_t>(i - cu[b]);
        const int32_t idx = static_cast<int32_t>(pos / static_cast<uint32_t>(p.page_size));
        const int32_t off = static_cast<int32_t>(pos - static_cast<uint32_t>(idx) * p.page_size);
        const int32_t page = idx < held[b] ? p.table[static_cast<int64_t>(b) * p.max_pages + idx]
                                           : p.free_list[avail - 1 - (fresh_cu[b] + idx - held[b])];
        if (page >= 0 && page < p.num_pages) slot = static_cast<int64_t>(page) * p.page_size + off;
        else bad_page = GDN_STATUS_BAD_PAGE;
      }
    }
    p.slot_map[i] = slot;
  }
  if (bad_page != 0u) atomic_status(p.status, bad_page);
}

// One CTA: the requests' page counts are summed so that each knows where its pages go, and
// the warps copy them. Finished requests are few; nothing here is worth more CTAs.
__global__ void __launch_bounds__(kPlanThreads) gdn_kv_release_kernel(const KvReleaseParams p) {
  __shared__ int64_t warp_sums[kPlanThreads / 32];
  __shared__ int32_t at[kPlanThreads], row[kPlanThreads], count[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  uint32_t bad = 0;
  int64_t top = p.free_count[0];
  __syncthreads();  // read by all before thread 0 writes it at the end
  if (top < 0 || top > p.num_pages) {
    if (tid == 0) atomic_status(p.status, GDN_STATUS_BAD_LEN);
    return;
  }
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + tid;
    int32_t b = i < p.n ? p.requests[i] : -1;
    if (b >= p.B) {
      bad |= GDN_STATUS_BAD_SLOT;
      b = -1;
    }
    int32_t h = b >= 0 ? p.held[b] : 0;
    if (h < 0 || h > p.max_pages) {
      bad |= GDN_STATUS_BAD_LEN;
      h = 0;
      b = -1;
    }
    int64_t total;
    const int64_t upto = block_scan<kPlanThreads>(h, warp_sums, &total);
    // past the list's end this request and the later ones of the chunk keep their pages
    const bool fits = top + upto <= p.num_pages;
    if (h > 0 && !fits) bad |= GDN_STATUS_BAD_LEN;
    at[tid] = static_cast<int32_t>(top + upto - h);
    row[tid] = b;
    count[tid] = fits ? h : 0;
    if (h > 0 && fits) p.held[b] = 0;
    int64_t kept;
    block_scan<kPlanThreads>(fits ? h : 0, warp_sums, &kept);
    __syncthreads();
    for (int j = warp; j < kPlanThreads; j += kPlanThreads / 32) {
      const int32_t* from = p.table + static_cast<int64_t>(row[j]) * p.max_pages;
      for (int k = lane; k < count[j]; k += 32) p.free_list[at[j] + k] = from[k];
    }
    top += kept;
    __syncthreads();
  }
  if (bad != 0u) atomic_status(p.status, bad);
  if (tid == 0) p.free_count[0] = static_cast<int32_t>(top);
}

// ---- rows to their slots ----------------------------------------------------------------
constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One thread an 8-element vector: one 16-byte load (two for fp32) and one 16-byte store.
// Neighbouring threads take neighbouring vectors of a row.
__global__ void __launch_bounds__(kAppendThreads) gdn_kv_append_kernel(const KvAppendParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t va = p.a.vecs * p.heads, vb = p.b.vecs * p.heads, row_vecs = va + vb;
  const int64_t all = static_cast<int64_t>(p.n) * row_vecs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kAppendThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x; i < all; i += step) {
    const int64_t r = i / row_vecs;
    uint32_t v = static_cast<uint32_t>(i - r * row_vecs);
    const int64_t slot = p.slot_map[r];
    if (slot < 0) continue;
    if (slot >= p.num_slots) {
      if (v == 0) atomic_status(p.status, GDN_STATUS_BAD_SLOT);
      continue;
    }
    const bool second = v >= va;
    if (second) v -= va;
    const KvRows& s = second ? p.b : p.a;
    const uint32_t head = v / s.vecs, e = (v - head * s.vecs) * 8;
    const int64_t from = r * s.src_row + head * s.src_head + e;
    uint4 x;
    if (p.bf16) {
      x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s.src) + from);
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(s.src) + from);
      const float4 lo = f[0], hi = f[1];
      x = make_uint4(pack_bf16(lo.x, lo.y), pack_bf16(lo.z, lo.w), pack_bf16(hi.x, hi.y), pack_bf16(hi.z, hi.w));
    }
    const int64_t page = slot / p.page_size, pos = slot - page * p.page_size;
    uint16_t* to = static_cast<uint16_t*>(s.dst) + page * s.dst_page + pos * s.dst_pos + head * s.dst_head + e;
    *reinterpret_cast<uint4*>(to) = x;
  }
}

// Launch with programmatic stream serialisation: the kernel waits itself (griddep_wait)
// before its first read, so its launch overlaps the previous kernel's tail.
template <class P>
cudaError_t launch_overlapped(void (*kernel)(const P), const P& p, unsigned grid, unsigned threads, size_t smem,
                              unsigned cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1u, 1u};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t stream) {
  const size_t smem = (5u * p.B + 1u) * sizeof(int32_t);
  const cudaError_t err = cudaFuncSetAttribute(gdn_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (5 * kMaxPlanBatch + 1) * static_cast<int>(sizeof(int32_t)));
  if (err != cudaSuccess) return err;
  // a few rounds of one CTA cost less than the cluster's start and barrier
  const unsigned ctas = p.slot_capacity > 4 * kPlanThreads || p.B > 4 * kPlanThreads ? kPlanCluster : 1;
  return launch_overlapped(gdn_kv_plan_kernel, p, ctas, kPlanThreads, smem, ctas, stream);
}

cudaError_t launch_kv_release(const KvReleaseParams& p, cudaStream_t stream) {
  return launch_overlapped(gdn_kv_release_kernel, p, 1u, kPlanThreads, 0, 1u, stream);
}

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  const int64_t all = static_cast<int64_t>(p.n) * (p.a.vecs + p.b.vecs) * p.heads;
  const int64_t blocks = (all + kAppendThreads - 1) / kAppendThreads;
  const unsigned grid = static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8);
  return launch_overlapped(gdn_kv_append_kernel, p, grid, kAppendThreads, 0, 1u, stream);
}

}  // namespace gdn
