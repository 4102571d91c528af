// gdn_kv.cu -- the paged cache: pages and slots for new tokens (gdn_kv_plan), pages given
// back (gdn_kv_release) and rows written to their slots (gdn_kv_append).
#include "gdn_device.cuh"
#include "gdn_kv.h"

namespace gdn {

namespace {

constexpr int kReleaseThreads = 512;
constexpr int kPlanCluster = 8;
constexpr int kAtOnce = 4;  // tokens a thread gives slots to at a time

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

// Largest b in [0, n) with sums[b] <= x (sums rise; sums[0] = 0), for COUNT values at once: their
// searches wait for shared memory together.
template <int COUNT>
__device__ __forceinline__ void find_rows(const int32_t* sums, int n, const int (&x)[COUNT], int (&b)[COUNT]) {
#pragma unroll
  for (int k = 0; k < COUNT; ++k) b[k] = 0;
  for (int half = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; half > 0; half >>= 1) {
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
      const int mid = b[k] + half;
      if (mid < n && sums[mid] <= x[k]) b[k] = mid;
    }
  }
}

// Every CTA takes the whole batch's sums for itself, in shared memory: that is 12 bytes read a
// request and spares a second launch or a grid barrier. Then the CTAs share the tokens and the
// pages. Where outputs are the inputs' own arrays (in_place), no CTA may write before all have
// read: the grid is one cluster then, with its barrier in between.
// Bound by instructions for prompts: a token costs a search over the sums and a division, so
// they want many SMs (512 requests, 131,000 tokens, pages of 16: 6.5 us; 21 us in place, on one
// cluster of 8 CTAs). Bound by latency for a decode step (256 requests: 3.8 us in one CTA).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) gdn_kv_plan_kernel(const KvPlanParams p) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_sums[THREADS / 32];
  __shared__ int32_t handed;            // free pages handed out
  int32_t* cu = sm;                     // [B + 1] tokens before request b
  int32_t* fresh_cu = cu + p.B + 1;     // [B] pages handed out before request b
  int32_t* start = fresh_cu + p.B;      // [B] cached length; -1 for a request without slots
  int32_t* held = start + p.B;          // [B] pages the request had
  int32_t* held_new = held + p.B;       // [B] and has now
  int32_t* len_new = held_new + p.B;    // [B] kv_len
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();

  uint32_t bad = 0;
  int32_t avail = p.free_count[0];
  const int32_t given = avail;
  if (avail < 0 || avail > p.free_capacity) {
    avail = 0;
    bad |= GDN_STATUS_BAD_LEN;
  }
  if (tid == 0) handed = 0;
  int64_t tokens = 0, pages = 0;  // of the requests before this chunk
  for (int base = 0; base < p.B; base += THREADS) {
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
    const int64_t upto = tokens + block_scan<THREADS>(n, warp_sums, &total);
    tokens += total;
    const int64_t length = static_cast<int64_t>(c) + n;
    const int64_t need = (length + p.page_size - 1) / p.page_size;
    if (!skip && (h < 0 || h > p.max_pages || need > p.max_pages || length > 0x7fffffffLL ||
                  upto > p.slot_capacity)) {
      skip = true;
      bad |= GDN_STATUS_BAD_LEN;
    }
    const int64_t want = skip || need <= h ? 0 : need - h;
    const int64_t pages_upto = pages + block_scan<THREADS>(want, warp_sums, &total);
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
      start[b] = skip ? -1 : c;
      len_new[b] = !skip ? c + n : c == -1 ? 0 : c;
      held[b] = h;
      held_new[b] = fits ? h + static_cast<int32_t>(want) : h;
    }
  }
  if (bad != 0u && blockIdx.x == 0) atomic_status(p.status, bad);
  if (p.in_place && gridDim.x > 1) cluster_sync_all(); else __syncthreads();

  const int first = blockIdx.x * THREADS + tid, step = gridDim.x * THREADS;
  for (int b = first; b <= p.B; b += step) {
    p.cu_new[b] = cu[b];
    if (b == p.B) {
      // a count outside the list is left for the caller to see
      p.free_count_out[0] = given != avail ? given : avail - handed;
      break;
    }
    p.kv_len[b] = len_new[b];
    p.held_out[b] = held_new[b];
  }
  uint32_t bad_page = 0;
  for (int f = first; f < handed; f += step) {
    const int wanted[1] = {f};
    int found[1];
    find_rows(fresh_cu, p.B, wanted, found);
    const int b = found[0];
    int32_t page = p.free_list[avail - 1 - f];
    if (page < 0 || page >= p.num_pages) {
      page = -1;
      bad_page = GDN_STATUS_BAD_PAGE;
    }
    p.table[static_cast<int64_t>(b) * p.max_pages + held[b] + (f - fresh_cu[b])] = page;
  }
  const int32_t all = cu[p.B];
  for (int64_t i0 = first; i0 < p.slot_capacity; i0 += static_cast<int64_t>(step) * kAtOnce) {
    int i[kAtOnce], row[kAtOnce], off[kAtOnce], page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t at = i0 + static_cast<int64_t>(k) * step;
      i[k] = at < all ? static_cast<int>(at) : -1;
    }
    find_rows(cu, p.B, i, row);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int b = row[k];
      const int32_t c = start[b];
      page[k] = -1;
      off[k] = 0;
      if (i[k] < 0 || c < 0) continue;
      const uint32_t pos = static_cast<uint32_t>(c) + static_cast<uint32_t>(i[k] - cu[b]);
      const int32_t idx = static_cast<int32_t>(pos / static_cast<uint32_t>(p.page_size));
      off[k] = static_cast<int32_t>(pos - static_cast<uint32_t>(idx) * p.page_size);
      page[k] = idx < held[b] ? p.table[static_cast<int64_t>(b) * p.max_pages + idx]
                              : p.free_list[avail - 1 - (fresh_cu[b] + idx - held[b])];
      if (page[k] < 0 || page[k] >= p.num_pages) {
        page[k] = -1;
        bad_page = GDN_STATUS_BAD_PAGE;
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t at = i0 + static_cast<int64_t>(k) * step;
      if (at < p.slot_capacity) p.slot_map[at] = page[k] < 0 ? -1 : static_cast<int64_t>(page[k]) * p.page_size + off[k];
    }
  }
  if (bad_page != 0u) atomic_status(p.status, bad_page);
}

// One CTA: the requests' page counts are summed so that each knows where its pages go, and
// the warps copy them. Finished requests are few; nothing here is worth more CTAs.
__global__ void __launch_bounds__(kReleaseThreads) gdn_kv_release_kernel(const KvReleaseParams p) {
  __shared__ int64_t warp_sums[kReleaseThreads / 32];
  __shared__ int32_t at[kReleaseThreads], row[kReleaseThreads], count[kReleaseThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  uint32_t bad = 0;
  int64_t top = p.free_count[0];
  __syncthreads();  // read by all before thread 0 writes it at the end
  if (top < 0 || top > p.free_capacity) {
    if (tid == 0) atomic_status(p.status, GDN_STATUS_BAD_LEN);
    return;
  }
  for (int base = 0; base < p.n; base += kReleaseThreads) {
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
    const int64_t upto = block_scan<kReleaseThreads>(h, warp_sums, &total);
    // past the list's end this request and the later ones of the chunk keep their pages
    const bool fits = top + upto <= p.free_capacity;
    if (h > 0 && !fits) bad |= GDN_STATUS_BAD_LEN;
    at[tid] = static_cast<int32_t>(top + upto - h);
    row[tid] = b;
    count[tid] = fits ? h : 0;
    if (h > 0 && fits) p.held[b] = 0;
    int64_t kept;
    block_scan<kReleaseThreads>(fits ? h : 0, warp_sums, &kept);
    __syncthreads();
    for (int j = warp; j < kReleaseThreads; j += kReleaseThreads / 32) {
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

// A token's 8-element vectors (of both sources) are copied by a warp, or by 2^k lanes of one where
// they are that few, with kFlight of them a lane in flight: the slot and its page are looked up
// once a token, neighbouring lanes move neighbouring 16 bytes, and a lane's loads are all under
// way before its first store. Bound by HBM: 32,749 tokens of 8 + 8 heads of 128 (bf16) take 42 us,
// 0.93 of the measured copy bandwidth.
template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads) gdn_kv_append_kernel(const KvAppendParams p) {
  constexpr int kFlight = BF16 ? 8 : 4;
  griddep_launch_dependents();
  griddep_wait();
  const int lanes = p.lanes, lane = threadIdx.x & (lanes - 1);
  const uint32_t va = p.a.vecs * p.a.heads, all = va + p.b.vecs * p.b.heads;
  const int64_t rows_at_once = static_cast<int64_t>(gridDim.x) * (kAppendThreads / lanes);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / lanes) + threadIdx.x / lanes; r < p.n; r += rows_at_once) {
    const int64_t slot = p.slot_map[r];
    for (uint32_t v0 = lane; v0 < all; v0 += lanes * kFlight) {
      uint4 x[kFlight], y[kFlight];  // y: the second half of fp32 vectors
      int64_t to[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        uint32_t v = v0 + k * lanes;
        if (v >= all) break;
        const bool second = v >= va;
        if (second) v -= va;
        const KvRows& s = second ? p.b : p.a;
        const uint32_t head = s.heads == 1 ? 0u : v / s.vecs, e = (v - head * s.vecs) * 8;
        const int64_t from = r * s.src_row + head * s.src_head + e;
        to[k] = head * s.dst_head + e;
        const uint4* f = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(s.src) + from * (BF16 ? 2 : 4));
        x[k] = f[0];
        if (!BF16) y[k] = f[1];
      }
      // what was read is dropped where the token has no slot: the loads need not wait for it
      if (slot < 0) break;
      if (slot >= p.num_slots) {
        if (v0 == 0) atomic_status(p.status, GDN_STATUS_BAD_SLOT);
        break;
      }
      // 32 bits hold most slots, and their division is several times shorter
      const int64_t page = slot <= 0x7fffffff ? static_cast<int64_t>(static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size))
                                              : slot / p.page_size;
      const int64_t pos = slot - page * p.page_size;
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const uint32_t v = v0 + k * lanes;
        if (v >= all) break;
        const KvRows& s = v >= va ? p.b : p.a;
        uint4 z = x[k];
        if (!BF16) {
          auto f = [](uint32_t bits) { return __uint_as_float(bits); };
          z = make_uint4(pack_bf16(f(x[k].x), f(x[k].y)), pack_bf16(f(x[k].z), f(x[k].w)), pack_bf16(f(y[k].x), f(y[k].y)),
                         pack_bf16(f(y[k].z), f(y[k].w)));
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.dst) + page * s.dst_page + pos * s.dst_pos + to[k]) = z;
      }
    }
  }
}

}  // namespace

namespace {

template <int THREADS>
cudaError_t launch_plan(const KvPlanParams& p, unsigned ctas, cudaStream_t stream) {
  const size_t smem = (6u * p.B + 1u) * sizeof(int32_t);
  // static shared memory, up to 300 bytes of it here, counts towards the 48 KB too
  if (smem > 47 * 1024) {
    static std::atomic<bool> allowed[kDevices];
    const cudaError_t err = allow_shared(reinterpret_cast<const void*>(gdn_kv_plan_kernel<THREADS>),
                                         (6 * kMaxPlanBatch + 1) * static_cast<int>(sizeof(int32_t)), allowed);
    if (err != cudaSuccess) return err;
  }
  return launch_overlapped(gdn_kv_plan_kernel<THREADS>, p, dim3(ctas), THREADS, smem, p.in_place ? ctas : 1u, stream);
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams& given, cudaStream_t stream) {
  KvPlanParams p = given;
  p.in_place = p.kv_len == p.cached || p.held_out == p.held || p.free_count_out == p.free_count;
  // A decode step is one round of a small CTA (256 requests: 3.8 us, 4.1 with 512 threads).
  if (p.slot_capacity <= 1024 && p.B <= 1024) return launch_plan<256>(p, 1, stream);
  if (p.in_place) return launch_plan<1024>(p, kPlanCluster, stream);
  const unsigned ctas = (p.slot_capacity + 256u * kAtOnce - 1) / (256u * kAtOnce);
  return launch_plan<256>(p, ctas < 1 ? 1 : ctas < kSms ? ctas : kSms, stream);
}

cudaError_t launch_kv_release(const KvReleaseParams& p, cudaStream_t stream) {
  return launch_overlapped(gdn_kv_release_kernel, p, dim3(1), kReleaseThreads, 0, 1u, stream);
}

cudaError_t launch_kv_append(const KvAppendParams& given, cudaStream_t stream) {
  KvAppendParams p = given;
  uint32_t all = 0;
  for (KvRows* s : {&p.a, &p.b}) {
    if (s->heads > 1 && s->src_head == s->vecs * 8 && s->dst_head == s->vecs * 8) {  // heads in one piece
      s->vecs *= s->heads;
      s->heads = 1;
    }
    all += s->vecs * s->heads;
  }
  p.lanes = 1;
  while (p.lanes < 32 && static_cast<uint32_t>(p.lanes) < all) p.lanes *= 2;
  const int64_t rows = kAppendThreads / p.lanes, blocks = (p.n + rows - 1) / rows;
  const unsigned grid = static_cast<unsigned>(blocks < kSms * 32 ? blocks : kSms * 32);
  return launch_overlapped(p.bf16 ? gdn_kv_append_kernel<true> : gdn_kv_append_kernel<false>, p, dim3(grid), kAppendThreads, 0,
                           1u, stream);
}

}  // namespace gdn
