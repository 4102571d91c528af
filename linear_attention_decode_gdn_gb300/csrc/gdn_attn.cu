// gdn_attn.cu -- attention over the paged cache on the CUDA cores (every shape), and the
// kernel that joins the partial results of split units for both attention kernels.
#include "gdn_attn.cuh"

#include <cuda_bf16.h>

namespace gdn {

namespace {

using namespace attn;

constexpr int kThreads = 128;  // one thread a position of the tile
constexpr int kCols = 8;       // query rows a CTA takes at a time
constexpr int kMaxDk = 576, kMaxDv = 512;
constexpr int kPairs = kMaxDv / (2 * kThreads);  // pairs of value elements a thread sums

__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

struct GeneralSmem {
  float q[kMaxDk][kCols];  // element-major: a thread reads its columns as two vectors
  float w[kTile][kCols];
  int64_t v_at[kTile];     // element offset of the position's value row; -1: not in use
  float warp_max[kThreads / 32][kCols], warp_sum[kThreads / 32][kCols];
};

// One online softmax over the unit's tiles, in fp32 throughout. Scores: a thread owns a
// position and reads its key row in 16-byte vectors, the query elements are broadcast from
// shared memory. Sums: a thread owns pairs of value elements and runs over the positions.
// This is the kernel for shapes that have no tensor-core instance, so it trades speed for
// having no shape conditions but multiples of eight. Bound by the fp32 pipes and by shared-memory
// broadcasts: 128 requests x 32 heads of 128 over 8 kv heads, 4100 positions on average, took it
// 4.2 ms (0.5 TB/s), where the tensor-core kernel takes 0.32.
__global__ void __launch_bounds__(kThreads) gdn_attn_general_kernel(const AttnParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  GeneralSmem& sm = *reinterpret_cast<GeneralSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  write_empty<kThreads>(p, tid);
  const Share share = find_share(p, blockIdx.x);
  if (tid == 0) write_record(p, share, blockIdx.x);
  Walk walk(share);
  Segment seg;
  uint32_t bad = 0;
  while (walk.next(p, &seg)) {
    const int cols = min(p.ncol, p.cols - seg.col_base);
    __syncthreads();  // the last segment's shared arrays are free
    for (int i = tid; i < p.dk / 8 * kCols; i += kThreads) {
      const int c = i % kCols, e = i / kCols * 8;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (c < cols) {
        const int col = seg.col_base + c, t = col / p.group, h = seg.kv_head * p.group + (col - t * p.group);
        x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + seg.b * p.q_b + t * p.q_t +
                                              h * p.q_h + e);
      }
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sm.q[e + 2 * k][c] = lo_bf16(u[k]);
        sm.q[e + 2 * k + 1][c] = hi_bf16(u[k]);
      }
    }
    float m[kCols], l[kCols], acc[kPairs][kCols][2];
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      m[c] = -INFINITY;
      l[c] = 0.0f;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) acc[j][c][0] = acc[j][c][1] = 0.0f;
    }
    const int32_t lower = lower_bound_of(p, seg.n, seg.col_base / p.group);
    __syncthreads();

    for (int tile = seg.tile; tile < seg.tile + seg.tiles; ++tile) {
      const int32_t pos = tile * kTile + tid;
      float s[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) s[c] = 0.0f;
      int64_t v_at = -1;
      if (pos < seg.n && pos >= lower) {
        const int32_t page = p.table[static_cast<int64_t>(seg.b) * p.max_pages + pos / p.page_size];
        if (page < 0 || page >= p.num_pages) {
          bad = GDN_STATUS_BAD_PAGE;
        } else {
          const int32_t in = pos % p.page_size;
          v_at = page * p.v_page + in * p.v_pos + seg.kv_head * p.v_head;
          const uint16_t* k = static_cast<const uint16_t*>(p.k) + page * p.k_page + in * p.k_pos + seg.kv_head * p.k_head;
          for (int e = 0; e < p.dk; e += 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(k + e);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float kj = j & 1 ? hi_bf16(u[j >> 1]) : lo_bf16(u[j >> 1]);
#pragma unroll
              for (int c = 0; c < kCols; ++c) s[c] = fmaf(kj, sm.q[e + j][c], s[c]);
            }
          }
        }
      }
      sm.v_at[tid] = v_at;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const int col = seg.col_base + c, t = col / p.group;
        const int32_t last = seg.n - p.T + t;
        const bool seen = c < cols && v_at >= 0 && pos <= last && (p.window <= 0 || pos > last - p.window);
        s[c] = seen ? s[c] * p.scale_log2 : -INFINITY;
        float x = s[c];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        if (lane == 0) sm.warp_max[warp][c] = x;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float top = m[c];
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, sm.warp_max[w][c]);
        const float ref = top == -INFINITY ? 0.0f : top;  // nothing seen yet: every weight is 0
        const float f = exp2f(m[c] - ref);
        m[c] = top;
        const float w = exp2f(s[c] - ref);
        l[c] = l[c] * f + w;
        sm.w[tid][c] = w;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          acc[j][c][0] *= f;
          acc[j][c][1] *= f;
        }
      }
      __syncthreads();
      for (int i = 0; i < kTile; ++i) {
        const int64_t at = sm.v_at[i];
        if (at < 0) continue;
        float w[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) w[c] = sm.w[i][c];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const int d = 2 * (tid + j * kThreads);
          if (d >= p.dv) continue;
          const uint32_t x = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.v) + at + d);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            // a weight of zero leaves the value out, whatever it holds
            if (w[c] == 0.0f) continue;
            acc[j][c][0] = fmaf(w[c], lo_bf16(x), acc[j][c][0]);
            acc[j][c][1] = fmaf(w[c], hi_bf16(x), acc[j][c][1]);
          }
        }
      }
      __syncthreads();  // weights, offsets and maxima are read
    }

    // the threads' sums of weights, added
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const float x = warp_sum(l[c]);
      if (lane == 0) sm.warp_sum[warp][c] = x;
    }
    __syncthreads();
    float* part = partial_of(p, blockIdx.x, seg.index == 0 ? 0 : 1);
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      if (c >= cols) continue;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) sum += sm.warp_sum[w][c];
      if (seg.whole) {
        const int64_t row = row_of(p, seg.b, seg.kv_head, seg.col_base + c);
        const float inv = sum > 0.0f ? 1.0f / sum : (sum == sum ? 0.0f : sum);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const int d = 2 * (tid + j * kThreads);
          if (d < p.dv)
            *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.o) + row * p.dv + d) =
                __floats2bfloat162_rn(acc[j][c][0] * inv, acc[j][c][1] * inv);
        }
        if (tid == 0 && p.lse != nullptr) p.lse[row] = lse_of(m[c], sum);
      } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const int d = 2 * (tid + j * kThreads);
          if (d < p.dv) *reinterpret_cast<float2*>(part + c * p.dv + d) = make_float2(acc[j][c][0], acc[j][c][1]);
        }
        if (tid == 0) {
          part[p.ncol * p.dv + c] = m[c];
          part[p.ncol * p.dv + p.ncol + c] = sum;
        }
      }
    }
  }
  if (bad != 0u) atomic_status(p.status, bad);
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWidth = 128;  // value elements a warp adds: four a lane

// Block (i, .) looks at the border between the shares of workers i and i + 1. Where it is the
// first border inside a unit, its warps add the unit's partial results, each for one column and
// kJoinWidth value elements, in the order of the workers, so the sums do not depend on timing:
// m = max m_j, l = sum 2^(m_j - m) l_j, o = sum 2^(m_j - m) o_j / l.
// Bound by latency, so a warp waits for two loads only: the record, then references, sums and
// the first parts together (one request of 131,071 positions, 8 units in 19 parts: about 3 us of
// 86 with the launch; a block a column that walked the records took 8). AHEAD parts are in
// flight: more shorten long lists of parts, fewer leave registers for more blocks.
template <int AHEAD>
__global__ void __launch_bounds__(kJoinThreads) gdn_attn_join_kernel(const AttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.x + 1, lane = threadIdx.x & 31;
  const uint4 r = *reinterpret_cast<const uint4*>(p.records + static_cast<size_t>(i) * kRecordInts);
  if (r.x == 0) return;
  const int parts = static_cast<int>(r.x), slot0 = static_cast<int>(r.y), b = static_cast<int>(r.z), unit = static_cast<int>(r.w);
  const int kv_head = unit / p.col_groups, col_base = (unit - kv_head * p.col_groups) * p.ncol;
  const int cols = min(p.ncol, p.cols - col_base);
  const int widths = (p.dv + kJoinWidth - 1) / kJoinWidth;
  const int task = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int c = task / widths, d = (task - c * widths) * kJoinWidth + lane * 4;
  if (c >= cols) return;
  const size_t floats = partial_floats(p);
  const float* const first = partial_of(p, i - 1, slot0);
  const float* const second = partial_of(p, i, 0);  // and so on, two apart
  auto part = [&](int j) { return j == 0 ? first : second + (j - 1) * 2 * floats; };
  const int64_t at = static_cast<int64_t>(c) * p.dv + d, ref = static_cast<int64_t>(p.ncol) * p.dv + c;
  const bool mine = d < p.dv;

  float4 ahead[AHEAD];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (mine && j < parts) ahead[j] = *reinterpret_cast<const float4*>(part(j) + at);
  float m = -INFINITY;
  bool lost = false;
  for (int j = lane; j < parts; j += 32) {
    const float mj = part(j)[ref];
    lost |= mj != mj;
    m = fmaxf(m, mj);
  }
  // a worker that gave up left nothing to add: the row stays as it is, and the status tells
  if (__any_sync(0xffffffffu, lost)) return;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float zero = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](float w, const float4& x) {
    o.x = fmaf(w, x.x, o.x);
    o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z);
    o.w = fmaf(w, x.w, o.w);
  };
  for (int j0 = 0; j0 < parts; j0 += 32) {
    const bool have = j0 + lane < parts;
    const float w = have ? exp2f(part(j0 + lane)[ref] - zero) : 0.0f;
    if (have) l = fmaf(w, part(j0 + lane)[ref + p.ncol], l);
    const int count = min(32, parts - j0);
    for (int j1 = 0; j1 < count; j1 += AHEAD) {
      if (j0 + j1 > 0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (mine && j1 + j < count) ahead[j] = *reinterpret_cast<const float4*>(part(j0 + j1 + j) + at);
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, (j1 + j) & 31);
        if (mine && j1 + j < count) add(wj, ahead[j]);
      }
    }
  }
  l = warp_sum(l);
  const int64_t row = row_of(p, b, kv_head, col_base + c);
  if (mine) {
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    __nv_bfloat162* const to = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.o) + row * p.dv + d);
    to[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    to[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  }
  if (d == 0 && p.lse != nullptr) p.lse[row] = lse_of(m, l);
}

}  // namespace

// The tensor-core kernel needs rows made of whole 64-element chunks, pages that fill a tile in
// whole boxes, and strides that a tensor map can hold.
//
// Columns: the narrowest of 16, 32 and 64 that holds the query rows of a kv head; more rows are
// column groups that read the cache again, from L2 as their tiles are side by side in time. A
// latent row's 64 columns cost 83 us where 32 cost 61 and 16 cost 57 (4 x 65,535 positions).
// What a unit counts for beyond its tiles was swept over 1, 2, 3, 5 and 8: heads of 64 gain from 3
// (a verify step of 32 requests with a window: 30.4 us at 1, 23.4 at 3), latent rows from 3 (128
// requests: 119.4 us at 1, 114.5 at 3), heads of 128 and 256 are within 1% of each other.
AttnPlan attn_plan(const gdn_paged_kv& kv, int cols) {
  const bool latent = kv.v == nullptr;
  const bool heads = latent ? kv.dk == 576 && kv.dv == 512
                            : kv.dk == kv.dv && (kv.dk == 64 || kv.dk == 128 || kv.dk == 256);
  const int ps = kv.page_size;
  const bool pages = ps == 16 || ps == 32 || ps == 64 || ps % kTile == 0;
  auto strides = [&](const int64_t* s) {
    const int32_t extent[3] = {kv.num_pages, kv.page_size, kv.num_kv_heads};
    for (int i = 0; i < 3; ++i)
      if (extent[i] > 1 && (s[i] <= 0 || s[i] >= (int64_t{1} << 39))) return false;
    return true;
  };
  if (!heads || !pages || !strides(kv.k_strides) || (!latent && !strides(kv.v_strides))) return {false, kCols, kMaxAttnCtas, 1};
  // a latent cache is read by pairs of CTAs
  return {true, cols <= 16 ? 16 : cols <= 32 ? 32 : 64, latent ? kSms / 2 : kSms, latent ? 3 : kv.dk == 256 ? 1 : kv.dk == 128 ? 2 : 3};
}

size_t attn_workspace_bytes(const AttnPlan& plan, int dv) {
  return kRecordBytes + static_cast<size_t>(plan.max_workers) * 2 * plan.ncol * (dv + 2) * sizeof(float);
}

cudaError_t launch_attn_general(AttnParams& p, cudaStream_t stream) {
  static std::atomic<bool> allowed[kDevices];
  const cudaError_t err =
      allow_shared(reinterpret_cast<const void*>(gdn_attn_general_kernel), static_cast<int>(sizeof(GeneralSmem)), allowed);
  if (err != cudaSuccess) return err;
  return launch_overlapped(gdn_attn_general_kernel, p, dim3(p.workers), kThreads, sizeof(GeneralSmem), 1u, stream);
}

cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t stream) {
  const unsigned cols = static_cast<unsigned>(p.cols < p.ncol ? p.cols : p.ncol);
  const unsigned tasks = cols * ((p.dv + kJoinWidth - 1) / kJoinWidth), warps = kJoinThreads / 32;
  const dim3 grid(p.workers - 1, (tasks + warps - 1) / warps);
  // By the parts that units of equal length would have. One request on 2 kv heads (76 parts): 21.9,
  // 17.1, 15.4 us for the whole call with 4, 8, 16 ahead; one on 2 kv heads in 8 parts: 9.3, 8.9,
  // 9.3; 67 requests on latent rows: 25.7, 26.4, 29.4.
  const int64_t units = static_cast<int64_t>(p.B) * p.heads_kv * p.col_groups;
  auto kernel = p.workers >= 16 * units ? gdn_attn_join_kernel<16>
                : p.workers >= 4 * units ? gdn_attn_join_kernel<8> : gdn_attn_join_kernel<4>;
  return launch_overlapped(kernel, p, grid, kJoinThreads, 0, 1u, stream);
}

cudaError_t launch_attn(const AttnPlan& plan, AttnParams& p, cudaStream_t stream) {
  p.ncol = plan.ncol;
  p.unit_cost = plan.unit_cost;
  p.col_groups = (p.cols + p.ncol - 1) / p.ncol;
  // at most one worker a tile that there could be
  const int64_t positions = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int64_t per_unit = (positions + kTile - 1) / kTile;
  const int64_t most = per_unit * p.B * p.heads_kv * p.col_groups;
  p.workers = static_cast<uint32_t>(most < plan.max_workers ? most : plan.max_workers);
  const cudaError_t err = plan.tensor ? launch_attn_tc(p, stream) : launch_attn_general(p, stream);
  if (err != cudaSuccess) return err;
  // a unit of one tile is never split
  return p.workers > 1 && per_unit > 1 ? launch_attn_join(p, stream) : cudaSuccess;
}

}  // namespace gdn
