// gdn_ssm.cu -- the selective state space recurrence over prompts (gdn_ssm_scan) and for one token
// of every request (gdn_ssm_step):
//
//   s = softplus(dt + dt_bias),  h <- exp(s a) h + s u b,  y = (c . h + skip u) silu(z)
//
// for every channel, with a state of N values.
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kSsmThreads = 128;

// log(1 + e^x) without overflow and without cancellation.
__device__ __forceinline__ float softplusf_(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// N / 4 neighbouring lanes share a channel, four states each, and run over the positions.
template <int N, bool BF16>
__global__ void __launch_bounds__(kSsmThreads) gdn_ssm_kernel(const SsmParams p) {
  constexpr int kLanes = N / 4;
  const gdn_ssm& s = p.s;
  griddep_launch_dependents();
  griddep_wait();
  const int per = s.channels * kLanes;
  const int blocks = (per + kSsmThreads - 1) / kSsmThreads;
  const int b = blockIdx.x / blocks;
  const int item = (blockIdx.x - b * blocks) * kSsmThreads + threadIdx.x;
  const int slot = s.slot[b];
  if (slot < 0) return;
  const int len = s.seq_lens != nullptr ? s.seq_lens[b] : s.num_tokens;
  const bool bad_slot = slot >= s.num_slots, bad_len = len < 0 || len > s.num_tokens;
  if (bad_slot || bad_len) {
    if (item == 0) atomic_status(p.status, bad_slot ? GDN_STATUS_BAD_SLOT : GDN_STATUS_BAD_LEN);
    return;
  }
  if (len == 0) return;
  const bool live = item < per;  // all lanes of a warp run, for the sums over lanes
  const int d = live ? item / kLanes : 0, part = item % kLanes, n = part * 4;
  const int g = d / (s.channels / s.num_groups);
  float* const state = s.state + (static_cast<int64_t>(slot) * s.channels + d) * N + n;
  const float4 h4 = *reinterpret_cast<const float4*>(state);
  const float4 a4 = *reinterpret_cast<const float4*>(s.a + static_cast<int64_t>(d) * N + n);
  float h[4] = {h4.x, h4.y, h4.z, h4.w};
  const float a[4] = {a4.x, a4.y, a4.z, a4.w};
  const float skip = s.skip != nullptr ? s.skip[d] : 0.0f, bias = s.dt_bias != nullptr ? s.dt_bias[d] : 0.0f;
  for (int t = 0; t < len; ++t) {
    const float u = elem<BF16>(s.u, b * s.u_strides[0] + t * s.u_strides[1] + d);
    float dt = elem<BF16>(s.dt, b * s.dt_strides[0] + t * s.dt_strides[1] + d) + bias;
    if (s.flags & GDN_DT_SOFTPLUS) dt = softplusf_(dt);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float bj = elem<BF16>(s.b, b * s.b_strides[0] + t * s.b_strides[1] + g * s.b_strides[2] + n + j);
      const float cj = elem<BF16>(s.c, b * s.c_strides[0] + t * s.c_strides[1] + g * s.c_strides[2] + n + j);
      h[j] = fmaf(expf(dt * a[j]), h[j], dt * u * bj);
      sum = fmaf(h[j], cj, sum);
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (live && part == 0) {
      float y = fmaf(skip, u, sum);
      if (s.z != nullptr) y *= siluf_(elem<BF16>(s.z, b * s.z_strides[0] + t * s.z_strides[1] + d));
      set_elem<BF16>(s.y, (static_cast<int64_t>(b) * s.num_tokens + t) * s.channels + d, y);
    }
  }
  if (live) *reinterpret_cast<float4*>(state) = make_float4(h[0], h[1], h[2], h[3]);
}

template <bool BF16>
cudaError_t launch_type(const SsmParams& p, cudaStream_t stream) {
  const int64_t per = static_cast<int64_t>(p.s.channels) * (p.s.state_size / 4);
  const unsigned grid = static_cast<unsigned>((per + kSsmThreads - 1) / kSsmThreads * p.s.batch);
  switch (p.s.state_size) {
    case 8: return launch_overlapped(gdn_ssm_kernel<8, BF16>, p, dim3(grid), kSsmThreads, 0, 1u, stream);
    case 16: return launch_overlapped(gdn_ssm_kernel<16, BF16>, p, dim3(grid), kSsmThreads, 0, 1u, stream);
    case 32: return launch_overlapped(gdn_ssm_kernel<32, BF16>, p, dim3(grid), kSsmThreads, 0, 1u, stream);
    default: return launch_overlapped(gdn_ssm_kernel<64, BF16>, p, dim3(grid), kSsmThreads, 0, 1u, stream);
  }
}

}  // namespace

cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t stream) {
  return (p.s.flags & GDN_QKV_BF16) != 0u ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

}  // namespace gdn
