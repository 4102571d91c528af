// gdn_ssm.cu -- the selective state space recurrence for one token of every request (gdn_ssm_step):
//
//   s = softplus(dt + dt_bias),  h <- exp(s a) h + s u b,  y = (c . h + skip u) silu(z)
//
// for every channel, with a state of N values. Its bytes are the states', read and written: HBM.
//   512 requests x 4096 channels x 16 states (bf16 inputs): 47 us, 6.1 TB/s (0.89 of the measured copy
//     bandwidth); 112 us with lanes that load every scalar for themselves.
//   64 requests: 7.2 us. One request x 2048 channels: 3.1 us, two dependent loads.
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kStepWarps = 4;  // of a CTA; they have nothing in common. Eight CTAs an SM: 47.7 us, 57 without that limit, 55 with ten

struct StepParams {
  gdn_ssm s;
  int32_t* status;
  int32_t per_group, blocks;  // channels of a group, and blocks of them
  int32_t columns;            // warps of a request
  int32_t rows;               // requests of a warp
};

// The states of a request are read and written once, and nothing else is of that size. A warp takes
// CH channels: LANES lanes hold a channel's states, four each, in PASSES of 32 / LANES channels, so
// that every access is 512 bytes in a row and a thread's are in flight together. What a channel
// takes once (steps, gate, readout) is done by the lane that the sums over the states end up in,
// and comes to the others by shuffles.
template <int N, bool BF16>
__global__ void __launch_bounds__(kStepWarps * 32, 8) gdn_ssm_step_kernel(const StepParams p) {
  constexpr int LANES = N / 4, PASSES = LANES < 4 ? LANES : 4, WIDTH = 32 / LANES, CH = PASSES * WIDTH, SHARE = LANES / PASSES;
  const gdn_ssm& s = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t task = blockIdx.x * kStepWarps + warp, first = task / p.columns;
  const int block = static_cast<int>(task - first * p.columns), group = block / p.blocks, in_group = (block - group * p.blocks) * CH;
  const int c0 = group * p.per_group + in_group, count = min(CH, p.per_group - in_group);
  const int part = lane % LANES, at = lane / LANES;  // states 4 part .. of channel pass * WIDTH + at
  float a[PASSES][4];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i * WIDTH + at < count) x = *reinterpret_cast<const float4*>(s.a + static_cast<int64_t>(c0 + i * WIDTH + at) * N + part * 4);
    a[i][0] = x.x * kLog2e, a[i][1] = x.y * kLog2e, a[i][2] = x.z * kLog2e, a[i][3] = x.w * kLog2e;
  }
  // the channel that this lane reads out: sums end up in lane part = SHARE * pass
  const int own = part / SHARE * WIDTH + at, d = c0 + own;
  const bool owns = part % SHARE == 0 && own < count;
  const bool softplus = (s.flags & GDN_DT_SOFTPLUS) != 0u;
  const float bias = owns && s.dt_bias != nullptr ? s.dt_bias[d] : 0.0f, skip = owns && s.skip != nullptr ? s.skip[d] : 0.0f;
  for (int r = 0; r < p.rows; ++r) {
    const int b = static_cast<int>(first) * p.rows + r;
    if (b >= s.batch) return;
    const int slot = s.slot[b];
    if (slot < 0) continue;
    if (slot >= s.num_slots) {
      if (block == 0 && lane == 0) atomic_status(p.status, GDN_STATUS_BAD_SLOT);
      continue;
    }
    float* const state = s.state + (static_cast<int64_t>(slot) * s.channels + c0 + at) * N + part * 4;
    float4 h[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      if (i * WIDTH + at < count) h[i] = *reinterpret_cast<const float4*>(state + i * WIDTH * N);
    float bn[4], cn[4], u = 0.0f, dt = 0.0f, z = 0.0f;
    auto four = [&](const void* base, const int64_t* strides, float (&x)[4]) {
      const int64_t from = b * strides[0] + group * strides[2] + part * 4;
      if constexpr (BF16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + from);
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + from);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      }
    };
    four(s.b, s.b_strides, bn);
    four(s.c, s.c_strides, cn);
    if (owns) {
      u = elem<BF16>(s.u, b * s.u_strides[0] + d);
      dt = elem<BF16>(s.dt, b * s.dt_strides[0] + d);
      if (s.z != nullptr) z = elem<BF16>(s.z, b * s.z_strides[0] + d);
    }
    dt += bias;
    if (softplus) dt = fmaxf(dt, 0.0f) + log1pf(expf(-fabsf(dt)));
    const float du = dt * u;
    float sum[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int from = at * LANES + i * SHARE;
      const float st = __shfl_sync(0xffffffffu, dt, from), su = __shfl_sync(0xffffffffu, du, from);
      h[i].x = fmaf(ex2(st * a[i][0]), h[i].x, su * bn[0]);
      h[i].y = fmaf(ex2(st * a[i][1]), h[i].y, su * bn[1]);
      h[i].z = fmaf(ex2(st * a[i][2]), h[i].z, su * bn[2]);
      h[i].w = fmaf(ex2(st * a[i][3]), h[i].w, su * bn[3]);
      if (i * WIDTH + at < count) *reinterpret_cast<float4*>(state + i * WIDTH * N) = h[i];
      sum[i] = fmaf(h[i].x, cn[0], fmaf(h[i].y, cn[1], fmaf(h[i].z, cn[2], h[i].w * cn[3])));
    }
    // Sums over a channel's lanes: a lane keeps half of its passes and gives the other half away until
    // it has one; further lanes add what is left.
#pragma unroll
    for (int off = LANES / 2, n = PASSES; off > 0; off /= 2, n = n > 1 ? n / 2 : 1) {
      const bool upper = (part & off) != 0;
      if (n == 1) {
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], off);
        continue;
      }
#pragma unroll
      for (int i = 0; i < n / 2; ++i)
        sum[i] = (upper ? sum[n / 2 + i] : sum[i]) + __shfl_xor_sync(0xffffffffu, upper ? sum[i] : sum[n / 2 + i], off);
    }
    if (owns) {
      float y = fmaf(skip, u, sum[0]);
      if (s.z != nullptr) y *= siluf_(z);
      set_elem<BF16>(s.y, static_cast<int64_t>(b) * s.channels + d, y);
    }
  }
}

template <int N, bool BF16>
cudaError_t launch_step(const SsmParams& given, cudaStream_t stream) {
  constexpr int LANES = N / 4, CH = (LANES < 4 ? LANES : 4) * (32 / LANES);
  StepParams p{given.s, given.status, given.s.channels / given.s.num_groups, 0, 0, 1};
  p.blocks = (p.per_group + CH - 1) / CH;
  p.columns = p.blocks * p.s.num_groups;
  const int64_t all = static_cast<int64_t>(p.columns) * p.s.batch;
  p.rows = all >= 32768 ? 2 : 1;  // a is loaded once for both: 47.7 us at 2, 48.3 at 4, 50.3 at 1 (512 x 4096 channels)
  const int64_t warps = static_cast<int64_t>(p.columns) * ((p.s.batch + p.rows - 1) / p.rows);
  return launch_overlapped(gdn_ssm_step_kernel<N, BF16>, p, dim3(static_cast<unsigned>((warps + kStepWarps - 1) / kStepWarps)),
                           kStepWarps * 32, 0, 1u, stream);
}

template <bool BF16>
cudaError_t launch_type(const SsmParams& p, cudaStream_t stream) {
  switch (p.s.state_size) {
    case 8: return launch_step<8, BF16>(p, stream);
    case 16: return launch_step<16, BF16>(p, stream);
    case 32: return launch_step<32, BF16>(p, stream);
    default: return launch_step<64, BF16>(p, stream);
  }
}

}  // namespace

cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t stream) {
  return (p.s.flags & GDN_QKV_BF16) != 0u ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

}  // namespace gdn
