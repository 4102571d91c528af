// gdn_norm.cu -- the residual's addition and the root-mean-square norm of a row, with an output in
// bf16, fp32 or e4m3 with scales (gdn_add_rms_norm).
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kMaxThreads = 1024;
constexpr float kTop = 448.0f;    // the largest e4m3 value
constexpr float kLeast = 1e-30f;  // scales are made as if the largest value were at least this

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row a CTA, in registers between its two passes: V vectors of 8 elements a thread.
template <bool XB, bool RB, int OT, int V>
__global__ void __launch_bounds__(kMaxThreads) gdn_norm_kernel(const gdn_norm p) {
  __shared__ float sums[32], tops[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  float y[V][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * blockDim.x + tid) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[j][k] = 0.0f;
    if (e >= p.width) continue;
    floats8<XB>(load8<XB>(p.x, row * p.x_stride + e), y[j]);
    if (p.residual != nullptr) {
      float r[8];
      floats8<RB>(load8<RB>(p.residual, row * p.residual_stride + e), r);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[j][k] += r[k];
      store8<RB>(p.residual, row * p.residual_stride + e, raw8<RB>(y[j]));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(y[j][k], y[j][k], sum);
  }
  sum = warp_sum(sum);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  sum = warp_sum(lane < warps ? sums[lane] : 0.0f);
  const float inv = 1.0f / sqrtf(sum / static_cast<float>(p.width) + p.eps);
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * blockDim.x + tid) * 8;
    float w[8];
    if (p.weight != nullptr && e < p.width) floats8<false>(load8<false>(p.weight, e), w);
    float group_top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[j][k] *= inv;
      if (p.weight != nullptr && e < p.width) y[j][k] *= w[k];
      group_top = max_nan(group_top, fabsf(y[j][k]));
    }
    if (OT != GDN_TYPE_E4M3) {
      if (e < p.width) store8<OT == GDN_TYPE_BF16>(p.o, row * p.width + e, raw8<OT == GDN_TYPE_BF16>(y[j]));
    } else if (p.group != 0) {
      // 16 neighbouring lanes hold a group's 128 channels
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) group_top = max_nan(group_top, __shfl_xor_sync(0xffffffffu, group_top, off));
      const float s = max_nan(group_top, kLeast) / kTop, to = 1.0f / s;
      if (e < p.width) {
        if ((lane & 15) == 0) p.scales[row * ((p.width + kNormGroup - 1) / kNormGroup) + e / kNormGroup] = s;
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 8; k += 4)
          q[k / 4] = pack_e4m3(y[j][k] * to, y[j][k + 1] * to) | pack_e4m3(y[j][k + 2] * to, y[j][k + 3] * to) << 16;
        *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p.o) + row * p.width + e) = make_uint2(q[0], q[1]);
      }
    } else {
      top = max_nan(top, group_top);
    }
  }
  if (OT == GDN_TYPE_E4M3 && p.group == 0) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = lane < warps ? tops[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float s = max_nan(top, kLeast) / kTop, to = 1.0f / s;
    if (tid == 0) p.scales[row] = s;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = (j * blockDim.x + tid) * 8;
      if (e >= p.width) continue;
      uint32_t q[2];
#pragma unroll
      for (int k = 0; k < 8; k += 4)
        q[k / 4] = pack_e4m3(y[j][k] * to, y[j][k + 1] * to) | pack_e4m3(y[j][k + 2] * to, y[j][k + 3] * to) << 16;
      *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p.o) + row * p.width + e) = make_uint2(q[0], q[1]);
    }
  }
}

template <bool XB, bool RB, int OT>
cudaError_t launch_row(const gdn_norm& p, cudaStream_t stream) {
  const int vecs = p.width / 8;
  const unsigned one = static_cast<unsigned>((vecs + 31) / 32 * 32), two = static_cast<unsigned>(((vecs + 1) / 2 + 31) / 32 * 32);
  if (one <= kMaxThreads) return launch_overlapped(gdn_norm_kernel<XB, RB, OT, 1>, p, dim3(p.rows), one, 0, 1u, stream);
  return launch_overlapped(gdn_norm_kernel<XB, RB, OT, 2>, p, dim3(p.rows), two, 0, 1u, stream);
}

template <bool XB, bool RB>
cudaError_t launch_out(const gdn_norm& p, cudaStream_t stream) {
  switch (p.o_type) {
    case GDN_TYPE_BF16: return launch_row<XB, RB, GDN_TYPE_BF16>(p, stream);
    case GDN_TYPE_FP32: return launch_row<XB, RB, GDN_TYPE_FP32>(p, stream);
    default: return launch_row<XB, RB, GDN_TYPE_E4M3>(p, stream);
  }
}

}  // namespace

cudaError_t launch_add_rms_norm(const gdn_norm& p, cudaStream_t stream) {
  const bool xb = p.x_type == GDN_TYPE_BF16, rb = p.residual_type == GDN_TYPE_BF16;
  return xb ? (rb ? launch_out<true, true>(p, stream) : launch_out<true, false>(p, stream))
            : (rb ? launch_out<false, true>(p, stream) : launch_out<false, false>(p, stream));
}

}  // namespace gdn
