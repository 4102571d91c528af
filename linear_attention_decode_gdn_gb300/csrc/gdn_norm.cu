// gdn_norm.cu -- the residual's addition and the root-mean-square norm of a row, with an output in
// bf16, fp32 or e4m3 with scales (gdn_add_rms_norm):
//
//   r = x + residual,  y = r / sqrt(mean r^2 + eps) w,  and in 8 bits  s = max |y| / 448,  q = y / s
//
// One pass over memory: the row waits in registers for its sum, and then for its largest value. Bound
// by HBM for many rows, by latency (one load, one or two block sums) for few.
//   32749 x 4096, bf16 with a bf16 residual into e4m3 with a scale for 128: 142 us, 6.6 TB/s (0.98 of
//     the measured copy bandwidth; 202 us with one vector a thread).
//   256 x 4096 into e4m3 with a scale a row: 4.2 us. One row of 2048: 2.5 us, a launch's own time.
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

#include <cfloat>

namespace gdn {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kRowWarps = 4;  // rows of a CTA where a warp takes one: up to 256 channels (16384 x 256: 7.0 us, 18.0 a CTA each)
// Vectors of a thread, by the time at 64 / 256 / 1024 / 4096 / 16384 rows (bf16 into e4m3, a scale for 128):
//   4096 channels: one 2.9 3.9 7.7 26.7 92 us, two 3.5 3.9 7.0 24.6 82, four 4.2 4.9 8.2 24.4 77;
//   1024 channels: one 2.7 2.9 3.8 7.2 23.4, two 3.5 3.5 3.6 7.6 22.5, four in a warp 4.2 4.2 4.3 8.1 23.8.
// So one where a row has an SM to itself, or where two would leave a warp or two; four from kManyVecs on
// (2^24 elements), where they come from HBM and a thread should wait for much at once; else two.
constexpr int64_t kManyVecs = 1 << 21;
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

// A row stays in registers between the passes over it, V vectors of 8 elements a thread. It belongs to
// a CTA, or (WARP) to a warp of one.
template <bool XB, bool RB, int OT, int V, bool WARP>
__global__ void __launch_bounds__(V > 2 ? 512 : kMaxThreads) gdn_norm_kernel(const gdn_norm p) {
  __shared__ float sums[WARP ? 1 : 32], tops[WARP ? 1 : 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARP ? lane : threadIdx.x, threads = WARP ? 32 : blockDim.x, warps = threads >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (WARP && row >= p.rows) return;
  // over the row's threads, every one of which gets the result
  auto whole_sum = [&](float x) {
    x = warp_sum(x);
    if (WARP) return x;
    if (lane == 0) sums[warp] = x;
    __syncthreads();
    return warp_sum(lane < warps ? sums[lane] : 0.0f);
  };
  auto warp_top = [](float x, int lanes) {
    for (int off = lanes / 2; off > 0; off >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
  };
  auto whole_top = [&](float x) {
    x = warp_top(x, 32);
    if (WARP) return x;
    if (lane == 0) tops[warp] = x;
    __syncthreads();
    return warp_top(lane < warps ? tops[lane] : 0.0f, 32);
  };

  Raw8<XB> in[V];
  Raw8<RB> old[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * threads + tid) * 8;
    if (e >= p.width) continue;
    in[j] = load8<XB>(p.x, row * p.x_stride + e);
    if (p.residual != nullptr) old[j] = load8<RB>(p.residual, row * p.residual_stride + e);
  }
  float y[V][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * threads + tid) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[j][k] = 0.0f;
    if (e >= p.width) continue;
    floats8<XB>(in[j], y[j]);
    if (p.residual != nullptr) {
      float r[8];
      floats8<RB>(old[j], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[j][k] += r[k];
      store8<RB>(p.residual, row * p.residual_stride + e, raw8<RB>(y[j]));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(y[j][k], y[j][k], sum);
  }
  const float inv = 1.0f / sqrtf(whole_sum(sum) / static_cast<float>(p.width) + p.eps);

  // y / s rounded to fp32 and then to 8 bits. The product with 1 / s alone is up to one and a half
  // roundings off, which puts quotients next to a border on its other side (three of 10^7 values). One
  // step of its remainder, which is exact, gives the rounded quotient (Markstein, IBM J. Res. Dev. 34,
  // 1990): 0.4 us more for 256 x 4096 with a scale a row, nothing for many rows (142 us; 188 by division).
  auto store_e4m3 = [&](int e, const float (&v)[8], float s) {
    const float to = 1.0f / s, by = fminf(s, FLT_MAX);  // an infinite s makes what is finite 0
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = v[k] * to;
      x[k] = fmaf(fmaf(-x[k], by, v[k]), to, x[k]);
    }
    uint32_t q[2];
#pragma unroll
    for (int k = 0; k < 8; k += 4) q[k / 4] = pack_e4m3(x[k], x[k + 1]) | pack_e4m3(x[k + 2], x[k + 3]) << 16;
    *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p.o) + row * p.width + e) = make_uint2(q[0], q[1]);
  };
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * threads + tid) * 8;
    float w[8], group_top = 0.0f;
    const bool weighed = p.weight != nullptr && e < p.width;
    if (weighed) floats8<false>(load8<false>(p.weight, e), w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[j][k] *= inv;
      if (weighed) y[j][k] *= w[k];
      if (OT == GDN_TYPE_E4M3) group_top = max_nan(group_top, fabsf(y[j][k]));
    }
    if (OT != GDN_TYPE_E4M3) {
      if (e < p.width) store8<OT == GDN_TYPE_BF16>(p.o, row * p.width + e, raw8<OT == GDN_TYPE_BF16>(y[j]));
    } else if (p.group != 0) {
      const float s = max_nan(warp_top(group_top, kNormGroup / 8), kLeast) / kTop;  // 16 neighbouring lanes hold a group
      if (e < p.width) {
        if ((lane & 15) == 0) p.scales[row * ((p.width + kNormGroup - 1) / kNormGroup) + e / kNormGroup] = s;
        store_e4m3(e, y[j], s);
      }
    } else {
      top = max_nan(top, group_top);
    }
  }
  if (OT == GDN_TYPE_E4M3 && p.group == 0) {
    const float s = max_nan(whole_top(top), kLeast) / kTop;
    if (tid == 0) p.scales[row] = s;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = (j * threads + tid) * 8;
      if (e < p.width) store_e4m3(e, y[j], s);
    }
  }
}

template <bool XB, bool RB, int OT>
cudaError_t launch_row(const gdn_norm& p, cudaStream_t stream) {
  const int vecs = p.width / 8;
  auto threads = [&](int v) { return static_cast<unsigned>(((vecs + v - 1) / v + 31) / 32 * 32); };
  if (vecs <= 32) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.rows) + kRowWarps - 1) / kRowWarps);
    return launch_overlapped(gdn_norm_kernel<XB, RB, OT, 1, true>, p, dim3(grid), kRowWarps * 32, 0, 1u, stream);
  }
  if (vecs >= 512 && static_cast<int64_t>(p.rows) * vecs >= kManyVecs)
    return launch_overlapped(gdn_norm_kernel<XB, RB, OT, 4, false>, p, dim3(p.rows), threads(4), 0, 1u, stream);
  if (vecs <= 128 || (p.rows <= kSms && vecs <= kMaxThreads))
    return launch_overlapped(gdn_norm_kernel<XB, RB, OT, 1, false>, p, dim3(p.rows), threads(1), 0, 1u, stream);
  return launch_overlapped(gdn_norm_kernel<XB, RB, OT, 2, false>, p, dim3(p.rows), threads(2), 0, 1u, stream);
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
