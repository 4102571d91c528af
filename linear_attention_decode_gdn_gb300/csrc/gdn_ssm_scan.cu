// gdn_ssm_scan.cu -- the selective state space recurrence over prompts (gdn_ssm_scan):
//
//   s = softplus(dt + dt_bias),  h <- exp(s a) h + s u b,  y = (c . h + skip u) silu(z)
//
// for every channel, with a state of N values.
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4;            // of a CTA; they have nothing in common
constexpr float kLog2e = 1.44269504088896340736f;

// ---- pairs of fp32, one instruction each ----------------------------------------------------
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 x) {
  const float2 v = unpack2(x);
  return pack2(ex2(v.x), ex2(v.y));
}

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1]. log(1 + e) = 2 artanh(q) with
// q = e / (2 + e) <= 1/3: the odd series to q^13 is off by less than 2^-26 of it, for any e.
__device__ __forceinline__ float softplus_series(float x) {
  const float e = expf(-fabsf(x)), q = __fdividef(e, 2.0f + e), q2 = q * q;
  float r = fmaf(q2, 2.0f / 13, 2.0f / 11);
  r = fmaf(r, q2, 2.0f / 9);
  r = fmaf(r, q2, 2.0f / 7);
  r = fmaf(r, q2, 2.0f / 5);
  r = fmaf(r, q2, 2.0f / 3);
  r = fmaf(r, q2, 2.0f);
  return fmaf(r, q, fmaxf(x, 0.0f));
}
__device__ __forceinline__ float silu_fast(float z) { return __fdividef(z, 1.0f + expf(-z)); }

// A thread owns four states of four channels: LANES neighbouring lanes a set of four channels, CH
// channels a warp. STEPS positions are staged in shared memory at a time.
template <int N_, bool BF16_>
struct Cfg {
  static constexpr int N = N_;
  static constexpr bool BF16 = BF16_;
  static constexpr int LANES = N / 4, CH = 4 * (32 / LANES);
  static constexpr int STEPS = BF16 && N > 8 ? 16 : 8;
  static constexpr int ROW = CH / 8, ITEMS = STEPS * ROW, U = (ITEMS + 31) / 32;            // vectors of u, dt, z
  static constexpr int NROW = N / 8, NITEMS = 2 * STEPS * NROW, V = (NITEMS + 31) / 32;     // and of b and c
};

// A warp's part of shared memory. b and c are held twice each, next to one another, so that a pair
// of channels meets them as a pair.
template <class C>
struct WarpSmem {
  float dt[C::STEPS][C::CH], du[C::STEPS][C::CH], y[C::STEPS][C::CH];
  float bc[2][C::STEPS][2 * C::N];
  float bias[C::CH], skip[C::CH];
};

struct ScanParams {
  gdn_ssm s;
  int32_t* status;
  int32_t per_group, blocks;  // channels of a group, and blocks of them
  uint32_t warps;             // tasks: (request, channel block)
};

template <class C>
__global__ void __launch_bounds__(kWarps * 32) gdn_ssm_scan_kernel(const ScanParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  constexpr bool BF16 = C::BF16;
  const gdn_ssm& s = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  WarpSmem<C>& sm = reinterpret_cast<WarpSmem<C>*>(smem_raw)[warp];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t task = blockIdx.x * kWarps + warp;
  if (task >= p.warps) return;
  const int all_blocks = p.blocks * s.num_groups;
  const int b = static_cast<int>(task / all_blocks), block = static_cast<int>(task - b * static_cast<uint32_t>(all_blocks));
  const int group = block / p.blocks, in_group = (block - group * p.blocks) * C::CH;
  const int c0 = group * p.per_group + in_group, count = min(C::CH, p.per_group - in_group);
  const int slot = s.slot[b];
  if (slot < 0) return;
  const int len = s.seq_lens != nullptr ? s.seq_lens[b] : s.num_tokens;
  const bool bad_slot = slot >= s.num_slots, bad_len = len < 0 || len > s.num_tokens;
  if (bad_slot || bad_len) {
    if (block == 0 && lane == 0) atomic_status(p.status, bad_slot ? GDN_STATUS_BAD_SLOT : GDN_STATUS_BAD_LEN);
    return;
  }
  if (len == 0) return;
  const int begin = 0, end = len;

  // ---- this thread's states -----------------------------------------------------------------
  const int set = lane / C::LANES, part = lane % C::LANES;
  float* const state = s.state + (static_cast<int64_t>(slot) * s.channels + c0 + set * 4) * C::N + part * 4;
  const float* const a_at = s.a + static_cast<int64_t>(c0 + set * 4) * C::N + part * 4;
  f32x2 h[2][4], a[2][4];
  auto load_states = [&](const float* from, f32x2 (&to)[2][4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (set * 4 < count) {
        x = *reinterpret_cast<const float4*>(from + (2 * i) * C::N);
        y = *reinterpret_cast<const float4*>(from + (2 * i + 1) * C::N);
      }
      to[i][0] = pack2(x.x, y.x);
      to[i][1] = pack2(x.y, y.y);
      to[i][2] = pack2(x.z, y.z);
      to[i][3] = pack2(x.w, y.w);
    }
  };
  load_states(state, h);
  load_states(a_at, a);
  const f32x2 log2e = pack2(kLog2e, kLog2e);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) a[i][j] = mul2(a[i][j], log2e);
  for (int c = lane; c < C::CH; c += 32) {
    sm.bias[c] = s.dt_bias != nullptr && c < count ? s.dt_bias[c0 + c] : 0.0f;
    sm.skip[c] = s.skip != nullptr && c < count ? s.skip[c0 + c] : 0.0f;
  }
  __syncwarp();

  // ---- rows of the inputs: item i of a tile is vector i % ROW of position i / ROW ------------------
  const int vec = lane % C::ROW * 8;
  const bool vec_live = vec < count;
  const int64_t u_at = b * s.u_strides[0] + c0 + vec, dt_at = b * s.dt_strides[0] + c0 + vec, z_at = b * s.z_strides[0] + c0 + vec;
  const int64_t b_at = b * s.b_strides[0] + group * s.b_strides[2], c_at = b * s.c_strides[0] + group * s.c_strides[2];
  const int64_t y_at = static_cast<int64_t>(b) * s.num_tokens * s.channels + c0 + vec;
  const bool softplus = (s.flags & GDN_DT_SOFTPLUS) != 0u;
  Raw8<BF16> next_u[C::U], next_dt[C::U], next_bc[C::V];
  auto item_t = [&](int k) { return (lane + 32 * k) / C::ROW; };
  auto item_live = [&](int k, int t0) {
    return vec_live && (C::ITEMS % 32 == 0 || lane + 32 * k < C::ITEMS) && t0 + item_t(k) < end;
  };
  auto fetch = [&](int t0) {
#pragma unroll
    for (int k = 0; k < C::U; ++k) {
      next_u[k] = next_dt[k] = zero8<BF16>();
      if (!item_live(k, t0)) continue;
      const int64_t t = t0 + item_t(k);
      next_u[k] = load8<BF16>(s.u, u_at + t * s.u_strides[1]);
      next_dt[k] = load8<BF16>(s.dt, dt_at + t * s.dt_strides[1]);
    }
#pragma unroll
    for (int k = 0; k < C::V; ++k) {
      next_bc[k] = zero8<BF16>();
      const int item = lane + 32 * k, which = item / (C::STEPS * C::NROW), in = item % (C::STEPS * C::NROW);
      const int64_t t = t0 + in / C::NROW;
      if (item >= C::NITEMS || t >= end) continue;
      next_bc[k] = which == 0 ? load8<BF16>(s.b, b_at + t * s.b_strides[1] + in % C::NROW * 8)
                              : load8<BF16>(s.c, c_at + t * s.c_strides[1] + in % C::NROW * 8);
    }
  };

  fetch(begin);
  for (int t0 = begin; t0 < end; t0 += C::STEPS) {
    // ---- steps, inputs, b and c of the tile into shared memory -----------------------------------
    Raw8<BF16> u[C::U], z[C::U];
#pragma unroll
    for (int k = 0; k < C::U; ++k) {
      u[k] = next_u[k];
      float x[8], dt[8];
      floats8<BF16>(next_u[k], x);
      floats8<BF16>(next_dt[k], dt);
      const bool live = item_live(k, t0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dt[e] += sm.bias[vec + e];
        if (softplus) dt[e] = softplus_series(dt[e]);
        if (!live) dt[e] = 0.0f;  // the state passes a position of no prompt unchanged
        x[e] *= dt[e];
      }
      if (C::ITEMS % 32 == 0 || lane + 32 * k < C::ITEMS) {
        store8<false>(&sm.dt[item_t(k)][vec], 0, raw8<false>(dt));
        store8<false>(&sm.du[item_t(k)][vec], 0, raw8<false>(x));
      }
    }
#pragma unroll
    for (int k = 0; k < C::V; ++k) {
      const int item = lane + 32 * k, which = item / (C::STEPS * C::NROW), in = item % (C::STEPS * C::NROW);
      if (C::NITEMS % 32 != 0 && item >= C::NITEMS) continue;
      float x[8];
      floats8<BF16>(next_bc[k], x);
      float4* const to = reinterpret_cast<float4*>(&sm.bc[which][in / C::NROW][in % C::NROW * 16]);
#pragma unroll
      for (int e = 0; e < 4; ++e) to[e] = make_float4(x[2 * e], x[2 * e], x[2 * e + 1], x[2 * e + 1]);
    }
    if (s.z != nullptr) {
#pragma unroll
      for (int k = 0; k < C::U; ++k)
        if (item_live(k, t0)) z[k] = load8<BF16>(s.z, z_at + (t0 + static_cast<int64_t>(item_t(k))) * s.z_strides[1]);
    }
    if (t0 + C::STEPS < end) fetch(t0 + C::STEPS);
    __syncwarp();

    // ---- the recurrence ----------------------------------------------------------------------------
    const int steps = min(C::STEPS, (end - t0 + 3) & ~3);
#pragma unroll 4
    for (int t = 0; t < steps; ++t) {
      const ulonglong2 dt = *reinterpret_cast<const ulonglong2*>(&sm.dt[t][set * 4]);
      const ulonglong2 du = *reinterpret_cast<const ulonglong2*>(&sm.du[t][set * 4]);
      const ulonglong2* const bt = reinterpret_cast<const ulonglong2*>(&sm.bc[0][t][part * 8]);
      const ulonglong2* const ct = reinterpret_cast<const ulonglong2*>(&sm.bc[1][t][part * 8]);
      const ulonglong2 b01 = bt[0], b23 = bt[1], c01 = ct[0], c23 = ct[1];
      const f32x2 bb[4] = {b01.x, b01.y, b23.x, b23.y}, cc[4] = {c01.x, c01.y, c23.x, c23.y};
      const f32x2 dts[2] = {dt.x, dt.y}, dus[2] = {du.x, du.y};
      f32x2 sum[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][j] = fma2(ex2_2(mul2(dts[i], a[i][j])), h[i][j], mul2(dus[i], bb[j]));
          sum[i] = j == 0 ? mul2(h[i][j], cc[j]) : fma2(h[i][j], cc[j], sum[i]);
        }
      }
      // Sums over the set's lanes: a lane keeps half of its channels and gives the other half away,
      // twice; further lanes add what is left.
      f32x2 keep = sum[0];
      {
        const bool upper = (part & (C::LANES / 2)) != 0;
        const f32x2 give = upper ? sum[0] : sum[1];
        keep = upper ? sum[1] : sum[0];
        keep = add2(keep, __shfl_xor_sync(0xffffffffu, give, C::LANES / 2));
      }
      const float2 two = unpack2(keep);
      if constexpr (C::LANES == 2) {
        *reinterpret_cast<float2*>(&sm.y[t][set * 4 + part * 2]) = two;
      } else {
        const bool upper = (part & (C::LANES / 4)) != 0;
        float one = upper ? two.y : two.x;
        one += __shfl_xor_sync(0xffffffffu, upper ? two.x : two.y, C::LANES / 4);
#pragma unroll
        for (int off = C::LANES / 8; off > 0; off >>= 1) one += __shfl_xor_sync(0xffffffffu, one, off);
        if (part % (C::LANES / 4) == 0) sm.y[t][set * 4 + part / (C::LANES / 4)] = one;
      }
    }
    __syncwarp();

    // ---- readout ----------------------------------------------------------------------------------
#pragma unroll
    for (int k = 0; k < C::U; ++k) {
      if (!item_live(k, t0)) continue;
      float x[8], y[8], g[8];
      floats8<BF16>(u[k], x);
      floats8<false>(load8<false>(&sm.y[item_t(k)][vec], 0), y);
      if (s.z != nullptr) floats8<BF16>(z[k], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = fmaf(sm.skip[vec + e], x[e], y[e]);
        if (s.z != nullptr) y[e] *= silu_fast(g[e]);
      }
      store8<BF16>(s.y, y_at + (t0 + static_cast<int64_t>(item_t(k))) * s.channels, raw8<BF16>(y));
    }
  }

  if (set * 4 < count) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = unpack2(h[i][j]);
      *reinterpret_cast<float4*>(state + (2 * i) * C::N) = make_float4(x[0].x, x[1].x, x[2].x, x[3].x);
      *reinterpret_cast<float4*>(state + (2 * i + 1) * C::N) = make_float4(x[0].y, x[1].y, x[2].y, x[3].y);
    }
  }
}

template <class C>
cudaError_t launch_scan(const SsmParams& given, cudaStream_t stream) {
  ScanParams p{given.s, given.status, given.s.channels / given.s.num_groups, 0, 0};
  p.blocks = (p.per_group + C::CH - 1) / C::CH;
  const int64_t warps = static_cast<int64_t>(p.blocks) * p.s.num_groups * p.s.batch;
  if (warps > 0x7fffffff) return cudaErrorInvalidConfiguration;
  p.warps = static_cast<uint32_t>(warps);
  constexpr int kBytes = kWarps * static_cast<int>(sizeof(WarpSmem<C>));
  static std::atomic<bool> allowed[kDevices];
  const cudaError_t err = allow_shared(reinterpret_cast<const void*>(gdn_ssm_scan_kernel<C>), kBytes, allowed);
  if (err != cudaSuccess) return err;
  return launch_overlapped(gdn_ssm_scan_kernel<C>, p, dim3((p.warps + kWarps - 1) / kWarps), kWarps * 32, kBytes, 1u, stream);
}

template <bool BF16>
cudaError_t launch_type(const SsmParams& p, cudaStream_t stream) {
  switch (p.s.state_size) {
    case 8: return launch_scan<Cfg<8, BF16>>(p, stream);
    case 16: return launch_scan<Cfg<16, BF16>>(p, stream);
    case 32: return launch_scan<Cfg<32, BF16>>(p, stream);
    default: return launch_scan<Cfg<64, BF16>>(p, stream);
  }
}

}  // namespace

size_t ssm_workspace_bytes(int32_t, int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_ssm_scan(const SsmParams& p, void*, cudaStream_t stream) {
  return (p.s.flags & GDN_QKV_BF16) != 0u ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

}  // namespace gdn
