// gdn_vec.cuh -- what the kernels of the selective state space layers share: vectors of eight elements
// (one 16-byte access of bf16, two of fp32), pairs of fp32 and the functions of them.
#pragma once

#include "gdn_device.cuh"

namespace gdn {

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight elements as they lie in memory.
template <bool BF16>
struct Raw8 {
  uint4 v[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8(const void* base, int64_t at) {
  const uint4* from = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + at * (BF16 ? 2 : 4));
  Raw8<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = from[i];
  return r;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, const Raw8<BF16>& r) {
  uint4* to = reinterpret_cast<uint4*>(static_cast<unsigned char*>(base) + at * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) to[i] = r.v[i];
}

template <bool BF16>
__device__ __forceinline__ void floats8(const Raw8<BF16>& r, float (&x)[8]) {
  if constexpr (BF16) {
    unpack8(r.v[0], x);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.v[i].x);
      x[4 * i + 1] = __uint_as_float(r.v[i].y);
      x[4 * i + 2] = __uint_as_float(r.v[i].z);
      x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  }
}

// bf16: rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> raw8(const float (&x)[8]) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.v[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                          __float_as_uint(x[4 * i + 3]));
  }
  return r;
}

// Element i as float.
template <bool BF16>
__device__ __forceinline__ float elem(const void* base, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_float(static_cast<const uint16_t*>(base)[i]);
  return static_cast<const float*>(base)[i];
}

template <bool BF16>
__device__ __forceinline__ void set_elem(void* base, int64_t i, float x) {
  if constexpr (BF16)
    static_cast<uint16_t*>(base)[i] = static_cast<uint16_t>(pack_bf16(x, 0.0f));
  else
    static_cast<float*>(base)[i] = x;
}

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

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

__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f32x2 rcp_2(f32x2 x) {
  const float2 v = unpack2(x);
  return pack2(rcp(v.x), rcp(v.y));
}
// log(1 + 2^x2) for x2 = x log2(e), which is log(1 + e^x) = max(x, 0) + log(1 + e) with e = e^-|x| in
// (0, 1]. log(1 + e) = e p(e), p a minimax polynomial of degree 8 on [0, 1] (a Remez fit, 2^-23 off
// with its coefficients rounded): without cancellation however small e is.
__device__ __forceinline__ f32x2 softplus_2(f32x2 x2) {
  const float2 v = unpack2(x2);
  const f32x2 e = pack2(ex2(-fabsf(v.x)), ex2(-fabsf(v.y)));
  f32x2 p = fma2(e, both(0.0052326931f), both(-0.0295052398f));
  p = fma2(p, e, both(0.0782259554f));
  p = fma2(p, e, both(-0.1366324574f));
  p = fma2(p, e, both(0.1910600662f));
  p = fma2(p, e, both(-0.2484298199f));
  p = fma2(p, e, both(0.3331909776f));
  p = fma2(p, e, both(-0.4999949336f));
  p = fma2(p, e, both(0.9999999404f));
  return fma2(pack2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)), both(kLn2), mul2(p, e));
}

// z / (1 + e^-z). 2^-t, t = z log2(e), is off by |z| roundings, which EXACT takes out again (the
// factor 1 + r ln 2, r what the rounding of t lost): without it the result is off by |z| 2^-24 beside
// its own 2^-22 (2^-18 at |z| = 64), where bf16 keeps 2^-8.
template <bool EXACT>
__device__ __forceinline__ f32x2 silu_2(f32x2 z) {
  f32x2 e = ex2_2(mul2(z, both(-kLog2e)));
  if (EXACT) {
    const float2 v = unpack2(z), big = unpack2(e);
    // past 80 either way e is next to 0 or so large that r does not count; finite, as r may be 0
    const f32x2 near = pack2(fminf(fmaxf(v.x, -80.0f), 80.0f), fminf(fmaxf(v.y, -80.0f), 80.0f));
    const f32x2 r = fma2(near, both(-kLog2e), mul2(near, both(kLog2e)));
    e = pack2(fminf(big.x, 3e38f), fminf(big.y, 3e38f));
    e = fma2(e, mul2(r, both(kLn2)), e);
  }
  return mul2(z, rcp_2(add2(e, both(1.0f))));
}

}  // namespace gdn
