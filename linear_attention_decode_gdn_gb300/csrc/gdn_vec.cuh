// gdn_vec.cuh -- vectors of eight elements, in fp32 registers: what the kernels of the selective
// state space layers share. A vector of bf16 is one 16-byte access, one of fp32 two.
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
__device__ __forceinline__ Raw8<BF16> zero8() {
  Raw8<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = make_uint4(0u, 0u, 0u, 0u);
  return r;
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

}  // namespace gdn
