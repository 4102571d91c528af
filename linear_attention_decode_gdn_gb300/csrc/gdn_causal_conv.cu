// gdn_causal_conv.cu -- the causal convolution of width 4 with SiLU, for prompts and single tokens,
// on its own (gdn_causal_conv).
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kConvThreads = 128;
constexpr int kSteps = 32;  // positions a thread takes
constexpr int kAhead = 4;   // of them in flight

// The three inputs before position `at` (oldest first) of eight channels: of the prompt, or of the
// slot's row where they lie before it.
template <bool BF16>
__device__ __forceinline__ void inputs_before(const gdn_conv& c, const void* row, int64_t x, int at, int d, Raw8<BF16> (&w)[3]) {
  // [8 channels][3]: 24 elements that start on a 16-byte boundary
  uint4 old[BF16 ? 3 : 6];
  if (at < 3) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 3 : 6); ++i)
      old[i] = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(row) + d * 3 * (BF16 ? 2 : 4))[i];
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int from = at - 3 + j;  // position of the input; -3..-1: the row's columns 0..2
    if (from >= 0) {
      w[j] = load8<BF16>(c.x, x + from * c.x_strides[1]);
      continue;
    }
#pragma unroll
    for (int col = 0; col < 3; ++col) {
      if (from + 3 != col) continue;
      if constexpr (BF16) {
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = (reinterpret_cast<const uint32_t*>(old)[(k * 3 + col) / 2] >> (16 * ((k * 3 + col) & 1))) & 0xffffu;
        w[j].v[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      } else {
        const uint32_t* o = reinterpret_cast<const uint32_t*>(old);
        w[j].v[0] = make_uint4(o[col], o[3 + col], o[6 + col], o[9 + col]);
        w[j].v[1] = make_uint4(o[12 + col], o[15 + col], o[18 + col], o[21 + col]);
      }
    }
  }
}

// The slot's row of eight channels.
template <bool BF16>
__device__ __forceinline__ void write_row(void* row, int d, const Raw8<BF16> (&w)[3]) {
  uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(row) + d * 3 * (BF16 ? 2 : 4));
  uint32_t out[BF16 ? 12 : 24];
  if constexpr (BF16) {
    auto e = [&](int i) {  // element i of [8][3]
      const uint4& v = w[i % 3].v[0];
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
      return (words[i / 3 / 2] >> (16 * (i / 3 & 1))) & 0xffffu;
    };
#pragma unroll
    for (int i = 0; i < 12; ++i) out[i] = e(2 * i) | e(2 * i + 1) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 24; ++i) {
      const uint4& v = w[i % 3].v[i / 3 / 4];
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
      out[i] = words[i / 3 % 4];
    }
  }
#pragma unroll
  for (int i = 0; i < (BF16 ? 3 : 6); ++i)
    reinterpret_cast<uint4*>(to)[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
}

// A thread runs over kSteps positions of eight channels with the last three inputs in registers. The
// thread of a request's first positions is the only one that reads the slot's row, so it also
// writes it, from the prompt's end.
template <bool BF16>
__global__ void __launch_bounds__(kConvThreads) gdn_causal_conv_kernel(const ConvParams p) {
  const gdn_conv& c = p.c;
  griddep_launch_dependents();
  griddep_wait();
  const int vecs = c.channels / 8, chunks = (c.num_tokens + kSteps - 1) / kSteps;
  const int64_t per = static_cast<int64_t>(vecs) * chunks, item = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  if (item >= per * c.batch) return;
  const int b = static_cast<int>(item / per), in = static_cast<int>(item - b * per);
  const int chunk = in / vecs, vec = in - chunk * vecs, d = vec * 8;
  const int slot = c.slot[b];
  if (slot < 0) return;
  const int len = c.seq_lens != nullptr ? c.seq_lens[b] : c.num_tokens;
  const bool bad_slot = slot >= c.num_slots, bad_len = len < 0 || len > c.num_tokens;
  if (bad_slot || bad_len) {
    if (in == 0) atomic_status(p.status, bad_slot ? GDN_STATUS_BAD_SLOT : GDN_STATUS_BAD_LEN);
    return;
  }
  const int begin = chunk * kSteps, end = min(begin + kSteps, len);
  if (begin >= end) return;
  const int64_t x = b * c.x_strides[0] + d;
  void* const row = static_cast<unsigned char*>(c.pool) + static_cast<int64_t>(slot) * c.channels * (3 * (BF16 ? 2 : 4));
  Raw8<BF16> before[3];
  inputs_before<BF16>(c, row, x, begin, d, before);
  if (chunk == 0) {
    Raw8<BF16> last[3];
    inputs_before<BF16>(c, row, x, len, d, last);
    write_row<BF16>(row, d, last);
  }
  // pairs of channels from here on
  f32x2 w[4][4], bias[4], past[3][4];  // [tap][pair]
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 lo = reinterpret_cast<const float4*>(c.w)[d + 2 * k], hi = reinterpret_cast<const float4*>(c.w)[d + 2 * k + 1];
    w[0][k] = pack2(lo.x, hi.x), w[1][k] = pack2(lo.y, hi.y), w[2][k] = pack2(lo.z, hi.z), w[3][k] = pack2(lo.w, hi.w);
    bias[k] = c.bias != nullptr ? *reinterpret_cast<const f32x2*>(c.bias + d + 2 * k) : 0;
  }
  auto pairs = [](const Raw8<BF16>& r, f32x2 (&x)[4]) {
    float f[8];
    floats8<BF16>(r, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = pack2(f[2 * k], f[2 * k + 1]);
  };
#pragma unroll
  for (int j = 0; j < 3; ++j) pairs(before[j], past[j]);
  const bool silu = (c.flags & GDN_CONV_SILU) != 0u;
  Raw8<BF16> next[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (begin + j < end) next[j] = load8<BF16>(c.x, x + (begin + j) * c.x_strides[1]);
  int64_t to = (static_cast<int64_t>(b) * c.num_tokens + begin) * c.channels + d;
  for (int t0 = begin; t0 < end; t0 += kAhead) {
    Raw8<BF16> now[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      now[j] = next[j];
      if (t0 + kAhead + j < end) next[j] = load8<BF16>(c.x, x + (t0 + kAhead + j) * c.x_strides[1]);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (t0 + j >= end) break;
      f32x2 in[4];
      float o[8];
      pairs(now[j], in);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f32x2 sum = fma2(in[k], w[3][k], fma2(past[2][k], w[2][k], fma2(past[1][k], w[1][k], fma2(past[0][k], w[0][k], bias[k]))));
        if (silu) sum = silu_2<!BF16>(sum);
        const float2 v = unpack2(sum);
        o[2 * k] = v.x, o[2 * k + 1] = v.y;
        past[0][k] = past[1][k], past[1][k] = past[2][k], past[2][k] = in[k];
      }
      store8<BF16>(c.o, to, raw8<BF16>(o));
      to += c.channels;
    }
  }
}

}  // namespace

cudaError_t launch_causal_conv(const ConvParams& p, cudaStream_t stream) {
  const int64_t chunks = (p.c.num_tokens + kSteps - 1) / kSteps, items = chunks * p.c.batch * (p.c.channels / 8);
  const unsigned grid = static_cast<unsigned>((items + kConvThreads - 1) / kConvThreads);
  return launch_overlapped((p.c.flags & GDN_QKV_BF16) != 0u ? gdn_causal_conv_kernel<true> : gdn_causal_conv_kernel<false>, p,
                           dim3(grid), kConvThreads, 0, 1u, stream);
}

}  // namespace gdn
