// gdn_causal_conv.cu -- the causal convolution of width 4 with SiLU, for prompts and single tokens,
// on its own (gdn_causal_conv):
//
//   o_t = silu(bias + w_0 x_{t-3} + w_1 x_{t-2} + w_2 x_{t-1} + w_3 x_t)
//
// Two bytes in and two out an element, eight products and sums and a SiLU: bound by HBM, if enough
// loads are in flight. A thread runs along the positions of eight channels, so that an input is read
// once (but for three at the start of each thread's run).
//   2 x 16384 positions of 4096 channels (bf16): 89 us, 6.0 TB/s (0.89 of the measured copy bandwidth);
//     120 us with four positions in registers instead of sixteen in shared memory.
//   8 ragged prompts of up to 4093 positions, 4096 channels: 57 us, 5.3 TB/s; issue slots 59% busy.
//   one token of 64 requests x 6144 channels: 4.3 us, latency (5.6 with each thread loading its own
//     taps); of 512 x 4096: 7.5 us, 4.5 TB/s (9.0 with one request's row on its way at a time).
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kConvThreads = 128;
constexpr int kGroup = 4, kGroups = 4;  // positions that are loaded together, and groups of them that a thread has room for
// Positions a thread takes: as many as leave kEnough threads. Every thread begins with its taps, so
// fewer and longer runs win (one prompt of 4096 positions: 18.6 us at 40000 threads, 26 at 155000),
// until the GPU is half empty.
constexpr int kMinSteps = 8, kMaxSteps = 128;
constexpr int64_t kEnough = 40000;
// Requests that a thread takes one token of, from so many vectors in the batch on: of 512 x 4096 channels
// 7.5 us at 4, 8.5 at 2, 9.3 at 8, 11.9 at 1; of 256 x 4096 6.2 at 4, 7.5 at 1; but of 64 x 6144 (49152
// vectors) 4.3 at 1, 5.0 at 4.
constexpr int64_t kManyItems = 100000;
constexpr int kTokenRows = 4;

struct ConvTask {
  ConvParams p;
  int32_t steps;
};

// Eight channels of a slot's row: [8][3] elements, which start on a 16-byte boundary.
template <bool BF16>
struct Row {
  uint32_t w[BF16 ? 12 : 24];
};
template <bool BF16>
__device__ __forceinline__ void* row_at(const gdn_conv& c, int slot, int d) {
  return static_cast<unsigned char*>(c.pool) + (static_cast<int64_t>(slot) * c.channels + d) * (3 * (BF16 ? 2 : 4));
}
template <bool BF16>
__device__ __forceinline__ Row<BF16> load_row(const void* at) {
  Row<BF16> r;
#pragma unroll
  for (int i = 0; i < (BF16 ? 3 : 6); ++i) {
    const uint4 v = static_cast<const uint4*>(at)[i];
    r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
  }
  return r;
}
// Column `col` as a vector of the eight channels.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> column(const Row<BF16>& r, int col) {
  Raw8<BF16> x;
  uint32_t out[BF16 ? 4 : 8];
  if constexpr (BF16) {
    auto e = [&](int i) { return (r.w[i / 2] >> (16 * (i & 1))) & 0xffffu; };
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = e(6 * k + col) | e(6 * k + 3 + col) << 16;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = r.w[3 * k + col];
  }
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) x.v[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
  return x;
}
// The row of three columns.
template <bool BF16>
__device__ __forceinline__ void store_row(void* at, const Raw8<BF16> (&col)[3]) {
  uint32_t words[3][BF16 ? 4 : 8], out[BF16 ? 12 : 24];
#pragma unroll
  for (int j = 0; j < 3; ++j)
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i)
      words[j][4 * i] = col[j].v[i].x, words[j][4 * i + 1] = col[j].v[i].y, words[j][4 * i + 2] = col[j].v[i].z, words[j][4 * i + 3] = col[j].v[i].w;
#pragma unroll
  for (int i = 0; i < (BF16 ? 12 : 24); ++i) {
    if constexpr (BF16) {
      auto e = [&](int j) { return (words[j % 3][j / 6] >> (16 * (j / 3 & 1))) & 0xffffu; };
      out[i] = e(2 * i) | e(2 * i + 1) << 16;
    } else {
      out[i] = words[i % 3][i / 3];
    }
  }
#pragma unroll
  for (int i = 0; i < (BF16 ? 3 : 6); ++i) static_cast<uint4*>(at)[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
}

// a / b of what is not negative; most fit 32 bits, whose division is several times shorter.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Taps and bias of eight channels, as pairs of channels.
struct Weights {
  f32x2 w[4][4], bias[4];  // [tap][pair]
};
// Called by a whole warp, whose lanes hold consecutive vectors (those of lane 0's row and, past its
// last, again from the first on). A lane's taps are 128 bytes in a row, so that loads of its own
// would touch 32 lines each; the warp loads the 4 KB in order and hands them over in shared memory,
// with places exchanged so that eight lanes meet all banks both ways.
constexpr int kTapVecs = 256;
__device__ __forceinline__ void fetch_weights(const gdn_conv& c, int d, float4* taps) {
  const int lane = threadIdx.x & 31, first = __shfl_sync(0xffffffffu, d, 0);
#pragma unroll
  for (int j = 0; j < kTapVecs / 32; ++j) {
    const int i = 32 * j + lane;
    cp_async16(&taps[i ^ (i >> 3 & 7)], c.w + static_cast<int64_t>((first + i) % c.channels) * 4);
  }
}
// After what fetch_weights() asked for is there, for all lanes.
__device__ __forceinline__ Weights take_weights(const gdn_conv& c, int d, const float4* taps) {
  const int lane = threadIdx.x & 31;
  Weights r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 lo = taps[8 * lane + ((2 * k) ^ (lane & 7))], hi = taps[8 * lane + ((2 * k + 1) ^ (lane & 7))];
    r.w[0][k] = pack2(lo.x, hi.x), r.w[1][k] = pack2(lo.y, hi.y), r.w[2][k] = pack2(lo.z, hi.z), r.w[3][k] = pack2(lo.w, hi.w);
    r.bias[k] = c.bias != nullptr ? *reinterpret_cast<const f32x2*>(c.bias + d + 2 * k) : 0;
  }
  return r;
}
__device__ __forceinline__ void copies_arrived() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}
template <bool BF16>
__device__ __forceinline__ void pairs8(const Raw8<BF16>& r, f32x2 (&x)[4]) {
  float f[8];
  floats8<BF16>(r, f);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = pack2(f[2 * k], f[2 * k + 1]);
}
// The output of eight channels at a position, of the inputs there and at the three before.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> output(const Weights& s, const f32x2 (&past)[3][4], const f32x2 (&in)[4], bool silu) {
  float o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f32x2 sum = fma2(in[k], s.w[3][k], fma2(past[2][k], s.w[2][k], fma2(past[1][k], s.w[1][k], fma2(past[0][k], s.w[0][k], s.bias[k]))));
    if (silu) sum = silu_2<!BF16>(sum);
    const float2 v = unpack2(sum);
    o[2 * k] = v.x, o[2 * k + 1] = v.y;
  }
  return raw8<BF16>(o);
}

// The three inputs before position `at` (oldest first) of eight channels: of the prompt, or of the
// slot's row where they lie before it.
template <bool BF16>
__device__ __forceinline__ void inputs_before(const gdn_conv& c, const void* row, int64_t x, int at, Raw8<BF16> (&to)[3]) {
  if (at < 3) {
    const Row<BF16> old = load_row<BF16>(row);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      if (at + j < 3)
        to[j] = at == 0 ? column<BF16>(old, j) : at == 1 ? column<BF16>(old, j < 2 ? j + 1 : 2) : column<BF16>(old, 2);
      else
        to[j] = load8<BF16>(c.x, x + (at - 3 + j) * c.x_strides[1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j) to[j] = load8<BF16>(c.x, x + (at - 3 + j) * c.x_strides[1]);
  }
}

// One token of every request. A thread takes eight channels of `rows` requests, for which it loads the
// taps once.
struct TokenTask {
  ConvParams p;
  int32_t rows;
};
template <bool BF16>
__global__ void __launch_bounds__(kConvThreads) gdn_causal_conv_token_kernel(const TokenTask task) {
  // A lane's part of a slot's row is 48 (96) bytes, of which its own accesses would take 16 at a time, 48
  // apart. Where a warp's lanes are all of one row (WHOLE) they take it in order, through shared
  // memory, and kFlight requests' rows are on their way together.
  constexpr int kFlight = BF16 ? 4 : 2, kPart = sizeof(Row<BF16>), kPartVecs = kPart / 16;
  __shared__ float4 taps[kConvThreads / 32][kTapVecs];
  __shared__ uint4 parts[kConvThreads / 32][kFlight][32 * kPartVecs];
  const gdn_conv& c = task.p.c;
  griddep_launch_dependents();
  griddep_wait();
  const int vecs = c.channels / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const int first = static_cast<int>(quotient(item, vecs)), d = static_cast<int>(item - static_cast<int64_t>(first) * vecs) * 8;
  fetch_weights(c, d, taps[warp]);
  Weights weights;
  const bool silu = (c.flags & GDN_CONV_SILU) != 0u, whole = vecs % 32 == 0;
  for (int r0 = 0; r0 < task.rows; r0 += kFlight) {
    const int b0 = first * task.rows + r0;
    int slot[kFlight];
    Raw8<BF16> now[kFlight];
#pragma unroll
    for (int r = 0; r < kFlight; ++r) {
      slot[r] = -1;
      if (r0 + r >= task.rows || b0 + r >= c.batch) continue;
      slot[r] = c.slot[b0 + r];
      now[r] = load8<BF16>(c.x, (b0 + r) * c.x_strides[0] + d);
      const int len = c.seq_lens != nullptr ? c.seq_lens[b0 + r] : 1;
      if (slot[r] < 0 || (len == 1 && slot[r] < c.num_slots)) continue;
      const bool bad_slot = slot[r] >= c.num_slots;
      if (d == 0 && (bad_slot || len != 0)) atomic_status(task.p.status, bad_slot ? GDN_STATUS_BAD_SLOT : GDN_STATUS_BAD_LEN);
      slot[r] = -1;
    }
    if (whole) {
#pragma unroll
      for (int r = 0; r < kFlight; ++r) {
        if (slot[r] < 0) continue;
        const uint4* const from = static_cast<const uint4*>(row_at<BF16>(c, slot[r], d - 8 * lane));
#pragma unroll
        for (int i = 0; i < kPartVecs; ++i) cp_async16(&parts[warp][r][32 * i + lane], from + 32 * i + lane);
      }
    }
    copies_arrived();
    if (r0 == 0) weights = take_weights(c, d, taps[warp]);
#pragma unroll
    for (int r = 0; r < kFlight; ++r) {
      if (slot[r] < 0) continue;
      void* const row = row_at<BF16>(c, slot[r], d);
      void* const at = whole ? static_cast<void*>(&parts[warp][r][lane * kPartVecs]) : row;
      const Row<BF16> old = load_row<BF16>(at);
      const Raw8<BF16> cols[3] = {column<BF16>(old, 1), column<BF16>(old, 2), now[r]};
      store_row<BF16>(at, cols);
      f32x2 past[3][4], in[4];
      pairs8<BF16>(column<BF16>(old, 0), past[0]);
      pairs8<BF16>(cols[0], past[1]);
      pairs8<BF16>(cols[1], past[2]);
      pairs8<BF16>(now[r], in);
      store8<BF16>(c.o, static_cast<int64_t>(b0 + r) * c.channels + d, output<BF16>(weights, past, in, silu));
    }
    if (whole) {
      __syncwarp();
#pragma unroll
      for (int r = 0; r < kFlight; ++r) {
        if (slot[r] < 0) continue;
        uint4* const to = static_cast<uint4*>(row_at<BF16>(c, slot[r], d - 8 * lane));
#pragma unroll
        for (int i = 0; i < kPartVecs; ++i) to[32 * i + lane] = parts[warp][r][32 * i + lane];
      }
      __syncwarp();
    }
  }
}

// A thread runs over `steps` positions of eight channels with the last three inputs in registers. The
// thread of a request's first positions is the only one that reads the slot's row, so it also
// writes it, from the prompt's end.
template <bool BF16>
__global__ void __launch_bounds__(kConvThreads, 4) gdn_causal_conv_kernel(const ConvTask task) {
  const ConvParams& p = task.p;
  const gdn_conv& c = p.c;
  __shared__ float4 taps[kConvThreads / 32][kTapVecs];
  griddep_launch_dependents();
  griddep_wait();
  const int vecs = c.channels / 8, chunks = (c.num_tokens + task.steps - 1) / task.steps;
  const int64_t per = static_cast<int64_t>(vecs) * chunks, item = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const int b = static_cast<int>(quotient(item, per)), in = static_cast<int>(item - b * per);
  const int chunk = in / vecs, vec = in - chunk * vecs, d = vec * 8;
  const int slot = b < c.batch ? c.slot[b] : -1;
  fetch_weights(c, d, taps[threadIdx.x >> 5]);  // while the slot is looked up
  copies_arrived();
  const Weights weights = take_weights(c, d, taps[threadIdx.x >> 5]);
  if (slot < 0) return;
  const int len = c.seq_lens != nullptr ? c.seq_lens[b] : c.num_tokens;
  const bool bad_slot = slot >= c.num_slots, bad_len = len < 0 || len > c.num_tokens;
  if (bad_slot || bad_len) {
    if (in == 0) atomic_status(p.status, bad_slot ? GDN_STATUS_BAD_SLOT : GDN_STATUS_BAD_LEN);
    return;
  }
  const int begin = chunk * task.steps, end = min(begin + task.steps, len);
  if (begin >= end) return;
  const int64_t x = b * c.x_strides[0] + d;
  void* const row = row_at<BF16>(c, slot, d);
  Raw8<BF16> before[3];
  inputs_before<BF16>(c, row, x, begin, before);
  if (chunk == 0) {
    Raw8<BF16> last[3];
    inputs_before<BF16>(c, row, x, len, last);
    store_row<BF16>(row, last);
  }
  f32x2 past[3][4];
#pragma unroll
  for (int j = 0; j < 3; ++j) pairs8<BF16>(before[j], past[j]);
  const bool silu = (c.flags & GDN_CONV_SILU) != 0u;
  // Loads go through shared memory, where a thread reads what it has asked for itself: more of them
  // are in flight than registers would hold.
  extern __shared__ __align__(16) unsigned char ring[];
  constexpr int kVec = BF16 ? 16 : 32;
  unsigned char* const mine = ring + threadIdx.x * 16;
  auto place = [&](int t, int half) { return mine + ((t & (kGroup * kGroups - 1)) * (kVec / 16) + half) * (kConvThreads * 16); };
  const unsigned char* const from = static_cast<const unsigned char*>(c.x) + x * (kVec / 8);
  const int64_t stride = c.x_strides[1] * (kVec / 8);
  auto fetch = [&](int t0) {
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (t0 + j < end)
#pragma unroll
        for (int half = 0; half < kVec / 16; ++half) cp_async16(place(t0 + j - begin, half), from + (t0 + j) * stride + half * 16);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kGroups - 1; ++i) fetch(begin + i * kGroup);
  int64_t to = (static_cast<int64_t>(b) * c.num_tokens + begin) * c.channels + d;
  for (int t0 = begin; t0 < end; t0 += kGroup) {
    fetch(t0 + (kGroups - 1) * kGroup);
    asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory");
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      if (t0 + j >= end) break;
      Raw8<BF16> now;
#pragma unroll
      for (int half = 0; half < kVec / 16; ++half) now.v[half] = *reinterpret_cast<const uint4*>(place(t0 + j - begin, half));
      f32x2 in[4];
      pairs8<BF16>(now, in);
      store8<BF16>(c.o, to, output<BF16>(weights, past, in, silu));
#pragma unroll
      for (int k = 0; k < 4; ++k) past[0][k] = past[1][k], past[1][k] = past[2][k], past[2][k] = in[k];
      to += c.channels;
    }
  }
}

template <bool BF16>
cudaError_t launch_conv(const ConvTask& task, int64_t items, cudaStream_t stream) {
  constexpr int kBytes = kGroup * kGroups * (BF16 ? 16 : 32) * kConvThreads;
  static std::atomic<bool> allowed[kDevices];
  const cudaError_t err = allow_shared(reinterpret_cast<const void*>(gdn_causal_conv_kernel<BF16>), kBytes, allowed);
  if (err != cudaSuccess) return err;
  const unsigned grid = static_cast<unsigned>((items + kConvThreads - 1) / kConvThreads);
  return launch_overlapped(gdn_causal_conv_kernel<BF16>, task, dim3(grid), kConvThreads, kBytes, 1u, stream);
}

template <bool BF16>
cudaError_t launch_token(const ConvParams& p, cudaStream_t stream) {
  const int64_t vecs = p.c.channels / 8;
  TokenTask task{p, vecs * p.c.batch >= kManyItems ? kTokenRows : 1};
  const int64_t items = vecs * ((p.c.batch + task.rows - 1) / task.rows);
  const unsigned grid = static_cast<unsigned>((items + kConvThreads - 1) / kConvThreads);
  return launch_overlapped(gdn_causal_conv_token_kernel<BF16>, task, dim3(grid), kConvThreads, 0, 1u, stream);
}

}  // namespace

cudaError_t launch_causal_conv(const ConvParams& p, cudaStream_t stream) {
  if (p.c.num_tokens == 1) return (p.c.flags & GDN_QKV_BF16) != 0u ? launch_token<true>(p, stream) : launch_token<false>(p, stream);
  ConvTask task{p, kMaxSteps};
  const int64_t vecs = static_cast<int64_t>(p.c.batch) * (p.c.channels / 8);
  auto items = [&] { return (p.c.num_tokens + task.steps - 1) / task.steps * vecs; };
  while (task.steps > kMinSteps && items() < kEnough) task.steps /= 2;
  return (p.c.flags & GDN_QKV_BF16) != 0u ? launch_conv<true>(task, items(), stream) : launch_conv<false>(task, items(), stream);
}

}  // namespace gdn
