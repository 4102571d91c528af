// gdn_ssm_scan.cu -- the selective state space recurrence over prompts (gdn_ssm_scan):
//
//   s = softplus(dt + dt_bias),  h <- exp(s a) h + s u b,  y = (c . h + skip u) silu(z)
//
// for every channel, with a state of N values.
//
// The decays differ by channel, state and position, so there is no matrix product in it: an
// exponential, two products and two sums for each of positions x channels x states. Channels and
// states are laid over the threads, positions run in order. A warp works for itself: it copies tiles
// of eight positions into shared memory (asynchronously, one ahead), makes steps and steps times
// inputs of them once a channel, runs the recurrence, and reads out.
//
// What bounds it is neither HBM (16384 positions of 8192 channels are 1.08 GB, 158 us) nor the
// exponentials (32 a cycle and SM: 260 us) but operands: the packed fp32 instructions read up to six
// registers, of which the SM's quarter supplies two a cycle (measured: a packed multiply-add of three
// different operands takes 3 cycles, a product 2). A position of 16 states and 32 channels is 102
// instructions with, by count, some 290 operands, and takes 171 cycles of a quarter; issue slots are
// 60% busy, the exponentials' unit 46%, shared memory 50%. At 32 x 512 positions of 8192 channels:
//   two channels x eight states a thread 582 us; four x eight 710 (registers leave 12 warps an SM);
//   steps held twice each, as pairs, instead of splat in registers 626; products in single
//   instructions instead of pairs 598 to 650; three CTAs an SM instead of four 740 (695 with four then).
// Whole calls: 16384 x 8192 channels 943 us (582 of it the scan, the rest the parts' ends, below);
// 8 ragged prompts of up to 2045 positions x 4096 channels 291 us; one of 1021 x 2048 channels 35 us;
// 3 x 509 of 64 states in fp32 103 us.
#include "gdn_ssm.h"
#include "gdn_vec.cuh"

#include <cmath>
#include <type_traits>

namespace gdn {

namespace {

constexpr int kWarps = 4;  // of a CTA; they have nothing in common
constexpr int kCtas = 4;   // of an SM (two of fp32 with 8 states and two channels a thread, whose shared memory is 81 KB)

// Two elements as they lie in memory.
template <bool BF16>
using Raw2 = typename std::conditional<BF16, uint32_t, float2>::type;
template <bool BF16>
__device__ __forceinline__ f32x2 pair_of(const Raw2<BF16>& r) {
  if constexpr (BF16) return pack2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  else return pack2(r.x, r.y);
}
template <bool BF16>
__device__ __forceinline__ Raw2<BF16> raw_of(f32x2 x) {
  const float2 v = unpack2(x);
  if constexpr (BF16) return pack_bf16(v.x, v.y);
  else return v;
}

// Eight elements of shared memory as pairs.
template <bool BF16>
__device__ __forceinline__ void pairs8(const unsigned char* from, f32x2 (&x)[4]) {
  if constexpr (BF16) {
    const uint4 v = *reinterpret_cast<const uint4*>(from);
    x[0] = pair_of<true>(v.x), x[1] = pair_of<true>(v.y), x[2] = pair_of<true>(v.z), x[3] = pair_of<true>(v.w);
  } else {
    const ulonglong2 lo = reinterpret_cast<const ulonglong2*>(from)[0], hi = reinterpret_cast<const ulonglong2*>(from)[1];
    x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
  }
}

// 16 bytes to shared memory, zeros where `there` is false (then nothing is read)
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// A thread owns eight states of OWN channels (two, or one where prompts are few and short), the states
// in pairs: LANES neighbouring lanes hold the same channels, a warp CH, STEPS positions at a time in
// shared memory. Item i of a tile is the pair of channels i % ROW of position i / ROW.
template <int N_, bool BF16_, int OWN_>
struct Cfg {
  static constexpr int OWN = OWN_;
  static constexpr int N = N_;
  static constexpr bool BF16 = BF16_;
  static constexpr int LANES = N / 8, CH = OWN * (32 / LANES), ROW = CH / 2, STEPS = 8;
  static constexpr int ITEMS = STEPS * ROW, U = ITEMS / 32;  // of u, dt, z, y; a lane's
  static constexpr int ELEM = BF16 ? 2 : 4;
  // b and c in fp32 in shared memory; else every thread makes its own of bf16. A position's 2 N values
  // are converted by the warp for 512 / N channels: 582 against 612 us at N = 16 (scan of 32 x 512
  // positions, 8192 channels), but 740 against 670 at N = 32 and 461 against 346 at 64.
  static constexpr bool WIDEN = BF16 && N <= 16;
  static constexpr int COPY = STEPS * CH * ELEM / 16, NCOPY = STEPS * N * ELEM / 16;  // 16-byte copies of u, dt or z, and of b or c
  static_assert(CH % 8 == 0, "whole copies");
  static_assert(ITEMS % 32 == 0, "every lane has as many");
};

// A warp's part of shared memory: two tiles as they lie in memory, one of which is being loaded,
// and of the other, the tile at work, the items (the pair's steps, and steps times inputs) and the readout.
template <class C>
struct WarpSmem {
  struct Tile {
    alignas(16) unsigned char u[C::COPY * 16], dt[C::COPY * 16], z[C::COPY * 16], b[C::NCOPY * 16], c[C::NCOPY * 16];
  } raw[2];
  ulonglong2 in[C::ITEMS];
  float y[C::STEPS][C::CH];
  float b[C::WIDEN ? C::STEPS : 1][C::N], c[C::WIDEN ? C::STEPS : 1][C::N];
  // bias: with softplus its product with log2(e) and what its rounding lost. The step's argument is off
  // by one rounding of dt and one of the sum, and by none of bias.
  float bias[2][C::CH], skip[C::CH];
};

// Where the prompts' channels are too few for the GPU, prompts are cut into parts of `part` positions
// that are scanned side by side. A first kernel (SUMMARY) takes every part but the last from a state
// of zero: end[j], and sum[j], the sum of its steps. A second one goes through the parts with the
// prompt's state, h <- exp(sum[j] a) h + end[j], and leaves in end[j] the state after part j. (Every
// part's warps doing that for themselves read O(parts^2) states: 45 MB for one prompt of 1021
// positions and 2048 channels.)
struct ScanParams {
  gdn_ssm s;
  int32_t* status;
  int32_t per_group, blocks;  // channels of a group, and blocks of them
  int32_t parts, part;        // parts of a prompt at most, and positions of one
  uint32_t tasks;             // (request, part, channel block)
  float* init;                // [B][D][N]: the states before the prompts
  float* end;                 // [B][parts - 1][D][N]
  float* sum;                 // [B][parts - 1][D]
};

template <class C, bool SUMMARY>
__global__ void __launch_bounds__(kWarps * 32, kCtas) gdn_ssm_scan_kernel(const ScanParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const gdn_ssm& s = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  WarpSmem<C>& sm = reinterpret_cast<WarpSmem<C>*>(smem_raw)[warp];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t task = blockIdx.x * kWarps + warp;
  if (task >= p.tasks) return;
  const uint32_t all_blocks = static_cast<uint32_t>(p.blocks * s.num_groups), parts = SUMMARY ? p.parts - 1 : p.parts;
  const uint32_t row = task / all_blocks;
  const int block = static_cast<int>(task - row * all_blocks), b = static_cast<int>(row / parts), part_no = static_cast<int>(row - b * parts);
  const int group = block / p.blocks, in_group = (block - group * p.blocks) * C::CH;
  const int c0 = group * p.per_group + in_group, count = min(C::CH, p.per_group - in_group);
  const int slot = s.slot[b];
  if (slot < 0) return;
  const int len = s.seq_lens != nullptr ? s.seq_lens[b] : s.num_tokens;
  const bool bad_slot = slot >= s.num_slots, bad_len = len < 0 || len > s.num_tokens;
  if (bad_slot || bad_len) {
    if (block == 0 && part_no == 0 && lane == 0) atomic_status(p.status, bad_slot ? GDN_STATUS_BAD_SLOT : GDN_STATUS_BAD_LEN);
    return;
  }
  const int begin = part_no * p.part, end = min(len - begin, p.part) + begin;
  if (begin >= len) return;
  const bool last = end == len;
  if (SUMMARY && last && part_no > 0) return;  // nothing comes after it

  // ---- this thread's states -----------------------------------------------------------------
  const int set = lane / C::LANES, part = lane % C::LANES;
  const bool mine_live = set * C::OWN < count;
  float* const state = s.state + (static_cast<int64_t>(slot) * s.channels + c0 + set * C::OWN) * C::N + part * 8;
  f32x2 h[C::OWN][4], a[C::OWN][4];  // [channel][pair of states]
  auto load_states = [&](const float* from, f32x2 (&to)[C::OWN][4]) {
#pragma unroll
    for (int i = 0; i < C::OWN; ++i) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        ulonglong2 x = make_ulonglong2(0, 0);
        if (mine_live) x = *reinterpret_cast<const ulonglong2*>(from + i * C::N + j * 2);
        to[i][j] = x.x, to[i][j + 1] = x.y;
      }
    }
  };
  auto store_states = [&](float* to, const f32x2 (&from)[C::OWN][4]) {
    if (!mine_live) return;
#pragma unroll
    for (int i = 0; i < C::OWN; ++i)
#pragma unroll
      for (int j = 0; j < 4; j += 2) *reinterpret_cast<ulonglong2*>(to + i * C::N + j * 2) = make_ulonglong2(from[i][j], from[i][j + 1]);
  };
  load_states(s.a + static_cast<int64_t>(c0 + set * C::OWN) * C::N + part * 8, a);
#pragma unroll
  for (int i = 0; i < C::OWN; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) a[i][j] = mul2(a[i][j], both(kLog2e));
  // this thread's place in init, and in end and sum of part j
  const int64_t mine = static_cast<int64_t>(c0 + set * C::OWN) * C::N + part * 8, per_request = static_cast<int64_t>(s.channels) * C::N;
  auto end_of = [&](int j) { return p.end + (static_cast<int64_t>(b) * (p.parts - 1) + j) * per_request + mine; };
  auto sum_of = [&](int j) { return p.sum + (static_cast<int64_t>(b) * (p.parts - 1) + j) * s.channels + c0 + set * C::OWN; };
  load_states(p.parts == 1 || (SUMMARY && part_no == 0) ? state : part_no == 0 ? p.init + b * per_request + mine : end_of(part_no - 1), h);
  f32x2 steps_sum[C::OWN] = {};  // both halves alike
  if (SUMMARY) {
    // the last part's scan overwrites the slot's state while others still begin
    if (part_no == 0) store_states(p.init + b * per_request + mine, h);
    if (last) return;
#pragma unroll
    for (int i = 0; i < C::OWN; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) h[i][j] = 0;
  }
  const bool softplus = (s.flags & GDN_DT_SOFTPLUS) != 0u;
  for (int c = lane; c < C::CH; c += 32) {
    const float bias = s.dt_bias != nullptr && c < count ? s.dt_bias[c0 + c] : 0.0f;
    sm.bias[0][c] = softplus ? bias * kLog2e : bias;
    sm.bias[1][c] = softplus ? fmaf(bias, kLog2e, -(bias * kLog2e)) : 0.0f;
    sm.skip[c] = s.skip != nullptr && c < count ? s.skip[c0 + c] : 0.0f;
  }

  // ---- tiles of the inputs ----------------------------------------------------------------------
  constexpr int kE = C::ELEM, kPer = 16 / kE;  // elements of a copy
  constexpr int kRow = C::CH / kPer, kNRow = C::N / kPer;  // copies of a row
  const int col = lane % kRow * kPer, ncol = lane % kNRow * kPer;
  auto row_at = [&](const void* base, const int64_t* strides, int64_t first, int per) {
    return static_cast<const unsigned char*>(base) + (b * strides[0] + (begin + lane / per) * strides[1] + first) * kE;
  };
  // this lane's first copies of the next tile
  const unsigned char* u_at = row_at(s.u, s.u_strides, c0 + col, kRow);
  const unsigned char* dt_at = row_at(s.dt, s.dt_strides, c0 + col, kRow);
  const unsigned char* z_at = row_at(s.z, s.z_strides, c0 + col, kRow);
  const unsigned char* b_at = row_at(s.b, s.b_strides, group * s.b_strides[2] + ncol, kNRow);
  const unsigned char* c_at = row_at(s.c, s.c_strides, group * s.c_strides[2] + ncol, kNRow);
  const bool gated = !SUMMARY && s.z != nullptr, col_live = col < count;
  auto fetch = [&](int t0) {
    typename WarpSmem<C>::Tile& to = sm.raw[t0 / C::STEPS & 1];
    auto copies = [&](unsigned char* dst, const unsigned char*& src, int64_t stride, int per, int all, bool live) {
#pragma unroll
      for (int k = 0; k < (all + 31) / 32; ++k) {
        const int row = lane / per + 32 / per * k;
        if (all % 32 != 0 && lane + 32 * k >= all) continue;
        copy16(dst + (lane + 32 * k) * 16, src + (32 / per * k) * stride * kE, live && t0 + row < end);
      }
      src += C::STEPS * stride * kE;
    };
    copies(to.u, u_at, s.u_strides[1], kRow, C::COPY, col_live);
    copies(to.dt, dt_at, s.dt_strides[1], kRow, C::COPY, col_live);
    if (gated) copies(to.z, z_at, s.z_strides[1], kRow, C::COPY, col_live);
    copies(to.b, b_at, s.b_strides[1], kNRow, C::NCOPY, true);
    if (!SUMMARY) copies(to.c, c_at, s.c_strides[1], kNRow, C::NCOPY, true);
  };

  const int pair = lane % C::ROW;  // of all items of this lane: ROW divides 32
  const bool pair_live = pair * 2 < count;
  const int64_t y_row = static_cast<int64_t>(s.channels) * kE;
  unsigned char* y_at = static_cast<unsigned char*>(s.y) +
                        ((static_cast<int64_t>(b) * s.num_tokens + begin + lane / C::ROW) * s.channels + c0 + pair * 2) * kE;
  fetch(begin);
  for (int t0 = begin; t0 < end; t0 += C::STEPS) {
    const typename WarpSmem<C>::Tile& raw = sm.raw[t0 / C::STEPS & 1];
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();  // the tile is there, and the last one is done with
    if (t0 + C::STEPS < end) fetch(t0 + C::STEPS);

    // ---- steps, inputs, b and c of the tile, in fp32 -----------------------------------------------
    const f32x2 bias = *reinterpret_cast<const f32x2*>(&sm.bias[0][pair * 2]), rest = *reinterpret_cast<const f32x2*>(&sm.bias[1][pair * 2]);
#pragma unroll
    for (int k = 0; k < C::U; ++k) {
      const int i = lane + 32 * k;
      f32x2 dt = pair_of<C::BF16>(reinterpret_cast<const Raw2<C::BF16>*>(raw.dt)[i]);
      if (softplus)
        dt = softplus_2(add2(fma2(dt, both(kLog2e), rest), bias));
      else
        dt = add2(dt, bias);
      if (t0 + i / C::ROW >= end) dt = 0;  // the state passes a position of no prompt unchanged
      const f32x2 x = mul2(pair_of<C::BF16>(reinterpret_cast<const Raw2<C::BF16>*>(raw.u)[i]), dt);
      sm.in[i] = make_ulonglong2(dt, x);
    }
    if constexpr (C::WIDEN) {
#pragma unroll
      for (int k = 0; k < C::STEPS * C::N / 64; ++k) {
        const int i = lane + 32 * k;
        reinterpret_cast<f32x2*>(sm.b)[i] = pair_of<C::BF16>(reinterpret_cast<const Raw2<C::BF16>*>(raw.b)[i]);
        if (!SUMMARY) reinterpret_cast<f32x2*>(sm.c)[i] = pair_of<C::BF16>(reinterpret_cast<const Raw2<C::BF16>*>(raw.c)[i]);
      }
    }
    __syncwarp();

    // ---- the recurrence ----------------------------------------------------------------------------
#pragma unroll
    for (int t = 0; t < C::STEPS; ++t) {
      f32x2 dts[C::OWN], dus[C::OWN];
      if constexpr (C::OWN == 2) {
        const ulonglong2 in = sm.in[t * C::ROW + set];
        const float2 dt = unpack2(in.x), du = unpack2(in.y);
        dts[0] = both(dt.x), dts[1] = both(dt.y), dus[0] = both(du.x), dus[1] = both(du.y);
      } else {
        const float* const in = reinterpret_cast<const float*>(&sm.in[t * C::ROW + set / 2]) + set % 2;
        dts[0] = both(in[0]), dus[0] = both(in[2]);
      }
      f32x2 bb[4], cc[4] = {0, 0, 0, 0};
      if constexpr (C::WIDEN) {
        pairs8<false>(reinterpret_cast<const unsigned char*>(&sm.b[t][part * 8]), bb);
        if (!SUMMARY) pairs8<false>(reinterpret_cast<const unsigned char*>(&sm.c[t][part * 8]), cc);
      } else {
        pairs8<C::BF16>(raw.b + (t * C::N + part * 8) * kE, bb);
        if (!SUMMARY) pairs8<C::BF16>(raw.c + (t * C::N + part * 8) * kE, cc);
      }
      float sum[C::OWN];
#pragma unroll
      for (int i = 0; i < C::OWN; ++i) {
        f32x2 acc = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][j] = fma2(ex2_2(mul2(dts[i], a[i][j])), h[i][j], mul2(dus[i], bb[j]));
          if (!SUMMARY) acc = j == 0 ? mul2(h[i][j], cc[j]) : fma2(h[i][j], cc[j], acc);
        }
        const float2 v = unpack2(acc);
        sum[i] = v.x + v.y;
        if (SUMMARY) steps_sum[i] = add2(steps_sum[i], dts[i]);
      }
      if constexpr (!SUMMARY) {
        // Sums over the lanes of a pair of channels: a lane keeps one channel and gives the other
        // away; further lanes add what is left.
        if constexpr (C::OWN == 1) {
#pragma unroll
          for (int off = C::LANES / 2; off > 0; off >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], off);
          if (part == 0) sm.y[t][set] = sum[0];
        } else if constexpr (C::LANES == 1) {
          *reinterpret_cast<float2*>(&sm.y[t][set * 2]) = make_float2(sum[0], sum[1]);
        } else {
          constexpr int kOwn = C::LANES / 2;
          const bool second = (part & kOwn) != 0;
          float one = (second ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, second ? sum[0] : sum[1], kOwn);
#pragma unroll
          for (int off = kOwn / 2; off > 0; off >>= 1) one += __shfl_xor_sync(0xffffffffu, one, off);
          if (part % kOwn == 0) sm.y[t][set * 2 + part / kOwn] = one;
        }
      }
    }
    __syncwarp();

    // ---- readout ----------------------------------------------------------------------------------
    if constexpr (!SUMMARY) {
      const f32x2 skip = *reinterpret_cast<const f32x2*>(&sm.skip[pair * 2]);
#pragma unroll
      for (int k = 0; k < C::U; ++k) {
        const int i = lane + 32 * k, t = i / C::ROW;
        if (!pair_live || t0 + t >= end) continue;
        f32x2 y = fma2(skip, pair_of<C::BF16>(reinterpret_cast<const Raw2<C::BF16>*>(raw.u)[i]), reinterpret_cast<const f32x2*>(sm.y)[i]);
        if (gated) y = mul2(y, silu_2<!C::BF16>(pair_of<C::BF16>(reinterpret_cast<const Raw2<C::BF16>*>(raw.z)[i])));
        *reinterpret_cast<Raw2<C::BF16>*>(y_at + 32 / C::ROW * k * y_row) = raw_of<C::BF16>(y);
      }
      y_at += C::STEPS * y_row;
    }
  }

  if (SUMMARY) {
    store_states(end_of(part_no), h);
    if (mine_live && part == 0) {
#pragma unroll
      for (int i = 0; i < C::OWN; ++i) sum_of(part_no)[i] = unpack2(steps_sum[i]).x;
    }
  } else if (last) {
    store_states(state, h);
  }
}

// A state after a part. The decays of a part may pass fp32 together (a > 0) where none does by itself:
// a state of zero stays zero under them.
__device__ __forceinline__ float joined(float x, float h, float end) { return h == 0.0f ? end : fmaf(ex2(x), h, end); }

// Four states a thread, several parts' loads in flight.
constexpr int kJoinThreads = 128, kJoinAhead = 8;
__global__ void __launch_bounds__(kJoinThreads) gdn_ssm_join_kernel(const ScanParams p) {
  const gdn_ssm& s = p.s;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t states = static_cast<int64_t>(s.channels) * s.state_size;
  const uint32_t blocks = static_cast<uint32_t>((states / 4 + kJoinThreads - 1) / kJoinThreads);
  const int b = static_cast<int>(blockIdx.x / blocks);
  const int64_t at = (static_cast<int64_t>(blockIdx.x - b * blocks) * kJoinThreads + threadIdx.x) * 4;
  const int slot = s.slot[b], len = s.seq_lens != nullptr ? s.seq_lens[b] : s.num_tokens;
  if (at >= states || slot < 0 || slot >= s.num_slots || len <= p.part || len > s.num_tokens) return;
  const int parts = (len - 1) / p.part;  // that another one comes after
  const float4 a = *reinterpret_cast<const float4*>(s.a + at);
  float4 h = *reinterpret_cast<const float4*>(p.init + b * states + at);
  float* const end = p.end + b * (p.parts - 1) * states + at;
  const float* const sum = p.sum + static_cast<int64_t>(b) * (p.parts - 1) * s.channels + at / s.state_size;
  for (int j0 = 0; j0 < parts; j0 += kJoinAhead) {
    float4 e[kJoinAhead];
    float t[kJoinAhead];
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j) {
      if (j0 + j >= parts) break;
      e[j] = *reinterpret_cast<const float4*>(end + (j0 + j) * states);
      t[j] = sum[static_cast<int64_t>(j0 + j) * s.channels] * kLog2e;
    }
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j) {
      if (j0 + j >= parts) break;
      h = make_float4(joined(t[j] * a.x, h.x, e[j].x), joined(t[j] * a.y, h.y, e[j].y), joined(t[j] * a.z, h.z, e[j].z),
                      joined(t[j] * a.w, h.w, e[j].w));
      *reinterpret_cast<float4*>(end + (j0 + j) * states) = h;
    }
  }
}

// How prompts are cut: as a rough model of the times says, whose constants are measured. A position
// takes 0.18 us where a warp has its quarter of an SM to itself, 0.225 where two share one, and 0.09
// for each of more, up to the four that fit and in rounds beyond. With one channel a thread there are
// twice the warps, which take 0.13, 0.15 and 0.058 each: sooner through a prompt where they have room
// (64 positions of 2048 channels: 11.2 us, 14.5 with two), later where not (a full GPU: 656 and 584).
// Parts take two thirds more for their ends, two launches, and 6 us a further round to begin (3 prompts
// of 509 positions of 64 states, 768 warps: 103 us in 3 parts, 113 in 11). Cuts that fill the GPU one
// to four times are compared with none:
//   whole wins where there are enough warps (16 x 1024 positions of 4096 channels, 2048 warps: 342 us,
//   417 in two parts) or few positions (2048 channels, two a thread: 64 positions 14.5 us, 15.9 in two
//   parts, but 96 20.1 and 16.0; 768 warps: 200 positions 47.5 and 49.7);
//   parts elsewhere (16384 positions, 256 warps: 2906 us whole, 1009 in 9 parts, which fill 0.95 of the
//   GPU, 943 in 19, which fill it twice, 1126 in 10, which leave half of the second round empty), and
//   where prompts have lengths of their own, of which a whole one holds up the end (8 ragged prompts,
//   1024 warps: 457 us whole, 292 in 7 parts; of equal length 477 and 471): parts without positions
//   cost next to nothing, so 0.6 of the time is reckoned there.
// The model knows neither types nor groups: it takes four CTAs an SM also where two fit (kCtas), blocks
// of 512 / N channels also where groups end inside them, and prompts with seq_lens for ragged ones.
// A join goes through all parts in turn, so there are at most sqrt(T) of them, of 32 positions at least.
struct Cut {
  int32_t parts, part;
  int32_t own;  // channels of a thread
};
constexpr int32_t kShortest = 32, kRounds = 4;
constexpr int64_t kResident = kSms * kCtas * kWarps;  // warps of a full GPU
int64_t warps_of(int64_t batch, int32_t channels, int32_t state_size) {
  const int32_t of_warp = 512 / state_size;  // channels
  return batch * ((channels + of_warp - 1) / of_warp);
}
// of one prompt
int64_t most_parts(int32_t tokens) {
  const int64_t root = static_cast<int64_t>(std::sqrt(static_cast<double>(tokens))), whole = (tokens + kShortest - 1) / kShortest;
  return root < whole ? root : whole;
}
Cut cut_of(int32_t batch, int32_t tokens, int32_t channels, int32_t state_size, bool ragged) {
  constexpr int32_t kRound = 8, kQuarters = kSms * 4;
  const int64_t warps = warps_of(batch, channels, state_size);
  auto position = [](int64_t all_warps) {  // us
    const int64_t shared = (all_warps + kQuarters - 1) / kQuarters;
    return shared <= 1 ? 0.18 : shared <= 2 ? 0.225 : 0.09 * static_cast<double>(shared);
  };
  auto position_of_one = [](int64_t all_warps) {  // with a channel a thread
    const int64_t shared = (all_warps + kQuarters - 1) / kQuarters;
    return shared <= 1 ? 0.13 : shared <= 2 ? 0.15 : 0.058 * static_cast<double>(shared);
  };
  Cut best{1, tokens, 2};
  double least = 2.5 + tokens * position(warps);
  const double took_one = 2.5 + tokens * position_of_one(2 * warps);
  if (state_size < 64 && took_one < least) least = took_one, best.own = 1;
  const int64_t most = most_parts(tokens);
  for (int rounds = 1; rounds <= kRounds; ++rounds) {
    int64_t parts = kResident * rounds / warps;
    if (parts > most) parts = most;
    if (parts < 2) continue;
    int64_t part = (tokens + parts - 1) / parts;
    part = part > kShortest ? (part + kRound - 1) / kRound * kRound : kShortest;
    parts = (tokens + part - 1) / part;
    const double all = static_cast<double>(part) * (5.0 / 3.0) * position(warps * parts);
    const double took = ragged ? 5.0 + 0.6 * all : 6.0 * rounds - 1.0 + all;
    if (parts > 1 && took < least) least = took, best = {static_cast<int32_t>(parts), static_cast<int32_t>(part), 2};
  }
  return best;
}

template <class C, bool SUMMARY>
cudaError_t launch_parts(ScanParams p, cudaStream_t stream) {
  const int64_t tasks = static_cast<int64_t>(p.blocks) * p.s.num_groups * p.s.batch * (SUMMARY ? p.parts - 1 : p.parts);
  p.tasks = static_cast<uint32_t>(tasks);
  constexpr int kBytes = kWarps * static_cast<int>(sizeof(WarpSmem<C>));
  static std::atomic<bool> allowed[kDevices];
  const cudaError_t err = allow_shared(reinterpret_cast<const void*>(gdn_ssm_scan_kernel<C, SUMMARY>), kBytes, allowed);
  if (err != cudaSuccess) return err;
  return launch_overlapped(gdn_ssm_scan_kernel<C, SUMMARY>, p, dim3((p.tasks + kWarps - 1) / kWarps), kWarps * 32, kBytes, 1u, stream);
}

template <int N, bool BF16>
cudaError_t launch_scan(const SsmParams& given, void* workspace, cudaStream_t stream) {
  using C = Cfg<N, BF16, 2>;
  const gdn_ssm& s = given.s;
  const Cut cut = cut_of(s.batch, s.num_tokens, s.channels, s.state_size, s.seq_lens != nullptr);
  ScanParams p{s, given.status, s.channels / s.num_groups, 0, cut.parts, cut.part, 0, nullptr, nullptr, nullptr};
  if constexpr (N < 64) {  // a row of four channels would be no whole copy
    using One = Cfg<N, BF16, 1>;
    p.blocks = (p.per_group + One::CH - 1) / One::CH;
    if (cut.own == 1) return launch_parts<One, false>(p, stream);
  }
  p.blocks = (p.per_group + C::CH - 1) / C::CH;
  if (cut.parts > 1) {
    const int64_t states = static_cast<int64_t>(s.batch) * s.channels * s.state_size;
    p.init = static_cast<float*>(workspace);
    p.end = p.init + states;
    p.sum = p.end + states * (cut.parts - 1);
    cudaError_t err = launch_parts<C, true>(p, stream);
    if (err != cudaSuccess) return err;
    const int64_t blocks = (static_cast<int64_t>(s.channels) * s.state_size / 4 + kJoinThreads - 1) / kJoinThreads;
    err = launch_overlapped(gdn_ssm_join_kernel, p, dim3(static_cast<unsigned>(blocks * s.batch)), kJoinThreads, 0, 1u, stream);
    if (err != cudaSuccess) return err;
  }
  return launch_parts<C, false>(p, stream);
}

template <bool BF16>
cudaError_t launch_type(const SsmParams& p, void* workspace, cudaStream_t stream) {
  switch (p.s.state_size) {
    case 8: return launch_scan<8, BF16>(p, workspace, stream);
    case 16: return launch_scan<16, BF16>(p, workspace, stream);
    case 32: return launch_scan<32, BF16>(p, workspace, stream);
    default: return launch_scan<64, BF16>(p, workspace, stream);
  }
}

}  // namespace

// What every call of these channels and states needs that has no more requests and positions, so that a
// buffer of the largest serves all: prompts have at most most_parts() parts each and, as cuts fill the
// GPU at most kRounds times, all of them together at most so many as there is room for. Of n parts there
// are the states before them and after all but the last, and as many sums of steps.
size_t ssm_workspace_bytes(int32_t batch, int32_t tokens, int32_t channels, int32_t state_size) {
  const int64_t each = most_parts(tokens), all = kResident * kRounds / warps_of(1, channels, state_size);
  if (each < 2 || all < 2) return 0;
  const int64_t parts = batch * each < all ? batch * each : all;
  return static_cast<size_t>(parts) * channels * (state_size + 1) * sizeof(float);
}

bool ssm_scan_in_parts(const gdn_ssm& s) {
  return cut_of(s.batch, s.num_tokens, s.channels, s.state_size, s.seq_lens != nullptr).parts > 1;
}

cudaError_t launch_ssm_scan(const SsmParams& given, void* workspace, cudaStream_t stream) {
  SsmParams p = given;
  // The stride of a single token may be any, but copies of the positions past it, which read nothing,
  // still want an aligned address.
  if (p.s.num_tokens == 1) p.s.u_strides[1] = p.s.dt_strides[1] = p.s.z_strides[1] = p.s.b_strides[1] = p.s.c_strides[1] = 0;
  return (p.s.flags & GDN_QKV_BF16) != 0u ? launch_type<true>(p, workspace, stream) : launch_type<false>(p, workspace, stream);
}

}  // namespace gdn
