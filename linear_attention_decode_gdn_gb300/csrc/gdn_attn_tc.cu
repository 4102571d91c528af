// gdn_attn_tc.cu -- attention over the paged cache on the tensor cores: head sizes 64, 128 and
// 256, and latent rows of 512 + 64.
//
// Decode attention reads every cached byte once for a handful of query rows, so the matrix
// products are laid out around the cache: the tile's 128 positions are the 128 rows of a
// tcgen05 MMA, the query rows (16, 32 or 64 columns) its narrow side.
//
//   S^T [128 positions x N] = K [128 x dk] (q [N x dk])^T        A, B from shared memory
//   P^T = 2^(S^T - m), m one running maximum a column            in registers, a thread a position
//   O^T [dv x N] += V^T [dv x 128] P^T [128 x N]                 A = V as it lies in memory (its
//                                                                rows run along dv), B from shared
//
// So neither K nor V is transposed or padded, the accumulators take (2 + dv / 128) N columns of
// TMEM, and a query group of 4 or 16 costs the same as it streams by.
//
// One CTA an SM, 256 threads. Warp 0 gathers pages by TMA into a ring of 16 KB chunks (128
// positions x 64 elements, 128-byte swizzle; pages of 16 .. 128 positions are boxes of one
// chunk). Warp 1 issues the MMAs: scores of tile i + 1 before values of tile i, so the tensor
// core works while the softmax does. Warps 2 and 3 lay out the next unit's queries. Warps 4 - 7
// are the softmax: one thread a position, N columns each; sums of weights stay in the threads
// until the unit ends. The running maximum is raised (and O^T rescaled in TMEM) only where a
// score passes it by 2^8, so most tiles need one barrier and no reduction; weights up to 2^8
// lose nothing in bf16 or fp32.
#include "gdn_attn.cuh"
#include "gdn_tc.cuh"
#include "gdn_tmap.h"

#include <cuda_bf16.h>

namespace gdn {

namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kChunk = kTile * 128;          // bytes: 128 positions x 64 bf16
constexpr int kSmemMost = 227 * 1024;
constexpr int kMiscBytes = 3072;
constexpr float kRaise = 8.0f;               // log2 of what a weight may grow to

template <int DK_, int DV_, int N_, bool LATENT_>
struct Cfg {
  static constexpr int DK = DK_, DV = DV_, N = N_;
  static constexpr bool LATENT = LATENT_;
  static constexpr int KC = LATENT ? DV / 64 : DK / 64;   // key chunks of the ring
  static constexpr int VC = LATENT ? 0 : DV / 64;         // value chunks (a latent row's key is its value)
  static constexpr int PER = KC + VC;                     // ring chunks a tile
  static constexpr int TAILC = LATENT ? (DK - DV) / 64 : 0;  // chunks of the key's tail, in a ring of their own
  static constexpr int MB = DV > 128 ? DV / 128 : 1;      // blocks of 128 rows of O^T
  static constexpr int PB = LATENT && N > 16 ? 1 : 2;     // buffers of weights
  static constexpr int TAILS = LATENT ? (N > 16 ? 1 : 2) : 0;
  static constexpr int QBYTES = N * DK * 2, PBYTES = N * kTile * 2;
  static constexpr int FIXED = kMiscBytes + QBYTES + PB * PBYTES + TAILS * kChunk;
  static constexpr int FIT = (kSmemMost - FIXED) / kChunk;
  static constexpr int RING = (FIT > 12 ? 12 : FIT) & ~1;  // even: a block of V is two chunks side by side
  static constexpr size_t SMEM = static_cast<size_t>(FIXED) + RING * kChunk;
  static constexpr int TMEM_USED = (2 + MB) * N;
  static constexpr int TMEM = TMEM_USED <= 32 ? 32 : TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  // key chunks of the next tile that fit beside a tile whose values are still needed
  static constexpr int AHEAD = LATENT ? (RING - PER < KC ? RING - PER : KC) : KC;
  static_assert(RING >= PER && TAILC <= 1, "a tile fits the rings");
  static_assert(N % 16 == 0 && N <= 64 && SMEM <= kSmemMost && TMEM_USED <= 512, "fits");
};

struct Misc {
  uint64_t full[12], empty[12];
  uint64_t tail_full[2], tail_empty[2];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2];
  uint64_t drained;
  uint32_t tmem;
  uint32_t timeout;
  float m[64];
  float per_warp[4][64];
  int64_t rows[64];
  ShareScratch scratch;
};
static_assert(sizeof(Misc) <= kMiscBytes, "shared memory plan");

struct TcParams {
  AttnParams a;
  int32_t box;  // positions of one TMA box: min(page_size, 128)
  CUtensorMap k, v;
};

// ---- PTX ----------------------------------------------------------------------------------
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Operand tile of 128-byte rows, 128-byte swizzle (8 rows = 1024 bytes repeat).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return tc::smem_desc(saddr, lbo, sbo) | (2ull << 61);
}
// kind::f16, called by a whole warp with uniform operands; one elected lane issues.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 l;\n elect.sync l|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t head, int32_t pos,
                                        int32_t page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(head), "r"(pos), "r"(page)
      : "memory");
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n bar.red.or.pred b, 1, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sums of N columns over the warp's lanes: afterwards lane holds the sums of columns
// lane * N / 32 .. (N >= 32) or of column lane * N / 32 (N = 16).
template <int N>
__device__ __forceinline__ void column_sums(float (&v)[N], int lane) {
#pragma unroll
  for (int off = 16, n = N; off > 0; off >>= 1) {
    if (n > 1) {
      const int half = n / 2;
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        if (j >= half) continue;
        const float keep = upper ? v[j + half] : v[j], send = upper ? v[j] : v[j + half];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
      n = half;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    }
  }
}

// A wait with a limit. The first one that runs out raises a flag that ends every other wait of
// the CTA, so the kernel returns soon after (and reports GDN_STATUS_TIMEOUT).
__device__ __forceinline__ bool waited(uint64_t* bar, uint32_t parity, Misc& sm) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile uint32_t* const flag = &sm.timeout;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*flag != 0u) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *flag = 1u;
      return false;
    }
  }
  return true;
}
// The same for a whole warp that goes on together.
__device__ __forceinline__ bool warp_waited(uint64_t* bar, uint32_t parity, Misc& sm) {
  return __all_sync(0xffffffffu, waited(bar, parity, sm));
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1) gdn_attn_tc_kernel(const __grid_constant__ TcParams tp) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const AttnParams& p = tp.a;
  constexpr int N = C::N;
  constexpr uint32_t kTails = C::TAILS > 0 ? C::TAILS : 1;
  unsigned char* const ring = smem;
  unsigned char* const tails = ring + C::RING * kChunk;
  unsigned char* const weights = tails + C::TAILS * kChunk;
  unsigned char* const queries = weights + C::PB * C::PBYTES;
  Misc& sm = *reinterpret_cast<Misc*>(queries + C::QBYTES);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.tail_full[i], 1);
      mbar_init(&sm.tail_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 128);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.q_full, 64);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drained, 1);
    sm.timeout = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&sm.tmem, C::TMEM);
    tc::tmem_relinquish();
  }
  griddep_wait();
  write_empty<kThreads>(p);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const Share share = find_share<kThreads>(p, sm.scratch);
  if (tid == 0) write_record(p, share);

  Walk walk(share);
  Segment seg;

  if (warp == 0) {
    // ---- pages into the ring --------------------------------------------------------------
    uint32_t put = 0, tail_put = 0;  // chunks issued
    uint32_t bad = 0;
    const int boxes = kTile / tp.box;  // of one chunk; lane l issues box l
    bool ok = true;
    while (ok && walk.next(p, &seg)) {
      const int32_t lower = lower_bound_of(p, seg.n, seg.col_base / p.group);
      const int32_t* row = p.table + static_cast<int64_t>(seg.b) * p.max_pages;
      auto page_at = [&](int tile) -> int32_t {
        const int64_t at = static_cast<int64_t>(tile) * kTile + lane * tp.box;
        // a box that no query of the unit sees reads as zero, as one of a page that is none
        if (lane >= boxes || at >= seg.n || at + tp.box <= lower) return p.num_pages;
        const int32_t page = row[at / p.page_size];
        if (page >= 0 && page < p.num_pages) return page;
        bad = GDN_STATUS_BAD_PAGE;
        return p.num_pages;
      };
      int32_t page = page_at(seg.tile);
      for (int tile = seg.tile; ok && tile < seg.tile + seg.tiles; ++tile) {
        const int32_t next = tile + 1 < seg.tile + seg.tiles ? page_at(tile + 1) : 0;
        const int32_t pos = (tile * kTile + lane * tp.box) % p.page_size;
        for (int c = 0; c < C::PER; ++c, ++put) {
          const uint32_t slot = put % C::RING;
          ok = warp_waited(&sm.empty[slot], ((put / C::RING) & 1u) ^ 1u, sm);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], kChunk);
          __syncwarp();
          const bool value = !C::LATENT && c >= C::KC;
          if (lane < boxes)
            tma_box(smem_addr(ring) + slot * kChunk + lane * tp.box * 128, value ? &tp.v : &tp.k,
                    (value ? c - C::KC : c) * 64, seg.kv_head, pos, page, &sm.full[slot]);
        }
        if (C::TAILC > 0 && ok) {
          const uint32_t slot = tail_put % kTails;
          ok = warp_waited(&sm.tail_empty[slot], ((tail_put / kTails) & 1u) ^ 1u, sm);
          if (ok) {
            if (lane == 0) mbar_arrive_expect_tx(&sm.tail_full[slot], kChunk);
            __syncwarp();
            if (lane < boxes)
              tma_box(smem_addr(tails) + slot * kChunk + lane * tp.box * 128, &tp.k, C::KC * 64, seg.kv_head, pos, page,
                      &sm.tail_full[slot]);
            ++tail_put;
          }
        }
        page = next;
      }
    }
    if (!ok) {  // nothing may still be on its way into this CTA's memory when it ends
      for (uint32_t i = put > C::RING ? put - C::RING : 0; i < put; ++i)
        mbar_wait(&sm.full[i % C::RING], (i / C::RING) & 1u);
      for (uint32_t i = tail_put > kTails ? tail_put - kTails : 0; i < tail_put; ++i)
        mbar_wait(&sm.tail_full[i % kTails], (i / kTails) & 1u);
    }
    if (bad != 0u) atomic_status(p.status, bad);
  } else if (warp == 1) {
    // ---- matrix products --------------------------------------------------------------------
    constexpr uint32_t kScores = idesc_bf16(128, N, false, false), kValues = idesc_bf16(128, N, true, true);
    const uint32_t ring_at = smem_addr(ring), tails_at = smem_addr(tails), q_at = smem_addr(queries),
                   w_at = smem_addr(weights);
    uint32_t i = 0, units = 0;  // tiles and units begun
    bool ok = true;
    uint32_t first_of_last = 0;  // whether the last tile with scores was its unit's first

    // key chunks [from, to) of tile i against the queries
    auto scores = [&](int from, int to) {
      for (int c = from; c < to && ok; ++c) {
        const uint32_t n = i * C::PER + c, slot = n % C::RING;
        ok = warp_waited(&sm.full[slot], (n / C::RING) & 1u, sm);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t a = ring_at + slot * kChunk, b = q_at + c * (8 * N * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16(tmem + (i & 1u) * N, desc_sw128(a + k * 32, 16, 1024), tc::smem_desc(b + k * (2 * N * 16), N * 16, 128),
                   kScores, c > 0 || k > 0);
        if (!C::LATENT) tc::commit(&sm.empty[slot]);
      }
      if (C::TAILC > 0 && to == C::KC && ok) {
        const uint32_t slot = i % kTails;
        ok = warp_waited(&sm.tail_full[slot], (i / kTails) & 1u, sm);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t a = tails_at + slot * kChunk, b = q_at + C::KC * (8 * N * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16(tmem + (i & 1u) * N, desc_sw128(a + k * 32, 16, 1024), tc::smem_desc(b + k * (2 * N * 16), N * 16, 128),
                   kScores, 1);
        tc::commit(&sm.tail_empty[slot]);
      }
    };
    // values of tile j; `first`: of its unit
    auto values = [&](uint32_t j, uint32_t first) {
      const uint32_t buf = j % C::PB;
      ok = warp_waited(&sm.p_full[buf], (j / C::PB) & 1u, sm);
      if (!ok) return;
      tc::fence_after_sync();
      for (int m = 0; m < C::MB; ++m) {
        const uint32_t n = j * C::PER + (C::LATENT ? 0 : C::KC) + 2 * m, slot = n % C::RING;
        constexpr int kUse = C::DV >= 128 ? 2 : 1;
        if (!C::LATENT)
          for (int c = 0; c < kUse && ok; ++c) ok = warp_waited(&sm.full[slot + c], (n / C::RING) & 1u, sm);
        if (!ok) return;
        tc::fence_after_sync();
        // dv = 64 is the upper half of the 128 rows; the lower half multiplies the slot before (the
        // tile's keys, or what replaces them) and is never read
        const uint32_t a = ring_at + (C::DV >= 128 ? slot : slot - 1) * kChunk, b = w_at + buf * C::PBYTES;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16(tmem + 2 * N + m * N, desc_sw128(a + k * 2048, kChunk, 1024),
                   tc::smem_desc(b + k * 256, 128, kTile * 16), kValues, first == 0u || k > 0);
        for (int c = 0; c < kUse; ++c) tc::commit(&sm.empty[slot + c]);
      }
      tc::commit(&sm.pv_done[j & 1u]);
    };

    while (ok && walk.next(p, &seg)) {
      for (int t = 0; ok && t < seg.tiles; ++t) {
        if (t == 0) ok = warp_waited(&sm.q_full, units & 1u, sm);
        if (ok) ok = warp_waited(&sm.s_empty[i & 1u], ((i >> 1) & 1u) ^ 1u, sm);
        if (!ok) break;
        tc::fence_after_sync();
        if (C::AHEAD > 0) scores(0, C::AHEAD);
        if (C::AHEAD < C::KC) {
          if (ok && i > 0) values(i - 1, first_of_last);
          if (ok) scores(C::AHEAD, C::KC);
        }
        if (!ok) break;
        tc::commit(&sm.s_full[i & 1u]);
        if (t == seg.tiles - 1) tc::commit(&sm.q_empty);
        if (C::AHEAD == C::KC && i > 0) values(i - 1, first_of_last);
        first_of_last = t == 0;
        ++i;
      }
      ++units;
    }
    if (ok && i > 0) values(i - 1, first_of_last);
    // the last MMA has left TMEM and shared memory alone when this completes
    tc::commit(&sm.drained);
    if (!mbar_wait(&sm.drained, 0)) sm.timeout = 1u;
  } else if (warp < 4) {
    // ---- queries of the next unit -----------------------------------------------------------
    // K-major core matrices: 16 bytes of column n, element group e at (e * N + n) * 16
    uint32_t units = 0;
    while (walk.next(p, &seg)) {
      if (units > 0 && !waited(&sm.q_empty, (units - 1) & 1u, sm)) break;
      const int cols = min(N, p.cols - seg.col_base);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + seg.b * p.q_b;
      constexpr int kVecs = C::DK / 8;
#pragma unroll 4
      for (int v = tid - 64; v < N * kVecs; v += 64) {
        const int c = v / kVecs, e = v - c * kVecs;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (c < cols) {
          const int col = seg.col_base + c, t = col / p.group, h = seg.kv_head * p.group + (col - t * p.group);
          x = *reinterpret_cast<const uint4*>(q + t * p.q_t + h * p.q_h + e * 8);
        }
        *reinterpret_cast<uint4*>(queries + (e * N + c) * 16) = x;
      }
      tc::fence_smem_to_async();
      arrive(&sm.q_full);
      ++units;
    }
  } else {
    // ---- softmax ------------------------------------------------------------------------------
    const int r = tid - 128, w = warp - 4;  // this thread's position of the tile and TMEM lane
    const uint32_t lanes = tc::lane_base(w);
    uint32_t i = 0;
    // After a wait that ran out the threads still go through every barrier together (no later
    // wait holds them up) and write nothing more.
    bool ok = true;
    while (walk.next(p, &seg)) {
      const int cols = min(N, p.cols - seg.col_base);
      const int t_first = seg.col_base / p.group, t_last = (seg.col_base + cols - 1) / p.group;
      const int32_t lower = lower_bound_of(p, seg.n, t_first);
      const int32_t lower_last = lower_bound_of(p, seg.n, t_last);
      const int32_t* row = p.table + static_cast<int64_t>(seg.b) * p.max_pages;
      auto usable = [&](int tile) -> bool {
        const int64_t pos = static_cast<int64_t>(tile) * kTile + r;
        if (pos >= seg.n || pos < lower) return false;
        const int32_t page = row[pos / p.page_size];
        return page >= 0 && page < p.num_pages;
      };
      softmax_sync();  // the last unit's rows and maxima are read
      if (r < N) {
        sm.m[r] = -INFINITY;
        sm.rows[r] = r < cols ? row_of(p, seg.b, seg.kv_head, seg.col_base + r) : -1;
      }
      float l[N];
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] = 0.0f;
      softmax_sync();
      bool live = usable(seg.tile);
      for (int t = 0; t < seg.tiles; ++t, ++i) {
        const int tile = seg.tile + t;
        const int32_t begin = tile * kTile, pos = begin + r;
        const bool live_next = t + 1 < seg.tiles && usable(tile + 1);
        ok &= waited(&sm.s_full[i & 1u], (i >> 1) & 1u, sm);
        __syncwarp();
        tc::fence_after_sync();
        float s[N];
#pragma unroll
        for (int c = 0; c < N; c += 16) {
          float x[16];
          tc::ld16(tmem + lanes + (i & 1u) * N + c, x);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[c + j] = x[j];
        }
        tc::fence_before_sync();
        arrive(&sm.s_empty[i & 1u]);
        // every column sees every position of the tile, but where it is not live
        const bool plain = begin + kTile - 1 <= seg.n - p.T + t_first && begin >= lower_last;
        if (plain) {
#pragma unroll
          for (int c = 0; c < N; ++c) s[c] = live ? s[c] * p.scale_log2 : -INFINITY;
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int32_t last = seg.n - p.T + (seg.col_base + c) / p.group;
            const bool seen = live && pos <= last && (p.window <= 0 || pos > last - p.window);
            s[c] = seen ? s[c] * p.scale_log2 : -INFINITY;
          }
        }
        bool raise = false;
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&sm.m[c]);
          raise |= s[c] > m.x + kRaise || s[c + 1] > m.y + kRaise || s[c + 2] > m.z + kRaise || s[c + 3] > m.w + kRaise;
        }
        if (softmax_any(raise)) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const float x = warp_max(s[c]);
            if (lane == 0) sm.per_warp[w][c] = x;
          }
          softmax_sync();
          float f[N];
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const float old = sm.m[c];
            const float top = fmaxf(fmaxf(fmaxf(sm.per_warp[0][c], sm.per_warp[1][c]), fmaxf(sm.per_warp[2][c], sm.per_warp[3][c])), old);
            f[c] = top == old ? 1.0f : ex2(old - top);
            l[c] *= f[c];
          }
          softmax_sync();
          if (r < N)
            sm.m[r] = fmaxf(fmaxf(fmaxf(sm.per_warp[0][r], sm.per_warp[1][r]), fmaxf(sm.per_warp[2][r], sm.per_warp[3][r])), sm.m[r]);
          if (t > 0) {  // what has been summed so far; no MMA writes it until p_full
            ok &= waited(&sm.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, sm);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll
            for (int m = 0; m < C::MB; ++m) {
#pragma unroll
              for (int c = 0; c < N; c += 16) {
                float x[16];
                tc::ld16(tmem + lanes + 2 * N + m * N + c, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= f[c + j];
                tc::st16(tmem + lanes + 2 * N + m * N + c, x);
              }
            }
            tc::wait_st();
            tc::fence_before_sync();
          }
          softmax_sync();
        }
        // this tile's buffer of weights was last read by the products of tile i - PB
        if (i >= C::PB) {
          const uint32_t j = i - C::PB;
          ok &= waited(&sm.pv_done[j & 1u], (j >> 1) & 1u, sm);
        }
        unsigned char* const to = weights + (i % C::PB) * C::PBYTES + r * 16;
#pragma unroll
        for (int c = 0; c < N; c += 8) {
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            float4 m = *reinterpret_cast<const float4*>(&sm.m[c + j]);
            // a column that has seen nothing: 2^(-inf - 0) = 0
            m.x = m.x == -INFINITY ? 0.0f : m.x;
            m.y = m.y == -INFINITY ? 0.0f : m.y;
            m.z = m.z == -INFINITY ? 0.0f : m.z;
            m.w = m.w == -INFINITY ? 0.0f : m.w;
            const float w0 = ex2(s[c + j] - m.x), w1 = ex2(s[c + j + 1] - m.y), w2 = ex2(s[c + j + 2] - m.z),
                        w3 = ex2(s[c + j + 3] - m.w);
            l[c + j] += w0;
            l[c + j + 1] += w1;
            l[c + j + 2] += w2;
            l[c + j + 3] += w3;
            x[j / 2] = pack_bf16(w0, w1);
            x[j / 2 + 1] = pack_bf16(w2, w3);
          }
          *reinterpret_cast<uint4*>(to + (c / 8) * (kTile * 16)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
        if (begin + kTile > seg.n || begin < lower) {
          // Positions outside the request share its pages: whatever their values are (another
          // request's, or never written), a weight of zero has to meet a zero.
          constexpr int kValueChunks = C::DV / 64;
#pragma unroll
          for (int c = 0; c < kValueChunks; ++c) {
            const uint32_t n = i * C::PER + (C::LATENT ? 0 : C::KC) + c, slot = n % C::RING;
            ok &= waited(&sm.full[slot], (n / C::RING) & 1u, sm);
            if (ok && (pos >= seg.n || pos < lower)) {
              uint4* to16 = reinterpret_cast<uint4*>(ring + slot * kChunk + r * 128);
#pragma unroll
              for (int j = 0; j < 8; ++j) to16[(j + r) & 7] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        arrive(&sm.p_full[i % C::PB]);
        live = live_next;
      }

      // ---- the unit's (or the share's) end: sums over the positions, then O^T ---------------
      ok &= waited(&sm.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, sm);
      __syncwarp();
      tc::fence_after_sync();
      column_sums<N>(l, lane);
      softmax_sync();  // maxima of the last raise are read
      if (N >= 32) {
#pragma unroll
        for (int j = 0; j < N / 32; ++j) sm.per_warp[w][lane * (N / 32) + j] = l[j];
      } else if ((lane & 1) == 0) {
        sm.per_warp[w][lane / 2] = l[0];
      }
      softmax_sync();
      float* part = partial_of(p, blockIdx.x, seg.index == 0 ? 0 : 1);
      if (ok && r < cols) {
        const float sum = (sm.per_warp[0][r] + sm.per_warp[1][r]) + (sm.per_warp[2][r] + sm.per_warp[3][r]);
        if (!seg.whole) {
          part[p.ncol * C::DV + r] = sm.m[r];
          part[p.ncol * C::DV + p.ncol + r] = sum;
        } else if (p.lse != nullptr) {
          p.lse[sm.rows[r]] = lse_of(sm.m[r], sum);
        }
      }
#pragma unroll
      for (int m = 0; m < C::MB; ++m) {
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 16) {
          float x[16];
          tc::ld16(tmem + lanes + 2 * N + m * N + c0, x);
          const int d = C::DV >= 128 ? m * 128 + r : r - 64;
          if (ok && d >= 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int c = c0 + j;
              if (c >= cols) continue;
              if (seg.whole) {
                const float sum = (sm.per_warp[0][c] + sm.per_warp[1][c]) + (sm.per_warp[2][c] + sm.per_warp[3][c]);
                const float inv = sum > 0.0f ? 1.0f / sum : (sum == sum ? 0.0f : sum);
                static_cast<__nv_bfloat16*>(p.o)[sm.rows[c] * C::DV + d] = __float2bfloat16_rn(x[j] * inv);
              } else {
                part[c * C::DV + d] = x[j];
              }
            }
          }
        }
      }
      tc::fence_before_sync();  // read before the next unit's products write it (p_full)
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM);
  }
  if (tid == 0 && sm.timeout != 0u) atomic_status(p.status, GDN_STATUS_TIMEOUT);
}

template <class C>
cudaError_t launch_one(const TcParams& tp, cudaStream_t stream) {
  const cudaError_t err = cudaFuncSetAttribute(gdn_attn_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(C::SMEM));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tp.a.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdn_attn_tc_kernel<C>, tp);
}

template <int D>
cudaError_t launch_width(const TcParams& tp, cudaStream_t stream) {
  switch (tp.a.ncol) {
    case 16: return launch_one<Cfg<D, D, 16, false>>(tp, stream);
    case 32: return launch_one<Cfg<D, D, 32, false>>(tp, stream);
    default: return launch_one<Cfg<D, D, 64, false>>(tp, stream);
  }
}

// Pages as a 4-D tensor (element, head, position, page); boxes of 64 elements of one head,
// `box` positions of one page.
cudaError_t encode_pages(CUtensorMap* map, const AttnParams& p, const void* base, int d, int64_t head, int64_t pos,
                         int64_t page, int box) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.heads_kv),
                              static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.num_pages)};
  // a dimension of one element has no stride to speak of
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.heads_kv > 1 ? head : d) * 2u,
                                 static_cast<cuuint64_t>(pos) * 2u,
                                 static_cast<cuuint64_t>(p.num_pages > 1 ? page : d) * 2u};
  const cuuint32_t boxes[4] = {64u, 1u, static_cast<cuuint32_t>(box), 1u};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_attn_tc(AttnParams& p, cudaStream_t stream) {
  TcParams tp{};
  tp.a = p;
  tp.box = p.page_size < kTile ? p.page_size : kTile;
  cudaError_t err = encode_pages(&tp.k, p, p.k, p.dk, p.k_head, p.k_pos, p.k_page, tp.box);
  if (err == cudaSuccess) err = encode_pages(&tp.v, p, p.v, p.dv, p.v_head, p.v_pos, p.v_page, tp.box);
  if (err != cudaSuccess) return err;
  if (p.dk == 576)
    return p.ncol == 16 ? launch_one<Cfg<576, 512, 16, true>>(tp, stream) : launch_one<Cfg<576, 512, 32, true>>(tp, stream);
  if (p.dk == 64) return launch_width<64>(tp, stream);
  if (p.dk == 128) return launch_width<128>(tp, stream);
  return launch_width<256>(tp, stream);
}

}  // namespace gdn
