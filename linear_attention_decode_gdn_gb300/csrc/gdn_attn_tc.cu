// gdn_attn_tc.cu -- attention over the paged cache on the tensor cores: head sizes 64, 128 and
// 256, and latent rows of 512 + 64.
//
// Decode attention reads every cached byte once for a handful of query rows, so the matrix
// products are laid out around the cache: the tile's 128 positions are the 128 rows of a
// tcgen05 MMA, the query rows (16, 32 or 64 columns) its narrow side.
//
//   S^T [128 positions x N] = K [128 x dk] (q [N x dk])^T        A, B from shared memory
//   P^T = 2^(S^T - m), m one running reference a column          in registers, a thread a position
//   O^T [dv x N] += V^T [dv x 128] P^T [128 x N]                 A = V as it lies in memory (its
//                                                                rows run along dv), B from shared
//
// So neither K nor V is transposed or padded, and a query group of 4 or 16 costs the same as it
// streams by. The accumulators take 2 N columns of TMEM for two tiles' scores, and N for every 128
// value elements of this CTA (64 count as 128) and every softmax team.
//
// One CTA an SM. Warp 0 gathers pages by TMA into a ring of slots (128 positions x 64 or 128
// elements, 128-byte swizzle; pages of 16 .. 128 positions are boxes of a slot). Warp 1 issues
// the MMAs: scores of tile i + 1 before values of tile i (over latent rows, whichever is ready),
// so the tensor core works while the softmax does. Warps 2 and 3 lay out the next unit's queries.
// The other warps are the softmax, four for every 16 columns: one thread a position; sums of
// weights stay in the threads until the unit ends. The reference is the maximum of the tile that set it, times 2^8; it is raised
// (and O^T rescaled in TMEM) only where a score passes it, so most tiles need one barrier and no
// reduction, and no weight is above 1.
//
// Latent rows: the value is the key's own row, so a tile's 147 KB would have to stay until the
// values' product, and with them alone shared memory is full: loads, scores, softmax and values
// would take turns (128 requests x 32 heads: 300 us). A pair of CTAs (one cluster) therefore
// splits the row: each CTA holds half of the latent and of the tail, two to three tiles deep,
// forms its half of every score's sum, sends it to the other CTA's shared memory (st.async,
// counted on an mbarrier), and adds what it is sent. Both then take the same softmax (the sum of
// two is the same in either order) and each its half of O^T. No byte of the cache and no product
// is taken twice.
//
// Values that a product must not meet: the tensor core multiplies a weight of zero too, and 0 x NaN is
// NaN. Positions that no column sees are zeroed in shared memory; of those that some columns see and
// others do not (several positions a request: MULTI, a kernel of its own) NaN and infinities are
// taken out, and added at the unit's end for the columns that see them. 32 requests x 4 positions x 16
// heads on latent rows: 38.5 us, 115 where every request's newest value holds NaN.
//
// What bounds it, and what it takes (bf16 cache, one GB300):
//   full batch, 128 requests x 32 heads over 8 kv heads of 128, 2.17 GB: 315 to 327 us by the box,
//     6.6 to 6.9 TB/s: HBM. The same on 2 kv heads of 256, 1.08 GB: 169 us, 6.4 TB/s.
//   one request of 131,071 positions, same heads, 0.54 GB: 86 us, 6.2 TB/s: HBM, start and join.
//   128 requests x 32 heads on latent rows, 0.62 GB: 112 us, 5.5 TB/s: a tile's chain of load,
//     scores, exchange, softmax and values over a ring of two and a half tiles.
//   4 requests x 128 heads on latent rows, 65,535 positions: 141 us for two passes of 64 columns
//     (0.5 PFLOP/s): the same chain, 1850 cycles of it the exchange of 32 KB a tile.
//   one request, 16 heads over 2 kv heads of 256, 1021 positions: 9.1 us with the join: latency.
//   64 requests x 4 positions, 16 heads over 2 kv heads of 256, 0.28 GB: 55 us, 5.0 TB/s: 64 columns
//     leave a ring of one tile, so loads, scores and values of neighbouring tiles hardly overlap.
// The MMAs themselves take 34 to 42 cycles each at 16 to 64 columns, in every operand layout
// tried, and are not what bounds any of these.
#include "gdn_attn.cuh"
#include "gdn_tc.cuh"
#include "gdn_tmap.h"

#include <type_traits>

#include <cuda_bf16.h>

namespace gdn {

namespace {

using namespace attn;

constexpr int kChunk = kTile * 128;          // bytes: 128 positions x 64 bf16
constexpr int kSmemMost = 227 * 1024;
constexpr int kMiscBytes = 4096;
constexpr int kMaxSlots = 12;
constexpr int kAhead = 1;                    // tiles that latent rows are fetched into L2 before their load
constexpr float kHeadroom = 8.0f;            // log2 of what a score may grow by before weights are rescaled
constexpr float kNothing = -3.0e38f;         // the reference of a column that has seen nothing: finite, so
                                             // that no difference of infinities is ever taken

template <int DK_, int DV_, int N_, bool LATENT_>
struct Cfg {
  static constexpr int DK = DK_, DV = DV_, N = N_;
  static constexpr bool LATENT = LATENT_;
  static constexpr int CL = LATENT ? 2 : 1;                // CTAs that share a unit
  static constexpr int KCOLS = LATENT ? DV / CL : DK;      // key elements of this CTA, but for the tail
  static constexpr int VCOLS = DV / CL;                    // value elements of this CTA
  static constexpr int TCOLS = LATENT ? (DK - DV) / CL : 0;  // tail elements of this CTA
  static constexpr int SLOTC = VCOLS >= 128 ? 2 : 1;       // chunks of a slot
  static constexpr int SLOT = SLOTC * kChunk;
  static constexpr int KS = KCOLS / 64 / SLOTC;            // key slots of a tile
  static constexpr int VS = LATENT ? 0 : VCOLS / 64 / SLOTC;
  static constexpr int PER = KS + VS;
  static constexpr int MB = VCOLS > 128 ? VCOLS / 128 : 1; // blocks of 128 rows of O^T
  static constexpr int NC = 16, G = N / NC;                // columns of a softmax group (one load of TMEM), groups
  // Two softmax teams take turns at units, each with its own O^T: one ends a unit while the other
  // begins the next. Wider blocks have their threads in column groups, latent units are long.
  static constexpr int TEAMS = !LATENT && G == 1 ? 2 : 1;
  static constexpr int THREADS = 128 + 128 * G * TEAMS;
  static constexpr int PB = LATENT ? 1 : 2;                // buffers of weights
  static constexpr int QB = !LATENT && DK < 256 && N <= 32 ? 2 : 1;  // and of queries
  static constexpr int TAIL = kTile * TCOLS * 2;            // bytes of a tile's tail; there is one buffer
  static constexpr int QBYTES = N * (KCOLS + TCOLS) * 2, PBYTES = N * kTile * 2, RBYTES = LATENT ? N * kTile * 4 : 0;
  static constexpr int FIXED = kMiscBytes + QB * QBYTES + PB * PBYTES + RBYTES + TAIL;
  static constexpr int FIT = (kSmemMost - FIXED) / SLOT < kMaxSlots ? (kSmemMost - FIXED) / SLOT : kMaxSlots;
  static constexpr int SLOTS = SLOTC == 1 ? FIT & ~1 : FIT;
  static constexpr int SMEM = FIXED + SLOTS * SLOT;
  static constexpr int TMEM_USED = (2 + MB * TEAMS) * N;
  static constexpr int TMEM = TMEM_USED <= 32 ? 32 : TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  // the scores of a tile are taken while the values of the one before still need their slots
  static_assert(SLOTS >= KS + (LATENT ? KS : VS), "the ring holds what both products need");
  // A slot's barrier tells its fills apart by parity alone, so waiting for a fill is sound only where the
  // slot's fill before is known to have landed. With a tile's scores its keys have, and all fills before
  // them but the values of the tile before. Latent values are the keys; elsewhere every value slot's fill
  // before is among these where the ring holds a tile and its values, and where it does not (heads of 256
  // with more than 16 columns) the softmax first waits for the products of the tile before.
  static constexpr bool FILL_KNOWN = LATENT || SLOTS >= PER + VS;
  static_assert(FILL_KNOWN || TEAMS == 1, "that wait is for a tile of the same threads");
  static_assert(N % 16 == 0 && N <= 64 && SMEM <= kSmemMost && TMEM_USED <= 512, "fits");
};

struct Misc {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t tail_full, tail_empty;
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2];  // by tile
  uint64_t unit_begun[2], unit_done[2];  // by unit: its first scores, its O^T are complete
  uint64_t got[4], may_send[4];  // a group's scores received; the other CTA has read what was sent
  uint64_t drained;
  uint32_t tmem;
  uint32_t timeout;
  uint32_t cleaned[2];  // 1 + the unit of the share whose values held what is no number, by the unit's parity
  alignas(16) float m[64];  // read as vectors, like per_warp
  float inv[64];
  alignas(16) float per_warp[4][64];
  int32_t last[64];  // the last position that each column sees
  int32_t rows[64];  // the column's row of o
};
static_assert(sizeof(Misc) <= kMiscBytes, "shared memory plan");

struct TcParams {
  AttnParams a;
  int32_t box, box_shift;  // positions of one TMA box, min(page_size, 128), and its log2
  int32_t page_tiles;      // tiles of a page of 128 positions or more
  CUtensorMap k, v;        // v: the tail of a latent row
};

// ---- PTX ----------------------------------------------------------------------------------
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Operand tiles of 128-byte (64-byte) rows with the swizzle of that width; 8 rows repeat.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return tc::smem_desc(saddr, lbo, sbo) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return tc::smem_desc(saddr, lbo, sbo) | (4ull << 61);
}
// kind::f16, called by a whole warp with uniform operands; one elected lane issues.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 l;\n elect.sync l|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrival for a whole warp.
__device__ __forceinline__ void arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// The same where all of the warp's threads are `ok`; a warp that gave up arrives nowhere.
__device__ __forceinline__ void arrive_if(bool ok, uint64_t* bar, int lane) {
  if (__all_sync(0xffffffffu, ok)) arrive(bar, lane);
}
// One page's box; called by a whole warp with uniform operands, one elected lane issues.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t head, int32_t pos,
                                        int32_t page, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b32 l;\n elect.sync l|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n}\n" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(head), "r"(pos), "r"(page)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// 16 bytes to shared memory, zeros where `from_there` is false (then nothing is read)
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool from_there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(from_there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// 16 bytes to another CTA's shared memory, counted on that CTA's mbarrier
__device__ __forceinline__ void send16(uint32_t dst, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d)), "r"(bar)
               : "memory");
}
// An arrival at another CTA's mbarrier that publishes nothing: a release would wait for all that
// this thread has written.
__device__ __forceinline__ void arrive_there(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Barriers of four softmax warps.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(g + 1) : "memory"); }
__device__ __forceinline__ bool group_any(int g, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n bar.red.or.pred b, %2, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(g + 1)
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

// Sums of 16 columns over the warp's lanes: afterwards a lane holds the sum of column lane / 2.
__device__ __forceinline__ void column_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8, off = 16; half > 0; half >>= 1, off >>= 1) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float keep = upper ? v[j + half] : v[j], send = upper ? v[j] : v[j + half];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// mbar_try_wait that also sees what another CTA of the cluster has written
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0u;
}

// Whether the phase is complete, without waiting for it.
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0u;
}

// A wait with a limit. The first one that runs out raises a flag that ends every other wait of
// the CTA, so the kernel returns soon after (and reports GDN_STATUS_TIMEOUT). The other CTA of a
// pair is sent nothing more, so its own waits run out too.
template <bool CLUSTER = false>
__device__ __forceinline__ bool waited(uint64_t* bar, uint32_t parity, Misc& sm) {
  auto done = [&] { return CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return true;
  volatile uint32_t* const flag = &sm.timeout;
  const long long t0 = clock64();
  while (!done()) {
    if (*flag != 0u) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *flag = 1u;
      return false;
    }
  }
  return true;
}
// For a warp that polls several barriers: whether it has to stop.
__device__ __forceinline__ bool gave_up(long long since, Misc& sm) {
  volatile uint32_t* const flag = &sm.timeout;
  if (clock64() - since > kWaitLimitCycles) *flag = 1u;
  return __any_sync(0xffffffffu, *flag != 0u);
}
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, test_wait(bar, parity));
}
// A wait with a limit for a whole warp that goes on together.
__device__ __forceinline__ bool warp_waited(uint64_t* bar, uint32_t parity, Misc& sm) {
  return __all_sync(0xffffffffu, waited(bar, parity, sm));
}

__device__ __forceinline__ bool no_number(float x) { return !(fabsf(x) <= 3.4028235e38f); }

// 16 bytes of a value's row (bf16) with zeros for what is no number; whether there was any.
__device__ __forceinline__ bool clean16(uint4* at) {
  uint4 x = *at;
  uint32_t* const words[4] = {&x.x, &x.y, &x.z, &x.w};
  bool found = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t& u = *words[j];
    const bool lo = (u & 0x7f80u) == 0x7f80u, hi = (u & 0x7f800000u) == 0x7f800000u;
    found |= lo || hi;
    u &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0xffffu : 0xffffffffu);
  }
  if (found) *at = x;
  return found;
}

// What clean16 took out of a segment's values, for the columns that see it: w v of every value that is
// no number, for the `left` columns of a softmax group from c_base on and the elements d, d + 128, ..
// of each lane. refs and lasts: the group's references and last positions. Called by a whole warp, and
// only where something was found; looks at the positions that some columns of the unit see and others do not.
template <class C>
__device__ __noinline__ void sums_of_no_numbers(const AttnParams& p, const Segment& seg, const float* refs, const int32_t* lasts,
                                                int c_base, int left, int d, float (&sums)[C::MB][16]) {
  const int lane = threadIdx.x & 31;
  const int t_first = seg.col_base / p.group, t_last = (min(seg.col_base + C::N, p.cols) - 1) / p.group;
  const int32_t lower = lower_bound_of(p, seg.n, t_first), lower_last = lower_bound_of(p, seg.n, t_last);
  const int32_t begin = max(seg.tile * kTile, lower), end = min((seg.tile + seg.tiles) * kTile, seg.n);
  const int32_t all_see = max(seg.n - p.T + t_first, lower_last - 1);  // the last position that all columns see, if any does
  const int32_t* const row = p.table + static_cast<int64_t>(seg.b) * p.max_pages;
#pragma unroll
  for (int b = 0; b < C::MB; ++b)
#pragma unroll
    for (int c = 0; c < 16; ++c) sums[b][c] = 0.0f;
#pragma unroll 1
  for (int32_t pos = begin; pos < end; ++pos) {
    if (pos >= lower_last && pos <= all_see) {  // on to the first that is not seen by all
      pos = all_see;
      continue;
    }
    const int32_t page = row[pos / p.page_size], in = pos % p.page_size;
    if (page < 0 || page >= p.num_pages) continue;
    const uint16_t* const v = static_cast<const uint16_t*>(p.v) + page * p.v_page + in * p.v_pos + seg.kv_head * p.v_head + d;
    const uint16_t* const k = static_cast<const uint16_t*>(p.k) + page * p.k_page + in * p.k_pos + seg.kv_head * p.k_head;
    float x[C::MB];
    bool found = false;
#pragma unroll
    for (int b = 0; b < C::MB; ++b) {
      x[b] = __uint_as_float(static_cast<uint32_t>(v[b * 128]) << 16);
      found |= no_number(x[b]);
    }
    if (!__any_sync(0xffffffffu, found)) continue;
#pragma unroll 1
    for (int c = 0; c < left; ++c) {
      if (pos > lasts[c] || (p.window > 0 && pos <= lasts[c] - p.window)) continue;
      const int col = seg.col_base + c_base + c, t = col / p.group, h = seg.kv_head * p.group + (col - t * p.group);
      const uint16_t* const q = static_cast<const uint16_t*>(p.q) + seg.b * p.q_b + t * p.q_t + h * p.q_h;
      float s = 0.0f;
#pragma unroll 1
      for (int e = lane * 2; e < C::DK; e += 64) {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(k + e), b = *reinterpret_cast<const uint32_t*>(q + e);
        s = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), s);
        s = fmaf(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u), s);
      }
      const float w = ex2(warp_sum(s) * p.scale_log2 - refs[c]);
      if (w == 0.0f) continue;
#pragma unroll
      for (int b = 0; b < C::MB; ++b)
        if (no_number(x[b])) sums[b][c] = fmaf(w, x[b], sums[b][c]);
    }
  }
}

// MULTI: several positions a request, so the columns of a unit may see different positions.
template <class C, bool MULTI>
__global__ void __launch_bounds__(C::THREADS, 1) gdn_attn_tc_kernel(const __grid_constant__ TcParams tp) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const AttnParams& p = tp.a;
  constexpr int N = C::N, NC = C::NC;
  unsigned char* const ring = smem;
  unsigned char* const tail = ring + C::SLOTS * C::SLOT;
  unsigned char* const weights = tail + C::TAIL;
  unsigned char* const received = weights + C::PB * C::PBYTES;
  unsigned char* const queries = received + C::RBYTES;
  Misc& sm = *reinterpret_cast<Misc*>(queries + C::QB * C::QBYTES);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = C::CL > 1 ? cluster_rank() : 0u;
  const uint32_t worker = blockIdx.x / C::CL;

  griddep_launch_dependents();
  if (tid == 0) {
    // For tests, a barrier of the first two workers counts on an arrival that never comes (the first
    // one's share may end before its unit's first tile).
    const int32_t starve = worker < 2 && rank == 0 ? p.starve : 0;
    const bool starve_load = starve == GDN_STARVE_LOAD, starve_weights = starve == GDN_STARVE_WEIGHTS;
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&sm.full[i], i == 0 && starve_load ? 2 : 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 2);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 4 * C::G);
      mbar_init(&sm.p_full[i], 4 * C::G + (i == 0 && starve_weights ? 1 : 0));
      mbar_init(&sm.pv_done[i], 1);
      mbar_init(&sm.unit_begun[i], 1);
      mbar_init(&sm.unit_done[i], 1);
    }
    for (int i = 0; i < C::G; ++i) {
      mbar_init(&sm.got[i], 1);
      mbar_init(&sm.may_send[i], 1);
    }
    mbar_init(&sm.tail_full, 1);
    mbar_init(&sm.tail_empty, 1);
    mbar_init(&sm.drained, 1);
    sm.timeout = sm.cleaned[0] = sm.cleaned[1] = 0u;
    fence_mbar_init();
    if (C::LATENT)  // the first round of scores is expected from the start
      for (int i = 0; i < C::G; ++i) mbar_arrive_expect_tx(&sm.got[i], C::NC * kTile * 4);
  }
  if (warp == 1) {
    tc::tmem_alloc(&sm.tmem, C::TMEM);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (C::CL > 1) cluster_sync_all();  // the other CTA's barriers are there
  const uint32_t tmem = sm.tmem;
  griddep_wait();
  const Share share = find_share(p, worker);
  Walk walk(share);
  Segment seg;

  if (warp == 0) {
    // ---- pages into the ring --------------------------------------------------------------
    uint32_t slot = 0, round = 1, tile_no = 0;  // next slot, the parity its barrier has when free
    uint32_t put = 0, tails_put = 0;  // loads begun
    bool bad = false, ok = true;
    // BOXES of a chunk; lane l looks up the page of box l
    auto produce = [&](auto boxes_of_a_chunk) {
      constexpr int BOXES = decltype(boxes_of_a_chunk)::value, BOX = kTile / BOXES;
      while (ok && walk.next(p, &seg)) {
        const int32_t lower = lower_bound_of(p, seg.n, seg.col_base / p.group);
        const int32_t* row = p.table + static_cast<int64_t>(seg.b) * p.max_pages;
        // the entry is only looked at when its tile's turn comes, a tile later
        auto entry = [&](int tile) -> int32_t {
          const int32_t at = min(tile * kTile + (lane & (BOXES - 1)) * BOX, seg.n - 1);
          return row[BOXES > 1 ? at / BOX : tile / tp.page_tiles];
        };
        // a box that no query of the unit sees reads as zero, as one of a page that is none
        auto page_of = [&](int tile, int32_t page) -> int32_t {
          const int32_t at = tile * kTile + (lane & (BOXES - 1)) * BOX;
          const bool seen = at < seg.n && at + BOX > lower, valid = page >= 0 && page < p.num_pages;
          bad |= seen && !valid;
          return seen && valid ? page : p.num_pages;
        };
        const int end = seg.tile + seg.tiles;
        int32_t next = entry(seg.tile), ahead = 0;
        if (C::LATENT && seg.tile + kAhead < end) ahead = entry(seg.tile + kAhead);
        for (int tile = seg.tile; ok && tile < end; ++tile, ++tile_no) {
          int32_t page = page_of(tile, next);
          if (tile + 1 < end) next = entry(tile + 1);
          int32_t pages[BOXES];
#pragma unroll
          for (int b = 0; b < BOXES; ++b) pages[b] = __shfl_sync(0xffffffffu, page, b);
          const int32_t pos = BOXES > 1 ? 0 : tile % tp.page_tiles * kTile;
          for (int s = 0; s < C::PER; ++s) {
            ok = warp_waited(&sm.empty[slot], round, sm);
            if (!ok) break;
            const bool value = !C::LATENT && s >= C::KS;
            const CUtensorMap* map = value ? &tp.v : &tp.k;
            const int32_t x = (C::LATENT ? static_cast<int32_t>(rank) * C::KCOLS : 0) + (value ? s - C::KS : s) * (C::SLOTC * 64);
            const uint32_t dst = smem_addr(ring) + slot * C::SLOT;
            tc::expect_tx(&sm.full[slot], C::SLOT);
#pragma unroll
            for (int b = 0; b < BOXES; ++b)
#pragma unroll
              for (int c = 0; c < C::SLOTC; ++c)
                tma_box(dst + c * kChunk + b * BOX * 128, map, x + c * 64, seg.kv_head, pos, pages[b], &sm.full[slot]);
            ++put;
            if (++slot == C::SLOTS) {
              slot = 0;
              round ^= 1u;
            }
          }
          if (C::LATENT && ok) {
            ok = warp_waited(&sm.tail_empty, (tile_no & 1u) ^ 1u, sm);
            if (!ok) break;
            tc::expect_tx(&sm.tail_full, C::TAIL);
            ++tails_put;
#pragma unroll
            for (int b = 0; b < BOXES; ++b)
              tma_box(smem_addr(tail) + b * BOX * (C::TCOLS * 2), &tp.v, C::DV + static_cast<int32_t>(rank) * C::TCOLS,
                      0, pos, pages[b], &sm.tail_full);
          }
          if (C::LATENT && ok && tile + kAhead < end) {
            // The ring holds little more than two tiles, so a tile's loads begin when the one two
            // before is done with: from L2 they arrive sooner (128 requests: 135 us without this,
            // 127 with; two tiles ahead gain no more, three lose).
            const int32_t later = page_of(tile + kAhead, ahead);
            if (tile + kAhead + 1 < end) ahead = entry(tile + kAhead + 1);
#pragma unroll
            for (int j = 0; j < kTile; j += 32) {
              const int32_t in_tile = j + lane, first = (tile + kAhead) * kTile;
              const int32_t pg = __shfl_sync(0xffffffffu, later, in_tile / BOX);
              if (pg == p.num_pages || first + in_tile >= seg.n) continue;
              const int32_t in_page = BOXES > 1 ? in_tile % BOX : (tile + kAhead) % tp.page_tiles * kTile + in_tile;
              const uint16_t* from = static_cast<const uint16_t*>(p.k) + pg * p.k_page + in_page * p.k_pos + rank * C::KCOLS;
#pragma unroll
              for (int c = 0; c < C::KCOLS / 64; ++c) prefetch_l2(from + c * 64);
              prefetch_l2(from + C::DV - rank * (C::KCOLS - C::TCOLS));
            }
          }
        }
      }
    };
    switch (tp.box) {
      case 16: produce(std::integral_constant<int, 8>{}); break;
      case 32: produce(std::integral_constant<int, 4>{}); break;
      case 64: produce(std::integral_constant<int, 2>{}); break;
      default: produce(std::integral_constant<int, 1>{}); break;
    }
    // Nothing may still be on its way into this CTA's memory when it ends, whichever warp gave up.
    for (uint32_t i = put > C::SLOTS ? put - C::SLOTS : 0; i < put; ++i)
      mbar_wait(&sm.full[i % C::SLOTS], (i / C::SLOTS) & 1u);
    if (C::LATENT && tails_put > 0) mbar_wait(&sm.tail_full, (tails_put - 1) & 1u);
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomic_status(p.status, GDN_STATUS_BAD_PAGE);
  } else if (warp == 1) {
    // ---- matrix products --------------------------------------------------------------------
    constexpr uint32_t kScores = idesc_bf16(128, N, false, false), kValues = idesc_bf16(128, N, true, true);
    const uint32_t ring_at = smem_addr(ring), tail_at = smem_addr(tail), w_at = smem_addr(weights);
    uint32_t i = 0, units = 0;   // tiles and units begun
    uint32_t k_slot = 0, k_round = 0, v_slot = 0, v_round = 0;  // next slots of keys and of values
    // of the last tile with scores: whether it is its unit's first, its last, and that unit
    uint32_t first_of_last = 0, last_of_last = 0, unit_of_last = 0;
    bool ok = true;
    auto skip = [](uint32_t& slot, uint32_t& round, uint32_t n) {
      slot += n;
      if (slot >= C::SLOTS) {
        slot -= C::SLOTS;
        round ^= 1u;
      }
    };
    if (!C::LATENT) skip(v_slot, v_round, C::KS);

    auto scores = [&] {
      const uint32_t q_at = smem_addr(queries) + (C::QB > 1 ? (units & 1u) * C::QBYTES : 0);
      const uint32_t d = tmem + (i & 1u) * N;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        ok = warp_waited(&sm.full[k_slot], k_round, sm);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t a = ring_at + k_slot * C::SLOT, b = q_at + s * (C::SLOTC * 8 * N * 16);
#pragma unroll
        for (int k = 0; k < 4 * C::SLOTC; ++k)
          mma_bf16(d, desc_sw128(a + (k / 4) * kChunk + (k % 4) * 32, 16, 1024), tc::smem_desc(b + k * (2 * N * 16), N * 16, 128),
                   kScores, s > 0 || k > 0);
        if (!C::LATENT) tc::commit(&sm.empty[k_slot]);
        skip(k_slot, k_round, 1);
      }
      if (C::LATENT) {
        ok = warp_waited(&sm.tail_full, i & 1u, sm);
        if (!ok) return;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < C::TCOLS / 16; ++k)
          mma_bf16(d, desc_sw64(tail_at + k * 32, 16, 512),
                   tc::smem_desc(q_at + (C::KCOLS / 8 + 2 * k) * (N * 16), N * 16, 128), kScores, 1);
        tc::commit(&sm.tail_empty);
      }
      skip(k_slot, k_round, C::VS);
      tc::commit(&sm.s_full[i & 1u]);
    };
    // values of the last tile with scores, j
    auto values = [&](uint32_t j) {
      const uint32_t buf = j % C::PB, first = first_of_last;
      const uint32_t d = tmem + 2 * N + (unit_of_last % C::TEAMS) * (C::MB * N);
      ok = warp_waited(&sm.p_full[buf], (j / C::PB) & 1u, sm);
      if (!ok) return;
      tc::fence_after_sync();
#pragma unroll
      for (int m = 0; m < C::MB; ++m) {
        if (!C::LATENT) {
          ok = warp_waited(&sm.full[v_slot], v_round, sm);
          if (!ok) return;
          tc::fence_after_sync();
        }
        // dv = 64 is the upper half of the 128 rows; the lower half multiplies the slot before (the
        // tile's keys, or what replaces them) and is never read
        const uint32_t a = ring_at + (C::DV >= 128 ? v_slot : v_slot - 1) * C::SLOT, b = w_at + buf * C::PBYTES;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16(d + m * N, desc_sw128(a + k * 2048, kChunk, 1024), tc::smem_desc(b + k * 256, 128, kTile * 16),
                   kValues, first == 0u || k > 0);
        tc::commit(&sm.empty[v_slot]);
        skip(v_slot, v_round, 1);
      }
      if (!C::LATENT) skip(v_slot, v_round, C::KS);
      tc::commit(&sm.pv_done[j & 1u]);
      if (last_of_last != 0u) tc::commit(&sm.unit_done[unit_of_last & 1u]);
    };

    while (ok && walk.next(p, &seg)) {
      const uint32_t qb = units % C::QB;
      for (int t = 0; ok && t < seg.tiles; ++t) {
        if (t == 0) ok = warp_waited(&sm.q_full[qb], (units / C::QB) & 1u, sm);
        if (ok) ok = warp_waited(&sm.s_empty[i & 1u], ((i >> 1) & 1u) ^ 1u, sm);
        if (!ok) break;
        tc::fence_after_sync();
        // Whichever is ready first: the last tile's values (their slots are wanted) or these scores.
        bool due = i > 0;
        if (C::LATENT && due) {
          const uint32_t j = i - 1;
          const long long t0 = clock64();
          while (ok && !ready(&sm.full[k_slot], k_round)) {
            if (ready(&sm.p_full[j % C::PB], (j / C::PB) & 1u)) {
              values(j);
              due = false;
              break;
            }
            ok = !gave_up(t0, sm);
          }
          if (!ok) break;
        }
        scores();
        if (!ok) break;
        if (C::TEAMS > 1 && t == 0) tc::commit(&sm.unit_begun[units & 1u]);
        if (t == seg.tiles - 1) tc::commit(&sm.q_empty[qb]);
        if (due) values(i - 1);
        first_of_last = t == 0;
        last_of_last = t == seg.tiles - 1;
        unit_of_last = units;
        ++i;
      }
      ++units;
    }
    if (ok && i > 0) values(i - 1);
    // the last MMA has left TMEM and shared memory alone when this completes
    tc::commit(&sm.drained);
    if (!mbar_wait(&sm.drained, 0)) *static_cast<volatile uint32_t*>(&sm.timeout) = 1u;
  } else if (warp < 4) {
    // ---- queries of the next unit -----------------------------------------------------------
    // K-major core matrices: 16 bytes of column n, element group e at (e * N + n) * 16
    uint32_t units = 0;
    while (walk.next(p, &seg)) {
      const uint32_t qb = units % C::QB;
      if (!waited(&sm.q_empty[qb], ((units / C::QB) & 1u) ^ 1u, sm)) break;
      const int cols = min(N, p.cols - seg.col_base);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + seg.b * p.q_b;
      constexpr int kVecs = (C::KCOLS + C::TCOLS) / 8;
#pragma unroll 2
      for (int v = tid - 64; v < N * kVecs; v += 64) {
        const int c = v / kVecs, e = v - c * kVecs;
        const int col = seg.col_base + min(c, cols - 1), t = col / p.group, h = seg.kv_head * p.group + (col - t * p.group);
        const int at = C::LATENT ? (e < C::KCOLS / 8 ? static_cast<int>(rank) * C::KCOLS + e * 8
                                                     : C::DV + static_cast<int>(rank) * C::TCOLS + (e - C::KCOLS / 8) * 8)
                                 : e * 8;
        cp_async16_or_zero(queries + qb * C::QBYTES + (e * N + c) * 16, q + t * p.q_t + h * p.q_h + at, c < cols);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      tc::fence_smem_to_async();
      arrive(&sm.q_full[qb], lane);
      ++units;
    }
    if (tid == 64 && rank == 0) write_record(p, share, worker);
    write_empty<64>(p, tid - 64);
  } else {
    // ---- softmax ------------------------------------------------------------------------------
    const int quad = (warp - 4) / 4, g = C::TEAMS > 1 ? 0 : quad, w = warp & 3;  // its group of columns, its warp
    const uint32_t team = C::TEAMS > 1 ? quad : 0;
    const int r = w * 32 + lane;      // this thread's position of the tile and TMEM lane
    const int c_base = g * NC;        // its group's first column
    const int a_base = quad * NC;     // and its place in the arrays that are kept by column
    const uint32_t lanes = tc::lane_base(w);
    const uint32_t s_at = tmem + lanes + c_base, o_at = tmem + lanes + 2 * N + team * (C::MB * N) + c_base;
    // the group's part of what the CTAs send each other, and its barriers there
    const uint32_t mine = g * (NC * kTile * 4) + r * 16;
    const uint32_t there = C::LATENT ? in_cta(smem_addr(received), rank ^ 1u) + mine : 0u;
    const uint32_t got_there = C::LATENT ? in_cta(smem_addr(&sm.got[g]), rank ^ 1u) : 0u;
    const uint32_t may_send_there = C::LATENT ? in_cta(smem_addr(&sm.may_send[g]), rank ^ 1u) : 0u;
    uint32_t i = 0, units = 0;
    // After a wait that ran out the threads still go through the group's barriers together (no later
    // wait holds them up), but arrive at no other and write nothing more. So what is complete, here or in
    // the other CTA, was made of what all had waited for.
    bool ok = true;
    for (; walk.next(p, &seg); ++units) {
      if (C::TEAMS > 1 && (units & 1u) != team) {
        i += seg.tiles;
        continue;
      }
      const int cols = min(N, p.cols - seg.col_base);
      const int t_first = seg.col_base / p.group, t_last = (seg.col_base + cols - 1) / p.group;
      const int32_t lower = lower_bound_of(p, seg.n, t_first);
      const int32_t lower_last = lower_bound_of(p, seg.n, t_last);
      const int32_t* row = p.table + static_cast<int64_t>(seg.b) * p.max_pages;
      // the page of this thread's position; looked at a tile later
      auto entry = [&](int tile) -> int32_t {
        const int32_t at = min(tile * kTile + r, seg.n - 1);
        return row[tp.box < kTile ? at >> tp.box_shift : tile / tp.page_tiles];
      };
      int32_t next = entry(seg.tile);
      group_sync(quad);  // the last unit's rows and maxima are read
      if (r < NC) {
        const int a = a_base + r, col = seg.col_base + c_base + r;
        sm.m[a] = kNothing;
        sm.last[a] = seg.n - p.T + col / p.group;
        sm.rows[a] = static_cast<int32_t>(row_of(p, seg.b, seg.kv_head, col));
      }
      // Sums of weights, and references: in registers, but for the block of 640 threads, which has
      // 96 of them a thread and reads the references from shared memory.
      constexpr bool kKeep = C::G <= 2;
      float l[NC], kept[kKeep ? NC : 4];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        l[c] = 0.0f;
        if (kKeep) kept[c] = kNothing;
      }
      auto references = [&](int c) -> float4 {
        if (kKeep) return make_float4(kept[c], kept[c + 1], kept[c + 2], kept[c + 3]);
        return *reinterpret_cast<const float4*>(&sm.m[a_base + c]);
      };
      group_sync(quad);
      // A barrier's parity tells two rounds apart, so a team that has sat out a unit first waits for
      // its own unit's turn: the barriers of that unit's tiles are then at their rounds.
      if (C::TEAMS > 1) ok &= waited(&sm.unit_begun[units & 1u], (units >> 1) & 1u, sm);
      for (int t = 0; t < seg.tiles; ++t, ++i) {
        const int tile = seg.tile + t;
        const int32_t begin = tile * kTile, pos = begin + r;
        const bool live = pos < seg.n && pos >= lower && next >= 0 && next < p.num_pages;
        if (t + 1 < seg.tiles) next = entry(tile + 1);
        float s[NC];
        ok &= waited(&sm.s_full[i & 1u], (i >> 1) & 1u, sm);
        __syncwarp();
        tc::fence_after_sync();
        tc::ld16(s_at + (i & 1u) * N, s);
        tc::fence_before_sync();
        arrive_if(ok, &sm.s_empty[i & 1u], lane);
        if (C::LATENT) {
          // After a wait that ran out nothing is sent, expected or freed any more: the bytes that a
          // barrier counts would get ahead of the round that the other CTA is in. Its wait for them runs
          // out instead, and it stops as well.
          if (i > 0) ok &= waited(&sm.may_send[g], (i - 1) & 1u, sm);
          if (ok) {
#pragma unroll
            for (int c = 0; c < NC; c += 4) send16(there + (c / 4) * (kTile * 16), s[c], s[c + 1], s[c + 2], s[c + 3], got_there);
          }
          ok &= waited<true>(&sm.got[g], i & 1u, sm);
          if (ok && r == 0) mbar_arrive_expect_tx(&sm.got[g], NC * kTile * 4);  // the next tile's
          const unsigned char* from = received + mine;
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(from + (c / 4) * (kTile * 16));
            s[c] += x.x;
            s[c + 1] += x.y;
            s[c + 2] += x.z;
            s[c + 3] += x.w;
          }
        }
        // every column sees every position of the tile, but where it is not live
        const bool all_see = begin + kTile - 1 <= seg.n - p.T + t_first && begin >= lower_last;
        if (all_see) {
#pragma unroll
          for (int c = 0; c < NC; ++c) s[c] = live ? s[c] * p.scale_log2 : -INFINITY;
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int32_t last = sm.last[a_base + c];
            const bool seen = live && pos <= last && (p.window <= 0 || pos > last - p.window);
            s[c] = seen ? s[c] * p.scale_log2 : -INFINITY;
          }
        }
        bool raise = false;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 m = references(c);
          raise |= s[c] > m.x || s[c + 1] > m.y || s[c + 2] > m.z || s[c + 3] > m.w;
        }
        const bool any = group_any(quad, raise);
        // every thread of the group has used what it received: the other CTA may send more
        if (C::LATENT && ok && r == 0) arrive_there(may_send_there);
        if (any) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float x = warp_max(s[c]);
            if (lane == 0) sm.per_warp[w][a_base + c] = x;
          }
          group_sync(quad);
          if (t > 0) {  // O^T is complete up to the last tile, and no MMA writes it until p_full
            ok &= waited(&sm.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, sm);
            __syncwarp();
            tc::fence_after_sync();
          }
          float f[NC];
          if constexpr (kKeep) {
#pragma unroll
            for (int j = 0; j < NC; j += 4) {
              const int a = a_base + j;
              float top[4], x[4];
              auto load = [](float (&to)[4], const float* from) {
                const float4 v = *reinterpret_cast<const float4*>(from);
                to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
              };
              load(top, &sm.per_warp[0][a]);
#pragma unroll
              for (int v = 1; v < 4; ++v) {
                load(x, &sm.per_warp[v][a]);
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], x[k]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float to = top[k] > kept[j + k] ? top[k] + kHeadroom : kept[j + k];
                f[j + k] = ex2(kept[j + k] - to);
                l[j + k] *= f[j + k];
                kept[j + k] = to;
                if (r == j + k) sm.m[a + k] = to;
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
              const int a = a_base + j;
              const float top = fmaxf(fmaxf(sm.per_warp[0][a], sm.per_warp[1][a]), fmaxf(sm.per_warp[2][a], sm.per_warp[3][a]));
              const float m = sm.m[a];
              const float to = top > m ? top + kHeadroom : m;
              f[j] = ex2(m - to);
              l[j] *= f[j];
            }
          }
          if (t > 0) {
#pragma unroll 1
            for (int block = 0; block < C::MB; ++block) {
              float x[NC];
              tc::ld16(o_at + block * N, x);
#pragma unroll
              for (int j = 0; j < NC; ++j) x[j] *= f[j];
              tc::st16(o_at + block * N, x);
            }
          }
          if (t > 0) {
            tc::wait_st();
            tc::fence_before_sync();
          }
          if (!kKeep) {
            group_sync(quad);  // the old references are read
            if (r < NC) {
              const int a = a_base + r;
              const float top = fmaxf(fmaxf(sm.per_warp[0][a], sm.per_warp[1][a]), fmaxf(sm.per_warp[2][a], sm.per_warp[3][a]));
              if (top > sm.m[a]) sm.m[a] = top + kHeadroom;
            }
            group_sync(quad);
          }
        }
        // this tile's buffer of weights was last read by the products of tile i - PB
        if (i >= C::PB) {
          const uint32_t j = i - C::PB;
          ok &= waited(&sm.pv_done[j & 1u], (j >> 1) & 1u, sm);
        }
        // Weights are rounded to bf16 for the product with the values (2^-8 of a weight at most, as the
        // values and the output are bf16 themselves); their sums l, and so lse, take them in fp32.
        unsigned char* const to = weights + (i % C::PB) * C::PBYTES + (c_base / 8) * (kTile * 16) + r * 16;
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 m = references(c + j);
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
        if (begin + kTile > seg.n || begin < lower || (MULTI && !all_see)) {
          // Positions outside the request share its pages: whatever their values are (another
          // request's, or never written), a weight of zero has to meet a zero.
          constexpr int kSlots = C::LATENT ? C::KS : C::VS;
          const uint32_t fill = i * C::PER + (C::LATENT ? 0 : C::KS);
          if (!C::FILL_KNOWN && i > 0) ok &= waited(&sm.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, sm);
#pragma unroll 1
          for (int v = 0; v < kSlots; ++v) {
            const uint32_t slot = (fill + v) % C::SLOTS;
            ok &= waited(&sm.full[slot], ((fill + v) / C::SLOTS) & 1u, sm);
            if (pos >= seg.n || pos < lower) {
#pragma unroll
              for (int c = 0; c < C::SLOTC; ++c) {
                uint4* to16 = reinterpret_cast<uint4*>(ring + slot * C::SLOT + c * kChunk + r * 128);
#pragma unroll
                for (int j = 0; j < 8; ++j) to16[(j + r) & 7] = make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
          if (MULTI && !all_see) {
            // Of the values that only some columns see (a window's oldest, the request's newest: rows
            // old0 .. old1 - 1 and new0 .. new1 - 1) what is no number is taken out, a vector a thread,
            // and comes back at the unit's end for those that see it.
            constexpr int kVecs = C::VCOLS / 8;
            const int old0 = max(lower - begin, 0), old1 = min(min(lower_last, seg.n) - begin, kTile);
            const int new0 = max(max(seg.n - p.T + t_first + 1, lower_last) - begin, 0), new1 = min(seg.n - begin, kTile);
            const int olds = max(old1 - old0, 0), items = (olds + max(new1 - new0, 0)) * kVecs;
            bool found = false;
            for (int item = g * 128 + r; item < items; item += 128 * C::G) {
              const int at = item / kVecs, e = item - at * kVecs, to = at < olds ? old0 + at : new0 + at - olds;
              const uint32_t slot = (fill + e / (8 * C::SLOTC)) % C::SLOTS;
              found |= clean16(reinterpret_cast<uint4*>(ring + slot * C::SLOT + (e / 8) % C::SLOTC * kChunk + to * 128) + (e & 7));
            }
            if (found) *const_cast<volatile uint32_t*>(&sm.cleaned[units & 1u]) = units + 1;
          }
        }
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        arrive_if(ok, &sm.p_full[i % C::PB], lane);
      }

      // ---- the unit's (or the share's) end: sums over the positions, then O^T ---------------
      column_sums(l, lane);
      group_sync(quad);  // maxima of the last raise are read
      if ((lane & 1) == 0) sm.per_warp[w][a_base + lane / 2] = l[0];
      group_sync(quad);
      // Whoever of the group gave up raised the flag before its sum was exchanged above.
      ok &= *const_cast<volatile uint32_t*>(&sm.timeout) == 0u;
      float* const part = partial_of(p, worker, seg.index == 0 ? 0 : 1);
      if (r < NC) {
        const int a = a_base + r, c = c_base + r;
        const float sum = (sm.per_warp[0][a] + sm.per_warp[1][a]) + (sm.per_warp[2][a] + sm.per_warp[3][a]);
        sm.inv[a] = !seg.whole ? 1.0f : sum > 0.0f ? 1.0f / sum : (sum == sum ? 0.0f : sum);
        if (ok && c < cols && rank == 0) {
          if (!seg.whole) {
            part[N * C::DV + c] = sm.m[a];
            part[N * C::DV + N + c] = sum;
          } else if (p.lse != nullptr) {
            p.lse[sm.rows[a]] = lse_of(sm.m[a], sum);
          }
        }
      }
      group_sync(quad);
      ok &= waited(&sm.unit_done[units & 1u], (units >> 1) & 1u, sm);
      __syncwarp();
      tc::fence_after_sync();
      const int left = cols - c_base;  // columns that are rows of o
      float added[C::MB][NC];
      const bool cleaned = MULTI && *const_cast<volatile uint32_t*>(&sm.cleaned[units & 1u]) == units + 1;
      if (cleaned && (C::DV >= 128 || r >= 64)) {
        const Segment here = seg;  // a copy: what a call takes by address has no registers
        sums_of_no_numbers<C>(p, here, sm.m + a_base, sm.last + a_base, c_base, min(left, NC),
                              static_cast<int>(rank) * C::VCOLS + (C::DV >= 128 ? r : r - 64), added);
      }
#pragma unroll 1
      for (int block = 0; block < C::MB; ++block) {
        const int d = static_cast<int>(rank) * C::VCOLS + (C::DV >= 128 ? block * 128 + r : r - 64);
        float x[NC];
        tc::ld16(o_at + block * N, x);
        if (cleaned && d >= 0) {
#pragma unroll
          for (int j = 0; j < NC; ++j) x[j] += added[block][j];
        }
        if (ok && d >= 0 && seg.whole) {
          __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(p.o) + d;
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const int a = a_base + j;
            if (j < left) o[static_cast<int64_t>(sm.rows[a]) * C::DV] = __float2bfloat16_rn(x[j] * sm.inv[a]);
          }
        } else if (ok && d >= 0) {
          float* const to = part + c_base * C::DV + d;
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (j < left) to[j * C::DV] = x[j];
        }
        __syncwarp();
      }
      tc::fence_before_sync();  // read before the next unit's products write it (p_full)
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (C::CL > 1) {
    // What a CTA that gave up had sent may still be on its way, and only the receiver counts it: it
    // is given some 50 us, where it takes one.
    if (sm.timeout != 0u) {
      const long long t0 = clock64();
      while (clock64() - t0 < 100000) {
      }
    }
    cluster_sync_all();  // nothing more comes from, or goes to, the other CTA
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM);
  }
  if (sm.timeout != 0u) {
    // what this worker leaves to be joined is not all there: the join writes no row of it
    for (int c = tid; c < 2 * N; c += C::THREADS) partial_of(p, worker, c / N)[N * C::DV + c % N] = lost_reference();
    if (tid == 0) atomic_status(p.status, GDN_STATUS_TIMEOUT);
  }
}

template <class C, bool MULTI>
cudaError_t launch_form(const TcParams& tp, cudaStream_t stream) {
  static std::atomic<bool> allowed[kDevices];
  const cudaError_t err = allow_shared(reinterpret_cast<const void*>(gdn_attn_tc_kernel<C, MULTI>), C::SMEM, allowed);
  if (err != cudaSuccess) return err;
  return launch_overlapped(gdn_attn_tc_kernel<C, MULTI>, tp, dim3(tp.a.workers * C::CL), C::THREADS, C::SMEM, C::CL, stream);
}

template <class C>
cudaError_t launch_one(const TcParams& tp, cudaStream_t stream) {
  return tp.a.T > 1 ? launch_form<C, true>(tp, stream) : launch_form<C, false>(tp, stream);
}

template <int DK, int DV, bool LATENT>
cudaError_t launch_width(const TcParams& tp, cudaStream_t stream) {
  switch (tp.a.ncol) {
    case 16: return launch_one<Cfg<DK, DV, 16, LATENT>>(tp, stream);
    case 32: return launch_one<Cfg<DK, DV, 32, LATENT>>(tp, stream);
    default: return launch_one<Cfg<DK, DV, 64, LATENT>>(tp, stream);
  }
}

// Pages as a 4-D tensor (element, head, position, page); boxes of `width` elements of one head,
// `box` positions of one page.
cudaError_t encode_pages(CUtensorMap* map, const AttnParams& p, const void* base, int d, int64_t head, int64_t pos,
                         int64_t page, int box, int width) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.heads_kv),
                              static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.num_pages)};
  // a dimension of one element has no stride to speak of
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.heads_kv > 1 ? head : d) * 2u,
                                 static_cast<cuuint64_t>(pos) * 2u,
                                 static_cast<cuuint64_t>(p.num_pages > 1 ? page : d) * 2u};
  const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(width), 1u, static_cast<cuuint32_t>(box), 1u};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes,
                      width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace

cudaError_t launch_attn_tc(AttnParams& p, cudaStream_t stream) {
  const bool latent = p.dk == 576;
  TcParams tp{};
  tp.a = p;
  tp.box = p.page_size < kTile ? p.page_size : kTile;
  tp.box_shift = tp.box == 16 ? 4 : tp.box == 32 ? 5 : tp.box == 64 ? 6 : 7;
  tp.page_tiles = p.page_size < kTile ? 1 : p.page_size / kTile;
  cudaError_t err = encode_pages(&tp.k, p, p.k, p.dk, p.k_head, p.k_pos, p.k_page, tp.box, 64);
  if (err == cudaSuccess)
    err = latent ? encode_pages(&tp.v, p, p.k, p.dk, p.k_head, p.k_pos, p.k_page, tp.box, 32)
                 : encode_pages(&tp.v, p, p.v, p.dv, p.v_head, p.v_pos, p.v_page, tp.box, 64);
  if (err != cudaSuccess) return err;
  if (latent) return launch_width<576, 512, true>(tp, stream);
  if (p.dk == 64) return launch_width<64, 64, false>(tp, stream);
  if (p.dk == 128) return launch_width<128, 128, false>(tp, stream);
  return launch_width<256, 256, false>(tp, stream);
}

}  // namespace gdn
