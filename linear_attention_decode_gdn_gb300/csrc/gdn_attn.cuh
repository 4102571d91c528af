// gdn_attn.cuh -- what the attention kernels share: how the work is cut, and the places of
// the partial results.
//
// The work of a launch is a list of tiles, each kTile = 128 cache positions of one unit; a
// unit is one (request, kv head, column group), and its columns are the query rows that read
// the same keys: column c is query token c / group, head c % group of the kv head. The tiles
// of all units stand in one line, request by request, and every worker (a CTA, or a pair of
// them) takes an equal, unbroken share of the line, computed from kv_len on the device. So all
// are busy equally long whatever the lengths are, one long request is spread over the GPU, and
// a unit is cut only where two shares meet: of a worker's segments only the first and the last
// can be part of a unit. A unit also counts for p.unit_cost tiles that stand before its first
// one (its queries, first maximum and result take that long), so that a share of many short
// units is not the one that the others wait for; where workers have fewer than two tiles each,
// an even cut matters more and it counts for none. The cut units' workers leave unnormalised
// sums in the workspace, and gdn_attn_join_kernel adds them.
#pragma once

#include "gdn_device.cuh"
#include "gdn_kv.h"

namespace gdn {
namespace attn {

struct Tiles {
  int32_t first;  // first tile of the request that any of its queries sees
  int32_t count;  // 0: nothing to read
};

// Cached positions of request b; -1 where the request is to be skipped.
__device__ __forceinline__ int32_t length_of(const AttnParams& p, int b) {
  const int32_t n = p.kv_len[b];
  return n < 0 || n > static_cast<int64_t>(p.max_pages) * p.page_size ? -1 : n;
}

// First position that query t of a request of n positions sees.
__device__ __forceinline__ int32_t lower_bound_of(const AttnParams& p, int32_t n, int t) {
  if (p.window <= 0) return 0;
  const int32_t pos = n - p.T + t;
  return pos >= p.window ? pos - p.window + 1 : 0;
}

__device__ __forceinline__ Tiles tiles_of(const AttnParams& p, int32_t n) {
  if (n <= 0) return {0, 0};
  const int32_t first = lower_bound_of(p, n, 0) / kTile;
  return {first, (n - 1) / kTile + 1 - first};
}

// Line position where worker w's share begins (a worker: a CTA, or a pair of them).
__device__ __forceinline__ uint32_t share_start(uint32_t total, uint32_t workers, uint32_t w) {
  const uint32_t q = total / workers, r = total - q * workers;
  return w * q + min(w, r);
}
// The first worker whose share begins at or after line position `at`.
__device__ __forceinline__ uint32_t worker_from(uint32_t total, uint32_t workers, uint32_t at) {
  const uint32_t q = total / workers, r = total - q * workers, wide = r * (q + 1);
  if (at <= wide) return (at + q) / (q + 1);
  return r + (at - wide + q - 1) / q;  // at > wide: q > 0
}

// Where a worker's share begins: the request, the unit of it (kv head * col_groups + column
// group) and the position in the unit. The host keeps the line below 2^31.
struct Share {
  uint32_t total, count;
  uint32_t unit_start;  // line position of the first unit
  int32_t extra;        // what a unit counts for beyond its tiles
  int32_t b, unit, at;
};

// Called by all lanes of a warp; every warp finds the same share for itself, which costs one
// pass over the lengths and no barrier. A lane sums consecutive requests.
__device__ __forceinline__ Share find_share(const AttnParams& p, uint32_t worker) {
  const int lane = threadIdx.x & 31;
  const uint32_t units = static_cast<uint32_t>(p.heads_kv * p.col_groups);
  const int per = (p.B + 31) / 32, from = min(lane * per, p.B), to = min(from + per, p.B);
  uint32_t tiles = 0, requests = 0;
#pragma unroll 4
  for (int b = from; b < to; ++b) {
    const uint32_t count = static_cast<uint32_t>(tiles_of(p, length_of(p, b)).count);
    tiles += count;
    requests += count > 0 ? 1u : 0u;
  }
  Share s{};
  const uint32_t all_tiles = __reduce_add_sync(0xffffffffu, tiles) * units;
  // from two tiles a worker on: 8 latent requests of 192 query rows take 25.4 us (28.8 where it
  // starts at four); from one on, a single request on 2 kv heads takes 2% more
  s.extra = all_tiles >= 2u * p.workers ? p.unit_cost : 0;
  const uint32_t mine = tiles + requests * s.extra;
  uint32_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  s.total = __shfl_sync(0xffffffffu, upto, 31) * units;
  const uint32_t start = share_start(s.total, p.workers, worker);
  s.count = share_start(s.total, p.workers, worker + 1) - start;
  if (s.count == 0) return s;
  const bool here = start >= (upto - mine) * units && start < upto * units;
  uint32_t before = upto - mine;
  int32_t b = from;
  if (here) {
    for (;; ++b) {
      const uint32_t count = static_cast<uint32_t>(tiles_of(p, length_of(p, b)).count);
      if (count == 0) continue;
      const uint32_t cost = count + s.extra;
      if (start < (before + cost) * units) {
        const uint32_t in = start - before * units;
        s.unit = static_cast<int32_t>(in / cost);
        s.at = static_cast<int32_t>(in - s.unit * cost);
        break;
      }
      before += cost;
    }
  }
  const int owner = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  s.b = __shfl_sync(0xffffffffu, b, owner);
  s.unit = __shfl_sync(0xffffffffu, s.unit, owner);
  s.at = __shfl_sync(0xffffffffu, s.at, owner);
  s.unit_start = start - s.at;
  return s;
}

// A worker's run of tiles within one unit.
struct Segment {
  int32_t b, unit, kv_head, col_base;
  int32_t n;           // cached positions
  int32_t tile, tiles; // first tile (absolute) and how many, at least one
  int32_t index;       // 0 for the worker's first
  bool whole;          // covers the unit
};

// Walks the segments of a share; every thread that walks sees the same ones.
struct Walk {
  uint32_t left;
  int32_t extra, b, unit, at, index;

  __device__ __forceinline__ explicit Walk(const Share& s)
      : left(s.count), extra(s.extra), b(s.b), unit(s.unit), at(s.at), index(0) {}

  __device__ __forceinline__ bool next(const AttnParams& p, Segment* seg) {
    const int units = p.heads_kv * p.col_groups;
    while (left > 0) {
      int32_t n = length_of(p, b);
      Tiles t = tiles_of(p, n);
      if (unit >= units) {
        unit = 0;
        do {  // a later request has tiles, because some are left
          ++b;
          n = length_of(p, b);
          t = tiles_of(p, n);
        } while (t.count == 0);
      }
      const uint32_t rest = static_cast<uint32_t>(t.count + extra - at);
      const int32_t take = static_cast<int32_t>(left < rest ? left : rest);
      const int32_t first = max(at - extra, 0), end = max(at + take - extra, 0);
      seg->b = b;
      seg->unit = unit;
      seg->n = n;
      seg->tile = t.first + first;
      seg->tiles = end - first;
      seg->whole = end - first == t.count;
      left -= take;
      at = 0;
      ++unit;
      if (end == first) continue;  // the share ends before the unit's first tile
      seg->kv_head = seg->unit / p.col_groups;
      seg->col_base = (seg->unit - seg->kv_head * p.col_groups) * p.ncol;
      seg->index = index++;
      return true;
    }
    return false;
  }
};

// ---- the workspace ----------------------------------------------------------------------
// Record of a worker: what is to be joined at the border where its share begins: [parts, or 0 where
// that is not the first border inside a unit; the slot of the first part (the worker before's);
// request; unit]. A partial result: dv x ncol sums (column by column, fp32), then the columns'
// references (in the scaled log2 domain: sums are of 2^(s - m)) and sums.
__device__ __forceinline__ size_t partial_floats(const AttnParams& p) {
  return static_cast<size_t>(p.ncol) * (p.dv + 2);
}
__device__ __forceinline__ float* partial_of(const AttnParams& p, int worker, int slot) {
  return p.partials + (static_cast<size_t>(worker) * 2 + slot) * partial_floats(p);
}

// In place of the references of a worker that gave up; no column's reference is ever a NaN.
__device__ __forceinline__ float lost_reference() { return __int_as_float(0x7fffffff); }

__device__ __forceinline__ void write_record(const AttnParams& p, const Share& s, uint32_t worker) {
  uint4 r = make_uint4(0u, 0u, static_cast<uint32_t>(s.b), static_cast<uint32_t>(s.unit));
  if (s.count > 0 && worker > 0) {
    const uint32_t start = s.unit_start + s.at, before = share_start(s.total, p.workers, worker - 1);
    const uint32_t first_tile = s.unit_start + s.extra;
    const uint32_t end = first_tile + tiles_of(p, length_of(p, s.b)).count;
    if (start > first_tile && before <= first_tile) {
      r.x = worker_from(s.total, p.workers, end) - (worker - 1);  // workers worker - 1, worker, ...
      // the unit is that worker's last segment: its first one only where its share begins with it
      r.y = before >= s.unit_start ? 0u : 1u;
    }
  }
  *reinterpret_cast<uint4*>(p.records + static_cast<size_t>(worker) * kRecordInts) = r;
}

// Row of column c of a request and kv head: [B][T][H].
__device__ __forceinline__ int64_t row_of(const AttnParams& p, int b, int kv_head, int c) {
  const int t = c / p.group;
  return (static_cast<int64_t>(b) * p.T + t) * p.H + kv_head * p.group + (c - t * p.group);
}

// Requests with nothing in the cache belong to no share: their rows are written here, and
// lengths that cannot be are reported. Called by THREADS threads of the block, numbered `tid`.
template <int THREADS>
__device__ __forceinline__ void write_empty(const AttnParams& p, int tid) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int32_t raw = p.kv_len[b];
    if (raw > 0 && length_of(p, b) < 0 && tid == 0) atomic_status(p.status, GDN_STATUS_BAD_LEN);
    if (raw != 0) continue;
    const int64_t rows = static_cast<int64_t>(p.T) * p.H, at = b * rows;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + at * p.dv);
    for (int64_t i = tid; i < rows * (p.dv / 8); i += THREADS) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int64_t i = tid; i < rows; i += THREADS) p.lse[at + i] = __int_as_float(0xff800000);
  }
}

constexpr float kLn2 = 0.69314718055994530942f;

// m: the column's reference in the scaled log2 domain, l: its sum of 2^(s - m)
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.0f ? m * kLn2 + logf(l) : (l == l ? __int_as_float(0xff800000) : l);
}

}  // namespace attn
}  // namespace gdn
