// gdn_attn.cuh -- what the attention kernels share: how the work is cut, and the places of
// the partial results.
//
// The work of a launch is a list of tiles, each kTile = 128 cache positions of one unit; a
// unit is one (request, kv head, column group), and its columns are the query rows that read
// the same keys: column c is query token c / group, head c % group of the kv head. The tiles
// of all units stand in one line, request by request, and every CTA takes an equal, unbroken
// share of the line, computed from kv_len on the device. So the CTAs are busy equally long
// whatever the lengths are, one long request is spread over all of them, and a unit is cut
// only where two shares meet: of a CTA's segments only the first and the last can be part of
// a unit. Those leave unnormalised sums in the workspace, and gdn_attn_join_kernel adds them.
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

// Tiles of the line before the CTA's share begins.
__device__ __forceinline__ int64_t share_start(int64_t total, int ctas, int cta) {
  const int64_t q = total / ctas, r = total - q * ctas;
  return cta * q + (cta < r ? cta : r);
}

// Where a CTA's share begins: the request, the unit of it (kv head * col_groups + column
// group) and the tile in the unit.
struct Share {
  int64_t total, start, count;
  int64_t unit_start;  // line position of the first unit's first tile
  int32_t b, unit, tile;
};

// Called by all THREADS of the block; `scratch` is for this call alone (three barriers).
struct ShareScratch {
  int64_t warp_sums[32];
  Share share;
};

template <int THREADS>
__device__ __forceinline__ int64_t scan_tiles(int64_t x, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = static_cast<int64_t>(__shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(x), d));
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t s = warp_sums[w];
    before += w < warp ? s : 0;
    all += s;
  }
  *total = all;
  return x + before;
}

template <int THREADS>
__device__ __forceinline__ Share find_share(const AttnParams& p, ShareScratch& scratch) {
  const int tid = threadIdx.x;
  const int units = p.heads_kv * p.col_groups;
  // a batch of up to THREADS requests: one load a thread and one sum
  const int32_t mine = tid < p.B ? tiles_of(p, length_of(p, tid)).count : 0;
  int64_t all;
  int64_t upto = scan_tiles<THREADS>(mine, scratch.warp_sums, &all);
  int64_t total = all;
  for (int base = THREADS; base < p.B; base += THREADS) {
    const int b = base + tid;
    scan_tiles<THREADS>(b < p.B ? tiles_of(p, length_of(p, b)).count : 0, scratch.warp_sums, &all);
    total += all;
  }
  Share s{};
  s.total = total * units;
  s.start = share_start(s.total, gridDim.x, blockIdx.x);
  s.count = share_start(s.total, gridDim.x, blockIdx.x + 1) - s.start;
  int64_t before = 0;
  for (int base = 0; base < p.B; base += THREADS) {
    const int b = base + tid;
    int32_t count = mine;
    if (base > 0) {
      count = b < p.B ? tiles_of(p, length_of(p, b)).count : 0;
      upto = scan_tiles<THREADS>(count, scratch.warp_sums, &all);
    } else if (p.B > THREADS) {
      upto = scan_tiles<THREADS>(count, scratch.warp_sums, &all);
    }
    const int64_t lo = (before + upto - count) * units, hi = (before + upto) * units;
    if (count > 0 && s.count > 0 && s.start >= lo && s.start < hi) {
      Share f = s;
      const int64_t in = s.start - lo;
      f.b = b;
      f.unit = static_cast<int32_t>(in / count);
      f.tile = static_cast<int32_t>(in - static_cast<int64_t>(f.unit) * count);
      f.unit_start = s.start - f.tile;
      scratch.share = f;
    }
    before += all;
  }
  if (s.count == 0) return s;
  __syncthreads();
  return scratch.share;
}

// A CTA's run of tiles within one unit.
struct Segment {
  int32_t b, unit, kv_head, col_base;
  int32_t n;          // cached positions
  int32_t tile, tiles; // first tile (absolute) and how many
  int32_t index;      // 0 for the CTA's first
  bool whole;         // covers the unit
};

// Walks the segments of a share; every thread that walks sees the same ones.
struct Walk {
  int64_t left;
  int32_t b, unit, tile, index;

  __device__ __forceinline__ explicit Walk(const Share& s)
      : left(s.count), b(s.b), unit(s.unit), tile(s.tile), index(0) {}

  __device__ __forceinline__ bool next(const AttnParams& p, Segment* seg) {
    if (left <= 0) return false;
    const int units = p.heads_kv * p.col_groups;
    int32_t n = length_of(p, b);
    Tiles t = tiles_of(p, n);
    if (unit >= units) {
      unit = 0;
      do {  // a later request has tiles, because tiles are left
        ++b;
        n = length_of(p, b);
        t = tiles_of(p, n);
      } while (t.count == 0);
    }
    const int64_t rest = t.count - tile;
    const int32_t take = static_cast<int32_t>(left < rest ? left : rest);
    seg->b = b;
    seg->unit = unit;
    seg->kv_head = unit / p.col_groups;
    seg->col_base = (unit - seg->kv_head * p.col_groups) * p.ncol;
    seg->n = n;
    seg->tile = t.first + tile;
    seg->tiles = take;
    seg->index = index++;
    seg->whole = take == t.count;
    left -= take;
    tile = 0;
    ++unit;
    return true;
  }
};

// ---- the workspace ----------------------------------------------------------------------
// Record of a CTA: [start, share's end or -1 without work, unit_start, unit's end, b, unit] of
// its first segment's unit. A partial result: dv x ncol sums (column by column, fp32), then the
// columns' maxima (in the scaled log2 domain) and sums.
__device__ __forceinline__ size_t partial_floats(const AttnParams& p) {
  return static_cast<size_t>(p.ncol) * (p.dv + 2);
}
__device__ __forceinline__ float* partial_of(const AttnParams& p, int cta, int slot) {
  return p.partials + (static_cast<size_t>(cta) * 2 + slot) * partial_floats(p);
}

__device__ __forceinline__ void write_record(const AttnParams& p, const Share& s) {
  int64_t* r = p.records + static_cast<size_t>(blockIdx.x) * kRecordInts;
  r[0] = s.start;
  r[1] = s.count > 0 ? s.start + s.count : -1;
  if (s.count <= 0) return;
  r[2] = s.unit_start;
  r[3] = s.unit_start + tiles_of(p, length_of(p, s.b)).count;
  r[4] = s.b;
  r[5] = s.unit;
}

// Row of column c of a request and kv head: [B][T][H].
__device__ __forceinline__ int64_t row_of(const AttnParams& p, int b, int kv_head, int c) {
  const int t = c / p.group;
  return (static_cast<int64_t>(b) * p.T + t) * p.H + kv_head * p.group + (c - t * p.group);
}

// Requests with nothing in the cache belong to no share: their rows are written here, and
// lengths that cannot be are reported. Every thread of the block calls it.
template <int THREADS>
__device__ __forceinline__ void write_empty(const AttnParams& p) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int32_t raw = p.kv_len[b];
    if (raw > 0 && length_of(p, b) < 0 && threadIdx.x == 0) atomic_status(p.status, GDN_STATUS_BAD_LEN);
    if (raw != 0) continue;
    const int64_t rows = static_cast<int64_t>(p.T) * p.H, at = b * rows;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + at * p.dv);
    for (int64_t i = threadIdx.x; i < rows * (p.dv / 8); i += THREADS) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int64_t i = threadIdx.x; i < rows; i += THREADS) p.lse[at + i] = __int_as_float(0xff800000);
  }
}

constexpr float kLn2 = 0.69314718055994530942f;

// m: the column's maximum of scaled scores (log2 domain), l: its sum of 2^(s - m)
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.0f ? m * kLn2 + logf(l) : (l == l ? __int_as_float(0xff800000) : l);
}

}  // namespace attn
}  // namespace gdn
