// gdn_api.cpp -- the extern "C" entry points declared in include/gdn.h:
// argument validation, kernel selection and error reporting. No allocation.
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include <cuda_runtime_api.h>

#include "gdn.h"
#include "gdn_internal.h"
#include "gdn_kv.h"
#include "gdn_ssm.h"

namespace {

thread_local char g_last_error[512] = "";

constexpr uint32_t kKnownFlags = GDN_QKV_BF16 | GDN_FUSE_CONV | GDN_NO_QK_L2NORM | GDN_GATE_RAW |
                                 GDN_PLAIN_UPDATE | GDN_KLOG_FP32 | GDN_KLOG_PRENORM | GDN_ULOG_BF16 |
                                 GDN_GATE_KDA | GDN_OUT_NORM_GATE | GDN_SPLIT_DV |
                                 GDN_TEST_STARVE_WAIT;
constexpr int kMaxLogCapacity = 63;

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return code;
}

constexpr int kMaxVerifyTokens = 16;  // positions per request in one verify call

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0u; }

// What a call needs of dk and dv: the decode steps run every shape with a kernel
// (gdn::decode_shape_built: square heads of 16..128, dk = 128 / dv = 64, dk = 64 / dv = 128,
// and square heads of 64 or 128 split along dv); the host-side log sizes and the slot reset
// accept the same shapes; the input stage, verify and prefill square heads only.
enum class Shapes { kDecode, kSquare };

int check_dims(const gdn_dims* d, bool log_call, Shapes shapes = Shapes::kSquare) {
  if (d == nullptr) return fail(GDN_ERR_INVALID_ARG, "dims is NULL");
  if (d->batch < 0 || d->num_heads <= 0 || d->dk <= 0 || d->dv <= 0 || d->num_slots <= 0)
    return fail(GDN_ERR_INVALID_ARG, "batch must be >= 0 and num_heads, dk, dv, num_slots > 0");
  if (d->decay_per_key != 0 && d->decay_per_key != 1)
    return fail(GDN_ERR_INVALID_ARG, "decay_per_key must be 0 or 1");
  if ((d->flags & ~kKnownFlags) != 0u) return fail(GDN_ERR_INVALID_ARG, "unknown flag bits");
  const int ns = (d->flags & GDN_SPLIT_DV) ? 2 : 1;
  if (shapes == Shapes::kDecode) {
    if (!gdn::decode_shape_built(d->dk, d->dv, ns))
      return fail(GDN_ERR_UNSUPPORTED,
                  "decode shape dk=%d dv=%d%s not built (dk == dv in {16,32,64,128}, dk=128/dv=64, "
                  "dk=64/dv=128; GDN_SPLIT_DV: dk == dv in {64,128})",
                  d->dk, d->dv, ns > 1 ? " split along dv" : "");
    if (ns > 1 && (d->flags & (GDN_GATE_KDA | GDN_OUT_NORM_GATE)))
      return fail(GDN_ERR_UNSUPPORTED, "GDN_SPLIT_DV is built without the KDA gate and output epilogue");
  } else {
    if (d->dk != d->dv || (d->dk != 16 && d->dk != 32 && d->dk != 64 && d->dk != 128))
      return fail(GDN_ERR_UNSUPPORTED, "head size dk=%d dv=%d not built for this call (dk == dv in {16,32,64,128})",
                  d->dk, d->dv);
    if (ns > 1) return fail(GDN_ERR_UNSUPPORTED, "GDN_SPLIT_DV applies to the decode steps only");
  }
  if (static_cast<long long>(d->batch) * d->num_heads > 0x3fffffffLL)
    return fail(GDN_ERR_INVALID_ARG, "batch * num_heads too large");
  if (log_call) {
    if (d->log_capacity < 0) return fail(GDN_ERR_INVALID_ARG, "log_capacity < 0");
    if (d->log_capacity > kMaxLogCapacity)
      return fail(GDN_ERR_UNSUPPORTED, "log_capacity %d > %d", d->log_capacity, kMaxLogCapacity);
  }
  if ((d->flags & GDN_KLOG_PRENORM) &&
      ((d->flags & GDN_FUSE_CONV) || (d->flags & GDN_NO_QK_L2NORM)))
    return fail(GDN_ERR_UNSUPPORTED, "GDN_KLOG_PRENORM needs L2 normalisation and no fused conv");
  if ((d->flags & GDN_GATE_KDA) && (d->flags & GDN_GATE_RAW))
    return fail(GDN_ERR_INVALID_ARG, "GDN_GATE_KDA and GDN_GATE_RAW exclude each other");
  return GDN_OK;
}

int check_gate_inputs(const gdn_dims* d, const gdn_inputs* in) {
  if ((d->flags & GDN_GATE_KDA) && (in->a_log == nullptr || in->dt_bias == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "GDN_GATE_KDA needs a_log and dt_bias");
  if ((d->flags & GDN_OUT_NORM_GATE) && in->out_gate == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "GDN_OUT_NORM_GATE needs out_gate");
  return GDN_OK;
}

int check_inputs(const gdn_dims* d, const gdn_inputs* in) {
  if (in == nullptr) return fail(GDN_ERR_INVALID_ARG, "inputs is NULL");
  if (int rc = check_gate_inputs(d, in)) return rc;
  if (in->slot == nullptr || in->log_decay == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "slot and log_decay are required");
  if (d->flags & GDN_FUSE_CONV) {
    if (in->mixed_qkv == nullptr || in->conv_w == nullptr || in->conv_pool == nullptr)
      return fail(GDN_ERR_INVALID_ARG, "GDN_FUSE_CONV needs mixed_qkv, conv_w and conv_pool");
    if (!aligned16(in->mixed_qkv) || !aligned16(in->conv_w))
      return fail(GDN_ERR_UNSUPPORTED, "mixed_qkv and conv_w must be 16-byte aligned");
  } else {
    if (in->q == nullptr || in->k == nullptr || in->v == nullptr)
      return fail(GDN_ERR_INVALID_ARG, "q, k and v are required");
    if (!aligned16(in->q) || !aligned16(in->k) || !aligned16(in->v))
      return fail(GDN_ERR_UNSUPPORTED, "q, k and v must be 16-byte aligned");
  }
  return GDN_OK;
}

int check_log(const gdn_dims* d, const gdn_log* log) {
  if (log == nullptr) return fail(GDN_ERR_INVALID_ARG, "log is NULL");
  if (log->len == nullptr || log->ell == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "log->len and log->ell are required");
  if (d->log_capacity > 0) {
    if (log->k_log == nullptr || log->u_log == nullptr || log->lam_log == nullptr)
      return fail(GDN_ERR_INVALID_ARG, "k_log, u_log and lam_log are required when log_capacity > 0");
    if (!aligned16(log->k_log) || !aligned16(log->u_log))
      return fail(GDN_ERR_UNSUPPORTED, "k_log and u_log must be 16-byte aligned");
  }
  return GDN_OK;
}

gdn::DecodeParams make_params(const gdn_dims* d, const gdn_inputs* in) {
  gdn::DecodeParams p{};
  p.B = d->batch;
  p.H = d->num_heads;
  p.D = d->dk;
  p.DV = d->dv;
  p.num_slots = d->num_slots;
  p.C = d->log_capacity;
  p.dlam = d->decay_per_key ? d->dk : 1;
  p.channels = 2 * d->num_heads * d->dk + d->num_heads * d->dv;
  p.flags = d->flags;
  p.q_scale = d->q_scale;
  p.l2_eps = d->l2_eps;
  p.q = in->q;
  p.k = in->k;
  p.v = in->v;
  p.mixed = in->mixed_qkv;
  p.conv_w = in->conv_w;
  p.conv_b = in->conv_b;
  p.conv_pool = in->conv_pool;
  p.lam = in->log_decay;
  p.beta = in->beta;
  p.slot = in->slot;
  p.a_log = in->a_log;
  p.dt_bias = in->dt_bias;
  p.out_gate = in->out_gate;
  p.out_norm_w = in->out_norm_w;
  p.lower_bound = d->gate_lower_bound;
  p.out_eps = d->out_eps;
  return p;
}

int launched(cudaError_t err, const char* what) {
  if (err != cudaSuccess)
    return fail(GDN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(err), cudaGetErrorName(err));
  g_last_error[0] = '\0';
  return GDN_OK;
}

int decode_common(int mode, const gdn_dims* dims, const gdn_inputs* in, float* pool,
                  const gdn_log* log, float* o, int32_t* status, void* stream, const char* name) {
  const bool log_call = mode != gdn::MODE_DENSE;
  int rc = check_dims(dims, log_call, Shapes::kDecode);
  if (rc != GDN_OK) return rc;
  if (dims->batch == 0) return GDN_OK;
  if ((rc = check_inputs(dims, in)) != GDN_OK) return rc;
  if (pool == nullptr || o == nullptr) return fail(GDN_ERR_INVALID_ARG, "state/base pool and o are required");
  if (!aligned16(pool) || !aligned16(o))
    return fail(GDN_ERR_UNSUPPORTED, "state/base pool and o must be 16-byte aligned");
  if (log_call && (rc = check_log(dims, log)) != GDN_OK) return rc;
  if (mode == gdn::MODE_APPEND && dims->log_capacity < 1)
    return fail(GDN_ERR_INVALID_ARG, "append needs log_capacity >= 1");
  // the split path addresses the pool's rows with 32-bit tensor-copy coordinates
  if ((dims->flags & GDN_SPLIT_DV) &&
      static_cast<long long>(dims->num_slots) * dims->num_heads * dims->dk > 0x7fffffffLL)
    return fail(GDN_ERR_UNSUPPORTED, "GDN_SPLIT_DV: num_slots * num_heads * dk must stay below 2^31");
  if (gdn::decode_smem_bytes(mode, dims->dk, dims->dv, (dims->flags & GDN_SPLIT_DV) ? 2 : 1,
                             log_call ? dims->log_capacity : 0,
                             dims->decay_per_key ? dims->dk : 1,
                             (dims->flags & GDN_KLOG_FP32) ? 4 : 2,
                             (dims->flags & GDN_ULOG_BF16) ? 2 : 4) == 0)
    return fail(GDN_ERR_UNSUPPORTED, "log_capacity %d does not fit in shared memory for this shape",
                dims->log_capacity);
  gdn::DecodeParams p = make_params(dims, in);
  p.state = pool;
  p.o = o;
  p.status = status;
  if (log_call) {
    p.k_log = log->k_log;
    p.u_log = log->u_log;
    p.lam_log = log->lam_log;
    p.ell = log->ell;
    p.len = log->len;
  }
  return launched(gdn::launch_decode(mode, p, static_cast<cudaStream_t>(stream)), name);
}

// ---- the paged cache ---------------------------------------------------------------------
constexpr int kMaxCacheDk = 576, kMaxCacheDv = 512;
constexpr int kMaxAttnCols = 4096;  // query rows per kv head in one call

// Strides of dimensions with `extents`; a dimension of one element may have any.
template <int N>
bool strides_ok(const int64_t* s, const int32_t (&extents)[N], int multiple) {
  for (int i = 0; i < N; ++i)
    if (extents[i] > 1 && (s[i] < 0 || s[i] % multiple != 0)) return false;
  return true;
}

int check_kv(const gdn_paged_kv* kv) {
  if (kv == nullptr) return fail(GDN_ERR_INVALID_ARG, "kv is NULL");
  if (kv->num_pages <= 0 || kv->page_size <= 0 || kv->num_kv_heads <= 0 || kv->dk <= 0 || kv->dv <= 0)
    return fail(GDN_ERR_INVALID_ARG, "num_pages, page_size, num_kv_heads, dk and dv must be > 0");
  if (kv->k == nullptr) return fail(GDN_ERR_INVALID_ARG, "kv->k is required");
  if (kv->dk > kMaxCacheDk || kv->dv > kMaxCacheDv || kv->dk % 8 != 0 || kv->dv % 8 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "cache rows dk=%d dv=%d not built (multiples of 8, dk <= %d, dv <= %d)", kv->dk,
                kv->dv, kMaxCacheDk, kMaxCacheDv);
  if (kv->v == nullptr && (kv->num_kv_heads != 1 || kv->dv > kv->dk))
    return fail(GDN_ERR_INVALID_ARG, "a latent cache (v NULL) has one head and dv <= dk");
  const int32_t extents[3] = {kv->num_pages, kv->page_size, kv->num_kv_heads};
  if (!aligned16(kv->k) || !aligned16(kv->v) || !strides_ok(kv->k_strides, extents, 8) ||
      (kv->v != nullptr && !strides_ok(kv->v_strides, extents, 8)))
    return fail(GDN_ERR_UNSUPPORTED, "cache pages must be 16-byte aligned, with strides >= 0 that are multiples of 8");
  return GDN_OK;
}

int check_attn(const gdn_paged_kv* kv, const gdn_attn* a, const void* workspace) {
  if (int rc = check_kv(kv)) return rc;
  if (a == nullptr) return fail(GDN_ERR_INVALID_ARG, "attn is NULL");
  if (a->batch < 0 || a->num_tokens <= 0 || a->num_heads <= 0 || a->max_pages <= 0 || a->window < 0)
    return fail(GDN_ERR_INVALID_ARG, "batch and window must be >= 0, num_tokens, num_heads and max_pages > 0");
  if (a->num_heads % kv->num_kv_heads != 0)
    return fail(GDN_ERR_INVALID_ARG, "num_heads %d is not a multiple of num_kv_heads %d", a->num_heads, kv->num_kv_heads);
  if (static_cast<long long>(a->num_tokens) * (a->num_heads / kv->num_kv_heads) > kMaxAttnCols)
    return fail(GDN_ERR_UNSUPPORTED, "num_tokens * num_heads / num_kv_heads must be at most %d", kMaxAttnCols);
  if (static_cast<long long>(a->batch) * a->num_tokens * a->num_heads > 0x7fffffffLL ||
      static_cast<long long>(a->max_pages) * kv->page_size > 0x7fffff00LL)  // a tile past the last fits 32 bits
    return fail(GDN_ERR_INVALID_ARG, "batch * num_tokens * num_heads or max_pages * page_size too large");
  if (a->batch == 0) return GDN_OK;
  if (a->q == nullptr || a->block_table == nullptr || a->kv_len == nullptr || a->o == nullptr || workspace == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "q, block_table, kv_len, o and workspace are required");
  const int32_t extents[3] = {a->batch, a->num_tokens, a->num_heads};
  if (!aligned16(a->q) || !aligned16(a->o) || !aligned16(workspace) || !strides_ok(a->q_strides, extents, 8))
    return fail(GDN_ERR_UNSUPPORTED, "q, o and workspace must be 16-byte aligned, q strides >= 0 and multiples of 8");
  return GDN_OK;
}

int attend(const gdn_paged_kv* kv, const gdn_attn* a, void* workspace, size_t workspace_bytes, int32_t* status,
           void* stream, bool latent, const char* name, int32_t starve = 0) {
  if (int rc = check_attn(kv, a, workspace)) return rc;
  if ((kv->v == nullptr) != latent)
    return fail(GDN_ERR_INVALID_ARG, latent ? "gdn_latent_decode reads a latent cache (kv->v NULL)"
                                            : "gdn_attn_decode needs kv->v (gdn_latent_decode reads latent caches)");
  if (a->batch == 0) return GDN_OK;
  const int group = a->num_heads / kv->num_kv_heads;
  const gdn::AttnPlan plan = gdn::attn_plan(*kv, a->num_tokens * group);
  const size_t need = gdn::attn_workspace_bytes(plan, kv->dv);
  if (workspace_bytes < need)
    return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes, %zu are needed (gdn_attn_workspace)", workspace_bytes, need);
  const int64_t col_groups = (a->num_tokens * group + plan.ncol - 1) / plan.ncol;
  const int64_t tiles = (static_cast<int64_t>(a->max_pages) * kv->page_size + gdn::kTile - 1) / gdn::kTile;
  if ((tiles + plan.unit_cost) * a->batch > 0x7fffffffLL / (kv->num_kv_heads * col_groups))
    return fail(GDN_ERR_UNSUPPORTED, "the table could hold 2^31 tiles of %d positions or more", gdn::kTile);
  if (starve != 0 && !plan.tensor) return fail(GDN_ERR_UNSUPPORTED, "this shape's kernel has no waits");
  gdn::AttnParams p{};
  p.starve = starve;
  p.B = a->batch;
  p.T = a->num_tokens;
  p.H = a->num_heads;
  p.heads_kv = kv->num_kv_heads;
  p.group = group;
  p.dk = kv->dk;
  p.dv = kv->dv;
  p.num_pages = kv->num_pages;
  p.page_size = kv->page_size;
  p.max_pages = a->max_pages;
  p.window = a->window;
  p.cols = a->num_tokens * group;
  p.scale_log2 = a->scale * 1.44269504088896340736f;
  p.q = a->q;
  p.q_b = a->q_strides[0];
  p.q_t = a->q_strides[1];
  p.q_h = a->q_strides[2];
  const int64_t* vs = latent ? kv->k_strides : kv->v_strides;
  p.k = kv->k;
  p.v = latent ? kv->k : kv->v;
  p.k_page = kv->k_strides[0];
  p.k_pos = kv->k_strides[1];
  p.k_head = kv->k_strides[2];
  p.v_page = vs[0];
  p.v_pos = vs[1];
  p.v_head = vs[2];
  p.table = a->block_table;
  p.kv_len = a->kv_len;
  p.o = a->o;
  p.lse = a->lse;
  p.status = status;
  p.records = static_cast<uint32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + gdn::kRecordBytes);
  return launched(gdn::launch_attn(plan, p, static_cast<cudaStream_t>(stream)), name);
}

// ---- selective state space layers ----------------------------------------------------------
constexpr long long kMaxPositions = 1LL << 30;  // of a call: a tile past the last fits 32 bits
constexpr int kMaxChannels = 1 << 24;
constexpr long long kMaxStates = 1LL << 36;     // of a call's requests

// Rows of a [B][T][..] operand: 16-byte aligned, with strides that keep its rows so.
template <int N>
bool rows_ok(const void* p, const int64_t* strides, const int32_t (&extents)[N], bool bf16) {
  return aligned16(p) && strides_ok(strides, extents, bf16 ? 8 : 4);
}

// Memory of one tensor of a call: rows of `row` bytes, `extents` of them at `strides` bytes, the widest first.
struct Memory {
  const char* name;
  uintptr_t at, end;
  size_t row;
  bool dense = true;  // row after row
  int dims = 0;
  size_t strides[3], extents[3];
};
Memory whole(const char* name, const void* p, size_t bytes) {
  Memory m;
  m.name = name, m.row = bytes;
  m.at = reinterpret_cast<uintptr_t>(p), m.end = p == nullptr ? m.at : m.at + bytes;
  return m;
}
// Rows of `width` elements of `size` bytes, extents and strides as the call gives them.
template <int N>
Memory rows_of(const char* name, const void* p, size_t size, size_t width, const int64_t* strides, const int32_t (&extents)[N]) {
  Memory m = whole(name, p, size * width);
  if (p == nullptr) return m;
  size_t dense = width;
  for (int i = N - 1; i >= 0; --i) {
    const size_t stride = strides[i] * size, extent = extents[i];
    if (extent == 1) continue;
    m.dense = m.dense && static_cast<size_t>(strides[i]) == dense;
    dense *= extent;
    m.end += (extent - 1) * stride;
    int k = m.dims++;
    for (; k > 0 && m.strides[k - 1] < stride; --k) m.strides[k] = m.strides[k - 1], m.extents[k] = m.extents[k - 1];
    m.strides[k] = stride, m.extents[k] = extent;
  }
  return m;
}
// Whether a row of m meets [lo, hi), of the part of m that begins at `at` and has the dimensions from `dim` on.
// Of a dimension's parts those that reach into [lo, hi) are gone into. The first that lies in it whole
// ends the search, so that two at most, at its ends, are gone into for nothing.
bool meets(const Memory& m, uintptr_t lo, uintptr_t hi, int dim, uintptr_t at) {
  if (dim == m.dims) return at < hi && at + m.row > lo;
  size_t inner = m.row;  // bytes that one of the dimension's parts spans
  for (int i = dim + 1; i < m.dims; ++i) inner += (m.extents[i] - 1) * m.strides[i];
  const size_t step = m.strides[dim], last = step == 0 ? 0 : m.extents[dim] - 1;
  for (size_t i = step > 0 && lo >= at + inner ? (lo - at - inner) / step + 1 : 0; i <= last && at + i * step < hi; ++i)
    if (meets(m, lo, hi, dim + 1, at + i * step)) return true;
  return false;
}
bool meets(const Memory& m, uintptr_t lo, uintptr_t hi) {
  return m.at < hi && m.end > lo && m.at < m.end && lo < hi && meets(m, lo, hi, 0, m.at);
}

// A tensor that lies in one piece, against others of its call. Of those with `in_place` it may be the very
// same: the kernel reads an element only where, and before, it writes there.
struct Other {
  const Memory& m;
  bool in_place = false;
};
int check_apart(const Memory& out, std::initializer_list<Other> others) {
  for (const Other& x : others) {
    if (!meets(x.m, out.at, out.end)) continue;
    if (x.in_place && x.m.dense && x.m.at == out.at && x.m.end == out.end) continue;
    return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", out.name, x.m.name);
  }
  return GDN_OK;
}

int check_ssm_sizes(int32_t batch, int32_t num_tokens, int32_t channels, int32_t state_size) {
  if (batch < 0 || num_tokens < 0 || channels <= 0)
    return fail(GDN_ERR_INVALID_ARG, "batch and num_tokens must be >= 0, channels > 0");
  if (state_size != 8 && state_size != 16 && state_size != 32 && state_size != 64)
    return fail(GDN_ERR_UNSUPPORTED, "state_size %d not built (8, 16, 32, 64)", state_size);
  if (channels > kMaxChannels || static_cast<long long>(batch) * num_tokens > kMaxPositions ||
      static_cast<long long>(batch) * channels > kMaxStates / state_size)
    return fail(GDN_ERR_UNSUPPORTED, "channels must be at most 2^24, batch * num_tokens 2^30, batch * channels * state_size 2^36");
  return GDN_OK;
}

int check_ssm(const gdn_ssm* s) {
  if (s == nullptr) return fail(GDN_ERR_INVALID_ARG, "ssm is NULL");
  if (int rc = check_ssm_sizes(s->batch, s->num_tokens, s->channels, s->state_size)) return rc;
  if (s->num_groups <= 0 || s->num_slots <= 0) return fail(GDN_ERR_INVALID_ARG, "num_groups and num_slots must be > 0");
  if ((s->flags & ~(GDN_QKV_BF16 | GDN_DT_SOFTPLUS)) != 0u)
    return fail(GDN_ERR_INVALID_ARG, "a gdn_ssm knows GDN_QKV_BF16 and GDN_DT_SOFTPLUS only");
  if (s->num_groups > s->channels / 8 || s->channels % (8 * s->num_groups) != 0)
    return fail(GDN_ERR_UNSUPPORTED, "channels %d: not a multiple of 8 in each of %d groups", s->channels, s->num_groups);
  if (s->batch == 0 || s->num_tokens == 0) return GDN_OK;
  if (s->u == nullptr || s->dt == nullptr || s->b == nullptr || s->c == nullptr || s->a == nullptr || s->state == nullptr ||
      s->slot == nullptr || s->y == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "u, dt, a, b, c, state, slot and y are required");
  const bool bf16 = (s->flags & GDN_QKV_BF16) != 0u;
  const int32_t two[2] = {s->batch, s->num_tokens}, three[3] = {s->batch, s->num_tokens, s->num_groups};
  if (!rows_ok(s->u, s->u_strides, two, bf16) || !rows_ok(s->dt, s->dt_strides, two, bf16) ||
      !rows_ok(s->b, s->b_strides, three, bf16) || !rows_ok(s->c, s->c_strides, three, bf16) ||
      (s->z != nullptr && !rows_ok(s->z, s->z_strides, two, bf16)))
    return fail(GDN_ERR_UNSUPPORTED,
                "u, dt, b, c and z must be 16-byte aligned, with strides >= 0 that are multiples of 16 bytes");
  if (!aligned16(s->a) || !aligned16(s->skip) || !aligned16(s->dt_bias) || !aligned16(s->state) || !aligned16(s->y))
    return fail(GDN_ERR_UNSUPPORTED, "a, skip, dt_bias, state and y must be 16-byte aligned");
  return GDN_OK;
}

// Last of all: what a call writes shares no memory with what it reads.
int check_norm_apart(const gdn_norm& n) {
  const int32_t extents[1] = {n.rows};
  const size_t rows = n.rows, width = n.width, wide = n.group != 0 ? n.group : width;
  auto size = [](int type) -> size_t { return type == GDN_TYPE_FP32 ? 4 : type == GDN_TYPE_BF16 ? 2 : 1; };
  const Memory o = whole("o", n.o, rows * width * size(n.o_type)), weight = whole("weight", n.weight, width * 4);
  const Memory scales = whole("scales", n.o_type == GDN_TYPE_E4M3 ? n.scales : nullptr, rows * ((width + wide - 1) / wide) * 4);
  const Memory x = rows_of("x", n.x, size(n.x_type), width, &n.x_stride, extents);
  const Memory residual = rows_of("residual", n.residual, size(n.residual_type), width, &n.residual_stride, extents);
  if (int rc = check_apart(o, {{x, n.x_type == n.o_type}, {residual}, {weight}, {scales}})) return rc;
  if (int rc = check_apart(scales, {{x}, {residual}, {weight}})) return rc;
  if (int rc = check_apart(weight, {{residual}})) return rc;
  // x may be the residual itself. Rows of both at one distance meet in the first of either or nowhere; at
  // two distances each of x is looked at, which ends soon, as such rows meet soon.
  if (n.residual == nullptr || (x.at == residual.at && x.row == residual.row && (n.rows == 1 || n.x_stride == n.residual_stride)))
    return GDN_OK;
  bool met = meets(residual, x.at, x.at + x.row) || meets(x, residual.at, residual.at + residual.row);
  if (!met && x.dims > 0 && x.strides[0] != residual.strides[0] && meets(x, residual.at, residual.end))
    for (size_t i = 1; i < rows && !met; ++i) met = meets(residual, x.at + i * x.strides[0], x.at + i * x.strides[0] + x.row);
  return met ? fail(GDN_ERR_INVALID_ARG, "residual overlaps x") : GDN_OK;
}

int check_conv_apart(const gdn_conv& c) {
  const int32_t extents[2] = {c.batch, c.num_tokens};
  const size_t size = (c.flags & GDN_QKV_BF16) != 0u ? 2 : 4, D = c.channels, B = c.batch;
  const Memory x = rows_of("x", c.x, size, D, c.x_strides, extents), w = whole("w", c.w, D * 16);
  const Memory bias = whole("bias", c.bias, D * 4);
  const Memory slot = whole("slot", c.slot, B * 4), lens = whole("seq_lens", c.seq_lens, B * 4);
  const Memory pool = whole("pool", c.pool, c.num_slots * D * 3 * size), o = whole("o", c.o, B * c.num_tokens * D * size);
  if (int rc = check_apart(o, {{x}, {w}, {bias}, {pool}, {slot}, {lens}})) return rc;
  return check_apart(pool, {{x}, {w}, {bias}, {slot}, {lens}});
}

int check_ssm_apart(const gdn_ssm& s, const void* workspace, size_t workspace_bytes) {
  const int32_t two[2] = {s.batch, s.num_tokens}, three[3] = {s.batch, s.num_tokens, s.num_groups};
  const size_t size = (s.flags & GDN_QKV_BF16) != 0u ? 2 : 4, D = s.channels, N = s.state_size, B = s.batch;
  const Memory u = rows_of("u", s.u, size, D, s.u_strides, two), dt = rows_of("dt", s.dt, size, D, s.dt_strides, two);
  const Memory z = rows_of("z", s.z, size, D, s.z_strides, two), b = rows_of("b", s.b, size, N, s.b_strides, three);
  const Memory c = rows_of("c", s.c, size, N, s.c_strides, three), a = whole("a", s.a, D * N * 4), skip = whole("skip", s.skip, D * 4);
  const Memory bias = whole("dt_bias", s.dt_bias, D * 4), slot = whole("slot", s.slot, B * 4), lens = whole("seq_lens", s.seq_lens, B * 4);
  const Memory state = whole("state", s.state, s.num_slots * D * N * 4), y = whole("y", s.y, B * s.num_tokens * D * size);
  const Memory scratch = whole("workspace", workspace, workspace_bytes);
  if (int rc = check_apart(y, {{u, true}, {dt, true}, {z, true}, {b}, {c}, {a}, {skip}, {bias}, {slot}, {lens}, {state}})) return rc;
  if (int rc = check_apart(state, {{u}, {dt}, {z}, {b}, {c}, {a}, {skip}, {bias}, {slot}, {lens}})) return rc;
  return check_apart(scratch, {{u}, {dt}, {z}, {b}, {c}, {a}, {skip}, {bias}, {slot}, {lens}, {state}, {y}});
}

}  // namespace

extern "C" {

int gdn_version(void) { return GDN_API_VERSION; }

const char* gdn_strerror(int code) {
  switch (code) {
    case GDN_OK: return "ok";
    case GDN_ERR_INVALID_ARG: return "invalid argument";
    case GDN_ERR_UNSUPPORTED: return "unsupported shape, flag combination or alignment";
    case GDN_ERR_CUDA: return "CUDA launch failure";
    default: return "unknown error code";
  }
}

const char* gdn_last_error(void) { return g_last_error; }

int gdn_conv_l2norm(const gdn_dims* dims, const gdn_inputs* in, float* q_out, float* k_out,
                    float* v_out, int32_t* status, void* stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (!(dims->flags & GDN_FUSE_CONV))
    return fail(GDN_ERR_INVALID_ARG, "gdn_conv_l2norm needs GDN_FUSE_CONV in dims->flags");
  if (dims->batch == 0) return GDN_OK;
  if ((rc = check_inputs(dims, in)) != GDN_OK) return rc;
  if (q_out == nullptr || k_out == nullptr || v_out == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "q_out, k_out and v_out are required");
  gdn::DecodeParams p = make_params(dims, in);
  p.q_out = q_out;
  p.k_out = k_out;
  p.v_out = v_out;
  p.status = status;
  return launched(gdn::launch_conv_l2norm(p, static_cast<cudaStream_t>(stream)), "gdn_conv_l2norm");
}

int gdn_decode_dense(const gdn_dims* dims, const gdn_inputs* in, float* state_pool, float* o,
                     int32_t* status, void* stream) {
  return decode_common(gdn::MODE_DENSE, dims, in, state_pool, nullptr, o, status, stream,
                       "gdn_decode_dense");
}

int gdn_decode_append(const gdn_dims* dims, const gdn_inputs* in, const float* base_pool,
                      const gdn_log* log, float* o, int32_t* status, void* stream) {
  // The append kernel only reads the base.
  return decode_common(gdn::MODE_APPEND, dims, in, const_cast<float*>(base_pool), log, o, status,
                       stream, "gdn_decode_append");
}

int gdn_decode_merge(const gdn_dims* dims, const gdn_inputs* in, float* base_pool,
                     const gdn_log* log, float* o, int32_t* status, void* stream) {
  return decode_common(gdn::MODE_MERGE, dims, in, base_pool, log, o, status, stream,
                       "gdn_decode_merge");
}

int gdn_decode_step(const gdn_dims* dims, const gdn_inputs* in, float* base_pool,
                    const gdn_log* log, float* o, int32_t* status, void* stream) {
  return decode_common(gdn::MODE_STEP, dims, in, base_pool, log, o, status, stream,
                       "gdn_decode_step");
}

int gdn_decode_verify(const gdn_dims* dims, int32_t num_tokens, const gdn_inputs* in,
                      const int32_t* state_indices, const int32_t* num_accepted, float* state_pool,
                      float* o, int32_t* status, void* stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (num_tokens < 1 || num_tokens > kMaxVerifyTokens)
    return fail(GDN_ERR_UNSUPPORTED, "num_tokens %d outside [1, %d]", num_tokens, kMaxVerifyTokens);
  if (dims->flags & (GDN_KLOG_FP32 | GDN_KLOG_PRENORM | GDN_ULOG_BF16 | GDN_TEST_STARVE_WAIT))
    return fail(GDN_ERR_UNSUPPORTED, "verify runs the dense recurrence: no log flags");
  if (static_cast<long long>(dims->batch) * num_tokens * dims->num_heads > 0x7fffffffLL)
    return fail(GDN_ERR_INVALID_ARG, "batch * num_tokens * num_heads too large");
  if (dims->batch == 0) return GDN_OK;
  if (in == nullptr || in->log_decay == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "inputs and log_decay are required");
  if ((rc = check_gate_inputs(dims, in)) != GDN_OK) return rc;
  if (dims->flags & GDN_FUSE_CONV) {
    if (in->mixed_qkv == nullptr || in->conv_w == nullptr || in->conv_pool == nullptr)
      return fail(GDN_ERR_INVALID_ARG, "GDN_FUSE_CONV needs mixed_qkv, conv_w and conv_pool");
    if (!aligned16(in->mixed_qkv) || !aligned16(in->conv_w))
      return fail(GDN_ERR_UNSUPPORTED, "mixed_qkv and conv_w must be 16-byte aligned");
  } else {
    if (in->q == nullptr || in->k == nullptr || in->v == nullptr)
      return fail(GDN_ERR_INVALID_ARG, "q, k and v are required");
    if (!aligned16(in->q) || !aligned16(in->k) || !aligned16(in->v))
      return fail(GDN_ERR_UNSUPPORTED, "q, k and v must be 16-byte aligned");
  }
  if (state_indices == nullptr || num_accepted == nullptr || state_pool == nullptr || o == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "state_indices, num_accepted, state_pool and o are required");
  if (!aligned16(state_pool) || !aligned16(o))
    return fail(GDN_ERR_UNSUPPORTED, "state_pool and o must be 16-byte aligned");
  gdn::DecodeParams p = make_params(dims, in);
  p.T = num_tokens;
  p.state_indices = state_indices;
  p.num_accepted = num_accepted;
  p.state = state_pool;
  p.o = o;
  p.status = status;
  return launched(gdn::launch_verify(p, static_cast<cudaStream_t>(stream)), "gdn_decode_verify");
}

int gdn_prefill(const gdn_dims* dims, int32_t num_tokens, const gdn_inputs* in, const int32_t* seq_lens,
                float* state_pool, float* o, int32_t* status, void* stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (num_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "num_tokens < 0");
  if (dims->flags & (GDN_KLOG_FP32 | GDN_KLOG_PRENORM | GDN_ULOG_BF16 | GDN_TEST_STARVE_WAIT))
    return fail(GDN_ERR_UNSUPPORTED, "prefill: no DeltaLog flags");
  if (static_cast<long long>(dims->batch) * num_tokens * dims->num_heads > 0x7fffffffLL)
    return fail(GDN_ERR_INVALID_ARG, "batch * num_tokens * num_heads too large");
  if (dims->batch == 0 || num_tokens == 0) return GDN_OK;
  if ((rc = check_inputs(dims, in)) != GDN_OK) return rc;
  if (state_pool == nullptr || o == nullptr) return fail(GDN_ERR_INVALID_ARG, "state_pool and o are required");
  if (!aligned16(state_pool)) return fail(GDN_ERR_UNSUPPORTED, "state_pool must be 16-byte aligned");
  gdn::DecodeParams p = make_params(dims, in);
  p.T = num_tokens;
  p.seq_lens = seq_lens;
  p.state = state_pool;
  p.o = o;
  p.status = status;
  return launched(gdn::launch_prefill(p, static_cast<cudaStream_t>(stream)), "gdn_prefill");
}

int gdn_log_bytes(const gdn_dims* dims, gdn_log_sizes* out) {
  int rc = check_dims(dims, true, Shapes::kDecode);
  if (rc != GDN_OK) return rc;
  if (out == nullptr) return fail(GDN_ERR_INVALID_ARG, "out is NULL");
  const size_t sh = static_cast<size_t>(dims->num_slots) * dims->num_heads;
  const size_t C = static_cast<size_t>(dims->log_capacity);
  const size_t dlam = dims->decay_per_key ? static_cast<size_t>(dims->dk) : 1u;
  const size_t kb = (dims->flags & GDN_KLOG_FP32) ? 4u : 2u;
  out->k_log = sh * C * dims->dk * kb;
  out->u_log = sh * C * dims->dv * ((dims->flags & GDN_ULOG_BF16) ? 2u : 4u);
  out->lam_log = sh * C * dlam * 4u;
  out->ell = sh * dlam * 4u;
  out->len = sh * 4u;
  out->residency = out->k_log + out->u_log + out->lam_log + out->ell;
  out->total = out->residency + out->len;
  return GDN_OK;
}

int gdn_slot_reset(const gdn_dims* dims, const gdn_log* log, void* conv_pool, float* state_pool,
                   const int32_t* slots, int32_t n, int32_t* status, void* stream) {
  int rc = check_dims(dims, false, Shapes::kDecode);
  if (rc != GDN_OK) return rc;
  if (n < 0) return fail(GDN_ERR_INVALID_ARG, "n < 0");
  if (n == 0) return GDN_OK;
  if (slots == nullptr) return fail(GDN_ERR_INVALID_ARG, "slots is NULL");
  if (state_pool != nullptr && !aligned16(state_pool))
    return fail(GDN_ERR_UNSUPPORTED, "state_pool must be 16-byte aligned");
  gdn::ResetParams p{};
  p.H = dims->num_heads;
  p.D = dims->dk;
  p.DV = dims->dv;
  p.num_slots = dims->num_slots;
  p.dlam = dims->decay_per_key ? dims->dk : 1;
  p.channels = 2 * dims->num_heads * dims->dk + dims->num_heads * dims->dv;
  p.n = n;
  p.flags = dims->flags;
  p.slots = slots;
  p.ell = log ? log->ell : nullptr;
  p.len = log ? log->len : nullptr;
  p.conv_pool = conv_pool;
  p.state = state_pool;
  p.status = status;
  return launched(gdn::launch_slot_reset(p, static_cast<cudaStream_t>(stream)), "gdn_slot_reset");
}

int gdn_kv_plan(int32_t batch, int32_t max_pages, int32_t page_size, int32_t num_pages, int32_t free_capacity,
                int32_t slot_capacity, const int32_t* cached_len, const int32_t* new_len, const int32_t* held, int32_t* block_table,
                const int32_t* free_list, const int32_t* free_count, int32_t* kv_len, int32_t* cu_new,
                int64_t* slot_map, int32_t* held_out, int32_t* free_count_out, int32_t* status, void* stream) {
  if (batch < 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0 || free_capacity < 0 || slot_capacity < 0)
    return fail(GDN_ERR_INVALID_ARG,
                "batch, free_capacity and slot_capacity must be >= 0, max_pages, page_size and num_pages > 0");
  if (batch > gdn::kMaxPlanBatch)
    return fail(GDN_ERR_UNSUPPORTED, "batch %d > %d", batch, gdn::kMaxPlanBatch);
  if (batch == 0) return GDN_OK;
  if (cached_len == nullptr || held == nullptr || block_table == nullptr || (free_list == nullptr && free_capacity > 0) ||
      free_count == nullptr || kv_len == nullptr || cu_new == nullptr || held_out == nullptr ||
      free_count_out == nullptr || (slot_map == nullptr && slot_capacity > 0))
    return fail(GDN_ERR_INVALID_ARG, "every array but new_len and status is required (free_list and slot_map where they have room)");
  gdn::KvPlanParams p{};
  p.B = batch;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  p.slot_capacity = slot_capacity;
  p.cached = cached_len;
  p.fresh = new_len;
  p.held = held;
  p.table = block_table;
  p.free_list = free_list;
  p.free_count = free_count;
  p.kv_len = kv_len;
  p.cu_new = cu_new;
  p.slot_map = slot_map;
  p.held_out = held_out;
  p.free_count_out = free_count_out;
  p.status = status;
  return launched(gdn::launch_kv_plan(p, static_cast<cudaStream_t>(stream)), "gdn_kv_plan");
}

int gdn_kv_release(int32_t batch, int32_t max_pages, int32_t free_capacity, const int32_t* requests, int32_t n,
                   const int32_t* block_table, int32_t* held, int32_t* free_list, int32_t* free_count,
                   int32_t* status, void* stream) {
  if (batch < 0 || max_pages <= 0 || free_capacity <= 0 || n < 0)
    return fail(GDN_ERR_INVALID_ARG, "batch and n must be >= 0, max_pages and free_capacity > 0");
  if (n == 0) return GDN_OK;
  if (requests == nullptr || block_table == nullptr || held == nullptr || free_list == nullptr || free_count == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "requests, block_table, held, free_list and free_count are required");
  gdn::KvReleaseParams p{batch, max_pages, free_capacity, n, requests, block_table, held, free_list, free_count, status};
  return launched(gdn::launch_kv_release(p, static_cast<cudaStream_t>(stream)), "gdn_kv_release");
}

int gdn_kv_append(const gdn_paged_kv* kv, int32_t n, const void* k, const int64_t k_strides[2], const void* v,
                  const int64_t v_strides[2], const int64_t* slot_map, uint32_t flags, int32_t* status,
                  void* stream) {
  if (int rc = check_kv(kv)) return rc;
  if (n < 0) return fail(GDN_ERR_INVALID_ARG, "n < 0");
  if ((flags & ~GDN_QKV_BF16) != 0u) return fail(GDN_ERR_INVALID_ARG, "gdn_kv_append knows GDN_QKV_BF16 only");
  const bool latent = kv->v == nullptr;
  const int tail = latent ? kv->dk - kv->dv : kv->dv;
  if (n == 0) return GDN_OK;
  if (k == nullptr || k_strides == nullptr || slot_map == nullptr || (tail > 0 && (v == nullptr || v_strides == nullptr)))
    return fail(GDN_ERR_INVALID_ARG, "k, v, their strides and slot_map are required");
  const bool bf16 = (flags & GDN_QKV_BF16) != 0u;
  const int multiple = bf16 ? 8 : 4;
  const int32_t extents[2] = {n, kv->num_kv_heads};
  if (!aligned16(k) || !strides_ok(k_strides, extents, multiple) ||
      (tail > 0 && (!aligned16(v) || !strides_ok(v_strides, extents, multiple))))
    return fail(GDN_ERR_UNSUPPORTED, "k and v must be 16-byte aligned, with strides >= 0 that are multiples of 16 bytes");
  gdn::KvAppendParams p{};
  p.n = n;
  p.page_size = kv->page_size;
  p.num_slots = static_cast<int64_t>(kv->num_pages) * kv->page_size;
  p.bf16 = bf16;
  p.a = {k, k_strides[0], k_strides[1], kv->k, kv->k_strides[0], kv->k_strides[1], kv->k_strides[2],
         static_cast<uint32_t>((latent ? kv->dv : kv->dk) / 8), static_cast<uint32_t>(kv->num_kv_heads)};
  if (tail > 0) {
    const int64_t* to = latent ? kv->k_strides : kv->v_strides;
    void* dst = latent ? static_cast<void*>(static_cast<uint16_t*>(kv->k) + kv->dv) : kv->v;
    p.b = {v, v_strides[0], v_strides[1], dst, to[0], to[1], to[2], static_cast<uint32_t>(tail / 8), static_cast<uint32_t>(kv->num_kv_heads)};
  }
  p.slot_map = slot_map;
  p.status = status;
  return launched(gdn::launch_kv_append(p, static_cast<cudaStream_t>(stream)), "gdn_kv_append");
}

int gdn_attn_decode(const gdn_paged_kv* kv, const gdn_attn* attn, void* workspace, size_t workspace_bytes,
                    int32_t* status, void* stream) {
  return attend(kv, attn, workspace, workspace_bytes, status, stream, false, "gdn_attn_decode");
}

int gdn_latent_decode(const gdn_paged_kv* kv, const gdn_attn* attn, void* workspace, size_t workspace_bytes,
                      int32_t* status, void* stream) {
  return attend(kv, attn, workspace, workspace_bytes, status, stream, true, "gdn_latent_decode");
}

int gdn_attn_starve_wait(const gdn_paged_kv* kv, const gdn_attn* attn, int32_t wait, void* workspace, size_t workspace_bytes,
                         int32_t* status, void* stream) {
  if (wait != GDN_STARVE_LOAD && wait != GDN_STARVE_WEIGHTS) return fail(GDN_ERR_INVALID_ARG, "wait is one of GDN_STARVE_*");
  return attend(kv, attn, workspace, workspace_bytes, status, stream, kv != nullptr && kv->v == nullptr, "gdn_attn_starve_wait", wait);
}

int gdn_attn_workspace(const gdn_paged_kv* kv, int32_t batch, int32_t num_tokens, int32_t num_heads, size_t* bytes) {
  if (int rc = check_kv(kv)) return rc;
  if (bytes == nullptr) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
  if (batch < 0 || num_tokens <= 0 || num_heads <= 0 || num_heads % kv->num_kv_heads != 0)
    return fail(GDN_ERR_INVALID_ARG, "batch >= 0, num_tokens > 0 and num_heads a multiple of num_kv_heads");
  const long long cols = static_cast<long long>(num_tokens) * (num_heads / kv->num_kv_heads);
  if (cols > kMaxAttnCols)
    return fail(GDN_ERR_UNSUPPORTED, "num_tokens * num_heads / num_kv_heads must be at most %d", kMaxAttnCols);
  *bytes = gdn::attn_workspace_bytes(gdn::attn_plan(*kv, static_cast<int>(cols)), kv->dv);
  return GDN_OK;
}

int gdn_add_rms_norm(const gdn_norm* norm, void* stream) {
  if (norm == nullptr) return fail(GDN_ERR_INVALID_ARG, "norm is NULL");
  const gdn_norm& n = *norm;
  if (n.rows < 0 || n.width <= 0) return fail(GDN_ERR_INVALID_ARG, "rows must be >= 0 and width > 0");
  auto wide = [](int type) { return type == GDN_TYPE_BF16 || type == GDN_TYPE_FP32; };
  if (!wide(n.x_type) || !wide(n.residual_type) || !(wide(n.o_type) || n.o_type == GDN_TYPE_E4M3))
    return fail(GDN_ERR_INVALID_ARG, "x_type and residual_type are bf16 or fp32, o_type one of these or e4m3");
  if (n.group != 0 && (n.group != gdn::kNormGroup || n.o_type != GDN_TYPE_E4M3))
    return fail(GDN_ERR_UNSUPPORTED, "group is 0, or %d with an e4m3 output", gdn::kNormGroup);
  if (n.width % 8 != 0 || n.width > gdn::kMaxNormWidth)
    return fail(GDN_ERR_UNSUPPORTED, "width %d not built (a multiple of 8, at most %d)", n.width, gdn::kMaxNormWidth);
  if (n.rows == 0) return GDN_OK;
  if (n.x == nullptr || n.o == nullptr || (n.o_type == GDN_TYPE_E4M3 && n.scales == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "x, o and, with an e4m3 output, scales are required");
  const int32_t rows[1] = {n.rows};
  if (!rows_ok(n.x, &n.x_stride, rows, n.x_type == GDN_TYPE_BF16) ||
      (n.residual != nullptr && !rows_ok(n.residual, &n.residual_stride, rows, n.residual_type == GDN_TYPE_BF16)) ||
      !aligned16(n.weight) || !aligned16(n.o))
    return fail(GDN_ERR_UNSUPPORTED, "x, residual, weight and o must be 16-byte aligned, with row strides >= 0 that are multiples of 16 bytes");
  if (n.residual != nullptr && n.rows > 1 && n.residual_stride < n.width)
    return fail(GDN_ERR_INVALID_ARG, "rows of residual overlap");
  if (int rc = check_norm_apart(n)) return rc;
  return launched(gdn::launch_add_rms_norm(n, static_cast<cudaStream_t>(stream)), "gdn_add_rms_norm");
}

int gdn_causal_conv(const gdn_conv* conv, int32_t* status, void* stream) {
  if (conv == nullptr) return fail(GDN_ERR_INVALID_ARG, "conv is NULL");
  const gdn_conv& c = *conv;
  if (c.batch < 0 || c.num_tokens < 0 || c.channels <= 0 || c.num_slots <= 0)
    return fail(GDN_ERR_INVALID_ARG, "batch and num_tokens must be >= 0, channels and num_slots > 0");
  if ((c.flags & ~(GDN_QKV_BF16 | GDN_CONV_SILU)) != 0u)
    return fail(GDN_ERR_INVALID_ARG, "a gdn_conv knows GDN_QKV_BF16 and GDN_CONV_SILU only");
  if (c.channels % 8 != 0) return fail(GDN_ERR_UNSUPPORTED, "channels %d: not a multiple of 8", c.channels);
  if (c.channels > kMaxChannels || static_cast<long long>(c.batch) * c.num_tokens > kMaxPositions ||
      static_cast<long long>(c.batch) * c.num_tokens > (1LL << 38) / c.channels)
    return fail(GDN_ERR_UNSUPPORTED, "channels must be at most 2^24, batch * num_tokens 2^30, times channels 2^38");
  if (c.batch == 0 || c.num_tokens == 0) return GDN_OK;
  if (c.x == nullptr || c.w == nullptr || c.pool == nullptr || c.slot == nullptr || c.o == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "x, w, pool, slot and o are required");
  const int32_t two[2] = {c.batch, c.num_tokens};
  if (!rows_ok(c.x, c.x_strides, two, (c.flags & GDN_QKV_BF16) != 0u))
    return fail(GDN_ERR_UNSUPPORTED, "x must be 16-byte aligned, with strides >= 0 that are multiples of 16 bytes");
  if (!aligned16(c.w) || !aligned16(c.bias) || !aligned16(c.pool) || !aligned16(c.o))
    return fail(GDN_ERR_UNSUPPORTED, "w, bias, pool and o must be 16-byte aligned");
  if (int rc = check_conv_apart(c)) return rc;
  return launched(gdn::launch_causal_conv({c, status}, static_cast<cudaStream_t>(stream)), "gdn_causal_conv");
}

int gdn_ssm_scan(const gdn_ssm* ssm, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  if (int rc = check_ssm(ssm)) return rc;
  if (ssm->batch == 0 || ssm->num_tokens == 0) return GDN_OK;
  const size_t need = gdn::ssm_scan_in_parts(*ssm) ? gdn::ssm_workspace_bytes(ssm->batch, ssm->num_tokens, ssm->channels, ssm->state_size) : 0;
  if (workspace_bytes < need || (need > 0 && workspace == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes, %zu are needed (gdn_ssm_workspace)", workspace == nullptr ? 0 : workspace_bytes, need);
  if (need > 0 && !aligned16(workspace)) return fail(GDN_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  if (int rc = check_ssm_apart(*ssm, workspace, need)) return rc;
  return launched(gdn::launch_ssm_scan({*ssm, status}, workspace, static_cast<cudaStream_t>(stream)), "gdn_ssm_scan");
}

int gdn_ssm_step(const gdn_ssm* ssm, int32_t* status, void* stream) {
  if (int rc = check_ssm(ssm)) return rc;
  if (ssm->num_tokens != 1 || ssm->seq_lens != nullptr)
    return fail(GDN_ERR_INVALID_ARG, "gdn_ssm_step takes one token of every request: num_tokens 1, seq_lens NULL");
  if (ssm->batch == 0) return GDN_OK;
  if (int rc = check_ssm_apart(*ssm, nullptr, 0)) return rc;
  return launched(gdn::launch_ssm_step({*ssm, status}, static_cast<cudaStream_t>(stream)), "gdn_ssm_step");
}

int gdn_ssm_workspace(int32_t batch, int32_t num_tokens, int32_t channels, int32_t state_size, size_t* bytes) {
  if (bytes == nullptr) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
  if (int rc = check_ssm_sizes(batch, num_tokens, channels, state_size)) return rc;
  *bytes = gdn::ssm_workspace_bytes(batch, num_tokens, channels, state_size);
  return GDN_OK;
}

}  // extern "C"
