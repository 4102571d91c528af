// gdn_api.cpp -- the extern "C" entry points declared in include/gdn.h:
// argument validation, kernel selection and error reporting. No allocation.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <cuda_runtime_api.h>

#include "gdn.h"
#include "gdn_internal.h"
#include "gdn_kv.h"

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

}  // extern "C"
