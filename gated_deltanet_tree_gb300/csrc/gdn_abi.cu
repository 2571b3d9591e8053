// extern "C" entry points: argument checks, the factor-bank lifecycle and the
// kernel launches.  No entry point allocates memory or synchronises the host
// except gdn_check_error and gdn_check_error_words.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "gdn_accept.cuh"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"
#include "gdn_logprobs.cuh"
#include "gdn_seq.cuh"

namespace gdn {
namespace {
thread_local char g_msg[512] = "";
}

gdn_status fail(gdn_status st, const char* fmt, ...) {
  char tmp[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(tmp, sizeof(tmp), fmt, ap);
  va_end(ap);
  std::memcpy(g_msg, tmp, sizeof(tmp));
  return st;
}

void clear_error() { g_msg[0] = '\0'; }

}  // namespace gdn

using gdn::fail;

namespace {

constexpr size_t kAlign = 256;

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define GDN_CHECK_PTR(ptr, name)                                                         \
  do {                                                                                   \
    if ((ptr) == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", name);          \
    if (!aligned16(ptr)) return fail(GDN_ERR_INVALID_ARG, "%s is not 16-byte aligned", name); \
  } while (0)

int channels(const gdn_dims* d) { return 2 * d->Hk * d->dk + d->Hv * d->dv; }

gdn_status check_dims(const gdn_dims* d) {
  if (!d) return fail(GDN_ERR_INVALID_ARG, "dims is NULL");
  if (d->Hk < 1 || d->Hv < 1 || d->Hv % d->Hk != 0)
    return fail(GDN_ERR_INVALID_ARG, "heads Hk = %d, Hv = %d: need Hk >= 1 and Hv a multiple of Hk", d->Hk, d->Hv);
  if (!gdn::verify_supported(d->dk, d->dv))
    return fail(GDN_ERR_UNSUPPORTED, "head sizes dk = %d, dv = %d: supported are 32, 64 and 128", d->dk, d->dv);
  if (d->conv_mode != 0 && d->conv_mode != 1) return fail(GDN_ERR_INVALID_ARG, "conv_mode = %d", d->conv_mode);
  if (d->act != 0 && d->act != 1) return fail(GDN_ERR_INVALID_ARG, "act = %d", d->act);
  if (d->in_dtype != GDN_DTYPE_F32 && d->in_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARG, "in_dtype = %d", d->in_dtype);
  if (d->conv_mode == 1 && (d->K < 1 || d->K > GDN_MAX_TAPS))
    return fail(GDN_ERR_UNSUPPORTED, "conv taps K = %d outside 1..%d", d->K, GDN_MAX_TAPS);
  if (!std::isfinite(d->q_scale) || !std::isfinite(d->l2_eps) || d->l2_eps < 0.f)
    return fail(GDN_ERR_INVALID_ARG, "q_scale / l2_eps not finite or eps negative");
  return GDN_OK;
}

gdn_status check_sched(const gdn_batch_schedule* s) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "schedule is NULL");
  if (s->B < 1) return fail(GDN_ERR_INVALID_ARG, "schedule B = %d", s->B);
  if (s->n_max < 1 || s->n_max > GDN_MAX_NODES)
    return fail(GDN_ERR_UNSUPPORTED, "n_max = %d outside 1..%d", s->n_max, GDN_MAX_NODES);
  if (s->nb_max < 0 || s->nb_max > s->n_max) return fail(GDN_ERR_INVALID_ARG, "nb_max = %d", s->nb_max);
  GDN_CHECK_PTR(s->words, "schedule words");
  return GDN_OK;
}

gdn_status check_banks(const gdn_banks* bk, int B, int layers, int n_max) {
  if (!bk) return fail(GDN_ERR_INVALID_ARG, "banks is NULL");
  if (bk->B != B || bk->layers != layers || bk->n_max != n_max)
    return fail(GDN_ERR_CAPACITY, "banks sized for B=%d layers=%d n_max=%d, call has B=%d layers=%d n_max=%d", bk->B,
                bk->layers, bk->n_max, B, layers, n_max);
  if (bk->write_bank != 0 && bk->write_bank != 1) return fail(GDN_ERR_STATE, "banks not initialised (write_bank)");
  if (bk->pend_bank != -1 && bk->pend_bank != 1 - bk->write_bank)
    return fail(GDN_ERR_STATE, "banks lifecycle corrupted (pend_bank = %d, write_bank = %d)", bk->pend_bank,
                bk->write_bank);
  GDN_CHECK_PTR(bk->pend_path, "banks.pend_path");
  GDN_CHECK_PTR(bk->pend_len, "banks.pend_len");
  GDN_CHECK_PTR(bk->err, "banks.err");
  return GDN_OK;
}

gdn_status check_bank_fields(const gdn_banks* bk, const gdn_dims* d, int i, const char* which) {
  char name[64];
  std::snprintf(name, sizeof(name), "banks.k[%d] (%s)", i, which);
  GDN_CHECK_PTR(bk->k[i], name);
  std::snprintf(name, sizeof(name), "banks.u[%d] (%s)", i, which);
  GDN_CHECK_PTR(bk->u[i], name);
  std::snprintf(name, sizeof(name), "banks.a[%d] (%s)", i, which);
  GDN_CHECK_PTR(bk->a[i], name);
  if (d->conv_mode == 1) {
    std::snprintf(name, sizeof(name), "banks.x[%d] (%s)", i, which);
    GDN_CHECK_PTR(bk->x[i], name);
  }
  return GDN_OK;
}

gdn_status cuda_fail(cudaError_t e, const char* what) {
  return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

size_t ws_q_bytes(const gdn_dims* d, int B, int layers, int n_max) {
  return round_up(static_cast<size_t>(B) * layers * n_max * d->Hk * d->dk * sizeof(float), kAlign);
}

// Reads and clears device error words; the status of what they hold.
gdn_status read_error_words(int32_t* err, cudaStream_t stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronise");
  int32_t w[2] = {0, 0};
  e = cudaMemcpyAsync(w, err, sizeof(w), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "reading the error words");
  if (w[0] == 0) return GDN_OK;
  e = cudaMemsetAsync(err, 0, sizeof(w), stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the error words");
  if (w[0] & GDN_DEVERR_INVALID_PATH)
    return fail(GDN_ERR_INVALID_PATH, "accepted path of request %d is not a root path of its tree; nothing was "
                "committed for it", w[1] - 1);
  if (w[0] & GDN_DEVERR_TIMEOUT)
    return fail(GDN_ERR_TIMEOUT, "an asynchronous copy of request %d did not complete within the bounded wait; "
                "its outputs are incomplete", w[1] - 1);
  if (w[0] & GDN_DEVERR_SCHEDULE)
    return fail(GDN_ERR_SCHEDULE, "packed schedule of request %d is out of range (n, chains, boundary slots); "
                "the offending accesses were skipped", w[1] - 1);
  if (w[0] & GDN_DEVERR_CACHE)
    return fail(GDN_ERR_CACHE, "4-bit cache of request %d: a length, page number, path entry or row count is out of "
                "range; the offending accesses were skipped", w[1] - 1);
  if (w[0] & GDN_DEVERR_LOGITS)
    return fail(GDN_ERR_LOGITS, "request (or row) %d: a visited logits row holds no distribution, or its "
                "temperature is negative or not finite; nothing was taken from it", w[1] - 1);
  return fail(GDN_ERR_CUDA, "unknown device error word 0x%x", w[0]);
}

constexpr int kMaxAppendRows = 1 << 21;

int pages_of(int tokens) { return tokens / GDN_KV4_PAGE + (tokens % GDN_KV4_PAGE ? 1 : 0); }

gdn_status check_attn_dims(const gdn_attn_dims* d) {
  if (!d) return fail(GDN_ERR_INVALID_ARG, "dims is NULL");
  if (d->Hq < 1 || d->Hkv < 1 || d->Hq % d->Hkv != 0)
    return fail(GDN_ERR_INVALID_ARG, "heads Hq = %d, Hkv = %d: need Hkv >= 1 and Hq a multiple of Hkv", d->Hq, d->Hkv);
  if (d->Hq > 1024) return fail(GDN_ERR_UNSUPPORTED, "Hq = %d above 1024", d->Hq);
  if (d->D != 64 && d->D != 128 && d->D != 256)
    return fail(GDN_ERR_UNSUPPORTED, "head size D = %d: supported are 64, 128 and 256", d->D);
  if (d->dtype != GDN_DTYPE_F32 && d->dtype != GDN_DTYPE_BF16) return fail(GDN_ERR_INVALID_ARG, "dtype = %d", d->dtype);
  if (!std::isfinite(d->scale)) return fail(GDN_ERR_INVALID_ARG, "scale is not finite");
  const int vec = d->dtype == GDN_DTYPE_F32 ? 4 : 8;
  if (d->q_row != 0 && (d->q_row < d->Hq * d->D || d->q_row % vec))
    return fail(GDN_ERR_INVALID_ARG, "q_row = %d: below Hq * D or not a multiple of 16 bytes", d->q_row);
  if (d->kv_row != 0 && (d->kv_row < d->Hkv * d->D || d->kv_row % vec))
    return fail(GDN_ERR_INVALID_ARG, "kv_row = %d: below Hkv * D or not a multiple of 16 bytes", d->kv_row);
  return GDN_OK;
}

gdn_status check_cache(const gdn_kv4_cache* c, int layers) {
  if (!c) return fail(GDN_ERR_INVALID_ARG, "cache is NULL");
  if (c->B < 1 || c->layers < 1 || c->pages_max < 1 || c->n_pages < 1)
    return fail(GDN_ERR_INVALID_ARG, "cache B = %d, layers = %d, pages_max = %d, n_pages = %lld", c->B, c->layers,
                c->pages_max, static_cast<long long>(c->n_pages));
  if (c->pages_max > (INT32_MAX - GDN_KV4_PAGE) / GDN_KV4_PAGE || c->n_pages > INT32_MAX)
    return fail(GDN_ERR_UNSUPPORTED, "pages_max = %d, n_pages = %lld: lengths and page numbers are 32-bit", c->pages_max,
                static_cast<long long>(c->n_pages));
  if (c->layers != layers) return fail(GDN_ERR_CAPACITY, "cache of %d layers, call of %d", c->layers, layers);
  if (static_cast<long long>(c->B) * layers > INT32_MAX / 1024)
    return fail(GDN_ERR_UNSUPPORTED, "B * layers = %lld", static_cast<long long>(c->B) * layers);
  GDN_CHECK_PTR(c->pool, "cache.pool");
  GDN_CHECK_PTR(c->page_table, "cache.page_table");
  GDN_CHECK_PTR(c->seq_len, "cache.seq_len");
  GDN_CHECK_PTR(c->ticket, "cache.ticket");
  GDN_CHECK_PTR(c->err, "cache.err");
  return GDN_OK;
}

gdn::KvCacheView cache_view(const gdn_kv4_cache* c) {
  gdn::KvCacheView v{};
  v.pool = static_cast<char*>(c->pool);
  v.page_table = c->page_table; v.seq_len = c->seq_len; v.ticket = c->ticket; v.err = c->err;
  v.B = c->B; v.layers = c->layers; v.pages_max = c->pages_max; v.n_pages = c->n_pages;
  return v;
}

}  // namespace

#define GDN_TRY(expr)                 \
  do {                                \
    gdn_status st_ = (expr);          \
    if (st_ != GDN_OK) return st_;    \
  } while (0)

extern "C" {

int32_t gdn_abi_version(void) { return GDN_ABI_VERSION; }

const char* gdn_last_error(void) { return gdn::g_msg; }

gdn_status gdn_banks_init(gdn_banks* banks, int32_t B, int32_t layers, int32_t n_max) {
  gdn::clear_error();
  if (!banks) return fail(GDN_ERR_INVALID_ARG, "banks is NULL");
  if (B < 1 || layers < 1 || n_max < 1 || n_max > GDN_MAX_NODES)
    return fail(GDN_ERR_INVALID_ARG, "B = %d, layers = %d, n_max = %d", B, layers, n_max);
  banks->B = B;
  banks->layers = layers;
  banks->n_max = n_max;
  banks->write_bank = 0;
  banks->pend_bank = -1;
  banks->verified_bank = -1;
  return GDN_OK;
}

size_t gdn_workspace_bytes(const gdn_dims* d, int32_t B, int32_t layers, int32_t n_max) {
  if (!d || B < 1 || layers < 1 || n_max < 1) return 0;
  return ws_q_bytes(d, B, layers, n_max) +
         round_up(static_cast<size_t>(B) * layers * n_max * d->Hv * d->dv * sizeof(float), kAlign);
}

gdn_status gdn_tree_verify(const gdn_dims* d, int32_t layers, const gdn_batch_schedule* sched, const void* x_raw,
                           const float* conv_w, const void* beta, const void* log_g, float* state,
                           float* conv_state, float* out_o, float* boundary_states, gdn_banks* banks,
                           void* workspace, size_t workspace_bytes, int32_t flags, cudaStream_t stream) {
  gdn::clear_error();
  if (flags & ~(GDN_VERIFY_BOUNDARY_SCRATCH | GDN_VERIFY_CHAIN_WALK | GDN_VERIFY_UT_SIMT | GDN_VERIFY_TC_PER_HEAD |
                GDN_VERIFY_CHAINS))
    return fail(GDN_ERR_INVALID_ARG, "unknown verify flags 0x%x", flags);
  GDN_TRY(check_dims(d));
  GDN_TRY(check_sched(sched));
  if (layers < 1) return fail(GDN_ERR_INVALID_ARG, "layers = %d", layers);
  const int B = sched->B, n_max = sched->n_max;
  GDN_TRY(check_banks(banks, B, layers, n_max));
  GDN_CHECK_PTR(x_raw, "x_raw");
  GDN_CHECK_PTR(beta, "beta");
  GDN_CHECK_PTR(log_g, "log_g");
  GDN_CHECK_PTR(state, "state");
  GDN_CHECK_PTR(out_o, "out_o");
  GDN_CHECK_PTR(workspace, "workspace");
  if (d->conv_mode == 1) {
    GDN_CHECK_PTR(conv_w, "conv_w");
    if (d->K > 1) GDN_CHECK_PTR(conv_state, "conv_state");
  }
  if (sched->nb_max > 0) GDN_CHECK_PTR(boundary_states, "boundary_states");
  const size_t need = gdn_workspace_bytes(d, B, layers, n_max);
  if (workspace_bytes < need)
    return fail(GDN_ERR_CAPACITY, "workspace holds %zu bytes, the call needs %zu", workspace_bytes, need);
  const int cur = banks->write_bank;
  const int pend = banks->pend_bank;
  GDN_TRY(check_bank_fields(banks, d, cur, "write bank"));
  if (pend >= 0) GDN_TRY(check_bank_fields(banks, d, pend, "pending bank"));

  float* ws_q = static_cast<float*>(workspace);
  float* ws_v = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws_q_bytes(d, B, layers, n_max));

  gdn::ConvParams cp{};
  cp.B = B; cp.layers = layers; cp.n_max = n_max; cp.words = sched->words;
  cp.Hk = d->Hk; cp.Hv = d->Hv; cp.dk = d->dk; cp.dv = d->dv; cp.K = d->conv_mode ? d->K : 1;
  cp.C = channels(d); cp.conv_mode = d->conv_mode; cp.act = d->act; cp.in_dtype = d->in_dtype;
  cp.q_scale = d->q_scale; cp.l2_eps = d->l2_eps;
  cp.x_raw = x_raw; cp.conv_w = conv_w; cp.conv_state = conv_state;
  cp.fold = pend >= 0;
  cp.pend_x = pend >= 0 ? banks->x[pend] : nullptr;
  cp.pend_path = banks->pend_path; cp.pend_len = banks->pend_len;
  cp.q_out = ws_q; cp.v_out = ws_v; cp.k_out = banks->k[cur]; cp.x_out = banks->x[cur]; cp.err = banks->err;
  cudaError_t e = gdn::launch_conv(cp, stream);
  if (e != cudaSuccess) return cuda_fail(e, "conv-window launch");

  gdn::VerifyParams vp{};
  vp.B = B; vp.layers = layers; vp.n_max = n_max; vp.nb_max = sched->nb_max; vp.words = sched->words;
  vp.Hk = d->Hk; vp.Hv = d->Hv; vp.dk = d->dk; vp.dv = d->dv; vp.R = d->Hv / d->Hk; vp.in_dtype = d->in_dtype;
  vp.beta = beta; vp.log_g = log_g; vp.q_in = ws_q; vp.v_in = ws_v; vp.k_in = banks->k[cur];
  vp.u_out = banks->u[cur]; vp.a_out = banks->a[cur];
  vp.state = state; vp.out_o = out_o; vp.boundary = boundary_states;
  vp.boundary_out = (flags & GDN_VERIFY_BOUNDARY_SCRATCH) ? 0 : 1;
  // the UT form costs depth^2 per node and depth per (node, column): deep trees walk their chains, unless
  // the caller says every tree is a chain, which the tensor cores then solve in 16-node segments
  const bool chains_tc = (flags & GDN_VERIFY_CHAINS) && !(flags & (GDN_VERIFY_CHAIN_WALK | GDN_VERIFY_UT_SIMT)) &&
                         gdn::verify_tcp_supported(d->dk, d->dv, n_max, 1);
  vp.chain_walk = !chains_tc && ((flags & GDN_VERIFY_CHAIN_WALK) || sched->depth_max > GDN_UT_MAX_DEPTH) ? 1 : 0;
  vp.fold = pend >= 0;
  if (pend >= 0) {
    vp.pend_k = banks->k[pend]; vp.pend_u = banks->u[pend]; vp.pend_a = banks->a[pend];
  }
  vp.pend_path = banks->pend_path; vp.pend_len = banks->pend_len; vp.err = banks->err;
  // trees of 33 to 64 nodes, none deeper than 16 (as the packers report it): one segment on the tensor cores
  const bool wide_tc = !chains_tc && !vp.chain_walk && n_max > 32 && sched->depth_max >= 1 &&
                       sched->depth_max <= gdn::kWideMaxDepth &&
                       !(flags & (GDN_VERIFY_UT_SIMT | GDN_VERIFY_TC_PER_HEAD)) &&
                       gdn::verify_tcp_supported(d->dk, d->dv, n_max, 2);
  if (chains_tc) {
    e = gdn::launch_verify_tcp(vp, 1, stream);
    if (e != cudaSuccess) return cuda_fail(e, "tree-verify launch (tensor cores, chain segments)");
  } else if (wide_tc) {
    e = gdn::launch_verify_tcp(vp, 2, stream);
    if (e != cudaSuccess) return cuda_fail(e, "tree-verify launch (tensor cores, up to 64 nodes)");
  } else if (vp.chain_walk) {
    e = gdn::launch_verify(vp, stream);
    if (e != cudaSuccess) return cuda_fail(e, "chain-verify launch");
  } else if (!(flags & (GDN_VERIFY_UT_SIMT | GDN_VERIFY_TC_PER_HEAD)) &&
             gdn::verify_tcp_supported(d->dk, d->dv, n_max, 0)) {
    e = gdn::launch_verify_tcp(vp, 0, stream);
    if (e != cudaSuccess) return cuda_fail(e, "tree-verify launch (tensor cores, persistent)");
  } else if (!(flags & GDN_VERIFY_UT_SIMT) && gdn::verify_tc_supported(d->dk, d->dv, n_max)) {
    e = gdn::launch_verify_tc(vp, stream);
    if (e != cudaSuccess) return cuda_fail(e, "tree-verify launch (tensor cores)");
  } else {
    e = gdn::launch_verify_ut(vp, stream);
    if (e != cudaSuccess) return cuda_fail(e, "tree-verify launch");
  }

  banks->pend_bank = -1;
  banks->verified_bank = cur;
  return GDN_OK;
}

gdn_status gdn_commit_fold(const gdn_dims* d, int32_t layers, const gdn_batch_schedule* sched, const int32_t* path,
                           const int32_t* len, int32_t flags, gdn_banks* banks, cudaStream_t stream) {
  gdn::clear_error();
  GDN_TRY(check_dims(d));
  GDN_TRY(check_sched(sched));
  if (layers < 1) return fail(GDN_ERR_INVALID_ARG, "layers = %d", layers);
  GDN_TRY(check_banks(banks, sched->B, layers, sched->n_max));
  GDN_CHECK_PTR(path, "path");
  GDN_CHECK_PTR(len, "len");
  if (flags & ~GDN_COMMIT_COMPACT) return fail(GDN_ERR_INVALID_ARG, "unknown commit flags 0x%x", flags);
  const int vb = banks->verified_bank;
  if (vb < 0) return fail(GDN_ERR_STATE, "commit without a verify since the last commit");
  GDN_TRY(check_bank_fields(banks, d, vb, "verified bank"));

  gdn::CommitParams p{};
  p.B = sched->B; p.layers = layers; p.n_max = sched->n_max; p.words = sched->words;
  p.path = path; p.len = len; p.pend_path = banks->pend_path; p.pend_len = banks->pend_len; p.err = banks->err;
  p.k = banks->k[vb]; p.u = banks->u[vb]; p.a = banks->a[vb]; p.x = d->conv_mode == 1 ? banks->x[vb] : nullptr;
  p.k_words = d->Hk * d->dk; p.u_words = d->Hv * d->dv; p.a_words = d->Hv; p.x_words = channels(d);
  cudaError_t e = gdn::launch_commit(p, flags & GDN_COMMIT_COMPACT, stream);
  if (e != cudaSuccess) return cuda_fail(e, "commit launch");
  banks->pend_bank = vb;
  banks->write_bank = 1 - vb;
  banks->verified_bank = -1;
  return GDN_OK;
}

gdn_status gdn_finish(const gdn_dims* d, int32_t B, int32_t layers, float* state, float* conv_state,
                      gdn_banks* banks, cudaStream_t stream) {
  gdn::clear_error();
  GDN_TRY(check_dims(d));
  if (B < 1 || layers < 1) return fail(GDN_ERR_INVALID_ARG, "B = %d, layers = %d", B, layers);
  GDN_TRY(check_banks(banks, B, layers, banks ? banks->n_max : 0));
  const int pend = banks->pend_bank;
  if (pend < 0) return GDN_OK;
  GDN_CHECK_PTR(state, "state");
  if (d->conv_mode == 1 && d->K > 1) GDN_CHECK_PTR(conv_state, "conv_state");
  GDN_TRY(check_bank_fields(banks, d, pend, "pending bank"));

  cudaError_t e;
  if (d->conv_mode == 1 && d->K > 1) {
    gdn::ConvParams cp{};
    cp.B = B; cp.layers = layers; cp.n_max = banks->n_max; cp.words = nullptr;
    cp.Hk = d->Hk; cp.Hv = d->Hv; cp.dk = d->dk; cp.dv = d->dv; cp.K = d->K; cp.C = channels(d);
    cp.conv_mode = 1; cp.act = d->act; cp.in_dtype = d->in_dtype;
    cp.conv_state = conv_state; cp.fold = 1; cp.pend_x = banks->x[pend];
    cp.pend_path = banks->pend_path; cp.pend_len = banks->pend_len; cp.err = banks->err;
    cp.conv_w = nullptr;  // not read in fold-only mode
    e = gdn::launch_conv(cp, stream);
    if (e != cudaSuccess) return cuda_fail(e, "conv fold launch");
  }
  gdn::VerifyParams vp{};
  vp.B = B; vp.layers = layers; vp.n_max = banks->n_max; vp.words = nullptr;
  vp.Hk = d->Hk; vp.Hv = d->Hv; vp.dk = d->dk; vp.dv = d->dv; vp.R = d->Hv / d->Hk; vp.in_dtype = d->in_dtype;
  vp.state = state; vp.fold = 1;
  vp.pend_k = banks->k[pend]; vp.pend_u = banks->u[pend]; vp.pend_a = banks->a[pend];
  vp.pend_path = banks->pend_path; vp.pend_len = banks->pend_len; vp.err = banks->err;
  e = gdn::launch_verify(vp, stream);
  if (e != cudaSuccess) return cuda_fail(e, "state fold launch");
  banks->pend_bank = -1;
  return GDN_OK;
}

namespace {
// One CTA waits on an mbarrier armed for 16 bytes that no copy delivers: the bounded wait gives up and the
// CTA reports the timeout like the verify kernels do.
__global__ void selftest_wait_timeout_kernel(int32_t* err) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    gdn::mbar_init(&bar);
    gdn::mbar_expect(&bar, 16);
  }
  __syncthreads();
  if (!__syncthreads_and(gdn::mbar_wait(&bar, 0)) && threadIdx.x == 0) gdn::device_error(err, GDN_DEVERR_TIMEOUT, 0);
}
}  // namespace

gdn_status gdn_selftest_wait_timeout(gdn_banks* banks, cudaStream_t stream) {
  gdn::clear_error();
  if (!banks || !banks->err) return fail(GDN_ERR_INVALID_ARG, "banks / banks.err is NULL");
  if (!aligned16(banks->err)) return fail(GDN_ERR_INVALID_ARG, "banks.err is not 16-byte aligned");
  selftest_wait_timeout_kernel<<<1, 32, 0, stream>>>(banks->err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "self-test launch");
  return GDN_OK;
}

gdn_status gdn_check_error(gdn_banks* banks, cudaStream_t stream) {
  gdn::clear_error();
  if (!banks || !banks->err) return fail(GDN_ERR_INVALID_ARG, "banks / banks.err is NULL");
  return read_error_words(banks->err, stream);
}

gdn_status gdn_check_error_words(int32_t* err, cudaStream_t stream) {
  gdn::clear_error();
  GDN_CHECK_PTR(err, "err");
  return read_error_words(err, stream);
}

// ---- 4-bit key/value cache and its attention ----

size_t gdn_kv4_pool_bytes(const gdn_attn_dims* d, int32_t layers, int64_t n_pages) {
  if (check_attn_dims(d) != GDN_OK || layers < 1 || n_pages < 1) return 0;
  return static_cast<size_t>(layers) * static_cast<size_t>(n_pages) * d->Hkv * 72 * d->D;
}

gdn_status gdn_kv4_append(const gdn_attn_dims* d, int32_t layers, int32_t n_rows, const void* k_new,
                          const void* v_new, const int32_t* path, const int32_t* count, gdn_kv4_cache* cache,
                          cudaStream_t stream) {
  gdn::clear_error();
  GDN_TRY(check_attn_dims(d));
  GDN_TRY(check_cache(cache, layers));
  if (n_rows < 1 || n_rows > kMaxAppendRows)
    return fail(GDN_ERR_INVALID_ARG, "n_rows = %d outside 1..%d", n_rows, kMaxAppendRows);
  GDN_CHECK_PTR(k_new, "k_new");
  GDN_CHECK_PTR(v_new, "v_new");
  GDN_CHECK_PTR(count, "count");
  if (path) GDN_CHECK_PTR(path, "path");
  gdn::KvAppendParams p{};
  p.c = cache_view(cache);
  p.Hkv = d->Hkv; p.D = d->D; p.dtype = d->dtype; p.n_rows = n_rows;
  p.kv_row = d->kv_row ? d->kv_row : d->Hkv * d->D;
  p.k_new = k_new; p.v_new = v_new; p.path = path; p.count = count;
  cudaError_t e = gdn::launch_kv4_append(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
  return GDN_OK;
}

gdn_status gdn_kv4_read(const gdn_attn_dims* d, int32_t layers, int32_t n_rows, const int32_t* start,
                        int32_t out_dtype, void* k_out, void* v_out, const gdn_kv4_cache* cache,
                        cudaStream_t stream) {
  gdn::clear_error();
  GDN_TRY(check_attn_dims(d));
  GDN_TRY(check_cache(cache, layers));
  if (n_rows < 1 || n_rows > kMaxAppendRows)
    return fail(GDN_ERR_INVALID_ARG, "n_rows = %d outside 1..%d", n_rows, kMaxAppendRows);
  if (out_dtype != GDN_DTYPE_F32 && out_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARG, "out_dtype = %d", out_dtype);
  GDN_CHECK_PTR(k_out, "k_out");
  GDN_CHECK_PTR(v_out, "v_out");
  if (start) GDN_CHECK_PTR(start, "start");
  gdn::KvReadParams p{};
  p.c = cache_view(cache);
  p.Hkv = d->Hkv; p.D = d->D; p.out_dtype = out_dtype; p.n_rows = n_rows;
  p.start = start; p.k_out = k_out; p.v_out = v_out;
  cudaError_t e = gdn::launch_kv4_read(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  return GDN_OK;
}

size_t gdn_kv4_workspace_bytes(const gdn_attn_dims* d, int32_t B, int32_t layers, int32_t n_max, int32_t max_len) {
  if (check_attn_dims(d) != GDN_OK || B < 1 || layers < 1 || n_max < 1 || n_max > GDN_MAX_NODES || max_len < 0)
    return 0;
  return gdn::plan_kv4_attention(d->Hq, d->Hkv, d->D, d->dtype, B, layers, n_max, pages_of(max_len)).bytes;
}

gdn_status gdn_kv4_attention(const gdn_attn_dims* d, int32_t layers, const gdn_batch_schedule* sched, const void* q,
                             const void* k_new, const void* v_new, void* out, const gdn_kv4_cache* cache,
                             int32_t max_len, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  gdn::clear_error();
  GDN_TRY(check_attn_dims(d));
  GDN_TRY(check_cache(cache, layers));
  if (sched) {
    GDN_TRY(check_sched(sched));
    if (sched->B != cache->B)
      return fail(GDN_ERR_CAPACITY, "schedule of %d requests, cache of %d", sched->B, cache->B);
  }
  GDN_CHECK_PTR(q, "q");
  GDN_CHECK_PTR(out, "out");
  if ((k_new == nullptr) != (v_new == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "k_new and v_new: both or neither");
  if (k_new) {
    GDN_CHECK_PTR(k_new, "k_new");
    GDN_CHECK_PTR(v_new, "v_new");
  }
  if (max_len < 0) return fail(GDN_ERR_INVALID_ARG, "max_len = %d", max_len);
  GDN_CHECK_PTR(workspace, "workspace");
  const int n_max = sched ? sched->n_max : 1;
  const gdn::KvAttnPlan pl =
      gdn::plan_kv4_attention(d->Hq, d->Hkv, d->D, d->dtype, cache->B, layers, n_max, pages_of(max_len));
  if (!pl.kernel)
    return fail(GDN_ERR_UNSUPPORTED, "layers = %d, Hkv = %d, n_max = %d: above %d tiles of %d rows a request", layers, d->Hkv,
                n_max, gdn::kKvCounters, gdn::kKvDecRows);
  if (workspace_bytes < pl.bytes)
    return fail(GDN_ERR_CAPACITY, "workspace holds %zu bytes, the call needs %zu", workspace_bytes, pl.bytes);
  gdn::KvAttnParams p{};
  p.c = cache_view(cache);
  p.layers = layers; p.n_max = n_max; p.Hq = d->Hq; p.Hkv = d->Hkv; p.D = d->D; p.dtype = d->dtype;
  p.G = d->Hq / d->Hkv; p.scale = d->scale;
  p.q_row = d->q_row ? d->q_row : static_cast<long long>(d->Hq) * d->D;
  p.kv_row = d->kv_row ? d->kv_row : static_cast<long long>(d->Hkv) * d->D;
  p.words = sched ? sched->words : nullptr;
  p.q = q; p.k_new = k_new; p.v_new = v_new; p.out = out;
  p.ctas = pl.ctas; p.least = pl.least; p.row_tiles = pl.row_tiles;
  p.done = static_cast<int32_t*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.done_bytes);
  p.desc = reinterpret_cast<int4*>(p.done + gdn::kKvCounters);
  cudaError_t e =
      pl.kernel == gdn::kKvDec ? gdn::launch_kv4_attention_dec(p, stream) : gdn::launch_kv4_attention_tree(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cache attention launch");
  return GDN_OK;
}

// ---- acceptance of drafted tokens ----

size_t gdn_accept_workspace_bytes(int32_t B, int32_t n_max, int32_t V) {
  if (B < 1 || n_max < 1 || n_max > GDN_MAX_NODES || V < 1 || V > gdn::kMaxVocab) return 0;
  return round_up(static_cast<size_t>(B) * n_max * gdn::accept_slices(B, n_max, V, true) * 16 + 1, kAlign);
}

gdn_status gdn_tree_accept(const gdn_batch_schedule* sched, int32_t V, int32_t v_stride, int32_t logits_dtype,
                           const void* logits, const int32_t* tokens, const void* draft_probs, int32_t draft_dtype,
                           const float* uniform, const float* gumbel, const float* temperature, int32_t* path,
                           int32_t* len, int32_t* next, int32_t* err, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  gdn::clear_error();
  GDN_TRY(check_sched(sched));
  if (V < 1) return fail(GDN_ERR_INVALID_ARG, "V = %d", V);
  if (V > gdn::kMaxVocab) return fail(GDN_ERR_UNSUPPORTED, "V = %d above %d", V, gdn::kMaxVocab);
  if (v_stride != 0 && v_stride < V) return fail(GDN_ERR_INVALID_ARG, "v_stride = %d, V = %d", v_stride, V);
  if (logits_dtype != GDN_DTYPE_F32 && logits_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARG, "logits_dtype = %d", logits_dtype);
  if (draft_probs && draft_dtype != GDN_DTYPE_F32 && draft_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARG, "draft_dtype = %d", draft_dtype);
  GDN_CHECK_PTR(logits, "logits");
  GDN_CHECK_PTR(tokens, "tokens");
  if (draft_probs) GDN_CHECK_PTR(draft_probs, "draft_probs");
  if (temperature) {
    GDN_CHECK_PTR(temperature, "temperature");
    GDN_CHECK_PTR(uniform, "uniform");
    GDN_CHECK_PTR(gumbel, "gumbel");
  }
  GDN_CHECK_PTR(path, "path");
  GDN_CHECK_PTR(len, "len");
  GDN_CHECK_PTR(next, "next");
  GDN_CHECK_PTR(err, "err");
  GDN_CHECK_PTR(workspace, "workspace");
  const size_t need = gdn_accept_workspace_bytes(sched->B, sched->n_max, V);
  if (workspace_bytes < need)
    return fail(GDN_ERR_CAPACITY, "workspace holds %zu bytes, the call needs %zu", workspace_bytes, need);
  gdn::AcceptParams p{};
  p.B = sched->B; p.n_max = sched->n_max; p.V = V; p.logits_dtype = logits_dtype; p.draft_dtype = draft_dtype;
  p.v_stride = v_stride ? v_stride : V;
  p.words = sched->words; p.logits = logits; p.tokens = tokens; p.draft = draft_probs;
  p.uniform = uniform; p.gumbel = gumbel; p.temperature = temperature;
  p.path = path; p.len = len; p.next = next; p.err = err;
  p.n_slices = gdn::accept_slices(sched->B, sched->n_max, V, draft_probs != nullptr);
  p.slices = workspace;
  cudaError_t e = gdn::launch_accept(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "acceptance launch");
  return GDN_OK;
}

// ---- sequences through one layer ----

namespace {

bool known_dtype(int32_t t) { return t == GDN_DTYPE_F32 || t == GDN_DTYPE_BF16; }

// An output that is its input's buffer, or does not overlap it.
gdn_status check_moved(const void* in, const void* out, size_t bytes, const char* name) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  if (in && a != b && a < b + bytes && b < a + bytes)
    return fail(GDN_ERR_INVALID_ARG, "%s_out overlaps %s without being it", name, name);
  return GDN_OK;
}

// Everything that gdn_prefill and gdn_step share; fills p for the given layer.
gdn_status check_seq(const gdn_dims* d, int32_t layers, int32_t layer, int32_t B, const void* x_raw, int64_t x_row,
                     const float* conv_w, const void* beta, const void* log_g, int64_t gate_row, const float* state,
                     const float* conv_state, float* state_out, float* conv_out, void* out_o, int32_t out_dtype,
                     const gdn_banks* banks, int32_t* err, gdn::SeqParams& p) {
  GDN_TRY(check_dims(d));
  if (layers < 1 || layer < 0 || layer >= layers) return fail(GDN_ERR_INVALID_ARG, "layer %d of %d", layer, layers);
  if (B < 1) return fail(GDN_ERR_INVALID_ARG, "B = %d", B);
  const long long C = 2ll * d->Hk * d->dk + static_cast<long long>(d->Hv) * d->dv;
  // the kernels number a request's CTAs (up to eight a k-head) and channels with 32 bits
  if (C > (1 << 24) || static_cast<long long>(B) * d->Hk > (1 << 27) || static_cast<long long>(B) * d->Hv > (1 << 27))
    return fail(GDN_ERR_UNSUPPORTED, "B = %d, Hk = %d, Hv = %d: too many heads", B, d->Hk, d->Hv);
  if (!known_dtype(out_dtype)) return fail(GDN_ERR_INVALID_ARG, "out_dtype = %d", out_dtype);
  const int vec = d->in_dtype == GDN_DTYPE_F32 ? 4 : 8;
  if (x_row != 0 && (x_row < C || x_row % vec || x_row > INT32_MAX))
    return fail(GDN_ERR_INVALID_ARG, "x_row = %lld: below C = %lld, above 2^31 or not a multiple of 16 bytes",
                static_cast<long long>(x_row), C);
  if (gate_row != 0 && (gate_row < d->Hv || gate_row > INT32_MAX))
    return fail(GDN_ERR_INVALID_ARG, "gate_row = %lld, Hv = %d", static_cast<long long>(gate_row), d->Hv);
  const bool conv = d->conv_mode == 1, window = conv && d->K > 1;
  GDN_CHECK_PTR(x_raw, "x_raw");
  if (conv) GDN_CHECK_PTR(conv_w, "conv_w");
  // rows of gates lie where a fused projection puts them
  if (!beta || !log_g) return fail(GDN_ERR_INVALID_ARG, "beta or log_g is NULL");
  const uintptr_t one = d->in_dtype == GDN_DTYPE_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(beta) | reinterpret_cast<uintptr_t>(log_g)) & one)
    return fail(GDN_ERR_INVALID_ARG, "beta or log_g is not aligned to its elements");
  if (state) GDN_CHECK_PTR(state, "state");
  GDN_CHECK_PTR(state_out, "state_out");
  if (window) {
    if (conv_state) GDN_CHECK_PTR(conv_state, "conv_state");
    GDN_CHECK_PTR(conv_out, "conv_out");
  }
  GDN_CHECK_PTR(out_o, "out_o");
  GDN_CHECK_PTR(err, "err");
  const long long tile = static_cast<long long>(d->Hv) * d->dk * d->dv, rows = conv ? (d->K - 1) * C : 0;
  if (B * static_cast<long long>(layers) > (1ll << 60) / (4 * (tile > C * 8 ? tile : C * 8)))
    return fail(GDN_ERR_UNSUPPORTED, "B = %d, layers = %d", B, layers);
  GDN_TRY(check_moved(state, state_out, static_cast<size_t>(B) * layers * tile * sizeof(float), "state"));
  if (window) GDN_TRY(check_moved(conv_state, conv_out, static_cast<size_t>(B) * layers * rows * sizeof(float), "conv"));
  if (banks) {
    if (banks->B != B || banks->layers != layers)
      return fail(GDN_ERR_CAPACITY, "banks sized for B=%d layers=%d, call has B=%d layers=%d", banks->B, banks->layers, B,
                  layers);
    if (banks->verified_bank >= 0) return fail(GDN_ERR_STATE, "a verified tree is not committed (gdn_commit_fold, then gdn_finish)");
    if (banks->pend_bank >= 0) return fail(GDN_ERR_STATE, "a committed path is not in the state yet (gdn_finish folds it in)");
  }
  p.Hk = d->Hk; p.Hv = d->Hv; p.dk = d->dk; p.dv = d->dv; p.K = conv ? d->K : 1; p.C = static_cast<int>(C);
  p.conv_mode = d->conv_mode; p.act = d->act; p.in_dtype = d->in_dtype; p.out_dtype = out_dtype;
  p.q_scale = d->q_scale; p.l2_eps = d->l2_eps;
  p.x_row = x_row ? x_row : C; p.gate_row = gate_row ? gate_row : d->Hv;
  p.x = x_raw; p.beta = beta; p.log_g = log_g;
  p.conv_w = conv ? conv_w + static_cast<long long>(layer) * C * d->K : nullptr;
  p.state_in = state ? state + layer * tile : nullptr;
  p.state_out = state_out + layer * tile;
  p.conv_in = window && conv_state ? conv_state + layer * rows : nullptr;
  p.conv_out = window ? conv_out + layer * rows : nullptr;
  p.state_stride = layers * tile; p.conv_stride = layers * rows;
  p.out = out_o; p.err = err;
  return GDN_OK;
}

}  // namespace

size_t gdn_prefill_workspace_bytes(const gdn_dims* d) { return check_dims(d) == GDN_OK ? gdn::seq_workspace_bytes(*d) : 0; }

gdn_status gdn_prefill(const gdn_dims* d, int32_t layers, int32_t layer, int32_t B, const int32_t* lens,
                       const void* x_raw, int64_t x_row, const float* conv_w, const void* beta, const void* log_g,
                       int64_t gate_row, const float* state, const float* conv_state, float* state_out, float* conv_out,
                       void* out_o, int32_t out_dtype, const gdn_banks* banks, int32_t* err, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  gdn::clear_error();
  gdn::SeqParams p{};
  if (!lens) return fail(GDN_ERR_INVALID_ARG, "lens is NULL");
  long long rows = 0;
  for (int32_t b = 0; b < B; ++b) {
    if (lens[b] < 0) return fail(GDN_ERR_INVALID_ARG, "lens[%d] = %d", b, lens[b]);
    rows += lens[b];
  }
  if (rows > INT32_MAX - gdn::kChunk) return fail(GDN_ERR_UNSUPPORTED, "%lld rows", rows);   // a last chunk ends within 32 bits
  GDN_TRY(check_seq(d, layers, layer, B, x_raw, x_row, conv_w, beta, log_g, gate_row, state, conv_state, state_out,
                    conv_out, out_o, out_dtype, banks, err, p));
  GDN_CHECK_PTR(workspace, "workspace");
  const size_t need = gdn::seq_workspace_bytes(*d);
  if (workspace_bytes < need)
    return fail(GDN_ERR_CAPACITY, "workspace holds %zu bytes, the call needs %zu", workspace_bytes, need);
  cudaError_t e = gdn::launch_prefill(p, lens, B, workspace, stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
  return GDN_OK;
}

gdn_status gdn_step(const gdn_dims* d, int32_t layers, int32_t layer, int32_t B, const int32_t* live, const void* x_raw,
                    int64_t x_row, const float* conv_w, const void* beta, const void* log_g, int64_t gate_row,
                    const float* state, const float* conv_state, float* state_out, float* conv_out, void* out_o,
                    int32_t out_dtype, const gdn_banks* banks, int32_t* err, cudaStream_t stream) {
  gdn::clear_error();
  gdn::SeqParams p{};
  GDN_TRY(check_seq(d, layers, layer, B, x_raw, x_row, conv_w, beta, log_g, gate_row, state, conv_state, state_out,
                    conv_out, out_o, out_dtype, banks, err, p));
  if (live) GDN_CHECK_PTR(live, "live");
  p.live = live;
  cudaError_t e = cudaSuccess;
  if (!gdn::launch_seq_step(p, B, stream, e)) e = gdn::launch_seq_rec(p, nullptr, B, stream);
  if (e != cudaSuccess) return cuda_fail(e, "step launch");
  return GDN_OK;
}

// ---- log-probabilities ----

gdn_status gdn_top_logprobs(int32_t rows, int32_t V, int64_t v_stride, int32_t dtype, const void* logits,
                            const int32_t* tokens, int32_t top_k, float* top_logp, int32_t* top_token, float* given,
                            float* entropy, int32_t* err, cudaStream_t stream) {
  gdn::clear_error();
  if (rows < 1 || V < 1) return fail(GDN_ERR_INVALID_ARG, "rows = %d, V = %d", rows, V);
  if (V > gdn::kLogprobVocab) return fail(GDN_ERR_UNSUPPORTED, "V = %d above %d", V, gdn::kLogprobVocab);
  if (rows > INT32_MAX / 8) return fail(GDN_ERR_UNSUPPORTED, "rows = %d", rows);
  if (v_stride != 0 && v_stride < V)
    return fail(GDN_ERR_INVALID_ARG, "v_stride = %lld, V = %d", static_cast<long long>(v_stride), V);
  if (v_stride > (1ll << 60) / (4ll * rows))
    return fail(GDN_ERR_UNSUPPORTED, "v_stride = %lld", static_cast<long long>(v_stride));
  if (!known_dtype(dtype)) return fail(GDN_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (top_k < 1 || top_k > V) return fail(GDN_ERR_INVALID_ARG, "top_k = %d, V = %d", top_k, V);
  if (top_k > GDN_MAX_TOP) return fail(GDN_ERR_UNSUPPORTED, "top_k = %d above %d", top_k, GDN_MAX_TOP);
  // rows lie at any element: the kernel begins a row within sixteen aligned bytes
  if (!logits) return fail(GDN_ERR_INVALID_ARG, "logits is NULL");
  if (reinterpret_cast<uintptr_t>(logits) & (dtype == GDN_DTYPE_F32 ? 3 : 1))
    return fail(GDN_ERR_INVALID_ARG, "logits is not aligned to its elements");
  if ((tokens == nullptr) != (given == nullptr)) return fail(GDN_ERR_INVALID_ARG, "tokens and given: both or neither");
  if (tokens) {
    GDN_CHECK_PTR(tokens, "tokens");
    GDN_CHECK_PTR(given, "given");
  }
  GDN_CHECK_PTR(top_logp, "top_logp");
  GDN_CHECK_PTR(top_token, "top_token");
  if (entropy) GDN_CHECK_PTR(entropy, "entropy");
  GDN_CHECK_PTR(err, "err");
  gdn::LogprobParams p{};
  p.rows = rows; p.V = V; p.top = top_k; p.dtype = dtype; p.v_stride = v_stride ? v_stride : V;
  p.logits = logits; p.tokens = tokens; p.top_logp = top_logp; p.top_token = top_token;
  p.given = given; p.entropy = entropy; p.err = err;
  cudaError_t e = gdn::launch_logprobs(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "log-probability launch");
  return GDN_OK;
}

}  // extern "C"
