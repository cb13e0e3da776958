// C-ABI of the 4-bit paged key/value cache (declared in include/kvcache.h).
//
// Host side only: validation, the context (its shape and the error word), and
// the launches. The arithmetic runs in kv_append.hip, kv_attend.hip, kv_tree.hip
// and kv_verify.hip.
#include "kvcache.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <new>
#include <string>

#include "host_common.h"
#include "kv_checks.h"
#include "kv_internal.h"

using namespace agemm;

struct kvc_ctx {
  KvLayout L{};
  int device = 0;
  int num_cus = 0;
  int64_t patience = 0;  // ticks that a workgroup of a verification waits for the others
  uint64_t* err_host = nullptr;  // the last report (kv_report.h), 0: none
  uint64_t* err_dev = nullptr;
  std::string last_error;
};

namespace {

int fail(kvc_ctx* c, int code, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
int fail(kvc_ctx* c, int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(&c->last_error, code, "%s", buf);
}

int hip_fail(kvc_ctx* c, hipError_t e, const char* what) { return set_hip_error(&c->last_error, e, what); }

// Makes the context's device current for the life of the object.
struct OnDevice {
  int before = -1;
  hipError_t e;
  explicit OnDevice(int device) {
    e = hipGetDevice(&before);
    if (e == hipSuccess && before != device) e = hipSetDevice(device);
    else before = -1;
  }
  ~OnDevice() {
    if (before >= 0) (void)hipSetDevice(before);
  }
};

int attend(kvc_ctx* ctx, const void* pages, const kvc_attend_args* p, const uint64_t* mask, int32_t mask_words,
           void* workspace, int64_t workspace_bytes, void* stream) {
  KvPlan plan{};
  if (p && p->batch >= 0 && p->batch <= kKvMaxTokens && p->max_q >= 1 && p->max_q <= kKvMaxTokens &&
      p->max_kv >= 1)  // refused below otherwise
    plan = mask ? kv_tree_plan(ctx->L, p->batch, p->max_q, p->max_kv, p->out_f32 != 0, ctx->num_cus)
                : kv_attend_plan(ctx->L, p->batch, p->max_q, p->max_kv, ctx->num_cus);
  char why[kKvWhy];
  const int rc = kv_check_attend(ctx->L, pages, p, plan, workspace, workspace_bytes, why);
  if (rc) return rc == kKvNothing ? AGEMM_OK : fail(ctx, rc, "%s", why);

  KvAttendArgs a{};
  a.L = ctx->L;
  a.pages = static_cast<const char*>(pages);
  a.batch = p->batch;
  a.max_q = p->max_q;
  a.tokens = p->tokens;
  a.q = static_cast<const _Float16*>(p->q);
  a.q_ts = p->q_token_stride;
  a.q_hs = p->q_head_stride;
  a.q_start = p->q_start;
  a.kv_len = p->kv_len;
  a.q_off = p->q_off;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.table_width = p->table_width;
  a.causal = p->causal;
  a.scale = p->scale;
  a.out = p->out;
  a.lse = p->lse;
  a.tree = mask;
  a.tree_words = mask_words;
  if (!mask) kv_many_wide(plan, ctx->L, p->batch, p->max_q, p->max_kv, p->tokens, ctx->num_cus);
  a.plan = plan;
  a.ws = static_cast<float*>(workspace);
  a.joins = reinterpret_cast<int32_t*>(a.ws + plan.partials * plan.slot_floats);
  a.err = ctx->err_dev;
  OnDevice on(ctx->device);
  if (on.e != hipSuccess) return hip_fail(ctx, on.e, "hipSetDevice");
  const hipError_t e = launch_kv_attend(a, p->out_f32 != 0, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? AGEMM_OK : hip_fail(ctx, e, "attention launch");
}

}  // namespace

extern "C" {

int kvc_create(kvc_ctx** out, int Hq, int Hkv, int D, int page_tokens, int64_t num_pages) {
  if (!out) return AGEMM_EINVAL;
  *out = nullptr;
  const int rc = kv_check_create(Hq, Hkv, D, page_tokens, num_pages);
  if (rc) return rc;
  kvc_ctx* c = new (std::nothrow) kvc_ctx();
  if (!c) return AGEMM_ENOMEM;
  c->L = kv_layout(Hq, Hkv, D, page_tokens, num_pages);
  hipError_t e = hipGetDevice(&c->device);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&c->num_cus, hipDeviceAttributeMultiprocessorCount, c->device);
  int khz = 0;
  if (e == hipSuccess) e = hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, c->device);
  // Some forty times what a round takes with parts of 2048 tokens. What a workgroup waits for is by how much the others end
  // later, not a round: those of parts of 2^20 tokens (600 us) still go on by themselves. AGEMM_VERIFY_WAIT_US: a testing
  // hook (0: no wait, the last kernel does it all).
  const char* wait = std::getenv("AGEMM_VERIFY_WAIT_US");
  const long us = wait ? std::strtol(wait, nullptr, 10) : 200;
  c->patience = (int64_t)(us < 0 ? 0 : us < 100000 ? us : 100000) * khz / 1000;
  void* hp = nullptr;
  if (e == hipSuccess) e = hipHostMalloc(&hp, sizeof(uint64_t), hipHostMallocMapped | hipHostMallocCoherent);
  if (e == hipSuccess) {
    c->err_host = static_cast<uint64_t*>(hp);
    *c->err_host = 0;
    void* dp = nullptr;
    e = hipHostGetDevicePointer(&dp, hp, 0);
    c->err_dev = static_cast<uint64_t*>(dp);
  }
  if (e != hipSuccess) {
    if (hp) (void)hipHostFree(hp);
    delete c;
    return AGEMM_EHIP;
  }
  *out = c;
  return AGEMM_OK;
}

int kvc_destroy(kvc_ctx* ctx) {
  if (!ctx) return AGEMM_OK;
  {
    OnDevice on(ctx->device);
    (void)hipDeviceSynchronize();
    (void)hipHostFree(ctx->err_host);
  }
  delete ctx;
  return AGEMM_OK;
}

int kvc_page_bytes(const kvc_ctx* ctx, int64_t* bytes) {
  if (!ctx || !bytes) return AGEMM_EINVAL;
  *bytes = ctx->L.page_bytes;
  return AGEMM_OK;
}

int kvc_append(kvc_ctx* ctx, void* pages, const kvc_append_args* p, void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  const KvLayout& L = ctx->L;
  char why[kKvWhy];
  const int rc = kv_check_append(ctx->L, pages, p, why);
  if (rc) return rc == kKvNothing ? AGEMM_OK : fail(ctx, rc, "%s", why);

  KvAppendArgs a{};
  a.L = L;
  a.pages = static_cast<char*>(pages);
  a.tokens = p->tokens;
  a.q = static_cast<const _Float16*>(p->q);
  a.k = static_cast<const _Float16*>(p->k);
  a.v = static_cast<const _Float16*>(p->v);
  a.q_out = static_cast<_Float16*>(p->q_out);
  a.q_ts = p->q_token_stride;
  a.q_hs = p->q_head_stride;
  a.k_ts = p->k_token_stride;
  a.k_hs = p->k_head_stride;
  a.v_ts = p->v_token_stride;
  a.v_hs = p->v_head_stride;
  a.o_ts = p->out_token_stride;
  a.o_hs = p->out_head_stride;
  a.slots = p->slots;
  a.positions = p->positions;
  a.rope = p->rope;
  a.rope_len = p->rope_len;
  a.rope_dims = p->rope_dims;
  a.interleaved = p->interleaved;
  a.q_norm = static_cast<const _Float16*>(p->q_norm);
  a.k_norm = static_cast<const _Float16*>(p->k_norm);
  a.eps = p->eps;
  a.err = ctx->err_dev;
  OnDevice on(ctx->device);
  if (on.e != hipSuccess) return hip_fail(ctx, on.e, "hipSetDevice");
  const int64_t piece = kv_append_piece(L);
  for (a.first = 0; a.first < p->tokens; a.first += piece) {
    KvAppendArgs c = a;
    c.tokens = p->tokens - a.first < piece ? p->tokens - a.first : piece;
    if (c.q) c.q += a.first * a.q_ts, c.q_out += a.first * a.o_ts;
    if (c.k) c.k += a.first * a.k_ts, c.v += a.first * a.v_ts, c.slots += a.first;
    if (c.positions) c.positions += a.first;
    const hipError_t e = launch_kv_append(c, ctx->num_cus, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(ctx, e, "append launch");
  }
  return AGEMM_OK;
}

int kvc_attend_workspace(const kvc_ctx* ctx, int32_t batch, int32_t max_q, int64_t max_kv, int64_t* bytes) {
  if (!ctx || !bytes || batch < 0 || max_q < 1 || max_kv < 1) return AGEMM_EINVAL;
  if (batch > kKvMaxTokens || max_q > kKvMaxTokens) return AGEMM_ESHAPE;
  *bytes = kv_attend_bound(ctx->L, batch, max_q, max_kv, ctx->num_cus);
  const int64_t tree = kv_tree_bound(ctx->L, batch, max_q, max_kv, ctx->num_cus);
  if (*bytes < tree) *bytes = tree;
  return AGEMM_OK;
}

int kvc_attend(kvc_ctx* ctx, const void* pages, const kvc_attend_args* p, void* workspace, int64_t workspace_bytes,
               void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  return attend(ctx, pages, p, nullptr, 0, workspace, workspace_bytes, stream);
}

int kvc_attend_tree(kvc_ctx* ctx, const void* pages, const kvc_attend_args* p, const uint64_t* mask, int32_t mask_words,
                    void* workspace, int64_t workspace_bytes, void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  char why[kKvWhy];
  const int rc = kv_check_mask(p, mask, mask_words, why);
  if (rc) return fail(ctx, rc, "%s", why);
  return attend(ctx, pages, p, mask, mask_words, workspace, workspace_bytes, stream);
}

int kvc_tree(kvc_ctx* ctx, const kvc_tree_args* p, void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  char why[kKvWhy];
  int rc = kv_check_tree(p, why);
  if (!rc) rc = kv_check_tree_apart(p, why);
  if (rc) return rc == kKvNothing ? AGEMM_OK : fail(ctx, rc, "%s", why);

  KvTreeArgs a{};
  a.L = ctx->L;
  a.batch = p->batch;
  a.max_q = p->max_q;
  a.tokens = p->tokens;
  a.q_start = p->q_start;
  a.kv_len = p->kv_len;
  a.parent = p->parent;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.table_width = p->table_width;
  a.words = p->mask_words;
  a.mask = p->mask;
  a.positions = p->positions;
  a.slots = p->slots;
  a.total_len = p->total_len;
  a.err = ctx->err_dev;
  OnDevice on(ctx->device);
  if (on.e != hipSuccess) return hip_fail(ctx, on.e, "hipSetDevice");
  const hipError_t e = launch_kv_tree(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? AGEMM_OK : hip_fail(ctx, e, "tree launch");
}

int kvc_verify_workspace(const kvc_ctx* ctx, int32_t batch, int64_t vocab, int64_t* bytes) {
  if (!ctx || !bytes || batch < 0 || vocab < 1) return AGEMM_EINVAL;
  if (batch > kKvMaxSequences || vocab > (int64_t{1} << 28)) return AGEMM_ESHAPE;
  *bytes = kv_verify_bound(batch, vocab, ctx->num_cus);
  return AGEMM_OK;
}

int kvc_verify(kvc_ctx* ctx, const kvc_verify_args* p, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  KvVerifyPlan plan{};
  if (p && p->batch > 0 && p->batch <= kKvMaxSequences && p->vocab >= 1 && p->vocab <= (int64_t{1} << 28))  // refused below otherwise
    plan = kv_verify_plan(p->batch, p->vocab, p->q != nullptr, p->max_children, ctx->num_cus);
  char why[kKvWhy];
  const int64_t need = p ? kv_verify_bytes(plan, p->batch) : 0;
  int rc = kv_check_verify(p, need, workspace, workspace_bytes, why);
  if (!rc) rc = kv_check_verify_apart(p, workspace, need, why);
  if (rc) return rc == kKvNothing ? AGEMM_OK : fail(ctx, rc, "%s", why);

  KvVerifyArgs a{};
  a.batch = p->batch;
  a.max_q = p->max_q;
  a.tokens = p->tokens;
  a.q_start = p->q_start;
  a.parent = p->parent;
  a.token = p->token;
  a.p = p->p;
  a.q = p->q;
  a.p_stride = p->p_stride;
  a.q_stride = p->q_stride;
  a.vocab = (int32_t)p->vocab;
  a.u = p->u;
  a.path = p->path;
  a.count = p->count;
  a.next = p->next;
  a.plan = plan;
  // The states first, on lines of their own, as far as the workspace is aligned to lines.
  a.states = static_cast<KvVerifyState*>(workspace);
  a.sums = reinterpret_cast<double*>(a.states + p->batch);
  a.patience = ctx->patience;
  a.err = ctx->err_dev;
  OnDevice on(ctx->device);
  if (on.e != hipSuccess) return hip_fail(ctx, on.e, "hipSetDevice");
  const hipError_t e = launch_kv_verify(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? AGEMM_OK : hip_fail(ctx, e, "verification launch");
}

int kvc_commit(kvc_ctx* ctx, void* const* pages, int32_t layers, const kvc_commit_args* p, void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  char why[kKvWhy];
  int rc = kv_check_commit(ctx->L, pages, layers, p, why);
  if (!rc) rc = kv_check_commit_apart(p, why);
  if (rc) return rc == kKvNothing ? AGEMM_OK : fail(ctx, rc, "%s", why);

  KvCommitArgs a{};
  a.L = ctx->L;
  a.batch = p->batch;
  a.max_q = p->max_q;
  a.tokens = p->tokens;
  a.q_start = p->q_start;
  a.kv_len = p->kv_len;
  a.path = p->path;
  a.count = p->count;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.table_width = p->table_width;
  a.new_len = p->new_len;
  a.err = ctx->err_dev;
  OnDevice on(ctx->device);
  if (on.e != hipSuccess) return hip_fail(ctx, on.e, "hipSetDevice");
  const int piece = kv_commit_piece(ctx->L, p->batch);
  int i = 0;
  do {  // once without layers, for the lengths
    a.layers = layers - i < piece ? layers - i : piece;
    for (int j = 0; j < a.layers; ++j) a.pages[j] = static_cast<char*>(pages[i + j]);
    const hipError_t e = launch_kv_commit(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(ctx, e, "commit launch");
    a.new_len = nullptr;  // written by the first launch
    i += piece;
  } while (i < layers);
  return AGEMM_OK;
}

int kvc_read(kvc_ctx* ctx, const void* pages, int64_t tokens, const int64_t* slots, void* k_out, void* v_out,
             void* stream) {
  if (!ctx) return AGEMM_EINVAL;
  char why[kKvWhy];
  const int rc = kv_check_read(pages, tokens, slots, k_out, v_out, why);
  if (rc) return rc == kKvNothing ? AGEMM_OK : fail(ctx, rc, "%s", why);

  KvReadArgs a{};
  a.L = ctx->L;
  a.pages = static_cast<const char*>(pages);
  a.err = ctx->err_dev;
  OnDevice on(ctx->device);
  if (on.e != hipSuccess) return hip_fail(ctx, on.e, "hipSetDevice");
  const int64_t piece = kv_read_piece(ctx->L), row = (int64_t)ctx->L.Hkv * ctx->L.D;
  for (a.first = 0; a.first < tokens; a.first += piece) {
    a.tokens = tokens - a.first < piece ? tokens - a.first : piece;
    a.slots = slots + a.first;
    a.k_out = static_cast<_Float16*>(k_out) + a.first * row;
    a.v_out = static_cast<_Float16*>(v_out) + a.first * row;
    const hipError_t e = launch_kv_read(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(ctx, e, "read launch");
  }
  return AGEMM_OK;
}

int kvc_check(kvc_ctx* ctx) {
  if (!ctx) return AGEMM_EINVAL;
  const uint64_t word = __atomic_exchange_n(ctx->err_host, uint64_t{0}, __ATOMIC_ACQ_REL);
  if (word == 0) return AGEMM_OK;
  char what[kKvWhy];
  kv_report_text(what, sizeof what, word, ctx->L.num_pages << ctx->L.page_shift, ctx->L.num_pages);
  return fail(ctx, AGEMM_EINVAL, "%s", what);
}

const char* kvc_last_error(kvc_ctx* ctx) { return ctx ? ctx->last_error.c_str() : ""; }

}  // extern "C"
