// Checks of the arguments of the key/value cache's calls (kvcache.h), made
// before anything is launched. No HIP dependency: a CPU check compiles it as
// it is.
#pragma once

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "kv_layout.h"
#include "kvcache.h"

namespace agemm {

constexpr size_t kKvWhy = 256;  // bytes of a reason
constexpr int kKvNothing = -1;  // nothing to refuse and nothing to do

constexpr int64_t kKvMaxTokens = int64_t{1} << 23;  // rows of one call
constexpr int64_t kKvMaxItems = (int64_t{1} << 23) - 1;  // of an attention call: grids stay below 2^32 threads
constexpr int64_t kKvMaxStride = int64_t{1} << 40;

inline int kv_refuse(char* why, int code, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
inline int kv_refuse(char* why, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(why, kKvWhy, fmt, ap);
  va_end(ap);
  return code;
}

inline bool kv_aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class T>
inline bool kv_natural(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & (alignof(T) - 1)) == 0;
}

inline bool kv_stride_ok(int64_t s) { return s >= 0 && s <= kKvMaxStride && s % 8 == 0; }

// Rows (token, head) of D elements that no two (token, head) share.
inline bool kv_rows_apart(int64_t T, int64_t H, int64_t D, int64_t ts, int64_t hs) {
  const bool heads_inside = (H == 1 || hs >= D) && (T == 1 || ts >= (H - 1) * hs + D);
  const bool tokens_inside = (T == 1 || ts >= D) && (H == 1 || hs >= (T - 1) * ts + D);
  return heads_inside || tokens_inside;
}

// 0, kKvNothing, or the status to refuse the call with and the reason in why (kKvWhy bytes).
inline int kv_check_create(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages) {
  if (Hkv < 1 || Hq < Hkv || Hq > 1024 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return AGEMM_ESHAPE;
  if (page_tokens != 32 && page_tokens != 64 && page_tokens != 128 && page_tokens != 256) return AGEMM_ESHAPE;
  if (num_pages < 1 || num_pages > (int64_t{1} << 40) / page_tokens) return AGEMM_ESHAPE;
  return AGEMM_OK;
}

inline KvLayout kv_layout(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages) {
  KvLayout L;
  L.Hq = Hq;
  L.Hkv = Hkv;
  L.D = D;
  L.page_tokens = page_tokens;
  L.page_shift = __builtin_ctz((unsigned)page_tokens);
  L.num_pages = num_pages;
  L.page_bytes = (int64_t)Hkv * page_tokens * (D + 8);
  return L;
}

inline int kv_check_append(const KvLayout& L, const void* pages, const kvc_append_args* p, char* why) {
  if (!p) return kv_refuse(why, AGEMM_EINVAL, "args must be non-NULL");
  if (p->tokens < 0) return kv_refuse(why, AGEMM_EINVAL, "tokens must not be negative");
  if (p->tokens > kKvMaxTokens) return kv_refuse(why, AGEMM_ESHAPE, "more than %lld tokens in a call", (long long)kKvMaxTokens);
  if (p->tokens == 0) return kKvNothing;
  if (!p->q && !p->k) return kv_refuse(why, AGEMM_EINVAL, "neither q nor k given");
  if (!p->k != !p->v) return kv_refuse(why, AGEMM_EINVAL, "k and v go together");
  if (!p->q != !p->q_out) return kv_refuse(why, AGEMM_EINVAL, "q and q_out go together");
  if (!p->q && p->q_norm) return kv_refuse(why, AGEMM_EINVAL, "q_norm without q");
  if (!p->k && p->k_norm) return kv_refuse(why, AGEMM_EINVAL, "k_norm without k");
  if (p->k && !p->slots) return kv_refuse(why, AGEMM_EINVAL, "slots are required with k");
  if (p->rope && !p->positions) return kv_refuse(why, AGEMM_EINVAL, "positions are required with rope");
  if (p->rope && (p->rope_len < 1 || p->rope_dims < 1 || p->rope_dims > L.D || p->rope_dims % (L.D / 8)))
    return kv_refuse(why, AGEMM_EINVAL, "rope_dims must be a positive multiple of %d up to %d, rope_len positive", L.D / 8, L.D);
  if (p->interleaved != 0 && p->interleaved != 1) return kv_refuse(why, AGEMM_EINVAL, "interleaved must be 0 or 1");
  if ((p->q_norm || p->k_norm) && !(p->eps >= 0.f && isfinite(p->eps)))
    return kv_refuse(why, AGEMM_EINVAL, "eps must be finite and not negative");
  for (const void* x : {p->q, p->k, p->v, static_cast<const void*>(p->q_out), p->q_norm, p->k_norm})
    if (x && !kv_aligned16(x)) return kv_refuse(why, AGEMM_EINVAL, "q, k, v, q_out and the norm weights must be 16-byte aligned");
  if (p->k && !kv_aligned16(pages)) return kv_refuse(why, AGEMM_EINVAL, "pages must be non-NULL and 16-byte aligned");
  if (!kv_natural(p->slots) || !kv_natural(p->positions) || !kv_natural(p->rope))
    return kv_refuse(why, AGEMM_EINVAL, "slots, positions and rope must be aligned to their elements");
  if (p->q && (!kv_stride_ok(p->q_token_stride) || !kv_stride_ok(p->q_head_stride) || !kv_stride_ok(p->out_token_stride) ||
               !kv_stride_ok(p->out_head_stride)))
    return kv_refuse(why, AGEMM_EINVAL, "strides of q and q_out must be multiples of 8, not negative");
  if (p->k && (!kv_stride_ok(p->k_token_stride) || !kv_stride_ok(p->k_head_stride) || !kv_stride_ok(p->v_token_stride) ||
               !kv_stride_ok(p->v_head_stride)))
    return kv_refuse(why, AGEMM_EINVAL, "strides of k and v must be multiples of 8, not negative");
  if (p->q && !kv_rows_apart(p->tokens, L.Hq, L.D, p->out_token_stride, p->out_head_stride))
    return kv_refuse(why, AGEMM_EINVAL, "rows of q_out overlap");
  if (p->q && p->q == p->q_out && (p->q_token_stride != p->out_token_stride || p->q_head_stride != p->out_head_stride))
    return kv_refuse(why, AGEMM_EINVAL, "q_out in place of q needs the strides of q");
  return AGEMM_OK;
}

inline int kv_check_attend(const KvLayout& L, const void* pages, const kvc_attend_args* p, const KvPlan& plan,
                           const void* workspace, int64_t workspace_bytes, char* why) {
  if (!p) return kv_refuse(why, AGEMM_EINVAL, "args must be non-NULL");
  if (p->batch < 0 || p->tokens < 0) return kv_refuse(why, AGEMM_EINVAL, "batch and tokens must not be negative");
  if (p->max_q < 1 || p->max_kv < 1) return kv_refuse(why, AGEMM_EINVAL, "max_q and max_kv must be positive");
  if (p->tokens > kKvMaxTokens || p->max_q > kKvMaxTokens || p->batch > kKvMaxTokens)
    return kv_refuse(why, AGEMM_ESHAPE, "more than %lld rows in a call", (long long)kKvMaxTokens);
  if (p->batch == 0 || p->tokens == 0) return kKvNothing;
  if (plan.items > kKvMaxItems) return kv_refuse(why, AGEMM_ESHAPE, "batch and max_q too large for one call");
  if (p->causal != 0 && p->causal != 1) return kv_refuse(why, AGEMM_EINVAL, "causal must be 0 or 1");
  if (p->out_f32 != 0 && p->out_f32 != 1) return kv_refuse(why, AGEMM_EINVAL, "out_f32 must be 0 or 1");
  if (!(fabsf(p->scale) < 0x1p127f)) return kv_refuse(why, AGEMM_EINVAL, "scale must be below 2^127 in size");
  if (p->table_width < 1 || p->table_stride < 0 || (p->table_stride > 0 && p->table_stride < p->table_width))
    return kv_refuse(why, AGEMM_EINVAL, "table_width must be positive and table_stride 0 or at least the width");
  if ((int64_t)p->batch * p->table_width > (int64_t{1} << 30) / (L.page_tokens / 32))
    return kv_refuse(why, AGEMM_ESHAPE, "the page table names more than 2^35 tokens");
  if (!p->q_start && (p->max_q != 1 || p->batch > p->tokens))
    return kv_refuse(why, AGEMM_EINVAL, "without q_start max_q is 1 and every sequence has its row");
  if (!kv_stride_ok(p->q_token_stride) || !kv_stride_ok(p->q_head_stride))
    return kv_refuse(why, AGEMM_EINVAL, "strides of q must be multiples of 8, not negative");
  if (!kv_aligned16(pages) || !kv_aligned16(p->q) || !kv_aligned16(p->out))
    return kv_refuse(why, AGEMM_EINVAL, "pages, q and out must be non-NULL and 16-byte aligned");
  if (!p->kv_len || !p->page_table) return kv_refuse(why, AGEMM_EINVAL, "kv_len and page_table must be non-NULL");
  if (!kv_natural(p->q_start) || !kv_natural(p->kv_len) || !kv_natural(p->q_off) || !kv_natural(p->page_table) || !kv_natural(p->lse))
    return kv_refuse(why, AGEMM_EINVAL, "q_start, kv_len, q_off, page_table and lse must be aligned to their elements");
  if (plan.ws_bytes > 0 && (!kv_aligned16(workspace) || workspace_bytes < plan.ws_bytes))
    return kv_refuse(why, AGEMM_EINVAL, "workspace must be 16-byte aligned and hold %lld bytes", (long long)plan.ws_bytes);

  return AGEMM_OK;
}

inline int kv_check_read(const void* pages, int64_t tokens, const int64_t* slots, const void* k_out, const void* v_out,
                         char* why) {
  if (tokens < 0) return kv_refuse(why, AGEMM_EINVAL, "tokens must not be negative");
  if (tokens > kKvMaxTokens) return kv_refuse(why, AGEMM_ESHAPE, "more than %lld tokens in a call", (long long)kKvMaxTokens);
  if (tokens == 0) return kKvNothing;
  if (!slots || !kv_natural(slots)) return kv_refuse(why, AGEMM_EINVAL, "slots must be non-NULL and aligned to its elements");
  if (!kv_aligned16(pages) || !kv_aligned16(k_out) || !kv_aligned16(v_out))
    return kv_refuse(why, AGEMM_EINVAL, "pages, k_out and v_out must be non-NULL and 16-byte aligned");
  return AGEMM_OK;
}

}  // namespace agemm
