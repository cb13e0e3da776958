/*
 * C-ABI of the 4-bit paged key/value cache on one GPU (gfx950): appending to
 * it, attention over it, reading it back.
 *
 * It makes what the Flash-Decode combine (fdcombine.h) takes: each of W ranks
 * attends over its own shard of the cache (kvc_attend with a binary32 output)
 * and hands its normalised partial and log-sum-exp to fdc_produce as they are.
 *
 * What the cache holds. Per token and kv head, keys and values of D channels
 * as 4-bit numbers n_d with one pair (s, b) of binary16 numbers for the keys
 * and one for the values. n stands for the binary16 number nearest to
 *     (16 + n) s + b.
 * kvc_append chooses, from the D channels x of the row (in binary64),
 *     s = binary16((max x - min x) / 15),  b = binary16(min x - 16 s),
 *     n_d = clamp(rint((x_d - b) / s) - 16, 0, 15)   (n_d = 0 where s = 0),
 * s and b by way of binary32, rint to even.
 *
 * Pages (caller-owned device memory, num_pages x kvc_page_bytes, 16-byte
 * aligned): page p starts at byte p * page_bytes and holds page_tokens
 * consecutive tokens of one sequence; a token's slot is
 * p * page_tokens + its offset in the page. A page is Hkv x page_tokens / 32
 * blocks, [kv head][block of 32 tokens], each 32 (D + 8) bytes:
 *   16 D bytes  key nibbles: token t's row at t D / 2, channel d in byte d / 2,
 *               the even channel in the low half;
 *   16 D bytes  value nibbles: token t = 16 h + 4 q + i (h < 2, q, i < 4),
 *               channel d = c D / 16 + 4 g + j (c < 16, j < 4): nibble j of the
 *               16-bit word ((g 4 + q) 16 + c) 8 + 4 h + i;
 *   128 bytes   key pairs: (s, b) of token t at 4 t;
 *   128 bytes   value pairs: s of token t at 2 (8 q + 4 h + i), b 64 bytes on.
 * The layout is what the matrix instructions of kvc_attend take without a
 * shuffle. Bytes of tokens that no kvc_append wrote may hold anything; they
 * are never used, as long as lengths and page tables do not name them.
 *
 * Shapes: 1 <= Hkv, Hq a multiple of Hkv, Hq <= 1024; D in {64, 128, 256};
 * page_tokens in {32, 64, 128, 256}; num_pages * page_tokens <= 2^40. A call
 * takes up to 2^23 tokens; an attention call's batch * table_width *
 * page_tokens up to 2^35, and fewer than 2^23 workgroups' items (ESHAPE beyond).
 *
 * Every call returns an agemm_status (agemm.h), validates before launching (a
 * failed call launches nothing) and is asynchronous on the given stream (a
 * hipStream_t passed as void*; NULL = the null stream). It runs on the
 * context's device whichever is current. No call but kvc_create allocates,
 * and none synchronises, so all of them can be captured into a graph.
 * Calls of one context may run at the same time on several streams, as long
 * as each kvc_attend in flight has a workspace of its own, and no call reads
 * slots that another one writes. (The error text of kvc_last_error is per
 * context: use one context per host thread.)
 *
 * What only the device can see - page ids, lengths, positions, slots, values
 * - is checked there: the kernels use nothing out of range, leave out what
 * they cannot do, and note it in the context's error word for kvc_check.
 */
#ifndef KVCACHE_H_
#define KVCACHE_H_

#include <stdint.h>

#include "agemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvc_ctx kvc_ctx;

/* Creates a context for one cache shape on the current device. It owns only
 * an error word in pinned host memory; pages and workspaces are the caller's. */
int kvc_create(kvc_ctx** out, int Hq, int Hkv, int D, int page_tokens, int64_t num_pages);

/* Frees the context after synchronising its device. NULL is accepted. */
int kvc_destroy(kvc_ctx* ctx);

/* Bytes of one page: Hkv * page_tokens * (D + 8). */
int kvc_page_bytes(const kvc_ctx* ctx, int64_t* bytes);

/* Arguments of kvc_append. Matrices are binary16, channels contiguous,
 * element (token t, head h, d) at t * token_stride + h * head_stride + d; the
 * strides count elements, are multiples of 8 and may be 0 for inputs (a
 * broadcast row). Matrices, weights and pages 16-byte aligned; index arrays,
 * the rotation table and lse aligned to their elements. */
typedef struct {
  int64_t tokens;              /* T >= 0; 0 does nothing */
  const void* q;               /* T x Hq x D, or NULL: no queries */
  const void* k;               /* T x Hkv x D, or NULL with v: no keys and values */
  const void* v;               /* T x Hkv x D */
  void* q_out;                 /* T x Hq x D; required with q; may be q itself (same strides), else apart
                                  from q, k and v */
  int64_t q_token_stride, q_head_stride;
  int64_t k_token_stride, k_head_stride;
  int64_t v_token_stride, v_head_stride;
  int64_t out_token_stride, out_head_stride; /* rows of q_out must not overlap each other */
  const int64_t* slots;        /* T, device; required with k. A negative slot: the token's key and value
                                  are not kept (padding, or another rank's token) */
  const int64_t* positions;    /* T, device; required with rope */
  const float* rope;           /* rope_len x rope_dims binary32: a row holds rope_dims / 2 cosines, then as
                                  many sines; NULL: no rotation */
  int64_t rope_len;
  int32_t rope_dims;           /* rotated leading channels: a positive multiple of D / 8, <= D */
  int32_t interleaved;         /* 0: channel i pairs with i + rope_dims / 2; 1: 2 i with 2 i + 1 */
  const void* q_norm;          /* D binary16 weights of the RMS norm of each query head; NULL: none */
  const void* k_norm;          /* the same for key heads */
  float eps;                   /* added to the mean square, >= 0 and finite */
} kvc_append_args;

/* For each token: q_out = rope(norm(q)), rounded to binary16 once; the key
 * rope(norm(k)) and the value v go to the token's slot in 4 bits, rounded
 * once. Norm: x_d / sqrt(mean x^2 + eps) * w_d. Rotation of a pair (x, y):
 * (x cos - y sin, y cos + x sin). Sums and products in binary32; what is
 * quantised comes out as if all of it had been worked out in binary64.
 * A key or value channel outside +-20000 is held as that limit, a NaN as 0,
 * and kvc_check reports it: the cache holds finite numbers only, so a token
 * that a query's mask hides cannot reach its result. A position outside
 * 0..rope_len-1 is reported, and the token left out (q_out too); a slot past
 * the last page is reported, and its key and value left out. Two tokens of
 * one call must not name the same slot (that slot's content is then undefined). */
int kvc_append(kvc_ctx* ctx, void* pages, const kvc_append_args* args, void* stream);

/* Arguments of kvc_attend. */
typedef struct {
  int32_t batch;               /* sequences, >= 0 */
  int32_t max_q;               /* upper bound of the queries of one sequence, >= 1 */
  int64_t tokens;              /* rows T of q, out and lse */
  const void* q;               /* T x Hq x D binary16, strides as in kvc_append */
  int64_t q_token_stride, q_head_stride;
  const int32_t* q_start;      /* batch + 1, device: sequence i's queries are rows q_start[i] .. q_start[i+1]-1;
                                  NULL: one query a sequence, row i (batch <= T, max_q = 1) */
  const int32_t* kv_len;       /* batch, device: cached tokens of each sequence, >= 0 */
  const int32_t* q_off;        /* batch, device, or NULL: see below */
  const int32_t* page_table;   /* batch rows of table_width page ids, table_stride apart, device */
  int64_t table_stride;        /* in elements, >= table_width or 0 (a shared row) */
  int32_t table_width;         /* >= 1 */
  int32_t causal;              /* 1: query i of a sequence sees the first q_off + i + 1 of its cached tokens
                                  (no more than kv_len, none if that is <= 0); q_off NULL stands for
                                  kv_len - (its queries): they are the last of the cached tokens.
                                  0: every query sees all kv_len */
  int64_t max_kv;              /* the longest kv_len to expect, >= 1: it only chooses how work is split */
  float scale;                 /* factor of q . k, below 2^127 in size */
  int32_t out_f32;             /* out is binary32 (1) or binary16 (0) */
  void* out;                   /* T x Hq x D, contiguous, apart from q */
  float* lse;                  /* T x Hq, contiguous, or NULL */
} kvc_attend_args;

/* For each query row and head h, over the tokens j it sees, with kv head
 * h / (Hq / Hkv):
 *   S_j = scale * q . K_j,  out = sum_j e^(S_j) V_j / sum_j e^(S_j),
 *   lse = ln sum_j e^(S_j).
 * A row that sees no token: out = 0 and lse = -FLT_MAX, which the combine
 * takes as a partial without weight. Rows of q past the last sequence's are
 * left as they were in out and lse. Scores must be below 2^127 in size (times
 * log2(e) they fit binary32). Sums, maxima and statistics in binary32. The
 * softmax weights enter the product with the values in binary16: with a
 * binary32 out as two numbers, cut, which a weight w is off by at most
 * max(2^-21 w, 2^-36 of the row's largest weight) - over L tokens of tiny
 * weights up to L 2^-36 max |V| in out; with a binary16 out as one, rounded:
 * max(2^-11 w, 2^-37 of the largest). lse has all of every weight.
 * Reported by kvc_check: a page id outside the cache (its tokens count as not
 * seen), a length that is negative or does not fit the table (clamped), a
 * sequence with more than max_q queries, rows past T or a negative number of
 * them (its rows are left; where q_start descends, others' may be too).
 * The order of summation depends on the shapes and lengths alone: equal calls
 * give equal bits. workspace: at least kvc_attend_workspace bytes of bounds that
 * hold this call's batch, max_q and max_kv, 16-byte aligned (NULL if that is
 * 0); its contents before and after mean nothing. */
int kvc_attend(kvc_ctx* ctx, const void* pages, const kvc_attend_args* args, void* workspace,
               int64_t workspace_bytes, void* stream);

/* Workspace that holds every kvc_attend call of up to `batch` sequences, max_q
 * queries and max_kv tokens (any out type): one made for a server's largest
 * batch, chunk and length serves its smaller calls too, which may need more
 * than the largest one does. */
int kvc_attend_workspace(const kvc_ctx* ctx, int32_t batch, int32_t max_q, int64_t max_kv, int64_t* bytes);

/* Copies the keys and values of the tokens in `slots` (T, device) out of the
 * cache as the binary16 numbers they stand for: k_out and v_out T x Hkv x D,
 * contiguous. A negative slot leaves its rows as they were; one past the last
 * page does too, and is reported. */
int kvc_read(kvc_ctx* ctx, const void* pages, int64_t tokens, const int64_t* slots, void* k_out, void* v_out,
             void* stream);

/* AGEMM_EINVAL if a kernel met something it could not use since the last
 * check (the error word is then cleared; kvc_last_error names the last such
 * thing), else AGEMM_OK. Reads host memory: synchronise the streams first. */
int kvc_check(kvc_ctx* ctx);

/* Message of the last failed call on this context ("" if none). */
const char* kvc_last_error(kvc_ctx* ctx);

#ifdef __cplusplus
}
#endif

#endif /* KVCACHE_H_ */
