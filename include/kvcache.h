/*
 * C-ABI of the 4-bit paged key/value cache on one GPU (gfx950): appending to
 * it, attention over it, reading it back; and a step of speculative decoding on
 * it: drafted tokens in a tree, their attention, verification and commit.
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
 * as each kvc_attend, kvc_attend_tree and kvc_verify in flight has a workspace of
 * its own (two that share one mix their partials, sums and counters), and no call
 * reads slots that another one writes. (The error text of kvc_last_error is per
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

/* Workspace that holds every kvc_attend and kvc_attend_tree call of up to `batch` sequences, max_q
 * queries and max_kv tokens (any out type): one made for a server's largest
 * batch, chunk and length serves its smaller calls too, which may need more
 * than the largest one does. (It is the larger of what calls without and with
 * trees need, at most some two times the former.) */
int kvc_attend_workspace(const kvc_ctx* ctx, int32_t batch, int32_t max_q, int64_t max_kv, int64_t* bytes);

/* A step with drafted tokens. The tokens of a sequence's step form a tree of up
 * to 1024 nodes, in an order in which parents come first. Node 0 is the token
 * that the last step decided, whose keys and values are not cached yet; every
 * other node is a draft of the token that follows its parent. The nodes are the
 * rows q_start[i] .. q_start[i + 1] - 1 of sequence i, and node j's key and value
 * lie at place kv_len + j of the sequence until they are committed:
 *   kvc_tree         masks, positions and slots of the nodes;
 *   kvc_append       of the nodes with those, in every layer;
 *   kvc_attend_tree  with the masks, in every layer;
 *   kvc_verify       against the target's probabilities: the accepted path and
 *                    the token that follows it;
 *   kvc_commit       the path's keys and values go to places kv_len, kv_len + 1,
 *                    ..., in all layers; the lengths that the next step starts with.
 * Nothing of it needs the host, so a step can be captured into a graph. Up to
 * 2^20 sequences and 2^23 rows a call. q_start must ascend: where it descends, the
 * sequence with a negative number of rows is reported, and what the outputs hold in
 * rows that two sequences name, before q_start[0] and from q_start[batch] on is not
 * said. */

/* Arguments of kvc_tree. */
typedef struct {
  int32_t batch;               /* sequences, >= 0 */
  int32_t max_q;               /* upper bound of the nodes of one tree, 1 .. 64 mask_words */
  int64_t tokens;              /* rows T of parent and of the outputs but total_len */
  const int32_t* q_start;      /* batch + 1, device: sequence i's nodes are rows q_start[i] .. q_start[i+1]-1 */
  const int32_t* kv_len;       /* batch, device: cached tokens before the tree */
  const int32_t* parent;       /* T, device: the node that a node follows, counted from its sequence's first
                                  row; less than its own number; -1: it follows the cached tokens */
  const int32_t* page_table;   /* batch rows of table_width page ids, table_stride apart; required with slots */
  int64_t table_stride;        /* in elements, >= table_width or 0 (a shared row) */
  int32_t table_width;         /* >= 1 */
  int32_t mask_words;          /* 1 .. 16 */
  uint64_t* mask;              /* T x mask_words, contiguous: bit j % 64 of word j / 64 is node j */
  int64_t* positions;          /* T, or NULL */
  int64_t* slots;              /* T, or NULL */
  int32_t* total_len;          /* batch, or NULL */
} kvc_tree_args;

/* For each node: its mask has itself and its ancestors, its position is kv_len +
 * the number of its ancestors, its slot that of place kv_len + its number in the
 * page table. total_len = kv_len + the sequence's nodes. Rows of no sequence get
 * an empty mask, position 0 and slot -1, so that kvc_append keeps nothing of
 * them. The outputs must lie apart from the inputs and each other.
 * Reported by kvc_check: a parent that is no earlier node (taken as -1); a page
 * id outside the cache (slot -1); a sequence with more than max_q nodes, rows
 * past T or a negative number of them, or whose tree does not fit behind its
 * length (a negative one, or too long for the table): those of its rows that
 * there are count as rows of no sequence, and total_len is kv_len. */
int kvc_tree(kvc_ctx* ctx, const kvc_tree_args* args, void* stream);

/* kvc_attend (causal = 1) with a tree: query i of a sequence sees the first q_off
 * of its cached tokens, and token q_off + j where bit j of row i of `mask` is set
 * (no token past kv_len; q_off NULL stands for kv_len - its queries). mask: T x
 * mask_words (1 .. 16, and max_q up to 64 mask_words, as in kvc_tree), contiguous,
 * device, as kvc_tree leaves it. The queries need not be all of the tree's nodes:
 * with q_off given, those of its last level attend to what is cached of the others. Everything else as in kvc_attend; the
 * workspace too (kvc_attend_workspace). */
int kvc_attend_tree(kvc_ctx* ctx, const void* pages, const kvc_attend_args* args, const uint64_t* mask,
                    int32_t mask_words, void* workspace, int64_t workspace_bytes, void* stream);

/* Arguments of kvc_verify. */
typedef struct {
  int32_t batch;               /* sequences, >= 0 */
  int32_t max_q;               /* upper bound of the nodes of one tree, 1 .. 1024 */
  int64_t tokens;              /* rows T of token, parent, p, q, u and path */
  const int32_t* q_start;      /* batch + 1, device */
  const int32_t* parent;       /* T, device, as in kvc_tree; nodes that do not descend from node 0 are left out */
  const int64_t* token;        /* T, device: the drafted tokens; node 0's is not read */
  const float* p;              /* T x vocab, rows p_stride apart: the target's probabilities of the token that
                                  follows a node */
  const float* q;              /* T x vocab, rows q_stride apart: the draft's, from which a node's children were
                                  drawn one after another without replacement; NULL: the children are certain */
  int64_t p_stride, q_stride;  /* in elements, >= vocab or 0 (a shared row) */
  int64_t vocab;               /* 1 .. 2^28 */
  const float* u;              /* T, device: random numbers in [0, 1), one for each draft; node 0's is for the
                                  token at the end */
  int32_t max_children;        /* the most children of one node to expect, >= 1: it only chooses how work is split.
                                  With q, 1 is for chains: trees get the same results, but one workgroup a sequence
                                  for every sum (16 trees of 25 on 131072 tokens 147 to 476 us, 30 to 63 with what
                                  they have) */
  int32_t* path;               /* T: the accepted nodes, node 0 first, then -1 */
  int32_t* count;              /* batch: their number */
  int64_t* next;               /* batch: the token that follows them */
} kvc_verify_args;

/* Accepts drafts so that the accepted tokens and the one after them are
 * distributed as the target's are. At a node, from node 0 on, its children c are
 * tried in their order. With x = token[c], and for the first child w = p, d = q:
 * c is accepted if u[c] d(x) < w(x), and the walk goes on from it; else w becomes
 * max(0, w - d), normalised, and d loses x and is normalised, by the sum of what is
 * left of the row (only a whole row of p or q counts as a sum of 1). Without q, d is
 * 1 at x and 0 elsewhere for each child. Where no child is accepted (or none is
 * there) the walk ends, and next is the smallest token t with
 *   sum_{s <= t} w(s) > u[node 0] sum_s w(s).
 * A child whose token an earlier one of the same parent had is passed over, and so
 * are those behind children that left w 0 everywhere (next is drawn from p then) or
 * had all of d: 2^-57 of it a token of the vocabulary counts as nothing.
 * In 64 bits; the weights w of the sums as multiples of 2^-50, whose sums are
 * exact below 8 in any order (a token whose weight is 2^-51 or less has none, and
 * is never drawn), and d's in two parts, as a multiple of 2^-50 and the rest as one
 * of 2^-76: equal calls give equal results however they are split. Entries of p, q outside 0..1 count as the nearer end, NaN as 0; so does u,
 * its upper end the largest number below 1.
 * path, count, next and the workspace must lie apart from the inputs (what lies
 * between their rows counts as theirs) and each other.
 * A sequence without rows has count 0 and next -1. Reported by kvc_check: a
 * parent as in kvc_tree (of node 0, anything but -1), a drafted token outside the
 * vocabulary (passed over), a row of p without any weight (next -1), and rows as
 * in kvc_tree (count 0, next -1, path as it was). workspace: at least
 * kvc_verify_workspace bytes of bounds that hold this call's batch and vocab,
 * 16-byte aligned; its contents before and after mean nothing. */
int kvc_verify(kvc_ctx* ctx, const kvc_verify_args* args, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace that holds every kvc_verify call of up to `batch` sequences and `vocab` tokens. */
int kvc_verify_workspace(const kvc_ctx* ctx, int32_t batch, int64_t vocab, int64_t* bytes);

/* Arguments of kvc_commit. */
typedef struct {
  int32_t batch;               /* sequences, >= 0 */
  int32_t max_q;               /* upper bound of the nodes of one tree, 1 .. 1024 */
  int64_t tokens;              /* rows T of path */
  const int32_t* q_start;      /* batch + 1, device */
  const int32_t* kv_len;       /* batch, device: cached tokens before the tree */
  const int32_t* path;         /* T, device: the accepted nodes of a sequence in its first rows, ascending */
  const int32_t* count;        /* batch, device: their number, 0 .. the sequence's nodes */
  const int32_t* page_table;   /* as in kvc_tree; the trees of two sequences share no slot */
  int64_t table_stride;
  int32_t table_width;
  int32_t* new_len;            /* batch, or NULL: kv_len + count; apart from the inputs */
} kvc_commit_args;

/* Moves the key and value of node path[i] of each sequence to place kv_len + i of
 * it, bit for bit, in each of `layers` (0 .. 1024) caches of the context's shape (pages: a
 * host array of as many device pointers, no two of them equal), with the same
 * page table. Other slots stay as they are.
 * Reported by kvc_check, and that sequence left, its new_len kv_len: rows and
 * lengths as in kvc_tree, a count out of its range, a path that is not
 * ascending or leaves the tree. A page id outside the cache is reported, and the
 * nodes on it or bound for it are not moved. */
int kvc_commit(kvc_ctx* ctx, void* const* pages, int32_t layers, const kvc_commit_args* args, void* stream);

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
