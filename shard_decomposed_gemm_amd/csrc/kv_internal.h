// Internal interface between the key/value cache's C-ABI host code (kvc.cpp)
// and its gfx950 kernels (kv_append.hip, kv_attend.hip, kv_tree.hip, kv_verify.hip).
#pragma once

#include "agemm_internal.h"
#include "kv_layout.h"
#include "kv_report.h"

namespace agemm {

constexpr float kKvLimit = 20000.f;  // |x| held: (16 + n) s + b and b = -3.14 |x| at worst stay in binary16

struct KvAppendArgs {
  KvLayout L;
  char* pages;
  int64_t tokens;
  const _Float16 *q, *k, *v;
  _Float16* q_out;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
  const int64_t* slots;
  const int64_t* positions;
  const float* rope;
  int64_t rope_len;
  int32_t rope_dims, interleaved;
  const _Float16 *q_norm, *k_norm;
  float eps;
  int64_t first;  // number of the call's token that is token 0 here
  uint32_t quads, near;  // quads of a wave, workgroups of 32 tokens (the launch fills them in)
  uint64_t* err;  // kv_report.h
};

struct KvReadArgs {
  KvLayout L;
  const char* pages;
  int64_t tokens;
  const int64_t* slots;
  _Float16 *k_out, *v_out;
  int64_t first;  // number of the call's token that is token 0 here
  uint64_t* err;  // kv_report.h
};

struct KvAttendArgs {
  KvLayout L;
  const char* pages;
  int32_t batch, max_q;
  int64_t tokens;
  const _Float16* q;
  int64_t q_ts, q_hs;
  const int32_t *q_start, *kv_len, *q_off, *table;
  int64_t table_stride;
  int32_t table_width, causal;
  float scale;
  void* out;
  float* lse;
  const uint64_t* tree;  // masks of a tree's nodes, tree_words a row of q, or NULL
  int32_t tree_words;
  KvPlan plan;
  float* ws;  // plan.ws_bytes of partials
  int32_t* joins;  // with a tree, behind the partials: the number of KvJoin, and from 16 bytes on they themselves
  uint64_t* err;  // kv_report.h
};

// Rows of an item of several runs, for the join.
struct KvJoin {
  int64_t row0;        // its sequence's first row of q
  int32_t h, r0;       // kv head, first row of the head's
  int32_t rows, runs;  // rows of the head
  int32_t slot, step;  // the first run's partial, and from one run's to the next
};

struct KvTreeArgs {
  KvLayout L;
  int32_t batch, max_q;
  int64_t tokens;
  const int32_t *q_start, *kv_len, *parent, *table;
  int64_t table_stride;
  int32_t table_width, words;
  uint64_t* mask;
  int64_t *positions, *slots;
  int32_t* total_len;
  uint64_t* err;  // kv_report.h
};

// How far a sequence's verification has come (kv_verify.hip says what A, Z and D are).
struct KvWalk {
  double A, Z, D;
  double coarse, fine;     // D in two parts; as long as the row's sum is not known, less that
  int32_t node, last;      // where it is, the child tried last
  int32_t count, rejects;  // accepted nodes, tokens rejected at the last of them (without q)
  int32_t pending, wants;  // Z and D are out of date; the walk needs it to go on (else it has ended)
  int32_t done, known;     // known: q's sum of the row is in D's parts
};
// A line of its own: workgroups of all XCDs count in it.
struct KvVerifyState {
  KvWalk walk;
  uint32_t arrived;  // parts that are summed, over all rounds
  uint32_t turn;     // rounds after which the walk has gone on
  uint8_t rest[kKvStateBytes - sizeof(KvWalk) - 8];
};
static_assert(sizeof(KvVerifyState) == kKvStateBytes, "the workspace's bound counts them");

struct KvVerifyArgs {
  int32_t batch, max_q;
  int64_t tokens;
  const int32_t *q_start, *parent;
  const int64_t* token;
  const float *p, *q;
  int64_t p_stride, q_stride;
  int32_t vocab;
  const float* u;
  int32_t *path, *count;
  int64_t* next;
  KvVerifyPlan plan;
  KvVerifyState* states;  // batch
  double* sums;           // batch x kKvSums x segments of all parts
  int64_t patience;       // ticks of the wall clock that a workgroup of the rounds waits for the others
  uint64_t* err;  // kv_report.h
};

struct KvCommitArgs {
  KvLayout L;
  char* pages[kKvLayers];
  int32_t batch, layers;
  int32_t max_q;
  int64_t tokens;
  const int32_t *q_start, *kv_len, *path, *count, *table;
  int64_t table_stride;
  int32_t table_width;
  int32_t* new_len;
  uint64_t* err;  // kv_report.h
};

hipError_t launch_kv_tree(const KvTreeArgs& a, hipStream_t s);
hipError_t launch_kv_verify(const KvVerifyArgs& a, hipStream_t s);
hipError_t launch_kv_commit(const KvCommitArgs& a, hipStream_t s);
hipError_t launch_kv_append(const KvAppendArgs& a, int num_cus, hipStream_t s);
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s);
hipError_t launch_kv_attend(const KvAttendArgs& a, bool out_f32, hipStream_t s);

#ifdef __HIPCC__
// Launches and gives this launch's own status (hipGetLastError would give any
// earlier failure of the thread).
template <class A>
hipError_t kv_launch(void (*kernel)(A), dim3 grid, unsigned threads, hipStream_t s, A a) {
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, 0, s);
}

__device__ inline void kv_report(uint64_t* err, uint32_t code, int64_t index, int64_t seen) {
  __hip_atomic_store(err, kv_report_word(code, index, seen), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
}
#endif

}  // namespace agemm
