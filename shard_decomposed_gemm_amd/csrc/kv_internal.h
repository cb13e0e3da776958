// Internal interface between the key/value cache's C-ABI host code (kvc.cpp)
// and its gfx950 kernels (kv_append.hip, kv_attend.hip).
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
  KvPlan plan;
  float* ws;  // plan.ws_bytes of partials
  uint64_t* err;  // kv_report.h
};

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
