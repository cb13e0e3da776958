// Small shared functions of the key/value cache's kernels and host library as a
// CPU library, for tests/test_kv_units.py. No GPU, no HIP.
#include "kv_checks.h"

using namespace agemm;

extern "C" {

int kvu_blocks(int n) { return kv_blocks(n); }

// Workspace bytes that kvc_attend_workspace gives, and that kvc_attend asks for.
int64_t kvu_workspace(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  return kv_attend_bound(kv_layout(Hq, Hkv, D, 64, 1000), batch, max_q, max_kv, num_cus);
}
int64_t kvu_needs(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  return kv_attend_plan(kv_layout(Hq, Hkv, D, 64, 1000), batch, max_q, max_kv, num_cus).ws_bytes;
}

}  // extern "C"
