// Workspace bounds with and without trees as a CPU library, for
// tests/test_kv_tree_bounds.py. No GPU, no HIP.
#include "kv_checks.h"

using namespace agemm;

extern "C" {

int64_t kvb_plain(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  return kv_attend_bound(kv_layout(Hq, Hkv, D, 64, 1000), batch, max_q, max_kv, num_cus);
}
int64_t kvb_tree(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  return kv_tree_bound(kv_layout(Hq, Hkv, D, 64, 1000), batch, max_q, max_kv, num_cus);
}

}  // extern "C"
