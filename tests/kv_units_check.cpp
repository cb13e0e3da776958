// Small shared functions of the key/value cache's kernels and host library as a
// CPU library, for tests/test_kv_units.py. No GPU, no HIP.
#include "kv_checks.h"
#include "kv_report.h"

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

// The message of a report of these.
void kvu_report(uint32_t code, int64_t index, int64_t seen, int64_t slots, int64_t pages, char* buf) {
  kv_report_text(buf, kKvWhy, kv_report_word(code, index, seen), slots, pages);
}

}  // extern "C"
