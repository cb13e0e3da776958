// The argument checks, plans and reports of the calls with trees as a CPU
// library, for tests/test_kv_tree_host.py. No GPU, no HIP.
#include "kv_checks.h"
#include "kv_report.h"

using namespace agemm;

extern "C" {

int kvt_mask(const kvc_attend_args* p, const uint64_t* mask, int32_t words, char* why) { return kv_check_mask(p, mask, words, why); }
int kvt_tree(const kvc_tree_args* p, char* why) { return kv_check_tree(p, why); }
int kvt_verify(const kvc_verify_args* p, int64_t need, const void* ws, int64_t bytes, char* why) {
  return kv_check_verify(p, need, ws, bytes, why);
}
int kvt_commit(int Hkv, void* const* pages, int32_t layers, const kvc_commit_args* p, char* why) {
  return kv_check_commit(kv_layout(Hkv, Hkv, 64, 32, 10), pages, layers, p, why);
}
int kvt_commit_piece(int Hkv, int64_t batch) { return kv_commit_piece(kv_layout(Hkv, Hkv, 64, 32, 10), batch); }
// parts, part, rounds
void kvt_verify_plan(int64_t batch, int64_t vocab, int drawn, int64_t children, int num_cus, int32_t* out) {
  const KvVerifyPlan p = kv_verify_plan(batch, vocab, drawn != 0, children, num_cus);
  out[0] = p.parts;
  out[1] = p.part;
  out[2] = p.rounds;
}
int64_t kvt_verify_bound(int64_t batch, int64_t vocab, int num_cus) { return kv_verify_bound(batch, vocab, num_cus); }
void kvt_report(uint32_t code, int64_t index, int64_t seen, char* text) { kv_report_text(text, 256, kv_report_word(code, index, seen), 640, 10); }

}  // extern "C"
