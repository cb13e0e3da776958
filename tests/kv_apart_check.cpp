// Checks that outputs of calls with trees lie apart from what the kernels read, as
// a CPU library for tests/test_kv_tree_refusals.py. No GPU, no HIP.
#include "kv_checks.h"

using namespace agemm;

extern "C" {

int kva_tree(const kvc_tree_args* p, char* why) { return kv_check_tree_apart(p, why); }
int kva_verify(const kvc_verify_args* p, const void* ws, int64_t need, char* why) { return kv_check_verify_apart(p, ws, need, why); }
int kva_commit(const kvc_commit_args* p, char* why) { return kv_check_commit_apart(p, why); }

}  // extern "C"
