// Small shared functions of the key/value cache's kernels and host library as a
// CPU library, for tests/test_kv_units.py. No GPU, no HIP.
#include "kv_checks.h"

using namespace agemm;

extern "C" {

int kvu_blocks(int n) { return kv_blocks(n); }

}  // extern "C"
