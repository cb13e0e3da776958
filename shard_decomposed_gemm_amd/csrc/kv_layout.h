// Page layout of the 4-bit key/value cache (described in kvcache.h), shared by
// the kernels and the host library. No HIP dependency: a CPU check compiles it
// as it is.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define KV_HD __host__ __device__
#else
#define KV_HD
#endif

namespace agemm {

struct KvLayout {
  int32_t Hq, Hkv, D, page_tokens;
  int32_t page_shift;  // log2(page_tokens)
  int64_t num_pages;
  int64_t page_bytes;
};

// Block of 32 tokens of one kv head.
KV_HD inline int64_t kv_block_bytes(int D) { return 32 * (D + 8); }
// Byte of the block that holds tokens [32 i, 32 i + 32) of head h of a page.
KV_HD inline int64_t kv_block_at(const KvLayout& L, int64_t page, int h, int i) {
  return page * L.page_bytes + ((int64_t)h * (L.page_tokens >> 5) + i) * kv_block_bytes(L.D);
}
// Place of token t of a block among the eight of its quarter (value order).
KV_HD inline int kv_value_quarter(int t) { return (t >> 2) & 3; }
KV_HD inline int kv_value_place(int t) { return ((t >> 4) << 2) | (t & 3); }

}  // namespace agemm
