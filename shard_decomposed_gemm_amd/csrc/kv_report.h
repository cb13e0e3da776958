// What the key/value cache's kernels report for kvc_check: one 64-bit word in
// pinned host memory, written by one store, so that the reports of workgroups
// that write at the same time cannot mix. No HIP dependency: a CPU check
// compiles it as it is.
#pragma once

#include <stddef.h>
#include <stdio.h>

#include "kv_layout.h"

namespace agemm {

enum KvErr : uint32_t {  // 0: nothing; the value that a report holds
  kKvSlot = 1,      // slot past the last page
  kKvPosition = 2,  // position outside the rotation table
  kKvValue = 3,     // key or value not finite or beyond the limit: its kv head
  kKvPage = 4,      // page id outside the cache
  kKvLength = 5,    // length negative or beyond the page table
  kKvRows = 6,      // query rows beyond max_q or T, or not ascending: their number
};

// Case in bits 60..63, index of the token or sequence (a call has up to 2^23)
// in 36..59, value in 0..35, signed; a value beyond that is held at the end.
constexpr int64_t kKvMostSeen = (int64_t{1} << 35) - 1;
KV_HD inline uint64_t kv_report_word(uint32_t code, int64_t index, int64_t seen) {
  const int64_t v = seen > kKvMostSeen ? kKvMostSeen : seen < -kKvMostSeen - 1 ? -kKvMostSeen - 1 : seen;
  return (uint64_t)code << 60 | ((uint64_t)index & 0xffffff) << 36 | ((uint64_t)v & 0xfffffffffull);
}

// The message of a report, of a cache of `slots` slots and `pages` pages.
inline void kv_report_text(char* buf, size_t size, uint64_t word, int64_t slots, int64_t pages) {
  const unsigned code = (unsigned)(word >> 60), at = (unsigned)(word >> 36) & 0xffffff;
  const long long v = (long long)(word << 28) >> 28;
  const char* end = v == kKvMostSeen ? "from " : v == -kKvMostSeen - 1 ? "up to " : "";
  switch (code) {
    case kKvSlot: snprintf(buf, size, "token %u: slot %s%lld past the last page (%lld slots)", at, end, v, (long long)slots); break;
    case kKvPosition: snprintf(buf, size, "token %u: position %s%lld outside the rotation table", at, end, v); break;
    case kKvValue: snprintf(buf, size, "token %u: a key or value of kv head %lld not finite or beyond the limit", at, v); break;
    case kKvPage: snprintf(buf, size, "sequence %u: page id %lld outside the cache (%lld pages)", at, v, (long long)pages); break;
    case kKvLength: snprintf(buf, size, "sequence %u: length %lld negative or beyond its page table", at, v); break;
    case kKvRows: snprintf(buf, size, "sequence %u: %lld query rows, more than max_q, less than 0 or outside q", at, v); break;
    default: snprintf(buf, size, "unknown case %u", code);
  }
}

}  // namespace agemm
