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

// Plans of attention with a tree.
static KvPlan tree_plan;
extern "C" {

// rows, many, tiles, items, slots, places, least, most_runs, partials, join_rows, join_groups, join_grid, ws_bytes
void kvt_plan(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv, int f32, int num_cus, int64_t* out) {
  const KvPlan p = tree_plan = kv_tree_plan(kv_layout(Hq, Hkv, D, 64, 1000), batch, max_q, max_kv, f32 != 0, num_cus);
  const int64_t v[13] = {p.rows,      p.many,     p.tiles,     p.items,       p.slots,     p.places,  p.least,
                         p.most_runs, p.partials, p.join_rows, p.join_groups, p.join_grid, p.ws_bytes};
  for (int i = 0; i < 13; ++i) out[i] = v[i];
}
int64_t kvt_bound(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  return kv_tree_bound(kv_layout(Hq, Hkv, D, 64, 1000), batch, max_q, max_kv, num_cus);
}
// With the plan made last: work, partials and items to join of a batch with these blocks and queries, as the kernels
// share it out; its chunk.
int kvt_shared(int Hkv, int batch, const int32_t* blocks, const int32_t* queries, int64_t* work, int64_t* partials, int64_t* joins) {
  const KvPlan& p = tree_plan;
  auto tiles = [&](int b) { return ((int64_t)queries[b] * p.group + p.rows - 1) >> p.row_shift; };
  int64_t U = 0, items = 0;
  int longest = 0;
  for (int b = 0; b < batch; ++b) {
    U += blocks[b] * tiles(b) * Hkv;
    items += tiles(b) * Hkv;
    longest = longest > blocks[b] ? longest : blocks[b];
  }
  int c = batch == 1 ? kv_tree_chunk_of_one(p, (int)items, blocks[0]) : kv_tree_chunk(p, U, longest);
  auto runs = [&](int b) { return tiles(b) * Hkv * kv_tree_runs(c, blocks[b]); };
  if (batch > 1 && batch <= 64 && items <= p.places)
    for (int turn = 0; turn < 4 && c < longest; ++turn) {
      int64_t all = 0;
      for (int b = 0; b < batch; ++b) all += runs(b);
      if (all <= p.places) break;
      c = kv_tree_longer(p, c, (int)all);
    }
  *work = *partials = *joins = 0;
  for (int b = 0; b < batch; ++b) {
    *work += runs(b);
    if (kv_tree_runs(c, blocks[b]) > 1) *partials += runs(b), *joins += tiles(b) * Hkv;
  }
  return c;
}

}  // extern "C"
