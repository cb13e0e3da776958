// The key/value cache's argument checks and page layout as a CPU library: the
// host library's and the kernels' own headers behind C entries, for
// tests/test_kv_host.py. No GPU, no HIP.
#include "kv_checks.h"

using namespace agemm;

extern "C" {

int kvh_create(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages) {
  return kv_check_create(Hq, Hkv, D, page_tokens, num_pages);
}

int kvh_append(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages, const void* pages, const kvc_append_args* p,
               char* why) {
  return kv_check_append(kv_layout(Hq, Hkv, D, page_tokens, num_pages), pages, p, why);
}

int kvh_attend(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages, const void* pages, const kvc_attend_args* p,
               int64_t need, const void* workspace, int64_t workspace_bytes, char* why) {
  const KvLayout L = kv_layout(Hq, Hkv, D, page_tokens, num_pages);
  KvPlan plan{};
  if (p && p->batch >= 0 && p->max_q >= 1 && p->max_kv >= 1) plan = kv_attend_plan(L, p->batch, p->max_q, p->max_kv, 256);
  plan.ws_bytes = need;
  return kv_check_attend(L, pages, p, plan, workspace, workspace_bytes, why);
}

int kvh_read(const void* pages, int64_t tokens, const int64_t* slots, const void* k_out, const void* v_out, char* why) {
  return kv_check_read(pages, tokens, slots, k_out, v_out, why);
}

// Byte of the block of `slot` and kv head h, and the token's places in it.
int64_t kvh_block(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages, int64_t slot, int h, int* token,
                  int* quarter, int* place) {
  const KvLayout L = kv_layout(Hq, Hkv, D, page_tokens, num_pages);
  const int off = (int)(slot & (L.page_tokens - 1));
  *token = off & 31;
  *quarter = kv_value_quarter(*token);
  *place = kv_value_place(*token);
  return kv_block_at(L, slot >> L.page_shift, h, off >> 5);
}

// The work plan: many, rows, join_rows, join_groups, tiles, splits, chunk, items, slots, slot_floats, ws_bytes.
static KvPlan plan_of;
void kvh_plan(int Hq, int Hkv, int D, int page_tokens, int64_t num_pages, int64_t batch, int64_t max_q, int64_t max_kv,
              int num_cus, int64_t* out) {
  const KvPlan p = kv_attend_plan(kv_layout(Hq, Hkv, D, page_tokens, num_pages), batch, max_q, max_kv, num_cus);
  plan_of = p;
  const int64_t v[11] = {p.many, p.rows, p.join_rows, p.join_groups, p.tiles, p.splits, p.chunk, p.items,
                         p.slots, p.slot_floats, p.ws_bytes};
  for (int i = 0; i < 11; ++i) out[i] = v[i];
}
// Items of the launch of the plan that kvh_plan made last, widened if it can be; its rows and tiles.
int64_t kvh_many_items(int Hq, int Hkv, int D, int64_t batch, int64_t max_q, int64_t max_kv,
                       int64_t tokens, int num_cus, int64_t* rows, int64_t* tiles) {
  KvPlan p = plan_of;
  const KvLayout L = kv_layout(Hq, Hkv, D, 64, 1000);
  kv_many_wide(p, L, batch, max_q, max_kv, tokens, num_cus);
  *rows = p.rows;
  *tiles = p.tiles;
  return kv_many_items(p, L, batch, tokens);
}
// Blocks of a run in the plan that kvh_plan made last.
int kvh_chunk(int64_t U, int longest) { return kv_chunk(plan_of, U, longest); }
int kvh_item_runs(int chunk, int nblk) { return kv_item_runs(chunk, nblk); }
int kvh_run_blocks(int chunk, int splits, int nblk) { return kv_run_blocks(chunk, splits, nblk); }
int kvh_runs(int chunk, int splits, int nblk) { return kv_runs(chunk, splits, nblk); }

int64_t kvh_piece(int Hq, int Hkv, int D, int read) {
  const KvLayout L = kv_layout(Hq, Hkv, D, 64, 1000);
  return read ? kv_read_piece(L) : kv_append_piece(L);
}

}  // extern "C"
