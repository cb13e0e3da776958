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

// How one attention call's work is laid out. Rows of a kv head's item are its
// query heads of all queries, r = query * G + head. Each item's blocks of 32
// tokens go in runs of `chunk` to `splits` workgroups at most (longer runs
// where a sequence has more blocks than that); the partials of an item with
// several runs meet in the workspace, one slot per (item, run).
struct KvPlan {
  int32_t many;    // 0: the kernel for few rows, 1: for many
  int32_t rows;    // rows of one item
  int32_t join_rows, join_groups;  // the join: rows of a workgroup (a power of two), workgroups of an item
  int32_t tiles;   // items of one sequence and kv head
  int32_t splits;
  int32_t chunk;   // blocks of a run
  int64_t items;
  int64_t slot_floats;  // of one partial: rows x D, then rows x (exponent, sum)
  int64_t ws_bytes;
};

constexpr int kKvMaxSplits = 256;
constexpr int kKvWaves = 8;  // of a workgroup for few rows: each takes every eighth block of a run

// Blocks that a run of an item with nblk blocks has, and the runs.
KV_HD inline int kv_run_blocks(int chunk, int splits, int nblk) {
  const int need = (nblk + splits - 1) / splits;
  return need > chunk ? need : chunk;
}
KV_HD inline int kv_runs(int chunk, int splits, int nblk) {
  const int c = kv_run_blocks(chunk, splits, nblk);
  return nblk <= c ? 1 : (nblk + c - 1) / c;
}

inline KvPlan kv_attend_plan(const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  KvPlan p;
  const int64_t rows = max_q * (L.Hq / L.Hkv);
  p.many = rows > (L.D == 256 ? 16 : 32);
  p.rows = p.many ? 128 : rows > 16 ? 32 : 16;
  p.tiles = (int32_t)(p.many ? (rows + p.rows - 1) / p.rows : 1);
  p.items = batch * L.Hkv * p.tiles;
  const int64_t nblk = (max_kv + 31) / 32;
  int64_t chunk;
  if (p.many) {
    const int64_t places = (int64_t)num_cus * 4;
    chunk = (p.items * nblk + places - 1) / places;
    if (chunk < 32) chunk = 32;
  } else if (nblk <= 4 * kKvWaves) {
    chunk = nblk;  // four blocks a wave are done before a join would be
  } else {
    // As many runs as run at once, but none so long that the last of them
    // keep the chip waiting: the more items, the longer they may be.
    const int64_t places = (int64_t)num_cus * (L.D == 256 || p.rows == 32 ? 1 : 2);
    chunk = (p.items * nblk + places - 1) / places;
    if (chunk < kKvWaves) chunk = kKvWaves;
    const int64_t most = 16 * kKvWaves * ((p.items + places - 1) / places);
    if (chunk > most) chunk = most;
  }
  int64_t splits = (nblk + chunk - 1) / chunk;
  if (splits < 1) splits = 1;
  if (splits > kKvMaxSplits) {
    splits = kKvMaxSplits;
    chunk = (nblk + splits - 1) / splits;
  }
  p.chunk = (int32_t)(chunk < (int64_t{1} << 26) ? chunk : int64_t{1} << 26);
  p.splits = (int32_t)splits;
  const int64_t live = rows < p.rows ? rows : p.rows;  // rows of an item that can exist
  p.join_rows = p.items * live <= 2 * num_cus ? 1 : 2048 / L.D;
  p.join_groups = (int32_t)((live + p.join_rows - 1) / p.join_rows);
  p.slot_floats = (int64_t)p.rows * (L.D + 2);
  p.ws_bytes = p.splits > 1 ? p.items * p.splits * p.slot_floats * 4 : 0;
  return p;
}

}  // namespace agemm
