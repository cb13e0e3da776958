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
// Blocks of 32 tokens that n >= 0 tokens take (n + 31 passes 2^31 for the longest lengths).
KV_HD inline int kv_blocks(int n) { return (int)(((uint32_t)n + 31u) >> 5); }
// Place of token t of a block among the eight of its quarter (value order).
KV_HD inline int kv_value_quarter(int t) { return (t >> 2) & 3; }
KV_HD inline int kv_value_place(int t) { return ((t >> 4) << 2) | (t & 3); }

// Tokens of one launch of the append and of the read: grids stay below 2^32
// threads, and the append's quads of rows below 2^28.
inline int64_t kv_append_piece(const KvLayout& L) {
  const int64_t quads = (L.Hq + 3) / 4 > (L.Hkv + 3) / 4 * 2 ? (L.Hq + 3) / 4 : (L.Hkv + 3) / 4 * 2;
  return ((int64_t{1} << 28) - 64) / quads;
}
inline int64_t kv_read_piece(const KvLayout& L) { return ((int64_t{1} << 28) - 64) / L.Hkv; }

// How one attention call's work is laid out. Rows of a kv head's item are its
// query heads of all queries, r = query * G + head.
//
// Few rows (many = 0): an item is a (sequence, kv head). Its blocks of 32
// tokens go in runs of equal length, chosen on the device from the lengths of
// the whole batch (kv_chunk), sequence by sequence, within one run by run and
// head by head; a workgroup takes one run, and run i of the call leaves its
// partial in slot i. With slots == items every item is one run.
//
// Many rows (many = 1): an item is a (sequence, tile of 128 or 256 rows, kv head);
// its blocks go in runs of `chunk` to `splits` workgroups at most (longer runs
// where a sequence has more blocks than that), one slot per (item, run).
struct KvPlan {
  int32_t many;
  int32_t rows;    // rows of one item
  int32_t join_rows, join_groups;  // the join: rows of a workgroup (a power of two), workgroups of an item
  int32_t tiles;   // items of one sequence and kv head
  int32_t splits, chunk;   // many rows
  int32_t places, least, most;  // few rows: workgroups that run at once, the shortest and the longest run
  int64_t items, slots;    // slots: few rows, the call's runs at most
  int64_t slot_floats;     // of one partial: rows x D, then rows x (exponent, sum)
  int64_t ws_bytes;
};

constexpr int kKvMaxSplits = 256;
constexpr int kKvMaxBatch = 512;  // sequences whose lengths every workgroup looks through
constexpr int kKvWaves = 8;  // of a workgroup for few rows: each takes every eighth block of a run
constexpr int kKvWhole = 1 << 26;  // blocks of the longest sequence

// Few rows: blocks of a run for U blocks in all, `longest` in one item: as many
// runs as run at once, but none so long that the last of them keep the chip
// waiting, no more runs than slots (each item has less than one that is not
// full), and no more of an item than the join takes.
KV_HD inline int kv_chunk(const KvPlan& p, int64_t U, int longest) {
  if (p.slots <= p.items) return kKvWhole;
  int64_t c = (U + p.places - 1) / p.places;
  c = c < p.least ? p.least : c < p.most ? c : p.most;
  const int64_t fits = (U + p.slots - p.items - 1) / (p.slots - p.items);
  c = c > fits ? c : fits;
  const int64_t joined = ((int64_t)longest + kKvMaxSplits - 1) / kKvMaxSplits;
  c = c > joined ? c : joined;
  return (int)(c < kKvWhole ? c : kKvWhole);
}
// Few rows: runs of an item of nblk blocks (an item whose rows see nothing has one).
KV_HD inline int kv_item_runs(int chunk, int nblk) { return nblk <= chunk ? 1 : (nblk + chunk - 1) / chunk; }

// Many rows: blocks that a run of an item with nblk blocks has, and the runs.
KV_HD inline int kv_run_blocks(int chunk, int splits, int nblk) {
  const int need = (nblk + splits - 1) / splits;
  return need > chunk ? need : chunk;
}
KV_HD inline int kv_runs(int chunk, int splits, int nblk) {
  const int c = kv_run_blocks(chunk, splits, nblk);
  return nblk <= c ? 1 : (nblk + c - 1) / c;
}

// Blocks of a sequence of max_kv tokens, or of the longest there can be.
inline int64_t kv_expected_blocks(int64_t max_kv) {
  return max_kv < (int64_t)kKvWhole * 32 ? (max_kv + 31) / 32 : kKvWhole;
}

inline KvPlan kv_attend_plan(const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  KvPlan p{};
  const int64_t rows = max_q * (L.Hq / L.Hkv), nblk = kv_expected_blocks(max_kv);
  // As many rows as the kernel for few rows holds, it takes: 16 x 4 queries of 64
  // heads (8 kv heads, D 128) on 8192 tokens 44 us, the one for many 82; 16 x 2
  // of 16 heads (2, D 256) 26, 77. Rows above that fill a third of a 128-row tile
  // at first: 5 such queries take 82 us, 8 85, 16 111; of D 256 3 take 76, 8 90.
  // A form between the two would be for them.
  p.many = rows > (L.D == 256 ? 16 : 32);
  p.rows = p.many ? 128 : rows > 16 ? 32 : 16;
  p.tiles = (int32_t)(p.many ? (rows + p.rows - 1) / p.rows : 1);
  p.items = batch * L.Hkv * p.tiles;
  const int64_t live = rows < p.rows ? rows : p.rows;  // rows of an item that can exist
  p.join_rows = p.items * live <= 2 * num_cus ? 1 : 2048 / L.D;
  p.join_groups = (int32_t)((live + p.join_rows - 1) / p.join_rows);
  p.slot_floats = (int64_t)p.rows * (L.D + 2);
  p.splits = 1;
  p.slots = p.items;
  if (p.items == 0) return p;  // an empty batch
  if (p.many) {
    // As many runs as run at once, of equal length. A run's partial takes a
    // round through memory and the join a launch: in short runs only where
    // items leave CUs idle. In us, 32 heads, 8 kv heads, D 128:
    //   least run, blocks                     8    16    32   128  whole
    //   40 queries on 1000 tokens          19.5  25.7  31.8  31.6   31.7
    //   64 on 4096                         24.7  28.0  39.5   105    105
    //   4 x 40 on 16384                     106   105   106   131    403
    //   1777 on themselves (448 items)     74.1  73.7  73.4  59.8   57.6
    //   1024 on 16384 (256 items)           351   349   345   355    437
    const int64_t places = (int64_t)num_cus * 2, least = p.items >= num_cus ? 128 : 8;
    int64_t chunk = p.items < places ? (p.items * nblk + places - 1) / places : nblk;
    if (chunk < least) chunk = least;
    int64_t splits = (nblk + chunk - 1) / chunk;
    if (splits > kKvMaxSplits) splits = kKvMaxSplits;
    if (splits < 1) splits = 1;
    chunk = (nblk + splits - 1) / splits;
    p.chunk = (int32_t)(chunk < kKvWhole ? chunk : kKvWhole);
    p.splits = (int32_t)splits;
    p.ws_bytes = p.splits > 1 ? p.items * p.splits * p.slot_floats * 4 : 0;
  } else {
    p.places = num_cus * (L.D == 256 || p.rows == 32 ? 1 : 2);
    // One run an item: up to four blocks a wave are done before a join would
    // be, and where there are items enough anyway, longer ones too.
    if (nblk <= 4 * kKvWaves || batch > kKvMaxBatch || (p.items >= 2 * p.places && nblk * p.places <= 64 * p.items)) return p;
    // A run costs some 8 us beside its blocks (lengths, first loads, the
    // waves' join). A single sequence leaves most of the chip idle for them;
    // in a batch, four blocks a wave make up for it.
    p.least = batch > 1 ? 4 * kKvWaves : kKvWaves;
    const int64_t most = 16 * kKvWaves * ((p.items + p.places - 1) / p.places);  // the more items, the longer
    p.most = (int32_t)(most < kKvWhole ? most : kKvWhole);
    int64_t runs = (p.items * nblk + p.most - 1) / p.most;
    if (runs > 64 * p.places) runs = 64 * p.places;
    p.slots = p.items + (runs > p.places ? runs : p.places);
    p.ws_bytes = p.slots * p.slot_floats * 4;
  }
  return p;
}

// Workspace bytes that suffice for every call of up to `batch` sequences, max_q
// queries and max_kv tokens. (The plan's own need is not monotone: calls with
// fewer items have more runs an item, calls with many none.) Few rows: an item
// count that still splits, and the most runs that kv_attend_plan gives as many
// items or fewer. Many rows: splits > 1 takes items x nblk <= places x (nblk - 1),
// and then items x splits < places + items.
inline int64_t kv_attend_bound(const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  const int64_t G = L.Hq / L.Hkv, nblk = kv_expected_blocks(max_kv);
  const int few = L.D == 256 ? 16 : 32;  // rows of the kernel for few
  auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
  auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
  int64_t floats = 0;
  for (int rows = 16; rows <= few; rows *= 2) {
    const int64_t q = rows == 16 ? 1 : 16 / G + 1;  // the fewest queries of this form
    if (q > max_q || q * G > rows || nblk <= 4 * kKvWaves) continue;
    const int64_t places = (int64_t)num_cus * (L.D == 256 || rows == 32 ? 1 : 2);
    const int64_t items = least(least(batch, kKvMaxBatch) * L.Hkv, most(2 * places, (nblk * places + 63) / 64) - 1);
    if (items < L.Hkv) continue;
    const int64_t runs = least((least(items, places) * nblk + 16 * kKvWaves - 1) / (16 * kKvWaves), 64 * places);
    floats = most(floats, (items + most(runs, places)) * rows * (L.D + 2));
  }
  const int64_t places = (int64_t)num_cus * 2;
  const int64_t items = least(batch * L.Hkv * ((max_q * G + 127) / 128), (nblk - 1) * places / nblk);
  if (max_q * G > few && items >= L.Hkv && nblk > 8)
    floats = most(floats, least(places + items - 1, items * least(kKvMaxSplits, (nblk + 7) / 8)) * 128 * (L.D + 2));
  return floats * 4;
}

// Many rows: items that a call with `tokens` rows of q can have.
inline int64_t kv_many_items(const KvPlan& p, const KvLayout& L, int64_t batch, int64_t tokens) {
  if (batch == 1 || batch > kKvMaxBatch) return p.items;
  const int64_t items = (tokens * (L.Hq / L.Hkv) / p.rows + batch) * L.Hkv;
  return items < p.items ? items : p.items;
}

// Many rows, nothing to join: tiles of 256 rows (kv_attend.hip says why) where
// the rows still make four items a CU, of 64 blocks or more at the longest. 2 x
// 2048 queries on 8192 tokens (64 heads, 8 kv heads): 1085 us, in 128 rows 1190;
// 4 x 4096 on themselves (32, 8): 679, 714; but 64 x 256: 169, 128. With two items
// a CU, 1 x 4096 on itself, 256 rows would take 173, 128 take 197: the limit of
// four is on the safe side.
inline void kv_many_wide(KvPlan& p, const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, int64_t tokens,
                         int num_cus) {
  if (!p.many || p.splits > 1 || L.D != 128 || max_kv < 64 * 32) return;
  KvPlan w = p;
  w.rows = 256;
  w.tiles = (int32_t)((max_q * (L.Hq / L.Hkv) + 255) / 256);
  w.items = batch * L.Hkv * w.tiles;
  if (kv_many_items(w, L, batch, tokens) >= 4 * num_cus) p = w;
}

}  // namespace agemm
