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
  int32_t group, row_shift;  // with a tree: query heads of a kv head, log2(rows),
  int32_t join_grid;         // workgroups of the join (join_rows: of a wave; 0: one row a workgroup),
  int32_t most_runs;         // of an item,
  int64_t partials;          // partials that the workspace holds
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

// With a tree: blocks of a run, from the batch's real lengths. U blocks in all
// items, `longest` in one: `places` runs and a remainder of each item, none
// shorter than the least, no item of more runs than it has partials for. (Items of
// several runs, which have more than c blocks, then have 2 U / c <= 2 places runs.)
KV_HD inline int kv_quotient_up(int x, int d) { return (int)(((uint32_t)x + (uint32_t)d - 1) / (uint32_t)d); }
KV_HD inline int kv_tree_runs(int chunk, int nblk) { return nblk <= chunk ? 1 : kv_quotient_up(nblk, chunk); }
KV_HD inline int kv_tree_chunk(const KvPlan& p, int64_t U, int longest) {
  const int64_t many = U >> 31 ? (U + p.places - 1) / p.places : kv_quotient_up((int)U, p.places);
  const int c = (int)(many < kKvWhole ? many : kKvWhole);
  const int joined = kv_quotient_up(longest, p.most_runs);
  const int least = p.least > joined ? p.least : joined;
  return c < least ? least : c;
}
// A single sequence's, of `per` items: no more runs than run at once.
KV_HD inline int kv_tree_chunk_of_one(const KvPlan& p, int per, int nblk) {
  const int c = kv_tree_chunk(p, (int64_t)nblk * per, nblk);
  if (per == 0 || per > p.places) return c;
  const int even = kv_quotient_up(nblk, (int)((uint32_t)p.places / (uint32_t)per));
  return c > even ? c : even;
}
// The next try where `runs` runs of c blocks are more than run at once.
KV_HD inline int kv_tree_longer(const KvPlan& p, int c, int runs) {
  return c + 1 + (int)((float)c * (float)(runs - p.places) / (float)runs);
}

// A call with a tree. Its items are (sequence, tile of rows, kv head), whose rows
// all see nearly all of the sequence. Five forms take them: the kernel for few
// rows with tiles of 16, 32 or 64 rows, the one for many with 128 or 256. The
// former start fast and need no barrier, and the more rows unpack a block once
// the better; the latter unpack it once for four or eight waves. Which is faster
// follows from the work of a place (a workgroup that runs at once with others), by
// a model fitted to measured shapes with 8 kv heads (1 to 32 sequences of 200 to 32000
// tokens, equally long, 24 to 512 rows a kv head, binary16 outputs):
//   us = first + round max(1, items / places) + (block + full F) B + J (join + runs N / places)
// with B the blocks of a place, F the part of a tile's rows that exist, J whether
// items of several runs are joined, N the runs. Its choice takes 1.03 times the
// best form's time on average (1.4 at worst). Outside that range, on 23 shapes of 1
// to 20 kv heads, 60 to 8192 tokens and both outputs, 1.04 times (at worst 1.32: 24
// trees of 25 on 4099 tokens, 32 heads on 4, D 64, 70 us in tiles of 128 rows, 54 in
// tiles of 32; and 1.22: 4 of 16 on 4000, 16 on 1, D 128, binary32 out, 20 for 16).
// In us, of D 128, tiles of 16, 32, 64, 128 and 256 rows:
//   8 sequences of 500 tokens,    64 rows     9.8   12.2   16.0   19.5   17.4
//   8 of 16000,                   64         87.7   70.1   61.4   88.7   99.0
//   32 of 2000,                   64         47.7   48.2   37.7   53.1   55.3
//   8 of 16000,                  104          150    114   95.2    102    107
//   32 of 2000,                  200          131    145    125   89.1   80.0
//   8 of 16000,                  384                 324           311    261
// and of D 256, tiles of 16, 32 and 128:
//   8 of 500,                    104         23.3   17.5          39.2
//   8 of 8000,                   104          152    105           136
//   32 of 500,                   200          140    106          83.0
// A binary32 output of D 128 does not fit 64 rows' registers (8 of 16000, 64 rows:
// 85.9 us spilling, 76.0 with 32).
struct KvForm {
  int rows, places_per_cu, blocks;  // blocks: of a sequence that is one run for sure
  double first, round, block, full, join, runs;
};
inline int kv_tree_forms(int D, const KvForm** forms) {
  static const KvForm d64[] = {{16, 2, 64, 3.1, 3.4, .149, 0, 2.5, 7.0}, {32, 1, 32, 5.8, 1.8, .120, 0, 5.0, 0},
                               {64, 1, 32, 1.6, 7.4, .213, 0, 4.1, 2.9}, {128, 2, 32, 0, 5.2, .563, .186, 4.8, 12.7}};
  static const KvForm d128[] = {{16, 2, 64, 1.0, 4.6, .249, 0, .8, 12.8}, {32, 1, 32, 2.1, 6.3, .208, 0, 4.2, 2.7},
                                {64, 1, 32, 1.1, 9.7, .318, 0, 2.9, 5.6}, {128, 2, 32, 0, 4.8, .868, .342, 5.7, 19.6},
                                {256, 1, 32, 0, 8.5, .519, .555, 4.4, 15.6}};
  static const KvForm d256[] = {{16, 1, 64, 2.8, 6.1, .270, 0, 5.1, 4.0}, {32, 1, 32, 2.1, 8.9, .359, 0, 3.0, 6.2},
                                {128, 1, 32, 0, 12.6, 1.51, .186, 3.7, 16.3}};
  *forms = D == 64 ? d64 : D == 128 ? d128 : d256;
  return D == 64 ? 4 : D == 128 ? 5 : 3;
}
// The shortest run: four blocks a wave make up for what a run costs beside its
// blocks; a tile for many rows has large partials, and short runs only where few
// items leave most of the chip idle (64 rows x 8 heads of 2000 tokens, runs of 8
// blocks or more 27.8 us, 16 29.2, 32 39.3; 384 rows x 64 heads of 1000 46.8, 46.5,
// and 37.4 in one run).
inline int kv_tree_least(int rows, int64_t items, int64_t places) { return rows < 128 ? 32 : items * 8 <= places ? 8 : 16; }

// Runs of an item at most, and partials that items of several runs leave: such an
// item has more than c blocks, so that there are fewer than U / c <= places of them,
// and their runs, each less than its blocks / c + 1, are fewer than twice that.
inline int64_t kv_tree_most_runs(int64_t nblk, int64_t least) {
  const int64_t runs = (nblk + least - 1) / least;
  return runs < kKvMaxSplits ? runs : kKvMaxSplits;
}
inline int64_t kv_tree_partials(int64_t items, int64_t runs, int64_t places) {
  const int64_t most = places + (items < places ? items : places);
  return items < most && items * runs < most ? items * runs : most;
}

inline KvPlan kv_tree_plan_as(const KvForm& f, const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  KvPlan p{};
  const int64_t rows = max_q * (L.Hq / L.Hkv), nblk = kv_expected_blocks(max_kv);
  p.rows = f.rows;
  p.many = p.rows >= 128;
  p.group = L.Hq / L.Hkv;
  p.row_shift = __builtin_ctz((unsigned)p.rows);
  p.tiles = (int32_t)((rows + p.rows - 1) / p.rows);
  p.items = batch * L.Hkv * p.tiles;
  p.slot_floats = (int64_t)p.rows * (L.D + 2);
  p.splits = 1;
  p.slots = p.items;
  p.places = num_cus * f.places_per_cu;
  p.least = kv_tree_least(p.rows, p.items, p.places);
  // (So many items need no more runs, and their grid stays below 2^32 threads.)
  if (p.items == 0 || p.items > 1 << 22 || batch > kKvMaxBatch || nblk <= f.blocks) return p;
  p.slots = p.items + p.places;
  p.most_runs = (int32_t)kv_tree_most_runs(nblk, p.least);
  p.partials = kv_tree_partials(p.items, p.most_runs, p.places);
  const int64_t live = rows < p.rows ? rows : p.rows, joins = p.items < p.places ? p.items : p.places;
  // The join: a workgroup a row for few rows, some rows a wave for many.
  p.join_rows = joins * live <= 2 * num_cus ? 0 : 256 / L.D;
  p.join_groups = (int32_t)(p.join_rows ? (live + p.join_rows - 1) / p.join_rows : live);
  const int64_t grid = p.join_rows ? (joins * p.join_groups + 3) / 4 : joins * live;
  p.join_grid = (int32_t)(grid < 4 * num_cus ? grid : 4 * num_cus);
  p.ws_bytes = p.partials * p.slot_floats * 4 + 16 + joins * 32;
  return p;
}
inline double kv_tree_us(const KvForm& f, const KvPlan& p, int64_t rows, int64_t nblk) {
  const double per_place = (double)p.items / p.places;
  const bool split = p.slots > p.items;
  double chain = (double)(split && nblk > p.least ? p.least : nblk);
  if (per_place * nblk > chain) chain = per_place * nblk;
  double runs = chain > 0 ? per_place * nblk / chain : 0;
  if (runs < per_place) runs = per_place;
  const double fill = (double)rows / ((double)p.tiles * p.rows);
  return f.first + f.round * (per_place > 1 ? per_place : 1) + (f.block + f.full * fill) * chain +
         (split ? f.join + f.runs * (runs < 1 ? runs : 1) * fill : 0);
}
inline KvPlan kv_tree_plan(const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, bool out_f32, int num_cus) {
  const KvForm* forms;
  const int n = kv_tree_forms(L.D, &forms);
  const int64_t rows = max_q * (L.Hq / L.Hkv), nblk = kv_expected_blocks(max_kv);
  KvPlan best{};
  double least = 0;
  for (int i = 0; i < n; ++i) {
    if (forms[i].rows >= 128 && rows <= 32) break;  // their partials would be the most of a decoder's workspace
    if (forms[i].rows == 64 && (rows <= 32 || (L.D == 128 && out_f32))) continue;
    const KvPlan p = kv_tree_plan_as(forms[i], L, batch, max_q, max_kv, num_cus);
    const double us = kv_tree_us(forms[i], p, rows, nblk);
    if (i == 0 || us < least) best = p, least = us;
  }
  return best;
}
// Workspace bytes for every call with a tree within these bounds: each form's need grows with each of them.
inline int64_t kv_tree_bound(const KvLayout& L, int64_t batch, int64_t max_q, int64_t max_kv, int num_cus) {
  const KvForm* forms;
  const int n = kv_tree_forms(L.D, &forms);
  const int64_t rows = max_q * (L.Hq / L.Hkv), nblk = kv_expected_blocks(max_kv);
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) {
    const KvForm& f = forms[i];
    if (f.rows >= 128 && rows <= 32) break;
    if (nblk <= f.blocks || (f.rows == 64 && rows <= 32)) continue;
    const int64_t some = batch < kKvMaxBatch ? batch : kKvMaxBatch, places = (int64_t)num_cus * f.places_per_cu;
    const int64_t items = some * L.Hkv * ((rows + f.rows - 1) / f.rows);
    const int64_t need = kv_tree_partials(items, kv_tree_most_runs(nblk, f.rows < 128 ? 32 : 8), places) * f.rows * (L.D + 2) * 4 + 16 +
                         (items < places ? items : places) * 32;
    bytes = bytes > need ? bytes : need;
  }
  return bytes;
}

constexpr int kKvNodes = 1024;       // of one tree
constexpr int kKvMaskWords = kKvNodes / 64;
constexpr int kKvLayers = 64;        // of one launch of the commit

// Layers of one launch of the commit, a wave for each (layer, sequence, kv head).
inline int kv_commit_piece(const KvLayout& L, int64_t batch) {
  const int64_t fits = (int64_t{1} << 25) / (batch * L.Hkv);
  return (int)(fits < 1 ? 1 : fits < kKvLayers ? fits : kKvLayers);
}

// How a verification's rows of probabilities are summed: in `parts` parts of
// `part` tokens each, one workgroup a part; with rounds, again and again as the
// walk asks for sums, else once, for the last draw.
struct KvVerifyPlan {
  int32_t parts, part, rounds;
};
constexpr int kKvParts = 64;   // at most
constexpr int kKvStateBytes = 128;  // of a sequence: how far it has come, parts that are summed
inline int64_t kv_verify_parts(int64_t batch, int64_t vocab, int num_cus) {
  // Four workgroups a CU, of 2048 tokens at the least and, as far as 64 parts hold
  // the vocabulary so, 16384 at the most (the draw looks through a quarter of a part).
  int64_t parts = (4 * num_cus + batch - 1) / (batch > 0 ? batch : 1), most = (vocab + 2047) / 2048;
  const int64_t least = (vocab + 16383) / 16384;
  parts = parts > least ? parts : least;
  parts = parts < most ? parts : most;
  return parts < kKvParts ? parts : kKvParts;
}
inline KvVerifyPlan kv_verify_plan(int64_t batch, int64_t vocab, bool drawn, int64_t max_children, int num_cus) {
  KvVerifyPlan p{};
  int64_t parts = kv_verify_parts(batch, vocab, num_cus);
  const int64_t fits = (int64_t{1} << 23) / (batch > 0 ? batch : 1);  // grids stay below 2^32 threads
  parts = parts < fits ? parts : fits;
  const int64_t part = ((vocab + parts - 1) / parts + 1023) / 1024 * 1024;
  p.part = (int32_t)part;
  p.parts = (int32_t)((vocab + part - 1) / part);
  p.rounds = drawn && max_children > 1;
  return p;
}
constexpr int kKvSums = 3;  // of a segment, a quarter of a part: the weights, and q in two parts
constexpr int kKvPartBytes = 4 * kKvSums * 8;
inline int64_t kv_verify_bytes(const KvVerifyPlan& p, int64_t batch) { return batch * ((int64_t)p.parts * kKvPartBytes + kKvStateBytes); }
// Bytes for every verification of up to `batch` sequences and `vocab` tokens.
inline int64_t kv_verify_bound(int64_t batch, int64_t vocab, int num_cus) {
  const int64_t most = (vocab + 2047) / 2048 < kKvParts ? (vocab + 2047) / 2048 : kKvParts, all = batch * most;
  const int64_t some = batch * ((vocab + 16383) / 16384 + 1) + 4 * num_cus;
  return (some < all ? some : all) * kKvPartBytes + batch * kKvStateBytes;
}

}  // namespace agemm
