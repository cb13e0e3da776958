// Attention over the 4-bit paged cache on gfx950.
//
// The products run on the matrix units in binary16 with binary32 sums, keys
// and values as the binary16 numbers that their nibbles stand for, and
// transposed: S^T = K Q^T has keys as rows and queries as columns, so that a
// lane holds one query's scores for a few keys, and O^T = V^T P^T takes the
// weights P^T from the very registers that the scores came in. The matrix
// instructions ask for the operand of a product over keys with eight
// consecutive inner indices a lane; as the order of the inner index is free
// when both operands share it, the eight keys of a lane are those whose scores
// it holds, and the cache stores values in that order (kvcache.h). No lane
// exchanges data for the products.
//
// A nibble n becomes (16 + n) by an OR: n in bits 6..9 of a binary16 number
// with exponent 4. One packed multiply-add with (s, b) makes two channels'
// values: 3 operations for two.
//
// The running maximum m of the softmax is replaced only when a score passes it
// by 2^3: weights are kept as 2^(x - m + 12) (x the score in units of log 2),
// at most 2^15, so the usual block needs no maximum across lanes and no
// rescaling. The largest weight is at least 2^12 (short of scores of 2^26, base_of);
// binary16 has multiples of 2^-24 at the least, 2^-36 of that.
//
// With binary16 outputs a weight enters the product rounded to binary16 once
// (off by 2^-11 of it, as the output itself is, or half of 2^-24): a second
// number would be as many matrix instructions again for a bit that the output
// does not hold. Against 64 bits outputs are off by 2.4 to 2.9e-4 (norms),
// one rounding of them alone by 2.1e-4. With binary32 outputs it enters as two
// numbers, its value cut to binary16 and the rest cut again: off by less than
// 2^-21 of it or 2^-24, whichever is more. Cut, because one instruction cuts
// two numbers. The sum of the weights takes them whole.
#include <type_traits>

#include "kv_internal.h"

namespace agemm {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

constexpr float kLowest = -3.402823466e+38f;  // lse of a row that sees nothing
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kNoMax = -3.0e38f;  // exponent base before the first score
constexpr float kShift = 12.f;      // weights are 2^(x - m + kShift)
constexpr float kTop = 15.f;        // and at most 2^kTop
constexpr float kFar = 0x1p24f;     // from here on binary32 holds no fractions of an exponent

__device__ inline float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// The exponent base of a largest score `top`: kShift less, or top itself where
// binary32 would make more than kTop of that.
__device__ inline float base_of(float top) {
  const float b = top - kShift;
  return top - b > kTop ? top : b;
}
// Where a base is so large that binary32 holds no fractions of it, the product
// of a score and the factor is rounded before the base is taken off, so that
// equal scores have equal weights: a multiply-add, which has the exact product,
// would give each block's whatever the base's rounding leaves. Every block then
// goes the way of a new maximum.
__device__ inline bool is_far(float base) { return fabsf(base) >= kFar && base > kNoMax; }
__device__ inline float less_base(float rounded, float base) {
  asm("" : "+v"(rounded));  // no multiply-add
  return rounded - base;
}

// The constants that make (16 + n) of a nibble, in registers: with both as
// literals the compiler takes an AND and an OR, with registers one instruction.
struct Bits {
  uint32_t mask = 0x03C003C0u, exponent = 0x4C004C00u;
  __device__ Bits() {
    asm("" : "+s"(mask));
    asm("" : "+v"(exponent));
  }
};

// Two of a word's nibbles, j and j + 4, as (16 + n).
template <int j>
__device__ inline half2v sixteen_plus(const Bits& c, uint32_t w) {
  uint32_t x;
  if constexpr (j == 0) x = w << 6;
  else if constexpr (j == 1) x = w << 2;
  else if constexpr (j == 2) x = w >> 2;
  else x = w >> 6;
  return __builtin_bit_cast(half2v, (x & c.mask) | c.exponent);
}

// The largest of eight (fmaxf would first quiet every operand).
__device__ inline float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ inline float max8(const float* e) {
  return max3(max3(max3(e[0], e[1], e[2]), e[3], e[4]), max3(e[5], e[6], e[7]), e[7]);
}

// (Taken by value: of an element of a vector, __builtin_bit_cast reads a wrong one.)
__device__ inline half2v halves(uint32_t w) { return __builtin_bit_cast(half2v, w); }

__device__ inline half8v join4(half2v a, half2v b, half2v c, half2v d) {
  return half8v{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Eight channels of one key from a word of its row: channels 0 4 1 5 2 6 3 7.
__device__ inline half8v key_operand(const Bits& c, uint32_t w, half2v s, half2v b) {
  return join4(__builtin_elementwise_fma(sixteen_plus<0>(c, w), s, b), __builtin_elementwise_fma(sixteen_plus<1>(c, w), s, b),
               __builtin_elementwise_fma(sixteen_plus<2>(c, w), s, b), __builtin_elementwise_fma(sixteen_plus<3>(c, w), s, b));
}

// One channel (nibble j of the 16-bit words) of eight tokens; s and b of the tokens in pairs.
template <int j>
__device__ inline half8v value_operand(const Bits& c, uint4v w, const half2v (&s)[4], const half2v (&b)[4]) {
  return join4(__builtin_elementwise_fma(sixteen_plus<j>(c, w.x), s[0], b[0]),
               __builtin_elementwise_fma(sixteen_plus<j>(c, w.y), s[1], b[1]),
               __builtin_elementwise_fma(sixteen_plus<j>(c, w.z), s[2], b[2]),
               __builtin_elementwise_fma(sixteen_plus<j>(c, w.w), s[3], b[3]));
}

// A query's eight channels in the order of key_operand.
__device__ inline half8v query_operand(const _Float16* q) {
  const half8v v = *reinterpret_cast<const half8v*>(q);
  return half8v{v[0], v[4], v[1], v[5], v[2], v[6], v[3], v[7]};
}

// Weights p0 and p1 as elements i and i + 1 of the binary16 operand hi, with
// what the cut loses in lo (F32), or rounded (without lo).
template <bool F32>
__device__ inline void split_weight(float p0, float p1, half8v& hi, half8v& lo, int i) {
  if constexpr (F32) {
    const auto c = __builtin_amdgcn_cvt_pkrtz(p0, p1);
    hi[i] = (_Float16)c[0];
    hi[i + 1] = (_Float16)c[1];
    const uint32_t w = __builtin_bit_cast(uint32_t, c);
    float r0, r1;  // p0 and p1 less the halves of w, one instruction each
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r0) : "v"(w), "v"(p0));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r1) : "v"(w), "v"(p1));
    const auto d = __builtin_amdgcn_cvt_pkrtz(r0, r1);
    lo[i] = (_Float16)d[0];
    lo[i + 1] = (_Float16)d[1];
  } else {
    hi[i] = (_Float16)p0;
    hi[i + 1] = (_Float16)p1;
  }
}

// A sequence's rows and lengths, checked against what the call gave.
struct Sequence {
  int64_t row0;  // its first row of q
  int n;         // its queries, 0 if they cannot be used
  int len;       // cached tokens
  int64_t off;   // the first query sees off + 1 tokens
  int least;     // with a tree: its nodes less one, which are the most that any query sees beyond off; else 0

  __device__ int below_tree() const { return off < 0 ? 0 : off > len ? len : (int)off; }  // seen by every query
  __device__ int blocks() const { return n > 0 ? kv_blocks(seen(n - 1)) : 0; }  // that its last query sees
  __device__ int seen(int i) const {  // with a tree: at most
    const int64_t v = off + (i > least ? i : least) + 1;
    return v < 0 ? 0 : v > len ? len : (int)v;
  }
};

// A value that is the same in all lanes, kept in scalar registers.
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline int64_t uniform(int64_t x) {
  const uint64_t lo = (uint32_t)uniform((int)x), hi = (uint32_t)uniform((int)(x >> 32));
  return (int64_t)(hi << 32 | lo);
}
// Element i of an array that no kernel writes meanwhile, by a scalar load: its
// wait holds up none of the vector loads under way.
__device__ inline int scalar_load(const int32_t* p, int64_t i) {
  typedef const int32_t __attribute__((address_space(4))) * constant;
  return ((constant)(uintptr_t)p)[i];
}

// b the same in all lanes, or (EACH) one sequence a lane.
template <bool EACH = false>
__device__ inline Sequence sequence(const KvAttendArgs& a, int b, bool tell) {
  auto load = [](const int32_t* p, int64_t i) { return EACH ? p[i] : scalar_load(p, i); };
  Sequence s;
  int start = b, end = b + 1;
  if (a.q_start) {
    start = load(a.q_start, b);
    end = load(a.q_start, b + 1);
  }
  const int len = load(a.kv_len, b);
  const int64_t n = (int64_t)end - start;
  s.off = !a.causal ? (int64_t)1 << 32 : a.q_off ? (int64_t)load(a.q_off, b) : 0;
  const bool usable = n >= 0 && n <= a.max_q && start >= 0 && end <= a.tokens;
  if (!usable && tell) kv_report(a.err, kKvRows, b, n);
  s.n = usable ? (int)n : 0;
  s.row0 = start;
  const int64_t most = (int64_t)a.table_width << a.L.page_shift;
  const bool fits = len >= 0 && len <= most;
  if (!fits && tell) kv_report(a.err, kKvLength, b, len);
  s.len = len < 0 ? 0 : len <= most ? len : (int)most;
  if (a.causal && !a.q_off) s.off = (int64_t)s.len - n;
  s.least = a.tree ? 64 * a.tree_words - 1 : 0;
  return s;
}

// The tree's nodes that a row sees: the first 64 in registers, which is all for
// most trees, the others where they are asked for.
struct TreeRow {
  const uint32_t* mask;
  uint32_t m0, m1;
};
__device__ inline TreeRow tree_row(const KvAttendArgs& a, int64_t row) {
  TreeRow t;
  t.mask = reinterpret_cast<const uint32_t*>(a.tree) + row * (2 * a.tree_words);
  t.m0 = t.mask[0];
  t.m1 = t.mask[1];
  return t;
}
// Bit i: the row sees token first + i. first the same in all lanes; ones below
// the tree, zeros past the sequence's end.
__device__ inline uint32_t tree_seen(const KvAttendArgs& a, const TreeRow& t, const Sequence& s, int first) {
  const int64_t rel = first - s.off;
  const int left = s.len - first;
  if (left <= 0 || rel >= 64 * a.tree_words) return 0;
  uint32_t v = ~0u;
  if (rel > -32) {
    const int i = (int)(rel >> 5);
    uint32_t lo, hi;
    if (i < 1) {
      lo = i < 0 ? ~0u : t.m0;
      hi = i < 0 ? t.m0 : t.m1;
    } else {
      lo = t.mask[i];
      hi = i + 1 < 2 * a.tree_words ? t.mask[i + 1] : 0u;
    }
    v = (uint32_t)(((uint64_t)hi << 32 | lo) >> (rel & 31));
  }
  return left < 32 ? v & ((1u << left) - 1) : v;
}

// Sum of x over this lane and the earlier ones.
__device__ inline int sum_up_to(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);  // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);  // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);  // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return x;
}

// The largest x of this lane and the earlier ones (x >= 0).
__device__ inline int largest_up_to(int x) {
  auto with = [&](int y) { x = x > y ? x : y; };
  with(__builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
  return x;
}

// The sequence that lane l holds, in all lanes.
__device__ inline Sequence of_lane(const Sequence& s, int l) {
  auto wide = [&](int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), l) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)x, l));
  };
  Sequence r;
  r.row0 = wide(s.row0);
  r.n = __builtin_amdgcn_readlane(s.n, l);
  r.len = __builtin_amdgcn_readlane(s.len, l);
  r.off = wide(s.off);
  r.least = __builtin_amdgcn_readlane(s.least, l);
  return r;
}

// Few rows: the runs of a call, from its lengths. Every wave works them out
// for itself, 64 sequences at a time (kKvMaxBatch bounds them).
struct Runs {
  int chunk;     // blocks of a run
  int b;         // the sequence found, -1: none
  int64_t slot;  // its first run
  Sequence seq;
};
// The sequence with run `run`, or (run < 0) sequence b. Blocks of a head and
// runs of a head each sum up to at most 2^31 (the host sees to that).
__device__ inline Runs find_runs(const KvAttendArgs& a, int64_t run, int b, int lane, bool tell) {
  auto load = [&](int b0, bool report) {
    Sequence s{};
    if (b0 + lane < a.batch) s = sequence<true>(a, b0 + lane, report);
    return s;
  };
  const Sequence group0 = load(0, tell);
  const int first = group0.blocks();
  int all = __builtin_amdgcn_readlane(sum_up_to(first), 63), longest = __builtin_amdgcn_readlane(largest_up_to(first), 63);
  for (int b0 = 64; b0 < a.batch; b0 += 64) {
    const int x = load(b0, tell).blocks(), top = __builtin_amdgcn_readlane(largest_up_to(x), 63);
    all += __builtin_amdgcn_readlane(sum_up_to(x), 63);
    longest = longest > top ? longest : top;
  }
  const int chunk = kv_chunk(a.plan, (int64_t)all * a.L.Hkv, longest);
  int before = 0;  // runs of a head before this group of sequences
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Sequence s = b0 == 0 ? group0 : load(b0, false);
    const int mine = s.n > 0 ? kv_item_runs(chunk, s.blocks()) : 0;
    const int upto = before + sum_up_to(mine);
    const uint64_t at = run < 0 ? (b - b0 < 64 ? uint64_t{1} << (b - b0) : 0) : __ballot((int64_t)upto * a.L.Hkv > run);
    if (at) {
      const int l = __builtin_ctzll(at);
      return {chunk, b0 + l, (int64_t)(__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(mine, l)) * a.L.Hkv,
              of_lane(s, l)};
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return {chunk, -1, 0, Sequence{}};
}

// With a tree: the work of a call, (sequence, tile of its rows, kv head, run of
// its blocks), kv heads innermost, so that the tiles of a head go to one XCD and
// share its cache, then tiles, then runs. Runs are of the whole batch's lengths as
// for few rows; only items of several runs leave partials. b < 0: none.
struct Work {
  int b, tile, h, run;
  int chunk, runs;  // blocks of a run, runs of the item
  int per;          // items of the sequence
  int slot, join;   // the sequence's first partial and first item of several runs
  Sequence seq;
};
__device__ inline int tiles_of(const KvAttendArgs& a, const Sequence& s) {
  return (int)(((int64_t)s.n * a.plan.group + a.plan.rows - 1) >> a.plan.row_shift);
}
// Work `at` of the call, for a wave. Where runs are joined, the wave with work 0 of
// several sequences leaves the number of items to join.
__device__ inline Work find_work(const KvAttendArgs& a, int at, int lane, bool tell) {
  Work w;
  w.slot = w.join = 0;
  auto split = [&](int rest) {  // `rest`: work of the sequence
    w.run = (int)((uint32_t)rest / (uint32_t)w.per);
    const int r = rest - w.run * w.per;
    w.tile = (int)((uint32_t)r / (uint32_t)a.L.Hkv);
    w.h = r - w.tile * a.L.Hkv;
  };
  if (a.plan.slots <= a.plan.items) {  // one run an item
    w.per = a.plan.tiles * a.L.Hkv;
    w.b = (int)((uint32_t)at / (uint32_t)w.per);
    split(at - w.b * w.per);
    w.chunk = kKvWhole;
    w.runs = 1;
    w.seq = sequence(a, w.b, tell && w.tile == 0 && w.h == 0);
    return w;
  }
  if (a.batch == 1) {
    w.seq = sequence(a, 0, tell && at == 0);
    const int nblk = w.seq.blocks();
    w.per = tiles_of(a, w.seq) * a.L.Hkv;
    w.chunk = kv_tree_chunk_of_one(a.plan, w.per, nblk);
    w.runs = kv_tree_runs(w.chunk, nblk);
    w.b = at < w.per * w.runs ? 0 : -1;
    if (w.b == 0) split(at);
    return w;
  }
  auto load = [&](int b0, bool report) {
    Sequence s{};
    if (b0 + lane < a.batch) s = sequence<true>(a, b0 + lane, report);
    return s;
  };
  auto sum = [](int x) { return __builtin_amdgcn_readlane(sum_up_to(x), 63); };
  auto wide_sum = [&](int64_t x) { return ((int64_t)sum((int)(x >> 20)) << 20) + sum((int)(x & 0xfffff)); };
  const Sequence group0 = load(0, tell && at == 0);
  int64_t all = 0;
  int items = 0, longest = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Sequence s = b0 == 0 ? group0 : load(b0, tell && at == 0);
    const int x = s.blocks(), n = tiles_of(a, s), top = __builtin_amdgcn_readlane(largest_up_to(x), 63);
    all += wide_sum((int64_t)x * n);
    items += sum(n);
    longest = longest > top ? longest : top;
  }
  w.chunk = kv_tree_chunk(a.plan, all * a.L.Hkv, longest);
  if (a.batch <= 64 && items * a.L.Hkv <= a.plan.places) {
    // Remainders make more runs than run at once: longer ones, until they fit or nearly so.
    const int x = group0.blocks(), n = tiles_of(a, group0);
    for (int turn = 0; turn < 4 && w.chunk < longest; ++turn) {
      const int runs = sum(kv_tree_runs(w.chunk, x) * n) * a.L.Hkv;
      if (runs <= a.plan.places) break;
      w.chunk = kv_tree_longer(a.plan, w.chunk, runs);
    }
  }
  int before = 0, slots = 0, joins = 0;  // of a head, of the groups of sequences before
  w.b = -1;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Sequence s = b0 == 0 ? group0 : load(b0, false);
    const int runs = kv_tree_runs(w.chunk, s.blocks()), tiles = tiles_of(a, s), mine = runs * tiles;
    const int left = runs > 1 ? mine : 0, join = runs > 1 ? tiles : 0;
    const int to_mine = sum_up_to(mine), to_left = sum_up_to(left), to_join = sum_up_to(join);
    const uint64_t has = __ballot((before + to_mine) * a.L.Hkv > at);
    if (has && w.b < 0) {
      const int l = __builtin_ctzll(has);
      w.b = b0 + l;
      w.seq = of_lane(s, l);
      w.runs = __builtin_amdgcn_readlane(runs, l);
      w.per = __builtin_amdgcn_readlane(tiles, l) * a.L.Hkv;
      w.slot = (slots + __builtin_amdgcn_readlane(to_left - left, l)) * a.L.Hkv;
      w.join = (joins + __builtin_amdgcn_readlane(to_join - join, l)) * a.L.Hkv;
      split(at - (before + __builtin_amdgcn_readlane(to_mine - mine, l)) * a.L.Hkv);
      if (at > 0) return w;
    }
    before += __builtin_amdgcn_readlane(to_mine, 63);
    slots += __builtin_amdgcn_readlane(to_left, 63);
    joins += __builtin_amdgcn_readlane(to_join, 63);
  }
  if (at == 0 && tell && lane == 0) *a.joins = joins * a.L.Hkv;
  return w;
}
// The partial of a run, and (its first run's first wave) what there is to join.
__device__ inline int64_t partial_of(const KvAttendArgs& a, const Work& w, bool tell) {
  const int i = w.tile * a.L.Hkv + w.h;
  if (w.runs > 1 && w.run == 0 && tell && a.batch > 1)
    reinterpret_cast<KvJoin*>(a.joins + 4)[w.join + i] =
        KvJoin{w.seq.row0, w.h, w.tile << a.plan.row_shift, w.seq.n * a.plan.group, w.runs, w.slot + i, w.per};
  return w.slot + (int64_t)w.run * w.per + i;
}

// Many rows: the tile (sequence, tile of its rows) that is k-th of the call's,
// the last ones of all sequences first: those see the most keys. Every wave
// works it out for itself, from tiles that each lane holds of up to eight
// sequences. With more sequences than that, tiles that no sequence has are
// counted too. b < 0: none.
struct Tile {
  int b, tile;
};
__device__ inline Tile find_tile(const KvAttendArgs& a, int k, int lane, bool tell) {
  if (a.batch == 1 || a.batch > kKvMaxBatch) return {k % a.batch, a.plan.tiles - 1 - k / a.batch};
  constexpr int N = kKvMaxBatch / 64;
  const int G = a.L.Hq / a.L.Hkv;
  int tiles[N];
#pragma unroll
  for (int g = 0; g < N; ++g) {
    tiles[g] = 0;
    if (64 * g < a.batch && 64 * g + lane < a.batch)
      tiles[g] = (int)(((int64_t)sequence<true>(a, 64 * g + lane, tell).n * G + a.plan.rows - 1) / a.plan.rows);
  }
  auto from = [&](int t) {  // tiles of number t and later ones
    int n = 0;
#pragma unroll
    for (int g = 0; g < N; ++g) n += tiles[g] > t ? tiles[g] - t : 0;
    return __builtin_amdgcn_readlane(sum_up_to(n), 63);
  };
  if (from(0) <= k) return {-1, 0};
  int lo = 0, hi = a.plan.tiles;  // from(lo) > k >= from(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (from(mid) > k) lo = mid;
    else hi = mid;
  }
  int rank = k - from(hi);
#pragma unroll
  for (int g = 0; g < N; ++g) {
    const uint64_t has = __ballot(tiles[g] > lo);
    const int n = __builtin_popcountll(has);
    if (rank < n) {
      const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(has >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)has, 0));
      return {64 * g + (int)__builtin_ctzll(__ballot(tiles[g] > lo && before == rank)), lo};
    }
    rank -= n;
  }
  return {-1, 0};  // not reached
}

// Page id of block j of a sequence with `end` blocks to take, one at least (past them: some page id).
__device__ inline int page_of(const KvAttendArgs& a, int b, int j, int end) {
  return scalar_load(a.table, (int64_t)b * a.table_stride + ((j < end ? j : end - 1) >> (a.L.page_shift - 5)));
}
// Byte of block j on page `page`. `lost` keeps the last page id that is not in
// the cache, for a report after the loop (a store inside it would make every
// turn wait for all loads).
struct Lost {
  int page = 0;
  bool any = false;
};
__device__ inline int64_t block_on(const KvAttendArgs& a, int page, int h, int j, bool& there, Lost& lost) {
  there = page >= 0 && page < a.L.num_pages;
  if (!there) {
    lost.page = page;
    lost.any = true;
    page = 0;
  }
  return kv_block_at(a.L, page, h, j & ((a.L.page_tokens >> 5) - 1));
}
__device__ inline void report_lost(const KvAttendArgs& a, int b, const Lost& lost) {
  if (lost.any) kv_report(a.err, kKvPage, b, lost.page);
}

// Writes one row's channels d0 .. d0 + N - 1 of a finished output.
template <bool F32, int N>
__device__ inline void store_out(void* out, int64_t at, const float (&v)[N]) {
  if constexpr (F32) {
    float4v* p = reinterpret_cast<float4v*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) p[i] = float4v{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  } else {
    struct alignas(N * 2) H {
      _Float16 x[N];
    } h;
#pragma unroll
    for (int i = 0; i < N; ++i) h.x[i] = (_Float16)v[i];
    *reinterpret_cast<H*>(static_cast<_Float16*>(out) + at) = h;
  }
}

// ---------------------------------------------------------------- few rows

// For at most 16 NT rows a kv head (single tokens, drafts): HBM-bound, each
// cached byte read once. A workgroup takes a run of an item's blocks; its waves
// take every kWaves-th block each, with no barrier, and join their sums at the
// end. A wave holds all rows of the item as the 16 columns of its products (NT
// times), and a block of 32 keys as two tiles of 16. The next block's keys are
// loaded when this block's are used up, its values likewise, so that two
// workgroups a CU keep some 140 KB in flight. A block costs a wave some 260
// vector and 32 matrix instructions (D 128).
//
// Measured, this kernel alone: 262144 tokens of 8 kv heads (D 128, 12 rows) in
// 52 us, 5.5 TB/s of 7.14 that a plain read reaches; 32768 tokens of 96 kv
// heads (one row) in 72 us, 5.9 TB/s; 777 tokens, 8.2 us, all of it latency.
// The rest of each workgroup is lengths, page ids and first loads (3 to 6 us,
// one after the other) and the waves' join (3 us). A ragged batch (64 sequences
// up to 8192 tokens, 36 us for 18 of bytes) waits for its last runs: vector units
// are busy 43 % of the cycles, matrix units 7 %.
//
// With a tree an item is a tile of 16 NT rows of a sequence's head, and any number
// of rows comes here while the call is small. Unpacking a block is then shared by
// all of the tile's rows; softmax is not. A block takes a workgroup of D 128, as
// fitted to measured times, 0.25 us (16 rows, two workgroups a CU), 0.21 (32, one)
// or 0.32 (64, one): the taller tile does more rows for less.
constexpr int kWaves = kKvWaves;

template <int D>
struct RawKeys {  // a block's keys as a lane reads them
  uint32_t w[2][D / 32];
  half2v pair[2];
};
template <int D>
struct RawValues {
  uint4v w[D / 64];
  uint4v s, b;
};

// A block as a raw buffer: loads then take a 32-bit offset from the lane and
// the rest from scalars, and none can leave the block. They go past L2's
// retention (nontemporal): a cached byte is read once a call.
constexpr int kRawBuffer = 0x00020000;  // word 3: raw 32-bit buffer, gfx9 family
constexpr int kNontemporal = 2;
template <int D>
__device__ inline __amdgpu_buffer_rsrc_t block_buffer(const char* blk) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(blk), 0, 32 * (D + 8), kRawBuffer);
}

// `at`: this lane's byte of the first tile's keys; the other places of a block follow from it and the lane.
template <int D>
__device__ inline void load_keys(RawKeys<D>& r, __amdgpu_buffer_rsrc_t blk, uint32_t at, uint32_t pair) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if constexpr (D == 64) {
      const uint2v w = __builtin_bit_cast(uint2v, __builtin_amdgcn_raw_buffer_load_b64(blk, at + t * 8 * D, 0, kNontemporal));
      r.w[t][0] = w.x;
      r.w[t][1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4v w = __builtin_bit_cast(
            uint4v, __builtin_amdgcn_raw_buffer_load_b128(blk, at + (t * 8 * D + 16 * i), 0, kNontemporal));
        r.w[t][4 * i] = w.x;
        r.w[t][4 * i + 1] = w.y;
        r.w[t][4 * i + 2] = w.z;
        r.w[t][4 * i + 3] = w.w;
      }
    }
    const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(blk, pair + 64 * t, 32 * D, kNontemporal);
    r.pair[t] = halves(w);
  }
}
template <int D>
__device__ inline void load_values(RawValues<D>& r, __amdgpu_buffer_rsrc_t blk, uint32_t at, uint32_t pair) {
#pragma unroll
  for (int g = 0; g < D / 64; ++g)
    r.w[g] = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(blk, at + g * 1024, 16 * D, kNontemporal));
  r.s = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(blk, pair + 128, 32 * D, kNontemporal));
  r.b = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(blk, pair + 192, 32 * D, kNontemporal));
}

template <int D, int NT, bool F32, bool TREE>
__global__ __launch_bounds__(kWaves * 64, NT * D > 128 || NT > 1 ? 2 : 4) void kv_attend_few_kernel(KvAttendArgs a) {
  constexpr int MT = D / 16;
  constexpr int R = 16 * NT, LD = D + 4;  // rows of an item; a row's floats in LDS, padded off the same banks
  // Of many rows and channels the queries lie in LDS, for want of registers, and
  // the waves join some tiles at a time, for want of LDS.
  constexpr bool QL = NT * D > 256 || NT > 2;
  constexpr int PN = !QL ? NT : D == 256 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) float part[kWaves][16 * PN][LD];
  __shared__ half8v ql[QL ? NT : 1][QL ? D / 32 : 1][64];
  __shared__ TreeRow tl[QL ? R : 1];
  __shared__ float heads[kWaves][R][2];
  const uint32_t lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t col = lane & 15, quarter = lane >> 4;
  const int G = a.L.Hq / a.L.Hkv;
  int64_t slot_id = blockIdx.x;
  int b, h, run = 0, runs = 1, chunk = kKvWhole, r0 = 0;  // r0: the item's first row
  Sequence seq;
  if constexpr (TREE) {
    const Work w = find_work(a, blockIdx.x, lane, wave == 0);
    if (w.b < 0) return;
    b = w.b;
    h = w.h;
    run = w.run;
    runs = w.runs;
    chunk = w.chunk;
    seq = w.seq;
    r0 = w.tile * R;
    slot_id = partial_of(a, w, threadIdx.x == 0);
  } else if (a.plan.slots <= a.plan.items) {  // one run an item
    b = (int)blockIdx.x / a.L.Hkv;
    h = (int)blockIdx.x - b * a.L.Hkv;
    seq = sequence(a, b, h == 0 && threadIdx.x == 0);
  } else {
    if (a.batch == 1) {
      b = 0;
      seq = sequence(a, 0, blockIdx.x == 0 && threadIdx.x == 0);
      chunk = kv_chunk(a.plan, (int64_t)seq.blocks() * a.L.Hkv, seq.blocks());
      h = (int)blockIdx.x;
    } else {
      const Runs runs = find_runs(a, slot_id, 0, lane, blockIdx.x == 0 && wave == 0);
      if (runs.b < 0) return;
      b = runs.b;
      chunk = runs.chunk;
      seq = runs.seq;
      h = (int)(slot_id - runs.slot);
    }
    run = h / a.L.Hkv;
    h -= run * a.L.Hkv;
  }
  const int rows = TREE && seq.n * G - r0 > R ? R : seq.n * G - r0;
  const int nblk = seq.blocks();
  if constexpr (!TREE) runs = kv_item_runs(chunk, nblk);
  if (rows <= 0 || run >= runs) return;
  const int j1 = nblk - run * chunk < chunk ? nblk : (run + 1) * chunk;
  int j = run * chunk + wave;

  // A block without a page is read from the first page and hidden from every row.
  RawKeys<D> k;
  RawValues<D> v;
  bool paged = false;
  Lost lost;
  const char* blk = a.pages;
  const uint32_t key_at = col * (D / 2) + quarter * (D / 8);
  int page = 0;  // of the block after the next
  auto find = [&](int at) {
    blk = a.pages + uniform(block_on(a, page, h, at, paged, lost));
    page = page_of(a, b, at + kWaves, j1);  // of the block after this one
  };
  if (j < j1) {
    page = page_of(a, b, j, j1);
    find(j);
    load_keys<D>(k, block_buffer<D>(blk), key_at, 4 * col);
    load_values<D>(v, block_buffer<D>(blk), 16 * lane, 16 * quarter);
  }

  half8v q[QL ? 1 : NT][D / 32];
  float4v o[NT][MT];  // O^T: row 4 quarter + i of tile m is channel (4 quarter + i) D / 16 + m
  float base[NT];     // m - kShift
  float sum[NT];      // of this lane's weights
  int seen[NT];       // keys that the column's row sees (without a tree)
  TreeRow tree[QL ? 1 : NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // Columns past the last row repeat row 0: loads that some lanes leave out
    // would make the loop's first waits those for everything.
    const int r = r0 + (n * 16 + (int)col < rows ? n * 16 + col : 0);
    const int i = r / G;
    const _Float16* src = a.q + (seq.row0 + i) * a.q_ts + (int64_t)(h * G + r - i * G) * a.q_hs + quarter * (D / 4);
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
      if constexpr (!QL) q[n][x] = query_operand(src + 8 * x);
      else if ((n * (D / 32) + x) % kWaves == wave) ql[n][x][lane] = query_operand(src + 8 * x);
    if constexpr (TREE) {
      if constexpr (!QL) tree[n] = tree_row(a, seq.row0 + i);
      else if (wave == n % kWaves && quarter == 0) tl[n * 16 + col] = tree_row(a, seq.row0 + i);
    } else seen[n] = seq.seen(i);
    base[n] = kNoMax;
    sum[n] = 0.f;
#pragma unroll
    for (int m = 0; m < MT; ++m) o[n][m] = float4v{0.f, 0.f, 0.f, 0.f};
  }
  if constexpr (QL) __syncthreads();
  const int whole = TREE ? seq.below_tree() >> 5 : seq.seen(0) >> 5;  // blocks that every row sees whole
  const float factor = a.scale * kLog2e;
  float limit = kTop;  // of the exponents, the same in all lanes; -inf once some row's base is far
  const Bits bits;

  // One block; `more`: another follows, whose loads go out on the way.
  auto take = [&](auto next) {
    constexpr bool more = decltype(next)::value;
    const bool hide = j >= whole || !paged;
    int end = paged ? seq.len - j * 32 : 0;  // tokens of this block that hold anything
    if constexpr (more) find(j + kWaves);

    float4v s[NT][2];
    half8v qi[QL ? NT : 1];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      if constexpr (QL) {
#pragma unroll
        for (int n = 0; n < NT; ++n) qi[n] = ql[n][i][lane];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const half8v kk = key_operand(bits, k.w[t][i], half2v{k.pair[t].x, k.pair[t].x}, half2v{k.pair[t].y, k.pair[t].y});
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, QL ? qi[n] : q[n][i], s[n][t], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (more) load_keys<D>(k, block_buffer<D>(blk), key_at, 4 * col);

    half8v hi[NT], lo[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float e[8];
      float top;
      int left = TREE ? 0 : (end > 0 ? seen[n] - j * 32 : 0) - (int)quarter * 4;
      uint32_t bits_seen = 0;
      if constexpr (TREE)
        if (hide && end > 0) bits_seen = tree_seen(a, QL ? tl[n * 16 + col] : tree[QL ? 0 : n], seq, j * 32) >> (quarter * 4);
      auto exponents = [&](float bs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = __builtin_fmaf(s[n][i >> 2][i & 3], factor, -bs);
        if (hide) {
          asm volatile("" : "+v"(left), "+v"(bits_seen));  // keeps the comparisons in this branch
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (TREE ? !(bits_seen >> ((i >> 2) * 16 + (i & 3)) & 1) : (i >> 2) * 16 + (i & 3) >= left)
              e[i] = -__builtin_inff();
        }
        top = max8(e);
      };
      exponents(base[n]);
      if (__any(top > limit)) {  // a new maximum, for some column
        exponents(0.f);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float nb = fmaxf(base[n], base_of(top));
        if (__any(is_far(nb))) limit = -__builtin_inff();
        const float f = exp2_hw(base[n] - nb);
        sum[n] *= f;
#pragma unroll
        for (int m = 0; m < MT; ++m) o[n][m] *= f;
        base[n] = nb;
        if (limit == kTop) {
          exponents(nb);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = less_base(e[i], nb);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float p0 = exp2_hw(e[i]), p1 = exp2_hw(e[i + 1]);
        sum[n] += p0;
        sum[n] += p1;
        split_weight<F32>(p0, p1, hi[n], lo[n], i);
      }
    }

    half2v vs[4], vb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vs[i] = halves(v.s[i]);
      vb[i] = halves(v.b[i]);
    }
    if (hide) {  // what lies behind the sequence's end may be anything
      asm volatile("" : "+s"(end));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((e >> 2) * 16 + (int)quarter * 4 + (e & 3) >= end) vs[e >> 1][e & 1] = vb[e >> 1][e & 1] = (_Float16)0.f;
    }
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      auto multiply = [&](half8v vv, int m) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, hi[n], o[n][m], 0, 0, 0);
          if constexpr (F32) o[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, lo[n], o[n][m], 0, 0, 0);
        }
      };
      multiply(value_operand<0>(bits, v.w[g], vs, vb), 4 * g);
      multiply(value_operand<1>(bits, v.w[g], vs, vb), 4 * g + 1);
      multiply(value_operand<2>(bits, v.w[g], vs, vb), 4 * g + 2);
      multiply(value_operand<3>(bits, v.w[g], vs, vb), 4 * g + 3);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (more) load_values<D>(v, block_buffer<D>(blk), 16 * lane, 16 * quarter);
  };
  // The last block apart: were the loads conditional inside one loop, the
  // compiler would have to wait for all of them in every turn.
  for (; j + kWaves < j1; j += kWaves) take(std::true_type{});
  if (j < j1) take(std::false_type{});
  if (lane == 0) report_lost(a, b, lost);

  // Join the waves: all leave their sums in LDS, then each thread adds up four
  // channels of a row over the waves, in order.
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    sum[n] += __shfl_xor(sum[n], 16);
    sum[n] += __shfl_xor(sum[n], 32);
    const int r = n * 16 + col;
    if (r < rows && quarter == 0) {
      heads[wave][r][0] = base[n];
      heads[wave][r][1] = sum[n];
    }
  }
  float* slot = a.ws + slot_id * a.plan.slot_floats;
#pragma unroll
  for (int n0 = 0; n0 < NT; n0 += PN) {
    const int p0 = 16 * n0;
    if (QL && n0 > 0) {
      if (p0 >= rows) break;
      __syncthreads();
    }
#pragma unroll
    for (int n = n0; n < n0 + PN && n < NT; ++n) {
      const int r = n * 16 + col;
      if (r >= rows) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MT; m += 4)
          *reinterpret_cast<float4v*>(&part[wave][r - p0][(quarter * 4 + i) * MT + m]) =
              float4v{o[n][m][i], o[n][m + 1][i], o[n][m + 2][i], o[n][m + 3][i]};
    }
    __syncthreads();
    const int here = rows - p0 < 16 * PN ? rows - p0 : 16 * PN;
    for (int x = threadIdx.x; x < here * (D / 4); x += kWaves * 64) {
      const int l = x / (D / 4), r = p0 + l, d = 4 * (x % (D / 4));
      float top = kNoMax, all = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, heads[w][r][0]);
      float4v v4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = exp2_hw(heads[w][r][0] - top);
        all += heads[w][r][1] * f;
        v4 += *reinterpret_cast<const float4v*>(&part[w][l][d]) * f;
      }
      if (runs == 1) {
        const int i = (r0 + r) / G;
        const int64_t row = (seq.row0 + i) * a.L.Hq + h * G + r0 + r - i * G;
        const float inv = all != 0.f ? 1.f / all : 0.f;
        store_out<F32, 4>(a.out, row * D + d, {v4.x * inv, v4.y * inv, v4.z * inv, v4.w * inv});
        if (a.lse && d == 0) a.lse[row] = all != 0.f ? (top + log2f(all)) * kLn2 : kLowest;
      } else {
        *reinterpret_cast<float4v*>(slot + r * D + d) = v4;
        if (d == 0) {
          slot[a.plan.rows * D + 2 * r] = top;
          slot[a.plan.rows * D + 2 * r + 1] = all;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- many rows

// For more rows (prompts): bound by the matrix and vector units together. A
// workgroup of W waves takes 32 W rows of an item, 32 a wave, the columns of
// 32 x 32 products. The workgroup turns a tile of 64 W / D blocks into binary16
// operands in LDS, each thread one 16-byte piece of the keys and one of the
// values, while the waves multiply the tile before it; one barrier a tile. The
// next tile's bytes are on their way meanwhile. Two blocks' scores at a time
// are independent chains of products.
//
// Unpacking is half of the vector work at W = 4, and twice the rows share it at
// W = 8; four waves leave room for two workgroups a CU, whose starts and ends
// overlap, which short items need more (kv_many_wide has the figures).
//
// Measured: 2 x 2048 queries of 64 heads (8 kv heads, D 128) on 8192 tokens in
// 966 to 1085 us from part to part (call after call; the first twenty after a
// pause take up to 1400, until the clock settles), 962 GFLOP at 0.89 to 1.00
// PFLOP/s; a 8192^3 library product reaches 1.14. Matrix units busy 44 % and
// vector units 50 % of the cycles, at 1.9 GHz of 2.4: power seems to hold the clock.
// Binary32 out, which has twice the value products: 1394 us. D 64: 708 (binary32
// 883), D 256 with half the heads: 1552 (1850), one block a tile there.
// With a tree: 16 x 64 nodes of 64 heads (8 kv heads, D 128) on 8192 tokens in 285
// to 299 us with the join, 0.91 to 0.96 PFLOP/s; 48 nodes of 96 heads on 131072, binary32 out,
// 491 to 508, of 271 for the products and 406 with the second part of the weights.
template <int D, int W, bool F32, bool TREE>
__global__ __launch_bounds__(W * 64, D > 128 ? 1 : 2) void kv_attend_many_kernel(KvAttendArgs a) {
  constexpr int KB = W * 64 / D;   // blocks of a tile
  constexpr int KS = D / 16;       // inner steps of the scores
  constexpr int MT = D / 32;       // channel tiles of the output
  constexpr int RN = D / 32;       // 16-byte pieces of a key row
  constexpr int KFRAG = KB * KS * 64, VFRAG = KB * 2 * MT * 64;  // 16-byte operands of a tile: 256 W each
  __shared__ half8v kl[2][KFRAG];
  __shared__ half8v vl[2][VFRAG];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  const int G = a.L.Hq / a.L.Hkv;
  // Heads innermost: workgroups of one head go to one XCD and share its cache;
  // later tiles, which see more keys, first.
  const int item = blockIdx.x;
  int run = a.plan.splits - 1 - blockIdx.y, h = item % a.L.Hkv, b, tile, chunk = 0, runs = 1;
  int64_t slot_id = (int64_t)item * a.plan.splits + run;
  Sequence seq;
  if constexpr (TREE) {
    const Work w = find_work(a, item, lane, wave == 0);
    if (w.b < 0) return;
    b = w.b;
    tile = w.tile;
    h = w.h;
    run = w.run;
    runs = w.runs;
    chunk = w.chunk;
    seq = w.seq;
    slot_id = partial_of(a, w, tid == 0);
  } else {
    const bool tells = run == 0 && h == 0 && wave == 0;
    const Tile at = find_tile(a, item / a.L.Hkv, lane, tells && item == 0);
    b = at.b;
    tile = at.tile;
    if (b < 0) return;
    seq = sequence(a, b, (a.batch == 1 || a.batch > kKvMaxBatch) && tells && tile == 0 && lane == 0);
  }
  const int rows = seq.n * G;
  const int r0 = tile * (32 * W);
  if (r0 >= rows) return;
  const int r_last = (r0 + 32 * W - 1 < rows ? r0 + 32 * W - 1 : rows - 1);
  const int nblk = kv_blocks(seq.seen(r_last / G));
  if constexpr (!TREE) runs = kv_runs(a.plan.chunk, a.plan.splits, nblk);
  if (run >= runs) return;
  if constexpr (!TREE) chunk = kv_run_blocks(a.plan.chunk, a.plan.splits, nblk);
  const int j0 = TREE && runs == 1 ? 0 : run * chunk;
  const int j1 = nblk - j0 < chunk ? nblk : j0 + chunk;

  const int r = r0 + wave * 32 + col;
  const bool live = r < rows;
  const int qi = live ? r / G : 0;
  const int64_t orow = (seq.row0 + qi) * a.L.Hq + h * G + (r - qi * G);
  half8v q[KS];
  {
    const _Float16* src = a.q + (seq.row0 + qi) * a.q_ts + (int64_t)(h * G + r - qi * G) * a.q_hs + hh * 8;
#pragma unroll
    for (int u = 0; u < KS; ++u) q[u] = live ? query_operand(src + 16 * u) : half8v{};
  }
  const int seen = live ? seq.seen(qi) : seq.len;
  TreeRow tree;
  if constexpr (TREE) tree = tree_row(a, seq.row0 + qi);
  // Wave-uniform: blocks below `whole` are seen whole by every row of the wave, none at or past `none`.
  const int w0 = r0 + wave * 32, w1 = (w0 + 31 < rows ? w0 + 31 : rows - 1);
  const int whole = w0 >= rows ? 0 : TREE ? seq.below_tree() >> 5 : seq.seen(w0 / G) >> 5;
  const int none = w0 < rows ? kv_blocks(seq.seen(w1 / G)) : 0;
  const float factor = a.scale * kLog2e;
  const Bits bits;

  float16v o[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[m][i] = 0.f;
  float base = kNoMax, sum = 0.f;
  float limit = kTop;  // of the exponents, the same in all lanes; -inf once some row's base is far

  // This thread's piece of a tile: block, and within it the key row's piece and the value piece.
  const int piece = tid & (D - 1), pb = uniform(tid / D);
  const int ktok = piece / RN, krun = piece % RN;
  const int vq = (piece >> 4) & 3, vc = piece & 15, vg = piece >> 6;
  uint4v kr, vr, vsr, vbr;
  half2v kpr;
  bool have = false;  // this thread's block is there
  Lost lost;
  int next_page = j0 < j1 ? page_of(a, b, j0 + pb, j1) : 0;
  auto fetch = [&](int jt) {  // called for every tile in turn
    const int j = jt + pb;
    const int page = next_page;
    next_page = page_of(a, b, j + KB, j1);
    have = false;
    if (j >= j1) return;
    const char* blk = a.pages + uniform(block_on(a, page, h, j, have, lost));
    kr = *reinterpret_cast<const uint4v*>(blk + piece * 16);
    kpr = *reinterpret_cast<const half2v*>(blk + 32 * D + 4 * ktok);
    vr = *reinterpret_cast<const uint4v*>(blk + 16 * D + piece * 16);
    vsr = *reinterpret_cast<const uint4v*>(blk + 32 * D + 128 + vq * 16);
    vbr = *reinterpret_cast<const uint4v*>(blk + 32 * D + 192 + vq * 16);
  };
  __shared__ int there[2][KB];
  auto spread = [&](int jt, int buf) {
    const int j = jt + pb;
    half2v ks = kpr, vs[4], vb[4];
    // Nothing may come of tokens behind the sequence's end or without a page.
    const bool part = !have || seq.len - 32 * j < 32;  // the same in all lanes
    if (part && !(have && j * 32 + ktok < seq.len)) {
      ks = half2v{(_Float16)0.f, (_Float16)0.f};
      kr = uint4v{0, 0, 0, 0};
    }
    const half2v s2 = {ks.x, ks.x}, b2 = {ks.y, ks.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = krun * 4 + i;  // word of the row: step w / 2, half w & 1
      kl[buf][(pb * KS + (w >> 1)) * 64 + (((w & 1) * 32 + ktok) ^ (krun * (8 / RN)))] = key_operand(bits, kr[i], s2, b2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vs[i] = halves(vsr[i]);
      vb[i] = halves(vbr[i]);
    }
    if (part) {
      int left = have ? seq.len - (j * 32 + vq * 4) : 0;
      asm volatile("" : "+v"(left));  // keeps the comparisons in this branch
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((e >> 2) * 16 + (e & 3) >= left) vs[e >> 1][e & 1] = vb[e >> 1][e & 1] = (_Float16)0.f;
    }
    const half8v v[4] = {value_operand<0>(bits, vr, vs, vb), value_operand<1>(bits, vr, vs, vb), value_operand<2>(bits, vr, vs, vb),
                         value_operand<3>(bits, vr, vs, vb)};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      vl[buf][((pb * 2 + (vq >> 1)) * MT + 2 * vg + (x >> 1)) * 64 + (vq & 1) * 32 + (x & 1) * 16 + vc] = v[x];
    if (piece == 0) there[buf][pb] = have;
  };

  // NB blocks of a tile at once: their scores are independent chains of products.
  constexpr int NB = KB < 2 ? KB : 2;
  auto take = [&](int j, int buf, int kb) {
    float16v s[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[n][i] = 0.f;
    auto key = [&](int n, int u) { return kl[buf][((kb + n) * KS + u) * 64 + (lane ^ ((u >> 1) * (8 / RN)))]; };
    half8v k[2][NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) k[0][n] = key(n, 0);
#pragma unroll
    for (int u = 0; u < KS; ++u) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
        if (u + 1 < KS) k[(u + 1) & 1][n] = key(n, u + 1);
#pragma unroll
      for (int n = 0; n < NB; ++n) s[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[u & 1][n], q[u], s[n], 0, 0, 0);
    }
    // A block without a page, or past the run, is hidden from every row.
    bool hide = j + NB > whole;
    int left[NB];
    bool here[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      here[n] = j + n < j1 && uniform(there[buf][kb + n]);
      hide |= !here[n];
      left[n] = !TREE && here[n] ? seen - ((j + n) * 32 + hh * 4) : 0;
    }
    if constexpr (TREE) {  // bits of the tokens seen, in left
      if (hide) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
          if (here[n]) left[n] = (int)(tree_seen(a, tree, seq, (j + n) * 32) >> (hh * 4));
      }
    }
    float e[NB][16];
    float top;
    auto exponents = [&](float bs) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) e[n][i] = __builtin_fmaf(s[n][i], factor, -bs);
      if (hide) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          asm volatile("" : "+v"(left[n]));  // keeps the comparisons in this branch
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (TREE ? !((uint32_t)left[n] >> (8 * (i >> 2) + (i & 3)) & 1) : 8 * (i >> 2) + (i & 3) >= left[n])
              e[n][i] = -__builtin_inff();
        }
      }
      top = max3(max8(e[0]), max8(e[0] + 8), max8(e[NB - 1] + 8));
      if constexpr (NB > 1) top = max3(top, max8(e[1]), top);
    };
    exponents(base);
    if (__any(top > limit)) {
      exponents(0.f);
      top = fmaxf(top, __shfl_xor(top, 32));
      const float nb = fmaxf(base, base_of(top));
      if (__any(is_far(nb))) limit = -__builtin_inff();
      const float f = exp2_hw(base - nb);
      sum *= f;
#pragma unroll
      for (int m = 0; m < MT; ++m) o[m] *= f;
      base = nb;
      if (limit == kTop) {
        exponents(nb);
      } else {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) e[n][i] = less_base(e[n][i], nb);
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      half8v hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = exp2_hw(e[n][i]), p1 = exp2_hw(e[n][i + 1]);
        sum += p0;
        sum += p1;
        // group i / 4 of four keys: elements 0..3 of product 0 and 1, then 4..7
        split_weight<F32>(p0, p1, hi[(i >> 2) & 1], lo[(i >> 2) & 1], (i >> 3) * 4 + (i & 3));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const half8v v = vl[buf][(((kb + n) * 2 + u) * MT + m) * 64 + lane];
          o[m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, hi[u], o[m], 0, 0, 0);
          if constexpr (F32) o[m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, lo[u], o[m], 0, 0, 0);
        }
    }
  };

  if (j0 < j1) {
    fetch(j0);
    spread(j0, 0);
    if (j0 + KB < j1) fetch(j0 + KB);
    __syncthreads();
    int buf = 0;
    for (int jt = j0; jt < j1; jt += KB, buf ^= 1) {
#pragma unroll 1
      for (int kb = 0; kb < KB; kb += NB)
        if (jt + kb < j1 && jt + kb < none) take(jt + kb, buf, kb);
      if (jt + KB < j1) {
        spread(jt + KB, buf ^ 1);
        if (jt + 2 * KB < j1) fetch(jt + 2 * KB);
      }
      __syncthreads();
    }
  }

  if (lane == 0) report_lost(a, b, lost);
  sum += __shfl_xor(sum, 32);
  if (!live) return;
  // O^T: register i of tile m is row R = 8 (i / 4) + 4 hh + i % 4, channel (R % 16) D / 16 + 2 m + R / 16.
  const bool last = runs == 1;
  float* slot = last ? nullptr : a.ws + slot_id * a.plan.slot_floats;
  const int lr = r - r0;
  const float inv = !last ? 1.f : sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int y = 0; y < 8; ++y) {
    float v[2 * MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      v[2 * m] = o[m][y] * inv;
      v[2 * m + 1] = o[m][8 + y] * inv;
    }
    const int d0 = (8 * (y >> 2) + 4 * hh + (y & 3)) * (2 * MT);
    if (last) store_out<F32>(a.out, orow * D + d0, v);
    else store_out<true>(slot, (int64_t)lr * D + d0, v);
  }
  if (hh == 0) {
    if (last) {
      if (a.lse) a.lse[orow] = sum != 0.f ? (base + log2f(sum)) * kLn2 : kLowest;
    } else {
      slot[a.plan.rows * D + 2 * lr] = base;
      slot[a.plan.rows * D + 2 * lr + 1] = sum;
    }
  }
}

// ---------------------------------------------------------------- join

// Joins the partials of an item's runs. A workgroup takes `join_rows` of its
// rows: the weights 2^(exponent - largest) of the runs go to LDS, then each
// thread adds up four channels of a row over every S-th run, in order, and the
// S sums of a row meet in LDS. One row a workgroup (S = 2048 / D) where the call
// has few, so that many runs do not queue; a full workgroup of rows otherwise.
// Latency-bound: 4 to 8 us, of which the launch is 2; a join by the last
// workgroup of an item instead would need fences and counters to be cleared.
constexpr int kJoinThreads = 512;

// Joins R rows of an item, from row r0 + l0 of its kv head h on. RW: a power of two, R at the least.
template <int D, bool F32>
__device__ inline void join_rows(const KvAttendArgs& a, const float* part, int64_t step, int runs, int64_t row0, int h, int r0,
                                 int l0, int R, int RW) {
  constexpr int C = D / 4;  // threads of a row
  __shared__ float weight[kJoinThreads / C][kKvMaxSplits];
  __shared__ float4v meet[kJoinThreads];
  __shared__ float sums[kJoinThreads / C], tops[kJoinThreads / C];
  const int G = a.L.Hq / a.L.Hkv;
  const int lane = threadIdx.x & 63;
  for (int r = uniform((int)threadIdx.x >> 6); r < R; r += kJoinThreads / 64) {
    const float* head = part + a.plan.rows * D + 2 * (l0 + r);
    float e[kKvMaxSplits / 64], n[kKvMaxSplits / 64], top = kNoMax, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kKvMaxSplits / 64; ++i) {
      const int s = 64 * i + lane;
      e[i] = s < runs ? head[s * step] : kNoMax;
      n[i] = s < runs ? head[s * step + 1] : 0.f;
      top = fmaxf(top, e[i]);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
#pragma unroll
    for (int i = 0; i < kKvMaxSplits / 64; ++i) {
      const float f = exp2_hw(e[i] - top);
      sum += f * n[i];
      if (64 * i + lane < runs) weight[r][64 * i + lane] = f;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if (lane == 0) {
      sums[r] = sum;
      tops[r] = top;
    }
  }
  __syncthreads();

  const int S = kJoinThreads / (RW * C);
  const int d = 4 * ((int)threadIdx.x % C), r = (int)threadIdx.x / C % RW, slice = (int)threadIdx.x / (RW * C);
  float4v v = {0.f, 0.f, 0.f, 0.f};
  if (r < R) {
    const float* p = part + (int64_t)(l0 + r) * D + d;
#pragma unroll 8
    for (int s = slice; s < runs; s += S)
      v += *reinterpret_cast<const float4v*>(p + s * step) * weight[r][s];
  }
  if (S > 1) {
    meet[threadIdx.x] = v;
    __syncthreads();
    if (slice > 0) return;
    for (int s = 1; s < S; ++s) v += meet[s * RW * C + threadIdx.x];
  }
  if (r >= R) return;
  const int rr = r0 + l0 + r, i = rr / G;
  const int64_t row = (row0 + i) * a.L.Hq + h * G + rr - i * G;
  const float inv = sums[r] != 0.f ? 1.f / sums[r] : 0.f;
  store_out<F32, 4>(a.out, row * D + d, {v.x * inv, v.y * inv, v.z * inv, v.w * inv});
  if (a.lse && d == 0) a.lse[row] = sums[r] != 0.f ? (tops[r] + log2f(sums[r])) * kLn2 : kLowest;
}

template <int D, bool F32>
__global__ __launch_bounds__(kJoinThreads) void kv_attend_join_kernel(KvAttendArgs a) {
  const int rpi = a.plan.rows, RW = a.plan.join_rows;
  const int item = blockIdx.x, l0 = blockIdx.y * RW;
  const int G = a.L.Hq / a.L.Hkv;
  const int lane = threadIdx.x & 63;
  int b = 0, h, r0 = 0, runs;
  int64_t slot, step = 1;  // of the first partial, and to the next
  Sequence seq;
  if (a.plan.many) {
    h = item % a.L.Hkv;
    const Tile at = find_tile(a, item / a.L.Hkv, lane, false);
    if (at.b < 0) return;
    b = at.b;
    seq = sequence(a, b, false);
    r0 = at.tile * rpi;
    const int rows = seq.n * G;
    if (r0 >= rows) return;
    const int r_last = r0 + rpi - 1 < rows ? r0 + rpi - 1 : rows - 1;
    runs = kv_runs(a.plan.chunk, a.plan.splits, kv_blocks(seq.seen(r_last / G)));
    slot = (int64_t)item * a.plan.splits;
  } else {
    b = item / a.L.Hkv;
    h = item - b * a.L.Hkv;
    slot = h;
    int chunk;
    if (a.batch == 1) {
      seq = sequence(a, 0, false);
      chunk = kv_chunk(a.plan, (int64_t)seq.blocks() * a.L.Hkv, seq.blocks());
    } else {
      const Runs r = find_runs(a, -1, b, lane, false);
      seq = r.seq;
      chunk = r.chunk;
      slot += r.slot;
    }
    runs = kv_item_runs(chunk, seq.blocks());
    step = a.L.Hkv;
  }
  const int rows = seq.n * G;
  if (r0 + l0 >= rows) return;
  if (runs == 1) return;  // written by its only run
  const int R = rows - r0 - l0 < RW ? rows - r0 - l0 : RW;
  join_rows<D, F32>(a, a.ws + slot * a.plan.slot_floats, step * a.plan.slot_floats, runs, seq.row0, h, r0, l0, R, RW);
}

// With a tree: the items that the attention left in a list (a single sequence's
// follow from its lengths).
struct Joins {
  int count;
  KvJoin one;
  const KvJoin* list;

  __device__ explicit Joins(const KvAttendArgs& a) : one{}, list(reinterpret_cast<const KvJoin*>(a.joins + 4)) {
    if (a.batch > 1) {
      count = *a.joins;
      return;
    }
    const Sequence s = sequence(a, 0, false);
    const int per = tiles_of(a, s) * a.L.Hkv;
    one = KvJoin{s.row0, 0, 0, s.n * a.plan.group, kv_tree_runs(kv_tree_chunk_of_one(a.plan, per, s.blocks()), s.blocks()), 0, per};
    count = one.runs > 1 ? per : 0;
  }
  __device__ KvJoin at(const KvAttendArgs& a, int i) const {
    if (a.batch > 1) return list[i];
    KvJoin j = one;
    const int tile = (int)((uint32_t)i / (uint32_t)a.L.Hkv);
    j.h = i - tile * a.L.Hkv;
    j.r0 = tile << a.plan.row_shift;
    j.slot = i;
    return j;
  }
};

// Few rows in all: a workgroup each, whose slices take every S-th run.
template <int D, bool F32>
__global__ __launch_bounds__(kJoinThreads) void kv_tree_join_few_kernel(KvAttendArgs a) {
  const int groups = a.plan.join_groups;
  const Joins joins(a);
  for (int k = blockIdx.x, i; (i = (int)((uint32_t)k / (uint32_t)groups)) < joins.count; k += gridDim.x) {
    const KvJoin j = joins.at(a, i);
    const int l = k - i * groups;
    if (l >= j.rows - j.r0) continue;
    join_rows<D, F32>(a, a.ws + (int64_t)j.slot * a.plan.slot_floats, (int64_t)j.step * a.plan.slot_floats, j.runs, j.row0, j.h,
                      j.r0, l, 1, 1);
    __syncthreads();
  }
}

// Many rows: D / 4 lanes a row, four runs' numbers on their way at a time, nothing
// between the waves.
template <int D, bool F32>
__global__ __launch_bounds__(256) void kv_tree_join_many_kernel(KvAttendArgs a) {
  constexpr int C = D / 4, N = 64 / C;  // rows of a wave
  const int lane = threadIdx.x & 63, d = 4 * (lane % C);
  const int groups = a.plan.join_groups;
  const Joins joins(a);
  for (int k = uniform((int)(blockIdx.x * 4 + (threadIdx.x >> 6))), i; (i = (int)((uint32_t)k / (uint32_t)groups)) < joins.count;
       k += gridDim.x * 4) {
    const KvJoin j = joins.at(a, i);
    const int l = (k - i * groups) * N + lane / C;
    if (l >= j.rows - j.r0) continue;
    const float* part = a.ws + (int64_t)j.slot * a.plan.slot_floats;
    const int64_t step = (int64_t)j.step * a.plan.slot_floats;
    float top = kNoMax, sum = 0.f;
    float4v v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < j.runs; s += 4) {
      float e[4], n[4];
      float4v p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float* at = part + (s + x < j.runs ? s + x : s) * step;
        e[x] = at[a.plan.rows * D + 2 * l];
        n[x] = at[a.plan.rows * D + 2 * l + 1];
        p[x] = *reinterpret_cast<const float4v*>(at + l * D + d);
      }
      const float m = fmaxf(max3(e[0], e[1], e[2]), fmaxf(e[3], top));
      const float f = exp2_hw(top - m);
      sum *= f;
      v *= f;
      top = m;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float w = s + x < j.runs ? exp2_hw(e[x] - m) : 0.f;
        sum += w * n[x];
        v += w * p[x];
      }
    }
    const int r = j.r0 + l, q = (int)((uint32_t)r / (uint32_t)a.plan.group);
    const int64_t row = (j.row0 + q) * a.L.Hq + j.h * a.plan.group + r - q * a.plan.group;
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    store_out<F32, 4>(a.out, row * D + d, {v.x * inv, v.y * inv, v.z * inv, v.w * inv});
    if (a.lse && d == 0) a.lse[row] = sum != 0.f ? (top + log2f(sum)) * kLn2 : kLowest;
  }
}

template <int D, bool F32, bool TREE>
hipError_t launch_d(const KvAttendArgs& a, hipStream_t s) {
  const int64_t items = a.plan.many && !TREE ? kv_many_items(a.plan, a.L, a.batch, a.tokens) : a.plan.items;
  const dim3 grid((unsigned)(a.plan.many && !TREE ? items : a.plan.slots), (unsigned)a.plan.splits);
  hipError_t e = hipErrorInvalidValue;
  if (a.plan.many && a.plan.rows == 128) {
    e = kv_launch(kv_attend_many_kernel<D, 4, F32, TREE>, grid, 256, s, a);
  } else if (a.plan.many) {
    if constexpr (D == 128) e = kv_launch(kv_attend_many_kernel<D, 8, F32, TREE>, grid, 512, s, a);
  } else if (a.plan.rows == 16) {
    e = kv_launch(kv_attend_few_kernel<D, 1, F32, TREE>, grid, kWaves * 64, s, a);
  } else if constexpr (D <= 128 || TREE) {
    if (a.plan.rows == 32) e = kv_launch(kv_attend_few_kernel<D, 2, F32, TREE>, grid, kWaves * 64, s, a);
    if constexpr (TREE && D <= 128 && !(D == 128 && F32))
      if (a.plan.rows == 64) e = kv_launch(kv_attend_few_kernel<D, 4, F32, true>, grid, kWaves * 64, s, a);
  }
  if (a.plan.ws_bytes > 0 && e == hipSuccess)
    e = TREE ? a.plan.join_rows == 0
                   ? kv_launch(kv_tree_join_few_kernel<D, F32>, dim3((unsigned)a.plan.join_grid), kJoinThreads, s, a)
                   : kv_launch(kv_tree_join_many_kernel<D, F32>, dim3((unsigned)a.plan.join_grid), 256, s, a)
             : kv_launch(kv_attend_join_kernel<D, F32>, dim3((unsigned)items, (unsigned)a.plan.join_groups), kJoinThreads, s, a);
  return e;
}

template <bool F32, bool TREE>
hipError_t launch_out(const KvAttendArgs& a, hipStream_t s) {
  switch (a.L.D) {
    case 64: return launch_d<64, F32, TREE>(a, s);
    case 128: return launch_d<128, F32, TREE>(a, s);
    case 256: return launch_d<256, F32, TREE>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_kv_attend(const KvAttendArgs& a, bool out_f32, hipStream_t s) {
  if (a.tree) return out_f32 ? launch_out<true, true>(a, s) : launch_out<false, true>(a, s);
  return out_f32 ? launch_out<true, false>(a, s) : launch_out<false, false>(a, s);
}

}  // namespace agemm
