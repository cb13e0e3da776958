// Drafted tokens in a tree over the 4-bit paged cache on gfx950: laying them out
// before a step, and moving the accepted ones to their places after it.
#include "kv_internal.h"

namespace agemm {
namespace {

// ---------------------------------------------------------------- layout

// Place `at` of a sequence in its pages: the slot, -1 without a page that the cache has.
__device__ inline int64_t slot_of(const KvLayout& L, const int32_t* table, int64_t stride, int b, int64_t at, int* page) {
  *page = table[b * stride + (at >> L.page_shift)];
  if (*page < 0 || *page >= L.num_pages) return -1;
  return ((int64_t)*page << L.page_shift) + (at & (L.page_tokens - 1));
}

// What a sequence's tree may use. `fits`: its places lie in the table.
struct Nodes {
  int64_t row0;  // of its first node
  int64_t n;     // its nodes as given
  bool rows;     // they are rows of the call, max_q at most
  bool fits;
  int len;
};
template <class A>
__device__ inline Nodes nodes_of(const A& a, int b, bool table) {
  const int start = a.q_start[b], end = a.q_start[b + 1];
  Nodes s;
  s.row0 = start;
  s.n = (int64_t)end - start;
  s.rows = s.n >= 0 && s.n <= a.max_q && start >= 0 && end <= a.tokens;
  s.len = a.kv_len[b];
  const int64_t most = table ? (int64_t)a.table_width << a.L.page_shift : 0x7fffffff;
  s.fits = s.len >= 0 && s.len + s.n <= most && s.len + s.n <= 0x7fffffff;
  return s;
}

// One workgroup a sequence, a thread a node. With m_i the nodes that i has found
// so far, itself first, and up_i the next ancestor, a turn takes m_i |= m_up,
// up_i = up_up: after k turns every node has 2^k of its chain, so that a chain of
// n nodes takes log2 n turns and a usual tree two or three. The last workgroup
// marks the rows of no sequence.
//
// Latency-bound, by loads one after the other and the turns: a tree of 8 takes
// 2.2 us, 128 trees of up to 200 nodes 5.4.
template <int W>  // mask words at most
__global__ __launch_bounds__(64 * W) void kv_tree_kernel(KvTreeArgs a) {
  constexpr int N = 64 * W, LD = W | 1;  // odd: rows start in different banks
  __shared__ uint64_t mask[N][LD];
  __shared__ int16_t up[N], depth[N];
  const int i = threadIdx.x, words = a.words;
  auto pad = [&](int64_t row) {
    for (int w = 0; w < words; ++w) a.mask[row * words + w] = 0;
    if (a.positions) a.positions[row] = 0;
    if (a.slots) a.slots[row] = -1;
  };
  const int b = blockIdx.x;
  if (b == a.batch) {
    const int64_t first = a.batch ? a.q_start[0] : 0, last = a.batch ? a.q_start[a.batch] : 0;
    for (int64_t row = i; row < first && row < a.tokens; row += blockDim.x) pad(row);
    for (int64_t row = (last < 0 ? 0 : last) + i; row < a.tokens; row += blockDim.x) pad(row);
    return;
  }
  const Nodes s = nodes_of(a, b, a.slots != nullptr);
  if (!s.rows || !s.fits) {
    if (i == 0) {
      if (!s.rows) kv_report(a.err, kKvRows, b, s.n);
      else kv_report(a.err, kKvLength, b, s.len);
      if (a.total_len) a.total_len[b] = s.len;
    }
    for (int64_t row = (s.row0 < 0 ? 0 : s.row0) + i; row < s.row0 + s.n && row < a.tokens; row += blockDim.x) pad(row);
    return;
  }
  if (i == 0 && a.total_len) a.total_len[b] = s.len + (int)s.n;
  const int n = (int)s.n;
  const bool live = i < n;
  const int64_t row = s.row0 + i;
  int p = live ? a.parent[row] : -1;
  if (live && (p < -1 || p >= i)) {
    kv_report(a.err, kKvParent, row, p);
    p = -1;
  }
  int page = 0;
  int64_t slot = -1;
  if (live && a.slots) {
    slot = slot_of(a.L, a.table, a.table_stride, b, (int64_t)s.len + i, &page);
    if (slot < 0) kv_report(a.err, kKvPage, b, page);
  }
#pragma unroll
  for (int w = 0; w < W; ++w) mask[i][w] = w == i >> 6 ? uint64_t{1} << (i & 63) : 0;
  up[i] = (int16_t)p;
  int d = p >= 0;
  depth[i] = (int16_t)d;
  while (__syncthreads_or(p >= 0)) {
    uint64_t m[W];
    int next = -1;
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) m[w] = mask[p][w];
      d += depth[p];
      next = up[p];
    }
    __syncthreads();
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) mask[i][w] |= m[w];
      depth[i] = (int16_t)d;
      up[i] = (int16_t)next;
    }
    p = next;
  }
  if (!live) return;
  for (int w = 0; w < words; ++w) a.mask[row * words + w] = mask[i][w];
  if (a.positions) a.positions[row] = (int64_t)s.len + d;
  if (a.slots) a.slots[row] = slot;
}

// ---------------------------------------------------------------- commit

// Moves accepted nodes to the front of their tree, a wave for each (layer,
// sequence, kv head), 16 lanes a token: lane c has the c-th part of the key row
// and the channels of run c of the values. As a path ascends, path[i] >= i: the
// tokens of a chunk are all read before any is written, and what later chunks
// read lies behind what earlier ones wrote, so the move needs no second place.
//
// Latency-bound, by lengths, path, pages and tokens one after the other: 4.1 us for
// a path of one layer, 7.3 for 276 tokens in each of six (2.0 of bytes).
constexpr int kMove = 16;  // tokens of a chunk

template <int D>
__global__ __launch_bounds__(256) void kv_commit_kernel(KvCommitArgs a) {
  constexpr int KB = D / 32;  // bytes of a lane's part of a key row
  constexpr int G = D / 64;   // value words of a lane
  constexpr int U = kMove / 4;
  struct alignas(KB) Key {
    uint8_t x[KB];
  };
  const int lane = threadIdx.x & 63, part = lane & 15, sub = lane >> 4;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t heads = (int64_t)a.batch * a.L.Hkv;
  const int layer = (int)(item / heads);
  if (item >= heads * (a.layers > 0 ? a.layers : 1)) return;
  const int b = (int)((item - layer * heads) / a.L.Hkv), h = (int)(item - layer * heads - (int64_t)b * a.L.Hkv);
  const bool tells = layer == 0 && h == 0 && lane == 0;
  const Nodes s = nodes_of(a, b, true);
  const int count = a.count[b];
  const int32_t* path = a.path + s.row0;
  bool good = s.rows && s.fits && count >= 0 && count <= s.n;
  bool ascends = true;
  if (good)
    for (int i = lane; i < count; i += 64) {
      const int x = path[i], before = i > 0 ? path[i - 1] : -1;
      ascends &= x > before && x < s.n;
    }
  ascends = __all(ascends);
  if (tells) {
    if (!s.rows) kv_report(a.err, kKvRows, b, s.n);
    else if (!s.fits) kv_report(a.err, kKvLength, b, s.len);
    else if (!good || !ascends) kv_report(a.err, kKvPath, b, count);
    if (a.new_len) a.new_len[b] = s.len + (good && ascends ? count : 0);
  }
  if (!good || !ascends || a.layers == 0) return;

  char* pages = a.pages[layer];
  for (int c = 0; c < count; c += kMove) {
    char *from[U], *to[U];
    int ft[U], tt[U];  // tokens of their blocks
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = c + 4 * u + sub;
      from[u] = nullptr;
      const int x = i < count ? path[i] : i;
      if (x == i) continue;
      int page;
      auto place = [&](int at, int& token) -> char* {
        const int64_t slot = slot_of(a.L, a.table, a.table_stride, b, (int64_t)s.len + at, &page);
        if (slot < 0) {
          if (h == 0 && layer == 0 && part == 0) kv_report(a.err, kKvPage, b, page);
          return nullptr;
        }
        const int off = (int)(slot & (a.L.page_tokens - 1));
        token = off & 31;
        return pages + kv_block_at(a.L, slot >> a.L.page_shift, h, off >> 5);
      };
      from[u] = place(x, ft[u]);
      to[u] = place(i, tt[u]);
      if (!to[u]) from[u] = nullptr;
    }
    auto value_at = [&](char* blk, int g, int t) {
      return reinterpret_cast<uint16_t*>(blk + 16 * D) + ((g * 4 + kv_value_quarter(t)) * 16 + part) * 8 + kv_value_place(t);
    };
    // lane 0: the key pair, lanes 1 and 2: s and b of the value
    auto pair_at = [&](char* blk, int t) {
      return blk + 32 * D + (part == 0 ? 4 * t : 128 + (part == 2 ? 64 : 0) + 2 * (8 * kv_value_quarter(t) + kv_value_place(t)));
    };
    Key key[U];
    uint16_t value[U][G];
    uint32_t pair[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!from[u]) continue;
      key[u] = *reinterpret_cast<const Key*>(from[u] + ft[u] * (D / 2) + part * KB);
#pragma unroll
      for (int g = 0; g < G; ++g) value[u][g] = *value_at(from[u], g, ft[u]);
      if (part == 0) pair[u] = *reinterpret_cast<const uint32_t*>(pair_at(from[u], ft[u]));
      else if (part < 3) pair[u] = *reinterpret_cast<const uint16_t*>(pair_at(from[u], ft[u]));
    }
    // All of the chunk's loads are back before its first store.
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!from[u]) continue;
      *reinterpret_cast<Key*>(to[u] + tt[u] * (D / 2) + part * KB) = key[u];
#pragma unroll
      for (int g = 0; g < G; ++g) *value_at(to[u], g, tt[u]) = value[u][g];
      if (part == 0) *reinterpret_cast<uint32_t*>(pair_at(to[u], tt[u])) = pair[u];
      else if (part < 3) *reinterpret_cast<uint16_t*>(pair_at(to[u], tt[u])) = (uint16_t)pair[u];
    }
  }
}

}  // namespace

hipError_t launch_kv_tree(const KvTreeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.batch + 1);
  if (a.words == 1) return kv_launch(kv_tree_kernel<1>, grid, 64, s, a);
  if (a.words <= 4) return kv_launch(kv_tree_kernel<4>, grid, 256, s, a);
  return kv_launch(kv_tree_kernel<16>, grid, 1024, s, a);
}

hipError_t launch_kv_commit(const KvCommitArgs& a, hipStream_t s) {
  const int64_t items = (int64_t)a.batch * a.L.Hkv * (a.layers > 0 ? a.layers : 1);
  const dim3 grid((unsigned)((items + 3) / 4));
  switch (a.L.D) {
    case 64: return kv_launch(kv_commit_kernel<64>, grid, 256, s, a);
    case 128: return kv_launch(kv_commit_kernel<128>, grid, 256, s, a);
    case 256: return kv_launch(kv_commit_kernel<256>, grid, 256, s, a);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace agemm
