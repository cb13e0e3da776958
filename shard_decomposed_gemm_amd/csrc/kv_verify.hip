// Verification of drafted tokens against the target's probabilities on gfx950.
//
// At a node, after j rejected children of the draft q without replacement, the
// weights are w_j = max(0, w_{j-1} - c_j q_j) with q_j what is left of q,
// normalised, and c_j = sum w_{j-1}. As every term takes a multiple of q off, all
// of it is one number: w = max(0, p - A q) with A = sum_j Z_{j-1} / D_{j-1},
// Z the sum of w and D that of q without the rejected tokens. (A rejected token x
// has w(x) = 0 from then on: u q_j(x) Z >= w(x) with u < 1 makes the difference
// negative.) So a child is held against three numbers, and only another child
// after a rejection needs a pass over the vocabulary, for Z and D; without q not
// even that: Z = 1 - the p of the rejected ones.
//
// Weights are taken to multiples of 2^-50 (by adding and taking off 4, whose
// neighbours lie that far apart), so that sums in binary64 are exact up to 8 and
// do not depend on how the vocabulary is split.
//
// D divides, and a draft sure of its first token leaves little of it: 1 less the
// rejected q would be off by the binary32 roundings of the whole row (with 2^-23
// left, by a third of it), and 2^-50 is coarse for it too. So q is summed, as a
// multiple of 2^-50 and what that is off by as one of 2^-76, exactly both (of up to
// 2^28 numbers, the latter are below 2^-23 together), once a row, and the rejected
// tokens are taken off in the same two parts. D is off by 2^-77 a token then; below
// 2^-57 a token, where that might be a millionth of it, it counts as nothing. (To
// pass over the drafts that follow leaves the distribution as it is: the rest is
// drawn from w.)
//
// Where no sum but the last is expected, the workgroups of a row's parts each walk
// by themselves and sum, and a second kernel draws. Else one workgroup a sequence
// begins the walk, and the parts' workgroups then take turns: they sum the row
// that the walk has come to, and the one that is done last goes on with the walk
// and tells the others, which wait for that. A wait is bounded: what is not
// finished when one gives up, the last kernel finishes, a workgroup a sequence.
// As the sums are exact, who makes them does not matter.
#include "kv_internal.h"

namespace agemm {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(4))) Quad {  // rows of odd vocabularies are aligned to floats only
  float4v x;
};

constexpr double kGrid = 4.0;
constexpr float kBelowOne = 0x1.fffffep-1f;

__device__ inline float number(float u) { return u > 0.f ? fminf(u, kBelowOne) : 0.f; }
__device__ inline float unit(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // NaN: 0

constexpr int kThreads = 256;
constexpr int kSegments = kThreads / 64;  // of a part, a wave each

// A walk as the words that go between workgroups.
constexpr int kWords = sizeof(KvWalk) / 8;
struct KvWalkWords {
  uint64_t x[kWords];
};

struct Shared {
  int32_t token[kKvNodes];  // -1: outside the vocabulary
  float p[kKvNodes], q[kKvNodes], u[kKvNodes];
  int16_t parent[kKvNodes];
  int32_t path[kKvNodes];  // accepted nodes, then (without q) those rejected at the last of them
  KvWalkWords walk;
};

template <bool DRAWN>
__device__ inline double weight(double A, float p, float q) {
  double w = unit(p);
  if constexpr (DRAWN) w = __builtin_fma(-A, (double)unit(q), w);
  w = w > 0.0 ? w : 0.0;
  return (w + kGrid) - kGrid;
}

struct Parts {
  double coarse, fine;
};
__device__ inline Parts parts_of(float q) {
  constexpr double kFine = 0x1.8p-24;  // its neighbours are 2^-76 apart, on both sides
  const double x = unit(q), coarse = (x + kGrid) - kGrid;
  return {coarse, ((x - coarse) + kFine) - kFine};
}
constexpr double kLeast = 0x1p-57;  // of what is left of q, times the vocabulary

struct Rows {
  int64_t row0;
  int n;
  bool usable;
};
__device__ inline Rows rows_of(const KvVerifyArgs& a, int b) {
  const int start = a.q_start[b], end = a.q_start[b + 1];
  const int64_t n = (int64_t)end - start;
  const bool usable = n >= 0 && n <= a.max_q && start >= 0 && end <= a.tokens;
  return {start, usable ? (int)n : 0, usable};
}

// The tree, and p and q of every draft at its parent, to LDS.
template <bool DRAWN>
__device__ inline void load_tree(const KvVerifyArgs& a, const Rows& r, Shared& s, bool tell) {
  for (int i = threadIdx.x; i < r.n; i += kThreads) {
    const int64_t row = r.row0 + i;
    const int parent = a.parent[row];
    const int64_t token = a.token[row];
    const float u = a.u[row];
    const bool ok = i > 0 ? parent >= -1 && parent < i : parent == -1;
    const bool known = token >= 0 && token < a.vocab;
    if (tell && !ok) kv_report(a.err, kKvParent, row, parent);
    if (tell && i > 0 && !known) kv_report(a.err, kKvToken, row, token);
    s.parent[i] = (int16_t)(ok ? parent : -1);
    s.token[i] = known ? (int)token : -1;
    s.u[i] = number(u);
    if (ok && known && parent >= 0) {
      s.p[i] = unit(a.p[(r.row0 + parent) * a.p_stride + token]);
      if constexpr (DRAWN) s.q[i] = unit(a.q[(r.row0 + parent) * a.q_stride + token]);
    }
  }
}

// Goes on with the walk from w, by one wave, until it needs a sum or ends.
template <bool DRAWN>
__device__ inline void go_on(Shared& s, KvWalk w, int n, int lane) {
  w.wants = 0;
  // Node `base` + lane, in registers: most trees are one such group.
  int base = -1, parent, token;
  float np, nq = 0.f, nu;
  auto group = [&](int i0) {
    if (base == i0) return;
    base = i0;
    const int i = i0 + lane < n ? i0 + lane : n - 1;
    parent = i0 + lane < n ? s.parent[i] : -2;
    token = s.token[i];
    np = s.p[i];
    if constexpr (DRAWN) nq = s.q[i];
    nu = s.u[i];
  };
  auto number_of = [](float x, int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l)); };
  for (;;) {
    // the next child of the node, and whether an earlier one had its token
    int c = -1;
    for (int i0 = w.last & ~63; i0 < n && c < 0; i0 += 64) {
      group(i0);
      const uint64_t is = __ballot(i0 + lane > w.last && parent == w.node);
      if (is) c = i0 + __builtin_ctzll(is);
    }
    if (c < 0) break;
    const int l = c & 63, x = __builtin_amdgcn_readlane(token, l);
    bool again = x < 0 || __any(lane < l && parent == w.node && token == x);
    for (int i = (w.node & ~63) + lane; i < base && !again; i += 64) again = __any(s.parent[i] == w.node && s.token[i] == x);
    if (again || (!w.pending && !(w.Z > 0.0 && w.D > 0.0))) {
      w.last = c;
      continue;
    }
    if (w.pending) {
      w.wants = 1;
      break;
    }
    w.last = c;
    const double p = number_of(np, l), u = number_of(nu, l);
    bool take;
    if constexpr (DRAWN) {
      const double q = number_of(nq, l), left = __builtin_fma(-w.A, q, p);
      take = u * q * w.Z < (left > 0.0 ? left : 0.0) * w.D;
      if (!take) {
        const Parts x = parts_of((float)q);
        w.A += w.Z / w.D;
        w.coarse -= x.coarse;
        w.fine -= x.fine;
        w.pending = 1;
      }
    } else {
      take = u * w.Z < p;
      if (!take) {
        w.Z -= p;
        if (lane == 0) s.path[w.count + w.rejects] = c;
        ++w.rejects;
      }
    }
    if (take) {
      if (lane == 0) s.path[w.count] = c;
      ++w.count;
      w.node = c;
      w.rejects = w.pending = w.known = 0;
      w.A = w.coarse = w.fine = 0.0;
      w.Z = w.D = 1.0;
    }
  }
  if (lane == 0) s.walk = __builtin_bit_cast(KvWalkWords, w);
}

// x of another lane as the DPP control says, 0 where there is none.
template <int CTRL, int ROWS>
__device__ inline double moved(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over this lane and the earlier ones.
__device__ inline double sum_up_to(double x) {
  x += moved<0x111, 0xf>(x);  // row_shr:1
  x += moved<0x112, 0xf>(x);  // row_shr:2
  x += moved<0x114, 0xf>(x);  // row_shr:4
  x += moved<0x118, 0xf>(x);  // row_shr:8
  x += moved<0x142, 0xa>(x);  // row_bcast:15
  x += moved<0x143, 0xc>(x);  // row_bcast:31
  return x;
}
__device__ inline double lane_of(double x, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ inline double wave_sum(double x) { return lane_of(sum_up_to(x), 63); }

// Begins the walk of a sequence; `keeps`: and leaves how far it has come. False if there is nothing to walk.
template <bool DRAWN>
__device__ inline bool begin(const KvVerifyArgs& a, int b, Shared& s, bool keeps, int64_t& row0) {
  const int tid = threadIdx.x;
  const Rows r = rows_of(a, b);
  row0 = r.row0;
  if (r.n == 0) {
    if (keeps && tid == 0) {
      a.count[b] = 0;
      a.next[b] = -1;
      a.states[b].walk.done = 1;
      if (!r.usable) kv_report(a.err, kKvRows, b, (int64_t)a.q_start[b + 1] - a.q_start[b]);
    }
    return false;
  }
  load_tree<DRAWN>(a, r, s, keeps);
  if (tid == 0) s.path[0] = 0;
  __syncthreads();
  if (tid < 64) go_on<DRAWN>(s, KvWalk{0.0, 1.0, 1.0, 0.0, 0.0, 0, 0, 1, 0, 0, 0, 0, 0}, r.n, tid);
  __syncthreads();
  if (keeps) {
    const KvWalk w = __builtin_bit_cast(KvWalk, s.walk);
    // rejected ones as their tokens, which the draw leaves out
    for (int i = tid; i < r.n; i += kThreads)
      a.path[r.row0 + i] = i < w.count ? s.path[i] : i < w.count + w.rejects ? s.token[s.path[i]] : -1;
    if (tid == 0) a.states[b].walk = w;
  }
  return true;
}

// A wave's sums of tokens t0 .. t1 - 1 of a row: of the weights and the lanes' `sum`; with REST of q too.
struct Sums {
  double x[kKvSums];
  __device__ double of(int k) const { return k == 0 ? x[0] : k == 1 ? x[1] : x[2]; }
};
template <bool DRAWN, bool REST>
__device__ inline Sums sum_segment(const float* p, const float* q, double A, int t0, int t1, int lane, double sum) {
  Sums s = {{sum, 0.0, 0.0}};
  auto add = [&](float x, float y) {
    s.x[0] += weight<DRAWN>(A, x, y);
    if constexpr (REST) {
      const Parts z = parts_of(y);
      s.x[1] += z.coarse;
      s.x[2] += z.fine;
    }
  };
  int t = t0 + 4 * lane;
#pragma unroll 4
  for (; t + 4 <= t1; t += 256) {
    const float4v x = reinterpret_cast<const Quad*>(p + t)->x, y = DRAWN ? reinterpret_cast<const Quad*>(q + t)->x : x;
#pragma unroll
    for (int i = 0; i < 4; ++i) add(x[i], y[i]);
  }
  for (; t < t1; ++t) add(p[t], q[t]);
#pragma unroll
  for (int k = 0; k < (REST ? kKvSums : 1); ++k) s.x[k] = wave_sum(s.x[k]);
  return s;
}

__device__ inline double load_sum(const double* p) {
  return __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}
__device__ inline void store_sum(double* p, double x) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The row that a walk has come to, and its sums.
template <bool DRAWN>
struct Row {
  const float *p, *q;
  double A;
  int segment, vocab;

  __device__ Row(const KvVerifyArgs& a, int64_t row0, const KvWalk& w)
      : p(a.p + (row0 + w.node) * a.p_stride), q(DRAWN ? a.q + (row0 + w.node) * a.q_stride : p), A(w.A),
        segment(a.plan.part / kSegments), vocab(a.vocab) {}
  __device__ int first(int i) const {  // token of segment i
    const int64_t t = (int64_t)i * segment;
    return t < vocab ? (int)t : vocab;
  }
  // `rest`: of q too (what the walk wants to go on)
  __device__ Sums sum(int i, int lane, bool rest, double start = 0.0) const {
    if constexpr (DRAWN)
      if (rest) return sum_segment<true, true>(p, q, A, first(i), first(i + 1), lane, start);
    return sum_segment<DRAWN, false>(p, q, A, first(i), first(i + 1), lane, start);
  }
};

struct Meeting {
  double sums[kKvSums][kKvParts * kSegments];  // of the segments of all parts
  double waves[kKvSums][kSegments];
  int found, told;
};
__device__ inline double total_of(const Meeting& m, int segments, int k = 0) {  // the same in all waves
  double x = 0.0;
  for (int i = threadIdx.x & 63; i < segments; i += 64) x += m.sums[k][i];
  return wave_sum(x);
}
// The walk wants q's sum: once a row, as the rejected tokens' q comes off it.
__device__ inline bool wants_rest(const KvWalk& w) { return w.wants && !w.known; }
// The sums that the walk wanted are there.
__device__ inline void has_sums(KvWalk& w, const Meeting& m, int segments, int vocab) {
  w.Z = total_of(m, segments);
  if (!w.known) {
    w.coarse += total_of(m, segments, 1);
    w.fine += total_of(m, segments, 2);
    w.known = 1;
  }
  w.D = w.coarse + w.fine;
  if (!(w.D > vocab * kLeast)) w.D = 0.0;
  w.pending = 0;
}
template <bool DRAWN>
__device__ inline void sum_all(Meeting& m, const Row<DRAWN>& row, int segments, bool rest) {
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < segments; i += kSegments) {
    const Sums s = row.sum(i, lane, rest);
    if (lane < (rest ? kKvSums : 1)) m.sums[lane][i] = s.of(lane);
  }
  __syncthreads();
}

// Draws from the row that the walk w has ended at, whose sums are there, and
// writes the sequence's results. `tree`: s has the tree, which the path follows
// from; else the path is written, and s.token has the rejected tokens.
template <bool DRAWN>
__device__ inline void draw(const KvVerifyArgs& a, int b, Shared& s, Meeting& m, KvWalk w, Row<DRAWN> row, int64_t row0, int n,
                            float u0, bool tree) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, segments = a.plan.parts * kSegments;
  double all = total_of(m, segments);
  int rejects = w.rejects;
  if (!(all > 0.0)) {  // nothing left: p itself
    w.A = 0.0;
    rejects = 0;
    __syncthreads();
    row = Row<DRAWN>(a, row0, w);
    sum_all(m, row, segments, false);
    all = total_of(m, segments);
  }
  constexpr int kNone = 0x7fffffff;
  int token = -1;
  if (all > 0.0) {
    const double x = (double)number(u0) * all;
    // The first segment whose sum with those before it passes the number, in every wave: four segments a lane.
    static_assert(kKvParts * kSegments == 4 * 64, "all segments in a wave");
    double v[8], below = 0.0;
    int at = -1;
    {
      double own = 0.0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = 4 * lane + i < segments ? m.sums[0][4 * lane + i] : 0.0;
        own += v[i];
      }
      double run = sum_up_to(own) - own, before = 0.0;  // exact where all sums are
      int hit = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (hit < 0 && v[i] > 0.0 && run + v[i] > x) {
          hit = 4 * lane + i;
          before = run;
        }
        run += v[i];
      }
      const uint64_t hits = __ballot(hit >= 0);
      if (hits) {
        const int l = __builtin_ctzll(hits);
        at = __builtin_amdgcn_readlane(hit, l);
        below = lane_of(before, l);
      } else {  // only by rounding, where sums are not exact: the last one with a weight
        for (int i = 0; i < segments; ++i)
          if (m.sums[0][i] > 0.0) at = i;
        for (int i = 0; i < at; ++i) below += m.sums[0][i];
      }
    }
    // Then the first token. Rejected ones of the segment are left out.
    const int t1 = row.first(at + 1);
    __syncthreads();
    if (tid == 0) m.told = 0;
    __syncthreads();
    if constexpr (!DRAWN) {
      for (int k = tid; k < rejects; k += kThreads) {
        const int t = s.token[k];
        if (t >= row.first(at) && t < t1) s.path[atomicAdd(&m.told, 1)] = t;
      }
      __syncthreads();
    }
    const int out = m.told;
    int end = -1;
    for (int t0 = row.first(at); t0 < t1 && token < 0; t0 += 8 * kThreads) {
      const int t = t0 + 8 * tid;
      float px[8] = {}, qx[8] = {};
      if (t + 8 <= t1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4v p4 = reinterpret_cast<const Quad*>(row.p + t + 4 * i)->x;
          const float4v q4 = DRAWN ? reinterpret_cast<const Quad*>(row.q + t + 4 * i)->x : p4;
#pragma unroll
          for (int k = 0; k < 4; ++k) px[4 * i + k] = p4[k], qx[4 * i + k] = q4[k];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t + i < t1) px[i] = row.p[t + i], qx[i] = row.q[t + i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = weight<DRAWN>(w.A, px[i], qx[i]);
      if constexpr (!DRAWN)
        for (int k = 0; k < out; ++k) {
          const int z = s.path[k] - t;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (z == i) v[i] = 0.0;
        }
      double own = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (v[i] > 0.0) end = t + i;
        own += v[i];
      }
      const double upto = sum_up_to(own);
      if (lane == 63) m.waves[0][wave] = upto;
      if (tid == 0) m.found = kNone;
      __syncthreads();
      double run = below + (upto - own);
#pragma unroll
      for (int i = 0; i < kSegments; ++i) {
        if (i < wave) run += m.waves[0][i];
        below += m.waves[0][i];
      }
      int hit = kNone;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (hit == kNone && v[i] > 0.0 && run + v[i] > x) hit = t + i;
        run += v[i];
      }
      if (hit != kNone) atomicMin(&m.found, hit);
      __syncthreads();
      if (m.found != kNone) token = m.found;
      __syncthreads();
    }
    if (token < 0) {  // see above
      if (tid == 0) m.found = -1;
      __syncthreads();
      atomicMax(&m.found, end);
      __syncthreads();
      token = m.found;
    }
  } else if (tid == 0) {
    kv_report(a.err, kKvWeight, b, 0);
  }
  __syncthreads();
  if (tree && tid == 0)
    for (int i = w.count - 1, node = w.node; i >= 0; node = s.parent[node], --i) s.path[i] = node;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads)
    if (i >= w.count) a.path[row0 + i] = -1;
    else if (tree) a.path[row0 + i] = s.path[i];
  if (tid == 0) {
    a.count[b] = w.count;
    a.next[b] = token;
    a.states[b].walk.done = 1;
  }
}

// The rounds' beginning.
template <bool DRAWN>
__global__ __launch_bounds__(kThreads) void kv_verify_begin_kernel(KvVerifyArgs a) {
  __shared__ Shared s;
  int64_t row0;
  if (threadIdx.x == 0) a.states[blockIdx.x].arrived = a.states[blockIdx.x].turn = 0;
  begin<DRAWN>(a, blockIdx.x, s, true, row0);
}

// The rounds: 16 trees of 25 drawn nodes on 131072 tokens take 33 to 37 us a call
// where no tree wants more than four sums and 63 where one wants ten, 5.0 a turn,
// nearly all of it latency (without q's sums a call takes 1.4 to 2.1 less). What
// workgroups tell each other goes past the caches of their XCDs (relaxed accesses at
// the device's scope), and is there before the counter or turn that announces it: one
// wave stores and waits, which a release (the write-back of all of the cache, 20 us a
// call of 1024 workgroups) would do too.
__device__ inline void stores_are_there() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("" ::: "memory");
}
template <bool DRAWN>
__global__ __launch_bounds__(kThreads) void kv_verify_rounds_kernel(KvVerifyArgs a) {
  __shared__ Shared s;
  __shared__ Meeting m;
  const int b = blockIdx.x / a.plan.parts, part = blockIdx.x - b * a.plan.parts, segments = a.plan.parts * kSegments;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  KvVerifyState& state = a.states[b];
  KvWalk w = state.walk;
  if (w.done) return;
  const int64_t row0 = a.q_start[b];
  const int n = a.q_start[b + 1] - (int)row0;
  const float u0 = a.u[row0];
  load_tree<DRAWN>(a, Rows{row0, n, true}, s, false);
  double* sums = a.sums + (int64_t)b * kKvSums * segments;
  for (uint32_t turn = 1;; ++turn) {
    const Row<DRAWN> row(a, row0, w);
    const Sums mine = row.sum(part * kSegments + wave, lane, wants_rest(w));
    const int kinds = wants_rest(w) ? kKvSums : 1;
    if (lane < kinds) m.waves[lane][wave] = mine.of(lane);
    __syncthreads();
    if (wave == 0) {
      const int k = lane / kSegments, i = lane % kSegments;
      if (k < kinds) store_sum(sums + k * segments + part * kSegments + i, m.waves[k][i]);
      stores_are_there();
      if (lane == 0) m.found = __hip_atomic_fetch_add(&state.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == a.plan.parts * turn;
    }
    __syncthreads();
    if (m.found) {  // the last one
      if (tid < segments) {
        double x[kKvSums];
#pragma unroll
        for (int k = 0; k < kKvSums; ++k)  // all on their way at once
          if (k < kinds) x[k] = load_sum(sums + k * segments + tid);
#pragma unroll
        for (int k = 0; k < kKvSums; ++k)
          if (k < kinds) m.sums[k][tid] = x[k];
      }
      __syncthreads();
      if (!w.wants) {
        draw<DRAWN>(a, b, s, m, w, row, row0, n, u0, true);
        return;
      }
      has_sums(w, m, segments, a.vocab);
      if (wave == 0) {
        go_on<DRAWN>(s, w, n, lane);
        if (lane < kWords)
          __hip_atomic_store(reinterpret_cast<uint64_t*>(&state.walk) + lane, s.walk.x[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        stores_are_there();
        if (lane == 0) __hip_atomic_store(&state.turn, turn, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    } else {
      if (!w.wants) return;  // the last one draws
      if (wave == 0) {
        const uint64_t t0 = wall_clock64();
        bool told;
        while (!(told = __hip_atomic_load(&state.turn, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= turn) &&
               wall_clock64() - t0 < (uint64_t)a.patience)
          __builtin_amdgcn_s_sleep(1);
        asm volatile("" ::: "memory");
        if (told && lane < kWords)
          s.walk.x[lane] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(&state.walk) + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (lane == 0) m.told = told;
      }
      __syncthreads();
      if (!m.told) return;  // the last kernel finishes it
    }
    __syncthreads();
    w = __builtin_bit_cast(KvWalk, s.walk);
    __syncthreads();
  }
}

// Where the walk is expected to need no sum but the last: every part walks for
// itself and sums, and a second kernel draws. (With a kernel that begins, and the
// last part's workgroup drawing, 64 chains of 6 take 26 us, not 20.) Those chains,
// on 131072 tokens, take 13.8 us here, the rows at 4.9 TB/s with the walk that
// comes first; one chain on 32768 4.6, latency.
template <bool DRAWN>
__global__ __launch_bounds__(kThreads) void kv_verify_sum_kernel(KvVerifyArgs a) {
  __shared__ Shared s;
  const int b = blockIdx.x / a.plan.parts, part = blockIdx.x - b * a.plan.parts;
  const int lane = threadIdx.x & 63, i = part * kSegments + (threadIdx.x >> 6);
  int64_t row0;
  if (!begin<DRAWN>(a, b, s, part == 0, row0)) return;
  const KvWalk w = __builtin_bit_cast(KvWalk, s.walk);
  const Row<DRAWN> row(a, row0, w);
  double start = 0.0;
  if constexpr (!DRAWN)  // rejected tokens have no weight
    for (int k = lane; k < w.rejects; k += 64) {
      const int node = s.path[w.count + k], t = s.token[node];
      if (t >= row.first(i) && t < row.first(i + 1)) start -= weight<false>(0.0, s.p[node], 0.f);
    }
  const Sums mine = row.sum(i, lane, wants_rest(w), start);
  const int segments = a.plan.parts * kSegments;
  if (lane < (wants_rest(w) ? kKvSums : 1)) a.sums[((int64_t)b * kKvSums + lane) * segments + i] = mine.of(lane);
}
// SUMMED: the sums that the walk wants are there; else only what the rounds left is
// to do. Latency-bound: 4.0 us for a chain, 6.2 for 64, 4.6 with nothing left.
template <bool DRAWN, bool SUMMED>
__global__ __launch_bounds__(kThreads) void kv_verify_draw_kernel(KvVerifyArgs a) {
  __shared__ Shared s;
  __shared__ Meeting m;
  const int b = blockIdx.x, tid = threadIdx.x, segments = a.plan.parts * kSegments;
  KvWalk w = a.states[b].walk;
  const Rows r = rows_of(a, b);
  const int64_t row0 = r.row0;
  const int n = r.n;
  const double* sums = a.sums + (int64_t)b * kKvSums * segments + tid;
  if (SUMMED && tid < segments) m.sums[0][tid] = *sums;
  int known[kKvNodes / kThreads];
  if constexpr (!DRAWN) {
#pragma unroll
    for (int i = 0; i < kKvNodes / kThreads; ++i)
      if (tid + i * kThreads < n) known[i] = a.path[row0 + tid + i * kThreads];
  }
  if (w.done) return;
  Row<DRAWN> row(a, row0, w);
  const float u0 = a.u[row0];
  const bool tree = !SUMMED || w.wants;
  if (SUMMED && wants_rest(w) && tid < segments)
    for (int k = 1; k < kKvSums; ++k) m.sums[k][tid] = sums[k * segments];
  if (tree) {
    load_tree<DRAWN>(a, Rows{row0, n, true}, s, false);
  } else if constexpr (!DRAWN) {
#pragma unroll
    for (int i = 0; i < kKvNodes / kThreads; ++i) {
      const int k = tid + i * kThreads - w.count;
      if (k >= 0 && k < w.rejects) s.token[k] = known[i];
    }
  }
  __syncthreads();
  if (!SUMMED) sum_all(m, row, segments, wants_rest(w));
  while (w.wants) {
    has_sums(w, m, segments, a.vocab);
    __syncthreads();
    if (tid < 64) go_on<DRAWN>(s, w, n, tid);
    __syncthreads();
    w = __builtin_bit_cast(KvWalk, s.walk);
    row = Row<DRAWN>(a, row0, w);
    sum_all(m, row, segments, wants_rest(w));
  }
  draw<DRAWN>(a, b, s, m, w, row, row0, n, u0, tree);
}

template <bool DRAWN>
hipError_t launch(const KvVerifyArgs& a, hipStream_t s) {
  const dim3 sequences((unsigned)a.batch), parts((unsigned)(a.batch * a.plan.parts));
  hipError_t e;
  if constexpr (DRAWN)
    if (a.plan.rounds) {
      e = kv_launch(kv_verify_begin_kernel<true>, sequences, kThreads, s, a);
      if (e == hipSuccess) e = kv_launch(kv_verify_rounds_kernel<true>, parts, kThreads, s, a);
      return e == hipSuccess ? kv_launch(kv_verify_draw_kernel<true, false>, sequences, kThreads, s, a) : e;
    }
  e = kv_launch(kv_verify_sum_kernel<DRAWN>, parts, kThreads, s, a);
  return e == hipSuccess ? kv_launch(kv_verify_draw_kernel<DRAWN, true>, sequences, kThreads, s, a) : e;
}

}  // namespace

hipError_t launch_kv_verify(const KvVerifyArgs& a, hipStream_t s) {
  return a.q ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace agemm
