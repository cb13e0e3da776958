// Verification of drafted tokens against the target's probabilities on gfx950.
//
// At a node, after j rejected children of the draft q without replacement, the
// weights are w_j = max(0, w_{j-1} - c_j q_j) with q_j what is left of q,
// normalised, and c_j = sum w_{j-1}. As every term takes a multiple of q off, all
// of it is one number: w = max(0, p - A q) with A = sum_j Z_{j-1} / (1 - S_{j-1}),
// Z the sum of w and S the q of the rejected tokens. (A rejected token x has
// w(x) = 0 from then on: u q_j(x) Z >= w(x) with u < 1 makes the difference
// negative.) So a child is held against three numbers, and only another child
// after a rejection needs a pass over the vocabulary, for Z; without q not even
// that: Z = 1 - the p of the rejected ones.
//
// Weights are taken to multiples of 2^-50 (by adding and taking off 4, whose
// neighbours lie that far apart), so that sums in binary64 are exact up to 8 and
// do not depend on how the vocabulary is split.
//
// Bytes: the row of p (and q) that the last token is drawn from. The walk is
// latency: parents, tokens and numbers, then p and q of every draft, then some
// 0.2 us a level. Every workgroup of a part walks by itself, which costs no
// launch; the sums of the parts it stores are read by the next launch.
#include "kv_internal.h"

namespace agemm {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(4))) Quad {  // rows of odd vocabularies are aligned to floats only
  float4v x;
};

constexpr double kGrid = 4.0;
constexpr float kBelowOne = 0x1.fffffep-1f;

__device__ inline float unit(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // NaN: 0

struct Shared {
  int32_t token[kKvNodes];  // -1: outside the vocabulary
  float p[kKvNodes], q[kKvNodes], u[kKvNodes];
  int16_t parent[kKvNodes];
  int16_t path[kKvNodes];
  int32_t rejected[kKvNodes];  // tokens, at the current node, without q
  // what the walk left
  int32_t node, count, rejects, wants;  // wants: 1 if it needs a sum to go on, 0 at its end
  int32_t last;                         // the child tried last
  double A, S, Z;
  bool pending;  // Z is out of date
};

template <bool DRAWN>
__device__ inline double weight(double A, float p, float q) {
  double w = unit(p);
  if constexpr (DRAWN) w = __builtin_fma(-A, (double)unit(q), w);
  w = w > 0.0 ? w : 0.0;
  return (w + kGrid) - kGrid;
}

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
  for (int i = threadIdx.x; i < r.n; i += blockDim.x) {
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
    s.u[i] = u > 0.f ? fminf(u, kBelowOne) : 0.f;
    if (ok && known && parent >= 0) {
      s.p[i] = unit(a.p[(r.row0 + parent) * a.p_stride + token]);
      if constexpr (DRAWN) s.q[i] = unit(a.q[(r.row0 + parent) * a.q_stride + token]);
    }
  }
}

// Goes on with the walk, by one wave, until it needs a sum or ends.
template <bool DRAWN>
__device__ inline void walk(Shared& s, int n, int lane) {
  int cur = s.node, last = s.last, count = s.count, rejects = s.rejects;
  double A = s.A, S = s.S, Z = s.Z;
  bool pending = s.pending;
  int wants = 0;
  for (;;) {
    // the next child of cur, and whether an earlier one had its token
    int c = -1;
    for (int i0 = last & ~63; i0 < n && c < 0; i0 += 64) {
      const int i = i0 + lane;
      const uint64_t is = __ballot(i > last && i < n && s.parent[i] == cur);
      if (is) c = i0 + __builtin_ctzll(is);
    }
    if (c < 0) break;
    const int x = s.token[c];
    bool again = x < 0;
    for (int i0 = cur & ~63; i0 < c && !again; i0 += 64) {
      const int i = i0 + lane;
      again = __any(i > cur && i < c && s.parent[i] == cur && s.token[i] == x);
    }
    if (again || (DRAWN && !(S < 1.0)) || (!pending && !(Z > 0.0))) {
      last = c;
      continue;
    }
    if (pending) {
      wants = 1;
      break;
    }
    last = c;
    const double p = s.p[c], u = s.u[c];
    bool take;
    if constexpr (DRAWN) {
      const double q = s.q[c], w = __builtin_fma(-A, q, p);
      take = u * q * Z < (w > 0.0 ? w : 0.0) * (1.0 - S);
      if (!take) {
        A += Z / (1.0 - S);
        S += q;
        pending = true;
      }
    } else {
      take = u * Z < p;
      if (!take) {
        Z -= p;
        if (lane == 0) s.rejected[rejects] = x;
        ++rejects;
      }
    }
    if (take) {
      if (lane == 0) s.path[count] = (int16_t)c;
      ++count;
      cur = c;
      rejects = 0;
      A = S = 0.0;
      Z = 1.0;
      pending = false;
    }
  }
  if (lane == 0) {
    s.node = cur;
    s.last = last;
    s.count = count;
    s.rejects = rejects;
    s.A = A;
    s.S = S;
    s.Z = Z;
    s.pending = pending;
    s.wants = wants;
  }
}

__device__ inline void start_walk(Shared& s) {
  s.node = s.last = s.rejects = 0;
  s.count = 1;
  s.path[0] = 0;
  s.A = s.S = 0.0;
  s.Z = 1.0;
  s.pending = false;
}

__device__ inline double wave_sum(double x) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
  return x;
}

// Sum of the weights of tokens t0 .. t1 - 1 over a workgroup, valid in thread 0.
template <bool DRAWN, int THREADS>
__device__ inline double sum_part(const KvVerifyArgs& a, const Rows& r, const Shared& s, int t0, int t1, double* meet) {
  const float* p = a.p + (r.row0 + s.node) * a.p_stride;
  const float* q = DRAWN ? a.q + (r.row0 + s.node) * a.q_stride : p;
  const double A = s.A;
  double sum = 0.0;
  int t = t0 + 4 * (int)threadIdx.x;
#pragma unroll 4
  for (; t + 4 <= t1; t += 4 * THREADS) {
    const float4v x = reinterpret_cast<const Quad*>(p + t)->x, y = DRAWN ? reinterpret_cast<const Quad*>(q + t)->x : x;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += weight<DRAWN>(A, x[i], y[i]);
  }
  for (; t < t1; ++t) sum += weight<DRAWN>(A, p[t], q[t]);
  if constexpr (!DRAWN)  // rejected tokens have no weight
    for (int i = threadIdx.x; i < s.rejects; i += THREADS) {
      const int x = s.rejected[i];
      if (x >= t0 && x < t1) sum -= weight<false>(0.0, p[x], 0.f);
    }
  sum = wave_sum(sum);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) sum += meet[w];
  return sum;
}

// Round k: walks with the sums of the rounds before it, and sums this
// workgroup's part of what the walk asks for then, or of the last draw.
constexpr int kRoundThreads = 256;
template <bool DRAWN>
__global__ __launch_bounds__(kRoundThreads) void kv_verify_round_kernel(KvVerifyArgs a, int round) {
  __shared__ Shared s;
  __shared__ double meet[kRoundThreads / 64];
  const int b = blockIdx.x / a.plan.parts, part = blockIdx.x - b * a.plan.parts, lane = threadIdx.x & 63;
  const Rows r = rows_of(a, b);
  if (r.n == 0) return;
  load_tree<DRAWN>(a, r, s, part == 0 && round == 0);
  if (threadIdx.x == 0) start_walk(s);
  double* sums = a.ws + (int64_t)b * a.plan.rounds * a.plan.parts;
  __syncthreads();
  bool done = false;
  for (int k = 0; k <= round && !done; ++k) {
    if (threadIdx.x < 64) {
      if (k > 0) {
        const double z = wave_sum(lane < a.plan.parts ? sums[(k - 1) * a.plan.parts + lane] : 0.0);
        if (lane == 0) {
          s.Z = z;
          s.pending = false;
        }
      }
      walk<DRAWN>(s, r.n, lane);
    }
    __syncthreads();
    done = !s.wants;
    if (done && k < round) return;  // an earlier round summed the last draw
    __syncthreads();
  }
  const int t0 = part * a.plan.part, t1 = t0 + a.plan.part < a.vocab ? t0 + a.plan.part : a.vocab;
  const double sum = sum_part<DRAWN, kRoundThreads>(a, r, s, t0, t1, meet);
  if (threadIdx.x == 0) sums[round * a.plan.parts + part] = sum;
}

// Walks with the sums of all rounds and sums what they left, then draws: the
// part that holds the number, and in it the token.
constexpr int kPickThreads = 1024;
template <bool DRAWN>
__global__ __launch_bounds__(kPickThreads) void kv_verify_pick_kernel(KvVerifyArgs a) {
  __shared__ Shared s;
  __shared__ double meet[kPickThreads / 64];
  __shared__ double parts[kKvParts];
  __shared__ int found;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Rows r = rows_of(a, b);
  if (r.n == 0) {
    if (tid == 0) {
      a.count[b] = 0;
      a.next[b] = -1;
      if (!r.usable) kv_report(a.err, kKvRows, b, (int64_t)a.q_start[b + 1] - a.q_start[b]);
    }
    return;
  }
  load_tree<DRAWN>(a, r, s, false);
  if (tid == 0) start_walk(s);
  const double* sums = a.ws + (int64_t)b * a.plan.rounds * a.plan.parts;
  __syncthreads();
  // `parts` has the sums that the walk asks for next.
  auto fetch = [&](int k) {
    if (k < a.plan.rounds) {
      if (tid < a.plan.parts) parts[tid] = sums[k * a.plan.parts + tid];
    } else {
      for (int i = 0; i < a.plan.parts; ++i) {
        const int t0 = i * a.plan.part, t1 = t0 + a.plan.part < a.vocab ? t0 + a.plan.part : a.vocab;
        const double sum = sum_part<DRAWN, kPickThreads>(a, r, s, t0, t1, meet);
        if (tid == 0) parts[i] = sum;
      }
    }
    __syncthreads();
  };
  for (int k = 0;; ++k) {
    if (wave == 0) walk<DRAWN>(s, r.n, lane);
    __syncthreads();
    fetch(k);
    if (!s.wants) break;
    if (wave == 0) {
      const double z = wave_sum(lane < a.plan.parts ? parts[lane] : 0.0);
      if (lane == 0) {
        s.Z = z;
        s.pending = false;
      }
    }
    __syncthreads();
  }
  auto total = [&] { return wave_sum(lane < a.plan.parts ? parts[lane] : 0.0); };  // the same in all waves
  double all = total();
  if (!(all > 0.0)) {  // nothing left: p itself
    __syncthreads();
    if (tid == 0) {
      s.A = 0.0;
      s.rejects = 0;
    }
    __syncthreads();
    fetch(a.plan.rounds);
    all = total();
  }
  for (int i = tid; i < r.n; i += kPickThreads) a.path[r.row0 + i] = i < s.count ? s.path[i] : -1;
  if (tid == 0) a.count[b] = s.count;
  if (!(all > 0.0)) {
    if (tid == 0) {
      a.next[b] = -1;
      kv_report(a.err, kKvWeight, b, 0);
    }
    return;
  }

  // The first part whose sum with those before it passes the number.
  const double x = (double)s.u[0] * all;
  double below = 0.0;
  int part = 0;
  for (int last = 0;; ++part) {
    if (parts[part] > 0.0) last = part;
    if (below + parts[part] > x) break;
    if (part == a.plan.parts - 1) {  // only by rounding, where sums are not exact
      part = last;
      break;
    }
    below += parts[part];
  }
  const int t0 = part * a.plan.part, t1 = t0 + a.plan.part < a.vocab ? t0 + a.plan.part : a.vocab;
  const float* p = a.p + (r.row0 + s.node) * a.p_stride;
  const float* q = DRAWN ? a.q + (r.row0 + s.node) * a.q_stride : p;
  const double A = s.A;
  int best = -1;  // the last token with a weight so far, should none pass
  for (int tile = t0; tile < t1; tile += 4 * kPickThreads) {
    const int t = tile + 4 * tid;
    double w[4], mine = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = t + i < t1 ? weight<DRAWN>(A, p[t + i], q[t + i]) : 0.0;
      if constexpr (!DRAWN)
        for (int j = 0; j < s.rejects; ++j)
          if (s.rejected[j] == t + i) w[i] = 0.0;
      mine += w[i];
    }
    double upto = mine;  // over the lanes before and this one
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double y = __shfl_up(upto, m);
      if (lane >= m) upto += y;
    }
    __syncthreads();
    if (lane == 63) meet[wave] = upto;
    if (tid == 0) found = 0x7fffffff;
    __syncthreads();
    double before = below, whole = 0.0;
#pragma unroll
    for (int i = 0; i < kPickThreads / 64; ++i) {
      if (i < wave) before += meet[i];
      whole += meet[i];
    }
    double sum = before + (upto - mine);
    int hit = 0x7fffffff, any = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum += w[i];
      if (w[i] > 0.0) {
        any = t + i;
        if (sum > x && hit == 0x7fffffff) hit = t + i;
      }
    }
    if (hit != 0x7fffffff) atomicMin(&found, hit);
    __syncthreads();
    if (found != 0x7fffffff) {
      best = found;
      break;
    }
    best = any > best ? any : best;
    below += whole;
    __syncthreads();
  }
  if (found == 0x7fffffff) {  // see above
    __syncthreads();
    if (tid == 0) found = -1;
    __syncthreads();
    atomicMax(&found, best);
    __syncthreads();
    best = found;
  }
  if (tid == 0) a.next[b] = best;
}

template <class A>
hipError_t launch_round(void (*kernel)(A, int), dim3 grid, hipStream_t s, A a, int round) {
  void* args[] = {&a, &round};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kRoundThreads), args, 0, s);
}

template <bool DRAWN>
hipError_t launch(const KvVerifyArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  for (int k = 0; k < a.plan.rounds && e == hipSuccess; ++k)
    e = launch_round(kv_verify_round_kernel<DRAWN>, dim3((unsigned)(a.batch * a.plan.parts)), s, a, k);
  if (e == hipSuccess) e = kv_launch(kv_verify_pick_kernel<DRAWN>, dim3((unsigned)a.batch), kPickThreads, s, a);
  return e;
}

}  // namespace

hipError_t launch_kv_verify(const KvVerifyArgs& a, hipStream_t s) {
  return a.q ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace agemm
