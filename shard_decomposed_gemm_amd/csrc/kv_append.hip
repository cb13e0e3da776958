// Appending keys and values to the 4-bit paged cache, with the head norms and
// the position rotation of queries and keys in the same pass, and reading
// cached tokens back, on gfx950.
//
// A head row of D channels is the work of 16 lanes, D / 16 consecutive
// channels each, so that a lane's channels are exactly one run of the key
// row's nibbles and one value run c of the block layout, and no nibble changes
// lanes. A wave takes four rows of one token at a time: query rows are normed,
// rotated and written as binary16; key rows are normed, rotated and quantised;
// value rows are quantised. The rotation's partner of channel i, i +-
// rope_dims / 2, is in the lane rope_dims / 2 channels away. Sums and extremes
// over a row are four steps within a row of 16 lanes (DPP rotations).
//
// Bound by HBM: 2 bytes in and out a query channel, 2 in and 1/2 out a key or
// value channel, some 10 operations each. Measured on 16384 tokens of 64 + 2 x 8
// heads (D 128, whole rotation): queries 112 us, 4.8 TB/s of the 4.96 that a
// copy reaches; keys and values 51 us, 1.8 TB/s: some 40 operations a channel,
// and one quad in ten again in binary64, keep the vector units busy 55 % of the
// cycles, and a wave loads, works and stores one after the other.
#include <type_traits>

#include "kv_internal.h"

namespace agemm {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerPass = kThreads / 16;

template <int E>
struct alignas(E * 2) Halves {
  _Float16 x[E];
};

// x of the lane n places on in its row of 16.
template <int n>
__device__ inline float rotated(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + n, 0xf, 0xf, true));
}
template <int n>
__device__ inline double rotated(double x) {
  const int64_t v = __builtin_bit_cast(int64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), 0x120 + n, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (int64_t)hi << 32 | lo);
}
template <class T>
__device__ inline T sum16(T v) {
  v += rotated<8>(v);
  v += rotated<4>(v);
  v += rotated<2>(v);
  return v + rotated<1>(v);
}
__device__ inline float least(float a, float b) { return fminf(a, b); }
__device__ inline double least(double a, double b) { return fmin(a, b); }
template <class T>
__device__ inline T min16(T v) {
  v = least(v, rotated<8>(v));
  v = least(v, rotated<4>(v));
  v = least(v, rotated<2>(v));
  return least(v, rotated<1>(v));
}

// x (this lane's channels of a head row) normed and rotated in place. `partner`
// is the row's lane that holds the rotation's other channels.
enum Rope { kNone, kWhole, kOther };  // no rotation, halves of whole rows, anything else

template <class T, int E, int ROPE>
__device__ inline void norm_rope(T (&x)[E], bool norm, const Halves<E>& w, float eps, int d0, int R, bool interleaved,
                                 int partner, const float (&cs)[E], const float (&sn)[E]) {
  constexpr int D = 16 * E;
  if (norm) {
    T ss = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) ss += x[e] * x[e];
    const T inv = T(1) / sqrt(sum16(ss) * T(1.0 / D) + T(eps));
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] * inv * T((float)w.x[e]);
  }
  if constexpr (ROPE == kWhole) {  // the partner is the lane eight places on
    const T sign = d0 < D / 2 ? T(-1) : T(1);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] * T(cs[e]) + sign * rotated<8>(x[e]) * T(sn[e]);
  } else if constexpr (ROPE == kOther) {
    if (interleaved) {
      if (d0 < R) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const T u = x[e], y = x[e + 1];
          x[e] = u * T(cs[e]) - y * T(sn[e]);
          x[e + 1] = y * T(cs[e]) + u * T(sn[e]);
        }
      }
    } else {
      const T sign = d0 < (R >> 1) ? T(-1) : T(1);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const T y = __shfl(x[e], partner, 16);
        if (d0 < R) x[e] = x[e] * T(cs[e]) + sign * y * T(sn[e]);
      }
    }
  }
}

// Rounded to binary32, then to binary16. The compiler makes one rounding of the
// two, in some forty instructions, unless it is kept from seeing both.
__device__ inline _Float16 half_by_float(double x) {
  float f = (float)x;
  asm("" : "+v"(f));
  return (_Float16)f;
}

// The row's 4-bit form, 16-bit words of this lane's nibbles and the pair (s, b),
// in binary32; false where that cannot be told apart from what binary64 gives
// (some tenth of the quads of rows: of values for ties, which binary16 inputs
// often are).
// x is known to `off` times the row's largest size: s, b and (x - b) / s are
// recomputed at both ends of what their errors allow, or kept away from ties.
template <int E>
__device__ inline bool quantise_fast(const float (&x)[E], float off, uint32_t (&word)[E / 4], _Float16& s, _Float16& b) {
  float lo = x[0], hi = x[0], finite = 0.f;  // finite: a NaN if some x is not finite
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    finite = __builtin_fmaf(x[e], 0.f, finite);
  }
  lo = min16(lo);
  hi = -min16(-hi);
  const float size = fmaxf(-lo, hi), err = off * fmaxf(fabsf(lo), fabsf(hi));
  const float sf = (hi - lo) * (1.f / 15.f), es = err * (2.f / 15.f) + sf * 0x1p-21f;
  s = (_Float16)(sf - es);
  const float sh = (float)s, bf = lo - 16.f * sh;
  const float eb = off > 0.f ? err + fabsf(bf) * 0x1p-22f : 0.f;  // of exact x, bf is the exact number rounded to binary32
  b = (_Float16)(bf - eb);
  bool sure = finite == 0.f && size <= kKvLimit && sh > 0.f && s == (_Float16)(sf + es) && b == (_Float16)(bf + eb);
  const float bh = (float)b, inv = 1.f / sh;
  float k[E], far = 0.f;  // far: the largest distance of (x - b) / s from a whole number
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float t = (x[e] - bh) * inv;
    k[e] = rintf(t);
    far = fmaxf(far, fabsf(t - k[e]));
    k[e] = __builtin_amdgcn_fmed3f(k[e], 16.f, 31.f);
  }
  // x - b, 1 / s and their product: each within 2^-24 of a number below 32 + 1 steps
  sure = sure && far < 0.5f - (err * inv + 32.f * 0x1p-21f);
#pragma unroll
  for (int i = 0; i < E / 4; ++i)  // whole numbers below 2^18: exact
    word[i] = (uint32_t)__builtin_fmaf(__builtin_fmaf(__builtin_fmaf(k[4 * i + 3], 16.f, k[4 * i + 2]), 16.f, k[4 * i + 1]),
                                       16.f, k[4 * i]) - 16 * 0x1111;
  return sure;
}

// The same in binary64, where a nibble next to the border between two is
// decided as the definition says, ties of (x - b) / s to even. x - b and n s are exact for values of
// binary16, so the remainder tells a tie where the product with 1 / s cannot.
template <int E>
__device__ inline bool quantise(double (&x)[E], uint32_t (&word)[E / 4], _Float16& s, _Float16& b) {
  bool bad = false;
  double lo = kKvLimit, up = kKvLimit;  // up: the largest value's negative
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bad |= !(fabs(x[e]) <= kKvLimit);
    x[e] = x[e] == x[e] ? fmin(fmax(x[e], -(double)kKvLimit), (double)kKvLimit) : 0.0;
    lo = fmin(lo, x[e]);
    up = fmin(up, -x[e]);
  }
  lo = min16(lo);
  up = min16(up);
  s = half_by_float((-up - lo) / 15.0);
  const double sd = (double)s;
  b = half_by_float(lo - 16.0 * sd);
  const double bd = (double)b;
  const double inv = sd > 0.0 ? 1.0 / sd : 0.0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const double y = x[e] - bd;
    double k = rint(y * inv);
    const double rest = fma(-k, sd, y);
    if (fabs(rest) * 2.0 == sd && ((int)k & 1)) k += rest > 0.0 ? 1.0 : -1.0;
    const int i = (int)k - 16;  // s = 0: k = 0
    const uint32_t n = i < 0 ? 0 : i > 15 ? 15 : i;
    word[e / 4] = (e & 3 ? word[e / 4] : 0) | n << 4 * (e & 3);
  }
  return bad;
}

enum Role { kQueries, kKeysValues, kBoth };

// Element i of an array that no kernel writes meanwhile, by a scalar load.
__device__ inline int64_t scalar_load(const int64_t* p, uint32_t i) {
  typedef const int64_t __attribute__((address_space(4))) * constant;
  return ((constant)(uintptr_t)p)[i];
}

// A wave works on four rows of one token at a time, a quad: four query heads,
// four keys or four values, so that token, slot and page are scalars and keys
// and values do not diverge. It takes `a.quads` of them in turn, and loads all
// before it works on the first. Queries and keys with values have kernels of
// their own where there are many tokens: quantising takes more registers,
// which would halve the queries' occupancy. With few tokens one launch has
// both (blockIdx.y is the role). D = 16 E.
constexpr int kAhead = 4;

template <int E, int ROLE, int ROPE>
__global__ __launch_bounds__(kThreads, ROLE == kQueries ? (E > 8 ? 4 : 6) : E > 8 ? 2 : 4) void kv_append_kernel(KvAppendArgs a) {
  using H = Halves<E>;
  constexpr int D = 16 * E;
  const bool is_q = ROLE == kBoth ? blockIdx.y == 0 : ROLE == kQueries;
  const int heads = is_q ? a.L.Hq : a.L.Hkv;
  const uint32_t per_head4 = (uint32_t)(heads + 3) >> 2, quads = is_q ? per_head4 : 2 * per_head4;
  const uint32_t all = (uint32_t)a.tokens * quads;  // below 2^28
  // Workgroups go to the 8 XCDs in turn: those of the 32 tokens of a block,
  // whose values share lines, go to one, so that its L2 puts the lines
  // together. The last ones, short of 8 blocks, go as they come.
  uint32_t wg = blockIdx.x;
  if (!is_q) {
    const uint32_t n = a.near, g = wg / (8 * n), in = wg - g * 8 * n;
    if ((g + 1) * 8 * n <= gridDim.x) wg = g * 8 * n + (in & 7) * n + (in >> 3);
  }
  const uint32_t begin = (wg * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * a.quads;
  if (begin >= all) return;
  const uint32_t count = all - begin < a.quads ? all - begin : a.quads;
  const int lane = threadIdx.x & 15, sub = (threadIdx.x >> 4) & 3;  // of the row, row of the quad
  const int d0 = lane * E;

  struct Quad {
    uint32_t t, i;  // token, quad of the token
  };
  const uint32_t t0 = __builtin_amdgcn_readfirstlane(begin / quads);
  const Quad start = {t0, begin - t0 * quads};
  auto after = [&](Quad x) { return x.i + 1 < quads ? Quad{x.t, x.i + 1} : Quad{x.t + 1, 0}; };
  auto first_head = [&](Quad x) { return (int)(x.i < per_head4 ? x.i : x.i - per_head4) * 4; };

  // The rows, four ahead.
  const int64_t q_lane = sub * a.q_hs + d0, k_lane = sub * a.k_hs + d0, v_lane = sub * a.v_hs + d0;
  H ahead[kAhead];
  Quad x = start;
#pragma unroll
  for (uint32_t c = 0; c < kAhead; ++c) {
    if (c < count) {
      const int h = first_head(x);
      if (h + sub < heads) {
        const _Float16* src = is_q ? a.q + x.t * a.q_ts + h * a.q_hs + q_lane
                                   : x.i < per_head4 ? a.k + x.t * a.k_ts + h * a.k_hs + k_lane
                                                     : a.v + x.t * a.v_ts + h * a.v_hs + v_lane;
        ahead[c] = *reinterpret_cast<const H*>(src);
      }
      x = after(x);
    }
  }

  const int R = ROPE == kNone ? 0 : ROPE == kWhole ? D : a.rope_dims, half = R >> 1;
  int partner = lane;  // lane of the row that holds the rotation's other channels
  if (!a.interleaved && d0 < R) partner = d0 < half ? lane + half / E : lane - half / E;
  H wn{};
  const _Float16* weights = is_q ? a.q_norm : a.k_norm;
  if (weights) wn = *reinterpret_cast<const H*>(weights + d0);
  float cs[E], sn[E];  // this lane's cosines and sines, of the token at hand
#pragma unroll
  for (int e = 0; e < E; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }

  x = start;
  int64_t pos = 0, slot = 0;
#pragma unroll
  for (uint32_t c = 0; c < kAhead; ++c) {
    if (c >= count) break;
    const Quad now = x;
    x = after(x);
    const bool fresh = c == 0 || now.i == 0;
    const bool is_k = !is_q && now.i < per_head4;
    const int h0 = first_head(now);
    if (fresh) {
      if (!is_q) slot = scalar_load(a.slots, now.t);
      if (R) pos = scalar_load(a.positions, now.t);
    }
    if (R && (pos < 0 || pos >= a.rope_len)) {
      if (fresh && (threadIdx.x & 63) == 0) kv_report(a.err, kKvPosition, a.first + now.t, pos);
      continue;
    }
    if (!is_q && (slot < 0 || slot >= (a.L.num_pages << a.L.page_shift))) {
      if (slot >= 0 && fresh && (threadIdx.x & 63) == 0) kv_report(a.err, kKvSlot, a.first + now.t, slot);
      continue;
    }
    if (R && (is_q || is_k) && fresh && d0 < R) {
      const float* rp = a.rope + pos * R;
      if (ROPE == kOther && a.interleaved) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          cs[e] = rp[(d0 + e) >> 1];
          sn[e] = rp[half + ((d0 + e) >> 1)];
        }
      } else {
        const int i0 = d0 < half ? d0 : d0 - half;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          cs[e] = rp[i0 + e];
          sn[e] = rp[half + i0 + e];
        }
      }
    }
    if (h0 + sub >= heads) continue;
    const H in = ahead[c];
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (float)in.x[e];
    auto prepare = [&](auto& y) {
      typedef typename std::remove_reference<decltype(y[0])>::type T;
      if (is_q || is_k) norm_rope<T, E, ROPE>(y, weights != nullptr, wn, a.eps, d0, R, a.interleaved, partner, cs, sn);
    };
    prepare(v);
    if (is_q) {
      H out;
#pragma unroll
      for (int e = 0; e < E; ++e) out.x[e] = (_Float16)v[e];
      *reinterpret_cast<H*>(a.q_out + now.t * a.o_ts + h0 * a.o_hs + (sub * a.o_hs + d0)) = out;
      continue;
    }
    if constexpr (ROLE != kQueries) {
      uint32_t word[E / 4];  // channels 4 i .. 4 i + 3
      _Float16 s, b;
      // In units of 2^-24: a norm leaves a relative error below 16 (E + 4 additions, halved by the root, the root, a
      // quotient, two products); a rotation of (x, y) by (c, s) then one below 16 + 2 of |x c| + |y s|, which is at
      // most 2^(1/2) times the larger of the two results. 2^-19 covers 18 2^(1/2).
      // For whole rows: their lanes work together.
      if (__any(!quantise_fast<E>(v, is_k ? 0x1p-19f : 0.f, word, s, b))) {
        double y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (double)in.x[e];
        prepare(y);
        if (quantise<E>(y, word, s, b)) kv_report(a.err, kKvValue, a.first + now.t, h0 + sub);
      }
      const int off = (int)(slot & (a.L.page_tokens - 1));
      const int tok = off & 31;
      char* blk = a.pages + kv_block_at(a.L, slot >> a.L.page_shift, h0, off >> 5) +
                  (uint32_t)(sub * (a.L.page_tokens >> 5) * 32 * (D + 8));
      _Float16* par = reinterpret_cast<_Float16*>(blk + 32 * D);
      if (is_k) {
        struct alignas(E / 2) Row {
          uint16_t x[E / 4];
        } out;
#pragma unroll
        for (int w = 0; w < E / 4; ++w) out.x[w] = (uint16_t)word[w];
        *reinterpret_cast<Row*>(blk + tok * (D / 2) + lane * (E / 2)) = out;
        if (lane == 0) {
          struct alignas(4) Pair {
            _Float16 s, b;
          } pair = {s, b};
          *reinterpret_cast<Pair*>(par + 2 * tok) = pair;
        }
      } else {
        const int qr = kv_value_quarter(tok), e8 = kv_value_place(tok);
        uint16_t* vb = reinterpret_cast<uint16_t*>(blk + 16 * D);
#pragma unroll
        for (int w = 0; w < E / 4; ++w) vb[((w * 4 + qr) * 16 + lane) * 8 + e8] = (uint16_t)word[w];
        if (lane == 0) {
          par[64 + qr * 8 + e8] = s;
          par[96 + qr * 8 + e8] = b;
        }
      }
    }
  }
}

// One row of 16 lanes per (token, kv head). HBM-bound: 16384 tokens of 8 kv
// heads (D 128) in 17.4 us, 4.9 TB/s of bytes in and out.
template <int E>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs a) {
  using H = Halves<E>;
  constexpr int D = 16 * E;
  const int lane = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * kRowsPerPass + (threadIdx.x >> 4);
  if (row >= a.tokens * a.L.Hkv) return;
  const int64_t t = row / a.L.Hkv;
  const int h = (int)(row - t * a.L.Hkv);
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= (a.L.num_pages << a.L.page_shift)) {
    if (lane == 0 && h == 0) kv_report(a.err, kKvSlot, a.first + t, slot);
    return;
  }
  const int off = (int)(slot & (a.L.page_tokens - 1));
  const int tok = off & 31;
  const char* blk = a.pages + kv_block_at(a.L, slot >> a.L.page_shift, h, off >> 5);
  const int qr = kv_value_quarter(tok), e8 = kv_value_place(tok);
  const _Float16* par = reinterpret_cast<const _Float16*>(blk + 32 * D);
  const _Float16 ks = par[2 * tok], kb = par[2 * tok + 1], vs = par[64 + qr * 8 + e8], vb = par[96 + qr * 8 + e8];
  const uint16_t* kw = reinterpret_cast<const uint16_t*>(blk + tok * (D / 2)) + lane * (E / 4);
  const uint16_t* vw = reinterpret_cast<const uint16_t*>(blk + 16 * D);
  H ko, vo;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const uint32_t kn = kw[i], vn = vw[((i * 4 + qr) * 16 + lane) * 8 + e8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ko.x[4 * i + j] = __builtin_fmaf16((_Float16)(float)(16 + ((kn >> (4 * j)) & 15)), ks, kb);
      vo.x[4 * i + j] = __builtin_fmaf16((_Float16)(float)(16 + ((vn >> (4 * j)) & 15)), vs, vb);
    }
  }
  *reinterpret_cast<H*>(a.k_out + row * D + lane * E) = ko;
  *reinterpret_cast<H*>(a.v_out + row * D + lane * E) = vo;
}

}  // namespace

namespace {

template <int E, int ROPE>
hipError_t launch_append(KvAppendArgs a, int num_cus, hipStream_t s) {
  constexpr int waves = kThreads / 64;
  const int64_t nq = a.q ? (a.L.Hq + 3) / 4 : 0, nk = a.k ? (a.L.Hkv + 3) / 4 * 2 : 0;  // quads of a token
  // Few quads: one launch, which the host takes 2.5 us longer to make two of;
  // and with still fewer one to a wave, so that they spread over the chip.
  const int64_t all = a.tokens * (nq + nk);
  const bool few = all <= (int64_t)num_cus * 64;
  a.quads = all <= (int64_t)num_cus * 32 ? 1 : kAhead;
  a.near = (uint32_t)(32 * nk / (waves * a.quads) > 1 ? 32 * nk / (waves * a.quads) : 1);
  auto groups = [&](int64_t quads) { return (unsigned)((a.tokens * quads + waves * a.quads - 1) / (waves * a.quads)); };
  if (few && nq && nk) return kv_launch(kv_append_kernel<E, kBoth, ROPE>, dim3(groups(nq > nk ? nq : nk), 2), kThreads, s, a);
  hipError_t e = hipSuccess;
  if (nq) e = kv_launch(kv_append_kernel<E, kQueries, ROPE>, dim3(groups(nq)), kThreads, s, a);
  if (nk && e == hipSuccess) e = kv_launch(kv_append_kernel<E, kKeysValues, ROPE>, dim3(groups(nk)), kThreads, s, a);
  return e;
}

template <int E>
hipError_t launch_rope(const KvAppendArgs& a, int num_cus, hipStream_t s) {
  if (!a.rope) return launch_append<E, kNone>(a, num_cus, s);
  if (a.rope_dims == 16 * E && !a.interleaved) return launch_append<E, kWhole>(a, num_cus, s);
  return launch_append<E, kOther>(a, num_cus, s);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, int num_cus, hipStream_t s) {
  switch (a.L.D) {
    case 64: return launch_rope<4>(a, num_cus, s);
    case 128: return launch_rope<8>(a, num_cus, s);
    case 256: return launch_rope<16>(a, num_cus, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int64_t rows = a.tokens * a.L.Hkv;
  const dim3 grid((unsigned)((rows + kRowsPerPass - 1) / kRowsPerPass));
  switch (a.L.D) {
    case 64: return kv_launch(kv_read_kernel<4>, grid, kThreads, s, a);
    case 128: return kv_launch(kv_read_kernel<8>, grid, kThreads, s, a);
    case 256: return kv_launch(kv_read_kernel<16>, grid, kThreads, s, a);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace agemm
