// Appending keys and values to the 4-bit paged cache, with the head norms and
// the position rotation of queries and keys in the same pass, and reading
// cached tokens back, on gfx950.
//
// A head row of D channels is the work of 16 lanes, D / 16 consecutive
// channels each, so that a lane's channels are exactly one run of the key
// row's nibbles and one value run c of the block layout, and no nibble changes
// lanes. A workgroup of 256 threads takes 16 rows of one token at a time:
// query rows are normed, rotated and written as binary16; key rows are
// normed, rotated and quantised; value rows are quantised. The rotation's
// partner of channel i, i +- rope_dims / 2, is in the lane rope_dims / 2
// channels away.
//
// Bound by HBM: 2 bytes in and out a query channel, 2 in and 1/2 out a key or
// value channel, some 10 operations each.
#include "kv_internal.h"

namespace agemm {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerPass = kThreads / 16;

template <int E>
struct alignas(E * 2) Halves {
  _Float16 x[E];
};

template <class T>
__device__ inline T sum16(T v) {
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) v += __shfl_xor(v, m, 16);
  return v;
}
__device__ inline double min16(double v) {
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) v = fmin(v, __shfl_xor(v, m, 16));
  return v;
}

// x (this lane's channels of a head row) normed and rotated in place. `partner`
// is the row's lane that holds the rotation's other channels.
template <class T, int E>
__device__ inline void norm_rope(T (&x)[E], const _Float16* w, float eps, int d0, int R, bool interleaved, int partner,
                                 const float (&cs)[E], const float (&sn)[E]) {
  constexpr int D = 16 * E;
  if (w) {
    T ss = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) ss += x[e] * x[e];
    const T inv = T(1) / sqrt(sum16(ss) * T(1.0 / D) + T(eps));
    const Halves<E> wv = *reinterpret_cast<const Halves<E>*>(w + d0);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] * inv * T((float)wv.x[e]);
  }
  if (!R) return;
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
    T y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = __shfl(x[e], partner, 16);
    if (d0 < R) {
      const T sign = d0 < (R >> 1) ? T(-1) : T(1);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = x[e] * T(cs[e]) + sign * y[e] * T(sn[e]);
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

// The row's 4-bit form: nibbles n[] of this lane's channels and the pair (s, b).
// In binary64 (which this part multiplies and adds as fast as binary32): a
// nibble next to the border between two is then decided as the definition
// says, ties of (x - b) / s to even. x - b and n s are exact for values of
// binary16, so the remainder tells a tie where the product with 1 / s cannot.
template <int E>
__device__ inline bool quantise(double (&x)[E], uint32_t (&n)[E], _Float16& s, _Float16& b) {
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
    n[e] = (uint32_t)(i < 0 ? 0 : i > 15 ? 15 : i);
  }
  return bad;
}

// D = 16 E.
template <int E>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendArgs a) {
  using H = Halves<E>;
  constexpr int D = 16 * E;
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 15;  // of the row
  const int d0 = lane * E;
  const int nq = a.q ? a.L.Hq : 0;

  // This lane's cosines and sines: the same for every row of the token.
  const int R = a.rope ? a.rope_dims : 0;
  const int half = R >> 1;
  float cs[E], sn[E];
  int partner = lane;  // lane of the row that holds the rotation's other channels
  if (R) {
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.rope_len) {
      if (threadIdx.x == 0 && blockIdx.y == 0) kv_report(a.err, kKvPosition, t, pos, a.rope_len);
      return;
    }
    if (d0 < R) {
      const float* row = a.rope + pos * R;
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          cs[e] = row[(d0 + e) >> 1];
          sn[e] = row[half + ((d0 + e) >> 1)];
        }
      } else {
        const int i0 = d0 < half ? d0 : d0 - half;
        partner = d0 < half ? lane + half / E : lane - half / E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          cs[e] = row[i0 + e];
          sn[e] = row[half + i0 + e];
        }
      }
    }
  }
  int64_t slot = -1;
  if (a.k) {
    slot = a.slots[t];
    if (slot >= (a.L.num_pages << a.L.page_shift)) {
      if (threadIdx.x == 0 && blockIdx.y == 0) kv_report(a.err, kKvSlot, t, slot, a.L.num_pages << a.L.page_shift);
      slot = -1;
    }
  }

  // All 16 lanes of a row take the same path below; `r` is the same for them.
  for (int r = blockIdx.y * kRowsPerPass + (threadIdx.x >> 4); r < a.rows; r += gridDim.y * kRowsPerPass) {
    const bool is_q = r < nq;
    const bool is_k = !is_q && r < nq + a.L.Hkv;
    const int h = is_q ? r : is_k ? r - nq : r - nq - a.L.Hkv;
    if (!is_q && slot < 0) continue;
    const _Float16* src = is_q ? a.q + t * a.q_ts + h * a.q_hs
                               : is_k ? a.k + t * a.k_ts + h * a.k_hs : a.v + t * a.v_ts + h * a.v_hs;
    const H in = *reinterpret_cast<const H*>(src + d0);
    if (is_q) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = (float)in.x[e];
      norm_rope<float, E>(x, a.q_norm, a.eps, d0, R, a.interleaved, partner, cs, sn);
      H out;
#pragma unroll
      for (int e = 0; e < E; ++e) out.x[e] = (_Float16)x[e];
      *reinterpret_cast<H*>(a.q_out + t * a.o_ts + h * a.o_hs + d0) = out;
      continue;
    }
    double x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = (double)in.x[e];
    if (is_k) norm_rope<double, E>(x, a.k_norm, a.eps, d0, R, a.interleaved, partner, cs, sn);
    uint32_t n[E];
    _Float16 s, b;
    if (quantise<E>(x, n, s, b)) kv_report(a.err, kKvValue, t, h, 0);
    const int off = (int)(slot & (a.L.page_tokens - 1));
    const int tok = off & 31;
    char* blk = a.pages + kv_block_at(a.L, slot >> a.L.page_shift, h, off >> 5);
    uint32_t word[E / 4];  // 16 bits each: channels 4 i .. 4 i + 3
#pragma unroll
    for (int i = 0; i < E / 4; ++i) word[i] = n[4 * i] | n[4 * i + 1] << 4 | n[4 * i + 2] << 8 | n[4 * i + 3] << 12;
    _Float16* par = reinterpret_cast<_Float16*>(blk + 32 * D);
    if (is_k) {
      uint16_t* row = reinterpret_cast<uint16_t*>(blk + tok * (D / 2)) + lane * (E / 4);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) row[i] = (uint16_t)word[i];
      if (lane == 0) {
        par[2 * tok] = s;
        par[2 * tok + 1] = b;
      }
    } else {
      const int qr = kv_value_quarter(tok), e8 = kv_value_place(tok);
      uint16_t* vb = reinterpret_cast<uint16_t*>(blk + 16 * D);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) vb[((i * 4 + qr) * 16 + lane) * 8 + e8] = (uint16_t)word[i];
      if (lane == 0) {
        par[64 + qr * 8 + e8] = s;
        par[96 + qr * 8 + e8] = b;
      }
    }
  }
}

// One row of 16 lanes per (token, kv head).
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
    if (lane == 0 && h == 0) kv_report(a.err, kKvSlot, t, slot, a.L.num_pages << a.L.page_shift);
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

hipError_t launch_kv_append(const KvAppendArgs& a, int num_cus, hipStream_t s) {
  // One workgroup per token walks its rows, so that the rotation's row is
  // loaded once; with few tokens the rows go to several workgroups.
  const int passes = (a.rows + kRowsPerPass - 1) / kRowsPerPass;
  int64_t split = a.tokens >= 2 * num_cus ? 1 : (2 * num_cus + a.tokens - 1) / a.tokens;
  if (split > passes) split = passes;
  const dim3 grid((unsigned)a.tokens, (unsigned)split), block(kThreads);
  switch (a.L.D) {
    case 64: hipLaunchKernelGGL(kv_append_kernel<4>, grid, block, 0, s, a); break;
    case 128: hipLaunchKernelGGL(kv_append_kernel<8>, grid, block, 0, s, a); break;
    case 256: hipLaunchKernelGGL(kv_append_kernel<16>, grid, block, 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int64_t rows = a.tokens * a.L.Hkv;
  const dim3 grid((unsigned)((rows + kRowsPerPass - 1) / kRowsPerPass)), block(kThreads);
  switch (a.L.D) {
    case 64: hipLaunchKernelGGL(kv_read_kernel<4>, grid, block, 0, s, a); break;
    case 128: hipLaunchKernelGGL(kv_read_kernel<8>, grid, block, 0, s, a); break;
    case 256: hipLaunchKernelGGL(kv_read_kernel<16>, grid, block, 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace agemm
