// Attention over the 4-bit paged cache on gfx950.
//
// One workgroup per (query row, query head) walks the sequence's blocks of 32
// tokens with a running maximum m, sum l and weighted values acc of the
// softmax:
//   m' = max(m, S_j), l' = l e^(m-m') + sum_j e^(S_j-m'), acc alike.
// Eight threads share a key's product; then each thread owns a channel.
#include "kv_internal.h"

namespace agemm {
namespace {

constexpr int kThreads = 256;
constexpr float kLowest = -3.402823466e+38f;  // lse of a row that sees nothing

__device__ inline float held(uint32_t n, _Float16 s, _Float16 b) {
  return (float)__builtin_fmaf16((_Float16)(float)(16 + n), s, b);
}

template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void kv_attend_rows_kernel(KvAttendArgs a) {
  __shared__ float qs[D], sc[32];
  const int64_t row = blockIdx.x / a.L.Hq;
  const int hq = (int)(blockIdx.x - row * a.L.Hq);
  const int h = hq / (a.L.Hq / a.L.Hkv);
  const int tid = threadIdx.x;
  int b = (int)row, i = 0, n = 1;
  if (a.q_start) {  // the sequence whose rows hold this one (block-uniform search)
    for (b = 0; b < a.batch; ++b) {
      if (a.q_start[b + 1] < a.q_start[b] && tid == 0) kv_report(a.err, kKvRows, b, a.q_start[b + 1] - a.q_start[b], a.max_q);
      if (row >= a.q_start[b] && row < a.q_start[b + 1]) break;
    }
    if (b == a.batch) return;
    i = (int)(row - a.q_start[b]);
    n = a.q_start[b + 1] - a.q_start[b];
    if (n > a.max_q || a.q_start[b] < 0 || a.q_start[b + 1] > a.tokens) {
      if (tid == 0) kv_report(a.err, kKvRows, b, n, a.max_q);
      return;
    }
  }
  if (b >= a.batch) return;
  int64_t len = a.kv_len[b];
  const int64_t most = (int64_t)a.table_width << a.L.page_shift;
  if (len < 0 || len > most) {
    if (tid == 0) kv_report(a.err, kKvLength, b, len, most);
    len = len < 0 ? 0 : most;
  }
  if (a.causal) {
    const int64_t seen = (a.q_off ? (int64_t)a.q_off[b] : len - n) + i + 1;
    if (seen < len) len = seen < 0 ? 0 : seen;
  }
  for (int d = tid; d < D; d += kThreads) qs[d] = (float)a.q[row * a.q_ts + hq * a.q_hs + d];
  __syncthreads();

  float m = -__builtin_inff(), l = 0.f, acc = 0.f;
  for (int64_t at = 0; at < len; at += 32) {
    const int64_t page = a.table[b * a.table_stride + (at >> a.L.page_shift)];
    if (page < 0 || page >= a.L.num_pages) {
      if (tid == 0) kv_report(a.err, kKvPage, b, page, a.L.num_pages);
      continue;
    }
    const char* blk = a.pages + kv_block_at(a.L, page, h, (int)(at & (a.L.page_tokens - 1)) >> 5);
    const _Float16* par = reinterpret_cast<const _Float16*>(blk + 32 * D);
    const int key = tid >> 3, part = tid & 7;
    float s = 0.f;
    const uint8_t* kr = reinterpret_cast<const uint8_t*>(blk) + key * (D / 2) + part * (D / 16);
    for (int c = 0; c < D / 16; ++c) {
      const uint32_t w = kr[c];
      s += qs[part * (D / 8) + 2 * c] * held(w & 15, par[2 * key], par[2 * key + 1]);
      s += qs[part * (D / 8) + 2 * c + 1] * held(w >> 4, par[2 * key], par[2 * key + 1]);
    }
    for (int x = 1; x < 8; x <<= 1) s += __shfl_xor(s, x, 8);
    if (part == 0) sc[key] = at + key < len ? s * a.scale : -__builtin_inff();
    __syncthreads();
    float mn = m;
    for (int j = 0; j < 32; ++j) mn = fmaxf(mn, sc[j]);
    const float keep = mn == -__builtin_inff() ? 0.f : expf(m - mn);
    l *= keep;
    acc *= keep;
    const int c = tid / (D / 16), g = (tid % (D / 16)) >> 2, jn = tid & 3;
    const int top = (int)(len - at < 32 ? len - at : 32);
    for (int j = 0; j < top; ++j) {
      const float p = mn == -__builtin_inff() ? 0.f : expf(sc[j] - mn);
      l += p;
      if (tid < D) {
        const int qr = kv_value_quarter(j), e8 = kv_value_place(j);
        const uint32_t w = reinterpret_cast<const uint16_t*>(blk + 16 * D)[((g * 4 + qr) * 16 + c) * 8 + e8];
        acc += p * held((w >> (4 * jn)) & 15, par[64 + qr * 8 + e8], par[96 + qr * 8 + e8]);
      }
    }
    m = mn;
    __syncthreads();
  }
  const int64_t o = row * a.L.Hq + hq;
  if (tid < D) {
    const float v = l != 0.f ? acc / l : 0.f;
    if constexpr (F32) static_cast<float*>(a.out)[o * D + tid] = v;
    else static_cast<_Float16*>(a.out)[o * D + tid] = (_Float16)v;
  }
  if (a.lse && tid == 0) a.lse[o] = l != 0.f ? m + logf(l) : kLowest;
}

template <int D>
void launch_d(const KvAttendArgs& a, bool out_f32, hipStream_t s) {
  const dim3 grid((unsigned)(a.tokens * a.L.Hq)), block(kThreads);
  if (out_f32) hipLaunchKernelGGL((kv_attend_rows_kernel<D, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((kv_attend_rows_kernel<D, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_kv_attend(const KvAttendArgs& a, bool out_f32, hipStream_t s) {
  switch (a.L.D) {
    case 64: launch_d<64>(a, out_f32, s); break;
    case 128: launch_d<128>(a, out_f32, s); break;
    case 256: launch_d<256>(a, out_f32, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace agemm
