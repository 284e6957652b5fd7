// attention_q8.cuh -- what the kernels of the verify attention over the 8-bit
// cache share.
#pragma once

#include "common.cuh"
#include "kernels.cuh"

namespace spec {

constexpr float kLazyLog2 = 8.f;  // O is rescaled only when a row's maximum grows by more than 2^8
constexpr float kPBaseLog2 = 6.f; // P's row maximum when the reference is set: 2^6, so P <= 2^14 < 65504
constexpr int kQ8MaxCtas = 192;   // upper bound of a grid of one CTA a SM; sizes the partial slots
constexpr int kQ8SlotRows = 256;  // query rows of a slot at most
// the partial area: (m, l) of each slot's rows, the table of units cut over CTAs or warps, O of the slots
constexpr size_t kQ8BegunBytes = (size_t(kQ8MaxCtas) * 12 + 16) * 16;
constexpr size_t kQ8SlotMlBytes = size_t(2) * kQ8MaxCtas * kQ8SlotRows * 2 * 4 + kQ8BegunBytes;

int launch_attention_q8_tc(const AttentionQ8Params& p, cudaStream_t stream);

// History length and table row of a request, validated: a bad length is
// clamped, a bad row leaves no history.
struct ReqQ8 {
  int len, row;
};
__device__ __forceinline__ ReqQ8 req_q8(const AttentionQ8Params& a, int Lp, int rq, bool report) {
  const long long room = (long long)a.row_pages * a.page_size;
  const int most = room < a.max_seq_len ? int(room) : a.max_seq_len;
  if (Lp < 0 || Lp > most) {
    if (report) raise_error(a.error, SPEC_DEV_LENGTH);
    Lp = Lp < 0 ? 0 : most;
  }
  if (rq < 0 || rq >= a.req_rows) {
    if (report) raise_error(a.error, SPEC_DEV_INDEX);
    return ReqQ8{0, -1};
  }
  return ReqQ8{Lp, rq};
}

// The larger magnitude halfword by halfword (15 bits), inf and NaN counting as 0.
__device__ __forceinline__ uint32_t finite_bf16(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}
__device__ __forceinline__ bool nonfinite_bf16(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t max_abs_bf16(uint32_t m, uint32_t x) { return __vmaxu2(m, finite_bf16(x) & 0x7fff7fffu); }

// Exponent byte e of the power of two 2^(e - 127) that a row of largest finite
// magnitude `bits` is divided by to lie in [2^14, 2^15) (at least 2^-126).
__device__ __forceinline__ int norm_exp(uint32_t bits) {
  const int e = int(bits >> 7) - 14;
  return e < 1 ? 1 : e;
}
// 2^d, d clamped to [-126, 127]
__device__ __forceinline__ float ratio_scale(int d) {
  d = d < -126 ? -126 : d > 127 ? 127 : d;
  return __uint_as_float(uint32_t(127 + d) << 23);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// (Mx, Ls, acc) joined with another partial (m, l, o) of the same row
template <int N, typename O>
__device__ __forceinline__ void join(float& Mx, float& Ls, float (&acc)[N], float m, float l, const O& o) {
  if (!(l > 0.f || l != l)) return;  // nothing seen
  const float M2 = fmaxf(Mx, m);
  const float wa = Ls > 0.f || Ls != Ls ? exp2f(Mx - M2) : 0.f, wb = exp2f(m - M2);
  Ls = Ls * wa + l * wb;
#pragma unroll
  for (int q = 0; q < N; ++q) acc[q] = acc[q] * wa + o[q] * wb;
  Mx = M2;
}

}  // namespace spec
