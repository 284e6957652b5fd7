// attention_q8.cuh -- what the kernels of the verify attention over the 8-bit
// cache share.
#pragma once

#include "common.cuh"
#include "e4m3.cuh"
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

// Two bf16 values, inf and NaN replaced by 0.
__device__ __forceinline__ uint32_t finite_bf16(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}
__device__ __forceinline__ uint32_t max_abs_bf16(uint32_t m, uint32_t x) { return __vmaxu2(m, finite_bf16(x) & 0x7fff7fffu); }

// Exponent byte e of the power of two 2^(e - 127) that a row of largest finite
// magnitude `bits` is divided by to lie in [2^14, 2^15) (at least 2^-126).
__device__ __forceinline__ int norm_exp(uint32_t bits) {
  const int e = int(bits >> 7) - 14;
  return e < 1 ? 1 : e;
}

// A key's weight enters P with its value's exponent in it, 2^(x + d - m), d = e - base, and l without,
// 2^(x - m).  So that neither leaves fp32, however far the values of a kv head lie apart:
//   - d is at most kSpanUp.  A larger exponent raises the base: m falls by as much, so that P
//     stays as it was and l grows, while l is below 2^kMostLog2; the rest makes O smaller.
//   - l is won back from P, as P 2^-d, while d is at least -kSpanDown.  Below (a row or a page of zeros,
//     above all) l has a sum of its own, or the key counts as one of d = -kSpanDown whose values are
//     that much smaller.
//   - m is set against x + max(d, -kSpanDown), so that l stays below 2^78 a key.
// So l loses weights below 2^-37 of the largest only, and O bits of values 2^-70 below the largest of
// the kv head's, and those 2^-90 below.
constexpr int kSpanUp = 16, kSpanDown = 64, kMostLog2 = 64;
__device__ __forceinline__ int span_of(int d) { return max(d, -kSpanDown); }

// The base once an exponent `top` has come (base -1: none yet).
__device__ __forceinline__ int raised_base(int base, int top) { return base < 0 || top > base + kSpanUp ? top : base; }

// Of a base raised by `up`, what m falls by in a row of sum l.
__device__ __forceinline__ int raised_into_l(int up, float l) {
  return max(0, min(up, kMostLog2 + kExpBias - int(__float_as_uint(l) >> 23)));
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

// A partial's reference moves so that l lies in [1/2, 1); returns what O is multiplied by.  O then is an
// average of values, and 2^-kRoomLog2 of it: the sums of many values near the type's largest would not fit.
constexpr int kRoomLog2 = 8;
__device__ __forceinline__ float settle(float& m, float& l) {
  float f = 1.f;
  if (l > 0.f) {
    const int e = int(__float_as_uint(l) >> 23) - (kExpBias - 1);
    m += float(e);
    f = ratio_scale(-e);
    l *= f;
  }
  return f * (1.f / (1 << kRoomLog2));
}
// 1 / l, and for settled partials' sum
__device__ __forceinline__ float inverse_of(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }
__device__ __forceinline__ float settled_inverse(float l) { return l > 0.f || l != l ? float(1 << kRoomLog2) / l : 0.f; }

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
