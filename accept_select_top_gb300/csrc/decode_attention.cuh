// decode_attention.cuh -- what the kernels of the one-token attention over shared pages have in common.
#pragma once

#include "common.cuh"
#include "kernels.cuh"

namespace spec {

constexpr int kDecTile = 64;    // keys of a tile of the tcgen05 kernel
constexpr int kDecRows = 64;    // query rows of a unit
constexpr int kDecMaxCtas = 192;  // upper bound of a grid of one CTA a SM; sizes the fragment slots

// P at a row's maximum when its reference is set, and how far the maximum may grow before it is set again: P stays below
// 2^-32, so the sums of the 2^30 values that a request may have stay below a quarter of the largest of them.  (What that costs:
// products below 2^-126, of values below 2^-86.)
constexpr float kDecBase = -40.f, kDecLazy = 8.f;
constexpr float kDecUnit = 1099511627776.f;  // 2^-kDecBase

__device__ __forceinline__ uint32_t dec_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The weight of a partial result of reference m in one of reference M.  One that has seen nothing, or only scores of -inf or
// NaN, has m = -inf and the weight 0; it counts all the same where results are joined, for the NaN that its l or O may hold.  Only
// one whose O was not written is left out: its l is kDecNone.
constexpr float kDecNone = -1.f;
__device__ __forceinline__ float dec_weight(float m, float M) { return m == -INFINITY ? 0.f : exp2f(m - M); }
__device__ __forceinline__ float dec_inverse(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }
// (l is brought back to the weights' own scale first, where a row's largest is 1: the logarithm's rounding is then that of its sum)
__device__ __forceinline__ float dec_lse(float m, float l) {
  return l > 0.f || l != l ? ((m + kDecBase) + log2f(l * kDecUnit)) * 0.6931471805599453f : -INFINITY;
}

// Rows of a group's shared tokens (members times q heads of a kv head) above which the tcgen05 kernel takes them.  In us,
// there / in the other kernel: heads of 128, eight groups of 4096 tokens and 32 rows 50 / 56, 20 rows 47 / 54, two of 16384 and 32
// rows 47 / 54; heads of 64, 16 groups of 1024 and 24 rows 34 / 29.
constexpr int dec_flat_rows(int D) { return D == 128 ? 16 : 32; }
constexpr int kDecTallRows = 256;  // query rows of one of its units
constexpr int kDecTallEnd = 2;     // what a unit's end costs there in the division of the work, in tiles

// The two kernels of a call run side by side: of `ctas` SMs the tcgen05 kernel takes so many, by the ticks of both (one
// of its tiles takes as long as kDecTallCost of the other's ticks, and a unit there, of which a few SMs may have to take
// hundreds, kDecUnitCost more than its end's), and the rest of its CTAs leave at once, so that the other kernel's, launched
// behind them, find their SMs free.
constexpr int kDecTallCost = 4, kDecUnitCost = 2;
__device__ __forceinline__ int dec_tall_ctas(int tall, int flat, int units, int ctas) {
  if (tall == 0) return 0;
  const long long cost = (long long)tall * kDecTallCost, rest = flat + (long long)units * kDecUnitCost;
  const int n = int((cost * ctas + (cost + rest) / 2) / (cost + rest));
  return n < 1 || ctas == 1 ? 1 : n > ctas - 1 ? ctas - 1 : n;
}
constexpr int kDecTickKeys128 = 16;  // keys of a tick of the other kernel, of D 128 (64: twice as many)
constexpr int kDecEndTicks = 3;      // what a unit's end costs there
// ticks of a unit over keys [first, last), without its end's
template <int D>
__device__ __forceinline__ int dec_unit_ticks(int first, int last) {
  constexpr int kTick = kDecTickKeys128 * 128 / D, kTile = 4 * kTick;
  const int n = (last - first / kTile * kTile + kTick - 1) / kTick;
  return n < 1 ? 1 : n;
}

// What a group shares, from its bounds and its first member's length (0: nothing).
__device__ __forceinline__ int dec_shared(int shared, int first_len) { return shared > 0 && first_len >= shared ? shared : 0; }

// The workspace of a call.  plan: {ticks, CTAs, groups, -} and, for the joining kernel, what the first CTA of the main
// kernel found: ticks before each segment, and each request's group.
struct DecodeArgs {
  DecodeParams p;
  int shift;       // log2(page_size)
  int own_tiles;   // 64-row tiles of a kv head's rows of one request
  int flat_rows;   // dec_flat_rows
  int4* plan;
  int* pre;        // [groups + b + 1]
  int4* member;    // [b]: {group (-1: none), its first request, its members, tokens shared}
  // Partial results: (m, l) of each row, and O as words of four columns, [D / 4][rows].  Those of a unit's part:
  // [2 * CTA + i][..][64], i = 1: the unit that the CTA begins and does not finish.  Those of units that lie in one
  // CTA: from row r0 * Hq + h * (the segment's rows) + (the unit's first) on, as many rows as the unit has.
  float2* frag_ml;
  float2* own_ml;
  float2* shared_ml;
  float4* frag_o;
  float4* own_o;
  float4* shared_o;
  // the tcgen05 kernel's (tall 0: it is not launched): plan {ticks, CTAs, -, -}, ticks before each group, partial
  // results [2 * CTA + i][half][..][128], and of units that lie in one CTA, [half] first; halves: rows 128 .., or every
  // second tile where there are no more than 128
  int tall;
  int4* tall_plan;
  int* tall_pre;
  float2* tall_ml;
  float4* tall_o;
  float2* whole_ml;  // [half][b * Hq]
  float4* whole_o;
};

int launch_decode_tall(const DecodeArgs& args, int sms, cudaStream_t stream);

}  // namespace spec
