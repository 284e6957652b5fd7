// commit_kv_q8.cu -- bf16 K/V rows quantised into the 8-bit paged cache: the
// accepted rows of a verify step, or the rows of prompts.
//
// A unit is one (page, kv head) of K or of V in one layer.  With x the largest
// finite magnitude among the rows it receives, their scale is the smallest
// power of two s with x <= 448 s; a page that already holds rows keeps the
// larger of its scale and s, and where it grows, the held values are divided
// by the ratio (exact but below e4m3's normal range).  Dividing by a power of
// two is exact, so each value is rounded once, to nearest even.  +-inf saturates
// to +-448 s, NaN stays NaN; neither enters x.  Bytes behind a request's last
// row are left as they were.
//
// One warp holds sixteen rows of a unit in registers (16-byte loads, D / 8
// lanes a row), so a unit of a 16-, 32- or 64-token page is 1, 2 or 4 warps
// that share their maxima through shared memory: the rows are read once.
// Bound: bytes for prompts (2 read + 1 written a value): five of 4099 rows, four layers, 8 heads of 128,
// take 58 us (6.5 TB/s; 66 us when every value was looked at for infs and NaNs).  A verify step
// is the chain of dependent reads (lengths, table and row indices, rows, the held rows of a
// page whose scale grows): 32 trees, eight layers 5.1 us, 256 chains, two layers 8.2 us.
#include "common.cuh"
#include "kernels.cuh"

#include "e4m3.cuh"

namespace spec {

namespace {

constexpr int kQ8Threads = 256;
constexpr int kRowsPerWarp = 16;
// CTAs up to which K and V of every layer have one of their own; past it a CTA takes several in turn and
// looks up its rows once.  Five prompts of 4099 rows in four layers: 58 us by 4864, 61 us by 9728, 60 us by 2432.
constexpr long kMostCtas = 4864;

// the larger of |a| and |b| halfword by halfword, non-finite halves counting as 0
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
  x &= 0x7fff7fffu;
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return __vmaxu2(m, x);
}

template <int D, int WU>  // WU: warps a unit (page_size / 16)
__global__ void __launch_bounds__(kQ8Threads, 4) commit_kv_q8_kernel(const __grid_constant__ CommitQ8Params a) {
  constexpr int kLanesPerRow = D / 8, kRowsPerLoad = 32 / kLanesPerRow, kLoads = kRowsPerWarp / kRowsPerLoad;
  constexpr int PS = kRowsPerWarp * WU, kUnits = kQ8Threads / 32 / WU;
  __shared__ uint32_t s_max[2][kQ8Threads / 32];
  pdl_wait();
  pdl_trigger();
  // (every request's first page, then the second: the pages that are not touched come last)
  const int req = blockIdx.x % a.b, j = blockIdx.x / a.b;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.y * kUnits + w / WU, sub = w % WU;

  const int L = a.seq_lens[req], m = a.lens[req], rq = a.req_pool_idx[req];
  const bool first = blockIdx.y == 0 && blockIdx.z == 0 && j == 0 && threadIdx.x == 0;
  const bool len_ok = L >= 0 && m >= 0 && m <= a.max_len && (long long)L + m <= (long long)a.row_pages * PS;
  const bool rq_ok = rq >= 0 && rq < a.req_rows;
  if (first) {
    if (!len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
    if (!rq_ok) raise_error(a.error, SPEC_DEV_INDEX);
    a.new_seq_lens[req] = len_ok && rq_ok ? L + m : L;
  }
  if (!len_ok || !rq_ok) return;
  const int page = L / PS + j, base = page * PS;
  if (base >= L + m || m == 0) return;  // (the whole CTA)
  const int pid = a.page_table[size_t(rq) * a.row_pages + page];
  if (pid < 0 || pid >= a.num_pages) {
    if (threadIdx.x == 0) raise_error(a.error, SPEC_DEV_INDEX);
    return;
  }
  const int held = L > base ? L - base : 0;  // rows of the page that are there already
  const int upto = min(PS, L + m - base);    // first row of the page that stays as it is
  const bool on = head < a.Hkv;
  const size_t unit = size_t(pid) * a.Hkv + (on ? head : 0);

  // the rows, the same for K and V of every layer (-1: none)
  const int rsub = lane / kLanesPerRow, c = lane % kLanesPerRow;
  int rows[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = sub * kRowsPerWarp + i * kRowsPerLoad + rsub;
    rows[i] = -1;
    if (on && r >= held && r < upto) {
      const int k = base + r - L;
      const long long row = a.src_index ? a.src_index[size_t(req) * a.max_len + k] : (long long)a.src_start[req] + k;
      if (row < 0 || row >= a.num_rows) raise_error(a.error, SPEC_DEV_INDEX);
      else rows[i] = int(row);
    }
  }
#pragma unroll 1
  for (int z = blockIdx.z; z < 2 * a.num_layers; z += gridDim.z) {
    const int layer = z >> 1;
    const bool isv = (z & 1) != 0;
    const unsigned char* src =
        static_cast<const unsigned char*>(isv ? a.v_new[layer] : a.k_new[layer]) + size_t(on ? head : 0) * (D * 2);
    unsigned char* dst = static_cast<unsigned char*>(isv ? a.v_pages[layer] : a.k_pages[layer]) + unit * (size_t(PS) * D);
    uint8_t* scale = (isv ? a.v_scales[layer] : a.k_scales[layer]) + unit;
    const int had = held > 0 && on ? int(*scale) : 0;
    uint4 x[kLoads];
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      x[i] = rows[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + size_t(rows[i]) * a.new_ld * 2) + c)
                          : make_uint4(0u, 0u, 0u, 0u);
    // (an inf or a NaN shows as 0x7f80 or more; only then the finite ones are looked for)
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      mx = __vmaxu2(__vmaxu2(__vmaxu2(__vmaxu2(mx, x[i].x & 0x7fff7fffu), x[i].y & 0x7fff7fffu), x[i].z & 0x7fff7fffu), x[i].w & 0x7fff7fffu);
    mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    if (mx >= 0x7f80u) {
      mx = 0u;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) mx = max_abs2(max_abs2(max_abs2(max_abs2(mx, x[i].x), x[i].y), x[i].z), x[i].w);
      mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    }
    if (WU > 1) {
      uint32_t* sm = s_max[(z / gridDim.z) & 1];  // (the other one next time: one barrier is enough)
      if (lane == 0) sm[w] = mx;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < WU; ++q) mx = max(mx, sm[w - sub + q]);
    }
    const int need = scale_exp_of(mx), e = max(need, had);
    if (!on) continue;
    if (lane == 0 && sub == 0 && (held == 0 || e != had)) *scale = uint8_t(e);
    if (held > 0 && e > had) {  // the held rows move to the larger scale
      const float f = e - had < 64 ? exp_scale(kExpBias - (e - had)) : 0.f;
      const int most = min(held - sub * kRowsPerWarp, kRowsPerWarp);
      for (int r0 = 0; r0 < most; r0 += kRowsPerLoad)
        if (r0 + rsub < most) {
          uint2* p = reinterpret_cast<uint2*>(dst + size_t(sub * kRowsPerWarp + r0 + rsub) * D) + c;
          uint2 v = *p;
          auto move = [&](uint32_t q) {
            uint32_t h0 = e4m3x2_to_f16x2(q), h1 = e4m3x2_to_f16x2(q >> 16);
            const float2 a0 = __half22float2(*reinterpret_cast<__half2*>(&h0));
            const float2 a1 = __half22float2(*reinterpret_cast<__half2*>(&h1));
            return pack_e4m3(a0.x * f, a0.y * f) | (pack_e4m3(a1.x * f, a1.y * f) << 16);
          };
          *p = make_uint2(move(v.x), move(v.y));
        }
    }
    const float inv = inv_scale(e);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (rows[i] >= 0) {
        const int r = sub * kRowsPerWarp + i * kRowsPerLoad + rsub;
        auto put = [&](uint32_t u) { return pack_e4m3(bf16_lo(u) * inv, bf16_hi(u) * inv); };
        *(reinterpret_cast<uint2*>(dst + size_t(r) * D) + c) =
            make_uint2(put(x[i].x) | (put(x[i].y) << 16), put(x[i].z) | (put(x[i].w) << 16));
      }
  }
}

template <int D, int WU>
int launch_q8(const CommitQ8Params& p, cudaStream_t stream) {
  constexpr int kUnits = kQ8Threads / 32 / WU;
  const int pages = (p.max_len + 16 * WU - 2) / (16 * WU) + 1;
  // K and V of the layers: a CTA each, as long as there are no more than kMostCtas CTAs
  const long xy = long(p.b) * pages * ((p.Hkv + kUnits - 1) / kUnits);
  long z = kMostCtas / xy;
  z = z < 1 ? 1 : z > 2 * p.num_layers ? 2 * p.num_layers : z;
  const dim3 grid(unsigned(p.b) * unsigned(pages), unsigned((p.Hkv + kUnits - 1) / kUnits), unsigned(z));
  return launch_pdl(commit_kv_q8_kernel<D, WU>, grid, dim3(kQ8Threads), 0, stream, p) == cudaSuccess ? SPEC_OK
                                                                                                  : SPEC_ERR_LAUNCH;
}

}  // namespace

int launch_commit_kv_q8(const CommitQ8Params& p, cudaStream_t stream) {
  switch (p.D + p.page_size / 16) {
    case 64 + 1: return launch_q8<64, 1>(p, stream);
    case 64 + 2: return launch_q8<64, 2>(p, stream);
    case 64 + 4: return launch_q8<64, 4>(p, stream);
    case 128 + 1: return launch_q8<128, 1>(p, stream);
    case 128 + 2: return launch_q8<128, 2>(p, stream);
    case 128 + 4: return launch_q8<128, 4>(p, stream);
  }
  return SPEC_ERR_UNSUPPORTED;
}

}  // namespace spec
