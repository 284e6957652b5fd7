// attention_q8.cu -- tree-masked verify attention over the 8-bit paged cache, for
// few query rows a kv head (single tokens, short chains); attention_q8_tc.cu
// takes the larger trees.
//
// For row (node i, q head h): x_j = scale q . k_j over the history (e4m3 pages
// with a power-of-two scale for each page and kv head) and the visible tree
// nodes (the step's own bf16 rows), out = sum_j 2^(x_j log2e - m) v_j / l with
// a running maximum m and sum l.
//
// Everything is computed on f16 fragments with fp32 sums: an e4m3 value is an f16
// value, and a bf16 row divided by the power of two that puts its largest
// element into [2^14, 2^15) is one too, but for elements 2^-28 below that.  So
// the scales stay outside the products: a key's multiplies its column of S, and
// a value's, 2^e, is an exponent added to x: P_j = 2^(x_j + e_j - m), rounded
// once to f16 (2^-11), against a running maximum m of x + e.  So what P loses
// below f16's range is 2^-30 of the row's largest contribution p |v|, however
// far the value scales lie apart; l = sum P_j 2^-e_j (before the rounding).
//
// Bound: the cache's bytes.  A warp owns its work end to end: it takes an
// equal, contiguous range of 16-key tiles of all (request, kv head, 16-row
// tile) units laid end to end, copies each tile's K and V (2 x 16 x D bytes,
// contiguous in a page) into a private four-stage ring with 16-byte cp.async, and
// runs S = Q K^T and O += P V as register fragments (mma.sync m16n8k16: with at
// most 16 rows the tensor work of a 4 KB tile is 64 K multiply-adds, a third of
// the time the tile takes to arrive, and no operand passes through shared
// memory twice; a 128-row tcgen05 tile would be mostly padding).  The order of
// the head dimension inside a fragment is free as long as Q has the same, and
// that of the keys as long as P has the same, so both K and V fragments are
// read as whole 16-byte words.
//   There is no barrier before the end of the range.  Units cut by a range
// boundary leave fragments (O, m, l) in shared memory; the CTA joins those of
// its warps, and a unit cut over CTAs is joined by the CTA that arrives last on
// it (acquire-release counter).
#include "common.cuh"
#include "kernels.cuh"

#include "attention_q8.cuh"
#include "e4m3.cuh"

namespace spec {

namespace {

constexpr int kWarps = 8;
constexpr int kQ8AttThreads = 32 * kWarps;
constexpr int kRowsMost = 32;  // query rows a kv head up to which this kernel is taken
constexpr int kTile = 16;    // keys of a tile
constexpr int kRowTile = 16; // query rows of a unit
constexpr int kRing = 4;     // tiles in a warp's ring
constexpr int kMinTiles = 2; // a warp gets at least this many tiles before another warp is used

template <int D>
struct RowsSmem {
  static constexpr int kHalf = kTile * D;         // K (or V) bytes of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kFrag = kRowTile * D * 4;  // fp32 O of a fragment
  static constexpr int kWarp = kRing * kStage + kFrag + 2 * kRowTile * 8;  // ring | first fragment's O | (m, l) of both
  static_assert(kRing * kStage >= kFrag, "the last fragment's O takes the idle ring");
  static constexpr int kDesc = kWarps * kWarp;    // fragment descriptors: [warp][2] unit (-1: none)
  static constexpr int kScan = kDesc + 256;
  static size_t bytes(int b) { return size_t(kScan) + 12u * size_t(b + 1); }
};

struct RowsArgs {
  AttentionQ8Params p;
  int m_tiles;      // 16-row tiles of a kv head's n * G rows
  uint32_t* counters;  // [CTA]: arrivals on the unit that CTA begins and does not finish
  float* slot_o;    // [2 * CTA + i][16][D]
  float* slot_ml;   // [2 * CTA + i][16][2]
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bf16 values of a row (two 16-byte words) as f16x2, times inv
struct Raw16 {
  uint4 a, b;
};
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float inv) { return pack_f16(bf16_lo(w) * inv, bf16_hi(w) * inv); }
__device__ __forceinline__ uint32_t word_of(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

template <int D>
__global__ void __launch_bounds__(kQ8AttThreads, 1) attention_q8_rows_kernel(const __grid_constant__ RowsArgs args) {
  using L = RowsSmem<D>;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int KS = D / 16;   // k-steps of Q K^T
  constexpr int NT = D / 8;    // 8-column tiles of O
  const AttentionQ8Params& a = args.p;
  extern __shared__ __align__(128) unsigned char smem[];
  int* desc = reinterpret_cast<int*>(smem + L::kDesc);
  int* pre = reinterpret_cast<int*>(smem + L::kScan);  // [b + 1] tiles of one (kv head, row tile) before request r
  int* slen = pre + a.b + 1;                           // [b]
  int* srow = slen + a.b + 1;                          // [b] table row, -1 if bad
  __shared__ int wsum[kWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int G = a.Hq / a.Hkv, M = a.n * G, J = a.Hkv * args.m_tiles;
  const int tree_tiles = (a.n + kTile - 1) / kTile;
  if (tid < 2 * kWarps) desc[tid] = -1;

  pdl_wait();
  pdl_trigger();
  // ---- tiles before each request ----
  {
    int run = 0;
    for (int r0 = 0; r0 < a.b; r0 += kQ8AttThreads) {
      const int r = r0 + tid;
      int t = 0;
      if (r < a.b) {
        int Lp = a.seq_lens[r], rq = a.req_pool_idx[r];
        const ReqQ8 q = req_q8(a, Lp, rq, blockIdx.x == 0);
        slen[r] = q.len;
        srow[r] = q.row;
        t = (q.len + kTile - 1) / kTile + tree_tiles;
      }
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += y;
      }
      __syncthreads();
      if (lane == 31) wsum[w] = incl;
      __syncthreads();
      int before = run;
      for (int q = 0; q < kWarps; ++q) {
        if (q < w) before += wsum[q];
        run += wsum[q];
      }
      if (r < a.b) pre[r] = before + incl - t;
    }
    if (tid == 0) pre[a.b] = run;
    __syncthreads();
  }
  const long long T = (long long)pre[a.b] * J;  // (the host keeps it below 2^31)
  // wpc warps a CTA over `ctas` CTAs, every warp with at least one tile
  const long long grid = gridDim.x;
  int wpc = int((T + grid * kMinTiles - 1) / (grid * kMinTiles));
  wpc = wpc < 1 ? 1 : wpc > kWarps ? kWarps : wpc;
  long long ctas = (T + (long long)wpc * kMinTiles - 1) / ((long long)wpc * kMinTiles);
  if (ctas > grid) ctas = grid;
  const long long NW = ctas * wpc < T ? ctas * wpc : T;
  if (blockIdx.x * (long long)wpc >= NW) return;
  const long long me = blockIdx.x * (long long)wpc + w;
  const bool active = w < wpc && me < NW;
  const int S = active ? int(me * T / NW) : 0, E = active ? int((me + 1) * T / NW) : 0;
  auto warp_of = [&](long long x) { return ((x + 1) * NW - 1) / T; };  // the warp whose range holds tile x

  unsigned char* mine = smem + size_t(w) * L::kWarp;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  float* ffrag = reinterpret_cast<float*>(mine + kRing * L::kStage);
  float* fml = reinterpret_cast<float*>(mine + kRing * L::kStage + L::kFrag);  // [2][16][2]

  if (active) {
    auto req_of = [&](int f) {
      int lo = 0, hi = a.b;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)pre[mid] * J <= f) lo = mid;
        else hi = mid;
      }
      return lo;
    };
    // lane l looks up tile mb + l of the range: page, kv head, first key in
    // the page, keys that count; a tree tile (or a bad page) has page -1
    const int SHIFT = a.page_size == 16 ? 0 : a.page_size == 32 ? 1 : 2;  // log2(tiles a page)
    int mb = S - 32, l_unit = 0, l_off = 0, l_cnt = 0, l_exp = 0, p_exp = 0;
    auto load_meta = [&](int f0) {
      p_exp = l_exp;
      mb = f0;
      const int f = f0 + lane;
      l_unit = -1;
      l_off = l_cnt = l_exp = 0;
      if (f < E) {
        const int r = req_of(f), Tr = pre[r + 1] - pre[r];
        const int rem = f - pre[r] * J, j = rem / Tr, t = rem - j * Tr, h = j / args.m_tiles;
        if (t < Tr - tree_tiles && srow[r] >= 0) {
          const int pid = a.page_table[size_t(srow[r]) * a.row_pages + (t >> SHIFT)];
          if (pid < 0 || pid >= a.num_pages) {
            raise_error(a.error, SPEC_DEV_INDEX);
          } else {
            l_unit = pid * a.Hkv + h;
            l_off = (t & ((1 << SHIFT) - 1)) * kTile;
            l_cnt = min(kTile, slen[r] - t * kTile);
            l_exp = int(a.k_scales[l_unit]) | (int(a.v_scales[l_unit]) << 8) | 0x10000;
          }
        }
      }
    };
    constexpr int kChunks = D / 16;        // 16-byte chunks of a key
    constexpr int kCopies = kTile * kChunks / 32;
    auto issue = [&](int f) {
      if (f < E) {
        if (f - mb >= 32) load_meta(f);
        const int unit = __shfl_sync(FULL, l_unit, f - mb), off = __shfl_sync(FULL, l_off, f - mb),
                  cnt = __shfl_sync(FULL, l_cnt, f - mb);
        if (unit >= 0) {
          const size_t at = (size_t(unit) * a.page_size + off) * D;
          const uint32_t st = ring + uint32_t(f % kRing) * L::kStage;
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const int ch = i * 32 + lane, key = ch / kChunks, x = ch % kChunks;
            const int kx = D == 128 ? x ^ (4 * (key & 1)) : x;
            const int vx = D == 128 ? x ^ (((key >> 1) & 3) << 1) : x ^ (((key >> 1) & 1) << 1);
            const uint32_t nb = key < cnt ? 16u : 0u;  // (a key past the history reads as zeros)
            const size_t so = at + (key < cnt ? size_t(ch) * 16 : 0);
            cp16(st + uint32_t(key * D + kx * 16), a.k_pages + so, nb);
            cp16(st + L::kHalf + uint32_t(key * D + vx * 16), a.v_pages + so, nb);
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue(S + i);

    // ---- consumer state: the current unit and its running results ----
    int r = req_of(S), Tr = pre[r + 1] - pre[r];
    int j, t;
    {
      const int rem = S - pre[r] * J;
      j = rem / Tr;
      t = rem - j * Tr;
    }
    int t_first = t;
    uint32_t qf[KS][4];
    float xf[2];                // softmax factor of rows g, g + 8: scale * log2e * the row's power of two
    unsigned long long mask[2];
    float o[NT][4], m[2], l[2];
    int evb = 0;                // the exponent byte that the unit's value scales are taken relative to (its first tile's)
    unsigned long long nonfinite = 0;  // tree nodes whose V row holds an inf or a NaN
    bool fresh = true;
    for (int f = S; f < E; ++f) {
      cp_wait<kRing - 2>();
      __syncwarp();
      issue(f + kRing - 1);
      const int h = j / args.m_tiles, mt = j - h * args.m_tiles;
      if (fresh) {  // a unit begins: its Q rows as f16 fragments, masks, empty results
        fresh = false;
        t_first = t;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rg = mt * kRowTile + g + 8 * i;
          const bool on = rg < M;
          const int node = on ? rg / G : 0, hq = h * G + (on ? rg % G : 0);
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                            (size_t(r) * a.n + node) * a.q_ld + size_t(hq) * D);
          uint4 x[D / 32];
#pragma unroll
          for (int u = 0; u < D / 32; ++u)  // 16 elements from 16 c, and 64 + 16 c
            x[u] = on ? __ldg(src + (u >> 1) * 8 + 2 * c + (u & 1)) : make_uint4(0, 0, 0, 0);
          mask[i] = on ? a.mask_bits[size_t(r) * a.n + node] : 0ull;
          uint32_t mx = 0;
#pragma unroll
          for (int u = 0; u < D / 32; ++u)
            mx = max_abs_bf16(max_abs_bf16(max_abs_bf16(max_abs_bf16(mx, x[u].x), x[u].y), x[u].z), x[u].w);
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
          const int e = norm_exp(mx);
          const float inv = exp_scale(2 * kExpBias - e);
          xf[i] = a.scale * 1.4426950408889634f * exp_scale(e);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {  // words 2 kk, 2 kk + 1 of the thread's words
            const uint4& y = x[kk >> 1];
            qf[kk][i] = scaled_f16(word_of(y, (kk & 1) * 2), inv);
            qf[kk][2 + i] = scaled_f16(word_of(y, (kk & 1) * 2 + 1), inv);
          }
          m[i] = -INFINITY;
          l[i] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[q][i] = 0.f;
        evb = -1;
        nonfinite = 0;
      }

      float s[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[q][i] = 0.f;
      uint32_t vb[NT][2];  // V fragments: b0 (keys 2c, 2c+1), b1 (keys 2c+8, 2c+9) of column tile nt
      float dl[2][2];      // P's columns in l: 2^(evb - e) of key 8q + 2c + i
      const bool hist = t < Tr - tree_tiles;
      if (hist) {
        const int src = f - mb >= 0 ? f - mb : f - mb + 32;
        const int cur = __shfl_sync(FULL, l_exp, src & 31), prv = __shfl_sync(FULL, p_exp, src & 31);
        const int ex = f >= mb ? cur : prv;
        const float kf = exp_scale(ex & 255);
        const int ev = (ex >> 8) & 255;
        if (evb < 0) evb = ev;
        const float de = float(ev - evb);
        dl[0][0] = dl[0][1] = dl[1][0] = dl[1][1] = ratio_scale(evb - ev);
        const unsigned char* st = mine + (f % kRing) * L::kStage;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int key = 8 * q + g;
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {
            const int x = c + 4 * u, kx = D == 128 ? x ^ (4 * (key & 1)) : x;
            const uint4 y = *reinterpret_cast<const uint4*>(st + key * D + kx * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t wd = word_of(y, i);
              mma_f16(s[q], qf[4 * u + i], e4m3x2_to_f16x2(wd), e4m3x2_to_f16x2(wd >> 16));
            }
          }
        }
        const int cnt = min(kTile, slen[r] - t * kTile);
        const float x0 = xf[0] * kf, x1 = xf[1] * kf;
        const bool pageless = ex < 0x10000;  // (a page out of range: its keys do not count)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool on = 8 * q + 2 * c + i < cnt && !pageless;
            s[q][i] = on ? fmaf(s[q][i], x0, de) : -INFINITY;
            s[q][2 + i] = on ? fmaf(s[q][2 + i], x1, de) : -INFINITY;
          }
        const unsigned char* sv = st + L::kHalf;
        uint32_t v[4][D / 32];  // keys 2c, 2c+1, 2c+8, 2c+9; D / 8 bytes each
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 2 * c + (i & 1) + 8 * (i >> 1);
          if (D == 128) {
            const int vx = g ^ (((key >> 1) & 3) << 1);
            const uint4 y = *reinterpret_cast<const uint4*>(sv + key * D + vx * 16);
            v[i][0] = y.x;
            v[i][1] = y.y;
            v[i][D / 32 - 2] = y.z;
            v[i][D / 32 - 1] = y.w;
          } else {
            const int vx = (g >> 1) ^ (((key >> 1) & 1) << 1);
            const uint2 y = *reinterpret_cast<const uint2*>(sv + key * D + vx * 16 + (g & 1) * 8);
            v[i][0] = y.x;
            v[i][1] = y.y;
          }
        }
#pragma unroll
        for (int u = 0; u < D / 32; ++u)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t t0 = __byte_perm(v[0][u], v[1][u], hf ? 0x7362 : 0x5140);
            const uint32_t t1 = __byte_perm(v[2][u], v[3][u], hf ? 0x7362 : 0x5140);
            vb[4 * u + 2 * hf][0] = e4m3x2_to_f16x2(t0);
            vb[4 * u + 2 * hf][1] = e4m3x2_to_f16x2(t1);
            vb[4 * u + 2 * hf + 1][0] = e4m3x2_to_f16x2(t0 >> 16);
            vb[4 * u + 2 * hf + 1][1] = e4m3x2_to_f16x2(t1 >> 16);
          }
        if (pageless) {  // (the ring stage holds nothing of this tile)
#pragma unroll
          for (int q = 0; q < NT; ++q) vb[q][0] = vb[q][1] = 0u;
        }
      } else {
        // ---- tree nodes: the step's bf16 rows, each divided by its own power of two ----
        const int nb = (t - (Tr - tree_tiles)) * kTile;  // first node of the tile
        const uint16_t* kn = static_cast<const uint16_t*>(a.k_new) + size_t(h) * D;
        const uint16_t* vn = static_cast<const uint16_t*>(a.v_new) + size_t(h) * D;
        uint4 kx[2][D / 32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int node = nb + 8 * q + g;
          const uint4* src = reinterpret_cast<const uint4*>(kn + (size_t(r) * a.n + (node < a.n ? node : 0)) * a.new_ld);
#pragma unroll
          for (int u = 0; u < D / 32; ++u)
            kx[q][u] = node < a.n ? __ldg(src + (u >> 1) * 8 + 2 * c + (u & 1)) : make_uint4(0, 0, 0, 0);
        }
        float kf[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t mx = 0;
#pragma unroll
          for (int u = 0; u < D / 32; ++u)
            mx = max_abs_bf16(max_abs_bf16(max_abs_bf16(max_abs_bf16(mx, kx[q][u].x), kx[q][u].y), kx[q][u].z), kx[q][u].w);
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
          const int e = norm_exp(mx);
          const float inv = exp_scale(2 * kExpBias - e);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const uint4& y = kx[q][kk >> 1];
            mma_f16(s[q], qf[kk], scaled_f16(word_of(y, (kk & 1) * 2), inv), scaled_f16(word_of(y, (kk & 1) * 2 + 1), inv));
          }
          kf[q][0] = exp_scale(__shfl_sync(FULL, e, 8 * c));
          kf[q][1] = exp_scale(__shfl_sync(FULL, e, 8 * c + 4));
        }
        uint4 vx[4][D / 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int node = nb + 2 * c + (i & 1) + 8 * (i >> 1);
          const uint4* src = reinterpret_cast<const uint4*>(vn + (size_t(r) * a.n + (node < a.n ? node : 0)) * a.new_ld);
#pragma unroll
          for (int u = 0; u < D / 64; ++u)
            vx[i][u] = node < a.n ? __ldg(src + g * (D / 64) + u) : make_uint4(0, 0, 0, 0);
        }
        int evk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t mx = 0;
          bool nf = false;
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {
            nf = nf || nonfinite_bf16(vx[i][u].x) || nonfinite_bf16(vx[i][u].y) || nonfinite_bf16(vx[i][u].z) ||
                 nonfinite_bf16(vx[i][u].w);
            mx = max_abs_bf16(max_abs_bf16(max_abs_bf16(max_abs_bf16(mx, vx[i][u].x), vx[i][u].y), vx[i][u].z), vx[i][u].w);
          }
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(FULL, mx, 4));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 8));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 16));
          evk[i] = norm_exp(mx);
          // an inf or a NaN must reach the rows that see the node and no
          // other: it is left out of the product and added at the end
          const unsigned who = __ballot_sync(FULL, nf);
          if (who) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (who & (0x11111111u << q)) {
                const int node = nb + 2 * q + (i & 1) + 8 * (i >> 1);
                if (node < kMaxN) nonfinite |= 1ull << node;
              }
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
              vx[i][u].x = finite_bf16(vx[i][u].x);
              vx[i][u].y = finite_bf16(vx[i][u].y);
              vx[i][u].z = finite_bf16(vx[i][u].z);
              vx[i][u].w = finite_bf16(vx[i][u].w);
            }
          }
        }
        if (evb < 0) {
          evb = max(max(evk[0], evk[1]), max(evk[2], evk[3]));
          evb = max(evb, __shfl_xor_sync(FULL, evb, 1));
          evb = max(evb, __shfl_xor_sync(FULL, evb, 2));
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int node = nb + 8 * q + 2 * c + i;
            const bool in = node < a.n;
            const int d = evk[2 * q + i] - evb;
            s[q][i] = in && ((mask[0] >> (node & 63)) & 1) ? fmaf(s[q][i], xf[0] * kf[q][i], float(d)) : -INFINITY;
            s[q][2 + i] = in && ((mask[1] >> (node & 63)) & 1) ? fmaf(s[q][2 + i], xf[1] * kf[q][i], float(d)) : -INFINITY;
            dl[q][i] = ratio_scale(-d);
          }
        // the columns: element e of the thread's D / 8 is column tile e
#pragma unroll
        for (int e = 0; e < NT; ++e) {
          auto el = [&](int i) {
            const uint32_t wd = word_of(vx[i][e >> 3], (e & 7) >> 1);
            return ((e & 1) ? bf16_hi(wd) : bf16_lo(wd)) * exp_scale(2 * kExpBias - evk[i]);
          };
          vb[e][0] = pack_f16(el(0), el(1));
          vb[e][1] = pack_f16(el(2), el(3));
        }
      }

      // ---- running reference: P is kPBase at the row's maximum when it is
      // set, and it is moved only when P would pass 2^kLazyLog2 times that ----
      const float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      const float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      if (__any_sync(FULL, x0 > m[0] + (kLazyLog2 + kPBaseLog2) || x1 > m[1] + (kLazyLog2 + kPBaseLog2))) {
        float fac[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = i ? x1 : x0;
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
          const bool up = mx > m[i] + (kLazyLog2 + kPBaseLog2);
          fac[i] = up ? fast_exp2(m[i] + kPBaseLog2 - mx) : 1.f;  // (0 from an empty row)
          l[i] *= fac[i];
          if (up) m[i] = mx - kPBaseLog2;
        }
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          o[q][0] *= fac[0];
          o[q][1] *= fac[0];
          o[q][2] *= fac[1];
          o[q][3] *= fac[1];
        }
      }
      const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
      uint32_t pa[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float p00 = fast_exp2(s[q][0] - m0), p01 = fast_exp2(s[q][1] - m0);
        const float p10 = fast_exp2(s[q][2] - m1), p11 = fast_exp2(s[q][3] - m1);
        l[0] = fmaf(p00, dl[q][0], fmaf(p01, dl[q][1], l[0]));
        l[1] = fmaf(p10, dl[q][0], fmaf(p11, dl[q][1], l[1]));
        pa[2 * q] = pack_f16(p00, p01);
        pa[2 * q + 1] = pack_f16(p10, p11);
      }
#pragma unroll
      for (int q = 0; q < NT; ++q) mma_f16(o[q], pa, vb[q][0], vb[q][1]);

      // ---- the unit's or the range's end ----
      ++t;
      const bool unit_end = t == Tr;
      if (unit_end || f + 1 == E) {
        // rows g, g + 8; columns c D/4 .. + D/4: [0, D/8) from fragment columns 2c, [D/8, D/4) from 2c + 1
        float lt[2];
        const float vs = exp_scale(evb < 1 ? 1 : evb);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lt[i] = l[i] + __shfl_xor_sync(FULL, l[i], 1);
          lt[i] += __shfl_xor_sync(FULL, lt[i], 2);
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            o[q][2 * i] *= vs;
            o[q][2 * i + 1] *= vs;
          }
          if (nonfinite & mask[i])
            for (int node = 0; node < a.n; ++node)
              if ((nonfinite & mask[i]) >> node & 1) {
                const uint16_t* src = static_cast<const uint16_t*>(a.v_new) + (size_t(r) * a.n + node) * a.new_ld +
                                      size_t(h) * D + c * (D / 4);
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const float v = __uint_as_float(uint32_t(src[u * NT + q]) << 16);
                    if (!(fabsf(v) < INFINITY)) o[q][2 * i + u] += v;
                  }
              }
        }
        if (unit_end && t_first == 0) {  // the whole unit
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rg = mt * kRowTile + g + 8 * i;
            if (rg < M) {
              const size_t orow = (size_t(r) * a.n + rg / G) * a.Hq + h * G + rg % G;
              const float inv = lt[i] > 0.f || lt[i] != lt[i] ? 1.f / lt[i] : 0.f;
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + c * (D / 4));
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int q = 0; q < NT; q += 8) {
                  auto pk = [&](int e) { return pack_bf16x2(o[q + e][2 * i + u] * inv, o[q + e + 1][2 * i + u] * inv); };
                  dst[(u * NT + q) / 8] = make_uint4(pk(0), pk(2), pk(4), pk(6));
                }
              if (c == 0 && a.lse) a.lse[orow] = lse_of(m[i], lt[i]);
            }
          }
        } else {
          // a fragment: of a unit begun by an earlier warp (its own place), or one that goes on in a later one (the ring)
          const int which = unit_end ? 0 : 1;
          if (which == 1) {
            cp_wait<0>();
            __syncwarp();
          }
          float* fo = which == 0 ? ffrag : reinterpret_cast<float*>(mine);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float4* dst = reinterpret_cast<float4*>(fo + (g + 8 * i) * D + c * (D / 4));
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int q = 0; q < NT; q += 4)
                dst[(u * NT + q) / 4] = make_float4(o[q][2 * i + u], o[q + 1][2 * i + u], o[q + 2][2 * i + u], o[q + 3][2 * i + u]);
            if (c == 0) {
              fml[(which * 16 + g + 8 * i) * 2] = m[i];
              fml[(which * 16 + g + 8 * i) * 2 + 1] = lt[i];
            }
          }
          if (lane == 0) desc[2 * w + which] = r * J + j;  // (below 2^31: a unit has at least one tile)
        }
        fresh = true;
        if (unit_end) {
          t = 0;
          if (++j == J) {
            j = 0;
            ++r;
            if (r < a.b) Tr = pre[r + 1] - pre[r];
          }
        }
      }
    }
    cp_wait<0>();
  }
  __syncthreads();

  // ---- join the fragments: thread -> row tid / 16, D / 16 columns ----
  constexpr int CW = D / 16;  // 8 or 4 columns a thread
  const int row = tid >> 4, col = (tid & 15) * CW;
  int posted[2] = {-1, -1};  // units of this CTA that other CTAs share
  long long pstart[2] = {0, 0};
  int np = 0;
  auto finish = [&](int unit, float Mx, float Ls, const float (&acc)[CW]) {
    const int ur = unit / J, uj = unit - ur * J, uh = uj / args.m_tiles, um = uj - uh * args.m_tiles;
    const int rg = um * kRowTile + row;
    if (rg < M) {
      const size_t orow = (size_t(ur) * a.n + rg / G) * a.Hq + uh * G + rg % G;
      const float inv = Ls > 0.f || Ls != Ls ? 1.f / Ls : 0.f;
      uint32_t pk[CW / 2];
#pragma unroll
      for (int e = 0; e < CW / 2; ++e) pk[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + orow * D + col);
      if (CW == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[CW / 2 - 2], pk[CW / 2 - 1]);
      else *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
      if (col == 0 && a.lse) a.lse[orow] = lse_of(Mx, Ls);
    }
  };
  for (int i = 0; i < 2 * kWarps;) {
    const int unit = desc[i];
    if (unit < 0) {
      ++i;
      continue;
    }
    int e = i + 1;  // fragments [i, e) of this unit (in tile order; absent ones are -1)
    while (e < 2 * kWarps && (desc[e] == unit || desc[e] < 0)) ++e;
    float Mx = -INFINITY, Ls = 0.f, acc[CW];
#pragma unroll
    for (int q = 0; q < CW; ++q) acc[q] = 0.f;
    for (int x = i; x < e; ++x) {
      if (desc[x] < 0) continue;
      const unsigned char* base = smem + size_t(x >> 1) * L::kWarp;
      const float* ml = reinterpret_cast<const float*>(base + kRing * L::kStage + L::kFrag) + ((x & 1) * 16 + row) * 2;
      const float* fo = reinterpret_cast<const float*>(base + ((x & 1) ? 0 : kRing * L::kStage)) + row * D + col;
      join<CW>(Mx, Ls, acc, ml[0], ml[1], fo);
    }
    const int ur = unit / J, uj = unit - ur * J, Tu = pre[ur + 1] - pre[ur];
    const long long us = (long long)pre[ur] * J + (long long)uj * Tu;
    const long long ca = warp_of(us) / wpc, cb = warp_of(us + Tu - 1) / wpc;
    if (ca == cb) {
      finish(unit, Mx, Ls, acc);
    } else {
      const int slot = 2 * int(blockIdx.x) + (ca < blockIdx.x ? 0 : 1);
      float* so = args.slot_o + (size_t(slot) * kRowTile + row) * D + col;
#pragma unroll
      for (int q = 0; q < CW; q += 4) *reinterpret_cast<float4*>(so + q) = make_float4(acc[q], acc[q + 1], acc[q + 2], acc[q + 3]);
      if (col == 0) {
        args.slot_ml[(size_t(slot) * kRowTile + row) * 2] = Mx;
        args.slot_ml[(size_t(slot) * kRowTile + row) * 2 + 1] = Ls;
      }
      posted[np] = unit;  // (the CTA's first and last unit at most)
      pstart[np] = us;
      ++np;
    }
    i = e;
  }
  __shared__ int s_last;
  for (int x = 0; x < np; ++x) {
    const int unit = posted[x], ur = unit / J, Tu = pre[ur + 1] - pre[ur];
    const int ca = int(warp_of(pstart[x]) / wpc), cb = int(warp_of(pstart[x] + Tu - 1) / wpc);
    __syncthreads();
    if (tid == 0) s_last = atom_add_acq_rel(args.counters + ca) == uint32_t(cb - ca);
    __syncthreads();
    if (!s_last) continue;
    float Mx = -INFINITY, Ls = 0.f, acc[CW];
#pragma unroll
    for (int q = 0; q < CW; ++q) acc[q] = 0.f;
#pragma unroll 4
    for (int q = ca; q <= cb; ++q) {
      const int slot = 2 * q + (q == ca ? 1 : 0);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(args.slot_ml) + size_t(slot) * kRowTile + row);
      const float4* so = reinterpret_cast<const float4*>(args.slot_o + (size_t(slot) * kRowTile + row) * D + col);
      float v[CW];
#pragma unroll
      for (int u = 0; u < CW / 4; ++u) {
        const float4 y = __ldcg(so + u);
        v[4 * u] = y.x;
        v[4 * u + 1] = y.y;
        v[4 * u + 2] = y.z;
        v[4 * u + 3] = y.w;
      }
      join<CW>(Mx, Ls, acc, ml.x, ml.y, v);
    }
    finish(unit, Mx, Ls, acc);
    if (tid == 0) atomicExch(args.counters + ca, 0u);
  }
}

template <int D>
int launch_rows(const AttentionQ8Params& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return SPEC_ERR_LAUNCH;
  const size_t smem = RowsSmem<D>::bytes(p.b);
  if (cudaFuncSetAttribute(attention_q8_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
    return SPEC_ERR_LAUNCH;
  RowsArgs args{p, (p.n * (p.Hq / p.Hkv) + kRowTile - 1) / kRowTile, p.counters,
                reinterpret_cast<float*>(p.partials + kQ8SlotMlBytes), reinterpret_cast<float*>(p.partials)};
  const int grid = sms < kQ8MaxCtas ? sms : kQ8MaxCtas;
  const cudaError_t e = launch_pdl(attention_q8_rows_kernel<D>, dim3(grid), dim3(kQ8AttThreads), smem, stream, args);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace

size_t attention_q8_partial_bytes() { return kQ8SlotMlBytes + size_t(2) * kQ8MaxCtas * kQ8SlotRows * 128 * 4; }

int launch_attention_q8(const AttentionQ8Params& p, cudaStream_t stream) {
  if (p.n * (p.Hq / p.Hkv) > kRowsMost) return launch_attention_q8_tc(p, stream);
  return p.D == 128 ? launch_rows<128>(p, stream) : launch_rows<64>(p, stream);
}

}  // namespace spec
