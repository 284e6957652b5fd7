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
// below f16's range is 2^-24 of the row's largest contribution p |v|; l = sum
// P_j 2^-e_j (before the rounding), which is why e_j is kept within a span
// (attention_q8.cuh): alone, e = 1 of a row of zeros would take P below fp32's range.
//
// Bound: the cache's bytes.  A warp owns its work end to end: it takes an
// equal, contiguous range of 16-key tiles of all (request, kv head, 16-row
// tile) units laid end to end, copies each tile's K and V (2 x 16 x D bytes,
// contiguous in a page) into a private three-stage ring with 16-byte cp.async, and
// runs S = Q K^T and O += P V as register fragments (mma.sync m16n8k16: with at
// most 16 rows the tensor work of a 4 KB tile is 64 K multiply-adds, a third of
// the time the tile takes to arrive, and no operand passes through shared
// memory twice; a 128-row tcgen05 tile would be mostly padding).  The order of
// the head dimension inside a fragment is free as long as Q has the same, and
// that of the keys as long as P has the same, so both K and V fragments are
// read as whole 16-byte words.  What limits a warp is the issue of its ~340
// instructions a tile, so the history's loop is one short body, and what a unit's
// ends execute counts as much as what they read.
//   Few units: a cluster of CTAs takes each, its warps equal shares of the unit's
// tiles, and joins it through distributed shared memory.
//   Many: the warps of the whole GPU share all the tiles, and there is no
// barrier.  Units cut by a range boundary leave fragments (O, m, l)
// in the workspace, and a second, dependent launch joins them (joined in the same kernel,
// by the CTA's own warps behind a barrier and by the last CTA of a unit, they held a CTA 20 us
// on average, 57 us at most).  Only where all the warps of a CTA lie inside one unit does
// the CTA join its own first, so that a long context leaves few.
//   256 chains of four, contexts 256 to 4096, 32 / 8 heads of 128: 205 us (1.13 GB
// of cache at 5.5 TB/s); one token over 1000 keys 9.0 us.  A deeper ring is slower (four stages
// 215 us): with more bytes in flight than the memory needs, the dependent reads at a
// unit's ends only wait longer.
#include "common.cuh"
#include "kernels.cuh"

#include "attention_q8.cuh"
#include "cluster.cuh"
#include "e4m3.cuh"

namespace spec {

namespace {

constexpr int kWarps = 12;
constexpr int kQ8AttThreads = 32 * kWarps;
// Query rows a kv head up to which this kernel is taken (more, where clusters take the units): its time goes with
// the 16-row tiles, the tcgen05 kernel's hardly (in us, this one / that one; 8 kv heads of 128, no clusters): 32 rows,
// eight contexts of 16384 106 / 107, 64 ragged ones to 4096 104 / 228; 48 rows, 16 of 4096 81 / 72, 32 of 2048
// 85 / 91; 64 rows, 16 of 4096 96 / 72, eight of 16384 174 / 109.
constexpr int kRowsMost = 32;
constexpr int kTile = 16;    // keys of a tile
constexpr int kRowTile = 16; // query rows of a unit
constexpr int kRing = 3;     // tiles in a warp's ring
constexpr int kMinTicks = 2; // a warp gets at least this many ticks before another warp is used
// Ticks of a tree tile in the division of the work; a history tile is one.  A tree tile and the
// ends of its unit cost a warp some eight history tiles, nearly all latency: by 4, 6, 8 and 10 ticks the
// chains above take 214, 209, 205 and 202 us, 512 single tokens over 100 to 600 keys 115, 114, 121 and 125.
constexpr int kTreeTicks = 8;

// A cluster takes a unit and joins it by itself, in one launch, where the units are few enough for
// all of them to run at once (a GB300 holds 15 clusters of eight such CTAs, 36 of four, 76 of two) and a
// warp gets at most so many ticks; else the warps of the whole GPU share the work, and a second
// launch joins it.  In us, cluster / whole GPU, 32 / 8 heads of 128: one request, one token, 1000 keys 9.3 /
// 17.6, 8000 13.8 / 26.0, 32000 27.6 / 34.4, 60000 (39 ticks) 42.6 / 43.4; 16 requests of 4000 30.3 / 44.5.
// With more than kRowsMost query rows, against the tcgen05 kernel: one request of 2000 keys, 64 rows 14.3 / 29.4, 256 rows
// 20.6 / 26.5; of 4000, 256 rows (24 ticks) 29.5 / 30.0; two of 4000, 128 rows 28.5 / 33.2.
constexpr int kClusterTicks = 32, kClusterTicksTall = 20;
constexpr int kLargestCluster = 8;
inline int cluster_of(long long units, int sms) {
  return units <= 14 ? 8 : units <= 34 ? 4 : units <= 72 ? 2 : units <= sms ? 1 : 0;
}

template <int D>
struct RowsSmem {
  static constexpr int kHalf = kTile * D;         // K (or V) bytes of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kFrag = kRowTile * D * 4;  // fp32 O of a fragment
  static constexpr int kWarp = kRing * kStage;
  static_assert(kWarp >= kFrag, "a fragment takes the idle ring");
  static constexpr int kMl = kWarps * kWarp;      // [warp][16] (m, l)
  static constexpr int kMeta = kMl + kWarps * kRowTile * 8;  // [warp][stage] the tile's word
  static constexpr int kScan = kMeta + kWarps * kRing * 4;
  static size_t bytes(int b) { return size_t(kScan) + 12u * size_t(b + 1); }
  // (a cluster a unit: no scan, there the CTA's joined fragment: O, then (m, l))
  static constexpr int kUnitBytes = kScan + kFrag + kRowTile * 8;
};

// What the kernel leaves for the joining one: table[0] = {warps, warps a CTA},
// table[1 + warp] = the unit that the warp begins and does not finish
// {last warp on it (-1: none), request, (kv head, row tile)}.
struct RowsArgs {
  AttentionQ8Params p;
  int m_tiles;    // 16-row tiles of a kv head's n * G rows
  int4* table;
  float4* slot_o; // [2 * warp + i][D / 8][32], i = 1: the unit that the warp begins
  float2* slot_ml;  // [2 * warp + i][16]
};
static_assert((size_t(kQ8MaxCtas) * kWarps + 1) * 16 <= kQ8BegunBytes && 2 * kWarps * kRowTile <= 2 * kQ8SlotRows, "slots");

// The fragments of a unit on warps [wa, wb], wpc of them a CTA: a CTA whose warps lie
// strictly between has joined its own into its first warp's slot.
struct Fragments {
  int wa, wb, wpc, before, solid;  // warps before the first such CTA, and those CTAs
  __device__ Fragments(int a, int b, int c) : wa(a), wb(b), wpc(c) {
    const int k1 = wa / wpc + 1, k2 = wb / wpc - 1;
    solid = k2 >= k1 ? k2 - k1 + 1 : 0;
    before = solid ? k1 * wpc - wa : wb - wa + 1;
  }
  __device__ int count() const { return wb - wa + 1 - solid * (wpc - 1); }
  __device__ int warp(int i) const {
    return i < before ? wa + i : i < before + solid ? wa + before + (i - before) * wpc : wa + i + solid * (wpc - 1);
  }
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

// two bf16 values times inv, as f16x2
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float inv) { return pack_f16(bf16_lo(w) * inv, bf16_hi(w) * inv); }
__device__ __forceinline__ uint32_t word_of(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// The larger magnitude halfword by halfword, whatever it is: an inf or a NaN shows as 0x7f80 or
// more, and only then the finite ones are looked for (a third of the instructions).
__device__ __forceinline__ uint32_t raw_max(uint32_t m, const uint4& x) {
  m = __vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
  return __vmaxu2(__vmaxu2(m, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t finite_max(uint32_t m, const uint4& x) {
  return max_abs_bf16(max_abs_bf16(max_abs_bf16(max_abs_bf16(m, x.x), x.y), x.z), x.w);
}

// CLUSTER: a cluster of CTAs takes one unit (grid: cluster, units) and joins it by itself.
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kQ8AttThreads, 1) attention_q8_rows_kernel(const __grid_constant__ RowsArgs args) {
  using L = RowsSmem<D>;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int KS = D / 16;   // k-steps of Q K^T
  constexpr int NT = D / 8;    // 8-column tiles of O
  const AttentionQ8Params& a = args.p;
  extern __shared__ __align__(128) unsigned char smem[];
  int* pre = reinterpret_cast<int*>(smem + L::kScan);  // [b + 1] ticks of one (kv head, row tile) before request r
  int* slen = pre + a.b + 1;                           // [b]
  int* srow = slen + a.b + 1;                          // [b] table row, -1 if bad
  __shared__ int wsum[kWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int G = a.Hq / a.Hkv, M = a.n * G, J = a.Hkv * args.m_tiles;
  const int tree_tiles = (a.n + kTile - 1) / kTile, tree_ticks = kTreeTicks * tree_tiles;

  pdl_wait();
  pdl_trigger();
  // The warp's range of ticks [S, E) of T; its first unit (r, j), whose ticks are Tr, and tick t of it.
  long long T = 0, NW = 0;
  int wpc = kWarps, me0 = 0, me = 0, S = 0, E = 0, r = 0, Tr = 0, j = 0, t = 0;
  bool solid = CLUSTER;  // whether all of the CTA's warps lie (strictly between the first and the last of) one unit
  ReqQ8 own{0, -1};      // CLUSTER: the request's history
  auto req_of = [&](int f) {
    int lo = 0, hi = a.b;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * J <= f) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  if (CLUSTER) {
    r = blockIdx.y / J;
    j = blockIdx.y - r * J;
    own = req_q8(a, a.seq_lens[r], a.req_pool_idx[r], blockIdx.x == 0 && j == 0 && tid == 0);
    Tr = (own.len + kTile - 1) / kTile + tree_ticks;
    me = blockIdx.x * kWarps + w;
    const long long warps = gridDim.x * kWarps;
    S = t = int(me * (long long)Tr / warps);
    E = int((me + 1) * (long long)Tr / warps);
  } else {
    // ---- ticks before each request ----
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
          t = (q.len + kTile - 1) / kTile + tree_ticks;
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
    T = (long long)pre[a.b] * J;  // (the host keeps it below 2^31)
    // wpc warps a CTA over `ctas` CTAs, every warp with at least one tick
    const long long grid = gridDim.x;
    wpc = int((T + grid * kMinTicks - 1) / (grid * kMinTicks));
    wpc = wpc < 1 ? 1 : wpc > kWarps ? kWarps : wpc;
    long long ctas = (T + (long long)wpc * kMinTicks - 1) / ((long long)wpc * kMinTicks);
    if (ctas > grid) ctas = grid;
    NW = ctas * wpc < T ? ctas * wpc : T;
    if (blockIdx.x == 0 && tid == 0) args.table[0] = make_int4(int(NW), wpc, 0, 0);
    me0 = int(blockIdx.x) * wpc;
    me = me0 + w;
    if (w >= wpc || me >= NW) return;
    S = int(me * T / NW);
    E = int((me + 1) * T / NW);
    r = req_of(S);
    Tr = pre[r + 1] - pre[r];
    {
      const int rem = S - pre[r] * J;
      j = rem / Tr;
      t = rem - j * Tr;
    }
    // whether all of the CTA's warps lie strictly between the first and the last of one unit
    if (me0 + wpc < NW) {
      const long long u0 = S - t, c0 = me0 * T / NW, c1 = (long long)(me0 + wpc) * T / NW;
      solid = u0 < c0 && c1 < u0 + Tr;
    }
  }
  if (t > Tr - tree_ticks && (t - (Tr - tree_ticks)) % kTreeTicks) {  // inside a tree tile, which is the warp's that holds its first tick
    const int skip = kTreeTicks - (t - (Tr - tree_ticks)) % kTreeTicks;
    if (!CLUSTER && lane < kRowTile) args.slot_ml[size_t(2 * me) * kRowTile + lane] = make_float2(-INFINITY, 0.f);
    __syncwarp();
    S += skip;
    t += skip;
    if (!CLUSTER && t == Tr) {
      t = 0;
      if (++j == J) {
        j = 0;
        ++r;
        if (r < a.b) Tr = pre[r + 1] - pre[r];
      }
    }
  }
  if (!CLUSTER && lane == 0) args.table[1 + me] = make_int4(-1, 0, 0, 0);

  unsigned char* mine = smem + size_t(w) * L::kWarp;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  float2* fml = reinterpret_cast<float2*>(smem + L::kMl) + w * kRowTile;
  uint32_t* meta = reinterpret_cast<uint32_t*>(smem + L::kMeta) + w * kRing;
  if (lane < kRowTile) fml[lane] = make_float2(-INFINITY, 0.f);

  // Lane l looks up tick mb + l of the range: its (page, kv head) unit (-1: a tree
  // tile's), and in one word the first key in the page, the keys that count and the
  // exponents of the K and V scales.  A bad page has no key that counts.
  const int SHIFT = a.page_size == 16 ? 0 : a.page_size == 32 ? 1 : 2;  // log2(tiles a page)
  int mb = S - 32, l_unit = 0;
  uint32_t l_word = 0;
  auto load_meta = [&](int f0) {
    mb = f0;
    const int f = f0 + lane;
    l_unit = -1;
    l_word = 0;
    if (f < E) {
      const int fr = CLUSTER ? r : req_of(f), fT = CLUSTER ? Tr : pre[fr + 1] - pre[fr];
      const int rem = CLUSTER ? f : f - pre[fr] * J, fj = CLUSTER ? j : rem / fT, ft = CLUSTER ? f : rem - fj * fT;
      const int row = CLUSTER ? own.row : srow[fr], len = CLUSTER ? own.len : slen[fr];
      if (ft < fT - tree_ticks && row >= 0) {
        const int pid = a.page_table[size_t(row) * a.row_pages + (ft >> SHIFT)];
        if (pid < 0 || pid >= a.num_pages) {
          raise_error(a.error, SPEC_DEV_INDEX);
          l_unit = 0;
          l_word = uint32_t(kExpBias) << 16 | uint32_t(kExpBias) << 24;
        } else {
          l_unit = pid * a.Hkv + fj / args.m_tiles;
          l_word = uint32_t(ft & ((1 << SHIFT) - 1)) * kTile | uint32_t(min(kTile, len - ft * kTile)) << 8 |
                   uint32_t(a.k_scales[l_unit]) << 16 | uint32_t(a.v_scales[l_unit]) << 24;
        }
      }
    }
  };
  constexpr int kChunks = D / 16;  // 16-byte chunks of a key
  constexpr int kCopies = kTile * kChunks / 32, kKeys = 32 / kChunks;
  // where this lane's chunk of a copy goes: the K chunk order turns with the key's
  // parity, V's with the pair of keys, so that the fragment reads below meet no bank twice
  const int ckey = lane / kChunks, cx = lane % kChunks;
  const uint32_t kdst = ckey * D + (D == 128 ? cx ^ (4 * (ckey & 1)) : cx) * 16;
  auto vdst = [&](int i) {
    const int key = i * kKeys + ckey;
    return uint32_t(L::kHalf + ckey * D + (D == 128 ? cx ^ (((key >> 1) & 3) << 1) : cx ^ (((key >> 1) & 1) << 1)) * 16);
  };
  auto issue = [&](int f) {
    if (f < E) {
      if (f - mb >= 32) load_meta(f);
      const int unit = __shfl_sync(FULL, l_unit, f - mb);
      const uint32_t word = __shfl_sync(FULL, l_word, f - mb);
      if (unit >= 0) {
        const int cnt = (word >> 8) & 31;
        const size_t at = (size_t(unit) * a.page_size + (word & 63)) * D + lane * 16;
        const uint32_t st = ring + uint32_t(f % kRing) * L::kStage;
        const uint8_t *ks = a.k_pages + at, *vs = a.v_pages + at;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const uint32_t nb = i * kKeys + ckey < cnt ? 16u : 0u;  // (a key past the history reads as zeros)
          cp16(st + kdst + i * 512, ks + i * 512, nb);
          cp16(st + vdst(i) + i * 512, vs + i * 512, nb);
        }
        if (lane == 0) meta[f % kRing] = word;
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(S + i);

  const int kread = g * D + (D == 128 ? c ^ (4 * (g & 1)) : c) * 16;
  const int vread = L::kHalf + 2 * c * D + (D == 128 ? (g ^ (c << 1)) * 16 : ((g >> 1) ^ ((c & 1) << 1)) * 16 + (g & 1) * 8);
  for (int f = S; f < E;) {
    // ---- a unit, or the part of it in this range: its Q rows as f16 fragments, masks, empty results ----
    const int h = j / args.m_tiles, mt = j - h * args.m_tiles;
    const int t_first = t, f_first = f, Th = Tr - tree_ticks;
    uint32_t qf[KS][4];
    float xf[2];                // softmax factor of rows g, g + 8: scale * log2e * the row's power of two
    float o[NT][4], m[2], l[2];
    int evb = -1;               // the exponent byte that the unit's value scales are taken relative to (its first tile's)
    unsigned long long nonfinite = 0;  // tree nodes whose V row holds an inf or a NaN
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
      auto over_row = [&](uint32_t mx) {
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
        return max(mx, __shfl_xor_sync(FULL, mx, 2));
      };
      uint32_t mx = 0;
#pragma unroll
      for (int u = 0; u < D / 32; ++u) mx = raw_max(mx, x[u]);
      mx = over_row(mx);
      if (__any_sync(FULL, mx >= 0x7f80u)) {
        mx = 0;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) mx = finite_max(mx, x[u]);
        mx = over_row(mx);
      }
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
    // The reference m of a row: P is 2^kPBaseLog2 at the row's maximum when it is set,
    // and it moves only when P would pass 2^kLazyLog2 times that.
    constexpr float kMost = kLazyLog2 + kPBaseLog2;
    auto move = [&](const float (&x)[2][4]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        if (mx > m[i] + kMost) {
          const float fac = fast_exp2(m[i] + kPBaseLog2 - mx);  // (0 from an empty row)
          l[i] *= fac;
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            o[q][2 * i] *= fac;
            o[q][2 * i + 1] *= fac;
          }
          m[i] = mx - kPBaseLog2;
        }
      }
    };

    auto raise = [&](int top) {  // the base moves up to `top`
      const int up = evb >= 0 ? top - evb : 0;
      evb = top;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (the four lanes of a row keep one m: the largest of their sums decides)
        float most = fmaxf(l[i], __shfl_xor_sync(FULL, l[i], 1));
        most = fmaxf(most, __shfl_xor_sync(FULL, most, 2));
        if (up > 0 && m[i] > -INFINITY) {
          const float mn = floorf(m[i] - float(raised_into_l(up, most))), by = m[i] - mn;  // (exact)
          const float fac = fast_exp2(by - float(up));
          l[i] *= fast_exp2(by);
          m[i] = mn;
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            o[q][2 * i] *= fac;
            o[q][2 * i + 1] *= fac;
          }
        }
      }
    };
    // ---- history ----
    for (const int fh = min(E, f + (t < Th ? Th - t : 0)); f < fh; ++f) {
      cp_wait<kRing - 2>();
      __syncwarp();
      issue(f + kRing - 1);
      const unsigned char* st = mine + (f % kRing) * L::kStage;
      const uint32_t word = meta[f % kRing];
      const int cnt = (word >> 8) & 31, ev = word >> 24;
      const float kf = exp_scale((word >> 16) & 255);
      if (evb < 0) evb = ev;
      float s[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[q][i] = 0.f;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {  // key 8 q + g: chunks c and c + 4
          const uint4 y = *reinterpret_cast<const uint4*>(st + (kread ^ (64 * u)) + 8 * q * D);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            e4m3x4_to_f16x4(word_of(y, i), b0, b1);
            mma_f16(s[q], qf[4 * u + i], b0, b1);
          }
        }
      }
      // y = x - m with x = s * factor + (e - evb); a row without a reference yet has y = inf
      float de = float(ev - evb);
      const float x0 = xf[0] * kf, x1 = xf[1] * kf, d0 = de - m[0], d1 = de - m[1];
      const bool far = unsigned(ev - evb + kSpanDown) > unsigned(kSpanDown + kSpanUp);
      float y[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y[q][i] = fmaf(s[q][i], x0, d0);
          y[q][2 + i] = fmaf(s[q][2 + i], x1, d1);
        }
      if (cnt < kTile) {  // keys past the history
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (8 * q + 2 * c + (i & 1) >= cnt) y[q][i] = s[q][i] = -INFINITY;
      }
      const float ym = fmaxf(fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3])), fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
      const bool unset = m[0] == -INFINITY || m[1] == -INFINITY;
      float dl = ratio_scale(evb - ev);  // l's share of P (a sum of its own below the span)
      if (__any_sync(FULL, ym > kMost || unset || far)) {
        if (far) {
          if (ev > evb) raise(ev);
          de = float(span_of(ev - evb));
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[q][i] = 8 * q + 2 * c + (i & 1) < cnt ? fmaf(s[q][i], i < 2 ? x0 : x1, de) : -INFINITY;
        move(y);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[q][i] -= m[i >> 1] == -INFINITY ? 0.f : m[i >> 1];
        if (far) {
          dl = ev < evb ? 0.f : 1.f;
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (ev < evb) l[i >> 1] = fmaf(fast_exp2(y[q][i]), exp_scale(kExpBias + kSpanDown), l[i >> 1]);
              y[q][i] += float(ev - evb) - de;
            }
        }
      }
      uint32_t pa[4];
      float sum[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = fast_exp2(y[q][2 * i]), p1 = fast_exp2(y[q][2 * i + 1]);
          sum[i] = q == 0 ? p0 + p1 : sum[i] + (p0 + p1);
          pa[2 * q + i] = pack_f16(p0, p1);
        }
      l[0] = fmaf(sum[0], dl, l[0]);
      l[1] = fmaf(sum[1], dl, l[1]);
      // O += P V: b0 holds keys 2c, 2c+1, b1 keys 2c+8, 2c+9 of a column
      uint32_t v[4][D / 32];  // D / 8 bytes of each of the four keys
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char* sv = st + vread + ((i & 1) + 8 * (i >> 1)) * D;
        if (D == 128) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(sv);
          v[i][0] = w4.x;
          v[i][1] = w4.y;
          v[i][D / 32 - 2] = w4.z;
          v[i][D / 32 - 1] = w4.w;
        } else {
          const uint2 w2 = *reinterpret_cast<const uint2*>(sv);
          v[i][0] = w2.x;
          v[i][1] = w2.y;
        }
      }
#pragma unroll
      for (int u = 0; u < D / 32; ++u)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t a0, a1, c0, c1;
          e4m3x4_to_f16x4(__byte_perm(v[0][u], v[1][u], hf ? 0x7362 : 0x5140), a0, a1);
          e4m3x4_to_f16x4(__byte_perm(v[2][u], v[3][u], hf ? 0x7362 : 0x5140), c0, c1);
          mma_f16(o[4 * u + 2 * hf], pa, a0, c0);
          mma_f16(o[4 * u + 2 * hf + 1], pa, a1, c1);
        }
    }

    // ---- tree nodes: the step's bf16 rows, each divided by its own power of two ----
    const int f_end = f_first + (Tr - t_first);  // the tick behind the unit
    for (; f < E && f < f_end; f += kTreeTicks) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kTreeTicks; ++i) issue(f + kRing - 1 + i);
      const int nb = (t_first + (f - f_first) - Th) / kTreeTicks * kTile;  // first node of the tile
      unsigned long long mask[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rg = mt * kRowTile + g + 8 * i;
        mask[i] = rg < M ? a.mask_bits[size_t(r) * a.n + rg / G] : 0ull;
      }
      const uint16_t* kn = static_cast<const uint16_t*>(a.k_new) + size_t(h) * D;
      const bool upper = nb + 8 < a.n;  // whether the tile's second eight rows hold a node
      float s[2][4], kf[2][2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q == 1 && !upper) {
          kf[1][0] = kf[1][1] = 1.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) s[1][i] = 0.f;
          continue;
        }
        const int node = nb + 8 * q + g;
        const uint4* src = reinterpret_cast<const uint4*>(kn + (size_t(r) * a.n + (node < a.n ? node : 0)) * a.new_ld);
        uint4 kx[D / 32];
#pragma unroll
        for (int u = 0; u < D / 32; ++u)
          kx[u] = node < a.n ? __ldg(src + (u >> 1) * 8 + 2 * c + (u & 1)) : make_uint4(0, 0, 0, 0);
        auto over_row = [&](uint32_t mx) {
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
          return max(mx, __shfl_xor_sync(FULL, mx, 2));
        };
        uint32_t mx = 0;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) mx = raw_max(mx, kx[u]);
        mx = over_row(mx);
        if (__any_sync(FULL, mx >= 0x7f80u)) {
          mx = 0;
#pragma unroll
          for (int u = 0; u < D / 32; ++u) mx = finite_max(mx, kx[u]);
          mx = over_row(mx);
        }
        const int e = norm_exp(mx);
        const float inv = exp_scale(2 * kExpBias - e);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[q][i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const uint4& y = kx[kk >> 1];
          mma_f16(s[q], qf[kk], scaled_f16(word_of(y, (kk & 1) * 2), inv), scaled_f16(word_of(y, (kk & 1) * 2 + 1), inv));
        }
        kf[q][0] = exp_scale(__shfl_sync(FULL, e, 8 * c));
        kf[q][1] = exp_scale(__shfl_sync(FULL, e, 8 * c + 4));
      }
      auto vrow = [&](int node) {  // the thread's D / 8 elements of a node's V row
        return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v_new) + size_t(h) * D +
                                              (size_t(r) * a.n + (node < a.n ? node : 0)) * a.new_ld) + g * (D / 64);
      };
      // V's exponents; the rows themselves are read again for the product
      int evk[4];  // of nodes 2c, 2c+1, 2c+8, 2c+9
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= 2 && !upper) {
          evk[i] = evb >= 0 ? evb : 1;
          continue;
        }
        const int node = nb + 2 * c + (i & 1) + 8 * (i >> 1);
        const uint4* src = vrow(node);
        auto over_row = [&](uint32_t mx) {
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(FULL, mx, 4));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 8));
          return max(mx, __shfl_xor_sync(FULL, mx, 16));
        };
        uint4 x[D / 64];
        uint32_t mx = 0;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
          x[u] = node < a.n ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
          mx = raw_max(mx, x[u]);
        }
        mx = over_row(mx);
        // an inf or a NaN must reach the rows that see the node and no
        // other: it is left out of the product and added at the end
        const unsigned who = __ballot_sync(FULL, mx >= 0x7f80u);
        if (who) {
          mx = 0;
#pragma unroll
          for (int u = 0; u < D / 64; ++u) mx = finite_max(mx, x[u]);
          mx = over_row(mx);
        }
        evk[i] = node >= a.n && evb >= 0 ? evb : norm_exp(mx);
        if (who) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (who & (0x11111111u << q)) {
              const int at = nb + 2 * q + (i & 1) + 8 * (i >> 1);
              if (at < kMaxN) nonfinite |= 1ull << at;
            }
        }
      }
      const int most = max(max(evk[0], evk[1]), max(evk[2], evk[3])), least = min(min(evk[0], evk[1]), min(evk[2], evk[3]));
      if (__any_sync(FULL, evb < 0 || most > evb + kSpanUp || least < evb - kSpanDown)) {
        int top = max(most, __shfl_xor_sync(FULL, most, 1));
        top = max(top, __shfl_xor_sync(FULL, top, 2));
        if (evb < 0 || top > evb + kSpanUp) raise(top);
#pragma unroll
        for (int i = 0; i < 4; ++i) evk[i] = evb + span_of(evk[i] - evb);
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
        }
      move(s);
      const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
      uint32_t pa[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float p00 = fast_exp2(s[q][0] - m0), p01 = fast_exp2(s[q][1] - m0);
        const float p10 = fast_exp2(s[q][2] - m1), p11 = fast_exp2(s[q][3] - m1);
        const float dl0 = ratio_scale(evb - evk[2 * q]), dl1 = ratio_scale(evb - evk[2 * q + 1]);
        l[0] = fmaf(p00, dl0, fmaf(p01, dl1, l[0]));
        l[1] = fmaf(p10, dl0, fmaf(p11, dl1, l[1]));
        pa[2 * q] = pack_f16(p00, p01);
        pa[2 * q + 1] = pack_f16(p10, p11);
      }
      float inv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) inv[i] = exp_scale(2 * kExpBias - evk[i]);
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {  // eight column tiles: element e of the thread's D / 8 is column tile e
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int node = nb + 2 * c + (i & 1) + 8 * (i >> 1);
          x[i] = node < a.n ? __ldg(vrow(node) + u) : make_uint4(0, 0, 0, 0);
        }
        if (nonfinite) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = make_uint4(finite_bf16(x[i].x), finite_bf16(x[i].y), finite_bf16(x[i].z), finite_bf16(x[i].w));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          auto el = [&](int i) {
            const uint32_t wd = word_of(x[i], e >> 1);
            return ((e & 1) ? bf16_hi(wd) : bf16_lo(wd)) * inv[i];
          };
          mma_f16(o[8 * u + e], pa, pack_f16(el(0), el(1)), upper ? pack_f16(el(2), el(3)) : 0u);
        }
      }
    }

    // ---- the unit's or the range's end ----
    const bool unit_end = f == f_end && f <= E;  // (past E: the last ticks are another warp's, which has nothing to add)
    // rows g, g + 8; columns c D/4 .. + D/4: [0, D/8) from fragment columns 2c, [D/8, D/4) from 2c + 1
    const bool whole = !CLUSTER && unit_end && t_first == 0;
    float lt[2];
    const float vs = exp_scale(evb < 1 ? 1 : evb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lt[i] = l[i] + __shfl_xor_sync(FULL, l[i], 1);
      lt[i] += __shfl_xor_sync(FULL, lt[i], 2);
      const float inv = whole ? inverse_of(lt[i]) : settle(m[i], lt[i]);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        o[q][2 * i] = o[q][2 * i] * inv * vs;
        o[q][2 * i + 1] = o[q][2 * i + 1] * inv * vs;
      }
      if (nonfinite) {
        const int rg = mt * kRowTile + g + 8 * i;
        const unsigned long long seen = rg < M ? nonfinite & a.mask_bits[size_t(r) * a.n + rg / G] : 0ull;
        for (int node = 0; node < a.n; ++node)
          if (seen >> node & 1) {
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
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rg = mt * kRowTile + g + 8 * i;
        if (rg < M) {
          const size_t orow = (size_t(r) * a.n + rg / G) * a.Hq + h * G + rg % G;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + c * (D / 4));
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < NT; q += 8) {
              auto pk = [&](int e) { return pack_bf16x2(o[q + e][2 * i + u], o[q + e + 1][2 * i + u]); };
              dst[(u * NT + q) / 8] = make_uint4(pk(0), pk(2), pk(4), pk(6));
            }
          if (c == 0 && a.lse) a.lse[orow] = lse_of(m[i], lt[i]);
        }
      }
    } else {
      // a fragment, as the registers hold it: word e of a lane is columns
      // c D/4 + 4 (e % (D/16)) .. + 3 of row g + 8 (e / (D/16))
      const size_t slot = size_t(2 * me) + (t_first == 0 ? 1 : 0);
      if (solid) {
        cp_wait<0>();
        __syncwarp();
      }
      float4* dst = (solid ? reinterpret_cast<float4*>(mine) : args.slot_o + slot * (32 * NT)) + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int q = 0; q < NT; q += 4)
            dst[((i * 2 + u) * (NT / 4) + q / 4) * 32] = make_float4(o[q][2 * i + u], o[q + 1][2 * i + u], o[q + 2][2 * i + u], o[q + 3][2 * i + u]);
      float2* ml = solid ? fml : args.slot_ml + slot * kRowTile;
      if (c == 0) {
        ml[g] = make_float2(m[0], lt[0]);
        ml[g + 8] = make_float2(m[1], lt[1]);
      }
      if (!CLUSTER && lane == 0 && t_first == 0) args.table[1 + me] = make_int4(int(((long long)f_end * NW - 1) / T), r, j, 0);
    }
    if (!CLUSTER && unit_end) {
      t = 0;
      if (++j == J) {
        j = 0;
        ++r;
        if (r < a.b) Tr = pre[r + 1] - pre[r];
      }
    }
  }
  cp_wait<0>();
  if (!solid) return;
  // ---- the CTA's fragments are all of one unit: joined here, so that few are left of a long context ----
  __syncthreads();
  for (int x = tid; x < 32 * NT; x += 32 * wpc) {
    const int row = ((x & 31) >> 2) + 8 * (x / (16 * NT));
    const float2* ml = reinterpret_cast<const float2*>(smem + L::kMl) + row;
    float Mx = -INFINITY, Ls = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < wpc; ++q) {
      const float4 y = reinterpret_cast<const float4*>(smem + size_t(q) * L::kWarp)[x];
      const float v[4] = {y.x, y.y, y.z, y.w};
      join<4>(Mx, Ls, acc, ml[q * kRowTile].x, ml[q * kRowTile].y, v);
    }
    const float f = settle(Mx, Ls) * float(1 << kRoomLog2);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] *= f;
    const bool first = (x & 3) == 0 && (x / 32) % (NT / 2) == 0;
    if (CLUSTER) {
      reinterpret_cast<float4*>(smem + L::kScan)[x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (first) reinterpret_cast<float2*>(smem + L::kScan + L::kFrag)[row] = make_float2(Mx, Ls);
    } else {
      args.slot_o[size_t(2 * me0) * (32 * NT) + x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (first) args.slot_ml[size_t(2 * me0) * kRowTile + row] = make_float2(Mx, Ls);
    }
  }
  if (CLUSTER) {
    // ---- and the cluster's CTAs each a share of the words ----
    cluster_sync();
    const int share = 32 * NT / gridDim.x;  // (gridDim.x: 1, 2, 4 or 8 CTAs)
    for (int i = tid; i < share; i += kQ8AttThreads) {
      const int x = blockIdx.x * share + i, e = x >> 5, l = x & 31;
      const int row = (l >> 2) + 8 * (e / (NT / 2)), rg = (j % args.m_tiles) * kRowTile + row, h = j / args.m_tiles;
      float Mx = -INFINITY, Ls = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      float4 o[kLargestCluster];
      float2 ml[kLargestCluster];
#pragma unroll
      for (int q = 0; q < kLargestCluster; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        if (q < int(gridDim.x)) {
          ml[q] = cluster_ld2(cluster_addr(smem + L::kScan + L::kFrag + row * 8, q));
          o[q] = cluster_ld4(cluster_addr(smem + L::kScan + x * 16, q));
        }
      }
#pragma unroll
      for (int q = 0; q < kLargestCluster; ++q) {
        const float v[4] = {o[q].x, o[q].y, o[q].z, o[q].w};
        join<4>(Mx, Ls, acc, ml[q].x, ml[q].y, v);
      }
      if (rg < M) {
        const float inv = settled_inverse(Ls);
        const size_t orow = (size_t(r) * a.n + rg / G) * a.Hq + h * G + rg % G;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + (l & 3) * (D / 4) + 4 * (e % (NT / 2))) =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        if (a.lse && (l & 3) == 0 && e % (NT / 2) == 0) a.lse[orow] = lse_of(Mx, Ls);
      }
    }
    cluster_sync();  // (no CTA ends while another reads its shared memory)
  }
}

// Joins the units cut over warps: a block the unit that warp blockIdx.x begins and does not
// finish; a thread one 16-byte word of the fragments' layout.
template <int D>
__global__ void __launch_bounds__(4 * D, 3) attention_q8_rows_join_kernel(const __grid_constant__ RowsArgs args) {
  constexpr int NT = D / 8, kBatch4 = 4;
  pdl_wait();
  pdl_trigger();
  const AttentionQ8Params& a = args.p;
  const int4 head = __ldcg(args.table), unit = __ldcg(args.table + 1 + blockIdx.x);
  if (int(blockIdx.x) >= head.x || unit.x < 0) return;  // (an entry behind the warps that ran is not looked at)
  const Fragments fr(blockIdx.x, unit.x, head.y);
  const int nf = fr.count(), r = unit.y, j = unit.z, h = j / args.m_tiles, mt = j - h * args.m_tiles;
  const int G = a.Hq / a.Hkv, M = a.n * G, lane = threadIdx.x & 31, e = threadIdx.x >> 5;
  const int row = (lane >> 2) + 8 * (e / (NT / 2)), rg = mt * kRowTile + row;
  if (rg >= M) return;
  float Mx = -INFINITY, Ls = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int i0 = 0; i0 < nf; i0 += kBatch4) {
    float2 ml[kBatch4];
    float4 o[kBatch4];
#pragma unroll
    for (int i = 0; i < kBatch4; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i < nf) {
        const int slot = 2 * fr.warp(i0 + i) + (i0 + i == 0 ? 1 : 0);
        ml[i] = __ldcg(args.slot_ml + slot * kRowTile + row);
        o[i] = __ldcg(args.slot_o + size_t(slot) * (32 * NT) + threadIdx.x);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch4; ++i) {
      const float v[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
      join<4>(Mx, Ls, acc, ml[i].x, ml[i].y, v);
    }
  }
  const float inv = settled_inverse(Ls);
  const size_t orow = (size_t(r) * a.n + rg / G) * a.Hq + h * G + rg % G;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + (lane & 3) * (D / 4) + 4 * (e % (NT / 2))) =
      make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (a.lse && (lane & 3) == 0 && e % (NT / 2) == 0) a.lse[orow] = lse_of(Mx, Ls);
}

// The units of a call, the ticks of one at most, and the CTAs of a cluster that takes one (0: none does).
struct RowsPlan {
  int m_tiles, cluster;
  long long units, ticks;
  RowsPlan(const AttentionQ8Params& p, int sms) {
    const int rows = p.n * (p.Hq / p.Hkv);
    m_tiles = (rows + kRowTile - 1) / kRowTile;
    units = (long long)p.b * p.Hkv * m_tiles;
    ticks = (long long)(p.max_seq_len / kTile) + 1 + kTreeTicks * ((p.n + kTile - 1) / kTile);
    cluster = cluster_of(units, sms);
    if (ticks > (long long)(rows <= kRowsMost ? kClusterTicks : kClusterTicksTall) * cluster * kWarps) cluster = 0;
  }
};

template <int D>
int launch_rows(const AttentionQ8Params& p, const RowsPlan& plan, int sms, cudaStream_t stream) {
  RowsArgs args{p, plan.m_tiles,
                reinterpret_cast<int4*>(p.partials + kQ8SlotMlBytes - kQ8BegunBytes),
                reinterpret_cast<float4*>(p.partials + kQ8SlotMlBytes), reinterpret_cast<float2*>(p.partials)};
  if (plan.cluster > 0) {
    constexpr int bytes = RowsSmem<D>::kUnitBytes;
    if (cudaFuncSetAttribute(attention_q8_rows_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return SPEC_ERR_LAUNCH;
    return launch_cluster(attention_q8_rows_kernel<D, true>, plan.cluster, dim3(plan.cluster, unsigned(plan.units)), dim3(kQ8AttThreads), bytes,
                          stream, args) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_LAUNCH;
  }
  const size_t smem = RowsSmem<D>::bytes(p.b);
  if (cudaFuncSetAttribute(attention_q8_rows_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(RowsSmem<D>::bytes(kAttentionQ8MaxB))) != cudaSuccess)  // (the most, so that calls of two threads agree)
    return SPEC_ERR_LAUNCH;
  const int grid = sms < kQ8MaxCtas ? sms : kQ8MaxCtas;
  if (launch_pdl(attention_q8_rows_kernel<D, false>, dim3(grid), dim3(kQ8AttThreads), smem, stream, args) != cudaSuccess)
    return SPEC_ERR_LAUNCH;
  // (warps there can be at most: the second kernel's blocks beyond those that run leave at once)
  const long long most = plan.ticks * plan.units / kMinTicks + kWarps;
  const int warps = most < grid * kWarps ? int(most) : grid * kWarps;
  return launch_pdl(attention_q8_rows_join_kernel<D>, dim3(warps), dim3(4 * D), 0, stream, args) == cudaSuccess ? SPEC_OK
                                                                                                           : SPEC_ERR_LAUNCH;
}

}  // namespace

size_t attention_q8_partial_bytes() { return kQ8SlotMlBytes + size_t(2) * kQ8MaxCtas * kQ8SlotRows * 128 * 4; }

int launch_attention_q8(const AttentionQ8Params& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return SPEC_ERR_LAUNCH;
  const RowsPlan plan(p, sms);
  if (p.n * (p.Hq / p.Hkv) > kRowsMost && plan.cluster == 0) return launch_attention_q8_tc(p, stream);
  return p.D == 128 ? launch_rows<128>(p, plan, sms, stream) : launch_rows<64>(p, plan, sms, stream);
}

}  // namespace spec
