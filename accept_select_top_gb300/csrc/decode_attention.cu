// decode_attention.cu -- attention of one new token a request over the paged bf16
// cache.  Requests of a group share the pages of their first tokens.
//
// For request r and q head h: x_j = scale q . k_j over its tokens, out = sum_j
// 2^(x_j log2e - m) v_j / l with a running reference m and sum l.  The sums over
// the shared tokens and over a request's own ones are independent until the end,
// so a group's shared tokens are read once for all its rows.
//
// P is rounded to bf16, V's type (half a step 2^-8; with random values out is off by 1.4 times what its own rounding
// makes it); the sums l and O are fp32.  (P in two bf16 parts, whose products are exact to 2^-16, costs 2 to 11%: the batch
// below 388 us, not 363.)
//
// Bound: the cache's bytes.  A segment is a group's shared tokens (rows: every member's q heads of a kv head) or a
// request's own tokens; a unit is (segment, kv head, up to 64 rows).  One CTA a SM takes an equal contiguous
// range of all units, laid end to end as tiles of 32 KB.
//   Four producer warps look up the slots of the keys (two tiles ahead) and copy K and V rows with 16-byte
// cp.async into a ring of 160 KB; they do not care where units end, so the memory stays busy while one does.
//   Eight consumer warps compute on register fragments (mma.sync m16n8k16; rows are few, and a 128-row tcgen05 tile
// would be padding).  A unit's part of up to 16 rows belongs to four of them, which share each tile's keys (to one, if it
// is a single tile), and the parts take turns: what the ends of a part take (its Q, the results) is 3 us of latency,
// during which the others compute.  32 rows: two row tiles times four shares of the keys; 64: four times two.  The order of
// the head dimension inside a fragment is free as long as Q has the same, so K fragments are read as 16-byte words.
// At a unit's end the warps' results are joined through shared memory.
//   Units cut by a range boundary, and all of a grouped request, leave fp32 results in the workspace; a second,
// dependent launch joins them.  Where units are few and short, a cluster of CTAs takes each, an equal share of its tiles a
// CTA, and joins it through distributed shared memory in the same launch.  No atomics: a call's result is always the
// same.
//   256 requests of 256 to 4096 tokens, 32 / 8 heads of 128: 354 to 363 us (2.34 GB, 6.4 to 6.6 TB/s); 512 requests of 256
// tokens 113, of one token 36; one request of 1001 tokens 6.5.
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"

#include "cluster.cuh"
#include "decode_attention.cuh"

namespace spec {

namespace {

constexpr int kConsumers = 8, kProducers = 4;
constexpr int kDecThreads = 32 * (kConsumers + kProducers);
constexpr int kRing = 5;
// A cluster takes a unit where all of them run at once (a GB300 holds 15 clusters of eight CTAs of a SM each, 36 of four,
// 76 of two) and a CTA gets at most so many tiles; else the SMs share the work, and a second launch joins it.  In us, cluster /
// all SMs, 32 / 8 heads of 128: one request of 1000 tokens 6.5 / 12.4, 8192 (16 tiles a CTA) 13.9 / 17.7, 16384 22.6 / 22.1; eight
// of 1000 9.4 / 17.5, 2048 (16) 13.8 / 22.0, 4096 27 / 34.
constexpr int kClusterMost = 8, kClusterTiles = 24;
inline int cluster_of(long long units, int sms) { return units <= 14 ? 8 : units <= 34 ? 4 : units <= 72 ? 2 : units <= sms ? 1 : 0; }
constexpr int kOwners = kConsumers + 2;  // who may have a part to itself: a warp, or four of them
// A part of at most so many tiles, where the CTA's range is so many times longer, goes to one warp.
constexpr int kSoloTiles = 1, kSoloRange = 2;
// The work is divided in ticks of a quarter of a tile, so that short parts count by their keys; a tile belongs to the CTA
// that has its first tick.  A unit's end counts as kEndTicks.
constexpr int kEndTicks = kDecEndTicks;
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s: bound of every wait

template <int D>
struct DecSmem {
  static constexpr int kRow = 2 * D;               // bytes of a K (or V) row
  // Keys of a tile: 32 KB of K and V.  (Tiles of 64 keys for D 64, too, bounded it by what a tile costs besides its
  // bytes: 256 requests of 2048 tokens, 4 kv heads, 112 us, so 99.)
  static constexpr int kTile = 64 * 128 / D;
  static constexpr int kHalf = kTile * kRow;       // K of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kMerge = kRing * kStage;    // [warp][8 column tiles][32 lanes] float4
  static constexpr int kMl = kMerge + kConsumers * 8 * 32 * 16;  // [warp][16] (m, l)
  static constexpr int kMask = kMl + kConsumers * 16 * 8;        // [stage][4] keys that count, of a quarter of the tile each
  static constexpr int kBars = kMask + kRing * 4 * 4;            // full[5], empty[5], then [owner][5]
  static constexpr int kAbort = kBars + (2 + kOwners) * kRing * 8;
  static constexpr int kScan = kAbort + 16;        // pre [groups + b + 1], len [b], base [b]
  static size_t bytes(int b, int groups) { return size_t(kScan) + 4u * size_t(groups + 3 * b + 1); }
};
static_assert(DecSmem<128>::kScan + 4 * (4 * kDecodeMaxB + 1) + 256 <= 227 * 1024, "shared memory of one CTA");
static_assert(DecSmem<64>::kScan + 4 * (4 * kDecodeMaxB + 1) + 256 <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar, uint32_t count = 1) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// counts as an arrival once the thread's copies so far have landed
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
// Bounded wait for the phase of the given parity: false once kWaitCycles have passed or another warp has given up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try(bar, parity)) return true;
  const long long start = clock64();
  do {
    for (int i = 0; i < 64; ++i)
      if (mbar_try(bar, parity)) return true;
  } while (!*abort_flag && clock64() - start <= kWaitCycles);
  return false;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
  return x;
}
// four 8x8 matrices of 16-bit values, transposed
__device__ __forceinline__ uint4 ldsm_t(uint32_t a) {
  uint4 x;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(a)
               : "memory");
  return x;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void part_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// A unit of the tick space.  Segments: the groups' shared tokens, then the requests' own.
struct Unit {
  int seg, h, rt;        // segment, kv head, 64-row tile
  int row_tiles, ticks;  // of the segment; of the unit, without its end's
  int first, last;       // keys [first, last) of the table row that count
  int rows, r0;          // query rows of the segment; its first request
  int u0;                // the unit's first tick
  __device__ int tiles() const { return (ticks + 3) >> 2; }
  __device__ int row0() const { return rt * kDecRows; }
};

// CLUSTER: a cluster of CTAs takes one unit (grid: cluster, units) and joins it by itself.
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kDecThreads, 1) decode_attention_kernel(const __grid_constant__ DecodeArgs args) {
  using L = DecSmem<D>;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int NT = D / 8, kTile = L::kTile;
  static_assert(kTile == 4 * kDecTickKeys128 * 128 / D, "four ticks a tile");
  const DecodeParams& a = args.p;
  extern __shared__ __align__(128) unsigned char smem[];
  const int ng = a.num_groups, G = a.Hq / a.Hkv;
  int* pre = reinterpret_cast<int*>(smem + L::kScan);
  int* slen = pre + ng + a.b + 1;
  int* sbase = slen + a.b;
  int* sgroup = reinterpret_cast<int*>(smem);  // (the ring is not in use yet)
  int* sshared = sgroup + ng + 1;
  __shared__ int wsum[kDecThreads / 32];
  __shared__ int s_bad, s_tall;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const uint32_t full = smem_u32(smem + L::kBars), empty = full + 8 * kRing, owned = empty + 8 * kRing;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(full + 8 * i, kProducers * 33);
      mbar_init(empty + 8 * i, kConsumers);
    }
    for (int i = 0; i < kOwners * kRing; ++i) mbar_init(owned + 8 * i, kProducers * 33);
    *abort_flag = 0;
    s_bad = s_tall = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // (behind the tcgen05 kernel, which waits for what came before the call, this one starts where CTAs end: it reads
  // nothing of that kernel's, and waits for it at its own end)
  if (!args.tall) pdl_wait();
  pdl_trigger();

  // ---- segments ----
  const bool report = blockIdx.x == 0;
  Unit unit{};  // CLUSTER: the unit, and its tiles [S, E) of this CTA
  int S = 0, E = 0;
  const long long room = (long long)a.row_pages << args.shift;
  const int most = room < a.max_seq_len ? int(room) : a.max_seq_len;
  auto unit_ticks = [](int first, int last) { return dec_unit_ticks<D>(first, last); };
  if (CLUSTER) {
    const int r = blockIdx.y / a.Hkv;
    int len = a.seq_lens[r];
    const int row = a.req_pool_idx[r];
    unit.h = blockIdx.y - r * a.Hkv;
    const bool tell = report && unit.h == 0 && tid == 0;
    if (len < 0 || len > most) {
      if (tell) raise_error(a.error, SPEC_DEV_LENGTH);
      len = len < 0 ? 0 : most;
    }
    if (row < 0 || row >= a.req_rows) {
      if (tell) raise_error(a.error, SPEC_DEV_INDEX);
      len = 0;
    }
    unit.r0 = r;
    unit.rows = G;
    unit.row_tiles = 1;
    unit.last = len;
    const int tiles = (len + kTile - 1) / kTile;
    S = int((long long)blockIdx.x * tiles / gridDim.x);
    E = int((blockIdx.x + 1ll) * tiles / gridDim.x);
    __syncthreads();  // (the barriers)
  } else {
    for (int g = tid; g <= ng && ng > 0; g += kDecThreads) {
      sgroup[g] = a.group_start[g];
      if (g < ng) sshared[g] = a.shared_lens[g];
    }
    for (int r = tid; r < a.b; r += kDecThreads) {
      int len = a.seq_lens[r];
      const int row = a.req_pool_idx[r];
      if (len < 0 || len > most) {
        if (report) raise_error(a.error, SPEC_DEV_LENGTH);
        len = len < 0 ? 0 : most;
      }
      if (row < 0 || row >= a.req_rows) {
        if (report) raise_error(a.error, SPEC_DEV_INDEX);
        len = 0;
      }
      slen[r] = len;
    }
    __syncthreads();
    // groups that overlap or lie outside the batch: nothing is shared
    for (int g = tid; g < ng; g += kDecThreads)
      if (sgroup[g] < 0 || sgroup[g] > sgroup[g + 1] || sgroup[g + 1] > a.b) s_bad = 1;
    __syncthreads();
    const bool grouped = ng > 0 && !s_bad;
    if (report && tid == 0 && ng > 0 && s_bad) raise_error(a.error, SPEC_DEV_INDEX);
    for (int r = tid; r < a.b; r += kDecThreads) {
      int base = 0, g = -1;
      if (grouped && r >= sgroup[0] && r < sgroup[ng]) {
        int lo = 0, hi = ng;  // the last group that begins at or before r (empty ones are passed over)
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (sgroup[mid] <= r) lo = mid;
          else hi = mid;
        }
        g = lo;
        const int shared = sshared[g];
        if (report && r == sgroup[g] && (shared < 0 || shared > most)) raise_error(a.error, SPEC_DEV_LENGTH);
        const int s = dec_shared(shared, slen[sgroup[g]]);
        if (slen[r] >= s) base = s;
      }
      sbase[r] = base;
      if (report) {
        args.member[r] = g < 0 ? make_int4(-1, r, 1, 0) : make_int4(g, sgroup[g], sgroup[g + 1] - sgroup[g], base);
      }
    }
    __syncthreads();
    // the tcgen05 kernel's ticks
    int tall = 0;
    if (args.tall && grouped)
      for (int g = tid; g < ng; g += kDecThreads) {
        const int first = sgroup[g], rows = (sgroup[g + 1] - first) * G;
        if (rows > args.flat_rows && sbase[first] > 0)
          tall += a.Hkv * ((rows + kDecTallRows - 1) / kDecTallRows) * ((sbase[first] + kDecTile - 1) / kDecTile + kDecTallEnd);
      }
    tall = __reduce_add_sync(FULL, tall);
    if (args.tall && lane == 0 && tall) atomicAdd(&s_tall, tall);
    auto ticks_of = [&](int s) {
      if (s < ng) {
        const int first = grouped ? sgroup[s] : 0, rows = grouped ? (sgroup[s + 1] - first) * G : 0;
        const bool here = rows > 0 && sbase[first] > 0 && !(args.tall && rows > args.flat_rows);  // (else it is the tcgen05 kernel's)
        return here ? a.Hkv * ((rows + kDecRows - 1) / kDecRows) * (unit_ticks(0, sbase[first]) + kEndTicks) : 0;
      }
      return a.Hkv * args.own_tiles * (unit_ticks(sbase[s - ng], slen[s - ng]) + kEndTicks);
    };
    {
      const int segs = ng + a.b;
      int run = 0;
      for (int s0 = 0; s0 < segs; s0 += kDecThreads) {
        const int s = s0 + tid, t = s < segs ? ticks_of(s) : 0;
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
        for (int q = 0; q < kDecThreads / 32; ++q) {
          if (q < w) before += wsum[q];
          run += wsum[q];
        }
        if (s < segs) pre[s] = before + incl - t;
      }
      if (tid == 0) pre[segs] = run;
      __syncthreads();
      if (report)
        for (int s = tid; s <= segs; s += kDecThreads) args.pre[s] = pre[s];
    }
    const int T = pre[ng + a.b];  // (the host keeps it below 2^31)
    // (at least four ticks a CTA: each on a unit has one of its tiles)
    const int ctas = max(1, min(T >> 2, int(gridDim.x) - dec_tall_ctas(s_tall, T, a.b * a.Hkv * args.own_tiles, gridDim.x)));
    if (report && tid == 0) *args.plan = make_int4(T, ctas, ng, 0);
    if (int(blockIdx.x) >= ctas) {
      if (args.tall) pdl_wait();
      return;
    }
    S = int((long long)blockIdx.x * T / ctas);
    E = int((long long)(blockIdx.x + 1) * T / ctas);
  }

  auto open = [&](Unit& u, int seg) {  // the first unit of the first segment from `seg` on that has ticks
    while (seg < ng && pre[seg + 1] == pre[seg]) ++seg;
    u.seg = seg;
    u.h = u.rt = 0;
    if (seg < ng) {
      u.r0 = __ldg(a.group_start + seg);
      u.rows = (__ldg(a.group_start + seg + 1) - u.r0) * G;
      u.first = 0;
      u.last = sbase[u.r0];
      u.row_tiles = (u.rows + kDecRows - 1) / kDecRows;
    } else {
      u.r0 = seg - ng;
      u.rows = G;
      u.first = sbase[u.r0];
      u.last = slen[u.r0];
      u.row_tiles = args.own_tiles;
    }
    u.ticks = unit_ticks(u.first, u.last);
  };
  // the range's first unit, and the first of its tiles that is the CTA's
  auto locate = [&](Unit& u, int& t) {
    if (CLUSTER) {
      u = unit;
      t = S;
      return;
    }
    int lo = 0, hi = ng + a.b;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= S) lo = mid;
      else hi = mid;
    }
    open(u, lo);
    const int n = u.ticks + kEndTicks, j = (S - pre[u.seg]) / n;
    u.h = j / u.row_tiles;
    u.rt = j - u.h * u.row_tiles;
    u.u0 = pre[u.seg] + j * n;
    t = (S - u.u0 + 3) >> 2;
  };
  // the next unit; false behind the range
  auto next_unit = [&](Unit& u) {
    if (CLUSTER) return false;
    u.u0 += u.ticks + kEndTicks;
    if (u.u0 >= E) return false;
    if (++u.rt == u.row_tiles) {
      u.rt = 0;
      if (++u.h == a.Hkv) open(u, u.seg + 1);
    }
    return true;
  };
  // tiles of the unit in the range, from tile t on
  auto tiles_from = [&](const Unit& u, int t) { return CLUSTER ? E - t : min(u.tiles(), (E - u.u0 + 3) >> 2) - t; };
  // Who takes a part of n tiles of a unit: a warp (0 .. 7), four (8, 9), or all (-1).  parts: how many of either kind
  // came before in the range.
  auto owner_of = [&](const Unit& u, int n, int2& parts) {
    if (u.rows - u.row0() > 16) return -1;
    if (CLUSTER) return kConsumers;
    if (n <= kSoloTiles && E - S > kSoloRange * 4 * n) return parts.x++ % kConsumers;
    return kConsumers + (parts.y++ & 1);
  };
  // CLUSTER: the CTA's results lie where the ring was, O as [row][D], then each row's (m, l); the cluster's CTAs each join
  // a share of the words.
  auto join_cluster = [&] {
    cluster_sync();
    const int size = gridDim.x, words = G * (D / 4), w1 = int((blockIdx.x + 1ll) * words / size);
    for (int x = int((long long)blockIdx.x * words / size) + tid; x < w1; x += kDecThreads) {
      const int row = x / (D / 4), c = x - row * (D / 4);
      float2 ml[kClusterMost];
      float4 y[kClusterMost];
      float M = -INFINITY, Ls = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kClusterMost; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        if (q < size) {
          ml[q] = cluster_ld2(cluster_addr(smem + L::kStage + row * 8, q));
          y[q] = cluster_ld4(cluster_addr(smem + x * 16, q));
        }
      }
#pragma unroll
      for (int q = 0; q < kClusterMost; ++q) M = fmaxf(M, ml[q].x);
#pragma unroll
      for (int q = 0; q < kClusterMost; ++q) {
        if (q >= size) break;
        const float wt = dec_weight(ml[q].x, M);
        Ls = fmaf(ml[q].y, wt, Ls);
        acc = make_float4(fmaf(y[q].x, wt, acc.x), fmaf(y[q].y, wt, acc.y), fmaf(y[q].z, wt, acc.z), fmaf(y[q].w, wt, acc.w));
      }
      const float inv = dec_inverse(Ls);
      const size_t orow = size_t(unit.r0) * a.Hq + unit.h * G + row;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * c) =
          make_uint2(dec_pack(acc.x * inv, acc.y * inv), dec_pack(acc.z * inv, acc.w * inv));
      if (c == 0 && a.lse) a.lse[orow] = dec_lse(M, Ls);
    }
    cluster_sync();  // (no CTA ends while another reads its shared memory)
  };
  __syncthreads();  // (sgroup is not read any more)

  if (w >= kConsumers) {
    // ------------------------------------------------------------ producers
    const int p = w - kConsumers;
    constexpr int kChunks = D / 8;              // 16-byte chunks of a row
    constexpr int kKeys = 32 / kChunks;         // rows that a warp's copy spans
    constexpr int kMine = kTile / kProducers;   // keys of a tile that the warp copies
    const int cx = lane % kChunks, ck = lane / kChunks;
    const uint32_t slot_bytes = uint32_t(a.Hkv) * L::kRow;
    const unsigned char* const k0 = static_cast<const unsigned char*>(a.k_pool) + cx * 16;
    const long long to_v = static_cast<const unsigned char*>(a.v_pool) - static_cast<const unsigned char*>(a.k_pool);
    const uint32_t ring0 = smem_u32(smem) + (kMine * p + ck) * L::kRow;
    const uint32_t kdst = (cx ^ (4 * (ck & 1))) * 16, page_mask = (1u << args.shift) - 1u;
    Unit u;
    int t, n;
    locate(u, t);
    n = tiles_from(u, t);
    // What look() found: of each of two tiles the kv head (-1: none is left), the owner (-1: all warps), and the lane's key's
    // position (-1: none that counts) and page id.
    int x_pos[2] = {-1, -1}, x_id[2] = {-1, -1}, owner = -1, h_now = 0, x_now = 0, heads[2], owners[2];
    int2 parts = make_int2(0, 0);
    const int* row_now = nullptr;
    bool entered = false, more = true;
    auto look = [&](int half) {
      heads[half] = -1;
      while (n <= 0) {  // over a unit's end
        more = more && next_unit(u);
        if (!more) return;
        t = 0;
        n = tiles_from(u, 0);
        entered = false;
      }
      if (!entered) {
        entered = true;
        owner = owner_of(u, n, parts);
        h_now = u.h;
        row_now = a.page_table + (long long)__ldg(a.req_pool_idx + u.r0) * a.row_pages;
        x_now = (u.first / kTile + t) * kTile + kMine * p + lane;
      }
      heads[half] = h_now;
      owners[half] = owner;
      x_pos[half] = -1;
      if (lane < kMine && x_now >= u.first && x_now < u.last) {
        x_pos[half] = x_now;
        x_id[half] = __ldg(row_now + (x_now >> args.shift));
      }
      x_now += kTile;
      --n;
    };
    int stage = 0;
    uint32_t phase = 1;  // (an empty ring)
    bool dead = false;
    heads[1] = -1;
    look(0);
    if (heads[0] >= 0) look(1);
    while (heads[0] >= 0 && !dead) {
      const int h1 = heads[1];
      int slots[2];
      unsigned valids[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        slots[half] = 0;
        bool counts = x_pos[half] >= 0;
        if (counts) {
          if (uint32_t(x_id[half]) >= uint32_t(a.num_pages)) {
            raise_error(a.error, SPEC_DEV_INDEX);
            counts = false;
          } else {
            slots[half] = (x_id[half] << args.shift) + int(uint32_t(x_pos[half]) & page_mask);
          }
        }
        valids[half] = __ballot_sync(FULL, counts);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int h = half ? h1 : heads[0], who = owners[half], slot = slots[half];
        const unsigned valid = valids[half];
        if (h < 0 || dead) break;
        if (__any_sync(FULL, !mbar_wait(empty + 8 * stage, phase, abort_flag))) {
          dead = true;
          break;
        }
        const uint32_t st = ring0 + stage * L::kStage;
        const unsigned char* const from = k0 + uint32_t(h) * uint32_t(L::kRow);
        const unsigned mine = valid >> ck;
#pragma unroll
        for (int i = 0; i < kMine / kKeys; ++i) {
          const unsigned char* src = from + (unsigned long long)uint32_t(__shfl_sync(FULL, slot, i * kKeys + ck)) * slot_bytes;
          const uint32_t n = (mine >> (i * kKeys) & 1u) * 16u;  // (a key that does not count reads as zeros)
          const uint32_t to = st + i * kKeys * L::kRow;
          cp16(to + kdst, src, n);
          cp16(to + L::kHalf + (cx ^ ((i * kKeys + ck) & 7)) * 16, src + to_v, n);
        }
        const uint32_t tell = who < 0 ? full + 8 * stage : owned + 8 * (who * kRing + stage);
        if (lane == 0) {
          reinterpret_cast<volatile uint32_t*>(smem + L::kMask)[stage * 4 + p] = valid;
          mbar_arrive(tell);
        }
        mbar_arrive_copies(tell);
        if (++stage == kRing) {
          stage = 0;
          phase ^= 1;
        }
        if (half == 0) look(0);
      }
      const bool had = h1 >= 0 && heads[0] >= 0 && !dead;
      heads[1] = -1;
      if (had) look(1);
    }
    if (dead && lane == 0) {
      raise_error(a.error, SPEC_DEV_TIMEOUT);
      *abort_flag = 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (CLUSTER) join_cluster();
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const float xf = a.scale * 1.4426950408889634f;
  int stage = 0;
  int2 parts = make_int2(0, 0);
  uint32_t full_bits = 0, solo_bits = 0, four_bits = 0;  // parity of the next phase of each stage's barriers
  bool dead = false;
  float4* const merge = reinterpret_cast<float4*>(smem + L::kMerge);
  float2* const mls = reinterpret_cast<float2*>(smem + L::kMl);
  uint32_t qf[D / 16][4];
  float o[NT][4], m[2], l[2];
  auto wait_tile = [&](uint32_t bar, uint32_t parity) {
    if (!dead && __any_sync(FULL, !mbar_wait(bar, parity, abort_flag))) {
      dead = true;
      if (lane == 0) {
        raise_error(a.error, SPEC_DEV_TIMEOUT);
        *abort_flag = 1;
      }
    }
  };
  auto next_stage = [&] { stage = stage + 1 == kRing ? 0 : stage + 1; };
  // 16 query rows of the unit, from row x0 of the segment on, and empty results
  auto begin = [&](const Unit& u, int h, int x0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = x0 + g + 8 * i;
      const bool on = x < u.rows;
      const int f = on ? x / G : 0;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (size_t(u.r0) + f) * a.q_ld +
                                                        size_t(h * G + (on ? x - f * G : 0)) * D);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint4 y = on ? __ldg(src + 4 * k + c) : make_uint4(0, 0, 0, 0);
        qf[2 * k][i] = y.x;
        qf[2 * k][2 + i] = y.y;
        qf[2 * k + 1][i] = y.z;
        qf[2 * k + 1][2 + i] = y.w;
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[q][i] = 0.f;
  };
  // Keys [16 NB part, 16 NB (part + 1)) of the tile in `stage`.
  constexpr int NB = kTile / 64;
  auto block = [&](int part) {
    const uint32_t st = smem_u32(smem + stage * L::kStage);
    constexpr uint32_t kAll = NB == 2 ? 0xffffffffu : 0xffffu;
    const uint32_t mask = reinterpret_cast<volatile uint32_t*>(smem + L::kMask)[stage * 4 + part];
    if (mask == 0) return;
    float s[2 * NB][4];
#pragma unroll
    for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[q][e] = 0.f;
    const uint32_t krow = st + (16 * NB * part + g) * L::kRow;
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
#pragma unroll
      for (int q = 0; q < 2 * NB; ++q) {
        const uint4 y = lds16(krow + 8 * q * L::kRow + ((4 * k + c) ^ (4 * (g & 1))) * 16);
        mma_bf16(s[q], qf[2 * k], y.x, y.y);
        mma_bf16(s[q], qf[2 * k + 1], y.z, y.w);
      }
    auto masked = [&](float (&v)[2 * NB][4]) {
      if (mask != kAll) {
#pragma unroll
        for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(mask >> (8 * q + 2 * c + (e & 1)) & 1)) v[q][e] = -INFINITY;
      }
    };
    // y = x - m; a row without a reference has y = inf (NaN where x is -inf)
    float y[2 * NB][4], top = -INFINITY;
#pragma unroll
    for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[q][e] = fmaf(s[q][e], xf, -m[e >> 1]);
    masked(y);
#pragma unroll
    for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, y[q][e]);
    if (__any_sync(FULL, top > kDecBase + kDecLazy || m[0] == -INFINITY || m[1] == -INFINITY)) {
#pragma unroll
      for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[q][e] *= xf;
      masked(s);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2 * NB; ++q) mx = fmaxf(mx, fmaxf(s[q][2 * r], s[q][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        const float ref = mx - kDecBase;
        if (ref > m[r] + kDecLazy || m[r] == -INFINITY) {
          const float fac = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - ref);
          l[r] *= fac;
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            o[q][2 * r] *= fac;
            o[q][2 * r + 1] *= fac;
          }
          m[r] = ref;
        }
      }
#pragma unroll
      for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[q][e] = s[q][e] - (m[e >> 1] == -INFINITY ? 0.f : m[e >> 1]);
    }
    uint32_t pa[NB][4];
#pragma unroll
    for (int q = 0; q < 2 * NB; ++q)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = fast_exp2(y[q][2 * r]), p1 = fast_exp2(y[q][2 * r + 1]);
        l[r] += p0 + p1;
        pa[q >> 1][2 * (q & 1) + r] = dec_pack(p0, p1);
      }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int vkey = 16 * (NB * part + b) + (lane & 15);
      const uint32_t vrow = st + L::kHalf + vkey * L::kRow;
#pragma unroll
      for (int q = 0; q < NT / 2; ++q) {
        const uint4 v = ldsm_t(vrow + (((2 * q + (lane >> 4)) ^ (vkey & 7)) * 16));
        mma_bf16(o[2 * q], pa[b], v.x, v.y);
        mma_bf16(o[2 * q + 1], pa[b], v.z, v.w);
      }
    }
  };
  auto sum_l = [&] {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(FULL, l[r], 1);
      l[r] += __shfl_xor_sync(FULL, l[r], 2);
    }
  };
  // Two columns of a row's result (unnormalised, relative to M): out, or a partial result.
  auto put = [&](const Unit& u, int row, int col, bool whole, bool begun, float M, float Ls, float s0, float s1, bool note) {
    const int h = u.h, row0 = u.row0();
    if (CLUSTER) {
      *reinterpret_cast<float2*>(smem + (row * D + col) * 4) = make_float2(s0, s1);
      if (note) *reinterpret_cast<float2*>(smem + L::kStage + row * 8) = make_float2(M, Ls);
      return;
    }
    const bool own = u.seg >= ng;
    const int f = row / G;
    const size_t orow = (size_t(u.r0) + f) * a.Hq + h * G + (row - f * G);
    if (own && whole && u.first == 0) {
      const float inv = dec_inverse(Ls);
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + orow * D + col) = dec_pack(s0 * inv, s1 * inv);
      if (note && a.lse) a.lse[orow] = dec_lse(M, Ls);
    } else {
      const size_t first = whole ? size_t(u.r0) * a.Hq + size_t(h) * u.rows + row0 : size_t(2 * blockIdx.x + (begun ? 1 : 0)) * kDecRows;
      const int step = whole ? min(kDecRows, u.rows - row0) : kDecRows;
      float* fo = reinterpret_cast<float*>((whole ? (own ? args.own_o : args.shared_o) : args.frag_o) + first * (D / 4));
      *reinterpret_cast<float2*>(fo + 4 * ((col >> 2) * step + row - row0) + (col & 3)) = make_float2(s0, s1);
      if (note) (whole ? (own ? args.own_ml : args.shared_ml) : args.frag_ml)[first + row - row0] = make_float2(M, Ls);
    }
  };

  // A unit's part in the range, n tiles, by `who`: all warps (RT 2 or 4 row tiles of 16), or four of them (RT 1).
  auto work = [&](auto rt_const, const Unit& u, int t0, int n, int who) {
    constexpr int RT = decltype(rt_const)::value;
    constexpr int KS = RT == 1 ? 4 : kConsumers / RT;  // warps that hold a row tile
    constexpr int kThreads = 32 * RT * KS;
    const int rt = w % RT, share = RT == 1 ? w & 3 : w / RT, w0 = RT == 1 ? w & 4 : 0, id = RT == 1 ? 2 + (w >> 2) : 1;
    const int h = u.h, row0 = u.row0();
    uint32_t& bits = RT == 1 ? four_bits : full_bits;
    begin(u, h, row0 + rt * 16);
    for (int i = 0; i < n; ++i) {
      wait_tile(RT == 1 ? owned + 8 * (who * kRing + stage) : full + 8 * stage, bits >> stage & 1u);
      bits ^= 1u << stage;
      if (!dead) {
        if (RT == 4) {
          block(2 * share);
          block(2 * share + 1);
        } else {
          block(share);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * stage, kConsumers / (RT * KS));
      next_stage();
    }

    // ---- the warps' results joined ----
    sum_l();
    if (c == 0) {
      mls[w * 16 + g] = make_float2(m[0], l[0]);
      mls[w * 16 + g + 8] = make_float2(m[1], l[1]);
    }
    const bool begun = t0 == 0, whole = begun && n == u.tiles();
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        merge[(w * 8 + q) * 32 + lane] = make_float4(o[8 * half + q][0], o[8 * half + q][1], o[8 * half + q][2], o[8 * half + q][3]);
      part_sync(id, kThreads);
      for (int x = tid - 32 * w0; x < RT * 256; x += kThreads) {
        const int tile = x >> 8, q = (x >> 5) & 7, ln = x & 31, gg = ln >> 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = row0 + tile * 16 + gg + 8 * r;  // of the segment
          if (row >= u.rows) continue;
          float M = -INFINITY, Ls = 0.f, s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) M = fmaxf(M, mls[(w0 + RT * k + tile) * 16 + gg + 8 * r].x);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int ww = w0 + RT * k + tile;
            const float2 ml = mls[ww * 16 + gg + 8 * r];
            const float wt = dec_weight(ml.x, M);
            const float2 v = reinterpret_cast<const float2*>(merge + (ww * 8 + q) * 32 + ln)[r];
            Ls = fmaf(wt, ml.y, Ls);
            s0 = fmaf(wt, v.x, s0);
            s1 = fmaf(wt, v.y, s1);
          }
          put(u, row, 64 * half + 8 * q + 2 * (ln & 3), whole, begun, M, Ls, s0, s1, half == 0 && q == 0 && (ln & 3) == 0);
        }
      }
      part_sync(id, kThreads);
    }
  };
  // The same by one warp.
  auto work_alone = [&](const Unit& u, int t0, int n) {
    const int h = u.h, row0 = u.row0();
    begin(u, h, row0);
    for (int i = 0; i < n; ++i) {
      wait_tile(owned + 8 * (w * kRing + stage), solo_bits >> stage & 1u);
      solo_bits ^= 1u << stage;
      if (!dead) {
#pragma unroll 1
        for (int part = 0; part < 4; ++part) block(part);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * stage, kConsumers);
      next_stage();
    }
    sum_l();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (row >= u.rows) continue;
#pragma unroll
      for (int q = 0; q < NT; ++q)
        put(u, row, 8 * q + 2 * c, t0 == 0 && n == u.tiles(), t0 == 0, m[r], l[r], o[q][2 * r], o[q][2 * r + 1], q == 0 && c == 0);
    }
  };

  Unit u;
  int t;
  locate(u, t);
  do {
    const int n = tiles_from(u, t);
    if (n > 0 || CLUSTER) {  // (a CTA of a cluster without a tile leaves an empty result)
      const int who = owner_of(u, n, parts);
      if (who < 0) {
        if (u.rows - u.row0() <= 32) work(std::integral_constant<int, 2>{}, u, t, n, who);
        else work(std::integral_constant<int, 4>{}, u, t, n, who);
      } else if (who == w) {
        work_alone(u, t, n);
      } else if (who == kConsumers + (w >> 2)) {
        work(std::integral_constant<int, 1>{}, u, t, n, who);
      } else {
        stage = (stage + n) % kRing;
      }
    }
    t = 0;
  } while (next_unit(u));
  if (CLUSTER) join_cluster();
  else if (args.tall) pdl_wait();
}

// Joins the partial results: a thread a word of four columns of a row.  The rows of a group come in the order of its units,
// (kv head, member, q head), so that the words of neighbouring threads lie side by side.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeArgs args) {
  pdl_wait();
  pdl_trigger();
  const DecodeParams& a = args.p;
  constexpr int kRows = kJoinThreads / (D / 4);  // rows of a block
  const int c = threadIdx.x / kRows, at = blockIdx.x * kRows + threadIdx.x % kRows, total = a.b * a.Hq, G = a.Hq / a.Hkv;
  if (at >= total) return;
  const int4 plan = __ldcg(args.plan), tall_plan = args.tall ? __ldcg(args.tall_plan) : make_int4(0, 0, 0, 0);
  int r = at / a.Hq, head = at - r * a.Hq;
  const int4 mem = __ldcg(args.member + r);
  const int r0 = mem.y, all = mem.z * G;  // (all: the rows of a kv head)
  int base = mem.w;
  if (mem.x >= 0) {
    const int rem = at - r0 * a.Hq, hh = rem / all, x = rem - hh * all, f = x / G;
    r = r0 + f;
    head = hh * G + x - f * G;
    base = __ldcg(args.member + r).w;
  }
  const int h = head / G, i = head - h * G, x = (r - r0) * G + i;
  const size_t orow = size_t(r) * a.Hq + head;
  // The CTAs on a unit, the j-th of a segment of so many: [wa, wb].
  struct Span {
    int wa, wb;
  };
  auto span = [&](const int4& pl, const int* pre, int seg, int units, int j, int end, int tile) {  // tile: its ticks
    const int p0 = __ldcg(pre + seg), n = (__ldcg(pre + seg + 1) - p0) / units, u0 = p0 + j * n, last = u0 + (n - end - 1) / tile * tile;
    const long long T = pl.x, ctas = pl.y;
    return Span{int(((long long)(u0 + 1) * ctas - 1) / T), int(((long long)(last + 1) * ctas - 1) / T)};
  };
  const int own0 = i / kDecRows * kDecRows;
  const Span own = span(plan, args.pre, plan.z + r, a.Hkv * args.own_tiles, h * args.own_tiles + i / kDecRows, kEndTicks, 4);
  const bool done = own.wa == own.wb && base == 0;  // (already in out)
  if (done) return;
  const int n_own = own.wb - own.wa + 1;
  int n_sh = 0;
  // what the request shares: the first kernel's partial results, or the tcgen05 kernel's
  Span sh{0, 0};
  const bool tall = args.tall && all > args.flat_rows;
  const int size = tall ? kDecTallRows : kDecRows, x0 = x / size * size, rows = min(size, all - x0), xr = x - x0;
  const bool split = tall && rows <= 128;
  if (base > 0) {
    const int tiles = (all + size - 1) / size;
    sh = span(tall ? tall_plan : plan, tall ? args.tall_pre : args.pre, mem.x, a.Hkv * tiles, h * tiles + x / size, tall ? kDecTallEnd : kEndTicks, tall ? 1 : 4);
    n_sh = (sh.wb - sh.wa + 1) * (split ? 2 : 1);
  }
  const size_t sh_first = size_t(r0) * a.Hq + size_t(h) * all + x0;
  // part q: its (m, l), its first word, and how far its words lie apart
  struct Part {
    const float2* ml;
    const float4* o;
    int step;
  };
  auto part = [&](int q) {
    if (q < n_own) {
      const bool cut = own.wa != own.wb;
      const size_t first = cut ? size_t(2 * (own.wa + q) + (q == 0 ? 1 : 0)) * kDecRows : size_t(r) * a.Hq + h * G + own0;
      return Part{(cut ? args.frag_ml : args.own_ml) + first + i - own0, (cut ? args.frag_o : args.own_o) + first * (D / 4) + i - own0,
                  cut ? kDecRows : min(kDecRows, G - own0)};
    }
    q -= n_own;
    const bool cut = sh.wa != sh.wb;
    if (!tall) {
      const size_t first = cut ? size_t(2 * (sh.wa + q) + (q == 0 ? 1 : 0)) * kDecRows : sh_first;
      return Part{(cut ? args.frag_ml : args.shared_ml) + first + xr, (cut ? args.frag_o : args.shared_o) + first * (D / 4) + xr, cut ? kDecRows : rows};
    }
    const int cta = sh.wa + (split ? q >> 1 : q), half = split ? q & 1 : xr >> 7;
    const size_t first = cut ? ((size_t(2) * cta + (cta == sh.wa ? 1 : 0)) * 2 + half) * 128 : (split ? size_t(half) * total : 0) + sh_first;
    const int row = cut ? xr & 127 : xr;
    return Part{(cut ? args.tall_ml : args.whole_ml) + first + row, (cut ? args.tall_o : args.whole_o) + first * (D / 4) + row, cut ? 128 : rows};
  };
  const int np = n_own + n_sh;
  float M = -INFINITY, Ls = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kOnce = 8;
#pragma unroll 1
  for (int q0 = 0; q0 < np; q0 += kOnce) {
    float2 v[kOnce];
    float4 y[kOnce];
#pragma unroll
    for (int k = 0; k < kOnce; ++k) {
      v[k] = make_float2(-INFINITY, kDecNone);
      if (q0 + k < np) {
        const Part p = part(q0 + k);
        v[k] = __ldcg(p.ml);
        y[k] = __ldcg(p.o + size_t(c) * p.step);
      }
    }
    float M2 = M;
#pragma unroll
    for (int k = 0; k < kOnce; ++k) M2 = fmaxf(M2, v[k].x);
    const float was = dec_weight(M, M2);
    M = M2;
    Ls *= was;
    acc = make_float4(acc.x * was, acc.y * was, acc.z * was, acc.w * was);
#pragma unroll
    for (int k = 0; k < kOnce; ++k) {
      if (v[k].y < 0.f) continue;
      const float wt = dec_weight(v[k].x, M);
      Ls = fmaf(v[k].y, wt, Ls);
      acc = make_float4(fmaf(y[k].x, wt, acc.x), fmaf(y[k].y, wt, acc.y), fmaf(y[k].z, wt, acc.z), fmaf(y[k].w, wt, acc.w));
    }
  }
  const float inv = dec_inverse(Ls);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * c) =
      make_uint2(dec_pack(acc.x * inv, acc.y * inv), dec_pack(acc.z * inv, acc.w * inv));
  if (c == 0 && a.lse) a.lse[orow] = dec_lse(M, Ls);
}

template <int D>
int launch_decode(const DecodeArgs& args, int sms, cudaStream_t stream) {
  const DecodeParams& p = args.p;
  if (p.num_groups == 0 && args.own_tiles == 1) {
    const long long units = (long long)p.b * p.Hkv;
    const int size = cluster_of(units, sms);
    constexpr int tile = DecSmem<D>::kTile, smem = DecSmem<D>::kScan;
    if ((long long)size * kClusterTiles * tile >= p.max_seq_len && size > 0) {
      if (cudaFuncSetAttribute(decode_attention_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return SPEC_ERR_LAUNCH;
      return launch_cluster(decode_attention_kernel<D, true>, size, dim3(size, unsigned(units)), dim3(kDecThreads), smem, stream, args) == cudaSuccess
                 ? SPEC_OK
                 : SPEC_ERR_LAUNCH;
    }
  }
  const size_t smem = DecSmem<D>::bytes(p.b, p.num_groups);
  if (cudaFuncSetAttribute(decode_attention_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(DecSmem<D>::bytes(kDecodeMaxB, kDecodeMaxB))) != cudaSuccess)  // (the most, so that calls of two threads agree)
    return SPEC_ERR_LAUNCH;
  const int grid = sms < kDecMaxCtas ? sms : kDecMaxCtas;
  if (args.tall)
    if (const int rc = launch_decode_tall(args, sms, stream)) return rc;
  if (launch_pdl(decode_attention_kernel<D, false>, dim3(grid), dim3(kDecThreads), smem, stream, args) != cudaSuccess) return SPEC_ERR_LAUNCH;
  constexpr int rows = kJoinThreads / (D / 4);
  const unsigned blocks = unsigned((size_t(p.b) * p.Hq + rows - 1) / rows);
  return launch_pdl(decode_join_kernel<D>, dim3(blocks), dim3(kJoinThreads), 0, stream, args) == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

// Offsets of the workspace's parts.
struct DecodeLayout {
  size_t pre, member, frag_ml, own_ml, shared_ml, frag_o, own_o, shared_o, bytes;
  size_t tall_pre, tall_ml, whole_ml, tall_o, whole_o;
  DecodeLayout(int b, int Hq, int D, bool tall) {
    const size_t rows = size_t(b) * Hq, frags = size_t(2) * kDecMaxCtas * kDecRows, tall_frags = size_t(2) * kDecMaxCtas * kDecTallRows;
    size_t at = 256;
    auto take = [&](size_t n) {
      const size_t x = at;
      at += align256(n);
      return x;
    };
    pre = take(size_t(2 * b + 1) * 4);
    member = take(size_t(b) * 16);
    frag_ml = take(frags * 8);
    own_ml = take(rows * 8);
    shared_ml = take(rows * 8);
    frag_o = take(frags * D * 4);
    own_o = take(rows * D * 4);
    shared_o = take(rows * D * 4);
    tall_pre = tall_ml = whole_ml = tall_o = whole_o = at;
    if (tall) {
      tall_pre = take(size_t(b + 1) * 4);
      tall_ml = take(tall_frags * 8);
      whole_ml = take(2 * rows * 8);
      tall_o = take(tall_frags * D * 4);
      whole_o = take(2 * rows * D * 4);
    }
    bytes = at;
  }
};
// whether a group of the batch may have more rows than the register kernel takes
bool may_be_tall(int b, int Hq, int Hkv) { return (long long)b * (Hq / Hkv) > dec_flat_rows(128); }

}  // namespace

size_t decode_partial_bytes(int b, int Hq, int Hkv) { return DecodeLayout(b, Hq, 128, may_be_tall(b, Hq, Hkv)).bytes; }

int launch_decode_attention(const DecodeParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return SPEC_ERR_LAUNCH;
  // The groups are not known here, but their mean is: where it is far below what the tcgen05 kernel takes, its launch
  // (5 us) is left out, and a large group among small ones takes the other kernel's tiles of 64 rows.
  // (A scale of zero would take the -inf of a key that does not count to NaN there.)
  const bool tall = p.num_groups > 0 && may_be_tall(p.b, p.Hq, p.Hkv) && (long long)p.b * (p.Hq / p.Hkv) > dec_flat_rows(p.D) / 2 * (long long)p.num_groups &&
                    p.scale != 0.f;
  const DecodeLayout at(p.b, p.Hq, p.D, tall);
  unsigned char* ws = p.partials;
  DecodeArgs args{};
  args.p = p;
  for (args.shift = 0; (1 << args.shift) < p.page_size; ++args.shift) {
  }
  args.own_tiles = (p.Hq / p.Hkv + kDecRows - 1) / kDecRows;
  args.flat_rows = dec_flat_rows(p.D);
  args.plan = reinterpret_cast<int4*>(ws);
  args.pre = reinterpret_cast<int*>(ws + at.pre);
  args.member = reinterpret_cast<int4*>(ws + at.member);
  args.frag_ml = reinterpret_cast<float2*>(ws + at.frag_ml);
  args.own_ml = reinterpret_cast<float2*>(ws + at.own_ml);
  args.shared_ml = reinterpret_cast<float2*>(ws + at.shared_ml);
  args.frag_o = reinterpret_cast<float4*>(ws + at.frag_o);
  args.own_o = reinterpret_cast<float4*>(ws + at.own_o);
  args.shared_o = reinterpret_cast<float4*>(ws + at.shared_o);
  args.tall = tall;
  args.tall_plan = reinterpret_cast<int4*>(ws + 128);
  args.tall_pre = reinterpret_cast<int*>(ws + at.tall_pre);
  args.tall_ml = reinterpret_cast<float2*>(ws + at.tall_ml);
  args.tall_o = reinterpret_cast<float4*>(ws + at.tall_o);
  args.whole_ml = reinterpret_cast<float2*>(ws + at.whole_ml);
  args.whole_o = reinterpret_cast<float4*>(ws + at.whole_o);
  return p.D == 128 ? launch_decode<128>(args, sms, stream) : launch_decode<64>(args, sms, stream);
}

}  // namespace spec
