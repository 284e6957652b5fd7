// decode_attention_tc.cu -- the shared tokens of large groups in the one-token
// attention over shared pages, on the tcgen05 tensor cores (decode_attention.cu has the mathematics and takes
// everything else).
//
// A unit is (group, kv head, up to 256 query rows): row x is (member x / G, q head x % G of the kv head).  One CTA a
// SM takes an equal contiguous range of the 64-key tiles of all units laid end to end.  Warps:
//   0-3, 4-7  two softmax groups, one query row a thread.  More than 128 rows: group w has rows 128 w .. and both see
//             every tile; fewer: the groups take turns at the tiles (two partial results).
//   8-11      copy K and V rows with 16-byte cp.async into a ring of 128B-swizzled tiles
//   12, 13    issue S = Q K^T (M 128, N 64, K D) of groups 0, 1; 14, 15: O += P V (A = P from TMEM)
// TMEM: O0 O1 | two S buffers a group; P (bf16, two to a column) takes the place of its S, so that the scores of
// the next tile are computed, and the products of the last one added up, while a tile's softmax runs.
//   P is taken against a reference that moves only when a tile's sum of P passes 2^-32 (kDecBase, kDecLazy).
//   Every piece of a unit leaves an fp32 partial result; decode_attention.cu joins them.
//   Bound: up to 128 rows the cache's bytes (eight groups of 12 requests, 32768 shared tokens, 32 / 8 heads: 193 us a call,
// 1.1 GB); 256 rows: shared memory.  S with both operands there reads 6 KB in 32 cycles of the tensor cores, so that a tile
// is 1280 cycles of products and 256 of the copies' writes; it takes about 1790, and from memory it comes in 1340 (at the
// profiler's 1.8 GHz).  Two documents of 65536 tokens, 32 requests of 64 / 8 heads each: 132 us, 1.04 PF/s.  K and V in
// rings of their own, TMA boxes of 16 keys (what a page holds for certain; 30 GB/s a SM) and Q in TMEM, with one S a
// group, are slower by 8, 15 and 29%.
//   Every wait is bounded: on timeout the CTA sets SPEC_DEV_TIMEOUT, stops, drains its copies and MMAs and frees its TMEM.
#include "common.cuh"
#include "kernels.cuh"

#include "decode_attention.cuh"

namespace spec {

namespace {

constexpr int kRows = 128;
constexpr int kTallThreads = 16 * 32;
constexpr int kMostStages = 10;
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s: bound of every wait
constexpr float kSumMost = 2.3283064365386963e-10f;  // 2^(kDecBase + kDecLazy)
__host__ __device__ constexpr uint32_t col_o(int w) { return 128u * uint32_t(w); }
__host__ __device__ constexpr uint32_t col_s(int w, int b) { return 256u + 128u * uint32_t(w) + 64u * uint32_t(b); }

template <int D>
struct TallSmem {
  static constexpr int kStages = D == 128 ? 5 : 10;  // tiles in the ring
  static constexpr int kLag = D == 128 ? 2 : 5;      // tiles whose copies are in flight behind the one being issued
  static constexpr int kQBlock = kRows * 128;       // [128 rows x 64 bf16], 128B-swizzled
  static constexpr int kQTile = (D / 64) * kQBlock;
  static constexpr int kBlock = kDecTile * 128;     // [64 keys x 64 bf16]
  static constexpr int kHalf = (D / 64) * kBlock;   // K of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = 2 * kQTile;
  static constexpr int kBars = kRing + kStages * kStage;
  static constexpr int kNumBars = 2 * kMostStages + 2 + 2 + 4 + 4 + 4 + 4;
  static constexpr int kMask = kBars + 8 * kNumBars;   // [stage][4] keys that count, 16 bits each
  static constexpr int kWords = kMask + kStages * 16;  // TMEM address, abort flag, bad flag, the other kernel's ticks, then a word a warp
  static constexpr int kBytes = kWords + 16 + 4 * (kTallThreads / 32);
  // the ticks before each group are summed up where the ring will be
  static_assert(4 * (4 * kDecodeMaxB + 2) <= kStages * kStage, "scan space");
};
static_assert(TallSmem<128>::kBytes + 1024 <= 227 * 1024, "shared memory of one CTA");

enum {
  kFull0 = 0,              // + stage: the tile's copies have landed
  kEmpty0 = kMostStages,   // + stage: the products that read it are complete (one arrival a group)
  kQFull0 = 2 * kMostStages,  // + group
  kOFree0 = kQFull0 + 2,   // + group: the epilogue has read O
  kSFull0 = kOFree0 + 2,   // + 2 group + S buffer
  kPReady0 = kSFull0 + 4,
  kPvDone0 = kPReady0 + 4,
  kDrain0 = kPvDone0 + 4,  // + issuing warp
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// up to 128 tries without a time hint
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 128;\nAGAIN:\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n"
      " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra AGAIN;\nDONE:\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for the phase of the given parity: false once kWaitCycles have passed or another warp has given up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_poll(bar, parity)) return true;
  const long long start = clock64();
  do {
    if (mbar_poll(bar, parity)) return true;
  } while (!*abort_flag && clock64() - start <= kWaitCycles);
  return false;
}
// 16-byte global -> shared copy; 0 bytes: zeros
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor (128B swizzle, descriptor version 1) in two words: address and leading-dimension
// offset, then stride offset and flags.  The address is stepped in the low word alone.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
  return d;
}
// instruction descriptor of kind::f16: bf16 A and B, f32 accumulator, M = 128
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
}
// the lane of a converged warp that issues (always the same one)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

#define SPEC_R32(r)                                                                                                  \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),        \
      "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),         \
      "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),        \
      "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])

// 32 consecutive TMEM columns of this thread's lane (tmem_ld_wait completes the load)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SPEC_R32(r)
      : "r"(taddr)
      : "memory");
}
// 16 columns: the load is issued (tmem_ld_wait completes it)
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// columns stored (tmem_st_wait completes them)
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// 2^d of a whole number d <= 0; 0 below 2^-126 (as ex2 gives it: a larger factor would leave values of no weight standing)
__device__ __forceinline__ float pow2(float d) { return d >= -126.f ? __uint_as_float(uint32_t(127 + int(d)) << 23) : 0.f; }

// A place in the tick space: a group's shared tokens, (kv head, row block), tile.
struct Place {
  int g, j, t;
  int tiles, blocks, rows, r0, shared;  // of the group (tiles 0: it is none of this kernel's)
};

template <int D>
__global__ void __launch_bounds__(kTallThreads, 1) decode_attention_tc_kernel(const __grid_constant__ DecodeArgs args) {
  using L = TallSmem<D>;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int kStages = L::kStages, kLag = L::kLag;
  const DecodeParams& a = args.p;
  const int G = a.Hq / a.Hkv, ng = a.num_groups;
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;

  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  unsigned char* sp = smem_raw + (sbase - raw);
  auto bar = [&](int i) { return sbase + uint32_t(L::kBars) + 8u * uint32_t(i); };
  volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(sp + L::kMask);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sp + L::kWords);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + L::kWords + 4);
  volatile int* bad = reinterpret_cast<volatile int*>(sp + L::kWords + 8);
  int* s_flat = reinterpret_cast<int*>(sp + L::kWords + 12);
  int* wsum = reinterpret_cast<int*>(sp + L::kWords + 16);
  int* pre = reinterpret_cast<int*>(sp + L::kRing);  // [groups + 1] ticks before each group, until the roles start
  int* sgroup = pre + ng + 1;                        // [groups + 1]
  int* sshared = sgroup + ng + 1;                    // [groups]
  int* slen = sshared + ng;                          // [b]

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kFull0 + i), 4 * 32);
      mbar_init(bar(kEmpty0 + i), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kQFull0 + i), kRows);
      mbar_init(bar(kOFree0 + i), kRows);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kSFull0 + i), 1);
      mbar_init(bar(kPReady0 + i), kRows);
      mbar_init(bar(kPvDone0 + i), 1);
      mbar_init(bar(kDrain0 + i), 1);
    }
    *abort_flag = 0;
    *bad = 0;
    *s_flat = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_holder)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();  // nothing above reads global memory
  pdl_trigger();

  // ---- ticks before each group; this CTA's range ----
  const long long room = (long long)a.row_pages << args.shift;
  const int most = room < a.max_seq_len ? int(room) : a.max_seq_len;
  __syncthreads();
  for (int g = tid; g <= ng; g += kTallThreads) {
    const int s = a.group_start[g], e = g < ng ? a.group_start[g + 1] : a.b;
    if (g < ng && (s < 0 || s > e || e > a.b)) *bad = 1;
    sgroup[g] = s;
    if (g < ng) sshared[g] = a.shared_lens[g];
  }
  for (int r = tid; r < a.b; r += kTallThreads) {
    const int row = a.req_pool_idx[r], len = a.seq_lens[r];
    slen[r] = row < 0 || row >= a.req_rows ? 0 : min(max(len, 0), most);
  }
  __syncthreads();
  const bool grouped = *bad == 0;  // (the other kernel tells)
  auto fill = [&](Place& p, int r0, int members, int shared, auto&& len_of) {
    p.r0 = r0;
    p.rows = members * G;
    if (p.rows <= args.flat_rows) return;
    p.shared = dec_shared(shared, len_of(r0));
    p.blocks = (p.rows + kDecTallRows - 1) / kDecTallRows;
    p.tiles = (p.shared + kDecTile - 1) / kDecTile;
  };
  auto begin = [&](int g, Place& p) {
    p.g = g;
    p.j = p.t = p.tiles = 0;
    return grouped && g < ng;
  };
  // (all of it is read again where a role comes to the group)
  auto group = [&](int g, Place& p) {
    if (!begin(g, p)) return;
    const int r0 = __ldg(a.group_start + g);
    fill(p, r0, __ldg(a.group_start + g + 1) - r0, __ldg(a.shared_lens + g), [&](int r) {
      const int row = __ldg(a.req_pool_idx + r), len = __ldg(a.seq_lens + r);
      return row < 0 || row >= a.req_rows ? 0 : min(max(len, 0), most);
    });
  };
  auto known_group = [&](int g, Place& p) {  // from shared memory
    if (begin(g, p)) fill(p, sgroup[g], sgroup[g + 1] - sgroup[g], sshared[g], [&](int r) { return slen[r]; });
  };
  auto ticks_of = [&](const Place& p) { return p.tiles ? a.Hkv * p.blocks * (p.tiles + kDecTallEnd) : 0; };
  if (grouped) {  // the other kernel's ticks: each request's own tokens, and what smaller groups share
    const int own_tiles = args.own_tiles;
    int flat = 0;
    for (int r = tid; r < a.b; r += kTallThreads) {
      const int len = slen[r];
      int base = 0;
      if (r >= sgroup[0] && r < sgroup[ng]) {
        int lo = 0, hi = ng;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (sgroup[mid] <= r) lo = mid;
          else hi = mid;
        }
        const int first = sgroup[lo], rows = (sgroup[lo + 1] - first) * G, s = dec_shared(sshared[lo], slen[first]);
        base = len >= s ? s : 0;
        if (r == first && s > 0 && rows <= args.flat_rows) flat += a.Hkv * ((rows + kDecRows - 1) / kDecRows) * (dec_unit_ticks<D>(0, s) + kDecEndTicks);
      }
      flat += a.Hkv * own_tiles * (dec_unit_ticks<D>(base, len) + kDecEndTicks);
    }
    flat = __reduce_add_sync(FULL, flat);
    if (lane == 0) atomicAdd(s_flat, flat);
  }
  {
    int run = 0;
    for (int g0 = 0; g0 < ng; g0 += kTallThreads) {
      const int g = g0 + tid;
      Place p;
      known_group(g, p);
      const int t = ticks_of(p);
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += y;
      }
      __syncthreads();
      if (lane == 31) wsum[warp] = incl;
      __syncthreads();
      int before = run;
      for (int q = 0; q < kTallThreads / 32; ++q) {
        if (q < warp) before += wsum[q];
        run += wsum[q];
      }
      if (g < ng) pre[g] = before + incl - t;
    }
    if (tid == 0) pre[ng] = run;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_holder;
  const int T = pre[ng];
  const int ctas = min(T, dec_tall_ctas(T, *s_flat, a.b * a.Hkv * args.own_tiles, gridDim.x));
  const bool part = int(blockIdx.x) < ctas;
  const int S = part ? int((long long)blockIdx.x * T / ctas) : 0, E = part ? int((blockIdx.x + 1ll) * T / ctas) : 0;
  if (blockIdx.x == 0) {
    if (tid == 0) *args.tall_plan = make_int4(T, ctas, 0, 0);
    for (int g = tid; g <= ng; g += kTallThreads) args.tall_pre[g] = pre[g];
  }
  Place start{};
  if (part) {
    int lo = 0, hi = ng;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= S) lo = mid;
      else hi = mid;
    }
    known_group(lo, start);  // (the last that begins at or before S: it has ticks)
    const int rem = S - pre[lo];
    start.j = rem / (start.tiles + kDecTallEnd);
    start.t = rem - start.j * (start.tiles + kDecTallEnd);
  }
  __syncthreads();  // the scan's space becomes the ring
  auto next_unit = [&](Place& p) {
    p.t = 0;
    if (++p.j == a.Hkv * p.blocks) {
      int g = p.g;
      do {
        group(++g, p);
      } while (p.tiles == 0 && g < ng);
    }
  };
  auto block_rows = [&](const Place& p) { return min(kDecTallRows, p.rows - kDecTallRows * (p.j % p.blocks)); };
  // From place p, tick f of the range, on to the next piece of a unit in it: its tiles (0: none is left).
  auto piece = [&](Place& p, int& f) {
    while (f < E) {
      const int n = min(p.tiles - p.t, E - f);
      if (n > 0) return n;
      f += p.tiles + kDecTallEnd - p.t;
      if (f < E) next_unit(p);
    }
    return 0;
  };
  auto over = [&](Place& p, int& f, int n) {  // behind a piece of n tiles
    f += n;
    p.t += n;
  };
  auto fail = [&]() {
    raise_error(a.error, SPEC_DEV_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp >= 12) {
    // ============================ MMA issuers ============================
    // A whole warp runs the role, so that its addresses and descriptors stay uniform; one elected lane issues.
    const int w = warp & 1;
    const bool pv = warp >= 14;
    const uint32_t ub = __shfl_sync(FULL, sbase, 0), ut = __shfl_sync(FULL, tmem, 0);
    const uint32_t dq = desc_lo(ub + uint32_t(w) * L::kQTile, 16);
    const uint32_t db = pv ? desc_lo(ub + L::kRing + L::kHalf, L::kBlock) : desc_lo(ub + L::kRing, 16);
    bool ok = true;
    auto wait = [&](int b, int parity) { return mbar_wait(bar(b), uint32_t(parity), abort_flag); };
    Place p = start;
    int f = S, own = 0, cs = 0, stage = 0, ph = 0;  // pieces in which the group has a tile; steps issued
    for (int n; ok && (n = piece(p, f)) > 0; over(p, f, n)) {
      const bool split = block_rows(p) <= kRows;
      const int first = split ? w : 0;
      // (Q and O have a phase for each piece in which the group has a tile, the ring one for each tile, read or not)
      if (first < n) {
        ok = pv ? own == 0 || wait(kOFree0 + w, (own - 1) & 1) : wait(kQFull0 + w, own & 1);
        ++own;
      }
      ok = __all_sync(FULL, ok) != 0;
      for (int t = 0; ok && t < n; ++t) {
        const bool mine = !split || (t & 1) == w;
        const int sb = 2 * w + (cs & 1), sp_ = (cs >> 1) & 1;
        ok = wait(kFull0 + stage, ph);
        if (mine) ok = ok && (pv ? wait(kPReady0 + sb, sp_) : cs < 2 || wait(kPvDone0 + sb, sp_ ^ 1));
        if (!__all_sync(FULL, ok)) {
          ok = false;
          break;
        }
        tc_after();
        if (elect_one()) {
          const uint32_t ts = ut + col_s(w, cs & 1), dt = db + uint32_t(stage) * (L::kStage >> 4);
          if (mine && !pv) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(ts, desc(dq + uint32_t(((kk >> 2) * L::kQBlock + (kk & 3) * 32) >> 4)),
                     desc(dt + uint32_t(((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4)), idesc_bf16(kDecTile, false), kk > 0 ? 1u : 0u);
            mma_commit(bar(kSFull0 + sb));
          } else if (mine) {
#pragma unroll
            for (int kk = 0; kk < kDecTile / 16; ++kk)
              mma_ts(ut + col_o(w), ts + kk * 8, desc(dt + uint32_t((kk * 16 * 128) >> 4)), idesc_bf16(D, true), t != first || kk > 0 ? 1u : 0u);
            mma_commit(bar(kPvDone0 + sb));
            mma_commit(bar(kEmpty0 + stage));
          } else if (pv) {
            mbar_arrive(bar(kEmpty0 + stage));
          }
        }
        __syncwarp();
        cs += mine ? 1 : 0;
        if (++stage == kStages) {
          stage = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok && !*abort_flag) fail();
    // every MMA issued has completed before TMEM is released
    __syncwarp();
    if (elect_one()) mma_commit(bar(kDrain0 + (warp & 3)));
    for (int i = 0; i < 1000 && !mbar_poll(bar(kDrain0 + (warp & 3)), 0); ++i) {
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ============================ copies ============================
    const int c = warp - 8;
    constexpr int kChunks = D / 8;       // 16-byte chunks of a row
    constexpr int kKeys = 32 / kChunks;  // rows that a warp's copy spans
    const int cx = lane % kChunks, ck = lane / kChunks;
    const uint32_t slot_bytes = uint32_t(a.Hkv) * D * 2u, page_mask = (1u << args.shift) - 1u;
    const unsigned char* const k0 = static_cast<const unsigned char*>(a.k_pool) + cx * 16;
    const long long to_v = static_cast<const unsigned char*>(a.v_pool) - static_cast<const unsigned char*>(a.k_pool);
    const uint32_t ring0 = sbase + uint32_t(L::kRing) + uint32_t(cx >> 3) * L::kBlock + uint32_t(16 * c + ck) * 128u;
    Place p = start;
    int f = S, n = piece(p, f), i = 0;
    // What look() found: of each of two tiles the kv head (-1: none is left); lanes of a half of the warp hold their
    // key's position (-1: none that counts) and page id.
    int x_pos = -1, x_id = -1, h_now = 0, x_now = 0, heads[2];
    const int* row_now = nullptr;
    auto look = [&](int half) {
      if (i == n) {
        over(p, f, n);
        n = piece(p, f);
        i = 0;
      }
      heads[half] = -1;
      if (n == 0) return;
      if (i == 0) {
        h_now = p.j / p.blocks;
        row_now = a.page_table + (long long)__ldg(a.req_pool_idx + p.r0) * a.row_pages;
        x_now = p.t * kDecTile + 16 * c + (lane & 15);
      }
      heads[half] = h_now;
      if ((lane >> 4) == half) {
        x_pos = -1;
        if (x_now < p.shared) {
          x_pos = x_now;
          x_id = __ldg(row_now + (x_now >> args.shift));
        }
      }
      x_now += kDecTile;
      ++i;
    };
    int stage = 0, ph = 1, issued = 0, told = 0, told_stage = 0;
    bool ok = true;
    heads[1] = -1;
    look(0);
    if (heads[0] >= 0) look(1);
    while (ok && heads[0] >= 0) {
      const int h1 = heads[1];
      int slot = 0;
      bool counts = x_pos >= 0;
      if (counts) {
        if (uint32_t(x_id) >= uint32_t(a.num_pages)) {
          raise_error(a.error, SPEC_DEV_INDEX);
          counts = false;
        } else {
          slot = (x_id << args.shift) + int(uint32_t(x_pos) & page_mask);
        }
      }
      const unsigned valid = __ballot_sync(FULL, counts);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int h = half ? h1 : heads[0];
        if (h < 0 || !ok) break;
        ok = __all_sync(FULL, mbar_wait(bar(kEmpty0 + stage), uint32_t(ph), abort_flag)) != 0;
        if (!ok) break;
        const uint32_t st = ring0 + uint32_t(stage) * L::kStage;
        const unsigned char* const from = k0 + uint32_t(h) * uint32_t(D) * 2u;
        const unsigned mine = valid >> (half * 16 + ck);
#pragma unroll
        for (int q = 0; q < 16 / kKeys; ++q) {
          const unsigned char* src = from + (unsigned long long)uint32_t(__shfl_sync(FULL, slot, half * 16 + q * kKeys + ck)) * slot_bytes;
          const uint32_t bytes = (mine >> (q * kKeys) & 1u) * 16u;  // (a key that does not count reads as zeros)
          const uint32_t to = st + uint32_t(q * kKeys) * 128u + ((uint32_t(cx & 7) ^ uint32_t((q * kKeys + ck) & 7)) << 4);
          cp16(to, src, bytes);
          cp16(to + L::kHalf, src + to_v, bytes);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (lane == 0) masks[stage * 4 + c] = (valid >> (16 * half)) & 0xffffu;
        ++issued;
        if (issued - told > kLag) {  // the tile kLag back has landed: the MMAs may read it
          asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
          fence_async();
          mbar_arrive(bar(kFull0 + told_stage));
          ++told;
          told_stage = told_stage + 1 == kStages ? 0 : told_stage + 1;
        }
        if (++stage == kStages) {
          stage = 0;
          ph ^= 1;
        }
        // (the other half's next tile is looked up once both of this window have been copied)
        if (half == 0) look(0);
      }
      const bool had = ok && h1 >= 0 && heads[0] >= 0;
      heads[1] = -1;
      if (had) look(1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_async();
    for (; told < issued; ++told) {
      mbar_arrive(bar(kFull0 + told_stage));
      told_stage = told_stage + 1 == kStages ? 0 : told_stage + 1;
    }
    if (!ok && !*abort_flag) fail();
  } else {
    // ============================ softmax groups ============================
    // (every tcgen05.ld / st and every exit around them is warp-uniform)
    const int w = warp >> 2, r = tid & 127;
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t to = tl + col_o(w);
    const float xf = a.scale * 1.4426950408889634f;
    bool ok = true;
    int cs = 0, stage = 0;
    // A piece's Q rows go straight into their places of the operand tile (16 lanes a row, each warp its own 32 rows),
    // as soon as the piece before has its last scores.
    const uint32_t qtile = sbase + uint32_t(w) * L::kQTile;
    auto ask_q = [&](const Place& q) {
      constexpr int kChunks = D / 8, kRowsOp = 32 / kChunks;
      const int h = q.j / q.blocks, ch = lane % kChunks, x0 = kDecTallRows * (q.j % q.blocks) + (block_rows(q) <= kRows ? 0 : kRows * w);
#pragma unroll 1
      for (int rr = 32 * (warp & 3) + lane / kChunks, e = 0; e < 32 / kRowsOp; ++e, rr += kRowsOp) {
        const int x = x0 + rr;
        const bool on = x < q.rows;
        const int mem = on ? x / G : 0;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (size_t(q.r0) + mem) * a.q_ld + size_t(h * G + (on ? x - mem * G : 0)) * D + ch * 8;
        cp16(qtile + uint32_t(ch >> 3) * L::kQBlock + uint32_t(rr) * 128u + ((uint32_t(ch & 7) ^ uint32_t(rr & 7)) << 4), src, on ? 16u : 0u);
      }
    };
    auto has_tile = [&](const Place& q, int n) { return n > 0 && (block_rows(q) > kRows || w < n); };
    Place p = start, pn = start;
    int f = S, n = piece(p, f);
    if (has_tile(p, n)) ask_q(p);
    while (n > 0) {
      const bool split = block_rows(p) <= kRows;
      const int stride = split ? 2 : 1, first = split ? w : 0;
      const bool mine = first < n, whole = p.t == 0 && n == p.tiles;
      if (mine) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async();
        mbar_arrive(bar(kQFull0 + w));
      }
      pn = p;
      int fn = f;
      over(pn, fn, n);
      const int nn = piece(pn, fn);
      const bool ask = has_tile(pn, nn);
      if (!mine && ask) ask_q(pn);  // (no product reads it)
      float m = -INFINITY, l = 0.f;
      const int cs0 = cs;
      int st = stage + first >= kStages ? stage + first - kStages : stage + first;
      for (int t = first; t < n; t += stride) {
        if (!__all_sync(FULL, mbar_wait(bar(kSFull0 + 2 * w + (cs & 1)), (cs >> 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_after();
        const uint32_t ts = tl + col_s(w, cs & 1);
        if (t + stride >= n && ask) ask_q(pn);  // every product that reads this piece's Q is complete
        const uint32_t m0 = masks[st * 4] | masks[st * 4 + 1] << 16, m1 = masks[st * 4 + 2] | masks[st * 4 + 3] << 16;
        // The exponentials are taken against the reference as it is.  Their sum tells whether it will do; in the rare
        // case that it may not, the maximum is looked for, the reference moves and the tile is taken again.
#pragma unroll 1
        for (bool again = false;; again = true) {
          uint32_t u[64];
          tmem_ld32(ts, u);
          tmem_ld32(ts + 32, u + 32);
          const float mr = m == -INFINITY ? 0.f : m;
          tmem_ld_wait();
          if ((m0 & m1) != 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!((i < 32 ? m0 : m1) >> (i & 31) & 1u)) u[i] = xf < 0.f ? 0x7f800000u : 0xff800000u;
          }
          const float2 k2 = make_float2(xf, xf), o2 = make_float2(-mr, -mr);
          float2 s0 = make_float2(0.f, 0.f), s1 = s0;
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 y = fma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), k2, o2);
            const float2 q = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            if (i & 1) s1 = add2(s1, q);
            else s0 = add2(s0, q);
            pk[i] = dec_pack(q.x, q.y);
          }
          s0 = add2(s0, s1);
          const float sum = s0.x + s0.y;
          if (again || __all_sync(FULL, sum < kSumMost && m > -INFINITY)) {
            l += sum;
            tmem_st32(ts, pk);
            break;
          }
          float mx = -INFINITY;
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            uint32_t v[16];
            tmem_ld16(ts + 16 * g, v);
            const uint32_t bits = (g < 2 ? m0 : m1) >> (16 * (g & 1));
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (bits >> i & 1u) mx = fmaxf(mx, __uint_as_float(v[i]) * xf);
          }
          // the reference becomes a whole number, so that O and l are multiplied by a power of two, exactly (or by 0)
          float fac = 1.f;
          if (mx > m + kDecBase) {
            const float mn = ceilf(mx) - kDecBase;
            fac = m == -INFINITY ? 1.f : pow2(m - mn);
            l *= fac;
            m = mn;
          }
          if (cs > cs0 && __any_sync(FULL, fac != 1.f)) {
            if (!__all_sync(FULL, mbar_wait(bar(kPvDone0 + 2 * w + ((cs - 1) & 1)), ((cs - 1) >> 1) & 1, abort_flag))) {
              ok = false;
              break;
            }
            tc_after();
#pragma unroll 1
            for (int g = 0; g < D / 16; ++g) {
              uint32_t o[16];
              tmem_ld16(to + 16 * g, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac);
              tmem_st16(to + 16 * g, o);
            }
            tmem_st_wait();
          }
        }
        if (!ok) break;
        tmem_st_wait();
        tc_before();
        mbar_arrive(bar(kPReady0 + 2 * w + (cs & 1)));
        ++cs;
        st += stride;
        if (st >= kStages) st -= kStages;
      }
      if (!ok) break;
      stage = (stage + n) % kStages;

      // ---- the piece's partial result ----
      const int rows = block_rows(p), h = p.j / p.blocks, row = (split ? 0 : kRows * w) + r;  // row of the unit
      const size_t unit0 = size_t(p.r0) * a.Hq + size_t(h) * p.rows + kDecTallRows * (p.j % p.blocks);
      const size_t slot = (size_t(2) * blockIdx.x + (p.t == 0 ? 1 : 0)) * 2 + w;
      const size_t half = split ? size_t(w) * a.b * a.Hq : 0;
      float4* po = whole ? args.whole_o + (half + unit0) * (D / 4) + row : args.tall_o + slot * (D / 4) * kRows + r;
      float2* pm = whole ? args.whole_ml + half + unit0 + row : args.tall_ml + slot * kRows + r;
      const int step = whole ? rows : kRows;  // from one word of four columns to the next
      const bool valid = row < rows;
      if (mine) {
        if (!__all_sync(FULL, mbar_wait(bar(kPvDone0 + 2 * w + ((cs - 1) & 1)), ((cs - 1) >> 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_after();
#pragma unroll 1
        for (int g = 0; g < D / 16; ++g) {
          uint32_t o[16];
          tmem_ld16(to + 16 * g, o);
          tmem_ld_wait();
          if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              po[size_t(4 * g + i) * step] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                                         __uint_as_float(o[4 * i + 3]));
          }
        }
        tc_before();
        mbar_arrive(bar(kOFree0 + w));  // the next piece may write O
      }
      if (valid) *pm = make_float2(m, mine ? l : kDecNone);  // (without a tile: its O is not read)
      p = pn;
      f = fn;
      n = nn;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && !*abort_flag) fail();
  }

  // ---- teardown ----
  tc_before();
  __syncthreads();
  if (warp == 12) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D>
int launch(const DecodeArgs& args, int sms, cudaStream_t stream) {
  // at least 120 KB, so that two CTAs never share a SM (each holds all of TMEM)
  size_t smem = TallSmem<D>::kBytes + 1024;
  if (smem < 120 * 1024) smem = 120 * 1024;
  if (cudaFuncSetAttribute(decode_attention_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
    return SPEC_ERR_LAUNCH;
  const int grid = sms < kDecMaxCtas ? sms : kDecMaxCtas;
  return launch_pdl(decode_attention_tc_kernel<D>, dim3(grid), dim3(kTallThreads), smem, stream, args) == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace

int launch_decode_tall(const DecodeArgs& args, int sms, cudaStream_t stream) {
  return args.p.D == 128 ? launch<128>(args, sms, stream) : launch<64>(args, sms, stream);
}

}  // namespace spec
