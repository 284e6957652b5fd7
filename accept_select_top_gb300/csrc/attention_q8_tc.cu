// attention_q8_tc.cu -- tree-masked verify attention over the 8-bit paged cache on
// the tcgen05 tensor cores, for units of more query rows than the register
// kernel of attention_q8.cu takes (the mathematics is described there).
//
// A unit is (request, kv head, up to 256 query rows); row r is (node r / G, q
// head g G + r % G).  Its keys come in tiles: 128 history keys, then one tile of
// the (at most 64) tree nodes.  One CTA a SM takes an equal contiguous range of
// all tiles (units laid end to end, the row blocks of one kv head next to one
// another, so that the second finds its keys in L2).  Warps:
//   0-3, 4-7  two softmax groups, one query row a thread.  More than 128 rows:
//             group w has rows 128 w .. and both see every tile; fewer: the
//             groups take turns at the tiles (two partial results, joined).
//   8-11, 12-15  converters of K and of V: e4m3 becomes f16 (one instruction for
//             two values) in 128B-swizzled operand tiles, double buffered.  Tree
//             nodes are bf16 rows divided by their own power of two, and stored the
//             same way.
//   16-19     issue the MMAs: S = Q K^T (M 128, N 64, K D, both from shared
//             memory) and O += P V (A = P from TMEM), a warp each for each group.
//   20, 21    ask for the tiles: bulk copies bring their pages into shared memory as
//             they are.
// TMEM: O0 O1 | two S buffers a group; P (f16, two to a column) takes the place of
// its S.  A step is 64 keys: the scores of the next one are computed, and the
// products of the last one added up, while a step's softmax runs.  (One S buffer with
// places of their own for P made S always ready, but its softmax, which then has to
// settle a half's reference before S is gone, took 500 cycles longer.)
//
// Bound: 2 x 1024 cycles of MMA for 128 keys and 256 rows (f16 at 4096
// multiply-adds a cycle).  Per tile shared memory moves 64 KB of converted
// operands in, 128 KB for S (A and B) and 64 KB for P V; P through shared
// memory would add 128 KB, which is why it goes through TMEM (an MMA with A
// from TMEM measured the same 64 cycles as one with both operands in shared
// memory, once its descriptors are precomputed).
//   Measured: two contexts of 32768 to 131072, 64 nodes, 64 / 8 heads of 128: 267 us
// (1.29 PF/s; 277 us by eager calls); 32 requests of 2048, 64 nodes, 32 / 8 heads: 97 us (0.71 PF/s).  In the
// history a step of 64 keys takes a group some 1960 cycles, of which the softmax is 1500
// (two warps of it and two converters share a scheduler) and the MMAs of both groups
// 1280.  A unit's end costs about 25000 cycles more: the tree's rows are converted
// late, its softmax looks at masks and exponents node by node, and O leaves as 128 KB
// of fragments where a CTA's range cuts the unit.
//   Every wait is bounded: on timeout the CTA sets SPEC_DEV_TIMEOUT, stops,
// drains its MMAs and frees its TMEM.
#include "common.cuh"
#include "kernels.cuh"

#include "attention_q8.cuh"
#include "e4m3.cuh"

namespace spec {

namespace {

constexpr int kRows = 128;
constexpr int kKeys = 128;       // history keys of a tile
constexpr int kTreeKeys = 64;    // nodes of the tree tile
constexpr int kStep = 64;        // keys of a step of S, softmax and P V
constexpr float kPMost = 60000.f; // a sum of P below this holds no value that f16 does not
constexpr int kGroup = 16;       // keys with one page at least
constexpr int kGroups = kKeys / kGroup;
constexpr int kTcThreads = 24 * 32;
// Registers a thread, by warp group: the CTA is launched with kRegs each, and
// the groups trade (sums of four warps: what they take may not pass what was launched).
constexpr int kRegs = 80, kRegsSoft = 136, kRegsConv = 64, kRegsIssue = 40, kRegsAsk = 40;
static_assert(2 * kRegsSoft + 2 * kRegsConv + kRegsIssue + kRegsAsk <= 6 * kRegs, "register split");
constexpr int kConvThreads = 128;
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s: bound of every wait
__host__ __device__ constexpr uint32_t col_o(int w) { return 128u * uint32_t(w); }
__host__ __device__ constexpr uint32_t col_s(int w, int b) { return 256u + 128u * uint32_t(w) + 64u * uint32_t(b); }

// What the softmax needs of a tile: of a history tile, for each group of 16
// keys, {K scale, V exponent relative to the unit's base, its inverse factor in
// l (0: below the span, l's share is added up apart), keys that count (less kMark in
// a step's first group: the base has changed, or a group lies below the span)}; of the
// tree tile, each node's K and V exponent bytes, as the halves that hold 2^(K's - 127)
// and float(V's) in bf16.
constexpr float kMark = 1024.f;
__device__ __forceinline__ float keys_of(float w) { return w < 0.f ? w + kMark : w; }
struct TileMeta {
  union {
    float4 group[kGroups];
    uint32_t node[kTreeKeys];
  };
  unsigned long long nonfinite[4];  // tree nodes whose V row holds an inf or a NaN, a word a converter warp
  int top[4];                       // the tree's largest V exponent, a word a converter warp
  int base;                         // the history's V exponent base
  int pad[3];
};

template <int D>
struct TcSmem {
  static constexpr int kBlock = kRows * 128;       // [128 rows x 64 f16], 128B-swizzled
  static constexpr int kTile = (D / 64) * kBlock;  // an operand tile
  static constexpr int kRaw = kKeys * D;           // a tile as it is in memory (also 64 bf16 rows)
  static constexpr int kQ = 0;                     // two
  static constexpr int kK = 2 * kTile;             // two
  static constexpr int kV = 4 * kTile;             // two
  static constexpr int kRawK = 6 * kTile;
  static constexpr int kRawV = kRawK + kRaw;
  static constexpr int kMeta = kRawV + kRaw;       // four
  static constexpr int kInfo = kMeta + 4 * int(sizeof(TileMeta));  // [K, V][2][8]: keys of a raw tile's groups
  static constexpr int kBars = kInfo + 128;
  static constexpr int kAbort = kBars + 8 * 34 + 4;  // (after the barriers: TMEM address, abort flag)
  static constexpr int kKeep = kAbort + 4 + 4 * (kTcThreads / 32);  // behind the scan's words
  static constexpr int kBytes = kBars + 448;
  // the tiles before each request are summed up in what will hold operands
  static_assert(4 * (kAttentionQ8MaxB + 1) <= 2 * kTile, "scan space");
};
static_assert(TcSmem<128>::kBytes + 1024 <= 227 * 1024, "shared memory of one CTA");

enum {
  kKFull0 = 0,  // + buffer: converters stored the K tile (and the tile's meta)
  kKEmpty0 = 2, // + buffer: the S products that read it are complete (two arrivals)
  kVFull0 = 4,
  kVEmpty0 = 6,
  kQFull0 = 8,  // + group
  kOFree0 = 10,    // the epilogue has read O
  kFragFull = 12,  // group 1 stored its half of a unit that this CTA finishes
  kFragFree = 13,  // group 0 has read it
  kDrain0 = 14,    // + issuing warp
  kRawFull0 = 18,  // + (K, V): the raw tile has landed
  kRawEmpty0 = 20, // the converters have read it
  // + 2 group + S buffer: by buffer, so that nothing is ever two phases ahead of who waits for it
  kSFull0 = 22,
  kPReady0 = 26,
  kPvDone0 = 30,
  kNumBars = 34
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity), "r"(20000u)
               : "memory");
  return ok != 0;
}
// Up to 128 tries, in a loop of four instructions and without a time hint: the warps that wait
// take issue slots from the others (the long contexts 267 us so, 268 with a hint of 20 us, 275 by
// test_wait).
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
// Bounded wait for the phase of the given parity: false once kWaitCycles have
// passed or another warp has given up.  (That is looked at only where the phase does not
// come: a warp whose waits are still met goes on. With a look in every wait the long contexts take 272 us.)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_poll(bar, parity)) return true;
  const long long start = clock64();
  do {
    if (mbar_poll(bar, parity)) return true;
  } while (!*abort_flag && clock64() - start <= kWaitCycles);
  return false;
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// `bytes` (a multiple of 16) of global memory into shared memory, counted in on `bar`
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// 16-byte global -> shared copy; 0 bytes: zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& x) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
// one byte; the load stays ahead of the waits that follow it
__device__ __forceinline__ uint32_t ld_nc8(const uint8_t* p) {
  uint32_t x;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor (128B swizzle, descriptor version 1) in two
// words: address and leading-dimension offset, then stride offset and flags.  The
// address is stepped in the low word alone.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
  return d;
}
// instruction descriptor of kind::f16: f16 A and B, f32 accumulator, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
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
// 8, 16, 32 columns stored (tmem_st_wait completes them)
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
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

struct TcArgs {
  AttentionQ8Params p;
  int blocks;          // 256-row blocks of a kv head's n * G rows
  int4* begun;         // [CTA]: the unit that the CTA begins and does not finish {last CTA of it (-1: none), request, (head, block), -}
  float* slot_o;       // [2 * CTA + i][group][D / 4][128][4]
  float* slot_ml;      // [2 * CTA + i][group][128][2]
};

// a position in the tile space
struct Pos {
  int r, j, t, Tr;  // request, (kv head, row block), tile, tiles of the request
  int len, row;     // the request's history and table row (-1: none)
};

__device__ __forceinline__ void request_of(const AttentionQ8Params& a, Pos& p) {
  const ReqQ8 q = req_q8(a, a.seq_lens[p.r], a.req_pool_idx[p.r], false);
  p.len = q.len;
  p.row = q.row;
  p.Tr = (q.len + kKeys - 1) / kKeys + 1;
}
__device__ __forceinline__ void next_pos(const AttentionQ8Params& a, int J, Pos& p) {
  if (++p.t == p.Tr) {
    p.t = 0;
    if (++p.j == J) {
      p.j = 0;
      if (++p.r < a.b) request_of(a, p);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) attention_q8_tc_kernel(const __grid_constant__ TcArgs args) {
  using L = TcSmem<D>;
  constexpr unsigned FULL = 0xffffffffu;
  const AttentionQ8Params& a = args.p;
  const int G = a.Hq / a.Hkv, M = a.n * G, J = a.Hkv * args.blocks;
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;

  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  unsigned char* sp = smem_raw + (sbase - raw);
  TileMeta* metas = reinterpret_cast<TileMeta*>(sp + L::kMeta);
  const uint32_t bars = sbase + L::kBars;
  auto bar = [&](int i) { return bars + 8u * uint32_t(i); };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sp + L::kBars + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + L::kAbort);
  static_assert(L::kAbort == L::kBars + 8 * kNumBars + 4 && L::kKeep + 4 <= L::kBytes, "layout");
  int* wsum = reinterpret_cast<int*>(sp + L::kBars + 8 * kNumBars + 8);  // [24]
  int* keep = reinterpret_cast<int*>(sp + L::kKeep);  // the tiles in all
  int* pre = reinterpret_cast<int*>(sp);  // [b + 1] tiles of one (kv head, row block) before request r (until the roles start)

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKFull0 + i), kConvThreads);
      mbar_init(bar(kKEmpty0 + i), 2);
      mbar_init(bar(kVFull0 + i), kConvThreads);
      mbar_init(bar(kVEmpty0 + i), 2);
      mbar_init(bar(kQFull0 + i), kRows);
      mbar_init(bar(kOFree0 + i), kRows);
      mbar_init(bar(kRawFull0 + i), 1);
      mbar_init(bar(kRawEmpty0 + i), kConvThreads);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kSFull0 + i), 1);
      mbar_init(bar(kPReady0 + i), kRows);
      mbar_init(bar(kPvDone0 + i), 1);
      mbar_init(bar(kDrain0 + i), 1);
    }
    mbar_init(bar(kFragFull), kRows);
    mbar_init(bar(kFragFree), kRows);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_holder)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();  // nothing above reads global memory
  pdl_trigger();

  // ---- tiles before each request; this CTA's range ----
  {
    int run = 0;
    for (int r0 = 0; r0 < a.b; r0 += kTcThreads) {
      const int r = r0 + tid;
      int t = 0;
      if (r < a.b) {
        const ReqQ8 q = req_q8(a, a.seq_lens[r], a.req_pool_idx[r], blockIdx.x == 0);
        t = (q.len + kKeys - 1) / kKeys + 1;
      }
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
      for (int q = 0; q < kTcThreads / 32; ++q) {
        if (q < warp) before += wsum[q];
        run += wsum[q];
      }
      if (r < a.b) pre[r] = before + incl - t;
    }
    if (tid == 0) pre[a.b] = run;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_holder;
  const long long T = (long long)pre[a.b] * J;
  const long long ctas = T < gridDim.x ? T : gridDim.x;
  const bool part = blockIdx.x < ctas;
  const int S = part ? int(blockIdx.x * T / ctas) : 0, E = part ? int((blockIdx.x + 1ll) * T / ctas) : 0;
  Pos start;
  {
    int lo = 0, hi = a.b;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * J <= S) lo = mid;
      else hi = mid;
    }
    start.r = lo;
    start.Tr = pre[lo + 1] - pre[lo];
    const int rem = S - pre[lo] * J;
    start.j = rem / start.Tr;
    start.t = rem - start.j * start.Tr;
  }
  request_of(a, start);
  if (tid == 0) *keep = int(T);
  __syncthreads();  // the scan's space becomes operand tiles
  auto advance = [&](Pos& p) { next_pos(a, J, p); };
  // the piece of a unit that begins at position p, tile f of the range: its tiles
  auto piece_tiles = [&](const Pos& p, int f) { return min(p.Tr - p.t, E - f); };
  auto unit_rows = [&](int j) { return min(2 * kRows, M - 2 * kRows * (j % args.blocks)); };
  auto fail = [&]() {
    raise_error(a.error, SPEC_DEV_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp >= 20) {
    // ============================ asking for raw tiles ============================
    // Warp 20 K, 21 V (22 and 23 make up the warp group): one bulk copy a group of 16
    // keys (16 D contiguous bytes of a page), a lane each; of the tree tile, one a
    // node's row.  Page ids are read two tiles ahead, scale bytes one.  (Loads
    // through registers kept about 11 KB in flight a SM, as little L1 is left beside
    // the operands, and took three times the MMAs' time; asked for by the converters'
    // own first warps, the tiles came 2000 cycles later and bounded everything.)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsAsk));
    const int kv = warp & 1;
    const uint32_t rawt = sbase + (kv ? L::kRawV : L::kRawK);
    uint32_t* infos = reinterpret_cast<uint32_t*>(sp + L::kInfo) + kv * 2 * kGroups;
    const int SHIFT = a.page_size == 16 ? 0 : a.page_size == 32 ? 1 : 2;  // log2(groups a page)
    auto fetch = [&](const Pos& p) {  // the page id of the lane's group
      const int g0 = p.t * kGroups + lane;
      if (lane < kGroups && p.t < p.Tr - 1 && g0 * kGroup < p.len) return a.page_table[size_t(p.row) * a.row_pages + (g0 >> SHIFT)];
      return 0;
    };
    if (warp < 22 && S < E) {
      // the tile asked for next: where the lane's group (of the tree tile: row 0) lies, its bytes, its info word
      const uint8_t* src = nullptr;
      uint32_t bytes = 0, word = 0;
      bool tree = false;
      Pos p = start;  // and the one after
      int pid = fetch(p);
      auto prepare = [&]() {
        tree = p.t == p.Tr - 1;
        bytes = word = 0;
        if (tree) {
          src = static_cast<const uint8_t*>(kv ? a.v_new : a.k_new) + 2 * (size_t(p.r) * a.n * a.new_ld + size_t(p.j / args.blocks) * D);
        } else {
          const int g = p.t * kGroups + lane, left = p.len - g * kGroup;
          if (lane < kGroups && left > 0) {
            if (pid < 0 || pid >= a.num_pages) {
              raise_error(a.error, SPEC_DEV_INDEX);
            } else {
              const int unit = pid * a.Hkv + p.j / args.blocks, cnt = min(kGroup, left);
              bytes = uint32_t(cnt) * D;
              src = (kv ? a.v_pages : a.k_pages) + (size_t(unit) * a.page_size + (g & ((1 << SHIFT) - 1)) * kGroup) * D;
              word = uint32_t(cnt);
              if (kv == 0) word |= ld_nc8(a.k_scales + unit) << 8 | ld_nc8(a.v_scales + unit) << 16;
            }
          }
        }
      };
      const uint32_t full = bar(kRawFull0 + kv);
      bool ok = true;
      int ct = -1;
      for (;;) {
        if (ct >= 0) {
          if (ct > 0) {
            ok = __all_sync(FULL, mbar_wait(bar(kRawEmpty0 + kv), (ct - 1) & 1, abort_flag) && !*abort_flag) != 0;
            if (!ok) break;
          }
          if (lane < kGroups) infos[(ct & 1) * kGroups + lane] = word;
          const uint32_t all = tree ? uint32_t(a.n) * D * 2u : __reduce_add_sync(FULL, bytes);
          if (lane == 0) mbar_expect(full, all);
          __syncwarp();
          if (tree) {
            for (int i = lane; i < a.n; i += 32) bulk_copy(rawt + uint32_t(i * D * 2), src + size_t(i) * a.new_ld * 2, uint32_t(D) * 2u, full);
          } else if (bytes) {
            bulk_copy(rawt + uint32_t(lane * kGroup * D), src, bytes, full);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
        if (++ct == E - S) break;
        prepare();
        if (ct + 1 < E - S) {
          advance(p);
          pid = fetch(p);
        }
      }
      if (!ok && !*abort_flag) fail();
      // the last copy has landed before the CTA can end, whoever gave up
      for (int k = 0; k < 100 && !mbar_try(full, (ct - 1) & 1); ++k) {
      }
    }
  } else if (warp >= 16) {
    // ============================ MMA issuers ============================
    // Warps 16, 17: S = Q K^T of softmax groups 0, 1; warps 18, 19: O += P V.  A
    // step is 64 keys; its S goes into one of two buffers, as soon as P V of the
    // step before last has read it, so that the softmax of a step runs beside the
    // products of its neighbours.  Four warps, because a product's waits and
    // issue take one warp about as long as the product itself.  A whole warp runs
    // the role, so that its addresses and descriptors stay uniform (one lane
    // alone spent more time forming them than the MMAs take); one elected lane
    // issues.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    const int w = warp & 1;
    const bool pv = warp >= 18;
    const uint32_t ub = __shfl_sync(FULL, sbase, 0), ut = __shfl_sync(FULL, tmem, 0);
    const uint32_t dq = desc_lo(ub + L::kQ + uint32_t(w) * L::kTile, 16);
    const uint32_t db = pv ? desc_lo(ub + L::kV, L::kBlock) : desc_lo(ub + L::kK, 16);
    const int full0 = pv ? kVFull0 : kKFull0, empty0 = pv ? kVEmpty0 : kKEmpty0;
    bool ok = true;
    auto wait = [&](int b, int parity) { return mbar_wait(bar(b), uint32_t(parity), abort_flag); };
    Pos p = start;
    int ct0 = 0, own = 0, cs = 0;  // pieces in which the group has a tile; steps issued
    for (int f = S; ok && f < E;) {
      const int n = piece_tiles(p, f);
      const bool split = unit_rows(p.j) <= kRows;
      const int tree_at = p.t + n == p.Tr ? n - 1 : n, first = split ? w : 0;
      // Q and O have a phase for each piece in which the group has a tile, K and V one
      // for each tile, read or not: a phase let pass makes the next one's parity the wrong one.
      // Before S goes on to another piece, P V has to be through with the last: the softmax
      // then reads no more of its tiles' metas, whose places the converters take.
      if (!pv) ok = cs == 0 || wait(kPvDone0 + 2 * w + ((cs - 1) & 1), ((cs - 1) >> 1) & 1);
      if (first < n) {
        ok = ok && (pv ? own == 0 || wait(kOFree0 + w, (own - 1) & 1) : wait(kQFull0 + w, own & 1));
        ++own;
      }
      ok = __all_sync(FULL, ok) != 0;
      for (int t = 0, hf = 0; ok && t < n;) {
        const int ct = ct0 + t, buf = ct & 1, sb = 2 * w + (cs & 1), ph = (cs >> 1) & 1;
        if (split && (t & 1) != w) {  // the other group's tile
          ok = wait(full0 + buf, (ct >> 1) & 1);
          if (!__all_sync(FULL, ok)) {
            ok = false;
            break;
          }
          if (elect_one()) mbar_arrive(bar(empty0 + buf));
          __syncwarp();
          ++t;
          continue;
        }
        const bool last = hf == 1 || t == tree_at, begin = t == first && hf == 0;
        const uint32_t ts = ut + col_s(w, cs & 1);
        const uint32_t dt = db + uint32_t(buf) * (L::kTile >> 4) + uint32_t(hf) * (kStep * 128 >> 4);
        ok = hf == 1 || wait(full0 + buf, (ct >> 1) & 1);
        if (!pv) {
          ok = ok && (cs < 2 || wait(kPvDone0 + sb, ph ^ 1));
          // (the tree tile is one step, so its S alone does not tell that the softmax is through with the
          // group's tile before, whose place in the ring of metas the converters take once it is read)
          if (split && t == tree_at && cs > 0) ok = ok && wait(kPvDone0 + 2 * w + ((cs - 1) & 1), ((cs - 1) >> 1) & 1);
        } else {
          ok = ok && wait(kPReady0 + sb, ph);
        }
        if (!__all_sync(FULL, ok)) {
          ok = false;
          break;
        }
        tc_after();
        if (elect_one()) {
          if (!pv) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = uint32_t(((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4);
              mma_ss(ts, desc(dq + o), desc(dt + o), idesc_f16(kStep, false), kk > 0 ? 1u : 0u);
            }
            mma_commit(bar(kSFull0 + sb));
          } else {
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk)
              mma_ts(ut + col_o(w), ts + kk * 8, desc(dt + uint32_t((kk * 16 * 128) >> 4)), idesc_f16(D, true), !begin || kk > 0 ? 1u : 0u);
            mma_commit(bar(kPvDone0 + sb));
          }
          if (last) mma_commit(bar(empty0 + buf));
        }
        __syncwarp();
        ++cs;
        hf = last ? 0 : 1;
        t += last ? 1 : 0;
      }
      ct0 += n;
      f += n;
      p.t += n - 1;
      advance(p);
    }
    if (!ok && !*abort_flag) fail();
    // every MMA issued has completed before TMEM is released
    __syncwarp();
    if (elect_one()) mma_commit(bar(kDrain0 + (warp & 3)));
    for (int i = 0; i < 1000 && !mbar_try(bar(kDrain0 + (warp & 3)), 0); ++i) {
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ============================ converters ============================
    // Warps 8-11 K, 12-15 V: raw tile -> f16 operand tile.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    const int kv = warp >= 12 ? 1 : 0, cw = warp & 3, ct_id = tid & 127;
    const uint32_t rawt = sbase + (kv ? L::kRawV : L::kRawK);
    uint32_t* infos = reinterpret_cast<uint32_t*>(sp + L::kInfo) + kv * 2 * kGroups;
    const int full0 = kv ? kVFull0 : kKFull0, empty0 = kv ? kVEmpty0 : kKEmpty0;
    auto wait = [&](int b, int parity) {
      return __all_sync(FULL, mbar_wait(bar(b), uint32_t(parity), abort_flag)) != 0;
    };

    Pos p = start;
    constexpr int kLoads = D / 16;               // 16-byte words a thread of a raw tile
    constexpr int kLanesKey = D / 16;            // lanes a history key
    constexpr int kLanesRow = D / 8;             // lanes a tree row
    constexpr int kRowsLoad = kConvThreads / kLanesRow, kTreeLoads = kTreeKeys / kRowsLoad;
    // key (in the tile) of a thread's word i of a history tile, of the tree tile
    auto hist_key = [&](int i) { return D == 128 ? 16 * i + 4 * cw + lane / kLanesKey : 32 * i + 8 * cw + lane / kLanesKey; };
    auto tree_key = [&](int i) { return i * kRowsLoad + ct_id / kLanesRow; };
    // 16 e4m3 values -> two 16-byte chunks of their key's swizzled row
    auto store_hist = [&](uint32_t tile, const uint4 (&x)[kLoads]) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int key = hist_key(i);
        const int ch = lane % kLanesKey;  // elements 16 ch ..
        const uint32_t row = tile + uint32_t(ch >> 2) * L::kBlock + uint32_t(key) * 128u;
        const uint32_t c0 = uint32_t(2 * (ch & 3));
        // the second half's lanes store their upper chunk first: no two lanes of a phase share banks
        const bool swap = ch >= 4;
        const uint32_t a0 = swap ? x[i].z : x[i].x, a1 = swap ? x[i].w : x[i].y, b0 = swap ? x[i].x : x[i].z, b1 = swap ? x[i].y : x[i].w;
        const uint32_t at = row + (((c0 + (swap ? 1u : 0u)) ^ uint32_t(key & 7)) << 4);
        auto put = [&](uint32_t to, uint32_t w0, uint32_t w1) {
          uint4 y;
          e4m3x4_to_f16x4(w0, y.x, y.y);
          e4m3x4_to_f16x4(w1, y.z, y.w);
          sts16(to, y);
        };
        put(at, a0, a1);
        put(at ^ 16u, b0, b1);
      }
    };
    auto row_max = [&](const uint4& x) {  // a tree row's largest finite magnitude, from its lanes
      uint32_t mx = max_abs_bf16(max_abs_bf16(max_abs_bf16(max_abs_bf16(0u, x.x), x.y), x.z), x.w);
      mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
      for (int o = 1; o < kLanesRow; o <<= 1) mx = max(mx, __shfl_xor_sync(FULL, mx, o));
      return mx;
    };
    auto store_tree = [&](uint32_t tile, const uint4& x, int key, int e) {
      const float inv = exp_scale(2 * kExpBias - e);
      auto cv = [&](uint32_t w) { return pack_f16(bf16_lo(w) * inv, bf16_hi(w) * inv); };
      const int ch = ct_id % kLanesRow;
      sts16(tile + uint32_t(ch >> 3) * L::kBlock + uint32_t(key) * 128u + ((uint32_t(ch & 7) ^ uint32_t(key & 7)) << 4),
            make_uint4(cv(x.x), cv(x.y), cv(x.z), cv(x.w)));
    };
    int base = -1, last2 = -1, ct = 0;
    bool ok = true;
    for (int f = S; f < E; ++f, ++ct) {
      const int buf = ct & 1;
      const bool tree = p.t == p.Tr - 1, first = f == S || p.t == 0;
      const uint32_t* info = infos + buf * kGroups;
      const uint32_t tile = sbase + (kv ? L::kV : L::kK) + uint32_t(buf) * L::kTile;
      TileMeta& mt = metas[ct & 3];
      ok = wait(kRawFull0 + kv, ct & 1);
      if (!ok) break;
      // (K) the lane's group: keys that count, scale bytes
      const uint32_t word = lane < kGroups ? info[lane] : 0u;
      const int cnt = word & 255, ks0 = (word >> 8) & 255, vs0 = word >> 16;
      if (first) base = last2 = -1;
      bool mark = false;
      if (!tree && kv == 0 && cw == 0) {
        // (the base of the tile before last: the softmax groups may take the tiles in turn)
        const int last = base, top = int(__reduce_max_sync(FULL, cnt > 0 ? uint32_t(vs0) : 0u));
        if (top > 0) base = raised_base(base, top);
        mark = (last >= 0 && last != base) || (last2 >= 0 && last2 != base) || __any_sync(FULL, cnt > 0 && vs0 < base - kSpanDown);
        last2 = last;
      }
      if (!tree) {
        uint4 x[kLoads];  // the thread's words, zeros where there is no key
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int key = hist_key(i);
          x[i] = lds16(rawt + uint32_t(key * D + (lane % kLanesKey) * 16));
          if (uint32_t(key & 15) >= (info[key >> 4] & 255u)) x[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        mbar_arrive(bar(kRawEmpty0 + kv));
        ok = ct < 2 || wait(empty0 + buf, ((ct >> 1) - 1) & 1);
        if (!ok) break;
        if (kv == 0 && cw == 0 && lane < kGroups) {
          float4 y = cnt > 0 ? make_float4(exp_scale(ks0), float(vs0 - base), vs0 < base - kSpanDown ? 0.f : ratio_scale(base - vs0), float(cnt))
                             : make_float4(1.f, 0.f, 0.f, 0.f);
          if (mark && lane % (kStep / kGroup) == 0) y.w -= kMark;
          mt.group[lane] = y;
          if (lane == 0) mt.base = max(base, 0);
        }
        store_hist(tile, x);
      } else {
        ok = ct < 2 || wait(empty0 + buf, ((ct >> 1) - 1) & 1);
        if (!ok) break;
        constexpr int kRowsOnce = 4;  // (eight take more registers than there are)
        unsigned long long nf = 0;
        int top_e = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < kTreeLoads; i0 += kRowsOnce) {
          uint4 x[kRowsOnce];
#pragma unroll
          for (int i = 0; i < kRowsOnce; ++i) {
            const int key = tree_key(i0 + i);
            x[i] = lds16(rawt + uint32_t(key * D * 2 + (ct_id % kLanesRow) * 16));
            if (key >= a.n) x[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          // the rows' largest magnitudes; an inf or a NaN anywhere shows in them
          uint32_t top[kRowsOnce];
#pragma unroll
          for (int i = 0; i < kRowsOnce; ++i) {
            const uint32_t m2 = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu), __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
            top[i] = max(m2 & 0xffffu, m2 >> 16);
          }
#pragma unroll
          for (int o = 1; o < kLanesRow; o <<= 1)
#pragma unroll
            for (int i = 0; i < kRowsOnce; ++i) top[i] = max(top[i], __shfl_xor_sync(FULL, top[i], o));
          bool odd = false;
#pragma unroll
          for (int i = 0; i < kRowsOnce; ++i) odd = odd || top[i] >= 0x7f80u;
          if (__any_sync(FULL, odd)) {
#pragma unroll
            for (int i = 0; i < kRowsOnce; ++i) {
              const unsigned who = __ballot_sync(FULL, top[i] >= 0x7f80u);
              top[i] = row_max(x[i]);
              if (kv == 1) {
                // (an inf or a NaN of V is left out here and added to the rows that see it at the end)
                x[i] = make_uint4(finite_bf16(x[i].x), finite_bf16(x[i].y), finite_bf16(x[i].z), finite_bf16(x[i].w));
#pragma unroll 1
                for (int q = 0; q < 32 / kLanesRow; ++q)
                  if ((who >> (q * kLanesRow)) & 1u) nf |= 1ull << ((i0 + i) * kRowsLoad + cw * (32 / kLanesRow) + q);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kRowsOnce; ++i) {
            const int key = tree_key(i0 + i), e = norm_exp(top[i]);
            if (ct_id % kLanesRow == 0) reinterpret_cast<uint16_t*>(&mt.node[key])[kv] = uint16_t(kv == 0 ? uint32_t(e) << 7 : __float_as_uint(float(e)) >> 16);
            store_tree(tile, x[i], key, e);
            top_e = max(top_e, e);
          }
        }
        if (kv == 1) {
          top_e = int(__reduce_max_sync(FULL, uint32_t(top_e)));
          if (lane == 0) {
            mt.nonfinite[cw] = nf;
            mt.top[cw] = top_e;
          }
        }
        mbar_arrive(bar(kRawEmpty0 + kv));
      }
      fence_async();
      mbar_arrive(bar(full0 + buf));
      advance(p);
    }
    if (!ok && !*abort_flag) fail();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ============================ softmax groups ============================
    // (every tcgen05.ld / st and every exit around them is warp-uniform)
    const int w = warp >> 2, r = tid & 127;
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t to = tl + col_o(w);
    Pos p = start;
    int cs = 0, nfrag = 0, ct0 = 0;
    bool ok = true;
    // row of the thread (and of its warp's others) in a unit: among the kv head's n * G
    auto row_of = [&](const Pos& q, int rr) {
      return 2 * kRows * (q.j % args.blocks) + (unit_rows(q.j) <= kRows ? 0 : kRows * w) + rr;
    };
    // A piece's Q rows go straight into their places of the operand tile (16
    // lanes a row, coalesced; each warp its own 32 rows) and are divided and
    // converted in place when the piece begins.  They are asked for as soon as
    // the piece before has its last scores.
    const uint32_t qtile = sbase + L::kQ + uint32_t(w) * L::kTile;
    auto ask_q = [&](const Pos& q) {
      constexpr int kChunks = D / 8, kRowsOp = 32 / kChunks;
      const int h = q.j / args.blocks, ch = lane % kChunks;
      int rr = 32 * (warp & 3) + lane / kChunks, g = row_of(q, rr);
      int tok = g / G, hq = g - tok * G;  // (stepped: no division a row)
#pragma unroll 1
      for (int i = 0; i < 32 / kRowsOp; ++i, rr += kRowsOp, g += kRowsOp) {
        const bool on = g < M;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (size_t(q.r) * a.n + (on ? tok : 0)) * a.q_ld +
                              size_t(h * G + (on ? hq : 0)) * D + ch * 8;
        cp_async16(qtile + uint32_t(ch >> 3) * L::kBlock + uint32_t(rr) * 128u + ((uint32_t(ch & 7) ^ uint32_t(rr & 7)) << 4), src, on ? 16u : 0u);
        for (hq += kRowsOp; hq >= G; hq -= G) ++tok;
      }
    };
    // A piece's row of Q, divided by its power of two, as f16.
    float xf_next = 0.f;
    auto normalise_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      const uint32_t qrow = qtile + uint32_t(r) * 128u;
      auto chunk = [&](int i) { return qrow + uint32_t(i >> 3) * L::kBlock + ((uint32_t(i & 7) ^ uint32_t(r & 7)) << 4); };
      uint32_t mx = 0;
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        const uint4 x = lds16(chunk(i));
        mx = __vmaxu2(__vmaxu2(__vmaxu2(__vmaxu2(mx, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu), x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
      }
      if (max(mx & 0xffffu, mx >> 16) >= 0x7f80u) {  // an inf or a NaN: the largest of the others
        mx = 0;
#pragma unroll 1
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = lds16(chunk(i));
          mx = max_abs_bf16(max_abs_bf16(max_abs_bf16(max_abs_bf16(mx, x.x), x.y), x.z), x.w);
        }
      }
      const int e = norm_exp(max(mx & 0xffffu, mx >> 16));
      // the sign of the scale goes into Q, so that a larger score is a larger exponent
      const float inv = a.scale == 0.f ? 0.f : copysignf(exp_scale(2 * kExpBias - e), a.scale);
      // (a factor of 0 would take the -inf of a key that does not count to NaN: then Q is 0)
      xf_next = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f * exp_scale(e);
      auto cv = [&](uint32_t u) { return pack_f16(bf16_lo(u) * inv, bf16_hi(u) * inv); };
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        const uint4 x = lds16(chunk(i));
        sts16(chunk(i), make_uint4(cv(x.x), cv(x.y), cv(x.z), cv(x.w)));
      }
      fence_async();
      mbar_arrive(bar(kQFull0 + w));
    };
    auto has_tile = [&](const Pos& q, int f) { return unit_rows(q.j) > kRows || w < piece_tiles(q, f); };  // (the groups take tiles in turn, or all)
    if (S < E && has_tile(p, S)) ask_q(p);
    if (tid == 0) args.begun[blockIdx.x] = make_int4(-1, 0, 0, 0);
    // the piece at hand: tiles [f, f + n) of the range, from position p, and the next one's position
    Pos pn = start;
    int n = 0, node = 0, head = 0, h = 0, base = -1;
    bool split = false, complete = false, mine = false, valid = false;
    float m = -INFINITY, l = 0.f;
    unsigned long long mask = 0, nonfinite = 0;
    for (int f = S;;) {
      // The next piece's Q comes before this one's result, so that its first scores are
      // computed while the result is written.
      const bool more = f + n < E;
      const bool next = more && has_tile(pn, f + n);
      if (next) normalise_q();
      if (n > 0) {
        // ---- the piece's result ----
        if (mine) {
          const bool d_ok = mbar_wait(bar(kPvDone0 + 2 * w + ((cs - 1) & 1)), ((cs - 1) >> 1) & 1, abort_flag) && !*abort_flag;
          if (!__all_sync(FULL, d_ok)) {
            ok = false;
            break;
          }
          tc_after();
        }
        const float vs = exp_scale(base < 1 ? 1 : base);
        const bool direct = complete && !split;
        const int slot = 2 * int(blockIdx.x) + (complete || p.t == 0 ? 1 : 0);  // (0: a unit that an earlier CTA began)
        const bool local = complete && split;
        // a slot's O: 16-byte words [4 columns][row], so that a warp stores 512 contiguous bytes
        float4* so = reinterpret_cast<float4*>(args.slot_o) + (size_t(slot) * 2 + w) * kRows * (D / 4) + r;
        float2* sm = reinterpret_cast<float2*>(args.slot_ml) + (size_t(slot) * 2 + w) * kRows + r;
        const size_t orow = (size_t(p.r) * a.n + node) * a.Hq + head;
        float om = -INFINITY, ol = 0.f;  // group 1's half of a unit that group 0 finishes
        // (group 0 may not have read the last half that group 1 left in the slot)
        if (!direct && w == 1 && nfrag > 0 && !__all_sync(FULL, mbar_wait(bar(kFragFree), (nfrag - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (local) {
          if (w == 0) {
            if (!__all_sync(FULL, mbar_wait(bar(kFragFull), nfrag & 1, abort_flag))) {
              ok = false;
              break;
            }
            const float2 x = __ldcg(sm + kRows);
            om = x.x;
            ol = x.y;
          }
          ++nfrag;
        }
        const unsigned long long nf = nonfinite & mask;
        const bool any_nf = __any_sync(FULL, nf != 0ull);
        // out = O / l 2^base, averaged with the other half by their weights
        const bool has_o = ol > 0.f || ol != ol;
        const float M2 = has_o ? fmaxf(m, om) : m;
        const float la = has_o && m != M2 ? l * fast_exp2(m - M2) : l, lb = has_o ? fast_exp2(om - M2) : 0.f;
        const float Ls = has_o ? fmaf(ol, lb, la) : l;
        const bool result = direct || (local && w == 0);
        float fm = m, fl = l;
        const float inv = result ? inverse_of(l) : settle(fm, fl), wa = has_o ? la / Ls : 1.f, wb = lb * settled_inverse(Ls);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float v[16];
          if (mine) {
            uint32_t o[16];
            tmem_ld16(to + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(o[i]) * inv * vs;
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.f;
          }
          if (any_nf && nf) {
            for (int q = 0; q < a.n; ++q)
              if ((nf >> q) & 1ull) {
                const uint16_t* vr = static_cast<const uint16_t*>(a.v_new) + (size_t(p.r) * a.n + q) * a.new_ld + size_t(h) * D + 16 * c;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float y = __uint_as_float(uint32_t(vr[i]) << 16);
                  if (!(fabsf(y) < INFINITY)) v[i] += y;
                }
              }
          }
          if (result) {
            if (has_o) {
              const float4* oo = so + size_t(kRows) * (D / 4) + size_t(4 * c) * kRows;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 y = __ldcg(oo + i * kRows);
                v[4 * i] = v[4 * i] * wa + y.x * wb;
                v[4 * i + 1] = v[4 * i + 1] * wa + y.y * wb;
                v[4 * i + 2] = v[4 * i + 2] * wa + y.z * wb;
                v[4 * i + 3] = v[4 * i + 3] * wa + y.w * wb;
              }
            }
            if (valid) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D) + 2 * c;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                dst[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                    pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
            }
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) so[(4 * c + i) * kRows] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        if (result) {
          if (valid && a.lse) a.lse[orow] = lse_of(M2, Ls);
        } else if (valid) {
          *sm = make_float2(fm, fl);
        } else {
          *sm = make_float2(-INFINITY, 0.f);
        }
        // (a unit that goes on in later CTAs is joined by the second kernel)
        if (tid == 0 && !complete && p.t == 0) {
          const long long Tk = *keep, ck = Tk < gridDim.x ? Tk : gridDim.x;  // (the tiles in all, and the CTAs that share them)
          args.begun[blockIdx.x] = make_int4(int(((f + p.Tr) * ck - 1) / Tk), p.r, p.j, 0);
        }
        if (local) mbar_arrive(bar(w == 1 ? kFragFull : kFragFree));
        tc_before();
        if (mine) mbar_arrive(bar(kOFree0 + w));  // the next piece may write O
      }
      if (!more) break;
      ct0 += n;
      f += n;
      p = pn;
      n = piece_tiles(p, f);
      const int rows = unit_rows(p.j);
      split = rows <= kRows, complete = p.t == 0 && n == p.Tr;
      const int stride = split ? 2 : 1, first = split ? w : 0;
      const int rg = row_of(p, r);
      h = p.j / args.blocks;
      valid = rg < M;
      node = valid ? rg / G : 0, head = h * G + (valid ? rg % G : 0);
      mine = first < n;
      m = -INFINITY, l = 0.f;
      const float xf = xf_next;
      mask = valid ? a.mask_bits[size_t(p.r) * a.n + node] & (~0ull >> (kTreeKeys - a.n)) : 0ull;
      nonfinite = 0;
      base = -1;
      pn.t += n - 1;
      if (f + n < E) advance(pn);
      const bool ask = f + n < E && has_tile(pn, f + n);
      if (!mine && ask) ask_q(pn);  // (no product reads it)
      // The reference m is moved, to a whole number, when a score would put P above
      // 2^(kPBaseLog2 + kLazyLog2); O and l are multiplied by that power of two,
      // exactly, once the products so far are complete.
      // A base that has been raised (to `now`) moves it too.
      auto move = [&](float mx, int now, bool o_live) {
        float fac = 1.f;
        if (now != base) {
          const int d = m > -INFINITY ? now - base : 0, by = raised_into_l(d, l);
          l *= ratio_scale(by);
          m -= float(by);
          fac = ratio_scale(by - d);
          base = now;
        }
        if (mx > m + kPBaseLog2) {
          const float mn = ceilf(mx) - kPBaseLog2, by = m == -INFINITY ? 0.f : ratio_scale(int(fmaxf(m - mn, -126.f)));
          l *= by;
          fac *= by;
          m = mn;
        }
        if (!o_live || !__any_sync(FULL, fac != 1.f)) return true;
        if (!__all_sync(FULL, mbar_wait(bar(kPvDone0 + 2 * w + ((cs - 1) & 1)), ((cs - 1) >> 1) & 1, abort_flag))) return false;
        tc_after();
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(to + 16 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac);
          tmem_st16(to + 16 * c, o);
        }
        tmem_st_wait();
        return true;
      };
      const int cs0 = cs;
      int t = first, hf = 0;
      while (t < n) {
        // One step: 64 keys (half of a history tile, or the tree tile); P goes over
        // scores that have been read.  A short loop: unrolled, or with the tree's
        // case inside, the roles' code outran the instruction caches and half of
        // the warps' time went to fetching it.
        const bool s_ok = mbar_wait(bar(kSFull0 + 2 * w + (cs & 1)), (cs >> 1) & 1, abort_flag);
        if (!__all_sync(FULL, s_ok)) {
          ok = false;
          break;
        }
        tc_after();
        const TileMeta& mt = metas[(ct0 + t) & 3];
        const bool tree = p.t + t == p.Tr - 1, last = tree || hf == 1;
        const uint32_t ts = tl + col_s(w, cs & 1);
        if (last && t + stride >= n && ask) ask_q(pn);  // every product that reads this piece's Q is complete
        if (!tree) {
          // The exponentials are taken against the reference as it is.  Their sum
          // tells whether P holds them (none is larger than the sum, and f16 goes
          // to 65504); in the rare case that it may not, the maximum is looked
          // for, the reference moves and the step is taken again.
#pragma unroll 1
          for (bool again = false;; again = true) {
            uint32_t u[kStep];
            tmem_ld32(ts, u);
            tmem_ld32(ts + 32, u + 32);
            const float mr = m == -INFINITY ? 0.f : m;
            float4 e[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) e[g] = mt.group[4 * hf + g];
            tmem_ld_wait();
            bool marked = false;
            if (e[0].w + e[1].w + e[2].w + e[3].w < float(kStep)) {
              marked = e[0].w < 0.f;
              e[0].w = keys_of(e[0].w);
#pragma unroll
              for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (float(i) >= e[g].w) u[16 * g + i] = 0xff800000u;
            }
            float all = 0.f, ls = 0.f;
            uint32_t pk[32];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float xk = xf * e[g].x, off = e[g].y - mr;
              const float2 k2 = make_float2(xk, xk), o2 = make_float2(off, off);
              float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 y = fma2(make_float2(__uint_as_float(u[16 * g + 2 * i]), __uint_as_float(u[16 * g + 2 * i + 1])), k2, o2);
                const float2 q = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                if (i & 1) s1 = add2(s1, q);
                else s0 = add2(s0, q);
                pk[8 * g + i] = pack_f16(q.x, q.y);
              }
              s0 = add2(s0, s1);
              all += s0.x + s0.y;
              ls = fmaf(s0.x + s0.y, e[g].z, ls);
            }
            if (again || __all_sync(FULL, all < kPMost && m > -INFINITY && !marked)) {
              l += ls;
              tmem_st32(ts, pk);
              break;
            }
            float mx = -INFINITY;
#pragma unroll 1
            for (int g = 0; g < kStep / kGroup; ++g) {
              uint32_t v[16];
              tmem_ld16(ts + 16 * g, v);
              const float4 eg = mt.group[4 * hf + g];
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (float(i) < keys_of(eg.w)) mx = fmaxf(mx, fmaf(__uint_as_float(v[i]), xf * eg.x, fmaxf(eg.y, -float(kSpanDown))));
            }
            const int now = mt.base;
            if ((now != base || __any_sync(FULL, mx > m + kPBaseLog2)) && !move(mx, now, cs > cs0)) {
              ok = false;
              break;
            }
            if (marked) {
#pragma unroll 1
              for (int g = 0; g < kStep / kGroup; ++g) {
                const float4 eg = mt.group[4 * hf + g];
                if (eg.z != 0.f) continue;
                uint32_t v[16];
                tmem_ld16(ts + 16 * g, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (float(i) < keys_of(eg.w)) l += fast_exp2(fmaf(__uint_as_float(v[i]), xf * eg.x, -m));
              }
            }
          }
        } else {
          // (the V rows' exponents come with V)
          if (!__all_sync(FULL, mbar_wait(bar(kVFull0 + ((ct0 + t) & 1)), ((ct0 + t) >> 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          nonfinite = mt.nonfinite[0] | mt.nonfinite[1] | mt.nonfinite[2] | mt.nonfinite[3];
          const int now = raised_base(base, max(max(mt.top[0], mt.top[1]), max(mt.top[2], mt.top[3])));
          const float b0 = float(now);
          // x + add of node k, from its word; chunk: the mask's bits from the chunk's first node on
          auto score = [&](uint32_t v, uint32_t word, uint32_t chunk, int i, float add) {
            const float x = fmaf(__uint_as_float(v), xf * bf16_lo(word), add);
            return chunk & (1u << i) ? x : -INFINITY;
          };
          // (against which m is set)
          auto most = [&](uint32_t v, uint32_t word, uint32_t chunk, int i) { return score(v, word, chunk, i, fmaxf(bf16_hi(word) - b0, -float(kSpanDown))); };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kTreeKeys / 16; ++c) {
            uint32_t v[16];
            tmem_ld16(ts + 16 * c, v);
            const uint32_t bits = uint32_t(mask >> (16 * c));
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 wd = *reinterpret_cast<const uint4*>(mt.node + 16 * c + 4 * q);
              mx = fmaxf(mx, fmaxf(most(v[4 * q], wd.x, bits, 4 * q), most(v[4 * q + 1], wd.y, bits, 4 * q + 1)));
              mx = fmaxf(mx, fmaxf(most(v[4 * q + 2], wd.z, bits, 4 * q + 2), most(v[4 * q + 3], wd.w, bits, 4 * q + 3)));
            }
          }
          if (now != base || __any_sync(FULL, mx > m + (kLazyLog2 + kPBaseLog2))) ok = move(mx, now, cs > cs0);
          const float mr = m == -INFINITY ? 0.f : m, bm = b0 + mr;  // (whole numbers)
#pragma unroll 1
          for (int c = 0; ok && c < kTreeKeys / 16; ++c) {
            uint32_t v[16], pk[8];
            tmem_ld16(ts + 16 * c, v);
            const uint32_t bits = uint32_t(mask >> (16 * c));
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 wd = *reinterpret_cast<const uint4*>(mt.node + 16 * c + 4 * q);
              auto p_of = [&](uint32_t vv, uint32_t word, int i) {
                l += fast_exp2(score(vv, word, bits, i, -mr));
                return fast_exp2(score(vv, word, bits, i, bf16_hi(word) - bm));
              };
              const float q0 = p_of(v[4 * q], wd.x, 4 * q), q1 = p_of(v[4 * q + 1], wd.y, 4 * q + 1);
              const float q2 = p_of(v[4 * q + 2], wd.z, 4 * q + 2), q3 = p_of(v[4 * q + 3], wd.w, 4 * q + 3);
              pk[2 * q] = pack_f16(q0, q1);
              pk[2 * q + 1] = pack_f16(q2, q3);
            }
            tmem_st8(ts + 8 * c, pk);
          }
        }
        if (!ok) break;
        tmem_st_wait();
        tc_before();
        mbar_arrive(bar(kPReady0 + 2 * w + (cs & 1)));
        ++cs;
        hf = last ? 0 : 1;
        t += last ? stride : 0;
      }
      if (!ok) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && !*abort_flag) fail();
  }

  // ---- teardown ----
  tc_before();
  __syncthreads();
  if (warp == 16) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Joins the units that the kernel above left in fragments: block (c, slice) 32 rows
// of the unit that CTA c began and did not finish, a lane a row, an eighth of
// the columns a warp.  A launch of its own, because it wants the whole GPU: the last
// CTA of a unit, alone and with hardly any L1 beside its operands, took 23 us for
// the trees' 1.2 MB and 54 us for the long contexts'.
constexpr int kJoinThreads = 256, kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) attention_q8_join_kernel(const __grid_constant__ TcArgs args) {
  pdl_wait();
  pdl_trigger();
  const AttentionQ8Params& a = args.p;
  const int ca = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 unit = args.begun[ca];
  const int cb = unit.x, r = unit.y, j = unit.z;
  if (cb < 0) return;
  const int G = a.Hq / a.Hkv, M = a.n * G;
  const int rows = min(2 * kRows, M - 2 * kRows * (j % args.blocks)), h = j / args.blocks;
  const bool split = rows <= kRows;
  const int row = blockIdx.y * kJoinRows + lane;
  if (row >= rows) return;
  const int nf = (cb - ca + 1) * (split ? 2 : 1);
  auto at = [&](int y) {
    const int cta = ca + (split ? y >> 1 : y);
    return size_t(2 * cta + (cta == ca ? 1 : 0)) * 2 + (split ? y & 1 : row / kRows);
  };
  const float2* ml2 = reinterpret_cast<const float2*>(args.slot_ml) + row % kRows;
  float Mx = -INFINITY, Ls = 0.f;
  // (fragments two at a time: with four, fewer blocks fit a SM, and the trees take 111 us, not 97)
  constexpr int kAtOnce = 2;
#pragma unroll 1
  for (int y0 = 0; y0 < nf; y0 += 2 * kAtOnce) {
    float2 ml[2 * kAtOnce];
#pragma unroll
    for (int y = 0; y < 2 * kAtOnce; ++y) ml[y] = y0 + y < nf ? __ldcg(ml2 + at(y0 + y) * kRows) : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int y = 0; y < 2 * kAtOnce; ++y) {
      const bool has = ml[y].y > 0.f || ml[y].y != ml[y].y;  // (else it saw nothing, and its O is not read)
      const float M2 = has ? fmaxf(Mx, ml[y].x) : Mx;
      const float wa = Ls > 0.f || Ls != Ls ? exp2f(Mx - M2) : 0.f;
      Ls = has ? Ls * wa + ml[y].y * exp2f(ml[y].x - M2) : Ls;
      Mx = M2;
    }
  }
  const float inv = settled_inverse(Ls);
  constexpr int C4 = D / 4, C = C4 / (kJoinThreads / 32);  // 16-byte words a thread
  const int c = warp * C;
  float4 acc[C];
#pragma unroll
  for (int e = 0; e < C; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int y0 = 0; y0 < nf; y0 += kAtOnce) {
    float4 o4[kAtOnce][C];
    float2 ml[kAtOnce];
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      ml[y] = make_float2(-INFINITY, 0.f);
      if (y0 + y < nf) {
        const size_t slot = at(y0 + y);
        const float4* src = reinterpret_cast<const float4*>(args.slot_o) + (slot * C4 + c) * kRows + row % kRows;
        ml[y] = __ldcg(ml2 + slot * kRows);
#pragma unroll
        for (int e = 0; e < C; ++e) o4[y][e] = __ldcg(src + e * kRows);
      }
    }
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y)
      if (ml[y].y > 0.f || ml[y].y != ml[y].y) {
        const float k = exp2f(ml[y].x - Mx) * inv;
#pragma unroll
        for (int e = 0; e < C; ++e) {
          acc[e].x = fmaf(o4[y][e].x, k, acc[e].x);
          acc[e].y = fmaf(o4[y][e].y, k, acc[e].y);
          acc[e].z = fmaf(o4[y][e].z, k, acc[e].z);
          acc[e].w = fmaf(o4[y][e].w, k, acc[e].w);
        }
      }
  }
  const int rg = 2 * kRows * (j % args.blocks) + row;
  const size_t orow = (size_t(r) * a.n + rg / G) * a.Hq + h * G + rg % G;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * c);
#pragma unroll
  for (int e = 0; e < C; e += 2)
    dst[e / 2] = make_uint4(pack_bf16x2(acc[e].x, acc[e].y), pack_bf16x2(acc[e].z, acc[e].w),
                            pack_bf16x2(acc[e + 1].x, acc[e + 1].y), pack_bf16x2(acc[e + 1].z, acc[e + 1].w));
  if (warp == 0 && a.lse) a.lse[orow] = lse_of(Mx, Ls);
}

template <int D>
int launch_tc(const AttentionQ8Params& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return SPEC_ERR_LAUNCH;
  // the register split assumes what the CTA is launched with (the build checks it, too)
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, attention_q8_tc_kernel<D>) != cudaSuccess || attr.numRegs != kRegs) return SPEC_ERR_LAUNCH;
  // at least 120 KB, so that two CTAs never share a SM (each holds all of TMEM)
  size_t smem = TcSmem<D>::kBytes + 1024;
  if (smem < 120 * 1024) smem = 120 * 1024;
  if (cudaFuncSetAttribute(attention_q8_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
    return SPEC_ERR_LAUNCH;
  TcArgs args{p, (p.n * (p.Hq / p.Hkv) + 2 * kRows - 1) / (2 * kRows),
              reinterpret_cast<int4*>(p.partials + kQ8SlotMlBytes - kQ8BegunBytes),
              reinterpret_cast<float*>(p.partials + kQ8SlotMlBytes), reinterpret_cast<float*>(p.partials)};
  const int grid = sms < kQ8MaxCtas ? sms : kQ8MaxCtas;
  const cudaError_t e = launch_pdl(attention_q8_tc_kernel<D>, dim3(grid), dim3(kTcThreads), smem, stream, args);
  if (e != cudaSuccess) return SPEC_ERR_LAUNCH;
  const dim3 join(unsigned(grid), 2 * kRows / kJoinRows);
  return launch_pdl(attention_q8_join_kernel<D>, join, dim3(kJoinThreads), 0, stream, args) == cudaSuccess ? SPEC_OK
                                                                                                         : SPEC_ERR_LAUNCH;
}

}  // namespace

int launch_attention_q8_tc(const AttentionQ8Params& p, cudaStream_t stream) {
  return p.D == 128 ? launch_tc<128>(p, stream) : launch_tc<64>(p, stream);
}

}  // namespace spec
