// share_pages.cu -- pages of a cache held by several requests: forks, pages given
// back, and the pages in use moved to the lowest ids (tables only; copy_pages.cu
// moves what the pages hold).
//
// A page's count is its holders beyond the first, so what takes pages from the
// free list need not know of it: a fork adds one for each child, a release
// takes one off or, at zero, gives the page back.  Counts are changed by integer
// atomics and every list is ordered by prefix sums, so a call's results do not
// depend on the order in which its threads run.
//
// Bound: latency.  A step's forks and releases are some kB; the chain is lengths -> entries -> counts ->
// lists, dependent reads of about 1 us each.  What has to agree over the whole call (which of a page's holders
// gives it up first; how many pages lie before) is agreed within a cluster of CTAs by its barrier, so that a release is one
// launch and a compaction two.  In us: eight children of 1001 tokens 4 (two million slots of 64 children 9), their release 8;
// compaction of 17 thousand pages 11.
#include "common.cuh"
#include "kernels.cuh"

#include "cluster.cuh"
#include "share_pages.cuh"

namespace spec {

namespace {

constexpr int kForkThreads = 256;
constexpr int kClusterCtas = 8, kClusterThreads = 1024;

// ------------------------------------------------------------------- fork

// Child r: whole = len / page pages of the parent's row shared, one of its own behind them where len % page.
// The entries of all children, laid end to end, are shared out over the grid; a thread takes one.
__global__ void __launch_bounds__(kForkThreads) fork_pages_kernel(ForkParams a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int scan[];
  __shared__ int wsum[kForkThreads / 32];
  __shared__ SlotStage<kForkThreads> stage;
  int* pre = scan;             // [b + 1] entries before child r
  int* tails = pre + a.b + 1;  // [b + 1] pages of their own before child r
  const int tid = threadIdx.x;
  const bool report = blockIdx.x == 0;
  const int avail = *a.n_free;
  auto len_of = [&](int r, bool tell) {  // 0 for a child that gets nothing
    const int len = a.fork_lens[r], p = a.parents[r], c = a.children[r];
    const bool idx_ok = p >= 0 && p < a.req_rows && c >= 0 && c < a.req_rows && p != c;
    const bool len_ok = len >= 0 && len <= (long long)a.row_pages * a.page_size && (!a.req_to_token || len <= a.row_w);
    if (tell && !idx_ok) raise_error(a.error, SPEC_DEV_INDEX);
    if (tell && !len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
    return idx_ok && len_ok ? len : 0;
  };
  const int E = scan_counts<kForkThreads>(a.b, pre, wsum, [&](int r) { return pages_of(len_of(r, report), a.page_size); });
  const int T = scan_counts<kForkThreads>(a.b, tails, wsum, [&](int r) { return len_of(r, false) % a.page_size ? 1 : 0; });
  const bool fits = avail >= 0 && avail <= a.free_cap && T <= avail;
  if (tid == 0) {
    if (report && !fits) raise_error(a.error, SPEC_DEV_SPACE);
    // n_left may be n_free itself: it is written once every CTA has read that
    if (atom_add_acq_rel(a.counters) == gridDim.x - 1) {
      *a.n_left = fits ? avail - T : avail;
      *a.n_copies = fits ? T : 0;
      atomicExch(a.counters, 0u);
    }
  }
  if (!fits) return;
  for (int e0 = blockIdx.x * kForkThreads; e0 < E; e0 += gridDim.x * kForkThreads) {
    const int e = e0 + tid;
    int id = -1, count = 0;
    long long first = 0;
    if (e < E) {
      const int r = row_of_entry(pre, a.b, e), i = e - pre[r];
      const int len = a.fork_lens[r], child = a.children[r];
      const int theirs = a.page_table[(long long)a.parents[r] * a.row_pages + i];
      const bool ok = theirs >= 0 && theirs < a.num_pages;
      if (!ok) raise_error(a.error, SPEC_DEV_INDEX);
      if (i < len / a.page_size) {
        if (ok) {
          atomicAdd(a.share_counts + theirs, 1);
          id = theirs;
        }
      } else {
        const int j = tails[r], fresh = a.free_ids[avail - 1 - j];
        a.copy_src[j] = theirs;  // (a bad id is passed over by the copy)
        a.copy_dst[j] = fresh;
        if (fresh >= 0 && fresh < a.num_pages) id = fresh;
        else raise_error(a.error, SPEC_DEV_INDEX);
      }
      a.page_table[(long long)child * a.row_pages + i] = id;
      count = min(a.page_size, len - i * a.page_size);
      first = (long long)child * a.row_w + (long long)i * a.page_size;
    }
    if (a.req_to_token) write_slots<kForkThreads>(stage, a.req_to_token, first, id, count, a.page_size, a.vec_slots);
  }
}

// ---------------------------------------------------------------- release

// The occurrences (request, page) of the call, laid end to end, are cut into contiguous shares, one a CTA of the
// cluster, in rows of 1024.  note[p] = {times given up, -1 - the occurrence that speaks for the page}: times are counted by
// atomics, and whoever counts first speaks; a page is freed where more holders than its count give it up, and then its
// first occurrence speaks (by atomics, only where it is given up more than once).  So each page's count is stored once.
// Freed pages are pushed in descending order of occurrence: what alloc or fork took in one call goes back to where it was.
//   The page ids and what is known of them stay in registers for the first kKept rows of a share.
//   The CTAs meet four times.  Up to 16 are a cluster (16 of them where the device takes such); a call that may hold
// more occurrences than their registers is a cooperative launch over all SMs, as a SM's scattered accesses to the
// notes, one a cycle, are what a large call costs, and its CTAs meet at a counter.  In us, cluster of 16 / all SMs:
// 133 thousand pages 43 / 19, 328 thousand of 32 holders each 103 / 31 (its atomics meet at the same words);
// a few hundred pages: cluster of 8 8, all SMs 15 (a cooperative launch by itself costs 7).
constexpr int kKept = 8;
constexpr int kClusterMost = 16;
constexpr int kReleaseMostCtas = 192;
constexpr long long kBarrierCycles = 4000000000ll;  // about 2 s: bound of a wait for the other CTAs

// All CTAs of a cooperative launch, for the round-th time (from 1); what they wrote before is seen after.  False (in every
// thread) if they do not come.
__device__ __forceinline__ bool grid_sync(uint32_t* arrivals, uint32_t round, uint32_t* error) {
  __shared__ int s_ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t want = round * gridDim.x;
    bool ok = int(atom_add_acq_rel(arrivals) + 1 - want) >= 0;
    const long long start = clock64();
    while (!ok && clock64() - start <= kBarrierCycles) {
      uint32_t now;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(arrivals) : "memory");
      ok = int(now - want) >= 0;
    }
    if (!ok) raise_error(error, SPEC_DEV_TIMEOUT);
    s_ok = ok;
  }
  __syncthreads();
  return s_ok;
}
// Each CTA, once, behind its last meeting: the last of them takes the arrivals back to zero, wherever the meetings ended (the
// count of those that left wraps by itself).
__device__ __forceinline__ void grid_leave(uint32_t* counters) {
  if (threadIdx.x != 0) return;
  uint32_t before;
  asm volatile("atom.inc.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(counters + 1), "r"(gridDim.x - 1) : "memory");
  if (before == gridDim.x - 1) atomicExch(counters, 0u);
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kClusterThreads) release_pages_kernel(ReleaseParams a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ long long row_at[];  // [b] where the request's first page given up lies in page_table
  int* pre = reinterpret_cast<int*>(row_at + a.b);  // [b + 1]
  __shared__ int wsum[kClusterThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, me = blockIdx.x, ctas = gridDim.x;
  const int n_free = *a.n_free;
  uint32_t met = 0;
  auto meet = [&] {
    if (CLUSTER) {
      cluster_sync();
      return true;
    }
    const bool all = grid_sync(a.counters, ++met, a.error);
    if (!all || met == 4) grid_leave(a.counters);
    return all;
  };
  const int E = scan_counts<kClusterThreads>(a.b, pre, wsum, [&](int r) {
    const int len = a.seq_lens[r], keep = a.keep_lens ? a.keep_lens[r] : 0, row = a.req_pool_idx[r];
    const bool idx_ok = row >= 0 && row < a.req_rows;
    const bool len_ok = keep >= 0 && keep <= len && len <= (long long)a.row_pages * a.page_size;
    if (me == 0 && !idx_ok) raise_error(a.error, SPEC_DEV_INDEX);
    if (me == 0 && !len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
    if (!idx_ok || !len_ok) return 0;
    const int first = pages_of(keep, a.page_size);
    row_at[r] = (long long)row * a.row_pages + first;
    return pages_of(len, a.page_size) - first;
  });
  const int lo = int((long long)E * me / ctas), hi = int((long long)E * (me + 1) / ctas);
  const int rows = (hi - lo + kClusterThreads - 1) / kClusterThreads;
  auto page_at = [&](int e) {  // -1 for a bad one, or none
    if (e >= hi) return -1;
    const int r = row_of_entry(pre, a.b, e);
    const int p = __ldg(a.page_table + row_at[r] + (e - pre[r]));
    if (p >= 0 && p < a.num_pages) return p;
    raise_error(a.error, SPEC_DEV_INDEX);
    return -1;
  };
  int kept[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) kept[i] = page_at(lo + i * kClusterThreads + tid);
  // fn(occurrence, page) for the thread's other pages
  auto for_others = [&](auto&& fn) {
    for (int i0 = kKept; i0 < rows; i0 += kKept) {
      int p[kKept];
#pragma unroll
      for (int i = 0; i < kKept; ++i) p[i] = page_at(lo + (i0 + i) * kClusterThreads + tid);
#pragma unroll
      for (int i = 0; i < kKept; ++i)
        if (p[i] >= 0) fn(lo + (i0 + i) * kClusterThreads + tid, p[i]);
    }
  };
  auto occurrence = [&](int i) { return lo + i * kClusterThreads + tid; };
  // (in order, where that takes fewer stores of a warp)
  if (!CLUSTER && a.num_pages / 8 < E) {
    for (long long p = me * kClusterThreads + tid; p < a.num_pages; p += ctas * kClusterThreads) a.note[p] = make_int2(0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < kKept; ++i)
      if (kept[i] >= 0) a.note[kept[i]].x = 0;
    for_others([&](int, int p) { a.note[p].x = 0; });
  }
  if (!meet()) return;
  unsigned speaks = 0, freed = 0;  // bits: of the kept rows
  int x[kKept], y[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) x[i] = kept[i] >= 0 ? atomicAdd(&a.note[kept[i]].x, 1) : 1;
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (x[i] == 0) {
      a.note[kept[i]].y = -1 - occurrence(i);
      speaks |= 1u << i;
    }
  for_others([&](int e, int p) {
    if (atomicAdd(&a.note[p].x, 1) == 0) a.note[p].y = -1 - e;
  });
  if (!meet()) return;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    x[i] = kept[i] >= 0 ? __ldcg(&a.note[kept[i]].x) : 0;
    y[i] = kept[i] >= 0 ? a.share_counts[kept[i]] : 0;
  }
  auto give_up = [&](int e, int p, int times, int more) {
    if (times <= more) return false;
    if (times > 1) atomicMax(&a.note[p].y, -1 - e);
    if (times > more + 1) raise_error(a.error, SPEC_DEV_INVARIANT);
    return true;
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    if (give_up(occurrence(i), kept[i], x[i], y[i])) freed |= 1u << i;
    y[i] = max(0, y[i] - x[i]);  // (what its count will be)
  }
  for_others([&](int e, int p) { give_up(e, p, __ldcg(&a.note[p].x), a.share_counts[p]); });
  if (!meet()) return;
  // counts are not touched before the list is known to have room
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kKept; ++i) x[i] = freed >> i & 1 ? __ldcg(&a.note[kept[i]].y) : 0;
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (freed >> i & 1) {
      const bool first = x[i] == -1 - occurrence(i);
      mine += first;
      speaks = first ? speaks | 1u << i : speaks & ~(1u << i);
    }
  for_others([&](int e, int p) {
    if (__ldcg(&a.note[p].y) == -1 - e) mine += __ldcg(&a.note[p].x) > a.share_counts[p];
  });
  mine = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();
  if (lane == 0) wsum[w] = mine;
  __syncthreads();
  if (w == 0) {
    const int sum = __reduce_add_sync(0xffffffffu, wsum[lane]);
    if (lane == 0) a.totals[me] = sum;
  }
  if (!meet()) return;
  int total = 0, at = n_free;  // `at`: where the next page of this share goes
  {
    __syncthreads();
    int c[kReleaseMostCtas / 32];  // (each warp adds them up by itself)
    int behind = 0;
#pragma unroll
    for (int i = 0; i < kReleaseMostCtas / 32; ++i) {
      const int q = 32 * i + lane;
      c[i] = q < ctas ? __ldcg(a.totals + q) : 0;
      total += c[i];
      behind += q > me ? c[i] : 0;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    at += __reduce_add_sync(0xffffffffu, behind);
    mine = __ldcg(a.totals + me);
  }
  const bool fits = n_free >= 0 && n_free <= a.free_cap && total <= a.free_cap - n_free;
  if (me == 0 && tid == 0) {
    if (!fits) raise_error(a.error, SPEC_DEV_SPACE);
    *a.n_left = fits ? n_free + total : n_free;
  }
  if (!fits) return;
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (speaks >> i & 1) a.share_counts[kept[i]] = y[i];
  for (int i = rows - 1; i >= 0; --i) {
    const int e = lo + i * kClusterThreads + tid;
    int p = -1;
    bool go = false;
    if (i < kKept) {
#pragma unroll
      for (int q = 0; q < kKept; ++q)
        if (q == i) p = kept[q];
      go = speaks >> i & freed >> i & 1;
    } else {
      p = page_at(e);
      if (p >= 0 && __ldcg(&a.note[p].y) == -1 - e) {
        const int times = __ldcg(&a.note[p].x), more = a.share_counts[p];
        go = times > more;
        a.share_counts[p] = max(0, more - times);
      }
    }
    if (mine == 0) continue;  // (the CTA frees nothing)
    const unsigned m = __ballot_sync(0xffffffffu, go);
    __syncthreads();
    if (lane == 0) wsum[w] = __popc(m);
    __syncthreads();
    const int n = wsum[lane];  // (as many warps as lanes)
    const int behind = __reduce_add_sync(0xffffffffu, lane > w ? n : 0);
    if (go) a.free_ids[at + behind + __popc(m & ~((2u << lane) - 1u))] = p;
    at += __reduce_add_sync(0xffffffffu, n);
  }
}

// ---------------------------------------------------------------- compact

// Plan: the free list as a bitmap; every page below `limit` that is free is a hole, every one at or above it that
// is not is moved: the i-th moved page to the i-th hole, both ascending.  pre_hole / pre_live: holes and
// moved pages before each word of the bitmap, from which the second kernel finds any page's new id.
__global__ void __launch_bounds__(kClusterThreads) compact_plan_kernel(CompactParams a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int wsum[3][kClusterThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, me = blockIdx.x;
  const int N = int(a.num_pages), W = (N + 31) / 32;
  const int gid = me * kClusterThreads + tid;
  constexpr int kAll = kClusterCtas * kClusterThreads, kAhead = 4;
  int ahead[kAhead];  // (read before it is known how many of them count)
#pragma unroll
  for (int k = 0; k < kAhead; ++k) ahead[k] = gid + k * kAll < a.free_cap ? a.free_ids[gid + k * kAll] : -1;
  const int n_free = *a.n_free;
  const bool ok = n_free >= 0 && n_free <= a.free_cap;
  if (!ok) {  // (every CTA of the cluster)
    if (me == 0 && tid == 0) {
      raise_error(a.error, SPEC_DEV_SPACE);
      *a.plan = make_int4(0, 0, 0, 0);
      *a.n_left = n_free;
      *a.n_moves = 0;
    }
    return;
  }
  for (int i = gid; i < W; i += kAll) a.bits[i] = 0;
  cluster_sync();
  // the sums over the CTA's threads, in every thread
  auto block_sum = [&](int x, int y, int z) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    z = __reduce_add_sync(0xffffffffu, z);
    __syncthreads();
    if (lane == 0) {
      wsum[0][w] = x;
      wsum[1][w] = y;
      wsum[2][w] = z;
    }
    __syncthreads();
    return make_int3(__reduce_add_sync(0xffffffffu, wsum[0][lane]), __reduce_add_sync(0xffffffffu, wsum[1][lane]),
                     __reduce_add_sync(0xffffffffu, wsum[2][lane]));
  };
  auto mark = [&](int p) {
    if (p < 0 || p >= N) {
      raise_error(a.error, SPEC_DEV_INDEX);
    } else if (atomicOr(a.bits + (p >> 5), 1u << (p & 31)) >> (p & 31) & 1u) {
      raise_error(a.error, SPEC_DEV_INVARIANT);  // listed twice
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (gid + k * kAll < n_free) mark(ahead[k]);
  for (int i = gid + kAhead * kAll; i < n_free; i += kAll) mark(a.free_ids[i]);
  cluster_sync();
  // Each CTA counts for itself what lies in the whole bitmap, which takes less time than another meeting.
  int set = 0;
  for (int i = tid; i < W; i += kClusterThreads) set += __popc(__ldcg(a.bits + i));
  const int free_pages = block_sum(set, 0, 0).x;
  const int live = N - free_pages, limit = int(a.limit > live ? a.limit < N ? a.limit : N : live);
  // words of this CTA; a word's holes below the limit and moved pages from it on
  const int lo = int((long long)W * me / kClusterCtas), hi = int((long long)W * (me + 1) / kClusterCtas);
  auto parts = [&](int i, unsigned& hole, unsigned& moved) {
    const unsigned f = __ldcg(a.bits + i);
    const int under = limit - 32 * i, real = N - 32 * i;
    const unsigned below = under >= 32 ? ~0u : under <= 0 ? 0u : (1u << under) - 1u;
    const unsigned exists = real >= 32 ? ~0u : (1u << real) - 1u;
    hole = f & below;
    moved = ~f & ~below & exists;
  };
  int holes = 0, moved = 0, all_moved = 0;
  for (int i = tid; i < W; i += kClusterThreads) {
    unsigned h, m;
    parts(i, h, m);
    all_moved += __popc(m);
    if (i < lo) {
      holes += __popc(h);
      moved += __popc(m);
    }
  }
  const int3 sums = block_sum(holes, moved, all_moved);
  const int M = sums.z;
  int at_hole = sums.x, at_live = sums.y;
  if (me == 0 && tid == 0) {
    *a.plan = make_int4(1, limit, M, free_pages);
    *a.n_left = free_pages;
    *a.n_moves = M;
  }
  for (int i0 = lo; i0 < hi; i0 += kClusterThreads) {
    const int i = i0 + tid;
    unsigned h = 0, m = 0;
    if (i < hi) parts(i, h, m);
    int ch = __popc(h), cm = __popc(m), ih = ch, im = cm;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ih, o), z = __shfl_up_sync(0xffffffffu, im, o);
      if (lane >= o) {
        ih += y;
        im += z;
      }
    }
    __syncthreads();
    if (lane == 31) {
      wsum[0][w] = ih;
      wsum[1][w] = im;
    }
    __syncthreads();
    int bh = at_hole + ih - ch, bm = at_live + im - cm;
#pragma unroll
    for (int q = 0; q < kClusterThreads / 32; ++q) {
      if (q < w) {
        bh += wsum[0][q];
        bm += wsum[1][q];
      }
      at_hole += wsum[0][q];
      at_live += wsum[1][q];
    }
    if (i < hi) {
      a.pre_hole[i] = bh;
      a.pre_live[i] = bm;
      for (; h; h &= h - 1, ++bh) {
        const int p = 32 * i + __ffs(h) - 1;
        if (bh < M) a.move_dst[bh] = p;
        else a.new_free_ids[free_pages - 1 - (bh - M)] = p;  // a hole that stays: the lowest are handed out first
      }
      for (; m; m &= m - 1, ++bm) a.move_src[bm] = 32 * i + __ffs(m) - 1;
    }
  }
}

// The tables, slots, counts and the rest of the free list after the plan.  Each value has one thread, so that
// every output may be its input.  What the plan does not write is read while it runs: its CTAs let this kernel start once
// what came before the call is done.
__global__ void __launch_bounds__(kForkThreads) compact_tables_kernel(CompactParams a) {
  extern __shared__ int pre[];  // [b + 1]
  __shared__ int wsum[kForkThreads / 32];
  __shared__ SlotStage<kForkThreads> stage;
  const int tid = threadIdx.x, N = int(a.num_pages);
  auto pages_in = [&](int r, bool tell) {
    const int len = a.seq_lens[r], row = a.req_pool_idx[r];
    const bool idx_ok = row >= 0 && row < a.req_rows;
    const bool len_ok = len >= 0 && len <= (long long)a.row_pages * a.page_size && (!a.req_to_token || len <= a.row_w);
    if (tell && !idx_ok) raise_error(a.error, SPEC_DEV_INDEX);
    if (tell && !len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
    return idx_ok && len_ok ? pages_of(len, a.page_size) : 0;
  };
  const int E = scan_counts<kForkThreads>(a.b, pre, wsum, [&](int r) { return pages_in(r, false); });
  // of the thread's entry: its place in the row, the row, the request's length, the page
  int i = 0, row = 0, len = 0, id = -1;
  auto look = [&](int e) {
    if (e >= E) return;
    const int r = row_of_entry(pre, a.b, e);
    i = e - pre[r];
    row = a.req_pool_idx[r];
    len = a.seq_lens[r];
    id = a.page_table[(long long)row * a.row_pages + i];
  };
  look(blockIdx.x * kForkThreads + tid);
  pdl_wait();
  pdl_trigger();
  const int4 plan = *a.plan;
  const int limit = plan.y, M = plan.z, free_pages = plan.w;
  if (!plan.x) return;
  if (blockIdx.x == 0)
    for (int r = tid; r < a.b; r += kForkThreads) pages_in(r, true);
  for (int e0 = blockIdx.x * kForkThreads; e0 < E; e0 += gridDim.x * kForkThreads) {
    const bool on = e0 + tid < E;
    int count = 0;
    long long first = 0;
    if (on) {
      if (id < 0 || id >= N) {
        raise_error(a.error, SPEC_DEV_INDEX);
        id = -1;
      } else {
        const unsigned f = a.bits[id >> 5];
        if (f >> (id & 31) & 1u) {  // in use, but on the free list (below the limit it may be another page's place now)
          raise_error(a.error, SPEC_DEV_INVARIANT);
        } else if (id >= limit) {
          const int from = max(limit, id & ~31), at = a.pre_live[id >> 5];
          id = a.move_dst[at + __popc(~f & ((1u << (id & 31)) - 1u) & ~((1u << (from & 31)) - 1u))];
        }
      }
      a.new_page_table[(long long)row * a.row_pages + i] = id;
      count = min(a.page_size, len - i * a.page_size);
      first = (long long)row * a.row_w + (long long)i * a.page_size;
    }
    if (a.req_to_token) write_slots<kForkThreads>(stage, a.new_req_to_token, first, id, count, a.page_size, a.vec_slots);
    look(e0 + gridDim.x * kForkThreads + tid);
  }
  const int stride = gridDim.x * kForkThreads, gid = blockIdx.x * kForkThreads + tid;
  for (int i = gid; i < M; i += stride) {
    const int src = a.move_src[i], dst = a.move_dst[i], c = a.share_counts[src];
    a.new_share_counts[dst] = c;
    a.new_share_counts[src] = 0;
  }
  for (int p = gid; p < N; p += stride) {
    const unsigned f = a.bits[p >> 5], bit = 1u << (p & 31);
    const bool moved = p >= limit && !(f & bit);
    const bool filled = p < limit && (f & bit) && a.pre_hole[p >> 5] + __popc(f & (bit - 1u)) < M;
    if (!moved && !filled) a.new_share_counts[p] = a.share_counts[p];
  }
  for (int j = gid; j < N - limit && j < free_pages; j += stride) a.new_free_ids[j] = N - 1 - j;
}

int entry_ctas(long long entries) {
  const long long g = (entries + kForkThreads - 1) / kForkThreads;
  return int(g < 1 ? 1 : g > kTargetCtas ? kTargetCtas : g);
}

// (the most, so that calls of two threads agree)
template <typename K>
bool allow_smem(K kernel, size_t bytes, size_t most) {
  return bytes <= 16 * 1024 || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most)) == cudaSuccess;
}

}  // namespace

int launch_fork_pages(const ForkParams& p, cudaStream_t stream) {
  auto bytes = [](int b) { return size_t(b + 1) * 8; };
  if (!allow_smem(fork_pages_kernel, bytes(p.b), bytes(kAllocMaxB))) return SPEC_ERR_LAUNCH;
  const cudaError_t e = launch_pdl(fork_pages_kernel, dim3(entry_ctas((long long)p.b * p.row_pages)), dim3(kForkThreads), bytes(p.b), stream, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int launch_release_pages(const ReleaseParams& p, cudaStream_t stream) {
  auto bytes = [](int b) { return size_t(b + 1) * 12; };
  const size_t smem = bytes(p.b);
  const long long most = ((long long)p.b * p.row_pages + kKept * kClusterThreads - 1) / (kKept * kClusterThreads);
  if (most > kClusterMost) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        !allow_smem(release_pages_kernel<false>, smem, bytes(kAllocMaxB)))
      return SPEC_ERR_LAUNCH;
    const int ctas = sms < kReleaseMostCtas ? sms : kReleaseMostCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, release_pages_kernel<false>, p) == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
  }
  if (!allow_smem(release_pages_kernel<true>, smem, bytes(kAllocMaxB))) return SPEC_ERR_LAUNCH;
  const int ctas = most > kClusterCtas && cudaFuncSetAttribute(release_pages_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess
                       ? kClusterMost
                       : kClusterCtas;
  return launch_cluster(release_pages_kernel<true>, ctas, dim3(ctas), dim3(kClusterThreads), smem, stream, p) == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int launch_compact_pages(const CompactParams& p, cudaStream_t stream) {
  auto bytes = [](int b) { return size_t(b + 1) * 4; };
  if (!allow_smem(compact_tables_kernel, bytes(p.b), bytes(kAllocMaxB))) return SPEC_ERR_LAUNCH;
  if (launch_cluster(compact_plan_kernel, kClusterCtas, dim3(kClusterCtas), dim3(kClusterThreads), 0, stream, p) != cudaSuccess)
    return SPEC_ERR_LAUNCH;
  const long long work = (long long)p.b * p.row_pages > p.num_pages ? (long long)p.b * p.row_pages : p.num_pages;
  const cudaError_t e = launch_pdl(compact_tables_kernel, dim3(entry_ctas(work)), dim3(kForkThreads), bytes(p.b), stream, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

size_t release_partial_bytes(long long pages) { return kReleaseTotalsBytes + align256(size_t(pages) * 8); }
size_t compact_partial_bytes(long long pages) { return 256 + 3 * align256(size_t(pages + 31) / 32 * 4); }

}  // namespace spec
