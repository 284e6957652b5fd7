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
// gives it up first; how many pages lie before) is agreed within one cluster of eight CTAs by its barrier,
// so that a release is one launch and a compaction two.
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

// The occurrences (request, page) of the call, laid end to end, are cut into eight contiguous shares, one a CTA of
// the cluster.  note[p] = {times given up, first occurrence} is cleared, then filled by atomics; a page is
// freed where more holders than its count give it up, by its first occurrence.  Freed pages are pushed in
// descending order of occurrence: what alloc or fork took in one call goes back to where it was.
__global__ void __launch_bounds__(kClusterThreads) release_pages_kernel(ReleaseParams a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int pre[];  // [b + 1]
  __shared__ int wsum[kClusterThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, me = blockIdx.x;
  const int n_free = *a.n_free;
  auto first_of = [&](int r) { return a.keep_lens ? pages_of(a.keep_lens[r], a.page_size) : 0; };
  const int E = scan_counts<kClusterThreads>(a.b, pre, wsum, [&](int r) {
    const int len = a.seq_lens[r], keep = a.keep_lens ? a.keep_lens[r] : 0, row = a.req_pool_idx[r];
    const bool idx_ok = row >= 0 && row < a.req_rows;
    const bool len_ok = keep >= 0 && keep <= len && len <= (long long)a.row_pages * a.page_size;
    if (me == 0 && !idx_ok) raise_error(a.error, SPEC_DEV_INDEX);
    if (me == 0 && !len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
    return idx_ok && len_ok ? pages_of(len, a.page_size) - pages_of(keep, a.page_size) : 0;
  });
  const int lo = int((long long)E * me / kClusterCtas), hi = int((long long)E * (me + 1) / kClusterCtas);
  auto page_at = [&](int e) {  // -1 for a bad one
    const int r = row_of_entry(pre, a.b, e);
    const int p = a.page_table[(long long)a.req_pool_idx[r] * a.row_pages + first_of(r) + e - pre[r]];
    return p >= 0 && p < a.num_pages ? p : -1;
  };
  for (int e = lo + tid; e < hi; e += kClusterThreads) {
    const int p = page_at(e);
    if (p >= 0) a.note[p] = make_int2(0, INT_MAX);
    else raise_error(a.error, SPEC_DEV_INDEX);
  }
  cluster_sync();
  for (int e = lo + tid; e < hi; e += kClusterThreads) {
    const int p = page_at(e);
    if (p >= 0) {
      atomicAdd(&a.note[p].x, 1);
      atomicMin(&a.note[p].y, e);
    }
  }
  cluster_sync();
  // whether occurrence e frees its page; counts are not touched before the list is known to have room
  auto frees = [&](int e, int& p, int& left) {
    p = page_at(e);
    if (p < 0) return false;
    const int2 n = __ldcg(a.note + p);
    if (n.y != e) {
      p = -1;
      return false;
    }
    left = a.share_counts[p] - n.x;
    return left < 0;
  };
  int mine = 0;
  for (int e = lo + tid; e < hi; e += kClusterThreads) {
    int p, left;
    mine += frees(e, p, left);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();
  if (lane == 0) wsum[w] = mine;
  __syncthreads();
  if (tid == 0) {
    int sum = 0;
    for (int q = 0; q < kClusterThreads / 32; ++q) sum += wsum[q];
    a.totals[me] = sum;
  }
  cluster_sync();
  int total = 0, at = n_free;  // where the next page of this share goes
  for (int q = 0; q < kClusterCtas; ++q) {
    const int c = __ldcg(a.totals + q);
    total += c;
    if (q > me) at += c;
  }
  const bool fits = n_free >= 0 && n_free <= a.free_cap && total <= a.free_cap - n_free;
  if (me == 0 && tid == 0) {
    if (!fits) raise_error(a.error, SPEC_DEV_SPACE);
    *a.n_left = fits ? n_free + total : n_free;
  }
  if (!fits) return;
  for (int h = hi; h > lo; h -= kClusterThreads) {
    const int e = h - 1 - tid;
    int p = -1, left = 0;
    const bool go = e >= lo && frees(e, p, left);
    if (p >= 0) {
      if (left < -1) raise_error(a.error, SPEC_DEV_INVARIANT);
      a.share_counts[p] = left < 0 ? 0 : left;
    }
    const unsigned m = __ballot_sync(0xffffffffu, go);
    __syncthreads();
    if (lane == 0) wsum[w] = __popc(m);
    __syncthreads();
    int before = at;
#pragma unroll
    for (int q = 0; q < kClusterThreads / 32; ++q) {
      if (q < w) before += wsum[q];
      at += wsum[q];
    }
    if (go) a.free_ids[before + __popc(m & ((1u << lane) - 1u))] = p;
  }
}

// ---------------------------------------------------------------- compact

// Plan: the free list as a bitmap; every page below `limit` that is free is a hole, every one at or above it that
// is not is moved: the i-th moved page to the i-th hole, both ascending.  pre_hole / pre_live: holes and
// moved pages before each word of the bitmap, from which the second kernel finds any page's new id.
__global__ void __launch_bounds__(kClusterThreads) compact_plan_kernel(CompactParams a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int wsum[2][kClusterThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, me = blockIdx.x;
  const int N = int(a.num_pages), W = (N + 31) / 32;
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
  const int gid = me * kClusterThreads + tid;
  for (int i = gid; i < W; i += kClusterCtas * kClusterThreads) a.bits[i] = 0;
  cluster_sync();
  auto block_sum = [&](int x, int y, int2* to) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    __syncthreads();
    if (lane == 0) {
      wsum[0][w] = x;
      wsum[1][w] = y;
    }
    __syncthreads();
    if (tid == 0) {
      int2 s = make_int2(0, 0);
      for (int q = 0; q < kClusterThreads / 32; ++q) {
        s.x += wsum[0][q];
        s.y += wsum[1][q];
      }
      *to = s;
    }
  };
  int set = 0;
  for (int i = gid; i < n_free; i += kClusterCtas * kClusterThreads) {
    const int p = a.free_ids[i];
    if (p < 0 || p >= N) {
      raise_error(a.error, SPEC_DEV_INDEX);
    } else if (atomicOr(a.bits + (p >> 5), 1u << (p & 31)) >> (p & 31) & 1u) {
      raise_error(a.error, SPEC_DEV_INVARIANT);  // listed twice
    } else {
      ++set;
    }
  }
  block_sum(set, 0, a.totals + me);
  cluster_sync();
  int free_pages = 0;
  for (int q = 0; q < kClusterCtas; ++q) free_pages += __ldcg(a.totals + q).x;
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
  int holes = 0, moved = 0;
  for (int i = lo + tid; i < hi; i += kClusterThreads) {
    unsigned h, m;
    parts(i, h, m);
    holes += __popc(h);
    moved += __popc(m);
  }
  block_sum(holes, moved, a.totals + kClusterCtas + me);
  cluster_sync();
  int at_hole = 0, at_live = 0, M = 0;
  for (int q = 0; q < kClusterCtas; ++q) {
    const int2 c = __ldcg(a.totals + kClusterCtas + q);
    M += c.y;
    if (q < me) {
      at_hole += c.x;
      at_live += c.y;
    }
  }
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
// every output may be its input.
__global__ void __launch_bounds__(kForkThreads) compact_tables_kernel(CompactParams a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int pre[];  // [b + 1]
  __shared__ int wsum[kForkThreads / 32];
  __shared__ SlotStage<kForkThreads> stage;
  const int tid = threadIdx.x, N = int(a.num_pages);
  const bool report = blockIdx.x == 0;
  const int4 plan = *a.plan;
  const int limit = plan.y, M = plan.z, free_pages = plan.w;
  if (!plan.x) return;
  const int E = scan_counts<kForkThreads>(a.b, pre, wsum, [&](int r) {
    const int len = a.seq_lens[r], row = a.req_pool_idx[r];
    const bool idx_ok = row >= 0 && row < a.req_rows;
    const bool len_ok = len >= 0 && len <= (long long)a.row_pages * a.page_size && (!a.req_to_token || len <= a.row_w);
    if (report && !idx_ok) raise_error(a.error, SPEC_DEV_INDEX);
    if (report && !len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
    return idx_ok && len_ok ? pages_of(len, a.page_size) : 0;
  });
  for (int e0 = blockIdx.x * kForkThreads; e0 < E; e0 += gridDim.x * kForkThreads) {
    const int e = e0 + tid;
    int id = -1, count = 0;
    long long first = 0;
    if (e < E) {
      const int r = row_of_entry(pre, a.b, e), i = e - pre[r], row = a.req_pool_idx[r];
      id = a.page_table[(long long)row * a.row_pages + i];
      if (id < 0 || id >= N) {
        raise_error(a.error, SPEC_DEV_INDEX);
        id = -1;
      } else if (id >= limit) {
        const unsigned f = a.bits[id >> 5];
        const int from = max(limit, id & ~31), at = a.pre_live[id >> 5];
        if (f >> (id & 31) & 1u) raise_error(a.error, SPEC_DEV_INVARIANT);  // in use, but on the free list
        else id = a.move_dst[at + __popc(~f & ((1u << (id & 31)) - 1u) & ~((1u << (from & 31)) - 1u))];
      }
      a.new_page_table[(long long)row * a.row_pages + i] = id;
      count = min(a.page_size, a.seq_lens[r] - i * a.page_size);
      first = (long long)row * a.row_w + (long long)i * a.page_size;
    }
    if (a.req_to_token) write_slots<kForkThreads>(stage, a.new_req_to_token, first, id, count, a.page_size, a.vec_slots);
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
  auto bytes = [](int b) { return size_t(b + 1) * 4; };
  if (!allow_smem(release_pages_kernel, bytes(p.b), bytes(kAllocMaxB))) return SPEC_ERR_LAUNCH;
  const cudaError_t e = launch_cluster(release_pages_kernel, kClusterCtas, dim3(kClusterCtas), dim3(kClusterThreads), bytes(p.b), stream, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
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

size_t release_partial_bytes(long long pages) { return 256 + align256(size_t(pages) * 8); }
size_t compact_partial_bytes(long long pages) { return 256 + 3 * align256(size_t(pages + 31) / 32 * 4); }

}  // namespace spec
