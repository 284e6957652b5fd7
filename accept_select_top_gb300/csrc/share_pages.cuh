// share_pages.cuh -- table rows laid end to end, for the kernels that walk the pages of many requests.
#pragma once

#include "common.cuh"

namespace spec {

// Exclusive prefix sums of count(r), r < b, into pre[0 .. b] (shared memory); the total.  Every thread of
// the CTA; wsum: one int a warp.
template <int THREADS, typename F>
__device__ __forceinline__ int scan_counts(int b, int* pre, int* wsum, F&& count) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int run = 0;
  for (int r0 = 0; r0 < b; r0 += THREADS) {
    const int r = r0 + tid, t = r < b ? count(r) : 0;
    int incl = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    int before = run;
#pragma unroll
    for (int q = 0; q < THREADS / 32; ++q) {
      if (q < w) before += wsum[q];
      run += wsum[q];
    }
    if (r < b) pre[r] = before + incl - t;
  }
  if (tid == 0) pre[b] = run;
  __syncthreads();
  return run;
}

// The request that holds entry e: the last r with pre[r] <= e (those without an entry are passed over).
__device__ __forceinline__ int row_of_entry(const int* pre, int b, int e) {
  int lo = 0, hi = b;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(int len, int page) { return int((unsigned(len) + unsigned(page) - 1u) / unsigned(page)); }

// The slots of up to THREADS pages, written by the whole CTA: thread t's page `id` holds `count` tokens (0: none)
// from slots[first].  Staged in shared memory so that the stores of a page lie side by side; whole pages go as
// 16-byte stores where every page of the table starts on one (`vec`).
template <int THREADS>
struct SlotStage {
  long long first[THREADS];
  int id[THREADS], count[THREADS];
};
template <int THREADS>
__device__ __forceinline__ void write_slots(SlotStage<THREADS>& s, int32_t* slots, long long first, int id, int count, int page,
                                            bool vec) {
  const int tid = threadIdx.x;
  __syncthreads();
  s.first[tid] = first;
  s.id[tid] = id;
  s.count[tid] = count;
  __syncthreads();
  const int per = vec ? page / 4 : page;
  for (int x = tid; x < THREADS * per; x += THREADS) {
    const int t = x / per, off = (x - t * per) * (vec ? 4 : 1), n = s.count[t], p = s.id[t];
    if (off >= n) continue;
    int32_t* to = slots + s.first[t] + off;
    const int v = p * page + off;
    if (vec && off + 4 <= n) {
      *reinterpret_cast<int4*>(to) = p < 0 ? make_int4(-1, -1, -1, -1) : make_int4(v, v + 1, v + 2, v + 3);
    } else {
      for (int i = 0; i < (vec ? 4 : 1) && off + i < n; ++i) to[i] = p < 0 ? -1 : v + i;
    }
  }
}

}  // namespace spec
