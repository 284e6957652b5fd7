// alloc_slots.cu -- pages for new tokens, taken from the free list on the GPU:
// block table entries, the slot table, the ragged slot map and positions.
//
// With L = seq_lens[r] tokens cached and m = new_lens[r] to come, request r
// needs the pages [ceil(L / P), ceil((L + m) / P)) of its table row.  Pages are
// handed out in request order, then page order: the j-th of the call is
// free_ids[n_free - 1 - j].  So the page of every new token follows from two
// exclusive prefix sums over the requests (tokens and pages) and no CTA waits
// on another: each CTA scans all the lengths into shared memory itself (12
// bytes a request, from L2) and then takes an equal share of the call's
// tokens, whatever the lengths are.  A thread takes four consecutive tokens (one
// 16-byte store each to the slot map and the positions): one binary search in
// the prefix sums, then steps.  The token that opens a page writes its table
// entry.
//
// Bound: a decode step writes a few kB and is launch and round-trip latency
// (lengths, then free ids, then the stores); a batch of prompts is the 8
// bytes a token of its stores.
#include "common.cuh"
#include "kernels.cuh"

namespace spec {

namespace {

constexpr int kAllocThreads = 256;
constexpr int kPerThread = 4;

__device__ __forceinline__ unsigned ceil_div(unsigned a, unsigned d) { return a / d + (a % d ? 1u : 0u); }

__global__ void __launch_bounds__(kAllocThreads) alloc_slots_kernel(AllocParams a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ long long scan[];
  constexpr int kAllocWarps = kAllocThreads / 32;
  long long* const wsum[2] = {scan, scan + kAllocWarps};
  int* cu = reinterpret_cast<int*>(scan + 2 * kAllocWarps);  // [b + 1] tokens before request r
  int* cp = cu + a.b + 1;                                    // [b + 1] pages before request r
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const unsigned P = unsigned(a.page_size);
  const bool report = blockIdx.x == 0;
  const int avail = *a.n_free;

  long long run_t = 0, run_p = 0;
  for (int r0 = 0; r0 < a.b; r0 += kAllocThreads) {
    const int r = r0 + tid;
    int t = 0, pg = 0;
    if (r < a.b) {
      const int L = a.seq_lens[r], m = a.new_lens[r], rq = a.req_pool_idx[r];
      const bool idx_ok = rq >= 0 && rq < a.req_rows;
      bool len_ok = L >= 0 && m >= 0 && m <= a.max_new && (long long)L + m <= (long long)a.row_pages * a.page_size;
      if (a.req_to_token && (long long)L + m > a.row_w) len_ok = false;
      if (report && !idx_ok) raise_error(a.error, SPEC_DEV_INDEX);
      if (report && !len_ok) raise_error(a.error, SPEC_DEV_LENGTH);
      if (idx_ok && len_ok) {  // (a request with a bad row or length gets no token)
        t = m;
        pg = int(ceil_div(unsigned(L) + unsigned(m), P) - ceil_div(unsigned(L), P));
      }
    }
    long long it = t, ip = pg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, it, o), z = __shfl_up_sync(0xffffffffu, ip, o);
      if (lane >= o) {
        it += y;
        ip += z;
      }
    }
    __syncthreads();
    if (lane == 31) {
      wsum[0][w] = it;
      wsum[1][w] = ip;
    }
    __syncthreads();
    long long bt = run_t, bp = run_p;
    for (int q = 0; q < kAllocWarps; ++q) {
      if (q < w) {
        bt += wsum[0][q];
        bp += wsum[1][q];
      }
      run_t += wsum[0][q];
      run_p += wsum[1][q];
    }
    // (32-bit prefix sums: totals past slot_cap are refused below)
    if (r < a.b) {
      cu[r] = int(bt + it - t);
      cp[r] = int(bp + ip - pg);
    }
  }
  const bool fits = avail >= 0 && avail <= a.free_cap && run_p <= avail && run_t <= a.slot_cap;
  const int T = fits ? int(run_t) : 0;
  if (tid == 0) {
    cu[a.b] = int(run_t);
    if (report && !fits) raise_error(a.error, SPEC_DEV_SPACE);
    // n_left may be n_free itself: it is written once every CTA has read that
    if (atom_add_acq_rel(a.counters) == gridDim.x - 1) {
      *a.n_left = fits ? avail - int(run_p) : avail;
      atomicExch(a.counters, 0u);
    }
  }
  __syncthreads();
  if (report)
    for (int r = tid; r <= a.b; r += kAllocThreads) a.cu_new[r] = fits ? cu[r] : 0;

  const int groups = (T + kPerThread - 1) / kPerThread;
  for (int gidx = blockIdx.x * kAllocThreads + tid; gidx < groups; gidx += gridDim.x * kAllocThreads) {
    const int t0 = gidx * kPerThread;
    int lo = 0, hi = a.b;  // the last request with cu[r] <= t0 holds t0 (those of no token are passed over)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= t0) lo = mid;
      else hi = mid;
    }
    int r = lo, end = cu[lo + 1];
    int L = a.seq_lens[r], row = a.req_pool_idx[r];
    int slot[kPerThread], pos[kPerThread];
    unsigned last_page = 0xffffffffu;
    int last_id = -1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int t = t0 + i;
      slot[i] = pos[i] = 0;
      if (t < T) {
        if (t >= end) {
          do {
            ++r;
            end = cu[r + 1];
          } while (t >= end);
          L = a.seq_lens[r];
          row = a.req_pool_idx[r];
          last_page = 0xffffffffu;
        }
        const unsigned x = unsigned(L) + unsigned(t - cu[r]);
        const unsigned page = x / P, off = x - page * P;
        if (page != last_page) {
          const unsigned first = ceil_div(unsigned(L), P);
          int32_t* entry = a.page_table + size_t(row) * a.row_pages + page;
          last_id = page >= first ? a.free_ids[avail - 1 - (cp[r] + int(page - first))] : *entry;
          if (last_id < 0 || last_id >= a.num_pages) {
            raise_error(a.error, SPEC_DEV_INDEX);
            last_id = -1;
          }
          if (page >= first && off == 0) *entry = last_id;
          last_page = page;
        }
        pos[i] = int(x);
        slot[i] = last_id < 0 ? -1 : int(unsigned(last_id) * P + off);
        if (a.req_to_token) a.req_to_token[size_t(row) * a.row_w + x] = slot[i];
      }
    }
    if (t0 + kPerThread <= T) {
      *reinterpret_cast<int4*>(a.slot_map + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int i = 0; t0 + i < T; ++i) {
        a.slot_map[t0 + i] = slot[i];
        a.positions[t0 + i] = pos[i];
      }
    }
  }
}

}  // namespace

int launch_alloc_slots(const AllocParams& p, cudaStream_t stream) {
  // (all of the kernel's shared memory is dynamic: 48 KB of it need no leave)
  auto bytes = [](int b) { return size_t(2) * (kAllocThreads / 32) * sizeof(long long) + size_t(2) * (b + 1) * 4; };
  const size_t smem = bytes(p.b);
  // (the most, so that calls of two threads agree)
  if (smem > 48 * 1024 && cudaFuncSetAttribute(alloc_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(bytes(kAllocMaxB))) != cudaSuccess)
    return SPEC_ERR_LAUNCH;
  // as many CTAs as the largest possible call has shares, up to four a SM
  const long long most = (long long)p.b * p.max_new < p.slot_cap ? (long long)p.b * p.max_new : p.slot_cap;
  long long grid = (most + kAllocThreads * kPerThread - 1) / (kAllocThreads * kPerThread);
  if (grid > kTargetCtas) grid = kTargetCtas;
  if (grid < 1) grid = 1;
  const cudaError_t e = launch_pdl(alloc_slots_kernel, dim3(unsigned(grid)), dim3(kAllocThreads), smem, stream, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace spec
