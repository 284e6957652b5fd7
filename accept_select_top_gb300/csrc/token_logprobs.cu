// token_logprobs.cu -- log probabilities of given tokens, entropy and the k best
// alternatives of verify rows, in one pass over the logits.
//
// With M the row's maximum and y = (x - M) c, c = log2(e) / T:
//   s = sum 2^y,  t = sum y 2^y,
//   log p(v) = (x_v - M) / T - ln 2 log2 s,  H = ln 2 (log2 s - t / s).
// The difference comes before the factor: x c alone would overflow for masks of
// the type's lowest value, and its rounding would not cancel.  log p has a factor of its
// own: of such a mask, y is past fp32's range where log p is not.
//
// A CTA takes one chunk of one row (a whole row when there are rows enough to
// fill the GPU).  A thread reads batches of 64 bytes a load group, 32 logits:
// the batch maximum first (kept in shared memory), then the exponentials
// relative to the thread's running maximum.  The k best come out of the batch
// maxima: the CTA's 256 threads form 32 groups (by lane, so that short rows
// fill all of them), and the k-th largest of the 32 group maxima is a value
// that at least k logits reach; only the batches whose
// maximum reaches it are read again (from L2), their logits that reach it are
// ranked by counting.  Rows need no alignment: the logits before a row's first
// 16-byte boundary and behind its last are one more batch.
//   The chunks of a row are a cluster: each leaves (M, s, t) and its k best in its
// shared memory, and the first CTA joins them.
//
// Bound: the logits' bytes, read once, for many rows: 1024 fp32 rows of 129280 with 20
// alternatives take 90 us (5.9 TB/s).  Few rows are latency: 32 requests' 224 rows of
// 128256 bf16 logits, about half of them counting, 15 us, of which the selection and
// the join take some 5; four rows of 50257 6.5 us (8.3 us where the chunks met through
// the workspace and an arrival counter).
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.cuh"

namespace spec {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxBatches = 16;  // of a chunk: at most 131072 logits
constexpr int kListCap = 512;    // batches read again, and logits ranked; more (long ties) take the slow path
constexpr int kLpCluster = 8;    // chunks of a row at most: a cluster of CTAs
constexpr long kLpCtas = 912;    // CTAs up to which rows are cut
constexpr int kJoinCap = 128;  // entries ranked when chunks are joined; more take the slow path

struct LpArgs {
  LogprobParams p;
  int chunks, vpc;  // chunks of a row, 16-byte vectors of a chunk
};
struct LpPart {
  float M, s, t;
  int count;
};

template <typename T>
struct LpRow {
  const T* row;
  int V, head, nvec, tail;
  __device__ LpRow(const void* logits, long long idx, int v) : V(v) {
    constexpr int E = VecOps<T>::E;
    row = static_cast<const T*>(logits) + idx * (long long)v;
    const int off = int(reinterpret_cast<uintptr_t>(row) & 15) / int(sizeof(T));
    head = off ? min(E - off, v) : 0;
    nvec = (v - head) / E;
    tail = v - head - nvec * E;
  }
  __device__ const uint4* vecs() const { return reinterpret_cast<const uint4*>(row + head); }
  // the element that thread t < head + tail holds of the edge batch
  __device__ int edge(int t) const { return t < head ? t : V - tail + (t - head); }
};

// (T is the output row's request's, whichever request's verify row it reads)
__device__ __forceinline__ float inverse_temperature(const LogprobParams& a, int out_row) {
  const float T = a.temperatures ? a.temperatures[out_row / a.W] : 1.f;
  return T > 0.f ? 1.f / T : 1.f;
}

// A row's token and its logit, read before the row's statistics are there.
struct LpToken {
  int tok;
  float x;
};
template <typename T>
__device__ __forceinline__ LpToken token_of(const LogprobParams& a, int tok, long long idx) {
  const bool on = idx >= 0 && tok >= 0 && tok < a.V;
  return LpToken{tok, on ? LogitTraits<T>::load(static_cast<const T*>(a.logits) + idx * (long long)a.V, tok) : -INFINITY};
}

// Results of one row from its joined statistics and its k best (count of them
// with a value above -inf, in order); one warp.
__device__ void finish_row(const LogprobParams& a, int out_row, LpToken token, float M, float s, float t,
                           float inv_t, int count, const float* tv, int* ti) {
  const int lane = threadIdx.x & 31;
  const float ls = log2f(s);
  auto logp = [&](float x) {
    // (1 / T may be inf: of the maximum itself, 0 / T is 0)
    return M == -INFINITY || !(x > -INFINITY) ? -INFINITY : (x == M ? x - M : (x - M) * inv_t) - ls * 0.6931471805599453f;
  };
  if (lane == 0) {
    float lp = 0.f;
    if (token.tok >= a.V) raise_error(a.error, SPEC_DEV_INDEX);
    else if (token.tok >= 0) lp = logp(token.x);
    a.logprobs[out_row] = lp;
    if (a.entropy) a.entropy[out_row] = M == -INFINITY ? 0.f : (ls - t / s) * 0.6931471805599453f;
  }
  if (a.k > 0) {
    const float best = lane < count ? logp(tv[lane]) : -INFINITY;
    // fewer than k logits above -inf: the lowest other indices follow
    for (int base = 0; count < a.k && base < a.V; base += 32) {
      const int i = base + lane;
      bool other = i < a.V;
      for (int q = 0; q < count; ++q) other = other && ti[q] != i;
      const unsigned who = __ballot_sync(0xffffffffu, other);
      const int at = count + __popc(who & ((1u << lane) - 1u));
      __syncwarp();
      if (other && at < a.k) ti[at] = i;
      count = min(a.k, count + __popc(who));
      __syncwarp();
    }
    if (lane < a.k) {
      a.top_ids[size_t(out_row) * a.k + lane] = ti[lane];
      a.top_logprobs[size_t(out_row) * a.k + lane] = best;
    }
  }
}

__device__ void blank_row(const LogprobParams& a, int out_row) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    a.logprobs[out_row] = 0.f;
    if (a.entropy) a.entropy[out_row] = 0.f;
  }
  if (lane < a.k) {
    a.top_ids[size_t(out_row) * a.k + lane] = -1;
    a.top_logprobs[size_t(out_row) * a.k + lane] = 0.f;
  }
}

// (four CTAs a SM for fp32: with five, the compiler's own choice of 48 registers, fewer loads are in
// flight, 99 against 91 us)
template <typename T>
__global__ void __launch_bounds__(kLpThreads, sizeof(T) == 4 ? 4 : 1) token_logprobs_kernel(LpArgs args) {
  constexpr int E = VecOps<T>::E, U = kBatch / E;
  const LogprobParams& a = args.p;
  __shared__ float bmax[kMaxBatches + 1][kLpThreads];
  __shared__ float gmax[kLpWarps][32], red[2][kLpWarps];
  __shared__ float cv[kListCap];
  __shared__ int ci[kListCap], list[kListCap];
  __shared__ int n_list, n_cand;
  __shared__ float inv_t;
  __shared__ float tv[2][kLogprobMaxK];  // the chunk's best, the row's
  __shared__ int ti[2][kLogprobMaxK];
  __shared__ __align__(16) LpPart part;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // (the first row of every request, then the second: where only some count, those start together)
  const int rw = blockIdx.x / args.chunks, ch = blockIdx.x % args.chunks, out_row = rw % a.b * a.W + rw / a.b;
  long long idx = a.row_index ? a.row_index[out_row] : (long long)(out_row / a.W) * a.n + out_row % a.W;
  if (idx >= (long long)a.b * a.n) {
    if (ch == 0 && tid == 0) raise_error(a.error, SPEC_DEV_INDEX);
    idx = -1;
  }
  if (idx < 0) {  // (the whole cluster)
    if (ch == 0 && w == 0) blank_row(a, out_row);
    return;
  }
  float M = -INFINITY, s = 0.f, t = 0.f, c = 0.f;
  int count = 0;
  {
    const float it = inverse_temperature(a, out_row);
    if (tid == 0) {
      n_list = n_cand = 0;
      inv_t = it;
    }
    c = fminf(1.4426950408889634f * it, 3.402823466e38f);  // (0 inf would be NaN)
    const LpRow<T> row(a.logits, idx, a.V);
    const uint4* vp = row.vecs();
    const int v0 = ch * args.vpc, v1 = min(row.nvec, v0 + args.vpc);
    const int nb = v1 > v0 ? (v1 - v0 + U * kLpThreads - 1) / (U * kLpThreads) : 0;
    // ---- one pass: batch maxima, running maximum, s and t ----
    float m = -INFINITY;
    auto raise = [&](float bm) {  // the thread's maximum moves to bm
      if (s > 0.f) {
        const float d = fmaxf((m - bm) * c, -150.f), f = fast_exp2(d);
        t = f * fmaf(d, s, t);
        s *= f;
      }
      m = bm;
    };
    for (int q = 0; q < nb; ++q) {
      uint4 x[U];
      const int vb = v0 + q * U * kLpThreads + tid;
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = vb + u * kLpThreads < v1 ? ld_stream(vp + vb + u * kLpThreads) : VecOps<T>::neg_inf();
      float bm = VecOps<T>::vmax(x[0]);
#pragma unroll
      for (int u = 1; u < U; ++u) bm = fmaxf(bm, VecOps<T>::vmax(x[u]));
      bmax[q][tid] = bm;
      if (bm > m) raise(bm);
      if (m > -INFINITY) {
        float s2[2] = {0.f, 0.f}, t2[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            // (-inf, and NaN, count as 0: 2^-150 flushes)
            const float y = fmaxf((VecOps<T>::at(x[u], e) - m) * c, -150.f);
            const float p = fast_exp2(y);
            s2[e & 1] += p;
            t2[e & 1] = fmaf(y, p, t2[e & 1]);
          }
        s += s2[0] + s2[1];
        t += t2[0] + t2[1];
      }
    }
    const bool edges = ch == 0 && row.head + row.tail > 0;
    if (edges) {
      const float x = tid < row.head + row.tail ? LogitTraits<T>::load(row.row, row.edge(tid)) : -INFINITY;
      bmax[nb][tid] = x == x ? x : -INFINITY;
      if (x > m) raise(x);
      if (x > -INFINITY) {
        const float y = fmaxf((x - m) * c, -150.f), p = fast_exp2(y);
        s += p;
        t = fmaf(y, p, t);
      }
    }
    LpToken token{-1, 0.f};
    if (ch == 0 && tid == 0) token = token_of<T>(a, a.tokens[out_row], idx);
    // ---- the chunk's maximum and sums; the 32 group maxima ----
    gmax[w][lane] = m;
    __syncthreads();
    float gv = gmax[0][lane];
#pragma unroll
    for (int q = 1; q < kLpWarps; ++q) gv = fmaxf(gv, gmax[q][lane]);
    M = warp_max(gv);
    raise(M);
    s = warp_sum(s);
    t = warp_sum(t);
    if (lane == 0) {
      red[0][w] = s;
      red[1][w] = t;
    }
    float theta = -INFINITY;
    if (a.k > 0) {
      // the k-th largest group maximum (counting; ties by lane)
      int rank = 0;
#pragma unroll
      for (int o = 0; o < 32; ++o) {
        const float v = __shfl_sync(0xffffffffu, gv, o);
        rank += v > gv || (v == gv && o < lane);
      }
      const unsigned who = __ballot_sync(0xffffffffu, rank == a.k - 1);
      theta = __shfl_sync(0xffffffffu, gv, __ffs(who) - 1);
      const int all = nb + (edges ? 1 : 0);
      if (m >= theta)
        for (int q = 0; q < all; ++q) {
          const float bm = bmax[q][tid];
          if (bm >= theta && bm > -INFINITY) {
            const int at = atomicAdd(&n_list, 1);
            if (at < kListCap) list[at] = q * kLpThreads + tid;
          }
        }
    }
    __syncthreads();
    s = t = 0.f;
#pragma unroll
    for (int q = 0; q < kLpWarps; ++q) {
      s += red[0][q];
      t += red[1][q];
    }
    if (a.k > 0) {
      const int nl = n_list;
      if (nl <= kListCap) {
        for (int e = w; e < nl; e += kLpWarps) {
          const int q = list[e] / kLpThreads, th = list[e] % kLpThreads;
          int i = -1;
          if (q == nb) {
            if (lane == 0) i = row.edge(th);
          } else {
            const int v = v0 + (q * U + lane / E) * kLpThreads + th;
            if (v < v1) i = row.head + v * E + lane % E;
          }
          const float x = i >= 0 ? LogitTraits<T>::load(row.row, i) : -INFINITY;
          if (x >= theta && x > -INFINITY) {
            const int at = atomicAdd(&n_cand, 1);
            if (at < kListCap) {
              cv[at] = x;
              ci[at] = i;
            }
          }
        }
        __syncthreads();
      }
      const int nc = n_cand;
      if (nl <= kListCap && nc <= kListCap) {
        count = min(a.k, nc);
        for (int i = tid; i < nc; i += kLpThreads) {
          int rank = 0;
          for (int q = 0; q < nc; ++q) rank += better(cv[q], ci[q], cv[i], ci[i]);
          if (rank < a.k) {
            tv[0][rank] = cv[i];
            ti[0][rank] = ci[i];
          }
        }
      } else {
        // long ties: k rounds, each the best logit after the last one's
        float pv = INFINITY;
        int pi = -1;
        for (count = 0; count < a.k; ++count) {
          float bv = -INFINITY;
          int bi = INT_MAX;
          const int n_edge = edges ? row.head + row.tail : 0;
          const int elems = (v1 - v0) * E + n_edge;
          for (int q = tid; q < elems; q += kLpThreads) {
            const int i = q < n_edge ? row.edge(q) : row.head + v0 * E + (q - n_edge);
            const float x = LogitTraits<T>::load(row.row, i);
            if (x > -INFINITY && better(pv, pi, x, i) && better(x, i, bv, bi)) {
              bv = x;
              bi = i;
            }
          }
          warp_argmax(bv, bi);
          __syncthreads();
          if (lane == 0) {
            red[0][w] = bv;
            list[w] = bi;
          }
          __syncthreads();
          for (int q = 0; q < kLpWarps; ++q)
            if (better(red[0][q], list[q], bv, bi)) {
              bv = red[0][q];
              bi = list[q];
            }
          if (bi == INT_MAX) break;
          if (tid == 0) {
            tv[0][count] = bv;
            ti[0][count] = bi;
          }
          pv = bv;
          pi = bi;
        }
      }
      __syncthreads();
    }
    if (args.chunks == 1) {
      if (w == 0) finish_row(a, out_row, token, M, s, t, inv_t, count, tv[0], ti[0]);
      return;
    }
    if (tid == 0) part = LpPart{M, s, t, count};
    // ---- the row's first CTA joins the chunks, a lane a chunk ----
    cluster_sync();
    if (ch == 0 && w == 0) {
      const uint32_t heads = cluster_addr(&part, lane < args.chunks ? lane : 0);
      auto entry = [&](int q, int at) {
        return make_float2(cluster_ldf(cluster_addr(&tv[0][at], q)), cluster_ldf(cluster_addr(&ti[0][at], q)));
      };
      const int all = args.chunks * a.k;
      float4 h = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      float kth = 0.f;
      if (lane < args.chunks) {
        h = cluster_ld4(heads);
        if (a.k > 0) kth = entry(lane, a.k - 1).x;
      }
      float pM = -INFINITY, ps = 0.f, pt = 0.f;
      int pc = 0;
      float theta = -INFINITY;  // at least k logits reach it: the largest of the chunks' k-th best
      if (lane < args.chunks) {
        pM = h.x;
        ps = h.y;
        pt = h.z;
        pc = __float_as_int(h.w);
        if (pc == a.k) theta = kth;  // (else it was not written)
      }
      const float jM = warp_max(pM);
      const float d = fmaxf((pM - jM) * c, -150.f), f = fast_exp2(d);
      const float js = warp_sum(ps > 0.f ? f * ps : 0.f), jt = warp_sum(ps > 0.f ? f * fmaf(d, ps, pt) : 0.f);
      int got = 0;
      if (a.k > 0) {
        theta = warp_max(theta);
        // the entries that reach theta, ranked by counting
        float* qv = cv;
        int* qi = ci;
        int nc = 0;
#pragma unroll 4
        for (int base = 0; base < all; base += 32) {
          const int p = base + lane, pch = min(p / a.k, args.chunks - 1), at = p - pch * a.k;
          const int cnt = __shfl_sync(0xffffffffu, pc, pch);
          float2 x = make_float2(-INFINITY, 0.f);
          if (at < cnt) x = entry(pch, at);
          const bool in = at < cnt && x.x >= theta;
          const unsigned who = __ballot_sync(0xffffffffu, in);
          const int to = nc + __popc(who & ((1u << lane) - 1u));
          if (in && to < kJoinCap) {
            qv[to] = x.x;
            qi[to] = __float_as_int(x.y);
          }
          nc += __popc(who);
        }
        __syncwarp();
        if (nc <= kJoinCap) {
          got = min(a.k, nc);
          for (int i = lane; i < nc; i += 32) {
            int rank = 0;
            for (int q = 0; q < nc; ++q) rank += better(qv[q], qi[q], qv[i], qi[i]);
            if (rank < a.k) {
              tv[1][rank] = qv[i];
              ti[1][rank] = qi[i];
            }
          }
        } else {
          // long ties: the chunks' sorted lists, k times the best head
          int head = 0;
          for (; got < a.k; ++got) {
            float bv = -INFINITY;
            int bi = INT_MAX;
            if (head < pc) {
              const float2 x = entry(lane, head);
              bv = x.x;
              bi = __float_as_int(x.y);
            }
            const int hi = bi;
            warp_argmax(bv, bi);
            if (bi == INT_MAX || !(bv > -INFINITY)) break;
            if (lane == 0) {
              tv[1][got] = bv;
              ti[1][got] = bi;
            }
            if (hi == bi) ++head;
          }
        }
        __syncwarp();
      }
      finish_row(a, out_row, token, jM, js, jt, inv_t, got, tv[1], ti[1]);
    }
    cluster_sync();  // (no CTA ends while its shared memory is read)
  }
}

// Chunks of a row: a power of two, for at most kLpCtas CTAs in all (the 224 rows of the header's
// example in four chunks 15.2 us, in two 20.4, in eight 22.6), of 2048 logits at least
// and kMaxBatches batches at most.
int lp_chunks(long rows, int V) {
  int chunks = 1;
  while (chunks < kLpCluster && 2 * chunks * rows <= kLpCtas && 2 * chunks <= V / 2048) chunks *= 2;
  while (long(chunks) * kMaxBatches * kBatch * kLpThreads < V) chunks *= 2;  // (the API's largest V takes eight)
  return chunks;
}

}  // namespace

int launch_token_logprobs(const LogprobParams& p, cudaStream_t stream) {
  const long rows = long(p.b) * p.W;
  LpArgs args{p, lp_chunks(rows, p.V), 0};
  if (args.chunks > kLpCluster) return SPEC_ERR_UNSUPPORTED;
  const int E = p.dtype == SPEC_F32 ? 4 : 8;
  args.vpc = (p.V / E + args.chunks - 1) / args.chunks;
  if (args.vpc < 1) args.vpc = 1;
  const dim3 grid(unsigned(rows * args.chunks));
  const cudaError_t e =
      p.dtype == SPEC_F32 ? launch_cluster(token_logprobs_kernel<float>, args.chunks, grid, dim3(kLpThreads), 0, stream, args)
                          : launch_cluster(token_logprobs_kernel<uint16_t>, args.chunks, grid, dim3(kLpThreads), 0, stream, args);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace spec
