// copy_pages.cu -- pages of a cache copied within it, every layer's K and V and,
// for the 8-bit cache, their scales.
//
// Bound: HBM, two bytes moved for each byte of the pages.  Units of 4 KB, laid end to end (pair, then layer
// and K or V, then the page's bytes), go to the warps of a persistent grid in turn; a lane has eight 16-byte
// loads in flight before its first store.  4.3 GB moved (2.1 GB of pages): 661 us, 6.4 TB/s, 96% of a plain copy.
#include "common.cuh"
#include "kernels.cuh"

namespace spec {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kUnit = 4096;  // bytes of a page that a warp copies at a time
constexpr int kCtasPerSm = 4;

__global__ void __launch_bounds__(kCopyThreads, kCtasPerSm) copy_pages_kernel(const __grid_constant__ CopyParams a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  int n = *a.n_copies;
  if (n < 0 || n > a.max_copies) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.error, SPEC_DEV_LENGTH);
    n = n < 0 ? 0 : a.max_copies;
  }
  const unsigned per_page = unsigned((a.page_bytes + kUnit - 1) / kUnit), arrays = 2u * unsigned(a.num_layers);
  const long long units = (long long)n * arrays * per_page;
  const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
  for (long long u = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const long long unit = u / per_page;
    const unsigned part = unsigned(u - unit * per_page);
    const int pair = int(unit / arrays), which = int(unit - (long long)pair * arrays);
    const int src = a.src_ids[pair], dst = a.dst_ids[pair];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
      if (lane == 0) raise_error(a.error, SPEC_DEV_INDEX);
      continue;
    }
    unsigned char* pool = static_cast<unsigned char*>(which & 1 ? a.v_layers[which >> 1] : a.k_layers[which >> 1]);
    const uint4* from = reinterpret_cast<const uint4*>(pool + size_t(src) * a.page_bytes + size_t(part) * kUnit);
    uint4* to = reinterpret_cast<uint4*>(pool + size_t(dst) * a.page_bytes + size_t(part) * kUnit);
    const long long rest = (a.page_bytes - (long long)part * kUnit) / 16;
    const int vecs = rest < kUnit / 16 ? int(rest) : kUnit / 16;
    uint4 x[kUnit / 512];
#pragma unroll
    for (int i = 0; i < kUnit / 512; ++i)
      if (lane + 32 * i < vecs) x[i] = __ldcs(from + lane + 32 * i);
#pragma unroll
    for (int i = 0; i < kUnit / 512; ++i)
      if (lane + 32 * i < vecs) __stcs(to + lane + 32 * i, x[i]);
    if (part == 0 && a.scale_bytes) {
      uint8_t* scales = which & 1 ? a.v_scales[which >> 1] : a.k_scales[which >> 1];
      for (int i = lane; i < a.scale_bytes; i += 32)
        scales[size_t(dst) * a.scale_bytes + i] = scales[size_t(src) * a.scale_bytes + i];
    }
  }
}

}  // namespace

int launch_copy_pages(const CopyParams& p, int sms, cudaStream_t stream) {
  const long long units = (long long)p.max_copies * 2 * p.num_layers * ((p.page_bytes + kUnit - 1) / kUnit);
  long long grid = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  if (grid > (long long)sms * kCtasPerSm) grid = (long long)sms * kCtasPerSm;
  if (grid < 1) grid = 1;
  const cudaError_t e = launch_pdl(copy_pages_kernel, dim3(unsigned(grid)), dim3(kCopyThreads), 0, stream, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace spec
