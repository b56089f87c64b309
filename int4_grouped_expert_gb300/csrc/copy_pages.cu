// Copies whole pages of a paged cache, codes and scales, for a list of (from, to) pairs that lies on the device and for many
// caches (the layers of a model) in one launch.
//
// Bound by memory, each byte read and written once. A block takes pieces of 16 KB of a page's K or V codes, one after
// another through the whole list: four 16-byte loads of each thread on their way before the first is stored. The first
// piece's block takes the page's scales along. Pairs that lead nowhere cost a look at the list.
#include <algorithm>

#include "pages.cuh"

namespace strata {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;
constexpr int kCopyPiece = kCopyThreads * kCopyLoads * 16;

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a, int pieces) {
  griddep_wait();
  griddep_launch();
  int n = a.max_copies;
  if (a.n_copies) {
    n = *a.n_copies;
    if (n < 0 || n > a.max_copies) {
      if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
      n = min(max(n, 0), a.max_copies);
    }
  }
  const int per_pair = 2 * pieces * a.n_caches;
  const int64_t units = static_cast<int64_t>(n) * per_pair;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t pair = u / per_pair;
    const int at = static_cast<int>(u - pair * per_pair), cache = at / (2 * pieces), part = at - cache * 2 * pieces;
    const bool v = part >= pieces;
    const int piece = v ? part - pieces : part;
    const int64_t from = a.copies[2 * pair], to = a.copies[2 * pair + 1];
    if (from < 0 || to < 0) continue;
    if (from >= a.src_pages || to >= a.dst_pages) {
      if (at == 0 && threadIdx.x == 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
      continue;
    }
    const CopyPagesArgs::Cache& c = a.cache[cache];
    const int64_t begin = static_cast<int64_t>(piece) * kCopyPiece + threadIdx.x * 16;
    const uint8_t* src = (v ? c.v : c.k) + from * a.page_bytes;
    uint8_t* dst = (v ? c.v_to : c.k_to) + to * a.page_bytes;
    uint4 x[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j) {
      const int64_t i = begin + j * (kCopyThreads * 16);
      if (i < a.page_bytes) x[j] = __ldcs(reinterpret_cast<const uint4*>(src + i));
    }
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j) {
      const int64_t i = begin + j * (kCopyThreads * 16);
      if (i < a.page_bytes) __stcs(reinterpret_cast<uint4*>(dst + i), x[j]);
    }
    if (piece == 0 && static_cast<int>(threadIdx.x) < a.n_kv_heads) {  // (at most 256)
      const int64_t h = threadIdx.x;
      (v ? c.vs_to : c.ks_to)[to * a.n_kv_heads + h] = (v ? c.vs : c.ks)[from * a.n_kv_heads + h];
    }
  }
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesArgs& a, int num_sms, cudaStream_t stream) {
  const int pieces = static_cast<int>((a.page_bytes + kCopyPiece - 1) / kCopyPiece);
  const int64_t units = static_cast<int64_t>(a.max_copies) * 2 * pieces * a.n_caches;
  const int64_t grid = std::min<int64_t>(units, 8 * num_sms);
  return launch_kernel(copy_pages_kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), 0, stream, true, a, pieces);
}

}  // namespace strata
