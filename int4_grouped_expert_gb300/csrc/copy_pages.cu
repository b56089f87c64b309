// Copies whole pages of a paged cache, codes and scales, for a list of (from, to) pairs that lies on the device and for many
// caches (the layers of a model) in one launch.
//
// Bound by memory, each byte read and written once. A block takes a piece of 16 or 32 KB of a page's K or V codes, all of
// a thread's 16-byte loads on their way before the first is stored. The first piece's block takes the page's
// scales along. Pairs that lead nowhere cost a look at the list; the blocks are as many as max_copies asks for, for the count lies
// on the device. (us, no copies: 8 sequences of one cache 1.3, 64 of 48 caches of 8 heads of 128 and pages of 64 13, 256 of 48 40.)
#include <algorithm>

#include "pages.cuh"

namespace strata {

namespace {

constexpr int kCopyThreads = 256;
// Pieces of 16 KB, or of 32 KB where those fill the SMs several times.
template <int kCopyLoads>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a, int pieces) {
  constexpr int kCopyPiece = kCopyThreads * kCopyLoads * 16;
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

// (us, 3732 pages of 128 KB in each of three caches, 2.9 GB moved: blocks of four loads that go on by themselves, 8 an SM,
// 490; of eight 462; up to 16, 64, 256 blocks an SM of eight 442, 427, 423: 6.9 TB/s, the rate of a plain copy. Bulk copies
// through shared memory, 4 of 16 KB on their way in each of two blocks an SM, 461.)
constexpr int kCopyWide = 16, kCopyBlocks = 256;

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesArgs& a, int num_sms, cudaStream_t stream) {
  auto pieces = [&](int loads) { return static_cast<int>((a.page_bytes - 1) / (kCopyThreads * loads * 16) + 1); };
  auto units = [&](int loads) { return static_cast<int64_t>(a.max_copies) * 2 * pieces(loads) * a.n_caches; };
  const bool wide = units(8) >= kCopyWide * num_sms;
  // Blocks for up to kCopyBlocks an SM: one that ends makes room for the next at once, which keeps the memory busier than
  // blocks that go on by themselves.
  const int64_t grid = std::min<int64_t>(units(wide ? 8 : 4), kCopyBlocks * num_sms);
  return launch_kernel(wide ? copy_pages_kernel<8> : copy_pages_kernel<4>, dim3(static_cast<unsigned>(grid)),
                       dim3(kCopyThreads), 0, stream, true, a, pieces(wide ? 8 : 4));
}

}  // namespace strata
