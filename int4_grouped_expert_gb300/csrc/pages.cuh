// Launchers and argument blocks of the calls that manage the pages of a cache (pages.cu, copy_pages.cu).
#pragma once

#include "common.cuh"

namespace strata {

constexpr int kPagesCluster = 8;     // blocks of the cluster that settles one call's allocation
constexpr int kPagesThreads = 1024;
constexpr int kPagesMostSeq = 65535;  // sequences of a call

struct PagesExtendArgs {
  strata_kv_pages p;
  const int32_t* new_tokens;
  int T_max;
  int32_t *slots, *positions, *q_start, *copies, *n_copies;
  uint32_t* status;
};
cudaError_t launch_pages_extend(const PagesExtendArgs& a, cudaStream_t stream);

struct PagesForkArgs {
  strata_kv_pages p;
  const int32_t* parent;
  uint32_t* status;
};
cudaError_t launch_pages_fork(const PagesForkArgs& a, int num_sms, cudaStream_t stream);

struct PagesReleaseArgs {
  strata_kv_pages p;
  const int32_t* keep;  // null: no sequence is cut
  int window, n_sinks;  // window 0: nothing before a window is given back
  uint32_t* status;
};
cudaError_t launch_pages_release(const PagesReleaseArgs& a, int num_sms, cudaStream_t stream);

struct PagesCompactArgs {
  strata_kv_pages src, dst;
  int32_t *copies, *n_copies;
  int32_t* map;   // [src.n_pages]: a page's number in the other pool
  int32_t* live;  // pages in use, or -1: more than the other pool has
  uint32_t* status;
};
cudaError_t launch_pages_compact(const PagesCompactArgs& a, int num_sms, cudaStream_t stream);

constexpr int kCopyCaches = 48;  // caches of one launch
struct CopyPagesArgs {
  struct Cache {
    const uint8_t *k, *v;
    const float *ks, *vs;
    uint8_t *k_to, *v_to;
    float *ks_to, *vs_to;
  } cache[kCopyCaches];
  int n_caches, n_kv_heads;
  int64_t page_bytes, src_pages, dst_pages;
  const int32_t* copies;
  const int32_t* n_copies;  // null: max_copies
  int max_copies;
  uint32_t* status;
};
cudaError_t launch_copy_pages(const CopyPagesArgs& a, int num_sms, cudaStream_t stream);

}  // namespace strata
