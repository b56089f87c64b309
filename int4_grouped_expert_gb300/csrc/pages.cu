// Page tables of a cache on the device: room for new tokens, sequences that share pages, pages that are given back,
// and the move to another pool. The state is the table, the lengths and `refs`, the number of table entries
// that name each page; a page is free where that is zero. There is no list of free pages: the lowest free ones are
// taken in the order of the sequences, so the same calls give the same tables, whatever ran at the same time, and
// pools stay packed. Integer counts are added with atomics, whose order does not matter.
//
// What these calls move is small (4 bytes a page of the pool, 4 to 12 bytes a table entry): the chain of dependent
// steps is the time. Allocation needs sums over all pages and over all sequences before anybody can write, so one
// cluster of eight blocks does a whole call, with the cluster's barrier between its steps: one launch, no workspace,
// no counters in memory to wait for. Eight SMs read a pool of 65536 pages in about a microsecond.
#include <algorithm>

#include "pages.cuh"

namespace strata {

namespace {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}
// A 64-bit word of block `rank` of the cluster, at this block's address of it.
__device__ __forceinline__ uint64_t cluster_load(const uint64_t* p, int rank) {
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t theirs;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(theirs) : "r"(mine), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(theirs) : "memory");
  return v;
}

// Pages that `tokens` tokens take.
__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return tokens > 0 ? ((tokens - 1) >> shift) + 1 : 0;
}
__device__ __forceinline__ int shift_of(const strata_kv_pages& p) { return 31 - __clz(p.page_size); }
// A sequence's length, cut to what its table holds.
__device__ __forceinline__ int length_of(const strata_kv_pages& p, int len, uint32_t* status) {
  const int most = static_cast<int>(p.max_pages * p.page_size);  // (< 2^31, host)
  if (len >= 0 && len <= most) return len;
  set_status(status, STRATA_DEV_BAD_SLOT);
  return min(max(len, 0), most);
}
__device__ __forceinline__ bool is_page(const strata_kv_pages& p, int page) { return page >= 0 && page < p.n_pages; }

// Inclusive sums of a block's threads, and the block's total. Every thread calls it; `s` is free again after the
// next barrier of the block.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* s, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  if (lane == 31) s[warp] = v;
  __syncthreads();
  T w = s[lane];  // (32 warps)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += x;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return warp == 0 ? v : v + before;
}

// A block's share of n: whole chunks of `chunk`, in order.
struct Range {
  int64_t lo, hi;
};
__device__ __forceinline__ int64_t share_of(int64_t n, int chunk) {
  return ((n + kPagesCluster - 1) / kPagesCluster + chunk - 1) / chunk * chunk;
}
__device__ __forceinline__ Range range_of(int64_t n, int chunk, int rank) {
  const int64_t per = share_of(n, chunk), lo = min(n, rank * per);
  return {lo, min(n, lo + per)};
}
// The counts of four pages, and how many of them `want` holds for. Pages from hi on count as neither free nor in use.
constexpr int kPageChunk = 4 * kPagesThreads;
__device__ __forceinline__ int4 four_refs(const int32_t* refs, int64_t at, int64_t hi) {
  if (at + 4 <= hi) return *reinterpret_cast<const int4*>(refs + at);
  return make_int4(at < hi ? refs[at] : -1, at + 1 < hi ? refs[at + 1] : -1, at + 2 < hi ? refs[at + 2] : -1, -1);
}

// ------------------------------------------------------------------------------------------------ extend
// What a sequence asks for: `rows` new tokens (0: nothing, or something is wrong), pages for them, and whether its unfinished
// page is shared, so that it moves to a page of its own.
struct Ask {
  int rows, need, moved;
};
__device__ __forceinline__ Ask ask_of(const PagesExtendArgs& a, int s) {
  const strata_kv_pages& p = a.p;
  const int shift = shift_of(p), fresh = a.new_tokens[s];
  const int len = length_of(p, p.kv_len[s], a.status);
  Ask k{0, 0, 0};
  if (fresh == 0) return k;
  const int64_t most = p.max_pages * p.page_size;
  if (fresh < 0 || fresh > most - len) {
    set_status(a.status, STRATA_DEV_BAD_SLOT);
    return k;
  }
  if (len & (p.page_size - 1)) {
    const int page = p.page_table[s * p.table_stride + (len >> shift)];
    const int refs = is_page(p, page) ? p.refs[page] : 0;
    if (refs < 1) {
      set_status(a.status, STRATA_DEV_BAD_SLOT);
      return k;
    }
    k.moved = refs > 1;
  }
  k.rows = fresh;
  k.need = pages_of(len + fresh, shift) - pages_of(len, shift) + k.moved;
  return k;
}

// Sequences in order get room while pages and rows last. need <= rows for each (a page is for one new token at
// least, the page that a shared one moves to among them), so the list of pages has room where the rows' slots
// will be.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_extend_kernel(PagesExtendArgs a) {
  extern __shared__ int32_t seq_smem[];  // [3][share]: rows (negative: and the page moves), first row, first page
  __shared__ uint64_t s_rows[32], s_need[32];
  __shared__ int s_free[32];
  __shared__ uint64_t s_total[3], s_got[2];  // for the cluster: free pages, rows, pages; rows and pages that are given
  __shared__ uint32_t s_moves;
  griddep_wait();
  griddep_launch();
  const strata_kv_pages& p = a.p;
  const int rank = blockIdx.x, shift = shift_of(p);
  const int n_seq = p.n_seq, share = static_cast<int>(share_of(n_seq, kPagesThreads));
  int32_t *rows_of = seq_smem, *row_at = seq_smem + share, *page_at = seq_smem + 2 * share;
  const Range seqs = range_of(n_seq, kPagesThreads, rank), pages = range_of(p.n_pages, kPageChunk, rank);
  constexpr int kMoveBits = 17;  // (at most 65535 sequences move a page)

  // ---- free pages of this block's share, and what its sequences ask for
  int free = 0;
  for (int64_t at = pages.lo + 4 * threadIdx.x; at < pages.hi; at += kPageChunk) {
    const int4 r = four_refs(p.refs, at, pages.hi);
    free += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  uint64_t rows_sum = 0, need_sum = 0;  // (64 bits: nothing is cut before it is added)
  for (int64_t s0 = seqs.lo; s0 < seqs.hi; s0 += kPagesThreads) {
    const int s = static_cast<int>(s0) + threadIdx.x, i = s - static_cast<int>(seqs.lo);
    const Ask k = s < seqs.hi ? ask_of(a, s) : Ask{0, 0, 0};
    uint64_t rt, nt;
    const uint64_t rows = rows_sum + block_scan<uint64_t>(k.rows, s_rows, rt);
    const uint64_t need =
        need_sum + block_scan<uint64_t>(static_cast<uint64_t>(k.need) << kMoveBits | k.moved, s_need, nt);
    if (s < seqs.hi) {
      rows_of[i] = k.moved ? -k.rows : k.rows;
      // (sums beyond any limit are all the same: refused)
      row_at[i] = static_cast<int>(min(rows - k.rows, uint64_t(0x40000000)));
      page_at[i] = static_cast<int>(min((need >> kMoveBits) - k.need, uint64_t(0x40000000)));
    }
    rows_sum += rt;
    need_sum += nt;
    __syncthreads();
  }
  int free_total;
  block_scan(free, s_free, free_total);
  if (threadIdx.x == 0) {
    s_total[0] = free_total;
    s_total[1] = rows_sum;
    s_total[2] = need_sum;
    s_moves = 0;
  }
  cluster_sync();
  uint64_t free_before = 0, rows_before = 0, need_before = 0, free_all = 0;
  for (int b = 0; b < kPagesCluster; ++b) {
    const uint64_t f = cluster_load(s_total, b);
    if (b < rank) {
      free_before += f;
      rows_before += cluster_load(s_total + 1, b);
      need_before += cluster_load(s_total + 2, b);
    }
    free_all += f;
  }
  const uint64_t pages_before = need_before >> kMoveBits;
  // ---- who gets room: sums only grow, so it is the sequences up to some place. Rows and pages up to there.
  uint64_t rows_got = 0, pages_got = 0;
  for (int i = threadIdx.x; i < seqs.hi - seqs.lo; i += kPagesThreads) {
    const int n = abs(rows_of[i]);
    // (recomputed from the stored sums: the pages of sequence i end where the next one's begin)
    const uint64_t r1 = rows_before + row_at[i] + n;
    const int len = length_of(p, p.kv_len[seqs.lo + i], nullptr);
    const int need = n > 0 ? pages_of(len + n, shift) - pages_of(len, shift) + (rows_of[i] < 0) : 0;
    const uint64_t p1 = pages_before + page_at[i] + need;
    if (r1 <= static_cast<uint64_t>(a.T_max) && p1 <= free_all) {
      rows_got = max(rows_got, r1);
      pages_got = max(pages_got, p1);
      if (rows_of[i] < 0) atomicAdd(&s_moves, 1u);
    } else {
      if (n > 0) set_status(a.status, STRATA_DEV_NO_PAGES);
      rows_of[i] = 0;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    rows_got = max(rows_got, __shfl_xor_sync(0xffffffffu, rows_got, d));
    pages_got = max(pages_got, __shfl_xor_sync(0xffffffffu, pages_got, d));
  }
  if ((threadIdx.x & 31) == 0) {
    s_rows[threadIdx.x >> 5] = rows_got;
    s_need[threadIdx.x >> 5] = pages_got;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) {
      rows_got = max(rows_got, s_rows[w]);
      pages_got = max(pages_got, s_need[w]);
    }
    s_got[0] = rows_got;
    s_got[1] = pages_got << 32 | s_moves;
  }
  cluster_sync();
  uint32_t moves_before = 0, moves_all = 0;
  rows_got = pages_got = 0;
  for (int b = 0; b < kPagesCluster; ++b) {
    const uint64_t g = cluster_load(s_got + 1, b);
    rows_got = max(rows_got, cluster_load(s_got, b));
    pages_got = max(pages_got, g >> 32);
    if (b < rank) moves_before += static_cast<uint32_t>(g);
    moves_all += static_cast<uint32_t>(g);
  }
  const int R = static_cast<int>(rows_got);
  // ---- the lowest free pages, in order: noted where the slots will be
  uint64_t at_free = free_before;
  for (int64_t c = pages.lo; c < pages.hi && at_free < pages_got; c += kPageChunk) {
    const int64_t at = c + 4 * threadIdx.x;
    const int4 r = at < pages.hi ? four_refs(p.refs, at, pages.hi) : make_int4(-1, -1, -1, -1);
    const int here = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int total;
    uint64_t k = at_free + block_scan(here, s_free, total) - here;
    const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (v[j] != 0) continue;
      if (k < pages_got) {
        a.slots[k] = static_cast<int32_t>(at + j);
        p.refs[at + j] = 1;
      }
      ++k;
    }
    at_free += total;
    __syncthreads();
  }
  cluster_sync();
  // ---- tables and lengths: a lane a sequence, a warp where one has many pages
  uint32_t moves = moves_before;
  for (int64_t s0 = seqs.lo; s0 < seqs.hi; s0 += kPagesThreads) {
    const int s = static_cast<int>(s0) + threadIdx.x, i = s - static_cast<int>(seqs.lo);
    const bool on = s < seqs.hi;
    const int n = on ? abs(rows_of[i]) : 0, moved = on && rows_of[i] < 0;
    const int len = n > 0 ? length_of(p, p.kv_len[s], nullptr) : 0;
    int first = pages_of(len, shift) - moved;
    int need = n > 0 ? pages_of(len + n, shift) - first : 0;
    int from = n > 0 ? static_cast<int>(pages_before) + page_at[i] : 0;
    uint32_t total;
    const uint32_t m = moves + block_scan<uint32_t>(moved, reinterpret_cast<uint32_t*>(s_free), total) - moved;
    moves += total;
    if (on) a.q_start[s] = static_cast<int>(min(rows_before + row_at[i], rows_got));
    int32_t* row = p.page_table + static_cast<int64_t>(on ? s : 0) * p.table_stride;
    if (moved) {
      const int old = row[first], page = __ldcg(a.slots + from);
      atomicAdd(p.refs + old, -1);
      a.copies[2 * m] = old;
      a.copies[2 * m + 1] = page;
    }
    if (n > 0) p.kv_len[s] = len + n;
    if (need == 1) row[first] = __ldcg(a.slots + from);
    for (unsigned many = __ballot_sync(0xffffffffu, need > 1); many; many &= many - 1) {
      const int l = __ffs(many) - 1;
      const int64_t at = __shfl_sync(0xffffffffu, static_cast<int64_t>(row - p.page_table), l);
      const int f = __shfl_sync(0xffffffffu, first, l), k = __shfl_sync(0xffffffffu, need, l);
      const int src = __shfl_sync(0xffffffffu, from, l);
      for (int e = threadIdx.x & 31; e < k; e += 32) p.page_table[at + f + e] = __ldcg(a.slots + src + e);
    }
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.q_start[n_seq] = R;
    *a.n_copies = static_cast<int32_t>(moves_all);
  }
  cluster_sync();
  // ---- the rows, each by itself (the list of pages is not needed any more)
  for (int r = rank * kPagesThreads + threadIdx.x; r < a.T_max; r += kPagesCluster * kPagesThreads) {
    int slot = -1, pos = 0;
    if (r < R) {
      int lo = 0, hi = n_seq;  // the last sequence whose first row is not after r: q_start[lo] <= r < q_start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(a.q_start + mid) <= r) lo = mid;
        else hi = mid;
      }
      pos = __ldcg(p.kv_len + lo) - (__ldcg(a.q_start + lo + 1) - r);
      slot = (__ldcg(p.page_table + lo * p.table_stride + (pos >> shift)) << shift) + (pos & (p.page_size - 1));
    }
    a.slots[r] = slot;
    a.positions[r] = pos;
  }
}

// ------------------------------------------------------------------------------------------------ fork
// A block takes one child at a time: its length is read and written by that block alone.
constexpr int kForkThreads = 512;
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(PagesForkArgs a) {
  griddep_wait();
  griddep_launch();
  const strata_kv_pages& p = a.p;
  const int shift = shift_of(p);
  for (int s = blockIdx.x; s < p.n_seq; s += gridDim.x) {
    const int of = a.parent[s];
    if (of < 0) continue;
    // (a parent that is itself a child of this call, this sequence for one, is not settled yet)
    if (of >= p.n_seq || a.parent[of] >= 0 || p.kv_len[s] != 0) {
      if (threadIdx.x == 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
      continue;
    }
    const int len = length_of(p, p.kv_len[of], threadIdx.x == 0 ? a.status : nullptr), n = pages_of(len, shift);
    const int32_t* src = p.page_table + static_cast<int64_t>(of) * p.table_stride;
    int32_t* dst = p.page_table + static_cast<int64_t>(s) * p.table_stride;
    for (int e0 = threadIdx.x; e0 < n; e0 += 4 * kForkThreads) {
      int page[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) page[j] = e0 + j * kForkThreads < n ? src[e0 + j * kForkThreads] : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e0 + j * kForkThreads >= n) break;
        if (is_page(p, page[j])) {
          atomicAdd(p.refs + page[j], 1);
        } else {
          if (page[j] >= 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
          page[j] = -1;
        }
        dst[e0 + j * kForkThreads] = page[j];
      }
    }
    __syncthreads();  // every thread has seen that the child was empty
    if (threadIdx.x == 0) p.kv_len[s] = len;
  }
}

// ------------------------------------------------------------------------------------------------ release
// A block takes a stretch of entries of one sequence. What goes depends on the new length alone, which is the same
// before and after another block of the sequence has written it.
constexpr int kReleaseThreads = 256, kReleaseEntries = 4 * kReleaseThreads;
__global__ void __launch_bounds__(kReleaseThreads) pages_release_kernel(PagesReleaseArgs a, int stretches) {
  griddep_wait();
  griddep_launch();
  const strata_kv_pages& p = a.p;
  const int shift = shift_of(p);
  const int64_t units = static_cast<int64_t>(p.n_seq) * stretches;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int s = static_cast<int>(u / stretches), stretch = static_cast<int>(u % stretches);
    const int keep = a.keep ? a.keep[s] : -1;
    if (keep < 0 && a.window == 0) continue;
    const bool flag = stretch == 0 && threadIdx.x == 0;
    const int held = __ldcg(p.kv_len + s), old = length_of(p, held, flag ? a.status : nullptr);
    const int len = keep >= 0 ? min(keep, old) : old;
    // entries cut .. : behind the sequence; entries sinks .. gap - 1: whole between the first tokens and the window of
    // the next query, at position len (it sees tokens from len - window + 1 on)
    const int cut = keep >= 0 ? pages_of(len, shift) : 0x7FFFFFFF;
    const int sinks = pages_of(a.n_sinks, shift), gap = a.window > 0 && len >= a.window ? (len - a.window + 1) >> shift : 0;
    int32_t* row = p.page_table + static_cast<int64_t>(s) * p.table_stride;
    const int64_t e0 = static_cast<int64_t>(stretch) * kReleaseEntries + threadIdx.x;
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t e = e0 + j * kReleaseThreads;
      const bool goes = e < p.max_pages && (e >= cut || (e >= sinks && e < gap));
      page[j] = goes ? row[e] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (page[j] < 0) continue;
      row[e0 + j * kReleaseThreads] = -1;
      if (!is_page(p, page[j])) {
        set_status(a.status, STRATA_DEV_BAD_SLOT);
      } else if (atomicAdd(p.refs + page[j], -1) < 1) {  // (counted by nobody: left at zero)
        atomicAdd(p.refs + page[j], 1);
        set_status(a.status, STRATA_DEV_BAD_SLOT);
      }
    }
    if (stretch == 0 && threadIdx.x == 0 && keep >= 0 && len != held) p.kv_len[s] = len;
  }
}

// ------------------------------------------------------------------------------------------------ compact
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_map_kernel(PagesCompactArgs a) {
  __shared__ uint64_t s_total;
  __shared__ int s_scan[32];
  griddep_wait();
  griddep_launch();
  const int rank = blockIdx.x;
  const Range pages = range_of(a.src.n_pages, kPageChunk, rank);
  int live = 0, total;
  for (int64_t at = pages.lo + 4 * threadIdx.x; at < pages.hi; at += kPageChunk) {
    const int4 r = four_refs(a.src.refs, at, pages.hi);
    live += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  block_scan(live, s_scan, total);
  if (threadIdx.x == 0) s_total = total;
  cluster_sync();
  int64_t before = 0, all = 0;
  for (int b = 0; b < kPagesCluster; ++b) {
    const int64_t n = static_cast<int64_t>(cluster_load(&s_total, b));
    if (b < rank) before += n;
    all += n;
  }
  const bool fits = all <= a.dst.n_pages;
  for (int64_t c = pages.lo; c < pages.hi; c += kPageChunk) {
    const int64_t at = c + 4 * threadIdx.x;
    const int4 r = at < pages.hi ? four_refs(a.src.refs, at, pages.hi) : make_int4(-1, -1, -1, -1);
    const int v[4] = {r.x, r.y, r.z, r.w};
    const int here = (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    int k = static_cast<int>(before) + block_scan(here, s_scan, total) - here;
    before += total;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (at + j >= pages.hi) break;
      const bool on = v[j] > 0 && fits;
      a.map[at + j] = on ? k : -1;
      if (on) {
        a.dst.refs[k] = v[j];
        a.copies[2 * static_cast<int64_t>(k)] = static_cast<int32_t>(at + j);
        a.copies[2 * static_cast<int64_t>(k) + 1] = k;
      }
      k += v[j] > 0;
    }
    __syncthreads();
  }
  for (int64_t i = (fits ? all : 0) + rank * kPagesThreads + threadIdx.x; i < a.dst.n_pages;
       i += kPagesCluster * kPagesThreads)
    a.dst.refs[i] = 0;
  if (rank == 0 && threadIdx.x == 0) {
    *a.n_copies = fits ? static_cast<int32_t>(all) : 0;
    *a.live = fits ? static_cast<int32_t>(all) : -1;
    if (!fits) set_status(a.status, STRATA_DEV_NO_PAGES);
  }
  cluster_sync();  // (nobody leaves while another reads its total)
}

constexpr int kTableThreads = 256, kTableEntries = 4 * kTableThreads;
__global__ void __launch_bounds__(kTableThreads) pages_table_kernel(PagesCompactArgs a, int stretches) {
  griddep_wait();
  griddep_launch();
  const int shift = shift_of(a.src);
  const bool fits = *a.live >= 0;
  const int64_t units = static_cast<int64_t>(a.src.n_seq) * stretches;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int s = static_cast<int>(u / stretches), stretch = static_cast<int>(u % stretches);
    const bool first = stretch == 0 && threadIdx.x == 0;
    const int len = fits ? length_of(a.src, a.src.kv_len[s], first ? a.status : nullptr) : 0, n = pages_of(len, shift);
    const int32_t* src = a.src.page_table + static_cast<int64_t>(s) * a.src.table_stride;
    int32_t* dst = a.dst.page_table + static_cast<int64_t>(s) * a.dst.table_stride;
    const int64_t e0 = static_cast<int64_t>(stretch) * kTableEntries + threadIdx.x;
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) page[j] = e0 + j * kTableThreads < n ? src[e0 + j * kTableThreads] : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t e = e0 + j * kTableThreads;
      if (e >= a.dst.max_pages) break;
      int to = -1;
      if (page[j] >= 0) {
        if (is_page(a.src, page[j])) to = a.map[page[j]];
        if (to < 0) set_status(a.status, STRATA_DEV_BAD_SLOT);  // (no page, or one that nobody counts)
      }
      dst[e] = to;
    }
    if (first) a.dst.kv_len[s] = len;
  }
}

}  // namespace

cudaError_t launch_pages_extend(const PagesExtendArgs& a, cudaStream_t stream) {
  const int64_t share = ((a.p.n_seq + kPagesCluster - 1) / kPagesCluster + kPagesThreads - 1) / kPagesThreads * kPagesThreads;
  const size_t smem = 3 * sizeof(int32_t) * share;  // up to 96 KB
  if (smem > 40 << 10) {
    const cudaError_t e = cudaFuncSetAttribute(pages_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(pages_extend_kernel, dim3(kPagesCluster), dim3(kPagesThreads), smem, stream, true, a);
}

cudaError_t launch_pages_fork(const PagesForkArgs& a, int num_sms, cudaStream_t stream) {
  return launch_kernel(pages_fork_kernel, dim3(std::min(a.p.n_seq, 4 * num_sms)), dim3(kForkThreads), 0, stream, true, a);
}

cudaError_t launch_pages_release(const PagesReleaseArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t stretches = (a.p.max_pages + kReleaseEntries - 1) / kReleaseEntries;
  const int64_t grid = std::min<int64_t>(a.p.n_seq * stretches, 8 * num_sms);
  return launch_kernel(pages_release_kernel, dim3(static_cast<unsigned>(grid)), dim3(kReleaseThreads), 0, stream, true, a,
                       static_cast<int>(stretches));
}

cudaError_t launch_pages_compact(const PagesCompactArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_kernel(pages_map_kernel, dim3(kPagesCluster), dim3(kPagesThreads), 0, stream, true, a);
  if (e != cudaSuccess || a.src.n_seq == 0) return e;
  const int64_t stretches = (a.dst.max_pages + kTableEntries - 1) / kTableEntries;
  const int64_t grid = std::min<int64_t>(a.src.n_seq * stretches, 8 * num_sms);
  return launch_kernel(pages_table_kernel, dim3(static_cast<unsigned>(grid)), dim3(kTableThreads), 0, stream, true, a,
                       static_cast<int>(stretches));
}

}  // namespace strata
