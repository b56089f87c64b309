// Page tables of a cache on the device: room for new tokens, sequences that share pages, pages that are given back,
// and the move to another pool. The state is the table, the lengths and `refs`, the number of table entries
// that name each page; a page is free where that is zero. There is no list of free pages: the lowest free ones are
// taken in the order of the sequences, so the same calls give the same tables, whatever ran at the same time, and
// pools stay packed. Integer counts are added with atomics, whose order does not matter.
//
// What these calls move is small (4 bytes a page of the pool, 4 to 12 bytes a table entry): the chain of dependent
// steps is the time. Allocation needs sums over all pages and over all sequences before anybody can write, so one
// block does a whole call, or one cluster of eight with the cluster's barrier between its steps: one launch, no
// workspace, no counters in memory to wait for. (The figures are at kAlonePages; a release or a fork of 288 sequences takes
// 2 us. A first version, the cluster for every size with its sums one block after another, took 11 us for 8 sequences.)
#include <algorithm>

#include "pages.cuh"

namespace strata {

namespace {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}
// A word of block `rank` of the cluster, at this block's address of it.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, int rank) {
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t theirs, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(theirs) : "r"(mine), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(theirs) : "memory");
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
template <int kBlocks>
__host__ __device__ constexpr int64_t share_of(int64_t n, int chunk) {
  return ((n + kBlocks - 1) / kBlocks + chunk - 1) / chunk * chunk;
}
template <int kBlocks>
__device__ __forceinline__ Range range_of(int64_t n, int chunk, int rank) {
  const int64_t per = share_of<kBlocks>(n, chunk), lo = min(n, rank * per);
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
  const int shift = shift_of(p), fresh = a.new_tokens[s], len = p.kv_len[s];
  Ask k{0, 0, 0};
  if (fresh == 0) return k;
  if (fresh < 0 || len < 0 || fresh > p.max_pages * p.page_size - len) {
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

// Slots and positions of rows: a thread looks for the last sequence whose first row is not after its row.
template <int kBlocks, int U>
__device__ __forceinline__ void lay_out_rows(const PagesExtendArgs& a, const int32_t* row_at, int R, int rank) {
  const strata_kv_pages& p = a.p;
  const int n_seq = p.n_seq, shift = shift_of(p);
  auto start_of = [&](int s) { return kBlocks == 1 ? row_at[s] : __ldcg(a.q_start + s); };
  const int top = n_seq > 1 ? 1 << (31 - __clz(n_seq - 1)) : 0;
#pragma unroll 1
  for (int r0 = rank * kPagesThreads + threadIdx.x; r0 < a.T_max; r0 += U * kBlocks * kPagesThreads) {
    int of[U] = {}, pos[U], slot[U];
    auto row = [&](int j) { return r0 + j * kBlocks * kPagesThreads; };
#pragma unroll 1
    for (int d = top; d > 0; d >>= 1)
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int s = of[j] + d;
        if (row(j) < R && s < n_seq && start_of(s) <= row(j)) of[j] = s;
      }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      pos[j] = 0;
      if (row(j) < R)
        pos[j] = __ldcg(p.kv_len + of[j]) - ((of[j] + 1 < n_seq ? start_of(of[j] + 1) : R) - row(j));
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      slot[j] = -1;
      if (row(j) < R)
        slot[j] = (__ldcg(p.page_table + of[j] * p.table_stride + (pos[j] >> shift)) << shift) + (pos[j] & (p.page_size - 1));
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (row(j) >= a.T_max) break;
      a.slots[row(j)] = slot[j];
      a.positions[row(j)] = pos[j];
    }
  }
}

// Sequences in order get room while pages and rows last. need <= rows for each (a page is for one new token at
// least, the page that a shared one moves to among them), so the list of pages has room where the rows' slots
// will be. Sums stop at kMost, which is above every limit: what is beyond is refused, and nothing overflows.
// kBlocks: a cluster, or one block where a barrier between its threads costs less than the SMs that it does without.
constexpr uint32_t kMost = 1u << 28;
__device__ __forceinline__ uint32_t add_most(uint32_t a, uint32_t b) { return min(a + b, kMost); }

constexpr int kLaneNeed = 2;  // pages that a lane writes for its sequence by itself

template <int kBlocks>
__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kPagesThreads) pages_extend_kernel(PagesExtendArgs a) {
  extern __shared__ int32_t seq_smem[];  // [3][share]: rows (negative: and the page moves), first row, first page
  __shared__ uint32_t s_a[32], s_b[32], s_c[32], s_d[32];
  __shared__ int s_scan[32];
  __shared__ uint32_t s_total[3], s_got[3];  // for the cluster: free pages, rows, pages; rows, pages, moves that are given
  griddep_wait();
  griddep_launch();
  const strata_kv_pages& p = a.p;
  const int rank = kBlocks == 1 ? 0 : blockIdx.x, shift = shift_of(p), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_seq = p.n_seq, share = static_cast<int>(share_of<kBlocks>(n_seq, kPagesThreads));
  int32_t *rows_of = seq_smem, *row_at = seq_smem + share, *page_at = seq_smem + 2 * share;
  const Range seqs = range_of<kBlocks>(n_seq, kPagesThreads, rank);
  const Range pages = range_of<kBlocks>(p.n_pages, kPageChunk, rank);
  const int my_seqs = static_cast<int>(seqs.hi - seqs.lo);

  // ---- free pages of this block's share, and what its sequences ask for
  uint32_t free = 0;
  for (int64_t at = pages.lo + 4 * threadIdx.x; at < pages.hi; at += kPageChunk) {
    const int4 r = four_refs(p.refs, at, pages.hi);
    free += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  free = __reduce_add_sync(0xffffffffu, free);
  if (lane == 0) s_c[warp] = free;
  uint32_t rows_sum = 0, need_sum = 0;
  for (int i0 = 0; i0 < my_seqs; i0 += kPagesThreads) {
    const int i = i0 + threadIdx.x;
    const Ask k = i < my_seqs ? ask_of(a, static_cast<int>(seqs.lo) + i) : Ask{0, 0, 0};
    const uint32_t rows = min(static_cast<uint32_t>(k.rows), kMost), need = k.need;
    uint32_t r1 = rows, n1 = need;  // inclusive sums
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, r1, d), y = __shfl_up_sync(0xffffffffu, n1, d);
      if (lane >= d) r1 = add_most(r1, x), n1 = add_most(n1, y);
    }
    if (lane == 31) s_a[warp] = r1, s_b[warp] = n1;
    __syncthreads();
    uint32_t rw = s_a[lane], nw = s_b[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, rw, d), y = __shfl_up_sync(0xffffffffu, nw, d);
      if (lane >= d) rw = add_most(rw, x), nw = add_most(nw, y);
    }
    const uint32_t r_before = __shfl_sync(0xffffffffu, rw, max(warp - 1, 0)), n_before = __shfl_sync(0xffffffffu, nw, max(warp - 1, 0));
    if (warp > 0) r1 = add_most(r1, r_before), n1 = add_most(n1, n_before);
    if (i < my_seqs) {
      rows_of[i] = k.moved ? -k.rows : k.rows;
      // (exact below kMost, and refused from there on)
      row_at[i] = add_most(rows_sum, r1) < kMost ? rows_sum + r1 - rows : kMost;
      page_at[i] = add_most(need_sum, n1) < kMost ? need_sum + n1 - need : kMost;
    }
    rows_sum = add_most(rows_sum, __shfl_sync(0xffffffffu, rw, 31));
    need_sum = add_most(need_sum, __shfl_sync(0xffffffffu, nw, 31));
    __syncthreads();
  }
  __syncthreads();
  free = __reduce_add_sync(0xffffffffu, s_c[lane]);
  // what the blocks before this one have, and all of them (lane b asks block b)
  uint32_t free_before = 0, rows_before = 0, pages_before = 0, free_all = free;
  if constexpr (kBlocks > 1) {
    if (threadIdx.x == 0) s_total[0] = free, s_total[1] = rows_sum, s_total[2] = need_sum;
    cluster_sync();
    const uint32_t f = lane < kBlocks ? cluster_load(s_total, lane) : 0;
    free_all = __reduce_add_sync(0xffffffffu, f);
    free_before = __reduce_add_sync(0xffffffffu, lane < rank ? f : 0);
    rows_before = __reduce_add_sync(0xffffffffu, lane < rank ? cluster_load(s_total + 1, lane) : 0);
    pages_before = __reduce_add_sync(0xffffffffu, lane < rank ? cluster_load(s_total + 2, lane) : 0);
  }
  // ---- who gets room: sums only grow, so it is the sequences up to some place. Rows and pages up to there.
  uint32_t rows_got = 0, pages_got = 0, moves = 0;
  for (int i = threadIdx.x; i < my_seqs; i += kPagesThreads) {
    const int n = abs(rows_of[i]);
    const uint32_t r1 = rows_before + row_at[i] + min(static_cast<uint32_t>(n), kMost);
    const int len = length_of(p, p.kv_len[seqs.lo + i], nullptr);
    const int need = n > 0 ? pages_of(len + n, shift) - pages_of(len, shift) + (rows_of[i] < 0) : 0;
    const uint32_t p1 = pages_before + page_at[i] + need;
    if (r1 <= static_cast<uint32_t>(a.T_max) && p1 <= free_all) {
      rows_got = max(rows_got, r1);
      pages_got = max(pages_got, p1);
      moves += rows_of[i] < 0;
    } else {
      if (n > 0) set_status(a.status, STRATA_DEV_NO_PAGES);
      rows_of[i] = 0;
    }
  }
  rows_got = __reduce_max_sync(0xffffffffu, rows_got);
  pages_got = __reduce_max_sync(0xffffffffu, pages_got);
  moves = __reduce_add_sync(0xffffffffu, moves);
  if (lane == 0) s_a[warp] = rows_got, s_b[warp] = pages_got, s_d[warp] = moves;
  __syncthreads();
  rows_got = __reduce_max_sync(0xffffffffu, s_a[lane]);
  pages_got = __reduce_max_sync(0xffffffffu, s_b[lane]);
  moves = __reduce_add_sync(0xffffffffu, s_d[lane]);
  uint32_t moves_before = 0;
  if constexpr (kBlocks > 1) {
    if (threadIdx.x == 0) s_got[0] = rows_got, s_got[1] = pages_got, s_got[2] = moves;
    cluster_sync();
    rows_got = __reduce_max_sync(0xffffffffu, lane < kBlocks ? cluster_load(s_got, lane) : 0);
    pages_got = __reduce_max_sync(0xffffffffu, lane < kBlocks ? cluster_load(s_got + 1, lane) : 0);
    const uint32_t m = lane < kBlocks ? cluster_load(s_got + 2, lane) : 0;
    moves_before = __reduce_add_sync(0xffffffffu, lane < rank ? m : 0);
    moves = __reduce_add_sync(0xffffffffu, m);
  }
  const int R = static_cast<int>(rows_got);
  // ---- the lowest free pages, in order: noted where the slots will be
  uint32_t at_free = free_before;
  for (int64_t c = pages.lo; c < pages.hi && at_free < pages_got; c += kPageChunk) {
    const int64_t at = c + 4 * threadIdx.x;
    const int4 r = at < pages.hi ? four_refs(p.refs, at, pages.hi) : make_int4(-1, -1, -1, -1);
    const int here = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int total;
    uint32_t k = at_free + block_scan(here, s_scan, total) - here;
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
  if constexpr (kBlocks > 1) cluster_sync();
  else __syncthreads();
  // ---- tables and lengths: a lane a sequence, a warp where one has many pages
  for (int i0 = 0; i0 < my_seqs; i0 += kPagesThreads) {
    const int i = i0 + threadIdx.x, s = static_cast<int>(seqs.lo) + i;
    const bool on = i < my_seqs;
    const int n = on ? abs(rows_of[i]) : 0, moved = on && rows_of[i] < 0;
    const int len = n > 0 ? length_of(p, p.kv_len[s], nullptr) : 0;
    const int first = pages_of(len, shift) - moved;
    const int need = n > 0 ? pages_of(len + n, shift) - first : 0;
    const int from = n > 0 ? static_cast<int>(pages_before) + page_at[i] : 0;
    int32_t* row = p.page_table + static_cast<int64_t>(on ? s : 0) * p.table_stride;
    if (moves > 0) {
      int total;
      const uint32_t m = moves_before + block_scan(moved, s_scan, total) - moved;
      moves_before += total;
      if (moved) {
        const int old = row[first], page = __ldcg(a.slots + from);
        atomicAdd(p.refs + old, -1);
        a.copies[2 * m] = old;
        a.copies[2 * m + 1] = page;
      }
    }
    if (on) {
      const int q = static_cast<int>(min(rows_before + row_at[i], rows_got));
      a.q_start[s] = row_at[i] = q;  // (the block's place for it is read again below, if it is alone)
    }
    if (n > 0) p.kv_len[s] = len + n;
    if (need <= kLaneNeed) {
      int page[kLaneNeed];
#pragma unroll
      for (int e = 0; e < kLaneNeed; ++e) page[e] = e < need ? __ldcg(a.slots + from + e) : 0;
#pragma unroll
      for (int e = 0; e < kLaneNeed; ++e)
        if (e < need) row[first + e] = page[e];
    }
    for (unsigned many = __ballot_sync(0xffffffffu, need > kLaneNeed); many; many &= many - 1) {
      const int l = __ffs(many) - 1;
      const int64_t at = __shfl_sync(0xffffffffu, static_cast<int64_t>(row - p.page_table), l);
      const int f = __shfl_sync(0xffffffffu, first, l), k = __shfl_sync(0xffffffffu, need, l);
      const int src = __shfl_sync(0xffffffffu, from, l);
      for (int e = lane; e < k; e += 32) p.page_table[at + f + e] = __ldcg(a.slots + src + e);
    }
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.q_start[n_seq] = R;
    *a.n_copies = static_cast<int32_t>(moves);
  }
  if constexpr (kBlocks > 1) cluster_sync();
  else __syncthreads();
  // ---- the rows, each by itself (the list of pages is not needed any more); four of a thread at a time if it has some
  if (a.T_max <= kBlocks * kPagesThreads) lay_out_rows<kBlocks, 1>(a, row_at, R, rank);
  else lay_out_rows<kBlocks, 4>(a, row_at, R, rank);
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
template <int kBlocks>
__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kPagesThreads) pages_map_kernel(PagesCompactArgs a) {
  __shared__ uint32_t s_total;
  __shared__ int s_scan[32];
  griddep_wait();
  griddep_launch();
  const int rank = kBlocks == 1 ? 0 : blockIdx.x;
  const Range pages = range_of<kBlocks>(a.src.n_pages, kPageChunk, rank);
  int live = 0, total;
  for (int64_t at = pages.lo + 4 * threadIdx.x; at < pages.hi; at += kPageChunk) {
    const int4 r = four_refs(a.src.refs, at, pages.hi);
    live += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  block_scan(live, s_scan, total);
  uint32_t before = 0, all = total;
  if constexpr (kBlocks > 1) {
    if (threadIdx.x == 0) s_total = total;
    cluster_sync();
    const int lane = threadIdx.x & 31;
    const uint32_t n = lane < kBlocks ? cluster_load(&s_total, lane) : 0;
    before = __reduce_add_sync(0xffffffffu, lane < rank ? n : 0);
    all = __reduce_add_sync(0xffffffffu, n);
  } else {
    __syncthreads();  // (all have read the sums)
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
       i += kBlocks * kPagesThreads)
    a.dst.refs[i] = 0;
  if (rank == 0 && threadIdx.x == 0) {
    *a.n_copies = fits ? static_cast<int32_t>(all) : 0;
    *a.live = fits ? static_cast<int32_t>(all) : -1;
    if (!fits) set_status(a.status, STRATA_DEV_NO_PAGES);
  }
  if constexpr (kBlocks > 1) cluster_sync();  // (nobody leaves while another reads its total)
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

// Up to so many pages and rows, and a sequence a thread, one block makes room alone. (us, alone / the cluster, a row a sequence:
// 256 pages, 8 sequences 5.3 / 10.0; 16384, 256 7.1 / 10.6; 32768, 256 9.3 / 11.1; 49152, 256 11.4 / 12.5; 65536, 256 13.6 / 12.1;
// 262144, 8 37 / 17. More rows: 4096 pages, 8 sequences, 4096 rows 9.1 / 12.4, 8000 10.8 / 12.5, 16384 14.8 / 13.1; 16384 pages,
// 288 sequences, 3456 rows 9.7 / 11.8, 8064 13.1 / 12.0; 1000 sequences, 4000 rows 10.4 / 12.8, 16000 18.6 / 13.4.) Numbering pages
// goes over each of them twice (with the tables of 60 sequences: 500 pages 4.6 / 5.9, 4096 9.7 / 10.8, 6000 12.6 / 11.1, 12000
// 21.9 / 10.9).
constexpr int64_t kAlonePages = 32768, kAloneMapPages = 4096;
constexpr int kAloneRows = 4096;

}  // namespace

template <int kBlocks>
constexpr size_t extend_smem(int n_seq) {  // (up to 96 KB)
  return 3 * sizeof(int32_t) * share_of<kBlocks>(n_seq, kPagesThreads);
}
template <int kBlocks>
static cudaError_t launch_extend(const PagesExtendArgs& a, cudaStream_t stream) {
  const size_t smem = extend_smem<kBlocks>(a.p.n_seq);
  // The limit is what the largest call takes, not this one: threads with calls of different sizes share it.
  constexpr size_t most = extend_smem<kBlocks>(kBlocks == 1 ? kPagesThreads : kPagesMostSeq);
  if (smem > 40 << 10) {
    const cudaError_t e = cudaFuncSetAttribute(pages_extend_kernel<kBlocks>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(most));
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(pages_extend_kernel<kBlocks>, dim3(kBlocks), dim3(kPagesThreads), smem, stream, true, a);
}
cudaError_t launch_pages_extend(const PagesExtendArgs& a, cudaStream_t stream) {
  const bool alone = a.p.n_seq <= kPagesThreads && a.p.n_pages <= kAlonePages && a.T_max <= kAloneRows;
  return alone ? launch_extend<1>(a, stream) : launch_extend<kPagesCluster>(a, stream);
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
  const bool alone = a.src.n_pages <= kAloneMapPages && a.dst.n_pages <= kAloneMapPages;
  const cudaError_t e = launch_kernel(alone ? pages_map_kernel<1> : pages_map_kernel<kPagesCluster>,
                                      dim3(alone ? 1 : kPagesCluster), dim3(kPagesThreads), 0, stream, true, a);
  if (e != cudaSuccess || a.src.n_seq == 0) return e;
  // (a table without entries has its lengths written)
  const int64_t stretches = std::max<int64_t>(1, (a.dst.max_pages + kTableEntries - 1) / kTableEntries);
  const int64_t grid = std::min<int64_t>(a.src.n_seq * stretches, 8 * num_sms);
  return launch_kernel(pages_table_kernel, dim3(static_cast<unsigned>(grid)), dim3(kTableThreads), 0, stream, true, a,
                       static_cast<int>(stretches));
}

}  // namespace strata
