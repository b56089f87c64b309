// Causal attention over the paged cache of e4m3 codes with one scale per (page, K/V head):
//   o_i = sum_j softmax_j(scale * q_i . k_j) v_j   over the tokens j that query i sees,
// by one pass over the cache with a running reference and sum of the softmax.
//
// For few query rows the cache is the traffic, so the kernel streams it: each warp copies its own
// 32-token steps with cp.async into two private slots of shared memory (no block-wide waits) and
// multiplies one while the other fills. Rows of a K/V head (query rows x query heads that share it) are
// the N side of mma.sync m16n8k16 and 16 tokens its M side: S^T = K Q^T, then O^T += V^T P^T. Codes become
// f16 in registers, exactly (cvt e4m3x2 -> f16x2). The order of the contraction over a head's elements
// is free, so a lane takes 16 consecutive bytes of a K row; V bytes are paired token by token with
// PRMT, and the weights turn from S^T's layout to P^T's with movmatrix.
//
// Queries are f16, exact from bf16 (rows are held times a power of two); weights, with the page's V scale in their
// exponent (attention.cuh), are f16 (2^-11); sums, statistics and scales are fp32. The reference that is
// subtracted in the exponent moves only when one exceeds it by 8: weights up to 2^8 are as exact in f16 and the
// sums fp32, and the common step needs no reduction across lanes and no rescaling of O.
//
// The work is cut by the lengths that the call finds on the device, in one of two ways.
// Up to 228 pairs of (sequence, K/V head): a pair whose steps exceed an even share of all steps is cut into
// equal pieces, and a block takes one piece; its warps join in shared memory. The share is the smallest of
// three with which all blocks start at once: rounding up adds half a block a pair for mixed lengths, a
// whole one at worst. (Eight heads of 16 sequences of 8192: 512 blocks for 456 places took 66 us, 384 take 51.)
// More pairs: each warp takes an even share of all steps, through the middle of pairs, and goes through its
// pairs alone, copying ahead from one to the next. Blocks that start in later waves cost the time to find
// their work, fill their slots and join, about 8 us a wave: 500 sequences of 300 231 us against 74, 256 of
// 1000 118 against 97, 64 of 4096 106 against 99. With few pairs a share means two joins, one after the
// other, without help from other warps: 24 sequences of 8192 82 us against 70, one of 200 14 against 6.
// Either way pieces leave reference, sum and fp32 rows in the workspace, the last to arrive in a
// group of up to 8 (or the root of the count) joins the group's, and the last group the groups'. All sums are
// in the order of the pieces.
//
// Bound by memory, but for its start and end: 8 sequences of 131072 tokens 326 us (6.6 TB/s), one 51 us (5.2 TB/s), of
// which about 9 us are launch, the search for the piece, the first copies and the join.
#include <algorithm>

#include "attention.cuh"

namespace strata {

constexpr int kAttWarps = 4;
constexpr int kAttStep = 32;  // tokens of one warp step
constexpr int kAttSlots = 2;  // steps of a warp in shared memory
// A pair of up to kAttWholeSteps, two a warp, is not cut: a second step takes less than the join. Longer ones may
// be cut down to kAttMinSteps, one a warp. (us, pieces of 4 steps at least / of 8: 200 tokens 6.7 / 6.2,
// 500 7.2 / 8.0, 1000 7.6 / 8.3; of 16: 6.2, 8.5, 10.0.)
constexpr int kAttWholeSteps = 8, kAttMinSteps = 4;
constexpr int kAttMinShare = 2;      // steps that a warp's share has at least (200 sequences of 50: 2 12.3 us, 4 18.7)
constexpr int kAttResident = 456;    // blocks that run at once: three on each of 152 SMs

// Transposes an 8x8 matrix of 16-bit elements held one row per quad.
__device__ __forceinline__ uint32_t movm_trans(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// D += A * B, m16n8k16, f16 inputs, fp32 sums. (Not volatile: the compiler may interleave independent chains.)
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory, or zeros when there is nothing to copy.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

// Which token of a 16-token tile is row i (< 8) of an MMA tile, and i + 8 the one 8 further: chosen with
// the swizzle of the slots so that the lanes of a shared-memory phase read different banks, for K (rows i
// of a quad pair) and for V (rows 2t of the quads) alike.
template <int kD>
__device__ __forceinline__ int tile_token(int i) {
  // 128-wide: rows {0,4} {2,6} {5,1} {7,3}; 64-wide: {0,1} {3,2} {4,5} {7,6}
  return (kD == 128 ? 0x37156240u : 0x67542310u) >> (4 * i) & 15;
}
// Byte offset of 16-byte piece c of token row r in a slot.
template <int kD>
__device__ __forceinline__ int slot_offset(int r, int c) {
  return r * kD + ((c ^ (kD == 128 ? r & 7 : (r >> 1) & 2)) << 4);
}

// The steps of 32 tokens that a sequence's rows see; none if this kernel skips it.
template <bool kSink>
__device__ __forceinline__ Span<kSink> seq_steps(const AttnArgs& a, const SeqView& v) {
  const int64_t rows = static_cast<int64_t>(v.n) * a.group;
  if (rows == 0 || rows > a.rows_above) return {0, 0, 0, 0};
  Span<kSink> s = span_of<kSink, kAttStep>(a, first_seen(a, v.len - v.n), v.len);
  s.n = max(1, s.n);  // (no tokens: one empty step, zeros)
  return s;
}

__device__ __forceinline__ int pieces_of(int steps, int per) {
  return steps <= kAttWholeSteps ? (steps + kAttWholeSteps - 1) / kAttWholeSteps : (steps + per - 1) / per;
}
// This block's piece: found by a scan over the sequences, the same in every block.
struct Piece {
  int seq, head, index, of;  // piece `index` of `of`
  int slot0;                 // workspace slot of the (sequence, head)'s piece 0, if of > 1
};
template <bool kSink>
__device__ __forceinline__ bool find_piece(const AttnArgs& a, Piece& p) {
  if (a.b.n_seq == 1) {
    const int steps = seq_steps<kSink>(a, seq_view(a, 0, blockIdx.x == 0 && threadIdx.x == 0)).n, heads = a.c.n_kv_heads;
    int k = 1;
    for (int q = 2; q <= 4; ++q) {
      const int pieces = kAttResident - heads * q / 4;
      const int per = max(kAttMinSteps, static_cast<int>((static_cast<int64_t>(steps) * heads + pieces - 1) / pieces));
      k = pieces_of(steps, per);
      if (k * heads <= kAttResident) break;
    }
    if (static_cast<int>(blockIdx.x) >= k * heads) return false;
    const int head = blockIdx.x / k;
    p = {0, head, static_cast<int>(blockIdx.x) - head * k, k, head * k};
    return true;
  }
  // every warp scans for itself: a lane takes consecutive sequences
  const int lane = threadIdx.x & 31;
  const int per_lane = (a.b.n_seq + 31) / 32;
  const int s0 = min(a.b.n_seq, lane * per_lane), s1 = min(a.b.n_seq, s0 + per_lane);
  const bool flag = blockIdx.x == 0 && threadIdx.x < 32;
  int mine = 0;
  for (int s = s0; s < s1; ++s) mine += seq_steps<kSink>(a, seq_view(a, s, flag)).n;
  const int kept = mine;  // per_lane == 1: the lane's steps
  const int heads = a.c.n_kv_heads, pairs = heads * a.b.n_seq;
  const unsigned total = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine)) * heads;  // < 2^31 (host)
  int per = 0, blocks = 0, slots = 0;
  // blocks and workspace slots that a sequence's steps come to
  auto count = [&](int steps, int& blocks, int& slots) {
    const int k = pieces_of(steps, per) * heads;
    blocks += k;
    slots += k > heads ? k : 0;
  };
  // the smallest pieces of three that still start together
  for (int q = 2; q <= 4; ++q) {
    const int pieces = kAttResident - pairs * q / 4;
    per = max(kAttMinSteps, static_cast<int>((total + pieces - 1) / pieces));
    blocks = slots = 0;
    for (int s = s0; s < s1; ++s) count(per_lane == 1 ? kept : seq_steps<kSink>(a, seq_view(a, s, false)).n, blocks, slots);
    if (__reduce_add_sync(0xffffffffu, static_cast<unsigned>(blocks)) <= kAttResident) break;
  }
  int b_at = blocks, s_at = slots;  // inclusive scans
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, b_at, d), y = __shfl_up_sync(0xffffffffu, s_at, d);
    if (lane >= d) b_at += x, s_at += y;
  }
  const int id = blockIdx.x;
  const unsigned here = __ballot_sync(0xffffffffu, id < b_at);
  if (here == 0) return false;
  const int owner = __ffs(here) - 1;
  int seq = 0, local = 0, k = 1, slot0 = 0;
  if (lane == owner) {
    int b0 = b_at - blocks, l0 = s_at - slots;
    for (int s = s0; s < s1; ++s) {
      const int steps = per_lane == 1 ? kept : seq_steps<kSink>(a, seq_view(a, s, false)).n;
      int nb = 0, ns = 0;
      count(steps, nb, ns);
      if (id < b0 + nb) {
        seq = s;
        local = id - b0;
        k = pieces_of(steps, per);
        slot0 = l0;
        break;
      }
      b0 += nb;
      l0 += ns;
    }
  }
  seq = __shfl_sync(0xffffffffu, seq, owner);
  local = __shfl_sync(0xffffffffu, local, owner);
  k = __shfl_sync(0xffffffffu, k, owner);
  slot0 = __shfl_sync(0xffffffffu, slot0, owner);
  p = {seq, local / k, local % k, k, slot0 + local / k * k};
  return true;
}

// A place in the list of all steps: step `at` of the n of (sequence, head); sequences in order, heads within.
template <bool kSink>
struct Walk {
  int seq, head, at;
  Span<kSink> st;
  SeqView v;
  __device__ __forceinline__ void open(const AttnArgs& a, int s) {
    seq = s;
    v = seq_view(a, s, false);
    st = seq_steps<kSink>(a, v);
  }
  // Moves on by m steps of this head, which has at least as many left. (Not called past the last step.)
  __device__ __forceinline__ void move(const AttnArgs& a, int m) {
    at += m;
    if (at < st.n) return;
    at = 0;
    if (++head < a.c.n_kv_heads) return;
    head = 0;
    do open(a, seq + 1);
    while (st.n == 0 && seq + 1 < a.b.n_seq);
  }
};
// This warp's share of all steps: `per` of them from number `warp * per` on, and where that is.
struct Share {
  int per, total, todo;
};
template <bool kSink>
__device__ __forceinline__ bool find_share(const AttnArgs& a, Share& sh, Walk<kSink>& w) {
  const int lane = threadIdx.x & 31, heads = a.c.n_kv_heads;
  const int per_lane = (a.b.n_seq + 31) / 32;
  const int s0 = min(a.b.n_seq, lane * per_lane), s1 = min(a.b.n_seq, s0 + per_lane);
  const bool flag = blockIdx.x == 0 && threadIdx.x < 32;
  int mine = 0;
  for (int s = s0; s < s1; ++s) mine += seq_steps<kSink>(a, seq_view(a, s, flag)).n * heads;
  int end = mine;  // inclusive scan
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, end, d);
    if (lane >= d) end += x;
  }
  sh.total = __shfl_sync(0xffffffffu, end, 31);  // < 2^31 (host)
  const int warps = gridDim.x * kAttWarps, id = blockIdx.x * kAttWarps + (threadIdx.x >> 5);
  sh.per = max(kAttMinShare, (sh.total + warps - 1) / warps);
  const int64_t from = static_cast<int64_t>(id) * sh.per;
  if (from >= sh.total) return false;
  const int begin = static_cast<int>(from);
  sh.todo = min(sh.per, sh.total - begin);
  const int owner = __ffs(__ballot_sync(0xffffffffu, begin < end)) - 1;
  int seq = 0, left = begin - (end - mine);
  if (lane == owner) {
    for (seq = s0; seq < s1; ++seq) {
      const int n = seq_steps<kSink>(a, seq_view(a, seq, false)).n * heads;
      if (left < n) break;
      left -= n;
    }
  }
  seq = __shfl_sync(0xffffffffu, seq, owner);
  left = __shfl_sync(0xffffffffu, left, owner);
  w.open(a, seq);
  w.head = left / w.st.n;
  w.at = left % w.st.n;
  return true;
}

// kSolo: each warp takes an even share of all steps and goes through its (sequence, head) pairs alone.
// Otherwise a block takes one piece of a pair.
// kSink: there is a window, and a.sinks first tokens that stay visible before it.
template <int kD, int kNT, bool kSolo, bool kSink>
__global__ void __launch_bounds__(kAttWarps * 32, 3) attention_kernel(AttnArgs a) {
  constexpr int COLS = 8 * kNT;
  constexpr int KW = kD / 64;       // 16-byte pieces of a K row per lane
  constexpr int VW = kD / 32;       // words of a V row per lane
  constexpr int NJ = 2 * VW;        // output MMAs per token tile
  constexpr int KB = kAttStep * kD; // bytes of a step's K (and V)
  constexpr float kLag = 8.0f;      // how far a score may exceed the reference (log2)
  extern __shared__ __align__(1024) uint8_t att_smem[];
  // Beside the tensor-core kernel of the same call (launched first) this one starts at once: that kernel's
  // blocks have all waited for what came before the call. It still ends after it, so that whoever
  // waits for this kernel has waited for both.
  if (!a.beside) griddep_wait();
  griddep_launch();
  struct Last {
    bool wait;
    __device__ ~Last() { if (wait) griddep_wait(); }
  } last_wait{a.beside};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = a.group;
  Piece pc;
  Walk<kSink> now{}, ahead{};  // (kSolo) the step at hand, and the next to copy
  Share share;
  int h, s, rows;   // the (sequence, head) at hand and its rows: <= COLS
  SeqView sv;
  int p_lo, p_hi;   // positions of the first and last query
  int lo, hi;       // the tokens of the piece (kSink: numbers of steps times 32, and the sequence's tokens)
  int to = 0;       // (kSink) the last number of the piece, times 32
  Span<kSink> span{};
  int seen_lo = 0;  // first token that a row sees
  auto take = [&](int seq, int head, const SeqView& v) {
    s = seq, h = head, sv = v, rows = v.n * G;
    p_lo = v.len - v.n, p_hi = v.len - 1;
  };
  if constexpr (kSolo) {
    if (!find_share(a, share, now)) return;
    ahead = now;
  } else {
    if (!find_piece<kSink>(a, pc)) return;
    take(pc.seq, pc.head, seq_view(a, pc.seq, false));
    span = seq_steps<kSink>(a, sv);
    seen_lo = first_seen(a, sv.len - sv.n);
    lo = (span.first + static_cast<int>(static_cast<int64_t>(span.n) * pc.index / pc.of)) * kAttStep;
    to = (span.first + static_cast<int>(static_cast<int64_t>(span.n) * (pc.index + 1) / pc.of)) * kAttStep;
    hi = kSink ? sv.len : min(sv.len, to);
  }

  // ---- copies: a lane moves piece lane % PIECES of rows lane / PIECES, + 32 / PIECES, ...
  constexpr int PIECES = kD / 16, RPI = 32 / PIECES, NI = kAttStep / RPI;
  const int pshift = 31 - __clz(a.c.page_size), pmask = a.c.page_size - 1;
  uint8_t* ring = att_smem + warp * (kAttSlots * 2 * KB);
  const uint32_t ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  // of each slot's two tiles: K scale, V scale (negative: the tile lies in a page that does not exist)
  __shared__ float2 s_scale[kAttWarps][kAttSlots][2];
  const uint32_t scale_addr = static_cast<uint32_t>(__cvta_generic_to_shared(&s_scale[warp][0][0]));
  // (tokens lo .. hi - 1 are the ones that a row sees: of the others nothing is looked up or used)
  // where step number n / 32 of the block's pair begins, and whether it is the piece's
  auto ours = [&](int n) { return n < (kSink ? to : hi); };
  auto token = [&](int n) { return kSink && n >= span.gap_at * kAttStep ? n + span.gap * kAttStep : n; };
  auto issue = [&](int s, int h, int lo, int hi, int j0, int i_slot) {
    const int32_t* table = a.b.page_table + static_cast<int64_t>(s) * a.b.table_stride;
    const uint32_t slot = ring_addr + i_slot * 2 * KB;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = j0 + 16 * u;
      int page = -1;
      if (j < hi && (kSink ? j + 16 > lo || j < a.sinks : j + 16 > lo)) {
        page = input(a, table + (j >> pshift));
        if (page < 0 || page >= a.c.n_pages) {
          if (lane == 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
          page = -2;
        }
      }
      const int64_t ph = page < 0 ? 0 : static_cast<int64_t>(page) * a.c.n_kv_heads + h;
      // (the scales arrive with the codes: waiting for them here would cost a warp a DRAM latency per step)
      if (page >= 0 && !a.beside) {
        if (lane < 2) copy4(scale_addr + (i_slot * 2 + u) * 8 + lane * 4, (lane ? a.c.v_scales : a.c.k_scales) + ph);
      } else if (lane == 0) {
        s_scale[warp][i_slot][u] = page < 0 ? make_float2(0.f, page == -2 ? -1.f : 0.f)
                                            : make_float2(__ldcg(a.c.k_scales + ph), __ldcg(a.c.v_scales + ph));
      }
      const int64_t base = ((ph << pshift) + (j & pmask)) * kD + lane * 16;
      const int m = lo - j, n = page < 0 ? 0 : hi - j;  // rows m .. n - 1 of the tile; zeros elsewhere
#pragma unroll
      for (int i = 0; i < NI / 2; ++i) {
        const int r = lane / PIECES + RPI * i;
        const uint32_t dst = slot + slot_offset<kD>(16 * u + r, lane % PIECES);
        const bool on = (kSink ? r >= m || j + r < a.sinks : r >= m) && r < n;
        const int64_t at = on ? base + i * 512 : 0;
        copy16(dst, a.c.k_codes + at, on);
        copy16(dst + KB, a.c.v_codes + at, on);
      }
    }
  };
  int j_next = 0, to_copy = 0;
  auto issue_ahead = [&](int i_slot) {
    issue(ahead.seq, ahead.head, first_seen(a, ahead.v.len - ahead.v.n), ahead.v.len,
          ahead.st.at(ahead.at) * kAttStep, i_slot);
    if (--to_copy > 0) ahead.move(a, 1);
  };
  if constexpr (kSolo) {
    to_copy = share.todo;
#pragma unroll 1
    for (int i = 0; i < kAttSlots; ++i) {
      if (to_copy > 0) issue_ahead(i);
      cp_async_commit();
    }
  } else {
    j_next = lo + warp * kAttStep;
#pragma unroll 1
    for (int i = 0; i < kAttSlots; ++i, j_next += kAttWarps * kAttStep) {
      if (ours(j_next)) issue(s, h, seen_lo, hi, token(j_next), i);
      cp_async_commit();
    }
  }

  // ---- the queries of column g of each tile as f16 B fragments, times 2^-e
  uint32_t qf[kNT][4 * KW][2];
  float cmul[kNT][2];   // columns 2t, 2t+1: what turns a product into the exponent of 2
  uint32_t after;       // their positions after p_lo, a byte each (at most 16 rows)
  auto load_queries = [&] {
    after = 0;
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const int r = n * 8 + g;
      uint4 v[2 * KW];
      uint32_t mag = 0;
#pragma unroll
      for (int i = 0; i < 2 * KW; ++i) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const __nv_bfloat16* q = a.q + static_cast<int64_t>(sv.q0 + r / G) * a.q_stride +
                                   (h * G + r % G) * kD + (i >> 1) * 64 + t * 16;
          v[i] = input(a, reinterpret_cast<const uint4*>(q) + (i & 1));
        }
        mag = max(mag, bf16x8_mag(v[i]));
      }
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
      const int e = row_exp(mag);
      const float sc = exp2i(-e);
#pragma unroll
      for (int i = 0; i < 2 * KW; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qf[n][2 * i + (j >> 1)][j & 1] = pack_f16x2(bf16_lo_f32(w[j]) * sc, bf16_hi_f32(w[j]) * sc);
      }
      const float m = a.scale_log2 * exp2i(e);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cmul[n][i] = __shfl_sync(0xffffffffu, m, (2 * t + i) * 4);
        after |= static_cast<uint32_t>((n * 8 + 2 * t + i) / G) << (16 * n + 8 * i);
      }
    }
  };

  float o[kNT][NJ][4];
  // ref: the reference in use, or 0 before any score; limit: how much of a score above it moves it
  float ref[kNT][2], limit[kNT][2], sum[kNT][2];
  float lv_top;  // largest log2 of a V scale
  auto reset = [&] {
    lv_top = -INFINITY;
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      ref[n][0] = ref[n][1] = 0.f;
      limit[n][0] = limit[n][1] = -INFINITY;
      sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
    }
  };
  const int tok_g = tile_token<kD>(g);
  // addresses of this lane's K rows and V rows in a slot, 16 tokens apart for the second tile
  int k_at[KW], v_at[2];
#pragma unroll
  for (int w = 0; w < KW; ++w) k_at[w] = slot_offset<kD>(tok_g, t + 4 * w);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = tile_token<kD>(2 * t + i);
    v_at[i] = KB + (kD == 128 ? slot_offset<kD>(r, g) : slot_offset<kD>(r, g >> 1) + (g & 1) * 8);
  }

  auto step = [&](int j0, int i_slot) {
    const uint8_t* slot = ring + i_slot * 2 * KB;
    const float2 sc0 = s_scale[warp][i_slot][0], sc1 = s_scale[warp][i_slot][1];
    const float k_scale[2] = {sc0.x, sc1.x}, lv[2] = {log2_scale(sc0.y), log2_scale(sc1.y)};
    lv_top = fmaxf(lv_top, fmaxf(lv[0], lv[1]));
    const int lost = (sc0.y < 0.f ? 1 : 0) | (sc1.y < 0.f ? 2 : 0);
    // S^T: tokens tok_g, tok_g + 8 of each tile x columns 2t, 2t+1
    float sc[kNT][2][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][u][i] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint32_t w0[2][4], w1[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // (8 and 16 rows further the swizzle is the same)
        const uint4 x = *reinterpret_cast<const uint4*>(slot + k_at[w] + 16 * u * kD);
        const uint4 y = *reinterpret_cast<const uint4*>(slot + k_at[w] + (16 * u + 8) * kD);
        w0[u][0] = x.x; w0[u][1] = x.y; w0[u][2] = x.z; w0[u][3] = x.w;
        w1[u][0] = y.x; w1[u][1] = y.y; w1[u][2] = y.z; w1[u][3] = y.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t A[4] = {e4m3x2_f16x2(w0[u][j]), e4m3x2_f16x2(w1[u][j]), e4m3x2_f16x2(w0[u][j] >> 16),
                                 e4m3x2_f16x2(w1[u][j] >> 16)};
#pragma unroll
          for (int n = 0; n < kNT; ++n) mma_add(sc[n][u], A, qf[n][4 * w + j][0], qf[n][4 * w + j][1]);
        }
    }
    const int from = a.window > 0 ? p_hi - a.window + 1 : 0;  // (the last row's window)
    const bool whole = (kSink ? j0 >= from || j0 + kAttStep <= a.sinks : j0 >= from) && j0 + kAttStep - 1 <= p_lo &&
                       j0 + kAttStep <= hi && !lost;
    // exponents relative to the reference (in use or 0)
    bool over = false;
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float f = cmul[n][c] * k_scale[u], base = lv[u] - ref[n][c];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaf(sc[n][u][2 * i + c], f, base);
            if (!whole) {
              const int r = tok_g + 8 * i, j = j0 + 16 * u + r;
              const int pos = p_lo + static_cast<int>(after >> (16 * n + 8 * c) & 255u);
              const bool near = a.window <= 0 || j > pos - a.window;
              const bool seen = j < hi && j <= pos && (kSink ? near || j < a.sinks : near) && !(lost >> u & 1);
              if (!seen) x = -INFINITY;
            }
            sc[n][u][2 * i + c] = x;
            over |= x > limit[n][c];
          }
        }
      }
    if (__any_sync(0xffffffffu, over)) {  // some column's reference moves to its largest exponent so far
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float up = fmaxf(fmaxf(sc[n][0][c], sc[n][0][2 + c]), fmaxf(sc[n][1][c], sc[n][1][2 + c]));
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 4));
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 8));
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16));
          const bool had = limit[n][c] == kLag;
          if (had) up = fmaxf(up, 0.f);   // a reference never falls
          if (up == -INFINITY) up = 0.f;  // nothing seen yet
          else limit[n][c] = kLag;
          ref[n][c] += up;
          const float f = had ? exp2_approx(-up) : 1.f;  // (without a reference the sums are 0, or nan)
          sum[n][c] = sum_times_exp2(sum[n][c], had ? -up : 0.f);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            o[n][j][c] *= f;
            o[n][j][2 + c] *= f;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            sc[n][u][c] -= up;
            sc[n][u][2 + c] -= up;
          }
        }
    }
    // O^T += V^T P^T, tile by tile (the scale is the page's)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t pf[kNT][2];
      const float per_scale = exp2_approx(-lv[u]);
      const bool small = lv[u] < lv_top - kFarScale;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = exp2_approx(sc[n][u][i]);
        if (!small) {
          sum[n][0] = fmaf(p[0] + p[2], per_scale, sum[n][0]);
          sum[n][1] = fmaf(p[1] + p[3], per_scale, sum[n][1]);
        } else {
          sum[n][0] += exp2_approx(sc[n][u][0] - lv[u]) + exp2_approx(sc[n][u][2] - lv[u]);
          sum[n][1] += exp2_approx(sc[n][u][1] - lv[u]) + exp2_approx(sc[n][u][3] - lv[u]);
        }
        pf[n][0] = movm_trans(pack_f16x2(p[0], p[1]));
        pf[n][1] = movm_trans(pack_f16x2(p[2], p[3]));
      }
      uint32_t vr[4][VW];  // tokens 2t, 2t+1, 2t+8, 2t+9 of the MMA's order
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* at = slot + v_at[i & 1] + (16 * u + 8 * (i >> 1)) * kD;
        if (kD == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(at);
          vr[i][0] = v.x; vr[i][1] = v.y; vr[i][VW - 2] = v.z; vr[i][VW - 1] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(at);
          vr[i][0] = v.x; vr[i][1] = v.y;
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;  // bytes 0,1 or 2,3 of two tokens' words
        const uint32_t x0 = prmt(vr[0][j >> 1], vr[1][j >> 1], sel);
        const uint32_t x1 = prmt(vr[2][j >> 1], vr[3][j >> 1], sel);
        const uint32_t A[4] = {e4m3x2_f16x2(x0), e4m3x2_f16x2(x0 >> 16), e4m3x2_f16x2(x1),
                               e4m3x2_f16x2(x1 >> 16)};
#pragma unroll
        for (int n = 0; n < kNT; ++n) mma_add(o[n][j], A, pf[n][0], pf[n][1]);
      }
    }
  };

  // ---- pieces that are joined through the workspace: by teams, a block or (kSolo) a warp
  constexpr int TEAM = kSolo ? 32 : kAttWarps * 32;
  constexpr int64_t PART = COLS * (kD + 2);  // floats of a slot: rows, then (reference, sum) per column
  __shared__ float s_ref[kAttWarps][COLS], s_sum[kAttWarps][COLS];
  const int tid = kSolo ? lane : threadIdx.x, mine = kSolo ? warp : 0;
  auto sync = [&] {
    if constexpr (kSolo) __syncwarp();
    else __syncthreads();
  };
  int share0 = 0;
  // The slot of a pair's piece. (kSolo) A warp has one pair at most that began in an earlier share, and
  // one at most that begins in its own and goes on in the next: two slots.
  auto slot_of = [&](int i) -> int64_t {
    if constexpr (kSolo) return 2 * (share0 + i) + (i == 0);
    else return pc.slot0 + i;
  };
  // a column's sum over the tokens of the eight quads
  auto column_sum = [&](int n, int c) {
    float v = sum[n][c];
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    return v;
  };
  auto write = [&](int r, int e, const float (&y)[4], float l) {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(y[0] * inv, y[1] * inv);
    const __nv_bfloat162 b1 = __floats2bfloat162_rn(y[2] * inv, y[3] * inv);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&b0);
    w.y = *reinterpret_cast<const uint32_t*>(&b1);
    __nv_bfloat16* row = a.out + static_cast<int64_t>(sv.q0 + r / G) * a.out_stride + (h * G + r % G) * kD;
    *reinterpret_cast<uint2*>(row + e) = w;
  };
  // ---- pieces meet in groups, then the groups
  __shared__ int s_last[kAttWarps];
  // true in the last of n blocks to arrive at a counter, with what the others wrote visible
  auto arrive_last = [&](uint32_t* counter, int n) {
    sync();
    if (tid == 0) {  // wraps to zero at the last arrival: ready for the next call
      uint32_t old;
      asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(n - 1) : "memory");
      s_last[mine] = old == static_cast<uint32_t>(n - 1);
    }
    sync();
    return s_last[mine] != 0;
  };
  // joins the slots of n pieces, `step` apart from piece `from` on, into the first of them, or into the
  // output: each thread its elements, eight slots in flight
  auto join = [&](int from, int n, int step, bool final) {
    float* base = a.part + slot_of(from) * PART;
#pragma unroll 1
    for (int i = tid; i < rows * kD / 4; i += TEAM) {
      const int col = i / (kD / 4), e = i % (kD / 4) * 4;
      const int src = col * kD + e, stat = COLS * kD + 2 * col;
      float top = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int k0 = 0; k0 < n; k0 += 8) {
        float4 v[8];
        float2 ml[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool in = k0 + k < n;
          const float* at = a.part + slot_of(from + (k0 + k) * step) * PART;
          ml[k] = in ? __ldcg(reinterpret_cast<const float2*>(at + stat)) : make_float2(-INFINITY, 0.f);
          v[k] = in ? __ldcg(reinterpret_cast<const float4*>(at + src)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float now = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) now = fmaxf(now, ml[k].x);
        const float ref = now == -INFINITY ? 0.f : now;
        const float f = now == -INFINITY ? 1.f : exp2_approx(top - ref);
        l = sum_times_exp2(l, now == -INFINITY ? 0.f : top - ref);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] *= f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // (a slot that has seen nothing holds zeros; one that has seen nothing but nan, nan)
          const float w = exp2_approx(ml[k].x - ref);
          l += sum_times_exp2(ml[k].y, ml[k].x - ref);
          y[0] = fmaf(v[k].x, w, y[0]); y[1] = fmaf(v[k].y, w, y[1]);
          y[2] = fmaf(v[k].z, w, y[2]); y[3] = fmaf(v[k].w, w, y[3]);
        }
        top = now;
      }
      if (final) {
        write(col, e, y, l);
      } else {  // (this thread alone reads these elements of the slot; its statistics are read by others)
        *reinterpret_cast<float4*>(base + col * kD + e) = make_float4(y[0], y[1], y[2], y[3]);
        if (e == 0) {
          s_ref[mine][col] = top;
          s_sum[mine][col] = l;
        }
      }
    }
    if (!final) {
      sync();  // all have read the statistics
      if (tid < rows)
        *reinterpret_cast<float2*>(base + COLS * kD + 2 * tid) = make_float2(s_ref[mine][tid], s_sum[mine][tid]);
    }
  };
  // What a team does after it has left a piece in its slot. With first tokens up to 16 pieces meet at once, without up to 8: their
  // number is the order of a result's sums, and calls without first tokens keep theirs. (us, 16 / 8 at once, 32 and 8 heads, 4
  // first tokens: window 1024 of one sequence 8.5 / 9.4, of four 10.0 / 11.0, window 4096 of four 13.2 / 13.9: up to 16 pieces
  // are spared a second join. Of more it is the longer one: one sequence, window 2048 10.2 / 9.7, 4096 10.7 / 10.2, 16384
  // 13.7 / 13.2.)
  auto meet = [&](int index, int of) {
    int gs = min(kSink ? 16 : 8, of);
    while (gs * gs < of) ++gs;
    const int groups = (of + gs - 1) / gs, gi = index / gs, g0 = gi * gs, gn = min(gs, of - g0);
    if (!arrive_last(a.counters + slot_of(g0), gn)) return;
    if (groups == 1) {
      join(0, of, 1, true);
      return;
    }
    join(g0, gn, 1, false);
    // (the second counter of piece 0's slot counts the groups)
    if (arrive_last(a.counters + kAttMaxSlots + slot_of(0), groups)) join(0, groups, gs, true);
  };

  if constexpr (kSolo) {
    int i_slot = 0;
#pragma unroll 1
    for (int todo = share.todo; todo > 0;) {
      take(now.seq, now.head, now.v);
      const int m = min(todo, now.st.n - now.at);
      hi = sv.len;
      load_queries();
      reset();
      int j0 = now.st.at(now.at) * kAttStep;
#pragma unroll 1
      for (int i = 0; i < m; ++i, j0 = kSink ? now.st.at(now.at + i) * kAttStep : j0 + kAttStep) {
        cp_async_wait<kAttSlots - 1>();
        __syncwarp();
        step(j0, i_slot);
        __syncwarp();  // every lane has read the slot
        if (to_copy > 0) issue_ahead(i_slot);
        cp_async_commit();
        i_slot = i_slot + 1 == kAttSlots ? 0 : i_slot + 1;
      }
      // the pieces of this pair: in the shares from that of its first step to that of its last
      const int done = share.per * (blockIdx.x * kAttWarps + warp) + share.todo - todo - now.at;  // first step
      const bool whole = m == now.st.n;
      share0 = whole ? 0 : done / share.per;
      const int index = whole ? 0 : blockIdx.x * kAttWarps + warp - share0;
      const int of = whole ? 1 : (done + now.st.n - 1) / share.per - share0 + 1;
      float* part = a.part + slot_of(index) * PART;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = n * 8 + 2 * t + c;
          const float l = column_sum(n, c);
          const float f = whole ? (l == 0.f ? 0.f : 1.0f / l) : 1.f;
          if (col < rows) {
#pragma unroll
            for (int j = 0; j < NJ; j += 2) {
              const int e = g * (4 * VW) + 2 * j;
              const float y[4] = {o[n][j][c] * f, o[n][j][2 + c] * f, o[n][j + 1][c] * f, o[n][j + 1][2 + c] * f};
              if (whole) write(col, e, y, 1.f);
              else *reinterpret_cast<float4*>(part + col * kD + e) = make_float4(y[0], y[1], y[2], y[3]);
            }
            if (!whole && g == 0)
              *reinterpret_cast<float2*>(part + COLS * kD + 2 * col) =
                  make_float2(limit[n][c] == kLag ? ref[n][c] : -INFINITY, l);
          }
        }
      if (!whole) meet(index, of);
      todo -= m;
      if (todo > 0) now.move(a, m);
    }
    cp_async_wait<0>();
    return;
  } else {
    load_queries();
    reset();
    int i_slot = 0;
#pragma unroll 1
    for (int j0 = lo + warp * kAttStep; ours(j0); j0 += kAttWarps * kAttStep, j_next += kAttWarps * kAttStep) {
      cp_async_wait<kAttSlots - 1>();
      __syncwarp();
      step(token(j0), i_slot);
      __syncwarp();  // every lane has read the slot
      if (ours(j_next)) issue(s, h, seen_lo, hi, token(j_next), i_slot);
      cp_async_commit();
      i_slot = i_slot + 1 == kAttSlots ? 0 : i_slot + 1;
    }

    // ---- join the warps: every column to the largest reference, then the sums in the warps' order
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float v = column_sum(n, c);
        if (g == 0) {
          // (a column that has seen nothing but nan keeps its sum: nan)
          s_ref[warp][n * 8 + 2 * t + c] = limit[n][c] == kLag ? ref[n][c] : -INFINITY;
          s_sum[warp][n * 8 + 2 * t + c] = v;
        }
      }
    cp_async_wait<0>();
    __syncthreads();  // (and every warp is done with its slots)
    float* s_o = reinterpret_cast<float*>(att_smem);  // [kAttWarps][COLS][kD + 4]
    constexpr int OS = kD + 4;
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = n * 8 + 2 * t + c;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, s_ref[w][col]);
        const float f = top == -INFINITY ? 1.f : exp2_approx(s_ref[warp][col] - top);
        float* dst = s_o + (warp * COLS + col) * OS + g * (4 * VW);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[n][j][c] * f, o[n][j][2 + c] * f);
      }
    __syncthreads();
    // four elements of one column per thread
    float* part = a.part + slot_of(pc.index) * PART;
    for (int i = threadIdx.x; i < rows * kD / 4; i += kAttWarps * 32) {
      const int col = i / (kD / 4), e = i % (kD / 4) * 4;
      float top = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, s_ref[w][col]);
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        l += sum_times_exp2(s_sum[w][col], top == -INFINITY ? 0.f : s_ref[w][col] - top);
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * COLS + col) * OS + e);
        y[0] += v.x; y[1] += v.y; y[2] += v.z; y[3] += v.w;
      }
      if (pc.of == 1) {
        write(col, e, y, l);
      } else {
        *reinterpret_cast<float4*>(part + col * kD + e) = make_float4(y[0], y[1], y[2], y[3]);
        if (e == 0) *reinterpret_cast<float2*>(part + COLS * kD + 2 * col) = make_float2(top, l);
      }
    }
    if (pc.of > 1) meet(pc.index, pc.of);
  }
}

// Rows of a sequence and K/V head up to which its cache is streamed through this kernel; more go to
// attention_tc.cu. (us, streamed / there, 16 rows: one sequence of 32768 26 / 44, 16 of 4096 29 / 61,
// 64 of 2000 61 / 85; 12 rows, 4 of 8192 31 / 55. A third tile of 8 rows would not fit the registers.)
constexpr int kAttStreamRows = 16;
// (sequence, K/V head) pairs above which each warp goes its own way: the figures are at the top.
constexpr int kAttSoloPairs = kAttResident / 2;

AttnPlan attn_plan(const strata_kv_cache& c, const strata_kv_batch& b, int n_heads) {
  AttnPlan p{};
  const int64_t G = n_heads / c.n_kv_heads, most_rows = b.max_q * G;
  if (most_rows > kAttStreamRows) {
    p.tc = true;
    p.tc_slots = attn_tc_slots(c, b, G, 0, 0);
    p.tc_part_floats = attn_tc_part_floats(c, p.tc_slots);
    // sequences of equal length: none is below the limit
    if (b.T == static_cast<int64_t>(b.n_seq) * b.max_q) return p;
    p.stream_rows = kAttStreamRows;
  } else {
    p.stream_rows = 0x7FFFFFFF;
  }
  p.nt = std::min<int64_t>(most_rows, kAttStreamRows) <= 8 ? 1 : 2;
  const int64_t heads = static_cast<int64_t>(c.n_kv_heads) * b.n_seq;
  p.solo = heads > kAttSoloPairs;
  int64_t slots;
  static_assert(2 * kAttResident * kAttWarps <= kAttMaxSlots, "every slot has counters");
  if (p.solo) {
    p.grid = kAttResident;
    slots = 2 * kAttResident * kAttWarps;
  } else {
    p.grid = slots = kAttResident;
    const int64_t most_pieces = (b.max_kv + kAttStep * kAttMinSteps - 1) / (kAttStep * kAttMinSteps) + 1;
    if (most_pieces * heads < p.grid) p.grid = most_pieces * heads;
  }
  p.part_floats = static_cast<size_t>(slots) * (8 * p.nt) * (c.head_dim + 2);
  return p;
}

template <int kD, int kNT, bool kSolo, bool kSink>
static cudaError_t launch_attention_t(const AttnArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr size_t slots = static_cast<size_t>(kAttWarps) * kAttSlots * 2 * kAttStep * kD;
  constexpr size_t join = kSolo ? 0 : sizeof(float) * kAttWarps * 8 * kNT * (kD + 4);
  constexpr size_t smem = slots > join ? slots : join;
  const cudaError_t e = cudaFuncSetAttribute(attention_kernel<kD, kNT, kSolo, kSink>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attention_kernel<kD, kNT, kSolo, kSink>, dim3(static_cast<unsigned>(grid)), dim3(kAttWarps * 32),
                       smem, stream, true, a);
}

template <int kD, int kNT>
static cudaError_t launch_attention_t(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream) {
  if (a.sinks > 0)
    return p.solo ? launch_attention_t<kD, kNT, true, true>(a, p.grid, stream)
                  : launch_attention_t<kD, kNT, false, true>(a, p.grid, stream);
  return p.solo ? launch_attention_t<kD, kNT, true, false>(a, p.grid, stream)
                : launch_attention_t<kD, kNT, false, false>(a, p.grid, stream);
}

cudaError_t launch_attention(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream) {
  if (a.c.head_dim == 64)
    return p.nt == 1 ? launch_attention_t<64, 1>(a, p, stream) : launch_attention_t<64, 2>(a, p, stream);
  return p.nt == 1 ? launch_attention_t<128, 1>(a, p, stream) : launch_attention_t<128, 2>(a, p, stream);
}

}  // namespace strata
