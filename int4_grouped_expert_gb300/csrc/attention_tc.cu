// Causal attention over the paged cache of e4m3 codes for many query rows, on tcgen05 (the formula and
// the cache are those of attention.cu).
//
// A block owns up to 256 query rows of one sequence and K/V head (query rows x the heads that share it): two
// tiles of 128 rows, a TMEM lane each. It walks the cache in tiles of 64 tokens:
//   S_i = Q_i K^T (f16, fp32 sums in TMEM) -> softmax weights P_i (f16, in TMEM over S_i) -> O_i += P_i V
// Each row tile has two score buffers, so that its next scores are ready when a softmax ends, and the
// two row tiles are half a step apart. (With 128-token tiles and one score buffer the chain scores ->
// softmax -> product was the whole time: 5200 clocks per 128 tokens, of which the tensor cores
// needed 2048.)
//   warps 0, 1     an elected lane issues the MMAs of row tile 0, 1
//   warp 2         owns the TMEM allocation: the score buffers (4 x 64 columns), O_0, O_1 (head_dim each)
//   warp 3         looks up the pages' scales, many tiles ahead, and lays out a tile's with its stage
//   warps 4-11     softmax, one thread per row: running reference and sum in fp32. O is rescaled only when
//                  a score has grown by more than 2^8 over the reference (weights up to 2^8 are as exact
//                  in f16 and the sums fp32), which after the first tiles is rare
//   warps 12-19    codes -> f16 tiles in shared memory, K as it lies and V transposed (bytes of two
//                  tokens paired with PRMT), a ring of 4 stages: (K0, K1), (V0, K2), (V1, K3), ...
// Codes are f16 as they are, exactly; the scales of a tile's page, or of its pages of 16 or 32 tokens, go to the
// softmax (attention.cuh). That costs it a dozen instructions a row and tile, about 5% where it is the bound, against
// scaling the codes to the largest page of the block; that one left small pages few bits.
// Queries become f16 with a power of two per row; a token that no row sees or in a page that does not
// exist becomes zeros and a masked score, so what lies there does not matter.
//
// Measured: 2048 queries on 8192 tokens, 32 query and 8 K/V heads of 128: 252 us back to back, 954 TFLOP/s (254 as
// a public call); 8192 more tokens take 268 us, 1.05 us a tile over both rounds of blocks. Softmax and conversion
// instructions (issue 60% of active cycles), shared memory (66%) and the tensor pipe (46%) wait for one another over
// the score buffers; none is full.
// Every mbarrier wait is bounded in time; on time-out the kernel sets STRATA_DEV_TIMEOUT, every
// role leaves its loop, MMAs in flight are drained (bounded) and TMEM is freed.
#include <algorithm>

#include "attention.cuh"
#include "tc_ts_ptx.cuh"

namespace strata {

namespace {

constexpr int kAtTok = 64;      // tokens per tile
constexpr int kAtRing = 4;      // stages of two tiles of codes converted to f16
constexpr int kAtThreads = 640;
constexpr int kAtScales = 8;    // tiles whose scales are in shared memory
constexpr int kAtSms = 152;     // blocks that run at once
constexpr int kAtMaxSlots = 3 * kAtSms;
constexpr int kAtMinTiles = 4;  // tiles that a piece has at least
// What a block costs beside its tiles, in tiles of 1.17 us: to start and to fill its ring; the same and to
// leave a piece; for the kernel that joins (and half a tile a piece). Where a quarter of the SMs idle after
// full rounds, a tile takes a sixth less. (32 query heads, 8 K/V heads, us whole and cut: 64 queries on 4096
// tokens, 8 units, 77 and 28; 64 on 32768 582 and 60; 512 on 8192, 64 units, 141 and 97; 1280 on 8192, of whose
// 160 units 8 are cut, 244 and 170. Cutting 104 of 256 units took 276 for 245. Pieces of 4 tiles at
// least or of 8: 64 queries on 1600 tokens 23 / 28.)
constexpr int kAtStart = 4, kAtPiece = 8, kAtJoin = 6;
constexpr int kAtMostCut = kAtSms * 3 / 4;  // (more units than these are never worth cutting)

template <int kD>
struct AtCfg {
  static constexpr int QTILE = 128 * kD * 2;   // bytes of a row tile of Q in f16
  static constexpr int TILE = kAtTok * kD * 2; // of a tile of K or V
  static constexpr size_t SMEM = 2 * QTILE + static_cast<size_t>(kAtRing) * 2 * TILE + 1024 + 512;
};

// Two fp32 values as one operand of the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The units of a call: tc_rows rows of a (sequence, K/V head), sequence by sequence, those with the most tokens
// to see first. As many as fill all SMs a whole number of times stay whole; the others, which run last, are
// cut along the tokens where that ends sooner, into pieces of `per` tiles, at most k. The same in every warp, and in
// the kernel that joins: each product and sum is rounded where it is written, whatever the compiler fuses elsewhere.
struct Units {
  int whole, rest, k, per;
  int s0, s1, mine, end;  // this lane's sequences, their units, and the units up to there
};
__device__ __forceinline__ int units_of(const AttnArgs& a, const SeqView& v) {
  const int64_t rows = static_cast<int64_t>(v.n) * a.group;
  return rows > a.rows_below ? static_cast<int>((rows + a.tc_rows - 1) / a.tc_rows) * a.c.n_kv_heads : 0;
}
__device__ __forceinline__ Units find_units(const AttnArgs& a, bool flag) {
  Units u;
  const int lane = threadIdx.x & 31, per_lane = (a.b.n_seq + 31) / 32;
  u.s0 = min(a.b.n_seq, lane * per_lane), u.s1 = min(a.b.n_seq, u.s0 + per_lane);
  u.mine = 0;
  float tiles = 0.f, most = 0.f;
  for (int s = u.s0; s < u.s1; ++s) {
    const SeqView v = seq_view(a, s, flag);
    const int n = units_of(a, v);
    // tokens that a unit sees, on average
    float seen = fmaxf(0.f, __fsub_rn(static_cast<float>(v.len), __fmul_rn(0.5f, static_cast<float>(v.n))));
    if (a.window > 0)
      seen = fminf(seen, __fadd_rn(static_cast<float>(a.window), __fdiv_rn(static_cast<float>(a.tc_rows),
                                                                           static_cast<float>(a.group))));
    const float of_unit = __fadd_rn(__fmul_rn(seen, 1.f / kAtTok), 1.f);
    u.mine += n;
    tiles = __fadd_rn(tiles, __fmul_rn(static_cast<float>(n), of_unit));
    if (n > 0) most = fmaxf(most, of_unit);
  }
  u.end = u.mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, u.end, d);
    if (lane >= d) u.end += x;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) tiles = __fadd_rn(tiles, __shfl_xor_sync(0xffffffffu, tiles, d));
  const int all = __shfl_sync(0xffffffffu, u.end, 31);
  u.whole = all / kAtSms * kAtSms, u.rest = all - u.whole;
  u.k = 1;
  most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
  // (units that stay whole decide when a batch of very different lengths ends)
  if (u.rest > 0 &&
      (u.whole == 0 || __fmul_rn(most, static_cast<float>(all)) <= __fmul_rn(1.25f, tiles))) {
    // lane i weighs i + 1 pieces of the longest units, and in proportion of the others
    const int n = static_cast<int>(most), c = lane + 1;
    const float share = __fdiv_rn(__fdiv_rn(tiles, static_cast<float>(all)), most);
    const int pieces = max(u.rest, static_cast<int>(__fmul_rn(static_cast<float>(u.rest * c), share)));
    const int rounds = (pieces + kAtSms - 1) / kAtSms;
    int cost = c == 1 ? rounds * (n + 1 + kAtStart) : rounds * (n / c + 1 + kAtPiece) + kAtJoin + c / 2;
    if (c == 1 && u.whole > 0 && u.rest <= kAtMostCut) cost -= cost / 6;
    if (c > 1 && (n < c * kAtMinTiles || u.rest * c > a.tc_slots)) cost = 0x3FFFFFF;
    cost = min(cost, 0x3FFFFFF);
    u.k = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(cost) << 5 | lane) % 32 + 1;
  }
  u.per = max(kAtMinTiles, static_cast<int>(most) / u.k + 1);
  return u;
}
// One unit, and the tiles that its rows see.
struct Unit {
  int seq, head, row0, rows;  // first row; rows of the (sequence, head)
  SeqView sv;
  int tok_lo, tok_hi, j_lo, n_tiles, of;  // tokens tok_lo .. tok_hi - 1
};
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int seq, int head, int row0, int k, int per, bool flag) {
  Unit u;
  u.seq = seq, u.head = head, u.row0 = row0;
  u.sv = seq_view(a, seq, flag);
  u.rows = u.sv.n * a.group;
  const int p0 = u.sv.len - u.sv.n;  // position of the first query
  u.tok_hi = min(u.sv.len, p0 + (min(row0 + a.tc_rows, u.rows) - 1) / a.group + 1);
  u.tok_lo = first_seen(a, p0 + row0 / a.group);
  u.j_lo = u.tok_lo / kAtTok;
  u.n_tiles = u.tok_hi > u.tok_lo ? (u.tok_hi + kAtTok - 1) / kAtTok - u.j_lo : 0;
  u.of = min(k, max(1, (u.n_tiles + per - 1) / per));
  return u;
}
__device__ __forceinline__ Unit find_unit(const AttnArgs& a, const Units& us, int at) {
  const int heads = a.c.n_kv_heads;
  const int owner = __ffs(__ballot_sync(0xffffffffu, at < us.end)) - 1;
  int seq = 0, left = at - (us.end - us.mine), n = 0;
  if ((threadIdx.x & 31) == owner) {
    for (seq = us.s0; seq < us.s1; ++seq) {
      n = units_of(a, seq_view(a, seq, false));
      if (left < n) break;
      left -= n;
    }
  }
  seq = __shfl_sync(0xffffffffu, seq, owner);
  left = __shfl_sync(0xffffffffu, left, owner);
  n = __shfl_sync(0xffffffffu, n, owner);
  return unit_of(a, seq, left % heads, (n / heads - 1 - left / heads) * a.tc_rows, at < us.whole ? 1 : us.k, us.per,
                 false);
}

// The largest of 16 scores.
__device__ __forceinline__ float max16(const uint32_t* x) {
  float t = __uint_as_float(x[0]);
#pragma unroll
  for (int i = 1; i < 15; i += 2) t = max3(t, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
  return fmaxf(t, __uint_as_float(x[15]));
}

// kGroups: pairs of scales in a tile, 1 where it lies in one page (of 64 or 128 tokens), else one for every 16 tokens.
// (us, 1 / 4 of them, pages of 64: 2048 queries on 8192 tokens 252 / 268, 8 on 131072 141 / 144, 4096 on 4096 154 / 163.)
template <int kD, int kGroups>
__global__ void __launch_bounds__(kAtThreads, 1) attention_tc_kernel(AttnArgs a) {
  using C = AtCfg<kD>;
  constexpr int KC = kD / 64;   // 64-wide pieces of a head
  extern __shared__ uint8_t at_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(at_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + 2 * C::QTILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kAtRing * 2 * C::TILE);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + kAtRing;
  uint64_t* s_full = kv_empty + kAtRing;  // [row tile][buffer]
  uint64_t* p_full = s_full + 4;          // [row tile][buffer]
  uint64_t* pv_done = p_full + 4;         // [row tile][buffer]
  uint64_t* drain = pv_done + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  __shared__ int abort_flag_s;
  // of each group: K scale, log2 of the V scale, the inverse V scale (0 for a small one), and whether all is well (0), the
  // page does not exist (1), has a scale of inf or nan (2: nan for the rows that see it) or a small V scale (3:
  // kFarScale below the largest up to there)
  __shared__ float4 s_scale[kAtScales][kGroups];
  __shared__ volatile int s_any_small;  // a tile so far has a page of a small V scale
  __shared__ volatile int s_end[6];  // what is wanted again at the end only: not kept in registers
  volatile int* abort_flag = &abort_flag_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_wait();
  griddep_launch();
  const int id = blockIdx.x;
  int cut = 0, piece = 0;  // slot of the block's piece, its number among its unit's
  Unit u;
  if (a.tc_search) {
    const Units us = find_units(a, id == 0 && threadIdx.x < 32);
    cut = max(0, id - us.whole);
    const int at = cut > 0 ? us.whole + cut / us.k : id;
    if (at >= us.whole + us.rest) return;
    u = find_unit(a, us, at);
    piece = cut - max(0, at - us.whole) * us.k;
  } else {  // the same order, as if every sequence had max_q rows
    const int heads = a.c.n_kv_heads, of_seq = gridDim.x / a.b.n_seq, left = id % of_seq;
    u = unit_of(a, id / of_seq, left % heads, (of_seq / heads - 1 - left / heads) * a.tc_rows, 1, 1,
                left == 0 && threadIdx.x == 0);
    if (u.rows <= a.rows_below || u.row0 >= u.rows) return;
  }
  const int h = u.head, s = u.seq, row0 = u.row0, rows = u.rows, of = u.of;
  const SeqView sv = u.sv;
  const int G = a.group;
  const int tok_lo = u.tok_lo;  // before it, and from tok_hi on, nothing is looked up or used
  int j_lo = u.j_lo, n_tiles = u.n_tiles, tok_hi = u.tok_hi;
  if (piece >= of) return;
  if (of > 1) {
    const int from = n_tiles * piece / of, to = n_tiles * (piece + 1) / of;
    j_lo += from;
    n_tiles = to - from;
    tok_hi = min(tok_hi, (j_lo + n_tiles) * kAtTok);
  }
  const int row_end = min(row0 + a.tc_rows, rows);        // the rows from here on are another block's
  const int n_rt = row_end - row0 > 128 ? 2 : 1;          // row tiles in use
  const int P = a.c.page_size;
  const int32_t* table = a.b.page_table + static_cast<int64_t>(s) * a.b.table_stride;
  const bool softmax_warp = warp >= 4 && warp < 12;
  const int tile = (warp - 4) >> 2;                       // softmax warps: row tile
  const int row = row0 + tile * 128 + (warp & 3) * 32 + lane;

  if (n_tiles == 0) {  // nothing to see for any row: zeros
    if (softmax_warp && row < row_end) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(sv.q0 + row / G) * a.out_stride +
                                            (h * G + row % G) * kD);
      for (int i = 0; i < kD / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kAtRing; ++i) {
      tc::mbar_init(kv_full + i, 9);        // the conversion warps and the one of the scales
      tc::mbar_init(kv_empty + i, n_rt);  // each row tile's MMAs
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + 2 * i, 1);
      tc::mbar_init(s_full + 2 * i + 1, 1);
      tc::mbar_init(p_full + 2 * i, 4);
      tc::mbar_init(p_full + 2 * i + 1, 4);
      tc::mbar_init(pv_done + 2 * i, 1);
      tc::mbar_init(pv_done + 2 * i + 1, 1);
      tc::mbar_init(drain + i, 1);
    }
    tc::fence_barrier_init();
    abort_flag_s = 0;
    s_any_small = 0;
    s_end[0] = of > 1;
    s_end[1] = cut;  // (a unit's pieces have k slots, from its first block's number on)
    s_end[2] = sv.q0;
    s_end[3] = rows;
    s_end[4] = row0;
    s_end[5] = h;
  }
  if (warp == 2) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  float cmul = 0.f;  // softmax threads: what turns a product into the exponent of 2 (but for the K scale)
  if (softmax_warp) {
    // this thread's query row as f16 times 2^-e, in the swizzled layout of the A operand
    uint4 v[kD / 8];
    uint32_t mag = 0;
    const __nv_bfloat16* q = a.q + static_cast<int64_t>(sv.q0 + row / G) * a.q_stride + (h * G + row % G) * kD;
#pragma unroll
    for (int i = 0; i < kD / 8; ++i) {
      v[i] = row < row_end ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0u, 0u, 0u, 0u);
      mag = max(mag, bf16x8_mag(v[i]));
    }
    const int e = row_exp(mag);
    // a negative softmax scale goes into the queries, so that the largest product has the largest weight
    const float f = a.scale_log2 < 0.f ? -exp2i(-e) : exp2i(-e);
    cmul = fabsf(a.scale_log2) * exp2i(e);
    uint8_t* dst = smem + tile * C::QTILE + (row & 127) * 128;
#pragma unroll
    for (int i = 0; i < kD / 8; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack_f16x2(bf16_lo_f32(w[j]) * f, bf16_hi_f32(w[j]) * f);
      *reinterpret_cast<uint4*>(dst + (i >> 3) * (128 * 128) + (((i & 7) ^ (row & 7)) << 4)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    tc::fence_proxy_async_smem();
  }
  // the scales of a tile's groups: a lane a group, of kBatch tiles
  constexpr int kBatch = 32 / kGroups, kWide = kAtTok / kGroups;
  auto scales_of = [&](int batch) {
    const int t = batch * kBatch + lane / kGroups, tok = (j_lo + t) * kAtTok + lane % kGroups * kWide;
    float3 x = make_float3(0.f, 1.f, 0.f);
    if (t < n_tiles && tok < tok_hi && tok + kWide > tok_lo) {
      const int64_t page = table[tok >> (31 - __clz(P))];
      if (page >= 0 && page < a.c.n_pages) {
        x.x = a.c.k_scales[page * a.c.n_kv_heads + h];
        x.y = a.c.v_scales[page * a.c.n_kv_heads + h];
      } else {
        set_status(a.status, STRATA_DEV_BAD_SLOT);
        x.z = 1.f;
      }
    }
    return x;
  };
  float3 scales_now = {}, scales_next = {};
  if (warp == 3) scales_now = scales_of(0), scales_next = scales_of(1);
  // (the conversion warps start their first copies before they come to this barrier)
  uint32_t tmem = 0;
  if (warp < 12) {
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    tmem = *tmem_slot;
  }

  // registers: 5 warpgroups are launched with 96 a thread (61440 in all) and go on with
  // 48 + 2 * 120 + 2 * 96 (the same)
  // stage 0 holds K_0 and K_1, stage j + 1 V_j and K_(j+2): what the product of step j and the scores after
  // it read
  // O_i += P_i(j) V_j is done. Barriers of step j are per buffer (j & 1): whoever waits for one knows that
  // the step before it on the same buffer is over, and that no later one has begun.
  auto done = [&](int i, int j) {
    return tc::warp_wait(pv_done + 2 * i + (j & 1), (j >> 1) & 1, abort_flag, a.status);
  };
  if (warp < 4) {
    tc::reg_dec<48>();
    if (warp < n_rt) {
      // ---------------------------------------------------------------- MMA issuer of row tile i
      const int i = warp;
      const uint32_t id_s = tc::idesc_f16(128, kAtTok), id_o = tc::idesc_f16(128, kD);
      const uint32_t ts = tmem + i * 128, to = tmem + 256 + i * 128;
      const uint64_t q = tc::sw128_desc(tc::smem_u32(smem + i * C::QTILE));
      auto stage_at = [&](int t) { return tc::sw128_desc(tc::smem_u32(ring + (t % kAtRing) * 2 * C::TILE)); };
      auto full = [&](int t) {
        return tc::warp_wait(kv_full + t % kAtRing, (t / kAtRing) & 1, abort_flag, a.status);
      };
      // S(j) = Q K_j^T into buffer j & 1 (one lane)
      auto scores = [&](int j, uint64_t k) {
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)  // (64-wide pieces of Q are 16 KB apart, of K 8 KB, steps 32 bytes)
          tc::mma_f16_ss(ts + (j & 1) * 64, q + (kk >> 2) * 1024 + 2 * (kk & 3),
                         k + (kk >> 2) * (kAtTok * 8) + 2 * (kk & 3), id_s, kk ? 1u : 0u);
        tc::mma_commit(s_full + 2 * i + (j & 1));
      };
      constexpr uint64_t kSecond = C::TILE >> 4;  // descriptor distance of a stage's second tile
      bool ok = full(0);
      if (ok) {
        tc::tc_fence_after();
        const uint64_t k = stage_at(0);
        if (tc::elect_one()) {
          scores(0, k);
          if (n_tiles > 1) scores(1, k + kSecond);
          tc::mma_commit(kv_empty);
        }
        __syncwarp();
      }
      for (int j = 0; ok && j < n_tiles; ++j) {
        // O += P(j) V_j
        ok = full(j + 1) && tc::warp_wait(p_full + 2 * i + (j & 1), (j >> 1) & 1, abort_flag, a.status);
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t v = stage_at(j + 1);
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kAtTok / 16; ++kk)
            tc::mma_f16_ts(to, ts + (j & 1) * 64 + 32 + 8 * kk, v + 2 * kk, id_o, (j | kk) ? 1u : 0u);
          tc::mma_commit(pv_done + 2 * i + (j & 1));
        }
        __syncwarp();
        if (j + 2 >= n_tiles) continue;  // (the last stages are not filled again)
        // the next scores go where these weights are: once the product that reads them is done
        ok = done(i, j);
        if (!ok) break;
        tc::tc_fence_after();
        if (tc::elect_one()) {
          scores(j + 2, v + kSecond);
          tc::mma_commit(kv_empty + (j + 1) % kAtRing);
        }
        __syncwarp();
      }
      if (!ok) {  // drain every MMA issued so far before TMEM is released
        if (tc::elect_one()) tc::mma_commit(drain + i);
        __syncwarp();
        tc::mbar_wait_drain(drain + i, 0);
      }
    } else if (warp == 3) {
      // -------------------------------------------------------------- scales
      int batch = 0;
      float3 now = scales_now, next = scales_next;
      // (the largest up to the batch's end: what is called small a few tiles early is summed the other way, as well)
      float lv, top_lv = -INFINITY;
      bool fine;
      auto take = [&] {
        fine = now.x < INFINITY && now.y < INFINITY;
        lv = fine ? fminf(log2_scale(now.y), 126.f) : 0.f;
        float x = lv;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        top_lv = fmaxf(top_lv, x);
      };
      take();
      auto lay_out = [&](int t) {
        if (t >= n_tiles) return;
        if (t / kBatch > batch) {
          now = next;
          next = scales_of(++batch + 1);
          take();
        }
        const bool small = lv < top_lv - kFarScale;
        if (lane / kGroups == t % kBatch) {
          s_scale[t % kAtScales][lane % kGroups] =
              make_float4(fine ? now.x : 1.f, lv, small ? 0.f : exp2_approx(-lv),
                          now.z != 0.f ? now.z : !fine ? 2.f : small ? 3.f : 0.f);
          if (small) s_any_small = 1;
        }
      };
      for (int t = 0; t <= n_tiles; ++t) {  // stage t
        if (!tc::warp_wait(kv_empty + t % kAtRing, ((t / kAtRing) & 1) ^ 1, abort_flag, a.status)) break;
        if (t == 0) lay_out(0);
        lay_out(t + 1);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(kv_full + t % kAtRing);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    tc::reg_inc<120>();
    if (tile < n_rt) {
    // ------------------------------------------------------------------ softmax
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + 256 + tile * 128 + lanes;
    const int pos = sv.len - sv.n + row / G;
    float m = -INFINITY, l = 0.f;
    // The sum over pages of small scales has a reference of its own, the largest of their scores. (In local memory:
    // registers are short, and 2 KB more of shared memory would leave L1 28 KB instead of 60: 241 us became 314.)
    volatile float small_top = -INFINITY, small_sum = 0.f;
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const uint32_t ts = tmem + tile * 128 + (j & 1) * 64 + lanes;
      ok = tc::warp_wait(s_full + 2 * tile + (j & 1), (j >> 1) & 1, abort_flag, a.status);
      if (!ok) break;
      tc::tc_fence_after();
      const int j0 = (j_lo + j) * kAtTok;
      // columns lo .. hi of the tile are seen
      const int hi = min(pos, tok_hi - 1) - j0, lo = a.window > 0 ? pos - a.window + 1 - j0 : 0;
      const float4* scale = s_scale[j % kAtScales];
      // what turns a product into the exponent of 2 (never 0: a masked score, -inf, stays -inf under it)
      float cg[kGroups], lv[kGroups], per_scale;
      bool well = true;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float4 s = scale[g];
        cg[g] = fmaxf(cmul * s.x, 1.17549435e-38f);
        lv[g] = s.y;
        per_scale = s.z;  // (of several groups: looked up again, for want of registers)
        well = well && s.w == 0.f;
      }
      const bool whole = __all_sync(0xffffffffu, hi >= kAtTok - 1 && lo <= 0 && well);
      const bool odd = !whole && !__all_sync(0xffffffffu, well);
      if (odd) {
        float top = small_top, sum = small_sum;
#pragma unroll 1
        for (int c = 0; c < kAtTok; ++c) {  // (short code: it is rarely run)
          const float4 sc = scale[c * kGroups / kAtTok];
          const float score = __uint_as_float(tc::tmem_ld1(ts + c));
          const bool on = sc.w == 3.f && c <= hi && c >= lo;
          const float x = on ? score * fmaxf(cmul * sc.x, 1.17549435e-38f) : -INFINITY, before = top;
          top = fmaxf(top, x);
          const float ref = top == -INFINITY ? 0.f : top;
          sum = fmaf(sum, exp2_approx(before - ref), exp2_approx(x - ref));
          __syncwarp();
        }
        small_top = top, small_sum = sum;
      }
      uint32_t r[2][32];
      tc::tmem_ld32(ts, r[0]);
      tc::tmem_ld32(ts + 32, r[1]);
      tc::tmem_ld_wait();
      if (!whole) {
#pragma unroll
        for (int i = 0; i < kAtTok; ++i) {
          const bool seen = i <= hi && i >= lo;
          r[i / 32][i % 32] = seen ? r[i / 32][i % 32] : 0xFF800000u;  // -inf
        }
      }
      if (odd) {
#pragma unroll
        for (int i = 0; i < kAtTok; ++i) {
          const float state = scale[i * kGroups / kAtTok].w;
          if (state == 1.f) r[i / 32][i % 32] = 0xFF800000u;
          if (state == 2.f && i <= hi && i >= lo) r[i / 32][i % 32] = 0x7FC00000u;  // nan
        }
      }
      const float t[4] = {max16(r[0]), max16(r[0] + 16), max16(r[1]), max16(r[1] + 16)};
      const float top = kGroups == 1 ? fmaf(fmaxf(max3(t[0], t[1], t[2]), t[3]), cg[0], lv[0])
                                     : fmaxf(max3(fmaf(t[0], cg[0], lv[0]),
                                                  fmaf(t[1], cg[1 % kGroups], lv[1 % kGroups]),
                                                  fmaf(t[2], cg[2 % kGroups], lv[2 % kGroups])),
                                             fmaf(t[3], cg[3 % kGroups], lv[3 % kGroups]));
      if (__any_sync(0xffffffffu, top > m + 8.f)) {
        const float now = fmaxf(m, top);
        const float f = now == -INFINITY ? 1.f : exp2_approx(m - now);
        l = sum_times_exp2(l, now == -INFINITY ? 0.f : m - now);
        m = now;
        if (j > 0) {
          // the last product has to have added to O (the scores of this tile were issued before it)
          ok = done(tile, j - 1);
          if (!ok) break;
          tc::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kD; c += 16) {
            uint32_t x[16];
            tc::tmem_ld16(to + c, x);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
            tc::tmem_st16(to + c, x);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      uint64_t sum[4] = {0, 0, 0, 0};  // (pairs of zeros) of 16 columns each
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int g = (2 * q + i / 8) % kGroups;
          const uint64_t cc = pack_f32x2(cg[g], cg[g]), mm = pack_f32x2(lv[g] - ref, lv[g] - ref);
          const uint64_t x = pack_f32x2(__uint_as_float(r[q][2 * i]), __uint_as_float(r[q][2 * i + 1]));
          float2 e = unpack_f32x2(fma_f32x2(x, cc, mm));
          e.x = exp2_approx(e.x);
          e.y = exp2_approx(e.y);
          uint64_t& s = sum[kGroups == 1 ? i & 1 : 2 * q + i / 8];
          s = add_f32x2(s, pack_f32x2(e.x, e.y));
          p[i] = pack_f16x2(e.x, e.y);
        }
        tc::tmem_st16(ts + 32 + 16 * q, p);  // f16 pairs, over scores that this thread has read
      }
      if constexpr (kGroups == 1) sum[0] = add_f32x2(sum[0], sum[1]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float2 s = unpack_f32x2(sum[g]);
        l = fmaf(s.x + s.y, kGroups == 1 ? per_scale : scale[g].z, l);
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_full + 2 * tile + (j & 1));
    }
    if (ok) {
      ok = done(tile, n_tiles - 1);
      tc::tc_fence_after();
    }
    if (s_any_small) {  // (m is finite where top is)
      const float top = small_top, sum = small_sum;
      if (top != -INFINITY || sum != 0.f) l += sum_times_exp2(sum, top - (m == -INFINITY ? 0.f : m));
    }
    const int q0 = s_end[2], rows = s_end[3], h = s_end[5];
    const int row = s_end[4] + tile * 128 + (warp & 3) * 32 + lane;
    if (ok && s_end[0]) {
      // this piece: fp32 rows in the order [four elements][row], then (reference, sum)
      float* slot = a.tc_part + static_cast<int64_t>(s_end[1]) * (256 * (kD + 2));
      const int r0 = row - s_end[4];
#pragma unroll 1
      for (int c = 0; c < kD; c += 16) {
        uint32_t x[16];
        tc::tmem_ld16(to + c, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(slot + (c / 4 + i) * 1024 + r0 * 4) =
              make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]), __uint_as_float(x[4 * i + 2]),
                          __uint_as_float(x[4 * i + 3]));
      }
      *reinterpret_cast<float2*>(slot + 256 * kD + 2 * r0) = make_float2(m, l);
    } else if (ok) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(q0 + row / G) * a.out_stride +
                                            (h * G + row % G) * kD);
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(to + c, r);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * k]) * inv,
                                                           __uint_as_float(r[8 * i + 2 * k + 1]) * inv);
            o[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (row < rows) dst[c / 8 + i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    }
  } else {
    tc::reg_dec<96>();
    // ------------------------------------------------------------------ codes -> f16 tiles
    const int w = warp - 12;
    // K: this warp's 8 tokens of the tile (one page); a lane takes 16 bytes of row lane % 8 per 64-wide piece
    // V: a 32 x 32 piece (tokens x elements); a lane takes 4 elements of 8 tokens, chosen so that eight
    // lanes store to eight different 16-byte columns of the swizzled rows
    const bool v_on = w < 2 * kD / 32;               // (64-wide heads have 4 pieces)
    const int tg = lane & 3, dg = ((lane >> 2) & 1) | (lane >> 3) << 1;
    // codes of the tiles j (even) and j (odd), on their way two tiles ahead
    uint4 kr[2][KC];
    uint32_t vr[2][8];
    const int pshift = 31 - __clz(P);
    // whether a row sees any token of the group that tok is in, and their page (-1 if not); looked up one more
    // tile ahead
    constexpr int kLast = kAtTok / kGroups - 1;
    const int lo_g = tok_lo & ~kLast, n_g = ((tok_hi - 1) | kLast) + 1 - lo_g;
    auto seen = [&](int tok) { return static_cast<unsigned>(tok - lo_g) < static_cast<unsigned>(n_g); };
    auto page_of = [&](int tok) { return seen(tok) ? table[tok >> pshift] : -1; };
    auto in_span = [&](int tok) { return tok < tok_hi && tok >= tok_lo; };
    auto good = [&](int page) { return page >= 0 && page < a.c.n_pages; };
    const int k_tok = j_lo * kAtTok + w * 8, v_tok = j_lo * kAtTok + (w & 1) * 32 + tg * 8;
    int k_page = page_of(k_tok), v_page = page_of(v_tok);
    auto load_k = [&](int j, uint4 (&x)[KC]) {
      const int tok = k_tok + j * kAtTok;
      const bool on = good(k_page);
      const int64_t ph = on ? static_cast<int64_t>(k_page) * a.c.n_kv_heads + h : 0;
      const uint8_t* src = a.c.k_codes + ((ph << pshift) + (tok & (P - 1)) + (lane & 7)) * kD + (lane >> 3) * 16;
#pragma unroll
      for (int c = 0; c < KC; ++c)
        x[c] = on && in_span(tok + (lane & 7)) ? __ldcg(reinterpret_cast<const uint4*>(src + c * 64))
                                               : make_uint4(0u, 0u, 0u, 0u);
      k_page = page_of(tok + kAtTok);
    };
    auto load_v = [&](int j, uint32_t (&x)[8]) {
      const int tok = v_tok + j * kAtTok;
      const bool on = good(v_page) && v_on;
      const int64_t ph = on ? static_cast<int64_t>(v_page) * a.c.n_kv_heads + h : 0;
      const uint8_t* src = a.c.v_codes + ((ph << pshift) + (tok & (P - 1))) * kD + (w >> 1) * 32 + dg * 4;
#pragma unroll
      for (int t = 0; t < 8; ++t)
        x[t] = on && in_span(tok + t) ? __ldcg(reinterpret_cast<const uint32_t*>(src + t * kD)) : 0u;
      v_page = page_of(tok + kAtTok);
    };
    auto store_k = [&](uint8_t* dst, const uint4 (&x)[KC]) {
      uint8_t* rowp = dst + (w * 8 + (lane & 7)) * 128;
      const int ch = 2 * (lane >> 3);
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t y[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int b = 0; b < 2; ++b)
          *reinterpret_cast<uint4*>(rowp + c * (kAtTok * 128) + (((ch + b) ^ (lane & 7)) << 4)) =
              make_uint4(e4m3x2_f16x2(y[2 * b]), e4m3x2_f16x2(y[2 * b] >> 16), e4m3x2_f16x2(y[2 * b + 1]),
                         e4m3x2_f16x2(y[2 * b + 1] >> 16));
      }
    };
    auto store_v = [&](uint8_t* dst, const uint32_t (&x)[8]) {
      if (!v_on) return;
      const int ch = (w & 1) * 4 + tg;  // 8-token column
      uint32_t o[4][4];                 // [element][token pair]
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t y = prmt(x[2 * t], x[2 * t + 1], 0x5140), z = prmt(x[2 * t], x[2 * t + 1], 0x7362);
        o[0][t] = e4m3x2_f16x2(y);
        o[1][t] = e4m3x2_f16x2(y >> 16);
        o[2][t] = e4m3x2_f16x2(z);
        o[3][t] = e4m3x2_f16x2(z >> 16);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int d = (w >> 1) * 32 + dg * 4 + k;
        *reinterpret_cast<uint4*>(dst + d * 128 + ((ch ^ (d & 7)) << 4)) =
            make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
      }
    };
    bool ok = true;
    auto begin = [&](int t) {
      ok = tc::warp_wait(kv_empty + t % kAtRing, ((t / kAtRing) & 1) ^ 1, abort_flag, a.status);
      return ring + (t % kAtRing) * 2 * C::TILE;
    };
    auto end = [&](int t) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(kv_full + t % kAtRing);
    };
    // stage j + 1: V_j and K_(j+2); then the codes of V_(j+2) and K_(j+4) start
    auto put = [&](int j, uint32_t (&xv)[8], uint4 (&xk)[KC]) {
      if (j >= n_tiles || !ok) return;
      uint8_t* dst = begin(j + 1);
      if (!ok) return;
      store_v(dst, xv);
      if (j + 2 < n_tiles) store_k(dst + C::TILE, xk);
      end(j + 1);
      if (j + 2 < n_tiles) load_v(j + 2, xv);
      if (j + 4 < n_tiles) load_k(j + 4, xk);
    };
    load_k(0, kr[0]);
    load_k(1, kr[1]);
    load_v(0, vr[0]);
    load_v(1, vr[1]);
    __syncthreads();  // the barrier of the other warps above
    uint8_t* dst = begin(0);
    if (ok) {
      store_k(dst, kr[0]);
      store_k(dst + C::TILE, kr[1]);
      end(0);
      load_k(2, kr[0]);
      load_k(3, kr[1]);
    }
    for (int j = 0; ok && j < n_tiles; j += 2) {
      put(j, vr[0], kr[0]);
      put(j + 1, vr[1], kr[1]);
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the units that were cut: a block takes 16 rows of a unit at a time, so that all SMs read
// (one SM reads 65 GB/s from L2: the last piece's block took 16 us to join four).
constexpr int kAtJoinRows = 16;
template <int kD>
__global__ void __launch_bounds__(kAtJoinRows * kD / 8) attention_tc_join_kernel(AttnArgs a) {
  griddep_wait();
  griddep_launch();
  const Units us = find_units(a, false);
  if (us.k == 1) return;
  constexpr int SLICES = 256 / kAtJoinRows;
  const int r16 = threadIdx.x % kAtJoinRows, c = threadIdx.x / kAtJoinRows * 2;  // a thread: eight elements of a row
  for (int i = blockIdx.x; i < us.rest * SLICES; i += gridDim.x) {
    const Unit u = find_unit(a, us, us.whole + i / SLICES);
    const int r = i % SLICES * kAtJoinRows + r16, row = u.row0 + r;
    if (u.of == 1 || row >= u.rows) continue;
    constexpr int64_t PART = 256 * (kD + 2);
    const float* first = a.tc_part + static_cast<int64_t>(i / SLICES) * us.k * PART;
    float top = -INFINITY;
#pragma unroll 4
    for (int k = 0; k < u.of; ++k)
      top = fmaxf(top, __ldcg(reinterpret_cast<const float2*>(first + k * PART + 256 * kD) + r).x);
    const float ref = top == -INFINITY ? 0.f : top;
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < u.of; ++k) {
      const float* slot = first + k * PART;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot + 256 * kD) + r);
      const float4 v0 = __ldcg(reinterpret_cast<const float4*>(slot) + c * 256 + r);
      const float4 v1 = __ldcg(reinterpret_cast<const float4*>(slot) + (c + 1) * 256 + r);
      const float w = exp2_approx(ml.x - ref);
      sum += sum_times_exp2(ml.y, ml.x - ref);
      y[0] = fmaf(v0.x, w, y[0]); y[1] = fmaf(v0.y, w, y[1]); y[2] = fmaf(v0.z, w, y[2]); y[3] = fmaf(v0.w, w, y[3]);
      y[4] = fmaf(v1.x, w, y[4]); y[5] = fmaf(v1.y, w, y[5]); y[6] = fmaf(v1.z, w, y[6]); y[7] = fmaf(v1.w, w, y[7]);
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * k] * inv, y[2 * k + 1] * inv);
      o[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __nv_bfloat16* dst = a.out + static_cast<int64_t>(u.sv.q0 + row / a.group) * a.out_stride +
                         (u.head * a.group + row % a.group) * kD;
    reinterpret_cast<uint4*>(dst)[c / 2] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int kD>
cudaError_t launch_join_t(const AttnArgs& a, int64_t units, cudaStream_t stream) {
  const int64_t slices = units * (256 / kAtJoinRows);
  return launch_kernel(attention_tc_join_kernel<kD>, dim3(static_cast<unsigned>(std::min<int64_t>(slices, kAtSms * 4))),
                       dim3(kAtJoinRows * kD / 8), 0, stream, true, a);
}

template <int kD, int kGroups>
cudaError_t launch_tc_g(const AttnArgs& a, int64_t grid, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(attention_tc_kernel<kD, kGroups>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(AtCfg<kD>::SMEM));
  if (e != cudaSuccess) return e;
  return launch_kernel(attention_tc_kernel<kD, kGroups>, dim3(static_cast<unsigned>(grid)), dim3(kAtThreads),
                       AtCfg<kD>::SMEM, stream, true, a);
}
template <int kD>
cudaError_t launch_tc_t(const AttnArgs& a, int64_t grid, cudaStream_t stream) {
  return a.c.page_size >= kAtTok ? launch_tc_g<kD, 1>(a, grid, stream) : launch_tc_g<kD, 4>(a, grid, stream);
}

}  // namespace

// Units if every sequence had max_q rows, and a bound from the rows of all.
static int64_t full_units(const strata_kv_cache& c, const strata_kv_batch& b, int64_t group, int rows = 256) {
  return (b.max_q * group + rows - 1) / rows * b.n_seq * c.n_kv_heads;
}
static int64_t most_units(const strata_kv_cache& c, const strata_kv_batch& b, int64_t group, int rows = 256) {
  return std::min(full_units(c, b, group, rows), (b.T * group / rows + b.n_seq) * c.n_kv_heads);
}
// Pieces that may come to lie in the workspace; 0: no unit is cut. Above one and a half times the SMs the
// last units fill their gaps by themselves (512 units of 33 tiles: 165 us whole, 178 with 56 cut). Batches
// that are not cut do without the kernel that joins: 3 us.
int attn_tc_slots(const strata_kv_cache& c, const strata_kv_batch& b, int64_t group, int window) {
  const int64_t units = most_units(c, b, group);
  if (units > kAtSms * 3 / 2) return 0;
  // (of sequences of equal length the units are known)
  const bool equal = b.T == static_cast<int64_t>(b.n_seq) * b.max_q;
  const int64_t rest = units % kAtSms;
  if (equal && (rest == 0 || rest > kAtMostCut)) return 0;
  const int64_t seen = window > 0 ? std::min<int64_t>(b.max_kv, window + 256 / group) : b.max_kv;
  // What whole units take, of 128 rows where those start together, against pieces, in tiles as above; of unequal
  // sequences the longest are cut in two at least. (us, whole / cut, 1472 tokens: 64 queries 28.9 / 23.7,
  // 512 queries 29.3 / 40.0.)
  const int64_t n = seen / kAtTok + 1;
  const int64_t k = std::max<int64_t>(equal ? 1 : 2, std::min(n / kAtMinTiles, kAtSms / units));
  const int64_t whole = most_units(c, b, group, 128) <= kAtSms ? n * 3 / 4 + 8 : n + 1 + kAtStart;
  if (units <= kAtSms ? n / k + 1 + kAtPiece + kAtJoin + k / 2 >= whole : n < 24) return 0;
  const int64_t cut = std::min<int64_t>(seen / kAtTok / kAtMinTiles, 32);
  return static_cast<int>(std::min<int64_t>(kAtMaxSlots, std::min<int64_t>(units, kAtSms - 1) * cut));
}
size_t attn_tc_part_floats(const strata_kv_cache& c, int slots) {
  return static_cast<size_t>(slots) * 256 * (c.head_dim + 2);
}
cudaError_t launch_attention_tc_join(AttnArgs a, cudaStream_t stream) {
  a.tc_rows = 256;
  const int64_t units = most_units(a.c, a.b, a.group);
  return a.c.head_dim == 64 ? launch_join_t<64>(a, units, stream) : launch_join_t<128>(a, units, stream);
}
cudaError_t launch_attention_tc(AttnArgs a, cudaStream_t stream) {
  // Blocks find their units in the lengths where units are cut, or where blocks by max_q would mostly be
  // empty; the search is 1 us a block.
  // Units of one row tile where they still start together and are not cut: a tile takes them a sixth less.
  // (us, 256 / 128 rows, 8 K/V heads, 256 rows on 64 tokens 12.2 / 10.4, on 512 19.2 / 16.4, on 1024 27.4 / 23.3.)
  a.tc_rows = a.tc_slots == 0 && most_units(a.c, a.b, a.group, 128) <= kAtSms ? 128 : 256;
  const int64_t full = full_units(a.c, a.b, a.group, a.tc_rows), most = most_units(a.c, a.b, a.group, a.tc_rows);
  a.tc_search = a.tc_slots > 0 || full > 2 * most;
  const int64_t grid = a.tc_search ? most + a.tc_slots : full;
  return a.c.head_dim == 64 ? launch_tc_t<64>(a, grid, stream) : launch_tc_t<128>(a, grid, stream);
}

}  // namespace strata
