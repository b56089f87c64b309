// Causal attention over the paged cache of e4m3 codes for many query rows, on tcgen05 (the formula and
// the cache are those of attention.cu).
//
// A block owns 256 query rows of one sequence and K/V head (query rows x the heads that share it): two
// tiles of 128 rows, a TMEM lane each. It walks the cache in tiles of 128 tokens:
//   S_i = Q_i K^T (f16, fp32 sums in TMEM) -> softmax weights P_i (f16, in TMEM over S_i) -> O_i += P_i V
// with the two row tiles half a step apart, so that the tensor cores work on one while the softmax of
// the other runs.
//   warp 0         an elected lane issues the MMAs
//   warp 1         owns the TMEM allocation: S_0, S_1 (128 columns each), O_0, O_1 (head_dim each)
//   warps 4-11     softmax, one thread per row: running maximum and sum in fp32. O is rescaled only when
//                  a maximum has grown by more than 2^8 over the one in use (weights up to 2^8 are as
//                  exact in f16 and the sums fp32), which after the first tiles is rare
//   warps 12-19    codes -> f16 tiles in shared memory, K as it lies and V transposed (bytes of two
//                  tokens paired with PRMT), a ring of 4 tiles in the order K, V, K, V, ...
// A page's scale relative to the largest of the block's pages multiplies its codes on the way: exact for
// powers of two down to 2^-15, absolute error below 2^-25 of the largest scale beyond.
// Queries become f16 with a power of two per row; a token that no row sees or in a page that does not
// exist becomes zeros and a masked score, so what lies there does not matter.
//
// Bound by the MMAs (1024 clocks per row tile and 128 tokens at 128-wide heads) and the softmax's
// instructions, which overlap. Every mbarrier wait is bounded in time; on time-out the kernel sets
// STRATA_DEV_TIMEOUT, every role leaves its loop, MMAs in flight are drained (bounded) and TMEM is freed.
#include "attention.cuh"
#include "tc_ts_ptx.cuh"

namespace strata {

namespace {

constexpr int kAtTok = 128;     // tokens per tile
constexpr int kAtRing = 4;      // tiles of codes converted to f16
constexpr int kAtThreads = 640;
constexpr int kAtBad = 8;       // ring of per-tile masks of tokens in pages that do not exist

template <int kD>
struct AtCfg {
  static constexpr int TILE = 128 * kD * 2;  // bytes of a Q, K or V tile in f16
  static constexpr size_t SMEM = static_cast<size_t>(2 + kAtRing) * TILE + 1024 + 512;
};

__device__ __forceinline__ uint32_t scaled_codes(uint32_t two, __half2 s) {
  const uint32_t v = e4m3x2_f16x2(two);
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}

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

template <int kD>
__global__ void __launch_bounds__(kAtThreads, 1) attention_tc_kernel(AttnArgs a) {
  using C = AtCfg<kD>;
  constexpr int KC = kD / 64;   // 64-wide pieces of a head
  extern __shared__ uint8_t at_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(at_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + 2 * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kAtRing * C::TILE);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + kAtRing;
  uint64_t* s_full = kv_empty + kAtRing;  // [2]
  uint64_t* p_full = s_full + 2;          // [2]
  uint64_t* pv_done = p_full + 2;         // [2]
  uint64_t* drain = pv_done + 2;
  uint64_t* bad = drain + 1;              // [kAtBad], a byte per 16 tokens
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bad + kAtBad);
  __shared__ int abort_flag_s;
  __shared__ float s_ref[2][8];
  volatile int* abort_flag = &abort_flag_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_wait();
  griddep_launch();
  const int h = blockIdx.y, s = blockIdx.z;
  const SeqView sv = seq_view(a, s, threadIdx.x == 0 && blockIdx.x == 0 && h == 0);
  const int G = a.group, rows = sv.n * G;
  // the blocks with the most tokens to see start first
  const int rb = gridDim.x - 1 - blockIdx.x;
  const int row0 = rb * 256;
  if (rows <= a.rows_below || row0 >= rows) return;
  const int last_row = min(row0 + 256, rows) - 1;
  const int p_lo = sv.len - sv.n + row0 / G, p_hi = sv.len - sv.n + last_row / G;
  const int tok_hi = min(sv.len, p_hi + 1);
  const int tok_lo = a.window > 0 ? max(0, p_lo - a.window + 1) : 0;
  const int j_lo = tok_lo / kAtTok;
  const int n_tiles = tok_hi > tok_lo ? (tok_hi + kAtTok - 1) / kAtTok - j_lo : 0;
  const int n_rt = last_row - row0 >= 128 ? 2 : 1;        // row tiles in use
  const int P = a.c.page_size;
  const int32_t* table = a.b.page_table + static_cast<int64_t>(s) * a.b.table_stride;
  const bool softmax_warp = warp >= 4 && warp < 12;
  const int tile = (warp - 4) >> 2;                       // softmax warps: row tile
  const int row = row0 + tile * 128 + (warp & 3) * 32 + lane;

  if (n_tiles == 0) {  // nothing to see for any row: zeros
    if (softmax_warp && row < rows) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(sv.q0 + row / G) * a.out_stride +
                                            (h * G + row % G) * kD);
      for (int i = 0; i < kD / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kAtRing; ++i) {
      tc::mbar_init(kv_full + i, 8);
      tc::mbar_init(kv_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(pv_done + i, 1);
    }
    tc::mbar_init(drain, 1);
    tc::fence_barrier_init();
    abort_flag_s = 0;
  }
  if (warp == 1) {
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
      v[i] = row < rows ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0u, 0u, 0u, 0u);
      mag = max(mag, bf16x8_mag(v[i]));
    }
    const int e = row_exp(mag);
    // a negative softmax scale goes into the queries, so that the largest product has the largest weight
    const float f = a.scale_log2 < 0.f ? -exp2i(-e) : exp2i(-e);
    cmul = fabsf(a.scale_log2) * exp2i(e);
    uint8_t* dst = smem + tile * C::TILE + (row & 127) * 128;
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
  } else if (warp >= 12) {
    // the largest scales of the pages that are read
    float km = 0.f, vm = 0.f;
    const int first = j_lo * kAtTok / P, end = (tok_hi + P - 1) / P;
    for (int i = first + threadIdx.x - 12 * 32; i < end; i += 256) {
      const int64_t page = table[i];
      if (page < 0 || page >= a.c.n_pages) continue;
      km = fmaxf(km, a.c.k_scales[page * a.c.n_kv_heads + h]);
      vm = fmaxf(vm, a.c.v_scales[page * a.c.n_kv_heads + h]);
    }
    km = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(km)));
    vm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vm)));
    if (lane == 0) {
      s_ref[0][warp - 12] = km;
      s_ref[1][warp - 12] = vm;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float k_ref = 0.f, v_ref = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    k_ref = fmaxf(k_ref, s_ref[0][i]);
    v_ref = fmaxf(v_ref, s_ref[1][i]);
  }
  if (k_ref == 0.f) k_ref = 1.f;
  if (v_ref == 0.f) v_ref = 1.f;

  // registers: 5 warpgroups are launched with 96 a thread (61440 in all) and go on with
  // 48 + 2 * 136 + 2 * 80 (the same)
  if (warp < 4) {
    tc::reg_dec<48>();
    if (warp == 0) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t id_s = tc::idesc_f16(128, kAtTok), id_o = tc::idesc_f16(128, kD);
    auto tile_at = [&](int t) { return tc::smem_u32(ring + (t % kAtRing) * C::TILE); };
    auto full = [&](int t) {
      return tc::warp_wait(kv_full + t % kAtRing, (t / kAtRing) & 1, abort_flag, a.status);
    };
    auto scores = [&](int i, int j) {  // S_i = Q_i K_j^T
      const uint64_t q = tc::sw128_desc(tc::smem_u32(smem + i * C::TILE)), k = tc::sw128_desc(tile_at(2 * j));
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)  // (64-wide pieces are 16 KB apart, steps 32 bytes)
          tc::mma_f16_ss(tmem + i * 128, q + (kk >> 2) * 1024 + 2 * (kk & 3), k + (kk >> 2) * 1024 + 2 * (kk & 3),
                         id_s, kk ? 1u : 0u);
        tc::mma_commit(s_full + i);
        if (i == n_rt - 1) tc::mma_commit(kv_empty + (2 * j) % kAtRing);
      }
      __syncwarp();
    };
    bool ok = full(0);
    if (ok) {
      tc::tc_fence_after();
      for (int i = 0; i < n_rt; ++i) scores(i, 0);
    }
    for (int j = 0; ok && j < n_tiles; ++j) {
      for (int i = 0; i < n_rt; ++i) {
        ok = tc::warp_wait(p_full + i, j & 1, abort_flag, a.status) && (i > 0 || full(2 * j + 1));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t v = tc::sw128_desc(tile_at(2 * j + 1));
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kAtTok / 16; ++kk)  // (64-token halves are kD * 128 bytes apart)
            tc::mma_f16_ts(tmem + 256 + i * 128, tmem + i * 128 + 64 + 8 * kk, v + (kk >> 2) * (kD * 8) + 2 * (kk & 3), id_o,
                           (j | kk) ? 1u : 0u);
          tc::mma_commit(pv_done + i);
          if (i == n_rt - 1) tc::mma_commit(kv_empty + (2 * j + 1) % kAtRing);
        }
        __syncwarp();
        if (j + 1 < n_tiles) {
          // the next scores overwrite the weights: only once the product that reads them is done
          ok = (i > 0 || full(2 * j + 2)) && tc::warp_wait(pv_done + i, j & 1, abort_flag, a.status);
          if (!ok) break;
          tc::tc_fence_after();
          scores(i, j + 1);
        }
      }
    }
    if (!ok) {  // drain every MMA issued so far before TMEM is released
      if (tc::elect_one()) tc::mma_commit(drain);
      __syncwarp();
      tc::mbar_wait_drain(drain, 0);
    }
    }
    __syncwarp();
  } else if (warp < 12) {
    tc::reg_inc<136>();
    if (tile < n_rt) {
    // ------------------------------------------------------------------ softmax
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + tile * 128 + lanes, to = tmem + 256 + tile * 128 + lanes;
    const int pos = sv.len - sv.n + row / G;
    cmul = fmaxf(cmul * k_ref, 1.17549435e-38f);  // (never 0: a masked score, -inf, stays -inf under it)
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      ok = tc::warp_wait(s_full + tile, j & 1, abort_flag, a.status);
      if (!ok) break;
      tc::tc_fence_after();
      const int j0 = (j_lo + j) * kAtTok;
      // columns lo .. hi of the tile are seen
      const int hi = min(pos, sv.len - 1) - j0, lo = a.window > 0 ? pos - a.window + 1 - j0 : 0;
      const unsigned long long gone = bad[j % kAtBad];
      const bool whole = __all_sync(0xffffffffu, hi >= kAtTok - 1 && lo <= 0) && gone == 0;
      auto seen = [&](int c) { return c <= hi && c >= lo && !((gone >> (c / 16 * 8)) & 1); };
      // Scores are read 32 columns at a time, the next ones on their way, up for the maximum and down
      // again for the weights: the last columns are read once. The weights (16 columns of f16 pairs per
      // 32 scores) go to the upper half of the scores' columns, always over scores that have been read.
      uint32_t r[2][32];
      auto mask = [&](uint32_t (&x)[32], int q) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = seen(32 * q + i) ? x[i] : 0xFF800000u;  // -inf
      };
      float top = -INFINITY;
      tc::tmem_ld32(ts, r[0]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        tc::tmem_ld_wait();
        if (q < 3) tc::tmem_ld32(ts + 32 * (q + 1), r[(q + 1) & 1]);
        uint32_t (&x)[32] = r[q & 1];
        if (!whole) mask(x, q);
        float t0 = top, t1 = __uint_as_float(x[31]);
#pragma unroll
        for (int i = 0; i < 30; i += 4) {
          t0 = max3(t0, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          t1 = max3(t1, __uint_as_float(x[i + 2]), __uint_as_float(x[min(i + 3, 30)]));
        }
        top = fmaxf(t0, t1);
      }
      top *= cmul;
      if (__any_sync(0xffffffffu, top > m + 8.f)) {
        const float now = fmaxf(m, top);
        const float f = now == -INFINITY ? 1.f : exp2_approx(m - now);
        m = now;
        l *= f;
        if (j > 0) {  // (the product that adds to O is done: the scores of this tile came after it)
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
      const uint64_t cc = pack_f32x2(cmul, cmul), mm = pack_f32x2(-ref, -ref);
      uint64_t sum0 = 0, sum1 = 0;  // (two zeros)
#pragma unroll
      for (int q = 3; q >= 0; --q) {
        if (q < 3) tc::tmem_ld_wait();
        if (q > 0) tc::tmem_ld32(ts + 32 * (q - 1), r[(q - 1) & 1]);
        uint32_t (&x)[32] = r[q & 1];
        if (!whole && q < 3) mask(x, q);
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, mm));
          e.x = exp2_approx(e.x);
          e.y = exp2_approx(e.y);
          if (i & 1) sum1 = add_f32x2(sum1, pack_f32x2(e.x, e.y));
          else sum0 = add_f32x2(sum0, pack_f32x2(e.x, e.y));
          p[i] = pack_f16x2(e.x, e.y);
        }
        tc::tmem_st16(ts + 64 + 16 * q, p);
      }
      const float2 sums = unpack_f32x2(add_f32x2(sum0, sum1));
      l += sums.x + sums.y;
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_full + tile);
    }
    if (ok) {
      ok = tc::warp_wait(pv_done + tile, (n_tiles - 1) & 1, abort_flag, a.status);
      tc::tc_fence_after();
    }
    if (ok) {
      const float inv = l == 0.f ? 0.f : v_ref / l;
      uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(sv.q0 + row / G) * a.out_stride +
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
    tc::reg_dec<80>();
    // ------------------------------------------------------------------ codes -> f16 tiles
    const int w = warp - 12;
    // K: this warp's 16 tokens of the tile (one page); a lane takes 16 bytes of rows lane % 8 and + 8
    // V: 32 x 32 pieces (tokens x elements); a lane takes 4 elements of 8 tokens, chosen so that eight
    // lanes store to eight different 16-byte columns of the swizzled rows
    constexpr int VP = 2 * KC / 2;                 // V pieces per warp: 1 or 2
    const int tg = lane & 3, dg = ((lane >> 2) & 1) | (lane >> 3) << 1;
    uint4 kr[2][KC];
    uint32_t vr[VP][8];
    float k_scale, v_scale[VP];
    const int pshift = 31 - __clz(P);
    const float k_inv = 1.0f / k_ref, v_inv = 1.0f / v_ref;
    uint32_t k_gone = 0;
    // page of a token, -1 for one that no row sees; looked up a tile ahead
    auto page_of = [&](int tok) { return tok < tok_hi ? table[tok >> pshift] : -1; };
    auto good = [&](int page) { return page >= 0 && page < a.c.n_pages; };
    const int k_tok = j_lo * kAtTok + w * 16;
    int v_tok[VP], k_page = page_of(k_tok), v_page[VP];
#pragma unroll
    for (int p = 0; p < VP; ++p) {
      // piece: tokens (u % 4) * 32, elements (u / 4) * 32
      v_tok[p] = j_lo * kAtTok + ((w * VP + p) & 3) * 32 + tg * 8;
      v_page[p] = page_of(v_tok[p]);
    }
    auto load_k = [&](int j) {
      const int tok = k_tok + j * kAtTok;
      const bool on = good(k_page);
      k_gone = !on && tok < tok_hi;
      if (k_gone && lane == 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
      const int64_t ph = on ? static_cast<int64_t>(k_page) * a.c.n_kv_heads + h : 0;
      k_scale = on ? a.c.k_scales[ph] : 0.f;
      const uint8_t* src = a.c.k_codes + ((ph << pshift) + (tok & (P - 1)) + (lane & 7)) * kD + (lane >> 3) * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          kr[i][c] = make_uint4(0u, 0u, 0u, 0u);
          if (on && tok + (lane & 7) + 8 * i < tok_hi)
            kr[i][c] = __ldcg(reinterpret_cast<const uint4*>(src + 8 * i * kD + c * 64));
        }
      k_page = page_of(tok + kAtTok);
    };
    auto load_v = [&](int j) {
#pragma unroll
      for (int p = 0; p < VP; ++p) {
        const int u = w * VP + p, tok = v_tok[p] + j * kAtTok;
        const bool on = good(v_page[p]);
        const int64_t ph = on ? static_cast<int64_t>(v_page[p]) * a.c.n_kv_heads + h : 0;
        v_scale[p] = on ? a.c.v_scales[ph] : 0.f;
        const uint8_t* src = a.c.v_codes + ((ph << pshift) + (tok & (P - 1))) * kD + (u >> 2) * 32 + dg * 4;
        const int n = on ? tok_hi - tok : 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) vr[p][t] = t < n ? __ldcg(reinterpret_cast<const uint32_t*>(src + t * kD)) : 0u;
        v_page[p] = page_of(tok + kAtTok);
      }
    };
    auto store_k = [&](uint8_t* dst) {
      const float r = k_scale * k_inv;
      const __half2 ks2 = __floats2half2_rn(r, r);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const int t = w * 16 + (lane & 7) + 8 * i;
          const uint32_t x[4] = {kr[i][c].x, kr[i][c].y, kr[i][c].z, kr[i][c].w};
          uint8_t* rowp = dst + c * (128 * 128) + t * 128;
          const int ch = 2 * (lane >> 3);
#pragma unroll
          for (int b = 0; b < 2; ++b)
            *reinterpret_cast<uint4*>(rowp + (((ch + b) ^ (t & 7)) << 4)) =
                make_uint4(scaled_codes(x[2 * b], ks2), scaled_codes(x[2 * b] >> 16, ks2),
                           scaled_codes(x[2 * b + 1], ks2), scaled_codes(x[2 * b + 1] >> 16, ks2));
        }
    };
    auto store_v = [&](uint8_t* dst) {
#pragma unroll
      for (int p = 0; p < VP; ++p) {
        const int u = w * VP + p;
        const float r = v_scale[p] * v_inv;
        const __half2 vs2 = __floats2half2_rn(r, r);
        const int ch = (u & 1) * 4 + tg;           // 8-token column within a 64-token half
        uint8_t* base = dst + ((u & 3) >> 1) * (kD * 128);
        uint32_t o[4][4];                          // [element][token pair]
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t x = prmt(vr[p][2 * t], vr[p][2 * t + 1], 0x5140);
          const uint32_t y = prmt(vr[p][2 * t], vr[p][2 * t + 1], 0x7362);
          o[0][t] = scaled_codes(x, vs2);
          o[1][t] = scaled_codes(x >> 16, vs2);
          o[2][t] = scaled_codes(y, vs2);
          o[3][t] = scaled_codes(y >> 16, vs2);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int d = (u >> 2) * 32 + dg * 4 + k;
          *reinterpret_cast<uint4*>(base + d * 128 + ((ch ^ (d & 7)) << 4)) =
              make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
        }
      }
    };
    load_k(0);
    load_v(0);
    bool ok = true;
    for (int t = 0; ok && t < 2 * n_tiles; ++t) {
      const int j = t >> 1;
      ok = tc::warp_wait(kv_empty + t % kAtRing, ((t / kAtRing) & 1) ^ 1, abort_flag, a.status);
      if (!ok) break;
      uint8_t* dst = ring + (t % kAtRing) * C::TILE;
      if (t & 1) {
        store_v(dst);
        if (j + 1 < n_tiles) load_v(j + 1);
      } else {
        if (lane == 0) reinterpret_cast<volatile uint8_t*>(bad + j % kAtBad)[w] = static_cast<uint8_t>(k_gone);
        store_k(dst);
        if (j + 1 < n_tiles) load_k(j + 1);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(kv_full + t % kAtRing);
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int kD>
cudaError_t launch_tc_t(const AttnArgs& a, int blocks, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(attention_tc_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(AtCfg<kD>::SMEM));
  if (e != cudaSuccess) return e;
  return launch_kernel(attention_tc_kernel<kD>, dim3(blocks, a.c.n_kv_heads, a.b.n_seq), dim3(kAtThreads),
                       AtCfg<kD>::SMEM, stream, true, a);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnArgs& a, int blocks, cudaStream_t stream) {
  return a.c.head_dim == 64 ? launch_tc_t<64>(a, blocks, stream) : launch_tc_t<128>(a, blocks, stream);
}

}  // namespace strata
