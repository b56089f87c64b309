// Projections with group-quantized weights on tcgen05: out[t][n] = sum_c x[t][c] w[n][c], w = q * s ("Strata"
// MoE tuning notes, lpnh.cn/news/2730718, §2.1: G codes share one scale).
//
// Tile: 128 weight rows (the MMA's M, one TMEM lane each) x up to 256 tokens, contraction in 64-wide
// stages. The weights are the A operand and go to tensor memory, not shared memory: a thread
// dequantizes 64 codes of its row and stores them to its own TMEM lane, so shared memory carries only
// the activations. (Both operands in shared memory would move 96 KB a stage, 188 bytes a clock at the
// MMA's pace, and 128 is what shared memory has; this way it is 64 KB.)
//   warp 0       TMA (one elected lane): the stage's tokens (16-bit, 128-byte swizzle) -> a ring in
//                shared memory
//   warp 1       an elected lane issues tcgen05.mma (M = 128, N = tokens, K = 16)
//   warp 2       owns the TMEM allocation: the sums, then a ring of weight stages
//   warps 4-11   dequantize: two warps per 32 lanes, one for the even and one for the odd stages
//   warps 12-15  epilogue: TMEM -> registers -> bias, residual -> bf16
// Blocks are persistent over the tiles. Where the tiles are too few to fill the GPU, a cluster of 2 to
// 8 blocks shares a tile along the contraction; the sums meet in shared memory over the cluster, in
// the order of the ranks.
//
// Two operand forms:
//   up to 64 tokens (kMid)  unpacking the codes is what bounds it, so they are multiplied as exact
//       bf16 integers with x as it is (bf16, no pass before), group by group into one of four sums in
//       TMEM, which the epilogue warps multiply by the group's scale and add up in fp32 registers.
//   more tokens   the MMAs bound it: f16 operands, w = q * s rounded once (2^-11; bf16 would leave 2^-8), and
//       a pass before copies x to f16, each row times a power of two that keeps its range; the epilogue
//       multiplies it back.
//
// Measured at 4 bits: 64 tokens 7168 -> 9216 23 us (1.4 TB/s of codes); 4096 tokens 373 us, 1450 TFLOP/s, in short runs
// and 400 us, 1350 TFLOP/s, once the power limit holds the clocks (tensor pipe 65%; a stage's conversion and store to
// TMEM and the epilogue, which no other sum overlaps, are the rest).
//
// Every mbarrier wait is bounded in time; on time-out the kernel sets STRATA_DEV_TIMEOUT, every role
// leaves its loop, in-flight copies and MMAs are drained (bounded) and TMEM is freed.
#include <cudaTypedefs.h>

#include <algorithm>

#include "block.cuh"
#include "tc_ts_ptx.cuh"

namespace strata {

namespace {

constexpr int kLtRows = 128;  // weight rows per tile
constexpr int kLtBK = 64;     // contraction per stage
constexpr int kLtThreads = 512;
template <bool kMid>
struct LtCfg {
  static constexpr int TOK = kMid ? 64 : 256;        // tokens per tile
  static constexpr int BUFS = kMid ? 4 : 1;          // sums in TMEM (256 columns), then the weight stages
  static constexpr int STAGES = kMid ? 8 : 6;        // weights in TMEM (32 columns), tokens in shared memory
  static constexpr int B_BYTES = TOK * kLtBK * 2;
  static constexpr size_t SMEM = static_cast<size_t>(STAGES) * B_BYTES + 1024 + 512;
};

// bf16x2 of two codes, exact. 4 bits: codes 2 byte, 2 byte + 1 of an 8-code word; w4 is the word >> 4.
__device__ __forceinline__ __nv_bfloat162 lt_pair4_bf16(uint32_t w, uint32_t w4, int byte) {
  const uint32_t v = prmt(w, w4, byte | (byte + 4) << 8);  // low nibbles of bytes 0 and 2: the codes
  uint32_t d;  // (v & 0x000F000F) ^ 0x43084308: 136 + q
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(v), "n"(0x000F000F), "n"(0x43084308));
  return __hsub2(*reinterpret_cast<__nv_bfloat162*>(&d), __floats2bfloat162_rn(136.f, 136.f));
}
// 8 bits: 128 + (low 7 bits) minus 128, or 256 where the sign bit is set.
__device__ __forceinline__ __nv_bfloat162 lt_pair8_bf16(uint32_t w, int pair) {
  const uint32_t v = prmt(w, 0u, pair ? 0x4342 : 0x4140);
  const uint32_t m = (v & 0x007F007Fu) | 0x43004300u, b = (v & 0x00800080u) | 0x43004300u;
  return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&b));
}
// f16x2 of two codes, exact. 4 bits: codes 2 byte, 2 byte + 1 of an 8-code word; w4 is the word >> 4.
__device__ __forceinline__ __half2 lt_pair4(uint32_t w, uint32_t w4, int byte) {
  const uint32_t v = prmt(w, w4, byte | (byte + 4) << 8);  // low nibbles of bytes 0 and 2: the codes
  uint32_t d;  // (v & 0x000F000F) ^ 0x64086408: 1032 + q
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(v), "n"(0x000F000F), "n"(0x64086408));
  return __hsub2(*reinterpret_cast<__half2*>(&d), __floats2half2_rn(1032.f, 1032.f));
}
// 8 bits: the byte with its sign bit flipped in the low mantissa of 1024 is 1152 + q. u: the word ^ 0x80808080.
__device__ __forceinline__ __half2 lt_pair8(uint32_t u, int pair) {
  const uint32_t v = prmt(u, 0x64646464u, pair ? 0x4342 : 0x4140);
  return __hsub2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(1152.f, 1152.f));
}
__device__ __forceinline__ uint32_t lt_scaled(__half2 q, __half2 s) {
  const __half2 r = __hmul2(q, s);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// f16 copy of the rows of x, each times 2^-e (its largest entry in [8, 16)), and e.
__global__ void __launch_bounds__(256) linear_rows_kernel(const __nv_bfloat16* __restrict__ x, int64_t stride,
                                                          int K, __half* __restrict__ xh, int* __restrict__ xexp,
                                                          uint32_t* status) {
  __shared__ uint32_t s_mag[8];
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  const uint4* src = reinterpret_cast<const uint4*>(x + blockIdx.x * stride);
  uint4* dst = reinterpret_cast<uint4*>(xh + static_cast<int64_t>(blockIdx.x) * K);
  uint32_t m = 0;
  for (int c = threadIdx.x; c < K / 8; c += 256) m = max(m, bf16x8_mag(src[c]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) s_mag[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, s_mag[w]);
  const int e = row_exp(m);
  const float f = exp2i(-e);
  if (threadIdx.x == 0) xexp[blockIdx.x] = e;
  for (int c = threadIdx.x; c < K / 8; c += 256) {
    const uint4 v = src[c];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(bf16_lo_f32(w[j]) * f, bf16_hi_f32(w[j]) * f);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The residual of n_rows tokens from tok on, column n, as bf16 bits: all loads before the stores to out, which
// may be the same memory (loads between the stores wait for one another: 1186 tokens 3200 -> 3844 at 8 bits
// took 181 us).
template <int kRows>
__device__ __forceinline__ void lt_residual(const LinearArgs& a, int64_t tok, int n, int n_rows,
                                            uint32_t (&r)[kRows]) {
  const uint16_t* src = reinterpret_cast<const uint16_t*>(a.residual) + tok * a.residual_stride + n;
  if (n >= a.N) n_rows = 0;
  if (n_rows >= kRows) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) r[j] = src[j * a.residual_stride];
  } else {
#pragma unroll
    for (int j = 0; j < kRows; ++j) r[j] = j < n_rows ? src[j * a.residual_stride] : 0u;
  }
}

template <int kBits, bool kMid>
__global__ void __launch_bounds__(kLtThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, LinearArgs a, int ks, int box_rows) {
  using C = LtCfg<kMid>;
  extern __shared__ uint8_t lt_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lt_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::B_BYTES);
  uint64_t* full = bars;                  // a stage's weights and tokens are in place
  uint64_t* empty = full + C::STAGES;     // its MMAs are done
  uint64_t* acc_full = empty + C::STAGES;  // [BUFS]
  uint64_t* acc_empty = acc_full + C::BUFS;
  uint64_t* drain = acc_empty + C::BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(full + s, 5);   // the four dequant warps of a stage and the TMA
      tc::mbar_init(empty + s, 1);
    }
    for (int i = 0; i < C::BUFS; ++i) {
      tc::mbar_init(acc_full + i, 1);
      tc::mbar_init(acc_empty + i, 4);  // the epilogue warps
    }
    tc::mbar_init(drain, 1);
    tc::fence_barrier_init();
    abort_flag_s = 0;
  }
  if (warp == 2) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) tc::prefetch_tmap(&tmap_x);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_a = tmem + 256;
  griddep_wait();
  griddep_launch();
  if (kMid && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;  // (else the pass before has cleared it)

  // tile = (token block, 128 weight rows), weight rows fastest
  const int mtiles = (a.N + kLtRows - 1) / kLtRows;
  const int ttiles = static_cast<int>((a.T + box_rows - 1) / box_rows);
  const int n_items = mtiles * ttiles;
  const int rank = blockIdx.x % ks, step = gridDim.x / ks;
  // a sum's stages: a scale group, or the whole contraction; and this rank's share of them
  const int per = kMid ? a.group / kLtBK : a.K / kLtBK, share = kMid ? per : 1;
  const int parts = a.K / kLtBK / share;
  const int kb0 = parts * rank / ks * share, nk = parts * (rank + 1) / ks * share - kb0;
  const int n_sums = kMid ? nk / per : 1;   // sums per tile
  auto tokens = [&](int item) {
    return static_cast<int>(min(static_cast<int64_t>(box_rows), a.T - static_cast<int64_t>(item / mtiles) * box_rows));
  };

  if (warp == 0) {
    int it = 0;
    bool ok = true;
    for (int item = blockIdx.x / ks; ok && item < n_items; item += step) {
      const int t0 = item / mtiles * box_rows;
      for (int kb = 0; kb < nk; ++kb, ++it) {
        const int s = it % C::STAGES;
        ok = tc::warp_wait(empty + s, ((it / C::STAGES) & 1) ^ 1, abort_flag, a.status);
        if (!ok) break;
        if (tc::elect_one()) {
          // (one box: each costs the issuing warp about 130 clocks)
          tc::mbar_arrive_expect_tx(full + s, box_rows * kLtBK * 2);
          tc::tma_load_2d(smem + s * C::B_BYTES, &tmap_x, (kb0 + kb) * kLtBK, t0, full + s);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      // drain the copies that may still be in flight (a stage that its dequant warps have left does not
      // complete: the wait is bounded, and so is the copies' time)
      for (int j = (it > C::STAGES ? it - C::STAGES : 0); j < it; ++j)
        tc::mbar_wait_drain(full + (j % C::STAGES), (j / C::STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // The loop looks at the next stage's barrier while this stage's MMAs are issued: a wait costs about 100
    // clocks even when there is nothing to wait for.
    int s = 0, sum = 0;  // stage, and sums begun
    uint32_t ph = 0;
    bool ok = true, ready = false;
    const uint64_t db0 = tc::sw128_desc(tc::smem_u32(smem));
    for (int item = blockIdx.x / ks; ok && item < n_items; item += step) {
      const int n_mma = (tokens(item) + 15) & ~15;
      const uint32_t idesc = kMid ? tc::idesc_bf16(kLtRows, n_mma) : tc::idesc_f16(kLtRows, n_mma);
      int left = 0;      // stages of the sum in work still to come
      uint32_t dt = tmem;
      for (int kb = 0; kb < nk; ++kb) {
        const bool begins = kMid ? left == 0 : kb == 0;
        if (begins) {
          left = kMid ? per : nk;
          const int buf = sum % C::BUFS;
          dt = tmem + buf * C::TOK;
          ok = sum < C::BUFS || tc::warp_wait(acc_empty + buf, (sum / C::BUFS - 1) & 1, abort_flag, a.status);
          if (!ok) break;
          ++sum;
        }
        --left;
        if (!ready) {
          ok = tc::warp_wait(full + s, ph, abort_flag, a.status);
          if (!ok) break;
        }
        tc::tc_fence_after();
        const int s1 = s + 1 == C::STAGES ? 0 : s + 1;
        const uint32_t ph1 = s + 1 == C::STAGES ? ph ^ 1 : ph;
        const bool next = tc::mbar_test(full + s1, ph1);
        if (tc::elect_one()) {
          const uint64_t db = db0 + s * (C::B_BYTES >> 4);
          const uint32_t da = tmem_a + s * 32;
#pragma unroll
          for (int kk = 0; kk < kLtBK / 16; ++kk)
            tc::mma_f16_ts(dt, da + 8 * kk, db + 2 * kk, idesc, (kk > 0 || !begins) ? 1u : 0u);
          tc::mma_commit(empty + s);
          if (left == 0) tc::mma_commit(acc_full + (sum - 1) % C::BUFS);
        }
        __syncwarp();
        ready = __all_sync(0xffffffffu, next);
        s = s1;
        ph = ph1;
      }
    }
    if (!ok) {  // drain every MMA issued so far before TMEM is released
      if (tc::elect_one()) tc::mma_commit(drain);
      __syncwarp();
      tc::mbar_wait_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    const int q4 = warp & 3, par = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem_a + (static_cast<uint32_t>(q4 * 32) << 16);
    constexpr int NV = kBits * kLtBK / 128;      // 16-byte vectors of a row's stage: 2 or 4
    constexpr int PD = kBits == 4 ? 4 : 2;       // own stages in flight in registers
    const int gs = a.group == 64 ? 0 : a.group == 128 ? 1 : 2;
    const int64_t row_bytes = static_cast<int64_t>(a.K) * kBits / 8;
    const int ng = a.K / a.group;
    int it0 = 0;
    bool ok = true;
    for (int item = blockIdx.x / ks; ok && item < n_items; item += step, it0 += nk) {
      // rows past the end repeat the last one; their sums are not written
      const int64_t row = min(item % mtiles * kLtRows + q4 * 32 + lane, a.N - 1);
      const int first = (par ^ it0) & 1;
      const uint8_t* cp = a.codes + row * row_bytes + static_cast<int64_t>(kb0 + first) * (kLtBK * kBits / 8);
      const unsigned short* sp = reinterpret_cast<const unsigned short*>(a.scales) + row * ng;
      const int mine = nk > first ? (nk - first + 1) / 2 : 0;
      uint4 cw[PD][NV];
      unsigned short sw[PD];
      auto load = [&](int m, int u) {
        if (m >= mine) return;
        const uint4* p = reinterpret_cast<const uint4*>(cp + static_cast<int64_t>(m) * (2 * kLtBK * kBits / 8));
#pragma unroll
        for (int v = 0; v < NV; ++v) cw[u][v] = __ldg(p + v);
        if (!kMid) sw[u] = __ldg(sp + ((kb0 + first + 2 * m) >> gs));
      };
#pragma unroll
      for (int u = 0; u < PD; ++u) load(u, u);
      for (int m0 = 0; ok && m0 < mine; m0 += PD) {
#pragma unroll
        for (int u = 0; u < PD; ++u) {
          const int m = m0 + u;
          if (m >= mine) break;
          const int it = it0 + first + 2 * m, s = it % C::STAGES;
          const __half sh = __ushort_as_half(kMid ? 0 : sw[u]);
          const __half2 s2 = __halves2half2(sh, sh);
          uint32_t w[32];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const uint32_t c[4] = {cw[u][v].x, cw[u][v].y, cw[u][v].z, cw[u][v].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t other = kBits == 4 ? c[j] >> 4 : c[j] ^ 0x80808080u;
#pragma unroll
              for (int b = 0; b < 16 / kBits; ++b) {
                uint32_t& d = w[16 / kBits * (4 * v + j) + b];
                if (kMid) {
                  const __nv_bfloat162 q = kBits == 4 ? lt_pair4_bf16(c[j], other, b) : lt_pair8_bf16(c[j], b);
                  d = *reinterpret_cast<const uint32_t*>(&q);
                } else {
                  d = lt_scaled(kBits == 4 ? lt_pair4(c[j], other, b) : lt_pair8(other, b), s2);
                }
              }
            }
          }
          // weights of the largest fp16 magnitudes may round to inf: they stay finite (nan stays nan)
          if (!kMid && __half2float(sh) > 65504.f / (kBits == 4 ? 8 : 128)) {
            const __half2 top = __floats2half2_rn(65504.f, 65504.f);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const __half2 r = __hmin2_nan(__hmax2_nan(*reinterpret_cast<__half2*>(&w[i]), __hneg2(top)), top);
              w[i] = *reinterpret_cast<const uint32_t*>(&r);
            }
          }
          load(m + PD, u);
          // (the whole warp goes on or leaves: the TMEM instructions are warp-wide)
          ok = tc::warp_wait(empty + s, ((it / C::STAGES) & 1) ^ 1, abort_flag, a.status);
          if (!ok) break;
          tc::tc_fence_after();
          tc::tmem_st32(lane_addr + s * 32, w);
          tc::tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(full + s);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 12) {
    const int q4 = warp & 3;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    int sum = 0;
    bool ok = true;
    for (int item = blockIdx.x / ks; ok && item < n_items; item += step) {
      const int n = item % mtiles * kLtRows + q4 * 32 + lane;
      const int64_t t0 = static_cast<int64_t>(item / mtiles) * box_rows;
      const int nt = tokens(item);
      const float bias = a.bias && n < a.N ? a.bias[n] : 0.f;
      float* sums = reinterpret_cast<float*>(smem);  // ks > 1: [token][row], in place of the stages
      if constexpr (kMid) {
        float acc[C::TOK];
#pragma unroll
        for (int c = 0; c < C::TOK; ++c) acc[c] = 0.f;
        const __half* sp = a.scales + static_cast<int64_t>(min(n, a.N - 1)) * (a.K / a.group) + kb0 / per;
        __half next = n_sums > 0 ? __ldg(sp) : __half(0.f);
        for (int i = 0; i < n_sums; ++i, ++sum) {
          const int buf = sum % C::BUFS;
          const float sc = __half2float(next);
          if (i + 1 < n_sums) next = __ldg(sp + i + 1);
          ok = tc::warp_wait(acc_full + buf, (sum / C::BUFS) & 1, abort_flag, a.status);
          if (!ok) break;
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::TOK; c += 16) {
            if (c >= nt) break;
            uint32_t r[16];
            tc::tmem_ld16(lane_addr + buf * C::TOK + c, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(sc, __uint_as_float(r[j]), acc[c + j]);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(acc_empty + buf);
        }
        if (!ok) break;
        // (the last sum is complete, so this rank's stages are free for its sums)
#pragma unroll
        for (int c = 0; c < C::TOK; c += 16) {
          if (c >= nt) break;
          if (ks == 1 && a.residual) {
            uint32_t res[16];
            lt_residual(a, t0 + c, n, nt - c, res);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += __uint_as_float(res[j] << 16);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c + j >= nt) break;
            if (ks > 1)
              sums[(c + j) * kLtRows + q4 * 32 + lane] = acc[c + j];
            else if (n < a.N)
              a.out[(t0 + c + j) * a.out_stride + n] = __float2bfloat16_rn(acc[c + j] + bias);
          }
        }
      } else {
        const bool add = ks == 1 && a.residual;
        uint32_t res[32];  // one pass of 32 tokens ahead
        if (add) lt_residual(a, t0, n, nt, res);
        ok = tc::warp_wait_long(acc_full, sum & 1, abort_flag, a.status);
        if (!ok) break;
        ++sum;
        tc::tc_fence_after();
        for (int c = 0; c < nt; c += 32) {
          uint32_t r[32];
          tc::tmem_ld32(lane_addr + c, r);
          const float my_up = c + lane < nt ? exp2i(a.xexp[t0 + c + lane]) : 0.f;
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            r[j] = __float_as_uint(__uint_as_float(r[j]) * __shfl_sync(0xffffffffu, my_up, j));
          if (add) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(res[j] << 16));
            lt_residual(a, t0 + c + 32, n, nt - c - 32, res);
          }
          if (ks > 1) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < nt) sums[(c + j) * kLtRows + q4 * 32 + lane] = __uint_as_float(r[j]);
          } else if (n < a.N) {
            __nv_bfloat16* dst = a.out + (t0 + c) * a.out_stride + n;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < nt)
                dst[j * a.out_stride] = __float2bfloat16_rn(__uint_as_float(r[j]) + bias);
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(acc_empty);
      }
    }
  }
  __syncwarp();
  if (ks > 1) {
    // one tile per cluster: every rank sums its share of the tokens over the ranks, in their order
    tc::cluster_sync();
    const int item = blockIdx.x / ks;
    const int nt = tokens(item), n0 = item % mtiles * kLtRows;
    const int64_t t0 = static_cast<int64_t>(item / mtiles) * box_rows;
    const int c0 = nt * rank / ks, items = (nt * (rank + 1) / ks - c0) * (kLtRows / 4);  // (token, four rows)
    const uint32_t base = tc::smem_u32(smem);
    constexpr int U = 4;  // items on their way per thread
    for (int i0 = threadIdx.x; i0 < items && !abort_flag_s; i0 += U * kLtThreads) {
      float4 y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      float plus[U][4];  // bias and residual: before the stores, as above
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + u * kLtThreads, items - 1), n = n0 + i % (kLtRows / 4) * 4;
        const int64_t tok = t0 + c0 + i / (kLtRows / 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          plus[u][j] = a.bias && n + j < a.N ? a.bias[n + j] : 0.f;
          if (a.residual && n + j < a.N)
            plus[u][j] += __bfloat162float(a.residual[tok * a.residual_stride + n + j]);
        }
      }
      for (int k = 0; k < ks; ++k) {
        const uint32_t at = tc::cluster_map(base, k);
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * kLtThreads, items - 1);
          v[u] = tc::ld_cluster_f32x4(at + (c0 * (kLtRows / 4) + i) * 16);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          y[u].x += v[u].x; y[u].y += v[u].y; y[u].z += v[u].z; y[u].w += v[u].w;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kLtThreads;
        if (i >= items) break;
        const int64_t tok = t0 + c0 + i / (kLtRows / 4);
        const float f[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + i % (kLtRows / 4) * 4 + j;
          if (n < a.N) a.out[tok * a.out_stride + n] = __float2bfloat16_rn(f[j] + plus[u][j]);
        }
      }
    }
    tc::cluster_sync();  // no block leaves while another reads its sums
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

template <int kBits, bool kMid>
cudaError_t launch_tc_t(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  using C = LtCfg<kMid>;
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return cudaErrorInvalidValue;
  if (!kMid) {
    const cudaError_t e = launch_kernel(linear_rows_kernel, dim3(static_cast<unsigned>(a.T)), dim3(256), 0, stream,
                                        true, a.x, a.x_stride, a.K, a.xh, a.xexp, a.status);
    if (e != cudaSuccess) return e;
  }
  const int64_t mtiles = (a.N + kLtRows - 1) / kLtRows;
  int64_t items = mtiles * ((a.T + C::TOK - 1) / C::TOK);
  const int nk = a.K / kLtBK, parts = kMid ? a.K / a.group : nk;
  // contraction splits: stages of a share + about 8 stages' worth of start, drain and join, only while a
  // tile per cluster fits the GPU at once. Clusters of k blocks of this size that 152 SMs hold (the
  // GPU processing clusters leave some SMs over): 76, 46, 36, 28, 23, 15, 15 for k = 2 .. 8.
  constexpr int kHeld[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  int ks = 1;
  int64_t best = (items + num_sms - 1) / num_sms * (nk + 8);
  for (int k = 2; k <= 8 && nk >= 4 * k && parts >= k; ++k) {
    const int64_t cost = (parts + k - 1) / k * (nk / parts) + 8 + k;
    if (items * 152 <= static_cast<int64_t>(kHeld[k]) * num_sms && cost < best) best = cost, ks = k;
  }
  // Tokens of a tile: as few as take no more rounds of all SMs. (A round's time is mostly the conversion of
  // its weights, a little the tokens': 1186 tokens 3200 -> 3844 at 8 bits, 31 rows of 5 tiles in two
  // rounds, 59.5 us; 31 rows of 9 tiles of 144 tokens, in two rounds, 52.6.)
  int64_t ttiles = (a.T + C::TOK - 1) / C::TOK;
  if (!kMid && ks == 1) ttiles = std::max(ttiles, (items + num_sms - 1) / num_sms * num_sms / mtiles);
  const int box_rows = static_cast<int>(std::min<int64_t>(C::TOK, ((a.T + ttiles - 1) / ttiles + 15) / 16 * 16));
  items = mtiles * ((a.T + box_rows - 1) / box_rows);
  // the tokens (x itself, or its f16 copy) as a 2-d tensor: boxes of a tile's tokens x 64 columns (128 bytes),
  // zero fill past the last token
  CUtensorMap map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.T)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kMid ? a.x_stride : a.K) * 2};
  const cuuint32_t box[2] = {kLtBK, static_cast<cuuint32_t>(box_rows)}, estr[2] = {1, 1};
  if (enc(&map, kMid ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          kMid ? const_cast<void*>(static_cast<const void*>(a.x)) : static_cast<void*>(a.xh), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<kBits, kMid>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ks > 1 ? items * ks : std::min<int64_t>(items, num_sms)));
  cfg.blockDim = dim3(kLtThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<kBits, kMid>, map, a, ks, box_rows);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  if (a.T <= kLinearMidT)
    return a.bits == 4 ? launch_tc_t<4, true>(a, num_sms, stream) : launch_tc_t<8, true>(a, num_sms, stream);
  return a.bits == 4 ? launch_tc_t<4, false>(a, num_sms, stream) : launch_tc_t<8, false>(a, num_sms, stream);
}

}  // namespace strata
