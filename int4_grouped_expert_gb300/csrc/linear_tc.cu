// Projections with group-quantized weights for many tokens, on tcgen05: out[t][n] = sum_c x[t][c] w[n][c]
// with w = f16(q * s) ("Strata" MoE tuning notes, lpnh.cn/news/2730718, §2.1: G codes share one scale).
//
// Tile: 128 weight rows (the MMA's M, one TMEM lane each) x up to 256 tokens, contraction in 64-wide
// stages. The weights are the A operand and go to tensor memory, not shared memory: a thread
// dequantizes 64 codes of its row and stores them to its own TMEM lane, so shared memory carries only
// the activations. (Both operands in shared memory would move 96 KB a stage, 188 bytes a clock at the
// MMA's pace, and 128 is what shared memory has; this way it is 64 KB.)
//   warp 0       TMA (one elected lane): the stage's tokens (f16, 128-byte swizzle) -> a ring in shared memory
//   warp 1       an elected lane issues tcgen05.mma (f16, M = 128, N = tokens, K = 16)
//   warp 2       owns the TMEM allocation: 256 columns of sums, 8 stages x 32 columns of weights
//   warps 4-11   dequantize: two warps per 32 lanes, one for the even and one for the odd stages
//   warps 12-15  epilogue: TMEM -> registers -> bias, residual -> bf16
// Blocks are persistent over the tiles. Where the tiles are too few to fill the GPU, a cluster of 2 to
// 8 blocks shares a tile along the contraction; the sums meet in shared memory over the cluster, in
// the order of the ranks.
//
// Operands are f16: the weight is the exact code times the fp16 scale, rounded once (2^-11 relative; bf16
// would leave 2^-8), and a pass before this kernel copies x to f16, each row times a power of two that
// keeps its range; the epilogue multiplies it back.
//
// Every mbarrier wait is bounded in time; on time-out the kernel sets STRATA_DEV_TIMEOUT, every role
// leaves its loop, in-flight copies and MMAs are drained (bounded) and TMEM is freed.
#include <cudaTypedefs.h>

#include <algorithm>

#include "block.cuh"
#include "tc_ts_ptx.cuh"

namespace strata {

namespace {

constexpr int kLtRows = 128;              // weight rows per tile
constexpr int kLtTok = 256;               // tokens per tile
constexpr int kLtBK = 64;                 // contraction per stage
constexpr int kLtAStages = 8;             // weight stages in TMEM, 32 columns each
constexpr int kLtBStages = 6;             // activation stages in shared memory
constexpr int kLtBBytes = kLtTok * kLtBK * 2;
constexpr int kLtBox = 64;                // token rows per TMA box
constexpr int kLtThreads = 512;
constexpr size_t kLtSmem = static_cast<size_t>(kLtBStages) * kLtBBytes + 1024 + 512;

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
                                                          int K, __half* __restrict__ xh, int* __restrict__ xexp) {
  __shared__ uint32_t s_mag[8];
  griddep_wait();
  griddep_launch();
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

__device__ __forceinline__ float lt_epilogue(const LinearArgs& a, float y, float bias, int64_t tok, int n) {
  y += bias;
  if (a.residual) y += __bfloat162float(a.residual[tok * a.residual_stride + n]);
  return y;
}

template <int kBits>
__global__ void __launch_bounds__(kLtThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, LinearArgs a, int ks) {
  extern __shared__ uint8_t lt_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lt_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kLtBStages * kLtBBytes);
  uint64_t* full_a = bars;
  uint64_t* empty_a = full_a + kLtAStages;
  uint64_t* full_b = empty_a + kLtAStages;
  uint64_t* empty_b = full_b + kLtBStages;
  uint64_t* acc_full = empty_b + kLtBStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kLtAStages; ++s) {
      tc::mbar_init(full_a + s, 4);   // one warp per lane quarter
      tc::mbar_init(empty_a + s, 1);
    }
    for (int s = 0; s < kLtBStages; ++s) {
      tc::mbar_init(full_b + s, 1);
      tc::mbar_init(empty_b + s, 1);
    }
    tc::mbar_init(acc_full, 1);
    tc::mbar_init(acc_empty, 4);      // the epilogue warps
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
  const uint32_t tmem_a = tmem + kLtTok;
  griddep_wait();
  griddep_launch();

  // tile = (token block, 128 weight rows), weight rows fastest
  const int mtiles = (a.N + kLtRows - 1) / kLtRows;
  const int ttiles = static_cast<int>((a.T + kLtTok - 1) / kLtTok);
  const int n_items = mtiles * ttiles;
  const int rank = blockIdx.x % ks, step = gridDim.x / ks;
  const int nk_all = a.K / kLtBK;
  const int kb0 = nk_all * rank / ks, nk = nk_all * (rank + 1) / ks - kb0;  // this rank's stages
  auto tokens = [&](int item) {
    return static_cast<int>(min(static_cast<int64_t>(kLtTok), a.T - static_cast<int64_t>(item / mtiles) * kLtTok));
  };

  if (warp == 0) {
    int it = 0;
    bool ok = true;
    for (int item = blockIdx.x / ks; ok && item < n_items; item += step) {
      const int nbox = (tokens(item) + kLtBox - 1) / kLtBox;
      const int t0 = item / mtiles * kLtTok;
      for (int kb = 0; kb < nk; ++kb, ++it) {
        const int s = it % kLtBStages;
        ok = tc::warp_wait(empty_b + s, ((it / kLtBStages) & 1) ^ 1, abort_flag, a.status);
        if (!ok) break;
        if (tc::elect_one()) {
          tc::mbar_arrive_expect_tx(full_b + s, nbox * kLtBox * kLtBK * 2);
          for (int bx = 0; bx < nbox; ++bx)
            tc::tma_load_2d(smem + s * kLtBBytes + bx * kLtBox * kLtBK * 2, &tmap_x, (kb0 + kb) * kLtBK,
                            t0 + bx * kLtBox, full_b + s);
        }
        __syncwarp();
      }
    }
    if (!ok)  // drain the copies that may still be in flight
      for (int j = (it > kLtBStages ? it - kLtBStages : 0); j < it; ++j)
        tc::mbar_wait_drain(full_b + (j % kLtBStages), (j / kLtBStages) & 1);
    __syncwarp();
  } else if (warp == 1) {
    int it = 0, tcount = 0;
    bool ok = true;
    for (int item = blockIdx.x / ks; ok && item < n_items; item += step, ++tcount) {
      const uint32_t idesc = tc::idesc_f16(kLtRows, (tokens(item) + 15) & ~15);
      ok = tcount == 0 || tc::warp_wait(acc_empty, (tcount - 1) & 1, abort_flag, a.status);
      if (!ok) break;
      tc::tc_fence_after();
      for (int kb = 0; kb < nk; ++kb, ++it) {
        const int sa = it % kLtAStages, sb = it % kLtBStages;
        ok = tc::warp_wait(full_b + sb, (it / kLtBStages) & 1, abort_flag, a.status) &&
             tc::warp_wait(full_a + sa, (it / kLtAStages) & 1, abort_flag, a.status);
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t db = tc::sw128_desc(tc::smem_u32(smem + sb * kLtBBytes));
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kLtBK / 16; ++kk)
            tc::mma_f16_ts(tmem, tmem_a + sa * 32 + 8 * kk, db + 2 * kk, idesc, (kb | kk) ? 1u : 0u);
          tc::mma_commit(empty_a + sa);
          tc::mma_commit(empty_b + sb);
          if (kb == nk - 1) tc::mma_commit(acc_full);
        }
        __syncwarp();
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
        sw[u] = __ldg(sp + ((kb0 + first + 2 * m) >> gs));
      };
#pragma unroll
      for (int u = 0; u < PD; ++u) load(u, u);
      for (int m0 = 0; ok && m0 < mine; m0 += PD) {
#pragma unroll
        for (int u = 0; u < PD; ++u) {
          const int m = m0 + u;
          if (m >= mine) break;
          const int it = it0 + first + 2 * m, s = it % kLtAStages;
          const __half sh = __ushort_as_half(sw[u]);
          const __half2 s2 = __halves2half2(sh, sh);
          uint32_t w[32];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const uint32_t c[4] = {cw[u][v].x, cw[u][v].y, cw[u][v].z, cw[u][v].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (kBits == 4) {
                const uint32_t c4 = c[j] >> 4;
#pragma unroll
                for (int b = 0; b < 4; ++b) w[(16 * v + 4 * j + b) & 31] = lt_scaled(lt_pair4(c[j], c4, b), s2);
              } else {
                const uint32_t cu = c[j] ^ 0x80808080u;
#pragma unroll
                for (int b = 0; b < 2; ++b) w[(8 * v + 2 * j + b) & 31] = lt_scaled(lt_pair8(cu, b), s2);
              }
            }
          }
          // weights of the largest fp16 magnitudes may round to inf: they stay finite (nan stays nan)
          if (__half2float(sh) > 65504.f / (kBits == 4 ? 8 : 128)) {
            const __half2 top = __floats2half2_rn(65504.f, 65504.f);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const __half2 r = __hmin2_nan(__hmax2_nan(*reinterpret_cast<__half2*>(&w[i]), __hneg2(top)), top);
              w[i] = *reinterpret_cast<const uint32_t*>(&r);
            }
          }
          load(m + PD, u);
          // (the whole warp goes on or leaves: the TMEM instructions are warp-wide)
          ok = tc::warp_wait(empty_a + s, ((it / kLtAStages) & 1) ^ 1, abort_flag, a.status);
          if (!ok) break;
          tc::tc_fence_after();
          tc::tmem_st32(lane_addr + s * 32, w);
          tc::tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(full_a + s);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 12) {
    const int q4 = warp & 3;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    int tcount = 0;
    for (int item = blockIdx.x / ks; item < n_items; item += step, ++tcount) {
      if (!tc::warp_wait(acc_full, tcount & 1, abort_flag, a.status)) break;
      tc::tc_fence_after();
      const int n = item % mtiles * kLtRows + q4 * 32 + lane;
      const int64_t t0 = static_cast<int64_t>(item / mtiles) * kLtTok;
      const int nt = tokens(item);
      const float bias = a.bias && n < a.N ? a.bias[n] : 0.f;
      float* sums = reinterpret_cast<float*>(smem);  // ks > 1: [token][row], in place of the stages
      for (int c = 0; c < nt; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(lane_addr + c, r);
        const float my_up = c + lane < nt ? exp2i(a.xexp[t0 + c + lane]) : 0.f;
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          r[j] = __float_as_uint(__uint_as_float(r[j]) * __shfl_sync(0xffffffffu, my_up, j));
        if (ks > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < nt) sums[(c + j) * kLtRows + q4 * 32 + lane] = __uint_as_float(r[j]);
        } else if (n < a.N) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < nt)
              a.out[(t0 + c + j) * a.out_stride + n] =
                  __float2bfloat16_rn(lt_epilogue(a, __uint_as_float(r[j]), bias, t0 + c + j, n));
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(acc_empty);
    }
  }
  __syncwarp();
  if (ks > 1) {
    // one tile per cluster: every rank sums its share of the tokens over the ranks, in their order
    tc::cluster_sync();
    const int item = blockIdx.x / ks;
    const int nt = tokens(item), r = threadIdx.x & (kLtRows - 1);
    const int n = item % mtiles * kLtRows + r;
    const int64_t t0 = static_cast<int64_t>(item / mtiles) * kLtTok;
    if (n < a.N && !abort_flag_s) {
      const float bias = a.bias ? a.bias[n] : 0.f;
      const uint32_t base = tc::smem_u32(smem) + r * 4;
      for (int c = nt * rank / ks + (threadIdx.x >> 7); c < nt * (rank + 1) / ks; c += kLtThreads / kLtRows) {
        float y = 0.f;
        for (int k = 0; k < ks; ++k) y += tc::ld_cluster_f32(tc::cluster_map(base + c * kLtRows * 4, k));
        a.out[(t0 + c) * a.out_stride + n] = __float2bfloat16_rn(lt_epilogue(a, y, bias, t0 + c, n));
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

template <int kBits>
cudaError_t launch_tc_t(const CUtensorMap& map, const LinearArgs& a, int ks, unsigned grid, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<kBits>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kLtSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kLtThreads);
  cfg.dynamicSmemBytes = kLtSmem;
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
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<kBits>, map, a, ks);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return cudaErrorInvalidValue;
  cudaError_t e = launch_kernel(linear_rows_kernel, dim3(static_cast<unsigned>(a.T)), dim3(256), 0, stream, true,
                                a.x, a.x_stride, a.K, a.xh, a.xexp);
  if (e != cudaSuccess) return e;
  // the f16 rows as a 2-d tensor: boxes of 64 tokens x 64 columns (128 bytes), zero fill past the last token
  CUtensorMap map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.T)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.K) * 2};
  const cuuint32_t box[2] = {kLtBK, kLtBox}, estr[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.xh, dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int64_t items = static_cast<int64_t>((a.N + kLtRows - 1) / kLtRows) * ((a.T + kLtTok - 1) / kLtTok);
  const int nk = a.K / kLtBK;
  // contraction splits: rounds of blocks x (stages of a share + about 8 stages' worth of start, drain
  // and join), only while a tile per cluster fits the GPU at once
  int ks = 1;
  int64_t best = (items + num_sms - 1) / num_sms * (nk + 8);
  for (int k = 2; k <= 8 && items * k <= num_sms && nk >= 4 * k; k *= 2) {
    const int64_t cost = (nk + k - 1) / k + 8 + k;
    if (cost < best) best = cost, ks = k;
  }
  const unsigned grid = static_cast<unsigned>(ks > 1 ? items * ks : std::min<int64_t>(items, num_sms));
  return a.bits == 4 ? launch_tc_t<4>(map, a, ks, grid, stream) : launch_tc_t<8>(map, a, ks, grid, stream);
}

}  // namespace strata
