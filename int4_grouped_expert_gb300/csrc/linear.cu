// Projections with group-quantized weights for few tokens, or few weights:
//   y[t,n] = sum_g s[n,g] sum_{c in g} x[t,c] q[n,c],
// the format of "Strata" MoE tuning notes (lpnh.cn/news/2730718, §2.1: G codes share one fp16 scale).
//
// The weights are read once. A block owns 16 to 64 weight rows and its 8 warps take alternate pieces of the
// contraction; every lane loads its codes straight into registers and multiplies them on the tensor
// cores (mma.sync m16n8k16, 16 rows as A, 8 tokens as B). The order of a contraction is free, so lane t
// of a quad takes 16 or 32 consecutive codes of a row instead of the pairs the instruction names, and
// the matching activations. What bounds it: at one token and 4 bits the ALU pipe (70% busy: shifts and
// LOP3 that unpack the codes), with more tokens the reads of x from L2. Measured: 1 token at 4 bits 1024 ->
// 1024 1.8 us, 4096 -> 6144 6.6 us (2.0 TB/s); 16 tokens at 8 bits 4096 -> 6144 10.4 us (2.5 TB/s).
//
// The codes are exact in bf16 (|q| <= 128), the activations are bf16, their products are exact in
// fp32, and the group's scale multiplies the fp32 sum: nothing is rounded before the output.
#include <algorithm>

#include "block.cuh"

namespace strata {

// bf16x2 {q_0, q_1} and {q_2, q_3} of four int8 codes: 128 + (low 7 bits) minus 128 or, where the
// sign bit is set, 256. Both are exact bf16 values, and so is the difference.
__device__ __forceinline__ void codes8_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t v0 = prmt(w, 0u, 0x4140), v1 = prmt(w, 0u, 0x4342);
  const uint32_t m0 = (v0 & 0x007F007Fu) | 0x43004300u, b0 = (v0 & 0x00800080u) | 0x43004300u;
  const uint32_t m1 = (v1 & 0x007F007Fu) | 0x43004300u, b1 = (v1 & 0x00800080u) | 0x43004300u;
  __nv_bfloat162 r0 = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m0),
                              *reinterpret_cast<const __nv_bfloat162*>(&b0));
  __nv_bfloat162 r1 = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m1),
                              *reinterpret_cast<const __nv_bfloat162*>(&b1));
  lo = *reinterpret_cast<uint32_t*>(&r0);
  hi = *reinterpret_cast<uint32_t*>(&r1);
}

// D += A * B, m16n8k16, bf16 inputs, fp32 sums. (Not volatile: the compiler may interleave independent chains.)
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// kUnit: columns of one step, 128 (32 consecutive codes a lane), or 64 for 64-wide groups (16 a
// lane), so that a step's products share one scale per row. kMT: 16-row tiles of a block, which share the
// activations that a lane reads; kPF: steps whose codes are on their way.
template <int kBits, int kUnit, int kNT, int kMT, int kPF, int kLinWarps, int kBlocks>
__global__ void __launch_bounds__(kLinWarps * 32, kBlocks) linear_stream_kernel(LinearArgs a) {
  constexpr int CPL = kUnit / 4;            // codes a lane takes of a row
  constexpr int WPL = CPL * kBits / 32;     // words of them: 2, 4 or 8
  constexpr int COLS = 8 * kNT, ROWS = 16 * kMT;
  __shared__ float red[kLinWarps][ROWS][COLS + 1];
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * ROWS;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * COLS;
  const int64_t row_bytes = static_cast<int64_t>(a.K) * kBits / 8;
  const int ng = a.K / a.group, ushift = a.group == 256 ? 1 : 0;
  // rows g and g + 8 of each tile; rows past the end repeat the last one, and their sums are not written
  const uint8_t* cp[2 * kMT];
  const __half* sp[2 * kMT];
#pragma unroll
  for (int r = 0; r < 2 * kMT; ++r) {
    const int64_t row = min(n0 + 8 * r + g, a.N - 1);
    cp[r] = a.codes + row * row_bytes + t * (CPL * kBits / 8);
    sp[r] = a.scales + row * ng;
  }
  const __nv_bfloat16* xp[kNT];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const int64_t tok = t0 + n * 8 + g;
    xp[n] = tok < a.T ? a.x + tok * a.x_stride + t * CPL : nullptr;
  }
  float acc[kMT][kNT][4];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

  uint32_t w[kPF][2 * kMT][WPL];
  __half sc[kPF][2 * kMT];
  const int units = a.K / kUnit;
  auto load = [&](int u, int slot) {
    if (u >= units) return;
#pragma unroll
    for (int r = 0; r < 2 * kMT; ++r) {
      const uint8_t* p = cp[r] + static_cast<int64_t>(u) * (kUnit * kBits / 8);
      if (WPL == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[slot][r][0] = v.x; w[slot][r][1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < WPL / 4; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
          w[slot][r][4 * i] = v.x; w[slot][r][4 * i + 1] = v.y;
          w[slot][r][4 * i + 2] = v.z; w[slot][r][4 * i + 3] = v.w;
        }
      }
      sc[slot][r] = __ldg(sp[r] + (u >> ushift));
    }
  };
#pragma unroll
  for (int p = 0; p < kPF; ++p) load(warp + p * kLinWarps, p);
  for (int u0 = warp; u0 < units; u0 += kPF * kLinWarps) {
#pragma unroll
    for (int p = 0; p < kPF; ++p) {
      const int u = u0 + p * kLinWarps;
      if (u >= units) break;
      float part[kMT][kNT][4];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[m][n][i] = 0.f;
      // 8 columns at a time: two MMA steps of 4 columns per lane
#pragma unroll
      for (int j = 0; j < CPL / 8; ++j) {
        uint4 xv[kNT];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
          xv[n] = xp[n] ? *(reinterpret_cast<const uint4*>(xp[n] + u * kUnit) + j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          const uint32_t* w0 = w[p][2 * m];
          const uint32_t* w1 = w[p][2 * m + 1];
          uint32_t A[2][4];
          if (kBits == 4) {
            // pairs (0,4) (1,5) and (2,6) (3,7) of the 8 codes
            const uint32_t u0_ = w0[j] ^ 0x88888888u, u1_ = w1[j] ^ 0x88888888u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              A[h][0] = int4pair_to_bf16x2(u0_, 2 * h);
              A[h][1] = int4pair_to_bf16x2(u1_, 2 * h);
              A[h][2] = int4pair_to_bf16x2(u0_, 2 * h + 1);
              A[h][3] = int4pair_to_bf16x2(u1_, 2 * h + 1);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              codes8_bf16(w0[(2 * j + h) % WPL], A[h][0], A[h][2]);
              codes8_bf16(w1[(2 * j + h) % WPL], A[h][1], A[h][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            if (kBits == 4) {
              mma_bf16(part[m][n], A[0], prmt(xv[n].x, xv[n].z, 0x5410), prmt(xv[n].x, xv[n].z, 0x7632));
              mma_bf16(part[m][n], A[1], prmt(xv[n].y, xv[n].w, 0x5410), prmt(xv[n].y, xv[n].w, 0x7632));
            } else {
              mma_bf16(part[m][n], A[0], xv[n].x, xv[n].y);
              mma_bf16(part[m][n], A[1], xv[n].z, xv[n].w);
            }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        const float f0 = __half2float(sc[p][2 * m]), f1 = __half2float(sc[p][2 * m + 1]);
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          acc[m][n][0] = fmaf(f0, part[m][n][0], acc[m][n][0]);
          acc[m][n][1] = fmaf(f0, part[m][n][1], acc[m][n][1]);
          acc[m][n][2] = fmaf(f1, part[m][n][2], acc[m][n][2]);
          acc[m][n][3] = fmaf(f1, part[m][n][3], acc[m][n][3]);
        }
      }
      load(u + kPF * kLinWarps, p);
    }
  }
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][16 * m + g + 8 * (i >> 1)][n * 8 + 2 * t + (i & 1)] = acc[m][n][i];
  // what is added comes first, all of it at once: loads between the stores to out (which may be the
  // residual) would wait for one another
  constexpr int THREADS = kLinWarps * 32, ITEMS = (ROWS * COLS + THREADS - 1) / THREADS;
  float plus[ITEMS];
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const int i = threadIdx.x + u * THREADS, r = i % ROWS, c = i / ROWS;
    plus[u] = 0.f;
    if (c >= COLS || n0 + r >= a.N || t0 + c >= a.T) continue;
    if (a.bias) plus[u] = a.bias[n0 + r];
    if (a.residual) plus[u] += __bfloat162float(a.residual[(t0 + c) * a.residual_stride + n0 + r]);
  }
  __syncthreads();
  // the warps' sums in a fixed order, consecutive threads along the weight rows (output columns)
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const int i = threadIdx.x + u * THREADS, r = i % ROWS, c = i / ROWS;
    if (c >= COLS || n0 + r >= a.N || t0 + c >= a.T) continue;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < kLinWarps; ++k) y += red[k][r][c];
    a.out[(t0 + c) * a.out_stride + n0 + r] = __float2bfloat16_rn(y + plus[u]);
  }
}

constexpr int kLinSms = 152;
constexpr int kLinNarrowN = kLinSms * 16;  // up to here 16-row blocks take one round

// Whether more than 32 tokens are streamed too, 32 at a time, or go to linear_tc.cu: by what either was
// measured to take, in hundredths of us. A round of streaming blocks on all SMs grows with K; the other
// kernel's time is mostly its start, a cluster's join and, beyond 64 tokens, the pass before it. (us, streamed
// / tcgen05, at 4 bits: 64 tokens 1024 -> 1024 3.3 / 7.5, 4096 -> 1024 7.3 / 9.9, 4096 -> 2048 12.4 / 10.7;
// 256 tokens 4096 -> 256 7.2 / 19.5, 4096 -> 1024 23.5 / 20.9; 33 tokens 7168 -> 9216 38.9 / 22.4.)
bool linear_streams(int64_t T, int64_t K, int64_t N) {
  if (T <= kLinearStreamT) return true;
  const bool narrow = N <= kLinNarrowN;
  const int64_t rows = narrow ? 16 : 64;
  const int64_t rounds = ((N + rows - 1) / rows * ((T + 31) / 32) + kLinSms - 1) / kLinSms;
  const int64_t stream = narrow ? 200 + rounds * (60 + 115 * K / 1024) : 150 + rounds * (250 + 205 * K / 1024);
  const int64_t other = T <= kLinearMidT ? 550 + 65 * K / 1024 + 3 * T / 2
                                         : 830 + 85 * K / 1024 + 5 * std::min<int64_t>(T, 300) / 2;
  return stream < other;
}

template <int kBits, int kUnit, int kNT, int kMT, int kPF, int kLinWarps, int kBlocks>
static cudaError_t launch_stream_n(const LinearArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.N + 16 * kMT - 1) / (16 * kMT)),
                  static_cast<unsigned>((a.T + 8 * kNT - 1) / (8 * kNT)));
  return launch_kernel(linear_stream_kernel<kBits, kUnit, kNT, kMT, kPF, kLinWarps, kBlocks>, grid, kLinWarps * 32, 0,
                       stream, true, a);
}
// Up to 8 tokens the weights are all the traffic: 16 rows a block, the next step's codes on their way. With
// more, every block reads all of x, and wider blocks (32 rows, 64 beyond 16 tokens) read it less
// often; where 16-row blocks leave SMs idle, they are faster (us, wide / 16 rows: 16 tokens, 8 bits,
// 7168 -> 9216 19.6 / 32.1, 4 bits, 1024 -> 1024 2.7 / 2.2; 32 tokens 30.4 / 67 and 5.6 / 3.2). Blocks of 48
// rows and 16 warps, one an SM, where 32-row blocks, two an SM, put two on most SMs: x is read by fewer blocks. Their
// reduction over 16 warps pays from 384 columns a bit on. (us, 32 / 48 rows, 16 tokens, to 4868 and to 7296
// columns: 4 bits 1024 4.3 / 4.4, 4.5 / 4.4, 1536 5.2 / 4.9, 5.4 / 4.9, 4096 9.4 / 8.2, 9.7 / 8.2; 8 bits 1024 4.4 / 5.0, 4.6 /
// 4.9, 2048 6.4 / 6.8, 6.7 / 6.7, 3200 9.0 / 8.8, 9.4 / 9.0, 7168 16.0 / 14.9, 16.3 / 15.3; one 32-row block an SM:
// 4 bits 4096 -> 4096 5.9 / 8.2.)
template <int kBits, int kUnit>
static cudaError_t launch_stream_t(const LinearArgs& a, cudaStream_t stream) {
  const bool narrow = a.N <= kLinNarrowN;
  const bool wide = a.N > kLinSms * 32 && a.N <= kLinSms * 48 && a.K >= 384 * kBits;
  if (a.T <= 8) return launch_stream_n<kBits, kUnit, 1, 1, 2, 8, 3>(a, stream);
  if (a.T <= 16)
    return narrow ? launch_stream_n<kBits, kUnit, 2, 1, 1, 8, 3>(a, stream)
           : wide ? launch_stream_n<kBits, kUnit, 2, 3, 1, 16, 1>(a, stream)
                  : launch_stream_n<kBits, kUnit, 2, 2, 1, 8, 2>(a, stream);
  return narrow ? launch_stream_n<kBits, kUnit, 4, 1, 1, 8, 2>(a, stream)
                : launch_stream_n<kBits, kUnit, 4, 4, 1, 8, 1>(a, stream);
}

cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t stream) {
  if (a.bits == 4)
    return a.group == 64 ? launch_stream_t<4, 64>(a, stream) : launch_stream_t<4, 128>(a, stream);
  return a.group == 64 ? launch_stream_t<8, 64>(a, stream) : launch_stream_t<8, 128>(a, stream);
}

}  // namespace strata
