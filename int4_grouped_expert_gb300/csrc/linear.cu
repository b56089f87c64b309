// Projections with group-quantized weights for few tokens: y[t,n] = sum_g s[n,g] sum_{c in g} x[t,c] q[n,c],
// the format of "Strata" MoE tuning notes (lpnh.cn/news/2730718, §2.1: G codes share one fp16 scale).
//
// The weights are read once, so the kernel is bound by streaming their codes. A block owns 16 weight
// rows and its 8 warps take alternate pieces of the contraction; every lane loads its codes straight
// into registers and multiplies them on the tensor cores (mma.sync m16n8k16, the 16 rows as A, 8
// tokens as B). The order of a contraction is free, so lane t of a quad takes 16 or 32 consecutive
// codes of a row instead of the pairs the instruction names, and the matching activations.
//
// The codes are exact in bf16 (|q| <= 128), the activations are bf16, their products are exact in
// fp32, and the group's scale multiplies the fp32 sum: nothing is rounded before the output.
#include "block.cuh"

namespace strata {

constexpr int kLinWarps = 8;

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

// kUnit: columns of one step, 128 (32 consecutive codes a lane), or 64 for 64-wide groups (16 a
// lane), so that a step's products share one scale per row.
template <int kBits, int kNT, int kUnit>
__global__ void __launch_bounds__(kLinWarps * 32) linear_stream_kernel(LinearArgs a) {
  constexpr int CPL = kUnit / 4;            // codes a lane takes of a row
  constexpr int WPL = CPL * kBits / 32;     // words of them: 2, 4 or 8
  constexpr int COLS = 8 * kNT;
  __shared__ float red[kLinWarps][16][COLS + 1];
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * COLS;
  const int64_t row_bytes = static_cast<int64_t>(a.K) * kBits / 8;
  // rows past the end repeat the last one; their sums are not written
  const int64_t r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
  const uint8_t* c0 = a.codes + r0 * row_bytes + t * (CPL * kBits / 8);
  const uint8_t* c1 = a.codes + r1 * row_bytes + t * (CPL * kBits / 8);
  const int ng = a.K / a.group, ushift = a.group == 256 ? 1 : 0;
  const __half* s0 = a.scales + r0 * ng;
  const __half* s1 = a.scales + r1 * ng;
  float acc[kNT][4];
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;

  auto load_codes = [&](const uint8_t* p, uint32_t (&w)[WPL]) {
    if (WPL == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < WPL / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    }
  };

  const int units = a.K / kUnit;
  for (int u = warp; u < units; u += kLinWarps) {
    uint32_t w0[WPL], w1[WPL];
    load_codes(c0 + static_cast<int64_t>(u) * (kUnit * kBits / 8), w0);
    load_codes(c1 + static_cast<int64_t>(u) * (kUnit * kBits / 8), w1);
    const float f0 = __half2float(__ldg(s0 + (u >> ushift)));
    const float f1 = __half2float(__ldg(s1 + (u >> ushift)));
    float part[kNT][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
    // 8 columns at a time: two MMA steps of 4 columns per lane
#pragma unroll
    for (int j = 0; j < CPL / 8; ++j) {
      uint32_t A[2][4];
      if (kBits == 4) {
        // pairs (0,4) (1,5) and (2,6) (3,7) of the 8 codes
        const uint32_t u0 = w0[j] ^ 0x88888888u, u1 = w1[j] ^ 0x88888888u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          A[h][0] = int4pair_to_bf16x2(u0, 2 * h);
          A[h][1] = int4pair_to_bf16x2(u1, 2 * h);
          A[h][2] = int4pair_to_bf16x2(u0, 2 * h + 1);
          A[h][3] = int4pair_to_bf16x2(u1, 2 * h + 1);
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
        const int64_t tok = t0 + n * 8 + g;
        uint4 xv = make_uint4(0u, 0u, 0u, 0u);
        if (tok < a.T)
          xv = *(reinterpret_cast<const uint4*>(a.x + tok * a.x_stride + u * kUnit + t * CPL) + j);
        if (kBits == 4) {
          mma_bf16_16816(part[n], A[0], prmt(xv.x, xv.z, 0x5410), prmt(xv.x, xv.z, 0x7632), part[n]);
          mma_bf16_16816(part[n], A[1], prmt(xv.y, xv.w, 0x5410), prmt(xv.y, xv.w, 0x7632), part[n]);
        } else {
          mma_bf16_16816(part[n], A[0], xv.x, xv.y, part[n]);
          mma_bf16_16816(part[n], A[1], xv.z, xv.w, part[n]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      acc[n][0] = fmaf(f0, part[n][0], acc[n][0]);
      acc[n][1] = fmaf(f0, part[n][1], acc[n][1]);
      acc[n][2] = fmaf(f1, part[n][2], acc[n][2]);
      acc[n][3] = fmaf(f1, part[n][3], acc[n][3]);
    }
  }
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    red[warp][g][n * 8 + 2 * t] = acc[n][0];
    red[warp][g][n * 8 + 2 * t + 1] = acc[n][1];
    red[warp][g + 8][n * 8 + 2 * t] = acc[n][2];
    red[warp][g + 8][n * 8 + 2 * t + 1] = acc[n][3];
  }
  __syncthreads();
  // the warps' sums in a fixed order, consecutive threads along the weight rows (output columns)
  for (int i = threadIdx.x; i < 16 * COLS; i += kLinWarps * 32) {
    const int r = i & 15, c = i >> 4;
    const int64_t tok = t0 + c;
    if (n0 + r >= a.N || tok >= a.T) continue;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kLinWarps; ++w) y += red[w][r][c];
    if (a.bias) y += a.bias[n0 + r];
    if (a.residual) y += __bfloat162float(a.residual[tok * a.residual_stride + n0 + r]);
    a.out[tok * a.out_stride + n0 + r] = __float2bfloat16_rn(y);
  }
}

template <int kBits, int kUnit>
static cudaError_t launch_stream_t(const LinearArgs& a, cudaStream_t stream) {
  const unsigned gx = static_cast<unsigned>((a.N + 15) / 16);
  const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
  const dim3 grid(gx, static_cast<unsigned>((a.T + 8 * nt - 1) / (8 * nt)));
  if (nt == 1) return launch_kernel(linear_stream_kernel<kBits, 1, kUnit>, grid, kLinWarps * 32, 0, stream, true, a);
  if (nt == 2) return launch_kernel(linear_stream_kernel<kBits, 2, kUnit>, grid, kLinWarps * 32, 0, stream, true, a);
  return launch_kernel(linear_stream_kernel<kBits, 4, kUnit>, grid, kLinWarps * 32, 0, stream, true, a);
}

cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t stream) {
  if (a.bits == 4)
    return a.group == 64 ? launch_stream_t<4, 64>(a, stream) : launch_stream_t<4, 128>(a, stream);
  return a.group == 64 ? launch_stream_t<8, 64>(a, stream) : launch_stream_t<8, 128>(a, stream);
}

}  // namespace strata
