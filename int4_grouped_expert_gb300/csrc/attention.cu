// Causal attention over the paged cache of e4m3 codes with one scale per (page, K/V head):
//   o_i = sum_j softmax_j(scale * q_i . k_j) v_j   over the tokens j that query i sees,
// by one pass over the cache with the running maximum and sum of the softmax.
//
// The rows of a K/V head (query rows x query heads that share it) are the N side of mma.sync
// m16n8k16 and 16 tokens its M side: S^T = K Q^T, then O^T += V^T P^T. Codes go from global memory
// straight into registers and become f16 there, exactly (cvt e4m3x2 -> f16x2): each lane takes 16
// consecutive bytes of a K row (the order of the contraction over the head's elements is free) or of
// V rows, whose bytes are paired token by token with PRMT. The products use f16 queries (exact from
// bf16; rows of large entries are held times a power of two) and f16 probabilities (2^-11); sums, the
// statistics and the scales of the pages are fp32.
//
// A block's 8 warps take alternate 32-token steps of its range of the cache and join their results in
// shared memory. With few (sequence, head) pairs the cache is split over more blocks: each leaves
// its maximum, sum and fp32 rows in the workspace, and the last to arrive joins them in the order
// of the splits.
#include <algorithm>

#include "attention.cuh"

namespace strata {

constexpr int kAttWarps = 8;
constexpr int kAttStep = 32;  // tokens of one warp step

// Transposes an 8x8 matrix of 16-bit elements held one row per quad.
__device__ __forceinline__ uint32_t movm_trans(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

template <int kD, int kNT>
__global__ void __launch_bounds__(kAttWarps * 32) attention_kernel(AttnArgs a) {
  constexpr int COLS = 8 * kNT;
  constexpr int KW = kD / 64;       // 16-byte pieces of a K row per lane
  constexpr int VB = kD / 8;        // bytes of a V row per lane: 16 or 8
  constexpr int VW = VB / 4;        // words of them
  constexpr int NJ = 2 * VW;        // output MMAs per token tile
  extern __shared__ float att_smem[];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.n_split, rb = blockIdx.x / a.n_split;
  const int h = blockIdx.y, s = blockIdx.z;
  const SeqView sv = seq_view(a, s, threadIdx.x == 0 && split == 0 && rb == 0 && h == 0);
  const int G = a.group, rows = sv.n * G;
  const int row0 = rb * COLS;
  if (rows > a.rows_above || row0 >= rows) return;
  const int last_row = min(row0 + COLS, rows) - 1;
  // positions of the block's first and last query, and the tokens any of them sees
  const int p_lo = sv.len - sv.n + row0 / G, p_hi = sv.len - sv.n + last_row / G;
  const int tok_hi = min(sv.len, p_hi + 1);
  const int tok_lo = a.window > 0 ? max(0, p_lo - a.window + 1) : 0;
  const int first = tok_lo / a.split_tokens;
  const int last = tok_hi > tok_lo ? (tok_hi - 1) / a.split_tokens : first;  // splits with tokens
  if (split < first || split > last) return;
  const int n_here = last - first + 1;
  const int lo = max(tok_lo, split * a.split_tokens) / kAttStep * kAttStep;
  const int hi = min(tok_hi, (split + 1) * a.split_tokens);

  // the queries of column g of each tile as f16 B fragments, times 2^-e
  uint32_t qf[kNT][4 * KW][2];
  float cmul[kNT][2];   // columns 2t, 2t+1: what turns a product into the exponent of 2
  int pos[kNT][2];      // their positions
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const int r = row0 + n * 8 + g;
    uint4 v[2 * KW];
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < 2 * KW; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const __nv_bfloat16* q = a.q + static_cast<int64_t>(sv.q0 + r / G) * a.q_stride +
                                 (h * G + r % G) * kD + (i >> 1) * 64 + t * 16;
        v[i] = *(reinterpret_cast<const uint4*>(q) + (i & 1));
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
      pos[n][i] = sv.len - sv.n + (row0 + n * 8 + 2 * t + i) / G;
    }
  }

  float o[kNT][NJ][4];
  float mx[kNT][2], sum[kNT][2];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    mx[n][0] = mx[n][1] = -INFINITY;
    sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
  }

  const int P = a.c.page_size;
  const int32_t* table = a.b.page_table + static_cast<int64_t>(s) * a.b.table_stride;
  for (int j0 = lo + warp * kAttStep; j0 < hi; j0 += kAttWarps * kAttStep) {
    // two tiles of 16 tokens, each within one page
    uint4 kr[2][2][KW];
    uint32_t vr[2][4][VW];
    float ks[2], vs[2];
    int end[2];  // tokens of the tile that may be read
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = j0 + 16 * u;
      int64_t page = -1;
      end[u] = 0;
      if (j < hi) {
        page = table[j / P];
        if (page >= 0 && page < a.c.n_pages) end[u] = min(16, sv.len - j);
        else if (lane == 0) set_status(a.status, STRATA_DEV_BAD_SLOT);
      }
      const bool on = end[u] > 0;
      const int64_t ph = on ? page * a.c.n_kv_heads + h : 0;
      const int64_t base = (ph * P + j % P) * kD;
      ks[u] = on ? a.c.k_scales[ph] : 0.f;
      vs[u] = on ? a.c.v_scales[ph] : 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          kr[u][i][w] = make_uint4(0u, 0u, 0u, 0u);
          if (g + 8 * i < end[u])
            kr[u][i][w] = __ldcg(reinterpret_cast<const uint4*>(a.c.k_codes + base + (g + 8 * i) * kD + t * 16 + w * 64));
        }
      // V rows past the end are zero, whatever the cache holds there
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + 8 * (i >> 1);
#pragma unroll
        for (int w = 0; w < VW; ++w) vr[u][i][w] = 0u;
        if (r < end[u]) {
          const uint8_t* p = a.c.v_codes + base + r * kD + g * VB;
          if (VB == 16) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
            vr[u][i][0] = v.x; vr[u][i][1] = v.y; vr[u][i][VW - 2] = v.z; vr[u][i][VW - 1] = v.w;
          } else {
            const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
            vr[u][i][0] = v.x; vr[u][i][1] = v.y;
          }
        }
      }
    }
    // S^T: tokens g, g + 8 of each tile x columns 2t, 2t+1
    float sc[kNT][2][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][u][i] = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint32_t w0[4] = {kr[u][0][w].x, kr[u][0][w].y, kr[u][0][w].z, kr[u][0][w].w};
        const uint32_t w1[4] = {kr[u][1][w].x, kr[u][1][w].y, kr[u][1][w].z, kr[u][1][w].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t A[4] = {e4m3x2_f16x2(w0[j]), e4m3x2_f16x2(w1[j]), e4m3x2_f16x2(w0[j] >> 16),
                                 e4m3x2_f16x2(w1[j] >> 16)};
#pragma unroll
          for (int n = 0; n < kNT; ++n)
            mma_f16_16816(sc[n][u], A, qf[n][4 * w + j][0], qf[n][4 * w + j][1], sc[n][u]);
        }
      }
    // exponents, masked to -inf, and the new maxima
    const bool whole = j0 >= (a.window > 0 ? p_hi - a.window + 1 : 0) && j0 + kAttStep - 1 <= p_lo &&
                       j0 + kAttStep <= sv.len && end[0] == 16 && end[1] == 16;
    float corr[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = i & 1, r = g + 8 * (i >> 1);
          float v = sc[n][u][i] * (cmul[n][c] * ks[u]);
          if (!whole) {
            const int j = j0 + 16 * u + r;
            const bool seen = r < end[u] && j <= pos[n][c] && (a.window <= 0 || j > pos[n][c] - a.window);
            if (!seen) v = -INFINITY;
          }
          sc[n][u][i] = v;
          // a nan has to reach the sum, so it must not be lost in the maximum: exp2(nan - m) is nan
          top[c] = fmaxf(top[c], v);
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], 4));
        top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], 8));
        top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], 16));
        const float m = fmaxf(mx[n][c], top[c]);
        // a column that has seen nothing yet keeps 0: its sums are zero, and so is exp2(-inf - 0)
        const float ref = m == -INFINITY ? 0.f : m;
        corr[n][c] = exp2_approx(mx[n][c] - ref);
        mx[n][c] = m;
        float add = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p = exp2_approx(sc[n][u][2 * i + c] - ref);
            sc[n][u][2 * i + c] = p;
            add += p;
          }
        sum[n][c] = fmaf(sum[n][c], corr[n][c], add);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        o[n][j][0] *= corr[n][0]; o[n][j][1] *= corr[n][1];
        o[n][j][2] *= corr[n][0]; o[n][j][3] *= corr[n][1];
      }
    }
    // O^T += vs * V^T P^T, tile by tile (the scale is the page's)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t pf[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        pf[n][0] = movm_trans(pack_f16x2(sc[n][u][0], sc[n][u][1]));
        pf[n][1] = movm_trans(pack_f16x2(sc[n][u][2], sc[n][u][3]));
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;  // bytes 0,1 or 2,3 of two tokens' words
        const uint32_t x0 = prmt(vr[u][0][j >> 1], vr[u][1][j >> 1], sel);
        const uint32_t x1 = prmt(vr[u][2][j >> 1], vr[u][3][j >> 1], sel);
        const uint32_t A[4] = {e4m3x2_f16x2(x0), e4m3x2_f16x2(x0 >> 16), e4m3x2_f16x2(x1),
                               e4m3x2_f16x2(x1 >> 16)};
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16_16816(d, A, pf[n][0], pf[n][1], d);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][i] = fmaf(vs[u], d[i], o[n][j][i]);
        }
      }
    }
  }

  // join the warps: the common maximum of a column, then the sums pairwise, in a fixed order
  float* s_mx = att_smem;                        // [kAttWarps][COLS]
  float* s_sum = s_mx + kAttWarps * COLS;        // [kAttWarps][COLS]
  float* s_o = s_sum + kAttWarps * COLS;         // [kAttWarps / 2][32 lanes][kNT * NJ * 4 + pad]
  constexpr int OL = kNT * NJ * 4;
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v = sum[n][c];  // over the tokens of the eight quads
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (g == 0) {
        s_mx[warp * COLS + n * 8 + 2 * t + c] = mx[n][c];
        s_sum[warp * COLS + n * 8 + 2 * t + c] = v;
      }
    }
  __syncthreads();
  float m_all[kNT][2], l_all[kNT][2];
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = n * 8 + 2 * t + c;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) m = fmaxf(m, s_mx[w * COLS + col]);
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) l += s_sum[w * COLS + col] * exp2_approx(s_mx[w * COLS + col] - ref);
      m_all[n][c] = m;
      l_all[n][c] = l;
      const float f = exp2_approx(mx[n][c] - ref);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        o[n][j][c] *= f;
        o[n][j][2 + c] *= f;
      }
    }
#pragma unroll
  for (int half = kAttWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
      float* dst = s_o + (warp - half) * OL * 32 + lane;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[((n * NJ + j) * 4 + i) * 32] = o[n][j][i];
    }
    __syncthreads();
    if (warp < half) {
      const float* src = s_o + warp * OL * 32 + lane;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][i] += src[((n * NJ + j) * 4 + i) * 32];
    }
    __syncthreads();
  }

  const int64_t slot = (static_cast<int64_t>(s) * a.c.n_kv_heads + h) * a.row_blocks + rb;
  if (n_here > 1) {
    // leave (o, maximum, sum) in the workspace; the last split to arrive joins them all
    float* part = a.part + (slot * a.n_split + split) * (COLS * (kD + 2));
    if (warp == 0) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = n * 8 + 2 * t + c;
          float* dst = part + col * kD + g * VB;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[n][j][c], o[n][j][2 + c]);
          if (g == 0) {
            part[COLS * kD + 2 * col] = m_all[n][c];
            part[COLS * kD + 2 * col + 1] = l_all[n][c];
          }
        }
    }
    __threadfence();
    __shared__ int s_last;
    __syncthreads();
    if (threadIdx.x == 0)  // wraps to zero at the last arrival: ready for the next call
      s_last = atomicInc(a.counters + slot, n_here - 1) == static_cast<unsigned>(n_here - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const float* base = a.part + (slot * a.n_split + first) * (COLS * (kD + 2));
    const int64_t stride = static_cast<int64_t>(COLS) * (kD + 2);
    // four elements of one column per thread
    for (int i = threadIdx.x; i < COLS * kD / 4; i += kAttWarps * 32) {
      const int col = i / (kD / 4), e = i % (kD / 4) * 4, r = row0 + col;
      if (r >= rows) continue;
      float m = -INFINITY;
      for (int k = 0; k < n_here; ++k) m = fmaxf(m, __ldcg(base + k * stride + COLS * kD + 2 * col));
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < n_here; ++k) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(base + k * stride + COLS * kD + 2 * col));
        const float4 v = __ldcg(reinterpret_cast<const float4*>(base + k * stride + col * kD + e));
        const float f = exp2_approx(ml.x - ref);
        l = fmaf(ml.y, f, l);
        y[0] = fmaf(v.x, f, y[0]); y[1] = fmaf(v.y, f, y[1]);
        y[2] = fmaf(v.z, f, y[2]); y[3] = fmaf(v.w, f, y[3]);
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(y[0] * inv, y[1] * inv);
      const __nv_bfloat162 b1 = __floats2bfloat162_rn(y[2] * inv, y[3] * inv);
      uint2 w;
      w.x = *reinterpret_cast<const uint32_t*>(&b0);
      w.y = *reinterpret_cast<const uint32_t*>(&b1);
      *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(sv.q0 + r / G) * a.out_stride +
                                (h * G + r % G) * kD + e) = w;
    }
    return;
  }
  if (warp == 0) {
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = row0 + n * 8 + 2 * t + c;
        if (r >= rows) continue;
        const float inv = l_all[n][c] == 0.f ? 0.f : 1.0f / l_all[n][c];
        __nv_bfloat16* dst = a.out + static_cast<int64_t>(sv.q0 + r / G) * a.out_stride +
                             (h * G + r % G) * kD + g * VB;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          *reinterpret_cast<__nv_bfloat162*>(dst + 2 * j) =
              __floats2bfloat162_rn(o[n][j][c] * inv, o[n][j][2 + c] * inv);
      }
  }
}

// Rows of a sequence and K/V head up to which its cache is streamed through this kernel; more go to
// the tensor-core kernel.
constexpr int kAttStreamRows = 16;

AttnPlan attn_plan(const strata_kv_cache& c, const strata_kv_batch& b, int n_heads) {
  AttnPlan p{};
  const int64_t G = n_heads / c.n_kv_heads, most_rows = b.max_q * G;
  if (most_rows > kAttStreamRows) {
    p.tc_blocks = static_cast<int>((most_rows + 255) / 256);
    // sequences of equal length: none is below the limit
    if (b.T == static_cast<int64_t>(b.n_seq) * b.max_q) return p;
    p.stream_rows = kAttStreamRows;
  } else {
    p.stream_rows = 0x7FFFFFFF;
  }
  const int64_t rows = std::min<int64_t>(most_rows, kAttStreamRows);
  p.nt = rows <= 8 ? 1 : 2;
  p.row_blocks = static_cast<int>((rows + 8 * p.nt - 1) / (8 * p.nt));
  // enough blocks for four on each of 152 SMs, but no split shorter than 256 tokens
  const int64_t blocks = std::max<int64_t>(1, static_cast<int64_t>(p.row_blocks) * c.n_kv_heads * b.n_seq);
  const int64_t unit = kAttWarps * kAttStep;
  const int64_t most = std::max<int64_t>(1, (b.max_kv + unit - 1) / unit);
  const int64_t want = std::min(most, (4 * 152 + blocks - 1) / blocks);
  const int64_t per = (most + want - 1) / want;
  p.split_tokens = static_cast<int>(per * unit);
  p.n_split = static_cast<int>((most + per - 1) / per);
  if (p.n_split > 1) {
    p.n_counters = static_cast<size_t>(blocks);
    p.part_floats = static_cast<size_t>(blocks) * p.n_split * (8 * p.nt) * (c.head_dim + 2);
  }
  return p;
}

template <int kD, int kNT>
static cudaError_t launch_attention_t(const AttnArgs& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(float) * (2 * kAttWarps * 8 * kNT + kAttWarps / 2 * 32 * kNT * (kD / 16) * 4);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(attention_kernel<kD, kNT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(a.n_split * a.row_blocks), a.c.n_kv_heads, a.b.n_seq);
  return launch_kernel(attention_kernel<kD, kNT>, grid, dim3(kAttWarps * 32), smem, stream, true, a);
}

cudaError_t launch_attention(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream) {
  if (a.c.head_dim == 64)
    return p.nt == 1 ? launch_attention_t<64, 1>(a, stream) : launch_attention_t<64, 2>(a, stream);
  return p.nt == 1 ? launch_attention_t<128, 1>(a, stream) : launch_attention_t<128, 2>(a, stream);
}

}  // namespace strata
