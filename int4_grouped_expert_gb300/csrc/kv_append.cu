// Rotation of q and k by position and the append of k and v to a paged cache of e4m3 codes with one
// power-of-two scale per (page, head).
//
// A run is a stretch of rows with consecutive slots in one page, found from the slots alone; one block owns a
// run of one K/V head, so the scale of a (page, head) has one writer and needs no atomics. A row whose position
// is out of range is a hole in its run: not stored, and no part of the scale. The block holds the run's rows in
// registers as they came, finds the largest magnitude of the rotated rows, settles the new scale with
// the page's old one, rewrites the older codes if the scale grew, rotates again and writes the codes:
// the rotation is elementwise in fp32 with each product and sum rounded once, so both times give the
// same values. The call moves each byte of q, k and v once and is bound by memory for prompts, by the
// chain slot -> position -> table row -> codes for single tokens. Measured: 10798 tokens of 56 query and 8
// K/V heads of 128 68 us, 5.6 TB/s; 16 single tokens 4.1 us. Pages of 16 tokens leave most of a block idle: 2 prompts of
// up to 2184 tokens, 8 heads of 64, 21 us, 1.5 TB/s.
//
// A thread takes two chunks of 8 elements of a head's row that the rotation keeps to themselves: chunks c
// and c + rot / 16 where halves are paired, neighbouring chunks elsewhere; with them it needs 8 cosines
// and 8 sines, which serve all heads of a row that it takes.
#include "block.cuh"

namespace strata {

constexpr int kAppThreads = 256;
constexpr int kAppHeads = 8;  // query heads that a block takes at a time

// Two values as e4m3 codes (lo in the low byte), rounded to nearest-even. |x| <= 448 by the choice of
// the scale; larger ones (a scale that an earlier writer chose) saturate.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two e4m3 codes (low byte first) as f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(v)));
  return d;
}

// 2^e, e the smallest integer >= -100 with absmax <= 448 * 2^e (absmax finite, >= 0): 448 is
// 1.75 * 2^8, so e is the exponent less 8, one more where the mantissa is above 1.75.
__device__ __forceinline__ float append_scale(float absmax) {
  const uint32_t b = __float_as_uint(absmax);
  int e = static_cast<int>(b >> 23) - 127 - 8;
  if ((b & 0x7FFFFFu) > 0x600000u) ++e;
  return exp2i(max(e, -100));
}

// Two chunks of a row: their places, and how they turn.
struct Pair {
  int a, b;    // chunk indices
  int kind;    // 0: not rotated, 1: halves (a with b), 2: neighbours (within a, within b)
  int at;      // first of their 8 cosines in the table row
};
__device__ __forceinline__ Pair pair_of(int p, int rot, int neighbours) {
  const int turned = rot >> 4;  // pairs that are rotated
  if (p >= turned) return {2 * p, 2 * p + 1, 0, 0};
  if (neighbours) return {2 * p, 2 * p + 1, 2, 8 * p};
  return {p, p + turned, 1, 8 * p};
}
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ Turn turn_at(const KvAppendArgs& a, const Pair& p, int64_t position) {
  Turn t = {};
  if (p.kind == 0) return t;
  const float* cs = a.rope + position * a.rot_dim + p.at;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 c = *reinterpret_cast<const float4*>(cs + 4 * q);
    const float4 s = *reinterpret_cast<const float4*>(cs + (a.rot_dim >> 1) + 4 * q);
    t.c[4 * q] = c.x; t.c[4 * q + 1] = c.y; t.c[4 * q + 2] = c.z; t.c[4 * q + 3] = c.w;
    t.s[4 * q] = s.x; t.s[4 * q + 1] = s.y; t.s[4 * q + 2] = s.z; t.s[4 * q + 3] = s.w;
  }
  return t;
}
__device__ __forceinline__ Turn turn_of(const KvAppendArgs& a, const Pair& p, int row) {
  return turn_at(a, p, p.kind == 0 ? 0 : a.positions[row]);
}
__device__ __forceinline__ void to_f32(const uint4& w, float* x) {
  x[0] = bf16_lo_f32(w.x); x[1] = bf16_hi_f32(w.x); x[2] = bf16_lo_f32(w.y); x[3] = bf16_hi_f32(w.y);
  x[4] = bf16_lo_f32(w.z); x[5] = bf16_hi_f32(w.z); x[6] = bf16_lo_f32(w.w); x[7] = bf16_hi_f32(w.w);
}
// The 16 elements of a pair of chunks, rotated: fp32, every product and sum rounded once.
__device__ __forceinline__ void rotated(const uint4& wa, const uint4& wb, const Pair& p, const Turn& t, float (&y)[16]) {
  to_f32(wa, y);
  to_f32(wb, y + 8);
  if (p.kind == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = y[i], v = y[8 + i];
      y[i] = __fsub_rn(__fmul_rn(u, t.c[i]), __fmul_rn(v, t.s[i]));
      y[8 + i] = __fadd_rn(__fmul_rn(v, t.c[i]), __fmul_rn(u, t.s[i]));
    }
  } else if (p.kind == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = y[2 * i], v = y[2 * i + 1];
      y[2 * i] = __fsub_rn(__fmul_rn(u, t.c[i]), __fmul_rn(v, t.s[i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(v, t.c[i]), __fmul_rn(u, t.s[i]));
    }
  }
}

__device__ __forceinline__ bool finite16(const float (&y)[16]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) ok = ok && (__float_as_uint(y[i]) & 0x7F800000u) != 0x7F800000u;
  return ok;
}
__device__ __forceinline__ float max16(const float (&y)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}
__device__ __forceinline__ uint2 codes8(const float* y, float inv) {
  uint2 d;
  d.x = f32x2_to_e4m3x2(y[0] * inv, y[1] * inv) | f32x2_to_e4m3x2(y[2] * inv, y[3] * inv) << 16;
  d.y = f32x2_to_e4m3x2(y[4] * inv, y[5] * inv) | f32x2_to_e4m3x2(y[6] * inv, y[7] * inv) << 16;
  return d;
}

__device__ __forceinline__ bool in_cache(const KvAppendArgs& a, int slot) {
  return slot >= 0 && slot < a.c.n_pages * a.c.page_size;
}
__device__ __forceinline__ bool in_table(const KvAppendArgs& a, int position) {
  return position >= 0 && position < a.n_pos;
}
// 0: padding, 1: good, 2: out of range
__device__ __forceinline__ int row_state(const KvAppendArgs& a, int r) {
  const int s = a.slots[r];
  if (s < 0) return 0;
  return in_cache(a, s) && (a.rot_dim == 0 || in_table(a, a.positions[r])) ? 1 : 2;
}
// Row r, whose slot is in the cache, continues the run that row r - 1 is in, whether that one is stored or not.
__device__ __forceinline__ bool continues(const KvAppendArgs& a, int r) {
  const int s = a.slots[r];
  return r > 0 && s % a.c.page_size != 0 && a.slots[r - 1] == s - 1;
}

// The older codes of a (page, head) times old / now, when the scale grew.
__device__ __forceinline__ void rescale(uint8_t* codes, int bytes, float ratio) {
  for (int i = threadIdx.x * 16; i < bytes; i += kAppThreads * 16) {
    uint4 v = *reinterpret_cast<uint4*>(codes + i);
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = e4m3x2_to_f16x2(w[j]), hi = e4m3x2_to_f16x2(w[j] >> 16);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      w[j] = f32x2_to_e4m3x2(a.x * ratio, a.y * ratio) | f32x2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
    }
    *reinterpret_cast<uint4*>(codes + i) = v;
  }
}

// kIter: iterations that a page of rows takes.
template <int kD, int kIter>
__device__ __forceinline__ void append_run(const KvAppendArgs& a, int row0, int head) {
  constexpr int TPR = kD / 16;              // threads per row
  constexpr int RPI = kAppThreads / TPR;    // rows per iteration
  constexpr int WARPS = kAppThreads / 32;
  __shared__ int s_len[WARPS];
  __shared__ unsigned s_holes[WARPS];
  __shared__ float s_max[2][WARPS];
  const int P = a.c.page_size;
  const int slot = a.slots[row0], off = slot % P;
  const int64_t page = slot / P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the rows that may be the run's, on their way while its length is found
  const Pair kp = pair_of(threadIdx.x % TPR, a.rot_dim, a.neighbours);
  const Pair vp = {kp.a, kp.b, 0, 0};
  const int ri = threadIdx.x / TPR;
  const Turn none = {};
  uint4 kw[kIter][2], vw[kIter][2];
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int64_t r = row0 + j * RPI + ri;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const bool on = off + j * RPI + ri < P && r < a.T;
    const uint4* k = reinterpret_cast<const uint4*>(a.k + r * a.k_stride + head * kD);
    const uint4* v = reinterpret_cast<const uint4*>(a.v + r * a.v_stride + head * kD);
    kw[j][0] = on ? k[kp.a] : z;
    kw[j][1] = on ? k[kp.b] : z;
    vw[j][0] = on ? v[kp.a] : z;
    vw[j][1] = on ? v[kp.b] : z;
  }
  // its first row's cosines (a row with a position out of range is not stored: any table row will do) and the
  // page's scales as well
  Turn t_first = none;
  if (a.rot_dim > 0) {
    const int r = min(row0 + ri, a.T - 1);
    t_first = turn_at(a, kp, min(static_cast<int64_t>(max(a.positions[r], 0)), a.n_pos - 1));
  }
  const int64_t ph = page * a.c.n_kv_heads + head;
  const float k_old = off ? a.c.k_scales[ph] : 0.f, v_old = off ? a.c.v_scales[ph] : 0.f;
  // the run's length: the first row that does not continue it (P <= kAppThreads); and its holes
  {
    const int i = threadIdx.x, r = row0 + i;
    const bool in = off + i < P && r < a.T && a.slots[r] == slot + i;
    const unsigned out = __ballot_sync(0xffffffffu, !in);
    const unsigned holes = __ballot_sync(0xffffffffu, in && row_state(a, r) != 1);
    if (lane == 0) {
      s_len[warp] = out ? 32 * warp + __ffs(out) - 1 : kAppThreads;
      s_holes[warp] = holes;
    }
  }
  __syncthreads();
  constexpr int WORDS = kIter * RPI / 32;  // (a page has at most kIter * RPI rows)
  int n = kIter * RPI;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) n = min(n, s_len[w]);

  bool any = false;  // of n rows, one that is no hole
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
    if (32 * w < n) any |= (~s_holes[w] & (0xffffffffu >> max(0, 32 * w + 32 - n))) != 0;
  if (!any) {  // nothing changes
    __syncthreads();
    return;
  }
  unsigned skipped = 0;  // bit j: this thread's row of iteration j is past the run, or a hole in it
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int i = j * RPI + ri;
    if (i < n && !(s_holes[i >> 5] >> (i & 31) & 1u)) continue;
    skipped |= 1u << j;
    kw[j][0] = kw[j][1] = vw[j][0] = vw[j][1] = make_uint4(0u, 0u, 0u, 0u);
  }
  // a row is good when all its threads hold finite values
  auto good_row = [&](const float (&k)[16], const float (&v)[16]) {
    const unsigned bad = __ballot_sync(0xffffffffu, !(finite16(k) && finite16(v)));
    return ((bad >> (lane / TPR * TPR)) & ((1u << TPR) - 1u)) == 0;
  };
  float km = 0.f, vm = 0.f;
  unsigned bad_rows = 0;  // bit j: this thread's row of iteration j
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    if (j * RPI >= n) break;
    float k[16], v[16];
    const int i = j * RPI + ri;
    rotated(kw[j][0], kw[j][1], kp, j == 0 ? t_first : skipped >> j & 1u ? none : turn_of(a, kp, row0 + i), k);
    rotated(vw[j][0], vw[j][1], vp, none, v);
    if (good_row(k, v)) {
      km = fmaxf(km, max16(k));
      vm = fmaxf(vm, max16(v));
    } else if (!(skipped >> j & 1u)) {
      bad_rows |= 1u << j;
    }
  }
  km = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(km)));  // >= 0: bits order
  vm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vm)));
  if (lane == 0) {
    s_max[0][warp] = km;
    s_max[1][warp] = vm;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    km = fmaxf(km, s_max[0][w]);
    vm = fmaxf(vm, s_max[1][w]);
  }
  uint8_t* kc = a.c.k_codes + ph * P * kD;
  uint8_t* vc = a.c.v_codes + ph * P * kD;
  float ks = append_scale(km), vs = append_scale(vm);
  if (off) {
    if (ks > k_old) rescale(kc, off * kD, __fdiv_rn(k_old, ks)); else ks = k_old;
    if (vs > v_old) rescale(vc, off * kD, __fdiv_rn(v_old, vs)); else vs = v_old;
  }
  const float ki = __fdiv_rn(1.0f, ks), vi = __fdiv_rn(1.0f, vs);
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int i = j * RPI + ri;
    if (i >= n) break;
    if (skipped >> j & 1u) continue;
    float k[16], v[16];
    rotated(kw[j][0], kw[j][1], kp, j == 0 ? t_first : turn_of(a, kp, row0 + i), k);
    rotated(vw[j][0], vw[j][1], vp, none, v);
    const bool ok = !(bad_rows >> j & 1u);
    const uint2 nan8 = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), zero = make_uint2(0u, 0u);
    uint2* kd = reinterpret_cast<uint2*>(kc + static_cast<int64_t>(off + i) * kD);
    uint2* vd = reinterpret_cast<uint2*>(vc + static_cast<int64_t>(off + i) * kD);
    kd[kp.a] = ok ? codes8(k, ki) : nan8;
    kd[kp.b] = ok ? codes8(k + 8, ki) : nan8;
    vd[kp.a] = ok ? codes8(v, vi) : zero;
    vd[kp.b] = ok ? codes8(v + 8, vi) : zero;
  }
  __syncthreads();  // every thread has read the old scales (and the shared words, for the next run)
  if (threadIdx.x == 0) {
    a.c.k_scales[ph] = ks;
    a.c.v_scales[ph] = vs;
  }
  if (__any_sync(0xffffffffu, bad_rows != 0) && lane == 0) set_status(a.status, STRATA_DEV_NONFINITE);
}

// Queries: a block takes kAppThreads / (kD / 16 * kAppHeads) rows; a thread one pair of chunks of every
// kAppHeads-th head of a row.
template <int kD>
__device__ __forceinline__ void rotate_queries(const KvAppendArgs& a, int block) {
  constexpr int TPR = kD / 16, ROWS = kAppThreads / (TPR * kAppHeads);
  const int r = block * ROWS + threadIdx.x / (TPR * kAppHeads);
  if (r >= a.T || row_state(a, r) != 1) return;
  const Pair p = pair_of(threadIdx.x % TPR, a.rot_dim, a.neighbours);
  const Turn t = turn_of(a, p, r);
  const __nv_bfloat16* src = a.q + r * a.q_stride;
  __nv_bfloat16* dst = a.q_out + r * a.q_out_stride;
  constexpr int U = 4;  // heads on their way
  for (int h0 = threadIdx.x / TPR % kAppHeads; h0 < a.n_heads; h0 += U * kAppHeads) {
    uint4 wa[U], wb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * kAppHeads;
      if (h >= a.n_heads) break;
      wa[i] = reinterpret_cast<const uint4*>(src + h * kD)[p.a];
      wb[i] = reinterpret_cast<const uint4*>(src + h * kD)[p.b];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * kAppHeads;
      if (h >= a.n_heads) break;
      float y[16];
      rotated(wa[i], wb[i], p, t, y);
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
      // (q_out may be q: nobody else reads these chunks)
      reinterpret_cast<uint4*>(dst + h * kD)[p.a] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(dst + h * kD)[p.b] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <int kD, int kIter>
__global__ void __launch_bounds__(kAppThreads, kIter > 2 ? 1 : 3) kv_append_kernel(KvAppendArgs a, int kv_blocks) {
  griddep_wait();
  griddep_launch();
  if (blockIdx.x >= static_cast<unsigned>(kv_blocks)) {
    rotate_queries<kD>(a, blockIdx.x - kv_blocks);
    return;
  }
  const int head = blockIdx.x % a.c.n_kv_heads;
  const int lo = blockIdx.x / a.c.n_kv_heads * a.rows_per_block;  // rows_per_block <= kAppThreads
  const int r = lo + threadIdx.x;
  const int st = threadIdx.x < a.rows_per_block && r < a.T ? row_state(a, r) : 0;
  if (st == 2) set_status(a.status, STRATA_DEV_BAD_SLOT);
  __shared__ unsigned s_starts[kAppThreads / 32];
  const unsigned starts = __ballot_sync(0xffffffffu, st != 0 && in_cache(a, a.slots[r]) && !continues(a, r));
  if ((threadIdx.x & 31) == 0) s_starts[threadIdx.x >> 5] = starts;
  __syncthreads();
  for (int w = 0; w < kAppThreads / 32; ++w)
    for (unsigned m = s_starts[w]; m; m &= m - 1) append_run<kD, kIter>(a, lo + 32 * w + __ffs(m) - 1, head);
}

cudaError_t launch_kv_append(const KvAppendArgs& a0, int num_sms, cudaStream_t stream) {
  KvAppendArgs a = a0;
  const int D = a.c.head_dim, P = a.c.page_size;
  // Rows whose runs a block starts: single tokens are a run each, prompts one per page, so as few as keep the
  // blocks at about four per SM, and at most a page. (us, one row / this share / a page: 16 single tokens
  // 4.5 / 4.4 / 31.7, prompts of 10798 tokens 336 / 68 / 68, 512 tokens 16.4 / 7.6 / 7.7.)
  const int64_t share = (static_cast<int64_t>(a.T) * a.c.n_kv_heads + 4 * num_sms - 1) / (4 * num_sms);
  a.rows_per_block = static_cast<int>(share < P ? share : P);
  const int64_t kv_blocks = static_cast<int64_t>((a.T + a.rows_per_block - 1) / a.rows_per_block) * a.c.n_kv_heads;
  const int q_rows = kAppThreads / (D / 16 * kAppHeads);
  const int64_t grid = kv_blocks + (a.q ? (a.T + q_rows - 1) / q_rows : 0);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kern = D == 64 ? (P <= 64 ? kv_append_kernel<64, 1> : kv_append_kernel<64, 2>)
                      : (P <= 32   ? kv_append_kernel<128, 1>
                         : P <= 64 ? kv_append_kernel<128, 2>
                                   : kv_append_kernel<128, 4>);
  return launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(kAppThreads), 0, stream, true, a,
                       static_cast<int>(kv_blocks));
}

}  // namespace strata
