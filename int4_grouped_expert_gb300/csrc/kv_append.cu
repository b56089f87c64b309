// Rotation of q and k by position and the append of k and v to a paged cache of e4m3 codes with one
// power-of-two scale per (page, head).
//
// A run is a stretch of rows with consecutive slots in one page; one block owns a run of one K/V head,
// so the scale of a (page, head) has one writer and needs no atomics. The block finds the largest
// magnitude of the run (pass 1), settles the new scale with the page's old one, rewrites the older
// codes if the scale grew, and writes the codes (pass 2, from L1/L2). The rotation is elementwise
// in fp32 with each product and sum rounded once, so both passes see the same values. The call moves
// each byte of q, k and v once: it is bound by memory for prompts and by latency for single tokens.
#include "block.cuh"

namespace strata {

constexpr int kAppThreads = 128;

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

// Elements 8c .. 8c+7 of one head's row, rotated: fp32, every product and sum rounded once.
__device__ __forceinline__ void rotated8(const __nv_bfloat16* row, int c, const float* cs, int rot,
                                         int neighbours, float (&y)[8]) {
  const uint4 w = *(reinterpret_cast<const uint4*>(row) + c);
  float x[8] = {bf16_lo_f32(w.x), bf16_hi_f32(w.x), bf16_lo_f32(w.y), bf16_hi_f32(w.y),
                bf16_lo_f32(w.z), bf16_hi_f32(w.z), bf16_lo_f32(w.w), bf16_hi_f32(w.w)};
  const int i0 = 8 * c, h = rot >> 1;
  if (i0 >= rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  } else if (neighbours) {
    const float4 co = *reinterpret_cast<const float4*>(cs + i0 / 2);
    const float4 si = *reinterpret_cast<const float4*>(cs + h + i0 / 2);
    const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], cc[i]), __fmul_rn(x[2 * i + 1], ss[i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], cc[i]), __fmul_rn(x[2 * i], ss[i]));
    }
  } else {
    const bool first = i0 < h;  // rot % 16 == 0: a chunk lies in one half
    const int f = first ? i0 : i0 - h;
    const uint4 o = *(reinterpret_cast<const uint4*>(row) + (first ? i0 + h : f) / 8);
    const float z[8] = {bf16_lo_f32(o.x), bf16_hi_f32(o.x), bf16_lo_f32(o.y), bf16_hi_f32(o.y),
                        bf16_lo_f32(o.z), bf16_hi_f32(o.z), bf16_lo_f32(o.w), bf16_hi_f32(o.w)};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 co = *reinterpret_cast<const float4*>(cs + f + 4 * q);
      const float4 si = *reinterpret_cast<const float4*>(cs + h + f + 4 * q);
      const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * q + i;
        const float own = __fmul_rn(x[k], cc[i]), other = __fmul_rn(z[k], ss[i]);
        y[k] = first ? __fsub_rn(own, other) : __fadd_rn(own, other);
      }
    }
  }
}

__device__ __forceinline__ bool finite8(const float (&y)[8]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) ok = ok && (__float_as_uint(y[i]) & 0x7F800000u) != 0x7F800000u;
  return ok;
}
__device__ __forceinline__ float max8(const float (&y)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
  uint2 d;
  d.x = f32x2_to_e4m3x2(y[0] * inv, y[1] * inv) | f32x2_to_e4m3x2(y[2] * inv, y[3] * inv) << 16;
  d.y = f32x2_to_e4m3x2(y[4] * inv, y[5] * inv) | f32x2_to_e4m3x2(y[6] * inv, y[7] * inv) << 16;
  return d;
}

// 0: padding, 1: good, 2: out of range
__device__ __forceinline__ int row_state(const KvAppendArgs& a, int r) {
  const int s = a.slots[r];
  if (s < 0) return 0;
  if (s >= a.c.n_pages * a.c.page_size) return 2;
  if (a.rot_dim > 0) {
    const int p = a.positions[r];
    if (p < 0 || p >= a.n_pos) return 2;
  }
  return 1;
}
// Row r continues the run that row r - 1 is in.
__device__ __forceinline__ bool continues(const KvAppendArgs& a, int r) {
  if (r == 0 || row_state(a, r - 1) != 1) return false;
  const int s = a.slots[r];
  return s % a.c.page_size != 0 && s == a.slots[r - 1] + 1;
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

template <int kD>
__device__ __forceinline__ void append_run(const KvAppendArgs& a, int row0, int head) {
  constexpr int TPR = kD / 8;               // threads per row
  constexpr int RPI = kAppThreads / TPR;    // rows per iteration
  __shared__ int s_len[kAppThreads / 32];
  __shared__ float s_max[2][kAppThreads / 32];
  const int P = a.c.page_size;
  const int slot = a.slots[row0], off = slot % P;
  const int64_t page = slot / P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the run's length: the first row that does not continue it (P <= kAppThreads)
  {
    const int i = threadIdx.x, r = row0 + i;
    const bool in = off + i < P && r < a.T && a.slots[r] == slot + i && row_state(a, r) == 1;
    const unsigned out = __ballot_sync(0xffffffffu, !in);
    if (lane == 0) s_len[warp] = out ? 32 * warp + __ffs(out) - 1 : kAppThreads;
  }
  __syncthreads();
  int n = kAppThreads;
#pragma unroll
  for (int w = 0; w < kAppThreads / 32; ++w) n = min(n, s_len[w]);

  const int c = threadIdx.x % TPR, ri = threadIdx.x / TPR;
  const int rot = a.rot_dim;
  auto load = [&](int i, float (&k)[8], float (&v)[8]) {
    const int64_t r = row0 + i;
    const float* cs = rot ? a.rope + static_cast<int64_t>(a.positions[r]) * rot : nullptr;
    rotated8(a.k + r * a.k_stride + head * kD, c, cs, rot, a.neighbours, k);
    rotated8(a.v + r * a.v_stride + head * kD, c, nullptr, 0, 0, v);
  };
  // a row is good when all its threads hold finite values
  auto good_row = [&](const float (&k)[8], const float (&v)[8]) {
    const unsigned bad = __ballot_sync(0xffffffffu, !(finite8(k) && finite8(v)));
    return ((bad >> (lane / TPR * TPR)) & ((1u << TPR) - 1u)) == 0;
  };
  float km = 0.f, vm = 0.f;
  bool any_bad = false;
  for (int i0 = 0; i0 < n; i0 += RPI) {
    const int i = i0 + ri;
    float k[8] = {}, v[8] = {};
    if (i < n) load(i, k, v);
    const bool ok = good_row(k, v);
    any_bad |= !ok;
    if (ok) {
      km = fmaxf(km, max8(k));
      vm = fmaxf(vm, max8(v));
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
  for (int w = 0; w < kAppThreads / 32; ++w) {
    km = fmaxf(km, s_max[0][w]);
    vm = fmaxf(vm, s_max[1][w]);
  }
  const int64_t ph = page * a.c.n_kv_heads + head;
  uint8_t* kc = a.c.k_codes + ph * P * kD;
  uint8_t* vc = a.c.v_codes + ph * P * kD;
  float ks = append_scale(km), vs = append_scale(vm);
  if (off) {
    const float k_old = a.c.k_scales[ph], v_old = a.c.v_scales[ph];
    if (ks > k_old) rescale(kc, off * kD, __fdiv_rn(k_old, ks)); else ks = k_old;
    if (vs > v_old) rescale(vc, off * kD, __fdiv_rn(v_old, vs)); else vs = v_old;
  }
  const float ki = __fdiv_rn(1.0f, ks), vi = __fdiv_rn(1.0f, vs);
  for (int i0 = 0; i0 < n; i0 += RPI) {
    const int i = i0 + ri;
    float k[8] = {}, v[8] = {};
    if (i < n) load(i, k, v);
    const bool ok = good_row(k, v);
    if (i < n) {
      const int64_t at = static_cast<int64_t>(off + i) * kD + 8 * c;
      const uint32_t nan4 = 0x7F7F7F7Fu;
      *reinterpret_cast<uint2*>(kc + at) = ok ? codes8(k, ki) : make_uint2(nan4, nan4);
      *reinterpret_cast<uint2*>(vc + at) = ok ? codes8(v, vi) : make_uint2(0u, 0u);
    }
  }
  __syncthreads();  // every thread has read the old scales (and the shared words, for the next run)
  if (threadIdx.x == 0) {
    a.c.k_scales[ph] = ks;
    a.c.v_scales[ph] = vs;
  }
  if (__any_sync(0xffffffffu, any_bad) && lane == 0) set_status(a.status, STRATA_DEV_NONFINITE);
}

template <int kD>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(KvAppendArgs a, int kv_blocks) {
  griddep_wait();
  griddep_launch();
  if (blockIdx.x < static_cast<unsigned>(kv_blocks)) {
    const int head = blockIdx.x % a.c.n_kv_heads;
    const int lo = blockIdx.x / a.c.n_kv_heads * a.rows_per_block;  // rows_per_block <= kAppThreads
    const int r = lo + threadIdx.x;
    const int st = threadIdx.x < a.rows_per_block && r < a.T ? row_state(a, r) : 0;
    if (st == 2) set_status(a.status, STRATA_DEV_BAD_SLOT);
    __shared__ unsigned s_starts[kAppThreads / 32];
    const unsigned starts = __ballot_sync(0xffffffffu, st == 1 && !continues(a, r));
    if ((threadIdx.x & 31) == 0) s_starts[threadIdx.x >> 5] = starts;
    __syncthreads();
    for (int w = 0; w < kAppThreads / 32; ++w)
      for (unsigned m = s_starts[w]; m; m &= m - 1) append_run<kD>(a, lo + 32 * w + __ffs(m) - 1, head);
    return;
  }
  // queries: one thread per 8 elements
  const int64_t per_row = static_cast<int64_t>(a.n_heads) * (kD / 8);
  const int64_t i = static_cast<int64_t>(blockIdx.x - kv_blocks) * kAppThreads + threadIdx.x;
  const bool in = i < per_row * a.T;
  const int r = in ? static_cast<int>(i / per_row) : 0, j = in ? static_cast<int>(i % per_row) : 0;
  const bool on = in && row_state(a, r) == 1;
  float y[8] = {};
  if (on) {
    const int head = j / (kD / 8), c = j % (kD / 8);
    const float* cs = a.rot_dim ? a.rope + static_cast<int64_t>(a.positions[r]) * a.rot_dim : nullptr;
    rotated8(a.q + r * a.q_stride + head * kD, c, cs, a.rot_dim, a.neighbours, y);
  }
  __syncwarp();  // q_out may be q: a head's chunks are in one warp, all read before any is written
  if (on) {
    uint4 o;
    uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
      w[k] = *reinterpret_cast<uint32_t*>(&b);
    }
    *(reinterpret_cast<uint4*>(a.q_out + r * a.q_out_stride) + j) = o;
  }
}

cudaError_t launch_kv_append(const KvAppendArgs& a0, int num_sms, cudaStream_t stream) {
  KvAppendArgs a = a0;
  const int D = a.c.head_dim;
  // one row per block while that leaves the GPU room, a page of rows per block beyond
  a.rows_per_block = static_cast<int64_t>(a.T) * a.c.n_kv_heads <= 8 * num_sms ? 1 : a.c.page_size;
  const int64_t kv_blocks = static_cast<int64_t>((a.T + a.rows_per_block - 1) / a.rows_per_block) * a.c.n_kv_heads;
  const int64_t q_chunks = a.q ? static_cast<int64_t>(a.T) * a.n_heads * (D / 8) : 0;
  const int64_t grid = kv_blocks + (q_chunks + kAppThreads - 1) / kAppThreads;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_kernel(D == 64 ? kv_append_kernel<64> : kv_append_kernel<128>,
                       dim3(static_cast<unsigned>(grid)), dim3(kAppThreads), 0, stream, true, a,
                       static_cast<int>(kv_blocks));
}

}  // namespace strata
