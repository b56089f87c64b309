// Device helpers shared by the attention kernels.
#pragma once

#include "block.cuh"

namespace strata {

// Two e4m3 codes (low byte first) as f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(v)));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// How both kernels use a page's scales: the K scale multiplies the scores, in fp32, and the V scale goes into the
// exponent, so that a token's weight in the product with the V codes (exact in f16) is
//   w = 2^(score + log2(V scale) - ref),   ref a running reference of these exponents, per row,
// rounded to f16: 2^-11 of itself, or 2^-25 of the row's largest once it is below 2^-14 of that. The sum of the softmax
// takes w / V scale in fp32 and has the same reference, so output = (sum of w code) / (sum of w / V scale). A page
// that a row does not see, or whose tokens weigh little, changes nothing for the others, however large its scales are.
// Scales are positive; V scales below 2^-100, the least that the append writes, count as 2^-100.
__device__ __forceinline__ float log2_scale(float s) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s < 7.88860905e-31f ? 7.88860905e-31f : s));
  return y;
}
// Where log2(V scale) is this far below the largest met so far, w may be flushed to zero (2^-126) though its part in the
// sum is not negligible: there the sum takes 2^(score - ref) instead. (Pages of zeros have such scales. Nearer ones are
// flushed for weights below 2^-40 of the largest.)
constexpr float kFarScale = 78.f;
// A sum of the softmax times 2^d: to a reference that is -d above its own. Between pages of zeros and of large values
// that is more than the 2^-126 that one factor reaches, and such a sum is large (w / V scale).
__device__ __forceinline__ float sum_times_exp2(float sum, float d) {
  const float a = fmaxf(d, -100.f);
  return sum * exp2_approx(a) * exp2_approx(d - a);
}

// The rows and tokens of one sequence, cut to the call's limits.
struct SeqView {
  int q0, n;  // first row, rows
  int len;    // tokens in the cache
};
// A load of the call's inputs. A kernel that runs beside another of its call has not waited for the kernels
// before, whose results are in L2 by then: it does not look in L1.
template <class T>
__device__ __forceinline__ T input(const AttnArgs& a, const T* p) {
  return a.beside ? __ldcg(p) : *p;
}
__device__ __forceinline__ SeqView seq_view(const AttnArgs& a, int s, bool flag) {
  SeqView v;
  int q0 = input(a, a.b.q_start + s), q1 = input(a, a.b.q_start + s + 1), len = input(a, a.b.kv_len + s);
  const int T = static_cast<int>(a.b.T);
  bool bad = q0 < 0 || q1 < q0 || q1 > T || len < 0 || len > a.b.max_kv;
  q0 = min(max(q0, 0), T);
  q1 = min(max(q1, q0), T);
  bad |= q1 - q0 > a.b.max_q;
  v.q0 = q0;
  v.n = min(q1 - q0, a.b.max_q);
  v.len = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), a.b.max_kv));
  if (bad && flag) set_status(a.status, STRATA_DEV_BAD_SLOT);
  return v;
}
// First token that a row of the sequence sees whose first row stands at position p (below 0: before the first
// token). No step of it leaves 32 bits, whatever the window.
__device__ __forceinline__ int first_seen(const AttnArgs& a, int p) {
  return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

}  // namespace strata
