// Launchers and argument blocks of the attention half of a decoder block: quantized projections, the
// paged 8-bit cache and attention over it.
#pragma once

#include "common.cuh"

namespace strata {

// Up to this many tokens a projection streams its codes through registers (linear.cu), whatever its size
// (us, streamed / tcgen05, 32 tokens at 4 bits: 4096 -> 6144 12.7 / 14.8, 7168 -> 9216 22.1 / 21.9,
// 1024 -> 1024 3.2 / 6.7); beyond that linear_streams() weighs.
constexpr int kLinearStreamT = 32;
// Up to this many tcgen05 multiplies x with the integer codes (linear_tc.cu); more tokens take f16 operands
// (us, integers / f16, 4 bits: 33 tokens 4096 -> 6144 15.1 / 16.0, 1024 -> 1024 6.7 / 8.9; 64 tokens 7168 ->
// 9216 23.2 / 25.2; 128 tokens 4096 -> 6144 24 / 18.5).
constexpr int kLinearMidT = STRATA_LINEAR_EXACT_T;

// The power of two that a row of f16 operands is divided by, for its largest bf16 magnitude (key as
// bf16x8_mag): it brings the row's largest entry to [8, 16), so that rows of any size keep their
// precision (entries below 2^-17 of the largest begin to lose bits). A row of zeros takes 0.
__device__ __forceinline__ int row_exp(uint32_t mag_key) {
  return mag_key == 0 ? 0 : min(max(static_cast<int>(mag_key >> 7) - 127 - 3, -120), 120);
}

struct LinearArgs {
  const uint8_t* codes;   // [N, K/2] or [N, K]
  const __half* scales;   // [N, K/group]
  const float* bias;      // [N] or null
  const __nv_bfloat16* x; // [T, K], x_stride elements from row to row
  const __nv_bfloat16* residual;  // [T, N] or null
  __nv_bfloat16* out;     // [T, N]
  int64_t x_stride, residual_stride, out_stride;
  int64_t T;
  int N, K, group, bits;
  uint32_t* status;
  // many tokens (linear_tc.cu): scratch for the f16 copy of x [T, K] and the exponents of its rows
  __half* xh;
  int* xexp;
};
bool linear_streams(int64_t T, int64_t K, int64_t N);
cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t stream);
cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t stream);

struct KvAppendArgs {
  strata_kv_cache c;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int32_t *slots, *positions;
  const float* rope;
  int64_t n_pos;
  int T, n_heads, rot_dim, neighbours;
  int rows_per_block;     // rows whose runs one K/V block starts
  uint32_t* status;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, int num_sms, cudaStream_t stream);

// Slots of the attention workspace that have counters: the counters lie in the same place for every
// batch, so that a workspace can go from one to another without being cleared.
constexpr int kAttMaxSlots = 3648;

struct AttnArgs {
  strata_kv_cache c;
  strata_kv_batch b;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_stride, out_stride;
  int n_heads, group;     // query heads; query heads per K/V head
  float scale_log2;       // softmax scale * log2(e)
  int window;             // 0: none
  int rows_above;         // attention.cu takes the sequences with at most so many rows per K/V head,
  int rows_below;         // attention_tc.cu those with more
  // attention.cu
  bool beside;            // launched after attention_tc.cu's kernel, to run beside it
  float* part;            // partial results, a slot per piece of a cut (sequence, K/V head)
  uint32_t* counters;     // [2][kAttMaxSlots], zero between calls
  // attention_tc.cu
  int tc_rows;            // rows of a block at most: 256, or 128 (attention_tc_join_kernel: 256)
  bool tc_search;         // blocks find their units in the lengths
  int tc_slots;           // pieces that may be left in the workspace; 0: nothing is cut
  float* tc_part;
  uint32_t* status;
};
// How one attention call is laid out: chosen on the host from the limits the caller gives.
struct AttnPlan {
  int nt;                 // attention.cu: 8-row tiles of query rows per block, 1 or 2
  bool solo;              // attention.cu: shares for warps instead of pieces for blocks
  int64_t grid;
  size_t part_floats, tc_part_floats;
  int stream_rows;        // rows up to which a sequence goes to attention.cu: 0 none, INT_MAX all
  bool tc;                // attention_tc.cu is launched
  int tc_slots;           // its pieces in the workspace at most
};
AttnPlan attn_plan(const strata_kv_cache& c, const strata_kv_batch& b, int n_heads);
cudaError_t launch_attention(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream);
int attn_tc_slots(const strata_kv_cache& c, const strata_kv_batch& b, int64_t group, int window);
size_t attn_tc_part_floats(const strata_kv_cache& c, int slots);
cudaError_t launch_attention_tc(AttnArgs a, cudaStream_t stream);
cudaError_t launch_attention_tc_join(AttnArgs a, cudaStream_t stream);  // after both others

}  // namespace strata
