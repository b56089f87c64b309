// The C ABI of the attention half of a decoder block (include/strata.h): argument checks, workspace
// layout and launches. Every check runs before the first CUDA call of an entry point; nothing here
// allocates, throws or keeps state.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "block.cuh"
#include "pages.cuh"

namespace strata {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr size_t kWsAlign = 256;

size_t round_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
strata_status of(cudaError_t e) { return e == cudaSuccess ? STRATA_OK : STRATA_ERR_CUDA; }
// SMs of the current device, looked up once per device (a property that does not change).
bool sm_count(int* out) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const bool keep = dev >= 0 && dev < 64;
  int n = keep ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
    if (keep) known[dev].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return true;
}

strata_status check_linear(const strata_linear* w) {
  if (!w) return STRATA_ERR_INVALID_ARG;
  const int G = w->group_size == 0 ? STRATA_GROUP : w->group_size;
  const int bits = w->bits == 0 ? 4 : w->bits;
  if (G != 64 && G != 128 && G != 256) return STRATA_ERR_UNSUPPORTED;
  if (bits != 4 && bits != 8) return STRATA_ERR_UNSUPPORTED;
  if (w->N < 1 || w->N > (int64_t(1) << 20) || w->K < 1 || w->K > (int64_t(1) << 16) || w->K % G)
    return STRATA_ERR_SHAPE;
  if (!w->codes || !w->scales || !on(w->codes, 16) || !on(w->scales, 2) || (w->bias && !on(w->bias, 4)))
    return STRATA_ERR_INVALID_ARG;
  return STRATA_OK;
}

struct LinearLayout {
  size_t xexp, xh, total;
};
LinearLayout linear_layout(const strata_linear* w, int64_t T) {
  LinearLayout L{};
  L.xexp = sizeof(WsHeader);
  const int64_t rows = T > kLinearMidT ? T : 0;
  L.xh = round_up(L.xexp + sizeof(int) * rows);
  L.total = round_up(L.xh + sizeof(uint16_t) * rows * w->K);
  return L;
}

strata_status check_cache(const strata_kv_cache* c) {
  if (!c) return STRATA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return STRATA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return STRATA_ERR_UNSUPPORTED;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 256) return STRATA_ERR_UNSUPPORTED;
  if (c->n_pages < 0 || c->n_pages > 0x7FFFFFFF / c->page_size) return STRATA_ERR_SHAPE;
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return STRATA_ERR_INVALID_ARG;
  if (!on(c->k_codes, 16) || !on(c->v_codes, 16) || !on(c->k_scales, 4) || !on(c->v_scales, 4))
    return STRATA_ERR_INVALID_ARG;
  return STRATA_OK;
}

// bf16 rows read or written 16 bytes at a time
bool rows_ok(const void* p, int64_t stride, int64_t len) {
  return p && on(p, 16) && stride >= len && stride % 8 == 0;
}

strata_status check_batch(const strata_kv_cache* c, const strata_kv_batch* b, int32_t n_heads) {
  const strata_status s = check_cache(c);
  if (s != STRATA_OK) return s;
  if (!b) return STRATA_ERR_INVALID_ARG;
  if (n_heads < 1 || n_heads > 1024 || n_heads % c->n_kv_heads) return STRATA_ERR_UNSUPPORTED;
  if (b->n_seq < 0 || b->n_seq > 65535 || b->T < 0 || b->T > kMaxRows || b->max_q < 0 ||
      b->max_q > kMaxRows || b->max_kv < 0 || b->max_kv > 0x7FFFFFFF - 4096)
    return STRATA_ERR_SHAPE;
  if (b->n_seq == 0 || b->T == 0) return STRATA_OK;
  if (b->max_q < 1) return STRATA_ERR_SHAPE;
  if ((b->max_kv / 32 + 1) * b->n_seq > 0x7FFFFFFF / c->n_kv_heads) return STRATA_ERR_SHAPE;
  if (b->table_stride < 0 || b->max_kv > b->table_stride * c->page_size) return STRATA_ERR_SHAPE;
  if (!b->q_start || !b->kv_len || (!b->page_table && b->max_kv > 0)) return STRATA_ERR_INVALID_ARG;
  if (!on(b->q_start, 4) || !on(b->kv_len, 4) || !on(b->page_table, 4)) return STRATA_ERR_INVALID_ARG;
  return STRATA_OK;
}

// Least eps of a norm: squares that fp32 flushes to zero are far below it.
constexpr float kMinEps = 7.88860905e-31f;  // 2^-100

strata_status check_norm(const strata_qk_norm& n, int head_dim) {
  if (!std::isfinite(n.eps) || n.eps < kMinEps) return STRATA_ERR_INVALID_ARG;
  const struct {
    const float* weight;
    int64_t stride;
  } of[2] = {{n.q_weight, n.q_head_stride}, {n.k_weight, n.k_head_stride}};
  for (const auto& x : of) {
    if (!x.weight) continue;
    if (!on(x.weight, 16) || x.stride % 4 || (x.stride != 0 && x.stride < head_dim)) return STRATA_ERR_INVALID_ARG;
  }
  return STRATA_OK;
}

strata_status append(const strata_kv_cache* cache, const strata_qk_norm* norm, const void* q_bf16, int64_t q_stride,
                     int32_t n_heads, const void* k_bf16, int64_t k_stride,
                     const void* v_bf16, int64_t v_stride, int64_t T,
                     const int32_t* slots, const int32_t* positions, const float* rope,
                     int64_t n_pos, int32_t rot_dim, uint32_t flags, void* q_out,
                     int64_t q_out_stride, uint32_t* dev_status, strata_stream stream) {
  const strata_status s = check_cache(cache);
  if (s != STRATA_OK) return s;
  if (flags & ~STRATA_ROPE_NEIGHBOURS) return STRATA_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxRows) return STRATA_ERR_SHAPE;
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16) return STRATA_ERR_SHAPE;
  const bool with_q = q_bf16 || q_out;
  if (with_q && (n_heads < 1 || n_heads > 1024)) return STRATA_ERR_UNSUPPORTED;
  if (norm) {
    const strata_status ns = check_norm(*norm, cache->head_dim);
    if (ns != STRATA_OK) return ns;
  }
  if (T == 0) return STRATA_OK;
  const int64_t kv_len = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
  const int64_t q_len = static_cast<int64_t>(n_heads) * cache->head_dim;
  if (!rows_ok(k_bf16, k_stride, kv_len) || !rows_ok(v_bf16, v_stride, kv_len)) return STRATA_ERR_INVALID_ARG;
  if (with_q && (!rows_ok(q_bf16, q_stride, q_len) || !rows_ok(q_out, q_out_stride, q_len)))
    return STRATA_ERR_INVALID_ARG;
  if (with_q && q_bf16 == q_out && q_stride != q_out_stride) return STRATA_ERR_INVALID_ARG;
  if (!slots || !on(slots, 4) || (dev_status && !on(dev_status, 4))) return STRATA_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!positions || !on(positions, 4) || !rope || !on(rope, 16) || n_pos < 1))
    return STRATA_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(&sms)) return STRATA_ERR_CUDA;
  KvAppendArgs a{};
  a.c = *cache;
  a.q = static_cast<const __nv_bfloat16*>(q_bf16);
  a.k = static_cast<const __nv_bfloat16*>(k_bf16);
  a.v = static_cast<const __nv_bfloat16*>(v_bf16);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.slots = slots;
  a.positions = positions;
  a.rope = rope;
  a.n_pos = n_pos;
  a.T = static_cast<int>(T);
  a.n_heads = n_heads;
  a.rot_dim = rot_dim;
  a.neighbours = (flags & STRATA_ROPE_NEIGHBOURS) != 0;
  a.status = dev_status;
  if (norm) {
    a.q_weight = norm->q_weight;
    a.k_weight = norm->k_weight;
    a.q_weight_stride = norm->q_head_stride;
    a.k_weight_stride = norm->k_head_stride;
    a.eps = norm->eps;
  }
  return of(launch_kv_append(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

strata_status check_pages(const strata_kv_pages* p) {
  if (!p) return STRATA_ERR_INVALID_ARG;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return STRATA_ERR_UNSUPPORTED;
  if (p->n_seq < 0 || p->n_seq > kPagesMostSeq || p->n_pages < 0 || p->n_pages > 0x7FFFFFFF / p->page_size ||
      p->max_pages < 0 || p->max_pages > 0x7FFFFFFF / p->page_size || p->table_stride < p->max_pages)
    return STRATA_ERR_SHAPE;
  if ((p->n_seq > 0 && (!p->kv_len || (p->max_pages > 0 && !p->page_table))) || (p->n_pages > 0 && !p->refs))
    return STRATA_ERR_INVALID_ARG;
  if (!on(p->page_table, 4) || !on(p->kv_len, 4) || !on(p->refs, 16)) return STRATA_ERR_INVALID_ARG;
  return STRATA_OK;
}
// A word or array that a call writes or reads
bool ints_ok(const void* p) { return p && on(p, 4); }

// Caches of one shape: heads, head_dim, page_size and n_pages as the first one's
strata_status check_caches(const strata_kv_cache* c, int n, int64_t heads, int dim, int page_size) {
  for (int i = 0; i < n; ++i) {
    const strata_status s = check_cache(c + i);
    if (s != STRATA_OK) return s;
    if (c[i].n_kv_heads != heads || c[i].head_dim != dim || c[i].page_size != page_size || c[i].n_pages != c[0].n_pages)
      return STRATA_ERR_SHAPE;
  }
  return STRATA_OK;
}

struct AttnLayout {
  size_t counters, part, tc_part, total;
};
AttnLayout attn_layout(const AttnPlan& p) {
  AttnLayout L{};
  L.counters = sizeof(WsHeader);
  L.part = round_up(L.counters + 2 * sizeof(uint32_t) * kAttMaxSlots);
  L.tc_part = round_up(L.part + sizeof(float) * p.part_floats);
  L.total = round_up(L.tc_part + sizeof(float) * p.tc_part_floats);
  return L;
}

}  // namespace
}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_linear_workspace_size(const strata_linear* w, int64_t T_max) {
  if (check_linear(w) != STRATA_OK || T_max < 0 || T_max > kMaxRows) return 0;
  return linear_layout(w, T_max).total;
}

strata_status strata_linear_forward(const strata_linear* w, const void* x_bf16, int64_t x_stride,
                                    int64_t T, const void* residual_bf16, int64_t residual_stride,
                                    void* out_bf16, int64_t out_stride, void* workspace,
                                    size_t ws_bytes, strata_stream stream) {
  const strata_status s = check_linear(w);
  if (s != STRATA_OK) return s;
  if (T < 0 || T > kMaxRows) return STRATA_ERR_SHAPE;
  if (T == 0) return STRATA_OK;
  if (!rows_ok(x_bf16, x_stride, w->K) || !out_bf16 || !on(out_bf16, 2) || out_stride < w->N)
    return STRATA_ERR_INVALID_ARG;
  if (residual_bf16 && (!on(residual_bf16, 2) || residual_stride < w->N)) return STRATA_ERR_INVALID_ARG;
  if (residual_bf16 == out_bf16 && residual_stride != out_stride) return STRATA_ERR_INVALID_ARG;
  if (out_bf16 == x_bf16) return STRATA_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(w, T);
  if (!workspace || !on(workspace, kWsAlign) || ws_bytes < L.total) return STRATA_ERR_WORKSPACE;
  LinearArgs a{};
  a.codes = w->codes;
  a.scales = static_cast<const __half*>(w->scales);
  a.bias = w->bias;
  a.x = static_cast<const __nv_bfloat16*>(x_bf16);
  a.residual = static_cast<const __nv_bfloat16*>(residual_bf16);
  a.out = static_cast<__nv_bfloat16*>(out_bf16);
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.out_stride = out_stride;
  a.T = T;
  a.N = static_cast<int>(w->N);
  a.K = static_cast<int>(w->K);
  a.group = w->group_size == 0 ? STRATA_GROUP : w->group_size;
  a.bits = w->bits == 0 ? 4 : w->bits;
  char* base = static_cast<char*>(workspace);
  a.status = &reinterpret_cast<WsHeader*>(base)->status;
  a.xexp = reinterpret_cast<int*>(base + L.xexp);
  a.xh = reinterpret_cast<__half*>(base + L.xh);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (linear_streams(T, w->K, w->N)) return of(launch_linear_stream(a, st));
  int sms = 0;
  if (!sm_count(&sms)) return STRATA_ERR_CUDA;
  return of(launch_linear_tc(a, sms, st));
}

strata_status strata_kv_append(const strata_kv_cache* cache, const void* q_bf16, int64_t q_stride,
                               int32_t n_heads, const void* k_bf16, int64_t k_stride,
                               const void* v_bf16, int64_t v_stride, int64_t T,
                               const int32_t* slots, const int32_t* positions, const float* rope,
                               int64_t n_pos, int32_t rot_dim, uint32_t flags, void* q_out,
                               int64_t q_out_stride, uint32_t* dev_status, strata_stream stream) {
  return append(cache, nullptr, q_bf16, q_stride, n_heads, k_bf16, k_stride, v_bf16, v_stride, T, slots, positions, rope,
                n_pos, rot_dim, flags, q_out, q_out_stride, dev_status, stream);
}

strata_status strata_kv_append_normed(const strata_kv_cache* cache, const strata_qk_norm* norm, const void* q_bf16,
                                      int64_t q_stride, int32_t n_heads, const void* k_bf16, int64_t k_stride,
                                      const void* v_bf16, int64_t v_stride, int64_t T, const int32_t* slots,
                                      const int32_t* positions, const float* rope, int64_t n_pos, int32_t rot_dim,
                                      uint32_t flags, void* q_out, int64_t q_out_stride, uint32_t* dev_status,
                                      strata_stream stream) {
  if (!norm) return STRATA_ERR_INVALID_ARG;
  return append(cache, norm, q_bf16, q_stride, n_heads, k_bf16, k_stride, v_bf16, v_stride, T, slots, positions, rope,
                n_pos, rot_dim, flags, q_out, q_out_stride, dev_status, stream);
}

size_t strata_attention_workspace_size(const strata_kv_cache* cache, const strata_kv_batch* batch,
                                       int32_t n_heads) {
  if (check_batch(cache, batch, n_heads) != STRATA_OK) return 0;
  if (batch->n_seq == 0 || batch->T == 0) return sizeof(WsHeader);
  return attn_layout(attn_plan(*cache, *batch, n_heads)).total;
}

strata_status strata_attention_forward(const strata_kv_cache* cache, const strata_kv_batch* batch,
                                       const void* q_bf16, int64_t q_stride, int32_t n_heads,
                                       float scale, int32_t window, uint32_t flags, void* out_bf16,
                                       int64_t out_stride, void* workspace, size_t ws_bytes,
                                       strata_stream stream) {
  return strata_attention_sinks_forward(cache, batch, q_bf16, q_stride, n_heads, scale, window, 0, flags, out_bf16,
                                        out_stride, workspace, ws_bytes, stream);
}

strata_status strata_attention_sinks_forward(const strata_kv_cache* cache, const strata_kv_batch* batch,
                                             const void* q_bf16, int64_t q_stride, int32_t n_heads, float scale,
                                             int32_t window, int32_t n_sinks, uint32_t flags, void* out_bf16,
                                             int64_t out_stride, void* workspace, size_t ws_bytes,
                                             strata_stream stream) {
  const strata_status s = check_batch(cache, batch, n_heads);
  if (s != STRATA_OK) return s;
  if (flags & ~STRATA_WS_REUSE) return STRATA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || window < 0 || n_sinks < 0) return STRATA_ERR_INVALID_ARG;
  if (batch->n_seq == 0 || batch->T == 0) return STRATA_OK;
  const int64_t q_len = static_cast<int64_t>(n_heads) * cache->head_dim;
  if (!rows_ok(q_bf16, q_stride, q_len) || !rows_ok(out_bf16, out_stride, q_len) || q_bf16 == out_bf16)
    return STRATA_ERR_INVALID_ARG;
  const AttnPlan p = attn_plan(*cache, *batch, n_heads);
  const AttnLayout L = attn_layout(p);
  if (!workspace || !on(workspace, kWsAlign) || ws_bytes < L.total) return STRATA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(workspace);
  if (!(flags & STRATA_WS_REUSE) &&
      cudaMemsetAsync(base, 0, L.part, st) != cudaSuccess)
    return STRATA_ERR_CUDA;
  AttnArgs a{};
  a.c = *cache;
  a.b = *batch;
  a.q = static_cast<const __nv_bfloat16*>(q_bf16);
  a.out = static_cast<__nv_bfloat16*>(out_bf16);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_heads = n_heads;
  a.group = n_heads / cache->n_kv_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  // (a window that no position reaches past, but for first tokens that stay visible, is none: below max_kv,
  // position - window stays in 32 bits)
  a.window = window < batch->max_kv - n_sinks ? window : 0;
  a.sinks = a.window > 0 ? n_sinks : 0;
  a.part = reinterpret_cast<float*>(base + L.part);
  a.counters = reinterpret_cast<uint32_t*>(base + L.counters);
  // (a window shortens what is seen, and so the pieces; the workspace is laid out for none)
  a.tc_slots = p.tc ? std::min(p.tc_slots, attn_tc_slots(*cache, *batch, a.group, window, n_sinks)) : 0;
  a.tc_part = reinterpret_cast<float*>(base + L.tc_part);
  a.status = &reinterpret_cast<WsHeader*>(base)->status;
  a.rows_above = a.rows_below = p.stream_rows;
  if (p.tc) {
    const cudaError_t e = launch_attention_tc(a, st);
    if (e != cudaSuccess) return STRATA_ERR_CUDA;
  }
  a.beside = p.tc;
  if (p.stream_rows > 0 && launch_attention(a, p, st) != cudaSuccess) return STRATA_ERR_CUDA;
  return a.tc_slots > 0 ? of(launch_attention_tc_join(a, st)) : STRATA_OK;
}

strata_status strata_kv_pages_extend(const strata_kv_pages* pages, const int32_t* new_tokens, int64_t T_max,
                                     int32_t* slots, int32_t* positions, int32_t* q_start, int32_t* copies,
                                     int32_t* n_copies, uint32_t* dev_status, strata_stream stream) {
  const strata_status s = check_pages(pages);
  if (s != STRATA_OK) return s;
  if (T_max < 0 || T_max > kMaxRows) return STRATA_ERR_SHAPE;
  if (!ints_ok(q_start) || !ints_ok(n_copies) || (dev_status && !on(dev_status, 4))) return STRATA_ERR_INVALID_ARG;
  if (T_max > 0 && (!ints_ok(slots) || !ints_ok(positions))) return STRATA_ERR_INVALID_ARG;
  if (pages->n_seq > 0 && (!ints_ok(new_tokens) || !ints_ok(copies))) return STRATA_ERR_INVALID_ARG;
  PagesExtendArgs a{};
  a.p = *pages;
  a.new_tokens = new_tokens;
  a.T_max = static_cast<int>(T_max);
  a.slots = slots;
  a.positions = positions;
  a.q_start = q_start;
  a.copies = copies;
  a.n_copies = n_copies;
  a.status = dev_status;
  return of(launch_pages_extend(a, reinterpret_cast<cudaStream_t>(stream)));
}

strata_status strata_kv_pages_fork(const strata_kv_pages* pages, const int32_t* parent, uint32_t* dev_status,
                                   strata_stream stream) {
  const strata_status s = check_pages(pages);
  if (s != STRATA_OK) return s;
  if (dev_status && !on(dev_status, 4)) return STRATA_ERR_INVALID_ARG;
  if (pages->n_seq == 0) return STRATA_OK;
  if (!ints_ok(parent)) return STRATA_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(&sms)) return STRATA_ERR_CUDA;
  return of(launch_pages_fork({*pages, parent, dev_status}, sms, reinterpret_cast<cudaStream_t>(stream)));
}

strata_status strata_kv_pages_release(const strata_kv_pages* pages, const int32_t* keep, int32_t window, int32_t n_sinks,
                                      uint32_t* dev_status, strata_stream stream) {
  const strata_status s = check_pages(pages);
  if (s != STRATA_OK) return s;
  if (window < 0 || n_sinks < 0 || (dev_status && !on(dev_status, 4)) || (keep && !on(keep, 4)))
    return STRATA_ERR_INVALID_ARG;
  if (pages->n_seq == 0 || pages->max_pages == 0 || (!keep && window == 0)) return STRATA_OK;
  int sms = 0;
  if (!sm_count(&sms)) return STRATA_ERR_CUDA;
  return of(launch_pages_release({*pages, keep, window, n_sinks, dev_status}, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t strata_kv_pages_compact_workspace_size(const strata_kv_pages* src) {
  if (check_pages(src) != STRATA_OK) return 0;
  return round_up(sizeof(WsHeader) + sizeof(int32_t) * src->n_pages);
}

strata_status strata_kv_pages_compact(const strata_kv_pages* src, const strata_kv_pages* dst, int32_t* copies,
                                      int32_t* n_copies, void* workspace, size_t ws_bytes, uint32_t* dev_status,
                                      strata_stream stream) {
  strata_status s = check_pages(src);
  if (s == STRATA_OK) s = check_pages(dst);
  if (s != STRATA_OK) return s;
  if (src->n_seq != dst->n_seq || src->page_size != dst->page_size || dst->max_pages < src->max_pages)
    return STRATA_ERR_SHAPE;
  if ((src->page_table && src->page_table == dst->page_table) || (src->kv_len && src->kv_len == dst->kv_len) ||
      (src->refs && src->refs == dst->refs))
    return STRATA_ERR_INVALID_ARG;
  if (!ints_ok(n_copies) || (dst->n_pages > 0 && !ints_ok(copies)) || (dev_status && !on(dev_status, 4)))
    return STRATA_ERR_INVALID_ARG;
  if (!workspace || !on(workspace, kWsAlign) || ws_bytes < strata_kv_pages_compact_workspace_size(src))
    return STRATA_ERR_WORKSPACE;
  int sms = 0;
  if (!sm_count(&sms)) return STRATA_ERR_CUDA;
  PagesCompactArgs a{};
  a.src = *src;
  a.dst = *dst;
  a.copies = copies;
  a.n_copies = n_copies;
  a.live = &static_cast<WsHeader*>(workspace)->nseg;
  a.map = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + sizeof(WsHeader));
  a.status = dev_status;
  return of(launch_pages_compact(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

strata_status strata_kv_copy_pages(const strata_kv_cache* src, const strata_kv_cache* dst, int32_t n_caches,
                                   const int32_t* copies, const int32_t* n_copies, int64_t max_copies,
                                   uint32_t* dev_status, strata_stream stream) {
  if (n_caches < 0 || n_caches > 1024 || max_copies < 0 || max_copies > 0x7FFFFFFF / 16) return STRATA_ERR_SHAPE;
  if (n_caches > 0 && (!src || !dst)) return STRATA_ERR_INVALID_ARG;
  if (n_caches > 0) {
    strata_status s = check_caches(src, n_caches, src->n_kv_heads, src->head_dim, src->page_size);
    if (s == STRATA_OK) s = check_caches(dst, n_caches, src->n_kv_heads, src->head_dim, src->page_size);
    if (s != STRATA_OK) return s;
  }
  if ((n_copies && !on(n_copies, 4)) || (dev_status && !on(dev_status, 4))) return STRATA_ERR_INVALID_ARG;
  if (n_caches == 0 || max_copies == 0) return STRATA_OK;
  if (!ints_ok(copies)) return STRATA_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(&sms)) return STRATA_ERR_CUDA;
  CopyPagesArgs a{};
  a.n_kv_heads = src->n_kv_heads;
  a.page_bytes = static_cast<int64_t>(src->n_kv_heads) * src->page_size * src->head_dim;
  a.src_pages = src->n_pages;
  a.dst_pages = dst->n_pages;
  a.copies = copies;
  a.n_copies = n_copies;
  a.max_copies = static_cast<int>(max_copies);
  a.status = dev_status;
  for (int at = 0; at < n_caches; at += kCopyCaches) {
    a.n_caches = std::min(n_caches - at, kCopyCaches);
    for (int i = 0; i < a.n_caches; ++i) {
      const strata_kv_cache &x = src[at + i], &y = dst[at + i];
      a.cache[i] = {x.k_codes, x.v_codes, x.k_scales, x.v_scales, y.k_codes, y.v_codes, y.k_scales, y.v_scales};
    }
    if (launch_copy_pages(a, sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return STRATA_ERR_CUDA;
  }
  return STRATA_OK;
}

}  // extern "C"
