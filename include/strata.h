/*
 * strata.h — C ABI of the GB300 routed MoE FFN layer with int4 group-quantized experts.
 *
 * The operations follow the problem statement of five write-ups about the
 * "Strata" MoE engine (the pages have no titles; each is named by its address):
 *   [tuning-3090] xdnf.cn/news/329730            §3.2 tokens routed to one expert are
 *                                                gathered into one group of a single
 *                                                grouped-GEMM launch; §5.2 fixed,
 *                                                pre-allocated buffers
 *   [tuning-moe]  lpnh.cn/news/2730718           §2.1 group_quantize(weight, 128, 4):
 *                                                scale = absmax/7, clamp(-8, 7);
 *                                                §2.3 point 1: router softmax + top-k
 *                                                fused in one kernel
 *   [tok-102]     zwxr.cn/news/276292            §3.2 routing engine: logits in,
 *                                                softmax, partial sort, expert ids out
 *   [glm-4090]    haowenji.com/articles/x-2109226022155796480
 *                                                §01 experts are Gate/Up + Down
 *                                                projections; 8 routed + 1 shared
 *                                                expert per token
 *
 * Conventions for every call below.
 *  - All tensor pointers are DEVICE pointers owned by the caller, unless a
 *    parameter says "host". The library never allocates or frees memory and keeps
 *    no state between calls; scratch memory is a caller-owned workspace whose size
 *    the *_workspace_size queries return.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) unless documented as blocking.
 *  - Arguments are validated on the host before anything is launched; a failed
 *    check returns its status and has no side effects.
 *  - Launch failures return STRATA_ERR_CUDA (from cudaGetLastError).
 *  - Kernels never trap. Faults they detect in the data (a non-finite weight, an
 *    expert id out of range) set bits in a device status word, read back with
 *    strata_workspace_status / strata_read_status (these synchronize the stream).
 *  - Dtypes: bf16/fp16 tensors are passed as void* to raw 16-bit storage.
 *  - Layouts are row-major and contiguous unless stated.
 */
#ifndef STRATA_H_
#define STRATA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* strata_stream; /* identical to cudaStream_t */

typedef enum {
  STRATA_OK = 0,
  STRATA_ERR_INVALID_ARG = 1,   /* null pointer, bad flag, k > E, ... */
  STRATA_ERR_SHAPE = 2,         /* a dimension is not a multiple of 128, or out of range */
  STRATA_ERR_UNSUPPORTED = 3,   /* group size not 64/128/256, or a size above a limit */
  STRATA_ERR_WORKSPACE = 4,     /* workspace null, misaligned or smaller than required */
  STRATA_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed */
  STRATA_ERR_DEVICE_STATUS = 6, /* the device status word reported a data fault */
  STRATA_ERR_TIMEOUT = 7        /* a bounded device-side wait gave up */
} strata_status;

/* Flags of strata_route_topk / strata_moe_layer.flags. */
#define STRATA_RENORM 0x1u       /* renormalise the k gates of a token to sum to 1 (off by default:
                                    the pages never renormalise) */
#define STRATA_ADD_RESIDUAL 0x2u /* moe_forward only: out = bf16(x + MoE(x)), one rounding */
#define STRATA_ROUTER_FP16 0x4u  /* the router weights are fp16 [E, H] instead of fp32 ("Strata" MoE
                                    tuning notes, lpnh.cn/news/2730718, §2.1: the router kept in
                                    fp16); logits still accumulate in fp32 over exact products */
/* Kernel-path selection of moe_forward (results agree within the layer tolerance; default: the
   tensor-core path from 128 tokens up, the warp path below). For tests and tuning. */
#define STRATA_FORCE_WARP_PATH 0x100u /* mma.sync warp GEMMs, B from registers */
#define STRATA_FORCE_TC_PATH 0x200u   /* tcgen05 / TMEM GEMMs fed by TMA */
/* Forward entry points: the caller promises that the workspace is zero-filled or was last used by
   a completed forward call (of any layer) that reported no device timeout. The per-call clearing
   of the workspace header (one memset between the previous kernel and the router) is then
   skipped; the device status word is not cleared per call either, but accumulates until
   strata_workspace_status reads (and clears) it. After a call that timed out, zero the workspace
   again before reusing it with this flag. */
#define STRATA_WS_REUSE 0x8u

/* Flag of strata_kv_append. */
#define STRATA_ROPE_NEIGHBOURS 0x1u /* the rotation pairs elements (2i, 2i + 1) instead of
                                       (i, i + rot_dim / 2) */

/* Bits of the device status word. */
#define STRATA_DEV_NONFINITE 0x1u /* a quantized group held inf/nan (its scale is written as NaN,
                                     its codes as 0); strata_kv_append: a row of K or V held inf/nan */
#define STRATA_DEV_BAD_ID 0x2u    /* an expert id outside [0, E) reached the permutation */
#define STRATA_DEV_TIMEOUT 0x4u   /* a bounded device wait gave up */
#define STRATA_DEV_BAD_TOKENS 0x8u /* strata_moe_forward_padded: the device token count was outside
                                      [0, T_max]; the call ran with no live token */
#define STRATA_DEV_BAD_SLOT 0x10u /* strata_kv_append: a slot or a position out of range (the row was
                                     skipped); strata_attention_forward: a page index, row range or
                                     length out of range (what it names was left out);
                                     strata_kv_pages_*, strata_kv_copy_pages: the same of a page, a
                                     sequence, a length or a count */
#define STRATA_DEV_NO_PAGES 0x20u /* strata_kv_pages_extend: too few free pages or rows (the sequences from
                                     there on got none); strata_kv_pages_compact: the other pool is too small */

#define STRATA_GROUP 128     /* [tuning-moe] §2.1: 128 weights share one scale */
#define STRATA_MAX_EXPERTS 1024
#define STRATA_MAX_TOPK 32

/* Human-readable name of a status code (static string, never NULL). */
const char* strata_status_string(int status);

/* ABI version: major*10000 + minor*100 + patch. */
int strata_version(void);

/*
 * strata_quantize_groups — symmetric int4 group quantization, [tuning-moe] §2.1.
 *
 * For each row i of w and each group g of G = group_size consecutive columns:
 *   scale[i,g] = fp16_round_nearest_even(absmax(w[i, Gg : Gg+G]) / 7)
 *   q[i,c]     = clamp(round_half_even(w[i,c] / scale[i,g]), -8, 7)   (exact quotient)
 *   a group whose stored scale is 0 gets q = 0.
 * w_fp16      [n, k] fp16, row-major (device).
 * codes       [n, k/2] uint8 (device, written): byte c of row i holds q[i,2c] in bits 0-3 and
 *             q[i,2c+1] in bits 4-7, as 4-bit two's complement.
 * scales_fp16 [n, k/group_size] fp16 (device, written).
 * group_size  128 (the pages' choice) or 64 / 256 (the sizes they weigh against it);
 *             anything else -> STRATA_ERR_UNSUPPORTED; k % group_size != 0 -> STRATA_ERR_SHAPE;
 *             n == 0 is a no-op.
 * dev_status  optional device uint32 (NULL to skip): STRATA_DEV_NONFINITE is OR-ed in when a
 *             group holds inf/nan; such a group gets scale NaN and codes 0.
 * Buffers must be 16-byte aligned (STRATA_ERR_INVALID_ARG otherwise).
 */
strata_status strata_quantize_groups(const void* w_fp16, int64_t n, int64_t k, int32_t group_size,
                                     uint8_t* codes, void* scales_fp16, uint32_t* dev_status,
                                     strata_stream stream);

/*
 * strata_quantize_groups_bits — the same with the sketch's bit width as a parameter
 * ([tuning-moe] §2.1: scale = absmax / (2^(bits-1) - 1); the pages keep experts at 4 bits and
 * attention projections at 8).
 * bits  4: exactly strata_quantize_groups.
 *       8: scale[i,g] = fp16_round_nearest_even(absmax / 127),
 *          q[i,c] = clamp(round_half_even(w[i,c] / scale[i,g]), -128, 127) (exact quotient);
 *          codes [n, k] int8 (two's complement), one per byte, row-major.
 *       anything else -> STRATA_ERR_UNSUPPORTED.
 * Other arguments, errors and alignment as strata_quantize_groups.
 */
strata_status strata_quantize_groups_bits(const void* w_fp16, int64_t n, int64_t k,
                                          int32_t group_size, int32_t bits, uint8_t* codes,
                                          void* scales_fp16, uint32_t* dev_status,
                                          strata_stream stream);

/*
 * strata_route_topk — router GEMV + softmax + top-k + token grouping,
 * [tuning-moe] §2.3 point 1 and [tok-102] §3.2; grouping per [tuning-3090] §3.2.
 *
 *   logits[t,e] = sum_h x[t,h] * w_router[e,h] + bias[e]     (fp32 accumulation)
 *   p[t,:]      = softmax(logits[t,:])                        (fp32)
 *   ids[t,:]    = the k experts of largest logit, in descending order, ties to the lower id
 *   gates[t,j]  = p[t, ids[t,j]]   (divided by sum_j of them when flags & STRATA_RENORM)
 * and, when the pointers are non-NULL, the grouping of the T*k routed rows by expert, rows
 * ordered by (expert, token):
 *   counts[e]   rows routed to expert e;  offsets[e] = sum_{e'<e} counts[e'], offsets[E] = T*k
 *   perm[r]     token of row r;           inv[t,j] = row of (t, ids[t,j])
 * x_bf16 [T,H] bf16; w_router [E,H] fp32 (fp16 when flags & STRATA_ROUTER_FP16: cast the
 * pointer); bias [E] fp32 or NULL. flags: STRATA_RENORM | STRATA_ROUTER_FP16.
 * ids [T,k] int32, gates [T,k] fp32 (required); counts [E], offsets [E+1], perm [T*k],
 * inv [T,k] int32 (optional as a group: all four or none).
 * Limits: H % 128 == 0, 1 <= k <= min(E, 32), E <= 1024, T >= 0 (T == 0 writes counts/offsets
 * as zeros only). workspace >= strata_route_workspace_size(T, E, k) bytes, 256-byte aligned.
 */
size_t strata_route_workspace_size(int64_t T, int32_t E, int32_t k);
strata_status strata_route_topk(const void* x_bf16, const float* w_router, const float* bias,
                                int64_t T, int64_t H, int32_t E, int32_t k, uint32_t flags,
                                int32_t* ids, float* gates, int32_t* counts, int32_t* offsets,
                                int32_t* perm, int32_t* inv, void* workspace, size_t ws_bytes,
                                strata_stream stream);

/*
 * strata_route_topk_noalloc — strata_route_topk without a workspace argument, for callers that
 * may not allocate device memory when they call in: plugin interfaces whose enqueue step must not
 * allocate, code running while a CUDA graph is being captured (cudaMalloc is not allowed then),
 * processes whose device memory is all handed out up front by one custom allocator. The pages
 * have no counterpart: this is an interface convenience, not part of the method.
 *
 * Scratch: a fixed array of STRATA_NOALLOC_SCRATCH_BYTES in the library's device globals. Every
 * GPU that loads the library holds it until the process exits. Requests whose scratch would not
 * fit (strata_route_workspace_size(T, E, k) > STRATA_NOALLOC_SCRATCH_BYTES) return
 * STRATA_ERR_UNSUPPORTED before anything runs; everything else is identical to
 * strata_route_topk (same arguments, outputs and checks, applied in the same order, the size
 * limit last). Nothing is allocated or freed, by the library or any routine it calls.
 * Set-up: every call made while `stream` is not capturing looks up the array's device address in
 * the current context (cudaGetSymbolAddress, with the device current) and keeps it; a call made
 * while `stream` captures uses the address kept by the last uncaptured call on that device, and
 * returns STRATA_ERR_UNSUPPORTED if there was none. So make one call on each device (and again
 * after a device reset or a switch to another context) before capturing it.
 * All calls share the one array: calls that overlap on the GPU (different streams, or several
 * host threads) race and must be serialised by the caller. Each call clears the status header it
 * needs before its kernels run; the rest of the array keeps the previous call's contents.
 * Device status of the last call: strata_workspace_status is not available (no workspace
 * pointer); data faults still never trap.
 */
#define STRATA_NOALLOC_SCRATCH_BYTES (8u << 20) /* 8 MiB per device */
strata_status strata_route_topk_noalloc(const void* x_bf16, const float* w_router,
                                        const float* bias, int64_t T, int64_t H, int32_t E,
                                        int32_t k, uint32_t flags, int32_t* ids, float* gates,
                                        int32_t* counts, int32_t* offsets, int32_t* perm,
                                        int32_t* inv, strata_stream stream);

/*
 * strata_group_rows — the grouping step alone, for routes the caller computed ([tuning-3090]
 * §3.2: the rows routed to one expert are gathered into one group of the grouped GEMM): the
 * counts, offsets, perm and inv of strata_route_topk for a given ids [T,k] int32 (device), rows
 * ordered by (expert, token, slot) (a token may name one expert in several slots).
 * counts [E], offsets [E+1] (required); perm [T*k], inv [T,k] (required when T > 0); all int32,
 * device, 4-byte aligned. An id outside [0, E) sets STRATA_DEV_BAD_ID in the workspace status
 * word; its row is left out of every group (inv = -1, no perm entry) and offsets[E] counts the
 * valid rows only, which keep the positions they would have without the invalid ones.
 * Limits: 0 <= T <= 2^22, 1 <= k <= 32, 1 <= E <= 1024. workspace >=
 * STRATA_GROUP_WORKSPACE_BYTES, 256-byte aligned (it holds the status word only).
 */
#define STRATA_GROUP_WORKSPACE_BYTES 256u
strata_status strata_group_rows(const int32_t* ids, int64_t T, int32_t k, int32_t E,
                                int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv,
                                void* workspace, size_t ws_bytes, strata_stream stream);

/*
 * One routed MoE FFN layer. Expert weights are the outputs of strata_quantize_groups, stacked
 * over experts; the shared expert, when has_shared != 0, is index E of each stack.
 * Expert e computes y = (silu(x Wg_e^T) * (x Wu_e^T)) Wd_e^T   ([glm-4090] §01: Gate/Up, Down).
 */
typedef struct {
  int64_t H;             /* hidden size, % 128 == 0 */
  int64_t I;             /* expert intermediate size, % 128 == 0 */
  int32_t E;             /* routed experts, 1..1024 */
  int32_t k;             /* experts per token, 1..min(E, 32) */
  int32_t has_shared;    /* 0 or 1: expert E is always on, gate 1 */
  uint32_t flags;        /* STRATA_RENORM | STRATA_ADD_RESIDUAL | STRATA_ROUTER_FP16 |
                            STRATA_FORCE_*_PATH | STRATA_WS_REUSE */
  const float* w_router; /* [E, H] fp32, or fp16 with STRATA_ROUTER_FP16 (cast the pointer) */
  const float* bias;     /* [E] fp32 or NULL */
  const uint8_t* gate_codes; const void* gate_scales; /* [E+S, I, H/2] u8, [E+S, I, H/128] fp16 */
  const uint8_t* up_codes;   const void* up_scales;   /* same shapes */
  const uint8_t* down_codes; const void* down_scales; /* [E+S, H, I/2] u8, [E+S, H, I/128] fp16 */
  int32_t group_size;    /* scale group of all three projections: 128 (0 means 128), 64 or 256;
                            the scales above are then [.., K/group_size]. 256 on the decode path
                            needs H % 512 == 0 and I % 512 == 0 */
  int32_t bits;          /* code width of all three projections: 4 (0 means 4) or 8. With 8 the
                            codes are int8, one per byte (strata_quantize_groups_bits): gate/up
                            [E+S, I, H], down [E+S, H, I]; such layers run on the tensor-core
                            grouped GEMM at every batch size (STRATA_FORCE_WARP_PATH ->
                            STRATA_ERR_UNSUPPORTED) */
} strata_moe_layer;

/* Workspace bytes strata_moe_forward needs for up to T_max tokens (0 if the layer is invalid). */
size_t strata_moe_workspace_size(const strata_moe_layer* layer, int64_t T_max);

/*
 * strata_moe_forward — out[t] = sum_j gates[t,j] * y_{ids[t,j]}(x_t) + has_shared * y_E(x_t)
 * (+ x_t with STRATA_ADD_RESIDUAL), summed in fp32 and rounded once to bf16.
 * x_bf16 [T,H], out_bf16 [T,H] bf16 (device; out may not alias x). T == 0 is a no-op.
 * workspace: >= strata_moe_workspace_size(layer, T) bytes, 256-byte aligned, device. The
 * workspace needs no initialisation; one workspace serves one stream at a time.
 */
strata_status strata_moe_forward(const strata_moe_layer* layer, const void* x_bf16, int64_t T,
                                 void* out_bf16, void* workspace, size_t ws_bytes,
                                 strata_stream stream);

/*
 * strata_moe_forward_padded — strata_moe_forward at a fixed maximum batch whose live token count
 * is read on the device when the call runs, so that one CUDA graph captured at T_max serves every
 * batch of 0..T_max tokens ([tuning-3090] §3.2: the grouped GEMM captured as a fixed graph node
 * at a fixed maximum batch, smaller batches padded with empty tokens; §5.2: every buffer
 * allocated before the graph is built).
 * n_tokens  device int32, 4-byte aligned: T, the live tokens, rows 0..T-1 of x. It is read by the
 *           call's first kernel, so a graph replays with whatever it holds at that point (write it
 *           with a copy in stream order before the replay).
 * x_bf16    [T_max, H] bf16 (device); rows T..T_max-1 are never read and may hold anything.
 * out_bf16  [T_max, H] bf16 (device); rows 0..T-1 get exactly what strata_moe_forward gives for
 *           those T tokens up to the order of its contraction sums (the GEMMs' schedule, and with
 *           it how a contraction is split between CTAs, is chosen for T_max); rows T..T_max-1 are
 *           not written. The padding tokens route to no expert and cost no weight traffic: every
 *           grid is sized for T_max, every loop stops at T.
 * A count outside [0, T_max] sets STRATA_DEV_BAD_TOKENS in the device status word and the call
 * then runs with no live token (out untouched).
 * T_max: 1..64 (the fused decode router); 4-bit codes; not STRATA_FORCE_TC_PATH. Otherwise
 * STRATA_ERR_UNSUPPORTED (T_max < 1: STRATA_ERR_SHAPE). workspace >=
 * strata_moe_workspace_size(layer, T_max). Other errors as strata_moe_forward.
 */
strata_status strata_moe_forward_padded(const strata_moe_layer* layer, const void* x_bf16,
                                        const int32_t* n_tokens, int64_t T_max, void* out_bf16,
                                        void* workspace, size_t ws_bytes, strata_stream stream);

/*
 * strata_moe_stack_forward — n_layers MoE layers in sequence with a residual add between them:
 *   x_0 = x,  x_{l+1} = bf16(x_l + MoE_l(x_l)),  out = x_{n_layers}
 * (each layer as strata_moe_forward with STRATA_ADD_RESIDUAL; no normalisation is applied, none
 * being named for the stack). layers: host array of n_layers descriptors (1..256), all with the
 * same H. x_bf16, out_bf16: [T,H] bf16, device, distinct. workspace >=
 * strata_moe_stack_workspace_size (device, 256-byte aligned, caller-owned; it also holds the two
 * intermediate activation buffers). The device status word at the workspace start collects the
 * STRATA_DEV_* bits of every layer (strata_workspace_status reads it after the stack). Errors:
 * as strata_moe_forward, checked for every layer before the first launch; STRATA_ERR_SHAPE when
 * the layers' H differ.
 */
size_t strata_moe_stack_workspace_size(const strata_moe_layer* layers, int32_t n_layers,
                                       int64_t T_max);
strata_status strata_moe_stack_forward(const strata_moe_layer* layers, int32_t n_layers,
                                       const void* x_bf16, int64_t T, void* out_bf16,
                                       void* workspace, size_t ws_bytes, strata_stream stream);

/*
 * strata_moe_forward_ex — strata_moe_forward that also copies the routing out (each pointer
 * optional, device): ids [T,k], gates [T,k], counts [E], offsets [E+1], perm [T*k], inv [T,k],
 * with the meanings of strata_route_topk.
 */
strata_status strata_moe_forward_ex(const strata_moe_layer* layer, const void* x_bf16, int64_t T,
                                    void* out_bf16, int32_t* ids, float* gates, int32_t* counts,
                                    int32_t* offsets, int32_t* perm, int32_t* inv,
                                    void* workspace, size_t ws_bytes, strata_stream stream);

/*
 * strata_moe_forward_stats — strata_moe_forward that also accumulates expert-activation statistics
 * (the hot-expert list of "Strata" 3090 tuning, xdnf.cn/news/329730, §5.5): expert_rows[e] +=
 * rows routed to expert e in this batch, and expert_rows[E] += T for the shared expert.
 * expert_rows: [E + has_shared] uint64, device, 8-byte aligned, caller-owned and caller-zeroed;
 * calls on several streams may accumulate into the same array (atomic adds). Results and errors
 * are those of strata_moe_forward; STRATA_ERR_INVALID_ARG if expert_rows is NULL or unaligned.
 */
strata_status strata_moe_forward_stats(const strata_moe_layer* layer, const void* x_bf16,
                                       int64_t T, void* out_bf16, uint64_t* expert_rows,
                                       void* workspace, size_t ws_bytes, strata_stream stream);

/*
 * strata_moe_forward_profiled — strata_moe_forward that also records caller-created CUDA events
 * (cudaEvent_t, passed as void*) on `stream` at the stage boundaries, for per-kernel timing:
 *   events[0] before the router, [1] after the router (logits + top-k), [2] after the grouping,
 *   [3] after the gate/up grouped GEMM, [4] after the down grouped GEMM, [5] after the combine.
 * n_events must be 6; any NULL event is skipped. Results are identical to strata_moe_forward.
 */
#define STRATA_PROFILE_EVENTS 6
strata_status strata_moe_forward_profiled(const strata_moe_layer* layer, const void* x_bf16,
                                          int64_t T, void* out_bf16, void* workspace,
                                          size_t ws_bytes, strata_stream stream,
                                          void* const* events, int32_t n_events);

/*
 * strata_moe_forward_host — the same layer with HOST activations: copies x_host (bf16 [T,H],
 * host memory, best pinned) to the workspace, runs the layer, copies the result to out_host
 * (bf16 [T,H], host). BLOCKING: returns after out_host is written (synchronizes `stream`).
 * workspace >= strata_moe_workspace_size(layer, T) + strata_moe_host_staging_size(layer, T).
 */
size_t strata_moe_host_staging_size(const strata_moe_layer* layer, int64_t T_max);
strata_status strata_moe_forward_host(const strata_moe_layer* layer, const void* x_host,
                                      int64_t T, void* out_host, void* workspace, size_t ws_bytes,
                                      strata_stream stream);

/*
 * The attention half of a decoder block around the MoE layer: quantized projections, a paged cache
 * of 8-bit keys and values, and attention over it ([tuning-moe] §2.1: the engine keeps its
 * attention projections at 8 bits in the same group format, the output projection at 4). The pages
 * do not describe the cache; its format and the calls are this library's own.
 */

/* One dense projection: codes and scales are outputs of strata_quantize_groups_bits. */
typedef struct {
  int64_t N;           /* output features, 1 .. 2^20 */
  int64_t K;           /* input features, % group_size == 0, up to 2^16 */
  int32_t group_size;  /* 128 (0 means 128), 64 or 256 */
  int32_t bits;        /* 4 (0 means 4) or 8 */
  const uint8_t* codes; /* [N, K/2] (4 bits) or [N, K] int8 (8 bits), 16-byte aligned */
  const void* scales;  /* [N, K/group_size] fp16 */
  const float* bias;   /* [N] fp32 or NULL */
} strata_linear;

/*
 * strata_linear_forward — out[t,n] = sum_c x[t,c] * q[n,c] * scale[n, c / group_size] + bias[n]
 * (+ residual[t,n]), summed in fp32 and rounded once to bf16.
 * x_bf16 [T,K], out_bf16 [T,N], residual_bf16 [T,N] or NULL: bf16, device, consecutive elements in a
 * row; *_stride: elements from one row to the next (>= the row's length; x: a multiple of 8, and x
 * 16-byte aligned). out may be the residual itself (same address and stride); otherwise out
 * overlaps no input. T == 0 is a no-op.
 * Up to STRATA_LINEAR_EXACT_T tokens the codes are multiplied as exact integers and the sums scaled in fp32;
 * longer batches may multiply weights rounded once to f16 (2^-11 relative), with f16 copies of the
 * rows of x in the workspace, each times a power of two that keeps its range.
 * workspace >= strata_linear_workspace_size(w, T) bytes (0: the projection or T is invalid),
 * 256-byte aligned, device; it needs no initialisation. strata_workspace_status reads its status, that
 * of the last call: every call clears the word first.
 */
#define STRATA_LINEAR_EXACT_T 64
size_t strata_linear_workspace_size(const strata_linear* w, int64_t T_max);
strata_status strata_linear_forward(const strata_linear* w, const void* x_bf16, int64_t x_stride,
                                    int64_t T, const void* residual_bf16, int64_t residual_stride,
                                    void* out_bf16, int64_t out_stride, void* workspace,
                                    size_t ws_bytes, strata_stream stream);

/*
 * A paged cache of keys and values in 8 bits. A page holds page_size consecutive tokens of one
 * sequence for every head. Values are e4m3 codes times one fp32 scale per (page, head), one for K
 * and one for V. strata_kv_append writes power-of-two scales: a floating code loses nothing by
 * that, and a page whose range grows later is rescaled exactly (but for e4m3 subnormals).
 * Slot s of the cache is token s % page_size of page s / page_size. No initialisation is needed: a
 * page counts from the token that is put at its start.
 */
typedef struct {
  int32_t n_kv_heads; /* 1 .. 256 */
  int32_t head_dim;   /* 64 or 128 */
  int32_t page_size;  /* 16, 32, 64 or 128 */
  int64_t n_pages;    /* n_pages * page_size <= 2^31 - 1 */
  uint8_t* k_codes;   /* [n_pages, n_kv_heads, page_size, head_dim] e4m3, 16-byte aligned */
  uint8_t* v_codes;   /* the same */
  float* k_scales;    /* [n_pages, n_kv_heads], positive */
  float* v_scales;    /* the same */
} strata_kv_cache;

/*
 * strata_kv_append — rotates the T rows of k (and of q) by their positions and stores k and v in the
 * cache. Row t goes to slot slots[t]; a negative slot marks a padding row, of which nothing is
 * used or written (its elements may be loaded with those of the rows before it).
 *   rotation of pair (a, b) of a head's first rot_dim elements, in fp32:
 *     a' = a*cos - b*sin, b' = b*cos + a*sin,   cos = rope[pos][i], sin = rope[pos][rot_dim/2 + i]
 *     with a, b = elements i and i + rot_dim/2, or 2i and 2i + 1 with STRATA_ROPE_NEIGHBOURS
 *   scale of a page and head: 2^e, e the smallest integer >= -100 with absmax <= 448 * 2^e over
 *     the tokens of the page. Rows that begin inside a page (slot % page_size > 0) keep the tokens
 *     before them: the scale never falls, and if it grows the older codes are rewritten.
 *   codes: value / scale rounded to e4m3, nearest-even, once.
 * A (row, head) whose rotated k or v holds inf or nan sets STRATA_DEV_NONFINITE, gets k codes nan
 * and v codes 0, and has no part in the scale: the nan reaches the queries that see the token and
 * no others.
 * k, v [T, n_kv_heads * head_dim], q and q_out [T, n_heads * head_dim] bf16, device; rows
 * 16-byte aligned, strides in elements, multiples of 8. q, q_out NULL: keys and values only. q_out
 * may be q itself (same stride).
 * slots, positions [T] int32 (device); rope [n_pos, rot_dim] fp32, 16-byte aligned (device).
 * rot_dim: 0 (no rotation: rope and positions may be NULL) or a multiple of 16 up to head_dim.
 * The rows of a call that fall into one page must be consecutive rows with consecutive slots. A
 * slot >= n_pages * page_size or a position outside [0, n_pos) sets STRATA_DEV_BAD_SLOT and the row
 * is skipped: its slot keeps what it holds, and it has no part in the scale. (A page whose first token
 * was skipped by a call that stored nothing in it has not begun.) dev_status: device uint32 or NULL. T == 0 is a no-op; T <= 2^22.
 */
strata_status strata_kv_append(const strata_kv_cache* cache, const void* q_bf16, int64_t q_stride,
                               int32_t n_heads, const void* k_bf16, int64_t k_stride,
                               const void* v_bf16, int64_t v_stride, int64_t T,
                               const int32_t* slots, const int32_t* positions, const float* rope,
                               int64_t n_pos, int32_t rot_dim, uint32_t flags, void* q_out,
                               int64_t q_out_stride, uint32_t* dev_status, strata_stream stream);

/* Norms of queries and keys, one for each head of a row. */
typedef struct {
  const float* q_weight; /* [head_dim] fp32 for all query heads (q_head_stride 0), or a row a head; 16-byte aligned;
                            NULL: q is not normalised */
  int64_t q_head_stride; /* elements from one head's row to the next: 0, or >= head_dim and a multiple of 4 */
  const float* k_weight; /* the same for the K heads */
  int64_t k_head_stride;
  float eps;             /* finite, >= 2^-100 */
} strata_qk_norm;

/*
 * strata_kv_append_normed — strata_kv_append with a norm of each head's row of q and k ahead of the rotation:
 *   y[i] = x[i] / sqrt(mean_i(x[i]^2) + eps) * weight[i]      (i < head_dim; v is taken as it is)
 * in fp32: nothing is rounded between the norm and the rotated result (q_out bf16, k codes e4m3). A finite row of
 * any size has its norm: sums of squares do not overflow. A (row, head) of k that holds inf or nan, or becomes one by its
 * weights, is treated as one of strata_kv_append; such a row of q gives nan where it is not finite.
 * Arguments, errors and everything else as strata_kv_append; STRATA_ERR_INVALID_ARG also for a NULL norm, an eps out of
 * range, and weights that are not aligned or whose stride is below head_dim or no multiple of 4. Without either weight
 * the call is strata_kv_append.
 */
strata_status strata_kv_append_normed(const strata_kv_cache* cache, const strata_qk_norm* norm, const void* q_bf16,
                                      int64_t q_stride, int32_t n_heads, const void* k_bf16, int64_t k_stride,
                                      const void* v_bf16, int64_t v_stride, int64_t T, const int32_t* slots,
                                      const int32_t* positions, const float* rope, int64_t n_pos, int32_t rot_dim,
                                      uint32_t flags, void* q_out, int64_t q_out_stride, uint32_t* dev_status,
                                      strata_stream stream);

/* The sequences of one attention call. Arrays are on the device, int32. */
typedef struct {
  int32_t n_seq;            /* 0 .. 65535 */
  int32_t max_q;            /* at least the most query rows of one sequence */
  int64_t T;                /* rows of q and out, up to 2^22 */
  int64_t max_kv;           /* at least the largest kv_len; up to table_stride * page_size;
                               (max_kv / 32 + 1) * n_seq * n_kv_heads < 2^31 */
  const int32_t* q_start;   /* [n_seq + 1]: rows q_start[s] .. q_start[s+1] - 1 belong to sequence s */
  const int32_t* kv_len;    /* [n_seq]: tokens of the sequence in the cache, those of this call among them */
  const int32_t* page_table; /* [n_seq, table_stride]: the sequence's pages in order */
  int64_t table_stride;
} strata_kv_batch;

/*
 * strata_attention_forward — causal attention of q over the cache. Query i of a sequence with n
 * query rows and kv_len = L stands at position p = L - n + i and sees tokens j <= p, and
 * j > p - window when window > 0:
 *   out = sum_j softmax_j(scale * q . k_j) v_j     (statistics and sums in fp32; no token: zeros)
 * A token's weight times its page's V scale enters the sum of values in f16, relative to the row's
 * largest: rounded to 2^-11 of itself, or to 2^-25 of that largest one. Codes, queries (f16 times a
 * power of two a row, exact but for entries 2^-17 below the row's largest) and page scales are used
 * as they are, however far apart the scales of pages lie; V scales below 2^-100 count as 2^-100.
 * Head h reads K/V head h / (n_heads / n_kv_heads). q, out [T, n_heads * head_dim] bf16 (device,
 * 16-byte aligned rows, strides in elements, multiples of 8); rows of no sequence are not written.
 * Any lengths may be mixed in one call. What the cache holds past kv_len, or before the first token
 * that a row of the sequence sees through the window, is not used, whatever it is, and the page
 * table's entries for pages that lie there whole are not looked at: such pages may be given back.
 * A page index outside [0, n_pages) sets STRATA_DEV_BAD_SLOT and its tokens count as unseen;
 * so does a row range outside [0, T], a length below 0 or above max_kv, or more rows than max_q:
 * they are cut to the limit.
 * flags: STRATA_WS_REUSE (the workspace is zero-filled, or was left by a completed call of this
 * function: it is then not cleared first, and its status word accumulates).
 * workspace >= strata_attention_workspace_size(cache, batch, n_heads), 256-byte aligned (0: an
 * argument is invalid). n_seq == 0 or T == 0 is a no-op.
 */
size_t strata_attention_workspace_size(const strata_kv_cache* cache, const strata_kv_batch* batch,
                                       int32_t n_heads);
strata_status strata_attention_forward(const strata_kv_cache* cache, const strata_kv_batch* batch,
                                       const void* q_bf16, int64_t q_stride, int32_t n_heads,
                                       float scale, int32_t window, uint32_t flags, void* out_bf16,
                                       int64_t out_stride, void* workspace, size_t ws_bytes,
                                       strata_stream stream);

/*
 * strata_attention_sinks_forward — strata_attention_forward with a window and n_sinks first tokens of each sequence that
 * stay visible: a query at position p sees tokens j <= p with j > p - window or j < n_sinks (window 0: all j <= p,
 * whatever n_sinks is).
 * What the cache holds between the first tokens and the first token that a row of the sequence sees through the
 * window is not used, and the page table's entries for pages that lie there whole are not looked at: such pages may be
 * given back (strata_kv_pages_release does, and leaves -1). n_sinks >= 0; the workspace is that of
 * strata_attention_workspace_size, and may go from one of the two calls to the other. Arguments, errors and everything
 * else as strata_attention_forward, which is this call with n_sinks 0.
 */
strata_status strata_attention_sinks_forward(const strata_kv_cache* cache, const strata_kv_batch* batch,
                                             const void* q_bf16, int64_t q_stride, int32_t n_heads, float scale,
                                             int32_t window, int32_t n_sinks, uint32_t flags, void* out_bf16,
                                             int64_t out_stride, void* workspace, size_t ws_bytes,
                                             strata_stream stream);

/*
 * Pages of a cache and who holds them, on the device: the caller owns the arrays, the calls below change them, and a
 * page number means the same in every cache of a model's layers. Begin with refs and kv_len zero and page_table -1.
 */
typedef struct {
  int32_t n_seq;        /* 0 .. 65535 */
  int32_t page_size;    /* 16, 32, 64 or 128 */
  int64_t n_pages;      /* n_pages * page_size <= 2^31 - 1 */
  int64_t max_pages;    /* pages that a sequence can have; max_pages * page_size <= 2^31 - 1 */
  int64_t table_stride; /* entries from one sequence's row to the next, >= max_pages */
  int32_t* page_table;  /* [n_seq, max_pages]: a sequence's pages in order; -1 where there is none: behind its
                           tokens, or given back */
  int32_t* kv_len;      /* [n_seq]: tokens of each sequence */
  int32_t* refs;        /* [n_pages], 16-byte aligned: table entries that name the page; 0: it is free */
} strata_kv_pages;

/*
 * strata_kv_pages_extend — room for new_tokens[s] more tokens of each sequence, and their rows: what strata_kv_append
 * and strata_attention_forward want of them.
 * Sequence s gets the lowest free pages, the sequences in order, and kv_len[s] grows. Its new tokens are rows
 * q_start[s] .. q_start[s+1] - 1, at positions from the old length on. An unfinished page that other sequences
 * hold too is left to them: its place in the table gets a free page, and the pair (old page, new page) is listed
 * in copies, to be copied (strata_kv_copy_pages) before the append. Sequences that are extended in the same call count as
 * others: if all that hold the page are extended, all of them leave it, a free page each, and it is free.
 * new_tokens  [n_seq] int32, >= 0.           T_max  rows of slots and positions, up to 2^22.
 * slots, positions [T_max], q_start [n_seq + 1], copies [n_seq, 2], n_copies [1]: int32, written; rows
 *             without a token get slot -1 (padding of strata_kv_append) and position 0, copies from n_copies on keep
 *             what they hold.
 * From the first sequence on for which free pages or rows run out, no sequence gets any (STRATA_DEV_NO_PAGES); one with a
 * negative count or length, more tokens than its table holds, or an unfinished page that is none or that nobody counts
 * gets nothing (STRATA_DEV_BAD_SLOT): its length stays. dev_status here and below: device uint32 or NULL.
 */
strata_status strata_kv_pages_extend(const strata_kv_pages* pages, const int32_t* new_tokens, int64_t T_max,
                                     int32_t* slots, int32_t* positions, int32_t* q_start, int32_t* copies,
                                     int32_t* n_copies, uint32_t* dev_status, strata_stream stream);

/*
 * strata_kv_pages_fork — sequences that go on from where another one is: each s with parent[s] >= 0 takes that
 * sequence's length and pages, which both hold from then on (refs grows; nothing is copied before one of them is
 * extended). parent [n_seq] int32, -1: s stays as it is. s has to be empty (kv_len 0), and its parent may not have a
 * parent in the same call; otherwise, or for a parent >= n_seq, STRATA_DEV_BAD_SLOT is set and s stays as it is.
 */
strata_status strata_kv_pages_fork(const strata_kv_pages* pages, const int32_t* parent, uint32_t* dev_status,
                                   strata_stream stream);

/*
 * strata_kv_pages_release — gives pages back: their table entries become -1, and a page is free when nobody holds it.
 * keep [n_seq] int32 or NULL: sequence s is cut to min(kv_len[s], keep[s]) tokens (0: it ends), unless keep[s] < 0.
 * window > 0: of every sequence the pages that lie whole between its n_sinks first tokens and the window of its next
 * query (at position kv_len) go too: what strata_attention_sinks_forward with these numbers does not look at in later
 * calls. (Rows that are in the cache already and still to be attended to have earlier windows: release after them.)
 * A later cut moves the next query's window back, and what was before it is gone: attention leaves such tokens out, and
 * strata_kv_pages_extend gives nothing to a sequence whose unfinished page it was (both set STRATA_DEV_BAD_SLOT). Where a
 * sequence may come back to a length up to c tokens below one that it was released at (rejected drafts), release with window + c.
 */
strata_status strata_kv_pages_release(const strata_kv_pages* pages, const int32_t* keep, int32_t window, int32_t n_sinks,
                                      uint32_t* dev_status, strata_stream stream);

/*
 * strata_kv_pages_compact — the same sequences in another pool, a smaller or larger one: pages in use get the numbers
 * 0, 1, ... in the order of their old ones. dst's table, lengths and refs are written whole; copies
 * [dst->n_pages, 2] lists the pairs (old page, new page) and n_copies [1] their number, for
 * strata_kv_copy_pages from the caches of src to those of dst. src is not changed. n_seq and page_size are the same,
 * dst->max_pages >= src's (STRATA_ERR_SHAPE otherwise), and no array serves both (STRATA_ERR_INVALID_ARG).
 * If more pages are in use than dst has, dst is left empty and STRATA_DEV_NO_PAGES is set. An entry that names no
 * page or one that nobody counts becomes -1 (STRATA_DEV_BAD_SLOT).
 * workspace >= strata_kv_pages_compact_workspace_size(src) bytes (0: src is invalid), 256-byte aligned.
 */
size_t strata_kv_pages_compact_workspace_size(const strata_kv_pages* src);
strata_status strata_kv_pages_compact(const strata_kv_pages* src, const strata_kv_pages* dst, int32_t* copies,
                                      int32_t* n_copies, void* workspace, size_t ws_bytes, uint32_t* dev_status,
                                      strata_stream stream);

/*
 * strata_kv_copy_pages — copies whole pages, codes and scales: for each pair i < n_copies, page copies[i][0] of src[c] to
 * page copies[i][1] of dst[c], for all n_caches caches c (up to 1024, host arrays; the layers of a model).
 * copies [max_copies, 2], n_copies [1] or NULL (max_copies): int32, device. A pair with a negative page is no copy; one
 * with a page out of range, or a count outside 0 .. max_copies, sets STRATA_DEV_BAD_SLOT (no copy; the count is
 * cut). The pages written differ from one another and, where dst is src, from those read: the order of copies is
 * not defined. All caches have the same n_kv_heads, head_dim and page_size, those of src and those of dst each the
 * same n_pages (STRATA_ERR_SHAPE otherwise). dst may be src.
 */
strata_status strata_kv_copy_pages(const strata_kv_cache* src, const strata_kv_cache* dst, int32_t n_caches,
                                   const int32_t* copies, const int32_t* n_copies, int64_t max_copies,
                                   uint32_t* dev_status, strata_stream stream);

/*
 * Device status of a route/forward workspace: synchronizes `stream`, returns the status word in
 * *status_out (host) and clears it. Returns STRATA_ERR_TIMEOUT when STRATA_DEV_TIMEOUT was set (a
 * bounded device wait gave up: the call's outputs are incomplete), else STRATA_ERR_DEVICE_STATUS
 * when any other bit was set, else STRATA_OK.
 */
strata_status strata_workspace_status(void* workspace, strata_stream stream, uint32_t* status_out);

/* Same for a caller-owned device status word (e.g. the one given to strata_quantize_groups). */
strata_status strata_read_status(uint32_t* dev_status, strata_stream stream, uint32_t* status_out);

/*
 * strata_selftest_bounded_waits — a diagnostic of the failure path of the library's two bounded
 * device waits (no data path): the mbarrier wait of the TMA-fed grouped GEMMs and the counter
 * spin of the fused router run, one after the other, on a barrier and a counter that nothing
 * completes, each with a limit of limit_cycles SM clocks instead of its ~1-2 s. Each must give
 * up, OR STRATA_DEV_TIMEOUT into dev_words[0] and return, so the kernel ends after about
 * 2 * limit_cycles clocks and the context stays usable.
 * dev_words  [4] uint32, device, 16-byte aligned, caller-zeroed: [0] status word (read it with
 *            strata_read_status, which then returns STRATA_ERR_TIMEOUT), [1] the counter (must
 *            stay 0), [2] / [3] set to 1 when the mbarrier wait / the counter spin gave up.
 * limit_cycles 1 .. 4e9; outside -> STRATA_ERR_INVALID_ARG. Asynchronous on `stream`.
 */
strata_status strata_selftest_bounded_waits(uint32_t* dev_words, int64_t limit_cycles,
                                            strata_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* STRATA_H_ */
