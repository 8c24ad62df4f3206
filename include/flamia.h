/*
 * flamia.h — C ABI of the block-scaled causal attention training call
 * (FLAMIA-style MXFP8 and mixed NVFP4/FP8 paths) for one GB300 (sm_103a).
 *
 * Sources, by page title and section:
 *   [SUM]  "FLAMIA: FLAsh MIcroscaling Attention for Fast and Causally Safe
 *          Training on Blackwell" (paper summary), bullets under §3.1–§3.7,
 *          §4.1–§4.6.
 *   [READ] "因果安全的低精度注意力——FLAMIA Blackwell 训练内核精读"
 *          (close reading), 四 4.1–4.6 and 五 5.1–5.3.
 *
 * One training call is, in this order, on one CUDA stream:
 *   flamia_plan        -> work lists and document tables (once per cu_seqlens)
 *   flamia_quantize    -> role QKV: Q^, K^, V^ codes and scales
 *   flamia_fwd         -> O, per-row (m, l)
 *   flamia_quantize    -> role DO: dO^ codes and scales, D = rowsum(dO^ * O)
 *   flamia_bwd         -> dQ, dK, dV
 * ([READ] 五 5.1: the training call is forward + backward + quantization.)
 *
 * Conventions for every entry point:
 *   - Every pointer named "device" is a CUDA device pointer owned by the
 *     caller; the library never allocates, frees or synchronises inside
 *     plan/quantize/fwd/bwd, so the sequence can be captured in a CUDA graph.
 *   - Packed token-major layouts: activations [T][heads][d] (row-major, d
 *     contiguous); per-token metadata [heads][T].
 *   - Every device pointer must be 16-byte aligned (cu_seqlens: 4-byte);
 *     tensors are contiguous.
 *   - Arguments are validated on the host before any launch; a violation
 *     returns FLAMIA_ERR_INVALID_ARG or FLAMIA_ERR_UNSUPPORTED and launches
 *     nothing.  Launch failures return FLAMIA_ERR_CUDA.  Device-side
 *     conditions (a bounded wait that expired, an inconsistent cu_seqlens
 *     seen by a kernel) set the device status word in the workspace, read
 *     with flamia_get_device_status().
 *   - The workspace `ws` (size from flamia_workspace_size) holds the plan,
 *     the dQ accumulator (fp32, or FP16 with its prescale exponents), and
 *     the status word.  It must stay the same buffer from flamia_plan through
 *     flamia_bwd of one call.
 */
#ifndef FLAMIA_H_
#define FLAMIA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FLAMIA_OK = 0,
  FLAMIA_ERR_INVALID_ARG = 1,
  FLAMIA_ERR_UNSUPPORTED = 2,
  FLAMIA_ERR_WORKSPACE_TOO_SMALL = 3,
  FLAMIA_ERR_CUDA = 4,
  FLAMIA_ERR_TIMEOUT = 5,
  FLAMIA_ERR_BAD_SEQLENS = 6,
  FLAMIA_ERR_NO_PAGES = 7, /* paged cache: the free stack has too few pages */
  FLAMIA_ERR_BAD_PAGE = 8  /* paged cache: a page id, slot or free count out of range */
} flamia_status_t;

/* [SUM] §3.4: the two default training paths. */
typedef enum { FLAMIA_PATH_MXFP8 = 0, FLAMIA_PATH_NVFP4_FP8 = 1 } flamia_path_t;

typedef enum { FLAMIA_F32 = 0, FLAMIA_BF16 = 1, FLAMIA_E4M3 = 2, FLAMIA_E2M1 = 3 /* both: paged caches only */ } flamia_dtype_t;

typedef enum { FLAMIA_ROLE_QKV = 0, FLAMIA_ROLE_DO = 1 } flamia_role_t;

/* Problem description (host struct; cu_seqlens is a device pointer).
 *   T            total packed tokens (>= 1)
 *   H, Hkv       query heads and key/value heads; H % Hkv == 0 (GQA)
 *   d            head dimension: 64 or 128
 *   n_seq        documents; cu_seqlens[0] = 0, cu_seqlens[n_seq] = T,
 *                non-decreasing (device int32 [n_seq + 1]); an empty document
 *                is allowed.  Batched equal-length input is
 *                {0, L, 2L, ...} ([SUM] §3.6.2: packed documents in place).
 *   causal       1: query i sees keys j <= i of its own document; 0: the whole
 *                document.
 *   exact        1: the exact option ([SUM] §4.5): per-token Q, K and dO
 *                scales, per-(row, 32-key) dS exponents for dQ, deterministic
 *                dQ.  0: token-block scales over 32 document-local tokens.
 *   causal_dq_scale  with dq_fp16: 1 takes the power-of-two prescale of
 *                row i's FP16 dQ partials from keys j <= i only ([SUM] §4.5:
 *                removes the sequence-range dependency of the dQ
 *                accumulator); 0 from the whole document.
 *   dq_fp16      1: the default option's dQ partials (one per 128-key tile)
 *                are prescaled by a power of two per query row, rounded to
 *                FP16 and reduced into an FP16 accumulator ([READ] 四 4.4;
 *                the setting the Python training call uses by default: as
 *                fast as fp32 on short documents, faster on long and packed
 *                ones, where it halves the accumulator's traffic);
 *                0: fp32 partials into an fp32 accumulator.  No effect on the
 *                exact option and the mixed path, whose dQ sums in fp32 in
 *                a fixed order.
 *   deterministic 1: dQ's partials (one per 128-key tile) are added in
 *                key-tile order (a counter per query tile and head orders the
 *                bulk reduce-adds of the CTAs), so dQ is reproducible bit for
 *                bit; FP16 partials with dq_fp16 (then every FP16 addition
 *                happens in the order the per-tile model of [READ] 四 4.4
 *                states), else fp32.
 *   softmax_scale  0 selects 1/sqrt(d).
 *   path         flamia_path_t.
 *   in_dtype     dtype of Q, K, V, dO, O inputs (FLAMIA_BF16 or FLAMIA_F32).
 *   out_dtype    dtype of O, dQ, dK, dV outputs.
 *   bitexp       1: inference forward with bit-level exponentials ([SUM] §3.7
 *                Bit-Level Exponentials for Inference, §4.4): on key pairs 0-4
 *                of every 8 in each 32-key block, 2^z is the bf16 bit-field
 *                approximation 2^floor(z) (1 + frac z), fraction rounded to 7
 *                bits, with a zero-mean shift of 7 units (pattern
 *                RNE(128 z) + 16249, 0 for z <= -126.9453125); the other
 *                pairs use the hardware exponential.  l sums the same values.
 *                MXFP8 path, default option only (else
 *                FLAMIA_ERR_UNSUPPORTED); flamia_bwd rejects it
 *                (FLAMIA_ERR_UNSUPPORTED): the backward must rebuild the
 *                forward's P^ exactly.
 *   hadamard     1: Q and K are rotated by the Sylvester Hadamard matrix H_d
 *                (entries +-1) before quantization ([SUM] §4.3 Ablation Study
 *                and abstract: the fused quantizer's Hadamard rotation;
 *                [READ] 四 4.4: it spreads outlier channels and keeps dot
 *                products).  The rotated values are formed in fp32 by the
 *                fast Walsh-Hadamard transform (stages h = 1, 2, ..., d/2)
 *                inside flamia_quantize, the 1/d of H_d H_d = d I is folded
 *                into the softmax scale, and flamia_bwd rotates dQ and dK
 *                back, so O, dQ, dK, dV keep their meaning.  The Q/K payloads
 *                hold rotated codes.  MXFP8 path only (else
 *                FLAMIA_ERR_UNSUPPORTED); the workspace grows by
 *                4 T Hkv d bytes.
 *   clc          how flamia_fwd and flamia_bwd hand out the longest-first
 *                work items ([SUM] §3.6.2 Load-Balanced Scheduling and
 *                [READ] 四 4.4, GPU-side scheduling: cluster launch control
 *                for skewed and causal calls).  1: the grid has one CTA per
 *                item (item = blockIdx.x, (ceil(T/128) + n_seq) * heads CTAs,
 *                those past the plan's item count exit at once); a CTA that
 *                finishes its item cancels a CTA not yet launched
 *                (clusterlaunchcontrol.try_cancel) and takes that item, and
 *                stops when none is left.  0: a persistent grid of one CTA
 *                per SM takes items from a global counter.  Results are the
 *                same up to the order of the dQ partials' additions.  Not
 *                with the exact or deterministic options
 *                (FLAMIA_ERR_UNSUPPORTED): their ordered dQ reduction waits
 *                on items earlier in the list, which the counter hands out
 *                first and cancellation need not.
 */
typedef struct {
  int32_t T, H, Hkv, d, n_seq;
  const int32_t* cu_seqlens;
  int32_t causal, exact, causal_dq_scale, deterministic;
  float softmax_scale;
  int32_t path, in_dtype, out_dtype;
  int32_t dq_fp16;
  int32_t bitexp;
  int32_t hadamard;
  int32_t clc;
} flamia_problem_t;

/* A quantized operand (device pointers, caller-owned).
 *   codes    uint8 [T][heads][d] E4M3FN codes.  One payload serves both MMA
 *            orientations ([SUM] §3.1).
 *   scales   uint8 [heads][T] UE8M0 exponent byte (e + 127) of each token's
 *            block, replicated per token ([SUM] §3.6.2: per-token scale
 *            metadata).  V always has one exponent per key ([SUM] abstract).
 *   codes4   mixed path, Q and K only: uint8 [T][heads][d/2], two E2M1 codes
 *            per byte, element 2k in the low nibble.
 *   scales4  mixed path, Q and K only: uint8 [T][heads][d/16] E4M3 block scales.
 *   gscale4  mixed path, Q and K only: float [heads][T] per-token fp32 scale.
 *   On the mixed path flamia_fwd and flamia_bwd read codes4 and scales4 of Q
 *   and K directly as the operands of the block-scaled NVFP4 score MMA
 *   ([SUM] §3.4: QK^T and its recompute in NVFP4, one E4M3 scale per 16
 *   head-dimension elements), so they must stay unchanged between the calls.
 * Unused members may be NULL. */
typedef struct {
  void* codes;
  void* scales;
  void* codes4;
  void* scales4;
  void* gscale4;
} flamia_operand_t;

/* Bytes of device workspace needed by plan/quantize/fwd/bwd for `p`
 * (0 if `p` is invalid). */
size_t flamia_workspace_size(const flamia_problem_t* p);

/* Builds, on the GPU, the document tables and the longest-first work lists
 * ([SUM] §3.6.2 and [READ] 4.4: a fixed-pass merge sort on the GPU, once per
 * microbatch, items issued in descending cost to a persistent grid or, with
 * clc, by cluster launch control).  One launch when each list fits one sort
 * block (ceil(T/128) + n_seq <= 2048).
 * Forward items are (document, 128-query tile) with cost = key tiles visited;
 * backward items are (document, 128-key tile) with cost = query tiles
 * visited; ties keep document order.  Reads cu_seqlens on the device only.
 * Also clears the workspace's device status word and test hooks: the status
 * read after flamia_bwd covers one call, plan through backward. */
flamia_status_t flamia_plan(const flamia_problem_t* p, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Fused quantizer ([SUM] §3.1, §3.2; [READ] 4.4 fused quantization).
 * role FLAMIA_ROLE_QKV: in = {Q [T][H][d], K [T][Hkv][d], V [T][Hkv][d]},
 *   out = {Q^, K^, V^} operands.  Q and K: token-block exponent over 32
 *   document-local tokens x d (per token in the exact option); V: per key.
 *   Exponent = smallest e with max|x| <= 448 * 2^e (nothing clamps), clamped
 *   to [-127, 127]; all-zero blocks take e = 0; codes RNE(x * 2^-e).
 *   Mixed path: Q and K also get the NVFP4 payload (codes4/scales4/gscale4).
 * role FLAMIA_ROLE_DO: in = {dO [T][H][d]}, O = the forward output as stored
 *   (out_dtype), out = {dO^}; also writes D (device float [H][T]),
 *   D_i = sum_d dO^_id * O_id from the same dO^ that feeds dP ([SUM] §3.3).
 * Requires flamia_plan on the same workspace. */
flamia_status_t flamia_quantize(const flamia_problem_t* p, int32_t role, const void* const* in, const void* O,
                                const flamia_operand_t* out, float* D, void* ws, size_t ws_bytes,
                                cudaStream_t stream);

/* Forward ([SUM] §3.1–§3.3; [READ] 4.1–4.4): S = Q^ K^T (mixed path:
 * g_Q(i) g_K(j) sum_d (e2m1 s)_Q (e2m1 s)_K from the NVFP4 payload, [SUM]
 * §3.4), online softmax over key tiles with an integer row reference, P^ quantized to E4M3 with one
 * exponent per (row, 32-key block) after the per-key V factor is folded in,
 * O += P^ V^ by a block-scaled MMA, O = acc / l.
 *   O  device [T][H][d] out_dtype
 *   m  device int32 [H][T]: the row's integer reference exponent
 *   l  device float [H][T]: sum_j 2^(x_ij - m_i), x = S * softmax_scale * log2(e)
 * Requires flamia_plan on the same workspace. */
flamia_status_t flamia_fwd(const flamia_problem_t* p, const flamia_operand_t* q, const flamia_operand_t* k,
                           const flamia_operand_t* v, void* O, int32_t* m, float* l, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/* Backward ([SUM] §3.3; [READ] 4.3): recomputes S and P^ from the same Q^/K^
 * with the forward's tiling and exponent evaluation, dP = dO^ V^T,
 * dS = P (dP - D), dS quantized with one exponent per 32x32 block (the exact
 * option: per (row, 32 keys) for dQ), dV += P~^T dO^, dK += dS^T Q^,
 * dQ += dS K^; dK and dV accumulate in fp32; dQ's per-key-tile partials are
 * summed by bulk reduce-adds, in fp32, or (dq_fp16) prescaled by a power of
 * two per query row and summed in FP16 ([READ] 四 4.4); the exact and
 * deterministic options add the partials in key-tile order (the exact
 * option's in fp32); the mixed path takes the same route.
 * GQA sums dK/dV over the group.
 *   dQ device [T][H][d], dK/dV device [T][Hkv][d], out_dtype.
 * D, m, l as produced by flamia_quantize(DO) and flamia_fwd. */
flamia_status_t flamia_bwd(const flamia_problem_t* p, const flamia_operand_t* q, const flamia_operand_t* k,
                           const flamia_operand_t* v, const flamia_operand_t* dO, const float* D, const int32_t* m,
                           const float* l, void* dQ, void* dK, void* dV, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/* Reads and returns the device status word of `ws` (FLAMIA_OK,
 * FLAMIA_ERR_TIMEOUT or FLAMIA_ERR_BAD_SEQLENS).  Synchronises `stream`:
 * for tests and diagnostics, not for the hot path. */
flamia_status_t flamia_get_device_status(const void* ws, cudaStream_t stream);

/* Clears the device status word (stream-ordered, no synchronisation). */
flamia_status_t flamia_clear_device_status(void* ws, cudaStream_t stream);

/* Test hook (not for the hot path): make the next flamia_fwd / flamia_bwd
 * calls on workspace `ws` record, for every (query head h, query token i,
 * key token j) they evaluate, the P^ code in codes[(h*T + i)*T + j] (device
 * uint8 [H][T][T]) and each 32-key block's exponent in
 * exps[(h*T + i)*T + j0] at the block's first key j0 (device int32 [H][T][T]).
 * Both kernels write the P^ they use, so a caller can check that the backward
 * rebuilds the forward's P^ bit for bit ([SUM] §3.3).  NULL, NULL switches the
 * hook off.  Must be called after flamia_plan (which does not touch it) and
 * synchronises `stream`. */
flamia_status_t flamia_debug_set_phat_dump(void* ws, size_t ws_bytes, void* codes, int32_t* exps,
                                           cudaStream_t stream);

/* Regions of the workspace that tests read back (flamia_debug_workspace_offset). */
typedef enum {
  FLAMIA_WS_FWD_ITEMS = 0,    /* int32 pairs (document, 128-query tile), longest first */
  FLAMIA_WS_BWD_ITEMS = 1,    /* int32 pairs (document, 128-key tile), longest first */
  FLAMIA_WS_DQ_PRESCALE = 2   /* int8 [H][T]: exponent p of the FP16 dQ partials' prescale 2^p */
} flamia_ws_region_t;

/* Test hook: byte offset of a region inside the workspace of problem `p`
 * (0 for an invalid problem or region).  The dQ prescale exponents are
 * written by flamia_bwd on the dq_fp16 path. */
size_t flamia_debug_workspace_offset(const flamia_problem_t* p, int32_t region);

/* Test hook (not for the hot path): exercise the bounded waits.  While on,
 * each CTA of the next flamia_fwd / flamia_bwd launches withholds its first
 * work item, so its other roles' waits for that item run out after the
 * bounded-wait limit (about 2 s): the kernel records FLAMIA_ERR_TIMEOUT in the
 * device status word, every role leaves its loop and the CTA releases its
 * tensor memory and exits (nothing was issued, so no copy or MMA is in
 * flight).  The outputs of such a call are undefined.  Of flamia_paged_plan_shared
 * and flamia_paged_compact a CTA stays away from the last of the launch's
 * barriers over its CTAs, whose wait runs out likewise (about 2 s): no
 * page moves.  Process-wide (not per
 * workspace); flamia_plan switches it off.  Always returns FLAMIA_OK. */
flamia_status_t flamia_debug_withhold_first_item(int32_t on);

/* Test hooks (no device call): the tensor-core descriptors the kernels issue,
 * as the library's own builders encode them, so that a host test can check
 * each bit field against the field tables of the PTX ISA's tcgen05
 * "Instruction descriptor" and "Shared memory descriptor" sections.
 *
 * flamia_debug_mma_idesc: the 32-bit instruction descriptor of one
 *   tcgen05.mma of kind
 *     FLAMIA_MMA_F8F6F4   kind::f8f6f4, E4M3 x E4M3, fp32 accumulator;
 *     FLAMIA_MMA_MXF8F6F4 kind::mxf8f6f4.block_scale.scale_vec::1X, E4M3
 *                         operands, UE8M0 scales (one per 32 K-elements);
 *     FLAMIA_MMA_MXF4NVF4 kind::mxf4nvf4.block_scale.scale_vec::4X, E2M1
 *                         operands, UE4M3 scales (one per 16 K-elements);
 *     FLAMIA_MMA_BF16     kind::f16, BF16 x BF16, fp32 accumulator;
 *     FLAMIA_MMA_F16      kind::f16, F16 x F16, fp32 accumulator;
 *   for an M x N tile (cta_group::1: M = 64 with N a multiple of 8, or
 *   M = 128 with N a multiple of 16; 8 or 16 <= N <= 256).  a_mn / b_mn = 1
 *   selects an MN-major operand (0 or 1; 0 for the E2M1 kind), a_sf_id /
 *   b_sf_id the scale-factor ids of the block-scaled kinds (0..3; 0 for the
 *   E2M1 kind, 0 for kind::f8f6f4 and kind::f16).  Writes *out and returns FLAMIA_OK;
 *   FLAMIA_ERR_INVALID_ARG for a NULL out or an argument outside these
 *   ranges (then *out is untouched).
 * flamia_debug_smem_desc: the 64-bit shared-memory matrix descriptor for a
 *   tile at shared address saddr with leading- and stride-dimension byte
 *   offsets lbo / sbo (all multiples of 16 below 2^18) and swizzle mode
 *   FLAMIA_SWZ_NONE / _128B / _64B / _32B.  Same return rules. */
typedef enum {
  FLAMIA_MMA_F8F6F4 = 0,
  FLAMIA_MMA_MXF8F6F4 = 1,
  FLAMIA_MMA_MXF4NVF4 = 2,
  FLAMIA_MMA_BF16 = 4, /* the paged chunk kernel's */
  FLAMIA_MMA_F16 = 5   /* and its E2M1 tiles' */
} flamia_mma_kind_t;
typedef enum { FLAMIA_SWZ_NONE = 0, FLAMIA_SWZ_128B = 2, FLAMIA_SWZ_64B = 4, FLAMIA_SWZ_32B = 6 } flamia_swizzle_t;
flamia_status_t flamia_debug_mma_idesc(int32_t kind, uint32_t M, uint32_t N, int32_t a_mn, int32_t b_mn,
                                       int32_t a_sf_id, int32_t b_sf_id, uint32_t* out);
flamia_status_t flamia_debug_smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, int32_t swizzle,
                                       uint64_t* out);

/* Allocation-free work-list builder (this library's own addition; the
 * method's pages have no counterpart).  For callers that cannot allocate
 * device memory: code inside a CUDA graph under capture (cudaMalloc cannot be
 * captured), embeddings without an allocator, or frameworks that forbid
 * allocations outside their own caching allocator.  It builds the same two
 * longest-first work lists as flamia_plan, but its scratch (document
 * prefix tables, sort keys) lives in a file-scope device array of the library
 * (about 2.5 MiB, held by every GPU that loads the library until the process
 * exits) instead of a caller workspace; it calls no allocating routine.
 *   fwd_items, bwd_items  device int32 pairs (document, 128-token tile),
 *                         each [ceil(T/128) + n_seq] entries, caller-owned;
 *                         the first *n_items entries are written.
 *   n_items               device int32, receives the number of tiles (0 when
 *                         cu_seqlens is inconsistent with T).
 * Limits: ceil(T/128) + n_seq <= 65536 and n_seq <= 65536, else
 * FLAMIA_ERR_UNSUPPORTED.  The first call on each device looks up the array's
 * device address with that device current (make that first call before any
 * stream capture) and keeps it for the life of the process, so the entry
 * point must not be used on a device after cudaDeviceReset.  All calls share
 * the array and it keeps the last call's
 * contents: calls whose kernels may overlap on the GPU race with each other
 * and must be serialised by the caller. */
flamia_status_t flamia_plan_noalloc(const flamia_problem_t* p, int2* fwd_items, int2* bwd_items, int32_t* n_items,
                                    cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Serving from a paged key/value cache (this library's own addition; the
 * method's pages stop at the training call and the inference exponential).
 *
 * One serving step is, on one CUDA stream:
 *   flamia_paged_plan    once per step: pages, slots and the attention's work split
 *   per layer:
 *     flamia_paged_append  this step's K and V rows into the layer's cache
 *     flamia_paged_fwd     attention of this step's queries over the cache
 *
 * The cache of a layer is a pool of pages; a page holds `page_size`
 * consecutive tokens of one request for all key/value heads, head-major, so
 * that one head's tokens of a page are one contiguous run:
 *   K, V codes  [n_pages][Hkv][page_size][d]   bf16 or E4M3; E2M1:
 *               [n_pages][Hkv][page_size][d/2], two codes a byte, channel 2k in
 *               the low nibble (as flamia_operand_t's codes4)
 *   scales      [n_pages][Hkv][page_size]      E4M3 and E2M1: the UE8M0 byte of
 *               each (token, head) row, as flamia_quantize's exact option
 *               writes them for E4M3: the row's value is code * 2^(byte - 127).
 *               Byte 255 marks a row that holds a NaN or an infinity: all of it
 *               reads as NaN.  (A NaN code 0x7F or 0xFF under any other byte is
 *               not written by flamia_paged_append and must not occur.)
 *   blocks      [n_pages][Hkv][page_size][d/16]  E2M1 only: the E4M3 scale of
 *               each 16 channels of a row, not negative and (but under byte
 *               255) not the NaN code 0x7F: the value is
 *               code * block scale * 2^(byte - 127).  The exponent is a power of
 *               two, unlike gscale4 of flamia_operand_t, so that a value keeps
 *               at most six significant bits and is exact in bf16 and f16.
 * Token j of request r lies in page block_table[r][j / page_size], row
 * j % page_size; its slot is page * page_size + row.
 *
 * Problem description (host struct; pointers are device pointers).
 *   n_req        requests of the step, 1..8192
 *   T            rows of the packed per-token tensors (capacity).  Request r
 *                owns the rows [cu_q[r], cu_q[r+1]) of q, k, v, O and the slot
 *                map, all of which have T rows; rows behind cu_q[n_req] <= T
 *                belong to no request: what they hold does not matter, and
 *                they are not written (their slots are set to -1).
 *   max_q        upper bound of a request's new tokens, 1..T (0 selects T).  The
 *                kernel is chosen by it: up to max_q * H / Hkv = 32 rows a
 *                (request, key/value head) take the decode kernel.
 *   H, Hkv, d    query heads, key/value heads (H % Hkv == 0, H / Hkv <= 128),
 *                head dimension 64 or 128
 *   page_size    16, 32, 64 or 128
 *   n_pages      pages of the pool; n_pages * page_size < 2^31
 *   max_pages    columns of the block table; max_pages * page_size <= 2^30
 *                (2^25 where max_q * H / Hkv > 32)
 *   cache_dtype  FLAMIA_BF16, FLAMIA_E4M3 or FLAMIA_E2M1 (4 bits a value)
 *   in_dtype     dtype of the K and V rows given to flamia_paged_append:
 *                FLAMIA_BF16 or FLAMIA_F32
 *   causal       1: new token i of a request, at position kv_len - q_len + i,
 *                sees the keys up to its own position; 0: all kv_len keys
 *   softmax_scale  0 selects 1/sqrt(d)
 *   cu_q         int32 [n_req + 1], cu_q[0] = 0, non-decreasing
 *   kv_len       int32 [n_req]: the request's cached tokens after this step,
 *                its new ones included.  A request may have new tokens and
 *                kv_len 0 (an inactive slot of a captured batch), or fewer
 *                cached than new ones: rows without a key get O = 0 and
 *                lse = -inf, and slot -1.
 *   block_table  int32 [n_req][max_pages]; entries past a request's pages
 *                are not read
 *   q_stride, kv_stride  elements between two tokens' rows of q (and of k and
 *                v): 0 selects contiguous rows (H * d, Hkv * d); otherwise at
 *                least that, and a multiple of 16 bytes, so rows of a fused
 *                QKV projection can be passed in place
 * Conventions as above (16-byte alignment; the int32 arrays 4-byte).  cu_q,
 * kv_len and block_table must not change between flamia_paged_plan and the
 * last launch that uses its workspace.  One workspace serves one step at a
 * time: launches that may overlap (other streams, other graphs) need one each.
 * A launch whose workspace was not planned for the same sizes (everything
 * above but the dtypes, the scale, the strides and the pointers) writes nothing
 * and sets FLAMIA_ERR_INVALID_ARG.  The stream's device must be the current one. */
typedef struct {
  int32_t n_req, T, max_q, H, Hkv, d;
  int32_t page_size, n_pages, max_pages;
  int32_t cache_dtype, in_dtype, causal;
  float softmax_scale;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int32_t* block_table;
  int64_t q_stride, kv_stride;
} flamia_paged_t;

/* One layer's cache (device pointers, caller-owned; k_scales and v_scales
 * are NULL for bf16, k_blocks and v_blocks read for E2M1 only).  page_stride:
 * elements between two pages of k and of v (0: Hkv * page_size * d, contiguous;
 * else at least that, a multiple of 16 bytes), so that K and V pages can be
 * interleaved in one buffer. */
typedef struct {
  void* k;
  void* v;
  void* k_scales;
  void* v_scales;
  int64_t page_stride;
  void* k_blocks;
  void* v_blocks;
} flamia_cache_t;

/* Bytes of device workspace for `p` (0 if `p` is invalid). */
size_t flamia_paged_workspace_size(const flamia_paged_t* p);

/* Builds, in one launch, the step's block tables, slot map and attention
 * work split from the request lengths.  Clears the workspace's status word.
 *
 * Page management (old_len not NULL): request r held ceil(old_len[r] /
 * page_size) pages and needs ceil(kv_len[r] / page_size).  With
 * S = free_pages[0 .. *n_free) followed by the pages that shrinking requests
 * give back (request order, then table order), growing requests take pages
 * from the end of S (request order, then table order) and their new table
 * entries are written; what is left of S stays in free_pages and its length
 * goes to *n_free_out.  So a finished request passes kv_len 0, one whose
 * drafted tokens were rejected a smaller kv_len.  Pages must belong to one
 * request only (flamia_paged_plan_shared: to several).  Table entries outside
 * the taken pages are not written.
 *   old_len     int32 [n_req]
 *   free_pages  int32 [n_pages] stack of free page ids
 *   n_free, n_free_out  int32 [1]; may be the same word
 * If old_len is NULL, so must these three be: the table is used as it is.
 *
 * slot_map (may be NULL): int32 [T], the slot of each new token, -1 for rows
 * behind cu_q[n_req] and for positions below 0.
 *
 * Device-side conditions, all checked before anything is written:
 * FLAMIA_ERR_BAD_SEQLENS (cu_q, old_len or kv_len inconsistent, more than
 * max_q new tokens or more than max_pages pages), FLAMIA_ERR_BAD_PAGE (*n_free
 * outside [0, n_pages], or more pages given back than the stack has room
 * for), FLAMIA_ERR_NO_PAGES (fewer pages than the step needs),
 * FLAMIA_ERR_UNSUPPORTED (more attention than the work split counts: a
 * request's tiles of 256 rows of one key/value head times the blocks of 128
 * keys of its last tile above 2^31, or their sum over requests and heads above
 * 2^38, with two blocks more for each tile).  Then no page
 * moves, *n_free_out = *n_free, every slot is -1, and launches that use the
 * workspace write nothing.  A new token whose page id (of the table or the
 * stack) lies outside [0, n_pages) gets slot -2, which flamia_paged_append
 * reports. */
flamia_status_t flamia_paged_plan(const flamia_paged_t* p, int32_t* slot_map, const int32_t* old_len,
                                  int32_t* free_pages, const int32_t* n_free, int32_t* n_free_out, void* ws,
                                  size_t ws_bytes, cudaStream_t stream);

/* ---- Pages that requests share -------------------------------------------
 * One prompt's pages can serve many requests (answers sampled in parallel, the
 * beams of a beam search, cached prompts): their table entries name the same
 * page, and refs[page] counts them.  A step is then
 *   flamia_paged_plan_shared   in place of flamia_paged_plan
 *   flamia_paged_copy          its list of copies, in every layer
 *   per layer: append and attention as before.
 * These calls take a second workspace, `pages_ws` of
 * flamia_paged_pages_workspace_size bytes, which need not be initialised and
 * keeps nothing from call to call but its status word (flamia_paged_copy only
 * adds to that one).  One call at a time. */
size_t flamia_paged_pages_workspace_size(const flamia_paged_t* p);

/* The page management of a step whose requests may share pages, then what
 * flamia_paged_plan does with old_len NULL (slot map, work split).
 *   src       int32 [n_req] (may be NULL: src[r] = r): the request, as it was
 *             before the step, that request r continues; -1: none, it starts
 *             empty.  Several may continue one (a fork); a request that none
 *             continues ends.
 *   old_len   int32 [n_req]: tokens that the rows of block_table hold before
 *   refs      int32 [n_pages]: table entries that hold each page, plus holders
 *             that the caller counts beside the tables (such a page is neither
 *             freed nor written); 0 for free pages
 *   free_pages, n_free, n_free_out   as in flamia_paged_plan
 *   copies    int32 [n_req][2], n_copies int32 [1]: pages to copy in every
 *             layer before anything is appended, (source, destination).  No
 *             destination is a source.
 * With p the page size, q_r = cu_q[r+1] - cu_q[r] and w_r = max(0, kv_len[r] -
 * q_r) the tokens that request r keeps, its row gets the first
 *   keep_r = min(ceil(old_len[src[r]] / p), ceil(w_r / p))
 * entries of row src[r] as it was (0 for src[r] = -1).  Let total be each
 * page's count once every row holds these and no others.
 *   - A page of the old rows whose total is 0 goes onto the free stack, in the
 *     order of the old entries (row, then table order) that held it first.
 *   - Request r writes into entry w_r / p if q_r > 0, w_r < kv_len[r], w_r is
 *     no multiple of p and w_r / p < keep_r.  If that page has other holders
 *     than writers, each of its writers gets a new page in its place and a
 *     line in `copies` (in request order); if all its holders write, the first
 *     of them keeps it.
 *   - New pages come off the end of the stack in request order, table order:
 *     copies, and entries keep_r .. ceil(kv_len[r] / p) - 1.
 * Table entries from ceil(kv_len[r] / p) on are left as they were.  A page
 * must not occur twice in a row.
 * Device-side conditions, all checked before anything is written (in both
 * workspaces' status words): FLAMIA_ERR_BAD_SEQLENS (as in flamia_paged_plan;
 * src outside [-1, n_req)), FLAMIA_ERR_BAD_PAGE (*n_free out of range, a table
 * entry that the step reads or a free page that it may take, if every writer
 * takes a copy, outside [0, n_pages), counts below the entries that it sees,
 * more pages freed than the stack has room for),
 * FLAMIA_ERR_NO_PAGES.  Then nothing moves, *n_free_out = *n_free, *n_copies =
 * 0, every slot is -1, and launches that use `ws` write nothing.  So too after
 * FLAMIA_ERR_TIMEOUT (a CTA did not come to one of the launch's barriers).
 * FLAMIA_ERR_UNSUPPORTED (from the host) where the sizes allow a step that
 * flamia_paged_plan would refuse with it. */
flamia_status_t flamia_paged_plan_shared(const flamia_paged_t* p, int32_t* slot_map, const int32_t* src,
                                         const int32_t* old_len, int32_t* refs, int32_t* free_pages, const int32_t* n_free,
                                         int32_t* n_free_out, int32_t* copies, int32_t* n_copies, void* pages_ws,
                                         size_t pages_ws_bytes, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Copies pages in n_layers layers: for each of the first *n_copies (source,
 * destination) pairs of `copies` (int32 [max_copies][2]), page `source` of
 * src[l] to page `destination` of dst[l], whole, with its scales.  src and dst
 * are host arrays of n_layers caches and may be the same; of `p` Hkv, d,
 * page_size, n_pages and cache_dtype count.  No destination may be a source of
 * the same pool, nor occur twice.  *n_copies outside [0, max_copies] copies
 * nothing and sets FLAMIA_ERR_INVALID_ARG, a page outside [0, n_pages) skips
 * its pair and sets FLAMIA_ERR_BAD_PAGE (in pages_ws). */
flamia_status_t flamia_paged_copy(const flamia_paged_t* p, int32_t n_layers, const flamia_cache_t* src,
                                  const flamia_cache_t* dst, const int32_t* copies, int32_t max_copies,
                                  const int32_t* n_copies, void* pages_ws, size_t pages_ws_bytes, cudaStream_t stream);

/* Compacts the pool: with U = n_pages - *n_free pages in use, the k-th page in
 * use with an id >= U goes to the k-th free id < U, so that ids 0 .. U - 1 are
 * in use and the pool can be cut there.  Rewrites the entries of block_table
 * (request r holds ceil(len[r] / page_size); len int32 [n_req]), moves the
 * counts (refs may be NULL), sets free_pages[i] = n_pages - 1 - i for i <
 * *n_free, and writes the moves to copies (int32 [n_pages][2], 8-byte aligned)
 * and *n_copies for flamia_paged_copy, which must run before the pages are
 * used.  They are also the new ids of pages held beside the tables.
 * Conditions, checked before anything is written but `copies` (in pages_ws):
 * FLAMIA_ERR_BAD_SEQLENS (len), FLAMIA_ERR_BAD_PAGE (*n_free out of range, a
 * free page out of range or twice on the stack, a table entry out of range or
 * on the stack).  Then, and after FLAMIA_ERR_TIMEOUT, nothing moves and *n_copies
 * = 0. */
flamia_status_t flamia_paged_compact(const flamia_paged_t* p, const int32_t* len, int32_t* refs, int32_t* free_pages,
                                     const int32_t* n_free, int32_t* copies, int32_t* n_copies, void* pages_ws,
                                     size_t pages_ws_bytes, cudaStream_t stream);

/* Writes the step's K and V rows (in_dtype, [T][Hkv][d], kv_stride) into
 * their slots: rounded to bf16, or as E4M3 codes with the row's no-clamp
 * exponent (the smallest e with max|x| <= 448 2^e, clamped to [-127, 127]; 0
 * for a zero row), byte for byte those of flamia_quantize with `exact` for
 * finite rows; or as E2M1 codes: e is the smallest exponent with max|x| <=
 * 2688 2^e (2688 = 6 * 448; clamped alike, 0 for a zero row), a block scale s
 * the smallest E4M3 value with 6 s 2^e >= its 16 channels' max|x|, a code
 * RNE(x 2^-e / s) (0 where s is 0), of the exact quotient (values of a row
 * above 3.3e38 may so pass 2^128).  A slot of -1 skips the row; slots must be
 * distinct.  Any other slot outside the pool is skipped and sets
 * FLAMIA_ERR_BAD_PAGE.  Requires flamia_paged_plan on the same workspace. */
flamia_status_t flamia_paged_append(const flamia_paged_t* p, const void* k, const void* v, const int32_t* slot_map,
                                    const flamia_cache_t* cache, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Attention of the step's queries over the cache: with x_ij = softmax_scale
 * <q_i, k_j> over the keys j that row i sees,
 *   O_i = sum_j exp(x_ij - lse_i) v_j,   lse_i = ln sum_j exp(x_ij).
 * Query head h reads key/value head h / (H / Hkv).  Scores, softmax
 * statistics and accumulators are fp32.  Rounding of the weights for the P V
 * product, relative to each:
 *   chunk kernel                  bf16, 2^-8
 *   chunk kernel, E2M1            f16, 2^-11, and below that at most 2^-32 of
 *                                 the row's largest weight; bf16 in blocks of
 *                                 128 keys where a V row's scale byte is not
 *                                 112 to 127, and from one with a byte of 192
 *                                 or more (V of 2^66 or more) on for the rest
 *                                 of the tile, where V is exact down to 2^-118
 *   decode kernel, bf16 cache     two bf16 terms, 2^-16
 *   decode kernel, E4M3 or E2M1   f16, 2^-11, and below that at most 2^-20 of
 *                                 the row's largest weight; two bf16 terms
 *                                 where the scale bytes of the V rows that a
 *                                 warp takes lie more than 12 apart (E2M1,
 *                                 with a byte of 192 or more among them: V is
 *                                 exact down to 2^-102)
 * Keys that a row does not see, and what slots behind a request's last token
 * hold, change no row's precision beyond that.  Ranges: scores over a cache of
 * codes are formed from queries scaled to 2^13 and may overflow from K rows of
 * 2^116 on; sums of weights (at most 2^8 of the first ones) times V are fp32,
 * over E2M1 with V of 2^66 and more in units in which V of any size fits.  A
 * value of 2^128 of an E4M3 row counts as bf16's largest number.
 *   q    device bf16 [T][H][d] (q_stride)
 *   O    device bf16 [T][H][d], contiguous
 *   lse  device float [H][T], natural logarithm (may be NULL)
 * O must not overlap q or the cache.
 * A table entry outside [0, n_pages) sets FLAMIA_ERR_BAD_PAGE and leaves the
 * request's O and lse undefined; nothing outside the pool is read.  Requires
 * flamia_paged_plan on the same workspace; results do not depend on anything
 * else the workspace held. */
flamia_status_t flamia_paged_fwd(const flamia_paged_t* p, const void* q, const flamia_cache_t* cache, void* O,
                                 float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Static description of a status code. */
const char* flamia_status_string(flamia_status_t s);

#ifdef __cplusplus
}
#endif
#endif /* FLAMIA_H_ */
