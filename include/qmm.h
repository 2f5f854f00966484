/*
 * qmm.h -- C ABI of libqmm: block-quantized weight x q8_1 activation products on MI355X (gfx950).
 *
 * Sources (cited by page title and section):
 *   [PF] #2356 "pf_wmma: a second Volta prompt-expert kernel for IQ2_S gate/up and IQ4_NL down"
 *   [DQ] #1525 "prefill: dense IQ4_XS / Q8_0 to FP16 with 16-byte stores, swiglu + q8_1 and the
 *        MoE combine + hyper-connection write fused"
 *   [IQ] #242  "IQ kernels: decode each weight part once for every column and entry, bitwise identical"
 *   [GP] #1424 "Pascal GP100: a Q8_0 decode GEMV ... and IQ3_XXS / IQ3_S tables in shared memory"
 *
 * General rules for every entry point:
 *   - All pointers are DEVICE pointers unless a comment says "host".  The caller owns every
 *     buffer; the library allocates nothing and keeps no state between calls (reentrant),
 *     except where an entry point says otherwise (qmm_planes_alloc owns a packed copy until
 *     qmm_planes_release).
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).  Calls are
 *     asynchronous on that stream; outputs are ready when the stream reaches the call.
 *   - Argument errors are reported synchronously by the return value, before anything is
 *     launched; a launch error is reported as QMM_EHIP.  Faults inside a kernel surface at the
 *     caller's next synchronisation.
 *   - Weight formats (little-endian, every block starts with its fp16 scale d):
 *       QMM_Q8_0   34 B per 32 values : d, int8 q[32]                    value = d*q
 *       QMM_IQ4_NL 18 B per 32 values : d, 16 bytes of 4-bit indices into the sixteen IQ4_NL
 *                                       levels; value j<16 = low nibble of byte j, j>=16 = high
 *                                       nibble of byte j-16                value = d*level
 *       QMM_CB3   110 B per 256 values: d, qs[64], qh[8], signs[32], scales[4] (IQ3_S-like
 *                                       codebook: 9-bit index = qs[i] | bit i%8 of qh[i/8] << 8
 *                                       selects 4 magnitudes from `grid`; sign bit v%8 of
 *                                       signs[v/8]; sub-block s of 32 values has multiplier
 *                                       1 + 2*((scales[s/2] >> 4*(s%2)) & 15))
 *     A weight matrix is row-major: nrows rows of qmm_row_bytes(wtype, k) bytes each.
 *     `grid` (CB3 only) is 512 entries x 4 uint8 magnitudes (2048 bytes), each in [1, 63].
 *   - q8_1 activations: 36 B per 32 values = fp16 d, fp16 s, int8 q[32]; a column of k values
 *     is k/32 consecutive blocks, columns are consecutive ([ncols][k/32][36]).
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* weight formats */
#define QMM_Q8_0 1
#define QMM_IQ4_NL 2
#define QMM_CB3 3
#define QMM_F16 4 /* binary16 weights [rows][k] (qgemm_dense only): 2 bytes per value */

/* status codes */
#define QMM_OK 0
#define QMM_EINVAL (-1)       /* bad argument: null pointer, size out of range, ... */
#define QMM_EUNSUPPORTED (-2) /* a shape or format the kernels decline (caller keeps another path) */
#define QMM_EALIGN (-3)       /* a pointer or stride is not aligned as documented */
#define QMM_EHIP (-4)         /* the HIP runtime reported an error at launch */
#define QMM_ESPACE (-5)       /* workspace smaller than the *_workspace() query returned */

/* value types of the tensors of qmm_rmsnorm, qmm_dequantize_q8_1, qmm_moe_route, qmm_lora and qmm_kv_* */
#define QMM_TYPE_F32 1
#define QMM_TYPE_F16 2  /* binary16 */
#define QMM_TYPE_BF16 3 /* bfloat16 */

/* scores of qmm_moe_route */
#define QMM_SCORE_SOFTMAX 0
#define QMM_SCORE_SIGMOID 1

/* flags */
#define QMM_FLAG_DEBUG_INTERMEDIATES 1u /* also write fp32 intermediates into the workspace */

/* Version of this ABI (major*100 + minor). */
int qmm_version(void);

/* Host-only.  Human-readable text of a status code (never NULL). */
const char* qmm_status_str(int status);

/* Host-only.  Bytes of one weight row of k values, or 0 when k is not a positive multiple of
 * the format's block (32 values; 256 for CB3; 1 for QMM_F16) or wtype is unknown. */
int64_t qmm_row_bytes(int wtype, int64_t k);

/* q8_1 quantization of activations [DQ, Change: the q8_1 quantizer's 32-value blocks; GP, What
 * changed: q8_1 activations].  Per 32-value block: amax = max |x|; d = amax/127 (binary32);
 * q_j = x_j/d (binary32 division) rounded half away from zero; an all-zero block gives
 * d = q = s = 0; stored d = fp16(d), s = fp16(d * sum q).
 *   x   : float [ncols][ldx], column c's k values at x + c*ldx; ldx >= k; 4-byte aligned.
 *   xq  : output, ncols*(k/32)*36 bytes, 4-byte aligned.
 *   k   : multiple of 32, > 0.  ncols >= 1.
 * Errors: QMM_EINVAL (null, k, ncols, ldx), QMM_EALIGN. */
int qmm_quantize_q8_1(const float* x, int64_t k, int ncols, int64_t ldx, void* xq, void* stream);

/* FP16 dequantization [DQ, Change: dequant to FP16 with 16-byte stores; PF, Summary: the FP16
 * weights the tensor cores get].  out[r*ld + j] = binary16 nearest-even rounding of the exact
 * value of weight (r, j); columns k..ld-1 are not written.
 *   w    : nrows * qmm_row_bytes(wtype, k) bytes, 2-byte aligned.
 *   grid : CB3 codebook (2048 bytes), ignored (may be NULL) for other formats.
 *   out  : uint16 (binary16 bits) [nrows][ld], ld >= k, 2-byte aligned.  When out is 16-byte
 *          aligned and ld % 8 == 0 every thread writes 8 values with one 16-byte store.
 * Errors: QMM_EINVAL, QMM_EALIGN. */
int qmm_dequant_f16(int wtype, const void* w, const uint8_t* grid, int64_t nrows, int64_t k,
                    uint16_t* out, int64_t ld, void* stream);

/* Dense multi-column decode GEMV [IQ, What it does: the weight side is loaded and decoded once
 * and applied to every column, 1/2/4/8 columns per pass, 8 at a time beyond 8; GP, What
 * changed: 16-byte weight loads, activations staged once per workgroup].
 *   y[c*ldy + r] = sum over 32-value blocks b of  (d_w(r,b) * d_a(c,b)) * isum(r,b,c)
 * in binary32, isum the exact integer dot of the block's integer weight factors with the q8_1
 * int8 values (for CB3 the sub-block multiplier is folded into isum).  Every column of an
 * n-column call is bitwise equal to a one-column call on that column.
 *   w    : nrows x qmm_row_bytes(wtype, k) bytes, 4-byte aligned.
 *   grid : CB3 codebook or NULL.
 *   xq   : q8_1 [ncols][k/32][36], 4-byte aligned.   y: float, ldy >= nrows, 4-byte aligned.
 *   k    : multiple of 32 (of 256 for CB3), at most 32768.  ncols >= 1 (any count; passes
 *          of 8).
 * Errors: QMM_EINVAL (k not a multiple of 32 / 256, no rows or columns), QMM_EALIGN,
 *         QMM_EUNSUPPORTED (k above 32768, a buffer of 4 GiB or more). */
int qgemv_dense(int wtype, const void* w, const uint8_t* grid, int64_t nrows, int64_t k,
                const void* xq, int ncols, float* y, int64_t ldy, void* stream);

/* Decode GEMV on 1, 2 or 4 fp32 activation columns, quantized to q8_1 inside the kernel [IQ,
 * What it does: decode GEMV on q8_1 activations; DQ, Change: the q8_1 quantizer]: y equals
 * qgemv_dense(wtype, w, grid, nrows, k, qmm_quantize_q8_1(x), ncols, y, ldy) bit for bit, in
 * one launch instead of two (every workgroup quantizes the columns for itself; the q8_1 bytes
 * are not written out).
 *   w, grid : as qgemv_dense.   x: float [ncols][k], 4-byte aligned.
 *   y    : float, y[c*ldy + r], ldy >= nrows, 4-byte aligned.
 *   k    : multiple of 32 (of 256 for CB3), at most 3072 (rows of at most 96 blocks).
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED (ncols other than 1, 2, 4; k above 3072; a
 *         weight buffer of 4 GiB or more). */
int qgemv_dense_f32(int wtype, const void* w, const uint8_t* grid, int64_t nrows, int64_t k,
                    const float* x, int ncols, float* y, int64_t ldy, void* stream);

/* Test hook: the per-block integer sums isum(r, b, c) of qgemv_dense, computed by the same
 * device decode and dot code.  sums: int32 [ncols][nrows][k/32].  Same argument rules as
 * qgemv_dense. */
int qmm_debug_block_sums(int wtype, const void* w, const uint8_t* grid, int64_t nrows, int64_t k,
                         const void* xq, int ncols, int32_t* sums, void* stream);

/* Measurement hook: a plain streaming read of nbytes from p in one launch of `grid` workgroups
 * of `threads` threads (256, 512 or 1024): workgroup w reads the w-th of grid contiguous runs,
 * `unroll` (4, 8 or 16) 16-byte raw-buffer loads in flight per thread, no other work.  The
 * reference for the HBM time of the decode kernels at the same byte count.  Thread t of
 * workgroup w writes the XOR of the words it read to out[w * threads + t].
 *   p    : device, 16-byte aligned; nbytes a multiple of 16, below 4 GiB.
 *   out  : device uint32 [grid * threads], 4-byte aligned.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED (other threads / unroll), QMM_EHIP. */
int qmm_debug_stream_read(const void* p, uint64_t nbytes, uint32_t* out, int grid, int threads,
                          int unroll, void* stream);

/* Measurement hook: `grid` workgroups of 256 threads, each wave running 8 independent fp16 MFMA
 * accumulators (v_mfma_f32_32x32x16_f16, 32768 FLOP each) for `iters` rounds from registers
 * only: grid * 4 * 8 * iters * 32768 FLOP, the reference for the prefill GEMM's MFMA rate.
 *   out : device float [grid * 256] (the lanes' accumulator sums), 4-byte aligned.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EHIP. */
int qmm_debug_mfma_loop(float* out, int grid, int iters, void* stream);

/* Workspace bytes qgemv_grouped_experts needs (host). */
size_t qgemv_grouped_experts_workspace(int64_t inter, int nentries, unsigned flags);

/* Grouped MoE-expert decode [IQ, What it does: native_gu / native_down decode each weight part
 * once for every entry of a group; DQ, Change: swiglu then q8_1 of H for the down product].
 * Groups are experts; entries are the (token, slot) pairs routed to them.  For group g (expert
 * e = group_expert[g]) and every entry j in [group_entry_off[g], group_entry_off[g+1]):
 *   x  = q8_1 column entry_col[j] of xq (width hidden)
 *   gv = W_gate[e] x,  uv = W_up[e] x          (qgemv_dense arithmetic, inter rows)
 *   h  = silu(gv) * uv,  silu(z) = z / (1 + exp(-z)) in binary32 (device expf, <= 1 ulp;
 *        IEEE division)
 *   H  = q8_1(h) per 32 consecutive intermediate values          (workspace)
 *   y[j*hidden + r] = (W_down[e] H)[r]                            (binary32; unweighted)
 *   w_gate, w_up : expert e's matrix at byte offset e*gu_expert_stride, inter rows of width
 *                  hidden, format wtype_gu;  w_down: offset e*down_expert_stride, hidden rows of
 *                  width inter, format wtype_down; nexperts matrices each.  4-byte aligned;
 *                  strides multiples of 4 and at least one matrix.
 *   xq, xq_cols  : q8_1 activations [xq_cols][hidden/32][36]; an entry whose column is outside
 *                  [0, xq_cols) reads zeros.
 *   group_expert[ngroups], group_entry_off[ngroups+1], entry_col[nentries]: int32, device.
 *                  A group whose expert is outside [0, nexperts) is skipped; its entry range is
 *                  clamped to [0, nentries).  Entries of no group are not written.
 *   ws   : workspace of qgemv_grouped_experts_workspace() bytes, 16-byte aligned.  Layout:
 *          H q8_1 [nentries][inter/32][36] first; with QMM_FLAG_DEBUG_INTERMEDIATES then gv, uv
 *          as float [nentries][inter] (starting at the next 16-byte boundary).
 *   hidden, inter: multiples of 32 (256 where the format is CB3); a pass of 8 entries must fit
 *          the workgroup's 64 KiB of LDS (hidden, inter <= 6144 in practice).
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_ESPACE. */
int qgemv_grouped_experts(int wtype_gu, const void* w_gate, const void* w_up,
                          int64_t gu_expert_stride, int wtype_down, const void* w_down,
                          int64_t down_expert_stride, int nexperts, const uint8_t* grid,
                          int64_t hidden, int64_t inter, const void* xq, int xq_cols,
                          const int32_t* group_expert, const int32_t* group_entry_off, int ngroups,
                          const int32_t* entry_col, int nentries, float* y, void* ws,
                          size_t ws_bytes, unsigned flags, void* stream);

/* Allocation-free grouped decode, for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).  Computes exactly
 * what qgemv_grouped_experts computes with flags = 0 (same kernels: y is bitwise the same), but
 * keeps H in a fixed device array of the library instead of a caller workspace, and calls no
 * allocating routine.  Limit: H of nentries * (inter/32) * 36 bytes must fit the array's
 * qgemv_grouped_experts_noalloc_max_bytes() bytes (4 MiB: 3640 entries at inter 1024), else
 * QMM_ESPACE.  Every call on a GPU uses that GPU's one array, so calls that overlap on one GPU
 * (two streams, two threads) race; the array keeps the last call's H.  Each GPU the library runs
 * on holds its own array until the process ends.  Arguments otherwise as qgemv_grouped_experts.
 * Errors: as qgemv_grouped_experts; QMM_ESPACE (H beyond the array), QMM_EHIP (the array's
 * device address could not be obtained). */
size_t qgemv_grouped_experts_noalloc_max_bytes(void);
int qgemv_grouped_experts_noalloc(int wtype_gu, const void* w_gate, const void* w_up,
                                  int64_t gu_expert_stride, int wtype_down, const void* w_down,
                                  int64_t down_expert_stride, int nexperts, const uint8_t* grid,
                                  int64_t hidden, int64_t inter, const void* xq, int xq_cols,
                                  const int32_t* group_expert, const int32_t* group_entry_off,
                                  int ngroups, const int32_t* entry_col, int nentries, float* y,
                                  void* stream);

/* Workspace bytes qgemm_prefill_experts needs (host). */
size_t qgemm_prefill_experts_workspace(int nexperts, int64_t inter, int64_t nentries,
                                       unsigned flags);

/* Prefill grouped expert GEMM [PF, Summary: weights of one expert dequantized to FP16 in the
 * workgroup's shared memory, FP16 matrix-core math with FP32 sums, over the rows sorted per
 * expert].  For expert e, entries p in [expert_off[e], expert_off[e+1]), token t = sorted_tok[p]:
 *   G = X16[t] . Wg16[e]^T,  U = X16[t] . Wu16[e]^T     (FP16 products, FP32 sums; Wg16/Wu16 are
 *                                                        the qmm_dequant_f16 values)
 *   H16 = fp16(silu(G) * U)                              (workspace; silu in binary32 with the
 *                                                        device expf, error <= 1 ulp)
 *   y[p*hidden + j] = (H16 . Wd16[e]^T)[j]               (FP32, one row per sorted entry;
 *                                                        y 16-byte aligned)
 *   x_f16      : binary16 [ntok][hidden], 16-byte aligned.
 *   sorted_tok : int32 [nentries]; a token outside [0, ntok) reads zeros.  expert_off: int32
 *                [nexperts+1], non-decreasing, expert_off[nexperts] <= nentries (offsets are
 *                clamped to [0, nentries]; rows of no expert, as those past a qmm_moe_dispatch's
 *                last entry, are not written).
 *   w_gate, w_up (format wtype_gu, inter rows of width hidden) and w_down (wtype_down, hidden
 *   rows of width inter) at e * stride; Q8_0 or IQ4_NL (CB3: QMM_EUNSUPPORTED); 4-byte
 *   aligned, strides multiples of 4.
 *   ws : qgemm_prefill_experts_workspace() bytes, 16-byte aligned.  Layout: H16 [nentries][inter]
 *        binary16 first, then the tile schedule; with QMM_FLAG_DEBUG_INTERMEDIATES then G, U
 *        float [nentries][inter].
 *   hidden, inter: multiples of 64, at most 32768; ntok * hidden * 2, nentries * inter * 2 and
 *   each expert matrix below 4 GiB.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_ESPACE. */
int qgemm_prefill_experts(int wtype_gu, const void* w_gate, const void* w_up,
                          int64_t gu_expert_stride, int wtype_down, const void* w_down,
                          int64_t down_expert_stride, int nexperts, int64_t hidden, int64_t inter,
                          const uint16_t* x_f16, int64_t ntok, const int32_t* sorted_tok,
                          const int32_t* expert_off, int64_t nentries, float* y, void* ws,
                          size_t ws_bytes, unsigned flags, void* stream);

/* Workspace bytes qgemm_prefill_experts_q8 needs (host). */
size_t qgemm_prefill_experts_q8_workspace(int nexperts, int64_t hidden, int64_t inter, int64_t ntok,
                                          int64_t nentries, unsigned flags);

/* MMQ-style prefill grouped expert GEMM [DQ, Change: the prefill path on q8_1 activations
 * against the quantized weights, with SwiGLU and the q8_1 quantization of H fused between
 * gate/up and down, H never stored in fp32; IQ, What it does: the decode path's per-block
 * integer dot and float expression].  Computes, over the rows sorted per expert, exactly what
 * qgemv_grouped_experts computes with groups = experts and entry_col = sorted_tok:
 *   xq  = q8_1(X16 as binary32) per 32-value block               (the quantizer's arithmetic)
 *   g,u = per 32-value block b: (d_w d_a) * isum in binary32, summed over b in order
 *   H   = q8_1(silu(g) * u) per 32 consecutive intermediate values (silu in binary32 with the
 *         device expf, error <= 1 ulp, and v_rcp_f32)
 *   y[p*hidden + j] = the same block sum of W_down[e] against H   (binary32; sorted order)
 * The block dots run on int8 MFMA, the per-block scale products on fp32 MFMA.
 *   Arguments as qgemm_prefill_experts (Q8_0 or IQ4_NL; hidden, inter multiples of 64).
 *   ws : qgemm_prefill_experts_q8_workspace() bytes, 16-byte aligned.  Layout (each part at the
 *        next 16-byte boundary): the tokens' q8_1 as planes (int8 [ntok][hidden], then the
 *        binary16 scales [ntok][hidden/32]), H as planes (int8 [nentries][inter], then scales
 *        [nentries][inter/32]), the tile schedule, and with QMM_FLAG_DEBUG_INTERMEDIATES g, u
 *        as float [nentries][inter].
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_ESPACE. */
int qgemm_prefill_experts_q8(int wtype_gu, const void* w_gate, const void* w_up,
                             int64_t gu_expert_stride, int wtype_down, const void* w_down,
                             int64_t down_expert_stride, int nexperts, int64_t hidden,
                             int64_t inter, const uint16_t* x_f16, int64_t ntok,
                             const int32_t* sorted_tok, const int32_t* expert_off,
                             int64_t nentries, float* y, void* ws, size_t ws_bytes,
                             unsigned flags, void* stream);

/* Dense prompt projection [DQ, Change: dense Q8_0 / IQ4_XS weights dequantized to FP16 with
 * 16-byte stores for a matrix product over the prompt's tokens; PF, Summary: the FP16 weights the
 * matrix cores get, FP32 sums]:
 *   y[t*ldy + r] = sum over k of W16[r][k] * X16[t][k]      (FP16 products, FP32 sums)
 * with W16 the qmm_dequant_f16 values of w (wtype Q8_0 or IQ4_NL: converted in registers inside
 * the GEMM, bitwise those values) or w itself (wtype QMM_F16: binary16 [nrows][k], e.g. the
 * output of qmm_dequant_f16).  fp16 MFMA (32x32x16) with FP32 accumulation.
 *   w     : nrows x qmm_row_bytes(wtype, k) bytes (QMM_F16: 2k bytes per row, 16-byte aligned;
 *           the others 4-byte aligned).   x_f16: binary16 [ntok][k], 16-byte aligned.
 *   y     : float [ntok][ldy], ldy >= nrows, 4-byte aligned.
 *   k     : a multiple of 64, at most 32768.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED (k not a multiple of 64, buffers of 4 GiB or
 *         more). */
int qgemm_dense(int wtype, const void* w, int64_t nrows, int64_t k, const uint16_t* x_f16,
                int64_t ntok, float* y, int64_t ldy, void* stream);

/* Weight planes [GP, What changed: a device-side repack of the GGUF blocks into planes (an int8
 * plane plus scales) for the decode GEMV, the packed copy owned through pack / release calls].
 * Layout (Q8_0 and IQ4_NL): each row is cut into tiles of 16 consecutive blocks (the last tile
 * of a row holds the blocks left); a tile is its n blocks' factor bytes back to back in block
 * order (Q8_0: 32 int8; IQ4_NL: 16 index bytes), then their n fp16 scales in block order.  A row
 * keeps its size and place, so the planes of a matrix take exactly its blocks' bytes and every
 * factor run of a lane starts 16-byte aligned.
 *
 * qmm_pack_planes: writes the planes of the nrows x k matrix w into `planes` (caller-owned,
 *   nrows * qmm_row_bytes(wtype, k) bytes, must not overlap w).  Byte copies only.
 * qmm_planes_alloc: allocates the planes buffer (hipMalloc; the one allocating entry point of the
 *   library), packs w into it on `stream` and returns it in *planes; the caller owns it until
 *   qmm_planes_release (hipFree; synchronizes the device).  *planes is NULL on error.
 * qgemv_planes: qgemv_dense on a planes buffer: the same kernels with the realignment of each
 *   block left out, so y is bitwise qgemv_dense's on the original blocks.  planes 16-byte
 *   aligned, k a multiple of 512 (rows of whole tiles); other arguments as qgemv_dense.
 * Errors: QMM_EINVAL (format other than Q8_0 / IQ4_NL, null, sizes), QMM_EALIGN,
 *         QMM_EUNSUPPORTED (qgemv_planes: k not a multiple of 512, or as qgemv_dense),
 *         QMM_EHIP (allocation or launch). */
int qmm_pack_planes(int wtype, const void* w, int64_t nrows, int64_t k, void* planes, void* stream);
int qmm_planes_alloc(int wtype, const void* w, int64_t nrows, int64_t k, void** planes, void* stream);
int qmm_planes_release(void* planes);
int qgemv_planes(int wtype, const void* planes, int64_t nrows, int64_t k, const void* xq, int ncols,
                 float* y, int64_t ldy, void* stream);

/* MoE combine [DQ, Change: the combine sums a token's expert rows with one fixed
 * thread-to-element mapping and k order; profile block: moe_combine4 reads them at bandwidth].
 *   out[t*ldo + j] = sum over k = 0 .. topk-1 of  weights[t*topk + k] * y[r*hidden + j],
 *                    r = row_idx[t*topk + k]
 * in binary32, from +0, adding in k order, each product and each sum rounded once (no fused
 * multiply-add); an index outside [0, nrows) adds nothing.  Decode: y is a grouped call's
 * [nentries][hidden] output and row_idx the entries of each token; prefill: y is the sorted-
 * entry output and row_idx each token's positions in the sorted order.
 *   y       : float [nrows][hidden], 16-byte aligned.   out: float [ntok][ldo], 16-byte aligned.
 *   row_idx : int32 [ntok][topk];  weights: float [ntok][topk] (both 4-byte aligned).
 *   hidden, ldo: multiples of 4, ldo >= hidden (columns hidden..ldo-1 are not written).
 *   topk    : 1 .. 64.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED (hidden or ldo not a multiple of 4, topk
 *         above 64, sizes of 2^31 or more). */
int qmm_moe_combine(const float* y, int64_t nrows, int64_t hidden, const int32_t* row_idx,
                    const float* weights, int64_t ntok, int topk, float* out, int64_t ldo,
                    void* stream);

/* Root-mean-square norm with the residual's addition, for the activations the products take.
 * For row t, in binary32:
 *   r[j]  = x[j] + res[j]                          (r = x when res is NULL)
 *   y[j]  = (r[j] * (1 / sqrt(sum r^2 / hidden + eps))) * w[j]
 * and writes any of: res_out = r rounded once to rtype, y rounded once to ytype, yq = q8_1(y)
 * (qmm_quantize_q8_1's bytes for the binary32 y).  The norm is taken of the binary32 r, not of
 * the rounded res_out.  The sum of squares is binary32: rows whose sum passes its range give y = 0.
 *   x       : xtype [ntok][ldx], ldx >= hidden.
 *   res, res_out : rtype [ntok][ldr], [ntok][ldro]; either may be NULL.
 *   w       : float [hidden].   eps >= 0.
 *   y       : ytype [ntok][ldy], or NULL.   yq : q8_1 [ntok][hidden/32][36], or NULL.
 *   hidden  : 1 .. 32768; a multiple of 32 when yq is given.
 *   Pointers and strides need their type's alignment only (yq: 4 bytes); 16-byte aligned rows are
 *   read and written 16 bytes at a time.  res_out may be res, and y or res_out may be x, if the
 *   types and row strides agree; otherwise outputs must not overlap inputs.
 * Errors: QMM_EINVAL (no output, unknown type, sizes, strides, eps negative or not finite),
 *         QMM_EALIGN, QMM_EUNSUPPORTED (hidden above 32768, 2^22 rows or more). */
int qmm_rmsnorm(int xtype, const void* x, int64_t ldx, int rtype, const void* res, int64_t ldr,
                void* res_out, int64_t ldro, const float* w, float eps, int64_t ntok,
                int64_t hidden, int ytype, void* y, int64_t ldy, void* yq, void* stream);

/* The values q8_1 blocks stand for: out[c*ldo + j] = d * q_j of column c, the exact product rounded
 * once to the output type.
 *   xq   : q8_1 [ncols][k/32][36], 4-byte aligned.   k : a multiple of 32, > 0.
 *   out  : otype (QMM_TYPE_F32 or QMM_TYPE_F16) [ncols][ldo], ldo >= k.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED (more than 2^29 - 32 blocks). */
int qmm_dequantize_q8_1(const void* xq, int64_t k, int64_t ncols, int otype, void* out, int64_t ldo,
                        void* stream);

/* Routing of tokens to experts.  For each row of logits l[0..nexperts), in binary32:
 *   s[e] = softmax(l)[e]  or  1 / (1 + exp(-l[e]))                        (score)
 *   c[e] = s[e] + bias[e]   (bias NULL: s[e]; a softmax without bias whose groups, if any, go by
 *          their best member is compared by l[e] itself, the same order without its rounding)
 *   an expert whose l[e] is -inf or NaN is never chosen nor counted in the softmax; one whose c[e]
 *     is, by its bias, is never chosen but its s[e] counts in the softmax;
 *   ngroups > 1: the experts form ngroups equal runs; a run's score is the sum of its group_top
 *     (1 or 2) largest c (-inf where it has fewer), the topk_groups best runs stay, the experts of
 *     the others are not chosen;
 *   the topk largest c, in descending order; ties, of experts and of runs, go to the lowest index;
 *   weights = s of the chosen (without the bias), with QMM_ROUTE_RENORM divided by their sum (left
 *     at 0 where that sum is 0), times `scale`.
 * Where fewer than topk experts can be chosen the remaining ids are -1 and their weights 0 (a row
 * of -inf gives only those).  A softmax over +inf logits shares 1 among them.
 *   logits : ltype [ntok][ldl], ldl >= nexperts.   bias : float [nexperts] or NULL.
 *   ids : int32 [ntok][topk];  weights : float [ntok][topk].
 *   nexperts 1 .. 1024 and a multiple of ngroups; ngroups 1 .. 64; 1 <= topk_groups <= ngroups;
 *   group_top <= nexperts / ngroups; 1 <= topk <= min(64, topk_groups * nexperts / ngroups).
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED (nexperts above 1024, ngroups or topk above 64,
 *         2^25 rows or more). */
#define QMM_ROUTE_RENORM 1u
int qmm_moe_route(int ltype, const void* logits, int64_t ldl, const float* bias, int64_t ntok,
                  int nexperts, int score, int ngroups, int topk_groups, int group_top, int topk,
                  float scale, int32_t* ids, float* weights, unsigned flags, void* stream);

/* Workspace bytes qmm_moe_dispatch needs (host); 0 for sizes it does not take. */
size_t qmm_moe_dispatch_workspace(int64_t ntok, int topk, int nexperts);

/* The expert-sorted entry lists that the grouped products and the combine take, from a routing's
 * ids [ntok][topk]: the entries (t, k) whose id is in [0, nexperts), ordered by expert, then by token,
 * then by k; an id outside adds no entry.  With n entries in all:
 *   sorted_tok[p] = the token of entry p for p < n, -1 up to ntok*topk
 *                   (qgemm_prefill_experts' sorted_tok, qgemv_grouped_experts' entry_col);
 *   row_idx[t*topk + k] = the entry's p, or -1                    (qmm_moe_combine's row_idx);
 *   expert_off[e] = entries of experts below e, e = 0 .. nexperts (qgemm_prefill_experts');
 *   group_expert[g], group_off[g], g < G = min(nexperts, ntok*topk): the experts that have entries,
 *                   ascending, and their first entry; beyond them expert -1 and offset n;
 *                   group_off[G] = n  (qgemv_grouped_experts' groups).  Both NULL: not written.
 *   ws   : qmm_moe_dispatch_workspace() bytes, 4-byte aligned.
 *   nexperts 1 .. 1024, topk 1 .. 64, ntok * topk at most 2^30.  ntok 0 writes the offsets.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_ESPACE. */
int qmm_moe_dispatch(const int32_t* ids, int64_t ntok, int topk, int nexperts, int32_t* sorted_tok,
                     int32_t* row_idx, int32_t* expert_off, int32_t* group_expert, int32_t* group_off,
                     void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes qmm_lora needs (host); 0 for sizes it does not take. */
size_t qmm_lora_workspace(int64_t ntok, int max_rank);

/* Low-rank adapters of many requests beside a shared projection (qgemv_dense*, qgemm_dense): tokens
 * seg_off[s] .. seg_off[s+1]-1 belong to request s and use adapter i = seg_adapter[s]:
 *   y[t][r] = base[t][r] + scales[i] * sum_j B[i][r][j] * (sum_c A[i][j][c] * x[t][c]),  j < ranks[i]
 * with binary32 sums, of the inner product and, from those sums as they are, of the outer one.  A
 * segment whose adapter is outside [0, nadapters) gives y = base.
 *   x    : QMM_TYPE_F16 or QMM_TYPE_F32 [ntok][ldx], 16-byte aligned, ldx * element size a
 *          multiple of 16.
 *   a    : binary16 [nadapters][max_rank][k];  b : binary16 [nadapters][nrows][max_rank]; 16-byte
 *          aligned.  Rows / columns at ranks[i] and beyond are not used.
 *   ranks: int32 [nadapters] (clamped to [0, max_rank]);  scales : float [nadapters].
 *   seg_off : int32 [nseg + 1], non-decreasing (each offset is clamped to [0, ntok]; tokens of no
 *          segment are not written);  seg_adapter : int32 [nseg].
 *   base : float [ntok][ldbase], may be y (then ldbase = ldy; segments without adapter are not
 *          touched);  y : float [ntok][ldy]; strides >= nrows, 4-byte aligned.
 *   k    : a multiple of 32, at most 32768;  max_rank : a multiple of 8, at most 256;  ntok at most
 *          2^20, nseg at most 2^14, strides of y and base below 2^31.
 *   ws   : qmm_lora_workspace() bytes, 16-byte aligned.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_ESPACE. */
int qmm_lora(int xtype, const void* x, int64_t ldx, int64_t ntok, int64_t k, const uint16_t* a,
             const uint16_t* b, const int32_t* ranks, const float* scales, int nadapters,
             int max_rank, const int32_t* seg_off, const int32_t* seg_adapter, int nseg,
             const float* base, int64_t ldbase, float* y, int64_t ldy, int64_t nrows, void* ws,
             size_t ws_bytes, void* stream);

/* A paged key-value cache (host struct; k and v are device pointers).  Each of k and v is an array
 * of npages pages, kstride / vstride bytes apart; a page holds, for each of its nheads heads, a chunk of
 * page_size positions of head_dim values, page_size * qmm_row_bytes(type, head_dim) bytes:
 *   QMM_F16    : binary16 [page_size][head_dim];
 *   QMM_Q8_0, QMM_IQ4_NL : two planes, the blocks' factors [page_size][head_dim / 32 * 32 or 16 bytes],
 *                then their binary16 scales [page_size][head_dim / 32].  With nb = head_dim / 32, value
 *                16 i + n of block b (i = 0, 1; n = 0 .. 15) is int8 (n*nb + b)*2 + i of its position's
 *                factors, or the low (i = 0) or high (i = 1) half of byte n*nb + b: what one lane of a
 *                matrix instruction takes of every block is contiguous.  Values as in the weight formats,
 *                d * q and d * level.
 *   ktype, vtype : QMM_F16, QMM_Q8_0 or QMM_IQ4_NL.   k, v : 16-byte aligned; strides multiples of 16.
 *   page_size : a multiple of 16, at most 4096.   head_dim : 64, 96, 128, 192 or 256.
 *   nheads : 1 .. 1024.   npages : 1 .. 2^31 - 1.
 *
 * Sequence s of nseq has lens[s] positions in the cache, the new tokens of the call among them; position p
 * is place p % page_size of page pages[s*ldpages + p / page_size].  Its new tokens are seg_off[s] ..
 * seg_off[s+1]-1 of the call's ntok (NULL: nseq = ntok, token s alone); they are its last positions, token
 * t the position lens[s] - (seg_off[s+1] - t).  What the host cannot check is bounded on the device: offsets
 * are clamped to [0, ntok] and have to be non-decreasing, a position below 0, past max_pages or
 * on a page outside [0, npages) does not exist, and tokens of no sequence are left alone.
 *   pages : int32 [nseq][ldpages], ldpages >= max_pages; entries past a sequence's pages may hold anything (they, and what
 *           is on a page that they name, may be read, and have no effect).
 *   lens : int32 [nseq].   seg_off : int32 [nseq + 1] or NULL.   (4-byte aligned.)
 *   ntok at most 2^20, ntok * nheads at most 2^27, nseq at most 2^14, max_pages * page_size at most 2^30. */
typedef struct {
    int ktype, vtype;
    void *k, *v;
    int64_t kstride, vstride; /* bytes from a page to the next */
    int64_t npages;
    int page_size, nheads, head_dim;
} qmm_kv_cache;

/* Writes new tokens' keys and values to their positions, quantized per 32 values x_j of a head's row:
 *   QMM_Q8_0   : d = max |x| / 127, q_j = x_j / d rounded half away from zero;
 *   QMM_IQ4_NL : d = x_m / -127, x_m the value of largest magnitude (the first of them); the index of x_j
 *                the level nearest to x_j / d, ties to the lower one;
 *   in binary32 with IEEE divisions; d is stored as binary16.  Where d is 0 every value is 0 (scale +0, indices 8).
 *   QMM_F16    : x_j rounded to nearest even.
 * A block of a block format that holds an infinity or NaN does not read back as what it held; its
 * neighbours do.  A token whose position does not exist is not written.  The positions of one call
 * must be distinct.
 *   xtype : type of k and v, QMM_TYPE_*.   k, v : [ntok][ldk], [ntok][ldv], rows of nheads * head_dim
 *   values; one of them may be NULL: that cache is left alone.   cache : host pointer.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED. */
int qmm_kv_write(const qmm_kv_cache* cache, const int32_t* pages, int64_t ldpages, int64_t max_pages,
                 const int32_t* lens, const int32_t* seg_off, int nseq, int xtype, const void* k,
                 int64_t ldk, const void* v, int64_t ldv, int64_t ntok, void* stream);

/* Reads keys and values back, each value exact and rounded once to the output type: the last
 * seg_off[s+1] - seg_off[s] positions of each sequence (all of it where that is lens[s]); rows of zeros
 * where a position does not exist.  Arguments as qmm_kv_write; rows of k and v must not overlap. */
int qmm_kv_read(const qmm_kv_cache* cache, const int32_t* pages, int64_t ldpages, int64_t max_pages,
                const int32_t* lens, const int32_t* seg_off, int nseq, int otype, void* k, int64_t ldk,
                void* v, int64_t ldv, int64_t ntok, void* stream);

/* Workspace bytes qmm_kv_attend needs (host), enough for calls of smaller sizes too; 0 for sizes it does not take. */
size_t qmm_kv_attend_workspace(const qmm_kv_cache* cache, int64_t ntok, int nheads, int nseq,
                               int64_t max_pages);

/* Attention of new tokens over the cache, their own keys and values among it (qmm_kv_write first).  For
 * token t of sequence s at position p, head h, and the cache's head h / (nheads / cache->nheads):
 *   z_j = scale * sum_c q[t][h][c] * key_j[c],   j <= p, j > p - window if window > 0, j existing
 *   out[t][h] = sum_j exp(z_j - max z) * value_j / sum_j exp(z_j - max z),   lse[t][h] = log sum_j exp(z_j)
 * with binary32 scores, statistics and sums; query values and weights are kept to 2^-22 of themselves, or to 2^-38 of
 * the row's largest (query value; weight, times the largest scale seen of the block where values are blocks).  No j
 * (a token before position 0, an empty sequence, missing pages): out 0, lse -inf.  Positions a token does not see have no
 * effect on it, whatever they hold.  A row of q that is not finite gives NaN in its own outputs.  Infinities and NaN that it
 * sees in a binary16 cache count as the formulas say: a score of -inf has the weight 0, an infinite value gives its
 * infinity, or NaN beside the opposite one or at a weight of 0.  A block whose scale is not finite adds scale * (the sum of
 * its integers' products) to a score, and makes its own dims of the values NaN.  Nothing but scores of -inf: as no j.  Meant
 * for up to some tens of tokens a sequence (any count is right: each 16 or 32 rows of queries read the cache once).
 *   q    : qtype [ntok][ldq], rows of nheads * head_dim values.   nheads : a multiple of cache->nheads, at
 *          most 1024.   scale : finite.   window : >= 0.
 *   out  : otype [ntok][ldo], must not overlap q (out == q is refused).   lse : float [ntok][nheads] or NULL.
 *   cache->vtype holds at most as many bits as cache->ktype (an error of a key enters the exponent): QMM_EUNSUPPORTED
 *          for others, which qmm_kv_write and qmm_kv_read take.
 *   ws   : qmm_kv_attend_workspace() bytes, 16-byte aligned; nothing in it is kept between calls, and
 *          calls that may overlap in time need one each.
 * The same call gives the same bits, whatever the scheduling; in their last bits results depend on how the call is
 * split, which is by nseq, ntok, max_pages and all lengths.  Offsets that decrease so that sequences have more tokens than ntok in
 * all: nothing is written.
 * Errors: QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_ESPACE. */
int qmm_kv_attend(const qmm_kv_cache* cache, const int32_t* pages, int64_t ldpages, int64_t max_pages,
                  const int32_t* lens, const int32_t* seg_off, int nseq, int qtype, const void* q,
                  int64_t ldq, int64_t ntok, int nheads, float scale, int64_t window, int otype,
                  void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
