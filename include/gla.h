/* gla.h - C ABI of the GB300 Simple GLA mixer library (libgla.so).
 *
 * What it computes.  Source: "Beyond the KV cache: Training and serving i14's Laplace 3B linear
 * attention model on AWS Trainium2 with native PyTorch" (AWS blog post; Spanish and Chinese
 * copies carry the later sections and the figure captions).
 *   - Section "i14 and the Laplace 3B architecture", paragraph "GLA mixer": every head h keeps a
 *     d_k x d_v = 96 x 192 matrix state, decayed by a fixed per-head factor lambda_h and written
 *     with the rank-1 outer product of the current key and value; the readout queries the state.
 *     The equation images are missing from the text; this library computes
 *         S_t = lambda_h * S_{t-1} + k_t v_t^T ,      o_t = S_t^T (scale * q_t)
 *     with the readout after the update, S_0 = h0 (zeros when h0 is NULL) and hT = S_T.
 *   - Section "Challenge 1: Using native PyTorch on Trainium for GLA": the chunked form with
 *     128-token chunks (intra-chunk masked linear attention plus the carried state; the state
 *     advances with lambda^C, the decay compounded over the chunk).  gla_chunk_fwd computes that
 *     form; its result equals the recurrence above up to rounding.
 *   - Section "Challenge 3" (backward through the sequential state updates): gla_chunk_bwd is the
 *     adjoint of the recurrence.  lambda is fixed at initialisation, not learned ("Decay
 *     schedule"), so there is no gradient for it.
 *   - Section "Optimizing inference on Trainium2" (a wrapper reads and writes each sequence's
 *     recurrent state in a pool, one fixed page per sequence): gla_decode_step advances a pool of
 *     states by one token in place.
 *
 * Conventions shared by every entry point.
 *   - Sizes: only d_k = 96 and d_v = 192 are implemented; other values return
 *     GLA_ERR_UNSUPPORTED.  H >= 1.  Chunk size is 128 tokens (GLA_CHUNK).
 *   - Pointers are DEVICE pointers owned by the caller, 16-byte aligned (else GLA_ERR_ALIGN),
 *     except where a comment says "host".  The library never allocates, frees or keeps them.
 *   - Layouts are dense, C order, token-major:
 *       q, k     [n_seq, T, H, 96]   (or packed [T_total, H, 96] with cu_seqlens)
 *       v, o, dO [n_seq, T, H, 192]  (or packed [T_total, H, 192])
 *       h0, hT, dhT, dh0, state  [n_seq (or pool rows), H, 96, 192], always fp32
 *       log_lambda [H] fp32: natural log of lambda_h, <= 0 (-inf allowed: lambda = 0)
 *   - dtype (gla_dtype) is the type of q, k, v, o, dO, dq, dk, dv.  GLA_BF16 runs the tensor-core
 *     kernels (bf16 operands, fp32 accumulation and fp32 state); results are rounded to bf16
 *     nearest-even.  GLA_F32 runs the all-fp32 CUDA-core kernels.
 *   - scale multiplies q (1/sqrt(96) in the Laplace 3B configuration).
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream).
 *     Argument errors are detected on the host before anything is launched and return a negative
 *     gla_status; nothing aborts the process.  Faults found while a kernel runs (a bounded wait
 *     that timed out, a pool slot out of range) set a sticky per-device error word that
 *     gla_get_device_error() reports.
 *   - Empty work is valid: n_seq = 0, T = 0 or sequences of length 0 launch nothing for them;
 *     a length-0 sequence gives hT = h0 (zeros if h0 is NULL) and dh0 = dhT.
 *   - The library looks up the device addresses of its own device variables (the error word,
 *     the hand-over flags, the array of gla_chunk_fwd_noalloc) once per device and keeps them,
 *     and creates a few CUDA objects per device that live until the process exits (the
 *     backward's two side streams; the host-buffer forward's two copy streams and its events),
 *     so resetting a device (cudaDeviceReset) after the library's first call on it is not
 *     supported.
 */
#ifndef GLA_H_
#define GLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* gla_stream_t; /* identical to cudaStream_t */

typedef enum {
  GLA_OK = 0,
  GLA_ERR_NULL = -1,        /* a required pointer is NULL */
  GLA_ERR_SHAPE = -2,       /* negative size, bad cu_seqlens, pool slot out of range, or
                               n_seq * H * 96 or the token count reaches 2^31 */
  GLA_ERR_DTYPE = -3,       /* dtype is not a gla_dtype */
  GLA_ERR_ALIGN = -4,       /* a pointer is not 16-byte aligned */
  GLA_ERR_UNSUPPORTED = -5, /* d_k != 96, d_v != 192, or no sm_103 device current */
  GLA_ERR_WORKSPACE = -6,   /* workspace missing or smaller than gla_workspace_bytes() */
  GLA_ERR_LAUNCH = -7,      /* the CUDA runtime refused a launch */
  GLA_ERR_TIMEOUT = -8,     /* a bounded device-side wait gave up (kernel returned early) */
  GLA_ERR_BOUNDS = -9       /* debug-bounds build only: a device index fell outside its buffer
                               (the access was skipped; see gla_debug_bounds) */
} gla_status;

typedef enum { GLA_BF16 = 0, GLA_F32 = 1 } gla_dtype;

#define GLA_DK 96
#define GLA_DV 192
#define GLA_CHUNK 128

/* Bytes of device workspace that gla_chunk_fwd / gla_chunk_bwd need for `n_seq` packed
 * (cu_seqlens) sequences of H heads.  The workspace holds the longest-first schedule of the
 * (sequence, head) work.  Calls without cu_seqlens need none (pass NULL, 0). */
size_t gla_workspace_bytes(int n_seq, int H);

/* Chunked forward.
 *   q, k, v      inputs (layouts above), dtype `dtype`.
 *   log_lambda   [H] fp32 device.
 *   h0           [n_seq, H, 96, 192] fp32, or NULL for zero initial states.
 *   scale        multiplies q.
 *   o            output, same dtype and layout as v.
 *   hT           [n_seq, H, 96, 192] fp32 final states, or NULL to skip.
 *   cu_seqlens   NULL: n_seq sequences of T tokens each, layout [n_seq, T, H, d].
 *                else: [n_seq + 1] int32 device array of packed offsets, cu_seqlens[0] = 0,
 *                non-decreasing, cu_seqlens[n_seq] = T (the packed total); its values are read on
 *                the device only (no host synchronisation), so the caller guarantees them.
 *   workspace    >= gla_workspace_bytes(n_seq, H) bytes when cu_seqlens != NULL, else unused.
 * Returns GLA_OK once the work is queued on `stream`. */
int gla_chunk_fwd(const void* q, const void* k, const void* v, const float* log_lambda,
                  const float* h0, float scale, void* o, float* hT, const int32_t* cu_seqlens,
                  int n_seq, int T, int H, int dk, int dv, int dtype, void* workspace,
                  size_t ws_bytes, gla_stream_t stream);

/* Chunked forward with the self-augmentation step ("Beyond the KV cache", section "i14 and the
 * Laplace 3B architecture", the paragraph after the state readout): every output row also gains
 * a gated copy of its own value,
 *     o_t += sigmoid(q_t . (a_h * k_t)) v_t,
 * with a_h the head's aug_balance (a learned rescaling of the key's channels; a = 0 gives the
 * half-strength copy 0.5 v_t).  The query enters the gate unscaled.
 *   aug          [H, 96] fp32 device (non-NULL, 16-byte aligned); a NULL aug returns GLA_ERR_NULL.
 *   every other argument, and the results, as in gla_chunk_fwd (hT is not affected: the copy
 *   adds to the output only).
 * gla_chunk_bwd differentiates the mixer without this step. */
int gla_chunk_fwd_aug(const void* q, const void* k, const void* v, const float* log_lambda,
                      const float* h0, float scale, const float* aug, void* o, float* hT,
                      const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype,
                      void* workspace, size_t ws_bytes, gla_stream_t stream);

/* Bytes of device workspace that gla_chunk_bwd needs; n_seq, T, H as in that call, packed != 0
 * when cu_seqlens is given, dtype the gla_dtype.  In bf16 mode the workspace holds fp32 partial
 * sums of dq and dk (2 x T_total x H x 96 x 4 bytes) plus the packed schedule; in fp32 mode only
 * the packed schedule (0 extra bytes for fixed-length calls). */
size_t gla_bwd_workspace_bytes(int n_seq, int T, int H, int packed, int dtype);

/* Chunked backward: gradients of L(o, hT) given dO = dL/do and dhT = dL/dhT.
 *   q, k, v, log_lambda, h0, scale, cu_seqlens, n_seq, T, H, dtype: as in gla_chunk_fwd
 *                (h0 NULL = zeros).
 *   dO           same dtype and layout as v.
 *   dhT          [n_seq, H, 96, 192] fp32, or NULL for zero.
 *   dq, dk       outputs, layout of q; dv output, layout of v; all of dtype `dtype`.
 *   dh0          [n_seq, H, 96, 192] fp32 output, or NULL to skip.
 *   workspace    >= gla_bwd_workspace_bytes(n_seq, T, H, cu_seqlens != NULL, dtype) bytes.
 * The forward state is recomputed on chip; nothing from gla_chunk_fwd is needed.  In bf16 mode dv
 * and dh0 come from one reverse scan, dq and dk from scans over each 64-column tile of d_v whose
 * fp32 partial sums meet in the workspace before the final bf16 rounding. */
int gla_chunk_bwd(const void* q, const void* k, const void* v, const float* log_lambda,
                  const float* h0, float scale, const void* dO, const float* dhT, void* dq,
                  void* dk, void* dv, float* dh0, const int32_t* cu_seqlens, int n_seq, int T,
                  int H, int dk_size, int dv_size, int dtype, void* workspace, size_t ws_bytes,
                  gla_stream_t stream);

/* One decode step for N sequences, in place on a state pool.
 *   q, k         [N, H, 96]; v, o [N, H, 192]; dtype `dtype`.
 *   state        [pool_rows, H, 96, 192] fp32, updated in place: S <- lambda S + k v^T.
 *   slot         [N] int32 device array: sequence n uses pool row slot[n]; NULL = row n
 *                (then pool_rows >= N is required).  Rows must be distinct.  A slot outside
 *                [0, pool_rows) skips that sequence (state and o untouched) and records
 *                GLA_ERR_SHAPE in the device error word.
 *   o            readout o = S^T (scale q), taken after the update. */
int gla_decode_step(const void* q, const void* k, const void* v, const float* log_lambda,
                    float scale, float* state, const int32_t* slot, int pool_rows, void* o, int N,
                    int H, int dk, int dv, int dtype, gla_stream_t stream);

/* One decode step with the self-augmentation step: as gla_decode_step, and the output also gains
 * sigmoid(q . (a_h * k)) v (see gla_chunk_fwd_aug); aug [H, 96] fp32 device, non-NULL and
 * 16-byte aligned.  The state update is the same. */
int gla_decode_step_aug(const void* q, const void* k, const void* v, const float* log_lambda,
                        float scale, const float* aug, float* state, const int32_t* slot,
                        int pool_rows, void* o, int N, int H, int dk, int dv, int dtype,
                        gla_stream_t stream);

/* Per-tier Head RMSNorm and SiLU output gate ("Beyond the KV cache", section "i14 and the
 * Laplace 3B architecture": the per-head outputs pass through a Head RMSNorm within each decay
 * tier, then are gated by SiLU(g_t)).  For every row t and head h:
 *     y[t,h,:] = o[t,h,:] / sqrt(mean_c o[t,h,c]^2 + eps) * weight[tier[h],:] * SiLU(g[t,h,:]),
 * SiLU(x) = x sigmoid(x); the RMS runs over the head's 192 channels.
 *   o, g, y      [rows, H, 192], dtype `dtype` (o is a chunked-forward or decode output, g the
 *                gate stream); y may not alias o or g.
 *   weight       [n_tiers, 192] fp32 device, the gain of each tier's norm.
 *   tier         [H] int32 device: the tier of each head; a value outside [0, n_tiers) leaves
 *                that head's rows untouched and records GLA_ERR_SHAPE in the device error word.
 *   eps          >= 0, added to the mean square (not stated on the pages).
 * H <= 4096 (else GLA_ERR_UNSUPPORTED).  Pointers 16-byte aligned (tier 4-byte).  Returns GLA_OK once the work is queued on `stream`. */
int gla_head_norm_gate(const void* o, const void* g, const float* weight, const int32_t* tier,
                       int n_tiers, float eps, void* y, long long rows, int H, int dv, int dtype,
                       gla_stream_t stream);

/* One decode step whose readout goes straight through the per-tier Head RMSNorm and the SiLU
 * output gate ("Beyond the KV cache", section "i14 and the Laplace 3B architecture": the per-head
 * outputs pass through a Head RMSNorm within each decay tier, then the SiLU(g_t) gate; heads are
 * grouped into tiers that share a norm, section "Decay schedule's reach").  The state update is
 * that of gla_decode_step (aug NULL) or gla_decode_step_aug (aug non-NULL) on an fp32 pool; the
 * readout o (fp32, before any rounding) is not stored but normalised and gated in the same
 * kernel, and
 *     y[n,h,:] = o / sqrt(mean_c o_c^2 + eps) * weight[tier[h],:] * SiLU(g[n,h,:])
 * is written, as gla_head_norm_gate would compute from o.
 *   g            [N, H, 192] gate stream, dtype `dtype`, 16-byte aligned.
 *   weight       [n_tiers, 192] fp32, 16-byte aligned; tier [H] int32 (4-byte aligned).  A tier
 *                outside [0, n_tiers) leaves that head's y untouched (the state is still updated)
 *                and records GLA_ERR_SHAPE in the device error word.
 *   eps          >= 0; n_tiers >= 1 (else GLA_ERR_SHAPE).
 *   y            [N, H, 192] output, dtype `dtype`; may not alias g.
 * Every other argument as in gla_decode_step_aug. */
int gla_decode_step_norm_gate(const void* q, const void* k, const void* v, const float* log_lambda,
                              float scale, const float* aug, float* state, const int32_t* slot,
                              int pool_rows, const void* g, const float* weight, const int32_t* tier,
                              int n_tiers, float eps, void* y, int N, int H, int dk, int dv, int dtype,
                              gla_stream_t stream);

/* One decode step on a state pool stored in bf16 (no counterpart in the paper: a storage
 * variant that halves the state stream).  As gla_decode_step (aug NULL) or gla_decode_step_aug
 * (aug non-NULL), with `state` a [pool_rows, H, 96, 192] bf16 pool: each state is widened to
 * fp32, updated and read out in fp32 (the readout uses the update before rounding), and written
 * back rounded to bf16 (to nearest, ties to even).  The rounding error is kept in the state and
 * carried by later steps (relative 2^-9 per element per step, decayed by lambda), so long decodes
 * drift from the fp32-state result; the fp32 pool is the reference path. */
int gla_decode_step_bf16_state(const void* q, const void* k, const void* v, const float* log_lambda,
                               float scale, const float* aug, void* state, const int32_t* slot,
                               int pool_rows, void* o, int N, int H, int dk, int dv, int dtype,
                               gla_stream_t stream);

/* Decode step on a state pool stored as MXFP8 (no counterpart in the paper: a storage variant
 * that quarters the state stream; the pages keep fp32 states).  Format: OCP Microscaling (MX)
 * v1.0 MXFP8, E4M3 elements (OCP 8-bit floating point: bias 7, largest finite 448) with one E8M0
 * scale byte b (value 2^(b - 127)) per block of 32 consecutive values of a state row:
 *   state_codes   [pool_rows, H, 96, 192] uint8 E4M3 codes, 16-byte aligned;
 *   state_scales  [pool_rows, H, 96, 6] uint8 E8M0 scales of the blocks (columns 32j .. 32j+31),
 *                 16-byte aligned.
 * Each state is widened exactly to fp32, updated (S <- lambda S + k v^T) and read out
 * (o = S^T (scale q), from the update before it is stored) in fp32, and written back quantised:
 * per block, shared exponent se = floor(log2(max |x|)) - 8, plus one where the block maximum
 * would otherwise exceed 448 (the MX rule alone saturates such maxima to 448; here nothing
 * saturates), clamped to [-127, 127] (-127 for an all-zero block); codes = x 2^-se rounded to
 * E4M3, to nearest, ties to even.  The quantisation error (up to 2^-4 relative per element per
 * step, decayed by lambda) stays in the state, so long decodes drift from the fp32 result much
 * more than with the bf16 pool; the fp32 pool is the reference path.  Every other argument as in
 * gla_decode_step (aug NULL) or gla_decode_step_aug (aug non-NULL). */
int gla_decode_step_mxfp8_state(const void* q, const void* k, const void* v, const float* log_lambda,
                                float scale, const float* aug, uint8_t* state_codes, uint8_t* state_scales,
                                const int32_t* slot, int pool_rows, void* o, int N, int H, int dk, int dv,
                                int dtype, gla_stream_t stream);

/* Conversions between fp32 state rows and MXFP8 (the format of gla_decode_step_mxfp8_state), for
 * building a pool from fp32 states (a prefill's hT) and reading one back.  `rows` rows of 192
 * values: x [rows, 192] fp32, codes [rows, 192] uint8, scales [rows, 6] uint8; all 16-byte
 * aligned.  Quantisation as in gla_decode_step_mxfp8_state; dequantisation is exact. */
int gla_state_to_mxfp8(const float* x, uint8_t* codes, uint8_t* scales, long long rows, gla_stream_t stream);
int gla_state_from_mxfp8(const uint8_t* codes, const uint8_t* scales, float* x, long long rows,
                         gla_stream_t stream);

/* Sequence-split forward for long sequences (no counterpart in the paper).  A sequence's work
 * otherwise sits on one CTA per (head, 64-column tile of d_v), so one long sequence among few
 * keeps most SMs idle.  Here each sequence is cut into segments of at most seg_chunks chunks
 * (128 tokens each), and the forward runs in three steps: every segment from a zero state (its
 * final state U_i), a scan per (sequence, head) that chains them (S_in of the next segment =
 * lambda^(L_i) S_in + U_i; hT after the last), and every segment again from its S_in, writing o.
 * Same results as gla_chunk_fwd (the sums are only reassociated), about twice its reads of q, k
 * and v; worth it when the longest sequences dominate the call.
 *   cu_seqlens_host  [n_seq + 1] host array of packed offsets (cu_seqlens_host[0] = 0,
 *                    non-decreasing, cu_seqlens_host[n_seq] = T): the segments are planned on the
 *                    host, so no device offsets are needed (a fixed-length batch passes 0, T,
 *                    2T, ... with T = n_seq * T_seq and the [n_seq, T_seq, H, d] layout).
 *   aug              NULL, or aug_balance [H, 96] (the self-augmentation step of gla_chunk_fwd_aug).
 *   seg_chunks       >= 1, chunks per segment; 0: chosen by gla_split_choose_seg_chunks.  When
 *                    every sequence fits one segment the call is gla_chunk_fwd (or _aug).
 *   workspace        >= gla_split_workspace_bytes(cu_seqlens_host, n_seq, H, seg_chunks) bytes,
 *                    256-byte aligned: the plan, the segment states (two fp32 [segments, H, 96,
 *                    192] arrays) and the packed schedule.
 * Every other argument as in gla_chunk_fwd.  The plan is copied to the device with pageable
 * host-to-device copies (which may wait for the stream's earlier work).
 * gla_split_workspace_bytes returns 0 for a NULL cu_seqlens_host, n_seq < 0, H < 1, seg_chunks
 * < 0 or decreasing offsets.
 * gla_split_choose_seg_chunks: the segment length that seg_chunks = 0 uses, from a cost model of
 * the packed forward (one CTA per (segment, head, d_v tile) unit on each of 152 SMs, longest
 * units first, a unit costing its chunks plus a start-up cost; the split's two passes against the
 * plain forward's one), over lengths that cut the longest sequence into 2 .. 64 equal parts.
 * Returns 0 when no split is estimated faster, GLA_ERR_NULL / GLA_ERR_SHAPE on bad arguments.
 * Host only (no device needed). */
size_t gla_split_workspace_bytes(const int32_t* cu_seqlens_host, int n_seq, int H, int seg_chunks);
int gla_split_choose_seg_chunks(const int32_t* cu_seqlens_host, int n_seq, int H);
int gla_chunk_fwd_split(const void* q, const void* k, const void* v, const float* log_lambda,
                        const float* h0, float scale, const float* aug, void* o, float* hT,
                        const int32_t* cu_seqlens_host, int n_seq, int T, int H, int dk, int dv,
                        int dtype, int seg_chunks, void* workspace, size_t ws_bytes,
                        gla_stream_t stream);

/* The forward without any device allocation (no counterpart in the paper).  For callers that
 * cannot allocate device memory per call, such as a serving engine whose memory is all handed to
 * its own pool at start-up: same arguments and results as gla_chunk_fwd, minus the workspace.
 * The longest-first schedule of packed sequences lives instead in a library-owned device array of
 * GLA_NOALLOC_MAX_SEQS int32 (64 KB), kept by every GPU that loads the library until exit.
 *   Arguments are checked as in gla_chunk_fwd (the same status codes, including GLA_ERR_SHAPE for
 *   n_seq * H * 96 or the token count at 2^31 or beyond); then n_seq > GLA_NOALLOC_MAX_SEQS with
 *   cu_seqlens returns GLA_ERR_WORKSPACE (nothing launched).
 *   The first call on a device looks up the array's device address (cudaGetSymbolAddress); make
 *   that first call before any stream capture on the device.
 *   Calls share the array: calls that overlap on the GPU (unordered streams) race on it.  Calls
 *   ordered on one stream do not; each rewrites the entries it uses before reading them. */
#define GLA_NOALLOC_MAX_SEQS 16384
int gla_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const float* log_lambda,
                          const float* h0, float scale, void* o, float* hT,
                          const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv,
                          int dtype, gla_stream_t stream);

/* The chunked forward on HOST buffers ("Beyond the KV cache", section "Challenge 1: Using native
 * PyTorch on Trainium for GLA": sequences are independent, and within one the scan carries only
 * the state across a chunk boundary): q, k, v are read from host memory and o, hT written back
 * to host memory, the copies pipelined with the compute inside the call.  The batch is cut into
 * `pieces`: sub-batches of whole sequences (pieces <= n_seq), or, with pieces > n_seq, each
 * sequence cut into pieces / n_seq parts of a whole number of 128-token chunks (fewer when T does
 * not divide so), a part starting from the final state of the one before, which is the state the
 * uncut scan carries across that boundary: the results equal gla_chunk_fwd's on the same values.
 * Piece i is copied in on a library stream while piece i - 1 runs on `stream` and piece i - 2 is
 * copied out on another library stream; `stream` completes after the last copy out, so the host
 * outputs may be read once `stream` has been synchronised.
 *   q, k, v      HOST [n_seq, T, H, 96 / 192] of dtype `dtype` (page-locked memory lets the copies
 *                overlap the compute; pageable memory works, without the overlap).
 *   h0           HOST [n_seq, H, 96, 192] fp32, or NULL for zeros.
 *   o, hT        HOST outputs (o as v; hT [n_seq, H, 96, 192] fp32, or NULL to skip).
 *   log_lambda   DEVICE [H] fp32, 16-byte aligned.
 *   pieces       >= 1.
 *   workspace    DEVICE, 256-byte aligned, >= gla_chunk_fwd_host_workspace_bytes(n_seq, T, H,
 *                dtype) bytes: the staged batch (q, k, v, o) and three sets of states.
 * Fixed-length batches only.  Returns GLA_OK once the work is queued; argument errors as in
 * gla_chunk_fwd, GLA_ERR_WORKSPACE for a missing or short workspace, GLA_ERR_LAUNCH if a copy or
 * an event could not be queued.  Calls on one device are issued one at a time (a library mutex);
 * their work may still overlap on the GPU, so calls on streams that are not ordered with each
 * other need workspaces of their own (calls on one stream may share one).
 * gla_chunk_fwd_host_workspace_bytes returns 0 for n_seq < 0, T < 0, H < 1 or an unknown dtype. */
size_t gla_chunk_fwd_host_workspace_bytes(int n_seq, int T, int H, int dtype);
int gla_chunk_fwd_host(const void* q, const void* k, const void* v, const float* log_lambda,
                       const float* h0, float scale, void* o, float* hT, int n_seq, int T, int H,
                       int dk, int dv, int dtype, int pieces, void* workspace, size_t ws_bytes,
                       gla_stream_t stream);

/* Sequences that continue a shared prefix ("Beyond the KV cache", section "Optimizing inference on
 * Trainium2", keeps one page of state per sequence; the calls below, without counterpart there, serve
 * many sequences from one state).  A prefix - a prompt, a system message - is run once and leaves its
 * state S_p in a pool; a sequence that continues it keeps only its own tokens after the prefix, its
 * tail:
 *     S_n = lambda^L S_p + sum_{j < L} lambda^(L-1-j) k_j v_j^T     (L tokens in the tail).
 *   pool         [pool_rows, H, 96, 192] fp32 states (a forward's hT, a decode pool); read only.
 *   prefix_row   [n] int32 device: the pool row that each sequence continues.  Rows may repeat, in
 *                any order; sequences of one row that stand next to each other share one read of it.
 *   gla_tail     host struct of the tails, which live in device memory that the caller owns:
 *                  k [rows, H, cap, 96], v [rows, H, cap, 192], the head before the token;
 *                  GLA_TAIL_PLAIN: elements of the call's dtype; k_scales and v_scales unused.
 *                  GLA_TAIL_MXFP8: E4M3 codes with E8M0 scales k_scales [rows, H, cap, 3] and
 *                  v_scales [rows, H, cap, 6], one per 32 values, quantised by the rule of
 *                  gla_decode_step_mxfp8_state (no finite value saturates; an infinity costs its
 *                  block's other values).  In every call an element is code x scale in fp32: an
 *                  infinity stays one, a NaN stays one.
 *                cap >= 16 and a multiple of 16 (else GLA_ERR_SHAPE); every array 16-byte aligned.
 *   tail_slot    [n] int32 device: the tail row of each sequence, NULL = row n (then rows >= n is
 *                required).  Rows that a call writes must be distinct.
 *   tail_len     [n] int32 device: tokens in each tail, at places 0 .. tail_len - 1.  The calls
 *                read it and never change it: the caller advances it after a decode step.  Places
 *                from tail_len on may hold anything, NaN included.
 * In the decode step and the fold an infinity or a NaN in a state, a tail or a token stays with the outputs that it
 * enters.  Where operands are held as sums of several bf16 (bf16 calls, folds of bf16 and MXFP8 tails) an infinity may
 * come out as a NaN.
 * The self-augmentation step (gla_chunk_fwd_aug, gla_decode_step_aug) has no form among these calls.
 * A sequence whose row, slot, length or places lie outside the pool or its tail is skipped (its
 * outputs and its tail are left as they were) and records GLA_ERR_SHAPE in the device error word.
 * Each call returns once its work is queued on `stream`, may be captured into a graph (after a first
 * call of the library on the device), and needs no workspace except where it takes one. */
typedef enum { GLA_TAIL_PLAIN = 0, GLA_TAIL_MXFP8 = 1 } gla_tail_format;
typedef struct gla_tail {
  void* k;
  void* v;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int rows, cap, format;
} gla_tail;

/* One decode step for N sequences: with L = tail_len[n],
 *     o = scale (lambda^(L+1) S_p^T q + sum_{j < L} lambda^(L-j) (q . k_j) v_j + (q . k) v),
 * the readout after the token's own update, with the token's k and v as they are given; then k and
 * v are written to place L of the tail (quantised where it is MXFP8), which needs L < cap.
 * bf16 calls: sums in fp32; states, and the weights lambda^(L-j) (q . k_j), with 16 bits or more each, however far
 * apart the elements of a tail, its weights or its blocks lie; o rounded once.  fp32 calls: fp32 throughout.
 *   q, k [N, H, 96]; v, o [N, H, 192]; dtype `dtype`; N * H below 2^31.  One launch.
 * Tokens L from which a step over a state of its own (gla_tail_fold, then a decode step) moves fewer bytes:
 *     tail      fp32 pool   bf16 pool   MXFP8 pool
 *     bf16         256         128          66
 *     MXFP8        496         248         128
 * A tail's token is rounded once (MXFP8) or not at all; a bf16 or MXFP8 pool rounds the whole state at every step. */
int gla_prefix_decode_step(const void* q, const void* k, const void* v, const float* log_lambda, float scale,
                           const float* pool, int pool_rows, const int32_t* prefix_row, const gla_tail* tail,
                           const int32_t* tail_slot, const int32_t* tail_len, void* o, int N, int H, int dk, int dv,
                           int dtype, gla_stream_t stream);

/* Packed tokens written to the tails, and read back.
 *   k, v         packed [T, H, 96 / 192], dtype `dtype` (read by append, written by read).
 *   pos          [n_seq] int32 device: sequence n's tokens go to (come from) places pos[n],
 *                pos[n] + 1, ... of its tail (for an append, usually tail_len).
 *   cu_seqlens   [n_seq + 1] int32 device packed offsets, as in gla_chunk_fwd; rows from
 *                cu_seqlens[n_seq] on are left alone; offsets that decrease record GLA_ERR_SHAPE.  The row
 *                and places of a sequence without tokens are not looked at.  T <= 2^31 - 64.
 * An MXFP8 tail is quantised as it is written and widened as it is read: exactly, where dtype holds
 * the value (always, but for values of bf16's or fp32's subnormal range). */
int gla_tail_append(const void* k, const void* v, const gla_tail* tail, const int32_t* tail_slot, const int32_t* pos,
                    const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype, gla_stream_t stream);
int gla_tail_read(const gla_tail* tail, const int32_t* tail_slot, const int32_t* pos, const int32_t* cu_seqlens, void* k,
                  void* v, int n_seq, int T, int H, int dk, int dv, int dtype, gla_stream_t stream);

/* Tails folded into states of their own:
 *     out[out_row[n]] = lambda^L pool[prefix_row[n]] + sum_{j < L} lambda^(L-1-j) k_j v_j^T,
 * L = tail_len[n]; the state from which gla_decode_step, or more sequences, continue.
 *   out          [out_rows, H, 96, 192] fp32; out_row [N] int32 device, or NULL: row n (then
 *                out_rows >= N is required).  Rows must be distinct.  out may be the pool itself, and
 *                a sequence may be folded into the row it continues, as long as no other sequence of
 *                the call continues a row that the call writes.
 *   dtype        type of the tail's elements (GLA_TAIL_PLAIN).
 * Sums in fp32, of keys weighted in fp32: on the CUDA cores for fp32 tails, on the tensor cores (the
 * weighted key in three bf16 terms) for bf16 and MXFP8 ones. */
int gla_tail_fold(const float* log_lambda, const float* pool, int pool_rows, const int32_t* prefix_row,
                  const gla_tail* tail, const int32_t* tail_slot, const int32_t* tail_len, float* out, int out_rows,
                  const int32_t* out_row, int N, int H, int dk, int dv, int dtype, gla_stream_t stream);

/* gla_chunk_fwd and gla_chunk_bwd on packed sequences that continue shared states: sequence n's
 * initial state is pool[prefix_row[n]], read where it stands (no copies).  cu_seqlens is required;
 * every other argument as there.  A prefix_row outside the pool starts that sequence from zeros and
 * records GLA_ERR_SHAPE.  (bf16: as there, hT and dpool come from 16 bits of each operand, 2-3e-6 of the norm, and a
 * sequence's last chunk reads on into the next sequence with zero weights, so an infinity or a NaN in the first
 * 127 tokens of one can reach the one before.)
 *   dpool        [pool_rows, H, 96, 192] fp32 output, or NULL to skip: the pool's gradient, row p
 *                the sum of dh0 over the sequences that continue p, added in their order; zeros for
 *                a row that none continues.
 *   workspace    >= gla_workspace_bytes(n_seq, H) (forward) or gla_prefix_bwd_workspace_bytes(n_seq,
 *                T, H, dtype) bytes (backward: gla_chunk_bwd's and one state per sequence). */
int gla_prefix_fwd(const void* q, const void* k, const void* v, const float* log_lambda, const float* pool,
                   int pool_rows, const int32_t* prefix_row, float scale, void* o, float* hT,
                   const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype, void* workspace,
                   size_t ws_bytes, gla_stream_t stream);
size_t gla_prefix_bwd_workspace_bytes(int n_seq, int T, int H, int dtype);
int gla_prefix_bwd(const void* q, const void* k, const void* v, const float* log_lambda, const float* pool,
                   int pool_rows, const int32_t* prefix_row, float scale, const void* dO, const float* dhT, void* dq,
                   void* dk, void* dv, float* dpool, const int32_t* cu_seqlens, int n_seq, int T, int H, int dk_size,
                   int dv_size, int dtype, void* workspace, size_t ws_bytes, gla_stream_t stream);

/* The gated delta rule (no counterpart in the paper).  Per head the same 96 x 192 state, with a decay and a writing
 * strength of every token's own, both learned:
 *     S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   a_t = exp(g_t),
 *     o_t = S_t^T (scale q_t):
 * what the decayed state holds under the key is replaced, by the share beta_t, with the value.
 *   g, beta      [n_seq, T, H] (or packed [T_total, H]; [N, H] in the decode step), dtype `dtype`: the natural
 *                log of the decay (<= 0 in use; -inf allowed, a reset; values below -120 count as -120) and the
 *                strength.  beta times the squared length of k is meant to lie in [0, 2]: beyond that the
 *                recurrence itself grows.  (Keys of unit length and strengths in [0, 1] are the usual form.)  They
 *                and their gradients need the alignment of their type only: a slice of a packed array will do.
 * q, k, v, o, states, scale, cu_seqlens, dtype and the layouts are those of gla_chunk_fwd.  A call's tokens are
 * handled in chunks of 64; an infinity or a NaN in a token, or an infinity in a state, reaches every output of its chunk
 * and what follows it in its sequence and head (in the backward also what comes before), and nothing of another.  cu_seqlens is checked on the device: offsets that decrease or pass
 * T are clamped and record GLA_ERR_SHAPE.  Its last offset may stand below T (a step under its budget): the forward
 * leaves such rows of o as they were, the backward writes zeros to the gradients of such rows.
 * bf16 calls hold states in fp32 and what carries them from chunk to chunk in 16 to 24 bits (hT and dh0 are 0.2 to 1.2e-6
 * of the norm from the exact ones, up to 1e-5 where thousands of tokens forget nothing; where a state has been far larger
 * before, 3e-10 of its largest as well; where g is above 0, a state may grow by 2^8 within a chunk, which the fp32 call does
 * not ask).  o, dv and dbeta are their own
 * rounding away (1.7e-3 of the norm), dq and dk 1.7 to 2.3e-3, dg up to 2.9e-3: the states that they are made of are rounded
 * to bf16 on the way.  A caller who wants more makes the fp32 call on the same values: it keeps 22 bits of each operand of
 * a product, and everything else in fp32 (1 to 4e-7 of the norm, dg 8e-7).
 * Sizes: chunk places (n_seq * ceil(T / 64); packed T_total / 64 + n_seq) * H * 96, and rows of h0
 * and hT * H * 96, below 2^31, else GLA_ERR_SHAPE.
 * Workspaces: 33,344 bytes (fp32 34,048) for each chunk place and head in the forward, 235,520 (fp32 230,656) and 24 (48) a
 * token and head in the backward, which keeps every chunk's states: 0.14 GB and 1.0 GB (fp32 0.14 and 0.96) for 16,384
 * tokens of 16 heads in one sequence, in proportion to the tokens.
 * Calls may be captured into a graph after a first call of the same kind on the device; calls that may overlap need
 * workspaces of their own. */

/* Chunked forward.
 *   h0           [h0_rows, H, 96, 192] fp32 initial states, or NULL for zeros.
 *   h0_row       [n_seq] int32 device: sequence n starts from row h0_row[n] (rows may repeat), from zeros where it
 *                is -1; NULL = row n (then h0_rows >= n_seq).  Any other row outside h0 records GLA_ERR_SHAPE and
 *                starts from zeros.
 *   hT           [hT_rows, H, 96, 192] fp32 final states, or NULL to skip; hT_row [n_seq] int32 device: their
 *                rows, distinct, -1: not wanted; NULL = row n.  Any other row outside hT records GLA_ERR_SHAPE and
 *                is not written.  hT may be h0: a sequence may end in the row that it started from, as long as no
 *                other sequence of the call starts from a row that it writes.  Rows that no sequence has are left.
 *   workspace    >= gla_delta_workspace_bytes(n_seq, T, H, cu_seqlens != NULL, dtype) bytes.
 * A sequence without tokens ends in the state it starts from. */
size_t gla_delta_workspace_bytes(int n_seq, int T, int H, int packed, int dtype);
int gla_delta_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                  int h0_rows, const int32_t* h0_row, float scale, void* o, float* hT, int hT_rows,
                  const int32_t* hT_row, const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype,
                  void* workspace, size_t ws_bytes, gla_stream_t stream);

/* Chunked backward: gradients of L(o, hT) given dO = dL/do and dhT = dL/dhT.
 *   h0           [n_seq, H, 96, 192] fp32, or NULL for zeros; dhT the same, or NULL for zeros.
 *   dq, dk, dv   outputs, layouts of q, k, v; dg, dbeta outputs, layout of g; all of dtype `dtype`.
 *   dh0          [n_seq, H, 96, 192] fp32 output, or NULL to skip.
 *   workspace    >= gla_delta_bwd_workspace_bytes(n_seq, T, H, cu_seqlens != NULL, dtype) bytes.
 * The chunks' states are computed again; nothing of gla_delta_fwd is needed.  No sum depends on an order of
 * arrival: the same call gives the same bits. */
size_t gla_delta_bwd_workspace_bytes(int n_seq, int T, int H, int packed, int dtype);
int gla_delta_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                  float scale, const void* dO, const float* dhT, void* dq, void* dk, void* dv, void* dg, void* dbeta,
                  float* dh0, const int32_t* cu_seqlens, int n_seq, int T, int H, int dk_size, int dv_size, int dtype,
                  void* workspace, size_t ws_bytes, gla_stream_t stream);

/* One decode step for N sequences, in place on a pool of states, fp32 or (_bf16_state) bf16.
 *   q, k [N, H, 96]; v, o [N, H, 192]; g, beta [N, H]; state, slot, pool_rows as in gla_decode_step (rows distinct),
 *   but that a slot of -1 leaves its sequence alone (state and o untouched) without an error.  N * H below 2^31.
 * The readout uses the update before a bf16 pool rounds it.  Every sequence goes on from what its row holds: a row that
 * was another sequence's has to be cleared first, or left to the call below. */
int gla_delta_decode_step(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                          float* state, const int32_t* slot, int pool_rows, void* o, int N, int H, int dk, int dv,
                          int dtype, gla_stream_t stream);
int gla_delta_decode_step_bf16_state(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                     float scale, void* state, const int32_t* slot, int pool_rows, void* o, int N,
                                     int H, int dk, int dv, int dtype, gla_stream_t stream);

/* The same step where a sequence's state need not stand in the row that it ends in.
 *   state_dtype  GLA_F32 or GLA_BF16, the pool's type.
 *   start_row    [N] int32 device: the row that sequence n goes on from; -1: from zeros, and what the row of its slot
 *                holds is not read (not even a NaN); NULL: its slot's row.  Rows may repeat, and may be other rows than
 *                slot[n], as long as no other sequence of the call writes them.  Any other row outside the pool records
 *                GLA_ERR_SHAPE and starts from zeros.  Where slot is -1 the sequence is left alone as above. */
int gla_delta_decode_step_rows(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                               void* state, int state_dtype, const int32_t* slot, const int32_t* start_row, int pool_rows,
                               void* o, int N, int H, int dk, int dv, int dtype, gla_stream_t stream);

/* One serving step's maps, built on the device from the requests' lengths, so that a step needs no host
 * synchronisation (and can be captured: all sizes are fixed).
 *   new_len      [N] int32 device: tokens that request n brings; 0: none now (it keeps its row); negative: it has
 *                finished, and its row is free.
 *   held         [N] int32 device: the pool row that request n holds, -1: none.  Rows distinct (a row held twice
 *                records GLA_ERR_SHAPE).  Any other row outside [0, pool_rows) records GLA_ERR_SHAPE, and the
 *                request gets no row and no tokens.
 *   seen         [N] int32 device: tokens before this step, or NULL for zeros (used by token_pos).
 * Requests are served in order: one that brings tokens and holds no row takes the lowest free one (without one it gets
 * no tokens); each gets its tokens until `budget` tokens are handed out, the one at the limit a part of them.
 *   cu_seqlens   [N + 1]: packed offsets of the tokens handed out.
 *   slot         [N]: row of a request that has tokens in this step, else -1 (hT_row, and the decode step's slot).  A row that
 *                has become free is the next request's, and holds what the last one left: start_row goes with it.
 *   start_row    [N]: the row it goes on from, -1 where it is new or has no tokens (h0_row, and
 *                gla_delta_decode_step_rows' start_row).
 *   row          [N]: the row it holds after the step, -1: none (the next step's held).
 *   token_seq, token_pos   [budget]: request and place (seen + the place in this step) of each packed token, -1
 *                behind the last; both or neither NULL.
 * Inputs and outputs must not overlap, but that row may be held.  pool_rows from 1 to GLA_PLAN_MAX_ROWS, N up to
 * GLA_PLAN_MAX_REQUESTS, budget (where token_seq and token_pos are given) up to GLA_PLAN_MAX_BUDGET; else GLA_ERR_SHAPE
 * (too small) or GLA_ERR_UNSUPPORTED (too large).  Pointers 4-byte aligned. */
#define GLA_PLAN_MAX_ROWS (1 << 19)
#define GLA_PLAN_MAX_REQUESTS (1 << 20)
#define GLA_PLAN_MAX_BUDGET (1 << 30)
int gla_slot_plan(const int32_t* new_len, const int32_t* held, const int32_t* seen, int N, int pool_rows, int budget,
                  int32_t* cu_seqlens, int32_t* slot, int32_t* start_row, int32_t* row, int32_t* token_seq,
                  int32_t* token_pos, gla_stream_t stream);

/* Synchronises `stream`, then returns and clears the current device's sticky error word:
 * GLA_OK, GLA_ERR_TIMEOUT or GLA_ERR_SHAPE (or, in the debug-bounds build, GLA_ERR_BOUNDS);
 * GLA_ERR_LAUNCH if the stream itself failed.
 * There is one word per device, shared by every caller of the library on that device: the first
 * fault recorded since the last read is kept, and whichever caller reads next sees and clears it. */
int gla_get_device_error(gla_stream_t stream);

/* 1 in the library's debug-bounds build (libgla_debug.so, compiled with GLA_DEBUG_BOUNDS), 0 in
 * the release build (libgla.so).  The debug-bounds build is the same library with device-side
 * index checks at the kernels' computed global accesses (state rows, output and gradient rows,
 * partial-sum rows, packed-order and segment lookups, hand-over flags, TMA coordinates): an index
 * outside its buffer records GLA_ERR_BOUNDS in the device error word and the access is skipped.
 * It stands in for a memory checker; its results equal the release build's. */
int gla_debug_bounds(void);

/* Upper bound, in nanoseconds, of every device-side wait on an mbarrier (default 2e9).  A wait
 * that exceeds it records GLA_ERR_TIMEOUT, drains the copies its CTA has in flight, releases
 * tensor memory and returns.  Meant for tests of that path; applies to the current device. */
int gla_set_wait_limit_ns(unsigned long long ns);

/* For tests of that path, debug-bounds build only (GLA_ERR_UNSUPPORTED in the release build): from now on one
 * warp of every CTA of gla_prefix_decode_step's bf16 kernel (its second) and of gla_tail_fold's bf16 and MXFP8
 * kernel gives up its wait for chunk `chunk` (of its own, from 0; below 4,096) as if the limit had passed.  role:
 * the decode's wait for keys (0) or values (1); the fold's issuing (0), widening (1; from chunk 2 on) or, for the
 * last chunk, storing warps (2).  In the bf16 kernels of gla_delta_fwd and gla_delta_bwd `chunk` is 1024 x kernel (0: prep,
 * 1: either scan, 2: reverse scan, 3: gradients) + 32 x the mbarrier's number + its phase (below 32), and those of the
 * role that wait for it give up: the thread of the copies (0), that of the products (1) or the other warps (2).
 * role -1: no more. */
int gla_debug_give_up(int role, int chunk);

/* Human-readable name of a gla_status value. */
const char* gla_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* GLA_H_ */
