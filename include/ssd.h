/*
 * libssd: Mamba-2 structured-state-space-duality (SSD) chunked-scan forward
 * pass for NVIDIA GB300 (sm_103a), its backward pass and decoding step, and the operators around it (residual
 * norm, projection, gated recurrence).  C ABI: plain pointers and sizes only.
 *
 * The operation ("State Space Duality and Mamba-2", sections "The
 * Mathematical Bridge" and "The SSD Block Decomposition Algorithm"; the
 * discretisation is the selective-scan one of "NVIDIA Accelerates Mamba-2
 * Forward Kernel with CUDA Tile", where the decay and input matrices depend
 * on the step size dt):  per batch row b and head h, with group
 * g = h / (H / G),
 *
 *     h_t = exp(dt_t * A_h) * h_{t-1} + dt_t * x_t B_t^T        (P x N state)
 *     y_t = h_t C_t + D_h * x_t
 *
 * computed chunk by chunk: the intra-chunk block ((C B^T) o L) X with the
 * 1-semiseparable decay mask L_ij = exp(sum_{k=j+1..i} dt_k A_h), chunk
 * states B^T (decay o X), inter-chunk state passing and the off-diagonal
 * output C * state.  A sequence may also be cut into splits of split_len
 * tokens that run in parallel and are joined by composing their states
 * ("GPU Hierarchy Meets Structured Matrices", abstract: the split-sequence
 * algorithm; "Parallel Scan and Hardware-Aware SSM Kernels", "The scan": the
 * affine-step composition).  Packed documents (cu_seqlens) restart the state
 * at every document start (same page, "When it breaks"): document d starts
 * from initial_states[d] (or zero), which its first token decays like any
 * carried state.
 *
 * Layouts (all row-major, contiguous, device memory, 16-byte aligned bases):
 *   x, y            (batch, seqlen, nheads, headdim)      dtype
 *   dt              (batch, seqlen, nheads)               fp32, >= 0 (post-softplus)
 *   A, D            (nheads)                              fp32 (A <= 0; D optional)
 *   B, C            (batch, seqlen, ngroups, dstate)      dtype
 *   initial_states  (nstates, nheads, headdim, dstate)    fp32, optional (zeros)
 *   final_states    (nstates, nheads, headdim, dstate)    fp32, optional
 *   cu_seqlens      (ndocs + 1) int32, cu[0] = 0 < cu[1] < ... < cu[ndocs] = seqlen
 *                   (no empty document), optional.  The offsets are in device
 *                   memory, so the host cannot check them; the last launch of
 *                   ssd_fwd() / ssd_bwd() does, and records SSD_ERR_DEVICE_CHECK
 *                   (where 40) in the workspace status word when they break
 *                   this rule.  The kernels keep every index in bounds either
 *                   way; the outputs are then undefined.
 *   nstates = ndocs when cu_seqlens is given (then batch must be 1), else batch.
 *
 * Ownership: the caller owns every buffer; the library keeps no pointer past
 * a call and allocates no device memory.  Calls are asynchronous on the given
 * stream (a cudaStream_t passed as void*; NULL = legacy default stream).
 *
 * Errors: argument errors return a status before anything is launched and
 * nothing is written.  A failed launch returns SSD_ERR_CUDA.  Errors found on
 * the device (a bounded wait that ran out) are recorded in a status word at
 * the start of the workspace and are read by ssd_check_status().
 */
#ifndef SSD_H_
#define SSD_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SSD_API __attribute__((visibility("default")))
#else
#define SSD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SSD_OK = 0,
    SSD_ERR_INVALID_ARG = 1,   /* bad pointer, size, alignment or layout */
    SSD_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. chunk 256) */
    SSD_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
    SSD_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
    SSD_ERR_TIMEOUT = 5,       /* a device-side bounded wait ran out */
    SSD_ERR_DEVICE_CHECK = 6   /* a device-side consistency check failed (cu_seqlens) */
} ssd_status_t;

typedef enum {
    SSD_F32 = 0,
    SSD_BF16 = 1,
    SSD_E4M3 = 2   /* 8 bits (4 exponent, 3 mantissa, largest 448): ssd_add_norm's rows, ssd_linear's operands */
} ssd_dtype_t;

typedef struct {
    int64_t batch;      /* batch rows (1 when cu_seqlens is given)                  */
    int64_t seqlen;     /* tokens per row (total packed length with cu_seqlens)      */
    int32_t nheads;     /* H                                                         */
    int32_t headdim;    /* P                                                         */
    int32_t dstate;     /* N                                                         */
    int32_t ngroups;    /* G, H % G == 0; head h reads B, C of group h / (H / G)     */
    int32_t chunk;      /* Q: 64 or 128                                              */
    int32_t split_len;  /* tokens per split: a multiple of chunk; 0 = automatic;
                           >= seqlen = one split.  Never changes the result beyond
                           rounding.                                                 */
    int32_t ndocs;      /* documents when cu_seqlens is given, else 0                */
    int32_t dtype;      /* ssd_dtype_t of x, B, C and y                              */
} ssd_params_t;

/* Bytes of device workspace ssd_fwd() needs for these parameters (>= 256:
 * the first 256 bytes hold the device status word).  0 on invalid params. */
SSD_API size_t ssd_fwd_workspace_size(const ssd_params_t* p);

/* Zero the workspace's status word (async on `stream`).  Call once after
 * allocating a workspace; the status word then stays zero until a device
 * error is recorded, and ssd_check_status() clears it again. */
SSD_API int ssd_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/* The SSD forward pass: y (and optionally final_states) from x, dt, A, B, C
 * and the optional D, initial_states and cu_seqlens, as defined above.
 * `workspace` is device scratch of at least ssd_fwd_workspace_size(p) bytes,
 * initialised once by ssd_workspace_init(); calls that share a workspace must
 * be ordered on one stream.  y must not alias any input.  final_states may
 * alias initial_states.  Bitwise deterministic for fixed inputs and params. */
SSD_API int ssd_fwd(const ssd_params_t* p,
            const void* x, const float* dt, const float* A,
            const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* cu_seqlens,
            void* y, float* final_states,
            void* workspace, size_t workspace_bytes, void* stream);

/* ssd_fwd() for measurement: the same call, with a CUDA event recorded on
 * `stream` before and after each of its kernel launches.  Synchronises on the
 * last event, writes the first min(launches, max_launches) launch durations in
 * milliseconds to ms_per_launch (in launch order: for split plans the
 * aggregate pass, the composition, then the full pass) and the launch count
 * to *nlaunches.  Creates and destroys its events on every call: meant for
 * benchmarks, not for the hot path.  Errors as ssd_fwd(); SSD_ERR_INVALID_ARG
 * when ms_per_launch or nlaunches is NULL or max_launches < 1. */
SSD_API int ssd_fwd_timed(const ssd_params_t* p,
            const void* x, const float* dt, const float* A,
            const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* cu_seqlens,
            void* y, float* final_states,
            void* workspace, size_t workspace_bytes, void* stream,
            float* ms_per_launch, int max_launches, int* nlaunches);

/* ssd_fwd() for callers that cannot allocate device memory (for example a
 * plugin inside a host application that owns every device allocation, or a
 * C caller that only holds the input and output pointers it was given).
 * The paper has no counterpart of this entry point.
 *
 * Same operation, arguments and layouts as ssd_fwd(), without a workspace:
 * the workspace is a library-owned device array of 8 MiB that every GPU
 * loading the library reserves until process exit.  Problems whose
 * ssd_fwd_workspace_size() exceeds 8 MiB are rejected with
 * SSD_ERR_WORKSPACE before anything is launched; single-split problems need
 * less than 4.01 MiB: the 256-byte status header, the pieces' log-decays
 * (4 bytes each, rounded up to 256 bytes) and their states (at most 4 MiB),
 * for the pieces the leftover-unit plan cuts the last wave's units into.  The
 * caller still passes all inputs and outputs.
 * The first call on a device looks up the array's device address with that
 * device current (cudaGetSymbolAddress) and keeps it for the life of the
 * process; make no call after resetting the device (cudaDeviceReset), which
 * invalidates the kept address.  Every call uses the same array: calls whose GPU work
 * overlaps (other streams or other host threads) race on it.  The call
 * clears the status word, enqueues the work on `stream`, then synchronises
 * the stream and returns the device status (SSD_OK or the first device
 * error).  It calls no allocating routine. */
SSD_API int ssd_fwd_static_scratch(const ssd_params_t* p,
            const void* x, const float* dt, const float* A,
            const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* cu_seqlens,
            void* y, float* final_states, void* stream);

/* Bytes of device workspace ssd_bwd() needs for these parameters; 0 when the
 * parameters are invalid or the backward pass does not support them. */
SSD_API size_t ssd_bwd_workspace_size(const ssd_params_t* p);

/* Bytes of device workspace ssd_bwd() needs for packed documents (ndocs > 0)
 * when the call passes initial_states, dfinal_states or dinitial_states: that
 * call runs one unit per (head, document), in chunks from each document's first
 * token (on the tensor cores for their shape, 128 tokens; else on CUDA cores,
 * at most 32), so its chunk-state layout holds up to ndocs more chunks per head
 * than whole rows need.
 * 0 when the parameters are invalid, ndocs is 0 or the backward pass does not
 * support them. */
SSD_API size_t ssd_bwd_workspace_size_doc_states(const ssd_params_t* p);

/* Backward pass of ssd_fwd(): the gradients of the scalar
 *     <dy, y> + <dfinal_states, final_states>
 * with respect to every input, where y and final_states are ssd_fwd()'s outputs
 * for the same inputs.  The states are recomputed from the inputs, as "Parallel
 * Scan and Hardware-Aware SSM Kernels" ("Why the kernel matters more than the
 * algorithm") describes: only the state entering each backward chunk is kept, in
 * the workspace.  bf16 with headdim 64 and dstate 128 (the Mamba-2 head
 * shape) runs on the tensor cores: chunks of 128 tokens, every contraction a
 * bf16 x bf16 -> fp32 MMA (the decay-masked Q x Q products, the adjoint and
 * the incoming state are rounded to bf16 as MMA operands; sums, scans and
 * the adjoint recurrence stay fp32).  When rows x heads leave SMs idle it
 * cuts each sequence into splits that run in parallel ("GPU Hierarchy Meets
 * Structured Matrices": the split-sequence algorithm, here for the adjoint
 * too): the forward pass's split aggregates and their composition give the
 * state entering each split, and reverse aggregates (sum of 2^{P_i} dy_i C_i^T
 * over a split, P_i the log-decays from the split's start through i) composed
 * from dfinal_states give the adjoint leaving it.  split_len in p sets the
 * split (0: automatic; rounded up to a multiple of 128, at least 512).  Every other shape, and fp32, runs on
 * CUDA cores in fp32 (bf16 inputs widened, bf16 gradients rounded once at the
 * end).
 *
 * Inputs: x, dt, A, B, C, D (optional), initial_states (optional: zeros) exactly
 * as for ssd_fwd(); dy (batch, seqlen, nheads, headdim) dtype;
 * dfinal_states (batch, nheads, headdim, dstate) fp32 or NULL (zeros); with
 * cu_seqlens, initial_states, dfinal_states and dinitial_states are per
 * document, (ndocs, nheads, headdim, dstate).
 * Outputs (written, not accumulated into):
 *   dx               (batch, seqlen, nheads, headdim)   dtype
 *   ddt              (batch, seqlen, nheads)            fp32
 *   dA               (nheads)                           fp32
 *   dB, dC           (batch, seqlen, ngroups, dstate)   dtype (summed over each group's heads)
 *   dD               (nheads) fp32, or NULL; written only when D is given
 *   dinitial_states  (batch, nheads, headdim, dstate)   fp32, or NULL
 * All pointers are device memory with 16-byte aligned bases; no output may equal
 * an input.  Packed documents (cu_seqlens with ndocs, batch 1; strictly
 * increasing, from 0 to seqlen) are independent sequences: no state and no
 * gradient crosses a document boundary.  Without per-document states the
 * tensor-core path for its shape runs whole rows (a -inf log-decay at each
 * document start); with initial_states, dfinal_states or dinitial_states every
 * path runs one unit per (head, document), walking the document's own chunks
 * from its first token: each document
 * starts from its initial state (its first token's decay applied to it), its
 * final state receives dfinal_states[d], and dinitial_states[d] is the
 * gradient of initial_states[d].  headdim * dstate > 8192 and shapes whose
 * tiles do not fit in shared memory return SSD_ERR_UNSUPPORTED.
 * `chunk` and `split_len` in p are validated; they change only the rounding.
 * `workspace`: at least ssd_bwd_workspace_size(p) bytes, or
 * ssd_bwd_workspace_size_doc_states(p) for packed documents with any of the
 * three states, 256-byte aligned (else SSD_ERR_WORKSPACE).  Asynchronous on `stream`; a status-word reset
 * and two launches (six with splits: the two aggregate passes and their
 * compositions first).  The tensor-core path's device waits are bounded: one that
 * runs out records SSD_ERR_TIMEOUT (where codes 31-39, or 21-26 from the
 * split aggregates) in the status word at
 * the start of `workspace`, read by ssd_check_status(); the CUDA-core path has
 * no device waits.  Bitwise deterministic (fixed summation orders). */
SSD_API int ssd_bwd(const ssd_params_t* p,
            const void* x, const float* dt, const float* A,
            const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* cu_seqlens,
            const void* dy, const float* dfinal_states,
            void* dx, float* ddt, float* dA, void* dB, void* dC, float* dD,
            float* dinitial_states,
            void* workspace, size_t workspace_bytes, void* stream);

/* Gated RMS normalisation of the scan's output in one pass ("NVIDIA Accelerates
 * Mamba-2 Forward Kernel with CUDA Tile", operator fusion: the scan is followed
 * by gating and normalisation, fused so the gated values never leave the chip).
 * For each row r and each group of group_size consecutive channels:
 *
 *     g[r,k]   = y[r,k] * silu(z[r,k]),   silu(v) = v / (1 + exp(-v))
 *     out[r,k] = g[r,k] / sqrt(mean_{k' in group} g[r,k']^2 + eps) * weight[k]
 *
 * (the Mamba-2 block's output gate and its grouped RMS norm, gate applied before
 * the norm).  Layouts: y, z, out (rows, width) dtype, row-major, contiguous,
 * 16-byte aligned; weight (width) fp32, 16-byte aligned.  rows = batch * seqlen and width =
 * nheads * headdim for ssd_fwd's y.  width must be a multiple of group_size;
 * group_size a multiple of 8 (bf16) or 4 (fp32) and at most 8192 (else
 * SSD_ERR_UNSUPPORTED); eps >= 0 and finite.  out may be y itself (in place).
 * One launch on `stream`, no workspace; bitwise deterministic. */
SSD_API int ssd_gate_norm(int64_t rows, int32_t width, int32_t group_size, int32_t dtype,
             const void* y, const void* z, const float* weight, float eps, void* out, void* stream);

/* Root-mean-square norm with the residual's addition, in one pass: the pre-norm
 * of a layer, which also carries the residual stream.  Per row r of `width`
 * elements:
 *
 *     h[k]   = x[k] + residual[k]                 (residual NULL: h = x)
 *     rstd   = 1 / sqrt(mean_k h[k]^2 + eps)
 *     out[k] = h[k] * rstd * weight[k]
 *
 * out_dtype is dtype, or SSD_E4M3: then scales[r] = max(max_k |out[k]|, 1e-30) / 448
 * and out holds the fp32 quotient out[k] / scales[r], rounded to nearest even.  h is normalised as it was summed (fp32),
 * before it is rounded to residual_out's type.
 *   x             (rows, width) dtype (SSD_F32 or SSD_BF16)
 *   residual      (rows, width) residual_dtype, or NULL.  residual_dtype is SSD_F32,
 *                 or SSD_BF16 where dtype is.
 *   weight        (width) fp32
 *   out           (rows, width) out_dtype; may be x where the types are equal
 *   scales        (rows) fp32, for SSD_E4M3 (ignored otherwise)
 *   residual_out  (rows, width) residual_dtype, or NULL; may be residual (in place), or x where the types are equal
 *   rstd          (rows) fp32, or NULL: kept for ssd_add_norm_bwd()
 * Row-major, contiguous, each base aligned to its element (16-byte aligned bases
 * and widths of whole 16-byte vectors of x run faster).  rows >= 0 (0: nothing is launched); 1 <=
 * width <= 16384 (else SSD_ERR_UNSUPPORTED).  A NaN or an infinity makes its whole row NaN or
 * zero as the formula does.  One launch, no workspace; bitwise deterministic. */
SSD_API int ssd_add_norm(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, int32_t out_dtype,
             const void* x, const void* residual, const float* weight, float eps,
             void* out, float* scales, void* residual_out, float* rstd, void* stream);

/* Bytes of device workspace ssd_add_norm_bwd() needs (0 on invalid sizes or rows == 0). */
SSD_API size_t ssd_add_norm_bwd_workspace_size(int64_t rows, int32_t width);

/* Gradients of ssd_add_norm() (with out_dtype == dtype): of <dout, out> + <dresidual_out, residual_out>.
 * With xh = h * rstd and p = weight * dout,
 *
 *     dh = rstd * (p - xh * mean_k(p * xh)) + dresidual_out
 *     dweight = sum_rows dout * xh
 *
 * and dh is the gradient of x and of residual alike.
 *   dout           (rows, width) dtype
 *   h              (rows, width) residual_dtype: the forward's residual_out (or x where it had no residual)
 *   rstd           (rows) fp32, from the forward
 *   dresidual_out  (rows, width) residual_dtype, or NULL (zeros)
 *   dx             (rows, width) dtype, or NULL;          may be dout
 *   dresidual      (rows, width) residual_dtype, or NULL; may be dresidual_out
 *   dweight        (width) fp32, written
 * At least one of dx and dresidual is given.  Other layouts as ssd_add_norm(); rows == 0 writes zeros to dweight.
 * `workspace`: ssd_add_norm_bwd_workspace_size() bytes, 16-byte aligned.
 * Two launches; bitwise deterministic (dweight is summed in a fixed order). */
SSD_API int ssd_add_norm_bwd(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype,
             const void* dout, const void* h, const float* weight, const float* rstd, const void* dresidual_out,
             void* dx, void* dresidual, float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/* 8-bit rows, for activations that the backward pass reads again: each row's group of group_size columns
 * (group_size divides width; width: one scale a row) becomes e4m3 numbers and a scale,
 *
 *     scale = the smallest power of two with max |x| <= 448 scale over the group's finite x, at least 2^-108
 *     codes = x / scale, rounded once to nearest even;   an infinity or a NaN becomes NaN
 *
 * and stands for codes * scale, which is exact in bf16 and fp32.
 *   x        (rows, width) dtype (SSD_F32 or SSD_BF16), x_stride elements between rows (>= width)
 *   codes    (rows, width) e4m3, contiguous;  scales (rows, width / group_size) fp32
 * Bases aligned to their elements (16-byte aligned ones, with sizes and strides of whole 16-byte vectors of x, run faster);
 * no output may overlap an input.  rows >= 0 (0: nothing is launched), rows * groups < 2^31, group_size <= 16384, width and x_stride
 * < 2^30 (else SSD_ERR_UNSUPPORTED).  One launch, no workspace; bitwise deterministic. */
SSD_API int ssd_pack_rows(int64_t rows, int32_t width, int32_t group_size, int32_t dtype, int64_t x_stride,
             const void* x, void* codes, float* scales, void* stream);

/* out = codes * scale in fp32, then in dtype (both exact for the scales of ssd_pack_rows()).  codes, scales and limits
 * as there (any group_size that divides width); out (rows, width) contiguous. */
SSD_API int ssd_unpack_rows(int64_t rows, int32_t width, int32_t group_size, int32_t dtype,
             const void* codes, const float* scales, void* out, void* stream);

/* The gate and norm after the scan (ssd_gate_norm()) in training: with u = y * silu(z) per row and group of
 * group_size columns,
 *
 *     out = u * rstd * weight,   rstd = 1 / sqrt(mean_group(u^2) + eps),   silu(z) = z / (1 + exp(-z)) */
typedef struct {
    int64_t rows;
    int64_t z_stride;   /* elements between rows of z, >= width (z may be a column range of a projection's rows) */
    int64_t dz_stride;  /* ... of dz                                                                             */
    int32_t width;
    int32_t group_size; /* divides width; at most 8192 (else SSD_ERR_UNSUPPORTED)                                */
    int32_t dtype;      /* SSD_F32 or SSD_BF16: of out, dout, dy, dz, and of y and z unless they are 8-bit rows   */
    float eps;          /* >= 0, finite                                                                          */
} ssd_gate_norm_params_t;

/* out as above, and y and z as 8-bit rows for the backward pass (one scale a row and group).
 *   y (rows, width) dtype contiguous;  z (rows, width) dtype, row stride z_stride;  weight (width) fp32
 *   out (rows, width) dtype;  y_codes, z_codes (rows, width) e4m3;  y_scales, z_scales (rows, width / group_size) fp32
 * All contiguous but z; limits, alignment and overlaps as for ssd_pack_rows().  One launch, no workspace; bitwise deterministic. */
SSD_API int ssd_gate_norm_pack(const ssd_gate_norm_params_t* p, const void* y, const void* z, const float* weight,
             void* out, void* y_codes, float* y_scales, void* z_codes, float* z_scales, void* stream);

/* Gradients of <dout, out>.  With p = dout * weight and n = u * rstd,
 *
 *     du = rstd (p - n mean_group(p n));   dy = du silu(z);   dz = du y s (1 + z (1 - s)), s = 1 / (1 + exp(-z))
 *     dweight = sum_rows dout n
 *
 *   y, z               dtype, or e4m3 codes where y_scales, z_scales (one a row and group) are given; codes are contiguous
 *                      (z_stride == width)
 *   dout, dy           (rows, width) dtype, contiguous;  dz (rows, width) dtype, row stride dz_stride (it may be a
 *                      column range of a projection's gradient; columns outside of it are left alone)
 *   out                (rows, width) dtype, or NULL: the forward's result, computed again
 *   dweight            (width) fp32, written (zeros where rows == 0)
 * Sums are fp32, of u, or of codes * silu(z) with the scale joined to each thread's (8 or 16 elements): gates from 1e16 on may overflow
 * them.  One of y and z in 8 bits and the other not is slower (single elements instead of vectors).
 * `workspace`: ssd_gate_norm_bwd_workspace_size() bytes (0 on invalid parameters or rows == 0), 16-byte aligned, needs no
 * initialisation; calls that share it must be ordered on one stream.  No output may overlap an input.  Two launches;
 * bitwise deterministic (dweight is summed in a fixed order). */
SSD_API size_t ssd_gate_norm_bwd_workspace_size(const ssd_gate_norm_params_t* p);
SSD_API int ssd_gate_norm_bwd(const ssd_gate_norm_params_t* p, const void* dout, const void* y, const float* y_scales,
             const void* z, const float* z_scales, const float* weight, void* dy, void* dz, void* out, float* dweight,
             void* workspace, size_t workspace_bytes, void* stream);

/* The norm after a block, with the block's gate, the scaled addition to the residual stream and the next block's
 * norm, in one pass.  Per row:
 *
 *     u   = x * silu(gate)                                     (gate NULL: u = x)
 *     h   = residual + scale * (u * rstd1 * weight),           rstd1 = 1 / sqrt(mean(u^2) + eps)
 *     out = h * rstd2 * next_weight,                           rstd2 = 1 / sqrt(mean(h^2) + eps)  (h unrounded)
 */
typedef struct {
    int64_t rows;
    int64_t gate_stride;     /* elements between rows of gate, >= width (ignored without a gate) */
    int64_t dgate_stride;    /* ... of dgate                                                     */
    int32_t width;           /* 1 to 8192 (else SSD_ERR_UNSUPPORTED)                             */
    int32_t dtype;           /* SSD_F32 or SSD_BF16: of x, gate, dout, dx, dgate, and of out     */
    int32_t residual_dtype;  /* SSD_F32, or SSD_BF16 where dtype is: of residual, h, dresidual   */
    int32_t out_dtype;       /* dtype, or SSD_E4M3: out as 8-bit rows                            */
    float scale;             /* finite                                                           */
    float eps;               /* >= 0, finite                                                     */
} ssd_block_norm_params_t;

/*   x         (rows, width) dtype;  gate (rows, width) dtype, row stride gate_stride, or NULL
 *   residual  (rows, width) residual_dtype;  residual_out (h) of the same type, may be residual (in place)
 *   weight, next_weight (width) fp32; next_weight NULL: no second norm, and out and out_scales are ignored
 *   out       (rows, width) out_dtype;  out_scales (rows) fp32, with SSD_E4M3: rows as ssd_pack_rows() makes them
 *   x_codes (rows, width) e4m3, x_scales (rows) fp32 (and gate_codes, gate_scales with a gate): x and gate as 8-bit rows for
 *             the backward pass, all given or all NULL
 * All contiguous but gate; limits, alignment and (but for residual_out) overlaps as for ssd_pack_rows().  One launch, no
 * workspace; bitwise deterministic. */
SSD_API int ssd_block_norm(const ssd_block_norm_params_t* p, const void* x, const void* gate, const void* residual,
             const float* weight, const float* next_weight, void* residual_out, void* out, float* out_scales,
             void* x_codes, float* x_scales, void* gate_codes, float* gate_scales, void* stream);

/* Gradients of <dout, out> + <dresidual_out, residual_out>.  With p2 = dout * next_weight and n2 = h rstd2,
 *
 *     dh = dresidual_out + rstd2 (p2 - n2 mean(p2 n2))         (no next_weight: dh = dresidual_out)
 *     p1 = scale dh weight, n1 = u rstd1:  du = rstd1 (p1 - n1 mean(p1 n1))
 *     dx = du silu(gate), dgate = du x s (1 + gate (1 - s)), s = 1 / (1 + exp(-gate));   dresidual = dh
 *     dweight = sum_rows scale dh n1;   dnext_weight = sum_rows dout n2
 *
 *   x, gate, h      as the forward had and left them (h: its residual_out), or e4m3 codes where x_scales, gate_scales, h_scales
 *                   (one a row) are given; codes are contiguous.  h is ignored without next_weight
 *   dout            (rows, width) dtype, given with next_weight and only then
 *   dresidual_out   (rows, width) residual_dtype
 *   dx, dgate       (rows, width) dtype; dgate (with a gate) row stride dgate_stride;  dresidual (rows, width) residual_dtype
 *   dweight, dnext_weight  (width) fp32, written
 * `workspace`: ssd_block_norm_bwd_workspace_size() bytes (enough with and without next_weight).  Otherwise as for
 * ssd_gate_norm_bwd(). */
SSD_API size_t ssd_block_norm_bwd_workspace_size(const ssd_block_norm_params_t* p);
SSD_API int ssd_block_norm_bwd(const ssd_block_norm_params_t* p, const void* dout, const void* dresidual_out,
             const void* x, const float* x_scales, const void* gate, const float* gate_scales, const void* h, const float* h_scales,
             const float* weight, const float* next_weight, void* dx, void* dgate, void* dresidual, float* dweight,
             float* dnext_weight, void* workspace, size_t workspace_bytes, void* stream);

/* Matrix product with its epilogue, for the projections before and after the scan:
 *
 *     v[m,n] = sx[m] sw[n] sum_k x[m,k] w[n,k] + bias[n]       (the scales with SSD_E4M3 only)
 *     y[m,n] = act(v[m,n]) + residual[m,n]
 *
 * silu(v) = v / (1 + exp(-v));  gelu(v) = v / 2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))). */
typedef enum { SSD_ACT_NONE = 0, SSD_ACT_SILU = 1, SSD_ACT_GELU = 2 } ssd_act_t;
typedef struct {
    int64_t m;      /* rows of x and y (0: nothing is launched)                                        */
    int64_t ldx;    /* elements from one row of x to the next, >= k (x may be a column range)          */
    int32_t n;      /* columns of y, rows of w                                                         */
    int32_t k;      /* columns of x and w                                                              */
    int32_t dtype;  /* of x and w: SSD_BF16, or SSD_E4M3 with scales                                   */
    int32_t act;    /* ssd_act_t                                                                       */
} ssd_linear_params_t;

/* Bytes of device workspace for ssd_linear() and ssd_linear_bwd(); 0 on invalid parameters (bwd: also
 * unless dtype is SSD_BF16). */
SSD_API size_t ssd_linear_workspace_size(const ssd_linear_params_t* p);
SSD_API size_t ssd_linear_bwd_workspace_size(const ssd_linear_params_t* p);

/* y (and optionally v, for the backward pass) as defined above.
 *   x         (m, k) dtype, row stride ldx;  w (n, k) dtype, contiguous; both 16-byte aligned, with rows of
 *             whole 16-byte units: k and ldx multiples of 8 (bf16) or 16 (e4m3), else SSD_ERR_UNSUPPORTED
 *   x_scales  (m) fp32, w_scales (n) fp32: both with SSD_E4M3, both NULL otherwise
 *   bias      (n) fp32, or NULL
 *   residual  (m, n) bf16, contiguous, or NULL; may be y (in place)
 *   y         (m, n) bf16, contiguous
 *   pre       (m, n) bf16, or NULL: v, rounded
 * Sums are fp32 and y is rounded once.  `workspace`: ssd_linear_workspace_size(p) bytes, 256-byte
 * aligned; needs no initialisation; calls that share it must be ordered on one stream; where the size is 256 (only
 * the status word) it may be NULL, and nothing is recorded.  One launch, or two where
 * the contraction is split over CTAs.  The device waits are bounded: one that runs out records
 * SSD_ERR_TIMEOUT (where 61-65: stage free, stage loaded, accumulator free, accumulator done, drain) in the status word,
 * which each call clears, read by ssd_check_status().  Bitwise deterministic. */
SSD_API int ssd_linear(const ssd_linear_params_t* p, const void* x, const void* w, const float* x_scales,
             const float* w_scales, const float* bias, const void* residual, void* y, void* pre,
             void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of <dy, y> of ssd_linear() (dtype SSD_BF16):
 *
 *     dpre = dy * act'(pre);   dx = dpre w;   dw = dpre^T x;   dbias = sum_m dpre
 *
 * (the residual's gradient is dy itself.)  With an activation, or where n is not a multiple of 8, dpre is rounded
 * to bf16 in the workspace as the products' operand; dbias sums the unrounded values.
 *   x, w    as for the forward;   dy (m, n) bf16, contiguous, 16-byte aligned
 *   pre     (m, n) bf16: the forward's; NULL with SSD_ACT_NONE
 *   dx      (m, k) bf16, contiguous, or NULL;  dw (n, k) bf16, or NULL;  dbias (n) fp32, or NULL
 * m == 0 writes zeros to dw and dbias.  No output may overlap an input.  Workspace, errors and
 * determinism as for ssd_linear(), with ssd_linear_bwd_workspace_size(p). */
SSD_API int ssd_linear_bwd(const ssd_linear_params_t* p, const void* x, const void* w, const void* pre, const void* dy,
             void* dx, void* dw, float* dbias, void* workspace, size_t workspace_bytes, void* stream);

/* The same from 8-bit rows, p->dtype being that of w and dy (SSD_BF16): x is (m, k) e4m3 codes, row stride ldx >= k,
 * where x_scales (m) fp32 are given, and pre (m, n) e4m3 codes, contiguous, where pre_scales (m) fp32 are (neither: the
 * call above).  They stand for codes * scale: pre so in fp32; of x the codes times the scales' powers of two are the
 * product's operand, in bf16 in the workspace, which is exact, and the rest of the scales (1 for those of ssd_pack_rows()) is
 * in dpre before its rounding; where dpre is dy itself, x is codes * scale rounded to bf16.  Codes may start at any
 * byte; ldx is any number from k on then.  x may be NULL where dw is.  Where x_scales or dw is NULL no codes are expanded, and
 * ssd_linear_bwd_workspace_size() bytes are enough (it asks for an ldx of whole 16-byte units; k is one). */
SSD_API size_t ssd_linear_bwd_packed_workspace_size(const ssd_linear_params_t* p);
SSD_API int ssd_linear_bwd_packed(const ssd_linear_params_t* p, const void* x, const float* x_scales, const void* w,
             const void* pre, const float* pre_scales, const void* dy, void* dx, void* dw, float* dbias,
             void* workspace, size_t workspace_bytes, void* stream);


/* How a product of ssd_linear() or ssd_linear_bwd() runs (diagnostic, as ssd_fwd_plan(); needs no GPU).  product: 0 y,
 * 1 dx, 2 dw (both with SSD_BF16 only).  Returns SSD_OK, or the status that the call would return for these parameters;
 * m == 0 has no tiles. */
typedef struct {
    int64_t tiles;        /* tiles of the product                                                     */
    int64_t whole;        /* tiles computed by one worker each; the others are split along the contraction */
    int32_t splits;       /* parts of each of those others (1: all tiles are whole)                   */
    int32_t tile_rows;    /* 128: a worker is a CTA; 256: a pair of them                              */
    int32_t tile_cols;
    int32_t transposed;   /* 1: the tiles are those of the transposed product (y of up to 64 rows)    */
} ssd_linear_plan_t;
SSD_API int ssd_linear_plan(const ssd_linear_params_t* p, int product, ssd_linear_plan_t* plan);

/* Gated linear recurrence: one decay per channel and token (the scan above has one per head and token).
 * Per row b, token t and channel d, with gate logits g and inputs x,
 *
 *     a_t = 1 / (1 + exp(-g_t)),   h_t = a_t h_{t-1} + (1 - a_t) x_t,   y_t = h_t
 *
 * from h = initial_states (or zero).  Packed documents (cu_seqlens, batch 1) restart from
 * initial_states[document] (or zero) at each document's first token, as in ssd_fwd(). */
typedef struct {
    int64_t batch;      /* rows (1 when cu_seqlens is given)                                   */
    int64_t seqlen;     /* tokens per row (total packed length with cu_seqlens)                 */
    int64_t g_stride;   /* elements from one token of g (and dg) to the next, >= width          */
    int64_t x_stride;   /* the same of x (and dx): both may be column ranges of a wider matrix  */
    int32_t width;      /* channels                                                             */
    int32_t ndocs;      /* documents when cu_seqlens is given, else 0                           */
    int32_t dtype;      /* SSD_F32 or SSD_BF16: g, x, y and their gradients                     */
} ssd_gate_scan_params_t;

/* Bytes of device workspace ssd_gate_scan() and ssd_gate_scan_bwd() need; 0 on invalid parameters. */
SSD_API size_t ssd_gate_scan_workspace_size(const ssd_gate_scan_params_t* p);

/* The recurrence over whole sequences.
 *   g, x            (batch, seqlen, width) dtype, token strides g_stride, x_stride (row b starts at token
 *                   b * seqlen); each base aligned to its element
 *   initial_states  (nstates, width) fp32, or NULL (zeros); nstates = ndocs with cu_seqlens, else batch
 *   cu_seqlens      (ndocs + 1) int32, as for ssd_fwd(), or NULL
 *   y               (batch, seqlen, width) dtype, contiguous
 *   final_states    (nstates, width) fp32, or NULL; may not be initial_states
 * The state is fp32 throughout; y is rounded once.  No output may overlap an input.
 * `workspace`: at least ssd_gate_scan_workspace_size(p) bytes, 256-byte aligned (else
 * SSD_ERR_WORKSPACE); it needs no initialisation, and calls that share it must be ordered on one
 * stream; where the size is 256 (only the status word) it may be NULL, and nothing is recorded.  A clear of it (status word, tickets, states on their way) and one launch, asynchronous on `stream`; it
 * can be captured in a CUDA graph.  Tiles of a sequence hand their states on through the workspace; every wait is
 * bounded, and one that runs out records SSD_ERR_TIMEOUT (where 51: a tile's map, 52: a block's
 * state, 53-56: waits inside a CTA) in the status word read by ssd_check_status(), as offsets that break their rule
 * record SSD_ERR_DEVICE_CHECK.  Bitwise deterministic. */
SSD_API int ssd_gate_scan(const ssd_gate_scan_params_t* p, const void* g, const void* x, const float* initial_states,
             const int32_t* cu_seqlens, void* y, float* final_states, void* workspace, size_t workspace_bytes,
             void* stream);

/* Gradients of <dy, y> + <dfinal_states, final_states> of ssd_gate_scan():
 *
 *     lam_t = dy_t + a_{t+1} lam_{t+1}            (+ dfinal_states at a row's or document's last token)
 *     dx_t  = (1 - a_t) lam_t,   dg_t = lam_t (h_{t-1} - x_t) a_t (1 - a_t),   dinitial = a_1 lam_1
 *
 *   g, x, initial_states, cu_seqlens  as for the forward;  y  the forward's output (contiguous)
 *   dy             (batch, seqlen, width) dtype, contiguous
 *   dfinal_states  (nstates, width) fp32, or NULL (zeros)
 *   dg, dx         (batch, seqlen, width) dtype, token strides g_stride, x_stride; written
 *   dinitial_states (nstates, width) fp32, or NULL
 * h_{t-1} is recomputed in fp32 from the h of every 8th token (every 4th in fp32), which is read from y: where h lies close
 * to x, the difference in dg keeps the absolute error of y's rounding (2^-9 of h in bf16; none with fp32 tensors).
 * Workspace, launches, errors and aliasing as for ssd_gate_scan(). */
SSD_API int ssd_gate_scan_bwd(const ssd_gate_scan_params_t* p, const void* g, const void* x, const void* y,
             const float* initial_states, const int32_t* cu_seqlens, const void* dy, const float* dfinal_states,
             void* dg, void* dx, float* dinitial_states, void* workspace, size_t workspace_bytes, void* stream);

/* One token per row of the same recurrence from a resident state (decoding):
 *   g, x (batch, width) dtype, row strides g_stride, x_stride (elements, >= width); y (batch, width) dtype;
 *   state_in, state_out (batch, width) fp32: equal (in place) or disjoint.
 * batch >= 0 (0: nothing is launched).  One launch, no workspace. */
SSD_API int ssd_gate_scan_step(int64_t batch, int32_t width, int32_t dtype, int64_t g_stride, int64_t x_stride,
             const void* g, const void* x, const float* state_in, float* state_out, void* y, void* stream);

/* One autoregressive (decode) step: a single new token per batch row from a
 * resident state.  "State Space Duality and Mamba-2", section "Performance and
 * Serving Economics": generation keeps a fixed-size recurrent state and costs
 * constant time and memory per token.  The step is the recurrence above taken
 * once per (b, h), g = h / (H / G):
 *
 *     state'[b,h] = exp(dt[b,h] A_h) state[b,h] + dt[b,h] x[b,h] B[b,g]^T
 *     y[b,h]      = state'[b,h] C[b,g] + D_h x[b,h]
 *
 * so a prefill by ssd_fwd() (final_states) followed by steps gives the same
 * outputs, up to rounding, as one ssd_fwd() over the whole sequence.
 *
 * Layouts (row-major, contiguous, device memory): the forward's layouts with
 * one token per row (seqlen = 1):
 *   state_in, state_out (batch, nheads, headdim, dstate)  fp32, 16-byte aligned
 *   x, y                (batch, nheads, headdim)          dtype
 *   dt                  (batch, nheads)                   fp32, >= 0
 *   A, D                (nheads)                          fp32 (D optional)
 *   B, C                (batch, ngroups, dstate)          dtype
 * state_out may equal state_in (an in-place update) or be a disjoint buffer;
 * any other overlap is an argument error, as is y equal to an input.
 * dtype is an ssd_dtype_t.  dstate must be a multiple of 4 and at most 512,
 * headdim at most 2048 (else SSD_ERR_UNSUPPORTED).
 *
 * No workspace and no device-side waits: the call enqueues one kernel on
 * `stream` and returns (SSD_OK, an argument error before any launch, or
 * SSD_ERR_CUDA for a failed launch).  It can be captured in a CUDA graph.
 * Bitwise deterministic. */
SSD_API int ssd_step(int64_t batch, int32_t nheads, int32_t headdim, int32_t dstate, int32_t ngroups,
             int32_t dtype, const float* state_in, float* state_out,
             const void* x, const float* dt, const float* A, const void* B, const void* C,
             const float* D, void* y, void* stream);

/* Synchronise `stream`, read the device status word of `workspace`, clear it,
 * and return it (SSD_OK when no device error was recorded). */
SSD_API int ssd_check_status(void* workspace, void* stream);

/* ssd_check_status(), also returning in *where (if not NULL) which device wait
 * recorded the error: 0 with SSD_OK, else a code of the tensor-core full-pass
 * kernel (1 stage free, 2 stage loaded, 3 mask ready, 4 output buffer free,
 * 5 state summary buffer free, 6 scaled-X tile ready, 7 chunk values free,
 * 8 state summary done, 9 C B^T done, 10 chunk values ready, 11 off-diagonal
 * output done, 12 drain of copies or MMAs in flight, 13 diagonal output done,
 * 14 C init_d^T done, 15 state terms of a chunk with document starts ready)
 * or of the split-aggregate kernel (21 stage free, 22 stage loaded, 23 scaled
 * tile ready, 24 split contraction done, 25 drain of copies in flight, 26 the
 * other scaling group's decay product ready); with SSD_ERR_DEVICE_CHECK, 40:
 * the packed-document offsets are not 0 = cu[0] < ... < cu[ndocs] = seqlen. */
SSD_API int ssd_check_status_where(void* workspace, void* stream, uint32_t* where);

/* Test aid for the device-side failure path: ssd_fwd() with an injected stall.
 * The tensor-core kernel's TMA producer issues no loads, and every bounded
 * wait gives up after max_wait_rounds polls of its barrier (ordinary calls
 * allow 2^26 polls, and every wait gives up after 2 s).  The waits that depend on the loads run out;
 * the first records SSD_ERR_TIMEOUT and its code in the status word, and
 * every CTA stops waiting, lets its copies and MMAs finish, frees its tensor
 * memory and exits.  y and final_states are undefined afterwards;
 * ssd_check_status_where() reports the error and clears it, and the
 * workspace serves ordinary calls again.  Arguments as ssd_fwd(); returns
 * SSD_ERR_INVALID_ARG when max_wait_rounds < 4096 (the drain waits share the
 * cap) and SSD_ERR_UNSUPPORTED for problems the tensor-core kernel does not
 * run (the SIMT kernel has no device waits).  Not for production use. */
SSD_API int ssd_fwd_fault_inject(const ssd_params_t* p,
            const void* x, const float* dt, const float* A,
            const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* cu_seqlens,
            void* y, float* final_states,
            void* workspace, size_t workspace_bytes, uint32_t max_wait_rounds, void* stream);

/* Test aids for the failure paths of the operators around the scan: ssd_linear() and ssd_gate_scan() with an injected
 * stall.  Each CTA issues `loads` loads (blocks of the contraction, or tiles of the sequence) and no more; every bounded wait
 * gives up after max_wait_rounds polls.  What waits for the missing loads runs out; the first wait to do so records
 * SSD_ERR_TIMEOUT and its code, and every CTA lets its copies and MMAs finish, frees its tensor memory and exits.
 * ssd_gate_scan_fault_inject() with loads -1 loads everything, but no tile publishes its map, so the tiles after it wait in
 * vain.  Outputs are undefined afterwards; the workspace, which has to be given, serves ordinary calls again.  Arguments
 * as the ordinary calls; SSD_ERR_INVALID_ARG when max_wait_rounds < 4096 or loads is negative (below -1).  Not for
 * production use. */
SSD_API int ssd_linear_fault_inject(const ssd_linear_params_t* p, const void* x, const void* w, const float* x_scales,
             const float* w_scales, const float* bias, const void* residual, void* y, void* pre,
             void* workspace, size_t workspace_bytes, int32_t loads, uint32_t max_wait_rounds, void* stream);
SSD_API int ssd_gate_scan_fault_inject(const ssd_gate_scan_params_t* p, const void* g, const void* x,
             const float* initial_states, const int32_t* cu_seqlens, void* y, float* final_states, void* workspace,
             size_t workspace_bytes, int32_t loads, uint32_t max_wait_rounds, void* stream);

/* Human-readable name of a status code (static storage). */
SSD_API const char* ssd_status_string(int status);

/* Which kernel family ssd_fwd() uses for these params:
 * 0 = SIMT fp32 kernel, 1 = tcgen05 tensor-core kernel; -1 on invalid params.
 * *launches (if not NULL) receives the number of kernel launches per call. */
SSD_API int ssd_fwd_plan(const ssd_params_t* p, int has_initial_states, int has_final_states,
                 int* launches, int* nsplits);

/* The hierarchy-aware segsum device routines on their own (test aid).  Both
 * forms of csrc/segsum.cuh run here with the inputs the forward kernels give
 * them: the log-domain form, whose seg the SIMT kernel exponentiates, and the
 * linear-domain form, whose factors the tensor-core kernel multiplies in.
 * log2decay: (nrows, chunk) fp32 log2-domain log-decays (<= 0, may be -inf),
 * chunk 64 or 128.  Per row (each output may be NULL):
 *   seg_out  (chunk x chunk) seg[i][j] = sum_{k=j+1..i} log2decay[k] for j <= i,
 *            as the log-domain routine forms it (no prefix subtraction),
 *            -inf above the diagonal;
 *   L_out    (chunk x chunk) the decay mask prod_{k=j+1..i} a_k of the
 *            linear-domain routine, with a_k = ex2.approx(log2decay[k]) (the
 *            tensor-core kernel's factors): products grown from the diagonal
 *            on the 32 x 32 diagonal blocks, the rank-one product of the row
 *            factor and the column factor on the blocks left of them, 0 above
 *            the diagonal;
 *   pexp_out (chunk) the row prefixes prod_{k=0..i} a_k (decay of the state
 *            entering the chunk, at row i);
 *   sfx_out  (chunk) the column suffixes prod_{k=j+1..chunk-1} a_k (decay of
 *            token j's contribution to the state leaving the chunk).
 * Device pointers; async on `stream`.  Returns SSD_ERR_INVALID_ARG for a NULL
 * input or an unsupported chunk, SSD_ERR_CUDA for a failed launch.
 * Source: "GPU Hierarchy Meets Structured Matrices" (abstract): the 1-SS mask
 * as 1-SS diagonal blocks plus rank-one off-diagonal blocks. */
SSD_API int ssd_segsum_dump(const float* log2decay, int64_t nrows, int32_t chunk,
                    float* seg_out, float* L_out, float* pexp_out, float* sfx_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SSD_H_ */
