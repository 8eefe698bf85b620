/*
 * mlstm.h -- C ABI of the MI355X (gfx950) stabilized parallel mLSTM forward pass,
 * and, further down, of the gated delta rule, the block norm, the short causal
 * convolution, the selective scan and the gated feed-forward.
 *
 * The operation is the stabilized parallel forward pass of the mLSTM cell of
 * "xLSTM: Extended Long Short-Term Memory", Appendix A.3: the parallel form
 * ("Parallel mLSTM Forward Pass", Eqs. 71-77) in the stabilized version that
 * opens "Parallel mLSTM Backward Pass" (Eqs. 79-86), with the log forget gate
 * matrix of Eq. 101.  For one head with queries, keys, values Q, K, V (T x d)
 * and gate pre-activations f~, i~ (length T):
 *
 *   fbar_k   = log sigmoid(f~_k)                                   (Eq. 101)
 *   D~_ij    = sum_{k=j+1..i} fbar_k + i~_j  for j <= i, -inf above (Eqs. 79, 101, 72)
 *   m_i      = max_j D~_ij                                         (Eq. 80)
 *   D'_ij    = exp(D~_ij - m_i)                                    (Eq. 81)
 *   C~'_ij   = (q_i . k_j / sqrt(d)) D'_ij                          (Eq. 82)
 *   b_i      = sum_j C~'_ij                                        (Eq. 83)
 *   n_i      = max(|b_i|, exp(-m_i))                               (Eq. 84)
 *   h~_i     = sum_j C~'_ij v_j / n_i                              (Eqs. 85, 86)
 *
 * Heads are independent (the xLSTM cell has no memory mixing across heads),
 * so every call processes B x NH heads at once.
 *
 * Layouts (all row-major, contiguous, no strides):
 *   q, k, v, h_out  [B][NH][T][d]   element type given by `dtype`
 *   igate, fgate    [B][NH][T]      float32 (i~ and f~ pre-activations)
 *   m_out, n_out    [B][NH][T]      float32
 * k is passed UNSCALED: the library applies the 1/sqrt(d) of Eq. 82.
 *
 * Ownership: every pointer is device memory owned by the caller, on the
 * device that is current when the call is made.  The library never frees or
 * retains a caller pointer beyond the work it enqueues.  Outputs are fully
 * overwritten.  No output may overlap an input or another output (checked
 * from the pointers and sizes: MLSTM_ERR_ALIAS, nothing launched); inputs
 * may overlap each other.  The recurrent step alone may update C in place.
 *
 * Ordering: calls are asynchronous on the given HIP stream (NULL = the null
 * stream); results are valid once that stream has synchronized.  No host
 * synchronization happens inside the library.
 *
 * Errors: every argument check runs before any device work; on error nothing
 * is launched, no output is touched, and a negative status is returned.
 * Faults inside a kernel surface at the caller's next synchronization, as for
 * any stream API.  No C++ exception crosses this interface.
 *
 * Numerics: gates, m and n are float32.  For MLSTM_BF16 the two contractions
 * run on bf16 matrix cores with float32 accumulation; the row sums b are taken
 * from the float32 C~' before it is rounded to bf16; h_out is rounded to
 * nearest even.  Inputs must be finite; NaN/Inf propagate and are not checked.
 * Results are bitwise reproducible run to run (fixed reduction order, no
 * atomics).
 */
#ifndef MLSTM_H
#define MLSTM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element type of q, k, v, h_out */
enum { MLSTM_FP32 = 0, MLSTM_BF16 = 1 };

/* tile-kernel selector for mlstm_causal_tiles */
enum {
  MLSTM_KERNEL_AUTO = 0,   /* bf16 -> matrix-core kernel; fp32 -> float32 matrix-core kernel
                              (d a multiple of 32 up to 256, or 320, 384, 512), else vector kernel */
  MLSTM_KERNEL_MFMA = 1,   /* bf16 only: bf16 MFMA tiles (the production path) */
  MLSTM_KERNEL_VECTOR = 2, /* any dtype: float32 vector-ALU tiles, no bf16 rounding of C~' */
  MLSTM_KERNEL_MFMA_ALL_TILES = 3, /* as MLSTM_KERNEL_MFMA, but visiting every causal tile */
  MLSTM_KERNEL_MFMA_SINGLE = 4,    /* bf16 only, d <= 512: the one-wave-per-SIMD MFMA kernel */
  MLSTM_KERNEL_MFMA_WIDE = 5       /* bf16 only: the wide-head MFMA kernel, for any d */
};
/*
 * The bf16 MFMA path has three tile kernels, and a fourth on the one-launch
 * path.  For d <= 384 it runs 8 waves
 * per workgroup, two per SIMD: the two waves that share a SIMD share 32 query
 * rows, each forms C~' for its own 32 of every 64 keys and accumulates half
 * of the output columns, so one wave's copies and exponentials overlap the
 * other's matrix-core work.  On the one-launch path with d a multiple of 64
 * up to 192 it runs 4 waves, one per SIMD, each with 32 query rows and all
 * columns, and software-pipelines the key loop (the Q K^T product of one key
 * tile beside the C~' V product of the previous one, K and V staged through
 * registers); its sums are those of the one-wave kernel below.  For 384 < d <= 512 (and with
 * MLSTM_KERNEL_MFMA_SINGLE) it runs 4 waves, one per SIMD, each with 32 query
 * rows and all columns.  For d > 512 (and with MLSTM_KERNEL_MFMA_WIDE) four
 * waves share 32 query rows, each holding a quarter of the head dimension:
 * they add their partial Q K^T products through LDS, and each accumulates a
 * quarter of the output columns.  All give the same results up to float32
 * summation order.  Float32 inputs (MLSTM_KERNEL_AUTO) run on the float32
 * matrix instruction v_mfma_f32_32x32x2_f32: 4 waves, one per SIMD, each with
 * 32 query rows and their Q^T operands in registers, C~' kept in float32 and
 * fed from the first product's registers to the second; above d = 256 two
 * (at d = 512 four) workgroups per 128 query rows split the output columns.  Other
 * float32 head dimensions, and MLSTM_KERNEL_VECTOR, run the float32 vector
 * kernel.
 */
/*
 * Decay-aware tile skipping (MLSTM_KERNEL_AUTO and _MFMA on bf16).  From the
 * gate scan's terms the tile kernel bounds log2(D'_ij / sqrt(d)) over each
 * 32 x 32 block of Eqs. 79-81; where the bound is below -200 every entry's
 * float32 exponential is exactly 0, so the block adds nothing to b (Eq. 83)
 * or to C~'V and is not visited.  Outputs equal those of
 * MLSTM_KERNEL_MFMA_ALL_TILES (up to the sign of exact zeros).  Long
 * sequences with strong forgetting skip most of the causal triangle; the
 * counted work (2 T^2 d per head) is unchanged.
 */

/* status codes */
enum {
  MLSTM_OK = 0,
  MLSTM_ERR_NULL = -1,        /* a required pointer is NULL */
  MLSTM_ERR_SHAPE = -2,       /* B, NH, T or d < 1, or a size overflows */
  MLSTM_ERR_DTYPE = -3,       /* dtype not MLSTM_FP32 / MLSTM_BF16 */
  MLSTM_ERR_HEAD_DIM = -4,    /* d not a multiple of 16 in [16, 1024], or beyond a kernel's limit */
  MLSTM_ERR_ALIGN = -5,       /* a pointer is not 16-byte aligned */
  MLSTM_ERR_HIP = -6,         /* a HIP allocation or launch failed */
  MLSTM_ERR_WORKSPACE = -7,   /* caller workspace smaller than mlstm_workspace_bytes */
  MLSTM_ERR_KERNEL = -8,      /* unknown kernel selector, or an MFMA selector for fp32 */
  MLSTM_ERR_ALIAS = -9,       /* an output overlaps an input or another output */
  MLSTM_ERR_ACTIVATION = -10, /* unknown activation (forget gate, convolution, feed-forward) */
  MLSTM_ERR_SCRATCH = -11,    /* beyond the allocation-free entry point's fixed workspace */
  MLSTM_ERR_HEADS = -12,      /* NH not a multiple of NHK */
  MLSTM_ERR_NORM = -13,       /* unknown norm or gate activation, or eps not a number >= 0 */
  MLSTM_ERR_WIDTH = -14,      /* convolution width outside [2, 8], or scan states outside [1, 64] */
  MLSTM_ERR_ROW = -15         /* a row pitch shorter than its row, no multiple of 8, or too long */
};

/*
 * Forget-gate activation (the `forget_activation` argument of
 * mlstm_gate_scan, mlstm_parallel_fwd_train, mlstm_parallel_bwd and
 * mlstm_recurrent_step).  The mLSTM forward equations (Eq. 71) allow the
 * forget gate to be either sigma(f~) or exp(f~); every formula of the
 * parallel and recurrent forms uses it only through its logarithm
 * fbar = log f, which is log sigma(f~) or f~ itself.  With MLSTM_FORGET_EXP
 * the caller keeps f~ <= 0 if it wants f <= 1; nothing here requires it.
 * mlstm_parallel_fwd, _stream and _gated use MLSTM_FORGET_SIGMOID.
 */
enum { MLSTM_FORGET_SIGMOID = 0, MLSTM_FORGET_EXP = 1 };

/*
 * mlstm_parallel_fwd -- the whole forward pass (Eqs. 79-86) for B x NH heads.
 *   q, k, v   in   [B][NH][T][d], dtype
 *   igate     in   [B][NH][T] float32, i~ (input gate pre-activations, Eq. 72)
 *   fgate     in   [B][NH][T] float32, f~ (forget gate pre-activations, Eq. 71;
 *                  sigmoid forget activation; f~ at t = 0 never affects a result)
 *   h_out     out  [B][NH][T][d], dtype: h~ (Eq. 86), before any output gate
 *   m_out     out  [B][NH][T] float32: the row maximum m (Eq. 80)
 *   n_out     out  [B][NH][T] float32: the normalizer n (Eq. 84)
 *   B, NH, T  >= 1;  d a multiple of 16 in [16, 1024]
 *   dtype     MLSTM_FP32 or MLSTM_BF16
 * Runs on the null stream.  For bf16 with d <= 512 and T <= 2048, T a
 * multiple of 4, the pass is one kernel launch that needs no workspace: each
 * workgroup scans its head's gates itself (the gate-scan arithmetic in the
 * same order, so every output is bitwise that of the two stages with the same
 * tile arithmetic: the one-wave kernel where the pipelined kernel runs, the
 * kernel MLSTM_KERNEL_AUTO picks otherwise).  So is the pass for float32
 * inputs with T <= 2048: the float32 tile kernel (matrix-core where it takes
 * d, vector otherwise) scans its head's gates itself, bitwise as its two
 * stages would.  Otherwise the gate scan and the tile kernel run as two
 * launches on a library-allocated, stream-ordered workspace.
 * Returns MLSTM_OK or a negative status.
 */
int mlstm_parallel_fwd(const void* q, const void* k, const void* v,
                       const float* igate, const float* fgate,
                       void* h_out, float* m_out, float* n_out,
                       int64_t B, int64_t NH, int64_t T, int64_t d, int dtype);

/* As mlstm_parallel_fwd, enqueued on `stream` (a hipStream_t; NULL = null stream). */
int mlstm_parallel_fwd_stream(const void* q, const void* k, const void* v,
                              const float* igate, const float* fgate,
                              void* h_out, float* m_out, float* n_out,
                              int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                              void* stream);

/*
 * mlstm_parallel_fwd_noalloc -- mlstm_parallel_fwd_stream for callers that
 * cannot allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  It calls no allocating routine.
 * Its workspace is a fixed array of MLSTM_NOALLOC_SCRATCH_BYTES in the
 * library's device code, one per GPU, held until the process ends; a call
 * needs mlstm_workspace_bytes(B, NH, T) of it (about 20.5 bytes per position
 * of B * NH * T, T padded to a multiple of 128: up to ~800 K positions) and
 * returns MLSTM_ERR_SCRATCH, before any device work, for a problem that needs
 * more.  Where mlstm_parallel_fwd runs as a single launch (bf16, d <= 512,
 * T <= 2048, T a multiple of 4; float32, T <= 2048) no workspace is used
 * and any size is accepted.  All calls on one GPU share that GPU's array:
 * calls that overlap in time on one GPU (different streams, host threads)
 * race and must be serialized by the caller.  Nothing needs to be cleared between calls: each
 * call writes every workspace byte it reads.  Arguments, results and other
 * errors as for mlstm_parallel_fwd_stream; the first call on a device also
 * looks up the array's address on that device (MLSTM_ERR_HIP if that fails).
 */
enum { MLSTM_NOALLOC_SCRATCH_BYTES = 16 << 20 };
int mlstm_parallel_fwd_noalloc(const void* q, const void* k, const void* v,
                               const float* igate, const float* fgate,
                               void* h_out, float* m_out, float* n_out,
                               int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                               void* stream);

/*
 * mlstm_parallel_fwd_gated -- the forward pass followed by the output gate of
 * "Parallel mLSTM Forward Pass" (Eq. 78): H = sigma(O~) (.) H~, elementwise,
 * with the logistic sigmoid.  The gate is applied to the float32 h~ inside
 * the tile kernel's epilogue, before the result is rounded to `dtype`.
 *   ogate       in   [B][NH][T][d], dtype: O~ (output gate pre-activations); required
 *   h_out       out  [B][NH][T][d], dtype: H (Eq. 78)
 *   htilde_out  out  [B][NH][T][d], dtype: H~ (Eq. 86), bitwise what
 *                    mlstm_parallel_fwd writes to its h_out; may be NULL (not stored)
 *   all other arguments as for mlstm_parallel_fwd_stream.
 * ogate and htilde_out must be 16-byte aligned and must not alias any other
 * argument.  Errors as for mlstm_parallel_fwd (MLSTM_ERR_NULL for ogate NULL).
 */
int mlstm_parallel_fwd_gated(const void* q, const void* k, const void* v,
                             const float* igate, const float* fgate, const void* ogate,
                             void* h_out, void* htilde_out, float* m_out, float* n_out,
                             int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                             void* stream);

/*
 * The same pass split into its two stages with a caller-owned workspace, for
 * callers that time or schedule the stages separately.
 *
 * mlstm_workspace_bytes: bytes of device workspace the two stages need for
 * B x NH heads of length T (0 if the sizes are invalid).
 */
size_t mlstm_workspace_bytes(int64_t B, int64_t NH, int64_t T);

/*
 * mlstm_gate_scan -- stage 1: the gate-only part of Eqs. 79-81 and 101.
 * Computes fbar = log f (log sigmoid(f~), or f~ for MLSTM_FORGET_EXP), its
 * prefix sums, and the row maximum
 *   m_i = max_{j<=i} (sum_{k=j+1..i} fbar_k + i~_j)                 (Eq. 80)
 * through the equivalent recurrence m_i = max(m_{i-1} + fbar_i, i~_i),
 * m_0 = i~_0, before any Q K^T work.  Writes m_out and the per-row and
 * per-column exponent terms and block anchors the tile stage reads into
 * `workspace` (device memory, >= mlstm_workspace_bytes(B, NH, T) bytes,
 * 256-byte aligned).  `d` is needed for the 1/sqrt(d) folded into the
 * exponent terms.
 */
int mlstm_gate_scan(const float* igate, const float* fgate, float* m_out,
                    void* workspace, size_t workspace_bytes,
                    int64_t B, int64_t NH, int64_t T, int64_t d,
                    int forget_activation, void* stream);

/*
 * mlstm_causal_tiles -- stage 2: Eqs. 81-86 over causal tiles.  Reads q, k,
 * v, m (from stage 1) and the workspace stage 1 wrote on the same stream, and
 * writes h_out and n_out.  `kernel` is an MLSTM_KERNEL_* selector.
 */
int mlstm_causal_tiles(const void* q, const void* k, const void* v, const float* m,
                       const void* workspace, size_t workspace_bytes,
                       void* h_out, float* n_out,
                       int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                       int kernel, void* stream);

/*
 * mlstm_parallel_fwd_train -- mlstm_parallel_fwd_stream that also stores the
 * row sums b = C~' 1 (Eq. 83), which the backward pass needs (Eq. 90).
 *   b_out              out  [B][NH][T] float32 (required, 16-byte aligned)
 *   forget_activation  MLSTM_FORGET_SIGMOID or MLSTM_FORGET_EXP
 * Other arguments, layouts and errors as for mlstm_parallel_fwd_stream.
 */
int mlstm_parallel_fwd_train(const void* q, const void* k, const void* v,
                             const float* igate, const float* fgate,
                             void* h_out, float* m_out, float* n_out, float* b_out,
                             int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                             int forget_activation, void* stream);

/*
 * mlstm_parallel_bwd -- gradients of the stabilized parallel forward pass
 * ("Parallel mLSTM Backward Pass", Eqs. 87-105) with respect to q, k, v and
 * the gate pre-activations, given dh = dL/dH~.
 *   q, k, v, igate, fgate   in: the forward inputs
 *   h, m, n, b              in: the forward outputs of mlstm_parallel_fwd_train
 *                           (h~ before any output gate, [B][NH][T][d] dtype;
 *                           m, n, b [B][NH][T] float32)
 *   dh                      in  [B][NH][T][d], dtype
 *   dq, dk, dv              out [B][NH][T][d], dtype (float32 accumulation)
 *   digate, dfgate          out [B][NH][T] float32
 * m is held constant (its contributions cancel, as the pages note).  Eq. 90
 * is applied with the derivative of |b|, sign(b): the printed sign(n) is 1
 * for every row, since n > 0.  d(log sigma(x))/dx = sigma(-x) (Eq. 104);
 * with forget_activation MLSTM_FORGET_EXP, d(log f)/df~ = 1.  The forward
 * outputs must come from the same forget_activation.
 * dL/dn uses sum_j C~'_ij v_j = n_i h~_i, so for bf16 it carries the
 * rounding of the stored h~.  For bf16 with d <= 512 the contractions run
 * on the matrix cores (bf16 operands, float32 accumulation; the operand
 * E (.) dC~' of the dQ and dK products and C~'/n of the dV product are
 * rounded to bf16, the row and column sums of dD~ behind the gate gradients
 * are not); for float32 with d a multiple of 32 up to 384 they run on the
 * float32 matrix instruction (float32 operands and sums throughout; the
 * environment variable MLSTM_BWD_F32=vector, read at each call, selects the
 * vector passes instead); for the other float32 head dims, and for bf16
 * above d = 512, everything is float32 on the vector ALUs (above d = 512 in
 * head-dimension chunks, a correctness path far slower than the matrix
 * cores).  Results are bitwise reproducible.  The library allocates a stream-ordered workspace: per-row
 * terms and, for bf16 on the matrix cores, the bf16 operands of the dV and
 * dQ products, which the key pass stores so that the dV and dQ passes need
 * not recompute S and G: 8 KiB per head, 128-key block and 32-query tile of
 * the causal triangle for dV, 2 KiB per head and pair of 32-row tiles for dQ
 * (278 MB for 32 heads of 2048).  Above 2 GiB (or the byte count in the
 * environment variable MLSTM_BWD_STORE_MAX, read at each call) those passes
 * recompute them instead: dV is then bitwise the same, dQ, dK and the gate
 * gradients equal up to float32 rounding order.
 * Pointers 16-byte aligned; no output may alias an input.  Any d of the
 * forward pass (a multiple of 16 up to 1024).  Errors as for
 * mlstm_parallel_fwd.
 */
int mlstm_parallel_bwd(const void* q, const void* k, const void* v,
                       const float* igate, const float* fgate,
                       const void* h, const float* m, const float* n, const float* b,
                       const void* dh, void* dq, void* dk, void* dv,
                       float* digate, float* dfgate,
                       int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                       int forget_activation, void* stream);

/*
 * mlstm_recurrent_step -- one step of the recurrent mLSTM (the generation
 * form that the parallel pass reformulates; its equations are those the
 * recurrent backward pass of appendix A.3 differentiates, Eqs. 59-70), with
 * the states stabilized by the running maximum of the log gates, the same
 * recurrence as the parallel form's row maximum (Eq. 80):
 *   m_t  = max(fbar_t + m_{t-1}, i~_t),  fbar_t = log f_t (log sigmoid(f~_t),
 *          or f~_t with forget_activation MLSTM_FORGET_EXP)
 *   f'_t = exp(fbar_t + m_{t-1} - m_t),  i'_t = exp(i~_t - m_t)
 *   C_t  = f'_t C_{t-1} + i'_t v_t (k_t / sqrt(d))^T
 *   n_t  = f'_t n_{t-1} + i'_t k_t / sqrt(d)
 *   h~_t = C_t q_t / max(|n_t . q_t|, exp(-m_t))
 * These states are the unstabilized ones times exp(-m_t); h~_t, m_t and the
 * denominator equal row t of mlstm_parallel_fwd's h~, m and n.
 *   q, k, v      in   [B][NH][d], dtype: this step's query, key, value
 *   igate, fgate in   [B][NH] float32: i~_t, f~_t
 *   C_in, n_in, m_in   in  [B][NH][d][d], [B][NH][d], [B][NH] float32: the
 *                state after step t-1 (C rows index the value dimension);
 *                a fresh state is C = 0, n = 0, m = -inf
 *   C_out, n_out, m_out out: the state after step t.  C_out may be C_in
 *                (updated in place); n_out and m_out must not overlap n_in and
 *                m_in (MLSTM_ERR_ALIAS)
 *   h_out        out  [B][NH][d], dtype: h~_t (before any output gate)
 *   den_out      out  [B][NH] float32: max(|n_t . q_t|, exp(-m_t)); may be NULL
 *   d            a multiple of 16 in [16, 1024]
 * Vectors and C need 16-byte alignment, scalars 4-byte.  Asynchronous on
 * `stream`; no workspace.  Bound by memory bandwidth: the state is read and
 * written once per step.
 */
int mlstm_recurrent_step(const void* q, const void* k, const void* v,
                         const float* igate, const float* fgate,
                         const float* C_in, const float* n_in, const float* m_in,
                         float* C_out, float* n_out, float* m_out,
                         void* h_out, float* den_out,
                         int64_t B, int64_t NH, int64_t d, int dtype,
                         int forget_activation, void* stream);

/*
 * The gated delta rule: a matrix memory that corrects what it holds for a key
 * before it writes, with the same layouts, gate pre-activations and forget
 * activations as the mLSTM cell above.  Per head, with C (dv x dk, rows by
 * value), f_t = sigma(f~_t) or exp(f~_t) and a write strength beta_t,
 *
 *   C_t = f_t C_{t-1} + beta_t (v_t - f_t C_{t-1} k_t) k_t^T
 *   h_t = C_t q_t / sqrt(dk)
 *
 *   q, k     [B][NHK][T][dk]  dtype
 *   v, h     [B][NH][T][dv]   dtype; value head n reads key head n / (NH / NHK)
 *   beta     [B][NH][T]       float32, the strengths themselves
 *   fgate    [B][NH][T]       float32, the pre-activations f~
 *   C        [B][NH][dv][dk]  float32
 *   NHK      a divisor of NH;  dk a multiple of 16 in [16, 512];
 *   dv       a multiple of 16 in [16, 1024];  T >= 1;  fewer than 2^18 heads
 *            B NH, and 2^22 chunks B NH ceil(T / 64) (one token: fewer than 2^24
 *            value columns in sixteens, B NH dv / 16)
 * k is not normalized here.  The recurrence is stable for beta |k|^2 <= 2 (unit
 * keys and strengths in (0, 1), as a rule); near 2 and with keys that are all
 * alike the terms of a chunk cancel, and results keep 14 to 15 bits of float32's
 * 24.  A position with beta = 0 and f = 1 (f~ = +infinity, or 0 with
 * MLSTM_FORGET_EXP) leaves the memory as it is, which is how a batch is padded.
 * f~ = -infinity forgets everything.  f > 1 (MLSTM_FORGET_EXP) is taken as long as
 * the products of up to 64 neighbouring f are float32 numbers.  Inputs are
 * otherwise finite: NaN and infinities propagate, and may reach other positions of
 * the same 64.
 *
 * All sums, the memory and the products that feed it are float32 (bf16
 * operands are exact; float32 operands of a matrix product are split into
 * three bf16 planes), gate sums are float64; for MLSTM_BF16 h, dq, dk and dv are
 * rounded once, to nearest even.  Results are bitwise reproducible (no atomics, fixed order).
 */

/*
 * mlstm_delta_workspace_bytes -- workspace of mlstm_delta_fwd (or, with
 * backward != 0, of mlstm_delta_bwd) for these sizes; 0 for T = 1 forward, and
 * for sizes that the call refuses.
 */
size_t mlstm_delta_workspace_bytes(int64_t B, int64_t NHK, int64_t NH, int64_t T, int64_t dk,
                                   int64_t dv, int dtype, int backward);

/*
 * mlstm_delta_fwd -- a whole sequence, in chunks of 64 tokens.
 *   C_in       in   the memory before the sequence; NULL: zeros
 *   h          out
 *   C_out      out  the memory after it; may be C_in (updated in place)
 *   workspace  mlstm_delta_workspace_bytes bytes of device memory, 256-byte
 *              aligned, used by this call alone until it has run on `stream`
 * Where few heads leave the card idle a long sequence is cut into segments that
 * run side by side (each one's effect on a memory is taken first), so a position's
 * result may differ in its last bits from that of a shorter call.
 * Tensors 16-byte aligned (beta and fgate 4-byte).  Errors before any device
 * work.
 */
int mlstm_delta_fwd(const void* q, const void* k, const void* v, const float* beta,
                    const float* fgate, const float* C_in, void* h, float* C_out,
                    void* workspace, size_t workspace_bytes,
                    int64_t B, int64_t NHK, int64_t NH, int64_t T, int64_t dk, int64_t dv,
                    int dtype, int forget_activation, void* stream);

/*
 * mlstm_delta_bwd -- gradients of mlstm_delta_fwd.
 *   C_in            in   the memory before the sequence, or NULL (zeros)
 *   dh              in   dL/dh, [B][NH][T][dv] dtype
 *   dC_in           in   dL/dC after the sequence, or NULL (zeros)
 *   dq, dk, dv      out  dtype; dq and dk are summed over the value heads that
 *                        share a key head
 *   dbeta, dfgate   out  [B][NH][T] float32
 *   dC_out          out  dL/dC before the sequence, or NULL
 *   workspace       mlstm_delta_workspace_bytes(..., 1) bytes, 256-byte aligned:
 *                   chiefly the memory and its gradient at every 64th token
 *                   (8 dk dv bytes per head and chunk)
 * The forward pass is formed again; nothing of it is kept.  No output may
 * overlap an input.
 */
int mlstm_delta_bwd(const void* q, const void* k, const void* v, const float* beta,
                    const float* fgate, const float* C_in, const void* dh, const float* dC_in,
                    void* dq, void* dk, void* dv, float* dbeta, float* dfgate, float* dC_out,
                    void* workspace, size_t workspace_bytes,
                    int64_t B, int64_t NHK, int64_t NH, int64_t T, int64_t dk_dim,
                    int64_t dv_dim, int dtype, int forget_activation, void* stream);

/*
 * mlstm_delta_step -- one token (generation): q, k [B][NHK][dk], v, h
 * [B][NH][dv], beta, fgate [B][NH].  C_out may be C_in (updated in place).  No
 * workspace.  Bound by memory bandwidth: the memory is read and written once.
 */
int mlstm_delta_step(const void* q, const void* k, const void* v, const float* beta,
                     const float* fgate, const float* C_in, float* C_out, void* h,
                     int64_t B, int64_t NHK, int64_t NH, int64_t dk, int64_t dv,
                     int dtype, int forget_activation, void* stream);

/*
 * Block norm: what stands between a cell and the next block, in one pass.  Per
 * token, with the cell's output p in NH heads of d channels and D = NH d,
 *
 *   z = act(g) * w1 * norm(p)    norm over each head's d channels
 *   r = x + s * z                the residual stream, with its scale
 *   y = w2 * norm(r)             norm over all D channels: the next block's input
 *
 *   p            [B][NH][T][d]   dtype (NH = 1: plain rows of a block's output)
 *   gate g       [B][NH][T][d]   dtype, or NULL (act(g) = 1)
 *   residual x   [B][T][D]       dtype, or NULL (0)
 *   weight w1    [D]             float32
 *   scale s      [D]             float32, or NULL (1)
 *   next_weight w2 [D]           float32, or NULL (no y)
 *   r, y         [B][T][D]       dtype: rows, as a projection reads them
 *   d a multiple of 8, D <= 8192
 * norm is (a - mean) / sqrt(var + eps) (MLSTM_NORM_LAYER) or a / sqrt(mean(a^2)
 * + eps) (MLSTM_NORM_RMS); act is sigma(g) (MLSTM_GATE_SIGMOID) or g sigma(g)
 * (MLSTM_GATE_SILU).  Everything in between is float32; y is formed from r
 * before its rounding.  Inputs finite: a NaN or an infinity stays in its row (and
 * in the weights' gradients).  With eps = 0 a row without spread gives NaN.
 * Tensors 16-byte aligned; no output may overlap an input.  Bitwise reproducible.
 */
enum { MLSTM_NORM_LAYER = 0, MLSTM_NORM_RMS = 1 };
enum { MLSTM_GATE_SIGMOID = 0, MLSTM_GATE_SILU = 1 };

int mlstm_block_norm_fwd(const void* p, const void* gate, const void* residual,
                         const float* weight, const float* scale, const float* next_weight,
                         void* r_out, void* y_out,
                         int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                         int norm, int gate_activation, float eps, void* stream);

/*
 * mlstm_block_norm_bwd -- its gradients, from dr and dy.
 *   dr   [B][T][D] dtype, or NULL (0);  dy [B][T][D] dtype, with next_weight only
 *   dp   out [B][NH][T][d];  dgate, dresidual: out with gate, residual (else NULL)
 *   dweight [D], dscale [D], dnext_weight [D]: out float32, the last two with
 *        scale and next_weight (else NULL)
 *   workspace  mlstm_block_norm_workspace_bytes bytes, 256-byte aligned
 * Nothing of the forward pass is kept for it: it is formed again from p, gate
 * and residual, which the gradients need in any case.
 */
size_t mlstm_block_norm_workspace_bytes(int64_t B, int64_t NH, int64_t T, int64_t d);
int mlstm_block_norm_bwd(const void* p, const void* gate, const void* residual,
                         const float* weight, const float* scale, const float* next_weight,
                         const void* dr, const void* dy, void* dp, void* dgate, void* dresidual,
                         float* dweight, float* dscale, float* dnext_weight,
                         void* workspace, size_t workspace_bytes,
                         int64_t B, int64_t NH, int64_t T, int64_t d, int dtype,
                         int norm, int gate_activation, float eps, void* stream);

/*
 * Short causal convolution with an activation: what a recurrent cell's inputs
 * pass through, each channel by itself.  With z the state's W - 1 inputs followed
 * by x_0 .. x_{n-1},
 *
 *   a_t = bias + sum_{j < W} weight_j z_{t+j},   y_t = act(a_t)
 *
 *   x        [B][T] rows of C = NH d channels, dtype, x_row elements apart (a
 *            multiple of 8, at least C: x may be part of a wider projection)
 *   weight   [C][W] float32, the last one on the newest input;  bias [C] float32 or NULL
 *   state    [B][W - 1][C] dtype, oldest input first; the state before the
 *            sequence may be NULL (zeros)
 *   lengths  [B] int32 in device memory, or NULL (T).  Sequence b has the first
 *            lengths[b] positions (kept in [0, T]); beyond them y and dx are zeros,
 *            what the inputs hold is not used and the state stays as it is
 *   y        [B][NH][T][d] dtype, as the cells above read it (NH = 1: rows)
 *   W in [2, 8], d a multiple of 8, C <= 2^20, and B ceil(T / 64) ceil(C / 128) below
 * 2^24 (a launch's workgroups).  act: a sigma(a) (MLSTM_CONV_SILU)
 * or a.  Sums are float32, and a bf16 result is rounded once.  Tensors 16-byte
 * aligned (lengths 4).  Bitwise reproducible.  T = 1 is the step of generation.
 */
enum { MLSTM_CONV_NONE = 0, MLSTM_CONV_SILU = 1 };

/* state_out: the last W - 1 inputs after the sequence; may be state_in (in place) */
int mlstm_short_conv_fwd(const void* x, int64_t x_row, const float* weight, const float* bias,
                         const void* state_in, const int32_t* lengths, void* y, void* state_out,
                         int64_t B, int64_t NH, int64_t T, int64_t d, int64_t width, int dtype,
                         int activation, void* stream);

/*
 * mlstm_short_conv_bwd -- its gradients, from dy [B][NH][T][d] and dstate, that
 * of the state after the sequence ([B][W - 1][C] dtype, or NULL: zeros).
 *   dx [B][T][C] dtype;  dweight [C][W], dbias [C] float32 (dbias with bias, else
 *   NULL);  dstate_out: of the state before, or NULL
 *   workspace  mlstm_short_conv_workspace_bytes bytes, 256-byte aligned
 */
size_t mlstm_short_conv_workspace_bytes(int64_t B, int64_t NH, int64_t T, int64_t d,
                                        int64_t width, int dtype);
int mlstm_short_conv_bwd(const void* x, int64_t x_row, const float* weight, const float* bias,
                         const void* state_in, const int32_t* lengths, const void* dy,
                         const void* dstate, void* dx, float* dweight, float* dbias,
                         void* dstate_out, void* workspace, size_t workspace_bytes, int64_t B,
                         int64_t NH, int64_t T, int64_t d, int64_t width, int dtype,
                         int activation, void* stream);

/*
 * Selective state space scan: a recurrent cell of N states to a channel, whose
 * step and in- and output weights depend on the token.  Per channel c of group g,
 *
 *   Delta_t = softplus(dt_t + dt_bias_c)
 *   s_t = exp(Delta_t A_c) s_{t-1} + Delta_t u_t B_t
 *   y_t = (C_t . s_t + D_c u_t) z_t sigma(z_t)
 *
 *   u, dt, gate z  [batch][T] rows of `channels`, dtype, u_row, dt_row and gate_row
 *                  elements apart (multiples of 8; for T > 1 and backward all five
 *                  pitches are at most 2^23); gate NULL: no last factor
 *   A              [channels][N] float32 (negative, as a rule; any finite value)
 *   B, C           [batch][T] rows of [G][N] dtype, B_row and C_row elements apart;
 *                  channel c reads group c / (channels / G)
 *   D, dt_bias     [channels] float32, or NULL (0)
 *   state          [batch][channels][N] float32; before the sequence NULL: zeros
 *   lengths        [batch] int32 in device memory, or NULL, as above: positions
 *                  beyond are not used, y and gradients there are zeros and the
 *                  state stays as it is
 *   y              [batch][T][channels] dtype
 *   channels / G a multiple of 8, channels <= 2^20, N in [1, 64],
 *   batch T G N <= 2^31, batch channels <= 2^25
 * dt = -infinity gives Delta = 0, which leaves the state as it is; inputs are
 * otherwise finite, and a positive A is taken as long as exp(A sum Delta) over the
 * sequence is a float32 number.  All sums, Delta and the states are float32; a bf16 result is
 * rounded once.  Tensors 16-byte aligned (B and C to their elements, lengths 4).
 * Bitwise reproducible.
 */
size_t mlstm_scan_workspace_bytes(int64_t batch, int64_t T, int64_t channels, int64_t G, int64_t N,
                                  int dtype, int backward);

/*
 * mlstm_scan_fwd -- a sequence (T = 1: the step of generation, bound by the
 * state's traffic).  state_out: the state after it; may be state_in (in place).
 *   workspace  mlstm_scan_workspace_bytes(..., 0) bytes, 256-byte aligned: none for
 *              T = 1 and where the channels fill the card; else long sequences are
 *              cut into segments that run side by side, so a position's result may
 *              differ in its last bits from that of a shorter call
 */
int mlstm_scan_fwd(const void* u, int64_t u_row, const void* dt, int64_t dt_row, const float* A,
                   const void* B, int64_t B_row, const void* C, int64_t C_row, const float* D,
                   const void* gate, int64_t gate_row, const float* dt_bias,
                   const float* state_in, const int32_t* lengths, void* y, float* state_out,
                   void* workspace, size_t workspace_bytes, int64_t batch, int64_t T,
                   int64_t channels, int64_t G, int64_t N, int dtype, void* stream);

/*
 * mlstm_scan_bwd -- its gradients, from dy [batch][T][channels] and dstate, that of
 * the state after the sequence (or NULL: zeros).
 *   du, ddt, dgate  [batch][T][channels] dtype;  dB, dC [batch][T][G][N] dtype
 *   dA [channels][N], dD, ddt_bias [channels] float32
 *   dD, dgate and ddt_bias with D, gate and dt_bias, else NULL
 *   dstate_out      of the state before, or NULL
 *   workspace       mlstm_scan_workspace_bytes(..., 1) bytes, 256-byte aligned:
 *                   chiefly the states at every 16th token (8th for N > 32), and 8 N
 *                   bytes for each token and 64 channels
 * The forward pass is formed again; nothing of it is kept.
 */
int mlstm_scan_bwd(const void* u, int64_t u_row, const void* dt, int64_t dt_row, const float* A,
                   const void* B, int64_t B_row, const void* C, int64_t C_row, const float* D,
                   const void* gate, int64_t gate_row, const float* dt_bias,
                   const float* state_in, const int32_t* lengths, const void* dy,
                   const float* dstate, void* du, void* ddt, float* dA, void* dB, void* dC,
                   float* dD, void* dgate, float* ddt_bias, float* dstate_out, void* workspace,
                   size_t workspace_bytes, int64_t batch, int64_t T, int64_t channels, int64_t G,
                   int64_t N, int dtype, void* stream);

/*
 * Gated feed-forward: both input projections of a block's feed-forward, the
 * activation and the product,
 *
 *   h = act(x w_gate^T) * (x w_up^T)       act(g) = g sigma(g) or g Phi(g)
 *
 *   x [M][D], w_gate, w_up [F][D], h [M][F], all dtype, contiguous
 *   D and F multiples of 8, at most 2^16; M <= 2^20, M max(D, 2 F) <= 2^33
 * Products are summed in float32 (float32 operands as three bf16 planes, 24
 * bits), and a bf16 h is rounded once.  mlstm_gated_ffn_bwd forms both products
 * again; for bf16 their gradients have 16 bits as operands of the products behind dx,
 * dw_gate and dw_up, which are rounded once.  Inputs finite (float32 ones below 2^127 in
 * magnitude).  Tensors 16-byte aligned; workspace mlstm_gated_ffn_workspace_bytes bytes,
 * 256-byte aligned.  Bitwise reproducible.
 */
enum { MLSTM_FFN_SILU = 0, MLSTM_FFN_GELU = 1 };

size_t mlstm_gated_ffn_workspace_bytes(int64_t M, int64_t D, int64_t F, int dtype, int backward);
int mlstm_gated_ffn_fwd(const void* x, const void* w_gate, const void* w_up, void* h,
                        void* workspace, size_t workspace_bytes, int64_t M, int64_t D, int64_t F,
                        int dtype, int activation, void* stream);
/* dh [M][F] in; dx [M][D], dw_gate, dw_up [F][D] out, all dtype */
int mlstm_gated_ffn_bwd(const void* x, const void* w_gate, const void* w_up, const void* dh,
                        void* dx, void* dw_gate, void* dw_up, void* workspace,
                        size_t workspace_bytes, int64_t M, int64_t D, int64_t F, int dtype,
                        int activation, void* stream);

/*
 * mlstm_gated_ffn_tiles -- in what tiles a product of a call is taken (on the host; for
 * tests and timings): tiles[0], [1] columns and rows of a tile's outputs, [2] tiles taken
 * whole, [3] tiles whose sums are split, [4] into so many shares.  Zeros for the forward
 * of few rows, which has no tiles.
 */
enum { MLSTM_FFN_FORWARD = 0, MLSTM_FFN_AGAIN = 1, MLSTM_FFN_DX = 2, MLSTM_FFN_WEIGHTS = 3 };
int mlstm_gated_ffn_tiles(int64_t M, int64_t D, int64_t F, int dtype, int product,
                          int64_t tiles[5]);

/* Human-readable text of a status code (static storage). */
const char* mlstm_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* MLSTM_H */
