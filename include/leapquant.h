/*
 * leapquant.h -- C ABI of the LeapQuant decode hot path for AMD Instinct
 * MI355X (gfx950).
 *
 * The operations follow the pages about LeapQuant:
 *   [EL] "LeapQuant: Efficient Linear Attention with Accurate Recurrent State
 *        Quantization" (paper listing page): Abstract, Figure 2 (per-token
 *        vs per-window quantization), Figure 4 (state = quantized residual +
 *        compensator tokens + buffered updates), Appendix Table 4 (the
 *        delta-rule instances and the buffered record (d_i, k~_i, u_i)).
 *   [TM] "LeapQuant trims the memory burden of linear-attention models"
 *        (news write-up), section "Quantize less often, protect the
 *        outliers" (window, compensators, smoothing across channels).
 *
 * Model.  Each of n independent states S (dk x dv, one per sequence, head and
 * layer) evolves by the delta rule of [EL] Table 4:
 *     u_t = v_t - S_{t-1}^T b_t,   S_t = D_t S_{t-1} + k~_t u_t^T,   o_t = S_t^T q_t
 *   LQ_GATE_GDN (Gated DeltaNet row): D_t = alpha_t I, k~_t = beta_t k_t,
 *                b_t = alpha_t k_t (alpha_t one scalar per state).
 *   LQ_GATE_KDA (Kimi Delta Attention): D_t = Diag(alpha_t), k~_t = beta_t k_t,
 *                b_t = alpha_t * k_t (alpha_t one value per key channel).
 *   With the LQ_NO_DELTA flag, b_t = 0 (the other rows of Table 4).
 * Between window boundaries the state is kept as ([EL] Figure 2, Figure 4)
 *   B  = deQ(codes, a, s) + sum_c e_{idx_c} w_c^T      (fixed, low-bit)
 *   records (d_i, k~_i, u_i), i < t                    (fp32 buffer)
 * and S_{t-1} is exactly the recurrence started from B and replayed through
 * the records.  deQ(c, a, s)_ij = c_ij * a_i * s_j.  At the end of a window
 * the state is rebuilt and split again: the r rows of largest L2 norm become
 * compensator rows w_c (fp32, descending norm, ties to the lower row), the
 * remaining residual R is smoothed per value column by s_j = max_i |R_ij|
 * (1 for a zero column, or 1 everywhere with LQ_NO_SMOOTH) and quantized
 * per row: m_i = max_j |R_ij * (1/s_j)|, a_i = m_i / 127,
 * c_ij = clamp(rne(R_ij * (1/s_j) * (127/m_i)), -127, 127), all in fp32.
 *
 * Conventions for every entry point.
 *   - All array pointers are DEVICE memory owned by the caller; the library
 *     allocates, frees and synchronizes nothing and keeps no global state,
 *     so calls are reentrant.  lq_params and lq_state are host structs read
 *     only during the call.
 *   - Work is enqueued on `stream` (NULL = the default stream) and the call
 *     returns without waiting.  Device faults surface at the caller's next
 *     synchronization.  Every pointer is memory of the device the launch
 *     runs on; call with that device current (hipSetDevice), since the
 *     default stream belongs to the current device.  The library keeps no
 *     state of its own and allocates no memory (the kernels use only the
 *     caller's arrays, registers and LDS), so every call may be captured in
 *     a graph; calls on different streams or host threads do not interfere
 *     unless their arrays overlap.
 *   - Arrays are dense, row-major, in the shapes given below; n is the
 *     leading dimension of every per-state array.  The codes of one state
 *     are a 16 KiB block stored column-major in two 64-row halves: code
 *     (i, j) is byte (i >> 6) * 8192 + j * 64 + slot(i & 63), where
 *     slot(x) = (x & 0x0C) << 2 | (x & 0x30) >> 2 | (x & 3) swaps the two
 *     2-bit fields above the lowest two bits.  Both kernels then move codes
 *     as 16-byte column segments (the int8 MFMA operand of the decode GEMV
 *     and the accumulator rows of one lane in the window close).
 *   - Alignment: codes and every float array whose per-state extent is a
 *     multiple of 128 floats must be 16-byte aligned; beta, a scalar alpha,
 *     comp_idx and a scalar buf_gate need 4-byte alignment.
 *   - Argument errors are returned synchronously and nothing is launched:
 *       LQ_ERR_NULL        a required pointer is NULL
 *       LQ_ERR_SHAPE       n < 1, p outside [1, 64], r outside [0, 16],
 *                          unknown gate or flag, t or len out of range
 *       LQ_ERR_UNSUPPORTED dk != 128 or dv != 128
 *       LQ_ERR_ALIGN       a pointer violates the alignment above
 *       LQ_ERR_ALIAS       an output range overlaps an input range, or two
 *                          arrays of the lq_state overlap (checked by every
 *                          call that writes the state)
 *     A failed launch returns LQ_ERR_HIP.
 *   - Values are not checked: NaN or Inf inputs give unspecified (but
 *     in-bounds) results.  comp_idx entries outside [0, dk) are ignored when
 *     the state is read; the r entries of a state are distinct rows (the
 *     split always writes them so), and duplicates give unspecified results.
 */
#ifndef LEAPQUANT_H
#define LEAPQUANT_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The version of the structures' layouts and of the entry points up to
 * leapquant_stream_reference.  The sequence, head norm, convolution, scan and
 * block norm calls were added in version 6: whether a library of that version
 * has them, its symbols tell. */
#define LEAPQUANT_ABI_VERSION 6

typedef enum lq_status {
  LQ_OK = 0,
  LQ_ERR_NULL = -1,
  LQ_ERR_SHAPE = -2,
  LQ_ERR_UNSUPPORTED = -3,
  LQ_ERR_ALIGN = -4,
  LQ_ERR_ALIAS = -5,
  LQ_ERR_HIP = -6
} lq_status;

typedef enum lq_gate {
  LQ_GATE_GDN = 0, /* scalar decay per state and token (Gated DeltaNet)  */
  LQ_GATE_KDA = 1  /* per-key-channel decay (Kimi Delta Attention)       */
} lq_gate;

enum {
  LQ_NO_SMOOTH = 1u, /* ablation: s_j = 1 for every column                     */
  LQ_NO_DELTA = 2u,  /* b_t = 0, so u_t = v_t: the rows of [EL] Appendix Table 4
                        without the delta correction.  With LQ_GATE_GDN: linear
                        attention (alpha = 1, beta = 1), RetNet (alpha = gamma,
                        beta = 1), Mamba2 (beta = 1); with LQ_GATE_KDA: GLA /
                        RWKV6 / HGRN2 (beta = 1).  DeltaNet is LQ_GATE_GDN with
                        alpha = 1 and the flag clear.                          */
  LQ_DENSE_COMP = 4u /* compensator tokens with dense keys (below)             */
};

/* Dense compensator tokens (LQ_DENSE_COMP).  The compensators are r tokens
 * (k_c, w_c) with dense fp32 keys k_c (comp_key) and values w_c (comp_val):
 * the boundary state is B = deQ + sum_c k_c w_c^T, and a compensator enters
 * the window like a buffered record written before the window's first token
 * (decay Gamma, weight k_c . (Gamma * y), update w_c): it is updated
 * exactly like a real token ([EL] Abstract; in Figure 4 the compensators
 * hold the state's largest components).  The window
 * close joins them to the fp32 rebuild as r more records of the same MFMA
 * contraction (K = len + r).  The split finds the keys by comp_iters rounds
 * of subspace iteration on S S^T started from the one-hot keys of the r
 * largest-norm rows: K <- MGS(S S^T K), modified Gram-Schmidt in compensator
 * order, a key whose projected norm is zero or at most 2e-2 of its norm
 * before projection becoming the zero key.  Then w_c = S^T k_c and the
 * residual S - sum_c k_c w_c^T is smoothed and quantized as usual; comp_idx
 * receives the starting rows.  With comp_iters = 0 the keys are the one-hot
 * rows and every result equals the row extraction's.  Without the flag,
 * comp_key is neither read nor written and comp_iters is ignored. */

typedef struct lq_params {
  int32_t n;      /* number of independent states in the slab (>= 1)     */
  int32_t dk;     /* key dimension, rows of S; must be 128                */
  int32_t dv;     /* value dimension, columns of S; must be 128           */
  int32_t p;      /* window length in tokens, 1..64                       */
  int32_t r;      /* compensator rows per state, 0..16                    */
  int32_t gate;   /* lq_gate                                              */
  uint32_t flags; /* LQ_NO_SMOOTH | LQ_NO_DELTA | LQ_DENSE_COMP, or 0      */
  int32_t comp_iters; /* LQ_DENSE_COMP: subspace iterations, 0..8         */
} lq_params;

/* One slab of n states.  codes .. comp_val and comp_key are the boundary
 * state (the prefix-cache snapshot); buf_gate, buf_k and buf_u are the
 * window buffer.  For r == 0, comp_idx, comp_val and comp_key may be NULL;
 * comp_key may be NULL without LQ_DENSE_COMP.  The arrays a call uses must
 * not overlap one another, since a launch that writes some of them reads the
 * others: the calls that write the state return LQ_ERR_ALIAS otherwise. */
typedef struct lq_state {
  int8_t *codes;     /* [n][dk*dv]  int8 residual codes c_ij (layout above) */
  float *row_scale;  /* [n][dk]     a_i                                     */
  float *col_scale;  /* [n][dv]     s_j                                     */
  int32_t *comp_idx; /* [n][r]      row index of each compensator row       */
  float *comp_val;   /* [n][r][dv]  compensator rows w_c                    */
  float *buf_gate;   /* GDN: [n][p]; KDA: [n][p][dk]   d_i (alpha_i)        */
  float *buf_k;      /* [n][p][dk]  k~_i = beta_i k_i                       */
  float *buf_u;      /* [n][p][dv]  u_i                                     */
  float *comp_key;   /* [n][r][dk]  LQ_DENSE_COMP: compensator keys k_c     */
} lq_state;

/* Split fp32 states S [n][dk][dv] into the boundary state of `st` (codes,
 * row_scale, col_scale, comp_idx, comp_val); the window buffer is neither
 * read nor written.  This is the window-boundary split of [EL] Figure 4
 * applied to a state that has no buffered updates, i.e. the quantized
 * boundary state that precedes the first window of [EL] Figure 2.  S must
 * not overlap the boundary-state arrays. */
int leapquant_quantize_state(const lq_params *prm, const float *S,
                             const lq_state *st, hipStream_t stream);

/* Decode token t (0-based position inside the current window, 0 <= t < p)
 * for all n states ([EL] Figure 2, per-window quantization; [EL] Abstract,
 * compensators are updated like real tokens).  Reads the boundary
 * state and the records 0..t-1 of the buffer, writes
 *   o[n][dv] = S_t^T q_t, with S_t the exact recurrence from the boundary
 *              state through the buffered records and this token,
 * and appends record t: buf_gate[.][t] = alpha_t, buf_k[.][t] = beta_t k_t,
 * buf_u[.][t] = v_t - S_{t-1}^T b_t.
 * Inputs: q, k [n][dk]; v [n][dv]; beta [n]; alpha [n] (GDN) or [n][dk]
 * (KDA); all read-only.  o must not overlap any input or state array.
 * The caller closes the window (leapquant_window_close with len = p)
 * after t = p - 1 and before the next t = 0. */
int leapquant_decode_step(const lq_params *prm, const lq_state *st, int32_t t,
                          const float *q, const float *k, const float *v,
                          const float *beta, const float *alpha, float *o,
                          hipStream_t stream);

/* Close a window of len buffered records (1 <= len <= p; len < p only for
 * a final partial window): rebuild S_len = D_len..D_1 B + sum_i
 * (D_len..D_{i+1}) k~_i u_i^T in fp32, then split it into compensator rows,
 * smoothing scales, row scales and int8 codes, overwriting the boundary
 * state in place ([EL] Figure 2: quantize once per window; [EL] Figure 4).
 * The buffer is read, not cleared. */
int leapquant_window_close(const lq_params *prm, const lq_state *st,
                           int32_t len, hipStream_t stream);

/* Decode token t and close the window in one pass (the fused form of
 * leapquant_decode_step(t) followed by leapquant_window_close(len = t + 1);
 * [EL] Figure 2: the state is quantized once per window, at its last
 * token).  Reads the boundary state and the records 0..t-1, rebuilds
 * D_t S_{t-1} in fp32, writes o[n][dv] = S_t^T q_t with
 *   u_t = v_t - S_{t-1}^T b_t,  S_t = D_t S_{t-1} + k~_t u_t^T,
 * then splits S_t into the new boundary state, overwriting it in place.
 * Record t is not written to the buffer (the window is closed).  Arguments,
 * layouts, alignment and aliasing rules are those of leapquant_decode_step;
 * t is normally p - 1 (t < p - 1 closes a final partial window).  Results
 * agree with the two-call form to fp32 rounding, not bit for bit: the
 * fused form reads S_{t-1} from the rebuilt state instead of the windowed
 * sums. */
int leapquant_decode_close(const lq_params *prm, const lq_state *st, int32_t t,
                           const float *q, const float *k, const float *v,
                           const float *beta, const float *alpha, float *o,
                           hipStream_t stream);

/* Write the boundary state B = deQ(codes, a, s) + compensator rows as fp32
 * S_out [n][dk][dv]: the quantized residual plus the compensators that
 * [EL] Figure 4 splits the state into, i.e. the state the next window
 * starts from ([EL] Figure 2); used for state error tracking (the MSE of
 * [EL] Figure 3) and prefix-cache reads.  Row-major, 16-byte aligned;
 * S_out must not overlap `st` (LQ_ERR_ALIAS); other errors as for
 * leapquant_quantize_state. */
int leapquant_dequantize_state(const lq_params *prm, const lq_state *st,
                               float *S_out, hipStream_t stream);

/* ---- Continuous batching.  The slots of a slab hold sequences at
 * different positions of their own windows (requests join and finish
 * independently).  pos[n] and len[n] are int32 arrays in DEVICE memory,
 * read by the kernels (4-byte aligned, read-only, overlapping no state
 * array or output); the host keeps them up to date, typically with one
 * small device operation per token.
 *
 * leapquant_decode_step_slots: slot s decodes its token at window position
 * pos[s] exactly as leapquant_decode_step would with t = pos[s]; a slot with
 * pos[s] outside [0, p) is idle (its o row and state are left as they are).
 * leapquant_decode_close_slots: the same for the fused last-token decode
 * and close of leapquant_decode_close (slot s closes with pos[s] + 1
 * records); idle slots as above.
 * leapquant_window_close_slots: slot s is closed with len[s] records when
 * 1 <= len[s] <= p (len[s] < p closes a partial window at the end of a
 * sequence); other slots are left as they are.
 * The other arguments and the error codes are those of the uniform calls;
 * values in pos and len cannot be checked on the host. */
int leapquant_decode_step_slots(const lq_params *prm, const lq_state *st, const int32_t *pos,
                                const float *q, const float *k, const float *v,
                                const float *beta, const float *alpha, float *o,
                                hipStream_t stream);
int leapquant_decode_close_slots(const lq_params *prm, const lq_state *st, const int32_t *pos,
                                 const float *q, const float *k, const float *v,
                                 const float *beta, const float *alpha, float *o,
                                 hipStream_t stream);
int leapquant_window_close_slots(const lq_params *prm, const lq_state *st, const int32_t *len,
                                 hipStream_t stream);

/* Compacted closes.  At a given token only the slots whose windows end
 * close, about one slot in p; the _slots calls above still start one
 * workgroup per slot, and the idle ones cost launch time.  These calls take
 * list[count], int32 slot ids in DEVICE memory (4-byte aligned, read-only,
 * overlapping no state array, output or the per-slot array), and start
 * one workgroup per entry: listed slot s is processed exactly as the
 * matching _slots call processes it with pos[s] / len[s] (a listed slot
 * whose pos or len is out of range is idle); ids outside [0, n) are
 * skipped; unlisted slots are not touched.  0 <= count <= n (LQ_ERR_SHAPE
 * otherwise); count == 0 launches nothing and returns LQ_OK.  A slot listed
 * twice is closed twice concurrently, which races: the caller lists each
 * slot at most once (device values cannot be checked on the host).  The
 * other arguments and error codes are those of the _slots calls. */
int leapquant_decode_close_list(const lq_params *prm, const lq_state *st, const int32_t *pos,
                                const int32_t *list, int32_t count, const float *q,
                                const float *k, const float *v, const float *beta,
                                const float *alpha, float *o, hipStream_t stream);
int leapquant_window_close_list(const lq_params *prm, const lq_state *st, const int32_t *len,
                                const int32_t *list, int32_t count, hipStream_t stream);

/* One continuous-batching token in one launch ([EL] Figure 2: each slot
 * decodes against its fixed boundary state and closes its own window after
 * its p-th token).  Slot s with 0 <= pos[s] < p - 1 decodes its token
 * exactly as leapquant_decode_step_slots does; listed slot s with
 * pos[s] == p - 1 decodes its token and closes its window exactly as
 * leapquant_decode_close_list does.  Slots at position p - 1 that are not
 * listed, listed slots at any other position, ids outside [0, n) and slots
 * outside [0, p) are left as they are.  The result equals
 * leapquant_decode_step_slots over the positions with p - 1 replaced by -1
 * followed by leapquant_decode_close_list over the listed slots at p - 1,
 * bit for bit.  For slabs of more than 4,096 slots with 4 <= p <= 16 and
 * at most 8 compensator rows (no dense compensator tokens) it is a single
 * launch: the closing slots' workgroups run among the decode steps, which
 * keep memory busy around them, so the closes no longer cost a launch of
 * their own; other shapes run the two launches.  Arguments, list rules
 * and error codes are those of leapquant_decode_close_list. */
int leapquant_decode_step_close_list(const lq_params *prm, const lq_state *st, const int32_t *pos,
                                     const int32_t *list, int32_t count, const float *q,
                                     const float *k, const float *v, const float *beta,
                                     const float *alpha, float *o, hipStream_t stream);

/* ---- Uncompressed baselines ([EL] Table 2, rows "FP32 per-step" and
 * "BF16 per-step"): the same token update on a dense state that is read
 * and written in full every token.  Provided to measure the quantized path
 * against in the same harness; not part of the quantized decode. */
typedef enum lq_dense_dtype {
  LQ_DENSE_FP32 = 0, /* S is float [n][dk][dv]                            */
  LQ_DENSE_BF16 = 1  /* S is bfloat16 (uint16 bit patterns) [n][dk][dv];
                        computed in fp32, stored rounded to nearest even   */
} lq_dense_dtype;

/* One token for n dense states, in place: u_t = v_t - S^T b_t,
 * S <- D_t S + k~_t u_t^T, o[n][dv] = S^T q_t (the recurrence of [EL]
 * Table 4 with no quantization).  prm supplies n, dk, dv and gate (p, r
 * and flags must be valid but are not used).  S is row-major (row = key
 * channel), 16-byte aligned (fp32) or 8-byte aligned (bf16); the token
 * inputs follow leapquant_decode_step.  S and o must not overlap each other
 * or any input. */
int leapquant_dense_step(const lq_params *prm, void *S, int32_t dtype,
                         const float *q, const float *k, const float *v,
                         const float *beta, const float *alpha, float *o,
                         hipStream_t stream);

/* Static description of a status code (never NULL). */
const char *leapquant_status_string(int status);

/* ---- "BF16 + per-window" ([EL] Table 2, the row between BF16 per-step and
 * INT8 per-step): the boundary state is a dense bf16 state B [n][dk][dv]
 * (row-major, bfloat16 bit patterns), fixed for the window.  Within the
 * window the tokens are buffered in the fp32 records of `st` exactly as in
 * the int8 path (only buf_gate, buf_k and buf_u of `st` are used; r,
 * LQ_NO_SMOOTH and LQ_DENSE_COMP do not apply: flags may hold only
 * LQ_NO_DELTA).  The decode step reads B and the records.  The window close
 * rebuilds S = Gamma * B + K_w U in fp32 (rows scaled by the decay product
 * Gamma of the window) and writes it back into B rounded to bf16, nearest
 * with ties to even.  There is no fused last-token close for this row. */

/* Decode token t (0 <= t < p) of the window for all n states: reads B and
 * records 0 .. t-1, writes o and record t.  Errors as for
 * leapquant_decode_step; B must be 16-byte aligned and overlap neither the
 * buffer nor o. */
int leapquant_bf16w_decode_step(const lq_params *prm, const void *B, const lq_state *st, int32_t t,
                                const float *q, const float *k, const float *v, const float *beta,
                                const float *alpha, float *o, hipStream_t stream);

/* Close the window after len tokens (1 <= len <= p): B <- bf16(Gamma * B +
 * K_w U).  The buffer is read, not written. */
int leapquant_bf16w_window_close(const lq_params *prm, void *B, const lq_state *st, int32_t len,
                                 hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Whole sequences: prompts before decode, and training.
 *
 * The same recurrence ([EL] Appendix Table 4) over all tokens of a packed
 * batch of sequences, from fp32 states to fp32 states: what produces the
 * states that leapquant_quantize_state splits for decode, and its gradient.
 *
 * Tokens of all sequences lie behind one another: sequence i holds tokens
 * cu_seqlens[i] .. cu_seqlens[i + 1] - 1 (seqs + 1 int32 on the device,
 * ascending, within [0, tokens]; a sequence may be empty).  Tokens before
 * the first and behind the last sequence are neither read nor written.
 * Offsets are held to [0, tokens]; offsets that do not ascend give
 * unspecified (but in-bounds) results.  Value head h uses query and key
 * head h / (heads_v / heads_k).  State (i, h) is block i * heads_v + h of
 * S0 and S, [seqs * heads_v][dk][dv], the layout of leapquant_quantize_state.
 * q and k are used as given (unit-norm keys keep the recurrence stable; the
 * decode calls expect the same), with no scale.
 * Values are finite, below 2^127, and decays from 0 to 1 (both inclusive).
 * 64 tokens of a sequence may be computed together: a value that is not
 * finite reaches the outputs of tokens at and behind it, as the formulas say,
 * and may reach those of up to 63 tokens before it; never another sequence
 * nor, in the forward pass, another head's states.
 * ------------------------------------------------------------------------- */

typedef enum lq_dtype {
  LQ_F32 = 0,
  LQ_BF16 = 1,
  LQ_F16 = 2
} lq_dtype;

/* A strided array [tokens][heads][128] (or [tokens][heads] for scalars):
 * element (t, h, c) is ptr[t * token_stride + h * head_stride + c], strides
 * in elements and not negative.  The 128 values of a head are contiguous.
 * Arrays of heads need a 16-byte aligned ptr and strides that are whole
 * multiples of 16 bytes; scalars need 4-byte alignment.  Inputs may repeat
 * memory (stride 0); of an output, no two elements may be the same memory.
 * Slices of one larger row (q, k and v out of one projection, or their
 * gradients into one) are fine, also head by head.  Outputs share no memory
 * with inputs or other outputs (LQ_ERR_ALIAS): exact for arrays of one token
 * stride; arrays of other token strides whose ranges interleave, and more than
 * 65,536 pairs of heads in interleaved head strides that differ, count as
 * sharing. */
typedef struct lq_rows {
  void *ptr;
  int64_t token_stride;
  int64_t head_stride;
} lq_rows;

typedef struct lq_sequence {
  int64_t tokens;  /* rows of the token arrays, >= 0, below about 2^29        */
  int32_t seqs;    /* sequences, >= 1                                         */
  int32_t heads_k; /* query and key heads, >= 1                               */
  int32_t heads_v; /* value heads, a multiple of heads_k                      */
  int32_t dk;      /* must be 128                                             */
  int32_t dv;      /* must be 128                                             */
  int32_t gate;    /* lq_gate                                                 */
  uint32_t flags;  /* LQ_NO_DELTA or 0                                        */
  int32_t dtype;   /* lq_dtype of q, k, v, o and their gradients              */
} lq_sequence;

/* Bytes of workspace that are enough for every call with these parameters
 * and at most these tokens and seqs (0 is possible), or a negative
 * lq_status.  save: for a forward call that a backward call follows, and for
 * that backward call.  The workspace is 16-byte aligned device memory. */
int64_t leapquant_sequence_workspace(const lq_sequence *sq, int32_t save);

/* The forms of the forward call: token by token for few tokens a sequence,
 * 64 tokens together otherwise.  Without save the call goes by the average,
 * tokens / seqs (up to 24; up to 56 with fp32 operands or a decay a channel and
 * 256 states or more), as the lengths are on the device.  A long sequence among
 * many short ones therefore takes its tokens one by one (about 1 us each with
 * thousands of states): such a batch is better two calls, the long sequences'
 * and the short ones', on slices of the token arrays or, for a run of
 * sequences, on the same arrays with cu_seqlens, S0 and S from the run's first
 * sequence on (tokens, the arrays' rows, is what the average counts). */

/* Forward: for every sequence and value head, from state S0 (NULL: zeros),
 *   u_t = v_t - S_{t-1}^T b_t,  S_t = D_t S_{t-1} + k~_t u_t^T,  o_t = S_t^T q_t.
 * Inputs: q, k [tokens][heads_k][128] and v [tokens][heads_v][128] of dtype;
 * beta [tokens][heads_v] fp32; alpha fp32, [tokens][heads_v] (GDN) or
 * [tokens][heads_v][128] (KDA).  Outputs: o [tokens][heads_v][128] of dtype;
 * S the states after the last token (NULL: not wanted; may be S0 itself).
 * Sums and states are fp32; o is rounded once.  With save != 0 the workspace
 * afterwards holds what leapquant_sequence_backward reads.
 *   LQ_ERR_SHAPE also: workspace_bytes too small, an output whose elements
 *   coincide, more tokens, heads or sequences than a launch takes;
 *   LQ_ERR_UNSUPPORTED also: save with LQ_GATE_KDA. */
int leapquant_sequence_forward(const lq_sequence *sq, const int32_t *cu_seqlens,
                               const lq_rows *q, const lq_rows *k, const lq_rows *v,
                               const lq_rows *beta, const lq_rows *alpha, const lq_rows *o,
                               const float *S0, float *S, void *workspace,
                               int64_t workspace_bytes, int32_t save, hipStream_t stream);

/* Backward (LQ_GATE_GDN): from go, the gradient of o, and dS, that of S
 * (NULL: zeros), the gradients of q, k (summed over the value heads that
 * share them), v, beta, alpha and S0 (dS0 NULL: not wanted).  Call with the
 * parameters, cu_seqlens, q, k, beta and alpha of a forward call with save,
 * and its workspace, unchanged since (backward may be called more than once
 * on it).  Every result is summed in a fixed order. */
int leapquant_sequence_backward(const lq_sequence *sq, const int32_t *cu_seqlens,
                                const lq_rows *q, const lq_rows *k, const lq_rows *beta,
                                const lq_rows *alpha, const lq_rows *go, const float *dS,
                                const lq_rows *dq, const lq_rows *dk, const lq_rows *dv,
                                const lq_rows *dbeta, const lq_rows *dalpha, float *dS0,
                                void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Norm of query and key heads, with the position rotation.
 *
 * What makes the unit-norm queries and keys that the calls above and the
 * decode calls take: LQ_NORM_L2, or LQ_NORM_RMS with a weight that holds the
 * factor 128^-1/2 (an RMS-normed head of 128 values has norm 128^1/2, and keys
 * of a norm above 1 make the recurrence grow).  For each head x of 128 values
 * of token t:
 *   r = (sum x^2 + eps)^-1/2 (LQ_NORM_L2) or (sum x^2 / 128 + eps)^-1/2 (LQ_NORM_RMS)
 *   y = s * R(positions[t]) (w * x * r)
 * with w the weight of 128 values (NULL: ones), s = q_scale for queries and 1
 * for keys, and R the rotation of the first rot values in pairs (c, c + rot / 2),
 * or (2c, 2c + 1) with interleaved, by the angle positions[t] * inv_freq[c],
 * whose product is taken in 64 bits.  Sums of squares are fp32: values below
 * 2^60.
 * ------------------------------------------------------------------------- */

typedef enum lq_norm_kind {
  LQ_NORM_L2 = 0,
  LQ_NORM_RMS = 1
} lq_norm_kind;

typedef struct lq_head_norm {
  int64_t tokens;      /* >= 0; times runs of 16 heads below 2^25              */
  int32_t heads_q;     /* query heads, >= 0                                    */
  int32_t heads_k;     /* key heads, >= 0; at least one head in all            */
  int32_t dim;         /* must be 128                                          */
  int32_t kind;        /* lq_norm_kind                                         */
  int32_t dtype;       /* lq_dtype of q and k and of their gradients           */
  int32_t dtype_out;   /* lq_dtype of the outputs and of their gradients       */
  int32_t rot;         /* rotated values, 0 .. 128, a multiple of 16           */
  int32_t interleaved; /* 0: pairs (c, c + rot / 2); 1: pairs (2c, 2c + 1)     */
  float eps;           /* > 0                                                  */
  float q_scale;
  const float *q_weight;    /* [128], 16-byte aligned, or NULL                 */
  const float *k_weight;    /* [128], 16-byte aligned, or NULL                 */
  const int64_t *positions; /* [tokens]; NULL only with rot = 0                */
  const double *inv_freq;   /* [rot / 2] radians per position; NULL likewise   */
} lq_head_norm;

/* q, q_out [tokens][heads_q][128], k, k_out [tokens][heads_k][128].  An
 * output may be its own input (the same pointer, strides and dtype). */
int leapquant_head_norm(const lq_head_norm *nm, const lq_rows *q, const lq_rows *k,
                        const lq_rows *q_out, const lq_rows *k_out, hipStream_t stream);

/* Bytes of workspace of leapquant_head_norm_backward with weight gradients,
 * or a negative lq_status. */
int64_t leapquant_head_norm_workspace(int64_t tokens, int32_t heads_q, int32_t heads_k);

/* From the outputs' gradients gq, gk (dtype_out) and the inputs q, k, the
 * inputs' gradients dq, dk (dtype) and the weights' dq_weight, dk_weight
 * ([128] fp32, each NULL if not wanted; the sums over all tokens and heads in
 * a fixed order, zeros if there are none).  The workspace is used only with a
 * weight gradient. */
int leapquant_head_norm_backward(const lq_head_norm *nm, const lq_rows *q, const lq_rows *k,
                                 const lq_rows *gq, const lq_rows *gk, const lq_rows *dq,
                                 const lq_rows *dk, float *dq_weight, float *dk_weight,
                                 void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Around the recurrence: the short causal convolution that queries, keys and
 * values (or the inputs of a state space layer) pass before it, the selective
 * state space scan, and the norms before and after a block with its gate and
 * residual scale.
 *
 * Arrays of channels, [tokens][channels], are lq_rows whose head stride is not
 * used: element (t, c) is ptr[t * token_stride + c], aligned to its type, with
 * any stride and any number of channels.  Sequences are packed as above, with
 * the same rules for cu_seqlens and for tokens of no sequence.  Sums, states
 * and statistics are fp32 whatever the type of the arrays, results are rounded
 * once, and every sum is added in a fixed order.
 *
 * The calls for single tokens take one token of each of `tokens` rows; row i is
 * the next token of slot slots[i] (int32 on the device; NULL: of slot i, and
 * tokens <= n_slots).  Rows whose slot is outside [0, n_slots) are idle: their
 * outputs and every unlisted slot are left as they are.  A slot listed twice
 * races: the caller lists each at most once (device values cannot be checked
 * on the host).
 * ------------------------------------------------------------------------- */

typedef enum lq_activation {
  LQ_ACT_NONE = 0,
  LQ_ACT_SILU = 1,    /* x / (1 + e^-x) */
  LQ_ACT_SIGMOID = 2  /* 1 / (1 + e^-x) */
} lq_activation;

/* Convolution of every channel with `width` weights over its own past:
 *   v_t = bias + sum_{j < width} weight[c][j] x_{t - width + 1 + j},   y_t = act(v_t)
 * The width - 1 inputs before a sequence's first token are X0[seq][0 ..][c],
 * the last one next to it (NULL: zeros); X receives the last width - 1 inputs
 * of each sequence (NULL: not wanted), for its next tokens.  X0 and X
 * ([seqs][width - 1][channels] of dtype) may not overlap in the calls over
 * sequences. */
typedef struct lq_conv {
  int64_t tokens;      /* rows of the token arrays, >= 0                       */
  int32_t seqs;        /* sequences, >= 1 (not read for single tokens)         */
  int32_t channels;    /* 1 .. 2^20                                            */
  int32_t width;       /* 2, 3 or 4 (LQ_ERR_UNSUPPORTED otherwise)             */
  int32_t activation;  /* LQ_ACT_NONE or LQ_ACT_SILU                           */
  int32_t dtype;       /* lq_dtype of x, y, X0, X and their gradients          */
  const float *weight; /* [channels][width]                                    */
  const float *bias;   /* [channels] or NULL                                   */
} lq_conv;

int leapquant_conv_forward(const lq_conv *cv, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *y,
                           const void *X0, void *X, hipStream_t stream);

/* One token of each row: the slots' earlier inputs X0 [n_slots][width - 1]
 * [channels] in, the ones after the token out to X (may be X0). */
int leapquant_conv_step(const lq_conv *cv, const int32_t *slots, int32_t n_slots, const lq_rows *x, const lq_rows *y,
                        const void *X0, void *X, hipStream_t stream);

/* Bytes of workspace of leapquant_conv_backward with a weight or bias gradient,
 * enough for at most these tokens, or a negative lq_status (weight is not
 * read). */
int64_t leapquant_conv_workspace(const lq_conv *cv);

/* From dy, the gradient of y, and dX, that of X (NULL: zeros): dx, dX0,
 * dweight and dbias (fp32; the last three each NULL if not wanted).  X0 as
 * forward. */
int leapquant_conv_backward(const lq_conv *cv, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *dy,
                            const lq_rows *dx, const void *X0, const void *dX, void *dX0, float *dweight, float *dbias,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Selective state space scan.  Channel c of group g = c / (channels / groups)
 * has `states` states h_n with a decay each:
 *   d = dt + dt_bias, or log(1 + e^(dt + dt_bias)) with LQ_SCAN_SOFTPLUS
 *   h_n <- e^(d A_n) h_n + d B_n x,   y = (sum_n C_n h_n + D x) z / (1 + e^-z)
 * (without z: no last factor).  Where every channel of a head has one decay for
 * all states and steps and inputs are its keys and values, the recurrence is
 * that of leapquant_sequence_forward with LQ_NO_DELTA; here each channel and
 * state has its own.  e^(d A) is a decay: d A <= 0, values finite. */
enum { LQ_SCAN_SOFTPLUS = 1u };

typedef struct lq_scan {
  int64_t tokens;       /* rows of the token arrays, >= 0                      */
  int32_t seqs;         /* sequences, >= 1 (not read for single tokens)        */
  int32_t channels;     /* 1 .. 2^20, a multiple of groups                     */
  int32_t states;       /* 8, 16 or 32 (LQ_ERR_UNSUPPORTED otherwise)          */
  int32_t groups;       /* groups of channels that share B and C, >= 1         */
  int32_t dtype;        /* lq_dtype of the token arrays                        */
  uint32_t flags;       /* LQ_SCAN_SOFTPLUS or 0                               */
  const float *A;       /* [channels][states], 16-byte aligned                 */
  const float *D;       /* [channels] or NULL (zeros)                          */
  const float *dt_bias; /* [channels] or NULL (zeros)                          */
} lq_scan;

/* Bytes of workspace that are enough for every call with these parameters and
 * at most these tokens and seqs (0 is possible), or a negative lq_status.
 * save: for a forward call that a backward call follows, and for that call. */
int64_t leapquant_scan_workspace(const lq_scan *sc, int32_t save);

/* x, dt, z (NULL: none), y [tokens][channels]; B, C [tokens][groups][states]
 * (arrays of heads of `states` values: 16-byte aligned, also their strides);
 * S0, S [seqs][channels][states] fp32, the states before (NULL: zeros) and
 * after (NULL: not wanted; may be S0).  With save != 0 the workspace
 * afterwards holds what leapquant_scan_backward reads. */
int leapquant_scan_forward(const lq_scan *sc, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *dt,
                           const lq_rows *B, const lq_rows *C, const lq_rows *z, const lq_rows *y, const float *S0,
                           float *S, void *workspace, int64_t workspace_bytes, int32_t save, hipStream_t stream);

/* One token of each row: the slots' states S0 [n_slots][channels][states] in,
 * the ones after the token out to S (may be S0). */
int leapquant_scan_step(const lq_scan *sc, const int32_t *slots, int32_t n_slots, const lq_rows *x, const lq_rows *dt,
                        const lq_rows *B, const lq_rows *C, const lq_rows *z, const lq_rows *y, const float *S0, float *S,
                        hipStream_t stream);

/* From dy, the gradient of y, and dS, that of S (NULL: zeros), the gradients of
 * every input: dx, ddt, dB, dC, dz (NULL without z, and only then), dA, dD and
 * ddt_bias (these two NULL if not wanted, and without D and dt_bias) and dS0
 * (NULL: not wanted; may be dS).  Call with the parameters and inputs of a forward call
 * with save, and its workspace, unchanged since but by backward calls (there
 * may be more than one). */
int leapquant_scan_backward(const lq_scan *sc, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *dt,
                            const lq_rows *B, const lq_rows *C, const lq_rows *z, const lq_rows *dy, const lq_rows *dx,
                            const lq_rows *ddt, const lq_rows *dB, const lq_rows *dC, const lq_rows *dz, float *dA,
                            float *dD, float *ddt_bias, const float *dS, float *dS0, void *workspace,
                            int64_t workspace_bytes, hipStream_t stream);

/* Norms before and after a block.  For a row of `dim` values of a token and
 * head, with m(x) = (sum x^2 / dim + eps)^-1/2, from a block's output a,
 *   n = out_weight * a * m(a)   (out_norm; otherwise n = a)
 *   u = n * act(z)              (without a gate u = n)
 *   h = res + scale * u         (without res h = scale * u)
 *   y = in_weight * h * m(h)    (the input of the next block)
 * With heads of 128 values, out_norm and a SiLU gate it is the gated norm of a
 * recurrence's outputs; with one head of the model's width, res and y it joins
 * a block to the residual stream and norms it for the next one.  y is made of h
 * before h is rounded.  Values of a, z, res and h below 2^60, gradients below
 * 2^50. */
typedef struct lq_block_norm {
  int64_t tokens;          /* >= 0                                             */
  int32_t heads;           /* rows of a token, >= 1                            */
  int32_t dim;             /* values of a row, 8 .. 8192, a multiple of 8      */
  int32_t dtype;           /* lq_dtype of a, z, y and their gradients          */
  int32_t dtype_stream;    /* of res, h and their gradients: dtype or LQ_F32   */
  int32_t gate;            /* lq_activation of z, or LQ_ACT_NONE without z     */
  int32_t out_norm;        /* 1: norm of a                                     */
  float eps;               /* > 0                                              */
  float scale;
  const float *out_weight; /* [dim], 16-byte aligned, or NULL (ones)           */
  const float *in_weight;  /* [dim], 16-byte aligned, or NULL (ones)           */
} lq_block_norm;

/* Arrays of heads of dim values (lq_rows above; 16-byte aligned pointers and
 * strides).  z and res NULL without them; h and y each NULL if not wanted.  An
 * output may be a or res itself (the same pointer, strides and type). */
int leapquant_block_norm(const lq_block_norm *bn, const lq_rows *a, const lq_rows *z, const lq_rows *res, const lq_rows *h,
                         const lq_rows *y, hipStream_t stream);

/* Bytes of workspace of leapquant_block_norm_backward with a weight gradient,
 * enough for at most these tokens, or a negative lq_status. */
int64_t leapquant_block_norm_workspace(int64_t tokens, int32_t heads, int32_t dim);

/* From dh and dy, the gradients of h and y (one of them may be NULL: zeros),
 * and the inputs of the forward call (res is not read without dy): da, dz
 * (NULL without z, and only then), dres (NULL if not wanted; may be dh itself),
 * dout_weight and din_weight (fp32 [dim], each NULL if not wanted, and without
 * out_norm or dy). */
int leapquant_block_norm_backward(const lq_block_norm *bn, const lq_rows *a, const lq_rows *z, const lq_rows *res,
                                  const lq_rows *dh, const lq_rows *dy, const lq_rows *da, const lq_rows *dz,
                                  const lq_rows *dres, float *dout_weight, float *din_weight, void *workspace,
                                  int64_t workspace_bytes, hipStream_t stream);

/* ---- Measurement reference, no part of the method: a plain stream in
 * the decode step's launch shape.  One 64-lane wave per block of
 * read_bytes_per_wave bytes at src reads its block with 16-byte nontemporal
 * loads, 16 KiB per wave issued at a time, then sleeps idle_sleeps times
 * 512 cycles with nothing in flight (a stand-in for the work a decode wave
 * does after its loads return), then writes write_bytes_per_wave bytes at
 * dst + wave * write_bytes_per_wave (8 bytes per lane per 512-byte row, as
 * the decode step stores its output rows).  Timed beside the decode step
 * with idle_sleeps = 0, it gives the rate the device reaches for the same
 * bytes per wave, read/write mix and waves per launch with no arithmetic
 * between.  Also
 * writes waves * 64 checksum words to out (each the sum over the lane's
 * 16-byte loads of the XOR of their four 32-bit words).
 * read_bytes_per_wave a positive multiple of 1024, write_bytes_per_wave a
 * multiple of 512 (0 allowed, then dst may be NULL), both at most 2^30;
 * 0 <= idle_sleeps <= 4096; waves >= 1 (LQ_ERR_SHAPE otherwise); src and
 * dst 16-byte aligned, out
 * 4-byte aligned (LQ_ERR_ALIGN); dst and out must not overlap each other
 * or the bytes read (LQ_ERR_ALIAS). */
int leapquant_stream_reference(const void *src, int64_t read_bytes_per_wave, void *dst,
                               int64_t write_bytes_per_wave, int32_t idle_sleeps, int32_t waves,
                               uint32_t *out, hipStream_t stream);

/* LEAPQUANT_ABI_VERSION of the loaded library. */
int leapquant_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LEAPQUANT_H */
