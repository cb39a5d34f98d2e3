// Internal launch interface between the sequence entry points
// (lq_sequence_abi.cpp) and their gfx950 kernels (lq_sequence.hip,
// lq_sequence_grad.hip, lq_norm.hip).  Arguments are validated by the caller.
#pragma once
#include <stdint.h>
#include <hip/hip_runtime_api.h>

namespace lq {

constexpr int kChunk = 64;  // tokens of one chunk of the sequence kernels

// [tokens][heads][128] (or [tokens][heads] scalars) with element strides;
// the last axis is contiguous.
struct Rows {
  void *ptr;
  int64_t ts, hs;
};

// What the chunk kernels hand on, per chunk slot and head.  A slot is one
// chunk of one sequence: sequence i, chunk c has slot cu[i] / 64 + i + c, so
// `slots` = tokens / 64 + seqs slots cover any split of the tokens into
// sequences without a pass that counts them.  The matrices are kept as
// operands of the scans: bf16 parts in fragments of 16 rows x 32 contraction
// indexes (64 lanes x 16 bytes a part; n parts: 1 of bf16 inputs, 2 of fp16,
// 3 of fp32 ones).  With a decay for every channel K, Q and K^T hold decays:
// they are kept per value head, in 3 parts, and dec is the chunk's decay of
// every key row.
struct SeqSpace {
  uint16_t *T, *P;        // [slots][hv][4][2][3]  (I + M)^-1; decayed, beta-weighted q k^T
  uint16_t *K, *Q;        // [slots][hk][4][4][n]
  uint16_t *KT;           // [slots][hk][8][2][n]
  float *dec;             // [slots][hv][2][64]    decay from the chunk's start; beta times decay to its end
  // kept for the backward pass (else nullptr)
  uint16_t *TT, *PT;      // [slots][hv][4][2][3]  their transposes
  uint16_t *QT;           // [slots][hk][8][2][n]
  float *U;               // [slots][hv][64][128]  u_t
  float *S;               // [slots][hv][dk][dv]   state at the chunk's start
  float *X;               // [slots][hv][64][128]  backward: gradient of v
  float *G;               // [slots][hv][dk][dv]   backward: gradient of the state at the chunk's end
};

struct SeqArgs {
  int64_t tokens, slots;
  int seqs, hk, hv, group;
  const int32_t *cu;
  Rows q, k, v, beta, alpha, o;
  const float *S0;  // [seqs * hv][dk][dv] or nullptr (zeros)
  float *S;         // [seqs * hv][dk][dv] or nullptr
  SeqSpace w;
  // backward
  Rows go, dq, dk, dv, dbeta, dalpha;
  const float *dS;
  float *dS0;
};

struct NormArgs {
  int64_t tokens;
  int hq, hk;
  int rms, interleaved, rot;
  float eps, q_scale;
  Rows q, k;              // inputs
  Rows yq, yk;            // forward: outputs; backward: their gradients
  Rows dq, dk;            // backward: gradients of the inputs
  const float *wq, *wk;   // [128] or nullptr
  const int64_t *pos;     // [tokens]
  const double *freq;     // [rot / 2]
  float *dwq, *dwk;       // [128] or nullptr
  float *part;            // backward: [blocks][2][128] partial weight gradients
};

// Columns of the state that a workgroup of the scans takes: 32 halve the
// reads of the operands that its column blocks share, 16 double the
// workgroups of a few heads.  Wide once that gives `least` workgroups.
inline bool scan_wide(const SeqArgs &a, int least) { return (int64_t)a.seqs * a.hv * 4 >= least; }

// dtype: 0 fp32, 1 bf16, 2 fp16
hipError_t launch_seq_recurrent(const SeqArgs &a, int dtype, bool kda, bool delta, hipStream_t stream);
hipError_t launch_seq_chunked(const SeqArgs &a, int dtype, bool kda, bool delta, hipStream_t stream);
hipError_t launch_seq_backward(const SeqArgs &a, int dtype, bool delta, hipStream_t stream);
int64_t norm_blocks(int64_t tokens, int hq, int hk);  // workgroups of the backward pass
hipError_t launch_norm(const NormArgs &a, int in, int out, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs &a, int in, int out, hipStream_t stream);

}  // namespace lq
