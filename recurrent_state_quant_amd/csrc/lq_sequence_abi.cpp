// C ABI of the sequence operators (whole sequences, head norm): argument
// validation and launches.  Semantics are documented in include/leapquant.h.
#include <stdint.h>

#include <type_traits>

#include "leapquant.h"
#include "lq_abi_rows.h"
#include "lq_sequence.h"

namespace {

using namespace lq::abi;

constexpr int64_t kDim = 128, kState = kDim * kDim;
constexpr int64_t kMaxHeads = 65535;            // second grid dimension

// Sequences of few tokens on average run token by token in one launch, longer
// ones in chunks (lq_sequence.hip).  Measured where the two meet, in tokens a
// sequence: with operands of one or two parts at 22 (8 sequences x 32 heads),
// 28 (64 x 32) and 30 (1 x 32); with three parts (fp32, or a decay a channel)
// at 22 .. 34 for up to 32 states and at 52 .. 64 from 256 states on, where
// the chunks' operands outweigh the states.  The average decides, as the lengths
// are on the device: a long sequence among many short ones goes token by token
// too, 1.1 us a token with 8,192 states (4,096 tokens beside 255 of one, x 32
// heads, 4,466 us; the two parts in a call each, 372).
constexpr int64_t kShort = 24, kShortParts = 56, kManyStates = 256;

int64_t slots_of(int64_t tokens, int64_t seqs) { return tokens / lq::kChunk + seqs; }

int check_sequence(const lq_sequence *sq) {
  if (!sq) return LQ_ERR_NULL;
  if (sq->dk != kDim || sq->dv != kDim) return LQ_ERR_UNSUPPORTED;
  if (sq->tokens < 0 || sq->tokens > kMaxTokens || sq->seqs < 1 || sq->heads_k < 1 || sq->heads_v < 1 ||
      sq->heads_v > kMaxHeads || sq->heads_v % sq->heads_k)
    return LQ_ERR_SHAPE;
  if (sq->gate != LQ_GATE_GDN && sq->gate != LQ_GATE_KDA) return LQ_ERR_SHAPE;
  if (sq->flags & ~static_cast<uint32_t>(LQ_NO_DELTA)) return LQ_ERR_SHAPE;
  if (!dtype_ok(sq->dtype)) return LQ_ERR_SHAPE;
  // a launch has up to 8 workgroups for each state, or one for each chunk
  if (int64_t(sq->seqs) * sq->heads_v > kMaxGrid / 8 - 8 || slots_of(sq->tokens, sq->seqs) > kMaxGrid)
    return LQ_ERR_SHAPE;
  return LQ_OK;
}

bool chunked(const lq_sequence *sq, bool save) {
  const bool three = sq->gate == LQ_GATE_KDA || sq->dtype == LQ_F32;
  const bool many = int64_t(sq->seqs) * sq->heads_v >= kManyStates;
  return sq->tokens > 0 && (save || sq->tokens > (three && many ? kShortParts : kShort) * sq->seqs);
}

// The arrays of lq::SeqSpace, one behind another from `base`; returns the
// bytes they take (the sizes alone with base = nullptr).
int64_t space(const lq_sequence *sq, int64_t slots, bool save, char *base, lq::SeqSpace *w) {
  const bool kda = sq->gate == LQ_GATE_KDA;  // K and Q with decays: per value head, as fp32 values
  const int64_t hv = slots * sq->heads_v, hk = kda ? hv : slots * sq->heads_k;
  const int64_t parts = kda || sq->dtype == LQ_F32 ? 3 : sq->dtype == LQ_F16 ? 2 : 1;
  const int64_t square = lq::kChunk * lq::kChunk * 3 * 2, heads = lq::kChunk * kDim * parts * 2;
  const int64_t rows = lq::kChunk * kDim * 4, state = kDim * kDim * 4;
  int64_t used = 0;
  const auto take = [&](auto **p, int64_t bytes) {
    if (base) *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + used);
    used += bytes;
  };
  take(&w->T, hv * square);
  take(&w->P, hv * square);
  take(&w->K, hk * heads);
  take(&w->Q, hk * heads);
  take(&w->KT, hk * heads);
  take(&w->dec, hv * 2 * lq::kChunk * 4);
  if (save) {
    take(&w->TT, hv * square);
    take(&w->PT, hv * square);
    take(&w->QT, hk * heads);
    take(&w->U, hv * rows);
    take(&w->S, hv * state);
    take(&w->X, hv * rows);
    take(&w->G, hv * state);
  }
  return used;
}

int64_t space_bytes(const lq_sequence *sq, int64_t slots, bool save) {
  lq::SeqSpace none{};
  return space(sq, slots, save, nullptr, &none);
}

// What forward and backward check alike: cu_seqlens, q, k, beta, alpha and
// the workspace.
int check_common(const lq_sequence *sq, const int32_t *cu, const lq_rows *q, const lq_rows *k, const lq_rows *beta,
                 const lq_rows *alpha, void *ws, int64_t ws_bytes, bool save, Blocks *bl, lq::SeqArgs *a) {
  if (!cu) return LQ_ERR_NULL;
  if (!aligned(cu, 4)) return LQ_ERR_ALIGN;
  const int64_t T = sq->tokens, size = dtype_size(sq->dtype);
  const bool kda = sq->gate == LQ_GATE_KDA;
  Block b;
  int rc;
  bl->add_in(dense(cu, (int64_t(sq->seqs) + 1) * 4));
  if ((rc = check_rows(q, T, sq->heads_k, kDim, size, false, &b, &a->q))) return rc;
  bl->add_in(b);
  if ((rc = check_rows(k, T, sq->heads_k, kDim, size, false, &b, &a->k))) return rc;
  bl->add_in(b);
  if ((rc = check_rows(beta, T, sq->heads_v, 1, 4, false, &b, &a->beta))) return rc;
  bl->add_in(b);
  if ((rc = check_rows(alpha, T, sq->heads_v, kda ? kDim : 1, 4, false, &b, &a->alpha))) return rc;
  bl->add_in(b);
  const int64_t slots = slots_of(T, sq->seqs);
  const int64_t need = chunked(sq, save) ? space_bytes(sq, slots, save) : 0;
  if (need) {
    if (!ws) return LQ_ERR_NULL;
    if (!aligned(ws, 16)) return LQ_ERR_ALIGN;
    if (ws_bytes < need) return LQ_ERR_SHAPE;
    bl->add_out(dense(ws, need));
    space(sq, slots, save, static_cast<char *>(ws), &a->w);
  }
  a->tokens = T;
  a->slots = slots;
  a->seqs = sq->seqs;
  a->hk = sq->heads_k;
  a->hv = sq->heads_v;
  a->group = sq->heads_v / sq->heads_k;
  a->cu = cu;
  return LQ_OK;
}

int check_norm(const lq_head_norm *nm) {
  if (!nm) return LQ_ERR_NULL;
  if (nm->dim != kDim) return LQ_ERR_UNSUPPORTED;
  if (nm->tokens < 0 || nm->tokens > kMaxTokens || nm->heads_q < 0 || nm->heads_k < 0 || nm->heads_q > kMaxHeads ||
      nm->heads_k > kMaxHeads || nm->heads_q + nm->heads_k < 1)
    return LQ_ERR_SHAPE;
  if (nm->kind != LQ_NORM_L2 && nm->kind != LQ_NORM_RMS) return LQ_ERR_SHAPE;
  if (!dtype_ok(nm->dtype) || !dtype_ok(nm->dtype_out)) return LQ_ERR_SHAPE;
  if (nm->rot < 0 || nm->rot > kDim || nm->rot % 16 || (nm->interleaved != 0 && nm->interleaved != 1))
    return LQ_ERR_SHAPE;
  if (!(nm->eps > 0.f)) return LQ_ERR_SHAPE;
  if (nm->rot > 0 && nm->tokens > 0) {
    if (!nm->positions || !nm->inv_freq) return LQ_ERR_NULL;
    if (!aligned(nm->positions, 8) || !aligned(nm->inv_freq, 8)) return LQ_ERR_ALIGN;
  }
  if (!aligned(nm->q_weight, 16) || !aligned(nm->k_weight, 16)) return LQ_ERR_ALIGN;
  // four runs of sixteen heads a workgroup
  if (nm->tokens * ((nm->heads_q + nm->heads_k + 15) / 16) > kMaxGrid * 4) return LQ_ERR_SHAPE;
  return LQ_OK;
}

lq::NormArgs norm_args(const lq_head_norm *nm, Blocks *bl) {
  lq::NormArgs a{};
  a.tokens = nm->tokens;
  a.hq = nm->heads_q;
  a.hk = nm->heads_k;
  a.rms = nm->kind == LQ_NORM_RMS;
  a.interleaved = nm->interleaved;
  a.rot = nm->tokens > 0 ? nm->rot : 0;
  a.eps = nm->eps;
  a.q_scale = nm->q_scale;
  a.wq = nm->q_weight;
  a.wk = nm->k_weight;
  a.pos = nm->positions;
  a.freq = nm->inv_freq;
  bl->add_in(dense(a.wq, kDim * 4));
  bl->add_in(dense(a.wk, kDim * 4));
  if (a.rot) {
    bl->add_in(dense(a.pos, nm->tokens * 8));
    bl->add_in(dense(a.freq, nm->rot / 2 * 8));
  }
  return a;
}

bool same_rows(const lq::Rows &a, const lq::Rows &b) { return a.ptr == b.ptr && a.ts == b.ts && a.hs == b.hs; }

}  // namespace

extern "C" {

int64_t leapquant_sequence_workspace(const lq_sequence *sq, int32_t save) {
  const int rc = check_sequence(sq);
  if (rc) return rc;
  if (save && sq->gate == LQ_GATE_KDA) return LQ_ERR_UNSUPPORTED;
  if (save) return sq->tokens ? space_bytes(sq, slots_of(sq->tokens, sq->seqs), true) : 0;
  // the most sequences with which that many tokens are taken in chunks
  const int64_t most = sq->tokens > 0 ? (sq->tokens - 1) / kShort : 0;
  if (most < 1) return 0;
  return space_bytes(sq, slots_of(sq->tokens, most < sq->seqs ? most : sq->seqs), false);
}

int leapquant_sequence_forward(const lq_sequence *sq, const int32_t *cu_seqlens, const lq_rows *q, const lq_rows *k,
                               const lq_rows *v, const lq_rows *beta, const lq_rows *alpha, const lq_rows *o,
                               const float *S0, float *S, void *workspace, int64_t workspace_bytes, int32_t save,
                               hipStream_t stream) {
  int rc = check_sequence(sq);
  if (rc) return rc;
  const bool kda = sq->gate == LQ_GATE_KDA, delta = !(sq->flags & LQ_NO_DELTA);
  if (save && kda) return LQ_ERR_UNSUPPORTED;
  Blocks bl;
  lq::SeqArgs a{};
  if ((rc = check_common(sq, cu_seqlens, q, k, beta, alpha, workspace, workspace_bytes, save != 0, &bl, &a)))
    return rc;
  const int64_t size = dtype_size(sq->dtype), states = int64_t(sq->seqs) * sq->heads_v * kState * 4;
  Block b;
  if ((rc = check_rows(v, sq->tokens, sq->heads_v, kDim, size, false, &b, &a.v))) return rc;
  bl.add_in(b);
  if ((rc = check_rows(o, sq->tokens, sq->heads_v, kDim, size, true, &b, &a.o))) return rc;
  bl.add_out(b);
  if (!aligned(S0, 16) || !aligned(S, 16)) return LQ_ERR_ALIGN;
  if (S0 != S) bl.add_in(dense(S0, states));
  bl.add_out(dense(S, states));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.S0 = S0;
  a.S = S;
  if (!chunked(sq, save != 0)) return hip_status(lq::launch_seq_recurrent(a, sq->dtype, kda, delta, stream));
  return hip_status(lq::launch_seq_chunked(a, sq->dtype, kda, delta, stream));
}

int leapquant_sequence_backward(const lq_sequence *sq, const int32_t *cu_seqlens, const lq_rows *q, const lq_rows *k,
                                const lq_rows *beta, const lq_rows *alpha, const lq_rows *go, const float *dS,
                                const lq_rows *dq, const lq_rows *dk, const lq_rows *dv, const lq_rows *dbeta,
                                const lq_rows *dalpha, float *dS0, void *workspace, int64_t workspace_bytes,
                                hipStream_t stream) {
  int rc = check_sequence(sq);
  if (rc) return rc;
  if (sq->gate == LQ_GATE_KDA) return LQ_ERR_UNSUPPORTED;
  Blocks bl;
  lq::SeqArgs a{};
  if ((rc = check_common(sq, cu_seqlens, q, k, beta, alpha, workspace, workspace_bytes, true, &bl, &a))) return rc;
  const int64_t T = sq->tokens, size = dtype_size(sq->dtype), states = int64_t(sq->seqs) * sq->heads_v * kState * 4;
  Block b;
  if ((rc = check_rows(go, T, sq->heads_v, kDim, size, false, &b, &a.go))) return rc;
  bl.add_in(b);
  struct {
    const lq_rows *r;
    int64_t heads, width, size;
    lq::Rows *to;
  } outs[5] = {{dq, sq->heads_k, kDim, size, &a.dq},
               {dk, sq->heads_k, kDim, size, &a.dk},
               {dv, sq->heads_v, kDim, size, &a.dv},
               {dbeta, sq->heads_v, 1, 4, &a.dbeta},
               {dalpha, sq->heads_v, 1, 4, &a.dalpha}};
  for (const auto &x : outs) {
    if ((rc = check_rows(x.r, T, x.heads, x.width, x.size, true, &b, x.to))) return rc;
    bl.add_out(b);
  }
  if (!aligned(dS, 16) || !aligned(dS0, 16)) return LQ_ERR_ALIGN;
  if (dS != dS0) bl.add_in(dense(dS, states));
  bl.add_out(dense(dS0, states));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.dS = dS;
  a.dS0 = dS0;
  return hip_status(lq::launch_seq_backward(a, sq->dtype, !(sq->flags & LQ_NO_DELTA), stream));
}

int leapquant_head_norm(const lq_head_norm *nm, const lq_rows *q, const lq_rows *k, const lq_rows *q_out,
                        const lq_rows *k_out, hipStream_t stream) {
  int rc = check_norm(nm);
  if (rc) return rc;
  Blocks bl;
  lq::NormArgs a = norm_args(nm, &bl);
  const int64_t T = nm->tokens, si = dtype_size(nm->dtype), so = dtype_size(nm->dtype_out);
  Block bq, bk, oq, ok;
  if ((rc = check_rows(q, T, nm->heads_q, kDim, si, false, &bq, &a.q))) return rc;
  if ((rc = check_rows(k, T, nm->heads_k, kDim, si, false, &bk, &a.k))) return rc;
  if ((rc = check_rows(q_out, T, nm->heads_q, kDim, so, true, &oq, &a.yq))) return rc;
  if ((rc = check_rows(k_out, T, nm->heads_k, kDim, so, true, &ok, &a.yk))) return rc;
  // an output over its own input: each head is read whole before it is written
  const bool typed = nm->dtype == nm->dtype_out;
  if (!(typed && same_rows(a.q, a.yq))) bl.add_in(bq);
  if (!(typed && same_rows(a.k, a.yk))) bl.add_in(bk);
  bl.add_out(oq);
  bl.add_out(ok);
  if (bl.clash()) return LQ_ERR_ALIAS;
  if (T == 0) return LQ_OK;
  return hip_status(lq::launch_norm(a, nm->dtype, nm->dtype_out, stream));
}

int64_t leapquant_head_norm_workspace(int64_t tokens, int32_t heads_q, int32_t heads_k) {
  if (tokens < 0 || tokens > kMaxTokens || heads_q < 0 || heads_k < 0 || heads_q > kMaxHeads || heads_k > kMaxHeads ||
      heads_q + heads_k < 1)
    return LQ_ERR_SHAPE;
  return lq::norm_blocks(tokens, heads_q, heads_k) * 2 * kDim * 4;
}

int leapquant_head_norm_backward(const lq_head_norm *nm, const lq_rows *q, const lq_rows *k, const lq_rows *gq,
                                 const lq_rows *gk, const lq_rows *dq, const lq_rows *dk, float *dq_weight,
                                 float *dk_weight, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_norm(nm);
  if (rc) return rc;
  Blocks bl;
  lq::NormArgs a = norm_args(nm, &bl);
  const int64_t T = nm->tokens, si = dtype_size(nm->dtype), so = dtype_size(nm->dtype_out);
  Block b;
  if ((rc = check_rows(q, T, nm->heads_q, kDim, si, false, &b, &a.q))) return rc;
  bl.add_in(b);
  if ((rc = check_rows(k, T, nm->heads_k, kDim, si, false, &b, &a.k))) return rc;
  bl.add_in(b);
  if ((rc = check_rows(gq, T, nm->heads_q, kDim, so, false, &b, &a.yq))) return rc;
  bl.add_in(b);
  if ((rc = check_rows(gk, T, nm->heads_k, kDim, so, false, &b, &a.yk))) return rc;
  bl.add_in(b);
  if ((rc = check_rows(dq, T, nm->heads_q, kDim, si, true, &b, &a.dq))) return rc;
  bl.add_out(b);
  if ((rc = check_rows(dk, T, nm->heads_k, kDim, si, true, &b, &a.dk))) return rc;
  bl.add_out(b);
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return LQ_ERR_ALIGN;
  bl.add_out(dense(dq_weight, kDim * 4));
  bl.add_out(dense(dk_weight, kDim * 4));
  if (dq_weight || dk_weight) {
    const int64_t need = leapquant_head_norm_workspace(T, nm->heads_q, nm->heads_k);
    if (need) {
      if (!workspace) return LQ_ERR_NULL;
      if (!aligned(workspace, 16)) return LQ_ERR_ALIGN;
      if (workspace_bytes < need) return LQ_ERR_SHAPE;
      bl.add_out(dense(workspace, need));
    }
    a.part = static_cast<float *>(workspace);
  }
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  if (T == 0 && !dq_weight && !dk_weight) return LQ_OK;
  return hip_status(lq::launch_norm_backward(a, nm->dtype, nm->dtype_out, stream));
}

}  // extern "C"
