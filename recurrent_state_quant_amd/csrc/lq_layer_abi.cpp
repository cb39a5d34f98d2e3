// C ABI of the operators around the recurrence (short convolution, selective
// scan, block norms): argument validation and launches.  Semantics are
// documented in include/leapquant.h.
#include <stdint.h>

#include <type_traits>

#include "leapquant.h"
#include "lq_abi_rows.h"
#include "lq_layer.h"

namespace {

using namespace lq::abi;

constexpr int64_t kMaxChannels = int64_t(1) << 20;
constexpr int64_t kMaxGroups = 65535;
constexpr int64_t kMaxNorm = 8192;  // values of a row of the block norm

// ---- short convolution

int check_conv(const lq_conv *cv, bool step) {
  if (!cv) return LQ_ERR_NULL;
  if (cv->width < 2 || cv->width > 4) return LQ_ERR_UNSUPPORTED;
  if (cv->tokens < 0 || cv->tokens > kMaxTokens || cv->channels < 1 || cv->channels > kMaxChannels) return LQ_ERR_SHAPE;
  if (!step && cv->seqs < 1) return LQ_ERR_SHAPE;
  if (cv->activation != LQ_ACT_NONE && cv->activation != LQ_ACT_SILU) return LQ_ERR_SHAPE;
  if (!dtype_ok(cv->dtype)) return LQ_ERR_SHAPE;
  // four waves a workgroup; a wave takes at least 64 channels of 32 tokens, of one row or of one sequence
  const int64_t tiles = (cv->channels + 63) / 64, runs = step ? cv->tokens : (cv->tokens + 31) / 32 + cv->seqs;
  if (runs > kMaxGrid / tiles) return LQ_ERR_SHAPE;
  return LQ_OK;
}

int conv_weights(const lq_conv *cv, Blocks *bl, lq::ConvArgs *a) {
  if (!cv->weight) return LQ_ERR_NULL;
  if (!aligned(cv->weight, 4) || !aligned(cv->bias, 4)) return LQ_ERR_ALIGN;
  bl->add_in(dense(cv->weight, int64_t(cv->channels) * cv->width * 4));
  bl->add_in(dense(cv->bias, int64_t(cv->channels) * 4));
  a->tokens = cv->tokens;
  a->seqs = cv->seqs;
  a->channels = cv->channels;
  a->width = cv->width;
  a->silu = cv->activation == LQ_ACT_SILU;
  a->w = cv->weight;
  a->bias = cv->bias;
  return LQ_OK;
}

// [tokens][channels]
int check_channels(const lq_rows *r, int64_t tokens, int64_t channels, int64_t size, bool out, Block *b, lq::Rows *to) {
  return check_rows(r, tokens, 1, channels, size, out, b, to, size);
}

bool wide_rows(const lq::Rows &r, int64_t size) {
  return aligned(r.ptr, 16) && r.ts * size % 16 == 0;
}
bool wide_channels(int64_t channels, int64_t size) { return channels * size % 16 == 0; }

int64_t conv_space(const lq_conv *cv, int64_t blocks) { return blocks * (cv->width + 1) * cv->channels * 4; }

// ---- selective scan

int check_scan(const lq_scan *sc, bool step) {
  if (!sc) return LQ_ERR_NULL;
  if (sc->states != 8 && sc->states != 16 && sc->states != 32) return LQ_ERR_UNSUPPORTED;
  if (sc->tokens < 0 || sc->tokens > kMaxTokens || sc->channels < 1 || sc->channels > kMaxChannels || sc->groups < 1 ||
      sc->groups > kMaxGroups || sc->channels % sc->groups)
    return LQ_ERR_SHAPE;
  if (!step && sc->seqs < 1) return LQ_ERR_SHAPE;
  if (sc->flags & ~static_cast<uint32_t>(LQ_SCAN_SOFTPLUS)) return LQ_ERR_SHAPE;
  if (!dtype_ok(sc->dtype)) return LQ_ERR_SHAPE;
  if (step) {
    const int64_t blocks = (int64_t(sc->channels) * (sc->states / 4) + 255) / 256;
    return sc->tokens > kMaxGrid / blocks ? LQ_ERR_SHAPE : LQ_OK;
  }
  // the grids: chunks (at least one a sequence, four waves a workgroup), the
  // states of all sequences, and the gradient's sums of B and C
  const int64_t tiles = lq::scan_tiles(sc->channels, sc->groups);
  const int64_t slots = lq::scan_most_slots(sc->tokens, sc->seqs, sc->channels, sc->groups, sc->states, true);
  if (slots > kMaxGrid / ((tiles + 3) / 4)) return LQ_ERR_SHAPE;
  if (sc->seqs > kMaxGrid / ((int64_t(sc->channels) * sc->states + 255) / 256)) return LQ_ERR_SHAPE;
  if (sc->tokens > (kMaxGrid * 256) / (int64_t(sc->groups) * 2 * sc->states)) return LQ_ERR_SHAPE;
  return LQ_OK;
}

// The arrays of the workspace, one behind another from `base`; returns the
// bytes they take: room for the most slots, of the shortest chunks, so that more
// tokens or sequences never need less.  (Training 8,192 tokens x 2,048 channels x 16
// states in four sequences: states kept 269 MB, carried 68, steps' sums 4, shares of
// dB and dC 34, of dA, dD and dbias, of the gradient's whole chunks, 38.)
int64_t scan_space(const lq_scan *sc, bool save, char *base, lq::ScanArgs *a) {
  const int64_t channels = sc->channels, state = channels * sc->states * 4;
  const int64_t slots = lq::scan_most_slots(sc->tokens, sc->seqs, sc->channels, sc->groups, sc->states, save);
  int64_t used = 0;
  const auto take = [&](auto **p, int64_t bytes) {
    if (base) *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + used);
    used += (bytes + 15) / 16 * 16;
  };
  if (!save && sc->tokens <= lq::kScanLeast) return 0;  // no sequence has two chunks
  if (save) take(&a->check, lq::scan_checks(sc->tokens, sc->seqs) * state);
  take(&a->carry, slots * state);
  take(&a->sum, slots * channels * 4);
  if (save) {
    take(&a->part_bc, lq::scan_tiles(sc->channels, sc->groups) * sc->tokens * 2 * sc->states * 4);
    const int64_t chunks = lq::scan_most_chunks(sc->tokens, sc->seqs, sc->channels, sc->groups, sc->states);
    take(&a->part_a, chunks * (sc->states + 2) * channels * 4);
  }
  return used;
}
int64_t scan_need(const lq_scan *sc, bool save) {
  lq::ScanArgs none{};
  return scan_space(sc, save, nullptr, &none);
}

int scan_weights(const lq_scan *sc, Blocks *bl, lq::ScanArgs *a) {
  if (!sc->A) return LQ_ERR_NULL;
  if (!aligned(sc->A, 16) || !aligned(sc->D, 4) || !aligned(sc->dt_bias, 4)) return LQ_ERR_ALIGN;
  const int64_t channels = sc->channels;
  bl->add_in(dense(sc->A, channels * sc->states * 4));
  bl->add_in(dense(sc->D, channels * 4));
  bl->add_in(dense(sc->dt_bias, channels * 4));
  a->tokens = sc->tokens;
  a->seqs = sc->seqs;
  a->channels = sc->channels;
  a->groups = sc->groups;
  a->per = sc->channels / sc->groups;
  a->softplus = (sc->flags & LQ_SCAN_SOFTPLUS) != 0;
  a->A = sc->A;
  a->skip = sc->D;
  a->bias = sc->dt_bias;
  return LQ_OK;
}

// x, dt, B, C and z (which may be NULL)
int scan_inputs(const lq_scan *sc, const lq_rows *x, const lq_rows *dt, const lq_rows *B, const lq_rows *C,
                const lq_rows *z, Blocks *bl, lq::ScanArgs *a) {
  const int64_t T = sc->tokens, size = dtype_size(sc->dtype);
  Block b;
  int rc;
  if ((rc = check_channels(x, T, sc->channels, size, false, &b, &a->x))) return rc;
  bl->add_in(b);
  if ((rc = check_channels(dt, T, sc->channels, size, false, &b, &a->dt))) return rc;
  bl->add_in(b);
  if ((rc = check_rows(B, T, sc->groups, sc->states, size, false, &b, &a->B))) return rc;
  bl->add_in(b);
  if ((rc = check_rows(C, T, sc->groups, sc->states, size, false, &b, &a->C))) return rc;
  bl->add_in(b);
  if (z) {
    if ((rc = check_channels(z, T, sc->channels, size, false, &b, &a->z))) return rc;
    bl->add_in(b);
  }
  return LQ_OK;
}

// Offsets, chunks and workspace of the calls over sequences
int scan_chunks(const lq_scan *sc, const int32_t *cu, void *ws, int64_t ws_bytes, bool save, bool back, Blocks *bl,
                lq::ScanArgs *a) {
  if (!cu) return LQ_ERR_NULL;
  if (!aligned(cu, 4)) return LQ_ERR_ALIGN;
  bl->add_in(dense(cu, (int64_t(sc->seqs) + 1) * 4));
  a->cu = cu;
  a->chunk = (back ? lq::scan_grad_chunk : lq::scan_forward_chunk)(sc->tokens, sc->seqs, sc->channels, sc->groups,
                                                                  sc->states);
  a->part = back ? lq::scan_grad_part(a->chunk) : a->chunk;
  a->slots = lq::scan_slots(sc->tokens, sc->seqs, a->chunk);
  const int64_t need = scan_need(sc, save);
  if (need) {
    if (!ws) return LQ_ERR_NULL;
    if (!aligned(ws, 16)) return LQ_ERR_ALIGN;
    if (ws_bytes < need) return LQ_ERR_SHAPE;
    bl->add_out(dense(ws, need));
    scan_space(sc, save, static_cast<char *>(ws), a);
  }
  return LQ_OK;
}

// ---- block norm

int check_norm(const lq_block_norm *bn) {
  if (!bn) return LQ_ERR_NULL;
  if (bn->tokens < 0 || bn->tokens > kMaxTokens || bn->heads < 1 || bn->heads > kMaxGroups) return LQ_ERR_SHAPE;
  if (bn->dim < 8 || bn->dim > kMaxNorm || bn->dim % 8) return LQ_ERR_SHAPE;
  if (!dtype_ok(bn->dtype) || !dtype_ok(bn->dtype_stream)) return LQ_ERR_SHAPE;
  if (bn->dtype_stream != LQ_F32 && bn->dtype_stream != bn->dtype) return LQ_ERR_UNSUPPORTED;
  if (bn->gate != LQ_ACT_NONE && bn->gate != LQ_ACT_SILU && bn->gate != LQ_ACT_SIGMOID) return LQ_ERR_SHAPE;
  if (bn->out_norm != 0 && bn->out_norm != 1) return LQ_ERR_SHAPE;
  if (!(bn->eps > 0.f)) return LQ_ERR_SHAPE;
  if (!aligned(bn->out_weight, 16) || !aligned(bn->in_weight, 16)) return LQ_ERR_ALIGN;
  // sixteen rows a workgroup up to 128 values, four up to 1,024, one beyond
  const int64_t per = bn->dim <= 128 ? 16 : bn->dim <= 1024 ? 4 : 1;
  if (bn->tokens * bn->heads > kMaxGrid * per) return LQ_ERR_SHAPE;
  return LQ_OK;
}

int norm_inputs(const lq_block_norm *bn, const lq_rows *a, const lq_rows *z, const lq_rows *res, bool in_norm, Block *ba,
                Block *br, Blocks *bl, lq::BlockNormArgs *n) {
  const int64_t T = bn->tokens, size = dtype_size(bn->dtype), wide = dtype_size(bn->dtype_stream);
  Block b;
  int rc;
  if ((rc = check_rows(a, T, bn->heads, bn->dim, size, false, ba, &n->a))) return rc;
  if (bn->gate != LQ_ACT_NONE) {
    if ((rc = check_rows(z, T, bn->heads, bn->dim, size, false, &b, &n->z))) return rc;
    bl->add_in(b);
  } else if (z) {
    return LQ_ERR_SHAPE;
  }
  *br = Block{};
  if (res && (rc = check_rows(res, T, bn->heads, bn->dim, wide, false, br, &n->res))) return rc;
  if (bn->out_norm) bl->add_in(dense(bn->out_weight, int64_t(bn->dim) * 4));
  if (in_norm) bl->add_in(dense(bn->in_weight, int64_t(bn->dim) * 4));
  n->tokens = T;
  n->heads = bn->heads;
  n->dim = bn->dim;
  n->gate = bn->gate;
  n->out_norm = bn->out_norm;
  n->eps = bn->eps;
  n->scale = bn->scale;
  n->wo = bn->out_weight;
  n->wi = bn->in_weight;
  return LQ_OK;
}

bool same(const lq::Rows &a, const lq::Rows &b) { return a.ptr == b.ptr && a.ts == b.ts && a.hs == b.hs; }

}  // namespace

extern "C" {

int leapquant_conv_forward(const lq_conv *cv, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *y,
                           const void *X0, void *X, hipStream_t stream) {
  int rc = check_conv(cv, false);
  if (rc) return rc;
  Blocks bl;
  lq::ConvArgs a{};
  if ((rc = conv_weights(cv, &bl, &a))) return rc;
  if (!cu_seqlens) return LQ_ERR_NULL;
  if (!aligned(cu_seqlens, 4)) return LQ_ERR_ALIGN;
  bl.add_in(dense(cu_seqlens, (int64_t(cv->seqs) + 1) * 4));
  const int64_t size = dtype_size(cv->dtype), state = int64_t(cv->seqs) * (cv->width - 1) * cv->channels * size;
  Block b;
  if ((rc = check_channels(x, cv->tokens, cv->channels, size, false, &b, &a.x))) return rc;
  bl.add_in(b);
  if ((rc = check_channels(y, cv->tokens, cv->channels, size, true, &b, &a.y))) return rc;
  bl.add_out(b);
  if (!aligned(X0, size) || !aligned(X, size)) return LQ_ERR_ALIGN;
  bl.add_in(dense(X0, state));
  bl.add_out(dense(X, state));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.cu = cu_seqlens;
  a.X0 = X0;
  a.X = X;
  const bool wide = wide_channels(cv->channels, size) && wide_rows(a.x, size) && wide_rows(a.y, size) && aligned(X0, 16) &&
                    aligned(X, 16);
  return hip_status(lq::launch_conv(a, cv->dtype, wide, stream));
}

int leapquant_conv_step(const lq_conv *cv, const int32_t *slots, int32_t n_slots, const lq_rows *x, const lq_rows *y,
                        const void *X0, void *X, hipStream_t stream) {
  int rc = check_conv(cv, true);
  if (rc) return rc;
  if (n_slots < 1 || (!slots && cv->tokens > n_slots)) return LQ_ERR_SHAPE;
  if (!aligned(slots, 4)) return LQ_ERR_ALIGN;
  Blocks bl;
  lq::ConvArgs a{};
  if ((rc = conv_weights(cv, &bl, &a))) return rc;
  if (!X0 || !X) return LQ_ERR_NULL;
  bl.add_in(dense(slots, cv->tokens * 4));
  const int64_t size = dtype_size(cv->dtype), state = int64_t(n_slots) * (cv->width - 1) * cv->channels * size;
  Block b;
  if ((rc = check_channels(x, cv->tokens, cv->channels, size, false, &b, &a.x))) return rc;
  bl.add_in(b);
  if ((rc = check_channels(y, cv->tokens, cv->channels, size, true, &b, &a.y))) return rc;
  bl.add_out(b);
  if (!aligned(X0, size) || !aligned(X, size)) return LQ_ERR_ALIGN;
  if (X0 != X) bl.add_in(dense(X0, state));
  bl.add_out(dense(X, state));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.X0 = X0;
  a.X = X;
  a.slots = slots;
  a.n_slots = n_slots;
  const bool wide = wide_channels(cv->channels, size) && wide_rows(a.x, size) && wide_rows(a.y, size) && aligned(X0, 16) &&
                    aligned(X, 16);
  return hip_status(lq::launch_conv_step(a, cv->dtype, wide, stream));
}

int64_t leapquant_conv_workspace(const lq_conv *cv) {
  const int rc = check_conv(cv, false);
  return rc ? rc : conv_space(cv, lq::conv_grad_most(cv->tokens));
}

int leapquant_conv_backward(const lq_conv *cv, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *dy,
                            const lq_rows *dx, const void *X0, const void *dX, void *dX0, float *dweight, float *dbias,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_conv(cv, false);
  if (rc) return rc;
  Blocks bl;
  lq::ConvArgs a{};
  if ((rc = conv_weights(cv, &bl, &a))) return rc;
  if (!cu_seqlens) return LQ_ERR_NULL;
  if (!aligned(cu_seqlens, 4)) return LQ_ERR_ALIGN;
  bl.add_in(dense(cu_seqlens, (int64_t(cv->seqs) + 1) * 4));
  const int64_t size = dtype_size(cv->dtype), state = int64_t(cv->seqs) * (cv->width - 1) * cv->channels * size;
  Block b;
  if ((rc = check_channels(x, cv->tokens, cv->channels, size, false, &b, &a.x))) return rc;
  bl.add_in(b);
  if ((rc = check_channels(dy, cv->tokens, cv->channels, size, false, &b, &a.dy))) return rc;
  bl.add_in(b);
  if ((rc = check_channels(dx, cv->tokens, cv->channels, size, true, &b, &a.dx))) return rc;
  bl.add_out(b);
  if (!aligned(X0, size) || !aligned(dX, size) || !aligned(dX0, size) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return LQ_ERR_ALIGN;
  bl.add_in(dense(X0, state));
  bl.add_in(dense(dX, state));
  bl.add_out(dense(dX0, state));
  bl.add_out(dense(dweight, int64_t(cv->channels) * cv->width * 4));
  bl.add_out(dense(dbias, int64_t(cv->channels) * 4));
  if (dweight || dbias) {
    const int64_t need = conv_space(cv, lq::conv_grad_blocks(cv->tokens, lq::conv_grad_run(cv->tokens, cv->channels)));
    if (need) {
      if (!workspace) return LQ_ERR_NULL;
      if (!aligned(workspace, 16)) return LQ_ERR_ALIGN;
      if (workspace_bytes < need) return LQ_ERR_SHAPE;
      bl.add_out(dense(workspace, need));
    }
    a.part = static_cast<float *>(workspace);
  }
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.cu = cu_seqlens;
  a.X0 = X0;
  a.dX = dX;
  a.dX0 = dX0;
  a.dw = dweight;
  a.dbias = dbias;
  const bool wide = wide_channels(cv->channels, size) && wide_rows(a.x, size) && wide_rows(a.dy, size) &&
                    wide_rows(a.dx, size) && aligned(X0, 16) && aligned(dX, 16) && aligned(dX0, 16);
  return hip_status(lq::launch_conv_backward(a, cv->dtype, wide, stream));
}

int64_t leapquant_scan_workspace(const lq_scan *sc, int32_t save) {
  const int rc = check_scan(sc, false);
  if (rc) return rc;
  return scan_need(sc, save != 0);
}

int leapquant_scan_forward(const lq_scan *sc, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *dt,
                           const lq_rows *B, const lq_rows *C, const lq_rows *z, const lq_rows *y, const float *S0,
                           float *S, void *workspace, int64_t workspace_bytes, int32_t save, hipStream_t stream) {
  int rc = check_scan(sc, false);
  if (rc) return rc;
  Blocks bl;
  lq::ScanArgs a{};
  if ((rc = scan_weights(sc, &bl, &a))) return rc;
  if ((rc = scan_inputs(sc, x, dt, B, C, z, &bl, &a))) return rc;
  if ((rc = scan_chunks(sc, cu_seqlens, workspace, workspace_bytes, save != 0, false, &bl, &a))) return rc;
  Block b;
  if ((rc = check_channels(y, sc->tokens, sc->channels, dtype_size(sc->dtype), true, &b, &a.y))) return rc;
  bl.add_out(b);
  if (!aligned(S0, 16) || !aligned(S, 16)) return LQ_ERR_ALIGN;
  const int64_t states = int64_t(sc->seqs) * sc->channels * sc->states * 4;
  if (S0 != S) bl.add_in(dense(S0, states));
  bl.add_out(dense(S, states));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.S0 = S0;
  a.S = S;
  return hip_status(lq::launch_scan(a, sc->dtype, sc->states, stream));
}

int leapquant_scan_step(const lq_scan *sc, const int32_t *slots, int32_t n_slots, const lq_rows *x, const lq_rows *dt,
                        const lq_rows *B, const lq_rows *C, const lq_rows *z, const lq_rows *y, const float *S0, float *S,
                        hipStream_t stream) {
  int rc = check_scan(sc, true);
  if (rc) return rc;
  if (n_slots < 1 || (!slots && sc->tokens > n_slots)) return LQ_ERR_SHAPE;
  if (!aligned(slots, 4)) return LQ_ERR_ALIGN;
  Blocks bl;
  lq::ScanArgs a{};
  if ((rc = scan_weights(sc, &bl, &a))) return rc;
  if ((rc = scan_inputs(sc, x, dt, B, C, z, &bl, &a))) return rc;
  bl.add_in(dense(slots, sc->tokens * 4));
  Block b;
  if ((rc = check_channels(y, sc->tokens, sc->channels, dtype_size(sc->dtype), true, &b, &a.y))) return rc;
  bl.add_out(b);
  if (!S0 || !S) return LQ_ERR_NULL;
  if (!aligned(S0, 16) || !aligned(S, 16)) return LQ_ERR_ALIGN;
  const int64_t states = int64_t(n_slots) * sc->channels * sc->states * 4;
  if (S0 != S) bl.add_in(dense(S0, states));
  bl.add_out(dense(S, states));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.S0 = S0;
  a.S = S;
  a.which = slots;
  a.n_slots = n_slots;
  return hip_status(lq::launch_scan_step(a, sc->dtype, sc->states, stream));
}

int leapquant_scan_backward(const lq_scan *sc, const int32_t *cu_seqlens, const lq_rows *x, const lq_rows *dt,
                            const lq_rows *B, const lq_rows *C, const lq_rows *z, const lq_rows *dy, const lq_rows *dx,
                            const lq_rows *ddt, const lq_rows *dB, const lq_rows *dC, const lq_rows *dz, float *dA,
                            float *dD, float *ddt_bias, const float *dS, float *dS0, void *workspace,
                            int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_scan(sc, false);
  if (rc) return rc;
  Blocks bl;
  lq::ScanArgs a{};
  if ((rc = scan_weights(sc, &bl, &a))) return rc;
  if ((rc = scan_inputs(sc, x, dt, B, C, z, &bl, &a))) return rc;
  if ((rc = scan_chunks(sc, cu_seqlens, workspace, workspace_bytes, true, true, &bl, &a))) return rc;
  if (!dA || (dD && !sc->D) || (ddt_bias && !sc->dt_bias) || (dz && !z)) return LQ_ERR_NULL;
  const int64_t T = sc->tokens, size = dtype_size(sc->dtype), channels = sc->channels;
  Block b;
  if ((rc = check_channels(dy, T, channels, size, false, &b, &a.dy))) return rc;
  bl.add_in(b);
  if ((rc = check_channels(dx, T, channels, size, true, &b, &a.dx))) return rc;
  bl.add_out(b);
  if ((rc = check_channels(ddt, T, channels, size, true, &b, &a.ddt))) return rc;
  bl.add_out(b);
  if ((rc = check_rows(dB, T, sc->groups, sc->states, size, true, &b, &a.dB))) return rc;
  bl.add_out(b);
  if ((rc = check_rows(dC, T, sc->groups, sc->states, size, true, &b, &a.dC))) return rc;
  bl.add_out(b);
  if (z) {
    if ((rc = check_channels(dz, T, channels, size, true, &b, &a.dz))) return rc;
    bl.add_out(b);
  }
  if (!aligned(dA, 16) || !aligned(dD, 4) || !aligned(ddt_bias, 4) || !aligned(dS, 16) || !aligned(dS0, 16))
    return LQ_ERR_ALIGN;
  bl.add_out(dense(dA, channels * sc->states * 4));
  bl.add_out(dense(dD, channels * 4));
  bl.add_out(dense(ddt_bias, channels * 4));
  const int64_t states = int64_t(sc->seqs) * channels * sc->states * 4;
  if (dS != dS0) bl.add_in(dense(dS, states));
  bl.add_out(dense(dS0, states));
  if (bl.clash()) return LQ_ERR_ALIAS;
  a.dA = dA;
  a.dskip = dD;
  a.dbias = ddt_bias;
  a.dS = dS;
  a.dS0 = dS0;
  return hip_status(lq::launch_scan_backward(a, sc->dtype, sc->states, stream));
}

int leapquant_block_norm(const lq_block_norm *bn, const lq_rows *a, const lq_rows *z, const lq_rows *res, const lq_rows *h,
                         const lq_rows *y, hipStream_t stream) {
  int rc = check_norm(bn);
  if (rc) return rc;
  if (!h && !y) return LQ_ERR_NULL;
  Blocks bl;
  lq::BlockNormArgs n{};
  Block ba, br, b;
  if ((rc = norm_inputs(bn, a, z, res, y != nullptr, &ba, &br, &bl, &n))) return rc;
  const int64_t T = bn->tokens;
  if (h) {
    if ((rc = check_rows(h, T, bn->heads, bn->dim, dtype_size(bn->dtype_stream), true, &b, &n.h))) return rc;
    bl.add_out(b);
  }
  if (y) {
    if ((rc = check_rows(y, T, bn->heads, bn->dim, dtype_size(bn->dtype), true, &b, &n.y))) return rc;
    bl.add_out(b);
  }
  // an output over an input of its type: a lane reads its values before it writes them
  const bool typed = bn->dtype == bn->dtype_stream;
  if (!(y && same(n.a, n.y)) && !(h && typed && same(n.a, n.h))) bl.add_in(ba);
  if (res && !(h && same(n.res, n.h)) && !(y && typed && same(n.res, n.y))) bl.add_in(br);
  if (bl.clash()) return LQ_ERR_ALIAS;
  if (T == 0) return LQ_OK;
  return hip_status(lq::launch_block_norm(n, bn->dtype, bn->dtype_stream, stream));
}

int64_t leapquant_block_norm_workspace(int64_t tokens, int32_t heads, int32_t dim) {
  if (tokens < 0 || tokens > kMaxTokens || heads < 1 || heads > kMaxGroups || dim < 8 || dim > kMaxNorm || dim % 8)
    return LQ_ERR_SHAPE;
  return lq::block_norm_blocks(tokens * heads, dim) * 2 * dim * 4;
}

int leapquant_block_norm_backward(const lq_block_norm *bn, const lq_rows *a, const lq_rows *z, const lq_rows *res,
                                  const lq_rows *dh, const lq_rows *dy, const lq_rows *da, const lq_rows *dz,
                                  const lq_rows *dres, float *dout_weight, float *din_weight, void *workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_norm(bn);
  if (rc) return rc;
  if (!dh && !dy) return LQ_ERR_NULL;
  if ((dres && !res) || (din_weight && !dy)) return LQ_ERR_NULL;
  if (dout_weight && !bn->out_norm) return LQ_ERR_SHAPE;
  Blocks bl;
  lq::BlockNormArgs n{};
  Block ba, br, bh, b;
  if ((rc = norm_inputs(bn, a, z, res, dy != nullptr, &ba, &br, &bl, &n))) return rc;
  bl.add_in(ba);
  bl.add_in(br);
  const int64_t T = bn->tokens, size = dtype_size(bn->dtype), wide = dtype_size(bn->dtype_stream);
  bh = Block{};
  if (dh && (rc = check_rows(dh, T, bn->heads, bn->dim, wide, false, &bh, &n.dh))) return rc;
  if (dy) {
    if ((rc = check_rows(dy, T, bn->heads, bn->dim, size, false, &b, &n.dy))) return rc;
    bl.add_in(b);
  }
  if ((rc = check_rows(da, T, bn->heads, bn->dim, size, true, &b, &n.da))) return rc;
  bl.add_out(b);
  if (bn->gate != LQ_ACT_NONE) {
    if ((rc = check_rows(dz, T, bn->heads, bn->dim, size, true, &b, &n.dz))) return rc;
    bl.add_out(b);
  } else if (dz) {
    return LQ_ERR_SHAPE;
  }
  if (dres) {
    if ((rc = check_rows(dres, T, bn->heads, bn->dim, wide, true, &b, &n.dres))) return rc;
    bl.add_out(b);
  }
  // the stream's gradient in place
  if (!(dh && dres && same(n.dh, n.dres))) bl.add_in(bh);
  if (!aligned(dout_weight, 4) || !aligned(din_weight, 4)) return LQ_ERR_ALIGN;
  bl.add_out(dense(dout_weight, int64_t(bn->dim) * 4));
  bl.add_out(dense(din_weight, int64_t(bn->dim) * 4));
  if (dout_weight || din_weight) {
    const int64_t need = leapquant_block_norm_workspace(T, bn->heads, bn->dim);
    if (need) {
      if (!workspace) return LQ_ERR_NULL;
      if (!aligned(workspace, 16)) return LQ_ERR_ALIGN;
      if (workspace_bytes < need) return LQ_ERR_SHAPE;
      bl.add_out(dense(workspace, need));
    }
    n.part = static_cast<float *>(workspace);
  }
  if (bl.clash()) return LQ_ERR_ALIAS;
  n.dwo = dout_weight;
  n.dwi = din_weight;
  if (T == 0 && !dout_weight && !din_weight) return LQ_OK;
  return hip_status(lq::launch_block_norm_backward(n, bn->dtype, bn->dtype_stream, stream));
}

}  // extern "C"
