// Backward pass of the gated delta rule over whole sequences (scalar gate,
// gfx950), from what the chunked forward pass kept (T, P, U, the decays and
// the state at every chunk's start).  With dO the outputs' gradient and G
// that of the state at a chunk's end,
//   dU = P^T dO + kappa * (K G),   dX = T^T dU = dV,
//   dS0 = G_C G + Q^T (Gam * dO) - K^T (Gam * dX)           (scan, in reverse)
// and then, in every chunk by itself, with D1 = dO U^T, D2 = -dX U^T,
// E1 = L beta_j D1 (j <= i), E2 = L beta_j D2 (j < i), Z1 = dO S0^T,
// Z2 = dX S0^T, Z3 = U G^T, W = D1 * QK^T + D2 * KK^T:
//   dQ = Gam * Z1 + E1 K
//   dK = -Gam * Z2 + kappa * Z3 + E1^T Q + (E2 + E2^T) K
//   dbeta_j = sum_i L_ij W_ij + L_Cj k_j . Z3_j
//   dL_ij = beta_j W_ij;  dL_i0 = q_i . Z1_i - k_i . Z2_i (state column);
//   dL_Cj += beta_j k_j . Z3_j;  dL_C0 += <G, S0>
//   dalpha_t = sum_{j < t} L_{t-1,j} F_tj,   F_tj = dL_tj + alpha_{t+1} F_{t+1,j}
// The decays' gradient is taken from products of decays, not from a quotient
// by alpha_t: decays of zero have a gradient too.
// Without the delta correction T = I and the terms of dX in K drop out.
#include "lq_sequence_device.h"

namespace lq {

// ---------------------------------------------------------------------------
// Reverse scan: built as the forward scan (lq_sequence.hip): one workgroup of
// eight waves per (sequence, value head, block of CB columns), wave w holding
// rows 16 w .. + 15 of G; private operands in fragments straight from global
// memory, shared ones as bf16 parts through LDS, three barriers a chunk.
// Waves 0 .. 3 take the chain (K G, dU, T^T dU, dX), a token tile each; waves
// 4 .. 7 what does not depend on G: dO's parts and, one chunk ahead, P^T dO.
// ---------------------------------------------------------------------------
template <class E, bool DELTA, int CB>
__global__ __launch_bounds__(512) void seq_rscan_kernel(const SeqArgs A) {
  constexpr int NT = CB / 16, kBlocks = D / CB, NP = Parts<E>::n;
  constexpr int FS = 4 * NT, FX = 2 * NT;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wt = w & 3;
  const bool kwave = w < 4;
  const int64_t b = blockIdx.x;  // column blocks of a head on one XCD, as in the forward scan
  const int64_t unit = (b / (8 * kBlocks)) * 8 + (b & 7);
  if (unit >= (int64_t)A.seqs * A.hv) return;
  const int col0 = (int)((b >> 3) % kBlocks) * CB;
  const int seq = (int)(unit / A.hv), hv = (int)(unit % A.hv), hk = hv / A.group;
  const int start = seq_start(A, seq), end = seq_end(A, seq, start);
  __shared__ __align__(16) uint16_t sh_g[3 * FS * 512];               // G, [column][key row]
  __shared__ __align__(16) uint16_t sh_o[NP * FX * 512];              // dO of the next chunk, [column][token]
  __shared__ __align__(16) uint16_t sh_og[3 * FX * 512];              // Gam * dO
  __shared__ __align__(16) uint16_t sh_du[DELTA ? 3 * FX * 512 : 8];  // dU
  __shared__ __align__(16) uint16_t sh_x[DELTA ? 3 * FX * 512 : 8];   // -Gam * dX
  __shared__ floatx4 sh_pd[4 * NT * 64];                              // P^T dO, as the accumulators hold it
  const int i = lane & 15, g = lane >> 4, tok = 16 * wt + 4 * g;

  floatx4 s[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      s[n][r] = A.dS ? A.dS[(unit * D + 16 * w + 4 * g + r) * D + col0 + 16 * n + i] : 0.f;
  wait_loads();  // the loop below counts its own loads only

  // Loads as in the forward scan: at fixed places in the code, a row past the
  // end replaced by the chunk's first; dO is zero there, and so are its rows
  // of P^T and T^T and its columns of Q^T and K^T.  Pointers move back a chunk.
  bf8 fA[4][NP], fB[2][3], fQT[2][NP], fKT[2][NP];  // K; T^T or P^T
  E raw[NT][4] = {};
  float cur[NT][4], last;
  float4 gam, kap;
  const int slot0 = start / C + seq;
  const int chunks = (end - start + C - 1) / C;
  const int tl = start + (chunks - 1) * C;  // the last chunk's first token
  const E *pO = at<const E>(A.go, tl + tok, hv) + col0 + i;
  const int64_t backO = tok * A.go.ts;
  auto load_A = [&](int c) {
    if (kwave) {
      const size_t atk = (size_t)(slot0 + c) * A.hk + hk;
#pragma unroll
      for (int x = 0; x < 4; ++x) frag_load<NP>(fA[x], A.w.K + ((atk * 4 + wt) * 4 + x) * NP * 512, lane);
    }
  };
  auto load_do = [&](int c, int move) {
    const int len = end - start - c * C;
    if (!kwave) {
      pO -= move * (C * A.go.ts);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const E *p = tok + r < len ? pO + r * A.go.ts : pO - backO;
#pragma unroll
        for (int n = 0; n < NT; ++n) raw[n][r] = p[16 * n];
      }
    }
  };
  auto load_dec = [&](int c) {
    const float *dec = A.w.dec + ((size_t)(slot0 + c) * A.hv + hv) * 2 * C;
    gam = *reinterpret_cast<const float4 *>(dec + tok);
    kap = *reinterpret_cast<const float4 *>(dec + C + tok);
    last = dec[C - 1];
  };
  auto load_B = [&](int ck, int cq) {
    const size_t at_ = (size_t)(slot0 + (kwave ? ck : cq)) * A.hv + hv;
    const uint16_t *base = (kwave ? A.w.TT : A.w.PT) + (at_ * 4 + wt) * 2 * 3 * 512;
    frag_load<3>(fB[0], base + (wt >> 1) * 3 * 512, lane);  // tiles 2 and 3 have one step
    frag_load<3>(fB[1], base + 3 * 512, lane);
  };
  auto load_QK = [&](int c) {
    const size_t atk = (size_t)(slot0 + c) * A.hk + hk;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      frag_load<NP>(fQT[x], A.w.QT + ((atk * 8 + w) * 2 + x) * NP * 512, lane);
      if (DELTA) frag_load<NP>(fKT[x], A.w.KT + ((atk * 8 + w) * 2 + x) * NP * 512, lane);
    }
  };
  // dO of chunk c out of the loaded values: kept, and shared as parts
  auto share_do = [&](int c) {
    const int len = end - start - c * C;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 4; ++r) cur[n][r] = tok + r < len ? to_f(raw[n][r]) : 0.f;
      frag_share<NP, FX>(sh_o, 2 * n + (wt >> 1), wt & 1, lane, cur[n][0], cur[n][1], cur[n][2], cur[n][3]);
    }
  };
  // P^T dO of the chunk whose dO is shared and whose P^T is loaded
  auto product_do = [&]() {
    Acc2 y[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) y[n] = acc2_zero();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= (wt >> 1)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf8 fo[NP];
          frag_get<NP, FX>(fo, sh_o, 2 * n + x, lane);
          mma_parts<3, NP>(y[n], fB[x], fo);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) sh_pd[(wt * NT + n) * 64 + lane] = y[n].sum();
  };
  if (chunks) {
    const int c = chunks - 1, move = c > 0 ? 1 : 0;
    load_do(c, 0);
    load_B(c, c);
    load_A(c);
    load_dec(c);
    load_QK(c);
    if (!kwave) share_do(c);
    lds_barrier();
    if (!kwave) product_do();
    load_do(c - move, move);
    load_B(c, c - move);
  }
  for (int c = chunks - 1; c >= 0; --c) {
    const int t0 = start + c * C, len = end - t0;
    const int next = c > 0 ? c - 1 : 0, after = c > 1 ? c - 2 : 0;  // the two chunks before this one
    const size_t at_ = (size_t)(slot0 + c) * A.hv + hv;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      frag_share<3, FS>(sh_g, 4 * n + (w >> 1), w & 1, lane, s[n][0], s[n][1], s[n][2], s[n][3]);
#pragma unroll
      for (int r = 0; r < 4; ++r) A.w.G[(at_ * D + 16 * w + 4 * g + r) * D + col0 + 16 * n + i] = s[n][r];
    }
    lds_barrier();
    const float gm[4] = {gam.x, gam.y, gam.z, gam.w}, kp[4] = {kap.x, kap.y, kap.z, kap.w};
    const float la = last;
    floatx4 u[NT];
    if (kwave) {
      Acc2 y[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) y[n] = acc2_zero();
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf8 fg[3];
          frag_get<3, FS>(fg, sh_g, 4 * n + x, lane);
          mma_parts<NP, 3>(y[n], fA[x], fg);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const floatx4 pd = sh_pd[(wt * NT + n) * 64 + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) u[n][r] = fmaf(kp[r], y[n].a[r] + y[n].b[r], pd[r]);
        if (DELTA) frag_share<3, FX>(sh_du, 2 * n + (wt >> 1), wt & 1, lane, u[n][0], u[n][1], u[n][2], u[n][3]);
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        frag_share<3, FX>(sh_og, 2 * n + (wt >> 1), wt & 1, lane, gm[0] * cur[n][0], gm[1] * cur[n][1],
                          gm[2] * cur[n][2], gm[3] * cur[n][3]);
      share_do(next);
    }
    load_A(next);
    load_do(after, c > 1 ? 1 : 0);
    load_dec(next);
    lds_barrier();
    if (kwave) {
      if (DELTA) {
        Acc2 z[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) z[n] = acc2_zero();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x >= (wt >> 1)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              bf8 fu[3];
              frag_get<3, FX>(fu, sh_du, 2 * n + x, lane);
              mma_parts<3, 3>(z[n], fB[x], fu);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u[n] = z[n].sum();
          frag_share<3, FX>(sh_x, 2 * n + (wt >> 1), wt & 1, lane, -gm[0] * u[n][0], -gm[1] * u[n][1], -gm[2] * u[n][2],
                            -gm[3] * u[n][3]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          A.w.X[(at_ * C + tok + r) * D + col0 + 16 * n + i] = u[n][r];
          if (tok + r < len) at<E>(A.dv, t0 + tok + r, hv)[col0 + 16 * n + i] = from_f<E>(u[n][r]);
        }
    } else {
      product_do();
    }
    load_B(next, after);
    lds_barrier();
    Acc2 ds[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) ds[n] = acc2_zero();
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        bf8 fo[3], fx[3];
        frag_get<3, FX>(fo, sh_og, 2 * n + x, lane);
        mma_parts<NP, 3>(ds[n], fQT[x], fo);
        if (DELTA) {
          frag_get<3, FX>(fx, sh_x, 2 * n + x, lane);
          mma_parts<NP, 3>(ds[n], fKT[x], fx);
        }
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n] = s[n] * la + ds[n].sum();
    load_QK(next);
  }
  if (A.dS0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) A.dS0[(unit * D + 16 * w + 4 * g + r) * D + col0 + 16 * n + i] = s[n][r];
  }
}

// ---------------------------------------------------------------------------
// Gradients inside a chunk: one workgroup per (slot, key head), the value
// heads that share it in turn, so that dQ and dK are summed over them in a
// fixed order.  Wave w takes one token tile (16 rows).  Products are taken
// transposed (the token is the accumulators' column), so a lane holds four
// neighbouring values of one token's row.  U, S0 and G go through one LDS
// buffer as bf16 parts, 24 KiB at a time; the wave's own rows of Q, K, dO, dX
// and U come straight from global memory, a step ahead.  LDS and registers
// are held to what lets two workgroups share a CU: one loads while the other
// computes (with one, loads and products took turns: 350 us for the training
// step of 8,192 tokens and 16 heads).
// ---------------------------------------------------------------------------
__device__ __forceinline__ Raw8<F32> raw_f32(const float *p) { return raw_load(reinterpret_cast<const F32 *>(p)); }

template <class E, bool DELTA>
__global__ __launch_bounds__(256, 2) void seq_grad_kernel(const SeqArgs A) {
  // parts of E1 and E2: what dQ and dK can hold of them
  constexpr int NP = Parts<E>::n, NE = NP == 3 ? 3 : 2;
  const int slot = blockIdx.x, hk = blockIdx.y;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Chunk ch = find_chunk(A, slot, lane);
  if (ch.len == 0) return;
  __shared__ __align__(16) uint16_t sh_p[24 * 512];  // parts of U, S0 or G
  // two triangles each: E1 with its diagonal below, E2 transposed above; L
  // with its diagonal below, dL transposed above
  __shared__ __align__(16) float sh_e[C * LDC];
  __shared__ __align__(16) float sh_l[C * LDC];
  __shared__ __align__(16) float sh_a[C], sh_be[C], sh_gam[C], sh_kap[C];
  __shared__ __align__(16) float sh_db[4][C];
  __shared__ float sh_dgam[C], sh_kz[C], sh_gs[4], sh_f[4][C], sh_fa[4];
  // the tile's row of 64 x 64 products is the longer the later it is: the
  // two workgroups of a CU give a SIMD's waves opposite tiles
  const int wt = (blockIdx.x & 1) ? 3 - w : w;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  const size_t atk = (size_t)slot * A.hk + hk;

  floatx4 dq[8], dk[8];  // key columns 16 n + 4 g + r of token `row`
#pragma unroll
  for (int n = 0; n < 8; ++n) dq[n] = dk[n] = zero;

  for (int gr = 0; gr < A.group; ++gr) {
    // the lane is opaque in every round: else the addresses and conditions of
    // the whole round are computed ahead and kept, in scratch memory
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int row = 16 * wt + i;  // the lane's token
    const bool in = row < ch.len;
    const int rowc = in ? row : 0;
    const E *const pq = at<const E>(A.q, ch.t0 + rowc, hk), *const pk = at<const E>(A.k, ch.t0 + rowc, hk);
    const int hv = hk * A.group + gr;
    const size_t at_ = (size_t)slot * A.hv + hv;
    const float *U = A.w.U + at_ * C * D, *X = A.w.X + at_ * C * D;
    const float *S0 = A.w.S + at_ * D * D, *G = A.w.G + at_ * D * D;
    const E *go = at<const E>(A.go, ch.t0 + rowc, hv);
    __syncthreads();
    // operands of a step of the products below, loaded a step ahead
    Raw8<E> nq, nk, no;
    Raw8<F32> nx;
    const auto load_step = [&](int x) {
      nq = raw_load(pq + 8 * g + 32 * x);
      no = raw_load(go + 8 * g + 32 * x);
      if (DELTA) {
        nk = raw_load(pk + 8 * g + 32 * x);
        nx = raw_f32(X + row * D + 32 * x + 8 * g);
      }
    };
    load_step(0);
    if (tid < C) {
      const bool on = tid < ch.len;
      sh_a[tid] = on ? *at<const float>(A.alpha, ch.t0 + tid, hv) : 1.f;
      sh_be[tid] = on ? *at<const float>(A.beta, ch.t0 + tid, hv) : 0.f;
      sh_gam[tid] = A.w.dec[at_ * 2 * C + tid];
      sh_kap[tid] = A.w.dec[at_ * 2 * C + C + tid];
    }
    // U's parts, two steps at a time: wave w stores tile w
    Raw8<F32> nu[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) nu[e] = raw_f32(U + (16 * w + i) * D + 32 * e + 8 * g);
    lds_barrier();
    decay_matrix(sh_l, sh_a, w, lane);
    // ---- the 64 x 64 products (rows j of the accumulators, column `row`), lower tiles only
    floatx4 a1[4], a2[4], d1[4], d2[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) a1[n] = a2[n] = d1[n] = d2[n] = zero;
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
      if (!(x & 1)) {
        if (x) lds_barrier();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bf8 f[3];
          raw_parts<F32, 3>(f, nu[e]);
          frag_store<3>(sh_p + (w * 2 + e) * 3 * 512, f, lane);
          nu[e] = raw_f32(U + (16 * w + i) * D + 32 * (e + 2) + 8 * g);
        }
        lds_barrier();
      }
      bf8 fq[NP], fk[NP], fo[NP], fx[3];
      raw_parts<E, NP>(fq, nq);
      raw_parts<E, NP>(fo, no);
      if (DELTA) {
        raw_parts<E, NP>(fk, nk);
        raw_parts<F32, 3>(fx, nx);
      }
      if (x < 3) load_step(x + 1);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (n <= wt) {
          bf8 bk[NP], bu[3];
          const int j = 16 * n + i;
          parts_load<E, NP>(bk, at<const E>(A.k, ch.t0 + (j < ch.len ? j : 0), hk) + 32 * x + 8 * g);
          frag_load<3>(bu, sh_p + (n * 2 + (x & 1)) * 3 * 512, lane);
          mma_into<3, NP>(d1[n], bu, fo);
          if (DELTA) mma_into<3, 3>(d2[n], bu, fx);
          mma_into<NP, NP>(a1[n], bk, fq);
          if (DELTA) mma_into<NP, NP>(a2[n], bk, fk);
        }
      }
    }
    lds_barrier();  // L is whole, U's parts are read
    // S0's first 32 value columns: thread (key row, 16 columns)
    const int srow = tid >> 1, scol = 16 * (tid & 1);
    Raw8<F32> ns[2];
    const auto load_state = [&](const float *p, int x) {
#pragma unroll
      for (int e = 0; e < 2; ++e) ns[e] = raw_f32(p + srow * D + 32 * x + scol + 8 * e);
    };
    load_state(S0, 0);
    no = raw_load(go + 8 * g);
    if (DELTA) nx = raw_f32(X + row * D + 8 * g);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int j0 = 16 * n + 4 * g;
      float db[4] = {0.f, 0.f, 0.f, 0.f};
      if (n <= wt) {
        const float4 b4 = *reinterpret_cast<const float4 *>(sh_be + j0);
        const float4 l4 = *reinterpret_cast<const float4 *>(sh_l + row * LDC + j0);
        const float be[4] = {b4.x, b4.y, b4.z, b4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
        float e1[4], e2[4], dl[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // a token past the end took the first one's rows: nothing of it counts
          const float o = in ? d1[n][r] : 0.f, d = DELTA && in ? -d2[n][r] : 0.f;
          e1[r] = l[r] * be[r] * o;
          e2[r] = l[r] * be[r] * d;
          const float w1 = o * a1[n][r], wv = DELTA ? fmaf(d, a2[n][r], w1) : w1;
          dl[r] = be[r] * wv;
          db[r] = l[r] * wv;
          if (n == wt) {  // the diagonal: E1 alone; behind it: nothing
            const int j = j0 + r;
            db[r] = j < row ? db[r] : (j == row ? w1 : 0.f);
          }
          db[r] = row16_sum(db[r]);
        }
        if (n < wt) {
          *reinterpret_cast<float4 *>(sh_e + row * LDC + j0) = make_float4(e1[0], e1[1], e1[2], e1[3]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sh_e[(j0 + r) * LDC + row] = e2[r];
            sh_l[(j0 + r) * LDC + row] = dl[r];  // no lane reads L there
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = j0 + r, none = row * LDC + C;  // the row's padding, which no one reads
            sh_e[j <= row ? row * LDC + j : none] = e1[r];
            sh_e[j < row ? j * LDC + row : none] = e2[r];
            sh_l[j < row ? j * LDC + row : none] = dl[r];
          }
        }
      }
      if (i == 0) *reinterpret_cast<float4 *>(&sh_db[wt][j0]) = make_float4(db[0], db[1], db[2], db[3]);
    }
    // ---- Z1, Z2 with S0, then Z3 with G, transposed: rows 16 n + 4 g + r are key columns
    const float gam = sh_gam[row], kap = sh_kap[row];
    const int st = (srow >> 4) * 3 * 512, sl = (srow & 15) + 16 * 2 * (tid & 1);
    float dg = 0.f, kz = 0.f;
    {
      floatx4 z1[8], z2[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) z1[n] = z2[n] = zero;
#pragma unroll 1
      for (int x = 0; x < 4; ++x) {
        if (x) lds_barrier();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bf8 f[3];
          raw_parts<F32, 3>(f, ns[e]);
          frag_store<3>(sh_p + st, f, sl + 16 * e);
        }
        if (x < 3) load_state(S0, x + 1); else load_state(G, 0);
        lds_barrier();
        bf8 fo[NP], fx[3];
        raw_parts<E, NP>(fo, no);
        if (DELTA) raw_parts<F32, 3>(fx, nx);
        if (x < 3) {
          no = raw_load(go + 8 * g + 32 * (x + 1));
          if (DELTA) nx = raw_f32(X + row * D + 32 * (x + 1) + 8 * g);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          bf8 bs[3];
          frag_load<3>(bs, sh_p + n * 3 * 512, lane);
          mma_into<3, NP>(z1[n], bs, fo);
          if (DELTA) mma_into<3, 3>(z2[n], bs, fx);
        }
      }
      nu[0] = raw_f32(U + row * D + 8 * g);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float q[4], k[4];
        load4(pq + 16 * n + 4 * g, q);
        load4(pk + 16 * n + 4 * g, k);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dg = fmaf(q[r], z1[n][r], dg);
          dq[n][r] = fmaf(gam, z1[n][r], dq[n][r]);
          if (DELTA) {
            dg = fmaf(-k[r], z2[n][r], dg);
            dk[n][r] = fmaf(-gam, z2[n][r], dk[n][r]);
          }
        }
      }
    }
    float gs = 0.f;
    {
      floatx4 z3[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) z3[n] = zero;
#pragma unroll 1
      for (int x = 0; x < 4; ++x) {
        lds_barrier();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // <G, S0>: S0's values come again, out of the cache
          float xs[8], xg[8];
          load8(reinterpret_cast<const F32 *>(S0 + srow * D + 32 * x + scol + 8 * e), xs);
          const float4 u0 = __builtin_bit_cast(float4, ns[e].v[0]), u1 = __builtin_bit_cast(float4, ns[e].v[1]);
          xg[0] = u0.x; xg[1] = u0.y; xg[2] = u0.z; xg[3] = u0.w;
          xg[4] = u1.x; xg[5] = u1.y; xg[6] = u1.z; xg[7] = u1.w;
#pragma unroll
          for (int y = 0; y < 8; ++y) gs = fmaf(xs[y], xg[y], gs);
          bf8 f[3];
          split8<3>(xg, f);
          frag_store<3>(sh_p + st, f, sl + 16 * e);
        }
        if (x < 3) load_state(G, x + 1);
        lds_barrier();
        bf8 fu[3];
        raw_parts<F32, 3>(fu, nu[0]);
        if (x < 3) nu[0] = raw_f32(U + row * D + 32 * (x + 1) + 8 * g);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          bf8 bg[3];
          frag_load<3>(bg, sh_p + n * 3 * 512, lane);
          mma_into<3, 3>(z3[n], bg, fu);
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float k[4];
        load4(pk + 16 * n + 4 * g, k);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          kz = fmaf(k[r], z3[n][r], kz);
          dk[n][r] = fmaf(kap, z3[n][r], dk[n][r]);
        }
      }
    }
    gs = wave_sum(gs);
    if (lane == 0) sh_gs[w] = gs;
    dg += __shfl_xor(dg, 16);
    kz += __shfl_xor(kz, 16);
    dg += __shfl_xor(dg, 32);
    kz += __shfl_xor(kz, 32);
    if (g == 0) {
      sh_dgam[row] = in ? dg : 0.f;
      sh_kz[row] = in ? kz : 0.f;
    }
    lds_barrier();
    // ---- E1 K, E1^T Q, (E2 + E2^T) K
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      const float *pr = sh_e + row * LDC + 32 * x + 8 * g;    // the token's row: E1 up to the diagonal, E2^T behind
      const float *pc = sh_e + (32 * x + 8 * g) * LDC + row;  // its column: E2^T above the diagonal, E1 from there
      float vr[8], vc[8], v2[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = 32 * x + 8 * g + e;
        const float a = pr[e], b = pc[e * LDC];
        vr[e] = j <= row ? a : 0.f;
        vc[e] = j >= row ? b : 0.f;
        if (DELTA) v2[e] = j < row ? b : (j > row ? a : 0.f);
      }
      bf8 fr[NE], fc[NE], f2[NE];
      split8<NE>(vr, fr);
      split8<NE>(vc, fc);
      if (DELTA) split8<NE>(v2, f2);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const size_t f = ((atk * 8 + n) * 2 + x) * NP * 512;
        bf8 bk[NP], bq[NP];
        frag_load<NP>(bk, A.w.KT + f, lane);
        frag_load<NP>(bq, A.w.QT + f, lane);
        if (2 * x <= wt) mma_into<NP, NE, NE>(dq[n], bk, fr);
        if (2 * x + 1 >= wt) mma_into<NP, NE, NE>(dk[n], bq, fc);
        if (DELTA) mma_into<NP, NE, NE>(dk[n], bk, f2);
      }
    }
    // ---- dalpha: lane 0 has the state's column, lane j that of token j - 1;
    // wave w has tokens 16 w .. + 15, and what comes in from later ones is
    // added through the product of the decays between
    {
      const int j = lane - 1;
      float f[16], run = 0.f, pa = 1.f;
#pragma unroll
      for (int e = 15; e >= 0; --e) {
        const int t = 16 * w + e;
        float dl;
        if (lane == 0) {
          dl = sh_dgam[t];
          if (t == C - 1) dl += (sh_gs[0] + sh_gs[1]) + (sh_gs[2] + sh_gs[3]);
        } else {
          dl = t > j ? sh_l[j * LDC + t] : 0.f;
          if (t == C - 1) dl = fmaf(sh_be[j], sh_kz[j], dl);
        }
        const float a = t < C - 1 ? sh_a[t + 1] : 0.f;  // from the token behind
        run = fmaf(e < 15 ? a : 0.f, run, dl);
        pa *= a;
        f[e] = run;
      }
      sh_f[w][lane] = run;
      if (lane == 0) sh_fa[w] = pa;
      lds_barrier();
      float carry = 0.f;
      for (int s = 3; s > w; --s) carry = fmaf(sh_fa[s], carry, sh_f[s][lane]);
#pragma unroll
      for (int e = 15; e >= 0; --e) {
        const int t = 16 * w + e;
        carry *= t < C - 1 ? sh_a[t + 1] : 0.f;
        const float wg = lane == 0 ? (t > 0 ? sh_gam[t - 1] : 1.f) : (t > j ? sh_l[(t - 1) * LDC + j] : 0.f);
        const float x = wave_sum((f[e] + carry) * wg);
        if (lane == 0 && t < ch.len) *at<float>(A.dalpha, ch.t0 + t, hv) = x;
      }
      if (w == 0 && lane < ch.len) {
        float x = sh_l[(C - 1) * LDC + lane] * sh_kz[lane];
        for (int t = lane >> 4; t < 4; ++t) x += sh_db[t][lane];
        *at<float>(A.dbeta, ch.t0 + lane, hv) = x;
      }
    }
  }
  const int row = 16 * wt + (lane & 15), g = lane >> 4;
  if (row < ch.len) {
    E *oq = at<E>(A.dq, ch.t0 + row, hk) + 4 * g, *ok = at<E>(A.dk, ch.t0 + row, hk) + 4 * g;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      store4(oq + 16 * n, dq[n]);
      store4(ok + 16 * n, dk[n]);
    }
  }
}

// ---------------------------------------------------------------------------
// Launcher
// ---------------------------------------------------------------------------
template <class E, bool DELTA>
hipError_t backward(const SeqArgs &a, hipStream_t stream) {
  const int64_t units = ((int64_t)a.seqs * a.hv + 7) / 8 * 8;
  if (scan_wide(a))
    hipLaunchKernelGGL((seq_rscan_kernel<E, DELTA, 32>), dim3((unsigned)(units * 4)), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((seq_rscan_kernel<E, DELTA, 16>), dim3((unsigned)(units * 8)), dim3(512), 0, stream, a);
  hipLaunchKernelGGL((seq_grad_kernel<E, DELTA>), dim3((unsigned)a.slots, a.hk), dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <class E>
hipError_t backward(const SeqArgs &a, bool delta, hipStream_t stream) {
  return delta ? backward<E, true>(a, stream) : backward<E, false>(a, stream);
}
hipError_t launch_seq_backward(const SeqArgs &a, int dtype, bool delta, hipStream_t stream) {
  return dtype == 0 ? backward<F32>(a, delta, stream)
         : dtype == 1 ? backward<BF16>(a, delta, stream)
                      : backward<F16>(a, delta, stream);
}

}  // namespace lq
