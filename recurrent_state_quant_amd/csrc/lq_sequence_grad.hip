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
// Bound by the chain of a chunk, as that one, and its stores of dX, dV and G: 8,192
// tokens in 4 sequences x 16 heads 255 us.
// ---------------------------------------------------------------------------
template <class E, bool DELTA, int CB>
__global__ __launch_bounds__(512) void seq_rscan_kernel(const SeqArgs A) {
  constexpr int NT = CB / 16, kBlocks = D / CB, NP = Parts<E>::n;
  constexpr int FS = 4 * NT, FX = 2 * NT;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wt = w & 3;
  const bool kwave = w < 4;
  const int64_t b = blockIdx.x;  // column blocks of a head on one XCD, as in the forward scan
  const int64_t place = (b / (8 * kBlocks)) * 8 + (b & 7);
  if (place >= (int64_t)A.seqs * A.hv) return;
  const int seq = seq_place(A, (int)(place / A.hv), gridDim.x, lane);
  const int hv = (int)(place % A.hv), hk = hv / A.group;
  const int64_t unit = (int64_t)seq * A.hv + hv;
  const int start = seq_start(A, seq), end = seq_end(A, seq, start);
  __shared__ __align__(16) uint16_t sh_g[3 * FS * 512];               // G, [column][key row]
  __shared__ __align__(16) uint16_t sh_o[NP * FX * 512];              // dO of the next chunk, [column][token]
  __shared__ __align__(16) uint16_t sh_og[3 * FX * 512];              // Gam * dO
  __shared__ __align__(16) uint16_t sh_du[DELTA ? 3 * FX * 512 : 8];  // dU
  __shared__ __align__(16) uint16_t sh_x[DELTA ? 3 * FX * 512 : 8];   // -Gam * dX
  __shared__ floatx4 sh_pd[4 * NT * 64];                              // P^T dO, as the accumulators hold it
  const int i = lane & 15, g = lane >> 4, tok = 16 * wt + 4 * g;
  const int col = (int)((b >> 3) % kBlocks) * CB + NT * i;  // the lane's first column

  floatx4 s[NT];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float x[NT] = {};
    if (A.dS) load_n<NT>(A.dS + (unit * D + 16 * w + 4 * g + r) * D + col, x);
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][r] = x[n];
  }
  wait_loads();  // the loop below counts its own loads only

  // Loads as in the forward scan: at fixed places in the code, a row past the
  // end replaced by the chunk's first; dO is zero there, and so are its rows
  // of P^T and T^T and its columns of Q^T and K^T.  Pointers move back a chunk.
  bf8 fA[4][NP], fB[2][3], fQT[2][NP], fKT[2][NP];  // K; T^T or P^T
  E raw[4][NT] = {};
  float cur[NT][4], last;
  float4 gam, kap;
  const int slot0 = start / C + seq;
  const int chunks = (end - start + C - 1) / C;
  const int tl = start + (chunks - 1) * C;  // the last chunk's first token
  const E *pO = at<const E>(A.go, tl + tok, hv) + col;
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
      for (int r = 0; r < 4; ++r) load_raw<NT>(tok + r < len ? pO + r * A.go.ts : pO - backO, raw[r]);
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
      for (int r = 0; r < 4; ++r) cur[n][r] = tok + r < len ? to_f(raw[r][n]) : 0.f;
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
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) store_quad(A.w.G + at_ * D * D, 4 * w + g, col + n, s[n]);
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
    load_QK(next);
    if (kwave) {  // dX's and dV's stores, behind the products
      E *out = at<E>(A.dv, t0 + tok, hv) + col;
      E o[4][NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r][n] = from_f<E>(u[n][r]);
        store_quad(A.w.X + at_ * C * D, 4 * wt + g, col + n, u[n]);
      }
      if (len >= C) {  // a whole chunk: no branch for every row
#pragma unroll
        for (int r = 0; r < 4; ++r) store_raw<NT>(out + r * A.dv.ts, o[r]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tok + r < len) store_raw<NT>(out + r * A.dv.ts, o[r]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n] = s[n] * la + ds[n].sum();
  }
  if (A.dS0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) x[n] = s[n][r];
      store_n<NT>(A.dS0 + (unit * D + 16 * w + 4 * g + r) * D + col, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradients inside a chunk: one workgroup of eight waves per (slot, key head),
// the value heads that share it in turn, so that dQ and dK are summed over
// them in a fixed order.  A wave takes one token tile (16 rows) and half of
// the other axis: of the 64 x 64 products every other column tile, of the 64 x
// 128 ones 64 key columns.  Products are taken transposed (the token is the
// accumulators' column), so a lane holds four neighbouring values of one
// token's row.  U, then S0 and G 32 value columns at a time, go through LDS as
// bf16 parts; every other operand is a fragment of the wave's own.
// One workgroup a CU: with four waves and two workgroups the accumulators of
// 128 key columns did not fit (68 registers in scratch, no faster).
// Bound by the latency of a workgroup's steps (32 us for a chunk and head, of
// which the matrix products at their full rate are a third): 8,192 tokens x 16
// heads 270 us, 5,000 tokens x 16 value heads on 4 key heads in fp16 240 us.
// ---------------------------------------------------------------------------
// A tile of 16 rows of 128 values as the fragments of its four steps: lane (i,
// g) holds values 32 x + 8 g .. + 7 of row i.  Rows are read whole, 256 bytes a
// quarter wave, and turned in LDS that is the wave's own (no barrier); straight
// into fragments a load would touch sixteen rows and take four times as long.
// Rows at or past `len` repeat the first row.
template <class E> struct Row4 { Raw8<E> x[4]; };
constexpr int kTileBytes = 4 * LDC;  // a row in LDS: 256 bytes and padding
template <class E>
__device__ __forceinline__ void tile_load(Row4<E> &f, float *lds, const E *p, int64_t ts, int r0, int len, int lane) {
  constexpr int kHalves = sizeof(E) / 2;  // 256 bytes of a row at a time
  const int i = lane & 15, g = lane >> 4;
  char *const d = reinterpret_cast<char *>(lds);
  uint4 v[kHalves][4];
#pragma unroll
  for (int e = 0; e < kHalves; ++e)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + 4 * q + g;
      v[e][q] = reinterpret_cast<const uint4 *>(p + (r < len ? r : 0) * ts)[16 * e + i];
    }
#pragma unroll
  for (int e = 0; e < kHalves; ++e) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(d + (4 * q + g) * kTileBytes + 16 * i) = v[e][q];
#pragma unroll
    for (int x = 0; x < 4 / kHalves; ++x)
#pragma unroll
      for (int n = 0; n < kHalves; ++n)
        f.x[e * (4 / kHalves) + x].v[n] =
            *reinterpret_cast<const uint4 *>(d + i * kTileBytes + (32 * x + 8 * g) * (int)sizeof(E) + 16 * n);
  }
}

template <class E, bool DELTA>
__global__ __launch_bounds__(512) void seq_grad_kernel(const SeqArgs A) {
  constexpr int NP = Parts<E>::n;
  const int slot = blockIdx.x, hk = blockIdx.y;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Chunk ch = find_chunk(A, slot, threadIdx.x & 63);
  if (ch.len == 0) return;
  // dO's rows on their way to fragments; parts of U, then of S0 and G; then the terms of dalpha
  __shared__ __align__(16) uint16_t sh_p[48 * 512];
  __shared__ __align__(16) float sh_u[C * LDD];  // U
  __shared__ __align__(16) float sh_x[DELTA ? C * LDD : 4];  // dX
  // two triangles each: E1 with its diagonal below, E2 transposed above; L
  // with its diagonal below, dL transposed above
  __shared__ __align__(16) float sh_e[C * LDC];
  __shared__ __align__(16) float sh_l[C * LDC];
  __shared__ __align__(16) float sh_a[C + 4], sh_be[C], sh_gam[C], sh_kap[C];
  __shared__ __align__(16) float sh_db[4][C], sh_f[8][C];
  __shared__ float sh_dgam[2][C], sh_kz[2][C], sh_gs[8], sh_fa[8];
  // waves w and w + 4 share a SIMD: their token tiles together have the same
  // share of the triangle
  const int h = w >> 2, wt = h ? 7 - w : w;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  const size_t atk = (size_t)slot * A.hk + hk;
  const uint16_t *const Qf = A.w.Q + (atk * 4 + wt) * 4 * NP * 512, *const Kf = A.w.K + atk * 16 * NP * 512;

  floatx4 dq[4], dk[4];  // key columns 64 h + 16 n + 4 g + r of token `row`
#pragma unroll
  for (int n = 0; n < 4; ++n) dq[n] = dk[n] = zero;

  for (int gr = 0; gr < A.group; ++gr) {
    // the lane is opaque in every round: else the addresses and conditions of
    // the whole round are computed ahead and kept, in scratch memory
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int row = 16 * wt + i;  // the lane's token
    const bool in = row < ch.len;
    const int hv = hk * A.group + gr;
    const size_t at_ = (size_t)slot * A.hv + hv;
    const float *U = A.w.U + at_ * C * D, *X = A.w.X + at_ * C * D;
    const float *S0 = A.w.S + at_ * D * D, *G = A.w.G + at_ * D * D;
    __syncthreads();
    Row4<E> fo;  // dO's rows of the wave's tile
    float al = 1.f, be = 0.f, gm = 0.f, kp = 0.f;
    if (tid < C) {
      const int t = ch.t0 + (tid < ch.len ? tid : 0);
      al = *at<const float>(A.alpha, t, hv);
      be = *at<const float>(A.beta, t, hv);
      gm = A.w.dec[at_ * 2 * C + tid];
      kp = A.w.dec[at_ * 2 * C + C + tid];
    }
    {
      // thread: tokens 4 (tid >> 5) .. + 3 of two pairs of columns, 2 j and 2 j + 64 on
      const int quad = tid >> 5, j = tid & 31;
      floatx4 u[2][2], x[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int o = quad_at(quad, 64 * e + 2 * j + c);
          u[e][c] = reinterpret_cast<const floatx4 *>(U)[o];
          if (DELTA) x[e][c] = reinterpret_cast<const floatx4 *>(X)[o];
        }
      tile_load(fo, reinterpret_cast<float *>(sh_p) + w * 16 * LDC, at<const E>(A.go, ch.t0, hv), A.go.ts, 16 * wt,
                ch.len, lane);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int o = (4 * quad + r) * LDD + 64 * e + 2 * j;
          *reinterpret_cast<float2 *>(sh_u + o) = make_float2(u[e][0][r], u[e][1][r]);
          if (DELTA) *reinterpret_cast<float2 *>(sh_x + o) = make_float2(x[e][0][r], x[e][1][r]);
        }
    }
    if (tid < C) {
      sh_a[tid] = tid < ch.len ? al : 1.f;
      sh_be[tid] = tid < ch.len ? be : 0.f;
      sh_gam[tid] = gm;
      sh_kap[tid] = kp;
    }
    lds_barrier();
    // U's parts: wave w stores tile w >> 1, steps 2 (w & 1), + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ut = w >> 1, x = 2 * (w & 1) + e;
      bf8 f[3];
      raw_parts<F32, 3>(f, raw_load(reinterpret_cast<const F32 *>(sh_u + (16 * ut + i) * LDD + 32 * x + 8 * g)));
      frag_store<3>(sh_p + (ut * 4 + x) * 3 * 512, f, lane);
    }
    // L: column `lane`, rows 8 w .. + 7
    {
      float p = 1.f;
      for (int l = 0; l < 8 * w; l += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(sh_a + l);
        p *= l > lane ? a.x : 1.f;
        p *= l + 1 > lane ? a.y : 1.f;
        p *= l + 2 > lane ? a.z : 1.f;
        p *= l + 3 > lane ? a.w : 1.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = 8 * w + e;
        p *= r > lane ? sh_a[r] : 1.f;
        sh_l[r * LDC + lane] = r >= lane ? p : 0.f;
      }
    }
    // Q's and K's fragments for the products: all ahead where there is room
    bf8 fq[4][NP], fk[4][NP], fb[4][2][NP];
    const auto load_qk = [&](int x) {
      frag_load<NP>(fq[x], Qf + x * NP * 512, lane);
      if (DELTA) frag_load<NP>(fk[x], Kf + (wt * 4 + x) * NP * 512, lane);
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (2 * n + h <= wt) frag_load<NP>(fb[x][n], Kf + ((2 * n + h) * 4 + x) * NP * 512, lane);
    };
    if (NP == 1) {
#pragma unroll
      for (int x = 0; x < 4; ++x) load_qk(x);
    }
    lds_barrier();  // L is whole, U's parts are stored
    // ---- the 64 x 64 products (rows j of the accumulators, column `row`), lower tiles only
    floatx4 a1[2], a2[2], d1[2], d2[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) a1[n] = a2[n] = d1[n] = d2[n] = zero;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      bf8 po[NP], px[3];
      if (NP > 1) load_qk(x);
      raw_parts<E, NP>(po, fo.x[x]);
      if (DELTA) raw_parts<F32, 3>(px, raw_load(reinterpret_cast<const F32 *>(sh_x + row * LDD + 32 * x + 8 * g)));
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int t = 2 * n + h;
        if (t <= wt) {
          bf8 bu[3];
          frag_load<3>(bu, sh_p + (t * 4 + x) * 3 * 512, lane);
          mma_into<3, NP>(d1[n], bu, po);
          if (DELTA) mma_into<3, 3>(d2[n], bu, px);
          mma_into<NP, NP>(a1[n], fb[x][n], fq[x]);
          if (DELTA) mma_into<NP, NP>(a2[n], fb[x][n], fk[x]);
        }
      }
      if (NP > 1) __builtin_amdgcn_sched_barrier(0);
    }
    // 32 value columns of S0 and G: a thread has four key rows of two columns
    floatx4 xs[2], xg[2];
    const auto load_states = [&](int x) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int o = quad_at(tid >> 4, 32 * x + 2 * (tid & 15) + c);
        xs[c] = reinterpret_cast<const floatx4 *>(S0)[o];
        xg[c] = reinterpret_cast<const floatx4 *>(G)[o];
      }
    };
    // their parts as fragments, each group g of 16 lanes with its rows in the
    // order i ^ g: so the threads of a store ask 64 banks, not 16
    float gs = 0.f;
    const auto share_states = [&]() {
      const int j = tid & 15, c = j >> 2, r0 = 4 * ((tid >> 4) & 3);
      uint16_t *d = sh_p + (tid >> 6) * 3 * 512 + 16 * c * 8 + 2 * (j & 3);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint16_t *const to = d + (r0 + (r ^ c)) * 8;
        uint32_t p[3];
        split_pair<3>(xs[0][r], xs[1][r], p);
#pragma unroll
        for (int n = 0; n < 3; ++n) *reinterpret_cast<uint32_t *>(to + n * 512) = p[n];
        split_pair<3>(xg[0][r], xg[1][r], p);
#pragma unroll
        for (int n = 0; n < 3; ++n) *reinterpret_cast<uint32_t *>(to + (24 + n) * 512) = p[n];
        gs += xs[0][r] * xg[0][r] + xs[1][r] * xg[1][r];
      }
    };
    load_states(0);
    lds_barrier();  // U's parts are read
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int t = 2 * n + h, j0 = 16 * t + 4 * g;
      float db[4] = {0.f, 0.f, 0.f, 0.f};
      if (t <= wt) {
        const float4 b4 = *reinterpret_cast<const float4 *>(sh_be + j0);
        const float4 l4 = *reinterpret_cast<const float4 *>(sh_l + row * LDC + j0);
        const float be4[4] = {b4.x, b4.y, b4.z, b4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
        float e1[4], e2[4], dl[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // a token past the end took the first one's dO: nothing of it counts
          const float o = in ? d1[n][r] : 0.f, d = DELTA && in ? -d2[n][r] : 0.f;
          e1[r] = l[r] * be4[r] * o;
          e2[r] = l[r] * be4[r] * d;
          const float w1 = o * a1[n][r], wv = DELTA ? fmaf(d, a2[n][r], w1) : w1;
          dl[r] = be4[r] * wv;
          db[r] = l[r] * wv;
          if (t == wt) {  // the diagonal: E1 alone; behind it: nothing
            const int j = j0 + r;
            db[r] = j < row ? db[r] : (j == row ? w1 : 0.f);
          }
          db[r] = row16_sum(db[r]);
        }
        if (t < wt) {
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
    // ---- Z1, Z2 with S0, Z3 with G, transposed: rows 64 h + 16 n + 4 g + r are key columns
    floatx4 z1[4], z2[4], z3[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) z1[n] = z2[n] = z3[n] = zero;
    // the products' last operands: K^T and Q^T of the first 32 tokens
    bf8 bk[4][NP], bq[4][NP];
    const auto load_kq = [&](int x) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const size_t f = ((atk * 8 + 4 * h + n) * 2 + x) * NP * 512;
        frag_load<NP>(bk[n], A.w.KT + f, lane);
        frag_load<NP>(bq[n], A.w.QT + f, lane);
      }
    };
    // Q's and K's rows, for the sums along them
    float rq[4][4], rk[4][4];
    const auto load_rows = [&]() {
      const int tc = ch.t0 + (in ? row : 0);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        load4(at<const E>(A.q, tc, hk) + 64 * h + 16 * n + 4 * g, rq[n]);
        load4(at<const E>(A.k, tc, hk) + 64 * h + 16 * n + 4 * g, rk[n]);
      }
    };
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x) lds_barrier();
      share_states();
      if (x < 3) load_states(x + 1);
      if (NP == 1 && x == 2) load_rows();
      if (NP == 1 && x == 3) load_kq(0);
      lds_barrier();
      bf8 po[NP], px[3], pu[3];
      raw_parts<E, NP>(po, fo.x[x]);
      if (DELTA) raw_parts<F32, 3>(px, raw_load(reinterpret_cast<const F32 *>(sh_x + row * LDD + 32 * x + 8 * g)));
      raw_parts<F32, 3>(pu, raw_load(reinterpret_cast<const F32 *>(sh_u + row * LDD + 32 * x + 8 * g)));
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        bf8 bs[3], bg[3];
        frag_load<3>(bs, sh_p + (4 * h + n) * 3 * 512, lane ^ g);
        frag_load<3>(bg, sh_p + (8 + 4 * h + n) * 3 * 512, lane ^ g);
        mma_into<3, NP>(z1[n], bs, po);
        if (DELTA) mma_into<3, 3>(z2[n], bs, px);
        mma_into<3, 3>(z3[n], bg, pu);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (NP > 1) load_rows();
    const float gam = sh_gam[row], kap = sh_kap[row];
    float dg = 0.f, kz = 0.f;
    {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dg = fmaf(rq[n][r], z1[n][r], dg);
          kz = fmaf(rk[n][r], z3[n][r], kz);
          dq[n][r] = fmaf(gam, z1[n][r], dq[n][r]);
          dk[n][r] = fmaf(kap, z3[n][r], dk[n][r]);
          if (DELTA) {
            dg = fmaf(-rk[n][r], z2[n][r], dg);
            dk[n][r] = fmaf(-gam, z2[n][r], dk[n][r]);
          }
        }
    }
    gs = wave_sum(gs);
    dg += __shfl_xor(dg, 16);
    kz += __shfl_xor(kz, 16);
    dg += __shfl_xor(dg, 32);
    kz += __shfl_xor(kz, 32);
    if (g == 0) {
      sh_dgam[h][row] = in ? dg : 0.f;
      sh_kz[h][row] = in ? kz : 0.f;
    }
    if (lane == 0) sh_gs[w] = gs;
    lds_barrier();
    // ---- E1 K, E1^T Q, (E2 + E2^T) K
#pragma unroll
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
      if (NP > 1) load_kq(x);
      bf8 fr[3], fc[3], f2[3];
      split8<3>(vr, fr);
      split8<3>(vc, fc);
      if (DELTA) split8<3>(v2, f2);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        mma_into<NP, 3>(dq[n], bk[n], fr);
        mma_into<NP, 3>(dk[n], bq[n], fc);
        if (DELTA) mma_into<NP, 3>(dk[n], bk[n], f2);
      }
      if (NP == 1 && x == 0) load_kq(1);
    }
    // ---- dalpha: lane 0 has the state's column, lane j that of token j - 1;
    // wave w has tokens 8 w .. + 7, and what comes in from later ones is added
    // through the product of the decays between
    float *const sh_c = reinterpret_cast<float *>(sh_p);  // [64][LDC]
    {
      const int j = lane ? lane - 1 : 0;
      const float all = ((sh_gs[0] + sh_gs[1]) + (sh_gs[2] + sh_gs[3])) + ((sh_gs[4] + sh_gs[5]) + (sh_gs[6] + sh_gs[7]));
      const float end = lane ? sh_be[j] * (sh_kz[0][j] + sh_kz[1][j]) : all;  // into the last token
      float f[8], a[8], wg[8], run = 0.f, pa = 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 8 * w + e;
        const float s0 = sh_dgam[0][t] + sh_dgam[1][t], s1 = sh_l[j * LDC + t];
        const float g0 = t > 0 ? sh_gam[t > 0 ? t - 1 : 0] : 1.f, l0 = sh_l[(t > 0 ? t - 1 : 0) * LDC + j];
        f[e] = lane ? (t > j ? s1 : 0.f) : s0;
        wg[e] = lane ? (t > j ? l0 : 0.f) : g0;
        a[e] = t < C - 1 ? sh_a[t + 1] : 0.f;  // from the token behind
      }
      if (w == 7) f[7] += end;
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        run = fmaf(e < 7 ? a[e] : 0.f, run, f[e]);
        f[e] = run;
        pa *= a[e];
      }
      sh_f[w][lane] = run;
      if (lane == 0) sh_fa[w] = pa;
      lds_barrier();
      float carry = 0.f;
      for (int s = 7; s > w; --s) carry = fmaf(sh_fa[s], carry, sh_f[s][lane]);
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        carry *= a[e];
        sh_c[(8 * w + e) * LDC + lane] = (f[e] + carry) * wg[e];
      }
    }
    // a wave sums its own eight tokens' terms, eight lanes a token
    {
      const int t = 8 * w + (lane >> 3);
      const float4 c0 = *reinterpret_cast<const float4 *>(sh_c + t * LDC + 8 * (lane & 7));
      const float4 c1 = *reinterpret_cast<const float4 *>(sh_c + t * LDC + 8 * (lane & 7) + 4);
      float x = ((c0.x + c0.y) + (c0.z + c0.w)) + ((c1.x + c1.y) + (c1.z + c1.w));
      x += dpp<0xB1>(x);
      x += dpp<0x4E>(x);
      x += dpp<0x141>(x);
      const float kzt = sh_kz[0][t] + sh_kz[1][t];
      float y = sh_l[(C - 1) * LDC + t] * kzt;
      const int first = t >> 4;  // tiles before the token's have no terms
#pragma unroll
      for (int n = 0; n < 4; ++n) y += n >= first ? sh_db[n][t] : 0.f;
      if ((lane & 7) == 0 && t < ch.len) {
        *at<float>(A.dalpha, ch.t0 + t, hv) = x;
        *at<float>(A.dbeta, ch.t0 + t, hv) = y;
      }
    }
  }
  const int row = 16 * wt + (threadIdx.x & 15), g = (threadIdx.x & 63) >> 4;
  if (row < ch.len) {
    E *pq = at<E>(A.dq, ch.t0 + row, hk) + 64 * h + 4 * g, *pk = at<E>(A.dk, ch.t0 + row, hk) + 64 * h + 4 * g;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      store4(pq + 16 * n, dq[n]);
      store4(pk + 16 * n, dk[n]);
    }
  }
}

// ---------------------------------------------------------------------------
// Launcher
// ---------------------------------------------------------------------------
template <class E, bool DELTA>
hipError_t backward(const SeqArgs &a, hipStream_t stream) {
  const int64_t units = ((int64_t)a.seqs * a.hv + 7) / 8 * 8;
  // (8,192 tokens x 16 heads, 256 wide or 512 narrow workgroups: this scan 279
  // and 254 us, the forward one 246 and 261)
  if (scan_wide(a, 512))
    hipLaunchKernelGGL((seq_rscan_kernel<E, DELTA, 32>), dim3((unsigned)(units * 4)), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((seq_rscan_kernel<E, DELTA, 16>), dim3((unsigned)(units * 8)), dim3(512), 0, stream, a);
  if (a.tokens == 0) return hipGetLastError();  // (then there is no workspace either)
  hipLaunchKernelGGL((seq_grad_kernel<E, DELTA>), dim3((unsigned)a.slots, a.hk), dim3(512), 0, stream, a);
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
