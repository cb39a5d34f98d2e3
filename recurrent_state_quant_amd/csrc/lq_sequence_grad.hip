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
// Reverse scan: as the forward scan, one workgroup per (sequence, value head,
// block of CB columns), wave w holding rows 32 w .. + 31 of G.
// ---------------------------------------------------------------------------
template <class E, bool DELTA, int CB>
__global__ __launch_bounds__(256) void seq_rscan_kernel(const SeqArgs A) {
  constexpr int NT = CB / 16, kBlocks = D / CB;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int64_t b = blockIdx.x;  // column blocks of a head on one XCD, as in the forward scan
  const int64_t unit = (b / (8 * kBlocks)) * 8 + (b & 7);
  if (unit >= (int64_t)A.seqs * A.hv) return;
  const int col0 = (int)((b >> 3) % kBlocks) * CB;
  const int seq = (int)(unit / A.hv), hv = (int)(unit % A.hv), hk = hv / A.group;
  const int start = seq_start(A, seq), end = seq_end(A, seq, start);
  __shared__ float sh_k[C * LDD];
  __shared__ float sh_q[C * LDD];
  __shared__ float sh_P[C * LDC];
  __shared__ float sh_T[DELTA ? C * LDC : 1];
  __shared__ float sh_g[CB * LDD];  // G^T
  __shared__ float sh_o[CB * LDC];  // dO^T
  __shared__ float sh_og[CB * LDC]; // (Gam * dO)^T
  __shared__ float sh_u[CB * LDC];  // dU^T, then -(Gam * dX)^T
  const int i = lane & 15, g = lane >> 4, tok = 16 * w + 4 * g;

  floatx4 s[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        s[m][n][r] = A.dS ? A.dS[(unit * D + 32 * w + 16 * m + 4 * g + r) * D + col0 + 16 * n + i] : 0.f;

  const int chunks = (end - start + C - 1) / C;
  for (int c = chunks - 1; c >= 0; --c) {
    const int t0 = start + c * C, len = end - t0 < C ? end - t0 : C;
    const size_t at_ = (size_t)(start / C + seq + c) * A.hv + hv;
    const float *dec = A.w.dec + at_ * 2 * C;
    stage_rows<E>(sh_k, A.k, hk, t0, len, tid);
    stage_rows<E>(sh_q, A.q, hk, t0, len, tid);
    stage_f32<C>(sh_P, LDC, A.w.P + at_ * C * C, C, tid);
    if (DELTA) stage_f32<C>(sh_T, LDC, A.w.T + at_ * C * C, C, tid);
    float gam[4], kap[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      gam[r] = dec[tok + r];
      kap[r] = dec[C + tok + r];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = tok + r < len ? to_f(at<const E>(A.go, t0 + tok + r, hv)[col0 + 16 * n + i]) : 0.f;
      *reinterpret_cast<float4 *>(sh_o + (16 * n + i) * LDC + tok) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4 *>(sh_og + (16 * n + i) * LDC + tok) =
          make_float4(gam[0] * x[0], gam[1] * x[1], gam[2] * x[2], gam[3] * x[3]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 x = make_float4(s[m][n][0], s[m][n][1], s[m][n][2], s[m][n][3]);
        const int row = 32 * w + 16 * m + 4 * g, col = 16 * n + i;
        *reinterpret_cast<float4 *>(sh_g + col * LDD + row) = x;
        *reinterpret_cast<float4 *>(A.w.G + (at_ * D + col0 + col) * D + row) = x;
      }
    __syncthreads();
    floatx4 u[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) u[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int x = 0; x < D / 16; ++x) {
      const float4 fa = frag<false>(sh_k, LDD, 16 * w, x, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma(u[n], fa, frag<false>(sh_g, LDD, 16 * n, x, lane));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) u[n][r] *= kap[r];
    for (int x = w; x < C / 16; ++x) {
      const float4 fa = frag<true>(sh_P, LDC, 16 * w, x, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma(u[n], fa, frag<false>(sh_o, LDC, 16 * n, x, lane));
    }
    if (DELTA) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float4 *>(sh_u + (16 * n + i) * LDC + tok) =
            make_float4(u[n][0], u[n][1], u[n][2], u[n][3]);
        u[n] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
      __syncthreads();
      for (int x = w; x < C / 16; ++x) {
        const float4 fa = frag<true>(sh_T, LDC, 16 * w, x, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(u[n], fa, frag<false>(sh_u, LDC, 16 * n, x, lane));
      }
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        A.w.X[(at_ * C + tok + r) * D + col0 + 16 * n + i] = u[n][r];
        if (tok + r < len) at<E>(A.dv, t0 + tok + r, hv)[col0 + 16 * n + i] = from_f<E>(u[n][r]);
      }
      if (DELTA)
        *reinterpret_cast<float4 *>(sh_u + (16 * n + i) * LDC + tok) =
            make_float4(-gam[0] * u[n][0], -gam[1] * u[n][1], -gam[2] * u[n][2], -gam[3] * u[n][3]);
    }
    const float last = dec[C - 1];
    if (DELTA) __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[m][n] *= last;
      for (int x = 0; x < C / 16; ++x) {
        const float4 fa = frag<true>(sh_q, LDD, 32 * w + 16 * m, x, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(s[m][n], fa, frag<false>(sh_og, LDC, 16 * n, x, lane));
        if (DELTA) {
          const float4 fk = frag<true>(sh_k, LDD, 32 * w + 16 * m, x, lane);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(s[m][n], fk, frag<false>(sh_u, LDC, 16 * n, x, lane));
        }
      }
    }
    __syncthreads();
  }
  if (A.dS0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          A.dS0[(unit * D + 32 * w + 16 * m + 4 * g + r) * D + col0 + 16 * n + i] = s[m][n][r];
  }
}

// ---------------------------------------------------------------------------
// Gradients inside a chunk: one workgroup per (slot, key head), the value
// heads that share it in turn, so that dQ and dK are summed over them in a
// fixed order.  Wave w takes token tile w; rows of the products live in its
// accumulators.
// ---------------------------------------------------------------------------
template <class E, bool DELTA>
__global__ __launch_bounds__(256) void seq_grad_kernel(const SeqArgs A) {
  const int slot = blockIdx.x, hk = blockIdx.y;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const Chunk ch = find_chunk(A, slot, lane);
  if (ch.len == 0) return;
  __shared__ float sh_k[C * LDD];
  __shared__ float sh_b[C * LDD];   // U, then halves of S0 and G, then Q
  __shared__ float sh_l[C * LDC];   // L
  __shared__ float sh_dl[C * LDC];  // dL, then the terms of dalpha
  __shared__ float sh_e1[C * LDC];
  __shared__ float sh_e2[DELTA ? C * LDC : 1];
  __shared__ float sh_a[C], sh_be[C], sh_gam[C], sh_kap[C];
  __shared__ float sh_dgam[C], sh_kz[C], sh_db[4][C], sh_gs[4];
  const int i = lane & 15, g = lane >> 4, tok = 16 * w + 4 * g;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

  stage_rows<E>(sh_k, A.k, hk, ch.t0, ch.len, tid);
  floatx4 dq[8], dk[8];
#pragma unroll
  for (int n = 0; n < 8; ++n) dq[n] = dk[n] = zero;

  for (int gr = 0; gr < A.group; ++gr) {
    const int hv = hk * A.group + gr;
    const size_t at_ = (size_t)slot * A.hv + hv;
    const float *U = A.w.U + at_ * C * D, *X = A.w.X + at_ * C * D;
    const float *S0 = A.w.S + at_ * D * D, *G = A.w.G + at_ * D * D;
    __syncthreads();
    if (tid < C) {
      const bool in = tid < ch.len;
      sh_a[tid] = in ? *at<const float>(A.alpha, ch.t0 + tid, hv) : 1.f;
      sh_be[tid] = in ? *at<const float>(A.beta, ch.t0 + tid, hv) : 0.f;
      sh_gam[tid] = A.w.dec[at_ * 2 * C + tid];
      sh_kap[tid] = A.w.dec[at_ * 2 * C + C + tid];
    }
    stage_f32<D>(sh_b, LDD, U, C, tid);
    __syncthreads();
    decay_matrix(sh_l, sh_a, tid);
    __syncthreads();
    // ---- the four products of 64 x 64, lower tiles only
    {
      floatx4 a1[4], a2[4], d1[4], d2[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) a1[n] = a2[n] = d1[n] = d2[n] = zero;
      for (int x = 0; x < D / 16; ++x) {
        const float4 fq = frag_rows<E>(A.q, hk, ch.t0, ch.len, 16 * w, x, lane);
        const float4 fo = frag_rows<E>(A.go, hv, ch.t0, ch.len, 16 * w, x, lane);
        const float4 fk = frag<false>(sh_k, LDD, 16 * w, x, lane);
        const float4 fx = frag<false>(X, D, 16 * w, x, lane);
        for (int n = 0; n <= w; ++n) {
          const float4 bk = frag<false>(sh_k, LDD, 16 * n, x, lane);
          const float4 bu = frag<false>(sh_b, LDD, 16 * n, x, lane);
          mma(a1[n], fq, bk);
          mma(d1[n], fo, bu);
          if (DELTA) {
            mma(a2[n], fk, bk);
            mma(d2[n], fx, bu);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int j = 16 * n + i;
        const float be = sh_be[j];
        float db = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = tok + r;
          const float l = sh_l[row * LDC + j];  // 0 above the diagonal
          float wv = j <= row ? d1[n][r] * a1[n][r] : 0.f;
          sh_e1[row * LDC + j] = l * be * d1[n][r];
          if (DELTA) {
            const float d = j < row ? -d2[n][r] : 0.f;
            wv = fmaf(d, a2[n][r], wv);
            sh_e2[row * LDC + j] = l * be * d;
          }
          sh_dl[row * LDC + j] = be * wv;
          db = fmaf(l, wv, db);
        }
        db += __shfl_xor(db, 16);
        db += __shfl_xor(db, 32);
        if (g == 0) sh_db[w][j] = db;
      }
    }
    // ---- Z1, Z2 with S0 and <G, S0>
    {
      floatx4 z1[8], z2[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) z1[n] = z2[n] = zero;
      float gs = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // value columns 64 h .. + 63
        __syncthreads();
        for (int e = tid; e < 64 * (D / 4); e += 256) {
          const int r = e >> 5, c = (e & 31) * 4;
          const float4 x = *reinterpret_cast<const float4 *>(S0 + (64 * h + r) * D + c);
          const float4 y = *reinterpret_cast<const float4 *>(G + (64 * h + r) * D + c);
          *reinterpret_cast<float4 *>(sh_b + r * LDD + c) = x;
          gs += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
        __syncthreads();
        for (int x = 0; x < 4; ++x) {
          const float4 fo = frag_rows<E>(A.go, hv, ch.t0, ch.len, 16 * w, 4 * h + x, lane);
          const float4 fx = frag<false>(X, D, 16 * w, 4 * h + x, lane);
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float4 fs = frag<true>(sh_b, LDD, 16 * n, x, lane);
            mma(z1[n], fo, fs);
            if (DELTA) mma(z2[n], fx, fs);
          }
        }
      }
      gs = wave_sum(gs);
      if (lane == 0) sh_gs[w] = gs;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = tok + r;
        const float gam = sh_gam[row];
        float dg = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float q = row < ch.len ? to_f(at<const E>(A.q, ch.t0 + row, hk)[16 * n + i]) : 0.f;
          dg = fmaf(q, z1[n][r], dg);
          dq[n][r] = fmaf(gam, z1[n][r], dq[n][r]);
          if (DELTA) {
            dg = fmaf(-sh_k[row * LDD + 16 * n + i], z2[n][r], dg);
            dk[n][r] = fmaf(-gam, z2[n][r], dk[n][r]);
          }
        }
        dg = row16_sum(dg);
        if (i == 0) sh_dgam[row] = dg;
      }
    }
    // ---- Z3 with G
    {
      floatx4 z3[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) z3[n] = zero;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncthreads();
        stage_f32<D>(sh_b, LDD, G + 64 * h * D, 64, tid);
        __syncthreads();
        for (int x = 0; x < 4; ++x) {
          const float4 fu = frag<false>(U, D, 16 * w, 4 * h + x, lane);
#pragma unroll
          for (int n = 0; n < 8; ++n) mma(z3[n], fu, frag<true>(sh_b, LDD, 16 * n, x, lane));
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = tok + r;
        const float kap = sh_kap[row];
        float kz = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          kz = fmaf(sh_k[row * LDD + 16 * n + i], z3[n][r], kz);
          dk[n][r] = fmaf(kap, z3[n][r], dk[n][r]);
        }
        kz = row16_sum(kz);
        if (i == 0) sh_kz[row] = kz;
      }
    }
    // ---- E1 K, E1^T Q, (E2 + E2^T) K
    __syncthreads();
    stage_rows<E>(sh_b, A.q, hk, ch.t0, ch.len, tid);
    __syncthreads();
    for (int x = 0; x < 4; ++x) {
      if (x <= w) {
        const float4 f1 = frag<false>(sh_e1, LDC, 16 * w, x, lane);
        float4 f2 = f1;
        if (DELTA) f2 = frag<false>(sh_e2, LDC, 16 * w, x, lane);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 bk = frag<true>(sh_k, LDD, 16 * n, x, lane);
          mma(dq[n], f1, bk);
          if (DELTA) mma(dk[n], f2, bk);
        }
      }
      if (x >= w) {
        const float4 f1 = frag<true>(sh_e1, LDC, 16 * w, x, lane);
        float4 f2 = f1;
        if (DELTA) f2 = frag<true>(sh_e2, LDC, 16 * w, x, lane);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          mma(dk[n], f1, frag<true>(sh_b, LDD, 16 * n, x, lane));
          if (DELTA) mma(dk[n], f2, frag<true>(sh_k, LDD, 16 * n, x, lane));
        }
      }
    }
    // ---- dalpha: lane 0 runs the state's column, lane j that of token j - 1
    if (w == 0) {
      const int j = lane - 1;
      float f = 0.f;
      for (int t = C - 1; t >= 0; --t) {
        float dl, wgt;
        if (lane == 0) {
          dl = sh_dgam[t];
          if (t == C - 1) dl += sh_gs[0] + sh_gs[1] + sh_gs[2] + sh_gs[3];
          wgt = t > 0 ? sh_gam[t - 1] : 1.f;
        } else {
          dl = t > j ? sh_dl[t * LDC + j] : 0.f;
          if (t == C - 1) dl = fmaf(sh_be[j], sh_kz[j], dl);
          wgt = t > j ? sh_l[(t - 1) * LDC + j] : 0.f;
        }
        f = fmaf(t < C - 1 ? sh_a[t + 1] : 0.f, f, dl);
        sh_dl[t * LDC + (lane == 0 ? C - 1 : j)] = f * wgt;
      }
    }
    __syncthreads();
    {
      const int t = tid >> 2;  // four threads a token
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) x += sh_dl[t * LDC + 16 * (tid & 3) + e];
      x += dpp<0xB1>(x);
      x += dpp<0x4E>(x);
      if ((tid & 3) == 0 && t < ch.len) {
        *at<float>(A.dalpha, ch.t0 + t, hv) = x;
        const float lc = sh_l[(C - 1) * LDC + t];
        *at<float>(A.dbeta, ch.t0 + t, hv) =
            sh_db[0][t] + sh_db[1][t] + sh_db[2][t] + sh_db[3][t] + lc * sh_kz[t];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (tok + r < ch.len) {
      E *pq = at<E>(A.dq, ch.t0 + tok + r, hk), *pk = at<E>(A.dk, ch.t0 + tok + r, hk);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        pq[16 * n + i] = from_f<E>(dq[n][r]);
        pk[16 * n + i] = from_f<E>(dk[n][r]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Launcher
// ---------------------------------------------------------------------------
template <class E, bool DELTA>
hipError_t backward(const SeqArgs &a, hipStream_t stream) {
  const int64_t units = ((int64_t)a.seqs * a.hv + 7) / 8 * 8;
  hipLaunchKernelGGL((seq_rscan_kernel<E, DELTA, 16>), dim3((unsigned)(units * (D / 16))), dim3(256), 0, stream, a);
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
