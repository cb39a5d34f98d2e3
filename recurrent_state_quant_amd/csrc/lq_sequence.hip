// Forward pass of the gated delta rule over whole sequences (gfx950).
//
//   u_t = v_t - S_{t-1}^T b_t,  S_t = D_t S_{t-1} + k~_t u_t^T,  o_t = S_t^T q_t
//
// Two forms:
//   recurrent  token by token, the state in registers: every gate, any
//              length; one launch, so it also serves a few tokens per
//              sequence.
//   chunked    64 tokens at a time on the matrix path (scalar gate).  With
//              the decays L_ij = alpha_{j+1} .. alpha_i, G_i = alpha_1 ..
//              alpha_i and kappa_j = L_Cj beta_j of a chunk that starts at
//              state S0,
//                (I + M) U = V - G * (K S0),   M_ij = L_ij beta_j k_i.k_j  (j < i)
//                O = G * (Q S0) + P U,         P_ij = L_ij beta_j q_i.k_j  (j <= i)
//                S_C = G_C S0 + (kappa * K)^T U
//              in three launches: prep (T = (I + M)^-1 and P of every chunk,
//              in parallel), scan (U and S from chunk to chunk; the columns
//              of S are independent, so a head's scan is spread over
//              workgroups by columns), out (O of every chunk, in parallel).
#include "lq_sequence_device.h"

namespace lq {

// ---------------------------------------------------------------------------
// Recurrent form.  A wave holds all 128 rows of 8 * CC columns of one state:
// lane (column group cg = lane >> 3, row group rg = lane & 7) holds rows
// 16 rg .. 16 rg + 15 of CC columns.  Per token it needs S^T (D k) and S^T (D q)
// from the same S_{t-1} (o_t = S_{t-1}^T (D q) + (k~.q) u_t), so both sums are
// taken in one pass and reduced over the 8 row groups by DPP.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float row8_sum(float x) {
  x += dpp<0xB1>(x);   // quad_perm [1,0,3,2]
  x += dpp<0x4E>(x);   // quad_perm [2,3,0,1]
  x += dpp<0x141>(x);  // row_half_mirror: the other quad of the eight
  return x;
}

template <class E, bool KDA, bool DELTA, int CC>
__global__ __launch_bounds__(256) void seq_recurrent_kernel(const SeqArgs A) {
  constexpr int kBlocks = D / (32 * CC);  // workgroups per state
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int64_t unit = blockIdx.x / kBlocks;
  const int seq = (int)(unit / A.hv), hv = (int)(unit % A.hv), hk = hv / A.group;
  const int row0 = (lane & 7) * 16;
  const int col0 = (blockIdx.x % kBlocks) * 32 * CC + w * 8 * CC + (lane >> 3) * CC;
  const int start = seq_start(A, seq), end = seq_end(A, seq, start);

  float s[16][CC];
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int c = 0; c < CC; ++c)
      s[i][c] = A.S0 ? A.S0[(unit * D + row0 + i) * D + col0 + c] : 0.f;

  float k[16], q[16], a[KDA ? 16 : 1], v[CC], b = 0.f;
  auto fetch = [&](int t) {
    float x[8];
    const E *pk = at<const E>(A.k, t, hk) + row0, *pq = at<const E>(A.q, t, hk) + row0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load8(pk + 8 * h, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) k[8 * h + e] = x[e];
      load8(pq + 8 * h, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[8 * h + e] = x[e];
    }
    const float *pa = at<const float>(A.alpha, t, hv);
    if (KDA) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 y = reinterpret_cast<const float4 *>(pa + row0)[i];
        a[(4 * i) % (KDA ? 16 : 1)] = y.x;
        a[(4 * i + 1) % (KDA ? 16 : 1)] = y.y;
        a[(4 * i + 2) % (KDA ? 16 : 1)] = y.z;
        a[(4 * i + 3) % (KDA ? 16 : 1)] = y.w;
      }
    } else {
      a[0] = pa[0];
    }
    b = at<const float>(A.beta, t, hv)[0];
#pragma unroll
    for (int c = 0; c < CC; ++c) v[c] = to_f(at<const E>(A.v, t, hv)[col0 + c]);
  };
  if (start < end) fetch(start);
  for (int t = start; t < end; ++t) {
    float kt[16], y1[CC], y2[CC], kq = 0.f, u[CC];
    const float bt = b;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      kt[i] = bt * k[i];
      kq = fmaf(kt[i], q[i], kq);
    }
#pragma unroll
    for (int c = 0; c < CC; ++c) {
      float p1 = 0.f, p2 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i][c] *= a[KDA ? i : 0];
        if (DELTA) p1 = fmaf(s[i][c], k[i], p1);
        p2 = fmaf(s[i][c], q[i], p2);
      }
      y1[c] = p1;
      y2[c] = p2;
      u[c] = v[c];
    }
    if (t + 1 < end) fetch(t + 1);  // the next token's loads run behind the sums
    kq = row8_sum(kq);
    float o[CC];
#pragma unroll
    for (int c = 0; c < CC; ++c) {
      if (DELTA) u[c] -= row8_sum(y1[c]);
      o[c] = fmaf(kq, u[c], row8_sum(y2[c]));
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i][c] = fmaf(kt[i], u[c], s[i][c]);
    }
    if ((lane & 7) == 0) {
#pragma unroll
      for (int c = 0; c < CC; ++c) at<E>(A.o, t, hv)[col0 + c] = from_f<E>(o[c]);
    }
  }
  if (A.S) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < CC; ++c) A.S[(unit * D + row0 + i) * D + col0 + c] = s[i][c];
  }
}

// ---------------------------------------------------------------------------
// Prep: one workgroup per (slot, key head); the value heads that share it in
// turn.  q k^T and k k^T are taken once.  T by blocks of 16: each diagonal
// block by forward substitution (a column per lane), then T_ab = -T_aa sum_c
// M_ac T_cb by distance from the diagonal.
// ---------------------------------------------------------------------------
template <class E, bool DELTA>
__global__ __launch_bounds__(256) void seq_prep_kernel(const SeqArgs A) {
  const int slot = blockIdx.x, hk = blockIdx.y;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const Chunk ch = find_chunk(A, slot, lane);
  if (ch.len == 0) return;
  __shared__ float sh_k[C * LDD];
  __shared__ float sh_l[C * LDC];
  __shared__ float sh_m[C * LDC];
  __shared__ float sh_t[C * LDC];
  __shared__ float sh_a[C], sh_b[C];
  stage_rows<E>(sh_k, A.k, hk, ch.t0, ch.len, tid);
  __syncthreads();
  const int i0 = 16 * w + 4 * (lane >> 4), j0 = lane & 15;
  floatx4 qk[4], kk[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) qk[n] = kk[n] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int x = 0; x < D / 16; ++x) {
    const float4 fq = frag_rows<E>(A.q, hk, ch.t0, ch.len, 16 * w, x, lane);
    const float4 fk = frag<false>(sh_k, LDD, 16 * w, x, lane);
    for (int n = 0; n <= w; ++n) {
      const float4 fb = frag<false>(sh_k, LDD, 16 * n, x, lane);
      mma(qk[n], fq, fb);
      if (DELTA) mma(kk[n], fk, fb);
    }
  }
  for (int g = 0; g < A.group; ++g) {
    const int hv = hk * A.group + g;
    const size_t at_ = (size_t)slot * A.hv + hv;
    __syncthreads();
    if (w == 0) {
      const bool in = lane < ch.len;
      const float al = in ? *at<const float>(A.alpha, ch.t0 + lane, hv) : 1.f;
      const float be = in ? *at<const float>(A.beta, ch.t0 + lane, hv) : 0.f;
      sh_a[lane] = al;
      sh_b[lane] = be;
      // decay from the chunk's start (inclusive prefix product) and to its
      // end (exclusive suffix product)
      float pre = al, suf = __shfl_down(al, 1);  // (every lane takes part in a shuffle)
      suf = lane < 63 ? suf : 1.f;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const float x = __shfl_up(pre, d), y = __shfl_down(suf, d);
        if (lane >= d) pre *= x;
        if (lane + d < 64) suf *= y;
      }
      A.w.dec[at_ * 2 * C + lane] = pre;
      A.w.dec[at_ * 2 * C + C + lane] = suf * be;
    }
    __syncthreads();
    decay_matrix(sh_l, sh_a, tid);
    __syncthreads();
    float *P = A.w.P + at_ * C * C;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int j = 16 * n + j0;
      const float be = sh_b[j];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = i0 + r;
        const float lb = sh_l[i * LDC + j] * be;
        P[i * C + j] = j <= i ? lb * qk[n][r] : 0.f;
        if (DELTA) sh_m[i * LDC + j] = j < i ? lb * kk[n][r] : 0.f;
      }
    }
    if (!DELTA) continue;
    __syncthreads();
    // diagonal blocks: wave w, column lane & 15 (four lanes do the same)
    {
      const int d0 = 16 * w;
      float t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = i == j0 ? 1.f : 0.f;
#pragma unroll
        for (int l = 0; l < i; ++l) x = fmaf(-sh_m[(d0 + i) * LDC + d0 + l], t[l], x);
        t[i] = x;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (lane < 16) sh_t[(d0 + i) * LDC + d0 + j0] = t[i];
      }
    }
    const int bi = tid >> 4, bj = tid & 15;
    for (int dist = 1; dist < 4; ++dist) {
      __syncthreads();
      float x[3];
      for (int a = dist; a < 4; ++a) {
        const int b = a - dist;
        float y = 0.f;
        for (int c = b; c < a; ++c)
#pragma unroll
          for (int l = 0; l < 16; ++l)
            y = fmaf(sh_m[(16 * a + bi) * LDC + 16 * c + l], sh_t[(16 * c + l) * LDC + 16 * b + bj], y);
        // kept in the upper triangle of sh_m, which is not read
        sh_m[(16 * b + bi) * LDC + 16 * a + bj] = y;
      }
      __syncthreads();
      for (int a = dist; a < 4; ++a) {
        const int b = a - dist;
        float y = 0.f;
#pragma unroll
        for (int l = 0; l < 16; ++l)
          y = fmaf(sh_t[(16 * a + bi) * LDC + 16 * a + l], sh_m[(16 * b + l) * LDC + 16 * a + bj], y);
        x[a - 1] = -y;
      }
      for (int a = dist; a < 4; ++a) sh_t[(16 * a + bi) * LDC + 16 * (a - dist) + bj] = x[a - 1];
    }
    __syncthreads();
    float *T = A.w.T + at_ * C * C;
    for (int e = tid; e < C * C; e += 256) {
      const int i = e >> 6, j = e & 63;
      T[e] = (j >> 4) <= (i >> 4) ? sh_t[i * LDC + j] : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------
// Scan: one workgroup per (sequence, value head, block of CB columns).  Wave
// w holds rows 32 w .. 32 w + 31 of the state block in its accumulators and
// takes token tile w of the products with 64 rows.
// ---------------------------------------------------------------------------
template <class E, bool DELTA, int CB>
__global__ __launch_bounds__(256) void seq_scan_kernel(const SeqArgs A) {
  constexpr int NT = CB / 16, kBlocks = D / CB;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  // workgroups b, b + 8, .. run on one XCD: the column blocks of one head
  // are placed there, so that its L2 serves their common K and T
  const int64_t b = blockIdx.x;
  const int64_t unit = (b / (8 * kBlocks)) * 8 + (b & 7);
  if (unit >= (int64_t)A.seqs * A.hv) return;
  const int col0 = (int)((b >> 3) % kBlocks) * CB;
  const int seq = (int)(unit / A.hv), hv = (int)(unit % A.hv), hk = hv / A.group;
  const int start = seq_start(A, seq), end = seq_end(A, seq, start);
  __shared__ float sh_k[C * LDD];
  __shared__ float sh_T[DELTA ? C * LDC : 1];
  __shared__ float sh_s[CB * LDD];  // S^T
  __shared__ float sh_x[CB * LDC];  // X^T
  __shared__ float sh_u[CB * LDC];  // (kappa * U)^T
  const int i = lane & 15, g = lane >> 4;

  floatx4 s[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        s[m][n][r] = A.S0 ? A.S0[(unit * D + 32 * w + 16 * m + 4 * g + r) * D + col0 + 16 * n + i] : 0.f;

  for (int t0 = start, slot = start / C + seq; t0 < end; t0 += C, ++slot) {
    const int len = end - t0 < C ? end - t0 : C;
    const size_t at_ = (size_t)slot * A.hv + hv;
    const float *dec = A.w.dec + at_ * 2 * C;
    stage_rows<E>(sh_k, A.k, hk, t0, len, tid);
    if (DELTA) stage_f32<C>(sh_T, LDC, A.w.T + at_ * C * C, C, tid);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 x = make_float4(s[m][n][0], s[m][n][1], s[m][n][2], s[m][n][3]);
        const int row = 32 * w + 16 * m + 4 * g, col = 16 * n + i;
        *reinterpret_cast<float4 *>(sh_s + col * LDD + row) = x;
        *reinterpret_cast<float4 *>(A.w.S + (at_ * D + col0 + col) * D + row) = x;
      }
    __syncthreads();
    const int tok = 16 * w + 4 * g;
    floatx4 u[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) u[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (DELTA) {
      for (int x = 0; x < D / 16; ++x) {
        const float4 fa = frag<false>(sh_k, LDD, 16 * w, x, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(u[n], fa, frag<false>(sh_s, LDD, 16 * n, x, lane));
      }
    }
    float kap[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      kap[r] = dec[C + tok + r];
      const float gam = dec[tok + r];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float v = tok + r < len ? to_f(at<const E>(A.v, t0 + tok + r, hv)[col0 + 16 * n + i]) : 0.f;
        u[n][r] = v - gam * u[n][r];
      }
    }
    if (DELTA) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float4 *>(sh_x + (16 * n + i) * LDC + tok) =
            make_float4(u[n][0], u[n][1], u[n][2], u[n][3]);
        u[n] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
      __syncthreads();
      for (int x = 0; x <= w; ++x) {
        const float4 fa = frag<false>(sh_T, LDC, 16 * w, x, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(u[n], fa, frag<false>(sh_x, LDC, 16 * n, x, lane));
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 4; ++r) A.w.U[(at_ * C + tok + r) * D + col0 + 16 * n + i] = u[n][r];
      *reinterpret_cast<float4 *>(sh_u + (16 * n + i) * LDC + tok) =
          make_float4(kap[0] * u[n][0], kap[1] * u[n][1], kap[2] * u[n][2], kap[3] * u[n][3]);
    }
    const float last = dec[C - 1];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[m][n] *= last;
      for (int x = 0; x < C / 16; ++x) {
        const float4 fa = frag<true>(sh_k, LDD, 32 * w + 16 * m, x, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(s[m][n], fa, frag<false>(sh_u, LDC, 16 * n, x, lane));
      }
    }
    __syncthreads();
  }
  if (A.S) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          A.S[(unit * D + 32 * w + 16 * m + 4 * g + r) * D + col0 + 16 * n + i] = s[m][n][r];
  }
}

// ---------------------------------------------------------------------------
// Out: one workgroup per (slot, value head); wave w takes token tile w.
// ---------------------------------------------------------------------------
template <class E>
__global__ __launch_bounds__(256) void seq_out_kernel(const SeqArgs A) {
  const int slot = blockIdx.x, hv = blockIdx.y, hk = hv / A.group;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const Chunk ch = find_chunk(A, slot, lane);
  if (ch.len == 0) return;
  const size_t at_ = (size_t)slot * A.hv + hv;
  __shared__ float sh_b[C * LDD];
  const int i = lane & 15, g = lane >> 4, tok = 16 * w + 4 * g;
  floatx4 acc[8];
#pragma unroll
  for (int n = 0; n < 8; ++n) acc[n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // columns 64 h .. 64 h + 63 of S
    __syncthreads();
    stage_f32<D>(sh_b, LDD, A.w.S + (at_ * D + 64 * h) * D, 64, tid);
    __syncthreads();
    for (int x = 0; x < D / 16; ++x) {
      const float4 fa = frag_rows<E>(A.q, hk, ch.t0, ch.len, 16 * w, x, lane);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(acc[4 * h + n], fa, frag<false>(sh_b, LDD, 16 * n, x, lane));
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float gam = A.w.dec[at_ * 2 * C + tok + r];
#pragma unroll
    for (int n = 0; n < 8; ++n) acc[n][r] *= gam;
  }
  __syncthreads();
  stage_f32<D>(sh_b, LDD, A.w.U + at_ * C * D, C, tid);
  __syncthreads();
  const float *P = A.w.P + at_ * C * C;
  for (int x = 0; x <= w; ++x) {
    const float4 fa = frag<false>(P, C, 16 * w, x, lane);
#pragma unroll
    for (int n = 0; n < 8; ++n) mma(acc[n], fa, frag<true>(sh_b, LDD, 16 * n, x, lane));
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (tok + r < ch.len) {
      E *o = at<E>(A.o, ch.t0 + tok + r, hv);
#pragma unroll
      for (int n = 0; n < 8; ++n) o[16 * n + i] = from_f<E>(acc[n][r]);
    }
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <class E, bool KDA, bool DELTA>
hipError_t recurrent(const SeqArgs &a, hipStream_t stream) {
  const int64_t states = (int64_t)a.seqs * a.hv;
  // four columns a lane read the state in whole 128-byte lines and share k
  // and q among more columns; one column a lane has a quarter of the work in
  // each token's chain, and pays once there are few states
  if (states >= 256)
    hipLaunchKernelGGL((seq_recurrent_kernel<E, KDA, DELTA, 4>), dim3((unsigned)states), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((seq_recurrent_kernel<E, KDA, DELTA, 1>), dim3((unsigned)states * 4), dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <class E>
hipError_t recurrent(const SeqArgs &a, bool kda, bool delta, hipStream_t stream) {
  if (kda) return delta ? recurrent<E, true, true>(a, stream) : recurrent<E, true, false>(a, stream);
  return delta ? recurrent<E, false, true>(a, stream) : recurrent<E, false, false>(a, stream);
}
hipError_t launch_seq_recurrent(const SeqArgs &a, int dtype, bool kda, bool delta, hipStream_t stream) {
  return dtype == 0 ? recurrent<F32>(a, kda, delta, stream)
         : dtype == 1 ? recurrent<BF16>(a, kda, delta, stream)
                      : recurrent<F16>(a, kda, delta, stream);
}

template <class E, bool DELTA>
hipError_t chunked(const SeqArgs &a, hipStream_t stream) {
  const dim3 slots((unsigned)a.slots, a.hk), heads((unsigned)a.slots, a.hv);
  const int64_t units = ((int64_t)a.seqs * a.hv + 7) / 8 * 8;
  hipLaunchKernelGGL((seq_prep_kernel<E, DELTA>), slots, dim3(256), 0, stream, a);
  hipLaunchKernelGGL((seq_scan_kernel<E, DELTA, 16>), dim3((unsigned)(units * (D / 16))), dim3(256), 0, stream, a);
  hipLaunchKernelGGL((seq_out_kernel<E>), heads, dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <class E>
hipError_t chunked(const SeqArgs &a, bool delta, hipStream_t stream) {
  return delta ? chunked<E, true>(a, stream) : chunked<E, false>(a, stream);
}
hipError_t launch_seq_chunked(const SeqArgs &a, int dtype, bool delta, hipStream_t stream) {
  return dtype == 0 ? chunked<F32>(a, delta, stream)
         : dtype == 1 ? chunked<BF16>(a, delta, stream)
                      : chunked<F16>(a, delta, stream);
}

}  // namespace lq
