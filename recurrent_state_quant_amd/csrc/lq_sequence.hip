// Forward pass of the gated delta rule over whole sequences (gfx950).
//
//   u_t = v_t - S_{t-1}^T b_t,  S_t = D_t S_{t-1} + k~_t u_t^T,  o_t = S_t^T q_t
//
// Two forms:
//   recurrent  token by token, the state in registers, one launch: for few
//              tokens a sequence, where reading and writing the states is
//              the work.
//   chunked    64 tokens at a time on the matrix path.  With a scalar gate,
//              the decays L_ij = alpha_{j+1} .. alpha_i, G_i = alpha_1 ..
//              alpha_i and kappa_j = L_Cj beta_j of a chunk that starts at
//              state S0,
//                (I + M) U = V - G * (K S0),   M_ij = L_ij beta_j k_i.k_j  (j < i)
//                O = G * (Q S0) + P U,         P_ij = L_ij beta_j q_i.k_j  (j <= i)
//                S_C = G_C S0 + (kappa * K)^T U
//              (a decay for every key channel: at the prep kernel for it)
//              in two launches: prep (T = (I + M)^-1 and P of every chunk, in
//              parallel) and scan (U, O and S from chunk to chunk; the columns
//              of S are independent, so a head's scan is spread over
//              workgroups by columns).
// Every decay is a running product: no logarithm and no quotient, so alpha = 0
// (a state forgotten within a chunk) is exact.
#include "lq_sequence_device.h"

namespace lq {

// ---------------------------------------------------------------------------
// Recurrent form.  A wave holds all 128 rows of 8 * CC columns of one state:
// lane (column group cg = lane >> 3, row group rg = lane & 7) holds rows
// 16 rg .. 16 rg + 15 of CC columns.  Per token it needs S^T (D k) and S^T (D q)
// from the same S_{t-1} (o_t = S_{t-1}^T (D q) + (k~.q) u_t), so both sums are
// taken in one pass and reduced over the 8 row groups by DPP.
// With few tokens bound by the states' bytes: 201 tokens in 64 sequences x 32
// heads 52 us, 5.2 TB/s.  With many, by a token's chain (0.4 us, 1.1 us with four
// columns a lane), for which the chunked form is there.
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
  for (int i = 0; i < 16; ++i) {
    const float *p = A.S0 + (unit * D + row0 + i) * D + col0;
    if constexpr (CC == 4) {  // states pass once: streaming accesses
      const float4 x = A.S0 ? ld4(p) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
    } else {
      s[i][0] = A.S0 ? *p : 0.f;
    }
  }

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
    for (int i = 0; i < 16; ++i) {
      float *p = A.S + (unit * D + row0 + i) * D + col0;
      if constexpr (CC == 4)
        st4(p, make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
      else
        *p = s[i][0];
    }
  }
}

// ---------------------------------------------------------------------------
// T = (I + M)^-1 for the unit lower triangle I + M (M fp32 [64][LDC], below the
// diagonal; its blocks above are used on the way), by blocks of 16: each
// diagonal block by forward substitution (a column per lane), then 16 -> 32 ->
// 64 by T_ba = -T_b (M_ba T_a) on the fp32 matrix path.  Waves 0 .. 3 work;
// ends with a barrier.  T's blocks above the diagonal are not written.
__device__ __forceinline__ void invert_unit_lower(float *sh_t, float *sh_m, int w, int lane) {
  const int i = lane & 15, g = lane >> 4;
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  if (w < 4) {
    // diagonal block w, column i (the four groups of lanes do the same)
    const int d0 = 16 * w;
    float t[16];
#pragma unroll
    for (int a = 0; a < 16; ++a) {
      float x = a == i ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < a; ++l) x = fmaf(-sh_m[(d0 + a) * LDC + d0 + l], t[l], x);
      t[a] = x;
    }
    // group g stores rows 4 g .. + 3
#pragma unroll
    for (int a = 0; a < 16; ++a)
      if ((a >> 2) == g) sh_t[(d0 + a) * LDC + d0 + i] = t[a];
  }
  __syncthreads();
  if (w < 2) {
    const int b = 2 * w, a = b + 1;
    floatx4 y = zero, z = zero;
    mma(y, frag<false>(sh_m + 16 * b, LDC, 16 * a, 0, lane), frag<true>(sh_t + 16 * b * LDC, LDC, 16 * b, 0, lane));
    // the product, transposed, to block (b, a) of sh_m
    *reinterpret_cast<float4 *>(sh_m + (16 * b + i) * LDC + 16 * a + 4 * g) = make_float4(y[0], y[1], y[2], y[3]);
    mma(z, frag<false>(sh_t + 16 * a, LDC, 16 * a, 0, lane), frag<false>(sh_m + 16 * a, LDC, 16 * b, 0, lane));
#pragma unroll
    for (int r = 0; r < 4; ++r) sh_t[(16 * a + 4 * g + r) * LDC + 16 * b + i] = -z[r];
  }
  __syncthreads();
  const int a = 2 + (w >> 1), b = w & 1;
  if (w < 4) {
    floatx4 y = zero;
    for (int c = b; c < 2; ++c)
      mma(y, frag<false>(sh_m + 16 * c, LDC, 16 * a, 0, lane), frag<true>(sh_t + 16 * c * LDC, LDC, 16 * b, 0, lane));
    *reinterpret_cast<float4 *>(sh_m + (16 * b + i) * LDC + 16 * a + 4 * g) = make_float4(y[0], y[1], y[2], y[3]);
  }
  __syncthreads();
  if (w < 4) {
    floatx4 z = zero;
    for (int c = 2; c <= a; ++c)
      mma(z, frag<false>(sh_t + 16 * c, LDC, 16 * a, 0, lane), frag<false>(sh_m + 16 * c, LDC, 16 * b, 0, lane));
#pragma unroll
    for (int r = 0; r < 4; ++r) sh_t[(16 * a + 4 * g + r) * LDC + 16 * b + i] = -z[r];
  }
  __syncthreads();
}

// T and P as the scan's fragments: rows 16 w + i, columns 32 x + 8 g .. + 7;
// T's block above the diagonal in a step is not written in sh_t: zeros.
template <bool DELTA>
__device__ __forceinline__ void store_triangles(const SeqArgs &A, size_t at_, const float *sh_t, const float *sh_p, int w,
                                                int lane) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    if (2 * x > w) continue;
    const int row = 16 * w + i, col = 32 * x + 8 * g;
    float v[8];
    bf8 f[3];
    if (DELTA) {
      const bool in = (col >> 4) <= w;
      load8(reinterpret_cast<const F32 *>(sh_t + row * LDC + col), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = in && col + e <= row ? v[e] : 0.f;
      split8<3>(v, f);
      frag_store<3>(A.w.T + ((at_ * 4 + w) * 2 + x) * 3 * 512, f, lane);
    }
    load8(reinterpret_cast<const F32 *>(sh_p + row * LDC + col), v);
    split8<3>(v, f);
    frag_store<3>(A.w.P + ((at_ * 4 + w) * 2 + x) * 3 * 512, f, lane);
  }
}

// ---------------------------------------------------------------------------
// Prep: one workgroup per (slot, value head).  Writes, in the order in which
// the scans load them (matrix fragments, bf16 parts): T, P, and, for the first
// value head of a key head, K, Q and K^T; with SAVE also the transposes of T,
// P and Q for the backward scan.  M and T are fp32 (T's rounding enters every
// later chunk).  Four waves, a tile of 16 rows of M and P each.
// Bound by its bytes, nearly all of them written (T and P 18 KB each for a value
// head, K, Q and K^T 16 KB each for a bf16 key head): 4,096 tokens x 32 heads 224
// MB in 53 us, 4.2 TB/s; with SAVE and 8,192 tokens x 16 heads 325 MB in 64 us,
// 5.1 TB/s; 16,384 tokens x 16 key and 32 value heads 644 MB in 180 to 203 us, 3.2
// to 3.6 TB/s, the rest of it the latency of a workgroup's steps (load, decays,
// products, the inverse's five barriers).
// ---------------------------------------------------------------------------
template <class E, bool DELTA, bool SAVE>
__global__ __launch_bounds__(256) void seq_prep_kernel(const SeqArgs A) {
  constexpr int NP = Parts<E>::n, LDH = D + 8, kPlane = C * LDH;
  const int slot = blockIdx.x, hv = blockIdx.y, hk = hv / A.group;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Chunk ch = find_chunk(A, slot, lane);
  if (ch.len == 0) return;
  const size_t at_ = (size_t)slot * A.hv + hv, atk = (size_t)slot * A.hk + hk;
  const bool first = hv % A.group == 0;
  __shared__ __align__(16) uint16_t sh_k[NP * kPlane];  // K's parts; then (as fp32 [64][LDC]) T
  __shared__ __align__(16) float sh_l[C * LDC];         // L, then P
  __shared__ __align__(16) float sh_m[C * LDC];         // M; above its diagonal blocks: products on their way to T
  __shared__ __align__(16) float sh_a[C];
  __shared__ float sh_b[C];
  float *const sh_t = reinterpret_cast<float *>(sh_k);
  static_assert(sizeof(sh_k) >= sizeof(float) * C * LDC, "T fits over K");
  const int i = lane & 15, g = lane >> 4;

  {
    const int row = tid >> 2, c0 = (tid & 3) * 8;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bf8 f[NP];
#pragma unroll
      for (int n = 0; n < NP; ++n) f[n] = bf8{};
      if (row < ch.len) parts_load<E, NP>(f, at<const E>(A.k, ch.t0 + row, hk) + c0 + 32 * c);
#pragma unroll
      for (int n = 0; n < NP; ++n) *reinterpret_cast<bf8 *>(sh_k + n * kPlane + row * LDH + c0 + 32 * c) = f[n];
    }
  }
  bf8 fq[4][NP];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
#pragma unroll
    for (int n = 0; n < NP; ++n) fq[x][n] = bf8{};
    if (16 * w + i < ch.len) parts_load<E, NP>(fq[x], at<const E>(A.q, ch.t0 + 16 * w + i, hk) + 32 * x + 8 * g);
  }
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
  decay_matrix(sh_l, sh_a, w, lane);
  Acc2 aq[4], ak[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) aq[n] = ak[n] = acc2_zero();
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    bf8 fk[NP];
    if (DELTA || first) frag16<NP>(fk, sh_k, kPlane, LDH, 16 * w, 32 * x, lane);
    if (first) {
      frag_store<NP>(A.w.K + ((atk * 4 + w) * 4 + x) * NP * 512, fk, lane);
      frag_store<NP>(A.w.Q + ((atk * 4 + w) * 4 + x) * NP * 512, fq[x], lane);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (n <= w) {
        bf8 fb[NP];
        frag16<NP>(fb, sh_k, kPlane, LDH, 16 * n, 32 * x, lane);
        mma_parts<NP, NP>(aq[n], fq[x], fb);
        if (DELTA) mma_parts<NP, NP>(ak[n], fk, fb);
      }
    }
  }
  if (first) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // key rows 32 w .. + 31, token steps of 32
      const int mt = 2 * w + (e >> 1), x = e & 1;
      bf8 f[NP];
      frag_gather<NP>(f, sh_k, kPlane, LDH, 16 * mt, 32 * x, lane);
      frag_store<NP>(A.w.KT + ((atk * 8 + mt) * 2 + x) * NP * 512, f, lane);
    }
  }
  __syncthreads();  // L is whole, K's parts are read
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int j = 16 * n + i;
    const float be = sh_b[j];
    const floatx4 qk = aq[n].sum(), kk = ak[n].sum();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r;
      const float lb = sh_l[row * LDC + j] * be;
      sh_l[row * LDC + j] = j <= row ? lb * qk[r] : 0.f;
      if (DELTA && n <= w) sh_m[row * LDC + j] = j < row ? lb * kk[r] : 0.f;
    }
  }
  __syncthreads();
  if (DELTA) invert_unit_lower(sh_t, sh_m, w, lane);
  store_triangles<DELTA>(A, at_, sh_t, sh_l, w, lane);
  if (!SAVE) return;
  // transposes for the backward scan: columns 16 w + i, rows 32 x + 8 g .. + 7
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    if (x < (w >> 1)) continue;
    const int col = 16 * w + i, row = 32 * x + 8 * g;
    float v[8];
    bf8 f[3];
    if (DELTA) {
      const bool in = (row >> 4) >= w;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = in && row + e >= col ? sh_t[(row + e) * LDC + col] : 0.f;
      split8<3>(v, f);
      frag_store<3>(A.w.TT + ((at_ * 4 + w) * 2 + x) * 3 * 512, f, lane);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = sh_l[(row + e) * LDC + col];
    split8<3>(v, f);
    frag_store<3>(A.w.PT + ((at_ * 4 + w) * 2 + x) * 3 * 512, f, lane);
  }
  if (!first) return;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int n = 0; n < NP; ++n)
      *reinterpret_cast<bf8 *>(sh_k + n * kPlane + (16 * w + i) * LDH + 32 * x + 8 * g) = fq[x][n];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int mt = 2 * w + (e >> 1), x = e & 1;
    bf8 f[NP];
    frag_gather<NP>(f, sh_k, kPlane, LDH, 16 * mt, 32 * x, lane);
    frag_store<NP>(A.w.QT + ((atk * 8 + mt) * 2 + x) * NP * 512, f, lane);
  }
}

// ---------------------------------------------------------------------------
// Prep with a decay for every key channel c: the decays do not factor out of
// the products along c,
//   M_ij = beta_j sum_c k_ic k_jc alpha_{j+1,c} .. alpha_{i,c},
// so K, Q and K^T are written with their decays, per value head, in three
// parts.  A quotient of prefix products would overflow; instead, by blocks of
// 16 tokens: with a_i the decays from block I's start to token i, b_j those
// from token j to the end of block J, m those of the blocks between,
//   M_ij = beta_j sum_c (k a)_ic (m (k b))_jc
// are matrix products of factors that are all at most 1 (for alpha <= 1), and
// inside a block the sums are taken directly, the decay running from token to
// token (a lane has a token and 16 channels).  Decays of zero are exact.
// Eight waves, as LDS leaves room for one workgroup a CU (217 us with four):
// 3,001 tokens x 32 heads in fp32 152 us, of which the direct sums are 33 and
// the inverse 8; what it writes for the scan (180 KB a chunk and head) takes
// half of it at the rate of a copy.
// ---------------------------------------------------------------------------
template <class E, bool DELTA>
__global__ __launch_bounds__(512) void seq_prep_kda_kernel(const SeqArgs A) {
  const int slot = blockIdx.x, hv = blockIdx.y, hk = hv / A.group;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Chunk ch = find_chunk(A, slot, lane);
  if (ch.len == 0) return;
  const size_t at_ = (size_t)slot * A.hv + hv;
  __shared__ __align__(16) float sh_k[C * LDD];  // k, then k a; then T
  __shared__ __align__(16) float sh_q[C * LDD];  // q, then q a
  __shared__ __align__(16) float sh_a[C * LDD];  // alpha, then k b
  __shared__ __align__(16) float sh_p[C * LDC];  // P
  __shared__ __align__(16) float sh_m[C * LDC];  // M
  __shared__ __align__(16) float sh_bp[4][D];    // decays of the blocks
  __shared__ __align__(16) float sh_b[C];        // beta
  const int i = lane & 15, g = lane >> 4;
  {
    const int row = tid >> 3, c0 = (tid & 7) * 8, src = ch.t0 + (row < ch.len ? row : 0);
    const float *pa = at<const float>(A.alpha, src, hv) + c0;
    const E *pk = at<const E>(A.k, src, hk) + c0, *pq = at<const E>(A.q, src, hk) + c0;
    const bool on = row < ch.len;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x[8], y[8], z[8];
      load8(pk + 64 * c, x);
      load8(pq + 64 * c, y);
      load8(reinterpret_cast<const F32 *>(pa + 64 * c), z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = on ? x[e] : 0.f;
        y[e] = on ? y[e] : 0.f;
        z[e] = on ? z[e] : 1.f;
      }
      const int o = row * LDD + c0 + 64 * c;
      store8(reinterpret_cast<F32 *>(sh_k + o), x);
      store8(reinterpret_cast<F32 *>(sh_q + o), y);
      store8(reinterpret_cast<F32 *>(sh_a + o), z);
    }
  }
  if (tid < C) {
    const float be = *at<const float>(A.beta, ch.t0 + (tid < ch.len ? tid : 0), hv);
    sh_b[tid] = tid < ch.len ? be : 0.f;
  }
  __syncthreads();
  // ---- the products inside a block: a wave has half of one's tokens, a lane
  // (token i = lane >> 3, channels 16 (lane & 7) .. + 15), token j = i - o
  {
    const int blk = 16 * (w >> 1), ti = 8 * (w & 1) + (lane >> 3), row = blk + ti, c0 = 16 * (lane & 7);
    float d[16], ki[16], qi[16];
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(sh_k + row * LDD + c0 + c);
      const float4 y = *reinterpret_cast<const float4 *>(sh_q + row * LDD + c0 + c);
      ki[c] = x.x; ki[c + 1] = x.y; ki[c + 2] = x.z; ki[c + 3] = x.w;
      qi[c] = y.x; qi[c + 1] = y.y; qi[c + 2] = y.z; qi[c + 3] = y.w;
      d[c] = d[c + 1] = d[c + 2] = d[c + 3] = 1.f;
    }
    const int most = 8 * (w & 1) + 8;
#pragma unroll 2
    for (int o = 0; o < most; ++o) {
      const int j = ti - o < 0 ? 0 : ti - o;  // (tokens before the block: computed, not stored)
      const float *pk = sh_k + (blk + j) * LDD + c0, *pa = sh_a + (blk + j) * LDD + c0;
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(pk + c), y = *reinterpret_cast<const float4 *>(pa + c);
        const float kj[4] = {x.x, x.y, x.z, x.w}, aj[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float t = d[c + e] * kj[e];
          if (DELTA) sk = fmaf(ki[c + e], t, sk);
          sq = fmaf(qi[c + e], t, sq);
          d[c + e] *= aj[e];  // on to the token before
        }
      }
      if (DELTA) sk = row8_sum(sk);
      sq = row8_sum(sq);
      if ((lane & 7) == 0 && o <= ti) {
        const int col = blk + j;
        const float be = sh_b[col];
        sh_p[row * LDC + col] = be * sq;
        if (DELTA && o) sh_m[row * LDC + col] = be * sk;
      }
    }
    // the rest of the diagonal block: zeros
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 2 * (lane & 7) + e;
      if (col > ti) sh_p[row * LDC + blk + col] = 0.f;
      if (DELTA && col >= ti) sh_m[row * LDC + blk + col] = 0.f;
    }
  }
  __syncthreads();
  // ---- k a, q a, k b and the blocks' decays: thread (channel, block)
  {
    const int c = tid & 127, b = tid >> 7;
    float *pk = sh_k + 16 * b * LDD + c, *pq = sh_q + 16 * b * LDD + c, *pa = sh_a + 16 * b * LDD + c;
    float al[16], x = 1.f;
#pragma unroll
    for (int t = 0; t < 16; ++t) al[t] = pa[t * LDD];
#pragma unroll
    for (int t = 15; t >= 0; --t) {
      pa[t * LDD] = pk[t * LDD] * x;  // decays of the tokens behind t
      x *= al[t];
    }
    sh_bp[b][c] = x;
    x = 1.f;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      x *= al[t];
      pk[t * LDD] *= x;
      pq[t * LDD] *= x;
    }
  }
  __syncthreads();
  // ---- products between blocks, and K or Q with the decays from the chunk's
  // start: waves 0 .. 3 take K's rows 16 w .., waves 4 .. 7 Q's
  const int wt = w & 3;
  const bool kwave = w < 4;
  if (DELTA || !kwave) {
    const float *mine = (kwave ? sh_k : sh_q) + (16 * wt + i) * LDD;
    uint16_t *to = (kwave ? A.w.K : A.w.Q) + (at_ * 4 + wt) * 4 * 3 * 512;
    floatx4 acc[3];
#pragma unroll
    for (int n = 0; n < 3; ++n) acc[n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
      const int c0 = 32 * x + 8 * g;
      float k[8], m[8], v[8];
      bf8 fk[3], f[3];
      load8(reinterpret_cast<const F32 *>(mine + c0), k);
      split8<3>(k, fk);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = 1.f;  // decays of the blocks between
#pragma unroll
      for (int n = 2; n >= 0; --n) {
        if (n >= wt) continue;
        load8(reinterpret_cast<const F32 *>(sh_a + (16 * n + i) * LDD + c0), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= m[e];
        split8<3>(v, f);
        mma_into<3, 3>(acc[n], fk, f);
        load8(reinterpret_cast<const F32 *>(&sh_bp[n][c0]), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] *= v[e];
      }
      // m: now the decays of all blocks before the wave's
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] *= m[e];
      split8<3>(k, fk);
      frag_store<3>(to + x * 3 * 512, fk, lane);
    }
    float *const out = kwave ? sh_m : sh_p;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      if (n >= wt) continue;
      const float be = sh_b[16 * n + i];
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(16 * wt + 4 * g + r) * LDC + 16 * n + i] = be * acc[n][r];
    }
    // P's blocks above the diagonal in the steps that are stored: zeros
    if (!kwave)
      for (int n = wt + 1; n < 4; ++n)
        *reinterpret_cast<float4 *>(sh_p + (16 * wt + i) * LDC + 16 * n + 4 * g) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // ---- K^T with beta and the decays to the chunk's end: key rows 16 w .. + 15
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int mt = w, c = 16 * mt + i;
    // tokens 32 x + 8 g .. + 7 lie in block 2 x + (g >> 1)
    const float b1 = sh_bp[1][c], b2 = sh_bp[2][c], b3 = sh_bp[3][c];
    const int blk = 2 * x + (g >> 1);
    const float rest = blk == 0 ? b1 * b2 * b3 : (blk == 1 ? b2 * b3 : (blk == 2 ? b3 : 1.f));
    float v[8];
    bf8 f[3];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int tok = 32 * x + 8 * g + t;
      v[t] = sh_b[tok] * rest * sh_a[tok * LDD + c];
    }
    split8<3>(v, f);
    frag_store<3>(A.w.KT + ((at_ * 8 + mt) * 2 + x) * 3 * 512, f, lane);
  }
  if (tid < D) A.w.dec[at_ * 2 * C + tid] = (sh_bp[0][tid] * sh_bp[1][tid]) * (sh_bp[2][tid] * sh_bp[3][tid]);
  __syncthreads();
  if (DELTA) invert_unit_lower(sh_k, sh_m, w, lane);
  if (kwave) store_triangles<DELTA>(A, at_, sh_k, sh_p, w, lane);
}

// ---------------------------------------------------------------------------
// Scan: one workgroup per (sequence, value head, block of CB columns), chunk
// after chunk.  Wave w takes token tile w (16 rows) of the products with 64
// rows and rows 32 w .. + 31 of the state, whose block stays in its
// accumulators; column tile n of the block holds columns NT i + n, so that a
// lane's NT columns are neighbours in memory.
// The operands that do not depend on the state (K, Q, T, P, K^T) are private
// to a wave: they come straight from global memory in fragment order (a
// wave's load is one run of 1 KiB; rows of the inputs themselves would be
// sixteen pieces of 64 bytes and cost the address path four times as long),
// each reloaded for the next chunk right after its use, so the loads run
// behind the rest of the chunk.  What the waves share (S, X, U) goes through
// LDS as bf16 parts; three barriers a chunk.
// Bound by the chain of a chunk (K S, T X, K^T U and the barriers between), 1.9
// us with 16 columns: a prompt of 4,096 tokens x 32 heads 124 us; 16,384 tokens
// in 24 sequences x 32 heads, where two workgroups share a CU, 338 to 405 us.
// Eight waves, four of them for the output, were no faster (142 us).
// ---------------------------------------------------------------------------
// Workgroups that share a CU: the wide fp16 scan is held to the registers of two
// (256; it would take 260): 5,000 tokens in 19 sequences x 16 heads 104 us, 129
// with one
template <class E, bool KDA, int CB>
constexpr int scan_per_cu() { return !KDA && CB == 32 && Parts<E>::n == 2 ? 2 : 1; }

template <class E, bool KDA, bool DELTA, bool SAVE, int CB>
__global__ __launch_bounds__(256, (scan_per_cu<E, KDA, CB>())) void seq_scan_kernel(const SeqArgs A) {
  constexpr int NT = CB / 16, kBlocks = D / CB;
  // parts of K, Q and K^T; with a decay a channel they hold decays, per value head
  constexpr int NP = KDA ? 3 : Parts<E>::n;
  constexpr int FS = 4 * NT, FX = 2 * NT;  // fragments of a part of [CB][128], [CB][64]
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups b, b + 8, .. run on one XCD: the column blocks of one head
  // are placed there, so that its L2 serves their common operands
  const int64_t b = blockIdx.x;
  const int64_t place = (b / (8 * kBlocks)) * 8 + (b & 7);
  if (place >= (int64_t)A.seqs * A.hv) return;
  const int seq = seq_place(A, (int)(place / A.hv), gridDim.x, lane);
  const int hv = (int)(place % A.hv);
  const int64_t unit = (int64_t)seq * A.hv + hv;
  const int hk = KDA ? hv : hv / A.group, heads_k = KDA ? A.hv : A.hk;
  const int start = seq_start(A, seq), end = seq_end(A, seq, start);
  __shared__ __align__(16) uint16_t sh_s[3 * FS * 512];              // S, [column][key row]
  __shared__ __align__(16) uint16_t sh_x[DELTA ? 3 * FX * 512 : 8];  // X, [column][token]
  __shared__ __align__(16) uint16_t sh_u[KDA ? 8 : 3 * FX * 512];   // U
  __shared__ __align__(16) uint16_t sh_ku[3 * FX * 512];             // kappa * U; with a decay a channel U
  __shared__ __align__(16) float sh_dec[2][2 * C];                   // decays, of this chunk and the next
  const int i = lane & 15, g = lane >> 4, tok = 16 * w + 4 * g;
  const int col = (int)((b >> 3) % kBlocks) * CB + NT * i;  // the lane's first column

  floatx4 s[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x[NT] = {};
      if (A.S0) load_n<NT>(A.S0 + (unit * D + 32 * w + 16 * m + 4 * g + r) * D + col, x);
#pragma unroll
      for (int n = 0; n < NT; ++n) s[m][n][r] = x[n];
    }
  wait_loads();  // the loop below counts its own loads only

  // Loads stand at fixed places: with a branch around them the compiler could
  // not count what is in flight and would wait for all of it.  A row past the
  // end is the chunk's first row instead; its X is set to zero and its columns
  // of P and K^T are zero.  V's pointer moves on from chunk to chunk (`move`:
  // 1, or 0 where there is none: then the last chunk is read again).
  bf8 fk[4][NP], fq[4][NP], fT[2][3], fP[2][3], fKT[2][2][NP];
  E v[4][NT];
  float dec;  // thread t < 128: value t of the next chunk's decays
  const int slot0 = start / C + seq;
  const int chunks = (end - start + C - 1) / C;
  const E *pV = at<const E>(A.v, start + tok, hv) + col;
  const int64_t backV = tok * A.v.ts;
  auto load_k = [&](int c) {
    const size_t f = (((size_t)(slot0 + c) * heads_k + hk) * 4 + w) * 4 * NP * 512;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (DELTA) frag_load<NP>(fk[x], A.w.K + f + x * NP * 512, lane);
      frag_load<NP>(fq[x], A.w.Q + f + x * NP * 512, lane);
    }
  };
  auto load_v = [&](int c, int move) {
    const int len = end - start - c * C;
    pV += move * (C * A.v.ts);
#pragma unroll
    for (int r = 0; r < 4; ++r) load_raw<NT>(tok + r < len ? pV + r * A.v.ts : pV - backV, v[r]);
    dec = A.w.dec[((size_t)(slot0 + c) * A.hv + hv) * 2 * C + (threadIdx.x & 127)];
  };
  auto load_T = [&](int c) {
    const uint16_t *p = A.w.T + (((size_t)(slot0 + c) * A.hv + hv) * 4 + w) * 2 * 3 * 512;
    if (DELTA) {
      frag_load<3>(fT[0], p, lane);
      if (w >= 2) frag_load<3>(fT[1], p + 3 * 512, lane);
    }
  };
  auto load_P = [&](int c) {
    const uint16_t *p = A.w.P + (((size_t)(slot0 + c) * A.hv + hv) * 4 + w) * 2 * 3 * 512;
    frag_load<3>(fP[0], p, lane);
    if (w >= 2) frag_load<3>(fP[1], p + 3 * 512, lane);
  };
  auto load_KT = [&](int c) {
    const uint16_t *p = A.w.KT + (((size_t)(slot0 + c) * heads_k + hk) * 8 + 2 * w) * 2 * NP * 512;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int x = 0; x < 2; ++x) frag_load<NP>(fKT[m][x], p + (2 * m + x) * NP * 512, lane);
  };
  if (chunks) {
    load_k(0);
    load_v(0, 0);
    load_T(0);
    load_KT(0);
    load_P(0);
    if (threadIdx.x < 2 * C) sh_dec[0][threadIdx.x] = dec;
  }
  for (int c = 0; c < chunks; ++c) {
    const int t0 = start + c * C, len = end - t0;
    const int move = c + 1 < chunks ? 1 : 0, next = c + move;
    const size_t at_ = (size_t)(slot0 + c) * A.hv + hv;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        frag_share<3, FS>(sh_s, 4 * n + w, m, lane, s[m][n][0], s[m][n][1], s[m][n][2], s[m][n][3]);
      if (SAVE) {
#pragma unroll
        for (int n = 0; n < NT; ++n) store_quad(A.w.S + at_ * D * D, 8 * w + 4 * m + g, col + n, s[m][n]);
      }
    }
    lds_barrier();
    Acc2 yk[NT], yq[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) yk[n] = yq[n] = acc2_zero();
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        bf8 fs[3];
        frag_get<3, FS>(fs, sh_s, 4 * n + x, lane);
        if (DELTA) mma_parts<NP, 3>(yk[n], fk[x], fs);
        mma_parts<NP, 3>(yq[n], fq[x], fs);
      }
    load_k(next);
    const float *sd = sh_dec[c & 1];
    float gm[4], kp[4], la[2][4];
    if (KDA) {  // a decay for every row of the state, none for the tokens
#pragma unroll
      for (int r = 0; r < 4; ++r) gm[r] = kp[r] = 1.f;
#pragma unroll
      for (int m = 0; m < 2; ++m) load4(reinterpret_cast<const F32 *>(sd + 32 * w + 16 * m + 4 * g), la[m]);
    } else {
      load4(reinterpret_cast<const F32 *>(sd + tok), gm);
      load4(reinterpret_cast<const F32 *>(sd + C + tok), kp);
#pragma unroll
      for (int r = 0; r < 4; ++r) la[0][r] = la[1][r] = sd[C - 1];
    }
    floatx4 u[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const floatx4 y = yk[n].sum();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = to_f(v[r][n]);
        u[n][r] = tok + r < len ? (DELTA ? x - gm[r] * y[r] : x) : 0.f;
        yq[n].a[r] = gm[r] * (yq[n].a[r] + yq[n].b[r]);
        yq[n].b[r] = 0.f;
      }
    }
    load_v(next, move);
    if (DELTA) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        frag_share<3, FX>(sh_x, 2 * n + (w >> 1), w & 1, lane, u[n][0], u[n][1], u[n][2], u[n][3]);
      lds_barrier();
      Acc2 y[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) y[n] = acc2_zero();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (2 * x <= w) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            bf8 fx[3];
            frag_get<3, FX>(fx, sh_x, 2 * n + x, lane);
            mma_parts<3, 3>(y[n], fT[x], fx);
          }
        }
      }
      load_T(next);
#pragma unroll
      for (int n = 0; n < NT; ++n) u[n] = y[n].sum();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      frag_share<3, FX>(sh_ku, 2 * n + (w >> 1), w & 1, lane, kp[0] * u[n][0], kp[1] * u[n][1], kp[2] * u[n][2],
                        kp[3] * u[n][3]);
      if (!KDA) frag_share<3, FX>(sh_u, 2 * n + (w >> 1), w & 1, lane, u[n][0], u[n][1], u[n][2], u[n][3]);
    }
    if (SAVE) {
#pragma unroll
      for (int n = 0; n < NT; ++n) store_quad(A.w.U + at_ * C * D, 4 * w + g, col + n, u[n]);
    }
    lds_barrier();
    Acc2 ds[2][NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) ds[m][n] = acc2_zero();
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        bf8 fu[3];
        frag_get<3, FX>(fu, sh_ku, 2 * n + x, lane);
#pragma unroll
        for (int m = 0; m < 2; ++m) mma_parts<NP, 3>(ds[m][n], fKT[m][x], fu);
      }
    load_KT(next);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (2 * x <= w) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf8 fu[3];
          frag_get<3, FX>(fu, KDA ? sh_ku : sh_u, 2 * n + x, lane);
          mma_parts<3, 3>(yq[n], fP[x], fu);
        }
      }
    }
    load_P(next);
    if (threadIdx.x < 2 * C) sh_dec[(c + 1) & 1][threadIdx.x] = dec;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const floatx4 d = ds[m][n].sum();
#pragma unroll
        for (int r = 0; r < 4; ++r) s[m][n][r] = fmaf(s[m][n][r], la[m][r], d[r]);
      }
    E *o = at<E>(A.o, t0 + tok, hv) + col;
    E x[4][NT];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) x[r][n] = from_f<E>(yq[n].a[r] + yq[n].b[r]);
    if (len >= C) {  // a whole chunk: no branch for every row
#pragma unroll
      for (int r = 0; r < 4; ++r) store_raw<NT>(o + r * A.o.ts, x[r]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (tok + r < len) store_raw<NT>(o + r * A.o.ts, x[r]);
    }
  }
  if (A.S) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] = s[m][n][r];
        store_n<NT>(A.S + (unit * D + 32 * w + 16 * m + 4 * g + r) * D + col, x);
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
  // each token's chain.  4 tokens a sequence: 6.3 and 11.0 us at 64 states,
  // 8.8 and 11.6 at 128, 14.0 and 13.0 at 256, 24.1 and 20.6 at 512
  // (one column, four columns)
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

template <class E, bool KDA, bool DELTA, bool SAVE>
hipError_t chunked(const SeqArgs &a, hipStream_t stream) {
  const int64_t units = ((int64_t)a.seqs * a.hv + 7) / 8 * 8;
  const dim3 slots((unsigned)a.slots, a.hv);
  if constexpr (KDA)
    hipLaunchKernelGGL((seq_prep_kda_kernel<E, DELTA>), slots, dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((seq_prep_kernel<E, DELTA, SAVE>), slots, dim3(256), 0, stream, a);
  // (the scan wide and narrow: a prompt of 4,096 tokens x 32 heads, 128 or 256
  // workgroups, 174 and 124 us; 24 ragged sequences x 32 heads, many times what
  // the chip holds, 338 and 486.  Both launches of 1,536 tokens in bf16: 32
  // heads 90 and 74 us, 48 heads 96 and 94, 64 heads 102 and 105, 128 heads 201
  // and 257.  Operands of two or three parts leave the narrow scan one workgroup
  // a CU, and 33 to 63 states two rounds of them: fp16 48 heads 133 and 151, fp32
  // 203 and 244, and 32 heads 120 and 88, 153 and 124)
  if (scan_wide(a, 256))
    hipLaunchKernelGGL((seq_scan_kernel<E, KDA, DELTA, SAVE, 32>), dim3((unsigned)(units * 4)), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((seq_scan_kernel<E, KDA, DELTA, SAVE, 16>), dim3((unsigned)(units * 8)), dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <class E>
hipError_t chunked(const SeqArgs &a, bool kda, bool delta, hipStream_t stream) {
  const bool save = a.w.S != nullptr;
  if (kda) return delta ? chunked<E, true, true, false>(a, stream) : chunked<E, true, false, false>(a, stream);
  if (delta) return save ? chunked<E, false, true, true>(a, stream) : chunked<E, false, true, false>(a, stream);
  return save ? chunked<E, false, false, true>(a, stream) : chunked<E, false, false, false>(a, stream);
}
hipError_t launch_seq_chunked(const SeqArgs &a, int dtype, bool kda, bool delta, hipStream_t stream) {
  return dtype == 0 ? chunked<F32>(a, kda, delta, stream)
         : dtype == 1 ? chunked<BF16>(a, kda, delta, stream)
                      : chunked<F16>(a, kda, delta, stream);
}

}  // namespace lq
