// Gradient of the selective state space scan over packed sequences (gfx950).
// With v = dt + bias, d = softplus(v), a_n = e^(d A_n), p = sum_n C_n h_n + D x,
// s = 1 / (1 + e^-z) and dp = dy z s, backwards over a sequence's tokens (G: the
// gradient of the state behind a token, g: of the state after it),
//   g_n = G_n + C_n dp,  G_n <- a_n g_n,  e_n = g_n a_n h_n(before)
//   dC_n = sum_c dp h_n,  dB_n = sum_c g_n d x,  dA_n = sum_t e_n d
//   dx = d sum_n g_n B_n + D dp,  dd = sum_n e_n A_n + x sum_n g_n B_n
//   ddt = dd / (1 + e^-v),  dbias = sum_t ddt,  dD = sum_t dp x
//   dz = dy p s (1 + z (1 - s))
//
// As forward, a lane holds a channel and a wave 64 channels and a chunk; the
// gradients behind every chunk come from the chunks' own, begun from zero, as the
// states do.  The forward pass left the states before every fourth token: such a run
// is computed again from them, its states stay in registers, and it is taken
// backwards.
//
// Bound by vector instructions (of the time that its waves run, two a SIMD with 16
// states, they take 89 % of the issue slots; of the whole launch, as some waves end
// before others, 72 %): each token's decays
// are computed twice, and with the sums over the channels a state takes some 20
// instructions.  8,192 tokens x 2,048 channels x 16 states in bf16: chunks from zero
// 61 us, between them 10, main kernel 220, the sums of its waves 9.  1,021 tokens x
// 1,111 channels x 8 states in fp32: 9 + 5 + 22 + 4.  (As forward: with a warm chip;
// pairs of figures below were measured one against the other, most of them without.)
// With 32 states a lane's arrays do not fit the 256 registers that vector instructions
// take: 84 to 105 of them lie in accumulator registers and are copied, and up to 275
// scalars (fp32 with a gate; 13 to 47 otherwise) in lanes of vector registers.
#include "lq_scan_device.h"

namespace lq {

// The chunks' gradients behind from zero: what comes out of their first token.
template <class E, int N, bool GATE>
__global__ __launch_bounds__(256, N > 16 ? 3 : 4) void scan_grad_local_kernel(const ScanArgs A, int tiles, int64_t waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;
  const int slot = (int)(wave / tiles), tile = (int)(wave % tiles), tg = (A.per + 63) >> 6;
  const ScanChunk k = scan_chunk(A, A.part, slot, lane);
  if (!k.any || k.c == 0) return;  // nothing comes before the first chunk
  const ScanTile ch = scan_tile(A, tile / tg, tile % tg, lane);
  const int64_t width = A.channels;
  float a2[N], sum = 0.f;
  ScanState<N> g;
  scan_decays<N>(A, ch.c, a2);
  scan_zero<N>(g);
  const float bias = A.bias ? A.bias[ch.c] : 0.f;
  constexpr int ahead = 8;
  E rd[ahead], ry[ahead], rz[ahead];
  ScanLanes<E, N> rc[ahead];
  const auto load = [&](int t) {  // tokens t, t - 1 ..
    const ScanArgs &P = scan_args();
    const E *dt = at<const E>(P.dt, t, 0), *dy = at<const E>(P.dy, t, 0), *z = GATE ? at<const E>(P.z, t, 0) : dy;
    const E *cc = at<const E>(P.C, t, ch.g);
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      rd[u] = lane_load(dt, ch.c);
      ry[u] = lane_load(dy, ch.c);
      rc[u].load(cc, lane);
      if (GATE) rz[u] = lane_load(z, ch.c);
      if (t - u > k.t0) {
        dt -= P.dt.ts;
        dy -= P.dy.ts;
        cc -= P.C.ts;
        if (GATE) z -= P.z.ts;
      }
    }
  };
  load(k.t1 - 1);
  for (int t = k.t1 - 1; t >= k.t0; t -= ahead) {
    float fd[ahead], fy[ahead], fz[ahead], fc[ahead][ScanLanes<E, N>::rows];
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
#pragma unroll
      for (int r = 0; r < ScanLanes<E, N>::rows; ++r) fc[u][r] = to_f(rc[u].e[r]);
      fd[u] = to_f(rd[u]) + bias;
      fy[u] = to_f(ry[u]);
      fz[u] = GATE ? to_f(rz[u]) : 0.f;
    }
    // (as forward: converted before the next loads begin)
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      asm volatile("" : "+v"(fd[u]), "+v"(fy[u]));
      if (GATE) asm volatile("" : "+v"(fz[u]));
#pragma unroll
      for (int r = 0; r < ScanLanes<E, N>::rows; ++r) asm volatile("" : "+v"(fc[u][r]));
    }
    if (t - ahead >= k.t0) load(t - ahead);
    scan_steps<E>(A, fd);
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      if (t - u < k.t0) break;
      const float d = fd[u], dp = GATE ? fy[u] * (fz[u] * sigmoid_for<E>(fz[u])) : fy[u];
      sum += d;
      scan_add_outer<N>(g, fc[u], dp);
#pragma unroll
      for (int n = 0; n < N; ++n) g[n >> 2][n & 3] *= __builtin_amdgcn_exp2f(d * a2[n]);
    }
  }
  if (!ch.on) return;
  scan_store_fours<N>(A.carry + (int64_t)slot * N * width, (int)width, lane_offset(true, ch.c, 16), g);
  A.sum[slot * width + ch.c] = sum;
}

// The gradients behind every chunk of the sequences with several, over the
// chunks' own, as the states forward, the last chunk first.  dS is copied behind
// the last chunk, as dS0 may lie over it.
__global__ __launch_bounds__(256) void scan_grad_carry_kernel(const ScanArgs A, int states, int blocks) {
  const ScanCarry t = scan_carry(A, states, blocks);
  if (!t.any) return;
  const int chunks = t.chunks;
  const int64_t width = A.channels, step = states * width;
  const float a2 = A.A[t.state] * kLog2e;
  float g = A.dS ? A.dS[t.i * step + t.state] : 0.f;
  float *carry = A.carry + t.at;
  const float *sum = A.sum + t.at_sum;
  for (int k = chunks - 1; k >= 0; k -= kCarryAhead) {
    float v[kCarryAhead], s[kCarryAhead];
#pragma unroll
    for (int u = 0; u < kCarryAhead; ++u) {
      const int64_t at = max(k - u, 1);  // (chunk 0 has none: nothing comes before it)
      v[u] = carry[at * step];
      s[u] = sum[at * width];
    }
#pragma unroll
    for (int u = 0; u < kCarryAhead; ++u) {
      if (k - u < 0) break;
      carry[(k - u) * step] = g;
      g = fmaf(__builtin_amdgcn_exp2f(s[u] * a2), g, v[u]);
    }
  }
}

// Sums of many registers over the 16 lanes of a row at once: two registers become
// one, in which half of the lanes go on with the one and half with the other.
// Two instructions a step: a masked add writes the one's sum into half of the lanes
// of the other's.  The last two steps would need three, as the mask is of four
// lanes; the sixteen lanes that are left a sum meet in LDS.  8,192 tokens x 2,048
// channels with all four steps by selects, three instructions each, 281 us for 256;
// four-lane sums by products with ones on the matrix pipe, whose instructions wait
// for it and for one another, 350 for 296; the values through LDS, a lane adding
// four sums over eight channels, 302 for 290: fewer instructions, but waits that two
// waves a SIMD do not hide.
// Lanes with bits 3 and 2 of (0, 0), (1, 0), (0, 1), (1, 1) come to hold the sums of
// v[0], v[1], v[2], v[3] over four lanes: those of either bit 3 with this lane's bits 2
// to 0, and those with all three of them inverted (the half row mirrored).  So the lanes
// with one pair of bits 3 and 2, whose bits 1 and 0 differ, share the sixteen out among
// them, and the sum over the four of them is the whole.  (All lanes
// are active; the s_nops keep the two cycles between writing a register and
// reading it across lanes.)
__device__ __forceinline__ float fold4(const float (&v)[4]) {
  float x, y, r;
  asm("s_nop 1\n"
      "v_add_f32_dpp %0, %3, %3 row_ror:8 row_mask:0xf bank_mask:0xf\n"
      "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xf\n"
      "v_add_f32_dpp %0, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xc\n"
      "v_add_f32_dpp %1, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n"
      "s_nop 1\n"
      "v_add_f32_dpp %2, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n"
      "v_add_f32_dpp %2, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xa"
      : "=&v"(x), "=&v"(y), "=&v"(r)
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]));
  return r;
}
__device__ __forceinline__ int fold_place(int lane) { return 2 * (lane >> 2 & 1) + (lane >> 3 & 1); }

// The waves share nothing (a workgroup whose waves met after every run of tokens, to
// write a fourth of the sums, was no faster): each writes its sums over its channels
// for every token, as fold4 places them, sum 4 q + place at place * states / 2 + q.
template <class E, int N, bool GATE>
__global__ __launch_bounds__(256, scan_grad_waves(N)) void scan_grad_kernel(const ScanArgs A, int tiles, int64_t waves) {
  constexpr int sub = kScanSub, row = 2 * N + 4, Q = N / 2;  // Q: fours of sums, dB's and dC's
  __shared__ float sh[4][sub][16][row];
  const int lane = threadIdx.x & 63, w4 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wave = w4 + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;
  const int slot = (int)(wave / tiles), tile = (int)(wave % tiles), tg = (A.per + 63) >> 6, group = tile / tg;
  const ScanChunk k = scan_chunk(A, A.chunk, slot, lane);
  const ScanTile ch = scan_tile(A, group, tile % tg, lane);
  const int64_t width = A.channels;
  float a2[N], dskip = 0.f, dbias = 0.f;
  ScanState<N> g, dA;
  scan_zero<N>(g);
  scan_zero<N>(dA);
  if (k.any) {
    scan_decays<N>(A, ch.c, a2);
    if (ch.on) {
      if (k.chunks > 1)
        scan_load_fours<N>(A.carry + scan_last_part(A, k) * N * width, width, ch.c, g);
      else if (A.dS)
        scan_load_rows<N>(A.dS, k.i * width + ch.c, g);
    }
    const float bias = A.bias ? A.bias[ch.c] : 0.f, skip = A.skip ? A.skip[ch.c] : 0.f;
    const int len = k.t1 - k.t0, runs = (len + sub - 1) / sub;
    const int64_t first = k.start / sub + k.i + (k.t0 - k.start) / sub;
    const int place = fold_place(lane), row_bytes = (int)(width * sizeof(E));
    const uint32_t off = lane_offset(ch.on, ch.c, sizeof(E));
    E rx[sub], rd[sub], ry[sub], rz[sub];
    ScanLanes<E, N> rb[sub - 1], rc[sub];
    ScanState<N> start;  // the states before the run's tokens
    const auto load = [&](int r) {
      const int t = k.t0 + r * sub;
      const ScanArgs &P = scan_args();
      const E *x = at<const E>(P.x, t, 0), *dt = at<const E>(P.dt, t, 0), *dy = at<const E>(P.dy, t, 0);
      const E *z = GATE ? at<const E>(P.z, t, 0) : x, *b = at<const E>(P.B, t, group), *cc = at<const E>(P.C, t, group);
#pragma unroll
      for (int u = 0; u < sub; ++u) {
        rx[u] = lane_load(x, ch.c);
        if (u + 1 < sub) rb[u].load(b, lane);
        rc[u].load(cc, lane);
        rd[u] = lane_load(dt, ch.c);
        ry[u] = lane_load(dy, ch.c);
        if (GATE) rz[u] = lane_load(z, ch.c);
        if (t + u + 1 < k.t1) {
          x += P.x.ts;
          b += P.B.ts;
          cc += P.C.ts;
          dt += P.dt.ts;
          dy += P.dy.ts;
          if (GATE) z += P.z.ts;
        }
      }
    };
    const auto load_start = [&](int r) {
      scan_load_fours<N>(scan_args().check + (first + r) * N * width, width, ch.c, start);
    };
    if (runs) {
      load(runs - 1);
      load_start(runs - 1);
    }
    for (int r = runs - 1; r >= 0; --r) {
      const int t = k.t0 + r * sub, n_t = min(sub, k.t1 - t);
      float fx[sub], fd[sub], fy[sub], fz[sub], slope[sub];
      float fb[sub - 1][ScanLanes<E, N>::rows], fc[sub][ScanLanes<E, N>::rows];
      ScanState<N> hist[sub];
#pragma unroll
      for (int u = 0; u < sub; ++u) {
#pragma unroll
        for (int i = 0; i < ScanLanes<E, N>::rows; ++i) {
          fc[u][i] = to_f(rc[u].e[i]);
          if (u + 1 < sub) fb[u][i] = to_f(rb[u].e[i]);
        }
        fx[u] = ch.on ? to_f(rx[u]) : 0.f;
        fd[u] = to_f(rd[u]) + bias;
        fy[u] = ch.on ? to_f(ry[u]) : 0.f;
        fz[u] = GATE ? to_f(rz[u]) : 0.f;
      }
#pragma unroll
      for (int q = 0; q < N / 4; ++q) hist[0][q] = start[q];
      // the output rows of the run's last token, and the way to the one before:
      // reading them for each token would wait for the rows of B and C on their way
      const ScanArgs &P = scan_args();
      int64_t step_x = P.dx.ts, step_t = P.ddt.ts, step_z = GATE ? P.dz.ts : 0;
      E *out_x = at<E>(P.dx, t + n_t - 1, 0), *out_t = at<E>(P.ddt, t + n_t - 1, 0);
      E *out_z = GATE ? at<E>(P.dz, t + n_t - 1, 0) : nullptr;
      asm volatile("" : "+s"(step_x), "+s"(step_t), "+s"(step_z), "+s"(out_x), "+s"(out_t), "+s"(out_z));
      // the rows of B and C, of the tokens forwards and back
      const E *row_b = at<const E>(P.B, t + n_t - 1, group), *row_c = at<const E>(P.C, t + n_t - 1, group);
      int64_t step_b = P.B.ts, step_c = P.C.ts;
      asm volatile("" : "+s"(step_b), "+s"(step_c), "+s"(row_b), "+s"(row_c));
      ScanRow<E, N> B, C;
      B.load(row_b);
      C.load(row_c);
      scan_steps<E>(A, fd, slope);
#pragma unroll
      for (int u = 0; u + 1 < sub; ++u) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < N; ++n)
          hist[u + 1][n >> 2][n & 3] = __builtin_amdgcn_exp2f(fd[u] * a2[n]) * hist[u][n >> 2][n & 3];
        scan_add_outer<N>(hist[u + 1], fb[u], fd[u] * fx[u]);
      }
#pragma unroll
      for (int u = sub - 1; u >= 0; --u) {
        __builtin_amdgcn_sched_barrier(0);
        if (u == 1 && r > 0) {  // into the registers of the tokens that are done
          load(r - 1);
          load_start(r - 1);
        }
        if (u >= n_t) continue;  // past the chunk's end
        const ScanRow<E, N> b = B, cc = C;
        if (u > 0) {
          row_b -= step_b;
          row_c -= step_c;
          B.load(row_b);
          C.load(row_c);
        }
        float d = fd[u];
        // the decays again, but for those used next: keeping the run's spilled (643 us
        // for 294 of 8,192 tokens x 2,048 channels)
        if (u + 2 != sub || N > 16) asm("" : "+v"(d));
        const float xd = d * fx[u];
        float s = 0.f, dp = fy[u];
        if (GATE) {
          s = sigmoid_for<E>(fz[u]);
          dp *= fz[u] * s;
        }
        float p = skip * fx[u], gb = 0.f, ea = 0.f;
        float fold[Q];
        scan_add_outer<N>(g, fc[u], dp);
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
          float vb[4], vc[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int n = 4 * q + m;
            const float a = __builtin_amdgcn_exp2f(d * a2[n]);
            const float h = u + 1 < sub ? hist[u + 1 < sub ? u + 1 : u][q][m] : fmaf(a, hist[u][q][m], xd * b[n]);
            p = fmaf(cc[n], h, p);
            const float gn = g[q][m];
            gb = fmaf(gn, b[n], gb);
            g[q][m] = gn * a;
            const float e = g[q][m] * hist[u][q][m];
            ea = fmaf(e, a2[n], ea);
            dA[q][m] = fmaf(e, d, dA[q][m]);
            vb[m] = gn * xd;
            vc[m] = dp * h;
          }
          fold[q] = fold4(vb);
          fold[N / 4 + q] = fold4(vc);
        }
#pragma unroll
        for (int q = 0; q < Q; q += 4) {
          const floatx4 four = {fold[q], fold[q + 1], fold[q + 2], fold[q + 3]};
          *reinterpret_cast<floatx4 *>(&sh[w4][u][(lane >> 4) * 4 + (lane & 3)][place * Q + q]) = four;
        }
        const float ddt = fmaf(gb, fx[u], ea * kLn2) * slope[u];
        const float dz = fy[u] * p * (s * fmaf(fz[u], 1.f - s, 1.f));
        dskip = fmaf(dp, fx[u], dskip);
        dbias += ddt;
        lane_store(out_x, row_bytes, off, from_f<E>(fmaf(gb, d, skip * dp)));
        lane_store(out_t, row_bytes, off, from_f<E>(ddt));
        if (GATE) lane_store(out_z, row_bytes, off, from_f<E>(dz));
        out_x -= step_x;
        out_t -= step_t;
        if (GATE) out_z -= step_z;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // sixteen lanes a token, the sixteen shares of their sums in order
      constexpr int V = N / 8;
      const int u = lane >> 4, n = (lane & 15) * V;
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[e] = sh[w4][u][0][n + e];
#pragma unroll
        for (int i = 1; i < 16; ++i) y[e] += sh[w4][u][i][n + e];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (u < n_t) {
        float *to = A.part_bc + ((int64_t)tile * A.tokens + t + u) * 2 * N + n;
#pragma unroll
        for (int e = 0; e < V; ++e) to[e] = y[e];
      }
    }
    if (A.dS0 && k.c == 0 && ch.on) scan_store_rows<N>(A.dS0, k.i * width + ch.c, g);
  }
  if (!ch.on) return;
  // (slots without a chunk: zeros)
  float *part = A.part_a + (int64_t)slot * (N + 2) * width;
#pragma unroll
  for (int n = 0; n < N; ++n) part[n * width + ch.c] = dA[n >> 2][n & 3];
  part[N * width + ch.c] = dskip;
  part[(N + 1) * width + ch.c] = dbias;
}

// The sums of the waves and chunks, added in order, in one launch.  The first
// `blocks_bc` workgroups: dB and dC over the waves of a group, thread (token, group,
// place).  The others: dA, dD and dbias over the chunks, workgroup
// (64 channels, state), wave (a share of the slots).
template <class E>
__global__ __launch_bounds__(512) void scan_grad_sum_kernel(const ScanArgs A, int states, int tiles_group,
                                                            int64_t blocks_bc) {
  __shared__ float sh[8][64];
  if (blockIdx.x < blocks_bc) {
    const int64_t id = (int64_t)blockIdx.x * 512 + threadIdx.x;
    const int n = (int)(id % (2 * states)), g = (int)(id / (2 * states) % A.groups);
    const int64_t t = id / (2 * states) / A.groups;
    if (t < A.cu[0] || t >= A.cu[A.seqs] || t >= A.tokens) return;  // of no sequence
    float x = 0.f;
#pragma unroll 8
    for (int b = 0; b < tiles_group; ++b)
      x += A.part_bc[(((int64_t)g * tiles_group + b) * A.tokens + t) * 2 * states + n];
    const int half = states / 2, s = 4 * (n % half) + n / half;
    if (s < states)
      at<E>(A.dB, t, g)[s] = from_f<E>(x);
    else
      at<E>(A.dC, t, g)[s - states] = from_f<E>(x);
    return;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t block = blockIdx.x - blocks_bc;
  const int tiles = (A.channels + 63) >> 6, k = (int)(block / tiles);
  const int64_t width = A.channels, c = (block % tiles) * 64 + lane;
  float x = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int64_t s = w; s < A.slots; s += 8) x += A.part_a[(s * (states + 2) + k) * width + c];
  }
  sh[w][lane] = x;
  __syncthreads();
  if (w || c >= width) return;
  float y = 0.f;
#pragma unroll
  for (int v = 0; v < 8; ++v) y += sh[v][lane];
  if (k < states)
    A.dA[c * states + k] = y;
  else if (k == states && A.dskip)
    A.dskip[c] = y;
  else if (k > states && A.dbias)
    A.dbias[c] = y;
}

template <class E, int N>
static hipError_t scan_back(const ScanArgs &a, hipStream_t stream) {
  const int64_t tiles = scan_tiles(a.channels, a.groups), waves = tiles * a.slots;
  if (a.tokens > a.chunk) {
    const int64_t parts = tiles * scan_slots(a.tokens, a.seqs, a.part);
    const dim3 grid((unsigned)((parts + 3) / 4));
    if (a.z.ptr)
      hipLaunchKernelGGL((scan_grad_local_kernel<E, N, true>), grid, dim3(256), 0, stream, a, (int)tiles, parts);
    else
      hipLaunchKernelGGL((scan_grad_local_kernel<E, N, false>), grid, dim3(256), 0, stream, a, (int)tiles, parts);
    const int blocks = (a.channels * N + 255) / 256;
    hipLaunchKernelGGL(scan_grad_carry_kernel, dim3((unsigned)(a.seqs * (int64_t)blocks)), dim3(256), 0, stream, a, N,
                       blocks);
  }
  const dim3 grid((unsigned)((waves + 3) / 4));
  if (a.z.ptr)
    hipLaunchKernelGGL((scan_grad_kernel<E, N, true>), grid, dim3(256), 0, stream, a, (int)tiles, waves);
  else
    hipLaunchKernelGGL((scan_grad_kernel<E, N, false>), grid, dim3(256), 0, stream, a, (int)tiles, waves);
  const int64_t blocks_bc = (a.tokens * a.groups * 2 * N + 511) / 512;
  const int64_t blocks_sum = (int64_t)((a.channels + 63) / 64) * (N + 2);
  hipLaunchKernelGGL((scan_grad_sum_kernel<E>), dim3((unsigned)(blocks_bc + blocks_sum)), dim3(512), 0, stream, a, N,
                     (int)(tiles / a.groups), blocks_bc);
  return hipGetLastError();
}
template <class E>
static hipError_t scan_back(const ScanArgs &a, int states, hipStream_t stream) {
  return states == 8 ? scan_back<E, 8>(a, stream) : states == 16 ? scan_back<E, 16>(a, stream) : scan_back<E, 32>(a, stream);
}
hipError_t launch_scan_backward(const ScanArgs &a, int dtype, int states, hipStream_t stream) {
  return dtype == 0 ? scan_back<F32>(a, states, stream)
         : dtype == 1 ? scan_back<BF16>(a, states, stream)
                      : scan_back<F16>(a, states, stream);
}

}  // namespace lq
