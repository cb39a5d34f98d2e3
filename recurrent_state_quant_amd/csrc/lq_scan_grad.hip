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
// states do.  The forward pass left the state before every 8th token (4th with
// 32 states): a run of tokens is computed again from it, its states stay in
// registers, and the run is taken backwards.
#include "lq_scan_device.h"

namespace lq {

// The chunks' gradients behind from zero: what comes out of their first token.
template <class E, int N>
__global__ __launch_bounds__(256) void scan_grad_local_kernel(const ScanArgs A, int tiles, int64_t waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;
  const int slot = (int)(wave / tiles), tile = (int)(wave % tiles), tg = (A.per + 63) >> 6;
  const ScanChunk k = scan_chunk(A, slot, lane);
  if (!k.any || k.c == 0) return;  // nothing comes before the first chunk
  const ScanTile ch = scan_tile(A, tile / tg, tile % tg, lane);
  const int64_t width = A.channels;
  float a2[N], g[N], sum = 0.f;
  scan_decays<N>(A, ch.c, a2);
#pragma unroll
  for (int n = 0; n < N; ++n) g[n] = 0.f;
  const float bias = A.bias ? A.bias[ch.c] : 0.f;
  const bool gate = A.z.ptr;
  const E *dt = at<const E>(A.dt, 0, 0) + ch.c, *dy = at<const E>(A.dy, 0, 0) + ch.c;
  const E *z = gate ? at<const E>(A.z, 0, 0) + ch.c : dy;
  constexpr int ahead = 8;
  E rd[ahead], ry[ahead], rz[ahead];
  const auto load = [&](int t) {  // tokens t, t - 1 ..
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      const int64_t tt = max(t - u, k.t0);
      rd[u] = dt[tt * A.dt.ts];
      ry[u] = dy[tt * A.dy.ts];
      if (gate) rz[u] = z[tt * A.z.ts];
    }
  };
  load(k.t1 - 1);
  for (int t = k.t1 - 1; t >= k.t0; t -= ahead) {
    float fd[ahead], fy[ahead], fz[ahead];
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      fd[u] = to_f(rd[u]) + bias;
      fy[u] = to_f(ry[u]);
      fz[u] = gate ? to_f(rz[u]) : 0.f;
    }
    if (t - ahead >= k.t0) load(t - ahead);
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      if (t - u < k.t0) break;
      float cc[N];
      scan_row<E, N>(A.C, t - u, ch.g, cc);
      const float d = scan_step(A, fd[u]);
      const float dp = gate ? fy[u] * (fz[u] * sigmoid(fz[u])) : fy[u];
      sum += d;
#pragma unroll
      for (int n = 0; n < N; ++n) g[n] = __builtin_amdgcn_exp2f(d * a2[n]) * fmaf(cc[n], dp, g[n]);
    }
  }
  if (!ch.on) return;
  scan_store_cols<N>(A.carry + (int64_t)slot * N * width, width, ch.c, g);
  A.sum[slot * width + ch.c] = sum;
}

// The gradients behind every chunk of the sequences with several, over the
// chunks' own: thread (sequence, state, channel), the last chunk first.  dS is
// copied behind the last chunk, as dS0 may lie over it.
constexpr int kCarryAhead = 8;
__global__ __launch_bounds__(256) void scan_grad_carry_kernel(const ScanArgs A, int states, int64_t threads) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= threads) return;
  const int64_t width = A.channels, c = id % width, n = id / width % states, i = id / width / states;
  const auto offset = [&](int64_t s) {
    const int o = A.cu[s];
    return o < 0 ? 0 : (o > A.tokens ? (int)A.tokens : o);
  };
  const int start = offset(i), end = max(start, offset(i + 1));
  const int chunks = (end - start + (1 << A.shift) - 1) >> A.shift;
  if (chunks < 2) return;
  const int64_t slot = (start >> A.shift) + i;
  const float a2 = A.A[c * states + n] * kLog2e;
  float g = A.dS ? A.dS[(i * width + c) * states + n] : 0.f;
  float *carry = A.carry + (slot * states + n) * width + c;
  const float *sum = A.sum + slot * width + c;
  const int64_t step = states * width;
  for (int k = chunks - 1; k >= 0; k -= kCarryAhead) {
    float v[kCarryAhead], s[kCarryAhead];
#pragma unroll
    for (int u = 0; u < kCarryAhead; ++u) {
      const bool in = k - u > 0;
      v[u] = in ? carry[(k - u) * step] : 0.f;
      s[u] = in ? sum[(k - u) * width] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kCarryAhead; ++u) {
      if (k - u < 0) break;
      carry[(k - u) * step] = g;
      g = fmaf(__builtin_amdgcn_exp2f(s[u] * a2), g, v[u]);
    }
  }
}

// Sums across the wave of many values at once: each step halves the lanes that
// a value is spread over and packs two values into one register.
// Four values: afterwards rows of 16 lanes 0, 1, 2, 3 hold a, c, b, d.
__device__ __forceinline__ float fold4(float a, float b, float c, float d) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(c), __float_as_uint(d), false, false);
  const float x = __uint_as_float(p[0]) + __uint_as_float(p[1]), y = __uint_as_float(q[0]) + __uint_as_float(q[1]);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Two values into one register: lanes with `high` keep b.
template <int CTRL>
__device__ __forceinline__ float fold2(float a, float b, bool high) {
  return (high ? b : a) + dpp<CTRL>(high ? a : b);
}
// Q registers of fold4 into one: lane (row r, i) holds a sum of register q(i),
// the bits of q being bits 3, 2, 1, 0 of i in this order (as many as Q has).
template <int Q>
__device__ __forceinline__ float fold_row(float (&v)[Q], int lane) {
  static_assert(Q == 4 || Q == 8 || Q == 16, "");
  float a[Q / 2];
#pragma unroll
  for (int k = 0; k < Q / 2; ++k) a[k] = fold2<0x140>(v[2 * k], v[2 * k + 1], lane & 8);  // row_mirror
  float b[Q / 4];
#pragma unroll
  for (int k = 0; k < Q / 4; ++k) b[k] = fold2<0x141>(a[2 * k], a[2 * k + 1], lane & 4);  // row_half_mirror
  if constexpr (Q == 4) {
    b[0] += dpp<0x1B>(b[0]);  // quad_perm [3,2,1,0]
    return b[0] + dpp<0xB1>(b[0]);  // quad_perm [1,0,3,2]
  } else {
    float c[Q / 8];
#pragma unroll
    for (int k = 0; k < Q / 8; ++k) c[k] = fold2<0x1B>(b[2 * k], b[2 * k + 1], lane & 2);
    if constexpr (Q == 8) return c[0] + dpp<0xB1>(c[0]);
    if constexpr (Q == 16) return fold2<0xB1>(c[0], c[1], lane & 1);
  }
}
// The number of the sum that a lane holds after fold_row.
template <int Q>
__device__ __forceinline__ int fold_place(int lane) {
  const int row = lane >> 4;
  int q = (lane >> 3 & 1) | (lane >> 2 & 1) << 1;
  if (Q > 4) q |= (lane >> 1 & 1) << 2;
  if (Q > 8) q |= (lane & 1) << 3;
  return 4 * q + ((row & 1) << 1 | row >> 1);
}

// A block's four waves share a group and a chunk: their sums over the channels
// meet in LDS after every run of tokens.
template <class E, int N>
__global__ __launch_bounds__(256) void scan_grad_kernel(const ScanArgs A, int blocks_group) {
  constexpr int shift = scan_sub_shift(N), sub = 1 << shift, Q = N / 2;
  __shared__ float sh[2][4][sub][2 * N];
  const int lane = threadIdx.x & 63, w4 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = A.groups * blocks_group;
  const int slot = blockIdx.x / blocks, gb = blockIdx.x % blocks;
  const int group = gb / blocks_group, tile = gb % blocks_group * 4 + w4;
  const ScanChunk k = scan_chunk(A, slot, lane);
  const ScanTile ch = scan_tile(A, group, tile, lane);
  const int64_t width = A.channels;
  float a2[N], g[N], dA[N], dskip = 0.f, dbias = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) g[n] = dA[n] = 0.f;
  if (k.any) {
    scan_decays<N>(A, ch.c, a2);
    if (ch.on) {
      if (k.chunks > 1)
        scan_load_cols<N>(A.carry + (int64_t)slot * N * width, width, ch.c, g);
      else if (A.dS)
        scan_load_rows<N>(A.dS, k.i * width + ch.c, g);
    }
    const float bias = A.bias ? A.bias[ch.c] : 0.f, skip = A.skip ? A.skip[ch.c] : 0.f;
    const bool gate = A.z.ptr;
    const E *x = at<const E>(A.x, 0, 0) + ch.c, *dt = at<const E>(A.dt, 0, 0) + ch.c;
    const E *dy = at<const E>(A.dy, 0, 0) + ch.c, *z = gate ? at<const E>(A.z, 0, 0) + ch.c : x;
    E *out_x = at<E>(A.dx, 0, 0) + ch.c, *out_t = at<E>(A.ddt, 0, 0) + ch.c;
    E *out_z = gate ? at<E>(A.dz, 0, 0) + ch.c : out_x;
    const int len = k.t1 - k.t0, runs = (len + sub - 1) >> shift;
    const int64_t first = (k.start >> shift) + k.i + ((k.t0 - k.start) >> shift);
    const int place = fold_place<Q>(lane);
    const bool holder = Q == 16 || (Q == 8 ? !(lane & 1) : !(lane & 3));
    for (int r = runs - 1; r >= 0; --r) {
      const int t = k.t0 + (r << shift), n_t = min(sub, k.t1 - t);
      float fx[sub], fd[sub], fy[sub], fz[sub], slope[sub], hist[sub][N];
#pragma unroll
      for (int u = 0; u < sub; ++u) {
        const int64_t tt = min(t + u, k.t1 - 1);
        fx[u] = ch.on ? to_f(x[tt * A.x.ts]) : 0.f;
        fd[u] = to_f(dt[tt * A.dt.ts]) + bias;
        fy[u] = ch.on ? to_f(dy[tt * A.dy.ts]) : 0.f;
        fz[u] = gate ? to_f(z[tt * A.z.ts]) : 0.f;
      }
      // the states before the run's tokens
      scan_load_cols<N>(A.check + (first + r) * N * width, width, ch.c, hist[0]);
#pragma unroll
      for (int u = 0; u < sub; ++u) {
        fd[u] = scan_step(A, fd[u], slope[u]);
        if (u + 1 < sub) {
          float b[N];
          scan_row<E, N>(A.B, min(t + u, k.t1 - 1), ch.g, b);
          const float dx = fd[u] * fx[u];
#pragma unroll
          for (int n = 0; n < N; ++n)
            hist[u + 1][n] = fmaf(__builtin_amdgcn_exp2f(fd[u] * a2[n]), hist[u][n], dx * b[n]);
        }
      }
#pragma unroll
      for (int u = sub - 1; u >= 0; --u) {
        if (u >= n_t) continue;
        float b[N], cc[N];
        scan_row<E, N>(A.B, t + u, ch.g, b);
        scan_row<E, N>(A.C, t + u, ch.g, cc);
        const float d = fd[u], xd = d * fx[u];
        float s = 0.f, dp = fy[u];
        if (gate) {
          s = sigmoid(fz[u]);
          dp *= fz[u] * s;
        }
        float p = skip * fx[u], gb = 0.f, ea = 0.f, fold[Q];
#pragma unroll
        for (int n = 0; n < N; n += 4) {
          float vb[4], vc[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float a = __builtin_amdgcn_exp2f(d * a2[n + m]), ah = a * hist[u][n + m];
            const float h = fmaf(xd, b[n + m], ah);
            p = fmaf(cc[n + m], h, p);
            const float gn = fmaf(cc[n + m], dp, g[n + m]);
            gb = fmaf(gn, b[n + m], gb);
            const float e = gn * ah;
            ea = fmaf(e, a2[n + m], ea);
            dA[n + m] = fmaf(e, d, dA[n + m]);
            vb[m] = gn * xd;
            vc[m] = dp * h;
            g[n + m] = gn * a;
          }
          fold[n / 4] = fold4(vb[0], vb[1], vb[2], vb[3]);
          fold[Q / 2 + n / 4] = fold4(vc[0], vc[1], vc[2], vc[3]);
        }
        const float total = fold_row<Q>(fold, lane);
        if (holder) sh[r & 1][w4][u][place] = total;
        const float ddt = fmaf(gb, fx[u], ea * kLn2) * slope[u];
        dskip = fmaf(dp, fx[u], dskip);
        dbias += ddt;
        if (ch.on) {
          out_x[(t + u) * A.dx.ts] = from_f<E>(fmaf(gb, d, skip * dp));
          out_t[(t + u) * A.ddt.ts] = from_f<E>(ddt);
          if (gate) out_z[(t + u) * A.dz.ts] = from_f<E>(fy[u] * p * (s * fmaf(fz[u], 1.f - s, 1.f)));
        }
      }
      __syncthreads();  // (the other half of `sh` is written next)
      for (int v = threadIdx.x; v < n_t * 2 * N; v += 256) {
        const int u = v / (2 * N), n = v % (2 * N);
        A.part_bc[((int64_t)gb * A.tokens + t + u) * 2 * N + n] =
            ((sh[r & 1][0][u][n] + sh[r & 1][1][u][n]) + sh[r & 1][2][u][n]) + sh[r & 1][3][u][n];
      }
    }
    if (A.dS0 && k.c == 0 && ch.on) scan_store_rows<N>(A.dS0, k.i * width + ch.c, g);
  }
  if (!ch.on) return;
  // (slots without a chunk: zeros)
  float *part = A.part_a + (int64_t)slot * (N + 2) * width;
  scan_store_cols<N>(part, width, ch.c, dA);
  part[N * width + ch.c] = dskip;
  part[(N + 1) * width + ch.c] = dbias;
}

// dB and dC: the blocks' sums over the channels, added in order; thread (token,
// group, state of B or C)
template <class E>
__global__ __launch_bounds__(256) void scan_grad_bc_kernel(const ScanArgs A, int states, int blocks_group, int64_t threads) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= threads) return;
  const int n = (int)(id % (2 * states)), g = (int)(id / (2 * states) % A.groups);
  const int64_t t = id / (2 * states) / A.groups;
  const int lo = A.cu[0], hi = A.cu[A.seqs];
  if (t < lo || t >= hi) return;  // of no sequence
  float x = 0.f;
#pragma unroll 4
  for (int b = 0; b < blocks_group; ++b)
    x += A.part_bc[(((int64_t)g * blocks_group + b) * A.tokens + t) * 2 * states + n];
  if (n < states)
    at<E>(A.dB, t, g)[n] = from_f<E>(x);
  else
    at<E>(A.dC, t, g)[n - states] = from_f<E>(x);
}

// dA, dD and dbias: the chunks' sums, added in order.  Workgroup (64 channels,
// state), wave (a share of the slots).
__global__ __launch_bounds__(512) void scan_grad_sum_kernel(const ScanArgs A, int states) {
  __shared__ float sh[8][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int tiles = (A.channels + 63) >> 6, k = blockIdx.x / tiles;
  const int64_t width = A.channels, c = (int64_t)(blockIdx.x % tiles) * 64 + lane;
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
  const int64_t tiles = scan_tiles(a.channels, a.groups), waves = tiles * a.slots, blocks = scan_group_blocks(a.per);
  if (a.tokens > (int64_t(1) << a.shift)) {
    hipLaunchKernelGGL((scan_grad_local_kernel<E, N>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a,
                       (int)tiles, waves);
    const int64_t threads = (int64_t)a.seqs * a.channels * N;
    hipLaunchKernelGGL(scan_grad_carry_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, a, N,
                       threads);
  }
  hipLaunchKernelGGL((scan_grad_kernel<E, N>), dim3((unsigned)(a.slots * a.groups * blocks)), dim3(256), 0, stream, a,
                     (int)blocks);
  const int64_t threads = a.tokens * a.groups * 2 * N;
  if (threads)
    hipLaunchKernelGGL((scan_grad_bc_kernel<E>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, a, N,
                       (int)blocks, threads);
  hipLaunchKernelGGL(scan_grad_sum_kernel, dim3((unsigned)((a.channels + 63) / 64 * (N + 2))), dim3(512), 0, stream, a, N);
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
