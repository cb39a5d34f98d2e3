// Norms before and after a block with its gate and residual scale (gfx950),
// forward and backward.  For a row of `dim` values of a token and head, with
// m(x) = (sum x^2 / dim + eps)^-1/2,
//   n = wo a m(a)  (or a),   u = n act(z)  (or n),   h = res + scale u,   y = wi h m(h)
// Backward, from dh and dy,
//   H = dh + m(h) wi dy - h m(h)^3 sum(h wi dy) / dim,   dres = H,   du = scale H
//   dz = du n act'(z),   dn = du act(z)
//   da = m(a) wo dn - a m(a)^3 sum(a wo dn) / dim  (or dn)
//   dwi = sum of dy h m(h), dwo = sum of dn a m(a) over all rows
//
// LANES lanes hold a row, R pieces of eight values each (16-byte accesses in
// 16-bit types), so that every value is read and written once; statistics are
// in fp32.  Bound by memory traffic: 16,384 x 32 rows of 128 in bf16, normed and
// gated, 80 to 86 us (4.7 to 5.0 TB/s); 8,192 rows of 4,096 with gate, fp32 stream and
// both norms 87 us (5.4 TB/s, part of it from cache), backward 165 + 5 (4.5 TB/s).
#include "lq_layer_device.h"

namespace lq {

__device__ __forceinline__ float block_act(int gate, float z) {
  const float s = sigmoid(z);
  return gate == 1 ? z * s : s;
}

// Two sums of a row's values: LANES lanes side by side, or a workgroup of LANES
// threads, through `sh` ([2][LANES / 64], the halves in turn: a half is written
// again only behind the next sum's barrier).
template <int LANES>
__device__ __forceinline__ void row_sums(float &x, float &y, float2 *sh, int &turn) {
  if constexpr (LANES == 16) {
    x = row16_sum(x);
    y = row16_sum(y);
    return;
  }
  x = wave_sum(x);
  y = wave_sum(y);
  if constexpr (LANES == 64) return;
  constexpr int waves = LANES / 64;
  float2 *s = sh + (turn ^= waves);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = make_float2(x, y);
  __syncthreads();
  x = y = 0.f;
#pragma unroll
  for (int w = 0; w < waves; ++w) {
    x += s[w].x;
    y += s[w].y;
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x, float2 *sh, int &turn) {
  float none = 0.f;
  row_sums<LANES>(x, none, sh, turn);
  return x;
}

template <int LANES>
constexpr int norm_threads() { return LANES > 256 ? LANES : 256; }

// Values up to 2^60 have squares whose sum over 8,192 of them is 2^133.  So rows of
// more than 128 values sum those of x 2^-7, and 2^14 comes back with the reciprocal of
// their number: powers of two, so that nothing rounds otherwise.
template <int LANES>
constexpr float norm_root() { return LANES > 16 ? 0x1p-7f : 1.f; }
template <int LANES>
__device__ __forceinline__ float row_root(float squares, float inv, float eps) {
  constexpr float up = 1.f / (norm_root<LANES>() * norm_root<LANES>());
  return 1.f / sqrtf(fmaf(squares, inv * up, eps));
}

// A row's arguments as a lane uses them
struct BlockRow {
  int64_t t;
  int h, col;  // col: the lane's first value of piece 0; piece r is LANES * 8 further
  bool on;
};
template <int LANES>
__device__ __forceinline__ BlockRow block_row(const BlockNormArgs &A, int64_t row, int64_t rows) {
  BlockRow b;
  b.on = row < rows;
  const int64_t r = b.on ? row : rows - 1;
  b.t = r / A.heads;
  b.h = (int)(r % A.heads);
  b.col = (threadIdx.x & (LANES - 1)) * 8;
  return b;
}

template <class E>
__device__ __forceinline__ Raw8<E> block_load(const Rows &r, const BlockRow &b, int col, int dim) {
  // (past the row's end: its beginning again, not used)
  return raw_load(at<const E>(r, b.t, b.h) + (col < dim ? col : 0));
}
__device__ __forceinline__ void block_weights(const float *w, int col, int dim, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 1.f;
  if (w && col < dim) load8(reinterpret_cast<const F32 *>(w + col), x);
}

template <class E, class S, int LANES, int R>
__global__ __launch_bounds__(norm_threads<LANES>()) void block_norm_kernel(const BlockNormArgs A, int64_t rows) {
  __shared__ float2 sh[LANES > 64 ? 2 * (LANES / 64) : 1];
  int turn = 0;
  constexpr int per = norm_threads<LANES>() / LANES;
  constexpr float down = norm_root<LANES>() * norm_root<LANES>();
  const BlockRow b = block_row<LANES>(A, (int64_t)blockIdx.x * per + threadIdx.x / LANES, rows);
  const bool gate = A.gate, res = A.res.ptr;
  Raw8<E> ra[R], rz[R];
  Raw8<S> rr[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int col = b.col + r * LANES * 8;
    ra[r] = block_load<E>(A.a, b, col, A.dim);
    if (gate) rz[r] = block_load<E>(A.z, b, col, A.dim);
    if (res) rr[r] = block_load<S>(A.res, b, col, A.dim);
  }
  float x[R][8];
  float ss = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    raw_floats(x[r], ra[r]);
    if (b.col + r * LANES * 8 < A.dim) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[r][e] * down, x[r][e], ss);
    }
  }
  const float inv = 1.f / (float)A.dim;
  if (A.out_norm) {
    const float m = row_root<LANES>(row_sum<LANES>(ss, sh, turn), inv, A.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float w[8];
      block_weights(A.wo, b.col + r * LANES * 8, A.dim, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[r][e] *= m * w[e];
    }
  }
  ss = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int col = b.col + r * LANES * 8;
    if (gate) {
      float z[8];
      raw_floats(z, rz[r]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[r][e] *= block_act(A.gate, z[e]);
    }
    float s[8];
    if (res) raw_floats(s, rr[r]);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[r][e] = res ? fmaf(A.scale, x[r][e], s[e]) : A.scale * x[r][e];
    if (col < A.dim) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[r][e] * down, x[r][e], ss);
      if (A.h.ptr && b.on) store8(at<S>(A.h, b.t, b.h) + col, x[r]);
    }
  }
  if (!A.y.ptr) return;
  const float m = row_root<LANES>(row_sum<LANES>(ss, sh, turn), inv, A.eps);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int col = b.col + r * LANES * 8;
    float w[8];
    block_weights(A.wi, col, A.dim, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[r][e] *= m * w[e];
    if (col < A.dim && b.on) store8(at<E>(A.y, b.t, b.h) + col, x[r]);
  }
}

// Workgroups of the backward pass take rows in turn and hold their weight gradients
// in LDS, each lane's own columns for each row of a workgroup: in registers they
// would take the room of a third wave a SIMD.
// Three workgroups of 256 threads a CU where a lane has one piece, two with two
// pieces, one of 512 threads.  Of 8,192 rows of 4,096: 165 us; three of two pieces
// spill (327 us for 172), 512 lanes with one piece each, one workgroup a CU, 222 for 198.
// Two pieces of fp32 rows spill 7 to 10 registers a lane also at two workgroups (both
// calls of 8,192 rows of 4,096 take 366 us, at the copy's rate 270).
static int64_t norm_most_blocks(int dim) {
  return dim <= 512 ? 768 : dim <= 1024 ? 512 : dim <= 2048 ? 768 : dim <= 4096 ? 512 : 256;
}

template <class E, class S, int LANES, int R>
__global__ __launch_bounds__(norm_threads<LANES>(), R == 1 ? 3 : 2) void block_norm_backward_kernel(const BlockNormArgs A, int64_t rows) {
  constexpr int threads = norm_threads<LANES>(), per = threads / LANES;
  __shared__ float2 sh[LANES > 64 ? 2 * (LANES / 64) : 1];
  __shared__ float sum[per][2][LANES * R * 8];
  int turn = 0;
  const bool gate = A.gate, silu = A.gate == 1, res = A.res.ptr, dy = A.dy.ptr, dh = A.dh.ptr;
  constexpr float root = norm_root<LANES>(), down = root * root;
  const float inv = 1.f / (float)A.dim;
  const int group = threadIdx.x / LANES;
  const auto add = [&](int p, int r, const float (&x)[8]) {
    float y[8];
    F32 *at_s = reinterpret_cast<F32 *>(&sum[group][p][(threadIdx.x & (LANES - 1)) * 8 + r * LANES * 8]);
    load8(at_s, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += x[e];
    store8(at_s, y);
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    F32 *at_s = reinterpret_cast<F32 *>(&sum[group][0][(threadIdx.x & (LANES - 1)) * 8 + r * LANES * 8]);
    store8(at_s, zero);
    store8(at_s + LANES * R * 8, zero);
  }
  // whole rounds: every thread meets every barrier, past the end with the last row again
  // The next row's values are on their way while a row is computed.
  Raw8<E> na[R], nz[R], ny[R];
  Raw8<S> nr[R], nh[R];
  const auto load = [&](int64_t row) {
    const BlockRow b = block_row<LANES>(A, row, rows);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int col = b.col + r * LANES * 8;
      na[r] = block_load<E>(A.a, b, col, A.dim);
      if (gate) nz[r] = block_load<E>(A.z, b, col, A.dim);
      if (res && dy) nr[r] = block_load<S>(A.res, b, col, A.dim);
      if (dy) ny[r] = block_load<E>(A.dy, b, col, A.dim);
      if (dh) nh[r] = block_load<S>(A.dh, b, col, A.dim);
    }
  };
  const int64_t step = (int64_t)gridDim.x * per;
  load((int64_t)blockIdx.x * per + group);
  for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < rows; row0 += step) {
    const BlockRow b = block_row<LANES>(A, row0 + group, rows);
    Raw8<E> ra[R], rz[R], ry[R];
    Raw8<S> rr[R], rh[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ra[r] = na[r];
      rz[r] = nz[r];
      ry[r] = ny[r];
      rr[r] = nr[r];
      rh[r] = nh[r];
    }
    if (row0 + step < rows) load(row0 + step + group);
    float ma = 1.f, x[R][8], n[R][8], sg[R][8];  // h root; the normed a; 1 / (1 + e^-z)
    if (A.out_norm) {
      float ss = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (b.col + r * LANES * 8 >= A.dim) continue;
        float a[8];
        raw_floats(a, ra[r]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(a[e] * down, a[e], ss);
      }
      ma = row_root<LANES>(row_sum<LANES>(ss, sh, turn), inv, A.eps);
    }
    float ss = 0.f, hg = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int col = b.col + r * LANES * 8;
      raw_floats(n[r], ra[r]);
      if (A.out_norm) {
        float w[8];
        block_weights(A.wo, col, A.dim, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[r][e] *= ma * w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[r][e] = A.scale * root * n[r][e];
      if (gate) {
        float z[8];
        raw_floats(z, rz[r]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sg[r][e] = sigmoid_for<E>(z[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[r][e] *= sg[r][e];
        if (silu) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[r][e] *= z[e];
        }
      }
      if (dy && col < A.dim) {
        float w[8], g[8];
        if (res) {
          raw_floats(g, rr[r]);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[r][e] = fmaf(root, g[e], x[r][e]);
        }
        block_weights(A.wi, col, A.dim, w);
        raw_floats(g, ry[r]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[r][e], x[r][e], ss);
          hg = fmaf(x[r][e], w[e] * g[e], hg);
        }
      }
    }
    float mh = 0.f, c = 0.f;
    if (dy) {
      row_sums<LANES>(ss, hg, sh, turn);
      mh = row_root<LANES>(ss, inv, A.eps);
      c = hg * (inv / down) * mh * mh;
    }
    float dn[R][8], ag = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int col = b.col + r * LANES * 8;
      if (col >= A.dim) continue;
      float H[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) H[e] = 0.f;
      if (dh) raw_floats(H, rh[r]);
      if (dy) {
        float w[8], g[8];
        block_weights(A.wi, col, A.dim, w);
        raw_floats(g, ry[r]);
#pragma unroll
        for (int e = 0; e < 8; ++e) H[e] = fmaf(mh, fmaf(-x[r][e], c, w[e] * g[e]), H[e]);
        if (A.dwi && b.on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= x[r][e] * (mh / root);
          add(1, r, g);
        }
      }
      if (A.dres.ptr && b.on) store8(at<S>(A.dres, b.t, b.h) + col, H);
#pragma unroll
      for (int e = 0; e < 8; ++e) dn[r][e] = H[e] * A.scale;
      if (gate) {  // dz = du n act'(z), dn = du act(z)
        float z[8], dz[8];
        raw_floats(z, rz[r]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = sg[r][e], t = s * (1.f - s);
          dz[e] = dn[r][e] * n[r][e] * (silu ? fmaf(z[e], t, s) : t);
          dn[r][e] *= s;
        }
        if (silu) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dn[r][e] *= z[e];
        }
        if (b.on) store8(at<E>(A.dz, b.t, b.h) + col, dz);
      }
      if (A.out_norm) {
        float a[8], w[8];
        raw_floats(a, ra[r]);
        block_weights(A.wo, col, A.dim, w);
        if (A.dwo && b.on) {
          float g[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = dn[r][e] * (a[e] * ma);
          add(0, r, g);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dn[r][e] *= w[e];
          ag = fmaf(a[e], dn[r][e], ag);
        }
      }
    }
    if (A.out_norm) {
      const float ca = row_sum<LANES>(ag, sh, turn) * inv * ma * ma;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float a[8];
        raw_floats(a, ra[r]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dn[r][e] = ma * fmaf(-a[e], ca, dn[r][e]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int col = b.col + r * LANES * 8;
      if (col < A.dim && b.on) store8(at<E>(A.da, b.t, b.h) + col, dn[r]);
    }
  }
  if (!A.dwo && !A.dwi) return;  // the whole block
  // the rows of a workgroup, added in order
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * A.dim; d += threads) {
    const int p = d >= A.dim, col = d - p * A.dim;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < per; ++k) x += sum[k][p][col];
    A.part[((int64_t)blockIdx.x * 2 + p) * A.dim + col] = x;
  }
}

// The workgroups' weight gradients, added in order: workgroup (which, 64
// values), wave (a share of the workgroups)
__global__ __launch_bounds__(1024) void block_norm_weight_kernel(const BlockNormArgs A, int64_t blocks) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, p = blockIdx.x & 1;
  const int d = (int)(blockIdx.x >> 1) * 64 + lane;
  float x = 0.f;
  if (d < A.dim) {
#pragma unroll 8
    for (int64_t n = w; n < blocks; n += 16) x += A.part[(n * 2 + p) * A.dim + d];
  }
  sh[w][lane] = x;
  __syncthreads();
  float *out = p ? A.dwi : A.dwo;
  if (w || d >= A.dim || !out) return;
  float y = 0.f;
#pragma unroll
  for (int v = 0; v < 16; ++v) y += sh[v][lane];
  out[d] = y;
}

// Lanes of a row by its width: sixteen up to 128 values (the usual head), a
// wave up to 1,024, workgroups beyond (a wave with four pieces a lane has no
// registers left for the next row).
static int norm_lanes(int dim) { return dim <= 128 ? 16 : dim <= 1024 ? 64 : dim <= 4096 ? 256 : 512; }

int64_t block_norm_blocks(int64_t rows, int dim) {
  const int lanes = norm_lanes(dim), per = lanes < 256 ? 256 / lanes : 1;
  const int64_t b = (rows + per - 1) / per;
  return b < norm_most_blocks(dim) ? b : norm_most_blocks(dim);
}

template <class E, class S, int LANES, int R>
static hipError_t norm_rows(const BlockNormArgs &a, bool back, hipStream_t stream) {
  constexpr int threads = norm_threads<LANES>(), per = threads / LANES;
  const int64_t rows = a.tokens * a.heads;
  if (!back) {
    hipLaunchKernelGGL((block_norm_kernel<E, S, LANES, R>), dim3((unsigned)((rows + per - 1) / per)), dim3(threads), 0,
                       stream, a, rows);
    return hipGetLastError();
  }
  const int64_t blocks = block_norm_blocks(rows, a.dim);
  if (blocks)
    hipLaunchKernelGGL((block_norm_backward_kernel<E, S, LANES, R>), dim3((unsigned)blocks), dim3(threads), 0, stream, a,
                       rows);
  if (a.dwo || a.dwi)
    hipLaunchKernelGGL(block_norm_weight_kernel, dim3((unsigned)((a.dim + 63) / 64 * 2)), dim3(1024), 0, stream, a, blocks);
  return hipGetLastError();
}
template <class E, class S>
static hipError_t norm_dim(const BlockNormArgs &a, bool back, hipStream_t stream) {
  if (a.dim <= 128) return norm_rows<E, S, 16, 1>(a, back, stream);
  if (a.dim <= 512) return norm_rows<E, S, 64, 1>(a, back, stream);
  if (a.dim <= 1024) return norm_rows<E, S, 64, 2>(a, back, stream);
  if (a.dim <= 2048) return norm_rows<E, S, 256, 1>(a, back, stream);
  if (a.dim <= 4096) return norm_rows<E, S, 256, 2>(a, back, stream);
  return norm_rows<E, S, 512, 2>(a, back, stream);
}
static hipError_t norm_types(const BlockNormArgs &a, int dtype, int stream_dtype, bool back, hipStream_t stream) {
  if (dtype == 0) return norm_dim<F32, F32>(a, back, stream);
  if (dtype == 1)
    return stream_dtype == 0 ? norm_dim<BF16, F32>(a, back, stream) : norm_dim<BF16, BF16>(a, back, stream);
  return stream_dtype == 0 ? norm_dim<F16, F32>(a, back, stream) : norm_dim<F16, F16>(a, back, stream);
}
hipError_t launch_block_norm(const BlockNormArgs &a, int dtype, int stream_dtype, hipStream_t stream) {
  return norm_types(a, dtype, stream_dtype, false, stream);
}
hipError_t launch_block_norm_backward(const BlockNormArgs &a, int dtype, int stream_dtype, hipStream_t stream) {
  return norm_types(a, dtype, stream_dtype, true, stream);
}

}  // namespace lq
