// Short causal convolution of every channel over packed sequences (gfx950),
// forward, for single tokens, and backward.  With width K,
//   v_t = bias + sum_j w_j x_{t-K+1+j},   y_t = v_t or v_t / (1 + e^-v_t)
// where the K - 1 inputs before a sequence's first token come from X0 (zeros
// without it).  Backward, with dv_t = dy_t act'(v_t),
//   dx_t = sum_j w_j dv_{t+K-1-j}  (the last K - 1 tokens: plus dX)
//   dw_j = sum_t dv_t x_{t-K+1+j},  dbias = sum_t dv_t
//
// Bound by memory traffic.  A lane holds the weights and the last K - 1 inputs of
// 16 bytes of channels in registers and walks a run of tokens, so that every input
// is read once but for the K - 1 around a run.  With width 4 in bf16, 16,384 tokens
// x 8,192 channels of 24 sequences take 118 us (4.6 TB/s of input and output), 8,192
// x 6,144 43 us forward (4.7 TB/s) and 69 + 5 backward (4.4 TB/s of two inputs and an
// output).  Loads and stores past the caches gain nothing
// (48 us for 43 of inputs that are cached).
#include "lq_layer_device.h"

namespace lq {

// Rows loaded together: eight take 44 for 43 us of 8,192 tokens x 6,144 channels
// forward and, at the same three waves a SIMD, 76 for 72 backward.
constexpr int kConvAhead = 4;

// The sequence of a token: tokens [s, e) of sequence i (i = -1: none yet)
struct ConvSeq {
  int i, s, e;
};
__device__ __forceinline__ ConvSeq conv_seq(const ConvArgs &A, int i) {
  ConvSeq q{i, 0, 0};
  if (i >= 0) {
    q.s = seq_offset(A.cu, A.tokens, i);
    q.e = max(q.s, seq_offset(A.cu, A.tokens, i + 1));
  }
  return q;
}

// The K - 1 inputs before token t >= s of a sequence
template <class E, int V, int K>
__device__ __forceinline__ void conv_window(const ConvArgs &A, const ConvSeq &q, int t, int64_t c, float (&win)[K - 1][V]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int p = t - (K - 1) + j;
    if (p >= q.s) {
      vec_floats(win[j], vec_load<E, V>(at<const E>(A.x, p, 0) + c));
    } else if (A.X0) {
      const int64_t row = (int64_t)q.i * (K - 1) + (p - q.s + K - 1);
      vec_floats(win[j], vec_load<E, V>(static_cast<const E *>(A.X0) + row * A.channels + c));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = 0.f;
    }
  }
}

template <int V, int K>
__device__ __forceinline__ void conv_weights(const ConvArgs &A, int64_t c, float (&w)[K][V], float (&b)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][v] = A.w[(c + v) * K + j];
    b[v] = A.bias ? A.bias[c + v] : 0.f;
  }
}

// v_t of one token from its window and its own input
template <int V, int K>
__device__ __forceinline__ void conv_sum(const float (&w)[K][V], const float (&b)[V], const float (&win)[K - 1][V],
                                         const float (&x)[V], float (&out)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float s = b[v];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) s = fmaf(w[j][v], win[j][v], s);
    out[v] = fmaf(w[K - 1][v], x[v], s);
  }
}
template <int V, int K>
__device__ __forceinline__ void conv_shift(float (&win)[K - 1][V], const float (&x)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j + 1 < K - 1; ++j) win[j][v] = win[j + 1][v];
    win[K - 2][v] = x[v];
  }
}

// A wave takes 64 V channels and a run of tokens, whatever sequences they are of;
// the waves behind the runs take a sequence each and write its last inputs.
template <class E, int V, int K>
__global__ __launch_bounds__(256) void conv_kernel(const ConvArgs A, int tiles, int run_tokens, int64_t runs, int64_t waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;  // whole waves; the waves share nothing
  const int64_t run = wave / tiles;
  const int64_t c = ((int64_t)(wave % tiles) * 64 + lane) * V;
  const bool on = c < A.channels;
  if (run >= runs) {  // a sequence's last inputs
    const ConvSeq q = conv_seq(A, (int)(run - runs));
    if (!on) return;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int p = q.e - (K - 1) + j;
      Vec<E, V> r{};
      if (p >= q.s) {
        r = vec_load<E, V>(at<const E>(A.x, p, 0) + c);
      } else if (A.X0) {
        const int64_t row = (int64_t)q.i * (K - 1) + (p - q.s + K - 1);
        r = vec_load<E, V>(static_cast<const E *>(A.X0) + row * A.channels + c);
      }
      vec_store(static_cast<E *>(A.X) + ((int64_t)q.i * (K - 1) + j) * A.channels + c, r);
    }
    return;
  }
  const int t0 = (int)(run * run_tokens), t1 = (int)min((int64_t)t0 + run_tokens, A.tokens);
  ConvSeq q = conv_seq(A, seq_search(A.cu, A.tokens, A.seqs, 1, 0, t0, lane));
  if (!on) return;
  float w[K][V], b[V], win[K - 1][V];
  conv_weights<V, K>(A, c, w, b);
  int in = -1;  // the sequence that `win` is of
  Vec<E, V> next[kConvAhead];
  const auto load = [&](int t) {
#pragma unroll
    for (int u = 0; u < kConvAhead; ++u) next[u] = vec_load<E, V>(at<const E>(A.x, min(t + u, t1 - 1), 0) + c);
  };
  load(t0);
  for (int t = t0; t < t1; t += kConvAhead) {
    Vec<E, V> raw[kConvAhead];
#pragma unroll
    for (int u = 0; u < kConvAhead; ++u) raw[u] = next[u];
    if (t + kConvAhead < t1) load(t + kConvAhead);
#pragma unroll
    for (int u = 0; u < kConvAhead; ++u) {
      const int tt = t + u;
      if (tt >= t1) break;
      while (tt >= q.e && q.i + 1 < A.seqs) q = conv_seq(A, q.i + 1);
      if (tt < q.s || tt >= q.e) continue;  // of no sequence
      if (in != q.i) conv_window<E, V, K>(A, q, tt, c, win);
      in = q.i;
      float x[V], y[V];
      vec_floats(x, raw[u]);
      conv_sum<V, K>(w, b, win, x, y);
      if (A.silu) {
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] *= sigmoid_for<E>(y[v]);
      }
      vec_store(at<E>(A.y, tt, 0) + c, vec_round<E, V>(y));
      conv_shift<V, K>(win, x);
    }
  }
}

// One token of each row: slot s's inputs X0[s] and the row's own; the slot's
// last inputs go to X[s] (which may be X0: a lane reads its channels' inputs
// before it writes them).  64 rows x 8,192 channels: 6 us, which is a launch and
// three dependent loads (slot, inputs, output) more than their 8 MB.
template <class E, int V, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(const ConvArgs A, int tiles, int64_t waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;
  const int64_t row = wave / tiles;
  const int64_t c = ((int64_t)(wave % tiles) * 64 + lane) * V;
  const int64_t slot = A.slots ? A.slots[row] : row;
  if (c >= A.channels || slot < 0 || slot >= A.n_slots) return;
  const E *from = static_cast<const E *>(A.X0) + slot * (K - 1) * A.channels + c;
  E *to = static_cast<E *>(A.X) + slot * (K - 1) * A.channels + c;
  Vec<E, V> raw[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) raw[j] = vec_load<E, V>(from + (int64_t)j * A.channels);
  raw[K - 1] = vec_load<E, V>(at<const E>(A.x, row, 0) + c);
  float w[K][V], b[V], win[K - 1][V], x[V], y[V];
  conv_weights<V, K>(A, c, w, b);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) vec_floats(win[j], raw[j]);
  vec_floats(x, raw[K - 1]);
  conv_sum<V, K>(w, b, win, x, y);
  if (A.silu) {
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] *= sigmoid_for<E>(y[v]);
  }
  vec_store(at<E>(A.y, row, 0) + c, vec_round<E, V>(y));
#pragma unroll
  for (int j = 0; j < K - 1; ++j) vec_store(to + (int64_t)j * A.channels, raw[j + 1]);
}

// dv_t from v_t and dy_t
template <class E, int V>
__device__ __forceinline__ void conv_back(bool silu, const float (&v)[V], float (&d)[V]) {
  if (!silu) return;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float s = sigmoid_for<E>(v[e]);
    d[e] *= s * fmaf(v[e], 1.f - s, 1.f);
  }
}

// Backward.  A block's four waves take four neighbouring runs of the same
// channels.  A wave walks its run and the K - 1 tokens of the same sequence
// behind it; `acc` holds the gradients of the last K - 1 inputs, to which later
// tokens still add.  The waves' weight gradients meet in LDS, the blocks' are
// added by a second launch, all in a fixed order.
template <class E, int V, int K>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 3 : 2) void conv_backward_kernel(const ConvArgs A, int tiles, int run_tokens) {
  __shared__ float sh[4][K + 1][64 * V];
  const int lane = threadIdx.x & 63, w4 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block = blockIdx.x / tiles;
  const int64_t c = ((int64_t)(blockIdx.x % tiles) * 64 + lane) * V;
  const bool on = c < A.channels;
  float w[K][V], b[V], dw[K][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][v] = 0.f;
  }
  const int64_t first = (block * 4 + w4) * run_tokens;
  if (first < A.tokens) {
    const int t0 = (int)first, t1 = (int)min(first + run_tokens, A.tokens);
    ConvSeq q = conv_seq(A, seq_search(A.cu, A.tokens, A.seqs, 1, 0, t0, lane));
    if (on) {
      conv_weights<V, K>(A, c, w, b);
      float win[K - 1][V], acc[K - 1][V];
      int in = -1;  // the sequence that `win` and `acc` are of
      const int stop = (int)min((int64_t)t1 + K - 1, A.tokens);
      bool open = true;
      Vec<E, V> nx[kConvAhead], ng[kConvAhead];
      const auto load = [&](int t) {
#pragma unroll
        for (int u = 0; u < kConvAhead; ++u) {
          const int tt = min(t + u, stop - 1);
          nx[u] = vec_load<E, V>(at<const E>(A.x, tt, 0) + c);
          ng[u] = vec_load<E, V>(at<const E>(A.dy, tt, 0) + c);
        }
      };
      load(t0);
      for (int t = t0; t < stop && open; t += kConvAhead) {
        Vec<E, V> rx[kConvAhead], rg[kConvAhead];
#pragma unroll
        for (int u = 0; u < kConvAhead; ++u) {
          rx[u] = nx[u];
          rg[u] = ng[u];
        }
        if (t + kConvAhead < stop) load(t + kConvAhead);
#pragma unroll
        for (int u = 0; u < kConvAhead; ++u) {
          const int tt = t + u;
          if (tt >= stop || (tt >= t1 && (in != q.i || tt >= q.e))) {  // behind the run only the rest of its last sequence
            open = false;
            break;
          }
          while (tt >= q.e && q.i + 1 < A.seqs) q = conv_seq(A, q.i + 1);
          if (tt < q.s || tt >= q.e) continue;  // of no sequence
          if (in != q.i) {
            conv_window<E, V, K>(A, q, tt, c, win);
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
              for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
          }
          in = q.i;
          float x[V], d[V], y[V];
          vec_floats(x, rx[u]);
          vec_floats(d, rg[u]);
          conv_sum<V, K>(w, b, win, x, y);
          conv_back<E, V>(A.silu, y, d);
          if (tt < t1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
              db[v] += d[v];
#pragma unroll
              for (int j = 0; j < K - 1; ++j) dw[j][v] = fmaf(d[v], win[j][v], dw[j][v]);
              dw[K - 1][v] = fmaf(d[v], x[v], dw[K - 1][v]);
            }
          }
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[j][v] = fmaf(w[j][v], d[v], acc[j][v]);
          const int least = max(t0, q.s);
          if (tt - (K - 1) >= least) vec_store(at<E>(A.dx, tt - (K - 1), 0) + c, vec_round<E, V>(acc[0]));
#pragma unroll
          for (int v = 0; v < V; ++v) d[v] *= w[K - 1][v];
          conv_shift<V, K>(acc, d);
          conv_shift<V, K>(win, x);
          if (tt == q.e - 1) {  // the sequence's last K - 1 inputs
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
              const int p = q.e - (K - 1) + j;
              if (p < least || p >= t1) continue;
              if (A.dX) {
                float g[V];
                const int64_t row = (int64_t)q.i * (K - 1) + j;
                vec_floats(g, vec_load<E, V>(static_cast<const E *>(A.dX) + row * A.channels + c));
#pragma unroll
                for (int v = 0; v < V; ++v) acc[j][v] += g[v];
              }
              vec_store(at<E>(A.dx, p, 0) + c, vec_round<E, V>(acc[j]));
            }
          }
        }
      }
    }
  }
  if (!A.dw && !A.dbias) return;  // the whole block
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < K; ++j) sh[w4][j][v * 64 + lane] = dw[j][v];
    sh[w4][K][v * 64 + lane] = db[v];
  }
  __syncthreads();
  const int64_t c0 = (int64_t)(blockIdx.x % tiles) * 64 * V;
  for (int k = threadIdx.x; k < (K + 1) * 64 * V; k += 256) {
    const int j = k / (64 * V), at_c = k % (64 * V);  // channel c0 + at_c is value at_c % V of lane at_c / V
    const int from = (at_c % V) * 64 + at_c / V;
    if (c0 + at_c < A.channels)
      A.part[(block * (K + 1) + j) * A.channels + c0 + at_c] =
          ((sh[0][j][from] + sh[1][j][from]) + sh[2][j][from]) + sh[3][j][from];
  }
}

// The gradient of the inputs before each sequence: one wave a sequence and 64 V
// channels.
template <class E, int V, int K>
__global__ __launch_bounds__(256) void conv_before_kernel(const ConvArgs A, int tiles, int64_t waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;
  const ConvSeq q = conv_seq(A, (int)(wave / tiles));
  const int64_t c = ((int64_t)(wave % tiles) * 64 + lane) * V;
  if (c >= A.channels) return;
  float w[K][V], b[V], win[K - 1][V], acc[K - 1][V];
  conv_weights<V, K>(A, c, w, b);
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
  const int len = q.e - q.s;
  if (len > 0) conv_window<E, V, K>(A, q, q.s, c, win);
#pragma unroll
  for (int t = 0; t < K - 1; ++t) {
    if (t >= len) break;
    float x[V], d[V], y[V];
    vec_floats(x, vec_load<E, V>(at<const E>(A.x, q.s + t, 0) + c));
    vec_floats(d, vec_load<E, V>(at<const E>(A.dy, q.s + t, 0) + c));
    conv_sum<V, K>(w, b, win, x, y);
    conv_back<E, V>(A.silu, y, d);
    // token t's window begins with the inputs t .. K - 2 before the sequence
#pragma unroll
    for (int j = 0; j + t < K - 1; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[j + t][v] = fmaf(w[j][v], d[v], acc[j + t][v]);
    conv_shift<V, K>(win, x);
  }
#pragma unroll
  for (int r = 0; r < K - 1; ++r) {
    if (A.dX && r >= len) {  // still among the last inputs: row r - len of them
      float g[V];
      const int64_t row = (int64_t)q.i * (K - 1) + (r - len);
      vec_floats(g, vec_load<E, V>(static_cast<const E *>(A.dX) + row * A.channels + c));
#pragma unroll
      for (int v = 0; v < V; ++v) acc[r][v] += g[v];
    }
    vec_store(static_cast<E *>(A.dX0) + ((int64_t)q.i * (K - 1) + r) * A.channels + c, vec_round<E, V>(acc[r]));
  }
}

// The blocks' weight gradients, added in order: thread (channel, weight or bias)
__global__ __launch_bounds__(256) void conv_weight_kernel(const ConvArgs A, int64_t blocks) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = A.width + 1;
  if (k >= rows * A.channels) return;
  const int j = (int)(k / A.channels);
  const int64_t c = k % A.channels;
  float x = 0.f;
#pragma unroll 8
  for (int64_t n = 0; n < blocks; ++n) x += A.part[(n * rows + j) * A.channels + c];
  if (j == A.width) {
    if (A.dbias) A.dbias[c] = x;
  } else if (A.dw) {
    A.dw[c * A.width + j] = x;
  }
}

template <class E, int V, int K>
static hipError_t conv_forward(const ConvArgs &a, hipStream_t stream) {
  const int tiles = (a.channels + 64 * V - 1) / (64 * V);
  const int run = conv_run_tokens(a.tokens, tiles, 4);
  const int64_t runs = (a.tokens + run - 1) / run;
  const int64_t waves = (runs + (a.X ? a.seqs : 0)) * tiles;
  if (waves)
    hipLaunchKernelGGL((conv_kernel<E, V, K>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a, tiles, run,
                       runs, waves);
  return hipGetLastError();
}
template <class E, int V, int K>
static hipError_t conv_step(const ConvArgs &a, hipStream_t stream) {
  const int tiles = (a.channels + 64 * V - 1) / (64 * V);
  const int64_t waves = a.tokens * tiles;
  if (waves)
    hipLaunchKernelGGL((conv_step_kernel<E, V, K>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a, tiles,
                       waves);
  return hipGetLastError();
}
template <class E, int V, int K>
static hipError_t conv_backward(const ConvArgs &a, hipStream_t stream) {
  const int tiles = (a.channels + 64 * V - 1) / (64 * V);
  const int run = conv_grad_run(a.tokens, a.channels);
  const int64_t blocks = conv_grad_blocks(a.tokens, run);
  if (blocks)
    hipLaunchKernelGGL((conv_backward_kernel<E, V, K>), dim3((unsigned)(blocks * tiles)), dim3(256), 0, stream, a, tiles,
                       run);
  if (a.dw || a.dbias)
    hipLaunchKernelGGL(conv_weight_kernel, dim3((unsigned)(((int64_t)(K + 1) * a.channels + 255) / 256)), dim3(256), 0,
                       stream, a, blocks);
  if (a.dX0) {
    const int64_t waves = (int64_t)a.seqs * tiles;
    hipLaunchKernelGGL((conv_before_kernel<E, V, K>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a, tiles,
                       waves);
  }
  return hipGetLastError();
}

enum class ConvCall { forward, step, backward };
template <class E, int V, int K>
static hipError_t conv_run(const ConvArgs &a, ConvCall call, hipStream_t stream) {
  // backward holds twice the arrays: half the channels a lane
  if (call == ConvCall::backward) return conv_backward<E, (V > 4 ? 4 : V), K>(a, stream);
  return call == ConvCall::step ? conv_step<E, V, K>(a, stream) : conv_forward<E, V, K>(a, stream);
}
template <class E, int V>
static hipError_t conv_run(const ConvArgs &a, ConvCall call, hipStream_t stream) {
  return a.width == 2 ? conv_run<E, V, 2>(a, call, stream)
         : a.width == 3 ? conv_run<E, V, 3>(a, call, stream)
                        : conv_run<E, V, 4>(a, call, stream);
}
static hipError_t conv_run(const ConvArgs &a, int dtype, bool wide, ConvCall call, hipStream_t stream) {
  if (wide)
    return dtype == 0 ? conv_run<F32, 4>(a, call, stream)
           : dtype == 1 ? conv_run<BF16, 8>(a, call, stream)
                        : conv_run<F16, 8>(a, call, stream);
  return dtype == 0 ? conv_run<F32, 1>(a, call, stream)
         : dtype == 1 ? conv_run<BF16, 1>(a, call, stream)
                      : conv_run<F16, 1>(a, call, stream);
}

hipError_t launch_conv(const ConvArgs &a, int dtype, bool wide, hipStream_t stream) {
  return conv_run(a, dtype, wide, ConvCall::forward, stream);
}
hipError_t launch_conv_step(const ConvArgs &a, int dtype, bool wide, hipStream_t stream) {
  return conv_run(a, dtype, wide, ConvCall::step, stream);
}
hipError_t launch_conv_backward(const ConvArgs &a, int dtype, bool wide, hipStream_t stream) {
  return conv_run(a, dtype, wide, ConvCall::backward, stream);
}

}  // namespace lq
