// Norm of query and key heads with the position rotation (gfx950), forward
// and backward.  For a head x of 128 values,
//   r = (sum x^2 + eps)^-1/2 (L2) or (mean x^2 + eps)^-1/2 (RMS)
//   y = s R(pos) (w * x * r)
// with R turning the first `rot` values in pairs (i, i + rot / 2), or (2i,
// 2i + 1) when interleaved, by pos * freq_i; s is q_scale for queries, 1 for
// keys.  Backward, with g = s R(-pos) dy:
//   dx = w r g - x r^3 (x . (w g)) / (1 or 128),   dw = sum g * x * r
//
// A wave takes one token and a run of its heads, four heads at a time:
// sixteen lanes hold a head, eight values each (one 16-byte access in 16-bit
// types).  The token's turns are computed once per wave, one pair's angle per
// lane, and shared through LDS.  The angle is a product in 64 bits, reduced
// to a fraction of a turn there (positions times frequencies reach 10^5
// radians, where 32 bits leave 2^-7), and its sine and cosine are taken in 32
// bits.  Bound by memory traffic: each head is read and written once.
// 16,384 tokens x 32 heads in bf16 48 us, 5.6 TB/s; 256 tokens x 64 heads 5.4
// us, where the launch is the time.
#include "lq_sequence_device.h"

namespace lq {

constexpr int kNormHeads = 16;  // heads of one wave

// Which (token, run of heads) a wave has
struct NormWork {
  int64_t t;
  int h0, h1;
};
__device__ __forceinline__ NormWork norm_work(const NormArgs &A, int64_t wave) {
  const int heads = A.hq + A.hk, runs = (heads + kNormHeads - 1) / kNormHeads;
  NormWork n;
  n.t = wave / runs;
  n.h0 = (int)(wave % runs) * kNormHeads;
  n.h1 = n.h0 + kNormHeads < heads ? n.h0 + kNormHeads : heads;
  return n;
}

// The token's turns: lane f holds the cosine and sine of pair f
__device__ __forceinline__ float2 norm_turn(const NormArgs &A, int64_t t, int lane) {
  float2 cs = make_float2(1.f, 0.f);
  if (lane < A.rot / 2) {
    const double turns = (double)A.pos[t] * A.freq[lane] * 0.15915494309189535;  // 1 / (2 pi)
    const float f = (float)(turns - rint(turns));
    sincospif(2.f * f, &cs.y, &cs.x);
  }
  return cs;
}

// The eight values' cosines and sines of a lane: half-split pairs need eight
// pairs, interleaved ones four.  `first` is the lane's first value.
__device__ __forceinline__ void norm_pairs(const NormArgs &A, const float2 *turn, int first, float (&c)[8], float (&s)[8]) {
  const int half = A.rot / 2;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = first + e;
    const int f = A.interleaved ? d >> 1 : (d < half ? d : d - half);
    const float2 x = d < A.rot ? turn[f] : make_float2(1.f, 0.f);
    c[e] = x.x;
    // the partner's sign: the pair's first value gets -sin, the second +sin
    const bool second = A.interleaved ? (d & 1) : d >= half;
    s[e] = d < A.rot ? (second ? x.y : -x.y) : 0.f;
  }
}
// y = R x (or R^-1 x with the sines negated by `sign`)
__device__ __forceinline__ void norm_rotate(const NormArgs &A, float (&x)[8], const float (&c)[8], const float (&s)[8],
                                            float sign, int lane) {
  if (A.rot == 0) return;
  float p[8];
  if (A.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = x[e ^ 1];
  } else {
    // the partner is rot / 16 lanes on or back, among the head's first rot / 8
    const int in = lane & 15, span = A.rot >> 4;
    const int from = in < span ? lane + span : (in < 2 * span ? lane - span : lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __shfl(x[e], from);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fmaf(sign * s[e], p[e], c[e] * x[e]);
}

// The weight's eight values of a lane (queries or keys)
__device__ __forceinline__ void norm_weights(const float *w, int first, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 1.f;
  if (w) load8(reinterpret_cast<const F32 *>(w + first), x);
}

template <class EI, class EO>
__global__ __launch_bounds__(256) void norm_kernel(const NormArgs A) {
  __shared__ float2 sh_turn[4][64];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, first = (lane & 15) * 8;
  const NormWork n = norm_work(A, (int64_t)blockIdx.x * 4 + w);
  const bool on = n.t < A.tokens;
  if (!on) return;  // whole waves; the waves share nothing
  // every load first: the run's heads, four a quarter wave (past the run's end: its last head again)
  Raw8<EI> raw[kNormHeads / 4];
#pragma unroll
  for (int k = 0; k < kNormHeads / 4; ++k) {
    int h = n.h0 + (lane >> 4) + 4 * k;
    h = h < n.h1 ? h : n.h1 - 1;
    const bool isq = h < A.hq;
    raw[k] = raw_load(at<const EI>(isq ? A.q : A.k, n.t, isq ? h : h - A.hq) + first);
  }
  float wq[8], wk[8], c[8], s[8];
  norm_weights(A.wq, first, wq);
  norm_weights(A.wk, first, wk);
  if (A.rot) {
    sh_turn[w][lane] = norm_turn(A, n.t, lane);
    __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses stay in order
    norm_pairs(A, sh_turn[w], first, c, s);
  }
#pragma unroll
  for (int k = 0; k < kNormHeads / 4; ++k) {
    const int h = n.h0 + (lane >> 4) + 4 * k;
    if (n.h0 + 4 * k >= n.h1) break;
    const bool isq = h < A.hq;
    float x[8], ss = 0.f;
    raw_floats(x, raw[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    ss = row16_sum(ss);
    const float r = 1.f / sqrtf(ss * (A.rms ? 1.f / D : 1.f) + A.eps) * (isq ? A.q_scale : 1.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= r * (isq ? wq[e] : wk[e]);
    norm_rotate(A, x, c, s, 1.f, lane);
    if (h < n.h1) store8(at<EO>(isq ? A.yq : A.yk, n.t, isq ? h : h - A.hq) + first, x);
  }
}

// Backward.  Weight gradients: a lane sums its eight values over the wave's
// tokens and heads, the workgroup's waves meet in LDS, and the workgroups'
// sums in `part` are added by a second launch, all in a fixed order.
// 8,192 tokens x 32 heads in bf16 44 us, 4.6 TB/s, and 4.6 us for the weights.
constexpr int kNormBackWaves = 8, kNormBackBlocks = 512;

template <class EI, class EO>
__global__ __launch_bounds__(64 * kNormBackWaves, 4) void norm_backward_kernel(const NormArgs A) {
  __shared__ float2 sh_turn[kNormBackWaves][64];
  __shared__ float sh_dw[kNormBackWaves][2][D];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, first = (lane & 15) * 8;
  const int heads = A.hq + A.hk, runs = (heads + kNormHeads - 1) / kNormHeads;
  const int64_t waves = A.tokens * runs, step = (int64_t)gridDim.x * kNormBackWaves;
  float dw[2][8], wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
  norm_weights(A.wq, first, wq);
  norm_weights(A.wk, first, wk);
  for (int64_t wave = (int64_t)blockIdx.x * kNormBackWaves + w; wave < waves; wave += step) {
    const NormWork n = norm_work(A, wave);
    float c[8], s[8];
    if (A.rot) {
      __builtin_amdgcn_wave_barrier();
      sh_turn[w][lane] = norm_turn(A, n.t, lane);
      __builtin_amdgcn_wave_barrier();
      norm_pairs(A, sh_turn[w], first, c, s);
    }
#pragma unroll 1
    for (int k0 = 0; k0 < kNormHeads / 4; k0 += 2) {  // two heads a quarter wave in flight
      if (n.h0 + 4 * k0 >= n.h1) break;
      Raw8<EI> rx[2];
      Raw8<EO> rg[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int h = n.h0 + (lane >> 4) + 4 * (k0 + k);
        h = h < n.h1 ? h : n.h1 - 1;
        const bool isq = h < A.hq;
        rx[k] = raw_load(at<const EI>(isq ? A.q : A.k, n.t, isq ? h : h - A.hq) + first);
        rg[k] = raw_load(at<const EO>(isq ? A.yq : A.yk, n.t, isq ? h : h - A.hq) + first);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = n.h0 + (lane >> 4) + 4 * (k0 + k);
        const bool isq = h < A.hq, mine = h < n.h1;
        float x[8], gy[8], ss = 0.f, xg = 0.f;
        raw_floats(x, rx[k]);
        raw_floats(gy, rg[k]);
        norm_rotate(A, gy, c, s, -1.f, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        ss = row16_sum(ss);
        const float r = 1.f / sqrtf(ss * (A.rms ? 1.f / D : 1.f) + A.eps), sc = isq ? A.q_scale : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ge = sc * gy[e], t = mine ? ge * x[e] * r : 0.f;
          dw[0][e] += isq ? t : 0.f;
          dw[1][e] += isq ? 0.f : t;
          gy[e] = ge * (isq ? wq[e] : wk[e]);
          xg = fmaf(x[e], gy[e], xg);
        }
        xg = row16_sum(xg) * (A.rms ? 1.f / D : 1.f) * r * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r * (gy[e] - x[e] * xg);
        if (mine) store8(at<EI>(isq ? A.dq : A.dk, n.t, isq ? h : h - A.hq) + first, x);
      }
    }
  }
  if (!A.dwq && !A.dwk) return;
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x = dw[p][e];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      if (lane < 16) sh_dw[w][p][first + e] = x;
    }
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const int p = threadIdx.x >> 7, d = threadIdx.x & 127;
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < kNormBackWaves; ++v) x += sh_dw[v][p][d];
    A.part[(int64_t)blockIdx.x * 2 * D + threadIdx.x] = x;
  }
}

// dw: workgroup (queries or keys, 32 values), thread (value, one of 32 shares
// of the partial sums)
__global__ __launch_bounds__(1024) void norm_weight_kernel(const NormArgs A, int blocks) {
  __shared__ float sh[32][33];
  const int p = blockIdx.x >> 2, d = (blockIdx.x & 3) * 32 + (threadIdx.x & 31), e = threadIdx.x >> 5;
  float x = 0.f;
#pragma unroll 8
  for (int b = e; b < blocks; b += 32) x += A.part[((int64_t)b * 2 + p) * D + d];
  sh[e][threadIdx.x & 31] = x;
  __syncthreads();
  float *out = p ? A.dwk : A.dwq;
  if (e == 0 && out) {
    float y = 0.f;
#pragma unroll
    for (int v = 0; v < 32; ++v) y += sh[v][threadIdx.x];
    out[d] = y;
  }
}

static int64_t norm_waves(int64_t tokens, int hq, int hk) {
  return tokens * ((hq + hk + kNormHeads - 1) / kNormHeads);
}
// The backward pass holds its partial weight gradients in registers, so its
// workgroups stay and take waves in turn; 512 of eight waves fill the chip.
int64_t norm_blocks(int64_t tokens, int hq, int hk) {
  const int64_t b = (norm_waves(tokens, hq, hk) + kNormBackWaves - 1) / kNormBackWaves;
  return b < kNormBackBlocks ? b : kNormBackBlocks;
}

template <class EI, class EO>
hipError_t norm_run(const NormArgs &a, bool back, hipStream_t stream) {
  if (!back) {
    const int64_t b = (norm_waves(a.tokens, a.hq, a.hk) + 3) / 4;
    hipLaunchKernelGGL((norm_kernel<EI, EO>), dim3((unsigned)b), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  const int64_t b = norm_blocks(a.tokens, a.hq, a.hk);
  if (b) hipLaunchKernelGGL((norm_backward_kernel<EI, EO>), dim3((unsigned)b), dim3(64 * kNormBackWaves), 0, stream, a);
  if (a.dwq || a.dwk) hipLaunchKernelGGL(norm_weight_kernel, dim3(8), dim3(1024), 0, stream, a, (int)b);
  return hipGetLastError();
}
template <class EI>
hipError_t norm_run(const NormArgs &a, int out, bool back, hipStream_t stream) {
  return out == 0 ? norm_run<EI, F32>(a, back, stream)
         : out == 1 ? norm_run<EI, BF16>(a, back, stream)
                    : norm_run<EI, F16>(a, back, stream);
}
static hipError_t norm_run(const NormArgs &a, int in, int out, bool back, hipStream_t stream) {
  return in == 0 ? norm_run<F32>(a, out, back, stream)
         : in == 1 ? norm_run<BF16>(a, out, back, stream)
                   : norm_run<F16>(a, out, back, stream);
}
hipError_t launch_norm(const NormArgs &a, int in, int out, hipStream_t stream) {
  return norm_run(a, in, out, false, stream);
}
hipError_t launch_norm_backward(const NormArgs &a, int in, int out, hipStream_t stream) {
  return norm_run(a, in, out, true, stream);
}

}  // namespace lq
