// Device-side helpers of the operators around the recurrence: the sequence of
// a token, vectors of neighbouring elements, exponentials and the functions
// made of them.
#pragma once
#include "lq_layer.h"
#include "lq_sequence_device.h"

namespace lq {

// Offsets are device data: they are held to [0, tokens], so that wrong ones
// cannot lead outside the arrays.
__device__ __forceinline__ int seq_offset(const int32_t *cu, int64_t tokens, int i) {
  const int c = cu[i];
  return __builtin_amdgcn_readfirstlane(c < 0 ? 0 : (c > tokens ? (int)tokens : c));
}

// The last i of [0, seqs) with offset(i) / chunk + i * step <= at, or -1.
// All 64 lanes search together, 64 boundaries a step.
__device__ __forceinline__ int seq_search(const int32_t *cu, int64_t tokens, int seqs, int chunk, int step, int at,
                                          int lane) {
  int lo = 0, n = seqs;
  while (n > 0) {
    const int stride = (n + 63) >> 6;
    const int i = lo + lane * stride;
    bool below = false;
    if (lane * stride < n) {
      const int c = cu[i];
      const int o = c < 0 ? 0 : (c > tokens ? (int)tokens : c);
      below = o / chunk + i * step <= at;
    }
    const int m = __popcll(__ballot(below));
    if (m == 0) return lo - 1;  // (only in the first round: later ones begin below `at`)
    lo += (m - 1) * stride;
    if (stride == 1) return lo;
    const int left = n - (m - 1) * stride;
    n = left < stride ? left : stride;
  }
  return lo - 1;
}

// V neighbouring elements as loaded: 16 bytes (or 8), or one element
template <class E, int V> struct Vec { E e[V]; };
template <class E, int V>
__device__ __forceinline__ Vec<E, V> vec_load(const E *p) {
  constexpr int bytes = sizeof(E) * V;
  static_assert(V == 1 || bytes == 16 || bytes == 8, "one element, 8 or 16 bytes");
  Vec<E, V> r;
  if constexpr (V == 1) {
    r.e[0] = p[0];
  } else if constexpr (bytes == 16) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    __builtin_memcpy(&r, &a, 16);
  } else {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    __builtin_memcpy(&r, &a, 8);
  }
  return r;
}
template <class E, int V>
__device__ __forceinline__ void vec_store(E *p, const Vec<E, V> &r) {
  constexpr int bytes = sizeof(E) * V;
  if constexpr (V == 1) {
    p[0] = r.e[0];
  } else if constexpr (bytes == 16) {
    uint4 a;
    __builtin_memcpy(&a, &r, 16);
    *reinterpret_cast<uint4 *>(p) = a;
  } else {
    uint2 a;
    __builtin_memcpy(&a, &r, 8);
    *reinterpret_cast<uint2 *>(p) = a;
  }
}
template <class E, int V>
__device__ __forceinline__ void vec_floats(float (&x)[V], const Vec<E, V> &r) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = to_f(r.e[v]);
}
template <class E, int V>
__device__ __forceinline__ Vec<E, V> vec_round(const float (&x)[V]) {
  Vec<E, V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) r.e[v] = from_f<E>(x[v]);
  return r;
}

constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.925963033500e-8f, kLn2 = 0.69314718055994530942f;

// e^x: the product with log2 e rounds by up to |x| 2^-24 of an exponent, so
// its rest goes into the result (x = -7 otherwise leaves 3e-7)
__device__ __forceinline__ float exp_full(float x) {
  const float p = x * kLog2e;
  const float rest = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -p));
  const float e = __builtin_amdgcn_exp2f(p);
  // beyond the exponent's range the rest says nothing (an infinite x has none)
  return fabsf(x) < 87.f ? fmaf(e, rest * kLn2, e) : e;
}
// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_full(-x)); }
// The same of x made of inputs of type E, for results of type E: where these have 16
// bits, without the rest of the exponent's product (up to 1.25 |x| 2^-24 of e^-x), at
// half of the instructions.  The half step of a gate's input is 2^13 times that and
// more, also for the fp32 sums that it enters (gradients of weights and of an fp32
// stream).  Kernels that wait for memory anyway keep the full form: the norm forward
// and the single tokens' gate.
template <class E>
__device__ __forceinline__ float sigmoid_for(float x) {
  if constexpr (sizeof(E) == 4) return sigmoid(x);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

}  // namespace lq
