// Device-side helpers of the selective scan (lq_scan.hip, lq_scan_grad.hip).
#pragma once
#include <type_traits>

#include "lq_layer_device.h"

namespace lq {

// max(v, 0) + log(1 + e), e = e^-|v| in (0, 1].  log(1 + e) = 2 artanh(r) with
// r = e / (2 + e) <= 1/3, and artanh(r) = r (1 + r^2 P(r^2)) with a polynomial P
// fitted to the series 1/3 + r^2 / 5 + .. on [0, 1/9] (least largest error of the
// whole: 5.4e-9 relative): exact to rounding also where e is tiny, as it is for
// the small steps that such layers take.
__device__ __forceinline__ float softplus_of(float v, float e) {
  const float r = e * __builtin_amdgcn_rcpf(2.f + e), q = r * r;
  float p = fmaf(q, 0.14005996f, 0.14000902f);
  p = fmaf(p, q, 0.20010763f);
  p = fmaf(p, q, 0.33333209f);
  p = fmaf(p * q, r, r);
  return fmaf(2.f, p, fmaxf(v, 0.f));
}
// the step of a token and channel from its input v
__device__ __forceinline__ float scan_step(const ScanArgs &A, float v) {
  return A.softplus ? softplus_of(v, exp_full(-fabsf(v))) : v;
}
// The same with the step's derivative by v.
__device__ __forceinline__ float scan_step(const ScanArgs &A, float v, float &slope) {
  slope = 1.f;
  if (!A.softplus) return v;
  const float e = exp_full(-fabsf(v)), s = __builtin_amdgcn_rcpf(1.f + e);
  slope = v >= 0.f ? s : e * s;
  return softplus_of(v, e);
}

// A row of B or C: N values that are the same for the whole wave, through the
// scalar cache (the address is made of wave-uniform values), so that they cost
// the vector units nothing but their use as an operand.
template <class E, int N> struct ScanRow {
  static constexpr int words = N * (int)sizeof(E) / 4;
  uint32_t w[words];
  __device__ __forceinline__ void load(const Rows &r, int t, int g) {
    typedef const uint32_t __attribute__((address_space(4))) *scalars;
    const scalars p = (scalars)(uintptr_t)at<const E>(r, t, g);
#pragma unroll
    for (int i = 0; i < words; ++i) w[i] = p[i];
  }
  __device__ __forceinline__ float operator[](int n) const {
    if constexpr (sizeof(E) == 4)
      return __uint_as_float(w[n]);
    else
      return to_f(__builtin_bit_cast(E, (uint16_t)(w[n >> 1] >> (16 * (n & 1)))));
  }
};
// x b, as a fused product and sum with zero for fp16: that instruction takes an
// fp16 operand as it is
template <class E>
__device__ __forceinline__ float scan_times(float x, float b) {
  if constexpr (std::is_same_v<E, F16>) return fmaf(x, b, 0.f);
  return x * b;
}
// A wave's channels: 64 of one group, one a lane.
struct ScanTile {
  int g;        // group
  int c;        // this lane's channel (of lanes without one: the group's last)
  bool on;      // this lane has a channel
};
__device__ __forceinline__ ScanTile scan_tile(const ScanArgs &A, int g, int tile, int lane) {
  const int first = tile * 64 + lane;
  ScanTile r;
  r.g = g;
  r.on = first < A.per;
  r.c = g * A.per + (r.on ? first : A.per - 1);
  return r;
}

// The chunk of a slot
struct ScanChunk {
  int i, c, chunks;  // sequence, chunk, chunks of the sequence
  int start, t0, t1; // the sequence's first token, the chunk's tokens [t0, t1)
  bool any;          // the slot has a chunk (an empty sequence has one of no tokens)
};
__device__ __forceinline__ ScanChunk scan_chunk(const ScanArgs &A, int chunk, int slot, int lane) {
  ScanChunk k{0, 0, 0, 0, 0, 0, false};
  k.i = seq_search(A.cu, A.tokens, A.seqs, chunk, 1, slot, lane);
  if (k.i < 0) return k;
  k.start = seq_offset(A.cu, A.tokens, k.i);
  const int end = max(k.start, seq_offset(A.cu, A.tokens, k.i + 1));
  k.chunks = (end - k.start + chunk - 1) / chunk;
  k.c = slot - (k.start / chunk + k.i);
  if (k.c < 0 || (k.c >= k.chunks && k.c > 0)) return k;
  k.any = true;
  k.t0 = k.start + k.c * chunk;
  k.t1 = min(end, k.t0 + chunk);
  return k;
}

// Element c of a row whose address is the same for the wave: the address stays
// in scalar registers (it is hidden from the compiler, which would otherwise add
// it to the lane's offset first, in vector registers), the lane's offset is one
// register for all rows (of at most 2^20 elements).
template <class T> using lane_bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
template <class T>
__device__ __forceinline__ uintptr_t row_address(T *row) {
  uintptr_t p = reinterpret_cast<uintptr_t>(row);
  asm("" : "+s"(p));
  return p;
}
template <class T>
__device__ __forceinline__ T lane_load(const T *row, int c) {
  typedef const char __attribute__((address_space(1))) *bytes;
  typedef const lane_bits<T> __attribute__((address_space(1))) *global;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(T);
  return __builtin_bit_cast(T, *(global)((bytes)row_address(row) + off));
}
template <class T>
__device__ __forceinline__ void lane_store(T *row, int c, T x) {
  typedef char __attribute__((address_space(1))) *bytes;
  typedef lane_bits<T> __attribute__((address_space(1))) *global;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(T);
  *(global)((bytes)row_address(row) + off) = __builtin_bit_cast(lane_bits<T>, x);
}
// The kernel's arguments (its first) read again where they are used: pointers
// and strides of a dozen arrays do not stay in scalar registers that way.
__device__ __forceinline__ const ScanArgs &scan_args() {
  uintptr_t p = (uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm("" : "+s"(p));
  return *(const ScanArgs *)(const ScanArgs __attribute__((address_space(4))) *)p;
}
// The slot of the chunks from zero (M of them in one of k's) that chunk k begins
// with, and ends with.
__device__ __forceinline__ int64_t scan_first_part(const ScanArgs &A, const ScanChunk &k) {
  return k.start / A.part + k.i + (int64_t)k.c * (A.chunk / A.part);
}
__device__ __forceinline__ int64_t scan_last_part(const ScanArgs &A, const ScanChunk &k) {
  return k.start / A.part + k.i + (k.t1 - k.start + A.part - 1) / A.part - 1;
}
// A channel's states from or to [states][channels] or [channels][states]
template <int N>
__device__ __forceinline__ void scan_load_cols(const float *p, int64_t channels, int c, float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = lane_load(p + n * channels, c);
}
template <int N>
__device__ __forceinline__ void scan_store_cols(float *p, int64_t channels, int c, const float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) lane_store(p + n * channels, c, h[n]);
}
template <int N>
__device__ __forceinline__ void scan_load_rows(const float *p, int64_t row, float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; n += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p + row * N + n);
    h[n] = v.x; h[n + 1] = v.y; h[n + 2] = v.z; h[n + 3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void scan_store_rows(float *p, int64_t row, const float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; n += 4)
    *reinterpret_cast<float4 *>(p + row * N + n) = make_float4(h[n], h[n + 1], h[n + 2], h[n + 3]);
}
// decays as exponents of two: e^(d A) = 2^(d A log2 e)
template <int N>
__device__ __forceinline__ void scan_decays(const ScanArgs &A, int c, float (&a2)[N]) {
  scan_load_rows<N>(A.A, c, a2);
#pragma unroll
  for (int n = 0; n < N; ++n) a2[n] *= kLog2e;
}

}  // namespace lq
