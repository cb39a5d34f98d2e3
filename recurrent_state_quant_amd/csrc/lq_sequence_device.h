// Device-side helpers shared by the sequence kernels (lq_sequence.hip,
// lq_sequence_grad.hip): element types, chunk lookup, decays of a chunk, and
// fp32 matrix tiles out of LDS.
#pragma once
#include "lq_device.h"
#include "lq_sequence.h"

namespace lq {

constexpr int C = kChunk;
constexpr int LDD = D + 4;  // row of a [.][128] fp32 tile in LDS
constexpr int LDC = C + 4;  // row of a [.][64] fp32 tile in LDS

typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Element types of q, k, v, o and their gradients.
struct F32 { float x; };
struct BF16 { uint16_t x; };
struct F16 { _Float16 x; };

__device__ __forceinline__ float to_f(F32 e) { return e.x; }
__device__ __forceinline__ float to_f(BF16 e) { return __uint_as_float((uint32_t)e.x << 16); }
__device__ __forceinline__ float to_f(F16 e) { return (float)e.x; }
template <class E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ F32 from_f<F32>(float x) { return F32{x}; }
// results leave the kernels rounded once, to the nearest value of the type
template <> __device__ __forceinline__ BF16 from_f<BF16>(float x) {
  return BF16{__builtin_bit_cast(uint16_t, (__bf16)x)};
}
template <> __device__ __forceinline__ F16 from_f<F16>(float x) { return F16{(_Float16)x}; }

// eight elements at p (16-byte aligned)
__device__ __forceinline__ void load8(const F32 *p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const BF16 *p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const F16 *p, float (&x)[8]) {
  const f16x8 a = *reinterpret_cast<const f16x8 *>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)a[e];
}
__device__ __forceinline__ void store8(F32 *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(BF16 *p, const float (&x)[8]) {
  u16x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = from_f<BF16>(x[e]).x;
  *reinterpret_cast<u16x8 *>(p) = v;
}
__device__ __forceinline__ void store8(F16 *p, const float (&x)[8]) {
  f16x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (_Float16)x[e];
  *reinterpret_cast<f16x8 *>(p) = v;
}

// address of (token, head) of a strided array; every offset in 64 bits
template <class E>
__device__ __forceinline__ E *at(const Rows &r, int64_t t, int h) {
  return reinterpret_cast<E *>(r.ptr) + t * r.ts + (int64_t)h * r.hs;
}

// Sequence i's tokens.  Offsets are device data: they are held to
// [0, tokens], so that wrong ones cannot lead outside the arrays.
__device__ __forceinline__ int seq_start(const SeqArgs &A, int i) {
  const int c = A.cu[i];
  return c < 0 ? 0 : (c > A.tokens ? (int)A.tokens : c);
}
__device__ __forceinline__ int seq_end(const SeqArgs &A, int i, int start) {
  const int c = seq_start(A, i + 1);
  return c < start ? start : c;
}

struct Chunk {
  int t0, len;  // first token; tokens (0: the slot holds no chunk)
};
// The chunk of a slot: sequence i is the last with cu[i] / 64 + i <= slot.
// All 64 lanes search together, 64 boundaries a step.
__device__ __forceinline__ Chunk find_chunk(const SeqArgs &A, int slot, int lane) {
  int lo = 0, n = A.seqs;
  while (n > 0) {
    const int step = (n + 63) >> 6;
    const int i = lo + lane * step;
    const bool below = lane * step < n && seq_start(A, i) / C + i <= slot;
    const int m = __popcll(__ballot(below));
    if (m == 0) return Chunk{0, 0};
    lo += (m - 1) * step;
    const int left = n - (m - 1) * step;
    n = left < step ? left : step;
    if (step == 1) break;
  }
  const int start = seq_start(A, lo), end = seq_end(A, lo, start);
  const int c = slot - (start / C + lo);
  if (c < 0) return Chunk{0, 0};
  const int t0 = start + c * C;
  const int len = end - t0;
  return Chunk{t0, len < 0 ? 0 : (len > C ? C : len)};
}

// rows t0 .. t0 + 63 of head h as fp32 into lds [64][LDD], zeros past len;
// 256 threads
template <class E>
__device__ __forceinline__ void stage_rows(float *lds, const Rows &r, int h, int t0, int len, int tid) {
  const int row = tid >> 2, c0 = (tid & 3) * 8;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row < len) load8(at<const E>(r, t0 + row, h) + c0 + 32 * c, x);
    float4 *d = reinterpret_cast<float4 *>(lds + row * LDD + c0 + 32 * c);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// a dense fp32 [rows][cols] block into lds rows of ld; 256 threads
template <int COLS>
__device__ __forceinline__ void stage_f32(float *lds, int ld, const float *src, int rows, int tid) {
  constexpr int Q = COLS / 4;
  for (int e = tid; e < rows * Q; e += 256) {
    const int r = e / Q, c = e % Q;
    *reinterpret_cast<float4 *>(lds + r * ld + 4 * c) = reinterpret_cast<const float4 *>(src)[e];
  }
}

// Operand of a 16x16 tile of v_mfma_f32_16x16x4_f32 for sixteen steps of the
// contraction: lane (i = lane & 15, g = lane >> 4) holds row (or column) r0 +
// i at contraction indexes 16 kk + 4 g .. + 3.  The order of the contraction
// is the same permutation for both operands, so four 16x16x4 products cover
// sixteen indexes out of one 16-byte read per lane.
// TR: the array is stored with the contraction as its outer axis.
template <bool TR>
__device__ __forceinline__ float4 frag(const float *p, int ld, int r0, int kk, int lane) {
  const int i = lane & 15, g = lane >> 4;
  if (!TR) return *reinterpret_cast<const float4 *>(p + (r0 + i) * ld + 16 * kk + 4 * g);
  const float *s = p + (16 * kk + 4 * g) * ld + r0 + i;
  return make_float4(s[0], s[ld], s[2 * ld], s[3 * ld]);
}
// acc[r] is row 4 (lane >> 4) + r, column lane & 15 of the tile
__device__ __forceinline__ void mma(floatx4 &acc, float4 a, float4 b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x, b.x, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.y, b.y, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.z, b.z, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.w, b.w, acc, 0, 0, 0);
}

// The same operand straight from row t0 + r0 + i of a strided array.
template <class E>
__device__ __forceinline__ float4 frag_rows(const Rows &r, int h, int t0, int len, int r0, int kk, int lane) {
  const int i = r0 + (lane & 15), g = lane >> 4;
  if (i >= len) return make_float4(0.f, 0.f, 0.f, 0.f);
  const E *p = at<const E>(r, t0 + i, h) + 16 * kk + 4 * g;
  return make_float4(to_f(p[0]), to_f(p[1]), to_f(p[2]), to_f(p[3]));
}

// L[i][j] = product of al[j + 1 .. i] (1 on the diagonal, 0 above) into lds
// [64][LDC]: running products, no logarithm and no division, so decays of
// zero are exact.  Thread (column j, block of 16 rows); 256 threads.
__device__ __forceinline__ void decay_matrix(float *L, const float *al, int tid) {
  const int j = tid & 63, i0 = (tid >> 6) * 16;
  float p = 1.f;
  for (int l = j + 1; l < i0; ++l) p *= al[l];
  for (int i = i0; i < i0 + 16; ++i) {
    if (i > j) p *= al[i];
    L[i * LDC + j] = i >= j ? p : 0.f;
  }
}

}  // namespace lq
