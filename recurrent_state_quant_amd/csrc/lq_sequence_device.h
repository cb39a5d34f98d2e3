// Device-side helpers shared by the sequence kernels (lq_sequence.hip,
// lq_sequence_grad.hip): element types, chunk lookup, decays of a chunk, and
// matrix fragments in fp32 and in bf16 parts.
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

// N neighbouring values (N = 1 or 2, aligned to N elements), as loaded
template <int N, class E>
__device__ __forceinline__ void load_raw(const E *p, E (&x)[N]) {
  static_assert(N == 1 || N == 2, "one or two values");
  if constexpr (N == 1) {
    x[0] = p[0];
  } else if constexpr (sizeof(E) == 4) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    x[0] = __builtin_bit_cast(E, a.x);
    x[1] = __builtin_bit_cast(E, a.y);
  } else {
    const uint32_t a = *reinterpret_cast<const uint32_t *>(p);
    x[0] = __builtin_bit_cast(E, (uint16_t)a);
    x[1] = __builtin_bit_cast(E, (uint16_t)(a >> 16));
  }
}
template <int N, class E>
__device__ __forceinline__ void store_raw(E *p, const E (&x)[N]) {
  if constexpr (N == 1) {
    p[0] = x[0];
  } else if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(__builtin_bit_cast(uint32_t, x[0]), __builtin_bit_cast(uint32_t, x[1]));
  } else {
    *reinterpret_cast<uint32_t *>(p) =
        __builtin_bit_cast(uint16_t, x[0]) | (uint32_t)__builtin_bit_cast(uint16_t, x[1]) << 16;
  }
}
template <int N>
__device__ __forceinline__ void load_n(const float *p, float (&x)[N]) {
  if constexpr (N == 1) {
    x[0] = p[0];
  } else {
    const float2 a = *reinterpret_cast<const float2 *>(p);
    x[0] = a.x;
    x[1] = a.y;
  }
}
template <int N>
__device__ __forceinline__ void store_n(float *p, const float (&x)[N]) {
  if constexpr (N == 1)
    __builtin_nontemporal_store(x[0], p);
  else
    __builtin_nontemporal_store(vf2{x[0], x[1]}, reinterpret_cast<vf2 *>(p));
}
// [rows][128] fp32 arrays that the scans keep for the backward pass: four rows
// together, [rows / 4][column][4], as a lane's accumulator holds them, so that
// it is stored in one piece.  In a run of 32 columns the even ones come first:
// a store covers whole lines whether a lane has one column or two.  Streaming
// stores: these arrays outgrow the caches.
__device__ __forceinline__ int quad_at(int quad, int col) {
  return quad * D + (col & ~31) + (col & 1) * 16 + ((col & 31) >> 1);
}
__device__ __forceinline__ void store_quad(float *p, int quad, int col, floatx4 x) {
  __builtin_nontemporal_store(x, reinterpret_cast<floatx4 *>(p) + quad_at(quad, col));
}
// four values at p (aligned to four elements)
__device__ __forceinline__ void load4(const F32 *p, float (&x)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
__device__ __forceinline__ void load4(const BF16 *p, float (&x)[4]) {
  const uint2 a = *reinterpret_cast<const uint2 *>(p);
  x[0] = __uint_as_float(a.x << 16); x[1] = __uint_as_float(a.x & 0xFFFF0000u);
  x[2] = __uint_as_float(a.y << 16); x[3] = __uint_as_float(a.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const F16 *p, float (&x)[4]) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  const f16x4 a = *reinterpret_cast<const f16x4 *>(p);
  x[0] = (float)a[0]; x[1] = (float)a[1]; x[2] = (float)a[2]; x[3] = (float)a[3];
}
// four results, rounded, at p (aligned to four elements)
__device__ __forceinline__ void store4(F32 *p, floatx4 x) { *reinterpret_cast<floatx4 *>(p) = x; }
__device__ __forceinline__ void store4(BF16 *p, floatx4 x) {
  ushort4 v = make_ushort4(from_f<BF16>(x[0]).x, from_f<BF16>(x[1]).x, from_f<BF16>(x[2]).x, from_f<BF16>(x[3]).x);
  *reinterpret_cast<ushort4 *>(p) = v;
}
__device__ __forceinline__ void store4(F16 *p, floatx4 x) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<f16x4 *>(p) = f16x4{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
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

// The sequence of the n-th place in a scan's grid.  Where the grid is more than
// the chip holds at once (one or two workgroups a CU), the longest come first,
// so that the last workgroups to begin are short ones: 19 sequences x 16 heads
// 106 us, 130 in their order; 5 x 32 with a decay a channel 164, 179.  A wave
// ranks up to 64 lengths; more sequences even out by themselves.
__device__ __forceinline__ int seq_place(const SeqArgs &A, int n, int64_t workgroups, int lane) {
  if (workgroups <= 512 || A.seqs > 64 || A.seqs == 1) return n;
  int len = -1;
  if (lane < A.seqs) {
    const int start = seq_start(A, lane);
    len = seq_end(A, lane, start) - start;
  }
  int rank = 0;
  for (int j = 0; j < A.seqs; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    rank += other > len || (other == len && j < lane) ? 1 : 0;
  }
  return __builtin_amdgcn_readfirstlane(__ffsll(__ballot(lane < A.seqs && rank == n)) - 1);
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

// L[i][j] = product of al[j + 1 .. i] (1 on the diagonal, 0 above) into lds
// [64][LDC]: running products, no logarithm and no division, so decays of
// zero are exact.  Thread (column j, block of 16 rows, one a wave).
__device__ __forceinline__ void decay_matrix(float *L, const float *al, int w, int lane) {
  const int j = lane, i0 = 16 * w;
  float p = 1.f;
  for (int l = 0; l < i0; l += 4) {
    const float4 a = *reinterpret_cast<const float4 *>(al + l);
    p *= l > j ? a.x : 1.f;
    p *= l + 1 > j ? a.y : 1.f;
    p *= l + 2 > j ? a.z : 1.f;
    p *= l + 3 > j ? a.w : 1.f;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = i0 + e;
    p *= i > j ? al[i] : 1.f;
    L[i * LDC + j] = i >= j ? p : 0.f;
  }
}

// ---------------------------------------------------------------------------
// bf16 parts.  The matrix path runs bf16 eight times as fast as fp32, and an
// fp32 value is the exact sum of three bf16 parts (each the nearest to what
// the previous ones leave), an fp16 value of two, a bf16 value is one.  A
// product of two values takes the products of their parts that are not below
// 2^-24 of it: parts (i, j) with i + j <= 2, where a dropped product has the
// size of one fp32 rounding.  Sums are fp32 in the matrix unit.  Results in 16
// bits take no fewer parts: their terms may cancel (a token that overwrites a
// large state: Q S0 and P U), and the parts count beside the terms, not beside
// what is left of them.
// ---------------------------------------------------------------------------
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef float fl2 __attribute__((ext_vector_type(2)));

template <class E> struct Parts;
template <> struct Parts<BF16> { static constexpr int n = 1; };
template <> struct Parts<F16> { static constexpr int n = 2; };
template <> struct Parts<F32> { static constexpr int n = 3; };

__device__ __forceinline__ uint32_t pair_bf16(float x, float y) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((fl2){x, y}, bf2));
}
// N parts of the pair (x, y), as words
template <int N>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    p[n] = pair_bf16(x, y);
    if (n + 1 < N) {
      x -= __uint_as_float(p[n] << 16);
      y -= __uint_as_float(p[n] & 0xFFFF0000u);
    }
  }
}
template <int N>
__device__ __forceinline__ void split8(const float (&x)[8], bf8 (&out)[N]) {
  uint32_t w[N][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t p[N];
    split_pair<N>(x[2 * e], x[2 * e + 1], p);
#pragma unroll
    for (int n = 0; n < N; ++n) w[n][e] = p[n];
  }
#pragma unroll
  for (int n = 0; n < N; ++n) out[n] = __builtin_bit_cast(bf8, make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]));
}
// Operand fragments of v_mfma_f32_16x16x32_bf16: lane (i = lane & 15, g =
// lane >> 4) holds row (or column) i, contraction indexes 8 g .. 8 g + 7.
__device__ __forceinline__ floatx4 mma16(bf8 a, bf8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// All products of parts (i, j), i + j <= 2, small ones first, alternating
// between two sums: a product that adds to the previous one's result waits for
// it, and a wave has few tiles to change between.
struct Acc2 {
  floatx4 a, b;
  __device__ __forceinline__ floatx4 sum() const { return a + b; }
};
__device__ __forceinline__ Acc2 acc2_zero() {
  return Acc2{floatx4{0.f, 0.f, 0.f, 0.f}, floatx4{0.f, 0.f, 0.f, 0.f}};
}
template <int NA, int NB>
__device__ __forceinline__ void mma_parts(Acc2 &c, const bf8 (&a)[NA], const bf8 (&b)[NB]) {
  int k = 0;
#pragma unroll
  for (int t = 2; t >= 0; --t)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = t - i;
      if (j >= 0 && j < NB) {
        if (k++ & 1)
          c.b = mma16(a[i], b[j], c.b);
        else
          c.a = mma16(a[i], b[j], c.a);
      }
    }
}
// the same into one sum, for waves with many tiles to change between
template <int NA, int NB>
__device__ __forceinline__ void mma_into(floatx4 &c, const bf8 (&a)[NA], const bf8 (&b)[NB]) {
#pragma unroll
  for (int t = 2; t >= 0; --t)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = t - i;
      if (j >= 0 && j < NB) c = mma16(a[i], b[j], c);
    }
}
// N planes of a fragment out of LDS rows of ld elements, `plane` apart
template <int N>
__device__ __forceinline__ void frag16(bf8 (&f)[N], const uint16_t *p, int plane, int ld, int r0, int k0, int lane) {
  const uint16_t *s = p + (r0 + (lane & 15)) * ld + k0 + 8 * (lane >> 4);
#pragma unroll
  for (int n = 0; n < N; ++n) f[n] = *reinterpret_cast<const bf8 *>(s + n * plane);
}
// the same with the contraction as the array's outer axis
template <int N>
__device__ __forceinline__ void frag_gather(bf8 (&f)[N], const uint16_t *p, int plane, int ld, int r0, int k0, int lane) {
  const uint16_t *s = p + (k0 + 8 * (lane >> 4)) * ld + r0 + (lane & 15);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int t = 0; t < 8; ++t) f[n][t] = __builtin_bit_cast(__bf16, s[n * plane + t * ld]);
}
// N fragments stored one behind another in fragment order (64 lanes x 16 bytes)
template <int N>
__device__ __forceinline__ void frag_load(bf8 (&f)[N], const uint16_t *p, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n) f[n] = reinterpret_cast<const bf8 *>(p)[64 * n + lane];
}
template <int N>
__device__ __forceinline__ void frag_store(uint16_t *p, const bf8 (&f)[N], int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n) reinterpret_cast<bf8 *>(p)[64 * n + lane] = f[n];
}
// Fragments that the waves of a workgroup share, in LDS in fragment order
// (16 bytes a lane, one lane behind another: no bank is asked twice), parts
// F fragments apart.  A wave writes four values of column i out of its
// accumulators, contraction indexes 16 t + 4 g .. + 3 of a step of 32 (t: 0, 1).
template <int N, int F>
__device__ __forceinline__ void frag_share(uint16_t *p, int f, int t, int lane, float x0, float x1, float x2, float x3) {
  const int i = lane & 15, g = lane >> 4;
  uint32_t a[N], b[N];
  split_pair<N>(x0, x1, a);
  split_pair<N>(x2, x3, b);
  uint16_t *d = p + f * 512 + (i + 16 * (2 * t + (g >> 1))) * 8 + (g & 1) * 4;
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<uint2 *>(d + n * F * 512) = make_uint2(a[n], b[n]);
}
template <int N, int F>
__device__ __forceinline__ void frag_get(bf8 (&f)[N], const uint16_t *p, int at, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n) f[n] = *reinterpret_cast<const bf8 *>(p + (n * F + at) * 512 + lane * 8);
}
// N parts of eight values of a head's row
template <class E, int N>
__device__ __forceinline__ void parts_load(bf8 (&f)[N], const E *p) {
  if constexpr (N == 1) {
    f[0] = *reinterpret_cast<const bf8 *>(p);
  } else {
    float x[8];
    load8(p, x);
    split8<N>(x, f);
  }
}

// Eight values as loaded, and their parts
template <class E> struct Raw8 { uint4 v[sizeof(E) / 2]; };
template <class E>
__device__ __forceinline__ Raw8<E> raw_load(const E *p) {
  Raw8<E> r;
#pragma unroll
  for (int n = 0; n < (int)(sizeof(E) / 2); ++n) r.v[n] = reinterpret_cast<const uint4 *>(p)[n];
  return r;
}
__device__ __forceinline__ void raw_floats(float (&x)[8], const Raw8<F32> &r) {
  const float4 a = __builtin_bit_cast(float4, r.v[0]), b = __builtin_bit_cast(float4, r.v[1]);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void raw_floats(float (&x)[8], const Raw8<BF16> &r) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void raw_floats(float (&x)[8], const Raw8<F16> &r) {
  const f16x8 h = __builtin_bit_cast(f16x8, r.v[0]);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)h[e];
}
template <class E, int N>
__device__ __forceinline__ void raw_parts(bf8 (&f)[N], const Raw8<E> &r) {
  if constexpr (N == 1) {
    f[0] = __builtin_bit_cast(bf8, r.v[0]);
  } else {
    float x[8];
    raw_floats(x, r);
    split8<N>(x, f);
  }
}

// Every load so far is done (vmcnt(0)).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Barrier for data in LDS only: loads and stores of global memory stay in
// flight across it (__syncthreads waits for them too).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace lq
