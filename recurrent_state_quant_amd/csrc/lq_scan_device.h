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
// e^-|v|.  For inputs of 16 bits without the rest of the exponent's product, which
// with that of log2 e itself is up to 1.25 |v| 2^-24 of the result (5e-7 at v = -7),
// and so are the fp32 states and gradients that the steps enter.  With a bias the sum
// v = dt + bias has rounded by up to |v| 2^-24 already, which leaves as much; without
// one v is the input, whose own half step is 2^13 (fp16) or 2^16 (bf16) times that.
template <class E>
__device__ __forceinline__ float scan_exp(float v) {
  if constexpr (sizeof(E) == 4) return exp_full(-fabsf(v));
  return __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
}
// The steps of a lane's tokens from their inputs v (in one branch: one a token
// would keep the tokens' instructions apart)
template <class E, int K>
__device__ __forceinline__ void scan_steps(const ScanArgs &A, float (&v)[K]) {
  if (!A.softplus) return;
#pragma unroll
  for (int u = 0; u < K; ++u) v[u] = softplus_of(v[u], scan_exp<E>(v[u]));
}
// The same with the steps' derivatives by v.
template <class E, int K>
__device__ __forceinline__ void scan_steps(const ScanArgs &A, float (&v)[K], float (&slope)[K]) {
#pragma unroll
  for (int u = 0; u < K; ++u) slope[u] = 1.f;
  if (!A.softplus) return;
#pragma unroll
  for (int u = 0; u < K; ++u) {
    const float e = scan_exp<E>(v[u]), s = __builtin_amdgcn_rcpf(1.f + e);
    slope[u] = v[u] >= 0.f ? s : e * s;
    v[u] = softplus_of(v[u], e);
  }
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
// Stores of lanes that may have nothing to store, without a branch: one around
// them would leave the compiler with an unknown number of stores in flight, and so
// waiting for all of them wherever it needs a load that came before.  `bytes` is
// the row's length, at most 2^24; lanes of no channel have an offset behind it (and
// far enough from 2^32 that nothing wraps).
__device__ __forceinline__ uint32_t lane_offset(bool on, int c, int size) { return on ? (uint32_t)c * size : 1u << 30; }
template <class T>
__device__ __forceinline__ void lane_store(T *row, int bytes, uint32_t off, T x) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(row_address(row)), (short)0, bytes, 0x00020000);
  if constexpr (sizeof(T) == 2)
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(lane_bits<T>, x), r, (int)off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(lane_bits<T>, x), r, (int)off, 0, 0);
}

// A row of B or C: N values that are the same for the whole wave, through the
// scalar cache (the address is made of wave-uniform values), so that they cost
// the vector units nothing but their use as an operand.
template <class E, int N> struct ScanRow {
  static constexpr int words = N * (int)sizeof(E) / 4;
  uint32_t w[words];
  __device__ __forceinline__ void load(const E *row) {
    typedef const uint32_t __attribute__((address_space(4))) *scalars;
    const scalars p = (scalars)(uintptr_t)row;
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

// The same row as a matrix operand: lane l holds value l mod 16 (N = 8: mod 8) of
// each sixteen.  s[n] += row[n] x for every lane's own x is then one instruction
// for four n: sixteen products of a 4 x 1 block and a 1 x 4 block, the columns of
// block b the lanes 4 b .. 4 b + 3 with their x, and the four rows, broadcast from
// block q of every group of blocks, the values 4 q .. 4 q + 3.  The sum is in
// fp32, one rounding a value.  These instructions run beside other waves' vector
// instructions, of which each token has 16 fewer (of some 95 with 16 states): the
// chunks' outputs of 8,192 tokens x 2,048 channels 113 -> 104 us, of 16,384 x
// 4,096 340 -> 324, their states from zero 243 -> 217.  The sum over n of C_n h_n
// done likewise is slower (116 us of 8,192 x 2,048): four times the instructions,
// each waiting for the last.  The gradient's main kernel takes 249 us for 258.
template <class E, int N> struct ScanLanes {
  static constexpr int rows = (N + 15) / 16, period = N < 16 ? N : 16;
  E e[rows];
  __device__ __forceinline__ void load(const E *row, int lane) {
#pragma unroll
    for (int r = 0; r < rows; ++r) e[r] = lane_load(row + 16 * r, lane & (period - 1));
  }
};
template <int N> using ScanState = floatx4[N / 4];
template <int N, int Q = 0>
__device__ __forceinline__ void scan_add_outer(ScanState<N> &s, const float (&row)[(N + 15) / 16], float x) {
  constexpr int broadcast = N < 16 ? 1 : 2, block = Q & ((1 << broadcast) - 1);
  s[Q] = __builtin_amdgcn_mfma_f32_4x4x1f32(row[Q / 4], x, s[Q], broadcast, block, 0);
  if constexpr (Q + 1 < N / 4) scan_add_outer<N, Q + 1>(s, row, x);
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

// The kernel's arguments (its first) read again where they are used: pointers
// and strides of a dozen arrays do not stay in scalar registers that way.
__device__ __forceinline__ const ScanArgs &scan_args() {
  uintptr_t p = (uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm("" : "+s"(p));
  return *(const ScanArgs *)(const ScanArgs __attribute__((address_space(4))) *)p;
}
// The slots of the first and the last of the chunks from zero (one or two) that
// chunk k is made of.
__device__ __forceinline__ int64_t scan_first_part(const ScanArgs &A, const ScanChunk &k) {
  return k.start / A.part + k.i + (int64_t)k.c * (A.chunk / A.part);
}
__device__ __forceinline__ int64_t scan_last_part(const ScanArgs &A, const ScanChunk &k) {
  return k.start / A.part + k.i + (k.t1 - k.start + A.part - 1) / A.part - 1;
}

// A channel's states from or to [states / 4][channels][4], which a wave reads and
// writes in whole lines with four instructions for 16 states, or [channels][states]
template <int N>
__device__ __forceinline__ void scan_load_fours(const float *p, int64_t channels, int c, ScanState<N> &h) {
  typedef const char __attribute__((address_space(1))) *bytes;
  typedef const floatx4 __attribute__((address_space(1))) *global;
  const uint32_t off = (uint32_t)c * 16;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    h[q] = *(global)((bytes)row_address(p) + off);
    p += 4 * channels;
  }
}
template <int N>
__device__ __forceinline__ void scan_store_fours(float *p, int channels, uint32_t off, const ScanState<N> &h) {
  typedef unsigned int u4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const auto r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(row_address(p)), (short)0, channels * 16, 0x00020000);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, h[q]), r, (int)off, 0, 0);
    p += 4 * (int64_t)channels;
  }
}
template <int N>
__device__ __forceinline__ void scan_load_rows(const float *p, int64_t row, ScanState<N> &h) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) h[q] = *reinterpret_cast<const floatx4 *>(p + row * N + 4 * q);
}
template <int N>
__device__ __forceinline__ void scan_store_rows(float *p, int64_t row, const ScanState<N> &h) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) *reinterpret_cast<floatx4 *>(p + row * N + 4 * q) = h[q];
}
template <int N>
__device__ __forceinline__ void scan_zero(ScanState<N> &h) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) h[q] = floatx4{0.f, 0.f, 0.f, 0.f};
}
// What a thread of the launches between the chunks takes: a state of a channel of
// a sequence of several chunks
constexpr int kCarryAhead = 16;  // chunks whose states are loaded together
struct ScanCarry {
  bool any;
  int i, chunks;
  int state;           // channel * states + n
  int64_t at, at_sum;  // of the first chunk's states in ScanArgs::carry, of its steps in sum
};
__device__ __forceinline__ ScanCarry scan_carry(const ScanArgs &A, int states, int blocks) {
  ScanCarry r{};
  r.i = blockIdx.x / blocks;
  const int id = blockIdx.x % blocks * 256 + threadIdx.x;
  const int start = seq_offset(A.cu, A.tokens, r.i), end = max(start, seq_offset(A.cu, A.tokens, r.i + 1));
  r.chunks = (end - start + A.part - 1) / A.part;
  r.any = id < A.channels * states && r.chunks > 1;
  const int four = id / (4 * A.channels), c = id % (4 * A.channels) >> 2;
  const int64_t slot = start / A.part + r.i;
  r.state = c * states + 4 * four + (id & 3);
  r.at = slot * A.channels * states + id;
  r.at_sum = slot * A.channels + c;
  return r;
}

// decays as exponents of two: e^(d A) = 2^(d A log2 e)
template <int N>
__device__ __forceinline__ void scan_decays(const ScanArgs &A, int c, float (&a2)[N]) {
  ScanState<N> a;
  scan_load_rows<N>(A.A, c, a);
#pragma unroll
  for (int n = 0; n < N; ++n) a2[n] = a[n >> 2][n & 3] * kLog2e;
}

}  // namespace lq
