// Checks of the entry points over token arrays (lq_sequence_abi.cpp,
// lq_layer_abi.cpp): strided arrays, alignment, and whether two arrays share
// memory.
#pragma once
#include <stdint.h>

#include "leapquant.h"
#include "lq_sequence.h"

namespace lq {
namespace abi {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxGrid = (int64_t(1) << 23) - 1;  // workgroups of a launch: 512 lanes each stay below 2^32
constexpr int64_t kMaxPairs = 65536;                  // heads of two arrays that are compared one by one

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? LQ_OK : LQ_ERR_HIP; }

inline int64_t dtype_size(int32_t dtype) { return dtype == LQ_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype == LQ_F32 || dtype == LQ_BF16 || dtype == LQ_F16; }

// The memory of one argument: pieces of `width` bytes, `tokens` of them `ts`
// bytes apart for each of `heads`, which are `hs` bytes apart.
struct Block {
  uintptr_t lo, hi;
  int64_t tokens, heads, ts, hs, width;
};

inline Block dense(const void *p, int64_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return Block{b, p ? b + static_cast<uintptr_t>(bytes) : b, 1, 1, 0, 0, bytes};
}

// Do a piece of wa bytes and one of wb bytes meet that begins `off` bytes
// behind it, or there shifted by a whole number d of steps, least <= d <= most
// (least <= 0 <= most)?
inline bool meet(int64_t off, int64_t step, int64_t least, int64_t most, int64_t wa, int64_t wb) {
  if (step == 0) return off < wa && off > -wb;
  // the first d with off + d step > -wb
  const int64_t x = -wb - off;
  int64_t d = x / step - (x % step < 0 ? 1 : 0) + 1;
  if (d < least) d = least;
  return d <= most && off + d * step < wa;
}

// Exact for arrays with one token stride (or of one token, or one for all), as
// views of one buffer have; others whose ranges interleave count as overlapping.
inline bool overlap(const Block &a, const Block &b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.tokens > 1 && b.tokens > 1 && a.ts != b.ts) return true;
  const int64_t ts = a.tokens > 1 ? a.ts : b.ts;
  const int64_t off = static_cast<int64_t>(b.lo - a.lo);  // (the ranges meet: far below 2^63)
  const int64_t least = 1 - a.tokens, most = b.tokens - 1;
  // slices of one row: a row's heads as one piece
  if (!meet(off, ts, least, most, (a.heads - 1) * a.hs + a.width, (b.heads - 1) * b.hs + b.width)) return false;
  if (a.heads == 1 || b.heads == 1 || a.hs == b.hs) {
    const int64_t hs = a.heads > 1 ? a.hs : b.hs;
    for (int64_t d = 1 - a.heads; d < b.heads; ++d)
      if (meet(off + d * hs, ts, least, most, a.width, b.width)) return true;
    return false;
  }
  if (a.heads * b.heads > kMaxPairs) return true;
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j)
      if (meet(off + j * b.hs - i * a.hs, ts, least, most, a.width, b.width)) return true;
  return false;
}

// Are two elements of an array with these strides the same memory?
inline bool coincide(int64_t tokens, int64_t heads, int64_t ts, int64_t hs, int64_t width) {
  const int64_t row = (heads - 1) * hs + width, column = (tokens - 1) * ts + width;
  if ((tokens == 1 || ts >= row) && (heads == 1 || hs >= width)) return false;     // token by token
  if ((heads == 1 || hs >= column) && (tokens == 1 || ts >= width)) return false;  // head by head
  if (tokens > 1 && ts < width) return true;
  for (int64_t d = 1; d < heads; ++d)
    if (meet(d * hs, ts, 1 - tokens, tokens - 1, width, width)) return true;
  return false;
}

// Checks one strided array of heads (width 128) or scalars (width 1) of
// `size`-byte elements and gives its memory and the kernels' view of it.
// Without elements nothing is looked at.  align: of the pointer and the strides
// in bytes (0: 16 for heads, 4 for scalars, whose strides are whole elements).
inline int check_rows(const lq_rows *r, int64_t tokens, int64_t heads, int64_t width, int64_t size, bool out, Block *blk,
                      lq::Rows *to, int64_t align = 0) {
  if (!r) return LQ_ERR_NULL;
  *blk = Block{};
  *to = lq::Rows{nullptr, 0, 0};
  if (tokens == 0 || heads == 0) return LQ_OK;
  if (!r->ptr) return LQ_ERR_NULL;
  if (align == 0) align = width == 1 ? 4 : 16;
  if (!aligned(r->ptr, align)) return LQ_ERR_ALIGN;
  // the stride of an axis of one element is never used
  const int64_t ts = tokens > 1 ? r->token_stride : 0, hs = heads > 1 ? r->head_stride : 0;
  const int64_t most = int64_t(1) << 46;
  if (ts < 0 || hs < 0 || ts > most || hs > most) return LQ_ERR_SHAPE;
  if (width > 1 && ((ts * size) % align || (hs * size) % align)) return LQ_ERR_ALIGN;
  int64_t last;
  if (__builtin_mul_overflow(tokens - 1, ts, &last)) return LQ_ERR_SHAPE;
  const int64_t across = (heads - 1) * hs;  // heads < 2^16, hs <= 2^46
  if (last > (int64_t(1) << 58) || across > (int64_t(1) << 58)) return LQ_ERR_SHAPE;
  if (out && coincide(tokens, heads, ts, hs, width)) return LQ_ERR_SHAPE;
  *blk = dense(r->ptr, (last + across + width) * size);
  blk->tokens = ts ? tokens : 1;  // (stride 0: one and the same)
  blk->heads = hs ? heads : 1;
  blk->ts = ts * size;
  blk->hs = hs * size;
  blk->width = width * size;
  *to = lq::Rows{r->ptr, ts, hs};
  return LQ_OK;
}

// No output may overlap an input or another output.
struct Blocks {
  Block in[16], out[16];
  int n_in = 0, n_out = 0;
  void add_in(const Block &b) { in[n_in++] = b; }
  void add_out(const Block &b) { out[n_out++] = b; }
  bool clash() const {
    for (int i = 0; i < n_out; ++i) {
      for (int j = 0; j < n_in; ++j)
        if (overlap(out[i], in[j])) return true;
      for (int j = i + 1; j < n_out; ++j)
        if (overlap(out[i], out[j])) return true;
    }
    return false;
  }
};

}  // namespace abi
}  // namespace lq
