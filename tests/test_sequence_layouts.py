"""Which layouts of outputs the sequence entry points take (CPU): the library's
argument checks, built for the host with launches that do nothing, against
every byte of the arrays marked one by one."""
import os

import pytest

from tests.test_sanitizers import ROCM, ROOT, SAN, _run

DRIVER = r"""
#include <stdio.h>
#include <string.h>
#include <random>
#include <set>
#include "lq_sequence.h"
#include "leapquant.h"
namespace lq {
hipError_t launch_seq_recurrent(const SeqArgs &, int, bool, bool, hipStream_t) { return hipSuccess; }
hipError_t launch_seq_chunked(const SeqArgs &, int, bool, bool, hipStream_t) { return hipSuccess; }
hipError_t launch_seq_backward(const SeqArgs &, int, bool, hipStream_t) { return hipSuccess; }
int64_t norm_blocks(int64_t, int, int) { return 1; }
hipError_t launch_norm(const NormArgs &, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_backward(const NormArgs &, int, int, hipStream_t) { return hipSuccess; }
}  // namespace lq

static char *const kBase = (char *)0x7f0000000000;  // never dereferenced

// marks the 4-byte words of an array: is one of them its own already, or an array's before it?
struct Map {
  std::set<int64_t> all;
  bool self, other;
  void add(const lq_rows &r, int tokens, int heads, int width, int size) {
    self = other = false;
    std::set<int64_t> mine;
    for (int t = 0; t < tokens; ++t)
      for (int h = 0; h < heads; ++h) {
        const int64_t at = (char *)r.ptr - kBase + (t * r.token_stride + h * r.head_stride) * size;
        for (int64_t w = at; w < at + width * size; w += 4) {
          self |= !mine.insert(w).second;
          other |= all.count(w) > 0;
        }
      }
    all.insert(mine.begin(), mine.end());
  }
};

static int backward(int T, int hk, int hv, int dtype, const lq_rows (&out)[5], const lq_rows *go = nullptr) {
  lq_sequence sq = {T, 1, hk, hv, 128, 128, LQ_GATE_GDN, 0, dtype};
  lq_rows in = {(void *)0x600000000000, 0, 0}, sc = {(void *)0x610000000000, 0, 0};
  return leapquant_sequence_backward(&sq, (const int32_t *)0x620000000000, &in, &in, &sc, &sc, go ? go : &in, nullptr, &out[0],
                                     &out[1], &out[2], &out[3], &out[4], nullptr, (void *)0x630000000000,
                                     int64_t(1) << 40, nullptr);
}

#define EXPECT(call, want)                                                                \
  do {                                                                                    \
    const int rc_ = (call);                                                               \
    if (rc_ != (want)) {                                                                  \
      printf("%s: %d, expected %d\n", #call, rc_, (want));                                \
      ++wrong;                                                                            \
    }                                                                                     \
  } while (0)

// outputs as views of one buffer that a training program would hold
static int named() {
  int wrong = 0;
  const int T = 90, H = 4;
  lq_rows b = {kBase + (1 << 28), 2 * H, 2}, a = {kBase + (1 << 28) + 4, 2 * H, 2};  // [tokens][heads][2]
  // [tokens][heads][3][128], and [heads][tokens][3][128]
  for (int major = 0; major < 2; ++major) {
    const int64_t ts = major ? 384 : 384 * H, hs = major ? 384 * T : 384;
    const lq_rows o[5] = {{kBase, ts, hs}, {kBase + 256, ts, hs}, {kBase + 512, ts, hs}, b, a};
    EXPECT(backward(T, H, H, LQ_BF16, o), LQ_OK);
    const lq_rows wide[5] = {o[0], {kBase + 256 - 16, ts, hs}, o[2], b, a};
    EXPECT(backward(T, H, H, LQ_BF16, wide), LQ_ERR_ALIAS);
    const lq_rows twice[5] = {o[0], o[1], o[1], b, a};
    EXPECT(backward(T, H, H, LQ_BF16, twice), LQ_ERR_ALIAS);
  }
  // a row of 2 key heads, each q then k, and 4 value heads behind; the gates' gradients in its tail
  const int64_t row = 4 * 128 + 4 * 128 + 16;
  const lq_rows g[5] = {{kBase, row, 256}, {kBase + 512, row, 256}, {kBase + 4 * 512, row, 128},
                        {kBase + 8 * 512, row, 2}, {kBase + 8 * 512 + 4, row, 2}};
  EXPECT(backward(T, 2, 4, LQ_F32, g), LQ_OK);
  // two value heads beside each key head's q and k: [tokens][key heads][4][128]; the value heads' strides are not even
  const lq_rows v[5] = {{kBase, 1024, 512}, {kBase + 256, 1024, 512}, {kBase + 512, 1024, 128}, b, a};
  EXPECT(backward(T, 2, 4, LQ_BF16, v), LQ_ERR_ALIAS);
  // one token: its heads interleaved
  const lq_rows one[5] = {{kBase, 0, 384}, {kBase + 256, 0, 384}, {kBase + 512, 0, 384}, b, a};
  EXPECT(backward(1, H, H, LQ_BF16, one), LQ_OK);
  // one gradient of o for all tokens and heads, in a head of the first token's row that no output has
  const int64_t ts = 512 * H;
  const lq_rows q[5] = {{kBase, ts, 512}, {kBase + 256, ts, 512}, {kBase + 512, ts, 512}, b, a};
  const lq_rows none = {kBase + 768, 0, 0}, taken = {kBase + 512, 0, 0}, part = {kBase + 768 + 16, 0, 0};
  EXPECT(backward(T, H, H, LQ_BF16, q, &none), LQ_OK);
  EXPECT(backward(T, H, H, LQ_BF16, q, &taken), LQ_ERR_ALIAS);
  EXPECT(backward(T, H, H, LQ_BF16, q, &part), LQ_ERR_ALIAS);
  return wrong;
}

// random layouts: every answer against the marked words
static int drawn(int n) {
  std::mt19937 g(7);
  const auto any = [&](int lo, int hi) { return (int)(lo + g() % (unsigned)(hi - lo + 1)); };
  int wrong = 0, count[3] = {0, 0, 0};
  for (int i = 0; i < n; ++i) {
    const int T = any(1, 5), hk = any(1, 3), hv = hk * any(1, 2);
    const int dtype = any(0, 1), size = dtype == LQ_F32 ? 4 : 2, unit = 16 / size;
    const bool same = any(0, 3) > 0;  // one token stride for all
    // units of 16 bytes; heads are 128 values wide
    const int wide = 128 / unit, span = any(1, 3) * wide * any(1, 8);
    int64_t ts0 = any(0, 1) ? span + any(0, 3) : any(wide, 4 * wide);
    lq_rows o[5];
    Map m;
    bool self = false, other = false;
    int64_t lo[5], hi[5], ts[5];
    for (int x = 0; x < 5; ++x) {
      const int heads = x < 2 ? hk : hv, width = x < 3 ? 128 : 1, sz = x < 3 ? size : 4;
      const int64_t step = (same ? ts0 : any(0, 1) ? ts0 : any(wide, 6 * wide)) * 16;  // bytes
      const int64_t hs = (any(0, 3) ? any(wide, 3 * wide) : any(0, 2) ? wide * any(1, 9) : any(0, wide)) * 16;
      o[x] = lq_rows{kBase + 16 * any(0, 12 * wide) + (x < 3 ? 0 : 4 * any(0, 3)), step / sz, hs / sz};
      m.add(o[x], T, heads, width, sz);
      self |= m.self;
      other |= m.other;
      lo[x] = (char *)o[x].ptr - kBase;
      hi[x] = lo[x] + (T - 1) * step + (heads - 1) * hs + width * sz;
      ts[x] = T > 1 ? step : 0;
    }
    bool unlike = false;  // ranges that interleave with other token strides
    for (int x = 0; x < 5; ++x)
      for (int y = 0; y < x; ++y) unlike |= ts[x] != ts[y] && lo[x] < hi[y] && lo[y] < hi[x];
    const int want = self ? LQ_ERR_SHAPE : other || unlike ? LQ_ERR_ALIAS : LQ_OK;
    const int rc = backward(T, hk, hv, dtype, o);
    ++count[want == LQ_OK ? 0 : want == LQ_ERR_SHAPE ? 1 : 2];
    if (rc != want && ++wrong < 10) {
      printf("case %d: %d, expected %d; T %d hk %d hv %d size %d\n", i, rc, want, T, hk, hv, size);
      for (int x = 0; x < 5; ++x)
        printf("  %ld + t %ld + h %ld\n", (long)lo[x], (long)o[x].token_stride, (long)o[x].head_stride);
    }
  }
  printf("taken %d, coinciding elements %d, shared %d, wrong %d\n", count[0], count[1], count[2], wrong);
  return wrong || !count[0] || !count[1] || !count[2];
}

int main(int, char **argv) { return strcmp(argv[1], "named") ? drawn(5000) : named(); }
"""


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    d = tmp_path_factory.mktemp("layouts")
    (d / "driver.cpp").write_text(DRIVER)
    csrc = os.path.join(ROOT, "recurrent_state_quant_amd", "csrc")
    _run(["g++", "-std=c++17", "-O1", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", csrc,
          "-I", os.path.join(ROCM, "include"), "-o", str(d / "driver"), str(d / "driver.cpp"),
          os.path.join(csrc, "lq_sequence_abi.cpp")])
    return str(d / "driver")


@pytest.mark.parametrize("what", ["named", "drawn"])
def test_layouts_of_outputs(driver, what):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    print(_run([driver, what], env=env, timeout=120).stdout)
