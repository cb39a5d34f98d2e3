// The selective state space scan over packed sequences, and for single tokens
// (gfx950).  For every channel c of group g, with N states,
//   d = softplus(dt + bias),  h_n <- e^(d A_n) h_n + d B_n x,
//   y = (sum_n C_n h_n + D x) silu(z)
//
// A lane holds a channel with all of its states, so that B and C are the same
// for a wave and come through the scalar cache, and y needs no sum across
// lanes.  A wave takes 64 channels and one chunk of tokens; sequences of several
// chunks take three launches: every chunk's states from zero and the sum of its
// steps (the whole chunk decays by e^(A sum)), the states before every chunk
// from these, and the tokens again from there.
//
// Bound by vector instructions in the first and the third launch (of one prompt, with
// three waves a SIMD, they take 77 and 71 % of the issue slots while the chip is busy):
// with 16 states a token and channel take 16 exponentials, of two slots
// each, in both, and 32 to 48 products and sums.  One prompt of 4,096
// tokens x 4,096 channels in bf16: 54 + 7 + 75 us.  16,384 tokens x 4,096 of 24
// sequences in fp16: 179 + 25 + 260.  8,192 x 2,048 of four, states kept for the
// gradient: 55 + 13 + 93.  (These with a warm chip; pairs of figures further down were
// measured one against the other, most of them without.)  One launch that hands the states from chunk to chunk
// would halve the exponentials of a chunk only where the chunks ran one after the
// other, and so few waves do not fill the chip.  Keeping the steps of the first
// launch for the third would save it 7 us of the 89 it then took of the prompt,
// and cost reading and writing them.
#include "lq_scan_device.h"

namespace lq {

// kScanOut: the chunks' outputs from the states before them (kScanGated: gated by z,
// kScanSave: with the states kept for the gradient); kScanLocal: the chunks' states
// from zero.  Where there are outputs, four tokens' inputs are loaded together, which
// leaves room for a wave a SIMD more than eight do (324 us for 336 of 16,384 tokens x
// 4,096 channels, 82 for 83 of 4,096 x 4,096); where there are none, eight (206 us
// for 214).
enum { kScanLocal = 0, kScanOut = 1, kScanGated = 2, kScanSave = 4 };
template <class E, int N, int MODE>
__global__ __launch_bounds__(256, scan_forward_waves(N)) void scan_kernel(const ScanArgs A, int tiles, int64_t waves) {
  constexpr bool OUT = MODE & kScanOut, GATE = MODE & kScanGated, SAVE = MODE & kScanSave;
  constexpr int ahead = OUT ? 4 : 8;  // tokens whose inputs are loaded together
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + (int64_t)blockIdx.x * 4;
  if (wave >= waves) return;  // whole waves; the waves share nothing
  const int slot = (int)(wave / tiles), tile = (int)(wave % tiles), tg = (A.per + 63) >> 6;
  const ScanChunk k = scan_chunk(A, OUT ? A.chunk : A.part, slot, lane);
  if (!k.any || (!OUT && k.c + 1 >= k.chunks)) return;  // nothing comes behind the last chunk
  const ScanTile ch = scan_tile(A, tile / tg, tile % tg, lane);
  const int64_t width = A.channels;
  float a2[N], sum = 0.f;
  ScanState<N> h;
  scan_decays<N>(A, ch.c, a2);
  scan_zero<N>(h);
  if (OUT) {
    if (k.chunks > 1)
      scan_load_fours<N>(A.carry + scan_first_part(A, k) * N * width, width, ch.c, h);
    else if (A.S0)
      scan_load_rows<N>(A.S0, k.i * width + ch.c, h);
  }
  const float bias = A.bias ? A.bias[ch.c] : 0.f, skip = OUT && A.skip ? A.skip[ch.c] : 0.f;
  float *check = SAVE ? A.check + (k.start / kScanSub + k.i + (k.t0 - k.start) / kScanSub) * N * width : nullptr;
  const int row_bytes = (int)(width * sizeof(E));
  const uint32_t off_y = lane_offset(ch.on, ch.c, sizeof(E)), off_s = lane_offset(ch.on, ch.c, 16);
  E rx[ahead], rd[ahead], rz[ahead];
  ScanLanes<E, N> rb[ahead];
  const auto load = [&](int t) {
    const ScanArgs &P = scan_args();
    const E *x = at<const E>(P.x, t, 0), *dt = at<const E>(P.dt, t, 0), *z = GATE ? at<const E>(P.z, t, 0) : x;
    const E *b = at<const E>(P.B, t, ch.g);
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      rx[u] = lane_load(x, ch.c);
      rd[u] = lane_load(dt, ch.c);
      rb[u].load(b, lane);
      if (GATE) rz[u] = lane_load(z, ch.c);
      if (t + u + 1 < k.t1) {
        x += P.x.ts;
        dt += P.dt.ts;
        b += P.B.ts;
        if (GATE) z += P.z.ts;
      }
    }
  };
  // the output's row: reading the arguments for each token would wait for the row
  // of C on its way
  E *y = OUT ? at<E>(A.y, k.t0, 0) : nullptr;
  const E *row = OUT ? at<const E>(A.C, k.t0, ch.g) : nullptr;
  ScanRow<E, N> C;
  if (k.t0 < k.t1) {
    load(k.t0);
    if (OUT) C.load(row);
  }
  for (int t = k.t0; t < k.t1; t += ahead) {
    float fx[ahead], fd[ahead], fz[ahead], fb[ahead][ScanLanes<E, N>::rows];
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
#pragma unroll
      for (int r = 0; r < ScanLanes<E, N>::rows; ++r) fb[u][r] = to_f(rb[u].e[r]);
      fx[u] = to_f(rx[u]);
      fd[u] = to_f(rd[u]) + bias;
      fz[u] = GATE ? to_f(rz[u]) : 0.f;
    }
    // converted before the next loads begin, which take the same registers: converted
    // where they are used they would be copied (84 for 82 us of the prompt above)
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      asm volatile("" : "+v"(fx[u]), "+v"(fd[u]));
      if (GATE) asm volatile("" : "+v"(fz[u]));
#pragma unroll
      for (int r = 0; r < ScanLanes<E, N>::rows; ++r) asm volatile("" : "+v"(fb[u][r]));
    }
    if (t + ahead < k.t1) load(t + ahead);
    scan_steps<E>(A, fd);
#pragma unroll
    for (int u = 0; u < ahead; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      const int tt = t + u;
      if (tt >= k.t1) break;
      const ScanRow<E, N> cc = C;
      if (OUT) {
        row += tt + 1 < k.t1 ? A.C.ts : 0;
        C.load(row);
      }
      if (SAVE && u % kScanSub == 0) {
        scan_store_fours<N>(check, (int)width, off_s, h);
        check += N * width;
      }
      const float d = fd[u], x = fx[u];
      sum += d;
#pragma unroll
      for (int n = 0; n < N; ++n) h[n >> 2][n & 3] *= __builtin_amdgcn_exp2f(d * a2[n]);
      scan_add_outer<N>(h, fb[u], d * x);
      if (OUT) {
        float p0 = skip * x, p1 = 0.f;
#pragma unroll
        for (int n = 0; n < N; n += 2) {
          p0 = fmaf(cc[n], h[n >> 2][n & 3], p0);
          p1 = fmaf(cc[n + 1], h[n >> 2][(n & 3) + 1], p1);
        }
        float p = p0 + p1;
        if (GATE) p *= fz[u] * sigmoid_for<E>(fz[u]);
        lane_store(y, row_bytes, off_y, from_f<E>(p));
        y += A.y.ts;
      }
    }
  }
  if (!ch.on) return;
  if (!OUT) {
    scan_store_fours<N>(A.carry + (int64_t)slot * N * width, (int)width, off_s, h);
    A.sum[slot * width + ch.c] = sum;
  } else if (A.S && k.c + 1 >= k.chunks) {
    scan_store_rows<N>(A.S, k.i * width + ch.c, h);
  }
}

// The states before every chunk of the sequences with several, over the chunks'
// states from zero: blocks of a sequence, thread (four states, channel, one of
// them).  S0 is copied before the first chunk, as S may lie over it.
__global__ __launch_bounds__(256) void scan_carry_kernel(const ScanArgs A, int states, int blocks) {
  const ScanCarry t = scan_carry(A, states, blocks);
  if (!t.any) return;
  const int chunks = t.chunks;
  const int64_t width = A.channels, step = states * width;
  const float a2 = A.A[t.state] * kLog2e;
  float h = A.S0 ? A.S0[t.i * step + t.state] : 0.f;
  float *carry = A.carry + t.at;
  const float *sum = A.sum + t.at_sum;
  for (int k = 0; k < chunks; k += kCarryAhead) {
    float v[kCarryAhead], s[kCarryAhead];
#pragma unroll
    for (int u = 0; u < kCarryAhead; ++u) {
      const int64_t at = min(k + u, chunks - 2);  // (the last one has none: nothing comes behind it)
      v[u] = carry[at * step];
      s[u] = sum[at * width];
    }
#pragma unroll
    for (int u = 0; u < kCarryAhead; ++u) {
      if (k + u >= chunks) break;
      carry[(k + u) * step] = h;
      h = fmaf(__builtin_amdgcn_exp2f(s[u] * a2), h, v[u]);
    }
  }
}

// One token of each row.  Four states a lane, the lanes of a channel side by
// side, so that the states move in whole lines.  Bound by reading and writing
// them, past the caches, as a step's states are not read again before the next: 256
// rows x 4,096 channels x 16 states 32 to 34 us, 4.2 to 4.5 TB/s.
template <class E, int N>
__global__ __launch_bounds__(256) void scan_step_kernel(const ScanArgs A, int64_t blocks_row) {
  constexpr int lanes = N / 4;
  const int64_t row = blockIdx.x / blocks_row;
  const int64_t id = (blockIdx.x % blocks_row) * 256 + threadIdx.x;
  const int64_t slot = A.which ? A.which[row] : row;
  if (slot < 0 || slot >= A.n_slots) return;  // the whole block
  const bool on = id < (int64_t)A.channels * lanes;
  const int64_t c = on ? id / lanes : A.channels - 1;
  const int n = (int)(id % lanes) * 4, g = (int)(c / A.per);
  const int64_t at_s = (slot * A.channels + c) * N + n;
  const vf4 h0 = __builtin_nontemporal_load(reinterpret_cast<const vf4 *>(A.S0 + at_s));
  const float4 a = *reinterpret_cast<const float4 *>(A.A + c * N + n);
  const float x = to_f(at<const E>(A.x, row, 0)[c]);
  const float v = to_f(at<const E>(A.dt, row, 0)[c]) + (A.bias ? A.bias[c] : 0.f);
  float b[4], cc[4];
  load4(at<const E>(A.B, row, g) + n, b);
  load4(at<const E>(A.C, row, g) + n, cc);
  float steps[1] = {v};
  scan_steps<E>(A, steps);
  const float d = steps[0], dx = d * x, d2 = d * kLog2e;
  vf4 h;
  h.x = fmaf(__builtin_amdgcn_exp2f(d2 * a.x), h0.x, dx * b[0]);
  h.y = fmaf(__builtin_amdgcn_exp2f(d2 * a.y), h0.y, dx * b[1]);
  h.z = fmaf(__builtin_amdgcn_exp2f(d2 * a.z), h0.z, dx * b[2]);
  h.w = fmaf(__builtin_amdgcn_exp2f(d2 * a.w), h0.w, dx * b[3]);
  float p = fmaf(cc[0], h.x, cc[1] * h.y) + fmaf(cc[2], h.z, cc[3] * h.w);
  if (lanes >= 2) p += dpp<0xB1>(p);
  if (lanes >= 4) p += dpp<0x4E>(p);
  if (lanes >= 8) p += dpp<0x141>(p);
  if (!on) return;
  __builtin_nontemporal_store(h, reinterpret_cast<vf4 *>(A.S + at_s));
  if (n == 0) {
    p = fmaf(A.skip ? A.skip[c] : 0.f, x, p);
    if (A.z.ptr) {
      const float z = to_f(at<const E>(A.z, row, 0)[c]);
      p *= z * sigmoid(z);
    }
    at<E>(A.y, row, 0)[c] = from_f<E>(p);
  }
}

template <class E, int N>
static hipError_t scan_run(const ScanArgs &a, bool step, hipStream_t stream) {
  if (step) {
    const int64_t blocks_row = ((int64_t)a.channels * (N / 4) + 255) / 256;
    if (a.tokens)
      hipLaunchKernelGGL((scan_step_kernel<E, N>), dim3((unsigned)(a.tokens * blocks_row)), dim3(256), 0, stream, a,
                         blocks_row);
    return hipGetLastError();
  }
  const int64_t tiles = scan_tiles(a.channels, a.groups), waves = tiles * a.slots;
  if (a.tokens > a.chunk) {  // a sequence may have several chunks
    const int64_t parts = tiles * scan_slots(a.tokens, a.seqs, a.part);
    hipLaunchKernelGGL((scan_kernel<E, N, kScanLocal>), dim3((unsigned)((parts + 3) / 4)), dim3(256), 0, stream, a,
                       (int)tiles, parts);
    const int blocks = (a.channels * N + 255) / 256;
    hipLaunchKernelGGL(scan_carry_kernel, dim3((unsigned)(a.seqs * (int64_t)blocks)), dim3(256), 0, stream, a, N, blocks);
  }
  const dim3 grid((unsigned)((waves + 3) / 4));
  if (a.z.ptr && a.check)
    hipLaunchKernelGGL((scan_kernel<E, N, kScanOut | kScanGated | kScanSave>), grid, dim3(256), 0, stream, a, (int)tiles, waves);
  else if (a.z.ptr)
    hipLaunchKernelGGL((scan_kernel<E, N, kScanOut | kScanGated>), grid, dim3(256), 0, stream, a, (int)tiles, waves);
  else if (a.check)
    hipLaunchKernelGGL((scan_kernel<E, N, kScanOut | kScanSave>), grid, dim3(256), 0, stream, a, (int)tiles, waves);
  else
    hipLaunchKernelGGL((scan_kernel<E, N, kScanOut>), grid, dim3(256), 0, stream, a, (int)tiles, waves);
  return hipGetLastError();
}
template <class E>
static hipError_t scan_run(const ScanArgs &a, int states, bool step, hipStream_t stream) {
  return states == 8    ? scan_run<E, 8>(a, step, stream)
         : states == 16 ? scan_run<E, 16>(a, step, stream)
                        : scan_run<E, 32>(a, step, stream);
}
static hipError_t scan_run(const ScanArgs &a, int dtype, int states, bool step, hipStream_t stream) {
  return dtype == 0 ? scan_run<F32>(a, states, step, stream)
         : dtype == 1 ? scan_run<BF16>(a, states, step, stream)
                      : scan_run<F16>(a, states, step, stream);
}
hipError_t launch_scan(const ScanArgs &a, int dtype, int states, hipStream_t stream) {
  return scan_run(a, dtype, states, false, stream);
}
hipError_t launch_scan_step(const ScanArgs &a, int dtype, int states, hipStream_t stream) {
  return scan_run(a, dtype, states, true, stream);
}

}  // namespace lq
