// Internal launch interface between the entry points of the operators around
// the recurrence (lq_layer_abi.cpp) and their gfx950 kernels (lq_conv.hip,
// lq_scan.hip, lq_scan_grad.hip, lq_block_norm.hip).  Arguments are validated
// by the caller.
#pragma once
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "lq_sequence.h"

namespace lq {

// [tokens][channels] arrays are Rows whose head stride is not used.

struct ConvArgs {
  int64_t tokens;  // rows of the step
  int seqs, channels, width, silu;
  const int32_t *cu;
  Rows x, y;
  const float *w;     // [channels][width]
  const float *bias;  // [channels] or nullptr
  const void *X0;     // [seqs or slots][width - 1][channels] or nullptr (zeros)
  void *X;
  const int32_t *slots;  // step: [rows] or nullptr (row i has slot i)
  int n_slots;
  // backward
  Rows dy, dx;
  const void *dX;
  void *dX0;
  float *dw, *dbias;
  float *part;  // [blocks of runs][width + 1][channels]
};

// Tokens of a wave's run.  Longer runs share more of the tokens around them, once
// there are waves enough of them, `least` a SIMD.  Forward four: runs of 64 take 118
// us of 16,384 tokens x 16 tiles of channels, of 32 123 (four waves a SIMD with 64);
// but 97 for 85 us of 8,192 x 24 tiles (three), 49 for 43 of 8,192 x 12.  Backward
// three (256 channels a tile): 74 for 83 us of 8,192 x 24 tiles.
constexpr int kConvRunLeast = 32, kConvRunMost = 4096;
constexpr int64_t kConvBlocks = 256, kSimds = 4 * 256;
inline int conv_run_tokens(int64_t tokens, int64_t tiles, int least) {
  return tokens / (2 * kConvRunLeast) * tiles >= least * kSimds ? 2 * kConvRunLeast : kConvRunLeast;
}
// Of the backward pass: a block takes four runs of the same channels and joins their
// weight gradients, and runs grow once there are 256 blocks of them, so that the
// joined sums stay few.
inline int64_t conv_grad_blocks(int64_t tokens, int64_t run) { return (tokens + 4 * run - 1) / (4 * run); }
inline int conv_grad_run(int64_t tokens, int64_t channels) {
  int run = conv_run_tokens(tokens, (channels + 255) / 256, 3);
  while (run < kConvRunMost && conv_grad_blocks(tokens, run) > kConvBlocks) run *= 2;
  return run;
}
// The most blocks of any call with at most these tokens
inline int64_t conv_grad_most(int64_t tokens) {
  const int64_t few = conv_grad_blocks(tokens, kConvRunLeast), many = conv_grad_blocks(tokens, kConvRunMost);
  return few < kConvBlocks ? few : many > kConvBlocks ? many : kConvBlocks;
}

struct ScanArgs {
  int64_t tokens, slots;
  int seqs, channels, groups, per;  // per: channels of a group
  int chunk;                        // tokens of a chunk, a multiple of 8
  int part;                         // tokens of a chunk from zero: chunk, or half of it
  int softplus;
  const int32_t *cu;
  Rows x, dt, z, y, B, C;  // z.ptr may be nullptr
  const float *A, *skip, *bias;
  const float *S0;  // [seqs][channels][states] or nullptr (zeros)
  float *S;         // or nullptr
  float *check;     // [scan_checks][states / 4][channels][4] or nullptr: the states before every kScanSub-th token of a sequence
  float *carry;     // [part slots][states / 4][channels][4]  of sequences with several: the state before (backward: gradient behind)
  float *sum;       // [part slots][channels]          the sum of a part's steps
  // step
  const int32_t *which;  // [rows] or nullptr
  int n_slots;
  // backward
  Rows dy, dx, ddt, dB, dC, dz;
  float *dA, *dskip, *dbias;
  const float *dS;
  float *dS0;
  float *part_bc;  // [tiles][tokens][2 * states], in the order of the gradient's kernel
  float *part_a;   // [chunk slots][states + 2][channels]
};

// Tokens whose states the gradient holds in registers at once, and so how often
// the forward pass keeps a state.  Twice as many would halve the kept states'
// memory, but leave room for one wave a SIMD with 16 states.
constexpr int kScanSub = 4;
inline int64_t scan_checks(int64_t tokens, int64_t seqs) { return tokens / kScanSub + seqs; }

// Waves take 64 channels of one group and one chunk of tokens.
inline int64_t scan_tiles(int channels, int groups) {
  return int64_t(groups) * ((channels / groups + 63) / 64);
}
// Slots of chunks: sequence i, chunk c has slot cu[i] / chunk + i + c.
inline int64_t scan_slots(int64_t tokens, int64_t seqs, int chunk) { return tokens / chunk + seqs; }
// Tokens of a chunk.  A workgroup has a wave on each SIMD of a CU, and with w
// waves a token takes w + stall times a wave's own vector instructions (stall:
// what w waves leave unhidden; 1.4 measured forward, 0.7 in the gradient, whose
// instructions are three times as many).  `most` workgroups fit a CU; more run in
// rounds.  So the time is (chunk + what a wave's beginning takes, in tokens) times
// the rounds' w + stall, and the best length one that fills the CUs evenly.  All three
// forward launches of 4,096 tokens x 64 waves take 136 us in the chunks of 88 that are
// taken (2.9 waves a SIMD), 133 of 64 (4.0), 141 of 56 (4.6) and of 72 (3.6), 155 of 80
// (3.3), 178 of 120 (2.2); of 16,384 x 64 waves in 24 sequences 463 in chunks of 112,
// 453 of 72, 479 of 56, 471 of 104, 508 of 160.  The gradient's main launch of 8,192
// tokens x 32 waves in four sequences takes 220 us in chunks of 136, 225 of 40, 232 of
// 144, 266 of 96, 308 of 128.
// A call whose sequences may have several chunks takes two launches more, 25 tokens'
// time, and every chunk of a sequence lengthens the chain between them by 0.3
// of a token's; one that needs no chunks from zero takes 0.6 of the rest.  (200 tokens x
// 1,024 channels in chunks of 8 17.6 us, of 16 20.4, of 32 31.6.)  Chunks below 32
// tokens are for calls that do not fill the chip: at most `scan_few` of them, which
// bounds the workspace.
constexpr int kScanLeast = 8, kScanShort = 32, kScanMost = 512, kScanBegin = 12, kScanCus = 256;
inline int64_t scan_few(int64_t workgroups, int most) { return kScanCus * most / workgroups; }
inline int scan_chunk_tokens(int64_t tokens, int64_t seqs, int64_t workgroups, int most, double stall) {
  int best = kScanShort;
  double least = 0;
  const auto look = [&](int chunk) {
    if (chunk < kScanShort && scan_slots(tokens, seqs, chunk) > scan_few(workgroups, most)) return int64_t(2);
    // (half a chunk more for each sequence, as its last one is partly full)
    const int64_t each = ((tokens / chunk + (seqs + 1) / 2) * workgroups + kScanCus - 1) / kScanCus;
    const int64_t rounds = each / most, rest = each % most;
    double time = (chunk + kScanBegin) * (rounds * (most + stall) + (rest ? rest + stall : 0));
    time = tokens > chunk ? time + 25 + 0.3 * tokens / seqs / chunk : 0.6 * time;
    if (least == 0 || time < least) least = time, best = chunk;
    return each;
  };
  for (int chunk = kScanLeast; chunk <= kScanMost; chunk += 8)
    if (look(chunk) <= 1) break;
  if (tokens <= kScanMost) look(tokens <= kScanLeast ? kScanLeast : (int)(tokens + 7) / 8 * 8);
  return best;
}
// Waves of the forward kernel that a SIMD holds: of the chunks from zero, which take
// more registers than the outputs, of which one to three waves more fit
constexpr int scan_forward_waves(int states) { return states > 16 ? 3 : states > 8 ? 5 : 6; }
inline int scan_forward_chunk(int64_t tokens, int64_t seqs, int channels, int groups, int states) {
  return scan_chunk_tokens(tokens, seqs, (scan_tiles(channels, groups) + 3) / 4, scan_forward_waves(states), 1.4);
}
// Of the gradient; its chunks from zero are half as long where chunks fill the chip,
// as their kernel has room for more waves (1,021 tokens x 1,111 channels, which do
// not: 65.4 for 67.7 us with whole ones).
constexpr int scan_grad_waves(int states) { return states > 16 ? 1 : states > 8 ? 2 : 3; }
inline int scan_grad_chunk(int64_t tokens, int64_t seqs, int channels, int groups, int states) {
  return scan_chunk_tokens(tokens, seqs, (scan_tiles(channels, groups) + 3) / 4, scan_grad_waves(states), 0.7);
}
inline int scan_grad_part(int chunk) { return chunk >= kScanShort ? chunk / 2 : chunk; }
// The most slots of any call with at most these tokens and sequences, of chunks of
// `least` tokens and more, or shorter ones of calls that do not fill the chip
inline int64_t scan_most_of(int64_t tokens, int64_t seqs, int64_t workgroups, int waves, int least) {
  const int64_t all = scan_slots(tokens, seqs, kScanLeast), many = scan_slots(tokens, seqs, least);
  const int64_t few = scan_few(workgroups, waves);
  return few > all ? all : few > many ? few : many;
}
// Of the gradient's chunks,
inline int64_t scan_most_chunks(int64_t tokens, int64_t seqs, int channels, int groups, int states) {
  return scan_most_of(tokens, seqs, (scan_tiles(channels, groups) + 3) / 4, scan_grad_waves(states), kScanShort);
}
// and of the forward pass's, with `grad` also the gradient's and those from zero
inline int64_t scan_most_slots(int64_t tokens, int64_t seqs, int channels, int groups, int states, bool grad) {
  const int64_t workgroups = (scan_tiles(channels, groups) + 3) / 4;
  const int64_t most = scan_most_of(tokens, seqs, workgroups, scan_forward_waves(states), kScanShort);
  if (!grad) return most;
  const int64_t back = scan_most_of(tokens, seqs, workgroups, scan_grad_waves(states), scan_grad_part(kScanShort));
  return most > back ? most : back;
}

struct BlockNormArgs {
  int64_t tokens;
  int heads, dim;
  int gate, out_norm;  // gate: 0 none, 1 silu, 2 sigmoid
  float eps, scale;
  Rows a, z, res, h, y;  // res.ptr, h.ptr, y.ptr may be nullptr
  const float *wo, *wi;  // [dim] or nullptr (ones)
  // backward
  Rows dh, dy, da, dz, dres;  // dh.ptr, dy.ptr, dres.ptr may be nullptr
  float *dwo, *dwi;           // [dim] or nullptr
  float *part;                // [blocks][2][dim]
};

// dtype: 0 fp32, 1 bf16, 2 fp16
hipError_t launch_conv(const ConvArgs &a, int dtype, bool wide, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs &a, int dtype, bool wide, hipStream_t stream);
hipError_t launch_conv_backward(const ConvArgs &a, int dtype, bool wide, hipStream_t stream);
hipError_t launch_scan(const ScanArgs &a, int dtype, int states, hipStream_t stream);
hipError_t launch_scan_step(const ScanArgs &a, int dtype, int states, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs &a, int dtype, int states, hipStream_t stream);
int64_t block_norm_blocks(int64_t rows, int dim);  // workgroups of the backward pass
hipError_t launch_block_norm(const BlockNormArgs &a, int dtype, int stream_dtype, hipStream_t stream);
hipError_t launch_block_norm_backward(const BlockNormArgs &a, int dtype, int stream_dtype, hipStream_t stream);

}  // namespace lq
