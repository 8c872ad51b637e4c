// ssm.hpp -- internal launch interface of the state-space block's operators
// (short convolution, selective scan, residual norm, 8-bit product) between
// their C ABI (api_ssm.cpp) and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hyena {

// ------------------------------------------------------- short convolution
struct ConvArgs {
  const void* x;           // [B][D][L]; [B][D] for the step
  const float* w;          // [D][T]
  const float* bias;       // [D] or nullptr
  const void* state;       // [B][D][T-1] or nullptr
  const int32_t* lengths;  // [B] or nullptr
  void* y;
  void* state_out;         // or nullptr
  // backward
  const void* gy;
  const void* gstate_out;  // or nullptr
  void* gx;
  float* gw;               // [D][T]
  float* gbias;            // [D] or nullptr
  void* gstate;            // or nullptr
  float* partial;          // workspace, [parts][D][T+1]
  int B, D, T, silu, io;
  int64_t L;
};

// Rows share a workgroup of 256 threads when they are short: `per` threads
// (a power of two, `each` steps to a thread) to a row, or `blocks` workgroups
// of `span` steps along a long one.
struct ConvGrid {
  int per, lper;
  int64_t blocks, groups;
};
constexpr int64_t kConvStep = 2048;   // the forward's span: one word of 8 steps to a thread
inline ConvGrid conv_grid(int64_t B, int64_t D, int64_t L, int64_t span, int64_t each = 8) {
  ConvGrid g;
  const int64_t words = ((L < span ? L : span) + each - 1) / each;
  g.lper = 0;
  while (g.lper < 8 && (1 << g.lper) < words) ++g.lper;
  g.per = 1 << g.lper;
  g.blocks = (L + span - 1) / span;
  const int64_t rows = 256 >> g.lper;
  g.groups = (B * D + rows - 1) / rows * g.blocks;
  return g;
}

// Backward: a workgroup keeps to one channel and walks over `seqs` sequences
// (256 / per of them at a time) and kConvSpan steps of each, so that its sums
// over batch and time leave one partial.  Sequences are spread over
// workgroups until there are about eight to a compute unit.
constexpr int64_t kConvSpan = 16384;
// Steps to a thread of the backward: with up to 4 taps 16, of which 3 more
// have their p computed again instead of 3 of 8 (45 -> 39 us for 8 x 1536 x
// 2048 bf16); with more taps 8, for want of registers.
constexpr int conv_each(int T) { return T <= 4 ? 16 : 8; }
struct ConvBackwardGrid {
  int per, lper;
  int64_t blocks, groups, seqs, parts;   // blocks along time, groups of sequences
};
inline ConvBackwardGrid conv_backward_grid(int64_t B, int64_t D, int64_t L, int T) {
  const ConvGrid c = conv_grid(B, D, L, kConvSpan, conv_each(T));
  ConvBackwardGrid g;
  g.per = c.per;
  g.lper = c.lper;
  g.blocks = (L + kConvSpan - 1) / kConvSpan;
  const int64_t at_once = 256 >> c.lper, most = (B + at_once - 1) / at_once;
  int64_t n = (2048 + D * g.blocks - 1) / (D * g.blocks);
  if (n > most) n = most;
  g.seqs = (most + n - 1) / n * at_once;
  g.groups = (B + g.seqs - 1) / g.seqs;
  g.parts = g.blocks * g.groups;
  return g;
}

hipError_t short_conv(const ConvArgs& a, hipStream_t s);
hipError_t short_conv_step(const ConvArgs& a, hipStream_t s);
hipError_t short_conv_backward(const ConvArgs& a, hipStream_t s);

// ---------------------------------------------------------- selective scan
constexpr int kScanChunk = 128;     // steps that 16 lanes scan at once, 8 each
constexpr int kScanTile = 16;       // channels of a workgroup: 4 waves of 4 (a wave's 4 where they share the states)

struct ScanArgs {
  const void *u, *delta, *Bm, *Cm, *z;     // z: or nullptr
  const float *A, *skip, *dbias, *state;   // skip, dbias, state: or nullptr
  const int32_t* lengths;                  // or nullptr
  void* y;
  float* state_out;                        // or nullptr
  int B, D, G, N, softplus, io;
  int64_t L;
  int split;                               // waves that share a channel's states: 1 or 4
  // time axis split into `segs` segments of `seg` steps (a multiple of the
  // chunk): end states and sums of dt of all but the last, when segs > 1
  int segs;
  int64_t seg;
  float* hend;                             // [B][segs][D][N]
  float* sdt;                              // [B][segs][D]
  // backward
  const void* gy;
  const float* gstate_out;                 // or nullptr
  void *gu, *gdelta, *gB, *gC, *gz;        // gz: or nullptr
  float *gA, *gskip, *gdbias, *gstate;     // all but gA: or nullptr
  int chunks;                              // ceil(L / kScanChunk)
  int splits;                              // workgroups that share a chunk's channels
  float* hc;                               // [B][chunks][D][N] end states, then states at the chunks' starts, then gA's parts
  float* qc;                               // [B][chunks][D][N] carries towards the chunks' starts, then from their ends
  float* dts;                              // [B][chunks][D] sums of dt
  float* ps;                               // [B][chunks][D] gskip's parts
  float* pb;                               // [B][chunks][D] gdelta_bias's parts
  float* gbc;                              // [splits][2][B][G][N][L] parts of gB and gC, when splits > 1
};

// How the forward scan fills the chip.  It is bound by its arithmetic once a
// SIMD holds three waves; with k of them it takes t(k) of their single times
// (1.98, 2.4 and 3.15 of a saturated one measured for k = 1, 2, 3), k being
// what the fullest of 256 compute units gets.  Two ways to more waves:
//   split  4 waves share 4 channels, a quarter of the states each, instead of
//          16 channels with all states: what does not depend on the state
//          (3 states' worth of work, 6.5 with the meeting of the parts) is
//          done by all four.  1536 rows of 512 steps with 16 states: 23.0 us
//          alone, 14.8 shared; 4096 rows of 2048 steps: 83 alone, 92 shared;
//   segs   the time axis in segments of `seg` steps: a first pass over their
//          ends costs 0.72 of the scan and a launch (about 30 units of one
//          state of one chunk), and each workgroup joins the ends before it.
//          768 rows of 65536 fp32 steps: 581 us in 11 segments, 2.1
//          workgroups to a compute unit, 475 in 16, which are 3.
struct ScanPlan {
  int split, segs;
  int64_t seg;
};
inline ScanPlan scan_plan(int64_t B, int64_t D, int64_t N, int64_t L) {
  const int64_t groups = B * ((D + kScanTile - 1) / kScanTile), chunks = (L + kScanChunk - 1) / kScanChunk;
  ScanPlan best{1, 1, chunks * kScanChunk};
  double least = -1;
  for (int split = 1; split <= 4; split *= 4) {
    for (int64_t s = 1; s <= 256;) {
      const int64_t per = (chunks + s - 1) / s;       // s is the least number that gives segments of `per` chunks
      const int64_t k = (groups * split * s + 255) / 256;
      const double t = k == 1 ? 1.98 : k == 2 ? 2.4 : k == 3 ? 3.15 : (double)k;
      const double work = (split > 1 ? 6.5 : 3.1) + (double)((N + split - 1) / split);
      const double cost = t * work * (double)per * (s > 1 ? 1.72 : 1.0) + (s > 1 ? 30.0 + 0.4 * (double)s : 0.0);
      if (least < 0 || cost < least) {
        least = cost;
        best = ScanPlan{split, (int)s, per * kScanChunk};
      }
      if (per == 1) break;
      s = (chunks + per - 2) / (per - 1);
    }
  }
  return best;
}

// Channels of a workgroup of the backward's last pass.  Its LDS is 2.25 KB to
// a state (2.5 with 32 channels): beyond 32 states one workgroup fills a
// compute unit, and 8 waves, two to a SIMD, run it instead of 4 (6144 rows of
// 2048 steps, 64 states: 1.37 ms with 4, 1.08 ms with 8).
// A group of up to 16 channels fills no more than 4.
constexpr int scan_backward_tile(int64_t N, int64_t per_group) { return N > 32 && per_group > 16 ? 32 : 16; }

struct ScanBackwardLayout {
  int chunks, splits;
  int64_t hc, qc, dts, ps, pb, gbc, total;   // byte offsets
};

inline ScanBackwardLayout scan_backward_layout(int64_t B, int64_t D, int64_t G, int64_t N, int64_t L) {
  ScanBackwardLayout w;
  w.chunks = (int)((L + kScanChunk - 1) / kScanChunk);
  const int64_t tile = scan_backward_tile(N, D / G), tiles = (D / G + tile - 1) / tile;
  // about 1024 workgroups, four to a compute unit; of up to twice as many, the
  // number that shares the channels out most evenly (48 channels of 65536
  // steps: three workgroups of one tile rather than one of two and one of one)
  int64_t least = (1024 + B * G * w.chunks - 1) / (B * G * w.chunks), s = 1;
  if (least > tiles) least = tiles;
  for (int64_t k = least, slots = 0; k <= 2 * least && k <= tiles; ++k) {
    const int64_t n = (tiles + k - 1) / k * k;
    if (slots == 0 || n < slots) slots = n, s = k;
  }
  const int64_t per = (tiles + s - 1) / s;
  w.splits = (int)((tiles + per - 1) / per);
  const auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  const int64_t st = up(B * w.chunks * D * N * 4), rows = up(B * w.chunks * D * 4);
  w.hc = 0;
  w.qc = st;
  w.dts = 2 * st;
  w.ps = w.dts + rows;
  w.pb = w.ps + rows;
  w.gbc = w.pb + rows;
  w.total = w.gbc + (w.splits > 1 ? w.splits * 2 * B * G * N * L * 4 : 0);
  return w;
}

hipError_t selective_scan(const ScanArgs& a, hipStream_t s);
hipError_t selective_scan_step(const ScanArgs& a, hipStream_t s);
hipError_t selective_scan_backward(const ScanArgs& a, hipStream_t s);

// ------------------------------------------------------------ residual norm
struct NormArgs {
  const void *x, *residual;   // residual: or nullptr
  const float* weight;
  void* y;                    // I/O dtype, or
  uint8_t* q;                 // e4m3 codes with
  float* scales;              // [rows][ceil(D/128)]
  void* s_out;                // the sum; nullptr without residual
  int64_t rows;
  int D, io;
  float eps;
  // backward
  const void *gy, *gs;        // gs: or nullptr
  void* gx;
  float* gw;
  float* partial;             // workspace, [norm_backward_parts][D]
  // 8-bit cast without a norm: blocks of block_rows x 128
  int block_rows;
};

// Workgroups of the backward, which leave a partial each: they take 4 rows at
// a time up to D = 1024, one beyond.
inline int64_t norm_backward_parts(int64_t rows, int64_t D) {
  const int64_t n = D <= 1024 ? (rows + 3) / 4 : rows;
  return n < 1024 ? n : 1024;
}

hipError_t rms_norm(const NormArgs& a, hipStream_t s);
hipError_t rms_norm_backward(const NormArgs& a, hipStream_t s);
hipError_t quantize(const NormArgs& a, hipStream_t s);

// ------------------------------------------------------------ 8-bit product
struct ScaledArgs {
  const uint8_t* q;        // [M][K] e4m3
  const float* scales;     // [M][ceil(K/128)]
  const uint8_t* wq;       // [N][K] e4m3
  const float* wscales;    // [ceil(N/128)][ceil(K/128)]
  const float* bias;       // [N] or nullptr
  void* out;               // [M][N], or [M/L][N][L] (channel_major)
  int64_t M, N, K, L;
  int io, channel_major;
};

hipError_t scaled_matmul(const ScaledArgs& a, hipStream_t s);

}  // namespace hyena
