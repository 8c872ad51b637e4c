// linattn.hpp -- internal launch interface of the linear-attention block's
// operators (linear attention with decays, rotary positions, group norm)
// between their C ABI (api_linattn.cpp) and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hyena {

// An activation [B][L][heads][D]: elements between sequences, tokens and
// heads; a head's D values are contiguous.  Head h of the operator's H reads
// head h / share.
struct HeadView {
  const void* p;
  int64_t batch, token, head;
  int share;
  int64_t total;           // elements from the first to behind the last
};

// ------------------------------------------------------- linear attention
//
// One pass of the recurrence
//   S[t] = lambda S[t-1] + su k[t] v[t]^T,   out[t] = so S[t]^T q[t]
// over tokens in order, or from a sequence's last one to its first.  The
// forward is one pass, the backward three (LinArgs.pass).
struct LinPass {
  HeadView q, k, v;        // q, k of DK values to a head, v and out of DV
  void* out;               // [B][L][H][DV], I/O dtype or fp32 (out_f32)
  int out_f32;
  int DK, DV;
  float so, su;
  int reverse;             // from the last token; the first one finds the state undecayed
  const float* s0;         // [B][H][..] state or nullptr: element (dk, dv) at dk s0_k + dv s0_v
  int s0_k, s0_v;
  float* seg;              // split time axis: states behind all segments but the last, [B][H][segs - 1][..],
  int seg_k, seg_v;        // element (dk, dv) at dk seg_k + dv seg_v
  float* s_out;            // state after the last token ([DK][DV]), times lambda if reverse; or nullptr
};

struct LinArgs {
  LinPass pass[3];
  int passes;
  LinPass fill[2];         // what forms the states behind the segments: q, so and out unused, seg_v 1, all of the same sizes
  int fills;
  const float* log_decay;  // [H] or nullptr
  const int32_t* lengths;  // [B] or nullptr
  int B, H, io;
  int64_t L;
  int segs;                // the time axis in segments of `seg` tokens
  int64_t seg;
};

// How a pass fills the chip: the time axis in segments, so that there are as
// many workgroups (of 64 or 128 columns of the state) as the compute units
// hold at once.
constexpr int64_t kLinSegment = 256;   // the fewest tokens of a segment; a multiple of the kernels' blocks
struct LinPlan {
  int segs;
  int64_t seg;
};
inline int64_t lin_columns(int64_t DV) { return DV <= 64 ? 64 : 128; }
inline int64_t lin_resident(int64_t DK, int64_t DV) { return DK > 128 ? 256 : DK > 64 || DV > 64 ? 512 : 1024; }
inline LinPlan lin_plan(int64_t B, int64_t L, int64_t H, int64_t DK, int64_t DV) {
  const int64_t cols = lin_columns(DV), groups = B * H * ((DV + cols - 1) / cols);
  int64_t segs = lin_resident(DK, DV) / groups, most = (L + kLinSegment - 1) / kLinSegment;
  if (segs > most) segs = most;
  if (segs < 1) segs = 1;
  int64_t seg = (L + segs - 1) / segs;
  seg = (seg + 63) / 64 * 64;
  return LinPlan{(int)((L + seg - 1) / seg), seg};
}
// The backward's passes for gq and gk share a launch where both or neither are
// summed over shared heads.  In bf16 half as many segments as in the forward
// fill the chip: 4 x 2048 tokens of 12 heads 64 x 128 112 us (116 with as many
// as in the forward), 32768 of 6 heads 128 x 128 260 (274), of 12 heads 64 x 64
// 205 (210).  With k and v on fewer heads, where those passes share no launch:
// 32768 of 6 heads 128 x 128 on 2 344 (363), 4 x 2048 of 12 heads 64 x 64 on 4
// 91 and 91, of 64 x 128 154 (148), the one that half as many cost.  In fp32
// they cost: 16384 of 6 heads 128 x 128 352 us, 400 with half of them, on 2
// heads 388 and 433, 2 x 8192 of 12 heads 64 x 64 226 and 245.
inline LinPlan lin_backward_plan(int64_t B, int64_t L, int64_t H, int64_t Dk, int64_t Dv, int io) {
  return lin_plan(io ? 2 * B : B, L, H, Dk, Dv);
}
// The most workgroups of a launch of one pass with DV columns, counted by
// their 256 threads (128 columns may take 512).
inline int64_t lin_groups(const LinPlan& p, int64_t B, int64_t H, int64_t DV) {
  return B * H * p.segs * (DV <= 64 ? 1 : DV <= 128 ? 2 : 4);
}

struct LinStepArgs {
  HeadView q, k, v;        // token strides unused
  const float* log_decay;  // or nullptr
  float* state;            // [B][H][Dk][Dv]
  void* o;                 // [B][H][Dv]
  int B, H, Dk, Dv, io;
  float scale;
};

// A token's launch: words of 4 columns (1 where Dv is no multiple) of a head's
// state, `cols` of them (a power of two) to a workgroup.
struct LinStepPlan {
  int vec, cols, tiles;
};
inline LinStepPlan lin_step_plan(int Dv) {
  const int vec = Dv % 4 ? 1 : 4, words = Dv / vec;
  int cols = 1;
  while (cols < words && cols < 64) cols *= 2;
  return LinStepPlan{vec, cols, (words + cols - 1) / cols};
}

// Sums over the heads that share one: out[t][j][d] = sum of x[t][j share ..][d].
struct FoldArgs {
  const float* x[3];       // [tokens][heads share][D], or nullptr
  void* out[3];            // [tokens][heads][D]
  int heads[3], share[3], D[3];
  int64_t tokens;
  int io;
};

hipError_t linear_attention(const LinArgs& a, hipStream_t s);
hipError_t linear_attention_step(const LinStepArgs& a, hipStream_t s);
hipError_t fold_heads(const FoldArgs& a, hipStream_t s);

// -------------------------------------------------------- rotary positions
struct RotaryArgs {
  HeadView x, out;
  const double* freq;        // [R / 2]
  const int32_t* positions;  // or nullptr: the token's index
  int64_t pos_batch, pos_token;
  int64_t tokens, L;         // B L, L
  int H, D, R, interleaved, io, in_place;
  float scale, sine;         // sine: 1, or -1 for the inverse
};

// A launch: places of a head (two words of 16 bytes each, of the pairs that
// are turned, then of copied values), and threads that share a token's heads,
// enough for half a million threads in all.
inline int64_t rotary_word(const RotaryArgs& a) { return a.io ? 8 : 4; }
inline int64_t rotary_turning(const RotaryArgs& a) { return (a.R / 2 + rotary_word(a) - 1) / rotary_word(a); }
inline int64_t rotary_places(const RotaryArgs& a) {
  return rotary_turning(a) + (a.in_place ? 0 : (a.D - a.R + 2 * rotary_word(a) - 1) / (2 * rotary_word(a)));
}
inline int64_t rotary_shares(const RotaryArgs& a) {
  const int64_t want = ((int64_t)1 << 19) / (a.tokens * rotary_places(a)) + 1;
  return want < a.H ? want : a.H;
}
inline int64_t rotary_groups(const RotaryArgs& a) {
  return (a.tokens * rotary_places(a) * rotary_shares(a) + 255) / 256;
}

hipError_t rotary(const RotaryArgs& a, hipStream_t s);

// --------------------------------------------------------------- group norm
struct GroupNormArgs {
  const void *x, *z;           // [rows][G Dg]; z: or nullptr
  const float *weight, *bias;  // [G Dg] or nullptr
  void* y;
  int64_t rows;
  int G, Dg, silu, io;
  float eps;
  // backward
  const void* gy;
  void *gx, *gz;               // gz: or nullptr
  float *gw, *gb;              // or nullptr
  float* partial;              // workspace, [parts][2][G Dg]
};

hipError_t group_norm(const GroupNormArgs& a, hipStream_t s);
hipError_t group_norm_backward(const GroupNormArgs& a, hipStream_t s);

// How a launch covers rows of G groups of Dg values: `lanes` threads (a power
// of two up to 256) to a group, `words` words of 8 values to a thread; a
// workgroup of 256 threads takes `per` neighbouring groups of `rows` rows at
// a time.  Groups beyond 256 x 4 words (`words` 0) are not held: x is read three
// times, by the backward four times, and gy and z twice.
struct GroupNormPlan {
  int lanes, words, per, rows;
  int64_t blocks;              // workgroups across a row's groups
};
inline GroupNormPlan group_norm_plan(int64_t G, int64_t Dg) {
  GroupNormPlan p;
  const int64_t w = (Dg + 7) / 8;
  if (w <= 64) {
    p.lanes = 1;
    while (p.lanes < w) p.lanes *= 2;
    p.words = 1;
  } else if (w <= 128) {
    p.lanes = 64, p.words = 2;
  } else if (w <= 256) {
    p.lanes = 256, p.words = 1;
  } else if (w <= 512) {
    p.lanes = 256, p.words = 2;
  } else {
    p.lanes = 256, p.words = w <= 1024 ? 4 : 0;
  }
  // the most neighbouring groups (a power of two) that leave the fewest places idle: of 12 groups on 16 places 4
  // rows of 4 (the backward of 16384 rows of 12 x 128: 50 us, 55 with one row of 12 groups)
  const int units = 256 / p.lanes;
  p.per = 1;
  for (int n = 2; n <= units; n *= 2)
    if ((G + n - 1) / n * n <= (G + p.per - 1) / p.per * p.per) p.per = n;
  p.rows = units / p.per;
  p.blocks = (G + p.per - 1) / p.per;
  return p;
}
// Workgroups of the backward, which leave a partial each, along the rows.
inline int64_t group_norm_backward_parts(int64_t rows, int64_t G, int64_t Dg) {
  const GroupNormPlan p = group_norm_plan(G, Dg);
  const int64_t n = (rows + p.rows - 1) / p.rows, most = (2048 + p.blocks - 1) / p.blocks;
  return n < most ? n : most;
}

}  // namespace hyena
