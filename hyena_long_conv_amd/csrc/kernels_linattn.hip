// kernels_linattn.hip -- linear attention with a decay for each head: passes
// over whole sequences, single tokens, and sums over shared heads.
//
//   S[t] = lambda S[t-1] + su k[t] v[t]^T,  out[t] = so S[t]^T q[t].
//
// The forward is one pass.  With G[t] the loss's gradient with respect to
// S[t], gq[t] = S[t] go[t], gk[t] = G[t] v[t] and gv[t] = G[t]^T k[t], and G
// runs from the last token to the first as S does from the first to the last:
// the backward is three passes of the same kernel.
//
// What bounds them: the bytes of q, k, v and out at a copy's rate (5 TB/s)
// would take 31 us for 8 x 2048 tokens of 12 heads 64 x 128 in bf16, 81 us for
// 65536 tokens of 6 heads 128 x 128, 161 us for 65536 of 12 heads 64 x 64 in
// fp32.  So few heads do not fill the chip one token after the other; the time
// axis is split, and k and v are read twice, once for the states behind the
// segments (k_lin with FILL, then k_lin_join) and once for the outputs: 46 +
// 23 + 5, 128 + 54 + 14 and 214 + 100 + 13 us.  The main passes lose to their
// memory what the barriers between a block's phases leave idle (vector units
// 47% and matrix units 29% busy at 128 x 128; in fp32, whose matrix
// instructions take 16 times as long, 65% of those).
#include <hip/hip_runtime.h>

#include "linattn.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

// lambda^n = keep + f, kept as the pair that a state is multiplied by: near 1
// as 1 and expm1, since a rounded factor's error would come back with every
// block of a slow decay (over 2^16 tokens at log_decay -1e-4 that made 5e-5 of
// the result).  n = 0 gives 1 whatever the decay.
struct Decay { float f, keep; };
__device__ __forceinline__ Decay decay_of(float g, int64_t n) {
  if (n == 0) return {0.f, 1.f};
  const float x = g * (float)n;
  return x > -0.5f ? Decay{expm1f(x), 1.f} : Decay{expf(x), 0.f};
}
__device__ __forceinline__ float decayed(float s, Decay d, float add) { return fmaf(s, d.f, fmaf(s, d.keep, add)); }

// lambda^n.  The exponent's product with log2(e) is kept in two parts: its
// rounding, and log2(e)'s, would cost |log_decay n| units of the last place,
// alike in every block.
__device__ __forceinline__ float power_of(float g, int n) {
  if (n == 0) return 1.f;
  const float x = g * (float)n, hi = x * kLog2e;
  const float lo = fmaf(x, 1.92596299e-8f, fmaf(x, kLog2e, -hi)) + fmaf(g, (float)n, -x) * kLog2e;
  return x < -87.f ? 0.f : exp2_fast(hi) * fmaf(lo, 0.6931471805599453f, 1.f);
}

// -------------------------------------------------- passes over sequences
//
// A workgroup of 4 or 8 waves walks over a sequence (or a segment of it) in blocks
// of C tokens and keeps 16 NC columns of a head's state for each wave in the
// accumulators of its matrix instructions.  For a block with the state S
// in front of it, weights W = tril(lambda^(i-j)) and the rows k, q, v in LDS:
//   P   = so su W * (q k^T)                     shared out by tiles of 16 x 16,
//   out = so lambda^(i+1) (q S) + P v,
//   S   = lambda^C S + k^T (su lambda^(C-1-j) v).
// All products are formed transposed, with the state's and P's accumulators
// as operands of the next product as they lie: lane l of group g = l / 16
// holds rows 4 g .. 4 g + 3 of a tile's column l % 16, and two tiles make the
// 8 values that an operand holds for its row or column.  Tokens are taken in
// that order, 4 g .. 4 g + 3, 16 + 4 g .. 16 + 4 g + 3 of 32, and the state's
// rows are dealt to two tiles so that the 8 are 8 g .. 8 g + 7 of 32: what q
// and k hold in 16 bytes.  So the state never goes through LDS, and P does
// once, lane by lane.

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Eight values of an operand, as two halves of four.
template <int IOT> struct Frag;
template <> struct Frag<0> { f32x4v a, b; };
template <> struct Frag<1> { u32x2v a, b; };

__device__ __forceinline__ f32x4v mma(const Frag<1>& x, const Frag<1>& y, f32x4v c) {
  const u32x4v p = {x.a[0], x.a[1], x.b[0], x.b[1]}, q = {y.a[0], y.a[1], y.b[0], y.b[1]};
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, p), __builtin_bit_cast(bf16x8v, q), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4v mma(const Frag<0>& x, const Frag<0>& y, f32x4v c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.a[e], y.a[e], c, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.b[e], y.b[e], c, 0, 0, 0);
  return c;
}

// The product of the operands' first halves alone.
__device__ __forceinline__ f32x4v mma_half(const Frag<1>& x, u32x2v y, f32x4v c) {
  return mma(Frag<1>{x.a, u32x2v{0u, 0u}}, Frag<1>{y, u32x2v{0u, 0u}}, c);
}
__device__ __forceinline__ f32x4v mma_half(const Frag<0>& x, f32x4v y, f32x4v c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x.a[e], y[e], c, 0, 0, 0);
  return c;
}

// Rows of D values in LDS.  Word w of 16 bytes of row r lies in slot w ^ twist(r),
// which keeps 16 rows of a word apart, 8 rows of 4 neighbouring halves (v,
// transposed) and, in fp32, 4 rows, 4 apart, of 4 words that are neighbours or
// 2 apart; 8 rows of 4 halves, 16 bytes apart (k, transposed), meet in pairs.
// twist takes the row's last four bits and D is a power of two, so value d of
// row r0 + r, r0 a multiple of 16 and r < 16, is at (r0 D + base(r)) ^ d.
template <int IOT, int D> struct Lds;
template <int D> struct Lds<0, D> {
  typedef float T;
  typedef f32x4v Four;
  static __device__ __forceinline__ int base(int r) {
    return (r * D) ^ (((r & 3) << 1 | (r >> 2 & 1) | (r >> 3 & 1) << 3) << 2);
  }
  // eight values of a row from d, a multiple of 8
  static __device__ __forceinline__ Frag<0> row(const T* p, int base_r, int d) {
    return {*reinterpret_cast<const Four*>(p + (base_r ^ d)), *reinterpret_cast<const Four*>(p + (base_r ^ d ^ 4))};
  }
  // values of rows r .. r + 3 (a multiple of 4) at a column for each lane, which base_c = base(r) ^ column holds
  static __device__ __forceinline__ int next(int l) { return l; }             // 16 neighbouring columns
  static __device__ __forceinline__ int dealt(int l) { return 8 * (l >> 2) + (l & 3); }   // rows of a tile of the state
  static __device__ __forceinline__ int column_base(int r, int l, int column) { return base(r) ^ column; }
  static __device__ __forceinline__ Four column(const T* p, int base_c, int d) {
    return Four{p[base_c ^ d], p[base_c ^ d ^ base(1)], p[base_c ^ d ^ base(2)], p[base_c ^ d ^ base(3)]};
  }
};
template <int D> struct Lds<1, D> {
  typedef uint16_t T;
  typedef u32x2v Four;
  static __device__ __forceinline__ int base(int r) {
    const int twist = D >= 128 ? ((r & 7) << 1) | ((r >> 3) & 1) : (r & 6) | ((r >> 3) & 1);
    return (r * D) ^ (twist << 3);
  }
  static __device__ __forceinline__ Frag<1> row(const T* p, int base_r, int d) {
    const u32x4v v = *reinterpret_cast<const u32x4v*>(p + (base_r ^ d));
    return {u32x2v{v[0], v[1]}, u32x2v{v[2], v[3]}};
  }
  // the transposing read: lane l gives the address of row l / 4 and of columns that lanes 4 (l % 4) .. get
  static __device__ __forceinline__ int next(int l) { return 4 * (l & 3); }
  static __device__ __forceinline__ int dealt(int l) { return 8 * (l & 3); }
  static __device__ __forceinline__ int column_base(int r, int l, int column) { return base(r + (l >> 2)) ^ column; }
  static __device__ __forceinline__ Four column(const T* p, int base_c, int d) {
    return __builtin_bit_cast(Four, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + (base_c ^ d))));
  }
};

// Eight values behind an address that all lanes share, which is held in scalar
// registers, at a lane's own offset in bytes.
template <int IOT>
__device__ __forceinline__ Raw8<IOT> ld8_from(const char* p, uint32_t off) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  typedef const __attribute__((address_space(1))) char* global;
  const global q = reinterpret_cast<global>((uint64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                                            (uint32_t)__builtin_amdgcn_readfirstlane((int)v)) + off;
  Raw8<IOT> r;
  if constexpr (IOT == 0) {
    r.a = *reinterpret_cast<const __attribute__((address_space(1))) f32x4_e4*>(q);
    r.b = *reinterpret_cast<const __attribute__((address_space(1))) f32x4_e4*>(q + 16);
  } else {
    r.a = *reinterpret_cast<const __attribute__((address_space(1))) u32x4_e2*>(q);
  }
  return r;
}

// The same value, which the compiler cannot tell: what is computed from it is
// computed where it is used, instead of once and kept in registers.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ f32x4v here(f32x4v v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ u32x2v narrow4(f32x4v v) { return u32x2v{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])}; }
__device__ __forceinline__ f32x4v widen4(f32x4v v) { return v; }
__device__ __forceinline__ f32x4v widen4(u32x2v v) {
  return f32x4v{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
                __uint_as_float(v[1] & 0xffff0000u)};
}

// The first of four values that is not finite, or 4; and zeros in the place of all of them.
__device__ __forceinline__ bool is_bad(float v) { return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u; }
template <class Four>
__device__ __forceinline__ int first_bad(const Four& f) {
  const f32x4v v = widen4(f);
  return is_bad(v[0]) ? 0 : is_bad(v[1]) ? 1 : is_bad(v[2]) ? 2 : is_bad(v[3]) ? 3 : 4;
}
__device__ __forceinline__ void clear_bad(f32x4v& f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = is_bad(f[e]) ? 0.f : f[e];
}
__device__ __forceinline__ void clear_bad(u32x2v& f) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if ((f[e] & 0x7f80u) == 0x7f80u) f[e] &= 0xffff0000u;
    if ((f[e] & 0x7f800000u) == 0x7f800000u) f[e] &= 0xffffu;
  }
}

// fp32 values as operands: themselves in fp32, and in bf16 as a sum of bf16
// parts, each rounded from what the ones before leave: at most 2^-8 of a value
// after one part, 2^-17 after two, 2^-26, less than its last place, after three.
// The state's addends go in three, since their sum is an fp32 output (two would
// leave it off by 2.7e-6 of its norm and take 5 to 9% off the time).  A pair's
// weight and the state in its product with q go in two: at most 2^-17 of the
// sizes of an output's terms, |w| |v| and |q| |S|, are lost, which shows beside
// the output's own rounding only where the terms cancel to 2^-9 of their sizes
// or less.  One part of the state left 2^-8 of |q| |S|: 1.4 times the error of
// outputs of random values, 4 times where the keys share a direction that the
// queries lack.  Its second part costs 1 us of 45 in the main pass of 64 x 128
// heads and of 25 in that of 64 x 64, 16 of 113 at 128 x 128, 8 of 74 at 256 x 256.
template <int IOT> constexpr int kParts = IOT == 1 ? 3 : 1;     // of the state's addends
template <int IOT> constexpr int kFactors = IOT == 1 ? 2 : 1;   // of the pairs' weights
template <int IOT> constexpr int kStates = IOT == 1 ? 2 : 1;    // of the state where q meets it
template <int N>
__device__ __forceinline__ void parts_of(f32x4v a, f32x4v b, Frag<0> (&o)[N]) { o[0] = {a, b}; }
template <int N>
__device__ __forceinline__ void parts_of(f32x4v a, f32x4v b, Frag<1> (&o)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    o[k] = {narrow4(a), narrow4(b)};
    if (k < N - 1) a -= widen4(o[k].a), b -= widen4(o[k].b);
  }
}

// A block's rows of one operand on their way from global memory to LDS: W
// words of 8 values to a row, NW words to a thread, in one column of words.
// EVEN: heads of whole words, and rows near enough to each other for offsets
// of 32 bits inside a block; a word behind the block's tokens or the head's
// values is then read from the row or the head's start and set to zero on
// its way, so that no load waits for a condition.
template <int IOT, int C, int D, int THREADS, bool EVEN>
struct Rows {
  static constexpr int W = D / 8, NW = C * W > THREADS ? C * W / THREADS : 1, STEP = THREADS / W,
                       E = IOT == 0 ? 4 : 2;
  typedef Lds<IOT, D> M;
  static_assert(C * W % THREADS == 0 || THREADS % (C * W) == 0, "whole words for each thread, or one for some");
  Raw8<IOT> word[NW];
  const char* base;              // the head's first value of the sequence
  int64_t token;                 // elements between tokens
  int64_t last;                  // backward in time: the sequence's last token; otherwise -1
  int64_t total;                 // elements behind base
  int d, row, col;
  bool live;
  __device__ __forceinline__ void init(const HeadView& v, int64_t b, int h, int c0, int d_, int64_t n, bool reverse) {
    const int64_t at = b * v.batch + h / v.share * v.head + c0;
    base = static_cast<const char*>(v.p) + at * E;
    total = v.total - at;
    token = v.token;
    last = reverse ? n - 1 : -1;
    d = d_ - c0;
    row = threadIdx.x / W % C;
    col = 8 * (threadIdx.x % W);
    live = col < d;
  }
  // The block's `now` tokens from t0 on.
  __device__ __forceinline__ void load(int64_t t0, int now) {
    const bool back = last >= 0;
    if constexpr (EVEN) {
      const char* at = base + (back ? last - t0 - (now - 1) : t0) * token * E;   // its first value in memory
      const uint32_t inside = live ? col * E : 0, step = (uint32_t)token * E;
      if (now == C) {
        const uint32_t off = here((back ? C - 1 - row : row) * step + inside);
        if (!back) {
#pragma unroll
          for (int m = 0; m < NW; ++m) word[m] = ld8_from<IOT>(at + m * STEP * (int64_t)step, off);
        } else {
#pragma unroll
          for (int m = 0; m < NW; ++m) word[m] = ld8_from<IOT>(at - m * STEP * (int64_t)step, off);
        }
      } else {
#pragma unroll
        for (int m = 0; m < NW; ++m) {
          const int r = min(row + m * STEP, now - 1);
          word[m] = ld8_from<IOT>(at, (uint32_t)(back ? now - 1 - r : r) * step + inside);
        }
      }
    } else {
#pragma unroll
      for (int m = 0; m < NW; ++m) {
        const int r = row + m * STEP;
        const int64_t t = back ? last - t0 - r : t0 + r;
        word[m] = ld8n<IOT>(base, r < now ? t * token + col : 0, r < now ? d - col : 0, total);
      }
    }
  }
  // The words of the last load, `had` tokens of them.
  __device__ __forceinline__ void store(typename M::T* lds, int had) const {
    if (THREADS > C * W && threadIdx.x >= C * W) return;
    if (!EVEN || (had == C && d >= D)) put<false>(lds, had);
    else put<true>(lds, had);
  }
  template <bool MASK>
  __device__ __forceinline__ void put(typename M::T* lds, int had) const {
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      const Raw8<IOT> w = !MASK || (live && row + m * STEP < had) ? word[m] : zero8<IOT>();
      const int r = row + m * STEP, b = M::base(r & 15), r0 = (r & ~15) * D;
      if constexpr (IOT == 0) {
        *reinterpret_cast<f32x4v*>(lds + r0 + (b ^ col)) = w.a;
        *reinterpret_cast<f32x4v*>(lds + r0 + (b ^ (col + 4))) = w.b;
      } else {
        *reinterpret_cast<u32x4v*>(lds + r0 + (b ^ col)) = w.a;
      }
    }
  }
};

// The first n of four values to element i.
template <int IOT>
__device__ __forceinline__ void st4n(void* p, int64_t i, f32x4v v, int n) {
  if constexpr (IOT == 0) {
    float* q = static_cast<float*>(p) + i;
    if (n >= 4) {
      *reinterpret_cast<f32x4_e4*>(q) = v;
      return;
    }
  } else {
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    if (n >= 4) {
      const u32x2v w = narrow4(v);
      *reinterpret_cast<u2*>(static_cast<uint16_t*>(p) + i) = u2{w[0], w[1]};
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) st1<IOT>(p, i + e, v[e]);
}

template <int IOT> constexpr int kBlock = IOT == 1 ? 64 : 32;   // tokens of a block

template <int IOT, int DK, int WAVES, int NC, bool FILL>
constexpr int lin_lds_bytes() {
  constexpr int C = kBlock<IOT>, E = IOT == 0 ? 4 : 2, TILES = C / 16 * (C / 16 + 1) / 2;
  return (C * ((FILL ? 1 : 2) * DK + 16 * NC * WAVES) + (FILL ? 0 : TILES * 256 * kFactors<IOT>)) * E + (3 * C + 16) * 4;
}

// FILL: the state behind a segment alone, from nothing, for all but the last segment (LinArgs.fill).
template <int IOT, int DK, int WAVES, int NC, bool FILL, bool EVEN, bool OUT32>
__global__ __launch_bounds__(64 * WAVES, DK >= 256 || NC == 2 || (DK >= 128 && WAVES == 4 && !FILL) ? 2 : 4) void k_lin(LinArgs a, int first_pass) {
  constexpr int C = kBlock<IOT>, IT = C / 16, JJ = C / 32, KT = DK / 16, DVT = 16 * NC * WAVES, NP = kParts<IOT>, NF = kFactors<IOT>, NS = kStates<IOT>;
  constexpr int HELD = 4;                              // tiles of k's rows at a time
  typedef Lds<IOT, DK> MK;
  typedef Lds<IOT, DVT> MV;
  typedef typename MK::T T;
  typedef typename MK::Four Four;
  const LinPass& p = FILL ? a.fill[blockIdx.y] : a.pass[first_pass + blockIdx.y];
  extern __shared__ __attribute__((aligned(16))) unsigned char shared[];
  float* const weight = reinterpret_cast<float*>(shared);   // su lambda^(count-1-j) of a block's tokens,
  float* const through = weight + C;                         // and so lambda^(i+1)
  float* const apart = through + C;                          // so su lambda^n at C - 1 - n, zeros behind it
  T* const lk = reinterpret_cast<T*>(apart + C + 16);
  T* const lv = lk + C * DK;
  T* const lq = lv + C * DVT;
  T* const lp = lq + C * DK;   // tiles (i, j) of 16 x 16 at (i (i + 1) / 2 + j) NF + part, 4 values to a lane
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15, g = lane >> 4;

  const int tiles = (p.DV + DVT - 1) / DVT, segs = FILL ? a.segs - 1 : a.segs;
  const int tile = (int)(blockIdx.x % (unsigned)tiles), rest = (int)(blockIdx.x / (unsigned)tiles);
  // the last segments first: what the fill read last is what the Infinity Cache still holds (65536 fp32 tokens of 12
  // heads 64 x 64: 207 -> 199 us)
  const int bh = rest / segs, nth = rest - bh * segs, sg = FILL ? nth : segs - 1 - nth, b = bh / a.H, h = bh - b * a.H, c0 = tile * DVT;
  const int64_t n = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.L) : a.L;
  const int64_t t0 = sg * a.seg, end = min(n, t0 + a.seg), size = (int64_t)p.DK * p.DV;
  const float gd = a.log_decay ? a.log_decay[h] : 0.f;
  if (FILL && t0 >= n) return;

  // the state: rows 32 (k / 2) + 8 g + 4 (k % 2) + r, column 16 (NC wave + c) + l of the tile
  const int mine = 16 * NC * wave, dv = c0 + mine + l;
  f32x4v S[KT][NC];
  {
    const float* s0 = nullptr;
    int sk = 0, sv = 0;
    if (!FILL) {
      if (sg > 0) s0 = p.seg + ((int64_t)bh * (a.segs - 1) + sg - 1) * size, sk = p.seg_k, sv = p.seg_v;
      else if (p.s0) s0 = p.s0 + bh * size, sk = p.s0_k, sv = p.s0_v;
    }
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int dk = 32 * (k / 2) + 8 * g + 4 * (k & 1) + r, d = dv + 16 * c;
          S[k][c][r] = s0 && t0 < max(n, (int64_t)1) && dk < p.DK && d < p.DV ? s0[(int64_t)dk * sk + (int64_t)d * sv] : 0.f;
        }
  }

  if (t0 < end) {
    Rows<IOT, C, DK, 64 * WAVES, EVEN> rk, rq;
    Rows<IOT, C, DVT, 64 * WAVES, EVEN> rv;
    const int first = (int)min(end - t0, (int64_t)C);
    rk.init(p.k, b, h, 0, p.DK, n, p.reverse);
    rv.init(p.v, b, h, c0, p.DV, n, p.reverse);
    rk.load(t0, first);
    rv.load(t0, first);
    if (!FILL) {
      rq.init(p.q, b, h, 0, p.DK, n, p.reverse);
      rq.load(t0, first);
    }
    Decay whole{0.f, 1.f};
    const bool busy = c0 + mine < p.DV;                 // this wave has columns; all waves load, and form P
    // P's tiles on and below the diagonal, MINE at most for a wave
    constexpr int TILES = IT * (IT + 1) / 2, MINE = (TILES + WAVES - 1) / WAVES;
    if (!FILL && threadIdx.x < C + 16) apart[threadIdx.x] = threadIdx.x < C ? p.so * p.su * power_of(gd, C - 1 - threadIdx.x) : 0.f;
    // this lane's outputs: token l of a tile, values d0 + 16 c .. + 3
    const int d0 = c0 + mine + 4 * g;
    const int64_t out_step = (p.reverse ? -1 : 1) * (int64_t)a.H * p.DV * (OUT32 ? 4 : 2);
    char* out = nullptr;
    if (!FILL)
      out = static_cast<char*>(p.out) + (((b * a.L + (p.reverse ? n - 1 - t0 : t0)) * a.H + h) * p.DV + d0) * (OUT32 ? 4 : 2) + l * out_step;
    int count = 0;
    for (int64_t t = t0; t < end; t += C) {
      const int now = (int)min(end - t, (int64_t)C);
      __syncthreads();                                // the block before has been read
      if (now != count || t <= t0 + C) {              // from the last token on, the first one finds the state undecayed
        const int lead = p.reverse && t == 0 ? 0 : 1, i = threadIdx.x;
        count = now;
        if (i < C) {
          weight[i] = i < count ? p.su * power_of(gd, count - 1 - i) : 0.f;
          through[i] = p.so * power_of(gd, i + lead);
        }
        whole = decay_of(gd, count - 1 + lead);
      }
      rk.store(lk, now);
      rv.store(lv, now);
      if (!FILL) rq.store(lq, now);
      __syncthreads();
      if (t + C < end) {
        const int next = (int)min(end - t - C, (int64_t)C);
        rk.load(t + C, next);
        rv.load(t + C, next);
        if (!FILL) rq.load(t + C, next);
      }
      if constexpr (!FILL) {
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
          // turned by the workgroup, so that the idle waves of a compute unit's workgroups are not all on one SIMD
          const int k = ((wave + (int)blockIdx.x) & (WAVES - 1)) + WAVES * m;
          if (k >= TILES) break;
          const int i = k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3, j = k - i * (i + 1) / 2;
          f32x4v acc = {0.f, 0.f, 0.f, 0.f};
          const int at = MK::base(l) ^ (8 * g), of_k = here(at + 16 * j * DK), of_q = here(at + 16 * i * DK);
#pragma unroll
          for (int d = 0; d < DK; d += 32) acc = mma(MK::row(lk, of_k, d), MK::row(lq, of_q, d), acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] *= apart[C - 1 - 16 * (i - j) - l + 4 * g + r];
          if (i == j) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = l >= 4 * g + r ? acc[r] : 0.f;
          }
          Frag<IOT> w[NF];
          parts_of(acc, acc, w);
#pragma unroll
          for (int f = 0; f < NF; ++f) *reinterpret_cast<Four*>(lp + ((k * NF + f) * 64 + lane) * 4) = w[f].a;
        }
        __syncthreads();
      }
      if (!busy) continue;
      // v transposed: this wave's columns, 8 tokens to a lane
      const auto values = [&](int j, int c) {
        const int at = here(MV::column_base(4 * g, l, MV::next(l) + mine));
        return Frag<IOT>{MV::column(lv + 32 * j * DVT, at, 16 * c), MV::column(lv + (32 * j + 16) * DVT, at, 16 * c)};
      };
      if constexpr (!FILL) {
        const T* const pt = lp + lane * 4;
        const auto weights = [&](int i, int j, int f) {
          return *reinterpret_cast<const Four*>(pt + ((i * (i + 1) / 2 + j) * NF + f) * 256);
        };
        const auto put = [&](int i, int c, f32x4v o) {
          if (16 * i + l < count) {
            if (OUT32) st4n<0>(out + 16 * i * out_step, 16 * c, o, p.DV - d0 - 16 * c);
            else st4n<1>(out + 16 * i * out_step, 16 * c, o, p.DV - d0 - 16 * c);
          }
        };
        f32x4v acc[IT][NC];
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[i][c] = f32x4v{0.f, 0.f, 0.f, 0.f};
        const int at = here(MK::base(l) ^ (8 * g));
#pragma unroll
        for (int k = 0; k < KT / 2; ++k) {
          Frag<IOT> sf[NC][NS];
#pragma unroll
          for (int c = 0; c < NC; ++c) parts_of(S[2 * k][c], S[2 * k + 1][c], sf[c]);
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const Frag<IOT> q = MK::row(lq + 16 * i * DK, at, 32 * k);
#pragma unroll
            for (int f = NS - 1; f >= 0; --f)
#pragma unroll
              for (int c = 0; c < NC; ++c) acc[i][c] = mma(sf[c][f], q, acc[i][c]);
          }
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const float w = through[16 * i + l];
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[i][c] *= w;
        }
#pragma unroll
        for (int j = 0; j < JJ; ++j) {
          Frag<IOT> vt[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) vt[c] = values(j, c);
#pragma unroll
          for (int i = 2 * j; i < IT; ++i) {
#pragma unroll
            for (int f = NF - 1; f >= 0; --f) {
              Frag<IOT> w;
              w.a = weights(i, 2 * j, f);
              if (i > 2 * j) w.b = weights(i, 2 * j + 1, f);
#pragma unroll
              for (int c = 0; c < NC; ++c)
                acc[i][c] = i == 2 * j ? mma_half(vt[c], w.a, acc[i][c]) : mma(vt[c], w, acc[i][c]);
            }
          }
        }
        float bad = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) bad = fmaf(acc[i][c][r], 0.f, bad);
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
          for (int c = 0; c < NC; ++c) put(i, c, acc[i][c]);
        if (__any(bad != 0.f)) {
          // A value of v that is not finite has met the zeros of P above the diagonal.  The diagonal's tiles again
          // with zeros in its place, for the tokens in front of it, which then hold what they would without it.
#pragma unroll 1
          for (int i = 0; i < IT; ++i) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              Frag<IOT> own = values(i / 2, c);
              int from = 16;                          // the first such token of column l
              if (i & 1) from = first_bad(own.b);
              else from = first_bad(own.a);
              from = from < 4 ? 4 * g + from : 16;
              from = min(from, __shfl_xor(from, 16));
              from = min(from, __shfl_xor(from, 32));
              if (!__any(from < 16)) continue;
              f32x4v o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int k = 0; k < KT / 2; ++k) {
                const Frag<IOT> q = MK::row(lq + 16 * i * DK, at, 32 * k);
                Frag<IOT> sf[NS];
                parts_of(here(S[2 * k][c]), here(S[2 * k + 1][c]), sf);   // not kept from above: 35 spilled registers at 128 x 128
#pragma unroll
                for (int f = NS - 1; f >= 0; --f) o = mma(sf[f], q, o);
              }
              o *= through[16 * i + l];
#pragma unroll
              for (int j = 0; j < JJ; ++j)
                if (2 * j + 1 < i) {
#pragma unroll
                  for (int f = NF - 1; f >= 0; --f)
                    o = mma(values(j, c), Frag<IOT>{weights(i, 2 * j, f), weights(i, 2 * j + 1, f)}, o);
                }
              if (i & 1) clear_bad(own.b);
              else clear_bad(own.a);
#pragma unroll
              for (int f = NF - 1; f >= 0; --f)
                o = i & 1 ? mma(own, Frag<IOT>{weights(i, i - 1, f), weights(i, i, f)}, o) : mma_half(own, weights(i, i, f), o);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int behind = __shfl(from, 4 * g + r);
                if (l < behind && behind < 16 && 16 * i + l < count && d0 + 16 * c + r < p.DV)
                  st1<OUT32 ? 0 : 1>(out + 16 * i * out_step, 16 * c + r, o[r]);
              }
            }
          }
        }
        out += C * out_step;
      }
      if (whole.keep != 0.f) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[k][c][r] = fmaf(S[k][c][r], whole.f, S[k][c][r]);
      } else {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int c = 0; c < NC; ++c) S[k][c] *= whole.f;
      }
      const int at = here(MK::column_base(4 * g, l, MK::dealt(l)));
#pragma unroll
      for (int j = 0; j < JJ; ++j) {
        Frag<IOT> vw[NC][NP];
        const float* at_j = weight + 32 * j + 4 * g;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const Frag<IOT> vt = values(j, c);
          const f32x4v x = widen4(vt.a) * *reinterpret_cast<const f32x4v*>(at_j);
          const f32x4v y = widen4(vt.b) * *reinterpret_cast<const f32x4v*>(at_j + 16);
          parts_of(x, y, vw[c]);
        }
#pragma unroll
        for (int k0 = 0; k0 < KT; k0 += HELD) {
          Frag<IOT> kt[HELD];
#pragma unroll
          for (int k = 0; k < HELD; ++k) {
            const int d = 32 * ((k0 + k) / 2) + 4 * (k & 1);
            kt[k] = {MK::column(lk + 32 * j * DK, at, d), MK::column(lk + (32 * j + 16) * DK, at, d)};
          }
#pragma unroll
          for (int q = NP - 1; q >= 0; --q)
#pragma unroll
            for (int k = 0; k < HELD; ++k)
#pragma unroll
              for (int c = 0; c < NC; ++c) S[k0 + k][c] = mma(kt[k], vw[c][q], S[k0 + k][c]);
          __builtin_amdgcn_sched_barrier(0);          // no more operands in flight than registers for them
        }
      }
    }
  }

  // the state behind the segment, or behind the sequence
  float* to = nullptr;
  if (FILL) to = p.seg + ((int64_t)bh * (a.segs - 1) + sg) * size;
  else if (p.s_out && (n == 0 ? sg == 0 : t0 < n && n <= t0 + a.seg)) to = p.s_out + bh * size;
  if (to) {
    const int sk = FILL ? p.seg_k : p.DV, sv = FILL ? p.seg_v : 1;
    const int dk0 = here(8 * g);
    const bool as_is = FILL || !p.reverse || n == 0;
    const Decay last = decay_of(gd, 1);
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int dk = 32 * (k / 2) + dk0 + 4 * (k & 1) + r, d = dv + 16 * c;
          if (dk < p.DK && d < p.DV)
            to[(int64_t)dk * sk + (int64_t)d * sv] = as_is ? S[k][c][r] : decayed(S[k][c][r], last, 0.f);
        }
  }
  if (FILL) return;
  // zeros behind the sequence
  const int64_t z0 = max(n, t0), z1 = min(a.L, t0 + a.seg);
  const int cols = min(DVT, p.DV - c0);
  for (int64_t i = threadIdx.x; i < (z1 - z0) * cols; i += 64 * WAVES) {
    const int64_t t = z0 + i / cols, at = ((b * a.L + t) * a.H + h) * p.DV + c0 + i % cols;
    if (OUT32) static_cast<float*>(p.out)[at] = 0.f;
    else static_cast<uint16_t*>(p.out)[at] = 0;
  }
}

// The states behind the segments one after the other: a segment's own, which
// stands in p.seg, and the state in front of it, decayed.  VEC neighbouring
// values to a thread; the loads wait for no condition (a segment without
// tokens left its slot as it was, and it stays so).
template <int VEC>
__global__ __launch_bounds__(256) void k_lin_join(LinArgs a) {
  typedef float vec __attribute__((ext_vector_type(VEC)));
  const LinPass& p = a.fill[blockIdx.y];
  const int size = p.DK * p.DV, blocks = (size / VEC + 255) / 256, slots = a.segs - 1;
  const int bh = (int)(blockIdx.x / (unsigned)blocks), i = ((int)(blockIdx.x - bh * blocks) * 256 + threadIdx.x) * VEC;
  if (i >= size) return;
  const int b = bh / a.H, h = bh - b * a.H, dk = i / p.seg_k, dv = i - dk * p.seg_k;   // seg_v is 1 where a pass fills
  float* const at = p.seg + (int64_t)bh * slots * size + i;
  constexpr int U = 8;                                // loads in flight
  vec own[U];
  const auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u) own[u] = *reinterpret_cast<const vec*>(at + (int64_t)min(s0 + u, slots - 1) * size);
  };
  load(0);
  const int64_t n = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.L) : a.L;
  const float gd = a.log_decay ? a.log_decay[h] : 0.f;
  vec s = {};
  if (p.s0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = p.s0[(int64_t)bh * size + (int64_t)dk * p.s0_k + (int64_t)(dv + e) * p.s0_v];
  }
  // tokens of the segments in front, whole ones but for the last; from a sequence's last token on, the first finds its state undecayed
  const int used = (int)min((n + a.seg - 1) / a.seg, (int64_t)slots);
  const Decay whole = decay_of(gd, a.seg), first = decay_of(gd, min(n, a.seg) - (p.reverse ? 1 : 0));
  const Decay part = decay_of(gd, n - (used - 1) * a.seg < a.seg ? n - (used - 1) * a.seg : a.seg);
  for (int s0 = 0; s0 < used; s0 += U) {
    vec now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = own[u];
    if (s0 + U < used) load(s0 + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = s0 + u;
      if (k < used) {
        const Decay d = k == 0 ? first : k == used - 1 ? part : whole;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = decayed(s[e], d, now[u][e]);
        *reinterpret_cast<vec*>(at + (int64_t)k * size) = s;
      }
    }
  }
}

// Launches: `sizes` names the heads' sizes, passes [first, first + count) of
// a.pass, or with FILL all of a.fill, share them.
template <int IOT, int DK, int WAVES, int NC, bool FILL, bool EVEN>
hipError_t launch_tiles(const LinArgs& a, int first, int count, hipStream_t s) {
  const LinPass& p = FILL ? a.fill[0] : a.pass[first];
  const int64_t tiles = (p.DV + 16 * NC * WAVES - 1) / (16 * NC * WAVES), bh = (int64_t)a.B * a.H;
  constexpr int bytes = lin_lds_bytes<IOT, DK, WAVES, NC, FILL>();
  static_assert(bytes <= 160 * 1024, "");
  const dim3 grid((unsigned)(bh * (FILL ? a.segs - 1 : a.segs) * tiles), count);
  if constexpr (FILL) {
    k_lin<IOT, DK, WAVES, NC, true, EVEN, false><<<grid, 64 * WAVES, bytes, s>>>(a, 0);
    if (const hipError_t e = hipGetLastError()) return e;
    const int vec = p.DV % 4 ? 1 : 4;
    const dim3 joins((unsigned)(bh * ((p.DK * p.DV / vec + 255) / 256)), count);
    if (vec == 4) k_lin_join<4><<<joins, 256, 0, s>>>(a);
    else k_lin_join<1><<<joins, 256, 0, s>>>(a);
  } else if (p.out_f32) {
    k_lin<IOT, DK, WAVES, NC, false, EVEN, true><<<grid, 64 * WAVES, bytes, s>>>(a, first);
  } else if constexpr (IOT == 1) {
    k_lin<IOT, DK, WAVES, NC, false, EVEN, false><<<grid, 64 * WAVES, bytes, s>>>(a, first);
  }
  return hipGetLastError();
}

// Columns of the state to a workgroup: 64 in 4 waves, or 128.  Those in 8
// waves of 16, four of which a SIMD holds, or in 4 of 32, which read the rows
// of q and k half as often but leave two to a SIMD.  bf16, 8 x 2048 tokens of 12 heads
// 64 x 128: 46 us in 8 waves, 52 in 4 (the fill 23 and 25); 65536 tokens of 6 heads
// 128 x 128: 128 in 4, 131 in 8, whose registers spill there (the fill, which
// needs fewer: 54 in 8, 59 in 4).  Heads of 129 to 256 values of k with up to 64
// of v spill 12 to 16 registers in 4 waves, which stay.
template <int IOT, bool FILL, bool EVEN>
hipError_t launch_sizes(const LinArgs& a, int first, int count, hipStream_t s) {
  const LinPass& p = FILL ? a.fill[0] : a.pass[first];
  const int dk = p.DK, dv = p.DV;
  if (dk > 128)
    return dv <= 64 ? launch_tiles<IOT, 256, 4, 1, FILL, EVEN>(a, first, count, s)
                    : launch_tiles<IOT, 256, 8, 1, FILL, EVEN>(a, first, count, s);
  if (dk > 64)
    return dv <= 64 ? launch_tiles<IOT, 128, 4, 1, FILL, EVEN>(a, first, count, s)
                    : launch_tiles<IOT, 128, FILL ? 8 : 4, FILL ? 1 : 2, FILL, EVEN>(a, first, count, s);
  return dv <= 64 ? launch_tiles<IOT, 64, 4, 1, FILL, EVEN>(a, first, count, s)
                  : launch_tiles<IOT, 64, 8, 1, FILL, EVEN>(a, first, count, s);
}

template <int IOT, bool FILL>
hipError_t launch_passes(const LinArgs& a, int first, int count, hipStream_t s) {
  bool even = true;
  for (int i = first; i < first + count; ++i) {
    const LinPass& p = FILL ? a.fill[i] : a.pass[i];
    even = even && p.DK % 8 == 0 && p.DV % 8 == 0;
    // 64 rows of them, in bytes, and a head's values fit 32 bits
    for (const HeadView* v : {&p.q, &p.k, &p.v}) even = even && v->token <= (1 << 23);
  }
  return even ? launch_sizes<IOT, FILL, true>(a, first, count, s) : launch_sizes<IOT, FILL, false>(a, first, count, s);
}

template <int IOT>
hipError_t launch(const LinArgs& a, hipStream_t s) {
  if (a.segs > 1)
    if (const hipError_t e = launch_passes<IOT, true>(a, 0, a.fills, s)) return e;
  // neighbouring passes of the same sizes go together
  for (int i = 0; i < a.passes;) {
    int n = 1;
    while (i + n < a.passes && a.pass[i + n].DK == a.pass[i].DK && a.pass[i + n].DV == a.pass[i].DV &&
           a.pass[i + n].out_f32 == a.pass[i].out_f32)
      ++n;
    if (const hipError_t e = launch_passes<IOT, false>(a, i, n, s)) return e;
    i += n;
  }
  return hipSuccess;
}

// ------------------------------------------------------------ single tokens
//
// Bound by the state's bytes, each read and written once.  A workgroup takes
// `cols` words of VEC columns of a head's state, 256 / cols threads to a word,
// which share its rows and meet in LDS for the output.
template <int IOT, int VEC>
__global__ __launch_bounds__(256) void k_lin_step(LinStepArgs a, int cols) {
  typedef float vec __attribute__((ext_vector_type(VEC)));
  __shared__ float lq[256], lk[256];
  __shared__ float part[256][VEC + 1];
  const int tid = threadIdx.x, c = tid & (cols - 1), g = tid / cols, groups = 256 / cols;
  const int tiles = (a.Dv / VEC + cols - 1) / cols, tile = (int)(blockIdx.x % (unsigned)tiles);
  const int64_t bh = blockIdx.x / (unsigned)tiles, b = bh / a.H;
  const int h = (int)(bh - b * a.H), dv = (tile * cols + c) * VEC;
  const bool live = dv < a.Dv;
  if (tid < a.Dk) {
    lq[tid] = ld1<IOT>(a.q.p, b * a.q.batch + h / a.q.share * a.q.head + tid);
    lk[tid] = ld1<IOT>(a.k.p, b * a.k.batch + h / a.k.share * a.k.head + tid);
  }
  float v[VEC], y[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    v[e] = live ? ld1<IOT>(a.v.p, b * a.v.batch + h / a.v.share * a.v.head + dv + e) : 0.f;
    y[e] = 0.f;
  }
  const Decay lam = decay_of(a.log_decay ? a.log_decay[h] : 0.f, 1);
  float* S = a.state + bh * a.Dk * a.Dv + dv;
  __syncthreads();
  if (live) {
    constexpr int U = 8;                              // rows in flight
    for (int r0 = g; r0 < a.Dk; r0 += U * groups) {
      vec s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = min(r0 + u * groups, a.Dk - 1);
        s[u] = *reinterpret_cast<const vec*>(S + (int64_t)r * a.Dv);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * groups;
        if (r < a.Dk) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            s[u][e] = decayed(s[u][e], lam, lk[r] * v[e]);
            y[e] = fmaf(lq[r], s[u][e], y[e]);
          }
          *reinterpret_cast<vec*>(S + (int64_t)r * a.Dv) = s[u];
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) part[tid][e] = y[e];
  __syncthreads();
  for (int i = tid; i < cols * VEC; i += 256) {
    const int d = tile * cols * VEC + i;
    float sum = 0.f;
    for (int j = 0; j < groups; ++j) sum += part[j * cols + i / VEC][i % VEC];
    if (d < a.Dv) st1<IOT>(a.o, bh * a.Dv + d, a.scale * sum);
  }
}

// ------------------------------------------------- sums over shared heads
template <int IOT>
__global__ __launch_bounds__(256) void k_fold(FoldArgs a) {
  const int k = blockIdx.y, D = a.D[k], share = a.share[k];
  if (!a.x[k]) return;
  const int64_t n = a.tokens * a.heads[k] * D;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t th = i / D;                         // (token, shared head)
    const float* x = a.x[k] + th * share * D + (i - th * D);
    float v = 0.f;
    for (int j = 0; j < share; ++j) v += x[(int64_t)j * D];
    st1<IOT>(a.out[k], i, v);
  }
}

}  // namespace

hipError_t linear_attention(const LinArgs& a, hipStream_t s) { return a.io ? launch<1>(a, s) : launch<0>(a, s); }

hipError_t linear_attention_step(const LinStepArgs& a, hipStream_t s) {
  const LinStepPlan p = lin_step_plan(a.Dv);
  const dim3 grid((unsigned)(p.tiles * ((int64_t)a.B * a.H)));
  if (a.io) {
    if (p.vec == 4) k_lin_step<1, 4><<<grid, 256, 0, s>>>(a, p.cols);
    else k_lin_step<1, 1><<<grid, 256, 0, s>>>(a, p.cols);
  } else {
    if (p.vec == 4) k_lin_step<0, 4><<<grid, 256, 0, s>>>(a, p.cols);
    else k_lin_step<0, 1><<<grid, 256, 0, s>>>(a, p.cols);
  }
  return hipGetLastError();
}

hipError_t fold_heads(const FoldArgs& a, hipStream_t s) {
  int64_t most = 0;
  for (int k = 0; k < 3; ++k) {
    const int64_t n = a.x[k] ? (a.tokens * a.heads[k] * a.D[k] + 255) / 256 : 0;
    if (n > most) most = n;
  }
  const dim3 grid((unsigned)(most < 8192 ? most : 8192), 3);
  if (a.io) k_fold<1><<<grid, 256, 0, s>>>(a);
  else k_fold<0><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace hyena
