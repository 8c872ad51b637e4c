// kernels_linattn.hip -- linear attention with a decay for each head: passes
// over whole sequences, single tokens, and sums over shared heads.
//
//   S[t] = lambda S[t-1] + su k[t] v[t]^T,  out[t] = so S[t]^T q[t].
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

// lambda^n with g2 = log2(e) log_decay
__device__ __forceinline__ float power_of(float g2, int n) { return n == 0 ? 1.f : exp2_fast(g2 * (float)n); }

// -------------------------------------------------- passes over sequences
//
// A workgroup of 4 waves walks over a sequence (or a segment of it) in blocks
// of C tokens and keeps DVT columns of a head's state, 16 NC for each wave, in
// the accumulators of its matrix instructions.  For a block with the state S
// in front of it, weights W = tril(lambda^(i-j)) and the rows k, q, v in LDS:
//   P   = so su W * (q k^T)                     shared out by tiles of 16 x 16,
//   out = so lambda^(i+1) (q S) + P v,
//   S   = lambda^C S + k^T (su lambda^(C-1-j) v).
// All products are formed transposed, with the state's and P's accumulators
// as operands of the next product as they lie: lane l of group g = l / 16
// holds rows 4 g .. 4 g + 3 of a tile's column l % 16, and two tiles make the
// 8 values of k that an operand holds for its row or column, in the order
// 4 g .. 4 g + 3, 16 + 4 g .. 16 + 4 g + 3, in which the other operand is read.
// So the state never goes through LDS, and P does once, lane by lane.

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

// Rows of LDS hold D values and a gap that keeps the reads below on all banks:
// 8 rows of 32 bytes (bf16, transposed), 4 rows of 64 (fp32, transposed).
template <int IOT> struct Lds;
template <> struct Lds<0> {
  typedef float T;
  static constexpr int GAP = 4;
  static __device__ __forceinline__ f32x4v four(const float* p) { return *reinterpret_cast<const f32x4v*>(p); }
  // values of four rows at one column: lane l of its 16 gets column l
  static __device__ __forceinline__ f32x4v four_rows(const float* p, int stride, int l) {
    p += l;
    return f32x4v{p[0], p[stride], p[2 * stride], p[3 * stride]};
  }
  static __device__ __forceinline__ f32x4v narrow(f32x4v v) { return v; }
  static __device__ __forceinline__ float one(float v) { return v; }
};
template <> struct Lds<1> {
  typedef uint16_t T;
  static constexpr int GAP = 16;
  static __device__ __forceinline__ u32x2v four(const uint16_t* p) { return *reinterpret_cast<const u32x2v*>(p); }
  // the transposing read: lane l gives the address of row l / 4, columns 4 (l % 4), and gets column l
  static __device__ __forceinline__ u32x2v four_rows(const uint16_t* p, int stride, int l) {
    const uint16_t* at = p + (l >> 2) * stride + 4 * (l & 3);
    return __builtin_bit_cast(u32x2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at));
  }
  static __device__ __forceinline__ u32x2v narrow(f32x4v v) { return u32x2v{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])}; }
  static __device__ __forceinline__ float one(uint16_t v) { return bf16_bits_to_f32(v); }
};

__device__ __forceinline__ f32x4v widen4(f32x4v v) { return v; }
__device__ __forceinline__ f32x4v widen4(u32x2v v) {
  return f32x4v{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
                __uint_as_float(v[1] & 0xffff0000u)};
}

// The state's addends are products in fp32 of bf16 values and fp32 weights.
// As matrix operands they go in three bf16 parts, 2^-24 of them left: with two
// the state would be off by 2.7e-6 of its norm, with one by 1.7e-3.
template <int IOT> constexpr int kParts = IOT == 1 ? 3 : 1;
__device__ __forceinline__ void parts_of(f32x4v a, f32x4v b, Frag<0> (&o)[1]) { o[0] = {a, b}; }
__device__ __forceinline__ void parts_of(f32x4v a, f32x4v b, Frag<1> (&o)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    o[k] = {Lds<1>::narrow(a), Lds<1>::narrow(b)};
    if (k < 2) a -= widen4(o[k].a), b -= widen4(o[k].b);
  }
}

// A block's rows of one operand on their way from global memory to LDS: W
// words of 8 values to a row, NW words to a thread, in one column of words.
template <int IOT, int C, int D>
struct Rows {
  static constexpr int W = D / 8, NW = C * W / 256, STEP = 256 / W, STRIDE = D + Lds<IOT>::GAP;
  static_assert(NW >= 1 && NW * 256 == C * W, "whole words for each thread");
  Raw8<IOT> word[NW];
  const char* base;      // the head's first value of the sequence
  int64_t first, step;   // elements to the walk's first token, and from one token to the next
  int64_t total;         // elements behind base
  int d, row, col;
  bool live;
  __device__ __forceinline__ void init(const HeadView& v, int64_t b, int h, int d_, int64_t n, bool reverse) {
    constexpr int E = IOT == 0 ? 4 : 2;
    const int64_t at = b * v.batch + h / v.share * v.head;
    base = static_cast<const char*>(v.p) + at * E;
    total = v.total - at;
    first = reverse ? (n - 1) * v.token : 0;
    step = reverse ? -v.token : v.token;
    d = d_;
    row = threadIdx.x / W;
    col = 8 * (threadIdx.x % W);
    live = col < d;
  }
  // The block at token t0 of the walk, zeros from token `end` on.
  __device__ __forceinline__ void load(int64_t t0, int64_t end) {
    if (t0 + C <= end && d % 8 == 0) {
      const int64_t at = first + (t0 + row) * step + (live ? col : 0);
#pragma unroll
      for (int m = 0; m < NW; ++m) word[m] = ld8<IOT>(base, at + m * STEP * step);
    } else {
#pragma unroll
      for (int m = 0; m < NW; ++m) {
        const int64_t t = t0 + row + m * STEP;
        word[m] = ld8n<IOT>(base, t < end ? first + t * step + col : 0, t < end ? d - col : 0, total);
      }
    }
  }
  __device__ __forceinline__ void store(typename Lds<IOT>::T* lds) const {
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      const Raw8<IOT> w = live ? word[m] : zero8<IOT>();
      auto* to = lds + (row + m * STEP) * STRIDE + col;
      if constexpr (IOT == 0) {
        *reinterpret_cast<f32x4v*>(to) = w.a;
        *reinterpret_cast<f32x4v*>(to + 4) = w.b;
      } else {
        *reinterpret_cast<u32x4v*>(to) = w.a;
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
      const u32x2v w = Lds<1>::narrow(v);
      *reinterpret_cast<u2*>(static_cast<uint16_t*>(p) + i) = u2{w[0], w[1]};
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) st1<IOT>(p, i + e, v[e]);
}

template <int IOT> constexpr int kBlock = IOT == 1 ? 64 : 32;   // tokens of a block

template <int IOT, int DK, int NC, bool FILL>
constexpr int lin_lds_bytes() {
  constexpr int C = kBlock<IOT>, E = sizeof(typename Lds<IOT>::T), G = Lds<IOT>::GAP;
  return (C * ((FILL ? 1 : 2) * (DK + G) + 64 * NC + G) + (FILL ? 0 : C * C)) * E;
}

// FILL: the state behind a segment alone, from nothing, for all but the last segment.
template <int IOT, int DK, int NC, bool FILL>
__global__ __launch_bounds__(256, 2) void k_lin(LinArgs a, int first_pass) {
  typedef typename Lds<IOT>::T T;
  constexpr int C = kBlock<IOT>, IT = C / 16, JJ = C / 32, KT = DK / 16, DVT = 64 * NC, NP = kParts<IOT>;
  const LinPass& p = a.pass[first_pass + blockIdx.y];
  if (FILL && !p.seg_fills) return;
  extern __shared__ __attribute__((aligned(16))) unsigned char shared[];
  T* const lk = reinterpret_cast<T*>(shared);
  T* const lv = lk + C * Rows<IOT, C, DK>::STRIDE;
  T* const lq = lv + C * Rows<IOT, C, DVT>::STRIDE;
  T* const lp = lq + C * Rows<IOT, C, DK>::STRIDE;   // tiles (i, j) of 16 x 16 at i IT + j, 4 values to a lane
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15, g = lane >> 4;

  const int tiles = (p.DV + DVT - 1) / DVT, segs = FILL ? a.segs - 1 : a.segs;
  const int tile = (int)(blockIdx.x % (unsigned)tiles), rest = (int)(blockIdx.x / (unsigned)tiles);
  const int bh = rest / segs, sg = rest - bh * segs, b = bh / a.H, h = bh - b * a.H, c0 = tile * DVT;
  const int64_t n = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.L) : a.L;
  const int64_t t0 = sg * a.seg, end = min(n, t0 + a.seg), size = (int64_t)p.DK * p.DV;
  const float gd = a.log_decay ? a.log_decay[h] : 0.f, g2 = gd * kLog2e;
  if (FILL && t0 >= n) return;

  // the state: rows 16 kt + 4 g + r, column 16 (NC wave + c) + l of the tile
  const int mine = c0 + 16 * NC * wave;
  f32x4v S[KT][NC];
  {
    const float* s0 = nullptr;
    int sk = 0, sv = 0;
    if (!FILL) {
      if (sg > 0) s0 = p.seg + ((int64_t)bh * (a.segs - 1) + sg - 1) * size, sk = p.seg_k, sv = p.seg_v;
      else if (p.s0) s0 = p.s0 + bh * size, sk = p.s0_k, sv = p.s0_v;
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int dk = 16 * kt + 4 * g + r, dv = mine + 16 * c + l;
          S[kt][c][r] = s0 && t0 < max(n, (int64_t)1) && dk < p.DK && dv < p.DV ? s0[(int64_t)dk * sk + (int64_t)dv * sv] : 0.f;
        }
  }

  if (t0 < end) {
    Rows<IOT, C, DK> rk, rq;
    Rows<IOT, C, DVT> rv;
    rk.init(p.k, b, h, p.DK, n, p.reverse);
    rv.init(p.v, b, h, p.DV, n, p.reverse);
    // this workgroup's columns of v
    rv.base += (int64_t)c0 * sizeof(T);
    rv.total -= c0;
    rv.d -= c0;
    rv.live = rv.col < rv.d;
    rk.load(t0, end);
    rv.load(t0, end);
    if (!FILL) {
      rq.init(p.q, b, h, p.DK, n, p.reverse);
      rq.load(t0, end);
    }
    // what depends on the tokens of a block and on whether the state decays before its first one
    float weight[JJ][8], through[IT];
    Decay whole{0.f, 1.f};
    auto powers = [&](int count, int lead) {
#pragma unroll
      for (int j = 0; j < JJ; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int left = count - 1 - (32 * j + 16 * (e >> 2) + 4 * g + (e & 3));
          weight[j][e] = left >= 0 ? p.su * power_of(g2, left) : 0.f;
        }
#pragma unroll
      for (int i = 0; i < IT; ++i) through[i] = p.so * power_of(g2, 16 * i + l + lead);
      whole = decay_of(gd, count - 1 + lead);
    };
    // P's tiles of this wave: number wave, wave + 4, .. of those on and below the diagonal
    constexpr int TILES = IT * (IT + 1) / 2, MINE = (TILES + 3) / 4;
    auto tile_at = [](int k, int& i, int& j) {
      i = k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3;
      j = k - i * (i + 1) / 2;
    };
    float pair[MINE][4];
    if (!FILL) {
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        int i, j;
        tile_at(wave + 4 * m, i, j);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int apart = 16 * (i - j) + l - 4 * g - r;
          pair[m][r] = apart >= 0 ? p.so * p.su * power_of(g2, apart) : 0.f;
        }
      }
    }
    int lead = p.reverse && sg == 0 ? 0 : 1, count = 0;
    for (int64_t t = t0; t < end; t += C) {
      const int now = (int)min(end - t, (int64_t)C);
      if (now != count || t <= t0 + C) {
        count = now;
        powers(count, t == t0 ? lead : 1);
      }
      __syncthreads();                                // the block before has been read
      rk.store(lk);
      rv.store(lv);
      if (!FILL) rq.store(lq);
      __syncthreads();
      if (t + C < end) {
        rk.load(t + C, end);
        rv.load(t + C, end);
        if (!FILL) rq.load(t + C, end);
      }
      if constexpr (!FILL) {
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
          const int k = wave + 4 * m;
          if (k >= TILES) break;
          int i, j;
          tile_at(k, i, j);
          f32x4v acc = {0.f, 0.f, 0.f, 0.f};
          const T* kr = lk + (16 * j + l) * (DK + Lds<IOT>::GAP) + 4 * g;
          const T* qr = lq + (16 * i + l) * (DK + Lds<IOT>::GAP) + 4 * g;
#pragma unroll
          for (int kk = 0; kk < DK / 32; ++kk)
            acc = mma(Frag<IOT>{Lds<IOT>::four(kr + 32 * kk), Lds<IOT>::four(kr + 32 * kk + 16)},
                      Frag<IOT>{Lds<IOT>::four(qr + 32 * kk), Lds<IOT>::four(qr + 32 * kk + 16)}, acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] = 16 * (i - j) + l >= 4 * g + r ? acc[r] * pair[m][r] : 0.f;
          // bf16: a pair's weight is rounded once, as an output is
          const auto w = Lds<IOT>::narrow(acc);
          *reinterpret_cast<decltype(Lds<IOT>::narrow(acc))*>(lp + ((i * IT + j) * 64 + lane) * 4) = w;
        }
        __syncthreads();
      }
      // v transposed: columns of this wave, 8 tokens to a lane
      Frag<IOT> vt[JJ][NC];
#pragma unroll
      for (int j = 0; j < JJ; ++j)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const T* at = lv + (32 * j + 4 * g) * Rows<IOT, C, DVT>::STRIDE + 16 * (NC * wave + c);
          vt[j][c] = {Lds<IOT>::four_rows(at, Rows<IOT, C, DVT>::STRIDE, l),
                      Lds<IOT>::four_rows(at + 16 * Rows<IOT, C, DVT>::STRIDE, Rows<IOT, C, DVT>::STRIDE, l)};
        }
      if constexpr (!FILL) {
        // bf16: the state is rounded once for its product with q, and stays fp32
        Frag<IOT> sf[KT / 2][NC];
#pragma unroll
        for (int k = 0; k < KT / 2; ++k)
#pragma unroll
          for (int c = 0; c < NC; ++c) sf[k][c] = {Lds<IOT>::narrow(S[2 * k][c]), Lds<IOT>::narrow(S[2 * k + 1][c])};
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          if (16 * i >= count) break;
          f32x4v acc[NC];
          // A value that is not finite meets the zeros of P above the diagonal; where an output shows one, the
          // tile is formed again with the diagonal's products one by one (`careful`), so that it reaches no earlier token.
          for (bool careful = false;; careful = true) {
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c] = f32x4v{0.f, 0.f, 0.f, 0.f};
            const T* qr = lq + (16 * i + l) * (DK + Lds<IOT>::GAP) + 4 * g;
#pragma unroll
            for (int k = 0; k < KT / 2; ++k) {
              const Frag<IOT> qf{Lds<IOT>::four(qr + 32 * k), Lds<IOT>::four(qr + 32 * k + 16)};
#pragma unroll
              for (int c = 0; c < NC; ++c) acc[c] = mma(sf[k][c], qf, acc[c]);
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c] *= through[i];
            const T* pt = lp + (i * IT * 64 + lane) * 4;
#pragma unroll
            for (int j = 0; j < JJ; ++j) {
              if (2 * j > i) break;
              Frag<IOT> pf{Lds<IOT>::four(pt + 2 * j * 256), {}}, zero{};
              if (2 * j + 1 <= i) pf.b = Lds<IOT>::four(pt + (2 * j + 1) * 256);
              else pf.b = zero.b;
              if (careful) {
                if (2 * j == i) continue;
                if (2 * j + 1 == i) pf.b = zero.b;
              }
#pragma unroll
              for (int c = 0; c < NC; ++c)
                acc[c] = mma(careful && 2 * j + 1 == i ? Frag<IOT>{vt[j][c].a, zero.b} : vt[j][c], pf, acc[c]);
            }
            if (careful) {
              for (int j = 0; j < 16; ++j) {
                const float w = Lds<IOT>::one(lp[((i * IT + i) * 64 + (j >> 2) * 16 + l) * 4 + (j & 3)]);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    const float v = Lds<IOT>::one(lv[(16 * i + j) * Rows<IOT, C, DVT>::STRIDE + 16 * (NC * wave + c) + 4 * g + r]);
                    acc[c][r] = j <= l ? fmaf(w, v, acc[c][r]) : acc[c][r];
                  }
              }
              break;
            }
            float bad = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
              for (int r = 0; r < 4; ++r) bad = fmaf(acc[c][r], 0.f, bad);
            if (!__any(bad != 0.f)) break;
          }
          const int64_t to = t + 16 * i + l;
          if (16 * i + l < count) {
            const int64_t at = ((b * a.L + (p.reverse ? n - 1 - to : to)) * a.H + h) * p.DV;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int dv = mine + 16 * c + 4 * g;
              if (p.out_f32) st4n<0>(p.out, at + dv, acc[c], p.DV - dv);
              else st4n<1>(p.out, at + dv, acc[c], p.DV - dv);
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[k][c][r] = decayed(S[k][c][r], whole, 0.f);
#pragma unroll
      for (int j = 0; j < JJ; ++j) {
        Frag<IOT> vw[NC][NP];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          f32x4v x = widen4(vt[j][c].a), y = widen4(vt[j][c].b);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= weight[j][e], y[e] *= weight[j][4 + e];
          parts_of(x, y, vw[c]);
        }
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const T* at = lk + (32 * j + 4 * g) * (DK + Lds<IOT>::GAP) + 16 * k;
          const Frag<IOT> kt{Lds<IOT>::four_rows(at, DK + Lds<IOT>::GAP, l),
                             Lds<IOT>::four_rows(at + 16 * (DK + Lds<IOT>::GAP), DK + Lds<IOT>::GAP, l)};
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int q = NP - 1; q >= 0; --q) S[k][c] = mma(kt, vw[c][q], S[k][c]);
        }
      }
    }
  }

  // the state behind the segment, or behind the sequence
  float* to = nullptr;
  if (FILL) {
    to = p.seg + ((int64_t)bh * (a.segs - 1) + sg) * size;
  } else if (p.s_out && (n == 0 ? sg == 0 : t0 < n && n <= t0 + a.seg)) {
    to = p.s_out + bh * size;
  }
  if (to) {
    const int sk = FILL ? p.seg_k : p.DV, sv = FILL ? p.seg_v : 1;
    const bool as_is = FILL || !p.reverse || n == 0;
    const Decay last = decay_of(gd, 1);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int dk = 16 * kt + 4 * g + r, dv = mine + 16 * c + l;
          if (dk < p.DK && dv < p.DV)
            to[(int64_t)dk * sk + (int64_t)dv * sv] = as_is ? S[kt][c][r] : decayed(S[kt][c][r], last, 0.f);
        }
  }
  if (FILL) return;
  // zeros behind the sequence
  const int64_t z0 = max(n, t0), z1 = min(a.L, t0 + a.seg);
  const int cols = min(DVT, p.DV - c0);
  for (int64_t i = threadIdx.x; i < (z1 - z0) * cols; i += 256) {
    const int64_t t = z0 + i / cols, at = ((b * a.L + t) * a.H + h) * p.DV + c0 + i % cols;
    if (p.out_f32) static_cast<float*>(p.out)[at] = 0.f;
    else static_cast<uint16_t*>(p.out)[at] = 0;
  }
}

// The states behind the segments one after the other: a segment's own, which
// stands in p.seg, and the state in front of it, decayed.
__global__ __launch_bounds__(256) void k_lin_join(LinArgs a, int first_pass) {
  const LinPass& p = a.pass[first_pass + blockIdx.y];
  if (!p.seg_fills) return;
  const int size = p.DK * p.DV, blocks = (size + 255) / 256;
  const int bh = (int)(blockIdx.x / (unsigned)blocks), i = (int)(blockIdx.x - bh * blocks) * 256 + threadIdx.x;
  if (i >= size) return;
  const int b = bh / a.H, h = bh - b * a.H, dk = i / p.seg_k, dv = i - dk * p.seg_k;   // seg_v is 1 where a pass fills
  const int64_t n = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.L) : a.L;
  const float gd = a.log_decay ? a.log_decay[h] : 0.f;
  float s = p.s0 ? p.s0[(int64_t)bh * size + (int64_t)dk * p.s0_k + (int64_t)dv * p.s0_v] : 0.f;
  float* at = p.seg + (int64_t)bh * (a.segs - 1) * size + i;
  const Decay whole = decay_of(gd, a.seg);
  constexpr int U = 8;                                // loads in flight
  for (int s0 = 0; s0 < a.segs - 1; s0 += U) {
    float own[U];
#pragma unroll
    for (int u = 0; u < U; ++u) own[u] = s0 + u < a.segs - 1 && (s0 + u) * a.seg < n ? at[(int64_t)(s0 + u) * size] : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t have = n - (s0 + u) * a.seg;
      if (s0 + u >= a.segs - 1 || have <= 0) continue;
      const bool full = have >= a.seg && (s0 + u > 0 || !p.reverse);
      s = decayed(s, full ? whole : decay_of(gd, min(have, a.seg) - (p.reverse && s0 + u == 0 ? 1 : 0)), own[u]);
      at[(int64_t)(s0 + u) * size] = s;
    }
  }
}

// One launch for passes [first, first + count), which share their sizes.
template <int IOT, int DK, int NC>
hipError_t launch_tiles(const LinArgs& a, int first, int count, hipStream_t s) {
  const LinPass& p = a.pass[first];
  const int64_t tiles = (p.DV + 64 * NC - 1) / (64 * NC), bh = (int64_t)a.B * a.H;
  bool fills = false;
  for (int i = first; i < first + count; ++i) fills = fills || a.pass[i].seg_fills;
  hipError_t e;
  if (a.segs > 1 && fills) {
    constexpr int bytes = lin_lds_bytes<IOT, DK, NC, true>();
    static_assert(bytes <= 160 * 1024, "");
    k_lin<IOT, DK, NC, true><<<dim3((unsigned)(bh * (a.segs - 1) * tiles), count), 256, bytes, s>>>(a, first);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t blocks = (p.DK * p.DV + 255) / 256;
    k_lin_join<<<dim3((unsigned)(bh * blocks), count), 256, 0, s>>>(a, first);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  constexpr int bytes = lin_lds_bytes<IOT, DK, NC, false>();
  static_assert(bytes <= 160 * 1024, "");
  k_lin<IOT, DK, NC, false><<<dim3((unsigned)(bh * a.segs * tiles), count), 256, bytes, s>>>(a, first);
  return hipGetLastError();
}

template <int IOT>
hipError_t launch_pass(const LinArgs& a, int first, int count, hipStream_t s) {
  const int dk = a.pass[first].DK, dv = a.pass[first].DV;
  if (dk > 128) return launch_tiles<IOT, 256, 1>(a, first, count, s);
  if (dk > 64) return dv > 64 ? launch_tiles<IOT, 128, 2>(a, first, count, s) : launch_tiles<IOT, 128, 1>(a, first, count, s);
  return dv > 64 ? launch_tiles<IOT, 64, 2>(a, first, count, s) : launch_tiles<IOT, 64, 1>(a, first, count, s);
}

template <int IOT>
hipError_t launch(const LinArgs& a, hipStream_t s) {
  if (a.passes == 1) return launch_pass<IOT>(a, 0, 1, s);
  // gv's states behind the segments are gk's too
  if (const hipError_t e = launch_pass<IOT>(a, 2, 1, s)) return e;
  return launch_pass<IOT>(a, 0, 2, s);
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
  const int vec = a.Dv % 4 ? 1 : 4, words = a.Dv / vec;
  int cols = 1;
  while (cols < words && cols < 64) cols *= 2;
  const dim3 grid((unsigned)((words + cols - 1) / cols * ((int64_t)a.B * a.H)));
  if (a.io) {
    if (vec == 4) k_lin_step<1, 4><<<grid, 256, 0, s>>>(a, cols);
    else k_lin_step<1, 1><<<grid, 256, 0, s>>>(a, cols);
  } else {
    if (vec == 4) k_lin_step<0, 4><<<grid, 256, 0, s>>>(a, cols);
    else k_lin_step<0, 1><<<grid, 256, 0, s>>>(a, cols);
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
