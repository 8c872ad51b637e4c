// kernels_rotary.hip -- rotary positions: pairs of a head's first R values
// turned by position * frequency, the rest copied.
//
// Bound by its bytes: every value is read and written once (8 x 2048 x 24 heads
// of 64 in bf16: 18.5 us, 5.4 TB/s, part of it from the Infinity Cache; 65536
// x 12 of 64 in fp32, half of each head turned: 84 us, 4.8 TB/s, a copy's rate;
// 104 with words of 32 bytes to a lane and the copies in a branch of their own).  What could cost
// more are the angles.  A thread forms the sines and cosines of 8 pairs (fp32: 4) of
// a token once and turns those pairs in several heads, which share them.
#include <hip/hip_runtime.h>

#include "linattn.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

// The cosine and sine of position * freq, freq in radians.  In fp32 the
// product of a position of 2^20 would be off by 2^-4 radians; in fp64 the
// turns are off by 2^-52 of their number, and what is left of them after the
// whole ones, at most half a turn, loses 2^-25 of itself when it is rounded.  The
// sines and cosines are fp32's and are rounded again with the scale: outputs in
// fp32 are off by 4.7e-8 of their norm where half of each head is turned, 3.6e-8
// with fp64's sines rounded once; in bf16 neither shows.
__device__ __forceinline__ void turn(double position, double freq, float scale, float sine, float& c, float& s) {
  const double turns = position * freq * 0.15915494309189535;
  float sn, cs;
  sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
  c = cs * scale;
  s = sn * scale * sine;
}

// A word: 16 bytes, 8 values of bf16 or 4 of fp32, so that the lanes of a load
// or a store cover whole lines.
template <int IOT> struct Word;
template <> struct Word<0> {
  static constexpr int N = 4;
  f32x4v v;
  // the first n values from element i of an array of `total`; the word is read whole where the array has it
  __device__ __forceinline__ Word(const void* p, int64_t i, int n, int64_t total) : v{0.f, 0.f, 0.f, 0.f} {
    if (n <= 0) return;
    const float* q = static_cast<const float*>(p) + i;
    if (i + N <= total) {
      v = *reinterpret_cast<const f32x4_e4*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < n) v[e] = q[e];
    }
  }
  __device__ __forceinline__ void widen(float (&o)[N]) const {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = v[e];
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&o)[N], int n) {
    float* q = static_cast<float*>(p) + i;
    if (n >= N) {
      *reinterpret_cast<f32x4_e4*>(q) = f32x4v{o[0], o[1], o[2], o[3]};
    } else {
#pragma unroll
      for (int e = 0; e < N - 1; ++e)
        if (e < n) q[e] = o[e];
    }
  }
};
template <> struct Word<1> {
  static constexpr int N = 8;
  Raw8<1> v;
  __device__ __forceinline__ Word(const void* p, int64_t i, int n, int64_t total) : v(ld8n<1>(p, i, n, total)) {}
  __device__ __forceinline__ void widen(float (&o)[N]) const { widen8<1>(v, o); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&o)[N], int n) { st8n<1>(p, i, o, n); }
};

// Thread -> token, share of its heads, place: two words of the pairs that are
// turned, then, out of place, two words of copied values.  Neighbours take
// neighbouring places, then heads.  All threads go the same way through the heads, two of them at a time,
// whether they turn or copy: the lanes of a wave that did the one would wait
// for those that do the other.
template <int IOT, bool IL>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a, int places, int turning, int groups) {
  typedef Word<IOT> W;
  constexpr int N = W::N;
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;   // a launch holds fewer than 2^32 threads
  const uint32_t rest = at / (uint32_t)places, token = rest / (uint32_t)groups;
  if (token >= a.tokens) return;
  const int w = (int)(at - rest * (uint32_t)places), h0 = (int)(rest - token * (uint32_t)groups);
  const uint32_t b32 = token / (uint32_t)a.L;
  const int64_t b = b32, t = token - b32 * (uint32_t)a.L;
  const int64_t xi = b * a.x.batch + t * a.x.token, oi = b * a.out.batch + t * a.out.token;
  const int half = a.R / 2;
  const bool turns = w < turning;
  // the words: the pairs' first and second values (interleaved: N / 2 pairs each), or copied ones
  int d0, d1, n0, n1;
  float c[N], s[N];
  if (turns) {
    const int pair = N * w, n = min(half - pair, N);
    d0 = IL ? 2 * pair : pair, d1 = IL ? 2 * pair + N : pair + half;
    n0 = IL ? min(2 * n, N) : n, n1 = IL ? 2 * n - N : n;
    const double pos = a.positions ? (double)a.positions[b * a.pos_batch + t * a.pos_token] : (double)t;
#pragma unroll
    for (int e = 0; e < N; ++e) turn(pos, a.freq[e < n ? pair + e : pair], a.scale, a.sine, c[e], s[e]);
  } else {
    d0 = a.R + 2 * N * (w - turning), d1 = d0 + N;
    n0 = min(a.D - d0, N), n1 = min(a.D - d1, N);
  }
  void* const out = const_cast<void*>(a.out.p);
  const auto head = [&](const W& ru, const W& rv, int h) {
    float u[N], v[N], p[N], q[N];
    ru.widen(u);
    rv.widen(v);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (!IL) {
        p[e] = fmaf(u[e], c[e], -v[e] * s[e]);
        q[e] = fmaf(u[e], s[e], v[e] * c[e]);
      } else if (e < N / 2) {
        p[2 * e] = fmaf(u[2 * e], c[e], -u[2 * e + 1] * s[e]);
        p[2 * e + 1] = fmaf(u[2 * e], s[e], u[2 * e + 1] * c[e]);
        q[2 * e] = fmaf(v[2 * e], c[e + N / 2], -v[2 * e + 1] * s[e + N / 2]);
        q[2 * e + 1] = fmaf(v[2 * e], s[e + N / 2], v[2 * e + 1] * c[e + N / 2]);
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = turns ? p[e] : u[e], q[e] = turns ? q[e] : v[e];
    W::store(out, oi + h * a.out.head + d0, p, n0);
    if (n1 > 0) W::store(out, oi + h * a.out.head + d1, q, n1);
  };
  const auto first = [&](int h) { return W(a.x.p, xi + h * a.x.head + d0, n0, a.x.total); };
  const auto second = [&](int h) { return W(a.x.p, xi + h * a.x.head + d1, n1, a.x.total); };
  int h = h0;
  for (; h + groups < a.H; h += 2 * groups) {
    const W u0 = first(h), v0 = second(h), u1 = first(h + groups), v1 = second(h + groups);
    head(u0, v0, h);
    head(u1, v1, h + groups);
  }
  if (h < a.H) {
    const W u0 = first(h), v0 = second(h);
    head(u0, v0, h);
  }
}

}  // namespace

hipError_t rotary(const RotaryArgs& a, hipStream_t s) {
  const int turning = (int)rotary_turning(a), places = (int)rotary_places(a), groups = (int)rotary_shares(a);
  const dim3 grid((unsigned)rotary_groups(a));
  if (a.io) {
    if (a.interleaved) k_rotary<1, true><<<grid, 256, 0, s>>>(a, places, turning, groups);
    else k_rotary<1, false><<<grid, 256, 0, s>>>(a, places, turning, groups);
  } else {
    if (a.interleaved) k_rotary<0, true><<<grid, 256, 0, s>>>(a, places, turning, groups);
    else k_rotary<0, false><<<grid, 256, 0, s>>>(a, places, turning, groups);
  }
  return hipGetLastError();
}

}  // namespace hyena
