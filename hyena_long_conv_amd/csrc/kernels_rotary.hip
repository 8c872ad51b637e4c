// kernels_rotary.hip -- rotary positions: pairs of a head's first R values
// turned by position * frequency, the rest copied.
//
// Bound by its bytes: every value is read and written once.  What could cost
// more are the angles.  A thread forms the sines and cosines of 8 pairs of a
// token once and turns those pairs in several heads, which share them.
#include <hip/hip_runtime.h>

#include "linattn.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

// The cosine and sine of position * freq, freq in radians.  In fp32 the
// product of a position of 2^20 would be off by 2^-4 radians; in fp64 the
// turns are off by 2^-52 of their number, and what is left of them after the
// whole ones, at most half a turn, loses 2^-25 of itself when it is rounded.
__device__ __forceinline__ void turn(double position, double freq, float scale, float sine, float& c, float& s) {
  const double turns = position * freq * 0.15915494309189535;
  float sn, cs;
  sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
  c = cs * scale;
  s = sn * scale * sine;
}

// Thread -> token, share of its heads, word: words of 8 pairs, then, out of
// place, words of 8 copied values.  Neighbours take neighbouring words, then heads.
template <int IOT, bool IL>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a, int words, int turning, int groups) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;   // a launch holds fewer than 2^32 threads
  const uint32_t rest = at / (uint32_t)words, token = rest / (uint32_t)groups;
  if (token >= a.tokens) return;
  const int w = (int)(at - rest * (uint32_t)words), h0 = (int)(rest - token * (uint32_t)groups);
  const uint32_t b32 = token / (uint32_t)a.L;
  const int64_t b = b32, t = token - b32 * (uint32_t)a.L;
  const int64_t xi = b * a.x.batch + t * a.x.token, oi = b * a.out.batch + t * a.out.token;
  const int half = a.R / 2;
  if (w >= turning) {                                 // copied values
    const int d = a.R + 8 * (w - turning), n = min(a.D - d, 8);
    for (int h = h0; h < a.H; h += groups) {
      float v[8];
      widen8<IOT>(ld8n<IOT>(a.x.p, xi + h * a.x.head + d, n, a.x.total), v);
      st8n<IOT>(const_cast<void*>(a.out.p), oi + h * a.out.head + d, v, n);
    }
    return;
  }
  const int pair = 8 * w, n = min(half - pair, 8);
  const double pos = a.positions ? (double)a.positions[b * a.pos_batch + t * a.pos_token] : (double)t;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) turn(pos, a.freq[e < n ? pair + e : pair], a.scale, a.sine, c[e], s[e]);
  // words (u, v): the pairs' first and second values, or, interleaved, 4 pairs each
  const int d0 = IL ? 2 * pair : pair, d1 = IL ? 2 * pair + 8 : pair + half;
  const int n0 = IL ? min(2 * n, 8) : n, n1 = IL ? 2 * n - 8 : n;
  for (int h = h0; h < a.H; h += groups) {
    float u[8], v[8], p[8], q[8];
    widen8<IOT>(ld8n<IOT>(a.x.p, xi + h * a.x.head + d0, n0, a.x.total), u);
    widen8<IOT>(ld8n<IOT>(a.x.p, xi + h * a.x.head + d1, n1, a.x.total), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (!IL) {
        p[e] = fmaf(u[e], c[e], -v[e] * s[e]);
        q[e] = fmaf(u[e], s[e], v[e] * c[e]);
      } else if (e < 4) {
        p[2 * e] = fmaf(u[2 * e], c[e], -u[2 * e + 1] * s[e]);
        p[2 * e + 1] = fmaf(u[2 * e], s[e], u[2 * e + 1] * c[e]);
        q[2 * e] = fmaf(v[2 * e], c[e + 4], -v[2 * e + 1] * s[e + 4]);
        q[2 * e + 1] = fmaf(v[2 * e], s[e + 4], v[2 * e + 1] * c[e + 4]);
      }
    }
    st8n<IOT>(const_cast<void*>(a.out.p), oi + h * a.out.head + d0, p, n0);
    if (n1 > 0) st8n<IOT>(const_cast<void*>(a.out.p), oi + h * a.out.head + d1, q, n1);
  }
}

}  // namespace

hipError_t rotary(const RotaryArgs& a, hipStream_t s) {
  const int turning = (int)rotary_turning(a), words = (int)rotary_words(a), groups = (int)rotary_shares(a);
  const dim3 grid((unsigned)rotary_groups(a));
  if (a.io) {
    if (a.interleaved) k_rotary<1, true><<<grid, 256, 0, s>>>(a, words, turning, groups);
    else k_rotary<1, false><<<grid, 256, 0, s>>>(a, words, turning, groups);
  } else {
    if (a.interleaved) k_rotary<0, true><<<grid, 256, 0, s>>>(a, words, turning, groups);
    else k_rotary<0, false><<<grid, 256, 0, s>>>(a, words, turning, groups);
  }
  return hipGetLastError();
}

}  // namespace hyena
