// kernels_conv.hip -- the short causal depthwise convolution as an operator
// of its own, forward, for single tokens, and backward.
//
//   p[t] = bias + sum_{j<T} w[j] x[t-j],   y = p  or  p * sigmoid(p)
//
// per channel; x[-1], x[-2], .. come from a carried state (zeros without
// one), and the last T-1 inputs are what the next call carries.  Taps are
// rounded up to TT = 4, 8 or 16 in the registers.  A thread holds 8
// consecutive outputs of a row and reads the TT values before them again,
// from the cache that its neighbours' loads have filled.  The taps behind T are
// passed over, not multiplied by zero: an infinity or NaN there is not theirs.
// The condition is the same for all lanes.  8 x 1536 x 2048 bf16,
// 4 taps, with silu: 20.4 us, 4.9 TB/s of x and y, a copy's rate; the vector
// units are busy 95% of that time (the sigmoid is a third of it), so the two
// bounds meet here.
#include <hip/hip_runtime.h>

#include "ssm.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

__device__ __forceinline__ int conv_length(const ConvArgs& a, int64_t b) {
  if (!a.lengths) return (int)a.L;
  const int n = a.lengths[b];
  return n < 0 ? 0 : (n > a.L ? (int)a.L : n);
}

// The input at t of row r, from the state before the row's start.
template <int IOT>
__device__ __forceinline__ float conv_at(const ConvArgs& a, int64_t r, int64_t t) {
  if (t >= 0) return ld1<IOT>(a.x, r * a.L + t);
  const int64_t i = t + a.T - 1;
  return a.state && i >= 0 ? ld1<IOT>(a.state, r * (a.T - 1) + i) : 0.f;
}

// v = inputs t .. t+7 of row r (t a multiple of 8, possibly negative; zeros from len on).
template <int IOT>
__device__ __forceinline__ void conv_word(const ConvArgs& a, int64_t r, int t, int len, float (&v)[8]) {
  if (t >= 0) {
    widen8<IOT>(ld8n<IOT>(a.x, r * a.L + t, len - t, (int64_t)a.B * a.D * a.L), v);
  } else {
    const int S = a.T - 1, i = t + S;                 // the state's place of v[0]
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = a.state && i + e >= 0 ? ld1<IOT>(a.state, r * S + i + e) : 0.f;
  }
}

// x = the H inputs before t, then those of t .. t + N - 1 (H, N multiples of 4).
template <int IOT, int H, int N>
__device__ __forceinline__ void conv_window(const ConvArgs& a, int64_t r, int t, int len, float (&x)[H + N]) {
  float v[8];
  if (t >= (H + 7) / 8 * 8 && t + (N + 7) / 8 * 8 <= len) {           // nothing to mask: most lanes
    const int64_t i = r * a.L + t;
#pragma unroll
    for (int k = 0; k < (H + 7) / 8; ++k) {
      widen8<IOT>(ld8<IOT>(a.x, i - 8 * (k + 1)), v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (H - 8 * (k + 1) + e >= 0) x[H - 8 * (k + 1) + e] = v[e];
    }
#pragma unroll
    for (int k = 0; k < (N + 7) / 8; ++k) {
      widen8<IOT>(ld8<IOT>(a.x, i + 8 * k), v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * k + e < N) x[H + 8 * k + e] = v[e];
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < (H + 7) / 8; ++k) {
    conv_word<IOT>(a, r, t - 8 * (k + 1), len, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (H - 8 * (k + 1) + e >= 0) x[H - 8 * (k + 1) + e] = v[e];
  }
#pragma unroll
  for (int k = 0; k < (N + 7) / 8; ++k) {
    conv_word<IOT>(a, r, t + 8 * k, len, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * k + e < N) x[H + 8 * k + e] = v[e];
  }
}

template <int TT>
__device__ __forceinline__ void conv_taps(const ConvArgs& a, int d, float (&w)[TT]) {
#pragma unroll
  for (int j = 0; j < TT; ++j) w[j] = j < a.T ? a.w[(int64_t)d * a.T + j] : 0.f;
}

template <int IOT, int TT>
__global__ __launch_bounds__(256) void k_conv(ConvArgs a, int per, int lper, int blocks) {
  const int tid = threadIdx.x;
  const uint32_t rb = blockIdx.x / (uint32_t)blocks;
  const int xb = (int)(blockIdx.x - rb * blocks);
  const int64_t r = (int64_t)rb * (256 >> lper) + (tid >> lper);
  if (r >= (int64_t)a.B * a.D) return;
  const uint32_t b = (uint32_t)r / (uint32_t)a.D;     // rows are at most 2^30
  const int d = (int)((uint32_t)r - b * (uint32_t)a.D), len = conv_length(a, b);
  const int i = xb * per + (tid & (per - 1)), t = 8 * i;
  if (a.state_out)
    for (int k = i; k < a.T - 1; k += blocks * per)
      st1<IOT>(a.state_out, r * (a.T - 1) + k, conv_at<IOT>(a, r, (int64_t)len - (a.T - 1) + k));
  if (t >= a.L) return;
  float x[TT + 8], w[TT], y[8];
  conv_taps<TT>(a, d, w);
  if (t < len) {
    conv_window<IOT, TT, 8>(a, r, t, len, x);
    const float bias = a.bias ? a.bias[d] : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = bias;
#pragma unroll
    for (int j = 0; j < TT; ++j)
      if (j < a.T) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(w[j], x[TT + e - j], y[e]);
      }
    if (a.silu) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= sigmoid_f(y[e]);
    }
    if (t + 8 > len) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = t + e < len ? y[e] : 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.f;
  }
  st8n<IOT>(a.y, r * a.L + t, y, (int)min(a.L - t, (int64_t)8));
}

// One token for each of B sequences: a thread to a channel; 16 x 1536 take 2.9
// us, a launch.  (The state's values are loaded one after the other, each
// under its tap's condition.)
template <int IOT, int TT>
__global__ __launch_bounds__(256) void k_conv_step(ConvArgs a) {
  const int64_t r = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (r >= (int64_t)a.B * a.D) return;
  const int d = (int)((uint32_t)r % (uint32_t)a.D), S = a.T - 1;
  float w[TT], x[TT];
  conv_taps<TT>(a, d, w);
  x[0] = ld1<IOT>(a.x, r);
#pragma unroll
  for (int j = 1; j < TT; ++j) x[j] = j <= S ? ld1<IOT>(a.state_out, r * S + S - j) : 0.f;
  float p = a.bias ? a.bias[d] : 0.f;
#pragma unroll
  for (int j = 0; j < TT; ++j) p = fmaf(w[j], x[j], p);
  st1<IOT>(a.y, r, a.silu ? p * sigmoid_f(p) : p);
#pragma unroll
  for (int j = 0; j < TT - 1; ++j)
    if (j < S) st1<IOT>(a.state_out, r * S + S - 1 - j, x[j]);
}

// Backward.  With gp = gy act'(p),
//   gx[t] = sum_j w[j] gp[t+j],  gw[j] = sum_t gp[t] x[t-j],  gbias = sum_t gp[t],
// and the carried inputs' gradients are gx at negative t; a gradient of the
// state that the call left behind adds to the last T-1 inputs'.  p is
// computed again, for a lane's 8 steps and the TT-1 behind them.  A workgroup
// sums over its sequences and steps in registers and leaves one partial for
// each tap, which k_conv_sum adds up in a fixed order.  8 x 1536 x 2048 bf16:
// 38 us and 4 for the sums, vector units 88% busy (a p, a sigmoid and a
// derivative for 19 steps of 16, the sums over taps twice); 31 us at a copy's
// rate.
template <int IOT, int TT, int E, bool EXACT>
__device__ __forceinline__ void conv_gp(const ConvArgs& a, int64_t r, int t, int len, const float (&w)[TT], float bias,
                                        float (&x)[2 * TT + E], float (&gp)[TT + E]) {
  conv_window<IOT, TT, TT + E>(a, r, t, len, x);
  const bool whole = t >= 0 && t + (TT + E + 7) / 8 * 8 <= len;
#pragma unroll
  for (int k = 0; k < (TT + E + 7) / 8; ++k) {
    float v[8];
    const int64_t i = r * a.L + t + 8 * k;
    widen8<IOT>(whole ? ld8<IOT>(a.gy, i) : ld8n<IOT>(a.gy, i, t + 8 * k < 0 ? 0 : len - t - 8 * k, (int64_t)a.B * a.D * a.L), v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * k + e < TT + E) gp[8 * k + e] = v[e];
  }
  if (a.silu) {
    float p[TT + E - 1];
#pragma unroll
    for (int e = 0; e < TT + E - 1; ++e) p[e] = bias;
#pragma unroll
    for (int j = 0; j < TT; ++j)
      if (EXACT || j < a.T) {
#pragma unroll
        for (int e = 0; e < TT + E - 1; ++e) p[e] = fmaf(w[j], x[TT + e - j], p[e]);
      }
#pragma unroll
    for (int e = 0; e < TT + E - 1; ++e) {
      const float s = sigmoid_f(p[e]);
      gp[e] *= s * fmaf(p[e], 1.f - s, 1.f);             // 0 before 0 and from len on
    }
  }
}

// EXACT: T = TT, and no condition at each tap (8 x 1536 x 2048 bf16: 16 taps
// 104 us, 13 taps, which need the conditions, 126; no difference with up to 8).
template <int IOT, int TT, bool EXACT>
__global__ __launch_bounds__(256) void k_conv_bwd(ConvArgs a, ConvBackwardGrid g) {
  constexpr int E = conv_each(TT);
  __shared__ float part[4][TT + 1];
  const int tid = threadIdx.x, per = g.per, at_once = 256 >> g.lper, S = a.T - 1;
  const uint32_t id = blockIdx.x / (uint32_t)a.D, grp = id / (uint32_t)g.blocks, xb = id - grp * (uint32_t)g.blocks;
  const int d = (int)(blockIdx.x - id * (uint32_t)a.D);
  float w[TT], sum[TT + 1];
  conv_taps<TT>(a, d, w);
  const float bias = a.bias ? a.bias[d] : 0.f;
#pragma unroll
  for (int j = 0; j <= TT; ++j) sum[j] = 0.f;
  const int t_end = (int)min(a.L, (xb + 1) * kConvSpan), b_end = (int)min((int64_t)a.B, (grp + 1) * g.seqs);
  for (int b = (int)(grp * g.seqs) + (tid >> g.lper); b < b_end; b += at_once) {
    const int64_t r = (int64_t)b * a.D + d;
    const int len = conv_length(a, b);
    // the row's words, then the carried inputs' (those before t = 0), one or two more to a row
    const int lane = tid & (per - 1);
    int t = (int)(xb * kConvSpan) + E * lane;
    for (bool carried = false;; t += carried ? -E * per : E * per) {
      if (!carried && t >= t_end) {
        if (!a.gstate || xb != 0) break;
        carried = true;
        t = -E * (lane + 1);
      }
      if (carried && t < -E * ((TT + E - 2) / E)) break;
      float gx[E];
#pragma unroll
      for (int e = 0; e < E; ++e) gx[e] = 0.f;
      // an empty sequence's state is handed on and read by no output: it may hold anything
      if (t < len && len > 0) {
        float x[2 * TT + E], gp[TT + E];
        conv_gp<IOT, TT, E, EXACT>(a, r, t, len, w, bias, x, gp);
#pragma unroll
        for (int j = 0; j < TT; ++j)
          if (EXACT || j < a.T) {
#pragma unroll
            for (int e = 0; e < E; ++e) gx[e] = fmaf(w[j], gp[e + j], gx[e]);
          }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          sum[TT] += gp[e];
#pragma unroll
          for (int j = 0; j < TT; ++j) sum[j] = fmaf(gp[e], x[TT + e - j], sum[j]);    // those behind T are not used
        }
      }
      if (t < len) {
        if (a.gstate_out && t + E > len - S) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int i = t + e - (len - S);
            if (i >= 0 && i < S) gx[e] += ld1<IOT>(a.gstate_out, r * S + i);
          }
        }
        if (t + E > len) {
#pragma unroll
          for (int e = 0; e < E; ++e) gx[e] = t + e < len ? gx[e] : 0.f;
        }
      }
      if (carried) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (t + e + S >= 0) st1<IOT>(a.gstate, r * S + t + e + S, gx[e]);
        continue;
      }
#pragma unroll
      for (int k = 0; k < E; k += 8) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = gx[k + e];
        if (t + k < a.L) st8n<IOT>(a.gx, r * a.L + t + k, o, (int)min(a.L - t - k, (int64_t)8));
      }
    }
  }
  // the workgroup's sums: within a wave, then over the waves
#pragma unroll
  for (int j = 0; j <= TT; ++j) {
    float v = row_sum(sum[j]);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if ((tid & 63) == 0) part[tid >> 6][j] = v;
  }
  __syncthreads();
  if (tid <= TT) {
    const float v = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    const int j = tid < TT ? tid : a.T;
    if (tid == TT || tid < a.T) a.partial[((int64_t)id * a.D + d) * (a.T + 1) + j] = v;
  }
}

__global__ __launch_bounds__(SUM_THREADS) void k_conv_sum(ConvArgs a, int64_t parts) {
  __shared__ float lds[32][33];
  const int64_t W = (int64_t)a.D * (a.T + 1), i = blockIdx.x * (int64_t)32 + (threadIdx.x & 31);
  const float v = column_sum(i < W ? a.partial + i : nullptr, parts, W, lds);
  if (threadIdx.x < 32 && i < W) {
    const int64_t d = i / (a.T + 1);
    const int j = (int)(i - d * (a.T + 1));
    if (j < a.T) a.gw[d * a.T + j] = v;
    else if (a.gbias) a.gbias[d] = v;
  }
}

template <int TT>
void conv_forward_tt(const ConvArgs& a, const ConvGrid& g, hipStream_t s) {
  if (a.io) k_conv<1, TT><<<(unsigned)g.groups, 256, 0, s>>>(a, g.per, g.lper, (int)g.blocks);
  else k_conv<0, TT><<<(unsigned)g.groups, 256, 0, s>>>(a, g.per, g.lper, (int)g.blocks);
}

template <int TT>
void conv_step_tt(const ConvArgs& a, hipStream_t s) {
  const unsigned n = (unsigned)(((int64_t)a.B * a.D + 255) / 256);
  if (a.io) k_conv_step<1, TT><<<n, 256, 0, s>>>(a);
  else k_conv_step<0, TT><<<n, 256, 0, s>>>(a);
}

template <int TT>
void conv_backward_tt(const ConvArgs& a, const ConvBackwardGrid& g, hipStream_t s) {
  const unsigned n = (unsigned)(g.parts * a.D);
  if (a.T == TT) {
    if (a.io) k_conv_bwd<1, TT, true><<<n, 256, 0, s>>>(a, g);
    else k_conv_bwd<0, TT, true><<<n, 256, 0, s>>>(a, g);
  } else {
    if (a.io) k_conv_bwd<1, TT, false><<<n, 256, 0, s>>>(a, g);
    else k_conv_bwd<0, TT, false><<<n, 256, 0, s>>>(a, g);
  }
}

}  // namespace

hipError_t short_conv(const ConvArgs& a, hipStream_t s) {
  const ConvGrid g = conv_grid(a.B, a.D, a.L, kConvStep);
  if (a.T <= 4) conv_forward_tt<4>(a, g, s);
  else if (a.T <= 8) conv_forward_tt<8>(a, g, s);
  else conv_forward_tt<16>(a, g, s);
  return hipGetLastError();
}

hipError_t short_conv_step(const ConvArgs& a, hipStream_t s) {
  if (a.T <= 4) conv_step_tt<4>(a, s);
  else if (a.T <= 8) conv_step_tt<8>(a, s);
  else conv_step_tt<16>(a, s);
  return hipGetLastError();
}

hipError_t short_conv_backward(const ConvArgs& a, hipStream_t s) {
  const ConvBackwardGrid g = conv_backward_grid(a.B, a.D, a.L, a.T);
  if (a.T <= 4) conv_backward_tt<4>(a, g, s);
  else if (a.T <= 8) conv_backward_tt<8>(a, g, s);
  else conv_backward_tt<16>(a, g, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t W = (int64_t)a.D * (a.T + 1);
  k_conv_sum<<<(unsigned)((W + 31) / 32), SUM_THREADS, 0, s>>>(a, g.parts);
  return hipGetLastError();
}

}  // namespace hyena
