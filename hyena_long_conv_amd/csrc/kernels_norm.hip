// kernels_norm.hip -- residual addition with a root-mean-square norm, its
// 8-bit output, its backward, and the 8-bit cast by itself.
//
//   s = x + residual (stored, and normed as stored),
//   y = s * r * weight,  r = 1 / sqrt(mean(s^2) + eps),
// along D; in 8 bits y goes out as e4m3 codes with one scale for each 128
// values of a row: scale = max|y| / 448 (1 for a block of zeros, and not
// below the least normal number, where a quotient would lose its digits),
// code = e4m3(y / scale), both divisions correctly rounded.
//
// All of these are bound by their bytes: a row is read once and held in
// registers between its sum and its output, a wave to a row up to D = 2048, a
// workgroup beyond, so that two to four words of 8 values to a thread are in
// flight.  bf16 with a residual: 16384 x 768 in 17 us (5.9 TB/s, part of it
// from the Infinity Cache), 8191 x 2048 to 8 bits in 30 us (3.9 TB/s; 4.7 in
// the best launch), backward of 16384 x 768 in 20 us and 4.6 for the sum over
// rows; a copy of 1 GiB runs at 4.8 TB/s.
#include <hip/hip_runtime.h>

#include "ssm.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int NORM_THREADS = 256;

__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// The size of a value as its bits, whose order as whole numbers is that of the
// sizes, with infinities and then NaN above all others.
__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Maximum over a row of 16 lanes, in every lane.
template <int K>
__device__ __forceinline__ uint32_t ror_bits(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + K, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, ror_bits<8>(v));
  v = max(v, ror_bits<4>(v));
  v = max(v, ror_bits<2>(v));
  return max(v, ror_bits<1>(v));
}

// The sum over the LANES threads (64 to 256, a row each) of a value.
template <int LANES>
__device__ __forceinline__ float group_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (LANES > 64) {
    const int w = threadIdx.x >> 6, first = w & ~(LANES / 64 - 1);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[w] = v;
    __syncthreads();
    v = lds[first];
#pragma unroll
    for (int k = 1; k < LANES / 64; ++k) v += lds[first + k];
  }
  return v;
}

// e4m3 codes of 8 values and their block's scale, from the block's largest
// size.  The quotients are correctly rounded: with r the rounded reciprocal
// of the scale, q = v r corrected once by its remainder is (Markstein 1990),
// as long as the remainder does not underflow; blocks that small are divided.
// Three instructions to a value instead of a division's dozen: 8191 rows of
// 2048 bf16 with a residual take 30 us instead of 35, the cast alone of 8192
// rows 10.9 instead of 13.3.
__device__ __forceinline__ uint2 codes8(const float (&y)[8], uint32_t top, float& scale) {
  const float t = __uint_as_float(top);
  scale = t > 0.f ? fmaxf(t / kE4m3Max, 1.17549435e-38f) : (t != t ? t : 1.f);
  float v[8];
  if (scale < 1e-18f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = y[e] / scale;
  } else {
    const float r = 1.f / scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = y[e] * r;
      v[e] = fmaf(fmaf(-q, scale, y[e]), r, q);
    }
  }
  uint2 q;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  q.x = (uint32_t)lo;
  q.y = (uint32_t)hi;
  return q;
}

__device__ __forceinline__ void st_codes(uint8_t* p, int64_t i, uint2 q, int n) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(1)));
  if (n >= 8) {
    *reinterpret_cast<u2*>(p + i) = u2{q.x, q.y};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[i + e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
  }
}

// LANES threads to a row, V words of 8 values to a thread: D <= 8 LANES V.
// MORE: longer rows, which are read again for the output.
template <int IOT, int LANES, int V, bool Q8, bool MORE>
__global__ __launch_bounds__(NORM_THREADS) void k_norm(NormArgs a) {
  __shared__ float lds[NORM_THREADS / 64];
  const int lane = threadIdx.x & (LANES - 1), D = a.D;
  const int64_t row = blockIdx.x * (int64_t)(NORM_THREADS / LANES) + threadIdx.x / LANES;
  const bool live = row < a.rows;
  const int64_t base = (live ? row : 0) * D;
  const int words = (D + 7) / 8, passes = MORE ? (words + LANES * V - 1) / (LANES * V) : 1;
  float f[V][8];
  // s of word w, stored on the way (`first`), zeros behind the row
  auto take = [&](int w, float (&o)[8], bool first) {
    const int n = live ? D - 8 * w : 0;
    const int64_t i = base + 8 * (int64_t)w;
    if (a.residual && !first) {
      widen8<IOT>(ld8n<IOT>(a.s_out, i, n, a.rows * D), o);
      return;
    }
    widen8<IOT>(ld8n<IOT>(a.x, i, n, a.rows * D), o);
    if (!a.residual) return;
    float r[8];
    widen8<IOT>(ld8n<IOT>(a.residual, i, n, a.rows * D), r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] += r[e];
      if constexpr (IOT == 1) o[e] = __uint_as_float(bf16x2_bits(o[e], 0.f) << 16);
    }
    if (n > 0) st8n<IOT>(a.s_out, i, o, n);
  };
  float ss = 0.f;
  for (int p = 0; p < passes; ++p) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      take(lane + LANES * (k + V * p), f[k], true);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[k][e], f[k][e], ss);
    }
  }
  ss = group_sum<LANES>(ss, lds);
  const float r = 1.f / sqrtf(ss / (float)D + a.eps);
  for (int p = 0; p < passes; ++p) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int w = lane + LANES * (k + V * p), n = live ? D - 8 * w : 0;
      float wt[8], y[8];
      if (MORE) take(w, f[k], false);
      widen8<0>(ld8n<0>(a.weight, 8 * (int64_t)w, D - 8 * w, D), wt);
      uint32_t top = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = f[k][e] * r * wt[e];
        top = max(top, size_bits(y[e]));
      }
      if constexpr (!Q8) {
        if (n > 0) st8n<IOT>(a.y, base + 8 * (int64_t)w, y, n);
      } else {
        // a block of 128 values is a row of 16 lanes
        float scale;
        const uint2 q = codes8(y, row_max(top), scale);
        if (n > 0) {
          st_codes(a.q, base + 8 * (int64_t)w, q, n);
          if ((w & 15) == 0) a.scales[row * ((D + 127) / 128) + (w >> 4)] = scale;
        }
      }
    }
  }
}

template <int IOT, bool Q8>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const auto grid = [&](int lanes) { return dim3((unsigned)((a.rows * lanes + NORM_THREADS - 1) / NORM_THREADS)); };
  if (a.D <= 512) k_norm<IOT, 64, 1, Q8, false><<<grid(64), NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 1024) k_norm<IOT, 64, 2, Q8, false><<<grid(64), NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 2048) k_norm<IOT, 64, 4, Q8, false><<<grid(64), NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 4096) k_norm<IOT, 256, 2, Q8, false><<<grid(256), NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 8192) k_norm<IOT, 256, 4, Q8, false><<<grid(256), NORM_THREADS, 0, s>>>(a);
  else k_norm<IOT, 256, 4, Q8, true><<<grid(256), NORM_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------- 8-bit cast alone
template <int IOT>
__global__ __launch_bounds__(256) void k_quantize_rows(NormArgs a) {
  const int kb = (a.D + 127) / 128;
  const int64_t blk = blockIdx.x * (int64_t)16 + (threadIdx.x >> 4);   // (row, block of 128)
  const int l = threadIdx.x & 15;
  const bool live = blk < a.rows * kb;
  const int64_t row = live ? blk / kb : 0;
  const int c = (int)(live ? blk - row * kb : 0) * 128 + 8 * l, n = live ? a.D - c : 0;
  float y[8], scale;
  uint32_t top = 0u;
  widen8<IOT>(ld8n<IOT>(a.x, row * a.D + c, n, a.rows * a.D), y);
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, size_bits(y[e]));
  const uint2 q = codes8(y, row_max(top), scale);
  if (n > 0) st_codes(a.q, row * a.D + c, q, n);
  if (live && l == 0) a.scales[blk] = scale;
}

// Blocks of 128 x 128: a workgroup each, 16 rows at a time.
template <int IOT>
__global__ __launch_bounds__(256) void k_quantize_tiles(NormArgs a) {
  __shared__ uint32_t lds[16];
  const int kb = (a.D + 127) / 128, rw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t rb = blockIdx.x / kb;
  const int c = (int)(blockIdx.x - rb * kb) * 128 + 8 * l;
  float y[8][8], scale;
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = rb * 128 + 16 * k + rw;
    widen8<IOT>(ld8n<IOT>(a.x, row * a.D + c, row < a.rows ? a.D - c : 0, a.rows * a.D), y[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, size_bits(y[k][e]));
  }
  top = row_max(top);
  if (l == 0) lds[rw] = top;
  __syncthreads();
  top = lds[0];
#pragma unroll
  for (int k = 1; k < 16; ++k) top = max(top, lds[k]);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = rb * 128 + 16 * k + rw;
    const uint2 q = codes8(y[k], top, scale);
    if (row < a.rows && c < a.D) st_codes(a.q, row * a.D + c, q, a.D - c);
  }
  if (threadIdx.x == 0) a.scales[blockIdx.x] = scale;
}

// --------------------------------------------------------------- backward
//
//   gx = r (weight gy - s r mean(s r weight gy)) + gs,  gweight = sum_rows gy s r.
// A workgroup walks over rows; a thread keeps its columns' share of gweight
// in registers, and the workgroup leaves one partial, which k_norm_sum adds up.
template <int IOT, int LANES, int V>
__global__ __launch_bounds__(NORM_THREADS) void k_norm_bwd(NormArgs a) {
  __shared__ float lds[NORM_THREADS / 64];
  const int lane = threadIdx.x & (LANES - 1), D = a.D;
  constexpr int RPW = NORM_THREADS / LANES;
  float wt[V][8], gw[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int w = lane + LANES * k;
    widen8<0>(ld8n<0>(a.weight, 8 * (int64_t)w, D - 8 * w, D), wt[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) gw[k][e] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * RPW;
  for (int64_t r0 = blockIdx.x * (int64_t)RPW; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + threadIdx.x / LANES;
    const bool live = row < a.rows;
    const int64_t base = (live ? row : 0) * D;
    float f[V][8], g[V][8], ss = 0.f, dot = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int w = lane + LANES * k, n = live ? D - 8 * w : 0;
      widen8<IOT>(ld8n<IOT>(a.x, base + 8 * (int64_t)w, n, a.rows * D), f[k]);
      widen8<IOT>(ld8n<IOT>(a.gy, base + 8 * (int64_t)w, n, a.rows * D), g[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(f[k][e], f[k][e], ss);
        dot = fmaf(g[k][e] * wt[k][e], f[k][e], dot);
      }
    }
    ss = group_sum<LANES>(ss, lds);
    dot = group_sum<LANES>(dot, lds);
    // a place behind the last row has no sum to divide by, and with eps = 0 nothing to add
    const float r = live ? 1.f / sqrtf(ss / (float)D + a.eps) : 0.f, m = dot * r * r / (float)D;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int w = lane + LANES * k, n = live ? D - 8 * w : 0;
      float o[8];
      if (a.gs) widen8<IOT>(ld8n<IOT>(a.gs, base + 8 * (int64_t)w, n, a.rows * D), o);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = r * fmaf(g[k][e], wt[k][e], -m * f[k][e]);
        gw[k][e] = fmaf(g[k][e], f[k][e] * r, gw[k][e]);
        o[e] = a.gs ? o[e] + v : v;
      }
      if (n > 0) st8n<IOT>(a.gx, base + 8 * (int64_t)w, o, n);
    }
  }
  if constexpr (RPW > 1) {                            // the workgroup's rows, in order
    __shared__ float sum[RPW - 1][V * LANES * 8];
    const int g = threadIdx.x / LANES;
    if (g > 0) {
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[g - 1][(8 * k + e) * LANES + lane] = gw[k][e];
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int j = 0; j < RPW - 1; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[k][e] += sum[j][(8 * k + e) * LANES + lane];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int w = lane + LANES * k;
    if (8 * w < D) st8n<0>(a.partial, blockIdx.x * (int64_t)D + 8 * (int64_t)w, gw[k], D - 8 * w);
  }
}

// Rows longer than a workgroup's registers: one workgroup for each partial,
// every row read twice.
template <int IOT>
__global__ __launch_bounds__(NORM_THREADS) void k_norm_bwd_long(NormArgs a, int64_t parts) {
  __shared__ float lds[NORM_THREADS / 64];
  const int tid = threadIdx.x, D = a.D, words = (D + 7) / 8;
  float* part = a.partial + blockIdx.x * (int64_t)D;
  bool fresh = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += parts) {
    const int64_t base = row * D;
    float ss = 0.f, dot = 0.f;
    for (int w = tid; w < words; w += NORM_THREADS) {
      float f[8], g[8], wt[8];
      const int n = D - 8 * w;
      widen8<IOT>(ld8n<IOT>(a.x, base + 8 * (int64_t)w, n, a.rows * D), f);
      widen8<IOT>(ld8n<IOT>(a.gy, base + 8 * (int64_t)w, n, a.rows * D), g);
      widen8<0>(ld8n<0>(a.weight, 8 * (int64_t)w, n, D), wt);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(f[e], f[e], ss);
        dot = fmaf(g[e] * wt[e], f[e], dot);
      }
    }
    ss = group_sum<NORM_THREADS>(ss, lds);
    dot = group_sum<NORM_THREADS>(dot, lds);
    const float r = 1.f / sqrtf(ss / (float)D + a.eps), m = dot * r * r / (float)D;
    for (int w = tid; w < words; w += NORM_THREADS) {
      float f[8], g[8], wt[8], o[8], gw[8];
      const int n = D - 8 * w;
      widen8<IOT>(ld8n<IOT>(a.x, base + 8 * (int64_t)w, n, a.rows * D), f);
      widen8<IOT>(ld8n<IOT>(a.gy, base + 8 * (int64_t)w, n, a.rows * D), g);
      widen8<0>(ld8n<0>(a.weight, 8 * (int64_t)w, n, D), wt);
      widen8<0>(fresh ? zero8<0>() : ld8n<0>(part, 8 * (int64_t)w, n, D), gw);   // this thread's own words
      if (a.gs) widen8<IOT>(ld8n<IOT>(a.gs, base + 8 * (int64_t)w, n, a.rows * D), o);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = r * fmaf(g[e], wt[e], -m * f[e]);
        gw[e] = fmaf(g[e], f[e] * r, gw[e]);
        o[e] = a.gs ? o[e] + v : v;
      }
      st8n<0>(part, 8 * (int64_t)w, gw, n);
      st8n<IOT>(a.gx, base + 8 * (int64_t)w, o, n);
    }
    fresh = false;
  }
}

__global__ __launch_bounds__(SUM_THREADS) void k_norm_sum(NormArgs a, int64_t parts) {
  __shared__ float lds[32][33];
  const int64_t i = blockIdx.x * (int64_t)32 + (threadIdx.x & 31);
  const float v = column_sum(i < a.D ? a.partial + i : nullptr, parts, a.D, lds);
  if (threadIdx.x < 32 && i < a.D) a.gw[i] = v;
}

template <int IOT>
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s) {
  const int64_t parts = norm_backward_parts(a.rows, a.D);   // a workgroup leaves one partial
  const dim3 grid((unsigned)parts);
  if (a.D <= 512) k_norm_bwd<IOT, 64, 1><<<grid, NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 1024) k_norm_bwd<IOT, 64, 2><<<grid, NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 2048) k_norm_bwd<IOT, 256, 1><<<grid, NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 4096) k_norm_bwd<IOT, 256, 2><<<grid, NORM_THREADS, 0, s>>>(a);
  else if (a.D <= 8192) k_norm_bwd<IOT, 256, 4><<<grid, NORM_THREADS, 0, s>>>(a);
  else k_norm_bwd_long<IOT><<<grid, NORM_THREADS, 0, s>>>(a, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_norm_sum<<<(unsigned)((a.D + 31) / 32), SUM_THREADS, 0, s>>>(a, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.q) return a.io ? launch_norm<1, true>(a, s) : launch_norm<0, true>(a, s);
  return a.io ? launch_norm<1, false>(a, s) : launch_norm<0, false>(a, s);
}

hipError_t rms_norm_backward(const NormArgs& a, hipStream_t s) {
  return a.io ? launch_norm_backward<1>(a, s) : launch_norm_backward<0>(a, s);
}

hipError_t quantize(const NormArgs& a, hipStream_t s) {
  const int64_t kb = (a.D + 127) / 128;
  if (a.block_rows == 1) {
    const unsigned n = (unsigned)((a.rows * kb + 15) / 16);
    if (a.io) k_quantize_rows<1><<<n, 256, 0, s>>>(a);
    else k_quantize_rows<0><<<n, 256, 0, s>>>(a);
  } else {
    const unsigned n = (unsigned)((a.rows + 127) / 128 * kb);
    if (a.io) k_quantize_tiles<1><<<n, 256, 0, s>>>(a);
    else k_quantize_tiles<0><<<n, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace hyena
