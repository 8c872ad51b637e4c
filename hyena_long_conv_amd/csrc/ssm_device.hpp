// ssm_device.hpp -- device helpers shared by the state-space block's kernels:
// eight-value accesses of fp32 or bf16 rows at any element alignment, the
// lane moves of 16-lane rows, and the two activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fft_engine.hpp"

namespace hyena {

constexpr float kLog2e = 1.4426950408889634f;

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
// Rows of an odd length start at any element: accesses of 16 bytes carry the
// element's alignment only (the memory pipe takes them at any byte).
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

template <int IOT> struct Raw8;
template <> struct Raw8<0> { f32x4v a, b; };
template <> struct Raw8<1> { u32x4v a; };

template <int IOT>
__device__ __forceinline__ float ld1(const void* p, int64_t i) {
  if constexpr (IOT == 0) return static_cast<const float*>(p)[i];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <int IOT>
__device__ __forceinline__ void st1(void* p, int64_t i, float v) {
  if constexpr (IOT == 0) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)bf16x2_bits(v, 0.f);
}

template <int IOT>
__device__ __forceinline__ Raw8<IOT> zero8() {
  Raw8<IOT> r;
  if constexpr (IOT == 0) { r.a = f32x4v{0.f, 0.f, 0.f, 0.f}; r.b = r.a; }
  else r.a = u32x4v{0u, 0u, 0u, 0u};
  return r;
}

// Eight values from element i, all of them in the array.
template <int IOT>
__device__ __forceinline__ Raw8<IOT> ld8(const void* p, int64_t i) {
  Raw8<IOT> r;
  if constexpr (IOT == 0) {
    const float* q = static_cast<const float*>(p) + i;
    r.a = *reinterpret_cast<const f32x4_e4*>(q);
    r.b = *reinterpret_cast<const f32x4_e4*>(q + 4);
  } else {
    r.a = *reinterpret_cast<const u32x4_e2*>(static_cast<const uint16_t*>(p) + i);
  }
  return r;
}

// The first n of eight values from element i of an array of `total`, zeros
// behind them.  The eight are read whole wherever the array has them and
// masked in registers: loads under a lane's condition wait for each other.
template <int IOT>
__device__ __forceinline__ Raw8<IOT> ld8n(const void* p, int64_t i, int n, int64_t total) {
  Raw8<IOT> r = zero8<IOT>();
  if (n <= 0) return r;
  if (i + 8 <= total) {
    r = ld8<IOT>(p, i);
    if (n < 8) {
      if constexpr (IOT == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          r.a[e] = e < n ? r.a[e] : 0.f;
          r.b[e] = e + 4 < n ? r.b[e] : 0.f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r.a[e] = 2 * e + 1 < n ? r.a[e] : (2 * e < n ? r.a[e] & 0xffffu : 0u);
      }
    }
    return r;
  }
  if constexpr (IOT == 0) {                           // the array's last values
    const float* q = static_cast<const float*>(p) + i;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e < n) r.a[e] = q[e];
      if (e + 4 < n) r.b[e] = q[e + 4];
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) r.a[e >> 1] |= (uint32_t)q[e] << (16 * (e & 1));
  }
  return r;
}

template <int IOT>
__device__ __forceinline__ void widen8(const Raw8<IOT>& r, float (&o)[8]) {
  if constexpr (IOT == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) { o[e] = r.a[e]; o[e + 4] = r.b[e]; }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[2 * e] = __uint_as_float(r.a[e] << 16);
      o[2 * e + 1] = __uint_as_float(r.a[e] & 0xffff0000u);
    }
  }
}

// The first n of eight values to element i (bf16: rounded to nearest even),
// n >= 1.
template <int IOT>
__device__ __forceinline__ void st8n(void* p, int64_t i, const float (&v)[8], int n) {
  if constexpr (IOT == 0) {
    float* q = static_cast<float*>(p) + i;
    if (n >= 8) {
      *reinterpret_cast<f32x4_e4*>(q) = f32x4v{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_e4*>(q + 4) = f32x4v{v[4], v[5], v[6], v[7]};
    } else {
      int e = 0;
      float x = v[0], y = v[1], z = v[2];
      if (n & 4) {
        *reinterpret_cast<f32x4_e4*>(q) = f32x4v{v[0], v[1], v[2], v[3]};
        e = 4, x = v[4], y = v[5], z = v[6];
      }
      if (n & 2) {
        q[e] = x, q[e + 1] = y;
        e += 2, x = z;
      }
      if (n & 1) q[e] = x;
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    const u32x4v w = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                      bf16x2_bits(v[6], v[7])};
    if (n >= 8) {
      *reinterpret_cast<u32x4_e2*>(q) = w;
    } else {
      typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
      typedef uint32_t u1 __attribute__((aligned(2)));
      int e = 0;
      uint32_t x = w[0], y = w[1];
      if (n & 4) {
        *reinterpret_cast<u2*>(q) = u2{w[0], w[1]};
        e = 4, x = w[2], y = w[3];
      }
      if (n & 2) {
        *reinterpret_cast<u1*>(q + e) = x;
        e += 2, x = y;
      }
      if (n & 1) q[e] = (uint16_t)x;
    }
  }
}

// Lane moves within rows of 16 lanes.  shr<k>: lane i gets lane i-k's value,
// shl<k>: lane i+k's; lanes without a source get 0, which lets the move become
// part of the instruction that uses it.  ror<k>: lane i gets lane (i-k) mod
// 16's.
template <int CTRL>
__device__ __forceinline__ float row_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int K> __device__ __forceinline__ float row_shr(float v) { return row_move<0x110 + K>(v); }
template <int K> __device__ __forceinline__ float row_shl(float v) { return row_move<0x100 + K>(v); }
template <int K> __device__ __forceinline__ float row_ror(float v) { return row_move<0x120 + K>(v); }

// The sum over a row of 16 lanes, in every lane.
__device__ __forceinline__ float row_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  v += row_ror<1>(v);
  return v;
}

// A workgroup of 1024 threads sums 32 columns of `parts` rows of partials in a
// fixed order: 32 threads to a column, whose sum thread (slice 0) returns.
// `col` is the column's first value (nullptr: none), `stride` a row's length.
constexpr int SUM_THREADS = 1024;
__device__ __forceinline__ float column_sum(const float* col, int64_t parts, int64_t stride, float (*lds)[33]) {
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  float v = 0.f;
  if (col) {
    int64_t p = k;
    for (; p + 96 < parts; p += 128) {               // four loads in flight
      const float a = col[p * stride], b = col[(p + 32) * stride];
      const float d = col[(p + 64) * stride], e = col[(p + 96) * stride];
      v += (a + b) + (d + e);
    }
    for (; p < parts; p += 32) v += col[p * stride];
  }
  lds[k][c] = v;
  __syncthreads();
  if (k == 0)
    for (int j = 1; j < 32; ++j) v += lds[j][c];
  return v;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }   // 1 ulp
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }     // 1 ulp

// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid_f(float x) { return rcp_fast(1.f + exp2_fast(-kLog2e * x)); }

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), with log1p(e) = 2 artanh(s),
// s = e / (2 + e) in (0, 1/3].  p = (artanh(s) / s - 1) / s^2 is interpolated
// at four Chebyshev nodes of s^2 in [0, 1/9]; s^2 p, which is what it adds to
// 1, is off by 1.7e-8 at most (2^-25.8; p itself by 1.5e-7), so the relative
// error is a few units of the last place over the whole range (a plain log of
// 1 + e would lose e's low bits, and small time steps with them).  The
// product with log2(e) is kept in two parts: its rounding alone would cost
// |x| / 2 units.  Below e^-87 the result is held at that value.
__device__ __forceinline__ float softplus_f(float x) {
  const float m = fmaxf(-fabsf(x), -87.f);
  const float hi = m * kLog2e, lo = fmaf(m, 1.92596299e-8f, fmaf(m, kLog2e, -hi));
  const float e = exp2_fast(hi) * fmaf(lo, 0.6931471805599453f, 1.f);
  const float s = e * rcp_fast(2.f + e), q = s * s;
  float p = 0.134257490f;
  p = fmaf(p, q, 0.141183099f);
  p = fmaf(p, q, 0.200037803f);
  p = fmaf(p, q, 0.333333202f);
  p = p * q;
  const float l = fmaf(2.f * s, p, 2.f * s);
  // a NaN passes through x + l, infinities through the maximum
  return (x > 0.f ? x : (x == x ? 0.f : x)) + l;
}

}  // namespace hyena
