// kernels_scaled_mm.hip -- matrix product of e4m3 operands with a scale for
// each 128 values along k of a left row and for each 128 x 128 block of the
// right operand:
//   out[m][n] = sum_kb scales[m][kb] wscales[n / 128][kb]
//                 sum_{k in kb} q[m][k] wq[n][k]  + bias[n].
#include <hip/hip_runtime.h>

#include "ssm.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a row from k, zeros behind K (a multiple of 16).
__device__ __forceinline__ i32x4 ld16(const uint8_t* row, int64_t k, int64_t K) {
  i32x4 v = {0, 0, 0, 0};
  if (k < K) v = *reinterpret_cast<const i32x4*>(row + k);
  return v;
}

// A lane's operand of v_mfma_f32_16x16x128: row lane & 15, 32 values of k.
__device__ __forceinline__ i32x8 operand(const uint8_t* row, int64_t k, int64_t K) {
  const i32x4 a = ld16(row, k, K), b = ld16(row, k + 16, K);
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// Eight codes as bf16, which holds every e4m3 value.
__device__ __forceinline__ bf16x8v widen_codes(int lo, int hi) {
  const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const bf16x2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const bf16x2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The sum over one block of 128.  The 8-bit matrix instructions drop low bits
// when they add up the products of a step: 1.4e-5 of the result's norm on
// normal data, far below a bf16 output's half step (2e-3) but not below an
// fp32 output's, which takes the codes as bf16 through the bf16 instructions
// (1e-8) at half their rate.
template <int IOT>
__device__ __forceinline__ f32x4v mfma128(i32x8 a, i32x8 b) {
  f32x4v z = {0.f, 0.f, 0.f, 0.f};
  if constexpr (IOT == 1) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(a[2 * i], a[2 * i + 1]),
                                                  widen_codes(b[2 * i], b[2 * i + 1]), z, 0, 0, 0);
    return z;
  }
}

// 64 x 64 outputs to a workgroup, 32 x 32 to a wave.
template <int IOT, bool CM>
__global__ __launch_bounds__(256) void k_scaled_mm(ScaledArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15, h = lane >> 4;
  const int64_t M = a.M, N = a.N, K = a.K, kb = (K + 127) / 128;
  const int64_t nt = (N + 63) / 64;
  const int64_t m0 = blockIdx.x / nt * 64 + (wave & 1) * 32, n0 = blockIdx.x % nt * 64 + (wave >> 1) * 32;
  f32x4v acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int64_t b = 0; b < kb; ++b) {
    i32x8 x[2], w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i] = operand(a.q + min(m0 + 16 * i + l, M - 1) * K, b * 128 + 32 * h, K);
      w[i] = operand(a.wq + min(n0 + 16 * i + l, N - 1) * K, b * 128 + 32 * h, K);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = min(n0 + 16 * j + (CM ? l : 4 * h), N - 1);
        const float sw = a.wscales[n / 128 * kb + b];
        const f32x4v p = CM ? mfma128<IOT>(x[i], w[j]) : mfma128<IOT>(w[j], x[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t m = min(m0 + 16 * i + (CM ? 4 * h + e : l), M - 1);
          acc[i][j][e] = fmaf(p[e], a.scales[m * kb + b] * sw, acc[i][j][e]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + 16 * i + (CM ? 4 * h + e : l), n = n0 + 16 * j + (CM ? l : 4 * h + e);
        if (m >= M || n >= N) continue;
        const float v = acc[i][j][e] + (a.bias ? a.bias[n] : 0.f);
        st1<IOT>(a.out, CM ? (m / a.L * N + n) * a.L + m % a.L : m * N + n, v);
      }
}

}  // namespace

hipError_t scaled_matmul(const ScaledArgs& a, hipStream_t s) {
  const unsigned n = (unsigned)(((a.M + 63) / 64) * ((a.N + 63) / 64));
  if (a.channel_major) {
    if (a.io) k_scaled_mm<1, true><<<n, 256, 0, s>>>(a);
    else k_scaled_mm<0, true><<<n, 256, 0, s>>>(a);
  } else {
    if (a.io) k_scaled_mm<1, false><<<n, 256, 0, s>>>(a);
    else k_scaled_mm<0, false><<<n, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace hyena
