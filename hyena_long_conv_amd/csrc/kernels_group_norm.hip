// kernels_group_norm.hip -- norm of each group of a row's channels (a head's
// outputs) with an activation or a gate, and its backward.
//
//   n = (x - mean) / sqrt(var + eps),  m = n weight + bias,
//   y = m, m sig(m) or m z sig(z).
//
// Bound by its bytes: a group is read once and held in registers between its
// sums and its output.  `lanes` threads share a group (group_norm_plan), so
// that a wave holds several narrow ones; a workgroup keeps to its groups and
// walks over rows, so that weight and bias are loaded once.  16384 rows of 12
// groups of 128 in bf16 with a gate: 27 us, 5.5 TB/s, part of it from the
// Infinity Cache (calls after each other on the same 150 MB); the backward 50
// us (5.0 TB/s) and 5 for the sums over its partials.
#include <hip/hip_runtime.h>

#include "linattn.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

constexpr int GN_THREADS = 256;

// The sum over LANES neighbouring threads (a power of two), in each of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, float* lds) {
  if constexpr (LANES >= 2) v += row_move<0xb1>(v);    // quad_perm: lanes 1 0 3 2
  if constexpr (LANES >= 4) v += row_move<0x4e>(v);    // quad_perm: lanes 2 3 0 1
  if constexpr (LANES >= 8) v += row_move<0x141>(v);   // half of a row mirrored
  if constexpr (LANES >= 16) v += row_move<0x140>(v);  // a row mirrored
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
  if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
  if constexpr (LANES > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  return v;
}

// sigmoid(z), and the derivative of z sigmoid(z).
__device__ __forceinline__ float slope_of(float z, float sig) { return sig * fmaf(z, 1.f - sig, 1.f); }

__device__ __forceinline__ void fill8(const float* p, int64_t i, int n, int64_t total, float none, float (&o)[8]) {
  if (p) {
    widen8<0>(ld8n<0>(p, i, n, total), o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = none;
  }
}

// Where a thread works: its group's first channel and its first word there,
// the first row and how many the workgroup takes at a time.
template <int LANES>
struct Place {
  int c0, lane, slot;      // slot: the row's, in the workgroup
  bool live;               // the group is there
  int64_t row, step;
  __device__ __forceinline__ Place(const GroupNormArgs& a, const GroupNormPlan& p) {
    lane = threadIdx.x & (LANES - 1);
    const int u = threadIdx.x / LANES, g = (int)(blockIdx.x % p.blocks) * p.per + u % p.per;
    slot = u / p.per;
    live = g < a.G && slot < p.rows;
    c0 = live ? g * a.Dg : 0;
    row = blockIdx.x / p.blocks * p.rows;
    step = gridDim.x / p.blocks * p.rows;
  }
};

template <int LANES, int V>
__device__ __forceinline__ void moments(const GroupNormArgs& a, float (&f)[V][8], int lane, float* lds, float& r) {
  float sum = 0.f, ss = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += f[k][e];
  const float mean = lanes_sum<LANES>(sum, lds) / (float)a.Dg;
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[k][e] = 8 * (lane + LANES * k) + e < a.Dg ? f[k][e] - mean : 0.f;
      ss = fmaf(f[k][e], f[k][e], ss);
    }
  r = 1.f / sqrtf(lanes_sum<LANES>(ss, lds) / (float)a.Dg + a.eps);
}

template <int IOT, int LANES, int V>
__global__ __launch_bounds__(GN_THREADS) void k_gnorm(GroupNormArgs a, GroupNormPlan p) {
  __shared__ float lds[GN_THREADS / 64];
  const Place<LANES> at(a, p);
  const int D = a.G * a.Dg;
  const int64_t total = a.rows * D;
  float wt[V][8], bs[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = 8 * (at.lane + LANES * k), n = at.live ? a.Dg - i : 0;
    fill8(a.weight, at.c0 + i, n, D, 1.f, wt[k]);
    fill8(a.bias, at.c0 + i, n, D, 0.f, bs[k]);
  }
  for (int64_t r0 = at.row; r0 < a.rows; r0 += at.step) {
    const int64_t row = r0 + at.slot, base = row * D + at.c0;
    const bool live = at.live && row < a.rows;
    float f[V][8], z[V][8], r;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = 8 * (at.lane + LANES * k), n = live ? a.Dg - i : 0;
      widen8<IOT>(ld8n<IOT>(a.x, base + i, n, total), f[k]);
      if (a.z) widen8<IOT>(ld8n<IOT>(a.z, base + i, n, total), z[k]);
    }
    moments<LANES, V>(a, f, at.lane, lds, r);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = 8 * (at.lane + LANES * k), n = live ? a.Dg - i : 0;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = fmaf(f[k][e] * r, wt[k][e], bs[k][e]);
        if (a.z) y[e] *= z[k][e] * sigmoid_f(z[k][e]);
        else if (a.silu) y[e] *= sigmoid_f(y[e]);
      }
      if (n > 0) st8n<IOT>(a.y, base + i, y, n);
    }
  }
}

// Groups wider than a workgroup's registers: a workgroup to a group, read three times.
template <int IOT>
__global__ __launch_bounds__(GN_THREADS) void k_gnorm_wide(GroupNormArgs a) {
  __shared__ float lds[GN_THREADS / 64];
  const int D = a.G * a.Dg, words = (a.Dg + 7) / 8, tid = threadIdx.x, c0 = (int)(blockIdx.x % a.G) * a.Dg;
  const int64_t base = (int64_t)(blockIdx.x / a.G) * D + c0, total = a.rows * D;
  float f[8], sum = 0.f, ss = 0.f;
  for (int w = tid; w < words; w += GN_THREADS) {
    widen8<IOT>(ld8n<IOT>(a.x, base + 8 * w, a.Dg - 8 * w, total), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += f[e];
  }
  const float mean = lanes_sum<GN_THREADS>(sum, lds) / (float)a.Dg;
  for (int w = tid; w < words; w += GN_THREADS) {
    widen8<IOT>(ld8n<IOT>(a.x, base + 8 * w, a.Dg - 8 * w, total), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = 8 * w + e < a.Dg ? f[e] - mean : 0.f;
      ss = fmaf(d, d, ss);
    }
  }
  const float r = 1.f / sqrtf(lanes_sum<GN_THREADS>(ss, lds) / (float)a.Dg + a.eps);
  for (int w = tid; w < words; w += GN_THREADS) {
    float wt[8], bs[8], z[8];
    const int n = a.Dg - 8 * w;
    widen8<IOT>(ld8n<IOT>(a.x, base + 8 * w, n, total), f);
    if (a.z) widen8<IOT>(ld8n<IOT>(a.z, base + 8 * w, n, total), z);
    fill8(a.weight, c0 + 8 * w, n, D, 1.f, wt);
    fill8(a.bias, c0 + 8 * w, n, D, 0.f, bs);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = fmaf((f[e] - mean) * r, wt[e], bs[e]);
      if (a.z) f[e] *= z[e] * sigmoid_f(z[e]);
      else if (a.silu) f[e] *= sigmoid_f(f[e]);
    }
    st8n<IOT>(a.y, base + 8 * w, f, n);
  }
}

// --------------------------------------------------------------- backward
//
// With gm the gradient of m (gy, gy z sig(z) or gy silu'(m)) and gn = gm weight:
//   gx = r (gn - mean(gn) - n mean(gn n)),  gz = gy m silu'(z),
//   gweight = sum_rows gm n,  gbias = sum_rows gm.
// A thread keeps its channels' shares of the last two in registers, and the
// workgroup leaves one partial, which k_gnorm_sum adds up.

// m's gradient from gy at one value, and z's.
__device__ __forceinline__ float of_m(const GroupNormArgs& a, float gy, float m, float z, float& gz) {
  if (a.z) {
    const float sig = sigmoid_f(z);
    gz = gy * m * slope_of(z, sig);
    return gy * z * sig;
  }
  return a.silu ? gy * slope_of(m, sigmoid_f(m)) : gy;
}

template <int IOT, int LANES, int V>
__global__ __launch_bounds__(GN_THREADS) void k_gnorm_bwd(GroupNormArgs a, GroupNormPlan p) {
  __shared__ float lds[GN_THREADS / 64];
  constexpr int UNITS = GN_THREADS / LANES;
  const Place<LANES> at(a, p);
  const int D = a.G * a.Dg;
  const int64_t total = a.rows * D;
  float wt[V][8], bs[V][8], gw[V][8], gb[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = 8 * (at.lane + LANES * k), n = at.live ? a.Dg - i : 0;
    fill8(a.weight, at.c0 + i, n, D, 1.f, wt[k]);
    fill8(a.bias, at.c0 + i, n, D, 0.f, bs[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) gw[k][e] = 0.f, gb[k][e] = 0.f;
  }
  for (int64_t r0 = at.row; r0 < a.rows; r0 += at.step) {
    const int64_t row = r0 + at.slot, base = row * D + at.c0;
    const bool live = at.live && row < a.rows;
    float f[V][8], g[V][8], z[V][8], r, s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = 8 * (at.lane + LANES * k), n = live ? a.Dg - i : 0;
      widen8<IOT>(ld8n<IOT>(a.x, base + i, n, total), f[k]);
      widen8<IOT>(ld8n<IOT>(a.gy, base + i, n, total), g[k]);
      if (a.z) widen8<IOT>(ld8n<IOT>(a.z, base + i, n, total), z[k]);
    }
    moments<LANES, V>(a, f, at.lane, lds, r);
    if (!live) r = 0.f;                               // a place without a group adds nothing, also with eps = 0
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = 8 * (at.lane + LANES * k), n = live ? a.Dg - i : 0;
      float gz[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[k][e] *= r;
        const float gm = of_m(a, g[k][e], fmaf(f[k][e], wt[k][e], bs[k][e]), a.z ? z[k][e] : 0.f, gz[e]);
        gw[k][e] = fmaf(gm, f[k][e], gw[k][e]);
        gb[k][e] += gm;
        g[k][e] = gm * wt[k][e];
        s1 += g[k][e];
        s2 = fmaf(g[k][e], f[k][e], s2);
      }
      if (a.z && n > 0) st8n<IOT>(a.gz, base + i, gz, n);
    }
    s1 = lanes_sum<LANES>(s1, lds) / (float)a.Dg;
    s2 = lanes_sum<LANES>(s2, lds) / (float)a.Dg;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = 8 * (at.lane + LANES * k), n = live ? a.Dg - i : 0;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = r * fmaf(-f[k][e], s2, g[k][e] - s1);
      if (n > 0) st8n<IOT>(a.gx, base + i, o, n);
    }
  }
  if (!a.partial) return;
  if constexpr (UNITS > 1) {                          // the workgroup's rows, in order, 8 values at a time
    __shared__ float sum[GN_THREADS][17];
    static_assert(V <= 2, "");
#pragma unroll
    for (int k = 0; k < V; ++k) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[threadIdx.x][e] = gw[k][e], sum[threadIdx.x][8 + e] = gb[k][e];
      __syncthreads();
      for (int j = 1; j < p.rows; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at.slot == 0) {
            gw[k][e] += sum[threadIdx.x + j * p.per * LANES][e];
            gb[k][e] += sum[threadIdx.x + j * p.per * LANES][8 + e];
          }
    }
  }
  if (at.slot > 0 || !at.live) return;
  float* part = a.partial + blockIdx.x / p.blocks * (int64_t)(2 * D);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = 8 * (at.lane + LANES * k), n = a.Dg - i;
    if (n > 0) {
      st8n<0>(part, at.c0 + i, gw[k], n);
      st8n<0>(part, D + at.c0 + i, gb[k], n);
    }
  }
}

template <int IOT>
__global__ __launch_bounds__(GN_THREADS) void k_gnorm_bwd_wide(GroupNormArgs a, int64_t parts) {
  __shared__ float lds[GN_THREADS / 64];
  const int D = a.G * a.Dg, words = (a.Dg + 7) / 8, tid = threadIdx.x, c0 = (int)(blockIdx.x % a.G) * a.Dg;
  const int64_t total = a.rows * D, part = blockIdx.x / a.G;
  bool fresh = true;
  for (int64_t row = part; row < a.rows; row += parts) {
    const int64_t base = row * D + c0;
    float f[8], sum = 0.f, ss = 0.f, s1 = 0.f, s2 = 0.f;
    for (int w = tid; w < words; w += GN_THREADS) {
      widen8<IOT>(ld8n<IOT>(a.x, base + 8 * w, a.Dg - 8 * w, total), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += f[e];
    }
    const float mean = lanes_sum<GN_THREADS>(sum, lds) / (float)a.Dg;
    for (int w = tid; w < words; w += GN_THREADS) {
      widen8<IOT>(ld8n<IOT>(a.x, base + 8 * w, a.Dg - 8 * w, total), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = 8 * w + e < a.Dg ? f[e] - mean : 0.f;
        ss = fmaf(d, d, ss);
      }
    }
    const float r = 1.f / sqrtf(lanes_sum<GN_THREADS>(ss, lds) / (float)a.Dg + a.eps);
    // n, gn and gm of word w; `first`: gz and the parameters' shares on the way
    auto word = [&](int w, bool first, float (&n8)[8], float (&gn)[8]) {
      float wt[8], bs[8], z[8], gz[8], gw[8], gb[8];
      const int n = a.Dg - 8 * w;
      widen8<IOT>(ld8n<IOT>(a.x, base + 8 * w, n, total), n8);
      widen8<IOT>(ld8n<IOT>(a.gy, base + 8 * w, n, total), gn);
      if (a.z) widen8<IOT>(ld8n<IOT>(a.z, base + 8 * w, n, total), z);
      fill8(a.weight, c0 + 8 * w, n, D, 1.f, wt);
      fill8(a.bias, c0 + 8 * w, n, D, 0.f, bs);
      float* mine = a.partial ? a.partial + part * (2 * (int64_t)D) : nullptr;   // this thread's own words
      if (first && mine) {
        widen8<0>(fresh ? zero8<0>() : ld8n<0>(mine, c0 + 8 * w, n, 2 * D), gw);
        widen8<0>(fresh ? zero8<0>() : ld8n<0>(mine, D + c0 + 8 * w, n, 2 * D), gb);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n8[e] = 8 * w + e < a.Dg ? (n8[e] - mean) * r : 0.f;
        const float gm = of_m(a, gn[e], fmaf(n8[e], wt[e], bs[e]), a.z ? z[e] : 0.f, gz[e]);
        gw[e] = fmaf(gm, n8[e], gw[e]);
        gb[e] += gm;
        gn[e] = gm * wt[e];
      }
      if (!first) return;
      if (a.z) st8n<IOT>(a.gz, base + 8 * w, gz, n);
      if (mine) {
        st8n<0>(mine, c0 + 8 * w, gw, n);
        st8n<0>(mine, D + c0 + 8 * w, gb, n);
      }
    };
    for (int w = tid; w < words; w += GN_THREADS) {
      float n8[8], gn[8];
      word(w, true, n8, gn);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1 += gn[e];
        s2 = fmaf(gn[e], n8[e], s2);
      }
    }
    s1 = lanes_sum<GN_THREADS>(s1, lds) / (float)a.Dg;
    s2 = lanes_sum<GN_THREADS>(s2, lds) / (float)a.Dg;
    for (int w = tid; w < words; w += GN_THREADS) {
      float n8[8], gn[8];
      word(w, false, n8, gn);
#pragma unroll
      for (int e = 0; e < 8; ++e) gn[e] = r * fmaf(-n8[e], s2, gn[e] - s1);
      st8n<IOT>(a.gx, base + 8 * w, gn, a.Dg - 8 * w);
    }
    fresh = false;
  }
}

__global__ __launch_bounds__(SUM_THREADS) void k_gnorm_sum(GroupNormArgs a, int64_t parts) {
  __shared__ float lds[32][33];
  const int64_t D = (int64_t)a.G * a.Dg, i = blockIdx.x * (int64_t)32 + (threadIdx.x & 31);
  const float v = column_sum(i < 2 * D ? a.partial + i : nullptr, parts, 2 * D, lds);
  if (threadIdx.x < 32 && i < 2 * D) {
    float* const to = i < D ? a.gw : a.gb;
    if (to) to[i < D ? i : i - D] = v;
  }
}

// CALL with the plan's LANES and V as constants.
#define HYENA_GN_DISPATCH(p, CALL)                                  \
  if (p.lanes == 1) CALL(1, 1);                                     \
  else if (p.lanes == 2) CALL(2, 1);                                \
  else if (p.lanes == 4) CALL(4, 1);                                \
  else if (p.lanes == 8) CALL(8, 1);                                \
  else if (p.lanes == 16) CALL(16, 1);                              \
  else if (p.lanes == 32) CALL(32, 1);                              \
  else if (p.lanes == 64 && p.words == 1) CALL(64, 1);              \
  else if (p.lanes == 64) CALL(64, 2);                              \
  else if (p.words == 1) CALL(256, 1);                              \
  else if (p.words == 2) CALL(256, 2);                              \
  else CALL(256, 4)

template <int IOT>
hipError_t launch_gnorm(const GroupNormArgs& a, hipStream_t s) {
  const GroupNormPlan p = group_norm_plan(a.G, a.Dg);
  if (!p.words) {
    k_gnorm_wide<IOT><<<(unsigned)(a.rows * a.G), GN_THREADS, 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t n = (a.rows + p.rows - 1) / p.rows, most = (4096 + p.blocks - 1) / p.blocks;
  const dim3 grid((unsigned)((n < most ? n : most) * p.blocks));
#define HYENA_GN_CALL(LANES, V) k_gnorm<IOT, LANES, V><<<grid, GN_THREADS, 0, s>>>(a, p)
  HYENA_GN_DISPATCH(p, HYENA_GN_CALL);
#undef HYENA_GN_CALL
  return hipGetLastError();
}

template <int IOT>
hipError_t launch_gnorm_backward(const GroupNormArgs& a, hipStream_t s) {
  const GroupNormPlan p = group_norm_plan(a.G, a.Dg);
  const int64_t parts = group_norm_backward_parts(a.rows, a.G, a.Dg);
  const dim3 grid((unsigned)(parts * p.blocks));
  if (!p.words) k_gnorm_bwd_wide<IOT><<<grid, GN_THREADS, 0, s>>>(a, parts);
  else {
#define HYENA_GN_CALL(LANES, V) k_gnorm_bwd<IOT, LANES, V><<<grid, GN_THREADS, 0, s>>>(a, p)
    HYENA_GN_DISPATCH(p, HYENA_GN_CALL);
#undef HYENA_GN_CALL
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partial) return e;
  k_gnorm_sum<<<(unsigned)((2 * (int64_t)a.G * a.Dg + 31) / 32), SUM_THREADS, 0, s>>>(a, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t group_norm(const GroupNormArgs& a, hipStream_t s) {
  return a.io ? launch_gnorm<1>(a, s) : launch_gnorm<0>(a, s);
}

hipError_t group_norm_backward(const GroupNormArgs& a, hipStream_t s) {
  return a.io ? launch_gnorm_backward<1>(a, s) : launch_gnorm_backward<0>(a, s);
}

}  // namespace hyena
