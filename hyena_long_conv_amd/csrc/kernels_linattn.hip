// kernels_linattn.hip -- linear attention with a decay for each head: passes
// over whole sequences, single tokens, and sums over shared heads.
//
//   S[t] = lambda S[t-1] + su k[t] v[t]^T,  out[t] = so S[t]^T q[t].
#include <hip/hip_runtime.h>

#include "linattn.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

__device__ __forceinline__ float decay_of(const float* log_decay, int h) {
  return log_decay ? expf(log_decay[h]) : 1.f;
}

// One token after the other: a workgroup keeps 64 columns of a head's state,
// 4 threads to a column.
template <int IOT, int KR>
__global__ __launch_bounds__(256) void k_lin_tokens(LinArgs a) {
  const LinPass& p = a.pass[blockIdx.z];
  const int tiles = (p.DV + 63) / 64, tile = (int)(blockIdx.x % 4);
  if (tile >= tiles) return;
  __shared__ float part[4][64], lq[4 * KR], lk[4 * KR];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6, dv = tile * 64 + c;
  const int64_t b = blockIdx.x / 4 / a.H;
  const int h = blockIdx.x / 4 - (int)b * a.H;
  const bool live = dv < p.DV;
  const int64_t n = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.L) : a.L;
  const float lam = decay_of(a.log_decay, h);
  float S[KR];
  const int64_t sb = (b * a.H + h) * (int64_t)p.DK * p.DV;
#pragma unroll
  for (int r = 0; r < KR; ++r) {
    const int dk = g * KR + r;
    S[r] = p.s0 && live && dk < p.DK ? p.s0[sb + (int64_t)dk * p.s0_k + (int64_t)dv * p.s0_v] : 0.f;
  }
  for (int64_t i = 0; i < a.L; ++i) {
    const int64_t t = i < n && p.reverse ? n - 1 - i : i, o = ((b * a.L + t) * a.H + h) * p.DV + dv;
    float y = 0.f;
    if (i < n) {
      __syncthreads();
      for (int d = threadIdx.x; d < 4 * KR; d += 256) {
        lq[d] = d < p.DK ? ld1<IOT>(p.q.p, b * p.q.batch + t * p.q.token + h / p.q.share * p.q.head + d) : 0.f;
        lk[d] = d < p.DK ? ld1<IOT>(p.k.p, b * p.k.batch + t * p.k.token + h / p.k.share * p.k.head + d) : 0.f;
      }
      const float v = live ? p.su * ld1<IOT>(p.v.p, b * p.v.batch + t * p.v.token + h / p.v.share * p.v.head + dv) : 0.f;
      __syncthreads();
      const float l = p.reverse && i == 0 ? 1.f : lam;
#pragma unroll
      for (int r = 0; r < KR; ++r) {
        S[r] = fmaf(lk[g * KR + r], v, l * S[r]);
        y = fmaf(lq[g * KR + r], S[r], y);
      }
      part[g][c] = y;
      __syncthreads();
      y = p.so * ((part[0][c] + part[1][c]) + (part[2][c] + part[3][c]));
    }
    if (g == 0 && live) {
      if (p.out_f32) static_cast<float*>(p.out)[o] = y;
      else st1<IOT>(p.out, o, y);
    }
  }
  if (!p.s_out || !live) return;
  const float l = p.reverse && n > 0 ? lam : 1.f;
#pragma unroll
  for (int r = 0; r < KR; ++r)
    if (g * KR + r < p.DK) p.s_out[sb + (int64_t)(g * KR + r) * p.DV + dv] = l * S[r];
}

template <int IOT>
hipError_t launch(const LinArgs& a, hipStream_t s) {
  int dk = 0;
  for (int i = 0; i < a.passes; ++i) dk = a.pass[i].DK > dk ? a.pass[i].DK : dk;
  const dim3 grid((unsigned)(4 * a.B * a.H), 1, (unsigned)a.passes);
  if (dk <= 64) k_lin_tokens<IOT, 16><<<grid, 256, 0, s>>>(a);
  else k_lin_tokens<IOT, 64><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
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
  const float lam = decay_of(a.log_decay, h);
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
            s[u][e] = fmaf(lk[r], v[e], lam * s[u][e]);
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
