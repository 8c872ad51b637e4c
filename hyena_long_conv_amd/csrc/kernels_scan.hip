// kernels_scan.hip -- the selective state-space scan, forward, for single
// tokens, and backward.
//
//   dt = softplus(delta + delta_bias),  a[t][n] = exp(dt[t] A[n]),
//   h[t][n] = a[t][n] h[t-1][n] + dt[t] u[t] B[t][n],
//   y[t] = (sum_n C[t][n] h[t][n] + skip u[t]) * silu(z[t])
//
// per channel d of each sequence; B and C are shared by the channels of a
// group.  Steps behind a sequence's length count as dt = u = B = C = 0: the
// state stays as it is, and the values stored there may be anything.
//
// The recurrence is a scan of the maps h -> a h + b, whose composition is
// (a2 a1, a2 b1 + b2).  16 lanes (one DPP row) hold 128 steps of one channel,
// 8 consecutive ones each: a lane composes its 8 steps, the row scans the 16
// results in 4 steps of 2 instructions, and the lane runs its 8 steps again
// from the right start.  A wave holds 4 channels, a workgroup 16, which share
// B and C in LDS as fp32.
//
// Arithmetic bounds it: to 8 (t, n) of a lane 8 products dt A, 9 exponentials
// (four issue slots each), 8 products with B, 7 + 8 steps of the recurrence, 8
// with C and about 12 for the row's scan, 88 slots.  8 x 1536 x 2048, 16
// states, bf16: 309 000 cycles of a compute unit, 94% of them with vector
// instructions: 134 us a call at some 2.3 GHz (147 to 153 where the clock is
// 2.0, as under the profiler); its bytes at a copy's rate are 42 us.  (A lane to a channel, with B and C as scalars, would need 64 slots
// and no scan, but 65536 channels to fill the chip, or a second pass over the
// exponentials.)
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ssm.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

constexpr int CH = kScanChunk, TILE = kScanTile, SCAN_THREADS = 256;

// Inclusive scan of the maps (P, H) over a row, lane 0 first.  A lane whose
// range reaches lane 0 has nothing more to take in: the zeros that come from
// outside the row leave its H as it is, and its P, which they clear, has no
// other use.
//
// H += P * (lane i-k's or i+k's H) as one instruction.  A lane move may read a
// register only two issue slots after it was written; the compiler sees to
// that around its own instructions, but not at either end of these.
template <int K> __device__ __forceinline__ void add_shr(float& H, float P) {
  asm("s_nop 1\n\tv_fmac_f32_dpp %0, %0, %1 row_shr:%2 row_mask:0xf bank_mask:0xf bound_ctrl:1\n\ts_nop 1" : "+v"(H) : "v"(P), "n"(K));
}
template <int K> __device__ __forceinline__ void add_shl(float& H, float P) {
  asm("s_nop 1\n\tv_fmac_f32_dpp %0, %0, %1 row_shl:%2 row_mask:0xf bank_mask:0xf bound_ctrl:1\n\ts_nop 1" : "+v"(H) : "v"(P), "n"(K));
}

__device__ __forceinline__ void row_scan(float P, float& H) {
  add_shr<1>(H, P);
  P *= row_shr<1>(P);
  add_shr<2>(H, P);
  P *= row_shr<2>(P);
  add_shr<4>(H, P);
  P *= row_shr<4>(P);
  add_shr<8>(H, P);
}

// The same, lane 15 first.
__device__ __forceinline__ void row_scan_back(float P, float& H) {
  add_shl<1>(H, P);
  P *= row_shl<1>(P);
  add_shl<2>(H, P);
  P *= row_shl<2>(P);
  add_shl<4>(H, P);
  P *= row_shl<4>(P);
  add_shl<8>(H, P);
}

// LDS place of step t's value among a state's 128: lanes read their 8 steps
// as two 16-byte words, the first halves of all lanes side by side, so that
// neither read has bank conflicts.
__device__ __forceinline__ void stage8(float* s, int l, const float (&v)[8]) {
  *reinterpret_cast<f32x4v*>(s + 4 * l) = f32x4v{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4v*>(s + 64 + 4 * l) = f32x4v{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void fetch8(const float* s, int l, float (&v)[8]) {
  const f32x4v x = *reinterpret_cast<const f32x4v*>(s + 4 * l);
  const f32x4v y = *reinterpret_cast<const f32x4v*>(s + 64 + 4 * l);
#pragma unroll
  for (int e = 0; e < 4; ++e) { v[e] = x[e]; v[e + 4] = y[e]; }
}

__device__ __forceinline__ int seq_length(const ScanArgs& a, int b) {
  if (!a.lengths) return (int)a.L;
  const int n = a.lengths[b];
  return n < 0 ? 0 : (n > a.L ? (int)a.L : n);
}

// dt and u of a lane's 8 steps (zeros behind the length).
template <int IOT>
__device__ __forceinline__ void steps8(const ScanArgs& a, const Raw8<IOT>& ru, const Raw8<IOT>& rd, float bias, int n,
                                       float (&u)[8], float (&dt)[8]) {
  widen8<IOT>(ru, u);
  widen8<IOT>(rd, dt);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = dt[i] + bias;
    dt[i] = a.softplus ? softplus_f(x) : x;
  }
  if (n < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dt[i] = i < n ? dt[i] : 0.f;
  }
}

// ---------------------------------------------------------------- forward
//
// One workgroup: 16 channels of a group (with SPLIT = 4: 4 channels, whose
// states its waves share) over one time segment, chunk after chunk.  END: only the state at the segment's end from a zero start, and the
// sum of dt, for the segments behind it (all but the last run this first
// when the time axis is split); a segment's decay is exp(A sum dt), so the
// start of segment s is a short recurrence over the ones before it, which
// each workgroup does for its own channels.
template <int IOT, int NV, int SPLIT, bool END>
__global__ __launch_bounds__(SCAN_THREADS) void k_scan(ScanArgs a) {
  extern __shared__ float lds[];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane >> 4, l = lane & 15;
  constexpr int TC = TILE / SPLIT;                   // channels of the workgroup
  const int N = a.N, Dg = a.D / a.G, tiles = (Dg + TC - 1) / TC;
  const int nseg = END ? a.segs - 1 : a.segs;
  int id = blockIdx.x;
  const int tile = id % tiles; id /= tiles;
  const int g = id % a.G; id /= a.G;
  const int seg = id % nseg;
  const int b = id / nseg;
  const int cw = SPLIT == 1 ? wave * 4 + row : row, dg = tile * TC + cw;
  // this wave's states
  const int share = (N + SPLIT - 1) / SPLIT, n_begin = SPLIT == 1 ? 0 : wave * share, n_end = min(N, n_begin + share);
  const bool first = SPLIT == 1 || wave == 0;
  const bool live = dg < Dg;
  const int d = g * Dg + (live ? dg : Dg - 1);
  const int64_t L = a.L;
  const int len = seq_length(a, b);
  const int64_t base = ((int64_t)b * a.D + d) * L;
  const int64_t bc = ((int64_t)b * a.G + g) * N * L;
  const int64_t total = (int64_t)a.B * a.D * L, bc_total = (int64_t)a.B * a.G * N * L;
  const int t_begin = (int)(seg * a.seg);
  const int t_end = (int)min(L, (int64_t)t_begin + a.seg);

  float* sB = lds;                                   // [N][128]
  float* sC = END ? lds : lds + N * CH;              // [N][128]
  float2* sS = reinterpret_cast<float2*>((END ? lds : sC) + N * CH);   // [TC][N]: A log2(e), the state at the chunk's start
  f32x4v* sY = reinterpret_cast<f32x4v*>(sS + TC * N);                 // SPLIT > 1: [SPLIT - 1][2][64] parts of y

  for (int i = tid; i < TC * N; i += SCAN_THREADS) {
    const int c = i / N, n = i - c * N, dc = tile * TC + c;
    float A2 = 0.f, h = 0.f;
    if (dc < Dg) {
      const int ch = g * Dg + dc;
      A2 = a.A[(int64_t)ch * N + n] * kLog2e;
      if constexpr (!END) {
        if (a.state) h = a.state[((int64_t)b * a.D + ch) * N + n];
        const float* ends = a.hend + ((int64_t)b * a.segs * a.D + ch) * N + n;
        const float* sums = a.sdt + (int64_t)b * a.segs * a.D + ch;
        for (int s0 = 0; s0 < seg; s0 += 16) {        // 16 segments' loads in flight
          float e[16], t[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int64_t at = (int64_t)min(s0 + k, seg - 1) * a.D;
            e[k] = ends[at * N];
            t[k] = sums[at];
          }
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (s0 + k < seg) h = fmaf(exp2_fast(A2 * t[k]), h, e[k]);
        }
      }
    }
    sS[i] = make_float2(A2, h);
  }
  const float bias = a.dbias ? a.dbias[d] : 0.f;
  const float skip = !END && a.skip ? a.skip[d] : 0.f;
  float dt_total = 0.f;

  // B and C of a chunk: 16 words of 8 steps for each state, NV for a thread
  constexpr int NW = END ? (NV + 1) / 2 : NV;
  const int words = (END ? N : 2 * N) * 16;
  Raw8<IOT> rbc[NW], ru, rd, rz;
  auto load = [&](int t0) {
    const int t = t0 + 8 * l;
    const auto word = [&](const void* p, int64_t i, int n, int64_t end) {
      return t0 + CH <= len ? ld8<IOT>(p, i) : ld8n<IOT>(p, i, n, end);     // the same way for the whole workgroup
    };
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int i = tid + SCAN_THREADS * k, v = i & 15, n = i >> 4;
      if (i < words) {
        const bool isC = n >= N;
        rbc[k] = word(isC ? a.Cm : a.Bm, bc + (int64_t)(isC ? n - N : n) * L + t0 + 8 * v, len - t0 - 8 * v, bc_total);
      }
    }
    // a wave's channels behind the group's last one read that one's row
    ru = word(a.u, base + t, len - t, total);
    rd = word(a.delta, base + t, len - t, total);
    if constexpr (!END)
      if (a.z) rz = word(a.z, base + t, len - t, total);
  };
  if (t_begin < len) load(t_begin);

  for (int t0 = t_begin; t0 < t_end; t0 += CH) {
    const int t = t0 + 8 * l, m = len - t;
    if (t0 >= len) {                                  // behind the sequence: zeros
      if constexpr (!END) {
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (first && live && t < L) st8n<IOT>(a.y, base + t, y, (int)min(L - t, (int64_t)8));
      }
      continue;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int i = tid + SCAN_THREADS * k;
      if (i < words) {
        float v[8];
        widen8<IOT>(rbc[k], v);
        stage8(lds + (i >> 4) * CH, i & 15, v);
      }
    }
    float u[8], dt[8], z[8], y[8];
    steps8<IOT>(a, ru, rd, bias, m, u, dt);
    if constexpr (!END)
      if (a.z) widen8<IOT>(rz, z);
    __syncthreads();
    if (t0 + CH < t_end && t0 + CH < len) load(t0 + CH);   // in flight over this chunk's scan

    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = first ? skip * u[i] : 0.f;
      u[i] *= dt[i];
      sum += dt[i];
    }
    dt_total += sum;
    // U states at once: their lane moves fill each other's waits
    auto states = [&](int n, auto count) {
      constexpr int U = decltype(count)::value;
      float x[U][8], al[U][8], h0[U], H[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float2 sc = sS[cw * N + n + k];
        h0[k] = sc.y;
        fetch8(sB + (n + k) * CH, l, x[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          al[k][i] = exp2_fast(dt[i] * sc.x);
          x[k][i] *= u[i];
        }
        H[k] = x[k][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) H[k] = fmaf(al[k][i], H[k], x[k][i]);
        const float P = exp2_fast(sc.x * sum);
        H[k] = fmaf(P, l == 0 ? h0[k] : 0.f, H[k]);
        row_scan(P, H[k]);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float r = row_ror<1>(H[k]);             // lane 0: the state at the chunk's end
        if (l == 0) sS[cw * N + n + k].y = r;
        if constexpr (!END) {
          float c[8];
          fetch8(sC + (n + k) * CH, l, c);
          float h = l == 0 ? h0[k] : r;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h = fmaf(al[k][i], h, x[k][i]);
            y[i] = fmaf(h, c[i], y[i]);
          }
        }
      }
    };
    int n = n_begin;
    for (; n + 2 <= n_end; n += 2) states(n, std::integral_constant<int, 2>());
    if (n < n_end) states(n, std::integral_constant<int, 1>());
    if constexpr (!END && SPLIT > 1) {                // the states' shares of y meet in the first wave
      if (wave > 0) {
        sY[(wave * 2 - 2) * 64 + lane] = f32x4v{y[0], y[1], y[2], y[3]};
        sY[(wave * 2 - 1) * 64 + lane] = f32x4v{y[4], y[5], y[6], y[7]};
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int k = 0; k < SPLIT - 1; ++k) {
          const f32x4v p = sY[2 * k * 64 + lane], q = sY[(2 * k + 1) * 64 + lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) { y[e] += p[e]; y[e + 4] += q[e]; }
        }
      }
    }
    if (!END && first) {
      if (a.z) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= z[i] * sigmoid_f(z[i]);
      }
      if (m < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = i < m ? y[i] : 0.f;
      }
      if (live && t < L) st8n<IOT>(a.y, base + t, y, (int)min(L - t, (int64_t)8));
    }
  }

  if constexpr (END) {
    dt_total = row_sum(dt_total);
    if (first && live && l == 0) a.sdt[((int64_t)b * a.segs + seg) * a.D + d] = dt_total;
  } else if (!a.state_out || seg != a.segs - 1) {
    return;
  }
  __syncthreads();
  for (int i = tid; i < TC * N; i += SCAN_THREADS) {
    const int c = i / N, n = i - c * N, dc = tile * TC + c;
    if (dc >= Dg) continue;
    const int ch = g * Dg + dc;
    if constexpr (END) a.hend[(((int64_t)b * a.segs + seg) * a.D + ch) * N + n] = sS[i].y;
    else a.state_out[((int64_t)b * a.D + ch) * N + n] = sS[i].y;
  }
}

template <int IOT, int NV, int SPLIT>
hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
  constexpr int TC = TILE / SPLIT;
  const int64_t tiles = (a.D / a.G + TC - 1) / TC, wgs = tiles * a.G * a.B;
  const size_t state = (size_t)TC * a.N * 8, bc = (size_t)a.N * CH * 4, parts = (SPLIT - 1) * 2048;
  if (a.segs > 1) {
    k_scan<IOT, NV, SPLIT, true><<<dim3((unsigned)(wgs * (a.segs - 1))), SCAN_THREADS, bc + state, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan<IOT, NV, SPLIT, false><<<dim3((unsigned)(wgs * a.segs)), SCAN_THREADS, 2 * bc + state + parts, s>>>(a);
  return hipGetLastError();
}

template <int IOT, int SPLIT>
hipError_t launch_scan_nv(const ScanArgs& a, hipStream_t s) {
  const int nv = (a.N + 7) / 8;
  return nv <= 1   ? launch_scan<IOT, 1, SPLIT>(a, s)
         : nv <= 2 ? launch_scan<IOT, 2, SPLIT>(a, s)
         : nv <= 4 ? launch_scan<IOT, 4, SPLIT>(a, s)
                   : launch_scan<IOT, 8, SPLIT>(a, s);
}

// ------------------------------------------------------------ single tokens
//
// 4 states to a lane, W lanes (a power of two, W * 4 >= N) to a channel of a
// sequence; the state's read and write are the call's traffic: 128 x 1536
// channels of 16 states in 8.8 us, 3.0 TB/s (5.6 us at a copy's rate).  What
// is above that is latency: u, delta and z, then A and the state, then B's
// and C's eight values, each a load under its lane's condition that is waited
// for before the next.
template <int IOT>
__global__ __launch_bounds__(256) void k_scan_step(ScanArgs a, int W, int lw, float* __restrict__ state) {
  const int64_t idx = blockIdx.x * (int64_t)256 + threadIdx.x, r = idx >> lw;
  const int l = (int)(idx & (W - 1)), N = a.N, n0 = 4 * l;
  const bool live = r < (int64_t)a.B * a.D;
  float part = 0.f, u = 0.f, z = 0.f, skip = 0.f;
  if (live) {
    const uint32_t b = (uint32_t)r / (uint32_t)a.D;   // rows are at most 2^30
    const int d = (int)((uint32_t)r - b * (uint32_t)a.D), g = a.G > 1 ? d / (a.D / a.G) : 0;
    u = ld1<IOT>(a.u, r);
    float dt = ld1<IOT>(a.delta, r) + (a.dbias ? a.dbias[d] : 0.f);
    if (a.z) z = ld1<IOT>(a.z, r);
    if (a.skip) skip = a.skip[d];
    const float* A = a.A + (int64_t)d * N + n0;
    float* h = state + r * N + n0;
    const int64_t bc = ((int64_t)b * a.G + g) * N + n0;
    float Av[4], hv[4], Bv[4], Cv[4];
    if ((N & 3) == 0) {
      if (n0 < N) {
        const f32x4v x = *reinterpret_cast<const f32x4v*>(A), y = *reinterpret_cast<const f32x4v*>(h);
#pragma unroll
        for (int e = 0; e < 4; ++e) { Av[e] = x[e]; hv[e] = y[e]; }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n0 + e < N) { Av[e] = A[e]; hv[e] = h[e]; }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = n0 + e < N;
      Bv[e] = in ? ld1<IOT>(a.Bm, bc + e) : 0.f;
      Cv[e] = in ? ld1<IOT>(a.Cm, bc + e) : 0.f;
    }
    if (a.softplus) dt = softplus_f(dt);
    const float du = dt * u;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n0 + e < N) {
        hv[e] = fmaf(exp2_fast(dt * (Av[e] * kLog2e)), hv[e], du * Bv[e]);
        part = fmaf(hv[e], Cv[e], part);
      }
    if ((N & 3) == 0) {
      if (n0 < N) *reinterpret_cast<f32x4v*>(h) = f32x4v{hv[0], hv[1], hv[2], hv[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n0 + e < N) h[e] = hv[e];
    }
  }
  for (int o = W >> 1; o > 0; o >>= 1) part += __shfl_xor(part, o);
  if (live && l == 0) {
    float y = fmaf(skip, u, part);
    if (a.z) y *= z * sigmoid_f(z);
    st1<IOT>(a.y, r, y);
  }
}

// --------------------------------------------------------------- backward
//
// With g[t] the gradient of h[t], q[t] = a[t] g[t] what it hands to h[t-1],
// gy' = gy silu(z) and g[t] = C[t] gy'[t] + q[t+1]:
//   gB[t] = sum_d g dt u,  gC[t] = sum_d h gy',  gA = sum_t q[t] h[t-1] dt[t],
//   gu = dt sum_n g B + skip gy',
//   gdt = u sum_n g B + sum_n q[t] h[t-1] A,  gdelta = gdt sigmoid(delta + bias),
//   gz = gy (sum_n C h + skip u) silu'(z).
// Three passes.  The first leaves each chunk's end state from a zero start
// and the carry q at its start from a zero end (and the sum of dt); the
// second joins them along time, both ways, into the state at each chunk's
// start and the carry at its end; the third then does all chunks at once.
// Its workgroup stays at one chunk and walks over channels, so that B and C
// are staged once and the sums over channels stay on the chip.  Rows of one
// chunk need the third pass only.
//
// 4 x 1536 x 2048, 16 states, bf16: 78 us for the first pass, 7 for the
// second, 194 for the third and 9 for the sums (298 in all as a call; 37 at a
// copy's rate): vector units 89% and 92% busy, some 75 and 200 instructions
// to 8 (t, n) of a lane.  Tried for the third pass and slower, on a card where
// it took 214 us: sums over channels kept per lane in LDS instead of folded
// over the wave (15% fewer instructions, but 84 KB of LDS: 239 us), 8 waves to
// a workgroup up to 32 states (248 us: twice the turns), two waves to a SIMD
// without the few spilled registers of three (220 us).

// Chunk sums: H, Q [N] and sum dt of 4 channels to a wave.
template <int IOT>
__global__ __launch_bounds__(SCAN_THREADS) void k_scan_bwd_ends(ScanArgs a) {
  extern __shared__ float lds[];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane >> 4, l = lane & 15;
  const int N = a.N, Dg = a.D / a.G, tiles = (Dg + TILE - 1) / TILE, per = (tiles + a.splits - 1) / a.splits;
  int id = blockIdx.x;
  const int split = id % a.splits; id /= a.splits;
  const int c = id % a.chunks; id /= a.chunks;
  const int g = id % a.G, b = id / a.G;
  const int64_t L = a.L;
  const int len = seq_length(a, b), t0 = c * CH, t = t0 + 8 * l, m = len - t;
  const int64_t bc = ((int64_t)b * a.G + g) * N * L;
  const int64_t total = (int64_t)a.B * a.D * L, bc_total = (int64_t)a.B * a.G * N * L;
  float* sB = lds;
  float* sC = lds + N * CH;
  for (int i = tid; i < 2 * N * 16; i += SCAN_THREADS) {
    const int v = i & 15, n = i >> 4;
    const bool isC = n >= N;
    float x[8];
    widen8<IOT>(ld8n<IOT>(isC ? a.Cm : a.Bm, bc + (int64_t)(isC ? n - N : n) * L + t0 + 8 * v, len - t0 - 8 * v, bc_total), x);
    stage8(lds + n * CH, v, x);
  }
  __syncthreads();
  const int tile_end = min(tiles, (split + 1) * per);
  for (int tile = split * per; tile < tile_end; ++tile) {
    const int dg = tile * TILE + wave * 4 + row;
    const bool live = dg < Dg;
    const int d = g * Dg + (live ? dg : Dg - 1), mm = live ? m : 0;
    const int64_t at = ((int64_t)b * a.D + d) * L + t;
    float u[8], dt[8], gy[8];
    const Raw8<IOT> rg = ld8n<IOT>(a.gy, at, mm, total);
    Raw8<IOT> rz;
    if (a.z) rz = ld8n<IOT>(a.z, at, mm, total);
    steps8<IOT>(a, ld8n<IOT>(a.u, at, mm, total), ld8n<IOT>(a.delta, at, mm, total), a.dbias ? a.dbias[d] : 0.f, mm, u, dt);
    widen8<IOT>(rg, gy);
    if (a.z) {
      float z[8];
      widen8<IOT>(rz, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) gy[i] *= z[i] * sigmoid_f(z[i]);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] *= dt[i];
      sum += dt[i];
    }
    const int64_t r = ((int64_t)b * a.chunks + c) * a.D + d;
    const float* A = a.A + (int64_t)d * N;
    for (int n = 0; n < N; ++n) {
      const float A2 = A[n] * kLog2e;
      float x[8], al[8], cc[8];
      fetch8(sB + n * CH, l, x);
      fetch8(sC + n * CH, l, cc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        al[i] = exp2_fast(dt[i] * A2);
        x[i] *= u[i];
      }
      float H = x[0], Q = al[7] * (cc[7] * gy[7]);
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        H = fmaf(al[i], H, x[i]);
        Q = al[7 - i] * fmaf(cc[7 - i], gy[7 - i], Q);
      }
      const float P = exp2_fast(A2 * sum);
      row_scan(P, H);
      row_scan_back(P, Q);
      if (live && l == 15) a.hc[r * N + n] = H;
      if (live && l == 0) a.qc[r * N + n] = Q;
    }
    sum = row_sum(sum);
    if (live && l == 0) a.dts[r] = sum;
  }
}

// Joins the chunks along time: hc becomes the state at each chunk's start,
// qc the carry that comes in behind its end.  A thread to a state and a
// direction (blockIdx.y); 16 chunks are read before the first of them is
// overwritten, since the time is that of their loads, one after the other.
__global__ __launch_bounds__(256) void k_scan_bwd_join(ScanArgs a) {
  constexpr int AHEAD = 16;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x, DN = (int64_t)a.D * a.N;
  if (i >= a.B * DN) return;
  const int64_t b = i / DN, dn = i - b * DN;
  const int d = (int)(dn / a.N), chunks = a.chunks;
  const bool back = blockIdx.y;
  const float A2 = a.A[dn] * kLog2e;
  float* part = (back ? a.qc : a.hc) + b * chunks * DN + dn;
  const float* dts = a.dts + b * chunks * (int64_t)a.D + d;
  const float* start = back ? a.gstate_out : a.state;
  float v = start ? start[i] : 0.f;
  for (int c0 = 0; c0 < chunks; c0 += AHEAD) {
    float e[AHEAD], t[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int c = min(c0 + k, chunks - 1), at = back ? chunks - 1 - c : c;
      e[k] = part[at * DN];
      t[k] = dts[(int64_t)at * a.D];
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int c = c0 + k, at = back ? chunks - 1 - c : c;
      if (c < chunks) {
        part[at * DN] = v;
        v = fmaf(exp2_fast(A2 * t[k]), v, e[k]);
      }
    }
  }
  if (back && a.gstate) a.gstate[i] = v;
}

// x + its partner across the wave's halves, for two values at once: the lower
// half holds x's sums, the upper half y's.
__device__ __forceinline__ float fold_halves(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same across neighbouring rows: even rows hold x's sums, odd rows y's.
__device__ __forceinline__ float fold_rows(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// W waves to a workgroup: 4, or 8 where a workgroup's LDS fills a compute unit.
template <int IOT, int W>
__global__ __launch_bounds__(64 * W, W == 8 ? 2 : 3) void k_scan_bwd(ScanArgs a) {
  constexpr int THREADS = 64 * W, TC = 4 * W;
  extern __shared__ float lds[];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane >> 4, l = lane & 15;
  const int N = a.N, Dg = a.D / a.G, tiles = (Dg + TC - 1) / TC, per = (tiles + a.splits - 1) / a.splits;
  int id = blockIdx.x;
  const int split = id % a.splits; id /= a.splits;
  const int c = id % a.chunks; id /= a.chunks;
  const int g = id % a.G, b = id / a.G;
  const int64_t L = a.L;
  const int len = seq_length(a, b), t0 = c * CH, t = t0 + 8 * l, m = len - t;
  const int room = (int)min(L - t, (int64_t)8);      // this lane's steps in the array (<= 0: none)
  const int64_t bc = ((int64_t)b * a.G + g) * N * L;
  const int64_t total = (int64_t)a.B * a.D * L, bc_total = (int64_t)a.B * a.G * N * L;
  float* sB = lds;                                             // [N][128]
  float* sC = sB + N * CH;                                     // [N][128]
  f32x4v* sG = reinterpret_cast<f32x4v*>(sC + N * CH);         // [N][64 lanes]: sums over channels
  f32x4v* sS = sG + N * 64;                                    // [TC][N]: A, start state, end carry, gA's part
  for (int i = tid; i < 2 * N * 16; i += THREADS) {
    const int v = i & 15, n = i >> 4;
    const bool isC = n >= N;
    float x[8];
    widen8<IOT>(ld8n<IOT>(isC ? a.Cm : a.Bm, bc + (int64_t)(isC ? n - N : n) * L + t0 + 8 * v, len - t0 - 8 * v, bc_total), x);
    stage8(lds + n * CH, v, x);
  }
  for (int i = tid; i < N * 64; i += THREADS) sG[i] = f32x4v{0.f, 0.f, 0.f, 0.f};

  __syncthreads();                                    // B, C and the zeros are there; the turns order the rest
  const int share = (N + W - 1) / W;
  int tile_end = min(tiles, (split + 1) * per);
  if (t0 >= len) {
    // Behind the sequence: zeros, without a look at the state, which an empty
    // sequence only hands on and which may hold anything.
    const int first = split * per * TC, count = min(Dg, tile_end * TC) - first;
    const int64_t ch = (int64_t)b * a.D + g * Dg + first, rc = ((int64_t)b * a.chunks + c) * a.D + g * Dg + first;
    const float none[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = tid; i < count * N; i += THREADS) {
      a.hc[rc * N + i] = 0.f;
      if (a.chunks == 1 && a.gstate) a.gstate[ch * N + i] = a.gstate_out ? a.gstate_out[ch * N + i] : 0.f;
    }
    for (int i = tid; i < count; i += THREADS) a.ps[rc + i] = a.pb[rc + i] = 0.f;
    if (room > 0)                                     // THREADS is a multiple of 16: a thread keeps its steps
      for (int i = tid >> 4; i < count; i += THREADS / 16) {
        const int64_t at = (ch + i) * L + t;
        if (a.z) st8n<IOT>(a.gz, at, none, room);
        st8n<IOT>(a.gu, at, none, room);
        st8n<IOT>(a.gdelta, at, none, room);
      }
    tile_end = 0;                                     // no tile; gB and gC below
  }
  for (int tile = split * per; tile < tile_end; ++tile) {
    const int cw = wave * 4 + row, dg = tile * TC + cw;
    const bool live = dg < Dg;
    const int d = g * Dg + (live ? dg : Dg - 1), mm = live ? m : 0;
    const int64_t at = ((int64_t)b * a.D + d) * L + t, r = ((int64_t)b * a.chunks + c) * a.D + d;
    const Raw8<IOT> ru = ld8n<IOT>(a.u, at, mm, total), rd = ld8n<IOT>(a.delta, at, mm, total), rg = ld8n<IOT>(a.gy, at, mm, total);
    Raw8<IOT> rz = zero8<IOT>();
    if (a.z) rz = ld8n<IOT>(a.z, at, mm, total);
    // this wave's channels only: no other wave reads or writes these words
    for (int n = l; n < N; n += 16) {
      const float A = a.A[(int64_t)d * N + n];
      float h = 0.f, q = 0.f;
      if (live) {
        const int64_t i = a.chunks > 1 ? r * N + n : ((int64_t)b * a.D + d) * N + n;
        const float *hp = a.chunks > 1 ? a.hc : a.state, *qp = a.chunks > 1 ? a.qc : a.gstate_out;
        if (hp) h = hp[i];
        if (qp) q = qp[i];
      }
      sS[cw * N + n] = f32x4v{A, h, q, 0.f};
    }
    // read by the row's other lanes: a wave's LDS accesses are done in order
    __builtin_amdgcn_wave_barrier();
    const float bias = a.dbias ? a.dbias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    float u[8], dt[8], du[8], gy[8], y[8], s1[8], s2[8];
    steps8<IOT>(a, ru, rd, bias, mm, u, dt);
    widen8<IOT>(rg, gy);
    if (a.z) {
      float z[8];
      widen8<IOT>(rz, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) gy[i] *= z[i] * sigmoid_f(z[i]);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = skip * u[i];
      du[i] = u[i] * dt[i];
      sum += dt[i];
      s1[i] = s2[i] = 0.f;
    }
    // the waves take the states in turn, so that each sum over channels
    // has one writer at a time and one order
    for (int turn = 0; turn < W; ++turn) {
      const int first = ((turn + wave) & (W - 1)) * share, last = min(N, first + share);
      for (int n = first; n < last; ++n) {
        const f32x4v sc = sS[cw * N + n];
        const float A = sc[0], A2 = A * kLog2e;
        float x[8], al[8], cc[8], h[8];
        fetch8(sB + n * CH, l, x);
        fetch8(sC + n * CH, l, cc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          al[i] = exp2_fast(dt[i] * A2);
          h[i] = du[i] * x[i];
        }
        float H = h[0], Q = al[7] * (cc[7] * gy[7]);
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          H = fmaf(al[i], H, h[i]);
          Q = al[7 - i] * fmaf(cc[7 - i], gy[7 - i], Q);
        }
        const float P = exp2_fast(A2 * sum);
        H = fmaf(P, l == 0 ? sc[1] : 0.f, H);
        Q = fmaf(P, l == 15 ? sc[2] : 0.f, Q);
        row_scan(P, H);
        row_scan_back(P, Q);
        // moved in all lanes, then chosen: the state before this lane's steps, the carry from behind them
        const float hm = row_shr<1>(H), qm = row_shl<1>(Q);
        const float hb = l == 0 ? sc[1] : hm;
        float q = l == 15 ? sc[2] : qm;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[i] = fmaf(al[i], i ? h[i - 1] : hb, h[i]);
          y[i] = fmaf(h[i], cc[i], y[i]);
        }
        float gA = 0.f;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const float gh = fmaf(cc[i], gy[i], q);
          q = al[i] * gh;
          s1[i] = fmaf(gh, x[i], s1[i]);
          const float w = q * (i ? h[i - 1] : hb);
          s2[i] = fmaf(w, A, s2[i]);
          gA = fmaf(w, dt[i], gA);
          cc[i] = fold_halves(gh * du[i], h[i] * gy[i]);
        }
        f32x4v acc = sG[n * 64 + lane];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += fold_rows(cc[2 * k], cc[2 * k + 1]);
        sG[n * 64 + lane] = acc;
        gA = row_sum(gA);
        if (l == 0) {
          sS[cw * N + n][3] = gA;
          if (a.chunks == 1 && a.gstate && live) a.gstate[((int64_t)b * a.D + d) * N + n] = q;
        }
      }
      __syncthreads();
    }
    // the chunk's parts of the sums over time, and the lane's own gradients
    for (int n = l; n < N; n += 16)
      if (live) a.hc[r * N + n] = sS[cw * N + n][3];
    float gz[8], sk = 0.f, sb = 0.f;
    if (a.z) {
      float z[8], g0[8];
      widen8<IOT>(rz, z);
      widen8<IOT>(rg, g0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sg = sigmoid_f(z[i]);
        gz[i] = g0[i] * y[i] * (sg * fmaf(z[i], 1.f - sg, 1.f));
      }
    }
    float pre[8];
    widen8<IOT>(rd, pre);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sk = fmaf(gy[i], u[i], sk);
      float gd = fmaf(s1[i], u[i], s2[i]);
      if (a.softplus) gd *= sigmoid_f(pre[i] + bias);
      gd = i < mm ? gd : 0.f;
      s2[i] = gd;
      sb += gd;
      s1[i] = fmaf(s1[i], dt[i], skip * gy[i]);
    }
    if (mm < 8) {                                     // zeros behind the sequence, whatever its state and carry are
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (a.z) gz[i] = i < mm ? gz[i] : 0.f;
        s1[i] = i < mm ? s1[i] : 0.f;
      }
    }
    sk = row_sum(sk);
    sb = row_sum(sb);
    if (live) {
      if (l == 0) { a.ps[r] = sk; a.pb[r] = sb; }
      if (room > 0) {
        if (a.z) st8n<IOT>(a.gz, at, gz, room);
        st8n<IOT>(a.gu, at, s1, room);
        st8n<IOT>(a.gdelta, at, s2, room);
      }
    }
  }
  // sums over channels: lane (row r, column l) of a state holds, in word k,
  // step 8 l + 2 k + (r & 1) of gB (r < 2) or gC
  __syncthreads();
  const float* sg = reinterpret_cast<const float*>(sG);
  for (int i = tid; i < 2 * N * CH; i += THREADS) {
    const int tt = i & (CH - 1), n = (i >> 7) % N, isC = (i >> 7) / N;
    if (t0 + tt >= L) continue;
    const float v = t0 + tt < len ? sg[(n * 64 + (isC * 2 + (tt & 1)) * 16 + (tt >> 3)) * 4 + ((tt & 7) >> 1)] : 0.f;
    const int64_t o = bc + (int64_t)n * L + t0 + tt;
    if (a.splits > 1) a.gbc[((int64_t)(split * 2 + isC) * a.B * a.G) * N * L + o] = v;
    else st1<IOT>(isC ? a.gC : a.gB, o, v);
  }
}

// The sums that are left, in one launch: the first `time_groups` workgroups
// add up the chunks' parts of gA, gskip and gdelta_bias, the others the
// splits' parts of gB and gC (256 values at a time, 4 threads to a value,
// whose loads are in flight eight at a time).
template <int IOT>
__global__ __launch_bounds__(SUM_THREADS) void k_scan_bwd_sums(ScanArgs a, int time_groups) {
  __shared__ float lds[32][33];
  if ((int)blockIdx.x < time_groups) {
    const int64_t DN = (int64_t)a.D * a.N, rows = (int64_t)a.B * a.chunks;
    // columns: gA's D*N, then gskip's D, then gdelta_bias's D
    const int64_t i = blockIdx.x * (int64_t)32 + (threadIdx.x & 31);
    const float* src = nullptr;
    int64_t stride = a.D;
    float* dst = nullptr;
    if (i < DN) { src = a.hc + i; stride = DN; dst = a.gA + i; }
    else if (i < DN + a.D && a.gskip) { src = a.ps + (i - DN); dst = a.gskip + (i - DN); }
    else if (i >= DN + a.D && i < DN + 2 * a.D && a.gdbias) { src = a.pb + (i - DN - a.D); dst = a.gdbias + (i - DN - a.D); }
    const float v = column_sum(src, rows, stride, lds);
    if (threadIdx.x < 32 && dst) *dst = v;
    return;
  }
  float* part = &lds[0][0];                           // [3][256]
  const int64_t n = (int64_t)a.B * a.G * a.N * a.L;
  const int c = threadIdx.x & 255, k = threadIdx.x >> 8;
  for (int64_t first = ((int64_t)blockIdx.x - time_groups) * 256; first < 2 * n;
       first += ((int64_t)gridDim.x - time_groups) * 256) {
    const int64_t i = first + c;
    float v = 0.f;
    if (i < 2 * n) {
      const float* p = a.gbc + i;
      int s = k;
      for (; s + 28 < a.splits; s += 32) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = p[(s + 4 * j) * 2 * n];
#pragma unroll
        for (int j = 0; j < 8; ++j) v += w[j];
      }
      for (; s < a.splits; s += 4) v += p[s * 2 * n];
    }
    if (k > 0) part[(k - 1) * 256 + c] = v;
    __syncthreads();
    if (k == 0 && i < 2 * n) {
      v = (v + part[c]) + (part[256 + c] + part[512 + c]);
      if (i < n) st1<IOT>(a.gB, i, v);
      else st1<IOT>(a.gC, i - n, v);
    }
    __syncthreads();
  }
}

template <int IOT>
hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
  const unsigned wgs = (unsigned)((int64_t)a.B * a.G * a.chunks * a.splits);
  const size_t bc = (size_t)2 * a.N * CH * 4;
  hipError_t e;
  if (a.chunks > 1) {
    k_scan_bwd_ends<IOT><<<dim3(wgs), SCAN_THREADS, bc, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    k_scan_bwd_join<<<dim3((unsigned)(((int64_t)a.B * a.D * a.N + 255) / 256), 2), 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const size_t sums = (size_t)a.N * 64 * 16, tile = scan_backward_tile(a.N, a.D / a.G);
  const size_t state = tile * a.N * 16;
  if (tile == 32) k_scan_bwd<IOT, 8><<<dim3(wgs), 512, bc + sums + state, s>>>(a);
  else k_scan_bwd<IOT, 4><<<dim3(wgs), 256, bc + sums + state, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int time_groups = (int)(((int64_t)a.D * (a.N + 2) + 31) / 32);
  const int64_t n = (int64_t)2 * a.B * a.G * a.N * a.L;
  const int64_t bc_groups = a.splits > 1 ? min((n + 255) / 256, (int64_t)1 << 18) : 0;
  k_scan_bwd_sums<IOT><<<dim3((unsigned)(time_groups + bc_groups)), SUM_THREADS, 0, s>>>(a, time_groups);
  return hipGetLastError();
}

}  // namespace

hipError_t selective_scan(const ScanArgs& a, hipStream_t s) {
  if (a.split > 1) return a.io ? launch_scan_nv<1, 4>(a, s) : launch_scan_nv<0, 4>(a, s);
  return a.io ? launch_scan_nv<1, 1>(a, s) : launch_scan_nv<0, 1>(a, s);
}

hipError_t selective_scan_step(const ScanArgs& a, hipStream_t s) {
  int lw = 0;
  while ((4 << lw) < a.N) ++lw;
  const int64_t threads = ((int64_t)a.B * a.D) << lw;
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (a.io) k_scan_step<1><<<grid, 256, 0, s>>>(a, 1 << lw, lw, a.state_out);
  else k_scan_step<0><<<grid, 256, 0, s>>>(a, 1 << lw, lw, a.state_out);
  return hipGetLastError();
}

hipError_t selective_scan_backward(const ScanArgs& a, hipStream_t s) {
  return a.io ? launch_scan_backward<1>(a, s) : launch_scan_backward<0>(a, s);
}

}  // namespace hyena
