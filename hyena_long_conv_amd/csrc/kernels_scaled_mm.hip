// kernels_scaled_mm.hip -- matrix product of e4m3 operands with a scale for
// each 128 values along k of a left row and for each 128 x 128 block of the
// right operand:
//   out[m][n] = sum_kb scales[m][kb] wscales[n / 128][kb]
//                 sum_{k in kb} q[m][k] wq[n][k]  + bias[n].
//
// 8192 x 8192 x 2048 to bf16: 143 us, 1.9 PFLOP/s (149 channel-major with a
// bias, 171 at the profiler's clock, where the matrix units are busy 44% of
// the cycles and the vector units, which scale and add every block's products,
// 46%); 2.15 at K = 8192.  (A library product without block scales reaches 2.6
// at 8192^3.)  To fp32, through the bf16 instructions: 292 us, 0.94 PFLOP/s;
// 227 us at the 1.21 of a library product in bf16.
#include <hip/hip_runtime.h>

#include "ssm.hpp"
#include "ssm_device.hpp"

namespace hyena {
namespace {

constexpr int KS = 128;                            // k of a step: one block of scales

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

// The sum over one block of 128: with SUM32 in fp32, the codes widened to
// bf16 and multiplied by the bf16 instructions, otherwise by the 8-bit ones at
// twice the rate.  Those add up 8 neighbouring products at 2^-13 of the
// largest one, the bits below cut towards zero (2^16 beside a product of 7 in
// its group loses the 7; the groups' sums keep some 23 bits).  What is lost of
// 8 products is below 7 * 2^-13 of the largest, 2^-10, while the codes of
// that product are each rounded by up to 2^-4 of it.  On normal data the sums
// are off by 1.4e-5 of the result's norm (1e-8 with SUM32), a bf16 output's
// rounding by 1.7e-3.  So: 8-bit sums for tiles with a bf16 output, which are
// bound by the matrix units (8192 x 8192 x 2048: 143 us, 294 with SUM32), and
// SUM32 for an fp32 output and for few rows, which are bound by the weights'
// bytes (16 rows of 4096 x 2048: 5.2 us, 5.3 with SUM32; 64 rows 9.3 and 9.8).
template <bool SUM32>
__device__ __forceinline__ f32x4v mfma128(i32x8 a, i32x8 b) {
  f32x4v z = {0.f, 0.f, 0.f, 0.f};
  if constexpr (!SUM32) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(a[2 * i], a[2 * i + 1]),
                                                  widen_codes(b[2 * i], b[2 * i + 1]), z, 0, 0, 0);
    return z;
  }
}

// ------------------------------------------------------------ tiles in LDS
//
// A workgroup of WM x WN waves computes BM = 16 IM WM rows by BN = 16 IN WN
// columns, one block of 128 along k at a time.  A step's operands go from
// global memory straight to one of two LDS stages while the other one is
// multiplied, and so do its rows' scales.  An LDS row is 128 bytes, 8 words
// of 16; word c of row r lies in slot c ^ swizzle(r).  A read takes word 2h or
// 2h + 1 of 16 rows; two rows span the 64 banks, so the 16 lanes of a turn
// have to hold all 8 slots of even and of odd rows.  The right operand's rows are the matrix instruction's rows: a lane
// then holds 4 neighbouring n of one m, one scale serves its 4 values, and
// wscales is one value for a wave, whose n stay in one block of 128.

typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr uint32_t OOB = 0x7ffffff0u;              // behind every buffer: reads as zeros

// Pairs of rows go through the 8 slots; the order also keeps turns apart that
// join 8 rows of one h with the 8 others of h + 1 (pairs 0, 1, 6, 7 and
// 2, 3, 4, 5 hold slot sets that are closed under ^ 2).
__device__ __forceinline__ int swizzle(int r) {
  return ((r >> 1) & 1) | ((r >> 2) & 2) | ((((r >> 2) ^ (r >> 3)) & 1) << 2);
}

template <int ROWS, int WAVES>
struct TileLoads {
  static constexpr int J = ROWS * 8 / 64 / WAVES;  // instructions of a wave: 8 rows each
  uint32_t off[J];
  uint32_t kq[J];
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ void init(const uint8_t* base, int64_t row0, int64_t rows, int K, int wave, int lane) {
    const int64_t left = rows - row0;
    const int have = left > ROWS ? ROWS : (int)left;
    rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base + row0 * K), (short)0, have * K, 0x00020000);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int s = (J * wave + j) * 64 + lane, r = s >> 3, c = (s & 7) ^ swizzle(r);
      kq[j] = 16u * c;
      off[j] = r < have ? (uint32_t)(r * K) + kq[j] : OOB;
    }
  }
  // The step at k0 into the stage's rows; K a multiple of 16, words behind it are zeros.
  __device__ __forceinline__ void issue(unsigned char* dst, int wave, int k0, int K) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t o = (uint32_t)k0 + kq[j] < (uint32_t)K && off[j] != OOB ? off[j] + (uint32_t)k0 : OOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(dst + (J * wave + j) * 1024), 16, (int)o, 0, 0, 0);
    }
  }
};

__device__ __forceinline__ i32x8 tile_operand(const unsigned char* rows, int l, int h) {
  const unsigned char* r = rows + l * KS;
  const i32x4 a = *reinterpret_cast<const i32x4*>(r + 16 * ((2 * h) ^ swizzle(l)));
  const i32x4 b = *reinterpret_cast<const i32x4*>(r + 16 * ((2 * h + 1) ^ swizzle(l)));
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Eight consecutive outputs of a row or, channel-major, of a channel.
template <int IOT, bool CM>
__device__ __forceinline__ void put8(const ScaledArgs& a, int64_t m, int64_t n, const float (&v)[8]) {
  if constexpr (!CM) {
    if (m < a.M && n < a.N) st8n<IOT>(a.out, m * a.N + n, v, (int)min(a.N - n, (int64_t)8));
  } else {
    if (n >= a.N || m >= a.M) return;
    const uint32_t L = (uint32_t)a.L, b = (uint32_t)m / L, t = (uint32_t)m - b * L;
    if (t + 8 <= L) {
      st8n<IOT>(a.out, ((int64_t)b * a.N + n) * a.L + t, v, 8);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {                     // across the end of a sequence
      const uint32_t me = (uint32_t)m + e, be = me / L;
      if (me < a.M) st1<IOT>(a.out, ((int64_t)be * a.N + n) * a.L + (me - be * L), v[e]);
    }
  }
}

// Workgroup -> tile: an XCD (workgroup id mod 8) takes a contiguous part of
// the tiles in an order that goes through panels of 8 tiles along m, so that
// the workgroups of an XCD share rows of both operands in its L2.
__device__ __forceinline__ bool tile_of(int64_t tm, int64_t tn, int64_t& m, int64_t& n) {
  const int64_t per = (tm * tn + 7) / 8, k = blockIdx.x / 8, t = (blockIdx.x & 7) * per + k;
  if (k >= per || t >= tm * tn) return false;
  const int64_t panel = t / (8 * tn), left = tm - panel * 8, wide = left < 8 ? left : 8, u = t - panel * 8 * tn;
  n = u / wide;
  m = panel * 8 + (u - n * wide);
  return true;
}

template <int IOT, bool CM, int IM, int IN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_scaled_mm(ScaledArgs a) {
  constexpr int BM = 16 * IM * WM, BN = 16 * IN * WN, STAGE = (BM + BN) * KS + BM * 4, W = WM * WN;
  static_assert(128 % (16 * IN) == 0, "a wave's n lie in one block of wscales");
  extern __shared__ __attribute__((aligned(1024))) unsigned char stage[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15, h = lane >> 4;
  const int K = (int)a.K, kb = (K + KS - 1) / KS;
  int64_t mt, nt;
  if (!tile_of((a.M + BM - 1) / BM, (a.N + BN - 1) / BN, mt, nt)) return;
  const int64_t m0 = mt * BM, n0 = nt * BN;
  const int wm = wave % WM, wn = wave / WM;
  TileLoads<BM, W> lx;
  TileLoads<BN, W> lw;
  lx.init(a.q, m0, a.M, K, wave, lane);
  lw.init(a.wq, n0, a.N, K, wave, lane);
  // scales of the tile's rows: waves 0 .. BM / 64 - 1 fetch 64 each; the wave's block of wscales
  const __amdgpu_buffer_rsrc_t rss = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(a.scales + m0 * kb), (short)0, (int)min(a.M - m0, (int64_t)BM) * kb * 4, 0x00020000);
  const uint32_t so = (uint32_t)(wave * 64 + lane) * (uint32_t)kb * 4u;
  const int64_t nw = n0 + wn * IN * 16;
  const float* sw = a.wscales + min(nw, a.N - 1) / 128 * kb;
  auto issue = [&](int b) {
    unsigned char* st = stage + (b & 1) * STAGE;
    lx.issue(st, wave, b * KS, K);
    lw.issue(st + BM * KS, wave, b * KS, K);
    // the scalar offset is outside the buffer's bounds check, so it stays in the row behind K
    if (wave < BM / 64)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rss, (lds_ptr_t)(st + (BM + BN) * KS + wave * 256), 4, (int)so,
                                               4 * min(b, kb - 1), 0, 0);
  };

  f32x4v acc[IM][IN];
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < IN; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
  float swn = sw[0];
  issue(0);
  for (int b = 0; b < kb; ++b) {
    // this wave's loads of the step are in LDS and its reads of the other
    // stage are done; the barrier makes both hold for all waves
    __builtin_amdgcn_s_waitcnt(0x0070);               // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    const unsigned char* X = stage + (b & 1) * STAGE + wm * IM * 16 * KS;
    const unsigned char* Y = stage + (b & 1) * STAGE + BM * KS + wn * IN * 16 * KS;
    const float* S = reinterpret_cast<const float*>(stage + (b & 1) * STAGE + (BM + BN) * KS) + wm * IM * 16 + l;
    float sc[IM];
#pragma unroll
    for (int i = 0; i < IM; ++i) sc[i] = S[16 * i] * swn;
    swn = sw[min(b + 1, kb - 1)];
    i32x8 w[IN], x = tile_operand(X, l, h);
#pragma unroll
    for (int j = 0; j < IN; ++j) w[j] = tile_operand(Y + j * 16 * KS, l, h);
    // The products of one row of tiles run while the one before is scaled and
    // added: a product is ready some 16 cycles after it was issued.  The first
    // ones start on the first operands, the others' reads follow between them,
    // then the next step's loads (behind K they write zeros that no one reads).
    f32x4v p[2][IN];
    i32x8 next = x;
    if constexpr (IM > 1) next = tile_operand(X + 16 * KS, l, h);
#pragma unroll
    for (int j = 0; j < IN; ++j) p[0][j] = mfma128<IOT == 0>(w[j], x);
    if constexpr (IOT == 1) {
      __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
      for (int j = 0; j < IN; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, IM, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    issue(b + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 1; i < IM; ++i) {
      x = next;
      if (i + 1 < IM) next = tile_operand(X + (i + 1) * 16 * KS, l, h);
#pragma unroll
      for (int j = 0; j < IN; ++j) {
        p[i & 1][j] = mfma128<IOT == 0>(w[j], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i - 1][j][e] = fmaf(p[(i - 1) & 1][j][e], sc[i - 1], acc[i - 1][j][e]);
      }
    }
#pragma unroll
    for (int j = 0; j < IN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[IM - 1][j][e] = fmaf(p[(IM - 1) & 1][j][e], sc[IM - 1], acc[IM - 1][j][e]);
    if constexpr (IOT == 1) {                         // that order, for the instruction scheduler
#pragma unroll
      for (int i = 1; i < IM; ++i) {
        if (i + 1 < IM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int j = 0; j < IN; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
      }
      __builtin_amdgcn_sched_group_barrier(0x002, 4 * IN, 0);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0070);                 // vmcnt(0): nothing more lands in LDS

  // Out through LDS, each wave its own part, 16 rows (or 16 IM tokens of 16
  // channels) at a time, so that global stores are whole words of a row.
  __syncthreads();
  float* ep = reinterpret_cast<float*>(stage) + wave * (CM ? 16 * (16 * IM + 4) : 16 * (16 * IN + 4));
  if constexpr (!CM) {
    constexpr int LD = 16 * IN + 4;
#pragma unroll
    for (int i = 0; i < IM; ++i) {
#pragma unroll
      for (int j = 0; j < IN; ++j) *reinterpret_cast<f32x4v*>(ep + l * LD + 16 * j + 4 * h) = acc[i][j];
      __builtin_amdgcn_wave_barrier();
      for (int s = lane; s < 16 * 2 * IN; s += 64) {
        const int r = s / (2 * IN), c = 8 * (s - r * 2 * IN);
        const int64_t n = nw + c;
        float v[8], bv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ep[r * LD + c + e];
        if (a.bias) {
          widen8<0>(ld8n<0>(a.bias, n, (int)min(a.N - n, (int64_t)8), a.N), bv);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += bv[e];
        }
        put8<IOT, false>(a, m0 + (wm * IM + i) * 16 + r, n, v);
      }
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    constexpr int LD = 16 * IM + 4;
#pragma unroll
    for (int j = 0; j < IN; ++j) {
#pragma unroll
      for (int i = 0; i < IM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ep[(4 * h + e) * LD + 16 * i + l] = acc[i][j][e];
      __builtin_amdgcn_wave_barrier();
      for (int s = lane; s < 16 * 2 * IM; s += 64) {
        const int r = s / (2 * IM), c = 8 * (s - r * 2 * IM);
        const int64_t n = nw + 16 * j + r;
        const float bias = a.bias && n < a.N ? a.bias[n] : 0.f;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ep[r * LD + c + e] + bias;
        put8<IOT, true>(a, m0 + wm * IM * 16 + c, n, v);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// ---------------------------------------------------------------- few rows
//
// Up to 64 rows: the weights' bytes are the call.  A workgroup takes 16
// columns and splits k over its 8 waves; a lane loads its operands straight
// into registers (a row of 128 bytes is one line), and the waves' sums meet
// in LDS.  1, 16, 32 and 64 rows of 4096 x 2048: 4.4, 5.3, 6.7 and 9.8 us (one
// round of loads to a wave, so latency counts: 1.6 TB/s with 16 rows), where
// tiles of 64 x 64 take 9 us, and far more with fewer columns, for want of
// workgroups.
template <int IOT, bool CM, int IM>
__global__ __launch_bounds__(512) void k_scaled_mm_rows(ScaledArgs a) {
  __shared__ float part[8][IM][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15, h = lane >> 4;
  const int64_t K = a.K, kb = (K + KS - 1) / KS, n0 = blockIdx.x * (int64_t)16;
  const uint8_t* w = a.wq + min(n0 + l, a.N - 1) * K + 32 * h;
  const float* sw = a.wscales + n0 / 128 * kb;
  f32x4v acc[IM];
#pragma unroll
  for (int i = 0; i < IM; ++i) acc[i] = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int64_t b0 = wave; b0 < kb; b0 += 16) {        // two blocks' loads in flight
    i32x8 y[2], x[2][IM];
    float sc[2][IM];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t b = b0 + 8 * u, bs = min(b, kb - 1);    // zeros behind K
      y[u] = operand(w, b * KS, K - 32 * h);
#pragma unroll
      for (int i = 0; i < IM; ++i) {
        const int64_t m = min((int64_t)(16 * i + l), a.M - 1);
        x[u][i] = operand(a.q + m * K + 32 * h, b * KS, K - 32 * h);
        sc[u][i] = a.scales[m * kb + bs] * sw[bs];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < IM; ++i) {
        const f32x4v p = mfma128<true>(y[u], x[u][i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(p[e], sc[u][i], acc[i][e]);
      }
  }
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][i][l][4 * h + e] = acc[i][e];
  __syncthreads();
  for (int s = tid; s < IM * 256; s += 512) {
    // neighbouring threads: neighbouring n, or tokens where those are contiguous
    const int i = s >> 8, r = CM ? s & 15 : (s >> 4) & 15, c = CM ? (s >> 4) & 15 : s & 15;
    const int64_t m = 16 * i + r, n = n0 + c;
    if (m >= a.M || n >= a.N) continue;
    float v = part[0][i][r][c];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += part[k][i][r][c];
    if (a.bias) v += a.bias[n];
    st1<IOT>(a.out, CM ? (m / a.L * a.N + n) * a.L + m % a.L : m * a.N + n, v);
  }
}

template <int IOT, bool CM, int IM, int IN, int WM, int WN>
hipError_t launch_tiles(const ScaledArgs& a, hipStream_t s) {
  constexpr int BM = 16 * IM * WM, BN = 16 * IN * WN;
  constexpr size_t stages = 2 * ((BM + BN) * KS + BM * 4), out = (size_t)WM * WN * 16 * (16 * (CM ? IM : IN) + 4) * 4;
  const int64_t tiles = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  k_scaled_mm<IOT, CM, IM, IN, WM, WN>
      <<<dim3((unsigned)((tiles + 7) / 8 * 8)), 64 * WM * WN, stages > out ? stages : out, s>>>(a);
  return hipGetLastError();
}

template <int IOT, bool CM>
hipError_t launch_rows(const ScaledArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16));
  if (a.M <= 16) k_scaled_mm_rows<IOT, CM, 1><<<grid, 512, 0, s>>>(a);
  else if (a.M <= 32) k_scaled_mm_rows<IOT, CM, 2><<<grid, 512, 0, s>>>(a);
  else k_scaled_mm_rows<IOT, CM, 4><<<grid, 512, 0, s>>>(a);
  return hipGetLastError();
}

template <int IOT, bool CM>
hipError_t launch_product(const ScaledArgs& a, hipStream_t s) {
  const auto tiles = [&](int64_t bm, int64_t bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  // The largest tiles that still fill the chip.  N = 4096, K = 2048, bf16, in
  // tiles of 256, 128 and 64: 4096 rows 38, 49 and 64 us (256 tiles of 256),
  // 2048 rows 33, 26 and 33 (128 of them; 512 of 128), 1024 rows 30, 18.6 and
  // 17.3 (256 of 128).  The two smaller ones' products lie in accumulator
  // registers and are each read back from there (64 and 16 reads to a step),
  // which these times include.
  if (a.M <= 64) return launch_rows<IOT, CM>(a, s);
  if constexpr (IOT == 1) {                           // widened operands leave no registers for these
    if (tiles(256, 256) >= 192) return launch_tiles<IOT, CM, 8, 4, 2, 4>(a, s);
  }
  if (tiles(128, 128) >= 384) return launch_tiles<IOT, CM, 4, 4, 2, 2>(a, s);
  return launch_tiles<IOT, CM, 2, 2, 2, 2>(a, s);
}

}  // namespace

hipError_t scaled_matmul(const ScaledArgs& a, hipStream_t s) {
  if (a.channel_major) return a.io ? launch_product<1, true>(a, s) : launch_product<0, true>(a, s);
  return a.io ? launch_product<1, false>(a, s) : launch_product<0, false>(a, s);
}

}  // namespace hyena
