// api_ssm.cpp -- the extern "C" entry points of the state-space block's
// operators (include/hyena.h): every argument is checked on the host before
// anything is enqueued, and nothing is allocated.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "hyena.h"
#include "ssm.hpp"

using namespace hyena;

static_assert(HYENA_MAX_SHORT == 16, "the short convolution's kernels hold at most 16 taps");
static_assert(HYENA_MAX_STATE == 64, "the scan's kernels hold at most 64 states");

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;   // B * D
constexpr int64_t kMaxDim = (int64_t)1 << 20;
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads in a launch (2^32 threads)

// Arrays of a call: null checks are the caller's, absent ones are skipped.
struct Span {
  const void* p;
  int64_t bytes;
  int64_t align;
};

hyena_status check_spans(const Span* out, int no, const Span* in, int ni) {
  for (int i = 0; i < no + ni; ++i) {
    const Span& s = i < no ? out[i] : in[i - no];
    if (s.p && reinterpret_cast<uintptr_t>(s.p) % (uintptr_t)s.align) return HYENA_ERR_ALIGN;
  }
  const auto meet = [](const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
  };
  for (int i = 0; i < no; ++i) {
    for (int k = 0; k < ni; ++k)
      if (meet(out[i], in[k])) return HYENA_ERR_ALIAS;
    for (int k = 0; k < i; ++k)
      if (meet(out[i], out[k])) return HYENA_ERR_ALIAS;
  }
  return HYENA_OK;
}

template <int NO, int NI>
hyena_status check_spans(const Span (&out)[NO], const Span (&in)[NI]) {
  return check_spans(out, NO, in, NI);
}

bool io_ok(hyena_dtype io) { return io == HYENA_FP32 || io == HYENA_BF16; }
int64_t size_of(hyena_dtype io) { return io == HYENA_FP32 ? 4 : 2; }
bool batch_ok(int64_t B, int64_t D, int64_t L) {
  return B >= 1 && B <= kMaxDim && D >= 1 && D <= kMaxDim && B * D <= kMaxRows && L >= 1 && L <= HYENA_MAX_L;
}
hyena_status from_hip(hipError_t e) { return e == hipSuccess ? HYENA_OK : HYENA_ERR_HIP; }

}  // namespace

extern "C" {

// ------------------------------------------------------- short convolution

static hyena_status conv_args(const hyena_short_conv_params* p, hyena_dtype io, int64_t L, ConvArgs* a) {
  if (!p || !p->w) return HYENA_ERR_NULL;
  if (!batch_ok(p->B, p->D, L) || p->T < 1 || p->T > HYENA_MAX_SHORT) return HYENA_ERR_SHAPE;
  if (p->silu != 0 && p->silu != 1) return HYENA_ERR_UNSUPPORTED;
  if (!io_ok(io)) return HYENA_ERR_UNSUPPORTED;
  if (conv_grid(p->B, p->D, L, kConvStep).groups > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  *a = ConvArgs{};
  a->w = p->w;
  a->bias = p->bias;
  a->B = (int)p->B;
  a->D = p->D;
  a->T = p->T;
  a->L = L;
  a->silu = p->silu;
  a->io = io == HYENA_BF16;
  return HYENA_OK;
}

hyena_status hyena_short_conv(const void* x, const hyena_short_conv_params* p, void* y, void* state_out,
                              hyena_dtype io, void* stream) {
  if (!x || !y) return HYENA_ERR_NULL;
  ConvArgs a;
  if (const hyena_status s = conv_args(p, io, p ? p->L : 1, &a)) return s;
  if (a.T == 1 && (p->state || state_out)) return HYENA_ERR_SHAPE;
  const int64_t e = size_of(io), act = p->B * a.D * a.L * e, st = p->B * a.D * (a.T - 1) * e;
  const Span out[] = {{y, act, 16}, {state_out, st, 16}};
  const Span in[] = {{x, act, 16}, {p->state, st, 16}, {p->w, (int64_t)a.D * a.T * 4, 4}, {p->bias, (int64_t)a.D * 4, 4},
                     {p->lengths, p->B * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.x = x;
  a.state = p->state;
  a.lengths = p->lengths;
  a.y = y;
  a.state_out = state_out;
  return from_hip(short_conv(a, (hipStream_t)stream));
}

hyena_status hyena_short_conv_step(const void* x, const hyena_short_conv_params* p, void* state, void* y,
                                   hyena_dtype io, void* stream) {
  if (!x || !y) return HYENA_ERR_NULL;
  ConvArgs a;
  if (const hyena_status s = conv_args(p, io, 1, &a)) return s;
  if (a.T == 1 && state) return HYENA_ERR_SHAPE;
  if (a.T > 1 && !state) return HYENA_ERR_NULL;
  const int64_t e = size_of(io), act = p->B * a.D * e;
  const Span out[] = {{y, act, 16}, {state, act * (a.T - 1), 16}};
  const Span in[] = {{x, act, 16}, {p->w, (int64_t)a.D * a.T * 4, 4}, {p->bias, (int64_t)a.D * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.x = x;
  a.y = y;
  a.state_out = state;
  return from_hip(short_conv_step(a, (hipStream_t)stream));
}

int64_t hyena_short_conv_backward_workspace_bytes(int64_t B, int32_t D, int32_t T, int64_t L) {
  if (!batch_ok(B, D, L) || T < 1 || T > HYENA_MAX_SHORT) return -1;
  return conv_backward_grid(B, D, L, T).parts * D * (T + 1) * 4;
}

hyena_status hyena_short_conv_backward(const void* x, const hyena_short_conv_params* p, const void* gy,
                                       const void* gstate_out, void* gx, float* gw, float* gbias, void* gstate,
                                       hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!x || !gy || !gx || !gw || !workspace) return HYENA_ERR_NULL;
  ConvArgs a;
  if (const hyena_status s = conv_args(p, io, p ? p->L : 1, &a)) return s;
  if (a.T == 1 && (p->state || gstate_out || gstate)) return HYENA_ERR_SHAPE;
  const int64_t e = size_of(io), act = p->B * a.D * a.L * e, st = p->B * a.D * (a.T - 1) * e;
  if (conv_backward_grid(p->B, a.D, a.L, a.T).parts * a.D > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const int64_t need = hyena_short_conv_backward_workspace_bytes(p->B, a.D, a.T, a.L);
  if (workspace_bytes < need) return HYENA_ERR_WORKSPACE;
  const Span out[] = {{gx, act, 16}, {gw, (int64_t)a.D * a.T * 4, 4}, {gbias, (int64_t)a.D * 4, 4}, {gstate, st, 16},
                      {workspace, need, 16}};
  const Span in[] = {{x, act, 16}, {gy, act, 16}, {gstate_out, st, 16}, {p->state, st, 16},
                     {p->w, (int64_t)a.D * a.T * 4, 4}, {p->bias, (int64_t)a.D * 4, 4}, {p->lengths, p->B * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.x = x;
  a.state = p->state;
  a.lengths = p->lengths;
  a.gy = gy;
  a.gstate_out = gstate_out;
  a.gx = gx;
  a.gw = gw;
  a.gbias = gbias;
  a.gstate = gstate;
  a.partial = static_cast<float*>(workspace);
  return from_hip(short_conv_backward(a, (hipStream_t)stream));
}

// ---------------------------------------------------------- selective scan

static hyena_status scan_args(const hyena_selective_scan_params* p, hyena_dtype io, int64_t L, ScanArgs* a) {
  if (!p || !p->u || !p->delta || !p->A || !p->Bm || !p->Cm) return HYENA_ERR_NULL;
  if (!batch_ok(p->B, p->D, L) || p->N < 1 || p->N > HYENA_MAX_STATE || p->G < 1 || p->G > p->D || p->D % p->G)
    return HYENA_ERR_SHAPE;
  if (p->softplus != 0 && p->softplus != 1) return HYENA_ERR_UNSUPPORTED;
  if (!io_ok(io)) return HYENA_ERR_UNSUPPORTED;
  *a = ScanArgs{};
  a->u = p->u;
  a->delta = p->delta;
  a->A = p->A;
  a->Bm = p->Bm;
  a->Cm = p->Cm;
  a->skip = p->skip;
  a->z = p->z;
  a->dbias = p->delta_bias;
  a->B = (int)p->B;
  a->D = p->D;
  a->G = p->G;
  a->N = p->N;
  a->L = L;
  a->softplus = p->softplus;
  a->io = io == HYENA_BF16;
  return HYENA_OK;
}

static int64_t scan_groups(const ScanArgs& a) {
  const int64_t tile = kScanTile / a.split;
  return (int64_t)a.B * a.G * ((a.D / a.G + tile - 1) / tile);
}

static int64_t scan_workspace(const ScanPlan& plan, int64_t B, int64_t D, int64_t N) {
  return plan.segs > 1 ? plan.segs * B * D * (N + 1) * 4 : 0;
}

int64_t hyena_selective_scan_workspace_bytes(int64_t B, int32_t D, int32_t N, int64_t L) {
  if (!batch_ok(B, D, L) || N < 1 || N > HYENA_MAX_STATE) return -1;
  return scan_workspace(scan_plan(B, D, N, L), B, D, N);
}

hyena_status hyena_selective_scan(const hyena_selective_scan_params* p, void* y, float* state_out, hyena_dtype io,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  if (!y) return HYENA_ERR_NULL;
  ScanArgs a;
  if (const hyena_status s = scan_args(p, io, p ? p->L : 1, &a)) return s;
  const ScanPlan plan = scan_plan(a.B, a.D, a.N, a.L);
  a.split = plan.split;
  a.segs = plan.segs;
  a.seg = plan.seg;
  if (scan_groups(a) * a.segs > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const int64_t need = scan_workspace(plan, a.B, a.D, a.N);
  if (need > 0 && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
  const int64_t e = size_of(io), rows = p->B * a.D, act = rows * a.L * e, bc = p->B * a.G * a.N * a.L * e;
  const int64_t st = rows * a.N * 4;
  const Span out[] = {{y, act, 16}, {state_out, st, 16}, {need > 0 ? workspace : nullptr, need, 16}};
  const Span in[] = {{a.u, act, 16}, {a.delta, act, 16}, {a.z, act, 16}, {a.Bm, bc, 16}, {a.Cm, bc, 16},
                     {a.A, (int64_t)a.D * a.N * 4, 4}, {a.skip, (int64_t)a.D * 4, 4}, {a.dbias, (int64_t)a.D * 4, 4},
                     {p->state, st, 16}, {p->lengths, p->B * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.state = p->state;
  a.lengths = p->lengths;
  a.y = y;
  a.state_out = state_out;
  if (need > 0) {
    a.hend = static_cast<float*>(workspace);
    a.sdt = a.hend + (int64_t)a.segs * rows * a.N;
  }
  return from_hip(selective_scan(a, (hipStream_t)stream));
}

hyena_status hyena_selective_scan_step(const hyena_selective_scan_params* p, float* state, void* y, hyena_dtype io,
                                       void* stream) {
  if (!state || !y) return HYENA_ERR_NULL;
  ScanArgs a;
  if (const hyena_status s = scan_args(p, io, 1, &a)) return s;
  const int64_t e = size_of(io), rows = p->B * a.D, act = rows * e, bc = p->B * a.G * a.N * e;
  if (rows * 16 / 256 > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const Span out[] = {{y, act, 16}, {state, rows * a.N * 4, 16}};
  const Span in[] = {{a.u, act, 16}, {a.delta, act, 16}, {a.z, act, 16}, {a.Bm, bc, 16}, {a.Cm, bc, 16},
                     {a.A, (int64_t)a.D * a.N * 4, 16}, {a.skip, (int64_t)a.D * 4, 4}, {a.dbias, (int64_t)a.D * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.y = y;
  a.state_out = state;
  return from_hip(selective_scan_step(a, (hipStream_t)stream));
}

int64_t hyena_selective_scan_backward_workspace_bytes(int64_t B, int32_t D, int32_t G, int32_t N, int64_t L) {
  if (!batch_ok(B, D, L) || N < 1 || N > HYENA_MAX_STATE || G < 1 || G > D || D % G) return -1;
  return scan_backward_layout(B, D, G, N, L).total;
}

hyena_status hyena_selective_scan_backward(const hyena_selective_scan_params* p, const void* gy,
                                           const float* gstate_out, const hyena_selective_scan_grads* g,
                                           hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!gy || !g || !g->gu || !g->gdelta || !g->gA || !g->gB || !g->gC || !workspace) return HYENA_ERR_NULL;
  ScanArgs a;
  if (const hyena_status s = scan_args(p, io, p ? p->L : 1, &a)) return s;
  if (!a.z != !g->gz) return HYENA_ERR_NULL;
  const ScanBackwardLayout w = scan_backward_layout(a.B, a.D, a.G, a.N, a.L);
  if (workspace_bytes < w.total) return HYENA_ERR_WORKSPACE;
  const int64_t e = size_of(io), rows = p->B * a.D, act = rows * a.L * e, bc = p->B * a.G * a.N * a.L * e;
  const int64_t st = rows * a.N * 4, dn = (int64_t)a.D * a.N * 4, dv = (int64_t)a.D * 4;
  // a workgroup of 32 channels has 512 threads, kMaxGroups counts 256
  const int64_t size = scan_backward_tile(a.N, a.D / a.G) / 16;
  if (p->B * a.G * w.chunks * w.splits * size > kMaxGroups || rows * a.N / 256 >= kMaxGroups)
    return HYENA_ERR_UNSUPPORTED;
  const Span out[] = {{g->gu, act, 16}, {g->gdelta, act, 16}, {g->gz, act, 16}, {g->gB, bc, 16}, {g->gC, bc, 16},
                      {g->gA, dn, 4}, {g->gskip, dv, 4}, {g->gdelta_bias, dv, 4}, {g->gstate, st, 16},
                      {workspace, w.total, 16}};
  const Span in[] = {{a.u, act, 16}, {a.delta, act, 16}, {a.z, act, 16}, {gy, act, 16}, {a.Bm, bc, 16}, {a.Cm, bc, 16},
                     {a.A, dn, 4}, {a.skip, dv, 4}, {a.dbias, dv, 4}, {p->state, st, 16}, {gstate_out, st, 16},
                     {p->lengths, p->B * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.state = p->state;
  a.lengths = p->lengths;
  a.gy = gy;
  a.gstate_out = gstate_out;
  a.gu = g->gu;
  a.gdelta = g->gdelta;
  a.gB = g->gB;
  a.gC = g->gC;
  a.gz = g->gz;
  a.gA = g->gA;
  a.gskip = g->gskip;
  a.gdbias = g->gdelta_bias;
  a.gstate = g->gstate;
  a.chunks = w.chunks;
  a.splits = w.splits;
  char* base = static_cast<char*>(workspace);
  a.hc = reinterpret_cast<float*>(base + w.hc);
  a.qc = reinterpret_cast<float*>(base + w.qc);
  a.dts = reinterpret_cast<float*>(base + w.dts);
  a.ps = reinterpret_cast<float*>(base + w.ps);
  a.pb = reinterpret_cast<float*>(base + w.pb);
  a.gbc = reinterpret_cast<float*>(base + w.gbc);
  return from_hip(selective_scan_backward(a, (hipStream_t)stream));
}

// ------------------------------------------------------------ residual norm

static hyena_status norm_sizes(int64_t rows, int32_t D, float eps, hyena_dtype io) {
  if (rows < 1 || rows > ((int64_t)1 << 31) || D < 1 || D > kMaxDim) return HYENA_ERR_SHAPE;
  if (!(eps >= 0.f) || std::isinf(eps) || !io_ok(io)) return HYENA_ERR_UNSUPPORTED;
  // a row takes a quarter of a workgroup at least, a whole one where it is long
  if ((D <= 2048 ? (rows + 3) / 4 : rows) > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  return HYENA_OK;
}

static hyena_status norm_forward(const void* x, const void* residual, const float* weight, void* y, void* q,
                                 float* scales, void* s_out, int64_t rows, int32_t D, float eps, hyena_dtype io,
                                 void* stream) {
  if (!x || !weight || (!y && (!q || !scales)) || !residual != !s_out) return HYENA_ERR_NULL;
  if (const hyena_status s = norm_sizes(rows, D, eps, io)) return s;
  const int64_t act = rows * D * size_of(io);
  const Span out[] = {{y, act, 16}, {q, rows * D, 16}, {scales, rows * ((D + 127) / 128) * 4, 4}, {s_out, act, 16}};
  const Span in[] = {{x, act, 16}, {residual, act, 16}, {weight, (int64_t)D * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.y = y;
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.s_out = s_out;
  a.rows = rows;
  a.D = D;
  a.io = io == HYENA_BF16;
  a.eps = eps;
  return from_hip(rms_norm(a, (hipStream_t)stream));
}

hyena_status hyena_rms_norm(const void* x, const void* residual, const float* weight, void* y, void* s_out,
                            int64_t rows, int32_t D, float eps, hyena_dtype io, void* stream) {
  if (!y) return HYENA_ERR_NULL;
  return norm_forward(x, residual, weight, y, nullptr, nullptr, s_out, rows, D, eps, io, stream);
}

hyena_status hyena_rms_norm_quantized(const void* x, const void* residual, const float* weight, void* q,
                                      float* scales, void* s_out, int64_t rows, int32_t D, float eps,
                                      hyena_dtype io, void* stream) {
  return norm_forward(x, residual, weight, nullptr, q, scales, s_out, rows, D, eps, io, stream);
}

int64_t hyena_rms_norm_backward_workspace_bytes(int64_t rows, int32_t D) {
  if (rows < 1 || rows > ((int64_t)1 << 31) || D < 1 || D > kMaxDim) return -1;
  return norm_backward_parts(rows, D) * D * 4;
}

hyena_status hyena_rms_norm_backward(const void* s, const float* weight, const void* gy, const void* gs, void* gx,
                                     float* gw, int64_t rows, int32_t D, float eps, hyena_dtype io, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  if (!s || !weight || !gy || !gx || !gw || !workspace) return HYENA_ERR_NULL;
  if (const hyena_status st = norm_sizes(rows, D, eps, io)) return st;
  const int64_t act = rows * D * size_of(io), need = hyena_rms_norm_backward_workspace_bytes(rows, D);
  if (workspace_bytes < need) return HYENA_ERR_WORKSPACE;
  const Span out[] = {{gx, act, 16}, {gw, (int64_t)D * 4, 4}, {workspace, need, 16}};
  const Span in[] = {{s, act, 16}, {gy, act, 16}, {gs, act, 16}, {weight, (int64_t)D * 4, 4}};
  if (const hyena_status st = check_spans(out, in)) return st;
  NormArgs a{};
  a.x = s;
  a.weight = weight;
  a.gy = gy;
  a.gs = gs;
  a.gx = gx;
  a.gw = gw;
  a.partial = static_cast<float*>(workspace);
  a.rows = rows;
  a.D = D;
  a.io = io == HYENA_BF16;
  a.eps = eps;
  return from_hip(rms_norm_backward(a, (hipStream_t)stream));
}

// ------------------------------------------------------------ 8-bit product

hyena_status hyena_quantize(const void* x, void* q, float* scales, int64_t rows, int32_t K, int32_t block_rows,
                            hyena_dtype io, void* stream) {
  if (!x || !q || !scales) return HYENA_ERR_NULL;
  if (rows < 1 || rows > ((int64_t)1 << 31) || K < 1 || K > kMaxDim) return HYENA_ERR_SHAPE;
  if ((block_rows != 1 && block_rows != 128) || !io_ok(io)) return HYENA_ERR_UNSUPPORTED;
  const int64_t kb = (K + 127) / 128, blocks = block_rows == 1 ? rows * kb : (rows + 127) / 128 * kb;
  if ((block_rows == 1 ? (blocks + 15) / 16 : blocks) > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const Span out[] = {{q, rows * K, 16}, {scales, blocks * 4, 4}};
  const Span in[] = {{x, rows * K * size_of(io), 16}};
  if (const hyena_status s = check_spans(out, in)) return s;
  NormArgs a{};
  a.x = x;
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.rows = rows;
  a.D = K;
  a.io = io == HYENA_BF16;
  a.block_rows = block_rows;
  return from_hip(quantize(a, (hipStream_t)stream));
}

hyena_status hyena_scaled_matmul(const void* q, const float* scales, const void* wq, const float* wscales,
                                 const float* bias, void* out, int64_t B, int64_t L, int32_t N, int32_t K,
                                 int32_t channel_major, hyena_dtype io, void* stream) {
  if (!q || !scales || !wq || !wscales || !out) return HYENA_ERR_NULL;
  constexpr int64_t kRows = (int64_t)1 << 31;
  if (B < 1 || B > kRows || L < 1 || L > kRows || B * L > kRows || N < 1 || N > kMaxDim || K < 1 || K > kMaxDim)
    return HYENA_ERR_SHAPE;
  // sequences are told apart in the channel-major layout only
  if (channel_major && (B > kMaxDim || L > HYENA_MAX_L)) return HYENA_ERR_SHAPE;
  if (K % 16 || (channel_major != 0 && channel_major != 1) || !io_ok(io)) return HYENA_ERR_UNSUPPORTED;
  const int64_t M = B * L, kb = (K + 127) / 128;
  if (((M + 63) / 64) * ((N + 63) / 64) > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const Span outs[] = {{out, M * N * size_of(io), 16}};
  const Span in[] = {{q, M * K, 16}, {wq, (int64_t)N * K, 16}, {scales, M * kb * 4, 4},
                     {wscales, (N + 127) / 128 * kb * 4, 4}, {bias, (int64_t)N * 4, 4}};
  if (const hyena_status s = check_spans(outs, in)) return s;
  ScaledArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.scales = scales;
  a.wq = static_cast<const uint8_t*>(wq);
  a.wscales = wscales;
  a.bias = bias;
  a.out = out;
  a.M = M;
  a.N = N;
  a.K = K;
  a.L = L;
  a.io = io == HYENA_BF16;
  a.channel_major = channel_major;
  return from_hip(scaled_matmul(a, (hipStream_t)stream));
}

}  // extern "C"
