// api_linattn.cpp -- the extern "C" entry points of the linear-attention
// block's operators (include/hyena.h): every argument is checked on the host
// before anything is enqueued, and nothing is allocated.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.hpp"
#include "hyena.h"
#include "linattn.hpp"

using namespace hyena;

static_assert(HYENA_MAX_HEAD == 256, "the attention's kernels hold at most 256 values of a head");

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 38;   // a view's bytes, up to 24 (2^20 of these), fit 63 bits

// Elements from a view's first to behind its last one; 0 for a stride out of range.
int64_t extent(const int64_t (&stride)[3], int64_t B, int64_t L, int64_t heads, int64_t D) {
  for (const int64_t s : stride)
    if (s < 0 || s > kMaxStride) return 0;
  return (B - 1) * stride[0] + (L - 1) * stride[1] + (heads - 1) * stride[2] + D;
}

HeadView view(const void* p, const int64_t (&stride)[3], int share, int64_t total) {
  return HeadView{p, stride[0], stride[1], stride[2], share, total};
}

HeadView dense(const void* p, int64_t B, int64_t L, int64_t H, int64_t D) {
  return HeadView{p, L * H * D, H * D, D, 1, B * L * H * D};
}

bool heads_ok(int64_t B, int64_t L, int64_t H, int64_t Hq, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv) {
  if (!batch_ok(B, H, L) || Dk < 1 || Dk > HYENA_MAX_HEAD || Dv < 1 || Dv > HYENA_MAX_HEAD) return false;
  for (const int64_t h : {Hq, Hk, Hv})
    if (h < 1 || h > H || H % h) return false;
  return true;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// Bytes of the states between the segments of one pass.
int64_t seg_bytes(const LinPlan& p, int64_t B, int64_t H, int64_t Dk, int64_t Dv) {
  return round16((p.segs - 1) * B * H * Dk * Dv * 4);
}

// The backward's workspace: states before and behind the segments, and fp32
// gradients of every head where heads share one.  For sizes that a launch
// takes (kMaxGroups), so B H < 2^24 and the sum stays below 2^58.
struct BackwardLayout {
  int64_t before, behind, part[3], total;
};
BackwardLayout backward_layout(const LinPlan& p, int64_t B, int64_t L, int64_t H, const int64_t (&heads)[3], int64_t Dk,
                               int64_t Dv) {
  BackwardLayout w;
  const int64_t D[3] = {Dk, Dk, Dv};
  w.before = 0;
  w.behind = seg_bytes(p, B, H, Dk, Dv);
  w.total = 2 * w.behind;
  for (int i = 0; i < 3; ++i) {
    w.part[i] = w.total;
    if (heads[i] < H) w.total += round16(B * L * H * D[i] * 4);
  }
  return w;
}

}  // namespace

extern "C" {

// -------------------------------------------------------- linear attention

static hyena_status lin_args(const hyena_linear_attention_params* p, hyena_dtype io, int64_t L, int64_t (&ext)[3]) {
  if (!p || !p->q || !p->k || !p->v) return HYENA_ERR_NULL;
  if (!heads_ok(p->B, L, p->H, p->Hq, p->Hk, p->Hv, p->Dk, p->Dv)) return HYENA_ERR_SHAPE;
  if (!io_ok(io) || !std::isfinite(p->scale)) return HYENA_ERR_UNSUPPORTED;
  ext[0] = extent(p->q_stride, p->B, L, p->Hq, p->Dk);
  ext[1] = extent(p->k_stride, p->B, L, p->Hk, p->Dk);
  ext[2] = extent(p->v_stride, p->B, L, p->Hv, p->Dv);
  return ext[0] && ext[1] && ext[2] ? HYENA_OK : HYENA_ERR_SHAPE;
}

int64_t hyena_linear_attention_workspace_bytes(int64_t B, int64_t L, int32_t H, int32_t Dk, int32_t Dv) {
  if (!heads_ok(B, L, H, H, H, H, Dk, Dv)) return -1;
  const LinPlan plan = lin_plan(B, L, H, Dk, Dv);
  return lin_groups(plan, B, H, Dv) > kMaxGroups ? -1 : seg_bytes(plan, B, H, Dk, Dv);
}

hyena_status hyena_linear_attention(const hyena_linear_attention_params* p, void* o, float* state_out, hyena_dtype io,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
  int64_t ext[3];
  if (const hyena_status s = lin_args(p, io, p ? p->L : 1, ext)) return s;
  if (!o) return HYENA_ERR_NULL;
  const int64_t e = size_of(io), st = p->B * p->H * p->Dk * p->Dv * 4;
  const LinPlan plan = lin_plan(p->B, p->L, p->H, p->Dk, p->Dv);
  if (lin_groups(plan, p->B, p->H, p->Dv) > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const int64_t need = seg_bytes(plan, p->B, p->H, p->Dk, p->Dv);
  if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
  const Span out[] = {{o, p->B * p->L * p->H * p->Dv * e, 16}, {state_out, st, 16}, {need ? workspace : nullptr, need, 16}};
  const Span in[] = {{p->q, ext[0] * e, e}, {p->k, ext[1] * e, e}, {p->v, ext[2] * e, e}, {p->state, st, 16},
                     {p->log_decay, p->H * 4, 4}, {p->lengths, p->B * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  LinArgs a{};
  LinPass& f = a.pass[0];
  f.q = view(p->q, p->q_stride, p->H / p->Hq, ext[0]);
  f.k = view(p->k, p->k_stride, p->H / p->Hk, ext[1]);
  f.v = view(p->v, p->v_stride, p->H / p->Hv, ext[2]);
  f.out = o;
  f.out_f32 = io == HYENA_FP32;
  f.DK = p->Dk;
  f.DV = p->Dv;
  f.so = p->scale;
  f.su = 1.f;
  f.s0 = p->state;
  f.s0_k = f.seg_k = p->Dv;
  f.s0_v = f.seg_v = 1;
  f.seg = static_cast<float*>(workspace);
  f.s_out = state_out;
  a.passes = a.fills = 1;
  a.fill[0] = f;
  a.log_decay = p->log_decay;
  a.lengths = p->lengths;
  a.B = (int)p->B;
  a.H = p->H;
  a.L = p->L;
  a.io = io == HYENA_BF16;
  a.segs = plan.segs;
  a.seg = plan.seg;
  return from_hip(linear_attention(a, (hipStream_t)stream));
}

hyena_status hyena_linear_attention_step(const hyena_linear_attention_params* p, float* state, void* o, hyena_dtype io,
                                         void* stream) {
  int64_t ext[3];
  if (const hyena_status s = lin_args(p, io, 1, ext)) return s;
  if (!o || !state) return HYENA_ERR_NULL;
  if (p->B * p->H * lin_step_plan(p->Dv).tiles > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const int64_t e = size_of(io), st = p->B * p->H * p->Dk * p->Dv * 4;
  const Span out[] = {{o, p->B * p->H * p->Dv * e, 16}, {state, st, 16}};
  const Span in[] = {{p->q, ext[0] * e, e}, {p->k, ext[1] * e, e}, {p->v, ext[2] * e, e}, {p->log_decay, p->H * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  LinStepArgs a{};
  a.q = view(p->q, p->q_stride, p->H / p->Hq, ext[0]);
  a.k = view(p->k, p->k_stride, p->H / p->Hk, ext[1]);
  a.v = view(p->v, p->v_stride, p->H / p->Hv, ext[2]);
  a.log_decay = p->log_decay;
  a.state = state;
  a.o = o;
  a.B = (int)p->B;
  a.H = p->H;
  a.Dk = p->Dk;
  a.Dv = p->Dv;
  a.io = io == HYENA_BF16;
  a.scale = p->scale;
  return from_hip(linear_attention_step(a, (hipStream_t)stream));
}

int64_t hyena_linear_attention_backward_workspace_bytes(int64_t B, int64_t L, int32_t H, int32_t Hq, int32_t Hk,
                                                        int32_t Hv, int32_t Dk, int32_t Dv) {
  if (!heads_ok(B, L, H, Hq, Hk, Hv, Dk, Dv)) return -1;
  const LinPlan plan = lin_backward_plan(B, L, H, Dk, Dv, 0);   // no fewer segments than bf16's
  return lin_groups(plan, B, H, Dk > Dv ? Dk : Dv) > kMaxGroups ? -1 : backward_layout(plan, B, L, H, {Hq, Hk, Hv}, Dk, Dv).total;
}

hyena_status hyena_linear_attention_backward(const hyena_linear_attention_params* p, const void* go,
                                             const float* gstate_out, const hyena_linear_attention_grads* g,
                                             hyena_dtype io, void* workspace, int64_t workspace_bytes, void* stream) {
  int64_t ext[3];
  if (const hyena_status s = lin_args(p, io, p ? p->L : 1, ext)) return s;
  if (!go || !g || !g->gq || !g->gk || !g->gv) return HYENA_ERR_NULL;
  const int64_t e = size_of(io), st = p->B * p->H * p->Dk * p->Dv * 4, tokens = p->B * p->L;
  const LinPlan plan = lin_backward_plan(p->B, p->L, p->H, p->Dk, p->Dv, io == HYENA_BF16);
  if (lin_groups(plan, p->B, p->H, p->Dk > p->Dv ? p->Dk : p->Dv) > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  const int64_t heads[3] = {p->Hq, p->Hk, p->Hv};
  const BackwardLayout w = backward_layout(plan, p->B, p->L, p->H, heads, p->Dk, p->Dv);
  if (w.total && (!workspace || workspace_bytes < w.total)) return HYENA_ERR_WORKSPACE;
  const Span out[] = {{g->gq, tokens * p->Hq * p->Dk * e, 16}, {g->gk, tokens * p->Hk * p->Dk * e, 16},
                      {g->gv, tokens * p->Hv * p->Dv * e, 16}, {g->gstate, st, 16},
                      {w.total ? workspace : nullptr, w.total, 16}};
  const Span in[] = {{p->q, ext[0] * e, e}, {p->k, ext[1] * e, e}, {p->v, ext[2] * e, e}, {go, tokens * p->H * p->Dv * e, 16},
                     {p->state, st, 16}, {gstate_out, st, 16}, {p->log_decay, p->H * 4, 4}, {p->lengths, p->B * 4, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  char* const ws = static_cast<char*>(workspace);
  const HeadView q = view(p->q, p->q_stride, p->H / p->Hq, ext[0]), k = view(p->k, p->k_stride, p->H / p->Hk, ext[1]),
                 v = view(p->v, p->v_stride, p->H / p->Hv, ext[2]), d = dense(go, p->B, p->L, p->H, p->Dv);
  void* const grads[3] = {g->gq, g->gk, g->gv};
  LinArgs a{};
  FoldArgs f{};
  bool fold = false;
  for (int i = 0; i < 3; ++i) {
    LinPass& r = a.pass[i];
    const bool shared = heads[i] < p->H;
    r.out = shared ? ws + w.part[i] : grads[i];
    r.out_f32 = shared || io == HYENA_FP32;
    r.DK = i == 2 ? p->Dk : p->Dv;
    r.DV = i == 2 ? p->Dv : p->Dk;
    r.so = i == 0 ? p->scale : 1.f;
    r.su = i == 0 ? 1.f : p->scale;
    r.reverse = i > 0;
    r.s0 = i == 0 ? p->state : gstate_out;              // [Dk][Dv]; the first two passes hold it transposed
    r.s0_k = i == 2 ? p->Dv : 1;
    r.s0_v = i == 2 ? 1 : p->Dv;
    r.seg = reinterpret_cast<float*>(ws + (i == 0 ? w.before : w.behind));
    r.seg_k = r.s0_k;
    r.seg_v = r.s0_v;
    f.x[i] = shared ? static_cast<const float*>(r.out) : nullptr;
    f.out[i] = grads[i];
    f.heads[i] = (int)heads[i];
    f.share[i] = p->H / (int)heads[i];
    f.D[i] = i == 2 ? p->Dv : p->Dk;
    fold = fold || shared;
  }
  a.pass[0].q = d, a.pass[0].k = v, a.pass[0].v = k;    // gq[t] = scale S[t] go[t]
  a.pass[1].q = v, a.pass[1].k = d, a.pass[1].v = q;    // gk[t] = G[t] v[t],  G[t] = lambda G[t+1] + scale q[t] go[t]^T
  a.pass[2].q = k, a.pass[2].k = q, a.pass[2].v = d;    // gv[t] = G[t]^T k[t]
  a.pass[2].s_out = g->gstate;
  a.passes = 3;
  a.fill[1] = a.pass[2];                                // G
  a.fill[0] = a.pass[2];                                // S, from k and v
  a.fill[0].k = k, a.fill[0].v = v;
  a.fill[0].su = 1.f;
  a.fill[0].reverse = 0;
  a.fill[0].s0 = p->state;
  a.fill[0].seg = a.pass[0].seg;
  a.fills = 2;
  a.log_decay = p->log_decay;
  a.lengths = p->lengths;
  a.B = (int)p->B;
  a.H = p->H;
  a.L = p->L;
  a.io = io == HYENA_BF16;
  a.segs = plan.segs;
  a.seg = plan.seg;
  if (const hipError_t err = linear_attention(a, (hipStream_t)stream)) return from_hip(err);
  if (!fold) return HYENA_OK;
  f.tokens = tokens;
  f.io = io == HYENA_BF16;
  return from_hip(fold_heads(f, (hipStream_t)stream));
}

// --------------------------------------------------------- rotary positions

hyena_status hyena_rotary(const hyena_rotary_params* p, const void* x, void* out, hyena_dtype io, void* stream) {
  if (!p || !p->freq || !x || !out) return HYENA_ERR_NULL;
  if (!batch_ok(p->B, p->H, p->L) || p->D < 2 || p->D > (1 << 16) || p->R < 2 || p->R > p->D || p->R % 2) return HYENA_ERR_SHAPE;
  const int64_t ext = extent(p->x_stride, p->B, p->L, p->H, p->D);
  if (!ext) return HYENA_ERR_SHAPE;
  int64_t pos = 0;
  if (p->positions) {
    for (const int64_t s : p->pos_stride)
      if (s < 0 || s > kMaxStride) return HYENA_ERR_SHAPE;
    pos = (p->B - 1) * p->pos_stride[0] + (p->L - 1) * p->pos_stride[1] + 1;
  }
  if ((p->interleaved != 0 && p->interleaved != 1) || (p->inverse != 0 && p->inverse != 1) || !io_ok(io) ||
      !std::isfinite(p->scale))
    return HYENA_ERR_UNSUPPORTED;
  const bool in_place = out == x;
  const int64_t e = size_of(io), tokens = p->B * p->L;
  RotaryArgs a{};
  a.tokens = tokens;
  a.L = p->L;
  a.H = p->H;
  a.D = p->D;
  a.R = p->R;
  a.in_place = in_place;
  a.io = io == HYENA_BF16;
  if (rotary_groups(a) > kMaxGroups) return HYENA_ERR_UNSUPPORTED;
  if (in_place) {                                      // heads apart from each other: every stride beyond what is inside it
    int64_t n[3] = {p->B, p->L, p->H}, span = p->D;
    for (int done = 0; done < 3; ++done) {
      int at = -1;                                     // the smallest stride that is left
      for (int i = 0; i < 3; ++i)
        if (n[i] && (at < 0 || p->x_stride[i] < p->x_stride[at])) at = i;
      if (n[at] > 1) {
        if (p->x_stride[at] < span) return HYENA_ERR_ALIAS;
        span += (n[at] - 1) * p->x_stride[at];
      }
      n[at] = 0;
    }
  }
  const Span outs[] = {{out, in_place ? ext * e : tokens * p->H * p->D * e, in_place ? e : 16}};
  const Span in[] = {{in_place ? nullptr : x, ext * e, e}, {p->freq, (int64_t)p->R * 4, 8}, {p->positions, pos * 4, 4}};
  if (const hyena_status s = check_spans(outs, in)) return s;
  a.x = view(x, p->x_stride, 1, ext);
  a.out = in_place ? a.x : dense(out, p->B, p->L, p->H, p->D);
  a.out.p = out;
  a.freq = p->freq;
  a.positions = p->positions;
  a.pos_batch = p->pos_stride[0];
  a.pos_token = p->pos_stride[1];
  a.interleaved = p->interleaved;
  a.scale = p->scale;
  a.sine = p->inverse ? -1.f : 1.f;
  return from_hip(rotary(a, (hipStream_t)stream));
}

// --------------------------------------------------------------- group norm

static bool group_sizes_ok(int64_t rows, int64_t D, int64_t G) {
  return rows >= 1 && rows <= ((int64_t)1 << 31) && D >= 1 && D <= kMaxDim && G >= 1 && G <= D && D % G == 0;
}

static bool group_launch_ok(int64_t rows, int64_t D, int64_t G) {   // a group wider than a workgroup's registers is a workgroup's
  return group_norm_plan(G, D / G).words || rows * G <= kMaxGroups;
}

static hyena_status group_args(const hyena_group_norm_params* p, hyena_dtype io, GroupNormArgs* a) {
  if (!p || !p->x) return HYENA_ERR_NULL;
  if (!group_sizes_ok(p->rows, p->D, p->G)) return HYENA_ERR_SHAPE;
  if ((p->silu != 0 && p->silu != 1) || (p->silu && p->z) || !io_ok(io) || !(p->eps >= 0.f) || !std::isfinite(p->eps))
    return HYENA_ERR_UNSUPPORTED;
  if (!group_launch_ok(p->rows, p->D, p->G)) return HYENA_ERR_UNSUPPORTED;
  *a = GroupNormArgs{};
  a->x = p->x;
  a->z = p->z;
  a->weight = p->weight;
  a->bias = p->bias;
  a->rows = p->rows;
  a->G = p->G;
  a->Dg = p->D / p->G;
  a->silu = p->silu;
  a->eps = p->eps;
  a->io = io == HYENA_BF16;
  return HYENA_OK;
}

hyena_status hyena_group_norm(const hyena_group_norm_params* p, void* y, hyena_dtype io, void* stream) {
  GroupNormArgs a;
  if (const hyena_status s = group_args(p, io, &a)) return s;
  if (!y) return HYENA_ERR_NULL;
  const int64_t act = p->rows * p->D * size_of(io), ch = (int64_t)p->D * 4;
  const Span out[] = {{y, act, 16}};
  const Span in[] = {{p->x, act, 16}, {p->z, act, 16}, {p->weight, ch, 4}, {p->bias, ch, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.y = y;
  return from_hip(group_norm(a, (hipStream_t)stream));
}

int64_t hyena_group_norm_backward_workspace_bytes(int64_t rows, int32_t D, int32_t G) {
  if (!group_sizes_ok(rows, D, G) || !group_launch_ok(rows, D, G)) return -1;
  return group_norm_backward_parts(rows, G, D / G) * 2 * D * 4;
}

hyena_status hyena_group_norm_backward(const hyena_group_norm_params* p, const void* gy, void* gx, float* gweight,
                                       float* gbias, void* gz, hyena_dtype io, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  GroupNormArgs a;
  if (const hyena_status s = group_args(p, io, &a)) return s;
  if (!gy || !gx || !p->z != !gz) return HYENA_ERR_NULL;
  const bool sums = gweight || gbias;
  const int64_t act = p->rows * p->D * size_of(io), ch = (int64_t)p->D * 4;
  const int64_t need = sums ? hyena_group_norm_backward_workspace_bytes(p->rows, p->D, p->G) : 0;
  if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
  const Span out[] = {{gx, act, 16}, {gz, act, 16}, {gweight, ch, 4}, {gbias, ch, 4}, {need ? workspace : nullptr, need, 16}};
  const Span in[] = {{p->x, act, 16}, {gy, act, 16}, {p->z, act, 16}, {p->weight, ch, 4}, {p->bias, ch, 4}};
  if (const hyena_status s = check_spans(out, in)) return s;
  a.gy = gy;
  a.gx = gx;
  a.gz = gz;
  a.gw = gweight;
  a.gb = gbias;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  return from_hip(group_norm_backward(a, (hipStream_t)stream));
}

}  // extern "C"
