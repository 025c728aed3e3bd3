// C-ABI front end of the expert feed-forward block (norms, routing, experts): argument
// validation on the host, before any HIP call, and launches on the caller's stream.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/w4a16.h"
#include "checks.h"
#include "w4a16_internal.h"

namespace {

using namespace w4a16::checks;

bool act_type(int dtype) { return dtype == W4A16_DTYPE_F16 || dtype == W4A16_DTYPE_BF16; }

bool aligned16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (!w4a16::checks::aligned16(p)) return false;
  return true;
}

// Whether an output overlaps another output, or an input that it may not replace:
// outputs[i] may be exactly one of the first `same` inputs.
bool overlaps(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs, int same) {
  for (const Range *o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Range *p = outputs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return true;
    int n = 0;
    for (const Range &i : inputs)
      if (n++ < same ? overlap_but_same(*o, i) : overlap(*o, i)) return true;
  }
  return false;
}

int status(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_EHIP; }

// ---- norms --------------------------------------------------------------------------

constexpr int64_t kMaxNormD = 16384;

static_assert(W4A16_NORM_NONE == 0 && W4A16_NORM_RMS == 1 && W4A16_NORM_LAYER == 2,
              "the kernels' norm numbers");

int check_norm(const w4a16_norm &n) {
  if (n.kind < W4A16_NORM_NONE || n.kind > W4A16_NORM_LAYER) return W4A16_EUNSUPPORTED;
  if (n.kind == W4A16_NORM_NONE) return n.weight || n.bias ? W4A16_EINVAL : W4A16_OK;
  return n.eps >= 0.f && isfinite(n.eps) ? W4A16_OK : W4A16_EINVAL;
}

int check_norm_shape(const w4a16_norm &post, const w4a16_norm &pre, const void *y, const void *gate,
                     int64_t T, int64_t D, int64_t gate_rows, int dtype) {
  if (T < 0 || T >= kMaxM || D < 1 || D > kMaxNormD) return W4A16_EINVAL;
  if (!act_type(dtype)) return W4A16_EUNSUPPORTED;
  if (int rc = check_norm(post)) return rc;
  if (int rc = check_norm(pre)) return rc;
  if (gate && gate_rows < 1) return W4A16_EINVAL;
  if (T > 0 && !y && (gate || post.kind != W4A16_NORM_NONE)) return W4A16_EINVAL;
  return W4A16_OK;
}

w4a16::NormSpec spec(const w4a16_norm &n) { return {n.kind, n.eps, n.weight, n.bias}; }

// Tokens per gate vector: all of them without a gate, and no more than there are.
int tokens_per_gate(const void *gate, int64_t gate_rows, int64_t T) {
  return (int)std::max<int64_t>(1, gate ? std::min(gate_rows, T) : T);
}

// (a gate's tokens are clamped before they are added to T: gate_rows may be any 64-bit number)
int64_t gates(int64_t T, int64_t gate_rows) {
  if (gate_rows < 1 || T < 1) return 0;
  const int64_t rows = std::min(gate_rows, T);
  return (T + rows - 1) / rows;
}

w4a16::NormGradDesc norm_grad_desc(const w4a16_norm_backward_call &c) {
  w4a16::NormGradDesc d = {};
  d.dr = c.dr;
  d.dh = c.dh;
  d.y = c.y;
  d.r = c.r;
  d.gate = c.gate;
  d.post = spec(c.post);
  d.pre = spec(c.pre);
  d.alpha = c.alpha;
  d.dx = c.dx;
  d.dy = c.dy;
  void *const sums[w4a16::kNormSums] = {c.dgate, c.dpost_weight, c.dpost_bias, c.dpre_weight, c.dpre_bias};
  for (int i = 0; i < w4a16::kNormSums; ++i) d.sums[i] = sums[i];
  d.T = (int)c.T;
  d.D = (int)c.D;
  d.gate_rows = tokens_per_gate(c.gate, c.gate_rows, c.T);
  d.bf16 = c.dtype == W4A16_DTYPE_BF16;
  return d;
}

int check_norm_backward(const w4a16_norm_backward_call &c) {
  if (int rc = check_norm_shape(c.post, c.pre, c.y, c.gate, c.T, c.D, c.gate_rows, c.dtype)) return rc;
  const bool pre = c.pre.kind != W4A16_NORM_NONE, post = c.post.kind != W4A16_NORM_NONE;
  if ((c.dgate && !c.gate) || (!post && (c.dpost_weight || c.dpost_bias)) ||
      (!pre && (c.dpre_weight || c.dpre_bias)))
    return W4A16_EINVAL;
  return W4A16_OK;
}

// ---- routing -------------------------------------------------------------------------

constexpr int64_t kMaxExperts = 1024, kMaxTopK = 64;

int check_routing(const w4a16_routing *r) {
  if (!r || r->T < 0 || r->T > kMaxM || r->E < 1 || r->E > kMaxExperts) return W4A16_EINVAL;
  if (r->score != W4A16_SCORE_SOFTMAX && r->score != W4A16_SCORE_SIGMOID) return W4A16_EUNSUPPORTED;
  if (!act_type(r->dtype) && r->dtype != W4A16_DTYPE_F32) return W4A16_EUNSUPPORTED;
  if (r->k < 1 || r->k > kMaxTopK || !isfinite(r->scale)) return W4A16_EINVAL;
  if (r->groups < 1 || r->groups > 64 || r->E % r->groups || r->topk_groups < 1 ||
      r->topk_groups > r->groups || r->k > r->topk_groups * (r->E / r->groups))
    return W4A16_EINVAL;
  return W4A16_OK;
}

w4a16::RouteDesc route_desc(const w4a16_routing &r) {
  w4a16::RouteDesc d = {};
  d.T = (int)r.T;
  d.E = (int)r.E;
  d.k = (int)r.k;
  d.type = r.dtype;
  d.sigmoid = r.score == W4A16_SCORE_SIGMOID;
  // (a choice among all groups is one among all experts)
  d.groups = r.topk_groups < r.groups ? r.groups : 1;
  d.topk_groups = d.groups > 1 ? r.topk_groups : 1;
  d.renormalize = r.renormalize != 0;
  d.scale = r.scale;
  return d;
}

size_t logit_bytes(const w4a16_routing &r) { return (size_t)(r.T * r.E) * (r.dtype == W4A16_DTYPE_F32 ? 4 : 2); }

// ---- experts -------------------------------------------------------------------------

constexpr int64_t kMaxExpertDim = int64_t(1) << 20;

int check_experts_shape(int64_t T, int64_t E, int64_t k, int64_t D, int64_t N, int act, int dtype) {
  if (T < 0 || T > kMaxM || E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK) return W4A16_EINVAL;
  if (D < W4A16_GROUP || N < W4A16_GROUP || D > kMaxExpertDim || N > kMaxExpertDim || D % W4A16_GROUP ||
      N % W4A16_GROUP || N * D / 2 > kMaxPackedBytes)
    return W4A16_EINVAL;
  return known_act(act) && act_type(dtype) ? W4A16_OK : W4A16_EUNSUPPORTED;
}

w4a16::ExpertsDesc experts_desc(const w4a16_experts_call &c) {
  auto weight = [](const w4a16_expert_weight &w) { return w4a16::ExpertWeight{w.Wq, w.scales, w.zeros}; };
  w4a16::ExpertsDesc d = {};
  d.X = c.X;
  d.ids = static_cast<const int32_t *>(c.ids);
  d.weights = static_cast<const float *>(c.weights);
  d.gate = weight(c.gate);
  d.up = weight(c.up);
  d.down = weight(c.down);
  d.s = c.s;
  d.s_down = c.s_down;
  d.residual = c.residual;
  d.G = c.G;
  d.U = c.U;
  d.Y = c.Y;
  d.T = (int)c.T;
  d.E = (int)c.E;
  d.k = (int)c.k;
  d.D = (int)c.D;
  d.N = (int)c.N;
  d.act = c.act;
  d.bf16 = c.dtype == W4A16_DTYPE_BF16;
  return d;
}

w4a16::ExpertsGradDesc experts_grad_desc(const w4a16_experts_backward_call &c) {
  auto weight = [](const w4a16_expert_transposed &w) { return w4a16::ExpertTransposed{w.Wt, w.meta}; };
  w4a16::ExpertsGradDesc d = {};
  d.dY = c.dY;
  d.ids = static_cast<const int32_t *>(c.ids);
  d.weights = static_cast<const float *>(c.weights);
  d.G = c.G;
  d.U = c.U;
  d.gate = weight(c.gate);
  d.up = weight(c.up);
  d.down = weight(c.down);
  d.s = c.s;
  d.s_down = c.s_down;
  d.add = c.add;
  d.dX = c.dX;
  d.dweights = c.dweights;
  d.dweights_f32 = c.dweights_f32 != 0;
  d.T = (int)c.T;
  d.E = (int)c.E;
  d.k = (int)c.k;
  d.D = (int)c.D;
  d.N = (int)c.N;
  d.act = c.act;
  d.bf16 = c.dtype == W4A16_DTYPE_BF16;
  return d;
}

}  // namespace

extern "C" {

int w4a16_norm_block(const w4a16_norm_call *c, void *stream) {
  if (!c) return W4A16_EINVAL;
  if (int rc = check_norm_shape(c->post, c->pre, c->y, c->gate, c->T, c->D, c->gate_rows, c->dtype))
    return rc;
  if (c->T == 0) return W4A16_OK;
  if (!c->x || (!c->r && !c->h) || (c->h != nullptr) != (c->pre.kind != W4A16_NORM_NONE))
    return W4A16_EINVAL;
  if (!aligned16({c->x, c->y, c->gate, c->r, c->h, c->post.weight, c->post.bias, c->pre.weight, c->pre.bias}))
    return W4A16_EALIGN;
  const size_t rows = (size_t)(c->T * c->D) * 2, row = (size_t)c->D * 2;
  if (overlaps({{c->r, rows}, {c->h, rows}},
               {{c->x, rows}, {c->y, rows}, {c->gate, gates(c->T, c->gate_rows) * row}, {c->post.weight, row},
                {c->post.bias, row}, {c->pre.weight, row}, {c->pre.bias, row}}, 2))
    return W4A16_EINVAL;
  w4a16::NormDesc d = {c->x, c->y, c->gate, spec(c->post), spec(c->pre), c->alpha, c->r, c->h,
                       (int)c->T, (int)c->D, tokens_per_gate(c->gate, c->gate_rows, c->T), c->dtype == W4A16_DTYPE_BF16};
  return status(w4a16::launch_norm(d, static_cast<hipStream_t>(stream)));
}

int w4a16_norm_block_backward_workspace_size(const w4a16_norm_backward_call *c, size_t *bytes) {
  if (!c || !bytes) return W4A16_EINVAL;
  if (int rc = check_norm_backward(*c)) return rc;
  *bytes = w4a16::norm_grad_workspace_bytes(norm_grad_desc(*c));
  return W4A16_OK;
}

int w4a16_norm_block_backward(const w4a16_norm_backward_call *c, void *workspace,
                              size_t workspace_bytes, void *stream) {
  if (!c) return W4A16_EINVAL;
  if (int rc = check_norm_backward(*c)) return rc;
  const bool pre = c->pre.kind != W4A16_NORM_NONE;
  if (c->T > 0 && ((pre && (!c->dh || !c->r)) || (!pre && (!c->dr || c->dh)) || (c->dy && !c->y)))
    return W4A16_EINVAL;
  if (!aligned16({c->dr, c->dh, c->y, c->r, c->gate, c->post.weight, c->post.bias, c->pre.weight, c->pre.bias,
                  c->dx, c->dy, c->dgate, c->dpost_weight, c->dpost_bias, c->dpre_weight, c->dpre_bias}))
    return W4A16_EALIGN;
  const w4a16::NormGradDesc d = norm_grad_desc(*c);
  const size_t need = w4a16::norm_grad_workspace_bytes(d);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_EINVAL;
  if (!aligned256(workspace)) return W4A16_EALIGN;
  const size_t rows = (size_t)(c->T * c->D) * 2, row = (size_t)c->D * 2;
  const size_t gate = (size_t)gates(c->T, c->gate_rows) * row;
  if (overlaps({{c->dx, rows}, {c->dy, rows}, {c->dgate, 2 * gate}, {c->dpost_weight, 2 * row},
                {c->dpost_bias, 2 * row}, {c->dpre_weight, 2 * row}, {c->dpre_bias, 2 * row}, {workspace, need}},
               {{c->dr, rows}, {c->dh, rows}, {c->y, rows}, {c->r, rows}, {c->gate, gate}, {c->post.weight, row},
                {c->post.bias, row}, {c->pre.weight, row}, {c->pre.bias, row}}, 0))
    return W4A16_EINVAL;
  return status(w4a16::launch_norm_grad(d, workspace, static_cast<hipStream_t>(stream)));
}

int w4a16_route(const w4a16_routing *r, const void *logits, const void *bias, void *ids,
                void *weights, void *stream) {
  if (int rc = check_routing(r)) return rc;
  if (r->T == 0) return W4A16_OK;
  if (!logits || !ids || !weights) return W4A16_EINVAL;
  if (!aligned16({logits, bias, ids, weights})) return W4A16_EALIGN;
  const size_t out = (size_t)(r->T * r->k) * 4;
  if (overlaps({{ids, out}, {weights, out}}, {{logits, logit_bytes(*r)}, {bias, (size_t)r->E * 4}}, 0))
    return W4A16_EINVAL;
  w4a16::RouteDesc d = route_desc(*r);
  d.logits = logits;
  d.bias = static_cast<const float *>(bias);
  d.ids = static_cast<int32_t *>(ids);
  d.weights = static_cast<float *>(weights);
  return status(w4a16::launch_route(d, false, static_cast<hipStream_t>(stream)));
}

int w4a16_route_backward(const w4a16_routing *r, const void *dweights, const void *logits,
                         const void *ids, void *dlogits, void *stream) {
  if (int rc = check_routing(r)) return rc;
  if (r->T == 0) return W4A16_OK;
  if (!dweights || !logits || !ids || !dlogits) return W4A16_EINVAL;
  if (!aligned16({dweights, logits, ids, dlogits})) return W4A16_EALIGN;
  const size_t slots = (size_t)(r->T * r->k) * 4, n = logit_bytes(*r);
  if (overlaps({{dlogits, n}}, {{logits, n}, {dweights, slots}, {ids, slots}}, 0)) return W4A16_EINVAL;
  w4a16::RouteDesc d = route_desc(*r);
  d.logits = logits;
  d.dweights = static_cast<const float *>(dweights);
  d.ids = const_cast<int32_t *>(static_cast<const int32_t *>(ids));
  d.dlogits = dlogits;
  return status(w4a16::launch_route(d, true, static_cast<hipStream_t>(stream)));
}

int w4a16_experts_workspace_size(const w4a16_experts_call *c, size_t *bytes) {
  if (!c || !bytes) return W4A16_EINVAL;
  if (int rc = check_experts_shape(c->T, c->E, c->k, c->D, c->N, c->act, c->dtype)) return rc;
  *bytes = w4a16::experts_workspace_bytes(experts_desc(*c));
  return W4A16_OK;
}

int w4a16_experts(const w4a16_experts_call *c, void *workspace, size_t workspace_bytes, void *stream) {
  if (!c) return W4A16_EINVAL;
  if (int rc = check_experts_shape(c->T, c->E, c->k, c->D, c->N, c->act, c->dtype)) return rc;
  if (c->T == 0) return W4A16_OK;
  if (!c->X || !c->ids || !c->weights || !c->Y || (c->G != nullptr) != (c->U != nullptr)) return W4A16_EINVAL;
  for (const w4a16_expert_weight *w : {&c->gate, &c->up, &c->down}) {
    if (!w->Wq || !w->scales || !w->zeros) return W4A16_EINVAL;
    if (!aligned16({w->Wq, w->scales, w->zeros})) return W4A16_EALIGN;
  }
  if (!aligned16({c->X, c->ids, c->weights, c->s, c->s_down, c->residual, c->G, c->U, c->Y})) return W4A16_EALIGN;
  const w4a16::ExpertsDesc d = experts_desc(*c);
  const size_t need = w4a16::experts_workspace_bytes(d);
  if (!workspace || workspace_bytes < need) return W4A16_EINVAL;
  if (!aligned256(workspace)) return W4A16_EALIGN;
  const size_t rows = (size_t)(c->T * c->D) * 2, slots = (size_t)(c->T * c->k), kept = slots * c->N * 2;
  const size_t codes = (size_t)(c->E * (c->N * c->D / 2)), E = (size_t)c->E;
  const size_t meta_in = E * c->N * (size_t)((c->D / W4A16_GROUP + 3) / 4 * 4) * 2;
  const size_t meta_down = E * c->D * (size_t)((c->N / W4A16_GROUP + 3) / 4 * 4) * 2;
  if (overlaps({{c->Y, rows}, {c->G, kept}, {c->U, kept}, {workspace, need}},
               {{c->X, rows}, {c->ids, slots * 4}, {c->weights, slots * 4}, {c->gate.Wq, codes}, {c->up.Wq, codes},
                {c->down.Wq, codes}, {c->gate.scales, meta_in}, {c->gate.zeros, meta_in}, {c->up.scales, meta_in},
                {c->up.zeros, meta_in}, {c->down.scales, meta_down}, {c->down.zeros, meta_down},
                {c->s, (size_t)c->D * 2}, {c->s_down, E * c->N * 2}}, 0) ||
      overlaps({{c->G, kept}, {c->U, kept}, {workspace, need}}, {{c->residual, rows}}, 0) ||
      overlaps({{c->Y, rows}}, {{c->residual, rows}}, 1))
    return W4A16_EINVAL;
  return status(w4a16::launch_experts(d, workspace, static_cast<hipStream_t>(stream)));
}

int w4a16_experts_backward_workspace_size(const w4a16_experts_backward_call *c, size_t *bytes) {
  if (!c || !bytes) return W4A16_EINVAL;
  if (int rc = check_experts_shape(c->T, c->E, c->k, c->D, c->N, c->act, c->dtype)) return rc;
  *bytes = w4a16::experts_grad_workspace_bytes(experts_grad_desc(*c));
  return W4A16_OK;
}

int w4a16_experts_backward(const w4a16_experts_backward_call *c, void *workspace, size_t workspace_bytes,
                           void *stream) {
  if (!c) return W4A16_EINVAL;
  if (int rc = check_experts_shape(c->T, c->E, c->k, c->D, c->N, c->act, c->dtype)) return rc;
  if (c->T == 0) return W4A16_OK;
  if (!c->dY || !c->ids || !c->weights || !c->G || !c->U || (!c->dX && (!c->dweights || c->add)))
    return W4A16_EINVAL;
  for (const w4a16_expert_transposed *w : {&c->gate, &c->up, &c->down}) {
    if (!w->Wt || !w->meta) return W4A16_EINVAL;
    if (!aligned16({w->Wt, w->meta})) return W4A16_EALIGN;
  }
  if (!aligned16({c->dY, c->ids, c->weights, c->G, c->U, c->s, c->s_down, c->add, c->dX, c->dweights}))
    return W4A16_EALIGN;
  const w4a16::ExpertsGradDesc d = experts_grad_desc(*c);
  const size_t need = w4a16::experts_grad_workspace_bytes(d);
  if (!workspace || workspace_bytes < need) return W4A16_EINVAL;
  if (!aligned256(workspace)) return W4A16_EALIGN;
  const size_t rows = (size_t)(c->T * c->D) * 2, slots = (size_t)(c->T * c->k), kept = slots * c->N * 2;
  const size_t codes = (size_t)(c->E * (c->N * c->D / 2)), E = (size_t)c->E;
  const size_t meta = (size_t)(c->E * (c->N / W4A16_GROUP) * (c->D / W4A16_GROUP) * 512);
  const size_t grads = slots * (c->dweights_f32 ? 4 : 2);
  if (overlaps({{c->dX, rows}, {c->dweights, grads}, {workspace, need}},
               {{c->dY, rows}, {c->ids, slots * 4}, {c->weights, slots * 4}, {c->G, kept}, {c->U, kept},
                {c->gate.Wt, codes}, {c->up.Wt, codes}, {c->down.Wt, codes}, {c->gate.meta, meta}, {c->up.meta, meta},
                {c->down.meta, meta}, {c->s, (size_t)c->D * 2}, {c->s_down, E * c->N * 2}}, 0) ||
      overlaps({{c->dweights, grads}, {workspace, need}}, {{c->add, rows}}, 0) ||
      overlaps({{c->dX, rows}}, {{c->add, rows}}, 1))
    return W4A16_EINVAL;
  return status(w4a16::launch_experts_grad(d, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
