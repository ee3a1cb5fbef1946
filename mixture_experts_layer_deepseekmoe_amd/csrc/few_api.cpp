// Host side of moe_forward_few (include/moe.h): argument validation, workspace
// carving and the launch sequence.
#include "api_common.hpp"

namespace {

using namespace moe::api;

constexpr int kMaxCols = 32768;   // of d and I: a token's and an expert's rows are addressed with 32-bit byte offsets

int validate_few(const moe_shape* s) {
  const int rc = layer_shape_status(s);
  if (rc != MOE_OK) return rc;
  if (s->T > moe::FEW_TOKENS || s->d > kMaxCols || s->inter > kMaxCols) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace map (byte offsets, each 256-byte aligned).
struct Layout {
  size_t taken, logits, idx, gate, h, hq, hs, uq, us, part, total;
  int slices, splits;
};

Layout make_layout(const moe_shape& s) {
  Layout L{};
  const size_t T = static_cast<size_t>(s.T), K = static_cast<size_t>(s.top_k), R = T * (K + s.n_shared);
  const size_t d = static_cast<size_t>(s.d), I = static_cast<size_t>(s.inter);
  const bool fp8 = s.w_dtype == MOE_DTYPE_E4M3;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align_up(bytes); return at; };
  L.slices = moe::few_slices(s.d, fmt_of(s.x_dtype));
  L.taken = take(4);
  L.logits = take(L.slices * T * s.n_routed * 4);
  L.idx = take(T * K * 4);
  L.gate = take(T * K * 4);
  L.h = take(R * I * 4);   // fp32 values or pairs of bf16 ones
  L.hq = take(fp8 ? R * I : 0);
  L.hs = take(fp8 ? R * (I / 128) * 4 : 0);
  L.uq = take(fp8 ? T * d : 0);
  L.us = take(fp8 ? T * (d / 128) * 4 : 0);
  L.splits = moe::few_splits(s.T, s.d, s.n_routed, s.n_shared, s.inter, s.top_k, fmt_of(s.w_dtype));
  L.part = take(L.splits > 1 ? L.splits * T * d * 4 : 0);
  L.total = o;
  return L;
}

}  // namespace

extern "C" {

int moe_few_workspace_size(const moe_shape* shape, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const int rc = validate_few(shape);
  if (rc != MOE_OK) return rc;
  *bytes = make_layout(*shape).total;
  return MOE_OK;
}

int moe_forward_few(const moe_shape* shape, const void* u, const void* centroids, const float* bias,
                    const moe_weights* wt, void* y, const moe_routing* routing, void* workspace, size_t workspace_bytes,
                    const moe_trace* trace, hipStream_t stream) {
  int rc = validate_few(shape);
  if (rc != MOE_OK) return rc;
  if ((rc = layer_args_status(shape, u, centroids, bias, wt, y)) != MOE_OK) return rc;
  const moe_shape& s = *shape;
  const Layout L = make_layout(s);
  if (s.T > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < L.total)) return MOE_ERR_WORKSPACE;
  moe_routing r{};
  if (routing != nullptr) r = *routing;
  moe::FewArgs a{};
  a.u = u;
  a.centroids = centroids;
  a.bias = bias;
  a.w_gate_up = wt->w_gate_up;
  a.w_down = wt->w_down;
  a.ws_gate_up = wt->ws_gate_up;
  a.ws_down = wt->ws_down;
  a.s_gate_up = wt->s_gate_up;
  a.s_down = wt->s_down;
  a.ss_gate_up = wt->ss_gate_up;
  a.ss_down = wt->ss_down;
  a.T = s.T;
  a.d = s.d;
  a.n_routed = s.n_routed;
  a.n_shared = s.n_shared;
  a.inter = s.inter;
  a.top_k = s.top_k;
  a.n_groups = layer_groups(s);
  a.topk_groups = layer_topk_groups(s);
  a.x_fmt = fmt_of(s.x_dtype);
  a.w_fmt = fmt_of(s.w_dtype);
  a.out_fmt = fmt_of(s.out_dtype);
  a.slices = L.slices;
  a.splits = L.splits;
  a.counts = r.expert_counts;
  a.offsets = r.expert_offsets;
  a.perm_token = r.perm_token;
  a.pos = r.pos;
  a.y = y;
  if (s.T > 0) {
    a.taken = at<int32_t>(workspace, L.taken);
    a.logits = at<float>(workspace, L.logits);
    a.idx = r.topk_idx != nullptr ? r.topk_idx : at<int32_t>(workspace, L.idx);
    a.gate = r.topk_gate != nullptr ? r.topk_gate : at<float>(workspace, L.gate);
    a.h = at<void>(workspace, L.h);
    a.h_lo = at<uint16_t>(workspace, L.h) + static_cast<size_t>(s.T) * (s.top_k + s.n_shared) * s.inter;
    a.hq = at<uint8_t>(workspace, L.hq);
    a.hs = at<float>(workspace, L.hs);
    a.uq = at<uint8_t>(workspace, L.uq);
    a.us = at<float>(workspace, L.us);
    a.part = at<float>(workspace, L.part);
  }
  // an empty batch still has a routing: no expert has a row
  const bool rows = s.T > 0, fp8 = s.w_dtype == MOE_DTYPE_E4M3;
  const Stages stg{trace, stream};
  stg.begin(MOE_STAGE_ROUTE);
  if (rows) rc = check_launch(moe::launch_few_route(a, stream));
  if (rc != MOE_OK) return rc;
  stg.end(MOE_STAGE_ROUTE);
  stg.begin(MOE_STAGE_GATE_UP);
  if (rows || a.counts != nullptr || a.offsets != nullptr) rc = check_launch(moe::launch_few_gateup(a, stream));
  if (rc != MOE_OK) return rc;
  stg.end(MOE_STAGE_GATE_UP);
  stg.begin(MOE_STAGE_QUANT);
  if (rows && fp8) rc = check_launch(moe::launch_few_quant(a, stream));
  if (rc != MOE_OK) return rc;
  stg.end(MOE_STAGE_QUANT);
  stg.begin(MOE_STAGE_DOWN);
  if (rows) rc = check_launch(moe::launch_few_down(a, stream));
  if (rc != MOE_OK) return rc;
  stg.end(MOE_STAGE_DOWN);
  for (const int i : {MOE_STAGE_GROUP, MOE_STAGE_COMBINE}) {   // parts of the others
    stg.begin(i);
    stg.end(i);
  }
  return debug_status(MOE_OK, stream, "moe_forward_few");
}

}  // extern "C"
