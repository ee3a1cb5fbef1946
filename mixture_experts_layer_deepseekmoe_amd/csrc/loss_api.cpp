// Host side of the moe_vocab_loss* entry points (include/moe.h): argument
// validation, workspace carving and the launch sequence.
#include "api_common.hpp"

namespace {

using namespace moe::api;

constexpr long long kMaxPartials = 64LL << 30;
constexpr int kMaxTokens = 1 << 22;   // (T + 64) rows of G's smallest piece stay below 2^32 bytes

int validate_shape(const moe_loss_shape* s) {
  if (s == nullptr || s->T < 0 || s->d <= 0 || s->V <= 0) return MOE_ERR_INVALID_ARG;
  for (const int dt : {s->dh_dtype, s->dw_dtype})
    if (dt != MOE_DTYPE_F32 && dt != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (s->d % 64 != 0 || s->d > 32768 || s->T >= kMaxTokens || s->V > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  // the hidden rows are addressed with 32-bit byte offsets, a K-step of rows past their end
  if ((static_cast<long long>(s->T) + 64) * s->d * 2 >= (1LL << 32)) return MOE_ERR_UNSUPPORTED;
  // the forward's (max, sum) of every token and tile of 256 entries: 64 GiB of workspace (the kernels
  // themselves walk any number of tiles)
  const long long tiles = (static_cast<long long>(s->T) + 255) / 256 * ((s->V + 255LL) / 256);
  if (tiles * 256 * static_cast<long long>(sizeof(float2)) > kMaxPartials) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace map (byte offsets, each 256-byte aligned).
struct Layout {
  size_t rows, pos, count, part, zlab, forward_total;
  size_t lab_lo, lab_first, lab_list, hc, g, acc, backward_total;
  int piece;
};

Layout make_layout(const moe_loss_shape& s) {
  Layout L{};
  const size_t T = static_cast<size_t>(s.T), nv = static_cast<size_t>(moe::loss_tiles(s.T, s.d, s.V));
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align_up(bytes); return at; };
  L.count = take(12);
  L.rows = take(T * 4);
  L.pos = take(T * 4);
  const size_t shared = o;
  L.part = take(nv * T * sizeof(float2));
  L.zlab = take(T * 4);
  L.forward_total = o;
  o = shared;
  const bool pairs = moe::loss_pairs(fmt_of(s.dh_dtype), fmt_of(s.dw_dtype));
  L.piece = moe::loss_piece(s.T, s.d, s.V, pairs);
  L.lab_lo = take(T * 4);
  const bool labels = moe::loss_labels(s.T, fmt_of(s.dw_dtype));
  L.lab_first = take(labels ? (static_cast<size_t>((s.V + moe::LOSS_TILE - 1) / moe::LOSS_TILE) + 1) * 4 : 0);
  L.lab_list = take(labels ? T * 4 : 0);
  L.hc = take(static_cast<size_t>(moe::loss_k_rows(s.T)) * s.d * 2);
  L.g = take(static_cast<size_t>(moe::loss_g_rows(s.T, pairs)) * L.piece * 2);
  L.acc = take(static_cast<size_t>(moe::loss_acc_rows(s.T, s.d, L.piece)) * s.d * 4);
  L.backward_total = o;
  return L;
}

moe::LossArgs make_args(const moe_loss_shape& s, const Layout& L, const void* h, const void* w, const int32_t* labels,
                        void* ws) {
  moe::LossArgs a{};
  a.h = static_cast<const uint16_t*>(h);
  a.w = static_cast<const uint16_t*>(w);
  a.labels = labels;
  a.T = s.T;
  a.d = s.d;
  a.V = s.V;
  a.rows = at<int32_t>(ws, L.rows);
  a.count = at<int32_t>(ws, L.count);
  return a;
}

bool rows_ok(const moe_loss_shape& s, const void* p) { return s.T == 0 || (p != nullptr && aligned16(p)); }

}  // namespace

extern "C" {

int moe_vocab_loss_workspace_size(const moe_loss_shape* shape, size_t* forward_bytes, size_t* backward_bytes) {
  if (forward_bytes == nullptr && backward_bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const Layout L = make_layout(*shape);
  if (forward_bytes != nullptr) *forward_bytes = L.forward_total;
  if (backward_bytes != nullptr) *backward_bytes = L.backward_total;
  return MOE_OK;
}

int moe_vocab_loss(const moe_loss_shape* shape, const void* h, const void* w, const int32_t* labels, float* loss,
                   float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_loss_shape& s = *shape;
  if (!rows_ok(s, h) || w == nullptr || !aligned16(w) || (s.T > 0 && (labels == nullptr || loss == nullptr || lse == nullptr)))
    return MOE_ERR_INVALID_ARG;
  const Layout L = make_layout(s);
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < L.forward_total) return MOE_ERR_WORKSPACE;
  if (s.T == 0) return MOE_OK;
  moe::LossArgs a = make_args(s, L, h, w, labels, workspace);
  a.loss = loss;
  a.lse = lse;
  a.part = at<float2>(workspace, L.part);
  a.zlab = at<float>(workspace, L.zlab);
  a.tiles = moe::loss_tiles(s.T, s.d, s.V);
  a.v_len = s.V;
  return debug_status(check_launch(moe::launch_loss_forward(a, stream)), stream, "moe_vocab_loss");
}

int moe_vocab_loss_backward(const moe_loss_shape* shape, const void* h, const void* w, const int32_t* labels,
                            const float* lse, const float* dloss, const float* dlse, void* dh, void* dw,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_loss_shape& s = *shape;
  if (!rows_ok(s, h) || !rows_ok(s, dh) || w == nullptr || !aligned16(w) || dw == nullptr || !aligned16(dw) ||
      (s.T > 0 && (labels == nullptr || lse == nullptr || dloss == nullptr)))
    return MOE_ERR_INVALID_ARG;
  const Layout L = make_layout(s);
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < L.backward_total) return MOE_ERR_WORKSPACE;
  moe::LossArgs a = make_args(s, L, h, w, labels, workspace);
  a.pos = at<int32_t>(workspace, L.pos);
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dlse = dlse;
  a.lab_lo = at<float>(workspace, L.lab_lo);
  a.lab_first = at<int32_t>(workspace, L.lab_first);
  a.lab_list = at<uint32_t>(workspace, L.lab_list);
  a.hc = at<uint16_t>(workspace, L.hc);
  a.g = at<uint16_t>(workspace, L.g);
  a.acc = at<float>(workspace, L.acc);
  a.ldg = L.piece;
  a.g_rows = moe::loss_g_rows(s.T, moe::loss_pairs(fmt_of(s.dh_dtype), fmt_of(s.dw_dtype)));
  a.acc_rows = moe::loss_acc_rows(s.T, s.d, L.piece);
  a.dh_fmt = fmt_of(s.dh_dtype);
  a.dw_fmt = fmt_of(s.dw_dtype);
  a.dh = dh;
  a.dw = dw;
  int r = check_launch(moe::launch_loss_rows(a, stream));
  if (r == MOE_OK) r = check_launch(moe::launch_loss_gather(a, stream));
  for (int v = 0; v < s.V && r == MOE_OK; v += L.piece) {
    a.v_first = v;
    a.v_len = s.V - v < L.piece ? s.V - v : L.piece;
    r = check_launch(moe::launch_loss_piece(a, stream));
  }
  if (r == MOE_OK) r = check_launch(moe::launch_loss_dh(a, stream));
  return debug_status(r, stream, "moe_vocab_loss_backward");
}

}  // extern "C"
