// Host side of the moe_block_* entry points (include/moe.h): argument
// validation and launches.
#include "api_common.hpp"

#include <math.h>

namespace {

using namespace moe::api;

constexpr int kMaxCols = 32768;      // a row in the registers of one block
constexpr int kMaxRows = 1 << 22;    // one block (of up to 1024 threads) per row in one launch

int validate_shape(const moe_block_shape* s) {
  if (s == nullptr || s->T < 0 || s->d <= 0 || s->gate_rows < 0) return MOE_ERR_INVALID_ARG;
  for (const int dt : {s->x_dtype, s->n_dtype, s->y_dtype})
    if (dt != MOE_DTYPE_F32 && dt != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(s->eps > 0.f) || !isfinite(s->eps) || !isfinite(s->res_scale)) return MOE_ERR_INVALID_ARG;
  if (s->d % 8 != 0 || s->d > kMaxCols || s->T >= kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

long long gate_len(const moe_block_shape& s) {   // rows per gate, at least 1
  const long long T = s.T > 0 ? s.T : 1;
  return s.gate_rows > 0 && s.gate_rows < T ? s.gate_rows : T;
}
long long gate_count(const moe_block_shape& s) {
  return s.gate_rows > 0 ? (static_cast<long long>(s.T) + s.gate_rows - 1) / s.gate_rows : 1;
}

// A required array of rows (none are read or written when T is 0).
bool rows_ok(const moe_block_shape& s, const void* p) { return s.T == 0 || (p != nullptr && aligned16(p)); }
bool optional_ok(const void* p) { return p == nullptr || aligned16(p); }

// A checkpoint is codes and scales together, over whole 128-column tiles.
int save_ok(const moe_block_shape& s, const moe_block_save* k) {
  if (k == nullptr) return MOE_OK;
  if ((k->codes == nullptr) != (k->scales == nullptr) || !optional_ok(k->codes)) return MOE_ERR_INVALID_ARG;
  if (k->codes != nullptr && s.d % 128 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t backward_bytes(const moe_block_shape& s) {
  const long long n = moe::block_bwd_floats(moe::block_bwd_plan(s.T, gate_len(s), gate_count(s), true), s.d);
  const long long T = s.T > 0 ? s.T : 1;
  const long long m = moe::block_bwd_floats(moe::block_bwd_plan(s.T, T, 1, false), s.d);
  return align_up(static_cast<size_t>(n > m ? n : m) * 4);
}

}  // namespace

extern "C" {

int moe_block_workspace_size(const moe_block_shape* shape, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  *bytes = backward_bytes(*shape);
  return MOE_OK;
}

int moe_block_in(const moe_block_shape* shape, const void* x, const float* w, void* n, const moe_block_save* save,
                 hipStream_t stream) {
  int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_block_shape& s = *shape;
  if (!rows_ok(s, x) || !rows_ok(s, n) || w == nullptr || !aligned16(w)) return MOE_ERR_INVALID_ARG;
  if ((rc = save_ok(s, save)) != MOE_OK) return rc;
  const moe_block_save k = save != nullptr ? *save : moe_block_save{};
  const moe::BlockInArgs a{x, w, s.T, s.d, fmt_of(s.x_dtype), fmt_of(s.n_dtype), s.eps, n, k.rstd, k.codes, k.scales};
  return debug_status(check_launch(moe::launch_block_in(a, stream)), stream, "moe_block_in");
}

int moe_block_out(const moe_block_shape* shape, const void* x, const void* y, const void* skip, const float* w,
                  const float* gate, const float* w_next, void* x_out, void* n_next, const moe_block_save* save,
                  const moe_block_save* save_next, hipStream_t stream) {
  int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_block_shape& s = *shape;
  if (!rows_ok(s, x) || !rows_ok(s, y) || !rows_ok(s, x_out) || !optional_ok(skip) || !optional_ok(w) ||
      !optional_ok(gate) || !optional_ok(w_next) || (w_next != nullptr && !rows_ok(s, n_next)))
    return MOE_ERR_INVALID_ARG;
  if (w_next == nullptr && save_next != nullptr) return MOE_ERR_INVALID_ARG;
  if ((rc = save_ok(s, save)) != MOE_OK || (rc = save_ok(s, save_next)) != MOE_OK) return rc;
  const moe_block_save k = save != nullptr ? *save : moe_block_save{};
  const moe_block_save kn = save_next != nullptr ? *save_next : moe_block_save{};
  moe::BlockOutArgs a{};
  a.x = x;
  a.y = y;
  a.skip = skip;
  a.w = w;
  a.gate = gate;
  a.w_next = w_next;
  a.T = s.T;
  a.d = s.d;
  a.x_fmt = fmt_of(s.x_dtype);
  a.n_fmt = fmt_of(s.n_dtype);
  a.y_fmt = fmt_of(s.y_dtype);
  a.gate_rows = s.gate_rows;
  a.gates = gate_count(s);
  a.eps = s.eps;
  a.res_scale = s.res_scale;
  a.x_out = x_out;
  a.n_next = n_next;
  a.rstd = k.rstd;
  a.codes = k.codes;
  a.scales = k.scales;
  a.rstd_next = kn.rstd;
  a.codes_next = kn.codes;
  a.scales_next = kn.scales;
  return debug_status(check_launch(moe::launch_block_out(a, stream)), stream, "moe_block_out");
}

int moe_block_in_backward(const moe_block_shape* shape, const float* dn, const float* dn_sub, const float* dout,
                          const void* x, const float* w, const moe_block_save* save, float* dx, float* dw,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_block_shape& s = *shape;
  if (!rows_ok(s, dn) || !rows_ok(s, dx) || !optional_ok(dn_sub) || !optional_ok(dout) || !optional_ok(x) ||
      w == nullptr || !aligned16(w) || dw == nullptr || !aligned16(dw))
    return MOE_ERR_INVALID_ARG;
  if ((rc = save_ok(s, save)) != MOE_OK) return rc;
  if (s.T > 0 && (save == nullptr || save->rstd == nullptr || (x == nullptr && save->codes == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < backward_bytes(s)) return MOE_ERR_WORKSPACE;
  const moe_block_save k = save != nullptr ? *save : moe_block_save{};
  moe::BlockBwdArgs a{};
  a.g = dn;
  a.g_sub = dn_sub;
  a.res = dout;
  a.v = x;
  if (x == nullptr) {
    a.codes = k.codes;
    a.scales = k.scales;
  }
  a.w = w;
  a.rstd = k.rstd;
  a.T = s.T;
  a.d = s.d;
  a.v_fmt = fmt_of(s.x_dtype);
  a.skip_fmt = moe::FMT_F32;
  a.gate_len = s.T > 0 ? s.T : 1;
  a.gates = 1;
  a.res_scale = s.res_scale;
  a.dv = dx;
  a.dw = dw;
  a.part = static_cast<float*>(workspace);
  return debug_status(check_launch(moe::launch_block_bwd(a, stream)), stream, "moe_block_in_backward");
}

int moe_block_out_backward(const moe_block_shape* shape, const float* dout, const void* y, const void* skip,
                           const float* w, const float* gate, const moe_block_save* save, float* dy, float* dw,
                           float* dgate, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_block_shape& s = *shape;
  if (!rows_ok(s, dout) || !rows_ok(s, dy) || !optional_ok(y) || !optional_ok(skip) || !optional_ok(w) ||
      !optional_ok(gate) || !optional_ok(dw) || !optional_ok(dgate))
    return MOE_ERR_INVALID_ARG;
  if ((w == nullptr) != (dw == nullptr) || (gate == nullptr) != (dgate == nullptr)) return MOE_ERR_INVALID_ARG;
  if (y == nullptr && skip != nullptr) return MOE_ERR_INVALID_ARG;
  if ((rc = save_ok(s, save)) != MOE_OK) return rc;
  const moe_block_save k = save != nullptr ? *save : moe_block_save{};
  if (s.T > 0 && w != nullptr && k.rstd == nullptr) return MOE_ERR_INVALID_ARG;
  if (s.T > 0 && (w != nullptr || gate != nullptr) && y == nullptr && k.codes == nullptr) return MOE_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < backward_bytes(s)) return MOE_ERR_WORKSPACE;
  moe::BlockBwdArgs a{};
  a.g = dout;
  a.v = y;
  a.skip = skip;
  if (y == nullptr) {
    a.codes = k.codes;
    a.scales = k.scales;
  }
  a.w = w;
  a.gate = gate;
  a.rstd = k.rstd;
  a.T = s.T;
  a.d = s.d;
  a.v_fmt = fmt_of(s.y_dtype);
  a.skip_fmt = fmt_of(s.n_dtype);
  a.gate_len = gate != nullptr ? gate_len(s) : (s.T > 0 ? s.T : 1);
  a.gates = gate != nullptr ? gate_count(s) : 1;
  a.res_scale = s.res_scale;
  a.dv = dy;
  a.dw = dw;
  a.dgate = dgate;
  a.part = static_cast<float*>(workspace);
  return debug_status(check_launch(moe::launch_block_bwd(a, stream)), stream, "moe_block_out_backward");
}

}  // extern "C"
