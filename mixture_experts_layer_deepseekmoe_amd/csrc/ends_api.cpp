// Host side of the moe_embed* and moe_grad_* entry points (include/moe.h):
// argument validation, workspace carving and the launch sequence.
#include "api_common.hpp"

#include <math.h>

#include <algorithm>
#include <new>

namespace {

using namespace moe::api;

constexpr int kMaxCols = 32768;      // a row in the registers of one block
constexpr int kMaxTokens = 1 << 22;  // one block per row in one launch
constexpr int kMaxVocab = 1 << 24;

int validate_shape(const moe_embed_shape* s) {
  if (s == nullptr || s->T < 0 || s->d <= 0 || s->V <= 0) return MOE_ERR_INVALID_ARG;
  for (const int dt : {s->table_dtype, s->x_dtype, s->n_dtype, s->grad_dtype})
    if (dt != MOE_DTYPE_F32 && dt != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (!isfinite(s->scale) || !(s->eps > 0.f) || !isfinite(s->eps)) return MOE_ERR_INVALID_ARG;
  if (s->d % 8 != 0 || s->d > kMaxCols || s->T >= kMaxTokens || s->V > kMaxVocab) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool rows_ok(const moe_embed_shape& s, const void* p) { return s.T == 0 || (p != nullptr && aligned16(p)); }
bool tokens_ok(const moe_embed_shape& s, const int32_t* p) { return s.T == 0 || (p != nullptr && aligned4(p)); }

// Workspace map of the backward (byte offsets, each 256-byte aligned).
struct Layout {
  size_t ids, order, ids2, order2, hist, part, part2, total;
};
Layout make_layout(const moe_embed_shape& s) {
  Layout L{};
  const size_t T = static_cast<size_t>(s.T), blocks = static_cast<size_t>(moe::embed_radix_blocks(s.T));
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align_up(bytes); return at; };
  L.ids = take(T * 4);
  L.order = take(T * 4);
  L.ids2 = take(blocks > 0 ? T * 4 : 0);
  L.order2 = take(blocks > 0 ? T * 4 : 0);
  L.hist = take(blocks * 256 * 4);
  L.part = take(T / moe::EMBED_CHUNK * s.d * 4);
  L.part2 = take(T >= moe::EMBED_PART2_T ? T / moe::EMBED_CHUNK2 * s.d * 4 : 0);
  L.total = o;
  return L;
}

// ---- gradient tensors

constexpr long long kMaxElements = 1LL << 43;   // of all tensors: their chunks are counted in 32 bits

int tensor_ok(const moe_tensor& t) {
  if (t.numel < 0 || (t.dtype != MOE_DTYPE_F32 && t.dtype != MOE_DTYPE_BF16)) return MOE_ERR_INVALID_ARG;
  if (t.numel > kMaxElements) return MOE_ERR_UNSUPPORTED;
  if (t.numel > 0 && (t.data == nullptr || reinterpret_cast<uintptr_t>(t.data) % elem_bytes(t.dtype) != 0))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct Range {
  uintptr_t lo, hi;
};

// Every tensor is valid, `out` (nullable) fits, and no two share memory, nor the sum or
// the norm (nullable) with any, but for an output that is its input.
int tensors_ok(const moe_tensor* in, const moe_tensor* out, int n, const double* sumsq, const float* norm) {
  if (n < 0 || (n > 0 && in == nullptr)) return MOE_ERR_INVALID_ARG;
  Range* const r = new (std::nothrow) Range[2 * static_cast<size_t>(n) + 2];
  if (r == nullptr) return MOE_ERR_UNSUPPORTED;
  int rc = MOE_OK;
  size_t m = 0;
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(sumsq), n0 = reinterpret_cast<uintptr_t>(norm);
  r[m++] = {s0, s0 + sizeof(double)};
  if (norm != nullptr) r[m++] = {n0, n0 + sizeof(float)};
  long long total = 0;
  for (int i = 0; i < n && rc == MOE_OK; ++i) {
    rc = tensor_ok(in[i]);
    if (rc != MOE_OK || in[i].numel == 0) {
      if (rc == MOE_OK && out != nullptr && out[i].numel != 0) rc = MOE_ERR_INVALID_ARG;
      continue;
    }
    total += in[i].numel;
    if (total > kMaxElements) rc = MOE_ERR_UNSUPPORTED;
    const uintptr_t a = reinterpret_cast<uintptr_t>(in[i].data);
    r[m++] = {a, a + static_cast<uintptr_t>(in[i].numel) * elem_bytes(in[i].dtype)};
    if (out == nullptr || rc != MOE_OK) continue;
    rc = tensor_ok(out[i]);
    if (rc == MOE_OK && out[i].numel != in[i].numel) rc = MOE_ERR_INVALID_ARG;
    if (rc != MOE_OK || (out[i].data == in[i].data && out[i].dtype == in[i].dtype)) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(out[i].data);
    r[m++] = {b, b + static_cast<uintptr_t>(out[i].numel) * elem_bytes(out[i].dtype)};
  }
  if (rc == MOE_OK) {
    std::sort(r, r + m, [](const Range& x, const Range& y) { return x.lo < y.lo; });
    for (size_t i = 1; i < m; ++i)
      if (r[i].lo < r[i - 1].hi) rc = MOE_ERR_INVALID_ARG;
  }
  delete[] r;
  return rc;
}

// Calls f with the tensors from `at` on that fit one launch, and returns where the next begin.
int fill(moe::GradArgs& a, const moe_tensor* in, const moe_tensor* out, int n, int at) {
  a.n = 0;
  a.first[0] = 0;
  for (; at < n && a.n < moe::GRAD_TENSORS; ++at) {
    if (in[at].numel == 0) continue;
    const int k = a.n++;
    const moe_tensor& o = out != nullptr ? out[at] : in[at];
    a.data[k] = in[at].data;
    a.out[k] = o.data;
    a.numel[k] = in[at].numel;
    a.bf16[k] = (in[at].dtype == MOE_DTYPE_BF16 ? 1 : 0) | (o.dtype == MOE_DTYPE_BF16 ? 2 : 0);
    a.first[k + 1] = a.first[k] + static_cast<uint32_t>((in[at].numel + moe::GRAD_CHUNK - 1) / moe::GRAD_CHUNK);
  }
  return at;
}

size_t grad_bytes(int n) {
  const size_t launches = (static_cast<size_t>(n) + moe::GRAD_TENSORS - 1) / moe::GRAD_TENSORS;
  return align_up((launches > 0 ? launches : 1) * moe::GRAD_BLOCKS * sizeof(double));
}

}  // namespace

extern "C" {

int moe_embed(const moe_embed_shape* shape, const int32_t* tokens, const void* table, const float* w_next, void* x,
              void* n_next, const moe_block_save* save_next, hipStream_t stream) {
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_embed_shape& s = *shape;
  if (!tokens_ok(s, tokens) || table == nullptr || !aligned16(table) || !rows_ok(s, x)) return MOE_ERR_INVALID_ARG;
  if (w_next != nullptr && (!aligned16(w_next) || !rows_ok(s, n_next))) return MOE_ERR_INVALID_ARG;
  if (w_next == nullptr && (n_next != nullptr || save_next != nullptr)) return MOE_ERR_INVALID_ARG;
  const moe_block_save k = save_next != nullptr ? *save_next : moe_block_save{};
  if ((k.codes == nullptr) != (k.scales == nullptr) || !aligned16(k.codes)) return MOE_ERR_INVALID_ARG;
  if (k.codes != nullptr && s.d % 128 != 0) return MOE_ERR_UNSUPPORTED;
  const moe::EmbedArgs a{tokens, table, w_next, s.T, s.d, s.V, fmt_of(s.table_dtype), fmt_of(s.x_dtype),
                         fmt_of(s.n_dtype), s.scale, s.eps, x, n_next, k.rstd, k.codes, k.scales};
  return debug_status(check_launch(moe::launch_embed(a, stream)), stream, "moe_embed");
}

int moe_embed_workspace_size(const moe_embed_shape* shape, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  *bytes = make_layout(*shape).total;
  return MOE_OK;
}

int moe_embed_backward(const moe_embed_shape* shape, const int32_t* tokens, const float* dx, void* dtable,
                       int32_t accumulate, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int rc = validate_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_embed_shape& s = *shape;
  if (!tokens_ok(s, tokens) || !rows_ok(s, dx) || dtable == nullptr || !aligned16(dtable)) return MOE_ERR_INVALID_ARG;
  const Layout L = make_layout(s);
  if (s.T > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < L.total)) return MOE_ERR_WORKSPACE;
  moe::EmbedBwdArgs a{};
  a.tokens = tokens;
  a.dx = dx;
  a.T = s.T;
  a.d = s.d;
  a.V = s.V;
  a.grad_fmt = fmt_of(s.grad_dtype);
  a.accumulate = accumulate != 0;
  a.scale = s.scale;
  a.dtable = dtable;
  if (s.T > 0) {
    a.ids = at<int32_t>(workspace, L.ids);
    a.order = at<int32_t>(workspace, L.order);
    a.ids2 = at<int32_t>(workspace, L.ids2);
    a.order2 = at<int32_t>(workspace, L.order2);
    a.hist = at<int32_t>(workspace, L.hist);
    a.part = at<float>(workspace, L.part);
    a.part2 = at<float>(workspace, L.part2);
  }
  return debug_status(check_launch(moe::launch_embed_bwd(a, stream)), stream, "moe_embed_backward");
}

int moe_grad_workspace_size(int32_t n, size_t* bytes) {
  if (bytes == nullptr || n < 0) return MOE_ERR_INVALID_ARG;
  *bytes = grad_bytes(n);
  return MOE_OK;
}

int moe_grad_sumsq(const moe_tensor* tensors, int32_t n, double* sumsq, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
  if (sumsq == nullptr || (reinterpret_cast<uintptr_t>(sumsq) & 7u) != 0) return MOE_ERR_INVALID_ARG;
  int rc = tensors_ok(tensors, nullptr, n, sumsq, nullptr);
  if (rc != MOE_OK) return rc;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < grad_bytes(n)) return MOE_ERR_WORKSPACE;
  double* const part = static_cast<double*>(workspace);
  long long parts = 0;
  moe::GradArgs a;
  for (int i = 0; i < n && rc == MOE_OK;) {
    i = fill(a, tensors, nullptr, n, i);
    rc = check_launch(moe::launch_grad_sumsq(a, part + parts, stream));
    parts += moe::grad_blocks(a);
  }
  if (rc == MOE_OK) rc = check_launch(moe::launch_grad_finish(part, parts, sumsq, stream));
  return debug_status(rc, stream, "moe_grad_sumsq");
}

int moe_grad_clip(const moe_tensor* tensors, const moe_tensor* out, int32_t n, const double* sumsq, double max_norm,
                  float* norm, hipStream_t stream) {
  if (sumsq == nullptr || (reinterpret_cast<uintptr_t>(sumsq) & 7u) != 0 || !aligned4(norm) || !(max_norm > 0.0))
    return MOE_ERR_INVALID_ARG;
  int rc = tensors_ok(tensors, out, n, sumsq, norm);
  if (rc != MOE_OK) return rc;
  // from the last tensors to the first, as the kernel goes through a launch's: what the sum read last
  moe::GradArgs a;
  const int launches = (n + moe::GRAD_TENSORS - 1) / moe::GRAD_TENSORS;
  for (int l = launches - 1; l >= 0 && rc == MOE_OK; --l) {
    const int first = l * moe::GRAD_TENSORS, last = n < first + moe::GRAD_TENSORS ? n : first + moe::GRAD_TENSORS;
    fill(a, tensors, out, last, first);
    rc = check_launch(moe::launch_grad_clip(a, sumsq, max_norm, l == 0 ? norm : nullptr, stream));
  }
  if (n == 0 && norm != nullptr) {
    a.n = 0;
    a.first[0] = 0;
    rc = check_launch(moe::launch_grad_clip(a, sumsq, max_norm, norm, stream));
  }
  return debug_status(rc, stream, "moe_grad_clip");
}

}  // extern "C"
