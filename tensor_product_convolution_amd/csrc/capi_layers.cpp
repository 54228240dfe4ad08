// C ABI of the layers around the convolution: argument checks (all before any
// HIP call) and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>

#include "capi_checks.hpp"

using namespace tpc;

namespace {

constexpr const char* kTooMany = "too many nodes or structures for one launch";

tp_status check_drop(const char* where, const tp_dropout* d, DropArgs* out) {
  if (!(d->p >= 0.0 && d->p < 1.0)) return fail(where, "dropout probability must be in [0, 1)");
  out->k0 = (uint32_t)d->seed;
  out->k1 = (uint32_t)(d->seed >> 32);
  out->o0 = (uint32_t)d->offset;
  out->o1 = (uint32_t)(d->offset >> 32);
  out->threshold = (uint32_t)(d->p * 4294967296.0);
  out->factor = (float)(1.0 / (1.0 - d->p));
  return TP_OK;
}

tp_status check_rows(const char* where, int32_t dtype, int64_t n_rows, int32_t n_cols) {
  if (!known(dtype)) return fail(where, "unknown element type");
  if (n_rows < 0 || n_cols < 0) return fail(where, "negative size");
  if (n_cols < 1 || n_cols > kNormMaxCols) return fail(where, "rows of 1 to 8192 values only", TP_ERR_UNSUPPORTED);
  if (n_rows > std::numeric_limits<int64_t>::max() / 64 / n_cols) return fail(where, "too many rows", TP_ERR_OVERFLOW);
  return TP_OK;
}

// sizes and options of an attention description (no pointers)
tp_status check_attn(const char* where, const tp_attn* a) {
  if (!a) return fail(where, "description is NULL");
  if (!known(a->dtype)) return fail(where, "unknown element type");
  if (a->n_nodes < 0 || a->n_segments < 0) return fail(where, "negative size");
  if (a->n_nodes > 0 && a->n_segments == 0) return fail(where, "nodes without a structure");
  // row numbers run up to eight tiles past the end, tile numbers to one for every 32 nodes and
  // one for every structure
  if (a->n_nodes > std::numeric_limits<int32_t>::max() - 4096 ||
      (int64_t)a->n_nodes / 32 + a->n_segments > std::numeric_limits<int32_t>::max())
    return fail(where, "too many nodes or structures for one launch", TP_ERR_OVERFLOW);
  if (a->n_heads < 1 || a->n_kv_heads < 1 || a->n_heads % a->n_kv_heads)
    return fail(where, "n_heads must be a positive multiple of n_kv_heads");
  if (a->n_heads > 1024) return fail(where, "at most 1024 heads", TP_ERR_UNSUPPORTED);
  if (a->head_dim < 8 || a->head_dim > 128 || a->head_dim % 8)
    return fail(where, "head_dim must be a multiple of 8 in 8..128", TP_ERR_UNSUPPORTED);
  const float size = std::fabs(a->scale);
  if (!(size == 0.f || (size >= 1e-8f && size <= 1e8f))) return fail(where, "scale must be 0 or of size 1e-8 to 1e8");
  if (a->n_buckets < 0) return fail(where, "negative n_buckets");
  if (a->n_buckets > 64) return fail(where, "at most 64 buckets", TP_ERR_UNSUPPORTED);
  if (a->n_buckets > 0) {
    if (a->steps != 1 && a->steps != 2 && a->steps != 4 && a->steps != 8) return fail(where, "steps must be 1, 2, 4 or 8");
    if (!(a->r_min >= 1e-15f && a->r_min <= 1e15f)) return fail(where, "r_min must be in [1e-15, 1e15]");
  }
  return TP_OK;
}

tp_status check_attn_pointers(const char* where, const tp_attn* a) {
  if (!a->seg_ptr) return fail(where, "seg_ptr is NULL");
  if (a->n_buckets > 0 && (!a->pos || !a->bias)) return fail(where, "a bias needs pos and bias");
  if (!aligned(a->seg_ptr, 4) || !aligned(a->pos, 4) || !aligned(a->bias, size_of(a->dtype)))
    return fail(where, "misaligned pointer");
  return TP_OK;
}

struct Rows {
  const void* p;
  int64_t stride;
  int heads;
};

// rows of heads x head_dim that move in 16-byte pieces
tp_status check_attn_rows(const char* where, const tp_attn& a, const Rows& r) {
  const int64_t es = size_of(a.dtype);
  if (a.n_nodes > 0 && !r.p) return fail(where, "NULL pointer");
  if (bad_stride(r.stride, (int64_t)r.heads * a.head_dim, a.n_nodes))
    return fail(where, "row stride below the row length, or too large");
  if (!aligned(r.p, 16) || r.stride * es % 16) return fail(where, "rows must be 16-byte aligned");
  return TP_OK;
}

}  // namespace

extern "C" {

tp_status tp_dropout_apply(int32_t dtype, int64_t n, const void* x, const void* residual, const tp_dropout* drop,
                           void* out, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_dropout_apply";
    if (!known(dtype)) return fail(me, "unknown element type");
    if (n < 0) return fail(me, "negative size");
    if (!drop) return fail(me, "drop is NULL");
    if (n > 0 && (!x || !out)) return fail(me, "NULL pointer");
    if (n >= (int64_t)1 << 40) return fail(me, "too many elements for one launch", TP_ERR_OVERFLOW);
    const int64_t es = size_of(dtype);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(out, es)) return fail(me, "misaligned pointer");
    DropArgs d;
    tp_status s = check_drop(me, drop, &d);
    if (s != TP_OK || n == 0) return s;
    hipError_t e = dropout_apply(dtype, n, x, residual, d, out, stream);
    return e == hipSuccess ? TP_OK : hip_error(e, "tp_dropout_apply launch");
  });
}

tp_status tp_layer_norm_forward(int32_t dtype, int64_t n_rows, int32_t n_cols, const void* x, int64_t x_stride,
                                const void* residual, const tp_dropout* drop, const float* gamma, const float* beta,
                                float eps, void* y, int64_t y_stride, void* h, float* mean, float* rstd,
                                hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_layer_norm_forward";
    tp_status s = check_rows(me, dtype, n_rows, n_cols);
    if (s != TP_OK) return s;
    if (bad_stride(x_stride, n_cols, n_rows) || bad_stride(y_stride, n_cols, n_rows))
      return fail(me, "row stride below the row length, or too large");
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(me, "eps must be finite and not negative");
    if (residual ? !h : (h || drop)) return fail(me, "h goes with a residual, drop too");
    if (n_rows > 0 && (!x || !gamma || !beta || !y || !mean || !rstd)) return fail(me, "NULL pointer");
    const int64_t es = size_of(dtype);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(h, es) || !aligned(gamma, 4) ||
        !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
      return fail(me, "misaligned pointer");
    NormArgs a;
    if (drop && (s = check_drop(me, drop, &a.drop)) != TP_OK) return s;
    if (n_rows == 0) return TP_OK;
    a.dtype = dtype;
    a.n_cols = n_cols;
    a.n_rows = n_rows;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.x = x;
    a.residual = residual;
    a.has_drop = drop != nullptr;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.y = y;
    a.h = h;
    a.mean = mean;
    a.rstd = rstd;
    a.stream = stream;
    hipError_t e = norm_forward(a);
    return e == hipSuccess ? TP_OK : hip_error(e, "tp_layer_norm_forward launch");
  });
}

tp_status tp_layer_norm_workspace(int32_t dtype, int64_t n_rows, int32_t n_cols, size_t* bytes) {
  return guarded([&]() -> tp_status {
    if (!bytes) return fail("tp_layer_norm_workspace", "bytes is NULL");
    tp_status s = check_rows("tp_layer_norm_workspace", dtype, n_rows, n_cols);
    if (s == TP_OK) *bytes = norm_workspace_bytes(dtype, n_rows, n_cols);
    return s;
  });
}

tp_status tp_layer_norm_backward(int32_t dtype, int64_t n_rows, int32_t n_cols, const void* grad_y, int64_t gy_stride,
                                 const void* h, int64_t h_stride, const float* gamma, const float* mean,
                                 const float* rstd, const void* grad_res, const tp_dropout* drop, void* grad_h,
                                 void* grad_x, float* grad_gamma, float* grad_beta, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_layer_norm_backward";
    tp_status s = check_rows(me, dtype, n_rows, n_cols);
    if (s != TP_OK) return s;
    if (bad_stride(gy_stride, n_cols, n_rows) || bad_stride(h_stride, n_cols, n_rows))
      return fail(me, "row stride below the row length, or too large");
    if (n_rows > 0 && (!grad_y || !h || !gamma || !mean || !rstd || !grad_h)) return fail(me, "NULL pointer");
    if (!grad_gamma != !grad_beta) return fail(me, "grad_gamma and grad_beta are given together");
    if (grad_x && !drop) return fail(me, "grad_x needs drop");
    const int64_t es = size_of(dtype);
    if (!aligned(grad_y, es) || !aligned(h, es) || !aligned(grad_res, es) || !aligned(grad_h, es) ||
        !aligned(grad_x, es) || !aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(grad_gamma, 4) || !aligned(grad_beta, 4) || !aligned(ws, 4))
      return fail(me, "misaligned pointer");
    if (grad_gamma) {
      const size_t need = norm_workspace_bytes(dtype, n_rows, n_cols);
      if (need && (!ws || ws_bytes < need)) return fail(me, "workspace missing or too small", TP_ERR_WORKSPACE);
    }
    NormBwdArgs a;
    if (drop && (s = check_drop(me, drop, &a.drop)) != TP_OK) return s;
    if (n_rows == 0 && !grad_gamma) return TP_OK;
    a.dtype = dtype;
    a.n_cols = n_cols;
    a.n_rows = n_rows;
    a.gy_stride = gy_stride;
    a.h_stride = h_stride;
    a.grad_y = grad_y;
    a.h = h;
    a.grad_res = grad_res;
    a.gamma = gamma;
    a.mean = mean;
    a.rstd = rstd;
    a.grad_h = grad_h;
    a.grad_x = grad_x;
    a.grad_gamma = grad_gamma;
    a.grad_beta = grad_beta;
    a.part = static_cast<float*>(ws);
    a.stream = stream;
    hipError_t e = norm_backward(a);
    return e == hipSuccess ? TP_OK : hip_error(e, "tp_layer_norm_backward launch");
  });
}

tp_status tp_attn_forward(const tp_attn* a, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, void* out, int64_t out_stride, float* lse,
                          hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_attn_forward";
    tp_status s = check_attn(me, a);
    if (s != TP_OK) return s;
    const Rows rows[] = {{q, q_stride, a->n_heads}, {k, k_stride, a->n_kv_heads}, {v, v_stride, a->n_kv_heads},
                         {out, out_stride, a->n_heads}};
    for (const Rows& r : rows)
      if ((s = check_attn_rows(me, *a, r)) != TP_OK) return s;
    if (a->n_nodes == 0) return TP_OK;
    if (!aligned(lse, 4)) return fail(me, "misaligned pointer");
    if ((s = check_attn_pointers(me, a)) != TP_OK) return s;
    AttnArgs args;
    args.d = *a;
    args.q = q;
    args.k = k;
    args.v = v;
    args.out = out;
    args.qs = q_stride;
    args.ks = k_stride;
    args.vs = v_stride;
    args.os = out_stride;
    args.lse = lse;
    args.stream = stream;
    return launched(me, attn_forward(args), kTooMany);
  });
}

tp_status tp_attn_backward_workspace(const tp_attn* a, size_t* bytes) {
  return guarded([&]() -> tp_status {
    if (!bytes) return fail("tp_attn_backward_workspace", "bytes is NULL");
    tp_status s = check_attn("tp_attn_backward_workspace", a);
    if (s == TP_OK) *bytes = attn_workspace(*a).floats * sizeof(float);
    return s;
  });
}

tp_status tp_attn_backward(const tp_attn* a, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const void* out, int64_t out_stride, const float* lse,
                           const void* grad_out, int64_t go_stride, void* grad_q, int64_t gq_stride, void* grad_k,
                           int64_t gk_stride, void* grad_v, int64_t gv_stride, void* grad_bias, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_attn_backward";
    tp_status s = check_attn(me, a);
    if (s != TP_OK) return s;
    const int hq = a->n_heads, hk = a->n_kv_heads;
    const Rows rows[] = {{q, q_stride, hq},   {k, k_stride, hk},       {v, v_stride, hk},
                         {out, out_stride, hq}, {grad_out, go_stride, hq}, {grad_q, gq_stride, hq},
                         {grad_k, gk_stride, hk}, {grad_v, gv_stride, hk}};
    for (const Rows& r : rows)
      if ((s = check_attn_rows(me, *a, r)) != TP_OK) return s;
    if (grad_bias && a->n_buckets == 0) return fail(me, "grad_bias without a bias");
    if (!aligned(grad_bias, size_of(a->dtype)) || !aligned(lse, 4) || !aligned(ws, 16))
      return fail(me, "misaligned pointer");
    if (a->n_nodes > 0) {
      if (!lse) return fail(me, "lse is NULL");
      if ((s = check_attn_pointers(me, a)) != TP_OK) return s;
    }
    const AttnWorkspace w = attn_workspace(*a);
    if (w.floats > 0 && (!ws || ws_bytes < w.floats * sizeof(float)))
      return fail(me, "workspace missing or too small", TP_ERR_WORKSPACE);
    if (a->n_nodes == 0 && !grad_bias) return TP_OK;
    AttnArgs args;
    args.d = *a;
    args.q = q;
    args.k = k;
    args.v = v;
    args.out_in = out;
    args.go = grad_out;
    args.gq = grad_q;
    args.gk = grad_k;
    args.gv = grad_v;
    args.gbias = grad_bias;
    args.qs = q_stride;
    args.ks = k_stride;
    args.vs = v_stride;
    args.os = out_stride;
    args.gos = go_stride;
    args.gqs = gq_stride;
    args.gks = gk_stride;
    args.gvs = gv_stride;
    args.lse_in = lse;
    args.delta = static_cast<float*>(ws);
    args.part = args.delta + w.part;
    args.kv_part = args.delta + w.kv_part;
    args.stream = stream;
    return launched(me, attn_backward(args), kTooMany);
  });
}

}  // extern "C"
