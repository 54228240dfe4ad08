// C ABI of what stands around the attention block: norm and rotation of queries and keys,
// routing, products by group, the AdamW step.  Argument checks (all before any HIP call) and
// dispatch.
#include <hip/hip_runtime.h>

#include <cmath>

#include "capi_checks.hpp"

using namespace tpc;

namespace {

constexpr int64_t kInt32Max = std::numeric_limits<int32_t>::max();

tp_status check_heads(const char* where, const tp_heads* h) {
  if (!h) return fail(where, "description is NULL");
  if (!known(h->dtype)) return fail(where, "unknown element type");
  if (h->n_rows < 0) return fail(where, "negative size");
  if (h->n_heads < 1 || h->n_kv_heads < 1) return fail(where, "n_heads and n_kv_heads must be positive");
  if (h->n_heads > 1024 || h->n_kv_heads > 1024) return fail(where, "at most 1024 heads", TP_ERR_UNSUPPORTED);
  if (h->head_dim < 1 || h->head_dim > kHeadsMaxDim) return fail(where, "head_dim must be 1 to 256", TP_ERR_UNSUPPORTED);
  if (!h->gamma_q != !h->gamma_k) return fail(where, "gamma_q and gamma_k are given together");
  if (!(h->eps >= 0.f) || std::isinf(h->eps)) return fail(where, "eps must be finite and not negative");
  if (h->n_pairs < 0 || 2 * (int64_t)h->n_pairs > h->head_dim) return fail(where, "n_pairs must be 0 to head_dim / 2");
  if (h->interleaved != 0 && h->interleaved != 1) return fail(where, "interleaved must be 0 or 1");
  if (h->n_pairs > 0) {
    if (h->axes < 1 || h->axes > 3) return fail(where, "1 to 3 axes only", TP_ERR_UNSUPPORTED);
    if (h->pos_type != TP_POS_F32 && h->pos_type != TP_POS_I32) return fail(where, "unknown type of positions");
  }
  if (h->n_rows > std::numeric_limits<int64_t>::max() / 65536 / 2048) return fail(where, "too many rows", TP_ERR_OVERFLOW);
  return TP_OK;
}

struct HeadRows {
  const void* p;
  int64_t stride;
  int heads;
};

tp_status check_head_rows(const char* where, const tp_heads& h, const HeadRows& r) {
  if (bad_stride(r.stride, (int64_t)r.heads * h.head_dim, h.n_rows))
    return fail(where, "row stride below the row length, or too large");
  if (h.n_rows > 0 && !r.p) return fail(where, "NULL pointer");
  if (!aligned(r.p, size_of(h.dtype))) return fail(where, "misaligned pointer");
  return TP_OK;
}

tp_status check_head_pointers(const char* where, const tp_heads& h) {
  if (h.n_rows > 0 && h.n_pairs > 0 && (!h.pos || !h.freq)) return fail(where, "a rotation needs pos and freq");
  if (!aligned(h.gamma_q, 4) || !aligned(h.gamma_k, 4) || !aligned(h.pos, 4) || !aligned(h.freq, 8))
    return fail(where, "misaligned pointer");
  return TP_OK;
}

HeadArgs head_args(const tp_heads& h) {
  HeadArgs a;
  a.n_rows = h.n_rows;
  a.hq = h.n_heads;
  a.hk = h.n_kv_heads;
  a.d = h.head_dim;
  a.pairs = h.n_pairs;
  a.axes = h.axes;
  a.pos_int = h.pos_type == TP_POS_I32;
  a.interleaved = h.interleaved != 0;
  a.pos = h.pos;
  a.freq = h.freq;
  a.gamma_q = h.gamma_q;
  a.gamma_k = h.gamma_k;
  a.eps = h.eps;
  return a;
}

tp_status check_route(const char* where, int32_t dtype, int64_t n_rows, int32_t n_groups, int32_t k, int32_t over_all) {
  if (!known(dtype)) return fail(where, "unknown element type");
  if (n_rows < 0) return fail(where, "negative size");
  if (n_groups < 1 || n_groups > kMaxGroups) return fail(where, "1 to 1024 groups only", TP_ERR_UNSUPPORTED);
  if (k < 1 || k > n_groups) return fail(where, "k must be 1 to n_groups");
  if (k > kMaxChoices) return fail(where, "at most 16 choices", TP_ERR_UNSUPPORTED);
  if (over_all != 0 && over_all != 1) return fail(where, "over_all must be 0 or 1");
  return TP_OK;
}

tp_status check_order(const char* where, int64_t n, int32_t n_groups) {
  if (n < 0) return fail(where, "negative size");
  if (n_groups < 1 || n_groups > kMaxGroups) return fail(where, "1 to 1024 groups only", TP_ERR_UNSUPPORTED);
  if (n > kInt32Max - 4096) return fail(where, "slots do not fit 32 bits", TP_ERR_OVERFLOW);
  return TP_OK;
}

tp_status check_grouped(const char* where, const tp_grouped* g) {
  if (!g) return fail(where, "description is NULL");
  if (!known(g->dtype)) return fail(where, "unknown element type");
  tp_status s = check_order(where, g->n_slots, g->n_groups);
  if (s != TP_OK) return s;
  if (g->n_in < 1 || g->n_out < 1) return fail(where, "n_in and n_out must be positive");
  if (g->n_in > 1 << 20 || g->n_out > 1 << 20) return fail(where, "rows of at most 2^20 values", TP_ERR_UNSUPPORTED);
  if (g->fan < 1 || g->n_slots % g->fan) return fail(where, "n_slots must be a multiple of fan, fan positive");
  for (int32_t r : {g->x_rows, g->y_rows})
    if (r != TP_ROWS_SOURCE && r != TP_ROWS_GROUPED) return fail(where, "unknown order of rows");
  return TP_OK;
}

tp_status check_grouped_pointers(const char* where, const tp_grouped& g, bool weights) {
  if (!g.ptr || (g.n_slots > 0 && !g.rows) || (weights && !g.w)) return fail(where, "NULL pointer");
  if (!aligned(g.ptr, 4) || !aligned(g.rows, 4) || !aligned(g.w, size_of(g.dtype))) return fail(where, "misaligned pointer");
  return TP_OK;
}

bool summed(const tp_grouped& g) { return g.x_rows == TP_ROWS_SOURCE && g.fan > 1; }
size_t grad_x_bytes(const tp_grouped& g) {
  return summed(g) ? ((size_t)g.n_slots * g.n_in * sizeof(float) + 15) / 16 * 16 : 0;
}
size_t grad_w_bytes(const tp_grouped& g) { return grouped_weight_workspace(g.dtype, g.n_slots, g.n_groups, g.n_in, g.n_out); }

tp_status check_combine(const char* where, int32_t dtype, int64_t n_rows, int32_t k, int32_t n_cols) {
  if (!known(dtype)) return fail(where, "unknown element type");
  if (n_rows < 0 || k < 1 || n_cols < 1) return fail(where, "sizes must be positive (n_rows not negative)");
  if (n_rows > std::numeric_limits<int64_t>::max() / 8 / k / n_cols) return fail(where, "too many rows", TP_ERR_OVERFLOW);
  return TP_OK;
}

tp_status check_tensors(const char* where, int32_t n_tensors, const int64_t* sizes) {
  if (n_tensors < 0) return fail(where, "negative size");
  if (n_tensors > 0 && !sizes) return fail(where, "sizes is NULL");
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (sizes[i] < 0) return fail(where, "negative size");
    if (sizes[i] > (int64_t)1 << 38) return fail(where, "tensors of at most 2^38 values", TP_ERR_OVERFLOW);
  }
  if (adamw_table_bytes(n_tensors, sizes) < 0) return fail(where, "too many values for one step", TP_ERR_OVERFLOW);
  return TP_OK;
}

}  // namespace

extern "C" {

tp_status tp_head_norm_rotate_forward(const tp_heads* h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                      void* q_out, int64_t qo_stride, void* k_out, int64_t ko_stride, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_head_norm_rotate_forward";
    tp_status s = check_heads(me, h);
    if (s != TP_OK) return s;
    for (const HeadRows& r : {HeadRows{q, q_stride, h->n_heads}, HeadRows{k, k_stride, h->n_kv_heads},
                              HeadRows{q_out, qo_stride, h->n_heads}, HeadRows{k_out, ko_stride, h->n_kv_heads}})
      if ((s = check_head_rows(me, *h, r)) != TP_OK) return s;
    if ((s = check_head_pointers(me, *h)) != TP_OK || h->n_rows == 0) return s;
    HeadArgs a = head_args(*h);
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.qo_stride = qo_stride;
    a.ko_stride = ko_stride;
    a.stream = stream;
    return launched(me, heads_forward(h->dtype, a));
  });
}

tp_status tp_head_norm_rotate_workspace(const tp_heads* h, size_t* bytes) {
  return guarded([&]() -> tp_status {
    if (!bytes) return fail("tp_head_norm_rotate_workspace", "bytes is NULL");
    tp_status s = check_heads("tp_head_norm_rotate_workspace", h);
    if (s == TP_OK) *bytes = heads_workspace_bytes(h->dtype, head_args(*h));
    return s;
  });
}

tp_status tp_head_norm_rotate_backward(const tp_heads* h, const void* grad_qo, int64_t gqo_stride, const void* grad_ko,
                                       int64_t gko_stride, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                       void* grad_q, int64_t gq_stride, void* grad_k, int64_t gk_stride, float* grad_gamma_q,
                                       float* grad_gamma_k, float* grad_pos, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_head_norm_rotate_backward";
    tp_status s = check_heads(me, h);
    if (s != TP_OK) return s;
    const int hq = h->n_heads, hk = h->n_kv_heads;
    for (const HeadRows& r : {HeadRows{grad_qo, gqo_stride, hq}, HeadRows{grad_ko, gko_stride, hk}, HeadRows{q, q_stride, hq},
                              HeadRows{k, k_stride, hk}, HeadRows{grad_q, gq_stride, hq}, HeadRows{grad_k, gk_stride, hk}})
      if ((s = check_head_rows(me, *h, r)) != TP_OK) return s;
    if ((s = check_head_pointers(me, *h)) != TP_OK) return s;
    if (!grad_gamma_q != !grad_gamma_k) return fail(me, "grad_gamma_q and grad_gamma_k are given together");
    if (grad_gamma_q && !h->gamma_q) return fail(me, "weight gradients without a norm");
    if (grad_pos && (h->n_pairs == 0 || h->pos_type != TP_POS_F32))
      return fail(me, "grad_pos needs a rotation by float32 positions");
    if (!aligned(grad_gamma_q, 4) || !aligned(grad_gamma_k, 4) || !aligned(grad_pos, 4) || !aligned(ws, 4))
      return fail(me, "misaligned pointer");
    HeadBwdArgs b;
    b.f = head_args(*h);
    if (grad_gamma_q) {
      const size_t need = heads_workspace_bytes(h->dtype, b.f);
      if (need && (!ws || ws_bytes < need)) return fail(me, "workspace missing or too small", TP_ERR_WORKSPACE);
    }
    if (h->n_rows == 0 && !grad_gamma_q) return TP_OK;
    b.f.q = q;
    b.f.k = k;
    b.f.q_stride = q_stride;
    b.f.k_stride = k_stride;
    b.f.stream = stream;
    b.gq_up = grad_qo;
    b.gk_up = grad_ko;
    b.gq_up_stride = gqo_stride;
    b.gk_up_stride = gko_stride;
    b.gq = grad_q;
    b.gk = grad_k;
    b.gq_stride = gq_stride;
    b.gk_stride = gk_stride;
    b.grad_gamma_q = grad_gamma_q;
    b.grad_gamma_k = grad_gamma_k;
    b.grad_pos = h->n_rows > 0 ? grad_pos : nullptr;         // without rows pos and freq may be NULL
    b.part = static_cast<float*>(ws);
    return launched(me, heads_backward(h->dtype, b));
  });
}

tp_status tp_route_forward(int32_t dtype, int64_t n_rows, int32_t n_groups, int32_t k, int32_t over_all, const void* logits,
                           int64_t logits_stride, float* weight, int32_t* index, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_route_forward";
    tp_status s = check_route(me, dtype, n_rows, n_groups, k, over_all);
    if (s != TP_OK) return s;
    if (bad_stride(logits_stride, n_groups, n_rows)) return fail(me, "row stride below the row length, or too large");
    if (n_rows > 0 && (!logits || !weight || !index)) return fail(me, "NULL pointer");
    if (!aligned(logits, size_of(dtype)) || !aligned(weight, 4) || !aligned(index, 4)) return fail(me, "misaligned pointer");
    if (n_rows == 0) return TP_OK;
    RouteArgs a;
    a.dtype = dtype;
    a.n_rows = n_rows;
    a.stride = logits_stride;
    a.n_groups = n_groups;
    a.k = k;
    a.over_all = over_all != 0;
    a.logits = logits;
    a.weight = weight;
    a.index = index;
    a.stream = stream;
    return launched(me, route_forward(a));
  });
}

tp_status tp_route_backward(int32_t dtype, int64_t n_rows, int32_t n_groups, int32_t k, int32_t over_all, const void* logits,
                            int64_t logits_stride, const float* weight, const int32_t* index, const float* grad_weight,
                            void* grad_logits, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_route_backward";
    tp_status s = check_route(me, dtype, n_rows, n_groups, k, over_all);
    if (s != TP_OK) return s;
    if (over_all && bad_stride(logits_stride, n_groups, n_rows)) return fail(me, "row stride below the row length, or too large");
    if (n_rows > 0 && ((over_all && !logits) || !weight || !index || !grad_weight || !grad_logits))
      return fail(me, "NULL pointer");
    const int64_t es = size_of(dtype);
    if (!aligned(logits, es) || !aligned(weight, 4) || !aligned(index, 4) || !aligned(grad_weight, 4) || !aligned(grad_logits, es))
      return fail(me, "misaligned pointer");
    if (n_rows == 0) return TP_OK;
    RouteArgs a;
    a.dtype = dtype;
    a.n_rows = n_rows;
    a.stride = logits_stride;
    a.n_groups = n_groups;
    a.k = k;
    a.over_all = over_all != 0;
    a.logits = logits;
    a.weight_in = weight;
    a.index_in = index;
    a.grad_weight = grad_weight;
    a.grad_logits = grad_logits;
    a.stream = stream;
    return launched(me, route_backward(a));
  });
}

tp_status tp_group_workspace(int64_t n, int32_t n_groups, size_t* bytes) {
  return guarded([&]() -> tp_status {
    if (!bytes) return fail("tp_group_workspace", "bytes is NULL");
    tp_status s = check_order("tp_group_workspace", n, n_groups);
    if (s == TP_OK) *bytes = group_workspace_bytes(n, n_groups);
    return s;
  });
}

tp_status tp_group_rows(const int32_t* index, int64_t n, int32_t n_groups, int32_t* ptr, int32_t* rows, void* ws,
                        size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_group_rows";
    tp_status s = check_order(me, n, n_groups);
    if (s != TP_OK) return s;
    if (!ptr || (n > 0 && (!index || !rows))) return fail(me, "NULL pointer");
    if (!aligned(index, 4) || !aligned(ptr, 4) || !aligned(rows, 4) || !aligned(ws, 4)) return fail(me, "misaligned pointer");
    const size_t need = group_workspace_bytes(n, n_groups);
    if (need && (!ws || ws_bytes < need)) return fail(me, "workspace missing or too small", TP_ERR_WORKSPACE);
    return launched(me, group_rows(index, n, n_groups, ptr, rows, ws, stream));
  });
}

tp_status tp_grouped_linear_forward(const tp_grouped* g, const void* x, int64_t x_stride, const void* bias, int32_t act, void* y,
                                    int64_t y_stride, void* pre, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_grouped_linear_forward";
    tp_status s = check_grouped(me, g);
    if (s != TP_OK) return s;
    if (act != TP_ACT_NONE && act != TP_ACT_SILU) return fail(me, "unknown activation");
    if (pre && act == TP_ACT_NONE) return fail(me, "pre goes with an activation");
    if (bad_stride(x_stride, g->n_in, g->n_slots) || bad_stride(y_stride, g->n_out, g->n_slots))
      return fail(me, "row stride below the row length, or too large");
    if (g->n_slots == 0) return TP_OK;
    if ((s = check_grouped_pointers(me, *g, true)) != TP_OK) return s;
    if (!x || !y) return fail(me, "NULL pointer");
    const int64_t es = size_of(g->dtype);
    if (!aligned(x, es) || !aligned(bias, es) || !aligned(y, es) || !aligned(pre, es)) return fail(me, "misaligned pointer");
    GroupedArgs a;
    a.dtype = g->dtype;
    a.n_groups = g->n_groups;
    a.act = act;
    a.n = g->n_slots;
    a.ptr = g->ptr;
    a.rows = g->rows;
    a.a = x;
    a.w = g->w;
    a.bias = bias;
    a.lda = x_stride;
    a.ldc = y_stride;
    a.a_div = g->x_rows == TP_ROWS_SOURCE ? g->fan : 0;
    a.c_div = g->y_rows == TP_ROWS_SOURCE ? 1 : 0;
    a.k = g->n_in;
    a.cols = g->n_out;
    a.c = y;
    a.pre_out = pre;
    a.stream = stream;
    return launched(me, grouped_product(a));
  });
}

tp_status tp_grouped_linear_workspace(const tp_grouped* g, int32_t want_x, int32_t want_w, size_t* bytes) {
  return guarded([&]() -> tp_status {
    if (!bytes) return fail("tp_grouped_linear_workspace", "bytes is NULL");
    tp_status s = check_grouped("tp_grouped_linear_workspace", g);
    if (s == TP_OK) *bytes = (want_x ? grad_x_bytes(*g) : 0) + (want_w ? grad_w_bytes(*g) : 0);
    return s;
  });
}

tp_status tp_grouped_linear_backward(const tp_grouped* g, const void* grad_z, int64_t gz_stride, const void* x, int64_t x_stride,
                                     const void* pre, int64_t pre_stride, void* grad_x, int64_t gx_stride, void* grad_w,
                                     void* grad_bias, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_grouped_linear_backward";
    tp_status s = check_grouped(me, g);
    if (s != TP_OK) return s;
    const int64_t n = g->n_slots, es = size_of(g->dtype);
    if (bad_stride(gz_stride, g->n_out, n) || (grad_w && bad_stride(x_stride, g->n_in, n)) ||
        (pre && bad_stride(pre_stride, g->n_in, n)) || (grad_x && bad_stride(gx_stride, g->n_in, n)))
      return fail(me, "row stride below the row length, or too large");
    if (grad_bias && !grad_w) return fail(me, "grad_bias goes with grad_w");
    if (pre && summed(*g)) return fail(me, "pre needs one slot for each row of x");
    if (grad_x && summed(*g) && gx_stride != g->n_in) return fail(me, "grad_x must be contiguous where rows have several slots");
    if (!grad_x && !grad_w) return TP_OK;
    if (n == 0 && !grad_w) return TP_OK;
    if ((s = check_grouped_pointers(me, *g, grad_x && n > 0)) != TP_OK) return s;
    if (n > 0 && (!grad_z || (grad_w && !x))) return fail(me, "NULL pointer");
    if (!aligned(grad_z, es) || !aligned(x, es) || !aligned(pre, es) || !aligned(grad_x, es) || !aligned(grad_w, es) ||
        !aligned(grad_bias, es) || !aligned(ws, 16))
      return fail(me, "misaligned pointer");
    const size_t for_x = grad_x ? grad_x_bytes(*g) : 0, need = for_x + (grad_w ? grad_w_bytes(*g) : 0);
    if (need && (!ws || ws_bytes < need)) return fail(me, "workspace missing or too small", TP_ERR_WORKSPACE);
    if (grad_w) {
      GroupedWeightArgs a;
      a.dtype = g->dtype;
      a.n_groups = g->n_groups;
      a.n = n;
      a.ldx = x_stride;
      a.ldg = gz_stride;
      a.ptr = g->ptr;
      a.rows = g->rows;
      a.x = x;
      a.gy = grad_z;
      a.x_div = g->x_rows == TP_ROWS_SOURCE ? g->fan : 0;
      a.g_div = g->y_rows == TP_ROWS_SOURCE ? 1 : 0;
      a.k = g->n_in;
      a.cols = g->n_out;
      a.grad_w = grad_w;
      a.grad_bias = grad_bias;
      a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + for_x);
      a.stream = stream;
      if ((s = launched(me, grouped_weight_grad(a))) != TP_OK) return s;
    }
    if (!grad_x || n == 0) return TP_OK;
    GroupedArgs a;
    a.dtype = g->dtype;
    a.n_groups = g->n_groups;
    a.n = n;
    a.ptr = g->ptr;
    a.rows = g->rows;
    a.a = grad_z;
    a.w = g->w;
    a.lda = gz_stride;
    a.a_div = g->y_rows == TP_ROWS_SOURCE ? 1 : 0;
    a.c_div = g->x_rows == TP_ROWS_SOURCE ? 1 : 0;
    a.k = g->n_out;
    a.cols = g->n_in;
    a.transposed = true;
    a.c = summed(*g) ? ws : grad_x;        // the slots' parts are float32: rounded once, as their sum
    a.wide = summed(*g);
    a.ldc = summed(*g) ? g->n_in : gx_stride;
    a.pre = pre;
    a.ldpre = pre_stride;
    a.stream = stream;
    if ((s = launched(me, grouped_product(a))) != TP_OK || !summed(*g)) return s;
    CombineArgs c;
    c.dtype = g->dtype;
    c.n_rows = n / g->fan;
    c.k = g->fan;
    c.n_cols = g->n_in;
    c.wide = true;
    c.y = ws;
    c.out = grad_x;
    c.stream = stream;
    return launched(me, combine_forward(c));
  });
}

tp_status tp_combine_forward(int32_t dtype, int64_t n_rows, int32_t k, int32_t n_cols, const void* y, const float* weight,
                             void* out, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_combine_forward";
    tp_status s = check_combine(me, dtype, n_rows, k, n_cols);
    if (s != TP_OK || n_rows == 0) return s;
    if (!y || !out) return fail(me, "NULL pointer");
    if (!aligned(y, size_of(dtype)) || !aligned(weight, 4) || !aligned(out, size_of(dtype))) return fail(me, "misaligned pointer");
    CombineArgs a;
    a.dtype = dtype;
    a.n_rows = n_rows;
    a.k = k;
    a.n_cols = n_cols;
    a.y = y;
    a.weight = weight;
    a.out = out;
    a.stream = stream;
    return launched(me, combine_forward(a));
  });
}

tp_status tp_combine_backward(int32_t dtype, int64_t n_rows, int32_t k, int32_t n_cols, const void* grad_out, const void* y,
                              const float* weight, void* grad_y, float* grad_weight, hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_combine_backward";
    tp_status s = check_combine(me, dtype, n_rows, k, n_cols);
    if (s != TP_OK || n_rows == 0) return s;
    if (!grad_out || !y || !weight || !grad_y || !grad_weight) return fail(me, "NULL pointer");
    const int64_t es = size_of(dtype);
    if (!aligned(grad_out, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(grad_y, es) || !aligned(grad_weight, 4))
      return fail(me, "misaligned pointer");
    CombineArgs a;
    a.dtype = dtype;
    a.n_rows = n_rows;
    a.k = k;
    a.n_cols = n_cols;
    a.go = grad_out;
    a.y = y;
    a.weight = weight;
    a.gy = grad_y;
    a.grad_weight = grad_weight;
    a.stream = stream;
    return launched(me, combine_backward(a));
  });
}

tp_status tp_adamw_sizes(int32_t n_tensors, const int64_t* sizes, size_t* table_bytes, int64_t* state_values,
                         size_t* ws_bytes) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_adamw_sizes";
    if (!table_bytes || !state_values || !ws_bytes) return fail(me, "NULL pointer");
    tp_status s = check_tensors(me, n_tensors, sizes);
    if (s != TP_OK) return s;
    *table_bytes = (size_t)adamw_table_bytes(n_tensors, sizes);
    *state_values = adamw_state_size(n_tensors, sizes);
    *ws_bytes = adamw_workspace_bytes(n_tensors, sizes);
    return TP_OK;
  });
}

tp_status tp_adamw_table(int32_t n_tensors, const int64_t* sizes, void* const* params, void* const* copies, const float* decay,
                         void* host_table) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_adamw_table";
    tp_status s = check_tensors(me, n_tensors, sizes);
    if (s != TP_OK || n_tensors == 0) return s;
    if (!params || !host_table) return fail(me, "NULL pointer");
    for (int32_t i = 0; i < n_tensors; ++i) {
      if (sizes[i] > 0 && !params[i]) return fail(me, "NULL pointer");
      if (!aligned(params[i], 4) || (copies && !aligned(copies[i], 2))) return fail(me, "misaligned pointer");
      if (decay && !std::isfinite(decay[i])) return fail(me, "decay must be finite");
    }
    adamw_table_fill(n_tensors, sizes, params, copies, decay, host_table);
    return TP_OK;
  });
}

tp_status tp_adamw_step(const tp_adamw* a, const void* const* grads, float* norm, void* ws, size_t ws_bytes,
                        hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_adamw_step";
    if (!a) return fail(me, "description is NULL");
    if (a->bits != 8 && a->bits != 32) return fail(me, "states of 8 or 32 bits only", TP_ERR_UNSUPPORTED);
    if (!known(a->grad_dtype)) return fail(me, "unknown element type");
    tp_status s = check_tensors(me, a->n_tensors, a->sizes);
    if (s != TP_OK) return s;
    if (!(a->beta1 >= 0 && a->beta1 < 1 && a->beta2 >= 0 && a->beta2 < 1)) return fail(me, "betas must be in [0, 1)");
    if (!(a->eps >= 0) || std::isinf(a->eps)) return fail(me, "eps must be finite and not negative");
    if (!a->lr_at && !std::isfinite(a->lr)) return fail(me, "lr must be finite");
    if (!(a->max_norm >= 0)) return fail(me, "max_norm must not be negative");
    if (!a->scalars || (norm && !(a->max_norm > 0))) return fail(me, !a->scalars ? "NULL pointer" : "norm needs max_norm");
    const bool some = adamw_state_size(a->n_tensors, a->sizes) > 0;
    if (some && (!a->table || !a->m || !a->v || !grads || (a->bits == 8 && (!a->m_unit || !a->v_unit))))
      return fail(me, "NULL pointer");
    if (!aligned(a->table, 16) || !aligned(a->m, 16) || !aligned(a->v, 16) || !aligned(a->scalars, 16) || !aligned(ws, 16) ||
        !aligned(a->m_unit, 4) || !aligned(a->v_unit, 4) || !aligned(a->lr_at, 4) || !aligned(norm, 4))
      return fail(me, "misaligned pointer");
    for (int32_t i = 0; i < a->n_tensors && some; ++i) {
      if (a->sizes[i] > 0 && !grads[i]) return fail(me, "NULL pointer");
      if (!aligned(grads[i], size_of(a->grad_dtype))) return fail(me, "misaligned pointer");
    }
    if (a->max_norm > 0) {
      const size_t need = adamw_workspace_bytes(a->n_tensors, a->sizes);
      if (need && (!ws || ws_bytes < need)) return fail(me, "workspace missing or too small", TP_ERR_WORKSPACE);
    }
    AdamArgs r;
    r.bits = a->bits;
    r.grad_dtype = a->grad_dtype;
    r.n_tensors = a->n_tensors;
    r.sizes = a->sizes;
    r.table = a->table;
    r.m = a->m;
    r.v = a->v;
    r.m_unit = a->m_unit;
    r.v_unit = a->v_unit;
    r.beta1 = a->beta1;
    r.beta2 = a->beta2;
    r.eps = a->eps;
    r.lr = a->lr;
    r.max_norm = a->max_norm;
    r.lr_at = a->lr_at;
    r.seed = a->seed;
    r.scalars = a->scalars;
    r.ws = ws;
    r.norm = norm;
    r.grads = grads;
    r.stream = stream;
    return launched(me, adamw_step(r), "too many values for one step");
  });
}

tp_status tp_adamw_values(int32_t second, int64_t n, const uint8_t* codes, const float* units, float* out,
                          hipStream_t stream) {
  return guarded([&]() -> tp_status {
    const char* me = "tp_adamw_values";
    if (n < 0 || n % kAdamBlock) return fail(me, "n must be a multiple of 256, not negative");
    if (n == 0) return TP_OK;
    if (!codes || !units || !out) return fail(me, "NULL pointer");
    if (!aligned(codes, 16) || !aligned(units, 4) || !aligned(out, 4)) return fail(me, "misaligned pointer");
    return launched(me, adamw_values(second, n, codes, units, out, stream), "too many values for one launch");
  });
}

}  // extern "C"
