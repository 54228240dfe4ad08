// Internal declarations shared by the library's translation units.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>
#include <vector>

#include "../../include/tpconv.h"
#include "philox.hpp"

namespace tpc {

// ---- error reporting --------------------------------------------------------
tp_status set_error(tp_status code, const std::string& msg);
tp_status hip_error(hipError_t e, const char* where);

// ---- kernel dispatch --------------------------------------------------------
struct ConvArgs {
  int32_t n_nodes = 0, n_edges = 0;
  const int32_t *row_ptr = nullptr, *col = nullptr;
  const int32_t *t_row_ptr = nullptr, *t_perm = nullptr, *t_col = nullptr;
  // sender_rows: the edge rows (w, Y and their gradients) are stored in the
  // sender grouping (row k = sender-grouped position k); e_pos[q] is then the
  // row of receiver-sorted edge q, which the forward reads
  bool sender_rows = false;
  const int32_t* e_pos = nullptr;
  // launch order of the receiver- and sender-grouped kernels (null: node id)
  const int32_t *r_order = nullptr, *s_order = nullptr;
  const float *x = nullptr, *Y = nullptr, *w = nullptr, *grad_out = nullptr;
  float *out = nullptr, *grad_x = nullptr, *grad_Y = nullptr, *grad_w = nullptr;
  // second-order backward: cotangents of (grad_x, grad_Y, grad_w), outputs
  const float *gg_x = nullptr, *gg_Y = nullptr, *gg_w = nullptr;
  float *d_x = nullptr, *d_Y = nullptr, *d_w = nullptr, *d_g = nullptr;
  // edge-vector form: r [E][3] in place of Y, grad_r [E][3] in place of grad_Y
  const float* r = nullptr;
  float* grad_r = nullptr;
  hipStream_t stream = nullptr;
};

using LaunchFn = hipError_t (*)(const ConvArgs&);

struct KernelSet {
  LaunchFn fwd = nullptr;       // receiver pass: out
  LaunchFn bwd_recv = nullptr;  // receiver pass: grad_w, grad_Y
  LaunchFn bwd_send = nullptr;  // sender pass: grad_x
  LaunchFn dbl_recv = nullptr;  // second order, receiver pass: d_grad_out, d_Y, d_w
  LaunchFn dbl_send = nullptr;  // second order, sender pass: d_x
  LaunchFn bwd_fused = nullptr; // sender-grouped pass: grad_x with grad_w and/or grad_Y
  LaunchFn fwd_r = nullptr;     // forward from edge vectors (harmonics on chip)
  LaunchFn bwd_r = nullptr;     // backward from edge vectors: grad_x, grad_w, grad_r
};

// radial-weight variant (edge weights from a radial network of the length)
struct RadialArgs {
  int32_t n_nodes = 0, n_edges = 0;
  const int32_t *row_ptr = nullptr, *col = nullptr;
  const int32_t *t_row_ptr = nullptr, *t_perm = nullptr, *t_col = nullptr;
  // launch order of the receiver- and sender-grouped passes (null: node id)
  const int32_t *r_order = nullptr, *s_order = nullptr;
  const float *x = nullptr, *Y = nullptr, *r_len = nullptr, *W1 = nullptr, *W2 = nullptr;
  const float* grad_out = nullptr;   // gradient w.r.t. the unmixed output
  float *out = nullptr, *grad_x = nullptr, *grad_Y = nullptr, *grad_W1 = nullptr, *grad_W2 = nullptr;
  float* grad_rlen = nullptr;        // gradient w.r.t. the edge lengths (through the basis)
  float r_cut = 0.f;
  // edge-vector form: Y holds r [E][3] (r_len unused), grad_Y receives grad_r
  // [E][3] (grad_rlen unused)
  bool geom = false;
  // second-order backward: cotangents of (grad_x, grad_Y, grad_rlen) and
  // outputs (out receives d_grad_out before the mix)
  const float *gg_x = nullptr, *gg_Y = nullptr, *gg_rlen = nullptr;
  float *d_x = nullptr, *d_Y = nullptr, *d_rlen = nullptr, *d_W1 = nullptr, *d_W2 = nullptr;
  void* ws = nullptr;
  hipStream_t stream = nullptr;
};
using RadialFn = hipError_t (*)(const RadialArgs&);
struct RadialSet {
  RadialFn fwd = nullptr;
  RadialFn bwd = nullptr;                        // grad_x, grad_Y, grad_rlen, grad_W1, grad_W2
  size_t (*bwd_workspace)(int n_nodes, int n_edges) = nullptr;
  RadialFn dbl = nullptr;                        // d_grad_out (unmixed), d_x, d_Y, d_rlen, d_W1, d_W2
  size_t (*dbl_workspace)(int n_nodes, int n_edges) = nullptr;
};
// fully connected per-edge weights (W_e = sum_h R_e[h] Theta[h]), reassociated
struct FcArgs {
  int32_t n_nodes = 0, n_edges = 0, outdim = 0;
  const int32_t *row_ptr = nullptr, *col = nullptr;
  const int32_t *t_row_ptr = nullptr, *t_perm = nullptr, *t_col = nullptr;
  const int32_t *r_order = nullptr, *s_order = nullptr;   // launch orders (null: node id)
  const float *x = nullptr, *Y = nullptr, *R = nullptr, *Theta = nullptr;
  float* out = nullptr;
  // backward: upstream gradient and outputs (NULL: skip)
  const float* gout = nullptr;
  float *grad_x = nullptr, *grad_Y = nullptr, *grad_R = nullptr, *grad_Theta = nullptr;
  bool state_saved = false;   // backward: ws already holds the forward's state S
  void* ws = nullptr;
  hipStream_t stream = nullptr;
};
// second-order backward: cotangents of (grad_x, grad_Y, grad_R, grad_Theta)
// (NULL: zero) and outputs (NULL: skip); the FcArgs carry the first-order inputs
struct FcDbl {
  const float *gg_x = nullptr, *gg_Y = nullptr, *gg_R = nullptr, *gg_Theta = nullptr;
  float *d_x = nullptr, *d_Y = nullptr, *d_R = nullptr, *d_Theta = nullptr, *d_g = nullptr;
};
struct FcSet {
  hipError_t (*fwd)(const FcArgs&) = nullptr;
  size_t (*workspace)(int n_nodes) = nullptr;
  int n_radial = 0;
  hipError_t (*bwd)(const FcArgs&) = nullptr;
  size_t (*bwd_workspace)(int n_nodes) = nullptr;
  hipError_t (*dbl)(const FcArgs&, const FcDbl&) = nullptr;
  size_t (*dbl_workspace)(int n_nodes, int n_edges) = nullptr;
};
const FcSet* fc_l012_s2(int mul, int n_radial);

// Gaunt (spherical-grid) product: input degrees deg[0..n_in) (distinct, <= 2),
// filter degrees 0..lmax_sh (<= 2), output degrees 0..lmax_out (<= 2)
struct GauntArgs {
  int32_t n_nodes = 0, n_edges = 0, U = 0, n_in = 0, deg[3] = {0, 0, 0};
  int32_t lmax_sh = 0, lmax_out = 0;
  const int32_t *row_ptr = nullptr, *col = nullptr;
  const float *x = nullptr, *Y = nullptr, *w = nullptr;
  float* out = nullptr;
  // backward: the upstream gradient, the sender grouping and the outputs (NULL: skip)
  const float* gout = nullptr;
  const int32_t *t_row_ptr = nullptr, *t_perm = nullptr, *t_col = nullptr;
  float *grad_x = nullptr, *grad_Y = nullptr, *grad_w = nullptr;
  const int32_t *r_order = nullptr, *s_order = nullptr;   // launch orders (null: node id)
  hipStream_t stream = nullptr;
};
hipError_t gaunt_forward(const GauntArgs& a);
hipError_t gaunt_backward(const GauntArgs& a);
// second-order backward: cotangents of (grad_x, grad_Y, grad_w) (NULL: zero),
// outputs (NULL: skip) and scratch of gaunt_double_workspace bytes
struct GauntDbl {
  const float *gg_x = nullptr, *gg_Y = nullptr, *gg_w = nullptr;
  float *d_x = nullptr, *d_Y = nullptr, *d_w = nullptr, *d_g = nullptr;
  void* ws = nullptr;
};
hipError_t gaunt_double_backward(const GauntArgs& a, const GauntDbl& d);
size_t gaunt_double_workspace(const GauntArgs& a);
int gaunt_grid_points();

const RadialSet* find_radial(const std::vector<int>& ls, int lmax_sh, int lmax_out, int mul, int nb,
                             int nh);
const RadialSet* radial_l012_s2(int mul, int nb, int nh);
const RadialSet* radial_l0123_s3(int mul, int nb, int nh);

// Lookup of the compiled specialisation for (input degrees, lmax_sh,
// lmax_out, multiplicity); nullptr if none.
const KernelSet* find_kernels(const std::vector<int>& ls, int lmax_sh, int lmax_out, int mul);

// Per-signature registries (one translation unit each).
const KernelSet* kernels_l01_s1(int mul);
const KernelSet* kernels_l01_s2(int mul);
const KernelSet* kernels_l01_s3(int mul);
const KernelSet* kernels_l012_s2(int mul);
const KernelSet* kernels_l0123_s3(int mul);

// output-irrep description for the channel mix: degree-block sizes (2l+1) and
// per-channel offsets of each output irrep
struct UvwIrreps {
  int n;
  int dim[8];
  int ko[8];
};

// ---- device helpers implemented in graph.hip / sh.hip / uvw.hip --------------
size_t graph_workspace_bytes(int n_nodes, int n_edges);
tp_status graph_build(const int32_t* src, const int32_t* dst, int n_edges, int n_nodes,
                      int32_t* row_ptr, int32_t* col, int32_t* perm, int32_t* t_row_ptr,
                      int32_t* t_perm, int32_t* t_col, void* ws, int32_t flags, hipStream_t st);
tp_status graph_build_static(const int32_t* src, const int32_t* dst, int n_edges, int n_nodes,
                             int32_t* row_ptr, int32_t* col, int32_t* perm, int32_t* t_row_ptr,
                             int32_t* t_perm, int32_t* t_col, int32_t flags, hipStream_t st);
tp_status gather_rows(const void* in, const int32_t* perm, int64_t n_rows, int64_t words, void* out,
                      hipStream_t st);
tp_status sender_positions(const int32_t* t_perm, int n_edges, int32_t* e_pos, hipStream_t st);
size_t order_workspace_bytes(int n_nodes);
tp_status launch_order(const int32_t* row_ptr, const int32_t* t_row_ptr, int n_nodes, int n_edges,
                       int32_t* order, int32_t* t_order, void* ws, hipStream_t st);
tp_status sph_harm(int lmax, const float* r, int n, float* Y, hipStream_t st);
tp_status sph_harm_bwd(int lmax, const float* r, int n, const float* gY, const float* grl, float* gr,
                       hipStream_t st);
size_t uvw_workspace_bytes(int n_irreps, int U);
tp_status uvw_forward(int n_nodes, int U, int outdim, const UvwIrreps& irr, const float* W,
                      const float* X, float* Z, bool trans_w, hipStream_t st);
tp_status uvw_grad_w(int n_nodes, int U, int outdim, const UvwIrreps& irr, const float* X,
                     const float* G, float* gradW, void* ws, hipStream_t st);


// ---- layers around the convolution (norm.hip, attn*.hip) ----------------------
struct NormArgs {
  int dtype = TP_F32, n_cols = 0;
  int64_t n_rows = 0, x_stride = 0, y_stride = 0;
  const void *x = nullptr, *residual = nullptr;   // residual null: h is x
  bool has_drop = false;
  DropArgs drop;
  const float *gamma = nullptr, *beta = nullptr;
  float eps = 0.f;
  void *y = nullptr, *h = nullptr;
  float *mean = nullptr, *rstd = nullptr;
  hipStream_t stream = nullptr;
};
struct NormBwdArgs {
  int dtype = TP_F32, n_cols = 0;
  int64_t n_rows = 0, gy_stride = 0, h_stride = 0;
  const void *grad_y = nullptr, *h = nullptr, *grad_res = nullptr;
  const float *gamma = nullptr, *mean = nullptr, *rstd = nullptr;
  DropArgs drop;                                  // used where grad_x is set
  void *grad_h = nullptr, *grad_x = nullptr;
  float *grad_gamma = nullptr, *grad_beta = nullptr, *part = nullptr;
  hipStream_t stream = nullptr;
};
constexpr int kNormMaxCols = 8192;
size_t norm_workspace_bytes(int dtype, int64_t n_rows, int n_cols);
hipError_t norm_forward(const NormArgs& a);
hipError_t norm_backward(const NormBwdArgs& a);
hipError_t dropout_apply(int dtype, int64_t n, const void* x, const void* r, const DropArgs& d, void* out,
                         hipStream_t st);

// The passes return hipErrorInvalidConfiguration, with nothing launched, where a grid would have
// more threads in a dimension than 32 bits count.
struct AttnArgs {
  tp_attn d;
  const void *q = nullptr, *k = nullptr, *v = nullptr, *out_in = nullptr, *go = nullptr;
  int64_t qs = 0, ks = 0, vs = 0, os = 0, gos = 0, gqs = 0, gks = 0, gvs = 0;   // row strides, elements
  void *out = nullptr, *gq = nullptr, *gk = nullptr, *gv = nullptr, *gbias = nullptr;
  float* lse = nullptr;
  const float* lse_in = nullptr;
  float *delta = nullptr, *part = nullptr, *kv_part = nullptr;   // workspace of the backward
  bool split = false;                             // query heads that share a key head apart
  bool dry = false;                               // the grid is checked, nothing launched
  hipStream_t stream = nullptr;
};
hipError_t attn_forward(const AttnArgs& a);
hipError_t attn_backward(const AttnArgs& a);
hipError_t attn_backward_q(const AttnArgs& a);   // its query side (attn_dq.hip)
// workspace of the backward, in floats: delta [n_heads][n_nodes] from 0, the bias
// gradient's parts, the parts of grad_k and grad_v
struct AttnWorkspace {
  size_t part = 0, kv_part = 0, floats = 0;
};
AttnWorkspace attn_workspace(const tp_attn& d);

// ---- norm and rotation of queries and keys (heads.hip) --------------------------
// hipErrorInvalidConfiguration, with nothing launched, where a grid would be too large
struct HeadArgs {
  int64_t n_rows = 0, q_stride = 0, k_stride = 0, qo_stride = 0, ko_stride = 0;
  int hq = 0, hk = 0, d = 0, pairs = 0, axes = 0;
  bool pos_int = false, interleaved = false;
  const void *q = nullptr, *k = nullptr, *pos = nullptr;
  const double* freq = nullptr;
  const float *gamma_q = nullptr, *gamma_k = nullptr;   // null: no norm
  float eps = 0.f;
  void *q_out = nullptr, *k_out = nullptr;
  int lg = 0, rows = 0;                           // set by the launch
  hipStream_t stream = nullptr;
};
struct HeadBwdArgs {
  HeadArgs f;
  int64_t gq_up_stride = 0, gk_up_stride = 0, gq_stride = 0, gk_stride = 0;
  const void *gq_up = nullptr, *gk_up = nullptr;
  void *gq = nullptr, *gk = nullptr;
  float *grad_gamma_q = nullptr, *grad_gamma_k = nullptr, *grad_pos = nullptr, *part = nullptr;
};
constexpr int kHeadsMaxDim = 256;
size_t heads_workspace_bytes(int dtype, HeadArgs a);
hipError_t heads_forward(int dtype, HeadArgs a);
hipError_t heads_backward(int dtype, HeadBwdArgs b);

// ---- routing and products by group (route.hip, grouped*.hip) ---------------------
constexpr int kMaxGroups = 1024, kMaxChoices = 16;
struct RouteArgs {
  int dtype = TP_F32;
  int64_t n_rows = 0, stride = 0;
  int n_groups = 0, k = 0;
  bool over_all = false;                          // weights are the softmax over all groups, not over the chosen
  const void* logits = nullptr;
  float* weight = nullptr;
  int32_t* index = nullptr;
  // backward
  const float *weight_in = nullptr, *grad_weight = nullptr;
  const int32_t* index_in = nullptr;
  void* grad_logits = nullptr;
  hipStream_t stream = nullptr;
};
hipError_t route_forward(const RouteArgs& a);
hipError_t route_backward(const RouteArgs& a);
size_t group_workspace_bytes(int64_t n, int n_groups);
hipError_t group_rows(const int32_t* index, int64_t n, int n_groups, int32_t* ptr, int32_t* rows, void* ws, hipStream_t st);
struct CombineArgs {
  int dtype = TP_F32;
  int64_t n_rows = 0;
  int k = 0, n_cols = 0;
  bool wide = false;                              // forward: y is float32 whatever the type
  const void *y = nullptr, *go = nullptr;
  const float* weight = nullptr;                  // null: 1
  void *out = nullptr, *gy = nullptr;
  float* grad_weight = nullptr;
  hipStream_t stream = nullptr;
};
// c[row] = a[row] w_e (+ bias) and what follows, for the rows of each group; slots from
// ptr[n_groups] on belong to no group and get zeros.  Rows of a and c: those of the slots in
// group order (div 0), or rows[slot] / div.
struct GroupedArgs {
  int dtype = TP_F32, n_groups = 0, act = 0;
  int64_t n = 0;                                  // slots, fewer than 2^31
  const int32_t *ptr = nullptr, *rows = nullptr;
  const void *a = nullptr, *w = nullptr, *bias = nullptr;
  int64_t lda = 0, ldc = 0;
  int a_div = 0, c_div = 0;
  int k = 0, cols = 0;                            // contraction, columns of c
  bool transposed = false;                        // w is [n_groups][cols][k], not [k][cols]
  bool wide = false;                              // transposed: c is float32 whatever the type
  void *c = nullptr, *pre_out = nullptr;          // pre_out: before the activation, rows of c
  const void* pre = nullptr;                      // c is multiplied by the activation's slope here; rows of c
  int64_t ldpre = 0;
  hipStream_t stream = nullptr;
};
hipError_t grouped_product(const GroupedArgs& a);
// grad_w[e] = sum over the rows of group e of x^T gy, grad_bias[e] = sum of gy
struct GroupedWeightArgs {
  int dtype = TP_F32, n_groups = 0;
  int64_t n = 0, ldx = 0, ldg = 0;
  const int32_t *ptr = nullptr, *rows = nullptr;
  const void *x = nullptr, *gy = nullptr;
  int x_div = 0, g_div = 0, k = 0, cols = 0;
  void *grad_w = nullptr, *grad_bias = nullptr;
  float* part = nullptr;
  hipStream_t stream = nullptr;
};
size_t grouped_weight_workspace(int dtype, int64_t n, int n_groups, int k, int cols);
hipError_t grouped_weight_grad(const GroupedWeightArgs& a);
hipError_t combine_forward(const CombineArgs& a);
hipError_t combine_backward(const CombineArgs& a);

// ---- the AdamW step (adamw.hip) -----------------------------------------------------
constexpr int kAdamBlock = 256;                   // state values that share a unit
struct AdamArgs {
  int bits = 32, grad_dtype = TP_F32, n_tensors = 0;
  const int64_t* sizes = nullptr;                 // host
  const void* table = nullptr;
  void *m = nullptr, *v = nullptr;
  float *m_unit = nullptr, *v_unit = nullptr;
  double beta1 = 0, beta2 = 0, eps = 0, lr = 0, max_norm = 0;
  const float* lr_at = nullptr;                   // device, null: lr
  uint64_t seed = 0;
  void *scalars = nullptr, *ws = nullptr;
  float* norm = nullptr;
  const void* const* grads = nullptr;             // host
  hipStream_t stream = nullptr;
};
// bytes of the table, elements of the state arrays, bytes of the workspace; -1: too many
int64_t adamw_table_bytes(int n_tensors, const int64_t* sizes);
int64_t adamw_state_size(int n_tensors, const int64_t* sizes);
size_t adamw_workspace_bytes(int n_tensors, const int64_t* sizes);
void adamw_table_fill(int n_tensors, const int64_t* sizes, void* const* params, void* const* copies, const float* decay,
                      void* table);
hipError_t adamw_step(const AdamArgs& a);
hipError_t adamw_values(int second, int64_t n, const uint8_t* codes, const float* units, float* out, hipStream_t st);

}  // namespace tpc
