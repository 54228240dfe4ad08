// Layer norm (forward, backward, weight gradients) with an optional dropout and
// residual in front, and dropout alone.
//
//   h = T(dropout(x) + residual) or x;  y = (h - mu) rstd gamma + beta
//   t = gamma gy, z = (h - mu) rstd
//   gh = rstd (t - mean(t) - z mean(t z)) + gres;  gx = dropout(gh)
//   ggamma = sum_rows gy z,  gbeta = sum_rows gy
//
// All of it is bound by HBM: every array is read or written once.  A row lives
// in the registers of TPR threads (4 .. 256, VPT 16-byte chunks each), so the
// mean and the squared deviations are two sums over registers (no second read,
// and no cancellation as in E[x^2] - E[x]^2).  Measured, of a copy's 5.07 TB/s: 100,000
// float32 rows of 128 values at a stride of 1,152: forward 18.2 us (5.6 TB/s), backward 27.2
// (5.6) and 3.9 for the weights' join; 32,768 bfloat16 rows of 1,024 with dropout and
// residual: forward 54.8 (4.9), backward 67.0 (4.0) and 4.9.
#include <algorithm>

#include "internal.hpp"
#include "rows.hpp"

namespace tpc {
namespace {

constexpr int kThreads = 256;
static_assert(kNormMaxCols <= 256 * 8 * Chunk<float>::kN && kNormMaxCols <= 256 * 4 * Chunk<bf16_t>::kN);

// Sum of a (and b) over the TPR threads of a row, in a fixed order.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* lds) {
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int m = W / 2; m > 0; m >>= 1) {
    a += __shfl_xor(a, m, 64);
    b += __shfl_xor(b, m, 64);
  }
  if (TPR > 64) {
    __syncthreads();                       // the previous sum has been read
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) {
      a += lds[i].x;
      b += lds[i].y;
    }
  }
  return make_float2(a, b);
}

// dropout(x) + residual of one element, each operation rounded once (no fused
// multiply-add), so h does not depend on how the compiler contracts it
__device__ __forceinline__ float drop_add(float x, bool keep, float factor, float r) {
#pragma clang fp contract(off)
  const float v = keep ? x * factor : 0.f;
  return v + r;
}

// How rows divide into chunks: into whole ones; with a last chunk that is moved back to
// end with the row and shares its first elements with the one before (both hold and
// store the same values, the sums over the row take them once); or a row is shorter than
// a chunk.  A partial chunk read and stored by the element costs the wave a chain of
// branches: 20,000 bfloat16 rows of 2,803, backward 136 us, with moved chunks 98.
enum Layout { kWhole, kMoved, kShort };

// A thread's chunks of the row's columns, at(0), at(1) ..
template <int N, int TPR, Layout L>
struct Cols {
  int tl, C;
  __device__ __forceinline__ int first(int i) const { return (tl + TPR * i) * N; }
  __device__ __forceinline__ bool has(int i) const { return first(i) < C; }
  __device__ __forceinline__ int at(int i) const { return L == kMoved ? min(first(i), C - N) : first(i); }
  __device__ __forceinline__ int count() const { return L == kShort ? C : N; }
  // element j of chunk i (which is there) counts in sums over the row
  __device__ __forceinline__ bool own(int i, int j) const {
    return L == kWhole ? true : L == kMoved ? at(i) + j >= first(i) : j < C;
  }
};

// float32 weights of a thread's chunks
template <int N, int TPR, int VPT, Layout L>
__device__ __forceinline__ void load_weights(const float* w, const Cols<N, TPR, L>& cols, float v[VPT][N]) {
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; j += 4)
      if (cols.has(i)) load_chunk(w + cols.at(i) + j, cols.count() - j, v[i] + j);
}

// Which elements of a thread's chunks of a row are kept.  Random words come in blocks of
// four, and a row of odd length starts inside a block: the threads then draw whole runs of
// N words from the row's first block on, one run a chunk, and pass the bits on in LDS
// (`runs`, a byte a run), as a chunk's bits lie in two of them.  60,000 bfloat16 rows of
// 999, fused: forward 111 us, backward 144; 119 and 148 where every chunk draws all the
// blocks that it touches.
template <int N, int TPR, int VPT, Layout L>
__device__ __forceinline__ void draw_keep(const DropArgs& d, int64_t row, const Cols<N, TPR, L>& cols, uint8_t* runs,
                                          bool keep[VPT][N]) {
  const uint64_t e = (uint64_t)row * cols.C;
  if (L == kWhole || cols.C % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (cols.has(i)) philox_keep<N>(d, (e + cols.at(i)) >> 2, keep[i]);
    return;
  }
  const int m = (int)(e & 3), end = (cols.C + m + N - 1) / N;      // runs that the row needs
  const auto draw = [&](int run) {
    bool k[N];
    uint32_t bits = 0;
    philox_keep<N>(d, (e >> 2) + run * (N / 4), k);
#pragma unroll
    for (int j = 0; j < N; ++j) bits |= (uint32_t)k[j] << j;
    runs[run] = (uint8_t)bits;
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (cols.tl + TPR * i < end) draw(cols.tl + TPR * i);
  if (TPR * VPT < end && cols.tl == 0) draw(TPR * VPT);
  if (TPR > 64) {
    __syncthreads();
  } else {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = cols.at(i) + m;
    if (cols.has(i)) {
      const uint32_t bits = ((uint32_t)runs[at / N + 1] << N | runs[at / N]) >> at % N;
#pragma unroll
      for (int j = 0; j < N; ++j) keep[i][j] = bits >> j & 1;
    }
  }
}
// the bytes of `runs` for a thread's row: one for each chunk, one more where the last run
// ends past them, one more that is read and not used
template <int TPR, int VPT>
struct Runs {
  static constexpr int kRow = TPR * VPT + 2, kBytes = kThreads / TPR * kRow;
  static __device__ __forceinline__ uint8_t* of(uint8_t* lds) { return lds + threadIdx.x / TPR * kRow; }
};

// The next row's chunks are loaded while the present row is reduced.
template <typename T, int TPR, int VPT, bool FUSED, Layout L>
__global__ void __launch_bounds__(kThreads)
    k_norm_fwd(NormArgs a) {
  constexpr int N = Chunk<T>::kN, RPB = kThreads / TPR;
  __shared__ float2 lds[4];
  __shared__ uint8_t runs[L == kWhole || !FUSED ? 1 : Runs<TPR, VPT>::kBytes];
  const int C = a.n_cols;
  const Cols<N, TPR, L> cols{(int)threadIdx.x % TPR, C};
  const float n = (float)C;                // sums are divided: a constant row has its exact mean
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool kHold = VPT * N <= 16;    // weights stay in registers
  float g[VPT][N], b[VPT][N];
  if (kHold) {
    load_weights<N, TPR, VPT, L>(a.gamma, cols, g);
    load_weights<N, TPR, VPT, L>(a.beta, cols, b);
  }
  RawChunk<T> x[VPT], r[VPT];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (cols.has(i)) {
        x[i].load((const T*)a.x + row * a.x_stride + cols.at(i), cols.count());
        if (FUSED) r[i].load((const T*)a.residual + row * C + cols.at(i), cols.count());
      }
    }
  };
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row < a.n_rows) fetch(row);
  for (; row < a.n_rows; row += step) {
    bool keep[VPT][N];
    if (FUSED && a.has_drop) draw_keep<N, TPR, VPT, L>(a.drop, row, cols, Runs<TPR, VPT>::of(runs), keep);
    float v[VPT][N];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool has = cols.has(i);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[i][j] = has ? x[i].at(j) : 0.f;
        if (FUSED && has) {
          v[i][j] = a.has_drop ? drop_add(v[i][j], keep[i][j], a.drop.factor, r[i].at(j)) : v[i][j] + r[i].at(j);
          // the norm is that of the stored row: the backward reads it back
          v[i][j] = (float)(T)v[i][j];
        }
        s += has && cols.own(i, j) ? v[i][j] : 0.f;
      }
    }
    if (a.n_rows - row > step) fetch(row + step);
    const float mu = row_sum<TPR>(s, 0.f, lds).x / n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = v[i][j] - mu;
        q += cols.has(i) && cols.own(i, j) ? d * d : 0.f;
      }
    // stored when the whole row has been read (h may take the place of x or residual)
    if (FUSED) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (cols.has(i)) store_chunk((T*)a.h + row * C + cols.at(i), cols.count(), v[i]);
    }
    const float var = row_sum<TPR>(q, 0.f, lds).x / n;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (cols.tl == 0) {
      a.mean[row] = mu;
      a.rstd[row] = rstd;
    }
    if (!kHold) {
      load_weights<N, TPR, VPT, L>(a.gamma, cols, g);
      load_weights<N, TPR, VPT, L>(a.beta, cols, b);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (cols.has(i)) {
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = (v[i][j] - mu) * rstd * g[i][j] + b[i][j];
        store_chunk((T*)a.y + row * a.y_stride + cols.at(i), cols.count(), o);
      }
    }
  }
}

// One pass over the rows: gh (and gx), and this workgroup's part of the weight
// gradients, summed over its rows in registers, then over its row groups in
// LDS.  part [gridDim.x][2][C]; a single workgroup writes the gradients itself.
template <typename T, int TPR, int VPT, Layout L>
__global__ void __launch_bounds__(kThreads)
    k_norm_bwd(NormBwdArgs a) {
  constexpr int N = Chunk<T>::kN, RPB = kThreads / TPR;
  __shared__ float2 lds[4];
  __shared__ uint8_t runs[L == kWhole ? 1 : Runs<TPR, VPT>::kBytes];
  extern __shared__ float sums[];          // [4 waves][TPR * VPT * N] where TPR <= 64
  const int C = a.n_cols;
  const Cols<N, TPR, L> cols{(int)threadIdx.x % TPR, C};
  const float n = (float)C;
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool kHold = VPT * N <= 16;
  float gg[VPT][N], gb[VPT][N], g[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) gg[i][j] = gb[i][j] = 0.f;
  if (kHold) load_weights<N, TPR, VPT, L>(a.gamma, cols, g);
  RawChunk<T> h[VPT], gy[VPT], gr[VPT];
  float mu = 0.f, rstd = 0.f;
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (cols.has(i)) {
        h[i].load((const T*)a.h + row * a.h_stride + cols.at(i), cols.count());
        gy[i].load((const T*)a.grad_y + row * a.gy_stride + cols.at(i), cols.count());
        if (a.grad_res) gr[i].load((const T*)a.grad_res + row * C + cols.at(i), cols.count());
      }
    }
    mu = a.mean[row];
    rstd = a.rstd[row];
  };
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row < a.n_rows) fetch(row);
  for (; row < a.n_rows; row += step) {
    bool keep[VPT][N];
    if (a.grad_x) draw_keep<N, TPR, VPT, L>(a.drop, row, cols, Runs<TPR, VPT>::of(runs), keep);
    if (!kHold) load_weights<N, TPR, VPT, L>(a.gamma, cols, g);
    float z[VPT][N], t[VPT][N], res[VPT][N];
    float s1 = 0.f, s2 = 0.f;
    const float scale = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (cols.has(i)) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          z[i][j] = (h[i].at(j) - mu) * scale;
          t[i][j] = gy[i].at(j);
          gg[i][j] += t[i][j] * z[i][j];
          gb[i][j] += t[i][j];
          t[i][j] *= g[i][j];
          s1 += cols.own(i, j) ? t[i][j] : 0.f;
          s2 += cols.own(i, j) ? t[i][j] * z[i][j] : 0.f;
          res[i][j] = a.grad_res ? gr[i].at(j) : 0.f;
        }
      }
    }
    if (a.n_rows - row > step) fetch(row + step);
    const float2 s = row_sum<TPR>(s1, s2, lds);
    const float m1 = s.x / n, m2 = s.y / n;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (cols.has(i)) {
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = scale * (t[i][j] - m1 - z[i][j] * m2) + res[i][j];
        store_chunk((T*)a.grad_h + row * C + cols.at(i), cols.count(), o);
        if (a.grad_x) {
#pragma unroll
          for (int j = 0; j < N; ++j) o[j] = keep[i][j] ? o[j] * a.drop.factor : 0.f;
          store_chunk((T*)a.grad_x + row * C + cols.at(i), cols.count(), o);
        }
      }
    }
  }
  if (!a.grad_gamma) return;
  float* pg = gridDim.x == 1 ? a.grad_gamma : a.part + (size_t)blockIdx.x * 2 * C;
  float* pb = gridDim.x == 1 ? a.grad_beta : pg + C;
  if (TPR > 64) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        if (cols.has(i)) {                 // columns that two chunks share have the same sums in both
          store_chunk(pg + cols.at(i) + j, N, gg[i] + j);
          store_chunk(pb + cols.at(i) + j, N, gb[i] + j);
        }
      }
    }
    return;
  }
  constexpr int kCols = TPR * VPT * N;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float s = pass ? gb[i][j] : gg[i][j];
#pragma unroll
        for (int m = TPR; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
        if (lane < TPR && cols.has(i)) sums[wv * kCols + cols.at(i) + j] = s;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += kThreads)
      (pass ? pb : pg)[c] = (sums[c] + sums[kCols + c]) + (sums[2 * kCols + c] + sums[3 * kCols + c]);
    __syncthreads();
  }
}

// Weight gradients from the workgroups' parts: 16 columns of [2][C] per
// workgroup, 64 threads per column, joined in LDS in a fixed order.
constexpr int kJoinCols = 16, kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads)
    k_norm_join(const float* __restrict__ part, int G, int C, float* __restrict__ gg, float* __restrict__ gb) {
  __shared__ float lds[kJoinThreads];
  const int col = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, grp = threadIdx.x / kJoinCols;
  float s = 0.f;
  if (col < 2 * C) {
#pragma unroll 8
    for (int b = grp; b < G; b += kJoinThreads / kJoinCols) s += part[(size_t)b * 2 * C + col];
  }
  lds[threadIdx.x] = s;
#pragma unroll
  for (int m = kJoinThreads / 2; m >= kJoinCols; m >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < m) lds[threadIdx.x] += lds[threadIdx.x + m];
  }
  if (grp == 0 && col < 2 * C) (col < C ? gg[col] : gb[col - C]) = lds[threadIdx.x];
}

// 16 bytes of the arrays per thread.  100,000 x 1,152 bfloat16: 121 us with a residual (5.7
// TB/s), 97 without (4.7: there the random words, 20 products a block of four, bound it).
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads)
    k_dropout(int64_t n, const T* x, const T* r, DropArgs d, T* out) {
  constexpr int N = Chunk<T>::kN;
  const int64_t e = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x) * N;
  if (e >= n) return;
  const int left = n - e < N ? (int)(n - e) : N;
  float v[N], q[N];
  load_chunk(x + e, left, v);
  if (RES) load_chunk(r + e, left, q);
  bool keep[N];
  philox_keep<N>(d, (uint64_t)e >> 2, keep);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = drop_add(v[j], keep[j], d.factor, RES ? q[j] : 0.f);
  store_chunk(out + e, left, v);
}

// (threads per row, chunks per thread, layout) for rows of n_cols values: the fewest threads
// that hold a row in one chunk each, up to a wave; then more chunks per lane; then the
// whole workgroup.  Two exceptions.  A float32 row of 33 to 48 chunks would leave up to half a
// wave idle: 16 x 3 (100,000 rows of 132, us: forward 17.7 against 22.5, backward 31.6 against
// 37.6).  A bfloat16 row of 129 to 256 chunks, 8 values each, would take 256 registers a
// lane: 256 x 1 (14,648 rows of 2,048: 21.7 against 24.2, 38.8 against 50.3); float32's
// half as large chunks are better off in one wave (29,296 rows of 1,024: 36.1 against 38.4).
template <int TPR, int VPT, typename F>
hipError_t pick_layout(bool whole, F&& f) {
  const std::integral_constant<int, TPR> tpr;
  const std::integral_constant<int, VPT> vpt;
  return whole ? f(tpr, vpt, std::integral_constant<Layout, kWhole>()) : f(tpr, vpt, std::integral_constant<Layout, kMoved>());
}
template <typename T, typename F>
hipError_t pick_shape(int n_cols, F&& f) {
  constexpr int N = Chunk<T>::kN;
  constexpr bool kSmall = N == 4;          // chunks of few values
  const int n = (n_cols + N - 1) / N;
  const bool whole = n_cols % N == 0;
  if (n_cols < N)
    return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>(), std::integral_constant<Layout, kShort>());
  if (n <= 4) return pick_layout<4, 1>(whole, f);
  if (n <= 8) return pick_layout<8, 1>(whole, f);
  if (n <= 16) return pick_layout<16, 1>(whole, f);
  if (n <= 32) return pick_layout<32, 1>(whole, f);
  if constexpr (kSmall)
    if (n <= 48) return pick_layout<16, 3>(whole, f);
  if (n <= 64) return pick_layout<64, 1>(whole, f);
  if (n <= 128) return pick_layout<64, 2>(whole, f);
  if (n <= 256) return pick_layout<kSmall ? 64 : 256, kSmall ? 4 : 1>(whole, f);
  if (n <= 512) return pick_layout<256, 2>(whole, f);
  if constexpr (kSmall)
    if (n > 1024) return pick_layout<256, 8>(whole, f);
  return pick_layout<256, 4>(whole, f);    // kNormMaxCols bfloat16 values are 1,024 chunks
}

// workgroups that walk the rows: enough waves to cover the latency, few enough that weights
// are loaded and partial gradients joined seldom (32,768 rows of 1,024 bfloat16, fused:
// forward 57.9 us with 4,096, 59.0 with 1,024; backward 66.7 with 512, 72.4 with 1,024, 74.6 with 1,536)
constexpr int kFwdBlocks = 4096, kBwdBlocks = 512;

template <typename T>
int64_t blocks_for(int64_t n_rows, int n_cols, int most) {
  int64_t rows = 1;                        // of one workgroup
  (void)pick_shape<T>(n_cols, [&](auto tpr, auto, auto) {
    rows = kThreads / tpr();
    return hipSuccess;
  });
  return std::max<int64_t>(1, std::min<int64_t>(most, (n_rows + rows - 1) / rows));
}

template <typename T>
hipError_t norm_fwd(const NormArgs& a) {
  const dim3 grid((unsigned)blocks_for<T>(a.n_rows, a.n_cols, kFwdBlocks));
  return pick_shape<T>(a.n_cols, [&](auto tpr, auto vpt, auto layout) {
    if (a.residual)
      hipLaunchKernelGGL((k_norm_fwd<T, tpr(), vpt(), true, layout()>), grid, dim3(kThreads), 0, a.stream, a);
    else
      hipLaunchKernelGGL((k_norm_fwd<T, tpr(), vpt(), false, layout()>), grid, dim3(kThreads), 0, a.stream, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t norm_bwd(const NormBwdArgs& a) {
  const int G = (int)blocks_for<T>(a.n_rows, a.n_cols, kBwdBlocks);
  hipError_t e = pick_shape<T>(a.n_cols, [&](auto tpr, auto vpt, auto layout) {
    const size_t lds = tpr() <= 64 ? (size_t)4 * tpr() * vpt() * Chunk<T>::kN * sizeof(float) : 0;
    hipLaunchKernelGGL((k_norm_bwd<T, tpr(), vpt(), layout()>), dim3(G), dim3(kThreads), lds, a.stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess || G == 1 || !a.grad_gamma) return e;
  hipLaunchKernelGGL(k_norm_join, dim3((2 * a.n_cols + kJoinCols - 1) / kJoinCols), dim3(kJoinThreads), 0, a.stream,
                     a.part, G, a.n_cols, a.grad_gamma, a.grad_beta);
  return hipGetLastError();
}

template <typename T>
hipError_t dropout(int64_t n, const void* x, const void* r, const DropArgs& d, void* out, hipStream_t st) {
  const int64_t per = (int64_t)kThreads * Chunk<T>::kN;
  // rows of 2^22 workgroups: a grid's dimension holds fewer than 2^32 threads
  const int64_t blocks = (n + per - 1) / per, row = std::min<int64_t>(blocks, 1 << 22);
  const dim3 grid((unsigned)row, (unsigned)((blocks + row - 1) / row));
  if (r)
    hipLaunchKernelGGL((k_dropout<T, true>), grid, dim3(kThreads), 0, st, n, (const T*)x, (const T*)r, d, (T*)out);
  else
    hipLaunchKernelGGL((k_dropout<T, false>), grid, dim3(kThreads), 0, st, n, (const T*)x, (const T*)r, d, (T*)out);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(int dtype, int64_t n_rows, int n_cols) {
  const int64_t G = dtype == TP_F32 ? blocks_for<float>(n_rows, n_cols, kBwdBlocks) : blocks_for<bf16_t>(n_rows, n_cols, kBwdBlocks);
  return G == 1 ? 0 : (size_t)G * 2 * n_cols * sizeof(float);
}

hipError_t norm_forward(const NormArgs& a) {
  return a.dtype == TP_F32 ? norm_fwd<float>(a) : norm_fwd<bf16_t>(a);
}

hipError_t norm_backward(const NormBwdArgs& a) {
  return a.dtype == TP_F32 ? norm_bwd<float>(a) : norm_bwd<bf16_t>(a);
}

hipError_t dropout_apply(int dtype, int64_t n, const void* x, const void* r, const DropArgs& d, void* out,
                         hipStream_t st) {
  return dtype == TP_F32 ? dropout<float>(n, x, r, d, out, st) : dropout<bf16_t>(n, x, r, d, out, st);
}

}  // namespace tpc
