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
// and no cancellation as in E[x^2] - E[x]^2).
#include <algorithm>

#include "internal.hpp"
#include "rows.hpp"

namespace tpc {
namespace {

constexpr int kThreads = 256;

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

// A thread's chunks of the row's columns: chunk i starts at N (tl + TPR i).  FULL: rows are
// whole chunks (n_cols a multiple of N), so a chunk is there or not.
template <int N, int TPR, bool FULL>
struct Cols {
  int tl, C;
  __device__ __forceinline__ int at(int i) const { return (tl + TPR * i) * N; }
  __device__ __forceinline__ int left(int i) const { return FULL ? (at(i) < C ? N : 0) : C - at(i); }
};

// float32 weights of a thread's chunks
template <int N, int TPR, int VPT, bool FULL>
__device__ __forceinline__ void load_weights(const float* w, const Cols<N, TPR, FULL>& cols, float v[VPT][N]) {
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; j += 4) load_chunk(w + cols.at(i) + j, cols.left(i) - j, v[i] + j);
}

// The next row's chunks are loaded while the present row is reduced.
template <typename T, int TPR, int VPT, bool FUSED, bool FULL>
__global__ void __launch_bounds__(kThreads)
    k_norm_fwd(NormArgs a) {
  constexpr int N = Chunk<T>::kN, RPB = kThreads / TPR;
  __shared__ float2 lds[4];
  const int C = a.n_cols;
  const Cols<N, TPR, FULL> cols{(int)threadIdx.x % TPR, C};
  const float n = (float)C;                // sums are divided: a constant row has its exact mean
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool kHold = VPT * N <= 16;    // weights stay in registers
  float g[VPT][N], b[VPT][N];
  if (kHold) {
    load_weights<N, TPR, VPT, FULL>(a.gamma, cols, g);
    load_weights<N, TPR, VPT, FULL>(a.beta, cols, b);
  }
  RawChunk<T> x[VPT], r[VPT];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int left = cols.left(i);
      if (left > 0) {
        x[i].load((const T*)a.x + row * a.x_stride + cols.at(i), left);
        if (FUSED) r[i].load((const T*)a.residual + row * C + cols.at(i), left);
      }
    }
  };
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row < a.n_rows) fetch(row);
  for (; row < a.n_rows; row += step) {
    bool keep[VPT][N];
    if (FUSED && a.has_drop) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) philox_keep<N, FULL>(a.drop, (uint64_t)row * C + cols.at(i), keep[i]);
    }
    float v[VPT][N];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int left = cols.left(i);
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = left > 0 ? x[i].at(j) : 0.f;
      if (FUSED && left > 0) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          v[i][j] = a.has_drop ? drop_add(v[i][j], keep[i][j], a.drop.factor, r[i].at(j)) : v[i][j] + r[i].at(j);
        store_chunk((T*)a.h + row * C + cols.at(i), left, v[i]);
        // the norm is that of the stored row: the backward reads it back
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = j < left ? (float)(T)v[i][j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) s += v[i][j];
    }
    if (a.n_rows - row > step) fetch(row + step);
    const float mu = row_sum<TPR>(s, 0.f, lds).x / n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = v[i][j] - mu;
        q += j < cols.left(i) ? d * d : 0.f;
      }
    const float var = row_sum<TPR>(q, 0.f, lds).x / n;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (cols.tl == 0) {
      a.mean[row] = mu;
      a.rstd[row] = rstd;
    }
    if (!kHold) {
      load_weights<N, TPR, VPT, FULL>(a.gamma, cols, g);
      load_weights<N, TPR, VPT, FULL>(a.beta, cols, b);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int left = cols.left(i);
      if (left > 0) {
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = (v[i][j] - mu) * rstd * g[i][j] + b[i][j];
        store_chunk((T*)a.y + row * a.y_stride + cols.at(i), left, o);
      }
    }
  }
}

// One pass over the rows: gh (and gx), and this workgroup's part of the weight
// gradients, summed over its rows in registers, then over its row groups in
// LDS.  part [gridDim.x][2][C]; a single workgroup writes the gradients itself.
template <typename T, int TPR, int VPT, bool FULL>
__global__ void __launch_bounds__(kThreads)
    k_norm_bwd(NormBwdArgs a) {
  constexpr int N = Chunk<T>::kN, RPB = kThreads / TPR;
  __shared__ float2 lds[4];
  extern __shared__ float sums[];          // [4 waves][TPR * VPT * N] where TPR <= 64
  const int C = a.n_cols;
  const Cols<N, TPR, FULL> cols{(int)threadIdx.x % TPR, C};
  const float n = (float)C;
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool kHold = VPT * N <= 16;
  float gg[VPT][N], gb[VPT][N], g[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) gg[i][j] = gb[i][j] = 0.f;
  if (kHold) load_weights<N, TPR, VPT, FULL>(a.gamma, cols, g);
  RawChunk<T> h[VPT], gy[VPT], gr[VPT];
  float mu = 0.f, rstd = 0.f;
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int left = cols.left(i);
      if (left > 0) {
        h[i].load((const T*)a.h + row * a.h_stride + cols.at(i), left);
        gy[i].load((const T*)a.grad_y + row * a.gy_stride + cols.at(i), left);
        if (a.grad_res) gr[i].load((const T*)a.grad_res + row * C + cols.at(i), left);
      }
    }
    mu = a.mean[row];
    rstd = a.rstd[row];
  };
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row < a.n_rows) fetch(row);
  for (; row < a.n_rows; row += step) {
    bool keep[VPT][N];
    if (a.grad_x) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) philox_keep<N, FULL>(a.drop, (uint64_t)row * C + cols.at(i), keep[i]);
    }
    if (!kHold) load_weights<N, TPR, VPT, FULL>(a.gamma, cols, g);
    float z[VPT][N], t[VPT][N], res[VPT][N];
    float s1 = 0.f, s2 = 0.f;
    const float scale = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (cols.left(i) > 0) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          z[i][j] = (h[i].at(j) - mu) * scale;
          t[i][j] = gy[i].at(j);
          gg[i][j] += t[i][j] * z[i][j];
          gb[i][j] += t[i][j];
          t[i][j] *= g[i][j];
          s1 += t[i][j];
          s2 += t[i][j] * z[i][j];
          res[i][j] = a.grad_res ? gr[i].at(j) : 0.f;
        }
      }
    }
    if (a.n_rows - row > step) fetch(row + step);
    const float2 s = row_sum<TPR>(s1, s2, lds);
    const float m1 = s.x / n, m2 = s.y / n;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int left = cols.left(i);
      if (left > 0) {
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = scale * (t[i][j] - m1 - z[i][j] * m2) + res[i][j];
        store_chunk((T*)a.grad_h + row * C + cols.at(i), left, o);
        if (a.grad_x) {
#pragma unroll
          for (int j = 0; j < N; ++j) o[j] = keep[i][j] ? o[j] * a.drop.factor : 0.f;
          store_chunk((T*)a.grad_x + row * C + cols.at(i), left, o);
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
      const int left = cols.left(i);
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        if (left - j > 0) {
          store_chunk(pg + cols.at(i) + j, left - j, gg[i] + j);
          store_chunk(pb + cols.at(i) + j, left - j, gb[i] + j);
        }
      }
    }
    return;
  }
  constexpr int L = TPR * VPT * N;
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
        if (lane < TPR) sums[wv * L + (lane + TPR * i) * N + j] = s;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += kThreads)
      (pass ? pb : pg)[c] = (sums[c] + sums[L + c]) + (sums[2 * L + c] + sums[3 * L + c]);
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

// 16 bytes of the arrays per thread.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads)
    k_dropout(int64_t n, const T* x, const T* r, DropArgs d, T* out) {
  constexpr int N = Chunk<T>::kN;
  const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * N;
  if (e >= n) return;
  const int left = n - e < N ? (int)(n - e) : N;
  float v[N], q[N];
  load_chunk(x + e, left, v);
  if (RES) load_chunk(r + e, left, q);
  bool keep[N];
  philox_keep<N, true>(d, (uint64_t)e, keep);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = drop_add(v[j], keep[j], d.factor, RES ? q[j] : 0.f);
  store_chunk(out + e, left, v);
}

// (threads per row, chunks per thread) for rows of n chunks: the fewest threads
// that hold a row in one chunk each, up to a wave; then more chunks per lane;
// then the whole workgroup.
template <typename F>
hipError_t pick_shape(int n, F&& f) {
  if (n <= 4) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
  if (n <= 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  if (n <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (n <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (n <= 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  if (n <= 128) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (n <= 256) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  if (n <= 512) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  if (n <= 1024) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 256>(), std::integral_constant<int, 8>());
}

// workgroups that walk the rows: enough waves to cover the latency, few enough that weights
// are loaded and partial gradients joined seldom (32,768 rows of 1,024 bfloat16, fused:
// forward 57.9 us with 4,096, 59.0 with 1,024; backward 66.7 with 512, 72.4 with 1,024, 74.6 with 1,536)
constexpr int kFwdBlocks = 4096, kBwdBlocks = 512;

int rows_per_block(int n) {
  return n <= 4 ? 64 : n <= 8 ? 32 : n <= 16 ? 16 : n <= 32 ? 8 : n <= 256 ? 4 : 1;
}

int chunks_of(int dtype, int n_cols) {
  const int k = dtype == TP_F32 ? 4 : 8;
  return (n_cols + k - 1) / k;
}

int64_t bwd_blocks(int dtype, int64_t n_rows, int n_cols) {
  const int rpb = rows_per_block(chunks_of(dtype, n_cols));
  return std::max<int64_t>(1, std::min<int64_t>(kBwdBlocks, (n_rows + rpb - 1) / rpb));
}

template <typename T>
hipError_t norm_fwd(const NormArgs& a) {
  const int n = chunks_of(a.dtype, a.n_cols), rpb = rows_per_block(n);
  const dim3 grid((unsigned)std::min<int64_t>(kFwdBlocks, (a.n_rows + rpb - 1) / rpb));
  const bool full = a.n_cols % Chunk<T>::kN == 0;
  return pick_shape(n, [&](auto tpr, auto vpt) {
    if (a.residual) {
      if (full)
        hipLaunchKernelGGL((k_norm_fwd<T, tpr(), vpt(), true, true>), grid, dim3(kThreads), 0, a.stream, a);
      else
        hipLaunchKernelGGL((k_norm_fwd<T, tpr(), vpt(), true, false>), grid, dim3(kThreads), 0, a.stream, a);
    } else {
      if (full)
        hipLaunchKernelGGL((k_norm_fwd<T, tpr(), vpt(), false, true>), grid, dim3(kThreads), 0, a.stream, a);
      else
        hipLaunchKernelGGL((k_norm_fwd<T, tpr(), vpt(), false, false>), grid, dim3(kThreads), 0, a.stream, a);
    }
    return hipGetLastError();
  });
}

template <typename T>
hipError_t norm_bwd(const NormBwdArgs& a) {
  const int n = chunks_of(a.dtype, a.n_cols);
  const int G = (int)bwd_blocks(a.dtype, a.n_rows, a.n_cols);
  hipError_t e = pick_shape(n, [&](auto tpr, auto vpt) {
    const size_t lds = tpr() <= 64 ? (size_t)4 * tpr() * vpt() * Chunk<T>::kN * sizeof(float) : 0;
    if (a.n_cols % Chunk<T>::kN == 0)
      hipLaunchKernelGGL((k_norm_bwd<T, tpr(), vpt(), true>), dim3(G), dim3(kThreads), lds, a.stream, a);
    else
      hipLaunchKernelGGL((k_norm_bwd<T, tpr(), vpt(), false>), dim3(G), dim3(kThreads), lds, a.stream, a);
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
  const dim3 grid((unsigned)((n + per - 1) / per));
  if (r)
    hipLaunchKernelGGL((k_dropout<T, true>), grid, dim3(kThreads), 0, st, n, (const T*)x, (const T*)r, d, (T*)out);
  else
    hipLaunchKernelGGL((k_dropout<T, false>), grid, dim3(kThreads), 0, st, n, (const T*)x, (const T*)r, d, (T*)out);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(int dtype, int64_t n_rows, int n_cols) {
  const int64_t G = bwd_blocks(dtype, n_rows, n_cols);
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
