// Products of rows with the weights of their group (element or expert), forward and with
// respect to the rows:
//
//   z_s = x_s W_e(s) + b_e(s),  y = z or silu(z);     grad x_s = grad z_s W_e(s)^T [silu'(pre_s)]
//
// over ragged groups that only the device knows.
#include <algorithm>

#include "grouped.hpp"

namespace tpc {
namespace {

// BM x BN tile of four waves, WM x WN each, S contraction values a step.  ALONG: w rows run along the contraction
// (transposed).  EVEN: contraction and columns are multiples of 8.
template <typename T, int BM, int BN, int WM, int WN, int S, bool ALONG, bool EVEN>
__global__ void __launch_bounds__(kGemmThreads)
    k_grouped(GroupedArgs a, int n_rows, int n_cols) {
  constexpr int P = kPlanes<T>, MB = WM / 32, NB = WN / 32;
  static_assert((BM / WM) * (BN / WN) * 64 == kGemmThreads);
  typedef AlongTile<T, BM, S> TA;
  typedef typename std::conditional<ALONG, AlongTile<T, BN, S>, AcrossTile<T, BN, S>>::type TB;
  constexpr int CA = BM * TA::kChunks / kGemmThreads, CB = BN * S / 8 / kGemmThreads;
  static_assert(CA >= 1 && CB >= 1);
  __shared__ __attribute__((aligned(16))) uint16_t lds[TA::kElems + TB::kElems];
  __shared__ int crow[BM];
  uint16_t *la = lds, *lb = lds + TA::kElems;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int rt, ct;
  place_tile(blockIdx.x, n_rows, n_cols, rt, ct);
  Part part;
  const int n = (int)a.n;
  if (!find_part(a.ptr, a.n_groups + 1, n, BM, rt, part) || part.first >= part.hi) return;
  const int rows = min(BM, part.hi - part.first), col0 = ct * BN;
  if (tid < BM) crow[tid] = tid < rows ? row_of(a.rows, part.first + tid, a.c_div, n) : -1;
  const bool none = part.group == a.n_groups;        // slots without a group
  f16v acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int wm = wave % (BM / WM), wn = wave / (BM / WM);
  if (!none) {
    const T* pa[CA];
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      // rows past the part's end repeat its last one; nothing of them is stored
      const int row = min((tid + i * kGemmThreads) / TA::kChunks, rows - 1);
      pa[i] = (const T*)a.a + (int64_t)row_of(a.rows, part.first + row, a.a_div, n) * a.lda;
    }
    const T* w = (const T*)a.w + (int64_t)part.group * a.k * a.cols;
    Octet<T> ra[CA], rb[CB];
    const auto fetch = [&](int k0) {
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int k = k0 + (tid + i * kGemmThreads) % TA::kChunks * 8;
        if (EVEN) {
          ra[i].load(pa[i] + min(k, a.k - 8));
          ra[i].keep(k < a.k);
        } else {
          ra[i].load(pa[i] + k, a.k - k);
        }
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int c = tid + i * kGemmThreads;
        if (ALONG) {
          const int k = k0 + c % TB::kChunks * 8, col = min(col0 + c / TB::kChunks, a.cols - 1);
          if (EVEN) {
            rb[i].load(w + (int64_t)col * a.k + min(k, a.k - 8));
            rb[i].keep(k < a.k);
          } else {
            rb[i].load(w + (int64_t)col * a.k + k, a.k - k);
          }
        } else {
          const int k = k0 + c / TB::kChunks, col = col0 + c % TB::kChunks * 8;
          if (EVEN) {
            rb[i].load(w + (int64_t)min(k, a.k - 1) * a.cols + min(col, a.cols - 8));
            rb[i].keep(k < a.k);
          } else {
            rb[i].load(w + (int64_t)min(k, a.k - 1) * a.cols + col, k < a.k ? a.cols - col : 0);
          }
        }
      }
    };
    fetch(0);
    for (int k0 = 0; k0 < a.k; k0 += S) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int c = tid + i * kGemmThreads;
        TA::put(la, c / TA::kChunks, c % TA::kChunks, ra[i]);
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int c = tid + i * kGemmThreads;
        TB::put(lb, c / TB::kChunks, c % TB::kChunks, rb[i]);
      }
      __syncthreads();
      if (k0 + S < a.k) fetch(k0 + S);
#pragma unroll
      for (int kk = 0; kk < S / 16; ++kk) {
        Frag<P> fa[MB], fb[NB];
#pragma unroll
        for (int i = 0; i < MB; ++i) fa[i] = TA::frag(la, wm * MB + i, kk, lane);
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[j] = TB::frag(lb, wn * NB + j, kk, lane);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) acc[i][j] = mma(fa[i], fb[j], acc[i][j]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int col = col0 + wn * WN + 32 * j + (lane & 31);
    if (col >= a.cols) continue;
    const float bias = a.bias && !none ? (float)((const T*)a.bias)[(int64_t)part.group * a.cols + col] : 0.f;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = crow[wm * WM + 32 * i + 8 * (r / 4) + 4 * (lane >> 5) + r % 4];
        if (row < 0) continue;
        float v = acc[i][j][r] + bias;
        if (a.pre) v = none ? 0.f : v * silu_slope((float)((const T*)a.pre)[row * a.ldpre + col]);
        if (a.act) {
          const T z = (T)v;                // the activation is that of the stored value
          if (a.pre_out) ((T*)a.pre_out)[row * a.ldc + col] = z;
          v = silu((float)z);
        }
        ((T*)a.c)[row * a.ldc + col] = (T)v;
      }
  }
}

template <typename T, int BM, int BN, int WM, int WN, int S>
hipError_t launch(const GroupedArgs& a) {
  const int64_t rows = a.n / BM + a.n_groups + 1, cols = (a.cols + BN - 1) / BN;
  if (rows * cols > 0xffffffffLL / kGemmThreads) return hipErrorInvalidConfiguration;
  const bool even = a.k % 8 == 0 && a.cols % 8 == 0;
  const auto go = [&](auto along, auto whole) {
    hipLaunchKernelGGL((k_grouped<T, BM, BN, WM, WN, S, along(), whole()>), dim3((unsigned)(rows * cols)), dim3(kGemmThreads), 0,
                       a.stream, a, (int)rows, (int)cols);
    return hipGetLastError();
  };
  const auto first = [&](auto along) { return even ? go(along, std::true_type()) : go(along, std::false_type()); };
  return a.transposed ? first(std::true_type()) : first(std::false_type());
}

template <typename T>
hipError_t product(const GroupedArgs& a) {
  if (a.n <= 32 * (int64_t)a.n_groups) return launch<T, 32, 128, 32, 32, 64>(a);
  return launch<T, 128, 128, 64, 64, kPlanes<T> == 3 ? 32 : 64>(a);
}

}  // namespace

hipError_t grouped_product(const GroupedArgs& a) {
  return a.dtype == TP_F32 ? product<float>(a) : product<bf16_t>(a);
}

}  // namespace tpc
