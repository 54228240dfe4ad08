// Weight gradients of the products by group: grad_w[e] = sum over the rows of group e of
// x^T gy, grad_bias[e] = sum of gy.
//
// Both operands have the contraction (the rows) across their tiles.  A group of more than
// `part` rows is summed in parts side by side, into the workspace, and joined in a fixed order;
// the others are written at once.
#include <algorithm>

#include "grouped.hpp"

namespace tpc {
namespace {

// The workspace's place of a part: at most two parts of groups cut into several start within the
// same `size` slots, one of them as its group's first.
__device__ __forceinline__ int64_t part_slot(const Part& p, int size) {
  return 2 * (int64_t)(p.first / size) + (p.first == p.lo);
}

template <typename T, int B, int W, bool EVEN>
__global__ void __launch_bounds__(kGemmThreads)
    k_grouped_weight(GroupedWeightArgs a, int size, int n_rows, int n_cols) {
  constexpr int S = std::is_same<T, float>::value ? 32 : 64, P = kPlanes<T>, NB = W / 32;
  static_assert((B / W) * (B / W) * 64 == kGemmThreads);
  typedef AcrossTile<T, B, S> Tile;
  constexpr int C = B * S / 8 / kGemmThreads, RPP = kGemmThreads / Tile::kChunks;    // rows of a pass of the threads
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * Tile::kElems];
  __shared__ float colsum[B];
  uint16_t *la = lds, *lb = lds + Tile::kElems;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = n_rows * n_cols, tile = blockIdx.x % tiles;
  Part part;
  const int n = (int)a.n;
  if (!find_part(a.ptr, a.n_groups + 1, n, size, blockIdx.x / tiles, part) || part.group == a.n_groups) return;
  const int k0 = tile / n_cols * B, c0 = tile % n_cols * B;
  const int end = min(part.hi, part.first + size);
  const bool bias = a.grad_bias && k0 == 0;
  f16v acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  float sums[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int wm = wave % (B / W), wn = wave / (B / W), chunk = tid % Tile::kChunks, trow = tid / Tile::kChunks;
  const int kc = k0 + chunk * 8, cc = c0 + chunk * 8;
  Octet<T> rx[C], rg[C];
  int ix[C], ig[C];
  const auto numbers = [&](int s0) {       // rows of the next step's slots
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int s = min(s0 + trow + i * RPP, end - 1);
      ix[i] = row_of(a.rows, s, a.x_div, n);
      ig[i] = row_of(a.rows, s, a.g_div, n);
    }
  };
  const auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const bool in = s0 + trow + i * RPP < end;
      const T *px = (const T*)a.x + ix[i] * a.ldx, *pg = (const T*)a.gy + ig[i] * a.ldg;
      if (EVEN) {
        rx[i].load(px + min(kc, a.k - 8));
        rg[i].load(pg + min(cc, a.cols - 8));
        rx[i].keep(in);
        rg[i].keep(in);
      } else {
        rx[i].load(px + kc, in ? a.k - kc : 0);
        rg[i].load(pg + cc, in ? a.cols - cc : 0);
      }
    }
  };
  if (part.first < end) {
    numbers(part.first);
    fetch(part.first);
    numbers(min(part.first + S, end - 1));
  }
  for (int s0 = part.first; s0 < end; s0 += S) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C; ++i) {
      Tile::put(la, trow + i * RPP, chunk, rx[i]);
      Tile::put(lb, trow + i * RPP, chunk, rg[i]);
      if (bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[j] += rg[i].at(j);
      }
    }
    __syncthreads();
    if (s0 + S < end) {
      fetch(s0 + S);
      numbers(min(s0 + 2 * S, end - 1));
    }
#pragma unroll
    for (int kk = 0; kk < S / 16; ++kk) {
      Frag<P> fa[NB], fb[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) fa[i] = Tile::frag(la, wm * NB + i, kk, lane);
#pragma unroll
      for (int j = 0; j < NB; ++j) fb[j] = Tile::frag(lb, wn * NB + j, kk, lane);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mma(fa[i], fb[j], acc[i][j]);
    }
  }
  const bool whole = part.hi - part.lo <= size;
  const int64_t mat = (int64_t)a.k * a.cols;
  float* to = whole ? nullptr : a.part + part_slot(part, size) * (mat + a.cols);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int col = c0 + wn * W + 32 * j + (lane & 31);
    if (col >= a.cols) continue;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = k0 + wm * W + 32 * i + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
        if (row >= a.k) continue;
        const int64_t at = (int64_t)row * a.cols + col;
        if (whole)
          ((T*)a.grad_w)[part.group * mat + at] = (T)acc[i][j][r];
        else
          to[at] = acc[i][j][r];
      }
  }
  if (!bias) return;
  // over the threads of a chunk's column, one after the other
  for (int i = 0; i < RPP; ++i) {
    __syncthreads();
    if (trow == i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) colsum[chunk * 8 + j] = (i ? colsum[chunk * 8 + j] : 0.f) + sums[j];
    }
  }
  __syncthreads();
  if (tid < B && c0 + tid < a.cols) {
    if (whole)
      ((T*)a.grad_bias)[(int64_t)part.group * a.cols + c0 + tid] = (T)colsum[tid];
    else
      to[mat + c0 + tid] = colsum[tid];
  }
}

// groups of several parts: their sum, in the parts' order
template <typename T>
__global__ void __launch_bounds__(kGemmThreads)
    k_grouped_join(GroupedWeightArgs a, int size) {
  const int n = (int)a.n, e = blockIdx.y;
  const int lo = min(max(a.ptr[e], 0), n), hi = min(max(a.ptr[e + 1], 0), n);
  if (hi - lo <= size) return;
  const int64_t mat = (int64_t)a.k * a.cols, all = mat + (a.grad_bias ? a.cols : 0);
  for (int64_t i = (int64_t)blockIdx.x * kGemmThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kGemmThreads) {
    float s = 0.f;
    for (int64_t f = lo; f < hi; f += size) s += a.part[(2 * (f / size) + (f == lo)) * (mat + a.cols) + i];
    if (i < mat)
      ((T*)a.grad_w)[e * mat + i] = (T)s;
    else
      ((T*)a.grad_bias)[(int64_t)e * a.cols + i - mat] = (T)s;
  }
}

// Tile width, and rows of a part: what even groups have and half as many again, fewer where
// tiles and groups alone would not fill the chip.
struct WeightShape {
  int tile, size;
  int64_t tiles;
};
WeightShape weight_shape(int64_t n, int n_groups, int k, int cols) {
  WeightShape s;
  s.tile = k > 64 && cols > 64 ? 128 : 64;
  s.tiles = (int64_t)((k + s.tile - 1) / s.tile) * ((cols + s.tile - 1) / s.tile);
  int64_t rows = n * 3 / (2 * n_groups);
  if (s.tiles * n_groups < 512) rows = std::min(rows, n * s.tiles / 512);
  s.size = (int)std::min<int64_t>(1 << 30, std::max<int64_t>(256, (rows + 63) / 64 * 64));
  return s;
}

template <typename T>
hipError_t weight_grad(const GroupedWeightArgs& a) {
  const WeightShape s = weight_shape(a.n, a.n_groups, a.k, a.cols);
  const int64_t parts = a.n / s.size + a.n_groups + 1;
  if (parts * s.tiles > 0xffffffffLL / kGemmThreads) return hipErrorInvalidConfiguration;
  const int nr = (a.k + s.tile - 1) / s.tile, nc = (a.cols + s.tile - 1) / s.tile;
  const dim3 grid((unsigned)(parts * s.tiles));
  const auto go = [&](auto b, auto w, auto even) {
    hipLaunchKernelGGL((k_grouped_weight<T, b(), w(), even()>), grid, dim3(kGemmThreads), 0, a.stream, a, s.size, nr, nc);
    return hipGetLastError();
  };
  const auto wide = [&](auto even) {
    return s.tile == 128 ? go(std::integral_constant<int, 128>(), std::integral_constant<int, 64>(), even)
                         : go(std::integral_constant<int, 64>(), std::integral_constant<int, 32>(), even);
  };
  hipError_t e = a.k % 8 == 0 && a.cols % 8 == 0 ? wide(std::true_type()) : wide(std::false_type());
  if (e != hipSuccess || a.n <= s.size) return e;
  const int64_t blocks = std::min<int64_t>(256, ((int64_t)a.k * a.cols + a.cols + kGemmThreads - 1) / kGemmThreads);
  hipLaunchKernelGGL(k_grouped_join<T>, dim3((unsigned)blocks, a.n_groups), dim3(kGemmThreads), 0, a.stream, a, s.size);
  return hipGetLastError();
}

}  // namespace

size_t grouped_weight_workspace(int, int64_t n, int n_groups, int k, int cols) {
  const WeightShape s = weight_shape(n, n_groups, k, cols);
  return n <= s.size ? 0 : 2 * ((size_t)(n / s.size) + 1) * ((size_t)k * cols + cols) * sizeof(float);
}

hipError_t grouped_weight_grad(const GroupedWeightArgs& a) {
  return a.dtype == TP_F32 ? weight_grad<float>(a) : weight_grad<bf16_t>(a);
}

}  // namespace tpc
