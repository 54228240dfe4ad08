// Weight gradients of the products by group: grad_w[e] = sum over the rows of group e of
// x^T gy, grad_bias[e] = sum of gy.
//
// Both operands have the contraction (the rows) across their tiles.  A group of more than
// `part` rows is summed in parts side by side, into the workspace, and joined in a fixed order;
// the others are written at once.
// Large groups are bound by the matrix units and by the LDS reads of two transposed operands (one group of 8,192 x 8,192 x
// 8,192 in bfloat16: 841 TFLOP/s), small matrices by the sums that the parts write and the join reads: 100,000 rows of
// 128 x 128 in float32, 89 groups, 43 us and 15.
#include <algorithm>

#include "grouped.hpp"

namespace tpc {
namespace {

// The workspace's place of a part: at most two parts of groups cut into several start within the
// same `size` slots, one of them as its group's first.
__device__ __forceinline__ int64_t part_slot(const Part& p, int size) {
  return 2 * (int64_t)(p.first / size) + (p.first == p.lo);
}

// Rows of any length and alignment: staged through registers.
template <typename T, int B, int W>
__global__ void __launch_bounds__(kGemmThreads, 2)
    k_grouped_weight(GroupedWeightArgs a, int size, int n_rows, int n_cols) {
  constexpr int S = std::is_same<T, float>::value ? 32 : 64, P = kPlanes<T>, NB = W / 32;
  static_assert((B / W) * (B / W) * 64 == kGemmThreads);
  typedef AcrossTile<T, B, S> Tile;
  constexpr int C = B * S / 8 / kGemmThreads, RPP = kGemmThreads / Tile::kChunks;    // rows of a pass of the threads
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * Tile::kElems];
  __shared__ float colsum[B];
  uint16_t *la = lds, *lb = lds + Tile::kElems;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = n_rows * n_cols, n = (int)a.n;
  const Parts parts(a.ptr, a.n_groups, a.n_groups, n, size, 1);
  if ((int)blockIdx.x >= parts.total * tiles) return;
  // tiles of a part on all dies: parts differ in length
  const int tile = blockIdx.x % tiles;
  const Part part = parts.at(blockIdx.x / tiles);
  const int k0 = tile / n_cols * B, c0 = tile % n_cols * B;
  const int end = part_end(part.first, part.hi, size);
  const bool bias = a.grad_bias && k0 == 0;
  Sums<T, NB, NB> acc;
  acc.clear();
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
      rx[i].load(px + kc, in ? a.k - kc : 0);
      rg[i].load(pg + cc, in ? a.cols - cc : 0);
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
        for (int j = 0; j < NB; ++j) acc.part[i][j] = mma(fa[i], fb[j], acc.part[i][j]);
    }
    if ((s0 - part.first + S) % acc.kTurn == 0) acc.gather();
  }
  acc.gather();
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
          ((T*)a.grad_w)[part.group * mat + at] = (T)acc.total(i, j)[r];
        else
          to[at] = acc.total(i, j)[r];
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

// Rows of whole 16-byte chunks: WM x WN waves, each MB x NB blocks of 32 x 32, D buffers.  The rows' numbers are
// loaded a step ahead of the rows, a lane each.
template <typename T, int WM, int WN, int MB, int NB, int D>
__global__ void __launch_bounds__(64 * WM * WN, 2)
    k_grouped_weight_fast(GroupedWeightArgs a, int size, int n_rows, int n_cols) {
  constexpr int W = WM * WN, BM = 32 * WM * MB, BN = 32 * WN * NB, S = kDeep<T>;
  typedef AcrossLds<T, BM, W> TA;
  typedef AcrossLds<T, BN, W> TB;
  TPC_BUFFERS(D, TA, TB, 1, 0);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = n_rows * n_cols, n = (int)a.n;
  const Parts parts(a.ptr, a.n_groups, a.n_groups, n, size, 1);
  if ((int)blockIdx.x >= parts.total * tiles) return;
  // tiles of a part on all dies: parts differ in length
  const int tile = blockIdx.x % tiles;
  const Part part = parts.at(blockIdx.x / tiles);
  const int k0 = tile / n_cols * BM, c0 = tile % n_cols * BN, end = part_end(part.first, part.hi, size);
  const int wm = wave / WN, wn = wave % WN;
  const bool bias = a.grad_bias && k0 == 0 && wm == 0;
  const T* zeros = reinterpret_cast<const T*>(kZeros);
  int next = 0;                            // the slot that this lane knows of the next step
  // of a step that is there: an empty group has no last slot, and without slots `rows` may be NULL
  const auto numbers = [&](int t) {
    const int place = part.first + t * S + (lane & (S - 1));
    next = a.x_div || a.g_div ? slot_at(a.rows, min(place, end - 1), n) : 0;
  };
  const auto load = [&](int t, auto buffer) {
    const int s0 = part.first + t * S;
#pragma unroll
    for (int q = 0; q < TA::Q; ++q) {
      const int r = TA::row(q, wave, lane), slot = __shfl(next, r, 64), row = a.x_div ? slot / a.x_div : s0 + r;
      const T* from = (const T*)a.x + row * a.ldx + min(k0 + TA::first(r, lane), a.k - TA::kPer);
      fetch16(s0 + r < end ? from : zeros, TA::place(buffers.a(buffer), q, wave));
    }
#pragma unroll
    for (int q = 0; q < TB::Q; ++q) {
      const int r = TB::row(q, wave, lane), slot = __shfl(next, r, 64), row = a.g_div ? slot : s0 + r;
      const T* from = (const T*)a.gy + row * a.ldg + min(c0 + TB::first(r, lane), a.cols - TB::kPer);
      fetch16(s0 + r < end ? from : zeros, TB::place(buffers.b(buffer), q, wave));
    }
    numbers(t + 1);
  };
  const int steps = part.first < end ? (end - part.first + S - 1) / S : 0;
  Sums<T, MB, NB> sums;
  float colsum[NB], colall[NB];            // of the bias, in two levels like the sums
  const auto gather = [&] {
    sums.gather();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      colall[j] += colsum[j];
      colsum[j] = 0.f;
    }
  };
  const auto all = [&](auto far) {
    sums.clear();
#pragma unroll
    for (int j = 0; j < NB; ++j) colsum[j] = colall[j] = 0.f;
    if (steps > 0) numbers(0);
    walk<D, TA::Q + TB::Q>(steps, load, [&](int t, auto buffer) {
      multiply<T, TA, TB, MB, NB, far(), true>(buffers.a(buffer), buffers.b(buffer), wm, wn, lane, sums, colsum, bias);
      if ((t + 1) % (Sums<T, MB, NB>::kTurn / S) == 0) gather();
    });
    gather();
  };
  all(std::false_type());
  if constexpr (sizeof(T) == 4) {          // infinities: again, with pieces that keep them
    if (__syncthreads_or(!sums.finite())) all(std::true_type());
  }
  __syncthreads();
  float* own = buffers.template own<32 * 32 * NB * (int)sizeof(float), W>(wave);
  const bool whole = part.hi - part.lo <= size;
  const int64_t mat = (int64_t)a.k * a.cols;
  float* to = whole ? nullptr : a.part + part_slot(part, size) * (mat + a.cols);
  const int col = c0 + 32 * NB * wn + lane % (4 * NB) * 8, left = a.cols - col;
  hand_out<T, MB, NB>(sums, own, lane, [&](int r, int, float* v) {
    const int row = k0 + 32 * MB * wm + r;
    if (row >= a.k || left <= 0) return;
    const int64_t at = (int64_t)row * a.cols + col;
    if (whole)
      store8((T*)a.grad_w + part.group * mat + at, left, v);
    else
      store8(to + at, left, v);
  });
  if (!bias) return;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const float s = colall[j] + __shfl_xor(colall[j], 32, 64);
    const int c = c0 + 32 * NB * wn + 32 * j + lane;
    if (lane >= 32 || c >= a.cols) continue;
    if (whole)
      ((T*)a.grad_bias)[(int64_t)part.group * a.cols + c] = (T)s;
    else
      to[mat + c] = s;
  }
}

// Groups of several parts: their sum.  `lanes` threads take every lanes-th part of four values each and are joined in
// LDS, in a fixed order.  FIND: blockIdx.y counts the groups of several parts, not all: there are at most n / size, and
// where that is much less than the groups, most workgroups would start to end at once (4,096 rows, 64 groups, 512 x
// 1,024: 32 against 44 us with the product; where all groups have several, looking for them costs 13 us more:
// 100,000 rows, 89 groups, 128 x 128).
template <typename T, bool FIND>
__global__ void __launch_bounds__(kGemmThreads)
    k_grouped_join(GroupedWeightArgs a, int size, int lanes) {
  __shared__ f4 sums[kGemmThreads];
  const int n = (int)a.n, wide = kGemmThreads / lanes, lane = threadIdx.x & 63;
  const auto start = [&](int g) { return min(max(a.ptr[g], 0), n); };
  int e = FIND ? -1 : (int)blockIdx.y, left = blockIdx.y;
  for (int g0 = 0; g0 < a.n_groups && e < 0; g0 += 64) {
    uint64_t several = __ballot(g0 + lane < a.n_groups && start(min(g0 + lane + 1, a.n_groups)) - start(min(g0 + lane, a.n_groups)) > size);
    const int here = __popcll(several);
    if (left < here) {
      for (; left > 0; --left) several &= several - 1;
      e = g0 + __ffsll((unsigned long long)several) - 1;
    } else {
      left -= here;
    }
  }
  if (e < 0) return;
  const int lo = start(e), hi = start(e + 1);
  if (hi - lo <= size) return;
  const int64_t mat = (int64_t)a.k * a.cols, all = mat + (a.grad_bias ? a.cols : 0), pitch = mat + a.cols;
  const int which = threadIdx.x / wide, parts = part_count(hi - lo, size, 1);
  for (int64_t i0 = (int64_t)blockIdx.x * wide * 4; i0 < all; i0 += (int64_t)gridDim.x * wide * 4) {
    const int64_t i = i0 + threadIdx.x % wide * 4;
    f4 s = {0.f, 0.f, 0.f, 0.f};
    if (i < all) {
#pragma unroll 4
      for (int p = which; p < parts; p += lanes) {
        const int64_t f = lo + (int64_t)p * size;
        float v[4];
        load_chunk(a.part + (2 * (f / size) + (p == 0)) * pitch + i, (int)min(all - i, (int64_t)4), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += v[j];
      }
    }
    for (int m = lanes >> 1; m > 0; m >>= 1) {
      __syncthreads();
      sums[threadIdx.x] = s;
      __syncthreads();
      if (which < m) s += sums[threadIdx.x + m * wide];
    }
    if (which == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j < mat)
          ((T*)a.grad_w)[e * mat + i + j] = (T)s[j];
        else if (i + j < all)
          ((T*)a.grad_bias)[(int64_t)e * a.cols + i + j - mat] = (T)s[j];
      }
    }
  }
}

// Tile width, rows of a part, tiles of a group
struct WeightShape {
  int tile, size;
  int64_t tiles;
};
WeightShape weight_shape(int dtype, int64_t n, int n_groups, int k, int cols) {
  WeightShape s;
  const auto count = [&](int t) { return (int64_t)((k + t - 1) / t) * ((cols + t - 1) / t); };
  // Wide tiles read less, where they are enough to fill the chip (bfloat16, 8,192 rows, 8 groups, 512 x 2,048, tiles of
  // 64, 128, 256: 50, 36, 105 us; 32,768 rows, 64 groups: 256, 175, 144; float32, 1,536 rows, 4 groups, 128 x 128, 64
  // and 128: 14 and 28).
  s.tile = k > 64 && cols > 64 && n / 256 * count(128) >= 256 ? 128 : 64;
  if (dtype == TP_BF16 && k > 128 && cols > 128 && count(256) * n_groups >= 256) s.tile = 256;
  s.tiles = count(s.tile);
  // A part is a group and a half on average, shorter where the tiles alone do not fill the chip; the sums of very
  // short ones would cost more to write and join than they bring (100,000 rows, 89 groups, 128 x 128, parts of
  // 128, 256, 512, 768 rows: float32 66, 57, 67, 78 us, bfloat16 44, 35, 34, 31; 1,536 rows, 4 groups, float32, of
  // 128 and 256: 14.1 and 15.8).
  int64_t rows = n * 3 / (2 * n_groups);
  const int fill = dtype == TP_F32 ? 512 : 384;
  if (s.tiles * n_groups < 512) rows = std::min(rows, n * s.tiles / fill);
  const int64_t least = s.tile > 64 && dtype == TP_BF16 ? 512 : s.tile == 64 && n < 8192 ? 128 : 256;
  s.size = (int)std::min<int64_t>(1 << 30, std::max<int64_t>(least, (rows + 63) / 64 * 64));
  return s;
}

template <typename T>
hipError_t weight_grad(const GroupedWeightArgs& a) {
  WeightShape s = weight_shape(a.dtype, a.n, a.n_groups, a.k, a.cols);
  constexpr int N = 16 / sizeof(T);
  const auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool fast = a.k % N == 0 && a.cols % N == 0 && a.ldx % N == 0 && a.ldg % N == 0 && aligned(a.x) && aligned(a.gy);
  // Of any alignment, wide tiles pay where they are many: 32,768 rows of 1,023 x 2,047, 16 groups, bfloat16, 680
  // against 714 us; 8,192 rows of 2,047 x 511, 8 groups, 137 against 108.
  const int64_t wide128 = (int64_t)((a.k + 127) / 128) * ((a.cols + 127) / 128) * (a.n / 256);
  const int tile = fast ? s.tile : a.k > 64 && a.cols > 64 && wide128 >= 8192 ? 128 : 64;
  const int nr = (a.k + tile - 1) / tile, nc = (a.cols + tile - 1) / tile;
  const int64_t blocks = (a.n / s.size + a.n_groups + 1) * nr * nc;
  if (blocks > 0xffffffffLL / 512) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  if (!fast && tile == 128)
    hipLaunchKernelGGL((k_grouped_weight<T, 128, 64>), grid, dim3(kGemmThreads), 0, a.stream, a, s.size, nr, nc);
  else if (!fast)
    hipLaunchKernelGGL((k_grouped_weight<T, 64, 32>), grid, dim3(kGemmThreads), 0, a.stream, a, s.size, nr, nc);
  else if (tile == 64)
    hipLaunchKernelGGL((k_grouped_weight_fast<T, 2, 2, 1, 1, 2>), grid, dim3(256), 0, a.stream, a, s.size, nr, nc);
  else if constexpr (sizeof(T) == 4)
    hipLaunchKernelGGL((k_grouped_weight_fast<T, 2, 2, 2, 2, 2>), grid, dim3(256), 0, a.stream, a, s.size, nr, nc);
  else if (tile == 128)
    hipLaunchKernelGGL((k_grouped_weight_fast<T, 2, 4, 2, 1, 2>), grid, dim3(512), 0, a.stream, a, s.size, nr, nc);
  else
    hipLaunchKernelGGL((k_grouped_weight_fast<T, 2, 4, 4, 2, 2>), grid, dim3(512), 0, a.stream, a, s.size, nr, nc);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n <= s.size) return e;
  int lanes = 1;                           // of the parts that one group can have
  while (lanes < 8 && 4 * lanes < a.n / s.size) lanes <<= 1;
  const int64_t wide = kGemmThreads / lanes * 4;
  const bool find = 2 * (a.n / s.size) < a.n_groups;
  const int64_t groups = find ? a.n / s.size : a.n_groups;
  const int64_t joins = std::min<int64_t>(std::max<int64_t>(256, 8192 / groups), ((int64_t)a.k * a.cols + a.cols + wide - 1) / wide);
  const dim3 joined((unsigned)joins, (unsigned)groups);
  if (find)
    hipLaunchKernelGGL((k_grouped_join<T, true>), joined, dim3(kGemmThreads), 0, a.stream, a, s.size, lanes);
  else
    hipLaunchKernelGGL((k_grouped_join<T, false>), joined, dim3(kGemmThreads), 0, a.stream, a, s.size, lanes);
  return hipGetLastError();
}

}  // namespace

size_t grouped_weight_workspace(int dtype, int64_t n, int n_groups, int k, int cols) {
  const WeightShape s = weight_shape(dtype, n, n_groups, k, cols);
  return n <= s.size ? 0 : 2 * ((size_t)(n / s.size) + 1) * ((size_t)k * cols + cols) * sizeof(float);
}

hipError_t grouped_weight_grad(const GroupedWeightArgs& a) {
  return a.dtype == TP_F32 ? weight_grad<float>(a) : weight_grad<bf16_t>(a);
}

}  // namespace tpc
