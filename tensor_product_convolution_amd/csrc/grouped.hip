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

// Rows of any length and alignment: staged through registers.  Bound by the loads: of one step they are all that a
// wave has in flight.  The launch bounds hold float32, with its two levels of sums, to two workgroups a compute unit
// (20,000 rows of 33 x 2,047: 92 against 178 us).  32,768 rows of 1,023 x 2,047, 16 groups: bfloat16 345 us (400
// TFLOP/s), float32 1,020 (134).  BM x BN tile of four waves, WM x WN
// each, S contraction values a step.  ALONG: w rows run along the contraction (transposed).
template <typename T, int BM, int BN, int WM, int WN, int S, bool ALONG>
__global__ void __launch_bounds__(kGemmThreads, 2)
    k_grouped(GroupedArgs a, int n_cols) {
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
  const int n = (int)a.n;
  const Parts parts(a.ptr, a.n_groups, a.n_groups + 1, n, BM, 0);
  if ((int)blockIdx.x >= parts.total * n_cols) return;
  int rt, ct;
  place_tile(place_of(blockIdx.x, parts.total * n_cols), parts.total, n_cols, rt, ct);
  const Part part = parts.at(rt);
  if (part.first >= part.hi) return;       // not with a valid ptr
  const int rows = min(BM, part.hi - part.first), col0 = ct * BN;
  if (tid < BM) crow[tid] = tid < rows ? row_of(a.rows, part.first + tid, a.c_div, n) : -1;
  const bool none = part.group == a.n_groups;        // slots without a group
  Sums<T, MB, NB> acc;
  acc.clear();
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
        ra[i].load(pa[i] + k, a.k - k);
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int c = tid + i * kGemmThreads;
        if (ALONG) {
          const int k = k0 + c % TB::kChunks * 8, col = min(col0 + c / TB::kChunks, a.cols - 1);
          rb[i].load(w + (int64_t)col * a.k + k, a.k - k);
        } else {
          const int k = k0 + c / TB::kChunks, col = col0 + c % TB::kChunks * 8;
          rb[i].load(w + (int64_t)min(k, a.k - 1) * a.cols + col, k < a.k ? a.cols - col : 0);
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
          for (int j = 0; j < NB; ++j) acc.part[i][j] = mma(fa[i], fb[j], acc.part[i][j]);
      }
      if ((k0 + S) % acc.kTurn == 0) acc.gather();
    }
    acc.gather();
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
        float v = acc.total(i, j)[r] + bias;
        if (a.pre) v = none ? 0.f : v * silu_slope<T>((float)((const T*)a.pre)[row * a.ldpre + col]);
        if (a.act) {
          const T z = (T)v;                // the activation is that of the stored value
          if (a.pre_out) ((T*)a.pre_out)[row * a.ldc + col] = z;
          v = silu<T>((float)z);
        }
        if (ALONG && a.wide)
          ((float*)a.c)[row * a.ldc + col] = v;
        else
          ((T*)a.c)[row * a.ldc + col] = (T)v;
      }
  }
}

// Rows of whole 16-byte chunks: WM x WN waves, each MB x NB blocks of 32 x 32, D buffers.  KS sets of such waves
// take the steps of the contraction in turn; their sums are joined in LDS.
// Large groups are bound by the matrix units and what feeds them: one group of 8,192 x 8,192 x 8,192 in bfloat16 runs at
// 1,069 TFLOP/s, transposed weights at 1,206 (a library product: 1,205); 65,536 rows of 4,096 x 1,024, 64 groups, 624 us
// (880), of 1,024 x 4,096 with the activation 795 (690): the activation and 512 MB of results follow each tile's 16 steps and
// nothing covers them in a workgroup that has the compute unit to itself.  float32 runs at 160 to 175 TFLOP/s (a library
// product: 154), bound by splitting as much as by the products; at 128 x 128 (100,000 rows, 89 groups) 45 us, twice what its
// bytes need.  Few rows are bound by their weights: 16 rows that
// choose 20 experts of 1,024 x 4,096, 37 us at 4.5 TB/s.
template <typename T, int WM, int WN, int MB, int NB, int D, int KS, bool ALONG>
__global__ void __launch_bounds__(64 * WM * WN * KS, 2)
    k_grouped_fast(GroupedArgs a, int n_cols) {
  constexpr int W = WM * WN, BM = 32 * WM * MB, BN = 32 * WN * NB, S = kDeep<T>;
  typedef AlongLds<T, BM, W> TA;
  typedef typename std::conditional<ALONG, AlongLds<T, BN, W>, AcrossLds<T, BN, W>>::type TB;
  __shared__ int arow[BM], crow[BM];
  const int tid = threadIdx.x, lane = tid & 63, id = __builtin_amdgcn_readfirstlane(tid >> 6), split = KS > 1 ? id / W : 0,
            wave = id - split * W;
  TPC_BUFFERS(D, TA, TB, KS, split);
  const int n = (int)a.n;
  const Parts parts(a.ptr, a.n_groups, a.n_groups + 1, n, BM, 0);
  if ((int)blockIdx.x >= parts.total * n_cols) return;
  int rt, ct;
  place_tile(place_of(blockIdx.x, parts.total * n_cols), parts.total, n_cols, rt, ct);
  const Part part = parts.at(rt);
  if (part.first >= part.hi) return;       // not with a valid ptr
  const int rows = min(BM, part.hi - part.first), col0 = ct * BN;
  for (int i = tid; i < BM; i += 64 * W * KS) {
    // rows past the part's end repeat its last one; nothing of them is stored
    const int place = part.first + min(i, rows - 1), slot = a.a_div || a.c_div ? slot_at(a.rows, place, n) : 0;
    arow[i] = a.a_div ? slot / a.a_div : place;
    crow[i] = i < rows ? (a.c_div ? slot : place) : -1;
  }
  const bool none = part.group == a.n_groups;        // slots without a group
  const int wm = wave / WN, wn = wave % WN;
  Sums<T, MB, NB> sums;
  sums.clear();
  if (!none) {
    const T *pa[TA::Q], *pb[TB::Q];
    const T* w = (const T*)a.w + (int64_t)part.group * a.k * a.cols;
    if constexpr (ALONG) {
#pragma unroll
      for (int q = 0; q < TB::Q; ++q)
        pb[q] = w + (int64_t)min(col0 + TB::row(q, wave, lane), a.cols - 1) * a.k + TB::first(lane);
    } else {
#pragma unroll
      for (int q = 0; q < TB::Q; ++q) {
        const int row = TB::row(q, wave, lane);
        pb[q] = w + (int64_t)row * a.cols + min(col0 + TB::first(row, lane), a.cols - TB::kPer);
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < TA::Q; ++q) pa[q] = (const T*)a.a + arow[TA::row(q, wave, lane)] * a.lda + TA::first(lane);
    const int steps = (a.k + S * KS - 1) / (S * KS);
    const T* zeros = reinterpret_cast<const T*>(kZeros);
    const auto load = [&](int t, auto buffer) {
      const int k0 = (t * KS + split) * S, mine = k0 + TA::first(lane);
      if (k0 + S <= a.k) {
#pragma unroll
        for (int q = 0; q < TA::Q; ++q) fetch16(pa[q] + k0, TA::place(buffers.a(buffer), q, wave));
#pragma unroll
        for (int q = 0; q < TB::Q; ++q)
          fetch16(pb[q] + (ALONG ? k0 : (int64_t)k0 * a.cols), TB::place(buffers.b(buffer), q, wave));
      } else {
#pragma unroll
        for (int q = 0; q < TA::Q; ++q) fetch16(mine < a.k ? pa[q] + k0 : zeros, TA::place(buffers.a(buffer), q, wave));
#pragma unroll
        for (int q = 0; q < TB::Q; ++q)
          fetch16((ALONG ? mine : k0 + TB::row(q, wave, lane)) < a.k ? pb[q] + (ALONG ? k0 : (int64_t)k0 * a.cols) : zeros,
                  TB::place(buffers.b(buffer), q, wave));
      }
    };
    const auto all = [&](auto far) {
      walk<D, TA::Q + TB::Q>(steps, load, [&](int t, auto buffer) {
        multiply<T, TA, TB, MB, NB, far()>(buffers.a(buffer), buffers.b(buffer), wm, wn, lane, sums);
        if ((t + 1) % (Sums<T, MB, NB>::kTurn / S) == 0) sums.gather();
      });
      sums.gather();
    };
    all(std::false_type());
    // an infinite operand has pieces that are not numbers: such a tile is formed again, with pieces
    // that keep infinities
    if constexpr (sizeof(T) == 4) {
      if (__syncthreads_or(!sums.finite())) {
        sums.clear();
        all(std::true_type());
      }
    }
  }
  __syncthreads();
  if constexpr (KS > 1) {
    constexpr int kOwn = 64 * 16 * MB * NB;
    static_assert(W * kOwn * sizeof(float) <= kBuffer);
    float* sum = reinterpret_cast<float*>(p0_) + wave * kOwn + lane;
    if (split > 0) sums.put(sum + split * (kBuffer / 4));
    __syncthreads();
    if (split > 0) return;
#pragma unroll
    for (int s = 1; s < KS; ++s) sums.add(sum + s * (kBuffer / 4));
  }
  float* own = buffers.template own<32 * 32 * NB * (int)sizeof(float), W>(wave);
  const int col = col0 + 32 * NB * wn + lane % (4 * NB) * 8, left = a.cols - col;
  float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.bias && !none && left > 0) load8((const T*)a.bias + (int64_t)part.group * a.cols + col, left, bias);
  hand_out<T, MB, NB>(sums, own, lane, [&](int r, int, float* v) {
    const int row = crow[32 * MB * wm + r];
    if (row < 0 || left <= 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += bias[j];
    if (a.pre) {
      float z[8];
      load8((const T*)a.pre + row * a.ldpre + col, left, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = none ? 0.f : v[j] * silu_slope<T>(z[j]);
    }
    if (a.act) {                           // the activation is that of the stored value
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)(T)v[j];
      if (a.pre_out) store8((T*)a.pre_out + row * a.ldc + col, left, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = silu<T>(v[j]);
    }
    if (ALONG && a.wide)
      store8((float*)a.c + row * a.ldc + col, left, v);
    else
      store8((T*)a.c + row * a.ldc + col, left, v);
  });
}

template <typename F>
hipError_t tiles(const GroupedArgs& a, int bm, int bn, F&& f) {
  const int64_t rows = a.n / bm + a.n_groups + 1, cols = (a.cols + bn - 1) / bn;
  if (rows * cols > 0xffffffffLL / 512) return hipErrorInvalidConfiguration;
  f(dim3((unsigned)(rows * cols)), (int)cols);
  return hipGetLastError();
}

template <typename T, int WM, int WN, int MB, int NB, int D, int KS = 1>
hipError_t fast(const GroupedArgs& a) {
  return tiles(a, 32 * WM * MB, 32 * WN * NB, [&](dim3 grid, int cols) {
    if (a.transposed)
      hipLaunchKernelGGL((k_grouped_fast<T, WM, WN, MB, NB, D, KS, true>), grid, dim3(64 * WM * WN * KS), 0, a.stream, a, cols);
    else
      hipLaunchKernelGGL((k_grouped_fast<T, WM, WN, MB, NB, D, KS, false>), grid, dim3(64 * WM * WN * KS), 0, a.stream, a, cols);
  });
}

template <typename T, int B, int W>
hipError_t any(const GroupedArgs& a) {
  constexpr int S = sizeof(T) == 4 ? 32 : 64;
  return tiles(a, B, B, [&](dim3 grid, int cols) {
    if (a.transposed)
      hipLaunchKernelGGL((k_grouped<T, B, B, W, W, S, true>), grid, dim3(kGemmThreads), 0, a.stream, a, cols);
    else
      hipLaunchKernelGGL((k_grouped<T, B, B, W, W, S, false>), grid, dim3(kGemmThreads), 0, a.stream, a, cols);
  });
}

template <typename T>
hipError_t product(const GroupedArgs& a) {
  constexpr int N = 16 / sizeof(T);
  const auto whole = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  // Only the device knows which groups occur: a table of which few do takes the tiles for few rows (1,536 rows of 4 out of
  // 118 groups against 4 of 4, float32, 256 x 256: 10.7 against 7.2 us; 128 x 128 6.2 and 5.9, bfloat16 4.5 and 4.1; from
  // 20,000 rows on within 5 %).
  const int64_t even = a.n / a.n_groups;
  const auto count = [&](int bm, int bn) { return (a.n / bm + a.n_groups / 2) * ((a.cols + bn - 1) / bn); };
  // Of any alignment: the wider tile reads the operands half as often, but has four times fewer workgroups, and
  // the loads through registers need many (bfloat16, 32,768 rows, 16 groups, 1,023 x 2,047: 382 against 434 us;
  // 8,192 rows, 8 groups, 511 x 2,047: 87 against 76).
  if (a.k % N || a.cols % N || a.lda % N || !whole(a.a) || !whole(a.w))
    return even >= 64 && count(128, 128) >= 2048 ? any<T, 128, 64>(a) : any<T, 64, 32>(a);
  // Few tiles leave most of the chip idle: four sets of waves share a tile's contraction where that is more than
  // two steps long (float32, 256 rows, 2 groups, 2,048 x 512: 24 against 48 us; 1,536 rows, 4 groups, 256 x 256:
  // 7.3 against 10.8; 288 such tiles, 512 x 2,048: 19 against 17).
  const int64_t small = count(32, 64);
  if (small <= 256 && a.k > 2 * kDeep<T>) return fast<T, 1, 2, 1, 1, 3, 4>(a);
  // Groups of few rows are bound by their weights, which narrow tiles with four buffers bring in best (bfloat16,
  // 32 rows, 32 groups, 2,048 x 512: 11.5 against 21 us).  So are bfloat16 tiles that are few (2,048 rows, 8
  // groups, 2,048 x 512, 544 tiles: 17.6 against 22.4; 4,096 rows, 1,024 x 512, 1,056 tiles: 18.2 against 15).
  if (even <= 32 || (sizeof(T) == 2 && small <= 768)) return fast<T, 1, 2, 1, 1, 4>(a);
  // Wide tiles read less and share the splitting of float32, where there are enough to fill the chip several times
  // (bfloat16, 65,536 rows, 8 groups, 512 x 2,048: 195 against 258 us; 8,192 rows: 43 against 35; float32, 16,384
  // rows: 242 against 275; 4,096 rows of 512 x 1,024: 50 against 47).
  if constexpr (sizeof(T) == 2) {
    if (even >= 192 && count(256, 256) >= 512) return fast<T, 2, 4, 4, 2, 2>(a);
    return fast<T, 1, 4, 2, 1, 2>(a);
  } else {
    if (count(128, 128) >= 1024) return fast<T, 2, 2, 2, 2, 2>(a);
    return fast<T, 2, 2, 1, 1, 2>(a);
  }
}

}  // namespace

hipError_t grouped_product(const GroupedArgs& a) {
  return a.dtype == TP_F32 ? product<float>(a) : product<bf16_t>(a);
}

}  // namespace tpc
