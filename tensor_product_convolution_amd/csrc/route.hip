// Routing of rows to groups: the choice of the k best groups of each row with their weights,
// the stable order of the choices by group, and the weighted sum over a row's choices.
//
//   chosen = the k largest logits of a row, the lowest index first among equals
//   w_j = softmax over the chosen (or over all) at the chosen
//   backward, over the chosen: grad l_j = w_j sum_i w_i (gw_j - gw_i)
//   out = sum_j w_j y_j;  grad y_j = w_j grad_out, grad w_j = grad_out . y_j
//
// The choice is one comparison of a 64-bit key a step: the logit as an ordered integer over the
// inverted index.  The order by group is a counting sort in which a wave numbers its 64
// entries at once: the lanes of one group find each other by a ballot per bit of the group.
// All of it is bound by HBM for many rows and by the launches for few: up to 8,192 entries are
// ordered by one launch, more by three.  4,096 rows of 8 logits take 4.7 us either way, 32,768 of 64 7.3; the order of
// 1,536 entries 5.4 us, of 8,192 11, of 100,000 in 89 groups 21 (8 us and less a launch, each little more than its
// chain of loads); the sums of 32,768 rows of 2 x 1,024 in bfloat16 33 us (201 MB, 6.1 TB/s, part of it still in the
// last cache).
#include <algorithm>

#include "internal.hpp"
#include "rows.hpp"

namespace tpc {
namespace {

constexpr int kThreads = 256;
typedef unsigned long long u64;

template <typename T>
__device__ __forceinline__ float value_of(const T* p) {
  return (float)*p;
}

// 0 for what no row may choose: minus infinity and NaN
__device__ __forceinline__ u64 key_of(float x, int e) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);          // -0 equals 0
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (u64)o << 32 | (0xffffffffu - (uint32_t)e);
}
__device__ __forceinline__ float logit_of(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int group_of(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int m = lanes >> 1; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}
__device__ __forceinline__ float lanes_max(float v, int lanes) {
  for (int m = lanes >> 1; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  return v;
}

// VPT logits a thread, `lanes` threads a row
template <typename T, int VPT>
__global__ void __launch_bounds__(kThreads)
    k_route_fwd(RouteArgs a, int lanes) {
  const int per = kThreads / lanes, lane = threadIdx.x % lanes;
  const int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / lanes;
  const bool has = row < a.n_rows;         // the same for all threads of a row
  const T* l = (const T*)a.logits + (has ? row : 0) * a.stride;
  u64 key[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = lane + i * lanes;
    key[i] = has && e < a.n_groups ? key_of(value_of(l + e), e) : 0;
  }
  float top = 0.f, all = 0.f;
  u64 won[kMaxChoices];
  // rolled: unrolled, 32,768 rows of 64 take 8.9 us against 6.9
#pragma unroll 1
  for (int j = 0; j < kMaxChoices; ++j) {
    if (j >= a.k) break;
    u64 best = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) best = key[i] > best ? key[i] : best;
    for (int m = lanes >> 1; m > 0; m >>= 1) {
      const u64 o = __shfl_xor(best, m, 64);
      best = o > best ? o : best;
    }
    won[j] = best;
    if (j == 0) {
      top = logit_of(best);
      if (a.over_all) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) s += key[i] ? expf(logit_of(key[i]) - top) : 0.f;
        all = lanes_sum(s, lanes);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) key[i] = key[i] == best ? 0 : key[i];
  }
  if (!has) return;
  float e[kMaxChoices], sum = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxChoices; ++j) {
    if (j >= a.k) break;
    e[j] = won[j] ? expf(logit_of(won[j]) - top) : 0.f;
    sum += e[j];
  }
  if (a.over_all) sum = all;
#pragma unroll
  for (int j = 0; j < kMaxChoices; ++j) {
    if (j >= a.k) break;
    if (j % lanes != lane) continue;
    a.weight[row * a.k + j] = won[j] ? e[j] / sum : 0.f;
    a.index[row * a.k + j] = won[j] ? group_of(won[j]) : -1;
  }
}

// Differences of the weights' gradients come first: where one weight is nearly 1, a gradient
// less the weighted mean would cancel.  Over all groups, those not chosen count as choices
// without a gradient.
template <typename T, int VPT>
__global__ void __launch_bounds__(kThreads)
    k_route_bwd(RouteArgs a, int lanes) {
  const int per = kThreads / lanes, lane = threadIdx.x % lanes;
  const int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / lanes;
  const bool has = row < a.n_rows;
  const int64_t at = has ? row : 0;
  float w[kMaxChoices], g[kMaxChoices];
  int idx[kMaxChoices];
#pragma unroll
  for (int j = 0; j < kMaxChoices; ++j) {
    const bool live = j < a.k && has;
    idx[j] = live ? a.index_in[at * a.k + j] : -1;
    w[j] = live && idx[j] >= 0 ? a.weight_in[at * a.k + j] : 0.f;
    g[j] = live && idx[j] >= 0 ? a.grad_weight[at * a.k + j] : 0.f;
  }
  float p[VPT], rest = 0.f, mean = 0.f;
  if (a.over_all) {
    const T* l = (const T*)a.logits + at * a.stride;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = lane + i * lanes;
      p[i] = has && e < a.n_groups ? value_of(l + e) : -INFINITY;
      p[i] = p[i] > -INFINITY ? p[i] : -INFINITY;
      top = fmaxf(top, p[i]);
    }
    top = lanes_max(top, lanes);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      p[i] = p[i] > -INFINITY ? expf(p[i] - top) : 0.f;
      sum += p[i];
    }
    sum = lanes_sum(sum, lanes);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      p[i] = sum > 0.f || sum != sum ? p[i] / sum : 0.f;
      bool chosen = false;
#pragma unroll
      for (int j = 0; j < kMaxChoices; ++j) chosen |= j < a.k && idx[j] == lane + i * lanes;
      rest += chosen ? 0.f : p[i];
    }
    rest = lanes_sum(rest, lanes);
#pragma unroll
    for (int j = 0; j < kMaxChoices; ++j) mean += w[j] * g[j];
  }
  if (!has) return;
  T* out = (T*)a.grad_logits + row * a.n_groups;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = lane + i * lanes;
    if (e >= a.n_groups) break;
    float d = a.over_all ? -p[i] * mean : 0.f;
#pragma unroll
    for (int j = 0; j < kMaxChoices; ++j) {
      if (j >= a.k) break;
      if (idx[j] != e) continue;
      float s = a.over_all ? g[j] * rest : 0.f;
#pragma unroll
      for (int i2 = 0; i2 < kMaxChoices; ++i2) s += w[i2] * (g[j] - g[i2]);
      d = w[j] * s;
    }
    out[e] = (T)d;
  }
}

// threads of a row: 4 logits each up to 256 groups, 16 beyond, so that a row stays in a wave
template <typename F>
hipError_t pick_route(const RouteArgs& a, F&& f) {
  const int vpt = a.n_groups > 256 ? 16 : 4;
  int lanes = 1;
  while (lanes * vpt < a.n_groups) lanes <<= 1;
  const int64_t blocks = (a.n_rows + kThreads / lanes - 1) / (kThreads / lanes);
  if (blocks > 0xffffffffLL / kThreads) return hipErrorInvalidConfiguration;
  const auto typed = [&](auto t) {
    return vpt == 16 ? f(t, std::integral_constant<int, 16>(), lanes, dim3((unsigned)blocks))
                     : f(t, std::integral_constant<int, 4>(), lanes, dim3((unsigned)blocks));
  };
  return a.dtype == TP_F32 ? typed(float()) : typed(bf16_t());
}

// ---- order by group -------------------------------------------------------------------
// Entries are numbered by waves, each over a run of consecutive ones.  Group n_groups is that
// of the entries without a group; lanes past the end have n_groups + 1.
constexpr int kSmallWaves = 16;

__device__ __forceinline__ int entry_group(const int32_t* index, int64_t i, int64_t end, int n_groups) {
  if (i >= end) return n_groups + 1;
  const int32_t g = index[i];
  return g >= 0 && g < n_groups ? g : n_groups;
}

// the lanes that hold the same group
__device__ __forceinline__ u64 same_group(int g, int bits) {
  u64 m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = g >> b & 1;
    const u64 v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

__device__ __forceinline__ void wave_order() {     // LDS accesses of a wave on its own stay in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's run goes in blocks of kBlock entries, kEach a lane, loaded together.
constexpr int kEach = 8, kBlock = 64 * kEach;
struct Block {
  int g[kEach];
  u64 same[kEach];
  __device__ __forceinline__ void load(const int32_t* index, int64_t first, int64_t end, int n_groups, int bits) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kEach; ++j) g[j] = entry_group(index, first + 64 * j + lane, end, n_groups);
#pragma unroll
    for (int j = 0; j < kEach; ++j) same[j] = same_group(g[j], bits);
  }
  __device__ __forceinline__ void count(int n_groups, int* cnt) const {
    const u64 before = (1ull << (threadIdx.x & 63)) - 1;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (g[j] <= n_groups && (same[j] & before) == 0) cnt[g[j]] += __popcll(same[j]);
      wave_order();
    }
  }
  __device__ __forceinline__ void place(int64_t first, int n_groups, int* at, int32_t* rows) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const u64 before = same[j] & ((1ull << lane) - 1);
      const int to = g[j] <= n_groups ? at[g[j]] : 0;
      wave_order();
      if (g[j] <= n_groups) {
        rows[to + __popcll(before)] = (int32_t)(first + 64 * j + lane);
        if (before == 0) at[g[j]] = to + __popcll(same[j]);
      }
      wave_order();
    }
  }
};

// v[i] for i < n in LDS becomes the sum of those before it; every thread takes a run
__device__ __forceinline__ void block_scan(int* v, int n, int* waves) {
  const int run = (n + (int)blockDim.x - 1) / (int)blockDim.x, first = threadIdx.x * run, last = min(n, first + run);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = 0;
  for (int i = first; i < last; ++i) s += v[i];
  int inc = s;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int o = __shfl_up(inc, m, 64);
    inc += lane >= m ? o : 0;
  }
  if (lane == 63) waves[wave] = inc;
  __syncthreads();
  int base = inc - s;
  for (int i = 0; i < wave; ++i) base += waves[i];
  for (int i = first; i < last; ++i) {
    const int t = v[i];
    v[i] = base;
    base += t;
  }
  __syncthreads();
}

// one workgroup for all: a wave has one block
__global__ void __launch_bounds__(64 * kSmallWaves)
    k_group_small(const int32_t* __restrict__ index, int n, int n_groups, int bits, int32_t* __restrict__ ptr,
                  int32_t* __restrict__ rows) {
  extern __shared__ int lds[];             // [waves][n_groups + 1], [n_groups + 1]
  __shared__ int sums[kSmallWaves];
  const int G = n_groups + 1, wave = threadIdx.x >> 6, threads = blockDim.x, waves = threads >> 6;
  int* total = lds + waves * G;
  const int first = wave * kBlock;
  Block block;
  block.load(index, first, n, n_groups, bits);
  for (int i = threadIdx.x; i < waves * G; i += threads) lds[i] = 0;
  __syncthreads();
  block.count(n_groups, lds + wave * G);
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += threads) {
    int s = 0;
    for (int w = 0; w < waves; ++w) {
      const int t = lds[w * G + g];
      lds[w * G + g] = s;
      s += t;
    }
    total[g] = s;
  }
  __syncthreads();
  block_scan(total, G, sums);
  for (int w = 0; w < waves; ++w)
    for (int g = threadIdx.x; g < G; g += threads) lds[w * G + g] += total[g];
  for (int g = threadIdx.x; g < G; g += threads) ptr[g] = total[g];
  __syncthreads();
  block.place(first, n_groups, lds + wave * G, rows);
}

// counts [n_groups + 1][units]: a wave is a unit of `run` entries
__global__ void __launch_bounds__(kThreads)
    k_group_count(const int32_t* __restrict__ index, int64_t n, int n_groups, int bits, int run, int units,
                  int32_t* __restrict__ counts) {
  extern __shared__ int lds[];             // [4][n_groups + 1]
  const int G = n_groups + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int unit = blockIdx.x * (kThreads / 64) + wave;
  int* cnt = lds + wave * G;
  for (int g = lane; g < G; g += 64) cnt[g] = 0;
  wave_order();
  if (unit >= units) return;
  const int64_t first = (int64_t)unit * run;
  const int64_t end = min(n, first + run);
  for (int64_t i = first; i < end; i += kBlock) {
    Block block;
    block.load(index, i, end, n_groups, bits);
    block.count(n_groups, cnt);
  }
  for (int g = lane; g < G; g += 64) counts[(int64_t)g * units + unit] = cnt[g];
}

// a workgroup per group: its counts become the entries of the group in the units before
__global__ void __launch_bounds__(kThreads)
    k_group_scan(int32_t* counts, int units, int32_t* total) {
  __shared__ int waves[kThreads / 64];
  int32_t* v = counts + (int64_t)blockIdx.x * units;
  int base = 0;
  for (int i0 = 0; i0 < units; i0 += kThreads) {
    const int i = i0 + threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = i < units ? v[i] : 0;
    int inc = s;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(inc, m, 64);
      inc += lane >= m ? o : 0;
    }
    __syncthreads();
    if (lane == 63) waves[wave] = inc;
    __syncthreads();
    int before = base;
    for (int w = 0; w < kThreads / 64; ++w) {
      before += w < wave ? waves[w] : 0;
      base += waves[w];
    }
    if (i < units) v[i] = before + inc - s;
  }
  if (threadIdx.x == 0) total[blockIdx.x] = base;
}

__global__ void __launch_bounds__(kThreads)
    k_group_place(const int32_t* __restrict__ index, int64_t n, int n_groups, int bits, int run, int units,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ total, int32_t* __restrict__ ptr,
                  int32_t* __restrict__ rows) {
  extern __shared__ int lds[];             // [4][n_groups + 1], [n_groups + 1]
  __shared__ int waves[kThreads / 64];
  const int G = n_groups + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int unit = blockIdx.x * (kThreads / 64) + wave;
  int* start = lds + (kThreads / 64) * G;
  for (int g = threadIdx.x; g < G; g += kThreads) start[g] = total[g];
  __syncthreads();
  block_scan(start, G, waves);
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < G; g += kThreads) ptr[g] = start[g];
  if (unit >= units) return;
  int* at = lds + wave * G;
  for (int g = lane; g < G; g += 64) at[g] = start[g] + counts[(int64_t)g * units + unit];
  wave_order();
  const int64_t first = (int64_t)unit * run;
  const int64_t end = min(n, first + run);
  for (int64_t i = first; i < end; i += kBlock) {
    Block block;
    block.load(index, i, end, n_groups, bits);
    block.place(i, n_groups, at, rows);
  }
}

// entries of a unit: whole blocks, at most 2,048 units (they are scanned group by group)
int unit_run(int64_t n) { return (int)((n / 2048 + kBlock) / kBlock * kBlock); }
// waves of the one workgroup, whose counters fit 64 KB of LDS (1,536 entries in one launch 5.5 us, in three 10.5; 8,192 in
// 64 groups 11.4 and 14)
int small_waves(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(kSmallWaves + 1, (n + kBlock - 1) / kBlock)); }
size_t small_lds(int64_t n, int n_groups) { return (small_waves(n) + 1) * (size_t)(n_groups + 1) * sizeof(int); }
bool is_small(int64_t n, int n_groups) { return small_waves(n) <= kSmallWaves && small_lds(n, n_groups) <= 65536 - 256; }
int unit_count(int64_t n) { return (int)((n + unit_run(n) - 1) / unit_run(n)); }

// ---- sums over a row's choices ------------------------------------------------------------
// Threads of a workgroup: `lanes` along the columns, the rest along the rows.
int combine_lanes(int n_cols, int per) {
  int lanes = 1;
  while (lanes < kThreads && lanes * per < n_cols) lanes <<= 1;
  return lanes;
}

// Y: type of y
template <typename T, typename Y>
__global__ void __launch_bounds__(kThreads)
    k_combine_fwd(CombineArgs a, int lanes) {
  constexpr int N = Chunk<T>::kN;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  if (row >= a.n_rows) return;
  // unsigned: a row may be so long that the place behind it passes 2^31
  for (uint32_t c = threadIdx.x % lanes * N; c < (uint32_t)a.n_cols; c += lanes * N) {
    const int left = a.n_cols - (int)c;
    float s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
#pragma unroll 2
    for (int j = 0; j < a.k; ++j) {
      const int64_t slot = row * a.k + j;
      const float w = a.weight ? a.weight[slot] : 1.f;
      float v[N];
#pragma unroll
      for (int i = 0; i < N; i += Chunk<Y>::kN) load_chunk((const Y*)a.y + slot * a.n_cols + c + i, left - i, v + i);
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = fmaf(w, v[i], s[i]);
    }
    store_chunk((T*)a.out + row * a.n_cols + c, left, s);
  }
}

// `lanes` (at most a wave) threads a choice
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_combine_bwd(CombineArgs a, int lanes) {
  constexpr int N = Chunk<T>::kN;
  const int64_t slot = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  if (slot >= a.n_rows * a.k) return;
  const int64_t row = slot / a.k;
  const float w = a.weight[slot];
  float s = 0.f;
  for (uint32_t c = threadIdx.x % lanes * N; c < (uint32_t)a.n_cols; c += lanes * N) {
    const int left = a.n_cols - (int)c;
    float g[N], v[N];
    load_chunk((const T*)a.go + row * a.n_cols + c, left, g);
    load_chunk((const T*)a.y + slot * a.n_cols + c, left, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s = fmaf(g[i], v[i], s);
      g[i] *= w;
    }
    store_chunk((T*)a.gy + slot * a.n_cols + c, left, g);
  }
  s = lanes_sum(s, lanes);
  if (threadIdx.x % lanes == 0) a.grad_weight[slot] = s;
}

}  // namespace

hipError_t route_forward(const RouteArgs& a) {
  return pick_route(a, [&](auto t, auto vpt, int lanes, dim3 grid) {
    hipLaunchKernelGGL((k_route_fwd<decltype(t), vpt()>), grid, dim3(kThreads), 0, a.stream, a, lanes);
    return hipGetLastError();
  });
}

hipError_t route_backward(const RouteArgs& a) {
  return pick_route(a, [&](auto t, auto vpt, int lanes, dim3 grid) {
    hipLaunchKernelGGL((k_route_bwd<decltype(t), vpt()>), grid, dim3(kThreads), 0, a.stream, a, lanes);
    return hipGetLastError();
  });
}

size_t group_workspace_bytes(int64_t n, int n_groups) {
  return is_small(n, n_groups) ? 0 : ((size_t)unit_count(n) + 1) * (n_groups + 1) * sizeof(int32_t);
}

hipError_t group_rows(const int32_t* index, int64_t n, int n_groups, int32_t* ptr, int32_t* rows, void* ws, hipStream_t st) {
  const int G = n_groups + 1;
  int bits = 1;
  while ((1 << bits) < n_groups + 2) ++bits;
  if (is_small(n, n_groups)) {
    hipLaunchKernelGGL(k_group_small, dim3(1), dim3(64 * small_waves(n)), small_lds(n, n_groups), st, index, (int)n, n_groups, bits, ptr, rows);
    return hipGetLastError();
  }
  const int run = unit_run(n), units = unit_count(n);
  const dim3 grid((units + kThreads / 64 - 1) / (kThreads / 64));
  int32_t *counts = static_cast<int32_t*>(ws), *total = counts + (size_t)units * G;
  const size_t lds = (kThreads / 64) * (size_t)G * sizeof(int);
  hipLaunchKernelGGL(k_group_count, grid, dim3(kThreads), lds, st, index, n, n_groups, bits, run, units, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_group_scan, dim3(G), dim3(kThreads), 0, st, counts, units, total);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(k_group_place, grid, dim3(kThreads), lds + G * sizeof(int), st, index, n, n_groups, bits, run, units, counts,
                     total, ptr, rows);
  return hipGetLastError();
}

hipError_t combine_forward(const CombineArgs& a) {
  const auto go = [&](auto t, auto y) {
    const int lanes = combine_lanes(a.n_cols, Chunk<decltype(t)>::kN);
    const int64_t blocks = (a.n_rows + kThreads / lanes - 1) / (kThreads / lanes);
    if (blocks > 0xffffffffLL / kThreads) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_combine_fwd<decltype(t), decltype(y)>), dim3((unsigned)blocks), dim3(kThreads), 0, a.stream, a, lanes);
    return hipGetLastError();
  };
  return a.dtype == TP_F32 ? go(float(), float()) : a.wide ? go(bf16_t(), float()) : go(bf16_t(), bf16_t());
}

hipError_t combine_backward(const CombineArgs& a) {
  const auto go = [&](auto t) {
    const int lanes = std::min(64, combine_lanes(a.n_cols, Chunk<decltype(t)>::kN));
    const int64_t blocks = (a.n_rows * a.k + kThreads / lanes - 1) / (kThreads / lanes);
    if (blocks > 0xffffffffLL / kThreads) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_combine_bwd<decltype(t)>), dim3((unsigned)blocks), dim3(kThreads), 0, a.stream, a, lanes);
    return hipGetLastError();
  };
  return a.dtype == TP_F32 ? go(float()) : go(bf16_t());
}

}  // namespace tpc
