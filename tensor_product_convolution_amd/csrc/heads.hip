// Norm of queries and keys over each head, with the rotation by position, in one pass.
//
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r gamma
//   t = sum_a pos_a freq_ia;  (a, b) -> (a cos t - b sin t, a sin t + b cos t)  for pair i of y
// and backward, with h the upstream gradient rotated back:
//   grad_gamma = sum_rows h x r;  s = h gamma;  grad_x = r (s - x r mean(s x r))
//   grad t_i = sum_heads (h_b a - h_a b);  grad_pos_a = sum_i grad t_i freq_ia
//
// Bound by HBM: q and k are read once and written once.  A few threads hold a head, each
// the two values of up to 4 (float32) or 8 (bfloat16) pairs, so that pairs need no exchange in
// either layout.  The angles of a block of rows are taken once, into LDS, and
// serve all heads: turns in 64 bits, so that far positions keep their angle.
// 100,000 rows of 16 + 4 heads of 64, 24 pairs, bfloat16: 115 us (512 MB, 4.5 TB/s; a large copy reaches 5.1);
// float32 204 (5.0 TB/s).  1,536 rows of 8 + 8 heads of 32: 5 us, most of it the launch.
#include <algorithm>

#include "internal.hpp"
#include "rows.hpp"

namespace tpc {
namespace {

constexpr int kThreads = 256;
constexpr int kTrig = 2048;                // angles that a workgroup holds
constexpr int kMaxAxes = 3;

// The pairs of a thread.  A head is cut into chunks of kN pairs: first those of the rotated
// part, then those of the rest, whose pairs turn by nothing.  A chunk is two runs of up to kN
// values: its pairs' first and second values (half layout), or adjacent pairs one after the
// other (interleaved; the rest always).
template <typename T, bool INTER>
struct Chunks {
  static constexpr int N = Chunk<T>::kN;
  int at[2], left[2];                      // first element and length of the runs (may be <= 0)
  int pair;                                // first pair, -1 in the rest
  int pairs;                               // rotated pairs of the chunk
  __device__ __forceinline__ Chunks(int c, int d, int n_pairs) {
    const int turned = (n_pairs + N - 1) / N;
    pair = c < turned ? c * N : -1;
    pairs = c < turned ? min(N, n_pairs - c * N) : 0;
    if (c < turned && !INTER) {
      at[0] = c * N;
      at[1] = n_pairs + c * N;
      left[0] = left[1] = pairs;
    } else {
      const int first = c < turned ? 2 * c * N : 2 * n_pairs + 2 * (c - turned) * N;
      const int n = c < turned ? 2 * pairs : max(0, min(2 * N, d - first));
      at[0] = first;
      at[1] = first + N;
      left[0] = min(N, n);
      left[1] = n - N;
    }
  }
  // value j of run i, i N + j in all, is first (0) or second (1) value of a pair
  static constexpr __device__ __forceinline__ int first(int j) { return INTER ? 2 * j : j; }
  static constexpr __device__ __forceinline__ int second(int j) { return INTER ? 2 * j + 1 : N + j; }
};

// The length of a run, compared anew at each use: a mask in registers for each of its values is more than there is
// room for.
__device__ __forceinline__ int length_of(int left) {
  asm volatile("" : "+v"(left));
  return left;
}

template <typename T, bool INTER>
struct RawPairs {
  RawChunk<T> run[2];
  __device__ __forceinline__ void load(const T* head, const Chunks<T, INTER>& c) {
    run[0].load(head + c.at[0], length_of(c.left[0]));
    run[1].load(head + c.at[1], length_of(c.left[1]));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < Chunk<T>::kN; ++j) run[i].v[j] = (T)0.f;
  }
  __device__ __forceinline__ float at(int j) const { return run[j / Chunk<T>::kN].at(j % Chunk<T>::kN); }
};

template <typename T, bool INTER>
__device__ __forceinline__ void store_pairs(T* head, const Chunks<T, INTER>& c, const float* v) {
  store_chunk(head + c.at[0], length_of(c.left[0]), v);
  store_chunk(head + c.at[1], length_of(c.left[1]), v + Chunk<T>::kN);
}

// float32 values laid out like a head
template <typename T, bool INTER>
__device__ __forceinline__ void load_like(const float* w, const Chunks<T, INTER>& c, float* v) {
  constexpr int N = Chunk<T>::kN;
#pragma unroll
  for (int i = 0; i < 2 * N; i += 4) load_chunk(w + c.at[i / N] + i % N, c.left[i / N] - i % N, v + i);
}

// cos and sin of a row's angle i: the angle in 64 bits, its functions in 32.
__device__ __forceinline__ float2 turn_of(const HeadArgs& a, int64_t row, int i) {
  double t = 0.0;
  for (int x = 0; x < a.axes; ++x) {
    const int64_t at = row * a.axes + x;
    const double p = a.pos_int ? (double)static_cast<const int32_t*>(a.pos)[at] : (double)static_cast<const float*>(a.pos)[at];
    t = fma(p, a.freq[(int64_t)i * a.axes + x], t);
  }
  t *= 0.15915494309189533577;             // 1 / (2 pi)
  t -= rint(t);
  const float f = (float)t;                // off by up to 2^-26 turns, 1.6 u of a radian: turned by the rest as well
  const float rest = (float)(t - (double)f) * 6.2831853071795865f;
  float s, c;
  sincospif(2.f * f, &s, &c);
  return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// The angles of a block of rows, the rows' pairs filled up to whole chunks with pairs that do not turn.
template <typename T>
struct Angles {
  static constexpr int N = Chunk<T>::kN;
  float2* cs;                              // [kTrig]
  int pitch, at;                           // of a row; this thread's chunk in row r: at + r pitch, where it turns
  __device__ __forceinline__ Angles(const HeadArgs& a, float2* cs, int pair) : cs(cs) {
    pitch = (a.pairs + N - 1) / N * N;
    at = pair;
  }
  __device__ __forceinline__ void fill(const HeadArgs& a, int64_t row0, int rows) const {
    for (int i = threadIdx.x; i < rows * pitch; i += kThreads) {
      const int row = i / pitch, pair = i - row * pitch;
      cs[i] = pair < a.pairs ? turn_of(a, row0 + row, pair) : make_float2(1.f, 0.f);
    }
  }
  __device__ __forceinline__ void get(int row, float2* o) const {
    const float4* from = reinterpret_cast<const float4*>(cs + at + row * pitch);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const float4 t = from[j / 2];
      o[j] = make_float2(t.x, t.y);
      o[j + 1] = make_float2(t.z, t.w);
    }
  }
};

// the value of another lane of the row of 16
template <int CTRL>
__device__ __forceinline__ float lane_of(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// sum over the 2^lg neighbouring threads of a head, in a fixed order: with the neighbour, the pair next to it,
// then the mirror image in 8 and in 16 lanes, whose parts hold one sum each by then
__device__ __forceinline__ float head_sum(float v, int lg) {
  if (lg > 0) v += lane_of<0xb1>(v);
  if (lg > 1) v += lane_of<0x4e>(v);
  if (lg > 2) v += lane_of<0x141>(v);
  if (lg > 3) v += lane_of<0x140>(v);
  for (int m = 16; m < 1 << lg; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// Which head of which row a thread has in turn `it` of a block of rows
struct Item {
  int row, head;
  __device__ __forceinline__ Item(const HeadArgs& a, int it) {
    const int i = (it * kThreads + (int)threadIdx.x) >> a.lg;
    row = i / (a.hq + a.hk);
    head = i - row * (a.hq + a.hk);
  }
};

template <typename T, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads)
    k_heads_fwd(HeadArgs a) {
  constexpr int V = 2 * Chunk<T>::kN;
  __shared__ __attribute__((aligned(16))) float2 cs[kTrig];
  const Chunks<T, INTER> c((int)threadIdx.x & ((1 << a.lg) - 1), a.d, a.pairs);
  const Angles<T> angles(a, cs, c.pair);
  const float part = 1.f / (float)a.d;
  float g[2][V];
  if (NORM) {
    load_like<T, INTER>(a.gamma_q, c, g[0]);
    load_like<T, INTER>(a.gamma_k, c, g[1]);
  }
  const int64_t row0 = (int64_t)blockIdx.x * a.rows;
  const int rows = (int)min((int64_t)a.rows, a.n_rows - row0), heads = a.hq + a.hk;
  const int turns = (rows * heads * (1 << a.lg) + kThreads - 1) / kThreads;
  const auto source = [&](const Item& it) {
    return it.head < a.hq ? (const T*)a.q + (row0 + it.row) * a.q_stride + it.head * a.d
                          : (const T*)a.k + (row0 + it.row) * a.k_stride + (it.head - a.hq) * a.d;
  };
  RawPairs<T, INTER> x;
  {                                        // in flight while the angles are taken
    const Item it(a, 0);
    if (it.row < rows)
      x.load(source(it), c);
    else
      x.clear();
  }
  angles.fill(a, row0, rows);
  __syncthreads();
  for (int n = 0; n < turns; ++n) {
    const Item it(a, n), next(a, n + 1);
    const bool has = it.row < rows;        // the same for all threads of a head
    float v[V];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = x.at(j);
      s += v[j] * v[j];
    }
    if (next.row < rows)
      x.load(source(next), c);
    else
      x.clear();
    if (NORM) {
      const float r = 1.f / sqrtf(head_sum(s, a.lg) * part + a.eps);
      const bool key = it.head >= a.hq;
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = v[j] * r * (key ? g[1][j] : g[0][j]);
    }
    if (!has) continue;
    if (c.pair >= 0) {                     // no turn by nothing for the rest: it would pass on what is not finite
      float2 t[V / 2];
      angles.get(it.row, t);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float p = v[c.first(j)], q = v[c.second(j)];
        v[c.first(j)] = p * t[j].x - q * t[j].y;
        v[c.second(j)] = p * t[j].y + q * t[j].x;
      }
    }
    store_pairs(it.head < a.hq ? (T*)a.q_out + (row0 + it.row) * a.qo_stride + it.head * a.d
                               : (T*)a.k_out + (row0 + it.row) * a.ko_stride + (it.head - a.hq) * a.d,
                c, v);
  }
}

// One pass over blocks of rows, first their queries, then their keys; a workgroup's part of the weight
// gradients stays in registers until its last block.  part [gridDim.x][2][d]; a single workgroup
// writes the gradients itself.  Products and sums are written as the fused operations they are, so that
// the variants round alike.  Weights and frequencies are read from LDS, by chunk: in registers they
// leave two waves a SIMD.
// bfloat16 is bound by vector instructions and loads together, float32 by HBM: 100,000 rows of 16 + 4 heads of 64 with
// the positions' gradient 191 us (768 MB, 4.0 TB/s; half the time is vector issue), without it 163, float32 299
// (5.1 TB/s); 30,000 rows of 16 + 16 heads of 128 176 and 150 us; 1,536 of 8 + 8 of 32 9 us and 4 for the join.  Masks of `has` for each value instead of zeroed
// loads, angles read pair by pair under a condition, and sums through LDS took 292.
template <typename T, bool INTER, bool NORM, bool POS>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : 3)
    k_heads_bwd(HeadBwdArgs b) {
  const HeadArgs& a = b.f;
  constexpr int V = 2 * Chunk<T>::kN;
  __shared__ __attribute__((aligned(16))) float2 cs[kTrig];     // at the end the waves' weight gradients
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int n_chunks = 1 << a.lg, lane_c = (int)threadIdx.x & (n_chunks - 1), heads = a.hq + a.hk, per_axis = a.rows * heads;
  float *gl = lds, *fl = gl + (NORM ? 2 * n_chunks * V : 0), *sums = fl + (POS ? kMaxAxes * n_chunks * V / 2 : 0);
  const Chunks<T, INTER> c(lane_c, a.d, a.pairs);
  const Angles<T> angles(a, cs, c.pair);
  const float part = 1.f / (float)a.d;
  if (NORM && (int)threadIdx.x < 2 * n_chunks) {
    float v[V];
    load_like<T, INTER>((int)threadIdx.x < n_chunks ? a.gamma_q : a.gamma_k, c, v);
#pragma unroll
    for (int j = 0; j < V; ++j) gl[threadIdx.x * V + j] = v[j];
  }
  if (POS) {                               // [axis][pair]: chunk c of a head has pairs from c V / 2 on
    const int most = n_chunks * V / 2;
    for (int i = threadIdx.x; i < kMaxAxes * most; i += kThreads) {
      const int x = i / most, pair = i - x * most;
      fl[i] = x < a.axes && pair < a.pairs ? (float)a.freq[(int64_t)pair * a.axes + x] : 0.f;
    }
  }
  float gg[2][V];
#pragma unroll
  for (int j = 0; j < V; ++j) gg[0][j] = gg[1][j] = 0.f;
  const int step = kThreads >> a.lg, first = (int)threadIdx.x >> a.lg;
  RawPairs<T, INTER> x, u;
  const auto fetch = [&](auto key, int64_t row, int64_t end, int head) {
    if (row >= end) {                      // zeros where there is no head
      x.clear();
      u.clear();
      return;
    }
    x.load((const T*)(key() ? a.k : a.q) + row * (key() ? a.k_stride : a.q_stride) + head * a.d, c);
    u.load((const T*)(key() ? b.gk_up : b.gq_up) + row * (key() ? b.gk_up_stride : b.gq_up_stride) + head * a.d, c);
  };
  // what a thread begins the queries or keys of a block with
  const auto begin = [&](auto key, int64_t row0) {
    const int H = key() ? a.hk : a.hq, row = first / H;
    fetch(key, row0 + row, min(row0 + a.rows, a.n_rows), first - row * H);
  };
  // the queries (KEY 0) or keys of a block of rows; the loads of what comes next are in flight throughout
  const auto side = [&](auto key, int64_t row0, int rows) {
    constexpr int KEY = key();
    const int H = KEY ? a.hk : a.hq, before = KEY ? a.hq : 0;
    const int step_row = step / H, step_head = step - step_row * H;
    T* out = (T*)(KEY ? b.gk : b.gq);
    const int64_t os = KEY ? b.gk_stride : b.gq_stride;
    int row = first / H, head = first - row * H;
    if (KEY == 0) {
      angles.fill(a, row0, rows);
      __syncthreads();
    }
    for (int n = (rows * H + step - 1) / step; n > 0; --n) {
      const bool has = row < rows;         // the same for all threads of a head
      float v[V], h[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j] = x.at(j);
        h[j] = u.at(j);
      }
      const int r0 = row, h0 = head;
      row += step_row;
      head += step_head;
      if (head >= H) {
        head -= H;
        ++row;
      }
      if (n > 1) {
        fetch(key, row0 + row, row0 + rows, head);
      } else if (KEY == 0) {
        begin(std::integral_constant<int, 1>(), row0);
      } else {
        begin(std::integral_constant<int, 0>(), row0 + (int64_t)gridDim.x * a.rows);
      }
      if (c.pair >= 0) {
        float2 t[V / 2];
        angles.get(has ? r0 : 0, t);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float p = h[c.first(j)], q = h[c.second(j)];
          h[c.first(j)] = fmaf(p, t[j].x, q * t[j].y);
          h[c.second(j)] = fmaf(q, t[j].x, -p * t[j].y);
        }
      }
      const float* g = gl + (KEY * n_chunks + lane_c) * V;
      float r = 1.f, m = 0.f;
      if (NORM) {
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          s1 = fmaf(v[j], v[j], s1);
          s2 = fmaf(h[j] * g[j], v[j], s2);
        }
        r = 1.f / sqrtf(head_sum(s1, a.lg) * part + a.eps);
        r = has ? r : 0.f;                 // eps may be 0, and zeros would be no numbers then
        m = head_sum(s2, a.lg) * r * part;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= r;
      }
      if (POS) {                           // of the angles, from the pairs before they are turned
        float w[kMaxAxes] = {0.f, 0.f, 0.f};
        if (c.pair >= 0) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const int p = c.first(j), q = c.second(j);
            const float gt = NORM ? h[q] * (v[p] * g[p]) - h[p] * (v[q] * g[q]) : h[q] * v[p] - h[p] * v[q];
#pragma unroll
            for (int k = 0; k < kMaxAxes; ++k) w[k] += gt * fl[(k * n_chunks + lane_c) * (V / 2) + j];
          }
        }
#pragma unroll
        for (int k = 0; k < kMaxAxes; ++k) {
          if (k >= a.axes) break;
          const float s = head_sum(w[k], a.lg);
          if (has && lane_c == 0) sums[k * per_axis + r0 * heads + before + h0] = s;
        }
      }
      if (NORM) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          gg[KEY][j] = fmaf(h[j], v[j], gg[KEY][j]);         // both are zero where there is no head
          h[j] = r * fmaf(-v[j], m, h[j] * g[j]);
        }
      }
      if (has) store_pairs(out + (row0 + r0) * os + h0 * a.d, c, h);
    }
  };
  begin(std::integral_constant<int, 0>(), (int64_t)blockIdx.x * a.rows);
  for (int64_t row0 = (int64_t)blockIdx.x * a.rows; row0 < a.n_rows; row0 += (int64_t)gridDim.x * a.rows) {
    const int rows = (int)min((int64_t)a.rows, a.n_rows - row0);
    side(std::integral_constant<int, 0>(), row0, rows);
    side(std::integral_constant<int, 1>(), row0, rows);
    __syncthreads();
    if (POS) {
      for (int i = threadIdx.x; i < rows * a.axes; i += kThreads) {
        const int row = i / a.axes, k = i - row * a.axes;
        float s = 0.f;
        for (int h = 0; h < heads; ++h) s += sums[k * per_axis + row * heads + h];
        b.grad_pos[(row0 + row) * a.axes + k] = s;
      }
      __syncthreads();
    }
  }
  if (!NORM || !b.grad_gamma_q) return;
  // over the threads that hold the same chunk: lanes of a wave, then the four waves
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, all = 2 * n_chunks * V;
  float* mine = reinterpret_cast<float*>(cs);
  static_assert(sizeof(cs) >= 4 * 2 * 2 * kHeadsMaxDim * sizeof(float));
  __syncthreads();
  const auto join = [&](auto&& other) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      gg[0][j] += other(gg[0][j]);
      gg[1][j] += other(gg[1][j]);
    }
  };
  // turned by 1, 2, 4, 8 in the row of 16 lanes, then the rows
  if (n_chunks <= 1) join([](float v) { return lane_of<0x121>(v); });
  if (n_chunks <= 2) join([](float v) { return lane_of<0x122>(v); });
  if (n_chunks <= 4) join([](float v) { return lane_of<0x124>(v); });
  if (n_chunks <= 8) join([](float v) { return lane_of<0x128>(v); });
  if (n_chunks <= 16) join([](float v) { return __shfl_xor(v, 16, 64); });
  if (n_chunks <= 32) join([](float v) { return __shfl_xor(v, 32, 64); });
  if (lane < n_chunks) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) mine[wave * all + (i * n_chunks + lane_c) * V + j] = gg[i][j];
  }
  __syncthreads();
  float* out[2] = {b.grad_gamma_q, b.grad_gamma_k};
  if (gridDim.x > 1) {
    out[0] = b.part + (size_t)blockIdx.x * 2 * a.d;
    out[1] = out[0] + a.d;
  }
  for (int i = threadIdx.x; i < all; i += kThreads) {
    const int side_of = i / (n_chunks * V), j = i % V;
    const Chunks<T, INTER> o(i / V % n_chunks, a.d, a.pairs);
    const int run = j / Chunk<T>::kN, in = j % Chunk<T>::kN;
    if (in < (run ? o.left[1] : o.left[0]))
      out[side_of][(run ? o.at[1] : o.at[0]) + in] = (mine[i] + mine[all + i]) + (mine[2 * all + i] + mine[3 * all + i]);
  }
}

// Weight gradients from the workgroups' parts [n][2][d], a wave per value, in a fixed order: 5 us for 768 parts of
// 2 x 64.
__global__ void __launch_bounds__(kThreads)
    k_heads_join(const float* __restrict__ part, int n, int d, float* __restrict__ gq, float* __restrict__ gk) {
  const int col = (blockIdx.x * kThreads + threadIdx.x) >> 6, lane = threadIdx.x & 63;
  if (col >= 2 * d) return;
  float s = 0.f;
#pragma unroll 4
  for (int i = lane; i < n; i += 64) s += part[(size_t)i * 2 * d + col];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m, 64);
  if (lane == 0) (col < d ? gq[col] : gk[col - d]) = s;
}

// Workgroups that walk the rows of the backward: as many as the chip holds at once (100,000 rows of 8 + 8 heads of 32 with
// 512, 768, 1,024 of them: bfloat16 107, 90, 114 us, float32 158, 132, 129).
constexpr int kBwdBlocks = 768, kBwdBlocksF32 = 1024;

// Workgroups that few rows are spread over (1,536 rows of 8 + 8 heads of 32, forward over 128, 1,024, 2,048: float32 5.5,
// 4.2, 4.7 us).  The backward's each write a part of the weight gradients (over 256 and 1,024: 12.9 and 16.5).
constexpr int kFwdFill = 1024, kBwdFill = 256;

// Threads per head (their binary logarithm) and rows per workgroup: enough items for a few
// turns of the workgroup, fewer where the rows would not fill the chip.
void shape_of(int dtype, HeadArgs& a, int64_t blocks) {
  const int n = dtype == TP_F32 ? Chunk<float>::kN : Chunk<bf16_t>::kN;
  const int chunks = (a.pairs + n - 1) / n + (a.d - 2 * a.pairs + 2 * n - 1) / (2 * n);
  a.lg = 0;
  while ((1 << a.lg) < chunks) ++a.lg;
  const int64_t most = std::max(1, std::min(kTrig / std::max(1, (a.pairs + n - 1) / n * n), (4 * kThreads) / ((a.hq + a.hk) << a.lg)));
  a.rows = (int)std::max<int64_t>(1, std::min<int64_t>({most, 64, (a.n_rows + blocks - 1) / blocks}));
}

int64_t bwd_blocks(int dtype, const HeadArgs& a) {
  return std::max<int64_t>(1, std::min<int64_t>(dtype == TP_F32 ? kBwdBlocksF32 : kBwdBlocks, (a.n_rows + a.rows - 1) / a.rows));
}

template <typename F>
hipError_t pick(int dtype, bool interleaved, bool norm, F&& f) {
  const auto two = [&](auto t, auto inter) { return norm ? f(t, inter, std::true_type()) : f(t, inter, std::false_type()); };
  const auto one = [&](auto t) { return interleaved ? two(t, std::true_type()) : two(t, std::false_type()); };
  return dtype == TP_F32 ? one(float()) : one(bf16_t());
}

}  // namespace

size_t heads_workspace_bytes(int dtype, HeadArgs a) {
  shape_of(dtype, a, kBwdFill);
  const int64_t n = bwd_blocks(dtype, a);
  return n == 1 ? 0 : (size_t)n * 2 * a.d * sizeof(float);
}

hipError_t heads_forward(int dtype, HeadArgs a) {
  shape_of(dtype, a, kFwdFill);
  const int64_t blocks = (a.n_rows + a.rows - 1) / a.rows;
  if (blocks > 0xffffffffLL / kThreads) return hipErrorInvalidConfiguration;
  return pick(dtype, a.interleaved, a.gamma_q != nullptr, [&](auto t, auto inter, auto norm) {
    hipLaunchKernelGGL((k_heads_fwd<decltype(t), inter(), norm()>), dim3((unsigned)blocks), dim3(kThreads), 0, a.stream, a);
    return hipGetLastError();
  });
}

hipError_t heads_backward(int dtype, HeadBwdArgs b) {
  HeadArgs& a = b.f;
  shape_of(dtype, a, kBwdFill);
  const int n = (int)bwd_blocks(dtype, a);
  hipError_t e = pick(dtype, a.interleaved, a.gamma_q != nullptr, [&](auto t, auto inter, auto norm) {
    constexpr int V = 2 * Chunk<decltype(t)>::kN;
    const size_t chunks = (size_t)V << a.lg;
    const size_t floats = (norm() ? 2 * chunks : 0) + (b.grad_pos ? kMaxAxes * (chunks / 2 + (size_t)a.rows * (a.hq + a.hk)) : 0);
    if (b.grad_pos)
      hipLaunchKernelGGL((k_heads_bwd<decltype(t), inter(), norm(), true>), dim3(n), dim3(kThreads), floats * sizeof(float), a.stream, b);
    else
      hipLaunchKernelGGL((k_heads_bwd<decltype(t), inter(), norm(), false>), dim3(n), dim3(kThreads), floats * sizeof(float), a.stream, b);
    return hipGetLastError();
  });
  if (e != hipSuccess || n == 1 || !b.grad_gamma_q) return e;
  hipLaunchKernelGGL(k_heads_join, dim3((2 * a.d + 3) / 4), dim3(kThreads), 0, a.stream, b.part, n, a.d, b.grad_gamma_q,
                     b.grad_gamma_k);
  return hipGetLastError();
}

}  // namespace tpc
