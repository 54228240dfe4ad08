// AdamW over many tensors in a few launches, states in 32 or 8 bits.
//
//   t = t + 1;  G = g min(1, max_norm / |g|)
//   m = b1 m + (1 - b1) G,  v = b2 v + (1 - b2) G^2
//   p = p (1 - lr decay) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by HBM: parameters, gradients and states are read and written once, the gradients
// twice where their norm limits the step.  The tensors are cut into chunks of 2,048 values, one
// a workgroup; a table on the device says whose chunk it is, and the gradients' addresses, which
// change from step to step, come with the launch.  64 million values, bfloat16 gradients and copies, 8-bit states: 40 us for
// the norm and 230 for the step (16 bytes a value, 4.5 TB/s, vector instructions for 0.8 of it); 300,000 values in
// 40 tensors, 32-bit states: 8 and 4 us.
//
// 8-bit states: 256 values share a float32 unit, the largest of them over 1.875 (2^127 at most: all codes have a value), and each is a
// code of unit times a small float: eight codes an octave, the lowest octave linear down to zero.
// First moments have a sign and 127 codes (2^17 between the smallest and largest), second moments
// 255 (2^33).  A moment moves by a tenth or a thousandth of its distance a step, far below half
// a code, and rounding to nearest would hold it where it is: codes are rounded up or down at random, by
// 16 bits each of the generator's word for the value (word i % 4 of block i / 4, key seed, offset
// t), so that the mean is right.  A gradient that is not finite (where no norm is taken) leaves zeros: nothing of it may
// reach the 255 others through the unit.  A second moment that is not zero keeps code 1 at least:
// the update would be divided by nothing.  Which code is taken is decided in 64 bits.
#include <algorithm>

#include "internal.hpp"
#include "rows.hpp"

namespace tpc {
namespace {

constexpr int kThreads = 256, kValues = 8, kChunk = kThreads * kValues;
constexpr int kTensors = 256;              // gradients' addresses of a launch: 2 KB of arguments
constexpr int kNormBlocks = 1024;          // workgroups of a launch that sums squares
constexpr int kFused = 256;                // so many join their sums themselves

struct Entry {
  float* p;
  bf16_t* copy;
  int64_t offset, n;                       // first state value (a multiple of kAdamBlock), values
  float decay;
  int32_t pad;
};
struct Piece {
  int32_t tensor, chunk;
};
struct Scalars {
  int64_t step;
  double factor;                           // of the gradients
  float c1, c2, lr;                        // 1 / (1 - beta^t)
  int32_t skip;
  uint32_t done;                           // workgroups that have summed their squares
};
static_assert(sizeof(Scalars) <= 64);

struct Grads {
  const void* g[kTensors];
};

// what the kernels read of the optimiser
struct Run {
  const Entry* entries;
  const Piece* pieces;
  int first_tensor, n_pieces;
  Scalars* s;
};

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// What a step starts from besides its gradients
struct Begin {
  double beta1, beta2, max_norm, lr;
  const float* lr_at;
  float* norm;
};

// The step's number and what follows from it and the norm.  A norm that is not finite skips the step.
__device__ __forceinline__ void begin(Scalars* s, const Begin& b, double squares) {
  const bool limited = b.max_norm > 0.0;
  const double size = sqrt(squares);
  if (b.norm) *b.norm = (float)size;
  const bool skip = limited && !(size < INFINITY);
  s->skip = skip;
  if (skip) return;
  const int64_t t = s->step + 1;
  s->step = t;
  s->factor = limited && size > b.max_norm ? b.max_norm / size : 1.0;
  s->c1 = (float)(1.0 / (1.0 - pow(b.beta1, (double)t)));
  s->c2 = (float)(1.0 / (1.0 - pow(b.beta2, (double)t)));
  s->lr = b.lr_at ? *b.lr_at : (float)b.lr;
}

__device__ __forceinline__ double block_sum(double x, double* waves) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = x;
  __syncthreads();
  return (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

// the workgroups' sums, joined in their order, and the step's beginning
__device__ __forceinline__ void join(Scalars* s, const double* part, int parts, const Begin& b, double* waves) {
  double x = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads)
    x += __hip_atomic_load(part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  x = block_sum(x, waves);
  if (threadIdx.x == 0) begin(s, b, x);
}

__global__ void __launch_bounds__(kThreads)
    k_adam_begin(Scalars* s, const double* part, int parts, Begin b) {
  __shared__ double waves[kThreads / 64];
  join(s, part, parts, b, waves);
}

// Squares of the gradients, summed in 64 bits: part[first + blockIdx.x].  Where `parts` is given the
// last of so many workgroups to finish joins them: a launch less (300,000 values in 40 tensors: a step 22
// against 25.5 us).  1,024 workgroups that count themselves on one word take 15 us to, so many leave it
// to a launch of its own.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_adam_norm(Run r, Grads grads, double* part, int first, int parts, Begin b) {
  constexpr int N = Chunk<T>::kN;
  __shared__ double waves[kThreads / 64];
  __shared__ bool last;
  double s = 0.0;
  // four chunks at a time: their places, then their values, each loaded together
  constexpr int kAtOnce = 4, kLoads = kValues / N;
  for (int i0 = blockIdx.x; i0 < r.n_pieces; i0 += gridDim.x * kAtOnce) {
    RawChunk<T> v[kAtOnce][kLoads];
    Piece q[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) q[u] = r.pieces[min(i0 + u * (int)gridDim.x, r.n_pieces - 1)];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t n = i0 + u * (int)gridDim.x < r.n_pieces ? r.entries[q[u].tensor].n : 0;
      const T* g = (const T*)grads.g[q[u].tensor - r.first_tensor];
#pragma unroll
      for (int c = 0; c < kLoads; ++c) {
        const int64_t at = (int64_t)q[u].chunk * kChunk + (c * kThreads + threadIdx.x) * N;
        v[u][c].load(g + at, (int)max((int64_t)0, min(n - at, (int64_t)N)));
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int c = 0; c < kLoads; ++c)
#pragma unroll
        for (int j = 0; j < N; ++j) s = fma((double)v[u][c].at(j), (double)v[u][c].at(j), s);
  }
  s = block_sum(s, waves);
  if (threadIdx.x == 0) {
    // The sum goes to memory itself, past the caches, and is there before it is counted: a release
    // would write back all that the L2 holds.
    __hip_atomic_store(part + first + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_waitcnt(0x0f70);    // vmcnt 0: stores too
    last = parts > 0 && __hip_atomic_fetch_add(&r.s->done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)parts - 1;
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) r.s->done = 0;
  join(r.s, part, parts, b, waves);
}

struct Rates {
  double beta1, beta2, rest1, rest2;       // rest = 1 - beta
  float eps;
};

// a parameter's step.  Square root and reciprocal to a unit in the last place: the step is of
// lr's size, its rounding far below the parameter's
// LOW: also where v is subnormal, which the square root's instruction need not take.
template <bool LOW>
__device__ __forceinline__ float moved(float p, float m, float v, float decay, const Scalars& s, float eps) {
  const bool low = LOW && v < 0x1p-96f;
  const float root = __builtin_amdgcn_sqrtf((low ? v * 0x1p64f : v) * s.c2), d = (low ? root * 0x1p-32f : root) + eps;
  return p * (1.f - s.lr * decay) - s.lr * (m * s.c1 * __builtin_amdgcn_rcpf(d));
}

// the same with moments of any size
__device__ __forceinline__ float moved_far(float p, double m, double v, float decay, const Scalars& s, float eps) {
  return p * (1.f - s.lr * decay) - s.lr * (float)(m * (double)s.c1 / (sqrt(v * (double)s.c2) + (double)eps));
}
// Second moments outside of these are not for moved<false>(): their roots are taken in 64 bits.  Below kLeast that
// matters only where eps is as small.
constexpr double kLeast = 0x1p-126, kMost = 0x1p100;
constexpr float kSmallEps = 0x1p-39f;

// eight values of a gradient or parameter, by the type's chunks
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t left, float* v) {
  constexpr int N = Chunk<T>::kN;
#pragma unroll
  for (int c = 0; c < kValues; c += N) load_chunk(p + c, (int)max((int64_t)0, min(left - c, (int64_t)N)), v + c);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t left, const float* v) {
  constexpr int N = Chunk<T>::kN;
#pragma unroll
  for (int c = 0; c < kValues; c += N) store_chunk(p + c, (int)max((int64_t)0, min(left - c, (int64_t)N)), v + c);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_adam32(Run r, Grads grads, float* m, float* v, Rates b) {
  const Scalars s = *r.s;
  if (s.skip) return;
  const Piece q = r.pieces[blockIdx.x];
  const Entry e = r.entries[q.tensor];
  const int64_t at = (int64_t)q.chunk * kChunk + threadIdx.x * kValues, left = e.n - at;
  if (left <= 0) return;
  float p[kValues], g[kValues], x[kValues], y[kValues];
  load8(e.p + at, left, p);
  load8((const T*)grads.g[q.tensor - r.first_tensor] + at, left, g);
  load8(m + e.offset + at, kValues, x);
  load8(v + e.offset + at, kValues, y);
  const float f = (float)s.factor, b1 = (float)b.beta1, b2 = (float)b.beta2, r1 = (float)b.rest1, r2 = (float)b.rest2;
#pragma unroll
  for (int j = 0; j < kValues; ++j) {
    const float w = g[j] * f;
    x[j] = b1 * x[j] + r1 * w;
    y[j] = b2 * y[j] + r2 * (w * w);
    p[j] = moved<true>(p[j], x[j], y[j], e.decay, s, b.eps);
  }
  store8(m + e.offset + at, kValues, x);
  store8(v + e.offset + at, kValues, y);
  store8(e.p + at, left, p);
  if (e.copy) store8(e.copy + at, left, p);
}

// A code's value over the unit: its bits as the upper bits of a float32, whose subnormals are
// the linear octave.
__device__ __forceinline__ float first_value(uint32_t c) {
  const float a = __builtin_bit_cast(float, (c & 127u) << 20) * 0x1p112f;
  return c & 128u ? -a : a;
}
__device__ __forceinline__ float second_value(uint32_t c) { return __builtin_bit_cast(float, c << 20) * 0x1p96f; }

// The code at or below a >= 0 (in units), or the next one, by u / 65,536.  Above the lowest octave
// the upper word of the double is the code with 17 more bits, and u is added behind it.  OCTAVES:
// codes of full precision are 8 .. 8 OCTAVES + 7.
template <int OCTAVES>
__device__ __forceinline__ uint32_t code_of(double a, uint32_t u) {
  constexpr uint32_t kFirst = (1023u - OCTAVES) * 8;
  constexpr double kLow = 1.0 / (double)(1ull << (OCTAVES - 1));
  const uint32_t hi = (uint32_t)(__builtin_bit_cast(uint64_t, a) >> 32);
  const uint32_t above = ((hi + 2 * u) >> 17) - kFirst;
  const uint32_t below = ((uint32_t)(a * (8.0 * 65536.0 / kLow)) + u) >> 16;
  return min(a < kLow ? below : above, 8u * OCTAVES + 7u);
}

// largest of the half wave that holds a block of states
__device__ __forceinline__ float block_max(float x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor(x, m, 64));
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_adam8(Run r, Grads grads, uint8_t* m, uint8_t* v, float* m_unit, float* v_unit, Rates b, uint32_t k0, uint32_t k1) {
  static_assert(kAdamBlock == 32 * kValues);
  const Scalars s = *r.s;
  if (s.skip) return;
  const Piece q = r.pieces[blockIdx.x];
  const Entry e = r.entries[q.tensor];
  const int64_t at = (int64_t)q.chunk * kChunk + threadIdx.x * kValues, left = e.n - at, state = e.offset + at;
  if ((at & ~(int64_t)(kAdamBlock - 1)) >= e.n) return;      // a block that is not there
  const int64_t block = state / kAdamBlock;
  float p[kValues], g[kValues];
  load8(e.p + at, left, p);
  load8((const T*)grads.g[q.tensor - r.first_tensor] + at, left, g);
  const uint2 mc = *reinterpret_cast<const uint2*>(m + state), vc = *reinterpret_cast<const uint2*>(v + state);
  const double mu = (double)m_unit[block], vu = (double)v_unit[block];
  double x[kValues], y[kValues], top_x = 0.0, top_y = 0.0;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kValues; ++j) {
    const double w = (double)g[j] * s.factor;
    const uint32_t cm = (j < 4 ? mc.x : mc.y) >> 8 * (j & 3) & 255u, cv = (j < 4 ? vc.x : vc.y) >> 8 * (j & 3) & 255u;
    x[j] = b.beta1 * ((double)first_value(cm) * mu) + b.rest1 * w;
    y[j] = b.beta2 * ((double)second_value(cv) * vu) + b.rest2 * (w * w);
    top_x = fmax(top_x, fabs(x[j]));
    top_y = fmax(top_y, y[j]);
    p[j] = moved<false>(p[j], (float)x[j], (float)y[j], e.decay, s, b.eps);
    bad |= !(fabsf(g[j]) < INFINITY);
  }
  const double least = b.eps < kSmallEps ? kLeast : 0.0;
  if (least > 0.0) {
#pragma unroll
    for (int j = 0; j < kValues; ++j) bad |= y[j] > 0.0 && y[j] < least;
  }
  if (bad || top_y >= kMost) {
    top_x = top_y = 0.0;
#pragma unroll
    for (int j = 0; j < kValues; ++j) {
      if (j < left && y[j] > 0.0 && (y[j] < least || y[j] >= kMost)) p[j] = moved_far(e.p[at + j], x[j], y[j], e.decay, s, b.eps);
      // no code stands for what is not finite, and its block's others go on
      if (!(fabsf(g[j]) < INFINITY)) x[j] = y[j] = 0.0;
      top_x = fmax(top_x, fabs(x[j]));
      top_y = fmax(top_y, y[j]);
    }
  }
  // rounding does not change which is the largest
  const float ux = fminf(block_max((float)(top_x * (1.0 / 1.875))), 0x1p127f);
  const float uy = fminf(block_max((float)(top_y * (1.0 / 1.875))), 0x1p127f);
  const double ix = ux > 0.f ? 1.0 / (double)ux : 0.0, iy = uy > 0.f ? 1.0 / (double)uy : 0.0;
  DropArgs d;
  d.k0 = k0;
  d.k1 = k1;
  d.o0 = (uint32_t)s.step;
  d.o1 = (uint32_t)(s.step >> 32);
  uint32_t om[2] = {0, 0}, ov[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4];
    philox4(d, (uint64_t)(state >> 2) + h, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double ax = fabs(x[4 * h + j]) * ix, ay = y[4 * h + j] * iy;
      uint32_t cx = code_of<15>(ax, w[j] & 0xffffu), cy = code_of<31>(ay, w[j] >> 16);
      cx |= cx && x[4 * h + j] < 0.0 ? 128u : 0u;
      cy = ay > 0.0 && cy == 0 ? 1u : cy;
      om[h] |= cx << 8 * j;
      ov[h] |= cy << 8 * j;
    }
  }
  *reinterpret_cast<uint2*>(m + state) = make_uint2(om[0], om[1]);
  *reinterpret_cast<uint2*>(v + state) = make_uint2(ov[0], ov[1]);
  if ((threadIdx.x & 31) == 0) {
    m_unit[block] = ux;
    v_unit[block] = uy;
  }
  if (left <= 0) return;
  store8(e.p + at, left, p);
  if (e.copy) store8(e.copy + at, left, p);
}

template <bool SECOND>
__global__ void __launch_bounds__(kThreads)
    k_adam_values(int64_t n, const uint8_t* __restrict__ codes, const float* __restrict__ units, float* __restrict__ out) {
  const int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kValues;
  if (at >= n) return;                     // n is a multiple of kAdamBlock
  const uint2 c = *reinterpret_cast<const uint2*>(codes + at);
  const float u = units[at / kAdamBlock];
  float o[kValues];
#pragma unroll
  for (int j = 0; j < kValues; ++j) {
    const uint32_t x = (j < 4 ? c.x : c.y) >> 8 * (j & 3) & 255u;
    o[j] = (SECOND ? second_value(x) : first_value(x)) * u;
  }
  store8(out + at, kValues, o);
}

// launches of up to kTensors tensors: f(first tensor, tensors, first chunk, chunks)
template <typename F>
hipError_t each_launch(int n_tensors, const int64_t* sizes, F&& f) {
  int64_t chunk = 0;
  for (int i = 0; i < n_tensors; i += kTensors) {
    const int n = std::min(kTensors, n_tensors - i);
    int64_t c = 0;
    for (int j = i; j < i + n; ++j) c += chunks_of(sizes[j]);
    const hipError_t e = c ? f(i, n, chunk, c) : hipSuccess;
    if (e != hipSuccess) return e;
    chunk += c;
  }
  return hipSuccess;
}

int64_t entries_bytes(int n_tensors) { return ((int64_t)n_tensors * sizeof(Entry) + 15) / 16 * 16; }

}  // namespace

int64_t adamw_table_bytes(int n_tensors, const int64_t* sizes) {
  int64_t c = 0;
  for (int i = 0; i < n_tensors; ++i) {
    c += chunks_of(sizes[i]);
    if (c > 0xffffffffLL / kThreads) return -1;    // a launch holds fewer than 2^32 threads
  }
  return entries_bytes(n_tensors) + c * (int64_t)sizeof(Piece);
}

int64_t adamw_state_size(int n_tensors, const int64_t* sizes) {
  int64_t s = 0;
  for (int i = 0; i < n_tensors; ++i) s += (sizes[i] + kAdamBlock - 1) / kAdamBlock * kAdamBlock;
  return s;
}

size_t adamw_workspace_bytes(int n_tensors, const int64_t* sizes) {
  size_t parts = 0;
  (void)each_launch(n_tensors, sizes, [&](int, int, int64_t, int64_t chunks) {
    parts += (size_t)std::min<int64_t>(kNormBlocks, chunks);
    return hipSuccess;
  });
  return parts * sizeof(double);
}

void adamw_table_fill(int n_tensors, const int64_t* sizes, void* const* params, void* const* copies, const float* decay,
                      void* table) {
  Entry* e = static_cast<Entry*>(table);
  Piece* q = reinterpret_cast<Piece*>(static_cast<char*>(table) + entries_bytes(n_tensors));
  int64_t offset = 0;
  for (int i = 0; i < n_tensors; ++i) {
    e[i] = Entry{static_cast<float*>(params[i]), static_cast<bf16_t*>(copies ? copies[i] : nullptr), offset, sizes[i],
                 decay ? decay[i] : 0.f, 0};
    offset += (sizes[i] + kAdamBlock - 1) / kAdamBlock * kAdamBlock;
    for (int64_t c = 0; c < chunks_of(sizes[i]); ++c) *q++ = Piece{i, (int32_t)c};
  }
}

hipError_t adamw_step(const AdamArgs& a) {
  const Entry* entries = static_cast<const Entry*>(a.table);
  const Piece* pieces = reinterpret_cast<const Piece*>(static_cast<const char*>(a.table) + entries_bytes(a.n_tensors));
  Scalars* s = static_cast<Scalars*>(a.scalars);
  const auto prepare = [&](int first, int n, int64_t chunk, int64_t chunks, Run& r, Grads& g) {
    r = Run{entries, pieces + chunk, first, (int)chunks, s};
    for (int i = 0; i < n; ++i) g.g[i] = a.grads[first + i];
  };
  const Begin start{a.beta1, a.beta2, a.max_norm, a.lr, a.lr_at, a.norm};
  const int parts = a.max_norm > 0 ? (int)(adamw_workspace_bytes(a.n_tensors, a.sizes) / sizeof(double)) : 0;
  hipError_t e = hipSuccess;
  bool fused = false;
  if (parts > 0) {
    int at = 0;
    fused = parts <= kFused;
    e = each_launch(a.n_tensors, a.sizes, [&](int first, int n, int64_t chunk, int64_t chunks) {
      Run r;
      Grads g;
      prepare(first, n, chunk, chunks, r, g);
      const int blocks = (int)std::min<int64_t>(kNormBlocks, chunks);
      double* to = static_cast<double*>(a.ws);
      if (a.grad_dtype == TP_F32)
        hipLaunchKernelGGL(k_adam_norm<float>, dim3(blocks), dim3(kThreads), 0, a.stream, r, g, to, at, fused ? parts : 0, start);
      else
        hipLaunchKernelGGL(k_adam_norm<bf16_t>, dim3(blocks), dim3(kThreads), 0, a.stream, r, g, to, at, fused ? parts : 0, start);
      at += blocks;
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!fused) {
    hipLaunchKernelGGL(k_adam_begin, dim3(1), dim3(kThreads), 0, a.stream, s, static_cast<const double*>(a.ws), parts, start);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  // the reciprocal's instruction need not take a subnormal eps
  const float eps = a.eps > 0 ? std::max((float)a.eps, 0x1p-126f) : 0.f;
  const Rates b{a.beta1, a.beta2, 1.0 - a.beta1, 1.0 - a.beta2, eps};
  return each_launch(a.n_tensors, a.sizes, [&](int first, int n, int64_t chunk, int64_t chunks) {
    Run r;
    Grads g;
    prepare(first, n, chunk, chunks, r, g);
    const dim3 grid((unsigned)chunks);
    const auto go = [&](auto t) {
      typedef decltype(t) T;
      if (a.bits == 32)
        hipLaunchKernelGGL(k_adam32<T>, grid, dim3(kThreads), 0, a.stream, r, g, (float*)a.m, (float*)a.v, b);
      else
        hipLaunchKernelGGL(k_adam8<T>, grid, dim3(kThreads), 0, a.stream, r, g, (uint8_t*)a.m, (uint8_t*)a.v, a.m_unit,
                           a.v_unit, b, (uint32_t)a.seed, (uint32_t)(a.seed >> 32));
      return hipGetLastError();
    };
    return a.grad_dtype == TP_F32 ? go(float()) : go(bf16_t());
  });
}

hipError_t adamw_values(int second, int64_t n, const uint8_t* codes, const float* units, float* out, hipStream_t st) {
  const int64_t blocks = (n + kChunk - 1) / kChunk;
  if (blocks > 0xffffffffLL / kThreads) return hipErrorInvalidConfiguration;
  if (second)
    hipLaunchKernelGGL(k_adam_values<true>, dim3((unsigned)blocks), dim3(kThreads), 0, st, n, codes, units, out);
  else
    hipLaunchKernelGGL(k_adam_values<false>, dim3((unsigned)blocks), dim3(kThreads), 0, st, n, codes, units, out);
  return hipGetLastError();
}

}  // namespace tpc
