// Pieces shared by the attention kernels (attn_fwd.hip, attn_dq.hip, attn_dkv.hip).
//
// A wave owns 32 rows (queries, or keys in the key-side backward) and walks the
// other side in tiles of 32 rows staged in LDS.  Products run on
// v_mfma_f32_32x32x16_bf16 with the staged tile as the A operand, so a score tile
// comes out transposed: lane l holds column l % 32 (its own row) and tile rows
// 8 (i / 4) + 4 (l / 32) + i % 4, i = 0..15.  Softmax statistics are then one
// value per lane, and the tile is already the B operand of the next product
// (the order of a contraction index is free as long as A uses the same one),
// with the A operand read column-wise through the LDS transpose loads.
// float32 operands go as three bfloat16 pieces (split.hpp).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.hpp"
#include "rows.hpp"
#include "split.hpp"

namespace tpc {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// scores at or below -1e30 count as masked; a little above it, so that rounding lets none through
constexpr float kLowest = -0.9999e30f;
constexpr int kTile = 32;
constexpr int kMaxBuckets = 64;

// geometry of a staged tile: 32 rows of KS * 16 values (zero-filled from
// head_dim on), rows padded by 16 bytes so that 16-byte reads of 32 rows spread over the
// banks (the row length in 16-byte units is odd)
template <typename T, int KS>
struct Tile {
  static constexpr int P = kPlanes<T>;
  static constexpr int MT = (KS + 1) / 2;            // 32-row blocks of the head dimension
  static constexpr int kRow = 32 * MT + 8;           // 16-bit elements per row
  static constexpr int kPlane = kTile * kRow;
  static constexpr int kElems = P * kPlane;
};

// eight consecutive values of a row, as loaded from memory
template <typename T>
struct Raw;
template <>
struct Raw<bf16_t> {
  u4 v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const u4*>(p); }
  __device__ __forceinline__ void keep(bool k) { v = k ? v : u4{0, 0, 0, 0}; }
  __device__ __forceinline__ void negate() { v ^= 0x80008000u; }
  template <bool FAR>
  __device__ __forceinline__ void frag(Frag<1>& f) const { f.p[0] = __builtin_bit_cast(b8, v); }
  __device__ __forceinline__ float at(int j) const { return (float)__builtin_bit_cast(b8, v)[j]; }
};
template <>
struct Raw<float> {
  f4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f4*>(p);
    b = *reinterpret_cast<const f4*>(p + 4);
  }
  __device__ __forceinline__ void keep(bool k) {
    a = k ? a : f4{0.f, 0.f, 0.f, 0.f};
    b = k ? b : f4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void negate() {
    a = -a;
    b = -b;
  }
  template <bool FAR>
  __device__ __forceinline__ void frag(Frag<3>& f) const {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    to_frag<FAR>(x, f);
  }
  __device__ __forceinline__ float at(int j) const { return j < 4 ? a[j] : b[j - 4]; }
};

// row operand: row l % 32, contraction elements 16 kk + 8 (l / 32) + 0..7
template <typename G>
__device__ __forceinline__ Frag<G::P> row_frag(const uint16_t* tile, int kk, int lane) {
  Frag<G::P> f;
#pragma unroll
  for (int p = 0; p < G::P; ++p)
    f.p[p] = *reinterpret_cast<const b8*>(tile + p * G::kPlane + (lane & 31) * G::kRow + 16 * kk + 8 * (lane >> 5));
  return f;
}

// column operand: element 32 mt + l % 32 of the head dimension, tile rows
// 16 kb + 4 (l / 32) + {0..3, 8..11}: the rows whose scores the lane holds.  The
// transpose load hands lane i of a group of 16 the i-th column of the 4 rows x 16
// columns that the group addresses (4 lanes a row).
template <typename G>
__device__ __forceinline__ Frag<G::P> col_frag(const uint16_t* tile, int mt, int kb, int lane) {
  Frag<G::P> f;
  const int row = 16 * kb + 4 * (lane >> 5) + ((lane & 15) >> 2), col = 32 * mt + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
  for (int p = 0; p < G::P; ++p) {
    const uint16_t* at = tile + p * G::kPlane + row * G::kRow + col;
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at);
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(at + 8 * G::kRow));
    f.p[p] = __builtin_bit_cast(b8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return f;
}

// store eight consecutive values into a staged tile
template <typename G, bool FAR, typename T>
__device__ __forceinline__ void put(uint16_t* tile, int row, int col8, const Raw<T>& r) {
  Frag<G::P> f;
  r.template frag<FAR>(f);
#pragma unroll
  for (int p = 0; p < G::P; ++p)
    *reinterpret_cast<b8*>(tile + p * G::kPlane + row * G::kRow + 8 * col8) = f.p[p];
}

// the larger of a lane's value and that of the lane 32 away (which holds the other
// half of the same row), and the same for sums
__device__ __forceinline__ float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
  return fmaxf(flt(r[0]), flt(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
  return flt(r[0]) + flt(r[1]);
}

// Tile t of the packed batch in tiles of `rows` rows: structure b's tiles start at
// number seg[b] / rows + b, which never overlap and leave at most one unused
// number per structure, so a grid of n_nodes / rows + n_segments tiles covers every
// batch without the host knowing the lengths.  The wave looks b up 64 entries
// at a time (1 step up to 64 structures, 2 up to 4,096).  False: an unused number.
__device__ __forceinline__ bool find_tile(const tp_attn& d, int rows, int t, int& lo, int& hi, int& first) {
  const int lane = threadIdx.x & 63, N = d.n_nodes;
  int b = 0, n = d.n_segments;
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int at = b + lane * step;
    bool le = false;
    if (lane * step < n) {
      const int s = min(max(d.seg_ptr[at], 0), N);
      le = s / rows + at <= t;
    }
    const int cnt = __popcll(__ballot(le));
    if (cnt == 0) return false;            // not a valid seg_ptr
    b += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  lo = min(max(d.seg_ptr[b], 0), N);
  hi = min(max(d.seg_ptr[b + 1], 0), N);
  const int64_t q = (int64_t)lo + (int64_t)(t - (lo / rows + b)) * rows;
  first = (int)q;
  return q >= lo && q < hi;
}

// Scores are formed as c S with S = sign q k + bias / |scale|, c = |scale| log2 e (base-2
// units): the bias starts the accumulator of the product and costs no instruction,
// and the running maximum is taken on S.  scale 0: sign 0, c = log2 e.
struct Scale {
  float sign, c, inv;
  __device__ __forceinline__ explicit Scale(float scale) {
    const float a = scale != 0.f ? fabsf(scale) : 1.f;
    sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
    c = a * kLog2e;
    inv = 1.f / a;
  }
};

// A row's lse in base-2 units, for p = exp2(c S - lse); a row without keys gets p = 0.
// lse and this product are off by up to 4 2^-24 of their size.  From 2^22 on, where a score's own
// rounding is half a unit, that may make p huge or, from 10^9 on, infinite (and 0 times it
// NaN): there lse is raised by 8 2^-24 of its size, which keeps p below 1.
__device__ __forceinline__ float row_lse(float e) {
  const float x = e * kLog2e, size = fabsf(x);
  return e == -INFINITY ? INFINITY : size > 4194304.f ? fmaf(size, 0x1p-21f, x) : x;
}

// LDS bias table of HG heads, [entry][HG][32], in units of S; 32 copies of every value,
// so that the lanes of a half wave, each with a bucket of its own, read 32 different
// banks.
__device__ __forceinline__ float bias_at(const tp_attn& d, int h, int b) {
  const size_t i = (size_t)h * d.n_buckets + b;
  return d.dtype == TP_F32 ? static_cast<const float*>(d.bias)[i] : (float)static_cast<const bf16_t*>(d.bias)[i];
}
// THREADS / 64 threads share an entry's eight 16-byte chunks.  They load its value early, with
// all else that the walk begins with, and later write its copies, starting at different
// columns for different banks.
template <int HG, int THREADS>
struct TableFill {
  static constexpr int kShare = THREADS / 64;
  static_assert(THREADS % 64 == 0 && 8 % kShare == 0 && kMaxBuckets == 64);
  float v[HG];
  static __device__ __forceinline__ int entry(int u) { return (int)threadIdx.x / kShare + 64 * u; }
  __device__ __forceinline__ void load(const tp_attn& d, int h0) {
#pragma unroll
    for (int u = 0; u < HG; ++u) v[u] = entry(u) < d.n_buckets * HG ? bias_at(d, h0 + entry(u) % HG, entry(u) / HG) : 0.f;
  }
  __device__ __forceinline__ void write(const tp_attn& d, float inv, float* tbl) const {
    const int ne = d.n_buckets > 0 ? d.n_buckets : 1;
#pragma unroll
    for (int u = 0; u < HG; ++u) {
      const int i = entry(u);
      if (i >= ne * HG) break;
      const float w = v[u] * inv;
#pragma unroll
      for (int j = threadIdx.x % kShare; j < 8; j += kShare)
        reinterpret_cast<f4*>(tbl)[8 * i + ((i + j) & 7)] = f4{w, w, w, w};
    }
  }
};

typedef __attribute__((address_space(3))) float lds_f;
__device__ __forceinline__ uint32_t lds_address(const float* p) { return (uint32_t)(uintptr_t)(lds_f*)p; }
__device__ __forceinline__ lds_f* lds_at(uint32_t address) { return (lds_f*)(uintptr_t)address; }

// bucket -> LDS address of this lane's copy in the table
template <int HG>
struct Buckets {
  static constexpr int kEntry = HG * 128;
  int shift;
  float lo, hi;
  uint32_t add, first;                     // first: the only entry where there is no bias
  __device__ __forceinline__ Buckets(const tp_attn& d, const float* tbl, int lane) {
    int lg = 0;
    while ((1 << lg) < d.steps) ++lg;
    shift = 23 - lg;
    const int base = (int)(bits(d.r_min * d.r_min) >> shift), nb = d.n_buckets > 0 ? d.n_buckets : 1;
    lo = flt((uint32_t)base << shift);
    // a range that passes the largest float ends at infinity: as a float beyond it is a NaN or
    // negative, and would let distances below lo through
    hi = flt(min(((uint32_t)(base + nb) << shift) - 1, 0x7f800000u));
    first = lds_address(tbl) + (lane & 31) * 4;
    add = first - base * kEntry;
  }
  // the squared distance, every operation rounded once (no fused multiply-add).  It is
  // clamped as a float: positive floats are ordered as their representations, and the median of NaN
  // is the lower bound (bucket 0).
  __device__ __forceinline__ uint32_t address(float ax, float ay, float az, float bx, float by, float bz) const {
#pragma clang fp contract(off)
    const float dx = ax - bx, dy = ay - by, dz = az - bz;
    const float xx = dx * dx, yy = dy * dy, zz = dz * dz;
    const float d2 = (xx + yy) + zz;
    return (bits(__builtin_amdgcn_fmed3f(d2, lo, hi)) >> shift) * kEntry + add;
  }
};

// table addresses of the 16 tile rows that a lane holds: bucket of (own position, row's
// position).  pos: LDS [3][32].
template <int HG>
__device__ __forceinline__ void tile_entries(const Buckets<HG>& bk, const float* pos, int half, float x, float y,
                                             float z, uint32_t ent[16]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int r = 8 * g + 4 * half;
    const f4 px = *reinterpret_cast<const f4*>(pos + r), py = *reinterpret_cast<const f4*>(pos + kTile + r),
             pz = *reinterpret_cast<const f4*>(pos + 2 * kTile + r);
#pragma unroll
    for (int j = 0; j < 4; ++j) ent[4 * g + j] = bk.address(x, y, z, px[j], py[j], pz[j]);
  }
}
// scores of tile rows that do not count (bit r of valid clear)
__device__ __forceinline__ void mask_scores(uint32_t valid, int half, f16v& s) {
  const uint32_t m = valid >> (4 * half);
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = (m >> (8 * (i / 4) + i % 4)) & 1 ? s[i] : -INFINITY;
}

// S of a tile: the bias of every pair, then the product of the staged rows with the
// wave's own rows
template <typename G, int KS, bool SWAPPED = false>
__device__ __forceinline__ f16v scores(const uint16_t* tile, const Frag<G::P> own[KS], const uint32_t ent[16], int hh,
                                       int lane) {
  f16v s;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = lds_at(ent[i])[hh * 32];
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) s = mma<SWAPPED>(row_frag<G>(tile, kk, lane), own[kk], s);
  return s;
}
// the same without a bias
template <typename G, int KS, bool SWAPPED = false>
__device__ __forceinline__ f16v product(const uint16_t* tile, const Frag<G::P> own[KS], int lane) {
  f16v s;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) s = mma<SWAPPED>(row_frag<G>(tile, kk, lane), own[kk], s);
  return s;
}

// Staging of a tile, NS head slots of two arrays each (array number 2 slot +
// which), by the NT threads that share it: every thread fetches its 8-value chunks
// into registers while an earlier tile is worked on, then puts them into LDS.  Rows
// past the end or masked are staged as zeros.
template <typename T, int KS, int NT, int NS>
struct Stager {
  using G = Tile<T, KS>;
  static constexpr int kArrays = NS * 2;
  static constexpr int kChunks = (kArrays * kTile * 2 * KS + NT - 1) / NT;
  static constexpr int kBytes = kArrays * G::kElems * 2;
  Raw<T> raw[kChunks];
  bool live[kChunks];
  uint8_t byte[kChunks];                   // the mask's
  const T* at[kChunks];                    // this thread's chunk of the next tile
  const T *safe0, *safe1;                  // what is loaded where a chunk does not exist
  int64_t step0, step1;
  int tid;
  bool whole;                              // every chunk of the tile fetched last exists

  __device__ __forceinline__ int chunk(int i) const { return tid + i * NT; }
  static __device__ __forceinline__ int col_of(int c) { return c % (2 * KS); }
  static __device__ __forceinline__ int row_of(int c) { return c / (2 * KS) % kTile; }
  static __device__ __forceinline__ int array_of(int c) { return c / (2 * KS * kTile); }

  // the tile of rows r0 .. is next, then every `stride` rows, of a structure that starts at
  // row lo; head(slot): the head of a slot
  template <typename Head>
  __device__ __forceinline__ void aim(int thread, const void* p0, int64_t s0, const void* p1, int64_t s1, int lo, int r0,
                                      int stride, int D, Head&& head) {
    tid = thread;
    step0 = s0 * stride;
    step1 = s1 * stride;
    safe0 = static_cast<const T*>(p0) + lo * s0;
    safe1 = static_cast<const T*>(p1) + lo * s1;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = chunk(i), t = array_of(c);
      const int64_t r = r0 + row_of(c) - lo;
      at[i] = (t & 1 ? safe1 + r * s1 : safe0 + r * s0) + head((t >> 1) % NS) * D + 8 * col_of(c);
    }
  }
  // back to the first of n tiles fetched since aim, `columns` to the right of it
  __device__ __forceinline__ void again(int n, int columns) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) at[i] += columns - n * (array_of(chunk(i)) & 1 ? step1 : step0);
  }
  // loads the tile that aim (or the previous fetch) has come to, rows r0 ..
  __device__ __forceinline__ void fetch(int r0, int end, int D, const uint8_t* mask) {
    constexpr bool kEven = kArrays * kTile * 2 * KS % NT == 0;
    whole = kEven && end - r0 >= kTile && D == 16 * KS && !mask;
    const T* p[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) p[i] = at[i];
    if (!whole) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = chunk(i), t = array_of(c), r = r0 + row_of(c);
        live[i] = t < kArrays && r < end && 8 * col_of(c) < D;
        if (!live[i]) p[i] = t & 1 ? safe1 : safe0;
        byte[i] = mask ? mask[r < end ? r : end - 1] : 1;
      }
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      raw[i].load(p[i]);
      at[i] += array_of(chunk(i)) & 1 ? step1 : step0;
    }
  }
  __device__ __forceinline__ void stage(uint16_t* tiles, bool far = false) {
    if (!whole) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) raw[i].keep(live[i] && byte[i] != 0);
    }
    if (far) put_all<true>(tiles);
    else put_all<false>(tiles);
  }
  template <bool FAR>
  __device__ __forceinline__ void put_all(uint16_t* tiles) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = chunk(i);
      if (array_of(c) < kArrays) put<G, FAR>(tiles + array_of(c) * G::kElems, row_of(c), col_of(c), raw[i]);
    }
  }
};

// positions and validity of a tile's rows, one per thread of the first 32 that share it.
// LDS: [3][32] positions, then the validity bits.
struct RowStager {
  static constexpr int kBytes = 3 * kTile * 4 + 16;
  float x = 0.f, y = 0.f, z = 0.f;
  bool live = false;
  uint8_t byte = 1;                        // the mask's
  __device__ __forceinline__ void fetch(int tid, const tp_attn& d, bool biased, int r0, int end, const uint8_t* mask) {
    if (tid < kTile) {
      const int r = r0 + tid, rc = r < end ? r : end - 1;
      live = r < end;
      if (mask) byte = mask[rc];
      if (biased) {
        x = d.pos[3 * (size_t)rc];
        y = d.pos[3 * (size_t)rc + 1];
        z = d.pos[3 * (size_t)rc + 2];
      }
    }
  }
  __device__ __forceinline__ void stage(int tid, float* lds) const {
    const uint32_t vote = (uint32_t)__ballot(live && byte != 0);
    if (tid < kTile) {
      lds[tid] = x;
      lds[kTile + tid] = y;
      lds[2 * kTile + tid] = z;
    }
    if (tid == 0) *reinterpret_cast<uint32_t*>(lds + 3 * kTile) = vote;
  }
  static __device__ __forceinline__ uint32_t valid(const float* lds) {
    return __builtin_amdgcn_readfirstlane(*reinterpret_cast<const uint32_t*>(lds + 3 * kTile));
  }
};

// Between a wave's own LDS accesses where lanes read what other lanes wrote, or write again
// what they read: the hardware executes a wave's LDS accesses in order, the fence keeps the
// compiler to it (a wave barrier alone restrains scheduling only).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Walks the tiles of one group of waves: prepare(i) starts tile i's loads into registers,
// stage(i, buffer) puts them into LDS, work(i, buffer) uses them.  A tile that several
// waves share is staged one tile ahead into the other of two buffers, with one barrier
// a tile, or, where LDS holds one buffer only, between two barriers.  A wave on its own
// needs no barrier and one buffer.  All groups
// of the workgroup take the same n.  The caller has done prepare(0), as early as it can.
template <bool SHARED, int BUFS, typename Prepare, typename Stage, typename Work>
__device__ __forceinline__ void walk(int n, Prepare&& prepare, Stage&& stage, Work&& work) {
  if (SHARED && BUFS == 2) {
    stage(0);
    if (n > 1) prepare(1);
    __syncthreads();
    for (int i = 0; i < n; ++i) {
      if (i + 1 < n) stage((i + 1) & 1);
      if (i + 2 < n) prepare(i + 2);
      work(i & 1);
      __syncthreads();
    }
  } else {
    for (int i = 0; i < n; ++i) {
      if (SHARED) __syncthreads();
      else wave_sync();
      stage(0);
      if (SHARED) __syncthreads();
      else wave_sync();
      if (i + 1 < n) prepare(i + 1);
      work(0);
    }
  }
}
// buffers of a tile that `share` waves share, `groups` of them side by side: LDS for two
// workgroups a CU beside their tables
constexpr int buffers(int bytes, int share, int groups) { return share > 1 && 2 * groups * bytes <= 60 * 1024 ? 2 : 1; }

// the wave's own rows as B operands, times sign (1, -1 or 0: exact): row `r`,
// contraction elements 16 kk + 8 half ..
template <typename T, int KS>
__device__ __forceinline__ void own_rows(const void* p, int64_t stride, int r, int head, int D, int half, bool keep,
                                         float sign, Frag<kPlanes<T>> f[KS], bool far = false) {
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    const int c = 16 * kk + 8 * half;
    Raw<T> w;
    w.load(static_cast<const T*>(p) + (size_t)r * stride + (size_t)head * D + (c < D ? c : 0));
    w.keep(keep && c < D && sign != 0.f);
    if (sign < 0.f) w.negate();
    if (far) w.template frag<true>(f[kk]);
    else w.template frag<false>(f[kk]);
  }
}

// four values of a row of a transposed accumulator (lane: own row; register 16 mt + 4 g + j:
// element 32 mt + 8 g + 4 half + j of the head dimension) to memory
template <typename T>
__device__ __forceinline__ void store4(void* p, int64_t stride, int r, int head, int D, int half, int mt, int g,
                                       const float v[4]) {
  const int e = 32 * mt + 8 * g + 4 * half;
  if (e < D) {
    T w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (T)v[j];
    T* o = static_cast<T*>(p) + (size_t)r * stride + (size_t)head * D + e;
    __builtin_memcpy(__builtin_assume_aligned(o, 4 * sizeof(T)), w, sizeof(w));
  }
}

// Accumulators of the waves that split the other side meet in LDS, [wave][part][register]
// [lane]; each of them then adds up and stores its share of the registers, four at a
// time.
template <int MT>
__device__ __forceinline__ void park(float* at, const f16v acc[MT]) {
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 16; ++i) at[64 * (16 * mt + i)] = acc[mt][i];
}
// sum over W waves of factor[w] times register group gi (at: of wave 0, waves `stride` floats apart)
template <int W>
__device__ __forceinline__ void sum_parked(const float* at, int stride, int gi, const float* factor, float v[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v[j] = fmaf(at[w * stride + 64 * (4 * gi + j)], factor ? factor[w] : 1.f, v[j]);
  }
}

template <int MT>
__device__ __forceinline__ void clear(f16v acc[MT]) {
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[mt][i] = 0.f;
}

constexpr size_t kLdsMax = 160 * 1024;
constexpr int kCUs = 256;

// How many waves a call can use: 32-row tiles times heads, the mean length of a structure.
// A batch of one long structure and many small ones has a small mean: its shape is that of the
// small ones.
struct Extent {
  int64_t units, mean;
  Extent(const tp_attn& d, int heads)
      : units(((int64_t)d.n_nodes / kTile + d.n_segments) * heads), mean(d.n_nodes / (d.n_segments > 0 ? d.n_segments : 1)) {}
};

// a launch with `bytes` of LDS, which above 64 KiB have to be asked for
template <typename K>
hipError_t launch_lds(K kernel, dim3 grid, int threads, size_t bytes, const AttnArgs& args) {
  if ((uint64_t)grid.x * threads > UINT32_MAX) return hipErrorInvalidConfiguration;
  if (args.dry) return hipSuccess;
  if (bytes > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kLdsMax);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, grid, dim3(threads), bytes, args.stream, args);
  return hipGetLastError();
}

}  // namespace tpc
