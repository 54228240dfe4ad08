// Pieces shared by the products by group (grouped.hip, grouped_weight.hip).
//
// A workgroup forms one tile of a group's product on v_mfma_f32_32x32x16_bf16, float32
// operands as three bfloat16 planes (split.hpp).  Tiles are staged in LDS in steps of the
// contraction, in one of two layouts: rows of the operand with the contraction along them
// (read 16 bytes a lane), or rows of the contraction with the operand's index along them (read
// through the LDS transpose loads).  In both the 16-byte chunks of a row are permuted by its
// number, so that reads spread over the banks without padding.
#pragma once
#include <hip/hip_runtime.h>

#include "internal.hpp"
#include "parts.hpp"
#include "rows.hpp"
#include "split.hpp"

namespace tpc {

constexpr int kGemmThreads = 256;

// eight consecutive values of a row
template <typename T>
struct Octet;
template <>
struct Octet<bf16_t> {
  RawChunk<bf16_t> v;
  __device__ __forceinline__ void load(const bf16_t* p, int left) { v.load(p, left); }
  __device__ __forceinline__ float at(int j) const { return v.at(j); }
  __device__ __forceinline__ void frag(Frag<1>& f) const { f.p[0] = __builtin_bit_cast(b8, v.v); }
};
template <>
struct Octet<float> {
  RawChunk<float> a, b;
  __device__ __forceinline__ void load(const float* p, int left) {
    a.load(p, left);
    b.load(p + 4, left - 4);
  }
  __device__ __forceinline__ float at(int j) const { return j < 4 ? a.at(j) : b.at(j - 4); }
  __device__ __forceinline__ void frag(Frag<3>& f) const {
    const float x[8] = {a.at(0), a.at(1), a.at(2), a.at(3), b.at(0), b.at(1), b.at(2), b.at(3)};
    to_frag<true>(x, f);                   // an infinity stays one
  }
};

// An operand tile with the contraction along its rows: R rows of S values (a step)
template <typename T, int R, int S>
struct AlongTile {
  static_assert(S == 32 || S == 64);
  static constexpr int P = kPlanes<T>, kChunks = S / 8, kPlane = R * S, kElems = P * kPlane;
  static __device__ __forceinline__ int at(int row, int chunk) {
    // eight rows at a time reach all banks: 128-byte rows by their number, of 64 bytes by every other
    return row * S + ((chunk ^ (S == 64 ? row & 7 : row >> 1 & 3)) * 8);
  }
  static __device__ __forceinline__ void put(uint16_t* t, int row, int chunk, const Octet<T>& o) {
    Frag<P> f;
    o.frag(f);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<b8*>(t + p * kPlane + at(row, chunk)) = f.p[p];
  }
  // rows 32 block + l % 32, contraction 16 kk + 8 (l / 32) + 0..7
  static __device__ __forceinline__ Frag<P> frag(const uint16_t* t, int block, int kk, int lane) {
    Frag<P> f;
#pragma unroll
    for (int p = 0; p < P; ++p)
      f.p[p] = *reinterpret_cast<const b8*>(t + p * kPlane + at(32 * block + (lane & 31), 2 * kk + (lane >> 5)));
    return f;
  }
};

// An operand tile with the contraction across its rows: S rows of R values
template <typename T, int R, int S>
struct AcrossTile {
  static_assert(R == 64 || R == 128);
  static constexpr int P = kPlanes<T>, kChunks = R / 8, kPlane = R * S, kElems = P * kPlane;
  static __device__ __forceinline__ int at(int row, int chunk) {
    // pairs of chunks stay together: a transpose load takes 4 rows of 32 bytes
    return row * R + ((chunk ^ 2 * (R == 128 ? row & 7 : row >> 1 & 3)) * 8);
  }
  static __device__ __forceinline__ void put(uint16_t* t, int row, int chunk, const Octet<T>& o) {
    Frag<P> f;
    o.frag(f);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<b8*>(t + p * kPlane + at(row, chunk)) = f.p[p];
  }
  // The transpose load hands lane i of a group of 16 the i-th column of the 4 rows x 16 columns
  // that the group addresses (4 lanes a row).
  static __device__ __forceinline__ Frag<P> frag(const uint16_t* t, int block, int kk, int lane) {
    Frag<P> f;
    const int row = 16 * kk + 8 * (lane >> 5) + ((lane & 15) >> 2), chunk = 4 * block + 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
    const int lo_at = at(row, chunk) + 4 * (lane & 1), hi_at = at(row + 4, chunk) + 4 * (lane & 1);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(t + p * kPlane + lo_at));
      const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(t + p * kPlane + hi_at));
      f.p[p] = __builtin_bit_cast(b8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return f;
  }
};

// The groups cut into parts of `size` slots, numbered without gaps.  A wave counts the parts of 64 runs
// of groups at once; the host knows n / size + groups as a bound of their number.  `groups` counts the one
// behind the last pointer where slots without a group are parts too; `least` is 1 where an empty group
// counts as one part.
struct Part {
  int group, lo, hi, first;                // slots of the group, first slot of the part
};
struct Parts {
  const int32_t* ptr;
  int groups, n_groups, n, size, least, run, total;
  int first_slot, end_slot, before;        // of this lane's run; parts of the lanes below
  __device__ __forceinline__ int start(int e) const { return e <= n_groups ? min(max(ptr[e], 0), n) : n; }
  __device__ __forceinline__ int count(int lo, int hi) const { return part_count(hi - lo, size, least); }
  // x plus that of the lanes `shift` below it in the same row of 16, or of the rows before
  template <int CONTROL, int ROWS>
  static __device__ __forceinline__ int add(int x) {
    return x + __builtin_amdgcn_update_dpp(0, x, CONTROL, ROWS, 0xf, false);
  }
  __device__ __forceinline__ Parts(const int32_t* p, int real, int all, int slots, int each, int at_least)
      : ptr(p), groups(all), n_groups(real), n(slots), size(each), least(at_least) {
    const int lane = threadIdx.x & 63;
    run = (groups + 63) >> 6;
    int c = 0;
    first_slot = end_slot = start(lane * run);
    if (run == 1) {
      end_slot = start(lane + 1);
      c = lane < groups ? count(first_slot, end_slot) : 0;
    } else {
      for (int i = lane * run; i < min(groups, lane * run + run); ++i) {
        const int hi = start(i + 1);
        c += count(end_slot, hi);
        end_slot = hi;
      }
    }
    int sum = add<0x111, 0xf>(c);          // the running sum over the lanes: 1, 2, 4, 8 lanes back,
    sum = add<0x112, 0xf>(sum);
    sum = add<0x114, 0xf>(sum);
    sum = add<0x118, 0xf>(sum);
    sum = add<0x142, 0xa>(sum);            // then the ends of the rows of 16 before
    sum = add<0x143, 0xc>(sum);
    before = sum - c;
    // a wrong ptr may count to anything: no more than the launch has, and no group that is not there
    total = min(max(__builtin_amdgcn_readlane(sum, 63), 0), n / size + groups);
  }
  // part t < total
  __device__ __forceinline__ Part at(int t) const {
    const int owner = max(__popcll(__ballot(before <= t)) - 1, 0);
    const int last = __builtin_amdgcn_readfirstlane(min(owner, (groups - 1) / run));
    int left = t - __builtin_amdgcn_readlane(before, last);
    Part p;
    p.group = last * run;
    p.lo = __builtin_amdgcn_readlane(first_slot, last);
    p.hi = __builtin_amdgcn_readlane(end_slot, last);
    if (run > 1) {
      p.hi = start(p.group + 1);
      for (;;) {
        const int c = count(p.lo, p.hi);
        if (left < c || p.group + 1 >= groups) break;
        left -= c;
        ++p.group;
        p.lo = p.hi;
        p.hi = start(p.group + 1);
      }
    }
    p.first = (int)min((int64_t)p.lo + (int64_t)left * size, (int64_t)n);
    return p;
  }
};

// a slot by its place in group order; what is out of range is clamped
__device__ __forceinline__ int slot_at(const int32_t* rows, int place, int n) {
  return (int)min((uint32_t)rows[place], (uint32_t)(n - 1));
}
// the row of a slot: itself, or rows[slot] / div
__device__ __forceinline__ int row_of(const int32_t* rows, int slot, int div, int n) {
  if (div == 0) return slot;
  const uint32_t r = min((uint32_t)rows[slot], (uint32_t)(n - 1));
  return (int)(div == 1 ? r : r / (uint32_t)div);
}

// Workgroups go round the 8 dies in turn; each die gets a run of consecutive ones of `total` tiles.
__device__ __forceinline__ int place_of(int id, int total) {
  constexpr int kDies = 8;
  const int whole = total / kDies, more = total % kDies, die = id % kDies;
  return die * whole + min(die, more) + id / kDies;
}
// Tile t of rows x cols: 8 row tiles by all columns at a time, so that what a die reads of both operands
// stays in its L2.
__device__ __forceinline__ void place_tile(int t, int rows, int cols, int& r, int& c) {
  constexpr int kBand = 8;
  const int band = t / (kBand * cols), first = band * kBand, high = min(kBand, rows - first), in = t - first * cols;
  r = first + in % high;
  c = in / high;
}

// The sigmoid s of z and 1 - s, from exp(-|z|), so that both are right relatively; exp and reciprocal to a unit in the
// last place.  float32: what the product by log2(e) loses goes on as a factor, 10 u of s in all (without it 0.75 |z| u
// more, 57 u at -50).  Below z = -87.3 the sigmoid is 0.
template <typename T>
struct Sigmoid {
  float s, rest;
  __device__ __forceinline__ explicit Sigmoid(float z) {
    constexpr float kLog2E = 0x1.715476p+0f, kMore = 0x1.4ae0cp-26f, kLn2 = 0.69314718f;    // log2(e) in two pieces
    const float a = fminf(fabsf(z), 100.f), t = a * -kLog2E, lost = fmaf(a, -kMore, fmaf(a, -kLog2E, -t));
    const float e = __builtin_amdgcn_exp2f(t) * fmaf(lost, kLn2, 1.f), q = __builtin_amdgcn_rcpf(1.f + e);
    s = z < 0.f ? e * q : q;
    rest = z < 0.f ? q : e * q;
  }
};
// bfloat16: s to (0.75 |z| + 4) u of itself, 1 - s to 4 u of 1, far below the 2^16 u of the results' rounding; the other
// form would be twice the instructions of the activation, which nothing covers in a large tile.
template <>
struct Sigmoid<bf16_t> {
  float s, rest;
  __device__ __forceinline__ explicit Sigmoid(float z) {
    s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
    rest = 1.f - s;
  }
};
template <typename T>
__device__ __forceinline__ float silu(float z) {
  return z * Sigmoid<T>(z).s;
}
template <typename T>
__device__ __forceinline__ float silu_slope(float z) {
  const Sigmoid<T> g(z);
  return g.s * (1.f + z * g.rest);
}

// ---- the fast path: operands straight to LDS --------------------------------------------
// Tiles of 16-byte chunks go from memory to LDS without passing registers (one instruction
// moves 64 chunks to consecutive places), in the operands' type; the permutation of a row's chunks is
// made by what each lane fetches.  Two to four buffers, so that a step's loads have the
// steps before to arrive in.  float32 is split into its three pieces as the fragments are read: pieces
// in LDS would take half as many bytes again and would be formed once for every tile that
// shares an operand anyway.  Needs rows of whole, aligned chunks; the rest of a step past the
// contraction's end is fetched from a chunk of zeros.
typedef __attribute__((address_space(1))) const void global_bytes;
typedef __attribute__((address_space(3))) void lds_bytes;
__device__ __forceinline__ void fetch16(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((global_bytes*)from, (lds_bytes*)to, 16, 0, 0);
}
static __device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// contraction values of a step: 128 bytes
template <typename T>
constexpr int kDeep = 128 / sizeof(T);

// R rows with the contraction along them.  A wave's instruction q takes rows 8 q .. 8 q + 7.
template <typename T, int R, int WAVES>
struct AlongLds {
  static constexpr int kBytes = R * 128, Q = R / 8 / WAVES, kPer = 16 / sizeof(T);
  static_assert(R % (8 * WAVES) == 0);
  static __device__ __forceinline__ int row(int q, int wave, int lane) { return 8 * (q * WAVES + wave) + (lane >> 3); }
  static __device__ __forceinline__ int first(int lane) { return ((lane & 7) ^ (lane >> 3)) * kPer; }   // value of the row
  static __device__ __forceinline__ uint8_t* place(uint8_t* t, int q, int wave) { return t + 1024 * (q * WAVES + wave); }
  static __device__ __forceinline__ const uint8_t* chunk(const uint8_t* t, int row, int c) {
    return t + row * 128 + (c ^ (row & 7)) * 16;
  }
  // rows 32 block + l % 32, contraction 16 kk + 8 (l / 32) + 0..7
  static __device__ __forceinline__ void read(const uint8_t* t, int block, int kk, int lane, Octet<T>& o) {
    const int r = 32 * block + (lane & 31);
    if constexpr (sizeof(T) == 2) {
      o.v.v = __builtin_bit_cast(Chunk<bf16_t>::vec, *reinterpret_cast<const b8*>(chunk(t, r, 2 * kk + (lane >> 5))));
    } else {
      o.a.v = __builtin_bit_cast(Chunk<float>::vec, *reinterpret_cast<const f4*>(chunk(t, r, 4 * kk + 2 * (lane >> 5))));
      o.b.v = __builtin_bit_cast(Chunk<float>::vec, *reinterpret_cast<const f4*>(chunk(t, r, 4 * kk + 2 * (lane >> 5) + 1)));
    }
  }
};

// Rows of the contraction, R values of the operand's index each.
template <typename T, int R, int WAVES>
struct AcrossLds {
  static constexpr int kRow = R * sizeof(T), kLanes = kRow / 16, kRows = 64 / kLanes;       // rows of an instruction
  static constexpr int kBytes = kDeep<T> * kRow, Q = kBytes / 1024 / WAVES, kPer = 16 / sizeof(T);
  static_assert(kLanes <= 64 && kBytes % (1024 * WAVES) == 0);
  static __device__ __forceinline__ int row(int q, int wave, int lane) { return kRows * (q * WAVES + wave) + lane / kLanes; }
  // pairs of chunks stay together for the transpose loads of 4 rows of 32 bytes; the two halves of a
  // wave read float32 rows 8 apart from different banks
  static __device__ __forceinline__ int turn(int row) {
    return sizeof(T) == 4 ? (row >> 3 & 1) * 8 : kRow >= 256 ? 2 * (row & 7) : 2 * (row >> 1 & 3);
  }
  static __device__ __forceinline__ int first(int row, int lane) { return ((lane % kLanes) ^ turn(row)) * kPer; }
  static __device__ __forceinline__ uint8_t* place(uint8_t* t, int q, int wave) { return t + 1024 * (q * WAVES + wave); }
  static __device__ __forceinline__ const uint8_t* at(const uint8_t* t, int row, int col) {
    return t + row * kRow + ((col / kPer) ^ turn(row)) * 16 + col % kPer * sizeof(T);
  }
  static __device__ __forceinline__ void read(const uint8_t* t, int block, int kk, int lane, Octet<T>& o) {
    if constexpr (sizeof(T) == 2) {
      const int r = 16 * kk + 8 * (lane >> 5) + ((lane & 15) >> 2), c = 32 * block + 16 * (lane >> 4 & 1) + 4 * (lane & 3);
      const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at(t, r, c));
      const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at(t, r + 4, c));
      o.v.v = __builtin_bit_cast(Chunk<bf16_t>::vec, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = 16 * kk + 8 * (lane >> 5), c = 32 * block + (lane & 31);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o.a.v[j] = *reinterpret_cast<const float*>(at(t, r + j, c));
        o.b.v[j] = *reinterpret_cast<const float*>(at(t, r + 4 + j, c));
      }
    }
  }
};

// An octet as an operand.  FAR: an infinity stays one (split.hpp).
template <bool FAR>
__device__ __forceinline__ Frag<1> operand(const Octet<bf16_t>& o) {
  Frag<1> f;
  f.p[0] = __builtin_bit_cast(b8, o.v.v);
  return f;
}
template <bool FAR>
__device__ __forceinline__ Frag<3> operand(const Octet<float>& o) {
  Frag<3> f;
  const float x[8] = {o.at(0), o.at(1), o.at(2), o.at(3), o.at(4), o.at(5), o.at(6), o.at(7)};
  to_frag<FAR>(x, f);
  return f;
}

// The accumulators of a wave: MB x NB blocks of 32 x 32, C transposed (lane l holds row l % 32 of
// a block and columns 8 (i / 4) + 4 (l / 32) + i % 4).  In float32 a sum of thousands of products, six
// pieces each, would round more than their products do: what has come together in `part` goes to `all`
// every kTurn contraction values.
template <typename T, int MB, int NB>
struct Sums {
  static constexpr bool kTwo = sizeof(T) == 4;
  static constexpr int kTurn = 256;
  f16v part[MB][NB], all[kTwo ? MB : 1][kTwo ? NB : 1];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          part[i][j][r] = 0.f;
          if constexpr (kTwo) all[i][j][r] = 0.f;
        }
  }
  __device__ __forceinline__ void gather() {
    if constexpr (kTwo) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            all[i][j][r] += part[i][j][r];
            part[i][j][r] = 0.f;
          }
    }
  }
  __device__ __forceinline__ const f16v& total(int i, int j) const {
    if constexpr (kTwo)
      return all[i][j];
    else
      return part[i][j];
  }
  // the totals, 64 floats apart
  __device__ __forceinline__ void put(float* to) const {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) to[64 * (16 * (i * NB + j) + r)] = total(i, j)[r];
  }
  __device__ __forceinline__ void add(const float* from) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float x = from[64 * (16 * (i * NB + j) + r)];
          if constexpr (kTwo)
            all[i][j][r] += x;
          else
            part[i][j][r] += x;
        }
  }
  __device__ __forceinline__ bool finite() const {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) ok &= fabsf(total(i, j)[r]) < INFINITY;
    return ok;
  }
};

// One staged step's products.  bias: colsum[j] takes the sum of the wave's B operand.
template <typename T, typename TA, typename TB, int MB, int NB, bool FAR, bool BIAS = false>
__device__ __forceinline__ void multiply(const uint8_t* ta, const uint8_t* tb, int wm, int wn, int lane, Sums<T, MB, NB>& s,
                                         float* colsum = nullptr, bool bias = false) {
  constexpr int K = kDeep<T> / 16;
  if constexpr (sizeof(T) == 2) {
    // fragments are read one block row ahead of their products, which the compiler keeps in this order
    Octet<T> a, next, b[NB], after[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) TB::read(tb, wn * NB + j, 0, lane, b[j]);
    TA::read(ta, wm * MB, 0, lane, a);
#pragma unroll
    for (int kk = 0; kk < K; ++kk) {
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if (i + 1 < MB) {
          TA::read(ta, wm * MB + i + 1, kk, lane, next);
        } else if (kk + 1 < K) {
          TA::read(ta, wm * MB, kk + 1, lane, next);
        }
        if (i == 0 && kk + 1 < K) {
#pragma unroll
          for (int j = 0; j < NB; ++j) TB::read(tb, wn * NB + j, kk + 1, lane, after[j]);
        }
        if (BIAS && bias && i == 0) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) colsum[j] += b[j].at(e);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) s.part[i][j] = mma(operand<FAR>(b[j]), operand<FAR>(a), s.part[i][j]);
        __builtin_amdgcn_sched_barrier(0);
        a = next;
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) b[j] = after[j];
    }
  } else {
#pragma unroll
    for (int kk = 0; kk < K; ++kk) {
      Frag<kPlanes<T>> fb[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        Octet<T> o;
        TB::read(tb, wn * NB + j, kk, lane, o);
        if (BIAS && bias) {
#pragma unroll
          for (int e = 0; e < 8; ++e) colsum[j] += o.at(e);
        }
        fb[j] = operand<FAR>(o);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        Octet<T> o;
        TA::read(ta, wm * MB + i, kk, lane, o);
        const Frag<kPlanes<T>> fa = operand<FAR>(o);
#pragma unroll
        for (int j = 0; j < NB; ++j) s.part[i][j] = mma(fb[j], fa, s.part[i][j]);
      }
    }
  }
}

// All waves meet: what this one fetched, but for the last LATE loads, is in LDS, what it read has been
// read.  The fences are the wave's, for the compiler alone.
template <int LATE>
__device__ __forceinline__ void meet() {
  static_assert(LATE < 64);
  // vmcnt LATE (bits 0-3 and 14-15), lgkmcnt 0 (bits 8-11)
  __builtin_amdgcn_s_waitcnt(0x0070 | (LATE & 15) | (LATE >> 4) << 14);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The loop over the steps with D buffers: load(step, buffer) fetches, LOADS loads a wave, D - 1 steps
// ahead; product(step, buffer) multiplies.  Loads come back in order, so a step's are there when no more
// than those of the D - 2 steps behind it are out.  The buffers are separate arrays and take turns by
// name (buffer is a constant), so that the compiler sees that what is fetched is not what is read, and
// waits for nothing in between.
template <int D, int LOADS, typename Load, typename Product>
__device__ __forceinline__ void walk(int steps, Load&& load, Product&& product) {
  static_assert(D >= 2 && D <= 4);
  const std::integral_constant<int, 0> b0;
  const std::integral_constant<int, 1> b1;
  const std::integral_constant<int, 2> b2;
  const std::integral_constant<int, 3> b3;
  const auto pick = [&](auto i, auto&& f) {
    if constexpr (i() % D == 0) f(b0);
    if constexpr (i() % D == 1) f(b1);
    if constexpr (i() % D == 2) f(b2);
    if constexpr (i() % D == 3) f(b3);
  };
  // step t's loads are here; out are those of the D - 2 steps after it, where there are so many
  const auto ready = [&](int t) {
    if (t + D - 2 < steps)
      meet<(D - 2) * LOADS>();
    else
      meet<0>();
  };
  const auto turn = [&](auto i, int t, auto sure) {          // step t, in buffer i
    if (sure() || t + D - 1 < steps) pick(std::integral_constant<int, i() + D - 1>(), [&](auto b) { load(t + D - 1, b); });
    pick(i, [&](auto b) { product(t, b); });
    if constexpr (sure())
      meet<(D - 2) * LOADS>();
    else
      ready(t + 1);
  };
  if (steps <= 0) return;
  // While every step has a load to issue there are no conditions: the compiler counts loads too.
  int t = 0;
  load(0, b0);
  if (steps >= 2 * D - 1) {
    if constexpr (D > 2) load(1, b1);
    if constexpr (D > 3) load(2, b2);
    meet<(D - 2) * LOADS>();
    const std::true_type sure;
    do {
      turn(b0, t, sure);
      turn(b1, t + 1, sure);
      if constexpr (D > 2) turn(b2, t + 2, sure);
      if constexpr (D > 3) turn(b3, t + 3, sure);
      t += D;
    } while (t + 2 * D - 1 <= steps);
  } else {
    if constexpr (D > 2)
      if (steps > 1) load(1, b1);
    if constexpr (D > 3)
      if (steps > 2) load(2, b2);
    ready(0);
  }
  const std::false_type unsure;            // up to 2 D - 2 steps are left
  if (t < steps) turn(b0, t, unsure);
  if (t + 1 < steps) turn(b1, t + 1, unsure);
  if constexpr (D == 2) {
    // t + 2 = steps
  } else if constexpr (D == 3) {
    if (t + 2 < steps) turn(b2, t + 2, unsure);
    if (t + 3 < steps) turn(b0, t + 3, unsure);
  } else {
    if (t + 2 < steps) turn(b2, t + 2, unsure);
    if (t + 3 < steps) turn(b3, t + 3, unsure);
    if (t + 4 < steps) turn(b0, t + 4, unsure);
    if (t + 5 < steps) turn(b1, t + 5, unsure);
  }
}

// The buffers of a kernel by number, the tile of the first operand and behind it that of the second, and
// a wave's own part of them for hand_out.
template <int D, int A_BYTES, int BYTES>
struct Buffers {
  uint8_t *p0, *p1, *p2, *p3;
  template <typename I>
  __device__ __forceinline__ uint8_t* a(I) const {
    if constexpr (I() == 0) return p0;
    if constexpr (I() == 1) return p1;
    if constexpr (I() == 2) return p2;
    if constexpr (I() == 3) return p3;
  }
  template <typename I>
  __device__ __forceinline__ uint8_t* b(I i) const {
    return a(i) + A_BYTES;
  }
  template <int OWN, int WAVES>
  __device__ __forceinline__ float* own(int wave) const {
    constexpr int kEach = BYTES / OWN;
    static_assert(2 * kEach >= WAVES);
    return reinterpret_cast<float*>(wave < kEach ? p0 + wave * OWN : p1 + (wave - kEach) * OWN);
  }
};
// Each of KS `split`s of the contraction has buffers of its own.
#define TPC_BUFFERS(D, TA, TB, KS, split)                                                                                 \
  constexpr int kBuffer = TA::kBytes + TB::kBytes;                                                                        \
  __shared__ __attribute__((aligned(16))) uint8_t p0_[KS * kBuffer], p1_[KS * kBuffer], p2_[D > 2 ? KS * kBuffer : 16],   \
      p3_[D > 3 ? KS * kBuffer : 16];                                                                                     \
  const int mine_ = (split) * kBuffer;                                                                                    \
  const Buffers<D, TA::kBytes, kBuffer> buffers{p0_ + mine_, p1_ + mine_, p2_ + (D > 2 ? mine_ : 0), p3_ + (D > 3 ? mine_ : 0)}

// eight values, loaded and stored by the type's chunks; left: values there are
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, float* v) {
  constexpr int N = Chunk<T>::kN;
#pragma unroll
  for (int c = 0; c < 8; c += N) load_chunk(p + c, left - c, v + c);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int left, const float* v) {
  constexpr int N = Chunk<T>::kN;
#pragma unroll
  for (int c = 0; c < 8; c += N) store_chunk(p + c, left - c, v + c);
}

__device__ __forceinline__ void wave_in_order() {  // LDS accesses of a wave on its own stay in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Hands a wave's sums out as rows: out(row of the wave's blocks, first column of eight, values), by
// way of 32 x 32 NB float32 of LDS that are the wave's own, whose 16-byte chunks are permuted by the row.
template <typename T, int MB, int NB, typename Out>
__device__ __forceinline__ void hand_out(const Sums<T, MB, NB>& s, float* lds, int lane, Out&& out) {
  constexpr int C = 8 * NB, L = 4 * NB, R = 64 / L;           // chunks of a row, lanes of a row, rows at a time
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    wave_in_order();
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f16v& v = s.total(i, j);
        const int row = lane & 31, c = 8 * j + 2 * q + (lane >> 5);
        reinterpret_cast<f4*>(lds)[row * C + (c ^ (row & (C - 1)))] = f4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    wave_in_order();
#pragma unroll
    for (int p = 0; p < 32 / R; ++p) {
      const int row = p * R + lane / L, c = lane % L * 2;
      const f4 a = reinterpret_cast<const f4*>(lds)[row * C + (c ^ (row & (C - 1)))];
      const f4 b = reinterpret_cast<const f4*>(lds)[row * C + ((c + 1) ^ (row & (C - 1)))];
      float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      out(32 * i + row, 4 * c, v);
    }
  }
}

}  // namespace tpc
