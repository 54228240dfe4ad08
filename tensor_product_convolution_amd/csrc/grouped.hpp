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
  __device__ __forceinline__ void load(const bf16_t* p) { v.v = *reinterpret_cast<const Chunk<bf16_t>::vec*>(p); }
  __device__ __forceinline__ void keep(bool k) {
    u4 b = __builtin_bit_cast(u4, v.v);
    b = k ? b : u4{0, 0, 0, 0};
    v.v = __builtin_bit_cast(Chunk<bf16_t>::vec, b);
  }
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
  __device__ __forceinline__ void load(const float* p) {
    a.v = *reinterpret_cast<const Chunk<float>::vec*>(p);
    b.v = *reinterpret_cast<const Chunk<float>::vec*>(p + 4);
  }
  __device__ __forceinline__ void keep(bool k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a.v[j] = k ? a.v[j] : 0.f;
      b.v[j] = k ? b.v[j] : 0.f;
    }
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

// Part t of the groups cut into parts of `size` slots: group e's parts start at number
// ptr[e] / size + e, which never overlap and leave at most one unused number per group, so
// n / size + groups numbers cover any groups without the host knowing them.  Looked up 64
// groups at a time.  `groups` counts the one behind the last pointer (slots without a group),
// which ends at n.  False: an unused number, but for the first of an empty group.
struct Part {
  int group, lo, hi, first;                // slots of the group, first slot of the part
};
__device__ __forceinline__ bool find_part(const int32_t* ptr, int groups, int n, int size, int t, Part& p) {
  const int lane = threadIdx.x & 63;
  const auto start = [&](int e) { return min(max(ptr[e], 0), n); };
  int b = 0, left = groups;
  while (left > 1) {
    const int step = (left + 63) >> 6, at = b + lane * step;
    const bool le = lane * step < left && start(at) / size + at <= t;
    const int cnt = __popcll(__ballot(le));
    if (cnt == 0) return false;            // not a valid ptr
    b += (cnt - 1) * step;
    left = min(step, left - (cnt - 1) * step);
  }
  p.group = __builtin_amdgcn_readfirstlane(b);
  p.lo = start(p.group);
  p.hi = p.group + 1 < groups ? start(p.group + 1) : n;
  const int64_t first = (int64_t)p.lo + (int64_t)(t - (p.lo / size + p.group)) * size;
  p.first = (int)min(first, (int64_t)n);
  return first == p.lo || (first > p.lo && first < p.hi);
}

// the row of a slot: itself, or rows[slot] / div
__device__ __forceinline__ int row_of(const int32_t* rows, int slot, int div, int n) {
  if (div == 0) return slot;
  const uint32_t r = min((uint32_t)rows[slot], (uint32_t)(n - 1));
  return (int)(div == 1 ? r : r / (uint32_t)div);
}

// Places of the tiles rows x cols in the order of the launch.  Workgroups go round the 8 dies in
// turn; each die gets a run of consecutive tiles, 8 row tiles by all columns at a time, so that
// what it reads of both operands stays in its L2.
__device__ __forceinline__ void place_tile(int id, int rows, int cols, int& r, int& c) {
  constexpr int kDies = 8, kBand = 8;
  const int total = rows * cols, whole = total / kDies, more = total % kDies, die = id % kDies;
  const int t = die * whole + min(die, more) + id / kDies;
  const int band = t / (kBand * cols), first = band * kBand, high = min(kBand, rows - first), in = t - first * cols;
  r = first + in % high;
  c = in / high;
}

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }
__device__ __forceinline__ float silu_slope(float z) {
  const float s = 1.f / (1.f + expf(-z));
  return s * (1.f + z * (1.f - s));
}

}  // namespace tpc
