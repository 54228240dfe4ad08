// Row access shared by the norm and dropout kernels: 16-byte chunks of float32 or
// bfloat16 at element alignment, widened to float32.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace tpc {

typedef __bf16 bf16_t;

// Rows of odd length start at any element, so the vector types ask for the
// element's alignment only; the hardware loads 16 bytes from any address.
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  static constexpr int kN = 4;
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Chunk<bf16_t> {
  static constexpr int kN = 8;
  typedef __bf16 vec __attribute__((ext_vector_type(8), aligned(2)));
};

// o[0..kN) = the chunk at p; entries from `left` on (past the row's end) are 0 and not read
template <typename T>
__device__ __forceinline__ void load_chunk(const T* p, int left, float* o) {
  constexpr int N = Chunk<T>::kN;
  if (left >= N) {
    const typename Chunk<T>::vec v = *reinterpret_cast<const typename Chunk<T>::vec*>(p);
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = (float)v[j];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = j < left ? (float)p[j] : 0.f;
  }
}

// the same as loaded: a chunk held for a row to come, widened when its turn comes
template <typename T>
struct RawChunk {
  typename Chunk<T>::vec v;
  __device__ __forceinline__ void load(const T* p, int left) {
    constexpr int N = Chunk<T>::kN;
    if (left >= N) {
      v = *reinterpret_cast<const typename Chunk<T>::vec*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = j < left ? p[j] : (T)0.f;
    }
  }
  __device__ __forceinline__ float at(int j) const { return (float)v[j]; }
};

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, int left, const float* o) {
  constexpr int N = Chunk<T>::kN;
  if (left >= N) {
    typename Chunk<T>::vec v;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = (T)o[j];
    *reinterpret_cast<typename Chunk<T>::vec*>(p) = v;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < left) p[j] = (T)o[j];
  }
}

}  // namespace tpc
