// Counter-based random words for dropout: Philox 4x32 with 10 rounds (Salmon,
// Moraes, Dror and Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3", SC
// 2011).  A block of four 32-bit words is a pure function of (key, counter), so
// the backward draws the forward's words again and no mask is stored.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace tpc {

// a dropout as the kernels take it: word >= threshold keeps, factor = 1 / (1 - p)
struct DropArgs {
  uint32_t k0 = 0, k1 = 0;    // seed
  uint32_t o0 = 0, o1 = 0;    // offset
  uint32_t threshold = 0;
  float factor = 1.f;
};

// words 4 blk .. 4 blk + 3.  Two 32 x 32 -> 64 bit products a round (one
// instruction each), 20 in all: what bounds the dropout kernels in 16-bit types.
__device__ __forceinline__ void philox4(const DropArgs& d, uint64_t blk, uint32_t w[4]) {
  uint32_t c0 = (uint32_t)blk, c1 = (uint32_t)(blk >> 32), c2 = d.o0, c3 = d.o1;
  uint32_t k0 = d.k0, k1 = d.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0;
  w[1] = c1;
  w[2] = c2;
  w[3] = c3;
}

// which of the N words (a multiple of 4) from block blk on keep their elements.  A comparison's
// result stays in scalar registers, one bit a lane.
template <int N>
__device__ __forceinline__ void philox_keep(const DropArgs& d, uint64_t blk, bool keep[N]) {
#pragma unroll
  for (int b = 0; b < N / 4; ++b) {
    uint32_t w[4];
    philox4(d, blk + b, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) keep[4 * b + j] = w[j] >= d.threshold;
  }
}

}  // namespace tpc
