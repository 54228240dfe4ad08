// Matrix-core operands shared by attention and the products by group: fragments of eight
// bfloat16 values a lane, and float32 values as three of them.
//
// float32 operands are split exactly into three bfloat16 pieces, x = hi + mid + lo
// (8 + 8 + 8 significand bits, taken by truncation: |mid| < 2^-7 |x|, |lo| < 2^-15 |x|), and a
// product is the six partial products down to 2^-16 relative.  What is left out, mid lo + lo mid
// + lo lo, is below 2^-21 of a product, always towards zero; 0.7 2^-24 on average over normal
// operands.  Pieces rounded to nearest would leave out 2^-24 at most, of either sign, but take 2
// to 6 % longer (4,096 atoms, 4 heads of 64, step: 609 against 572 us), and the sums' own
// rounding is of the same size: outputs are 0.6 to 1.9, gradients 0.7 to 1.7 times as far from
// 64 bits as float32 arithmetic brings them (60 to 2,000 atoms).  Six bfloat16 MFMA cost 192
// cycles per 32x32x16 against 512 for the float32 MFMA.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "rows.hpp"

namespace tpc {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4 lds_s4;

template <typename T>
constexpr int kPlanes = std::is_same<T, float>::value ? 3 : 1;

template <int P>
struct Frag {
  b8 p[P];
};

template <bool SWAPPED = false>
__device__ __forceinline__ f16v mma(const Frag<1>& a, const Frag<1>& b, f16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}
// Smallest partial products first.  SWAPPED takes the same products in the same order with
// the operands exchanged, so that the key side of the backward forms bit for bit the
// scores of the query side: its row sums then cancel.
template <bool SWAPPED = false>
__device__ __forceinline__ f16v mma(const Frag<3>& a, const Frag<3>& b, f16v c) {
  constexpr int f = SWAPPED ? 2 : 0, g = SWAPPED ? 1 : 0;
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[f], b.p[2 - f], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2 - f], b.p[f], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[g], b.p[1 - g], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1 - g], b.p[g], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float flt(uint32_t x) { return __builtin_bit_cast(float, x); }
// the upper halves of two words, the first in the low half
__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// eight float32 values as an operand: one rounding (bfloat16) or the exact split
__device__ __forceinline__ void to_frag(const float* x, Frag<1>& f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f.p[0][j] = (__bf16)x[j];
}
// FAR: an infinity is split into (largest bfloat16, the same, infinity), not into infinity and NaN,
// so that its products are infinite whatever the other operand's pieces are.
template <bool FAR = false>
__device__ __forceinline__ void to_frag(const float* x, Frag<3>& f) {
  const auto upper = [](float v) {
    return bits(FAR ? __builtin_amdgcn_fmed3f(v, -0x1.fep+127f, 0x1.fep+127f) : v) & 0xffff0000u;
  };
  u4 h, m, l;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = x[2 * j], b = x[2 * j + 1];
    const uint32_t ha = upper(a), hb = upper(b);
    const float ra = a - flt(ha), rb = b - flt(hb);
    const uint32_t ma = upper(ra), mb = upper(rb);
    const float sa = ra - flt(ma), sb = rb - flt(mb);
    h[j] = FAR ? high_halves(ha, hb) : high_halves(bits(a), bits(b));
    m[j] = FAR ? high_halves(ma, mb) : high_halves(bits(ra), bits(rb));
    l[j] = high_halves(bits(sa), bits(sb));          // at most 8 bits left: exact
  }
  f.p[0] = __builtin_bit_cast(b8, h);
  f.p[1] = __builtin_bit_cast(b8, m);
  f.p[2] = __builtin_bit_cast(b8, l);
}

}  // namespace tpc
