// Attention forward: out = softmax(scale q k^T + bias[bucket]) v per structure.
// One pass over the keys with a running maximum and sum per query (see attn.hpp
// for the tile layout); HG heads share the tile's distances and buckets.
//
// QW x KW waves: QW own 32 queries each, KW split the keys and are joined through
// LDS at the end (for batches with few query tiles).
#include "attn.hpp"

#include <algorithm>

namespace tpc {
namespace {

template <typename T, int KS, int HG, int NKV, int QW, int KW>
struct FwdShape {
  using G = Tile<T, KS>;
  static constexpr int kThreads = 64 * QW * KW, kRows = kTile * KW;
  using Stage = Stager<T, KS, kThreads, KW, NKV>;
  static constexpr int kPart = (G::MT * 16 + 2) * 64;                // floats of one wave's head to join
  static constexpr int kJoin = QW * (KW - 1) * HG * kPart * 4;
  static constexpr int kTileBytes = Stage::kBytes > kJoin ? Stage::kBytes : kJoin;
  static size_t lds_bytes(int nb) {
    return (size_t)kTileBytes + 12 * kRows + 16 * KW + (size_t)((nb > 0 ? nb : 1) + 1) * HG * 128;
  }
  // operands, accumulators and scores beside what the fetch holds
  static constexpr int kRegs = HG * (KS * G::P * 4 + G::MT * 16) + 60 + Stage::kChunks * (G::P == 1 ? 4 : 8);
};

template <typename T, int KS, int HG, int NKV, int QW, int KW>
__global__ void __launch_bounds__(64 * QW * KW, (FwdShape<T, KS, HG, NKV, QW, KW>::kRegs > 210 ? 1 : 2))
    k_attn_fwd(AttnArgs a) {
  using S = FwdShape<T, KS, HG, NKV, QW, KW>;
  using G = Tile<T, KS>;
  constexpr int P = G::P, MT = G::MT, NP = S::kRows;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  uint16_t* tiles = reinterpret_cast<uint16_t*>(lds);
  float* pos = reinterpret_cast<float*>(lds + S::kTileBytes);        // [3][NP]
  uint32_t* valid = reinterpret_cast<uint32_t*>(pos + 3 * NP);       // [KW], 16 bytes each
  float* tbl = reinterpret_cast<float*>(valid + 4 * KW);
  const tp_attn& d = a.d;
  int lo, hi, q0;
  if (!find_tile(d, kTile * QW, blockIdx.x, lo, hi, q0)) return;
  const int lane = threadIdx.x & 63, half = lane >> 5, wv = threadIdx.x >> 6;
  const int kw = wv % KW, qw = wv / KW;
  const int h0 = blockIdx.y * HG, rep = d.n_heads / d.n_kv_heads, D = d.head_dim;
  const bool biased = d.n_buckets > 0;
  fill_table<HG>(d, h0, tbl, S::kThreads);
  const Buckets<HG> bk(d, lane);

  // this lane's query
  const int q = q0 + 32 * qw + (lane & 31), qc = q < hi ? q : hi - 1;
  float x = 0.f, y = 0.f, z = 0.f;
  if (biased) {
    x = d.pos[3 * (size_t)qc];
    y = d.pos[3 * (size_t)qc + 1];
    z = d.pos[3 * (size_t)qc + 2];
  }
  Frag<P> Q[HG][KS];
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) own_rows<T, KS>(a.q, a.qs, qc, h0 + hh, D, half, true, Q[hh]);

  typename S::Stage st;
  PosStager<NP> ps;
  bool live = false;
  auto fetch = [&](int k0) {
    st.fetch(a.k, a.ks, a.v, a.vs, k0, hi, D, d.key_mask, [&](int slot) { return (h0 + slot) / rep; });
    if (biased) ps.fetch(d.pos, k0, hi);
    if ((int)threadIdx.x < NP) {
      const int k = k0 + threadIdx.x;
      live = k < hi && (!d.key_mask || d.key_mask[k] != 0);
    }
  };

  f16v O[HG][MT];
  float m[HG], l[HG];
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    m[hh] = kLowest;
    l[hh] = 0.f;
    clear<MT>(O[hh]);
  }
  const float c = d.scale * kLog2e;

  fetch(lo);
  for (int k0 = lo; k0 < hi; k0 += NP) {
    __syncthreads();                       // the previous step's tiles have been read
    st.stage(tiles);
    ps.stage(pos);
    const uint64_t vote = __ballot(live);
    if ((int)threadIdx.x < NP && (lane & 31) == 0) valid[4 * (threadIdx.x >> 5)] = (uint32_t)(vote >> (32 * half));
    __syncthreads();
    if (hi - k0 > NP) fetch(k0 + NP);
    if (32 * kw >= hi - k0) continue;      // this wave's tile lies past the end
    const uint32_t vm = __builtin_amdgcn_readfirstlane(valid[4 * kw]);
    if (vm == 0) continue;
    int off[16];
    tile_offsets<HG>(bk, biased, pos, NP, 32 * kw, half, x, y, z, off);
    if (vm != 0xffffffffu) mask_offsets<HG>(bk, vm, half, off);
#pragma unroll
    for (int hh = 0; hh < HG; ++hh) {
      const uint16_t* kt = tiles + (size_t)((kw * NKV + (NKV == 1 ? 0 : hh)) * 2) * G::kElems;
      f16v s;
      clear<1>(&s);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) s = mma(row_frag<T, KS>(kt, kk, lane), Q[hh][kk], s);
      float p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = fmaf(s[i], c, table(tbl, off[i], hh));
      float tm = fmaxf(p[0], p[1]);
#pragma unroll
      for (int i = 2; i < 16; ++i) tm = fmaxf(tm, p[i]);
      tm = pair_max(tm);
      // the maximum follows in steps of at least 2^8: probabilities up to 2^8 lose nothing,
      // and the accumulators are rescaled in few tiles
      if (__any(tm > m[hh] + 8.f)) {
        const float mn = fmaxf(m[hh], tm), f = __builtin_amdgcn_exp2f(m[hh] - mn);
        m[hh] = mn;
        l[hh] *= f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 16; ++i) O[hh][mt][i] *= f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = __builtin_amdgcn_exp2f(p[i] - m[hh]);
        l[hh] += p[i];
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Frag<P> pf;
        to_frag(p + 8 * kb, pf);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) O[hh][mt] = mma(col_frag<T, KS>(kt + G::kElems, mt, kb, lane), pf, O[hh][mt]);
      }
    }
  }

  if (KW > 1) {
    float* join = reinterpret_cast<float*>(lds) + (size_t)qw * (KW - 1) * HG * S::kPart + lane;
    __syncthreads();
    if (kw > 0) {
#pragma unroll
      for (int hh = 0; hh < HG; ++hh) {
        float* w = join + ((kw - 1) * HG + hh) * S::kPart;
        w[0] = m[hh];
        w[64] = l[hh];
        park<MT>(w + 128, O[hh]);
      }
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int hh = 0; hh < HG; ++hh)
      for (int o = 0; o < KW - 1; ++o) {
        const float* w = join + (o * HG + hh) * S::kPart;
        const float mn = fmaxf(m[hh], w[0]);
        const float f = __builtin_amdgcn_exp2f(m[hh] - mn), g = __builtin_amdgcn_exp2f(w[0] - mn);
        m[hh] = mn;
        l[hh] = l[hh] * f + w[64] * g;
        add_parked<MT>(w + 128, f, g, O[hh]);
      }
  }
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    const float sum = pair_sum(l[hh]);
    if (q < hi) {
      const bool none = sum == 0.f;        // NaN is not none: it has to show
      if (a.lse && half == 0)
        a.lse[(size_t)(h0 + hh) * d.n_nodes + q] = none ? -INFINITY : (m[hh] + __builtin_amdgcn_logf(sum)) * kLn2;
      store_rows<T, MT>(a.out, a.os, q, h0 + hh, D, half, O[hh], 1.f / sum, none);
    }
  }
}

template <typename T, int KS, int HG, int NKV, int QW, int KW>
hipError_t launch(const AttnArgs& a) {
  using S = FwdShape<T, KS, HG, NKV, QW, KW>;
  const dim3 grid((unsigned)(a.d.n_nodes / (kTile * QW) + a.d.n_segments), (unsigned)(a.d.n_heads / HG));
  return launch_lds(k_attn_fwd<T, KS, HG, NKV, QW, KW>, grid, S::kThreads, S::lds_bytes(a.d.n_buckets), a.stream, a);
}

template <typename T, int KS, int HG, int NKV>
hipError_t by_waves(const AttnArgs& a) {
  // tiles of 32 queries and heads: where they fill the chip, four query tiles share
  // the staged keys; else the waves split the keys of one tile, as far as LDS holds
  // the tiles
  constexpr int pair = Tile<T, KS>::kElems * 4 * NKV;
  constexpr int KW = pair * 4 <= 96 * 1024 ? 4 : 2;
  const int64_t tiles = ((int64_t)a.d.n_nodes / kTile + a.d.n_segments) * (a.d.n_heads / HG);
  const int64_t mean = a.d.n_nodes / std::max(1, a.d.n_segments);
  if (mean > 64 && tiles >= 4096) return launch<T, KS, HG, NKV, 4, 1>(a);
  if (mean > 64) return launch<T, KS, HG, NKV, 1, KW>(a);
  return launch<T, KS, HG, NKV, 1, 1>(a);
}

template <typename T, int KS>
hipError_t by_heads(const AttnArgs& a) {
  constexpr bool pairs = kPlanes<T> * KS <= 6;      // operands of two heads fit the registers
  const int rep = a.d.n_heads / a.d.n_kv_heads;
  if constexpr (pairs) {
    if (rep % 2 == 0) return by_waves<T, KS, 2, 1>(a);
    if (rep == 1 && a.d.n_heads % 2 == 0) return by_waves<T, KS, 2, 2>(a);
  }
  return by_waves<T, KS, 1, 1>(a);
}

template <typename T>
hipError_t by_width(const AttnArgs& a) {
  const int ks = (a.d.head_dim + 15) / 16;
  if (ks <= 1) return by_heads<T, 1>(a);
  if (ks <= 2) return by_heads<T, 2>(a);
  if (ks <= 3) return by_heads<T, 3>(a);
  if (ks <= 4) return by_heads<T, 4>(a);
  if (ks <= 6) return by_heads<T, 6>(a);
  return by_heads<T, 8>(a);
}

}  // namespace

hipError_t attn_forward(const AttnArgs& a) { return a.d.dtype == TP_F32 ? by_width<float>(a) : by_width<bf16_t>(a); }

}  // namespace tpc
