// Attention backward, key side: grad_k and grad_v.
//
//   grad_v = p^T grad_out,  grad_k = scale ds^T q,  summed over the query heads of a
//   key head;  p = exp(s - lse), ds = p (grad_out v^T - delta)
//
// A wave owns 32 keys of NKV key heads and walks the queries in tiles, HG query heads
// at a time (HG heads of one key head, or HG key heads with one query head each).
// KV x QS waves: KV own 32 keys each, QS split the queries and are joined through
// LDS at the end.
#include "attn.hpp"

#include <algorithm>

namespace tpc {
namespace {

template <typename T, int KS, int HG, int NKV, int KV, int QS>
struct DkvShape {
  using G = Tile<T, KS>;
  static constexpr int kThreads = 64 * KV * QS, kRows = kTile * QS;
  using Stage = Stager<T, KS, kThreads, QS, HG>;
  static constexpr int kPart = G::MT * 16 * 64 * 2;
  static constexpr int kJoin = KV * (QS - 1) * NKV * kPart * 4;
  static constexpr int kTileBytes = Stage::kBytes > kJoin ? Stage::kBytes : kJoin;
  static size_t lds_bytes(int nb) {
    return (size_t)kTileBytes + 12 * kRows + 8 * HG * kRows + (size_t)((nb > 0 ? nb : 1) + 1) * HG * 128;
  }
  static constexpr int kRegs = NKV * (2 * KS * G::P * 4 + 2 * G::MT * 16) + 76 + Stage::kChunks * (G::P == 1 ? 4 : 8);
};

template <typename T, int KS, int HG, int NKV, int KV, int QS>
__global__ void __launch_bounds__(64 * KV * QS, (DkvShape<T, KS, HG, NKV, KV, QS>::kRegs > 220 ? 1 : 2))
    k_attn_dkv(AttnArgs a) {
  using S = DkvShape<T, KS, HG, NKV, KV, QS>;
  using G = Tile<T, KS>;
  constexpr int P = G::P, MT = G::MT, NP = S::kRows;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  uint16_t* tiles = reinterpret_cast<uint16_t*>(lds);
  float* pos = reinterpret_cast<float*>(lds + S::kTileBytes);       // [3][NP]
  float* stat = pos + 3 * NP;                                       // [HG][2][NP]: lse (base 2), delta
  float* tbl = stat + 2 * HG * NP;
  const tp_attn& d = a.d;
  int lo, hi, k0;
  if (!find_tile(d, kTile * KV, blockIdx.x, lo, hi, k0)) return;
  const int lane = threadIdx.x & 63, half = lane >> 5, wv = threadIdx.x >> 6;
  const int qs = wv % QS, kv = wv / QS;
  const int g0 = blockIdx.y * NKV, rep = d.n_heads / d.n_kv_heads, D = d.head_dim;
  const bool biased = d.n_buckets > 0;
  const Buckets<HG> bk(d, lane);

  // this lane's key; a masked one is held as zeros and gets zero gradients
  const int k = k0 + 32 * kv + (lane & 31), kc = k < hi ? k : hi - 1;
  const bool live = !d.key_mask || d.key_mask[kc] != 0;
  float x = 0.f, y = 0.f, z = 0.f;
  if (biased) {
    x = d.pos[3 * (size_t)kc];
    y = d.pos[3 * (size_t)kc + 1];
    z = d.pos[3 * (size_t)kc + 2];
  }
  Frag<P> K[NKV][KS], V[NKV][KS];
  f16v dK[NKV][MT], dV[NKV][MT];
#pragma unroll
  for (int s = 0; s < NKV; ++s) {
    own_rows<T, KS>(a.k, a.ks, kc, g0 + s, D, half, live, K[s]);
    own_rows<T, KS>(a.v, a.vs, kc, g0 + s, D, half, live, V[s]);
    clear<MT>(dK[s]);
    clear<MT>(dV[s]);
  }
  const float c = d.scale * kLog2e;

  // steps: query heads of the key head, HG at a time, outside; query tiles inside
  typename S::Stage st;
  PosStager<NP> ps;
  float slse[HG], sdel[HG];
  auto fetch = [&](int h0, int q0) {
    st.fetch(a.q, a.qs, a.go, a.gos, q0, hi, D, nullptr, [&](int slot) { return h0 + slot; });
    if (biased) ps.fetch(d.pos, q0, hi);
    if ((int)threadIdx.x < NP) {
      const int q = q0 + threadIdx.x;
#pragma unroll
      for (int hh = 0; hh < HG; ++hh) {
        const size_t at = (size_t)(h0 + hh) * d.n_nodes + min(q, hi - 1);
        const float e = a.lse_in[at];
        slse[hh] = q < hi && e != -INFINITY ? e * kLog2e : INFINITY;
        sdel[hh] = q < hi ? a.delta[at] : 0.f;
      }
    }
  };
  const int h_lo = g0 * rep, h_hi = (g0 + NKV) * rep;
  fetch(h_lo, lo);
  for (int h0 = h_lo; h0 < h_hi; h0 += HG) {
    __syncthreads();
    fill_table<HG>(d, h0, tbl, S::kThreads);
    for (int q0 = lo; q0 < hi; q0 += NP) {
      __syncthreads();
      st.stage(tiles);
      ps.stage(pos);
      if ((int)threadIdx.x < NP) {
#pragma unroll
        for (int hh = 0; hh < HG; ++hh) {
          stat[(2 * hh) * NP + threadIdx.x] = slse[hh];
          stat[(2 * hh + 1) * NP + threadIdx.x] = sdel[hh];
        }
      }
      __syncthreads();
      if (hi - q0 > NP) fetch(h0, q0 + NP);
      else if (h0 + HG < h_hi) fetch(h0 + HG, lo);
      if (32 * qs >= hi - q0) continue;
      int off[16];
      tile_offsets<HG>(bk, biased, pos, NP, 32 * qs, half, x, y, z, 0xffffffffu, off);
#pragma unroll
      for (int hh = 0; hh < HG; ++hh) {
        const int s_ = NKV == 1 ? 0 : hh;
        const uint16_t* qt = tiles + (size_t)((qs * HG + hh) * 2) * G::kElems;
        f16v s, dp;
        clear<1>(&s);
        clear<1>(&dp);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) s = mma(row_frag<T, KS>(qt, kk, lane), K[s_][kk], s);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) dp = mma(row_frag<T, KS>(qt + G::kElems, kk, lane), V[s_][kk], dp);
        float p[16], ds[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = 32 * qs + 8 * g + 4 * half;
          const f4 le = *reinterpret_cast<const f4*>(stat + (2 * hh) * NP + r);
          const f4 de = *reinterpret_cast<const f4*>(stat + (2 * hh + 1) * NP + r);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 4 * g + j;
            p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, table(tbl, off[i], hh)) - le[j]);
            ds[i] = p[i] * (dp[i] - de[j]);
          }
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          Frag<P> pf, df;
          to_frag(p + 8 * kb, pf);
          to_frag(ds + 8 * kb, df);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            dV[s_][mt] = mma(col_frag<T, KS>(qt + G::kElems, mt, kb, lane), pf, dV[s_][mt]);
            dK[s_][mt] = mma(col_frag<T, KS>(qt, mt, kb, lane), df, dK[s_][mt]);
          }
        }
      }
    }
  }

  if (QS > 1) {
    float* join = reinterpret_cast<float*>(lds) + (size_t)kv * (QS - 1) * NKV * S::kPart + lane;
    __syncthreads();
    if (qs > 0) {
#pragma unroll
      for (int s = 0; s < NKV; ++s) {
        float* w = join + ((qs - 1) * NKV + s) * S::kPart;
        park<MT>(w, dK[s]);
        park<MT>(w + S::kPart / 2, dV[s]);
      }
    }
    __syncthreads();
    if (qs > 0) return;
#pragma unroll
    for (int s = 0; s < NKV; ++s)
      for (int o = 0; o < QS - 1; ++o) {
        const float* w = join + (o * NKV + s) * S::kPart;
        add_parked<MT>(w, 1.f, 1.f, dK[s]);
        add_parked<MT>(w + S::kPart / 2, 1.f, 1.f, dV[s]);
      }
  }
  if (k < hi) {
#pragma unroll
    for (int s = 0; s < NKV; ++s) {
      store_rows<T, MT>(a.gk, a.gks, k, g0 + s, D, half, dK[s], d.scale, !live);
      store_rows<T, MT>(a.gv, a.gvs, k, g0 + s, D, half, dV[s], 1.f, !live);
    }
  }
}

template <typename T, int KS, int HG, int NKV, int KV, int QS>
hipError_t launch(const AttnArgs& a) {
  using S = DkvShape<T, KS, HG, NKV, KV, QS>;
  const dim3 grid((unsigned)(a.d.n_nodes / (kTile * KV) + a.d.n_segments), (unsigned)(a.d.n_kv_heads / NKV));
  return launch_lds(k_attn_dkv<T, KS, HG, NKV, KV, QS>, grid, S::kThreads, S::lds_bytes(a.d.n_buckets), a.stream, a);
}

template <typename T, int KS, int HG, int NKV>
hipError_t by_waves(const AttnArgs& a) {
  constexpr int pair = Tile<T, KS>::kElems * 4 * HG;
  constexpr int QS = pair * 4 <= 96 * 1024 ? 4 : 2;
  const int64_t tiles = ((int64_t)a.d.n_nodes / kTile + a.d.n_segments) * (a.d.n_kv_heads / NKV);
  const int64_t mean = a.d.n_nodes / std::max(1, a.d.n_segments);
  if (mean > 64 && tiles >= 4096) return launch<T, KS, HG, NKV, 4, 1>(a);
  if (mean > 64) return launch<T, KS, HG, NKV, 1, QS>(a);
  return launch<T, KS, HG, NKV, 1, 1>(a);
}

template <typename T, int KS>
hipError_t by_heads(const AttnArgs& a) {
  const int rep = a.d.n_heads / a.d.n_kv_heads;
  if constexpr (kPlanes<T> * KS <= 4) {
    if (rep % 2 == 0) return by_waves<T, KS, 2, 1>(a);
    if constexpr (KS <= 2)
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

hipError_t attn_backward(const AttnArgs& a) {
  hipError_t e = attn_backward_q(a);       // also leaves delta for the key side
  if (e != hipSuccess || a.d.n_nodes == 0) return e;
  return a.d.dtype == TP_F32 ? by_width<float>(a) : by_width<bf16_t>(a);
}

}  // namespace tpc
