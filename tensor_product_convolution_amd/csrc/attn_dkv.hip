// Attention backward, key side: grad_k, grad_v and the bias gradient.
//
//   grad_v = p^T grad_out,  grad_k = scale ds^T q,  summed over the query heads of a
//   key head;  grad_bias[bucket] += ds;  p = exp(s - lse), ds = p (grad_out v^T - delta)
//
// A wave owns 32 keys of NKV key heads and walks the queries in tiles, HG query heads
// at a time (HG heads of one key head, or HG key heads with one query head each).
// KV x QS waves: KV own 32 keys each, QS split the queries and are joined through
// LDS at the end.
//
// The bias gradient goes into LDS columns private to the lane (no two lanes add to
// one word, so the order of the sums is fixed), summed per workgroup and joined by
// a second kernel.
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
  static size_t lds_bytes(int nb, bool grad) {
    const size_t entries = (nb > 0 ? nb : 1) + 1;
    return (size_t)kTileBytes + 12 * kRows + 8 * HG * kRows + entries * HG * 128 +
           (grad ? (size_t)KV * QS * entries * HG * 256 : 0);
  }
  static constexpr int kRegs = NKV * (2 * KS * G::P * 4 + 2 * G::MT * 16) + 76 + Stage::kChunks * (G::P == 1 ? 4 : 8);
};

template <typename T, int KS, int HG, int NKV, int KV, int QS>
__global__ void __launch_bounds__(64 * KV * QS, (DkvShape<T, KS, HG, NKV, KV, QS>::kRegs > 220 ? 1 : 2))
    k_attn_dkv(AttnArgs a) {
  using S = DkvShape<T, KS, HG, NKV, KV, QS>;
  using G = Tile<T, KS>;
  constexpr int P = G::P, MT = G::MT, NP = S::kRows, NW = KV * QS;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  uint16_t* tiles = reinterpret_cast<uint16_t*>(lds);
  float* pos = reinterpret_cast<float*>(lds + S::kTileBytes);       // [3][NP]
  float* stat = pos + 3 * NP;                                       // [HG][2][NP]: lse (base 2), delta
  float* tbl = stat + 2 * HG * NP;
  const tp_attn& d = a.d;
  const int nb = d.n_buckets, ne = (nb > 0 ? nb : 1) + 1;
  float* cols = tbl + ne * HG * 32;        // [NW][ne][HG][64] bias gradient columns
  const int g0 = blockIdx.y * NKV, rep = d.n_heads / d.n_kv_heads, D = d.head_dim;
  const int h_lo = g0 * rep, h_hi = (g0 + NKV) * rep;
  int lo, hi, k0;
  if (!find_tile(d, kTile * KV, blockIdx.x, lo, hi, k0)) {
    if (a.gbias)
      for (int i = threadIdx.x; i < (h_hi - h_lo) * nb; i += S::kThreads)
        a.part[((size_t)(h_lo + i / nb) * gridDim.x + blockIdx.x) * nb + i % nb] = 0.f;
    return;
  }
  const int lane = threadIdx.x & 63, half = lane >> 5, wv = threadIdx.x >> 6;
  const int qs = wv % QS, kv = wv / QS;
  const bool biased = nb > 0;
  const Buckets<HG> bk(d, lane);

  // this lane's key; a masked one is held as zeros and gets zero gradients
  const int k = k0 + 32 * kv + (lane & 31), kc = k < hi ? k : hi - 1;
  const bool live = k < hi && (!d.key_mask || d.key_mask[kc] != 0);
  const bool some_dead = __any(!live);
  // table offset -> byte offset of the lane's column of the same entry (twice as wide)
  char* mycol = reinterpret_cast<char*>(cols + (size_t)wv * ne * HG * 64) + 4 * lane - 8 * (lane & 31);
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
  fetch(h_lo, lo);
  for (int h0 = h_lo; h0 < h_hi; h0 += HG) {
    __syncthreads();
    fill_table<HG>(d, h0, tbl, S::kThreads);
    if (a.gbias)
      for (int i = threadIdx.x; i < NW * ne * HG * 64; i += S::kThreads) cols[i] = 0.f;
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
      tile_offsets<HG>(bk, biased, pos, NP, 32 * qs, half, x, y, z, off);
      if (some_dead) mask_offsets<HG>(bk, live ? 0xffffffffu : 0u, half, off);
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
        if (a.gbias) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            __hip_atomic_fetch_add(reinterpret_cast<float*>(mycol + 2 * off[i] + hh * 256), ds[i], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_WORKGROUP);
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
    if (a.gbias) {
      // an entry's 64 columns of every wave; lanes start at different columns so that
      // they read different banks
      __syncthreads();
      for (int i = threadIdx.x; i < nb * HG; i += S::kThreads) {
        const int b = i / HG, hh = i % HG;
        float s = 0.f;
        for (int w = 0; w < NW; ++w)
#pragma unroll 8
          for (int j = 0; j < 64; ++j) s += cols[((size_t)(w * ne + b) * HG + hh) * 64 + ((j + lane) & 63)];
        a.part[((size_t)(h0 + hh) * gridDim.x + blockIdx.x) * nb + b] = s;
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

// grad_bias[h][b] = sum over the tiles' parts, in a fixed order.
constexpr int kJoinThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    k_attn_join_bias(const float* __restrict__ part, int n, int nb, T* __restrict__ out) {
  __shared__ float lds[kJoinThreads];
  const int h = blockIdx.x, b = threadIdx.x & 63, g = threadIdx.x >> 6;
  float s = 0.f;
  if (b < nb) {
#pragma unroll 8
    for (int t = g; t < n; t += kJoinThreads / 64) s += part[((size_t)h * n + t) * nb + b];
  }
  lds[threadIdx.x] = s;
#pragma unroll
  for (int m = kJoinThreads / 2; m >= 64; m >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < m) lds[threadIdx.x] += lds[threadIdx.x + m];
  }
  if (g == 0 && b < nb) out[(size_t)h * nb + b] = (T)lds[b];
}

template <typename T>
hipError_t join_bias(const AttnArgs& a, int parts) {
  hipLaunchKernelGGL(k_attn_join_bias<T>, dim3(a.d.n_heads), dim3(kJoinThreads), 0, a.stream, a.part, parts,
                     a.d.n_buckets, static_cast<T*>(a.gbias));
  return hipGetLastError();
}

template <typename T, int KS, int HG, int NKV, int KV, int QS>
hipError_t launch(const AttnArgs& a) {
  using S = DkvShape<T, KS, HG, NKV, KV, QS>;
  const int tiles = a.d.n_nodes / (kTile * KV) + a.d.n_segments;
  hipError_t e = launch_lds(k_attn_dkv<T, KS, HG, NKV, KV, QS>, dim3(tiles, a.d.n_kv_heads / NKV), S::kThreads,
                            S::lds_bytes(a.d.n_buckets, a.gbias != nullptr), a.stream, a);
  return e != hipSuccess || !a.gbias ? e : join_bias<T>(a, tiles);
}

template <typename T, int KS, int HG, int NKV>
hipError_t by_waves(const AttnArgs& a) {
  constexpr int pair = Tile<T, KS>::kElems * 4 * HG;
  constexpr int QS = pair * 4 <= 64 * 1024 ? 4 : 2;
  const int64_t tiles = ((int64_t)a.d.n_nodes / kTile + a.d.n_segments) * (a.d.n_kv_heads / NKV);
  const int64_t mean = a.d.n_nodes / std::max(1, a.d.n_segments);
  const auto fits = [&](size_t bytes) { return bytes <= kLdsMax; };
  if (mean > 64 && tiles >= 4096 && fits(DkvShape<T, KS, HG, NKV, 4, 1>::lds_bytes(a.d.n_buckets, a.gbias != nullptr)))
    return launch<T, KS, HG, NKV, 4, 1>(a);
  if (mean > 64 && fits(DkvShape<T, KS, HG, NKV, 1, QS>::lds_bytes(a.d.n_buckets, a.gbias != nullptr)))
    return launch<T, KS, HG, NKV, 1, QS>(a);
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
  if (a.d.n_nodes == 0) return a.d.dtype == TP_F32 ? join_bias<float>(a, 0) : join_bias<bf16_t>(a, 0);
  hipError_t e = attn_backward_q(a);       // also leaves delta for the key side
  if (e != hipSuccess) return e;
  return a.d.dtype == TP_F32 ? by_width<float>(a) : by_width<bf16_t>(a);
}

size_t attn_delta_floats(const tp_attn& d) { return ((size_t)d.n_heads * d.n_nodes + 3) / 4 * 4; }
size_t attn_part_floats(const tp_attn& d) {
  return ((size_t)d.n_nodes / kTile + d.n_segments) * d.n_heads * d.n_buckets;
}

}  // namespace tpc
