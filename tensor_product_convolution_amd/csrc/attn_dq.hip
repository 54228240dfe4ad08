// Attention backward, query side: grad_q, and delta for the key side.
//
//   p = exp(s - lse),  dp = grad_out v^T,  ds = p (dp - delta),  grad_q = scale ds k,
//   delta = grad_out . out
//
// A wave owns 32 queries and walks the keys as the forward does, with delta formed
// from its own rows.  That delta carries the rounding of out (and the products
// theirs), so a row of ds does not quite sum to zero.  The bias gradient of a bucket
// that holds most pairs, a sum of millions of terms that nearly cancel, came out
// 5e-3 (bfloat16) and 2e-5 (float32) off at 1,536 atoms.  So the row sums
// r = sum_j ds_ij are kept too, and the key side, which forms ds again, takes
// delta + r.  In bfloat16 grad_q of short rows notices as well (structures of 62 atoms:
// 2.5e-3 off against 2.4e-3), so p k is summed beside ds k and r p k taken off at the end.
//
// bfloat16 rounds p and ds to the type for their products, as the forward does, for the same
// reason; r sums the unrounded ds.
//
// Bound as the forward is (vector units 40 % busy, latency of the rest).  1,536 atoms, 8 heads: of 32, bfloat16 26 us, of
// 16, float32 34 us; 4,096 atoms, 4 heads of 64, float32: 187 us.
#include "attn.hpp"

namespace tpc {
namespace {

template <typename T, int KS, int HG, int NKV, int QW, int KW>
struct DqShape {
  using G = Tile<T, KS>;
  static constexpr int kThreads = 64 * QW * KW;
  using Stage = Stager<T, KS, 64 * QW, NKV>;
  static constexpr int kBuf = Stage::kBytes + RowStager::kBytes, kBufs = buffers(kBuf, QW, KW);
  static constexpr int kPart = (G::MT * 16 + 1) * 64;
  static constexpr int kJoin = KW > 1 ? QW * KW * HG * kPart * 4 : 0;
  static constexpr int kWork = kBuf * kBufs * KW;
  static size_t lds_bytes(int nb) {
    const size_t walk = kWork + (size_t)(nb > 0 ? nb : 1) * HG * 128;
    return walk > kJoin ? walk : kJoin;    // the joined parts take the place of all else
  }
  static constexpr int kRegs = HG * (2 * KS * G::P * 4 + (G::P == 1 ? 2 : 1) * G::MT * 16) + 76 + Stage::kChunks * (G::P == 1 ? 6 : 10);
};

template <typename T, int KS, int HG, int NKV, int QW, int KW>
__global__ void __launch_bounds__(64 * QW * KW, (DqShape<T, KS, HG, NKV, QW, KW>::kRegs > 220 ? 1 : 2))
    k_attn_dq(AttnArgs a) {
  using S = DqShape<T, KS, HG, NKV, QW, KW>;
  using G = Tile<T, KS>;
  constexpr int P = G::P, MT = G::MT;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* tbl = reinterpret_cast<float*>(lds + S::kWork);
  const tp_attn& d = a.d;
  const int h0 = blockIdx.y * HG;
  int lo, hi, q0;
  if (!find_tile(d, kTile * QW, blockIdx.x, lo, hi, q0)) return;
  const int lane = threadIdx.x & 63, half = lane >> 5, wv = threadIdx.x >> 6;
  const int kw = wv % KW, qw = wv / KW;
  const int rep = d.n_heads / d.n_kv_heads, D = d.head_dim;
  const bool biased = d.n_buckets > 0;
  typename S::Stage st;
  RowStager rows;
  const int tid = qw * 64 + lane;          // among the threads that share a tile
  char* mine = lds + kw * S::kBufs * S::kBuf;
  const auto tiles_of = [&](int buf) { return reinterpret_cast<uint16_t*>(mine + buf * S::kBuf); };
  const auto rows_of = [&](int buf) { return reinterpret_cast<float*>(mine + buf * S::kBuf + S::Stage::kBytes); };
  const int k_first = lo + kTile * kw, step = kTile * KW;
  st.aim(tid, a.k, a.ks, a.v, a.vs, lo, k_first, step, D, [&](int slot) { return (h0 + slot) / rep; });
  const auto prepare = [&](int i) {
    st.fetch(k_first + i * step, hi, D, d.key_mask);
    rows.fetch(tid, d, biased, k_first + i * step, hi, d.key_mask);
  };
  prepare(0);

  const Scale scale(d.scale);
  TableFill<HG, S::kThreads> fill;
  fill.load(d, h0);
  const Buckets<HG> bk(d, tbl, lane);

  const int q = q0 + 32 * qw + (lane & 31), qc = q < hi ? q : hi - 1;
  float x = 0.f, y = 0.f, z = 0.f;
  if (biased) {
    x = d.pos[3 * (size_t)qc];
    y = d.pos[3 * (size_t)qc + 1];
    z = d.pos[3 * (size_t)qc + 2];
  }
  Frag<P> Q[HG][KS], dO[HG][KS];
  float lse[HG], delta[HG];
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    own_rows<T, KS>(a.q, a.qs, qc, h0 + hh, D, half, true, scale.sign, Q[hh]);
    own_rows<T, KS>(a.go, a.gos, qc, h0 + hh, D, half, true, 1.f, dO[hh]);
    float s = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int c = 16 * kk + 8 * half;
      if (c < D) {
        Raw<T> o, g;
        o.load(static_cast<const T*>(a.out_in) + (size_t)qc * a.os + (size_t)(h0 + hh) * D + c);
        g.load(static_cast<const T*>(a.go) + (size_t)qc * a.gos + (size_t)(h0 + hh) * D + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(o.at(j), g.at(j), s);
      }
    }
    delta[hh] = pair_sum(s);
    const size_t at = (size_t)(h0 + hh) * d.n_nodes + qc;
    lse[hh] = q < hi ? row_lse(a.lse_in[at]) : INFINITY;
  }

  constexpr bool kCorrect = P == 1;
  f16v dQ[HG][MT], PK[HG][kCorrect ? MT : 1];
  float r[HG];
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    r[hh] = 0.f;
    clear<MT>(dQ[hh]);
    if (kCorrect) clear<MT>(PK[hh]);
  }

  const auto stage = [&](int buf) {
    st.stage(tiles_of(buf));
    rows.stage(tid, rows_of(buf));
  };
  fill.write(d, scale.inv, tbl);
  __syncthreads();                         // the table
  uint32_t ent[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) ent[i] = bk.first;
  walk<(QW > 1), S::kBufs>((hi - lo + step - 1) / step, prepare, stage, [&](int buf) {
    const float* pos = rows_of(buf);
    const uint32_t vm = RowStager::valid(pos);
    if (vm == 0) return;                   // past the end, or all masked
    if (biased) tile_entries<HG>(bk, pos, half, x, y, z, ent);
#pragma unroll
    for (int hh = 0; hh < HG; ++hh) {
      const uint16_t* kt = tiles_of(buf) + (NKV == 1 ? 0 : hh * 2) * G::kElems;
      f16v s = scores<G, KS>(kt, Q[hh], ent, hh, lane);
      const f16v dp = product<G, KS>(kt + G::kElems, dO[hh], lane);
      if (vm != 0xffffffffu) mask_scores(vm, half, s);
      float p[16], ds[16], sum = 0.f;      // a sum per tile first: few additions to the running one
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], scale.c, -lse[hh]));
        ds[i] = p[i] * (dp[i] - delta[hh]);
        sum += ds[i];
      }
      r[hh] += sum;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Frag<P> f, w;
        to_frag(ds + 8 * kb, f);
        if (kCorrect) to_frag(p + 8 * kb, w);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const Frag<P> k = col_frag<G>(kt, mt, kb, lane);
          dQ[hh][mt] = mma(k, f, dQ[hh][mt]);
          if (kCorrect) PK[hh][mt] = mma(k, w, PK[hh][mt]);
        }
      }
    }
  });

  // row sums over all waves that share the row: delta for the key side, and grad_q's part of it
  float* join = reinterpret_cast<float*>(lds) + (size_t)qw * KW * HG * S::kPart + lane;
  if (KW > 1) {
    __syncthreads();
#pragma unroll
    for (int hh = 0; hh < HG; ++hh) join[(kw * HG + hh) * S::kPart] = pair_sum(r[hh]);
    __syncthreads();
  }
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    float sum = 0.f;
    if (KW > 1) {
#pragma unroll
      for (int w = 0; w < KW; ++w) sum += join[(w * HG + hh) * S::kPart];
    } else {
      sum = pair_sum(r[hh]);
    }
    if (q < hi && half == 0 && kw == 0) a.delta[(size_t)(h0 + hh) * d.n_nodes + q] = delta[hh] + sum;
    if (kCorrect) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dQ[hh][mt][i] = fmaf(-sum, PK[hh][mt][i], dQ[hh][mt][i]);
    }
    if (KW > 1) park<MT>(join + (kw * HG + hh) * S::kPart + 64, dQ[hh]);
  }
  if (KW > 1) __syncthreads();
  if (q >= hi) return;
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    if (KW > 1) {
      for (int gi = (kw + hh * 4 * MT) % KW; gi < 4 * MT; gi += KW) {
        float v[4];
        sum_parked<KW>(join + hh * S::kPart + 64, HG * S::kPart, gi, nullptr, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= d.scale;
        store4<T>(a.gq, a.gqs, q, h0 + hh, D, half, gi / 4, gi % 4, v);
      }
    } else {
#pragma unroll
      for (int gi = 0; gi < 4 * MT; ++gi) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = dQ[hh][gi / 4][gi % 4 * 4 + j] * d.scale;
        store4<T>(a.gq, a.gqs, q, h0 + hh, D, half, gi / 4, gi % 4, v);
      }
    }
  }
}

template <typename T, int KS, int HG, int NKV, int QW, int KW>
hipError_t launch(const AttnArgs& a) {
  using S = DqShape<T, KS, HG, NKV, QW, KW>;
  const dim3 grid((unsigned)(a.d.n_nodes / (kTile * QW) + a.d.n_segments), (unsigned)(a.d.n_heads / HG));
  return launch_lds(k_attn_dq<T, KS, HG, NKV, QW, KW>, grid, S::kThreads, S::lds_bytes(a.d.n_buckets), a);
}

// ---- which variant
// The waves of a workgroup: with enough query tiles to fill the chip, eight tiles share the
// staged keys; with few, two tiles share them and the other waves split the keys, four
// ways where LDS holds the tiles; of many structures under 1,024 atoms two tiles share
// keys; structures of a tile get one wave;
// where a workgroup for each tile leaves CUs idle, its waves all split the keys.  (us) 4,096 atoms, 8 heads of 32, bfloat16:
// 2x4 94, 8x1 261; 512 molecules of 62 atoms: 2x1 55, 1x1 60, 4x1 65; 120 structures of 300: 2x1
// 108, 4x1 103; 1,536 atoms, 5 heads of 64 (245 tiles): 1x8 26, 1x4 30, 2x4 34, with 8 heads
// (392 tiles) 1x8 32, 2x4 28.
// Eight waves leave a wave 256 registers; a kernel that needs more (wide heads) would spill
// its operands and takes four: 8,000 atoms, 8 heads of 128, bfloat16: 4x1 1,220, 8x1 3,508; of
// 96: 1,012, 1,174; 2,000 atoms: of 128 2x2 93, 2x4 244, of 96 79, 95.  (float32 heads of 64
// spill 51 registers at 2x4, 17 MiB of writes at 4,096 atoms, and keep it all the same: 211
// against 270.)
template <typename T, int KS, int HG, int NKV>
hipError_t by_waves(const AttnArgs& a, const Extent& x) {
  constexpr bool kWide = DqShape<T, KS, HG, NKV, 2, 4>::kRegs > 250;
  constexpr int KX = Tile<T, KS>::kElems * 4 * NKV * 4 <= 120 * 1024 && !kWide ? 4 : 2, QX = kWide ? 4 : 8;
  constexpr int64_t fill = kPlanes<T> * KS <= 2 ? 4096 : 2048;       // waves a chip holds of this kernel
  const int64_t waves = x.units / HG;
  if (x.mean <= kTile) return launch<T, KS, HG, NKV, 1, 1>(a);
  if constexpr (HG == 1 && Tile<T, KS>::kElems * 4 * 4 <= 120 * 1024) {
    constexpr int K1 = Tile<T, KS>::kElems * 4 * 8 <= 120 * 1024 && DqShape<T, KS, 1, 1, 1, 8>::kRegs <= 256 ? 8 : 4;
    if (x.units <= kCUs) return launch<T, KS, 1, 1, 1, K1>(a);
  }
  if (x.mean >= 1024 && waves >= fill) return launch<T, KS, HG, NKV, QX, 1>(a);
  if (x.mean >= 1024 || waves < 1024) return launch<T, KS, HG, NKV, 2, KX>(a);
  return launch<T, KS, HG, NKV, 2, 1>(a);
}

// Two heads to a wave share distances and buckets, where their operands fit the registers
// and half the waves still fill the chip (4,096 atoms, 8 heads of 32: 94 against 120 us;
// 1,536 atoms: 39 against 30 us).
template <typename T, int KS>
hipError_t by_heads(const AttnArgs& a) {
  const Extent x(a.d, a.d.n_heads);
  if constexpr (KS <= (kPlanes<T> == 1 ? 2 : 1)) {
    const int rep = a.d.n_heads / a.d.n_kv_heads;
    if (x.units >= 1024) {
      if (rep % 2 == 0) return by_waves<T, KS, 2, 1>(a, x);
      if (rep == 1 && a.d.n_heads % 2 == 0) return by_waves<T, KS, 2, 2>(a, x);
    }
  }
  return by_waves<T, KS, 1, 1>(a, x);
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

hipError_t attn_backward_q(const AttnArgs& a) { return a.d.dtype == TP_F32 ? by_width<float>(a) : by_width<bf16_t>(a); }

}  // namespace tpc
