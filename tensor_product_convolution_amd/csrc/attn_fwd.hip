// Attention forward: out = softmax(scale q k^T + bias[bucket]) v per structure.
// One pass over the keys with a running maximum and sum per query (see attn.hpp
// for the tile layout); HG heads share the tile's distances and buckets.
//
// bfloat16 probabilities are rounded to the type for p v, a choice: in two pieces (float32's
// would be three) that product would be twice as long, and out, which is rounded to the type
// itself, is 2.4e-3 off with and 1.7e-3 without.  The sum that divides it is of the unrounded ones.
//
// QW x KW waves: QW own 32 queries each and share staged keys, KW split the keys and
// are joined through LDS at the end (for batches with few query tiles).
//
// The vector units bound it, not the matrix units: a pair costs about 11 instructions for
// its distance and bucket, shared by HG heads, and 6 a head around the exponential,
// against one 32-cycle product per 32 x 32 x 16.  16,384 atoms, 8 heads of 64, bfloat16: 986 us
// (557 TFLOP/s, 45 % of a large library product's rate; vector units 59 %, LDS 41 %, matrix
// units 22 % busy at two waves a SIMD); 1,536 atoms, 8 heads: of 32, bfloat16 22 us, of 16,
// float32 30 us (192 workgroups: a quarter of the chip is idle); 4,096 atoms, 4 heads of 64,
// float32 133 us (matrix units 31 %: six products for one).
#include "attn.hpp"

namespace tpc {
namespace {

template <typename T, int KS, int HG, int NKV, int QW, int KW>
struct FwdShape {
  using G = Tile<T, KS>;
  static constexpr int kThreads = 64 * QW * KW;
  using Stage = Stager<T, KS, 64 * QW, NKV>;
  static constexpr int kBuf = Stage::kBytes + RowStager::kBytes, kBufs = buffers(kBuf, QW, KW);
  static constexpr int kPart = (G::MT * 16 + 2) * 64;                // floats of one wave's head to join
  static constexpr int kJoin = KW > 1 ? QW * KW * HG * kPart * 4 : 0;
  static constexpr int kWork = kBuf * kBufs * KW;
  static size_t lds_bytes(int nb) {
    const size_t walk = kWork + (size_t)(nb > 0 ? nb : 1) * HG * 128;
    return walk > kJoin ? walk : kJoin;    // the joined parts take the place of all else
  }
  // operands, accumulators and scores beside what the fetch holds
  static constexpr int kRegs = HG * (KS * G::P * 4 + G::MT * 16 + 16) + 60 + Stage::kChunks * (G::P == 1 ? 6 : 10);
};

// One workgroup's queries.  Float32 operands are split with FAR or without; true: without, and
// a sum came out that is not finite.
template <bool FAR, typename T, int KS, int HG, int NKV, int QW, int KW>
__device__ __forceinline__ bool attn_fwd(const AttnArgs& a, char* lds) {
  using S = FwdShape<T, KS, HG, NKV, QW, KW>;
  using G = Tile<T, KS>;
  constexpr int P = G::P, MT = G::MT;
  float* tbl = reinterpret_cast<float*>(lds + S::kWork);
  const tp_attn& d = a.d;
  int lo, hi, q0;
  if (!find_tile(d, kTile * QW, blockIdx.x, lo, hi, q0)) return false;
  const int lane = threadIdx.x & 63, half = lane >> 5, wv = threadIdx.x >> 6;
  const int kw = wv % KW, qw = wv / KW;
  const int h0 = blockIdx.y * HG, rep = d.n_heads / d.n_kv_heads, D = d.head_dim;
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
  for (int hh = 0; hh < HG; ++hh) own_rows<T, KS>(a.q, a.qs, qc, h0 + hh, D, half, true, scale.sign, Q[hh], FAR);

  f16v O[HG][MT];
  float m[HG], l[HG];                      // running maximum of S and sum
  bool wide[HG];                           // a row of the wave is far from 0 (below)
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    m[hh] = kLowest * scale.inv;
    wide[hh] = false;
    l[hh] = 0.f;
    clear<MT>(O[hh]);
  }

  const auto stage = [&](int buf) {
    st.stage(tiles_of(buf), FAR);
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
    // every head's scores first: a head's products run while another's softmax does
    const uint16_t* kt = tiles_of(buf);
    f16v sc[HG];
#pragma unroll
    for (int hh = 0; hh < HG; ++hh) sc[hh] = scores<G, KS>(kt + (NKV == 1 ? 0 : hh * 2) * G::kElems, Q[hh], ent, hh, lane);
    if (vm != 0xffffffffu) {
#pragma unroll
      for (int hh = 0; hh < HG; ++hh) mask_scores(vm, half, sc[hh]);
    }
#pragma unroll
    for (int hh = 0; hh < HG; ++hh) {
      const uint16_t* vt = kt + (NKV == 1 ? 1 : hh * 2 + 1) * G::kElems;
      // c S - (c m rounded) is one instruction, off by one factor of up to 2^(2^-24 |c m|) in all
      // of a row.  From 10^9 on that overflows, or leaves the row's largest term 0: rows beyond
      // |c m| = 2^12 take the difference first, in the branch below.
      float p[16], sum = 0.f, cm = m[hh] * scale.c;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(sc[hh][i], scale.c, -cm));
        sum += p[i];
      }
      // The running maximum is raised when the tile's sum shows that it has been passed by
      // far: probabilities up to 2^9 lose nothing, most tiles need no maximum at all, and
      // the accumulators are rescaled in few.  NaN takes this way in every tile.
      if (wide[hh] || __any(!(sum <= 512.f))) {
        const auto is_wide = [&]() { return fabsf(cm) > 4096.f && cm > 0.999999f * kLog2e * kLowest; };   // not before its first key
        // what happens to a row does not depend on the others of the wave
        const bool over = is_wide() || !(pair_sum(sum) <= 1024.f);
        float tm = fmaxf(sc[hh][0], sc[hh][1]);
#pragma unroll
        for (int i = 2; i < 16; ++i) tm = fmaxf(tm, sc[hh][i]);
        tm = pair_max(tm);
        const float mn = over ? fmaxf(m[hh], tm) : m[hh], f = __builtin_amdgcn_exp2f((m[hh] - mn) * scale.c);
        m[hh] = mn;
        l[hh] *= f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 16; ++i) O[hh][mt][i] *= f;
        cm = mn * scale.c;
        const bool w = is_wide();
        wide[hh] = __any(w);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = __builtin_amdgcn_exp2f(fmaf(sc[hh][i], scale.c, -cm));
          sum += p[i];
        }
        if (w) {
          sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            p[i] = __builtin_amdgcn_exp2f((sc[hh][i] - mn) * scale.c);
            sum += p[i];
          }
        }
      }
      l[hh] += sum;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Frag<P> pf;
        to_frag(p + 8 * kb, pf);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) O[hh][mt] = mma(col_frag<G>(vt, mt, kb, lane), pf, O[hh][mt]);
      }
    }
  });

  bool again = false;
  if (P > 1 && !FAR) {
    float t = 0.f;
#pragma unroll
    for (int hh = 0; hh < HG; ++hh)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * mt + 8 * (i / 4) < 16 * KS) t = fmaf(O[hh][mt][i], 0.f, t);   // columns that are staged
    again = __any(t != t);
    if (QW * KW > 1) {
      uint32_t* found = reinterpret_cast<uint32_t*>(lds);
      __syncthreads();                     // the tiles have been read
      if (lane == 0) found[wv] = again;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < QW * KW; ++w) again |= __builtin_amdgcn_readfirstlane(found[w]) != 0;
    }
  }

  // statistics of the row over all waves that share it
  float factor[HG][KW], sum[HG];
  float* join = reinterpret_cast<float*>(lds) + (size_t)qw * KW * HG * S::kPart + lane;
  if (KW > 1) {
    __syncthreads();
#pragma unroll
    for (int hh = 0; hh < HG; ++hh) {
      float* w = join + (kw * HG + hh) * S::kPart;
      w[0] = m[hh];
      w[64] = pair_sum(l[hh]);
      park<MT>(w + 128, O[hh]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    if (KW > 1) {
#pragma unroll
      for (int w = 0; w < KW; ++w) m[hh] = fmaxf(m[hh], join[(w * HG + hh) * S::kPart]);
      sum[hh] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        factor[hh][w] = __builtin_amdgcn_exp2f((join[(w * HG + hh) * S::kPart] - m[hh]) * scale.c);
        sum[hh] = fmaf(join[(w * HG + hh) * S::kPart + 64], factor[hh][w], sum[hh]);
      }
    } else {
      sum[hh] = pair_sum(l[hh]);
    }
  }
  if (q >= hi) return again;
#pragma unroll
  for (int hh = 0; hh < HG; ++hh) {
    const bool empty = sum[hh] == 0.f;     // NaN is not empty: it has to show
    const float inv = 1.f / sum[hh];
    if (a.lse && half == 0 && kw == 0)
      a.lse[(size_t)(h0 + hh) * d.n_nodes + q] = empty ? -INFINITY : (m[hh] * scale.c + __builtin_amdgcn_logf(sum[hh])) * kLn2;
    const auto store = [&](int gi, float v[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = empty ? 0.f : v[j] * inv;
      store4<T>(a.out, a.os, q, h0 + hh, D, half, gi / 4, gi % 4, v);
    };
    if (KW > 1) {
      for (int gi = (kw + hh * 4 * MT) % KW; gi < 4 * MT; gi += KW) {
        float v[4];
        sum_parked<KW>(join + hh * S::kPart + 128, HG * S::kPart, gi, factor[hh], v);
        store(gi, v);
      }
    } else {
#pragma unroll
      for (int gi = 0; gi < 4 * MT; ++gi) {
        float v[4] = {O[hh][gi / 4][gi % 4 * 4], O[hh][gi / 4][gi % 4 * 4 + 1], O[hh][gi / 4][gi % 4 * 4 + 2],
                      O[hh][gi / 4][gi % 4 * 4 + 3]};
        store(gi, v);
      }
    }
  }
  return again;
}

// The split of float32 operands turns infinities into NaN.  A workgroup that finds values which are
// not finite walks again with the longer split that keeps them.  The check takes 1 % of 4,096 atoms,
// 4 heads of 64 (123 against 121 us), 3 % of 1,536, 8 heads of 16; the longer split in every walk 3 %.
template <typename T, int KS, int HG, int NKV, int QW, int KW>
__global__ void __launch_bounds__(64 * QW * KW, (FwdShape<T, KS, HG, NKV, QW, KW>::kRegs > 210 ? 1 : 2))
    k_attn_fwd(AttnArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const bool again = attn_fwd<false, T, KS, HG, NKV, QW, KW>(a, lds);
  if (kPlanes<T> > 1 && __any(again)) {
    __syncthreads();
    (void)attn_fwd<true, T, KS, HG, NKV, QW, KW>(a, lds);
  }
}

template <typename T, int KS, int HG, int NKV, int QW, int KW>
hipError_t launch(const AttnArgs& a) {
  using S = FwdShape<T, KS, HG, NKV, QW, KW>;
  const dim3 grid((unsigned)(a.d.n_nodes / (kTile * QW) + a.d.n_segments), (unsigned)(a.d.n_heads / HG));
  return launch_lds(k_attn_fwd<T, KS, HG, NKV, QW, KW>, grid, S::kThreads, S::lds_bytes(a.d.n_buckets), a);
}

// ---- which variant
// The waves of a workgroup: with enough query tiles to fill the chip, eight tiles share the
// staged keys; with few, two tiles share them and the other waves split the keys, four
// ways where LDS holds the tiles; of many structures under 1,024 atoms four tiles share
// keys; structures of a tile get one wave;
// where a workgroup for each tile leaves CUs idle, its waves all split the keys.  Measured (us): 16,384 atoms, 8 heads of 64,
// bfloat16: 8x1 977, 2x4 1,674; 4,096 atoms, 8 heads of 32: 2x4 76, 8x1 215; 120 structures
// of 300 atoms: 4x1 74, 2x1 86, 1x1 88, 2x4 144 (float32: 141, 2x1 179, 8x1 227); 512
// molecules of 62 atoms, 64 buckets: 4x1 42, 2x1 44, 1x1 41, 2x4 110; 1,536 atoms, 5 heads of
// 64 (245 tiles): 1x8 18, 1x4 23, 2x4 26, with 8 heads (392 tiles) 1x8 27, 2x4 23.
template <typename T, int KS, int HG, int NKV>
hipError_t by_waves(const AttnArgs& a, const Extent& x) {
  constexpr int KX = Tile<T, KS>::kElems * 4 * NKV * 4 <= 120 * 1024 ? 4 : 2;
  constexpr int64_t fill = kPlanes<T> * KS <= 2 ? 4096 : 2048;       // waves a chip holds of this kernel
  const int64_t waves = x.units / HG;
  if (x.mean <= kTile) return launch<T, KS, HG, NKV, 1, 1>(a);
  if constexpr (HG == 1 && KX == 4) {
    constexpr int K1 = Tile<T, KS>::kElems * 4 * 8 <= 120 * 1024 ? 8 : 4;
    if (x.units <= kCUs) return launch<T, KS, 1, 1, 1, K1>(a);
  }
  if (x.mean >= 1024 && waves >= fill) return launch<T, KS, HG, NKV, 8, 1>(a);
  if (x.mean >= 1024 || waves < 1024) return launch<T, KS, HG, NKV, 2, KX>(a);
  return launch<T, KS, HG, NKV, 4, 1>(a);
}

// Two heads to a wave share distances and buckets, where their operands fit the registers
// and half the waves still fill the chip (16,384 atoms: 977 against 1,414 us; 4,096: 76
// against 104; 1,536: 32 against 24).
template <typename T, int KS>
hipError_t by_heads(const AttnArgs& a) {
  const Extent x(a.d, a.d.n_heads);
  if constexpr (kPlanes<T> * KS <= 4) {
    const int rep = a.d.n_heads / a.d.n_kv_heads;
    if (x.units >= 2048) {
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

hipError_t attn_forward(const AttnArgs& a) { return a.d.dtype == TP_F32 ? by_width<float>(a) : by_width<bf16_t>(a); }

}  // namespace tpc
