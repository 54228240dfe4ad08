// Attention backward, key side: grad_k, grad_v and the bias gradient.
//
//   grad_v = p^T grad_out,  grad_k = scale ds^T q,  summed over the query heads of a
//   key head;  grad_bias[bucket] += ds;  p = exp(s - lse), ds = p (grad_out v^T - delta)
//
// A wave owns 32 keys of one key head and walks the queries in tiles, one query head
// after another.  KV x QS waves: KV own 32 keys each and share staged queries, QS
// split the queries and are joined through LDS at the end.  Where key heads are
// shared and there are too few key tiles to fill the chip, every query head gets
// workgroups of its own, whose float32 parts a second kernel adds up.
//
// bfloat16 rounds p and ds to the type for their products, as the forward does; the bias
// gradient sums the unrounded ds.
//
// The bias gradient goes into LDS columns private to the lane (no two lanes add to
// one word, so plain reads and writes do and the order of the sums is fixed), two
// elements at a time, summed per workgroup and joined by a second kernel.  An LDS
// float atomic takes 190 cycles a wave on gfx950; a read, an addition and a write of
// a pair take 150 cycles of latency, which the distances of the next tile fill.
//
// About 420 vector instructions a tile of 32 x 32 pairs and head, and nearly as many LDS
// cycles; the columns (256 bytes a bucket and wave) keep it at one to two waves a SIMD,
// which do not cover each other's latency (vector units 35 % busy, LDS 27 %).  1,536 atoms, 8 heads, 32 buckets: of 32, bfloat16 34 us, of
// 16, float32 48 us; 4,096 atoms, 4 query heads of 64 on one key head, 64 buckets, float32: 300 us
// (six products for one: 114 TFLOP/s of float32 work).
#include "attn.hpp"

namespace tpc {
namespace {

// Two sums into words of the lane's own column, which may be the same word: read both, add,
// write in order (the later of two sums into one word stands).
struct ColumnPair {
  lds_f *u, *v;
  float x, y;
  bool same;
  __device__ __forceinline__ ColumnPair(uint32_t a, uint32_t b) : u(lds_at(a)), v(lds_at(b)), x(*u), y(*v), same(a == b) {}
  __device__ __forceinline__ void add(float a, float b) const {
    const float s = x + a;
    *u = s;
    *v = (same ? s : y) + b;
  }
};

template <typename T, int KS, int KV, int QS>
struct DkvShape {
  using G = Tile<T, KS>;
  static constexpr int kThreads = 64 * KV * QS;
  using Stage = Stager<T, KS, 64 * KV, 1>;
  static constexpr int kBuf = Stage::kBytes + RowStager::kBytes + 2 * kTile * 4, kBufs = buffers(kBuf, KV, QS);
  static constexpr int kPart = 2 * G::MT * 16 * 64;                  // floats of one wave to join
  static constexpr int kJoin = QS > 1 ? KV * QS * kPart * 4 : 0;
  static constexpr int kWork = kBuf * kBufs * QS;
  static constexpr size_t lds_bytes(int nb) {
    const size_t walk = kWork + (nb > 0 ? (size_t)nb * (128 + KV * QS * 256) : 128);
    return walk > kJoin ? walk : kJoin;    // the joined parts take the place of all else
  }
  static constexpr int kRegs = 2 * KS * G::P * 4 + 2 * G::MT * 16 + 124 + Stage::kChunks * (G::P == 1 ? 6 : 10);
};

template <typename T, int KS, int KV, int QS>
__global__ void __launch_bounds__(64 * KV * QS, (DkvShape<T, KS, KV, QS>::kRegs > 220 ? 1 : 2))
    k_attn_dkv(AttnArgs a) {
  using S = DkvShape<T, KS, KV, QS>;
  using G = Tile<T, KS>;
  constexpr int P = G::P, MT = G::MT, NW = KV * QS;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* tbl = reinterpret_cast<float*>(lds + S::kWork);
  const tp_attn& d = a.d;
  const int nb = d.n_buckets, ne = nb > 0 ? nb : 1;
  float* cols = tbl + ne * 32;             // [NW][ne][64] bias gradient columns
  const int rep = d.n_heads / d.n_kv_heads, D = d.head_dim;
  // query heads h_lo .. h_hi - 1 of key head g
  const int g = a.split ? blockIdx.y / rep : blockIdx.y;
  const int h_lo = a.split ? blockIdx.y : g * rep, h_hi = a.split ? h_lo + 1 : h_lo + rep;
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
  const Buckets<1> bk(d, tbl, lane);
  const Scale scale(d.scale);

  // this lane's key; a masked one is held as zeros and gets zero gradients
  const int k = k0 + 32 * kv + (lane & 31), kc = k < hi ? k : hi - 1;
  const bool live = k < hi && (!d.key_mask || d.key_mask[kc] != 0);
  const bool some_dead = __any(!live);
  // table address -> address of the lane's column of the same entry (twice as wide)
  float* my_cols = cols + (size_t)wv * ne * 64;
  const uint32_t col = lds_address(my_cols) + 4 * lane - 2 * bk.first, col0 = lds_address(my_cols) + 4 * lane;
  float x = 0.f, y = 0.f, z = 0.f;
  if (biased) {
    x = d.pos[3 * (size_t)kc];
    y = d.pos[3 * (size_t)kc + 1];
    z = d.pos[3 * (size_t)kc + 2];
  }
  Frag<P> K[KS], V[KS];
  own_rows<T, KS>(a.k, a.ks, kc, g, D, half, live, scale.sign, K);
  own_rows<T, KS>(a.v, a.vs, kc, g, D, half, live, 1.f, V);
  f16v dK[MT], dV[MT];
  clear<MT>(dK);
  clear<MT>(dV);

  typename S::Stage st;
  RowStager rows;
  float slse = 0.f, sdel = 0.f;            // of the rows that were fetched last
  const int tid = kv * 64 + lane;          // among the threads that share a tile
  char* mine = lds + qs * S::kBufs * S::kBuf;
  const auto tiles_of = [&](int buf) { return reinterpret_cast<uint16_t*>(mine + buf * S::kBuf); };
  const auto rows_of = [&](int buf) { return reinterpret_cast<float*>(mine + buf * S::kBuf + S::Stage::kBytes); };
  const auto stat_of = [&](int buf) { return rows_of(buf) + RowStager::kBytes / 4; };   // [2][32]: lse (base 2), delta
  const int q_first = lo + kTile * qs, step = kTile * QS, n = (hi - lo + step - 1) / step;
  // table addresses of the present tile; ds and column addresses of the previous one, which
  // wait to be added to the columns
  uint32_t ent[16], due[16];
  float ds[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) ent[i] = bk.first;
  int h = h_lo;
  const auto prepare = [&](int i) {
    const int q0 = q_first + i * step;
    st.fetch(q0, hi, D, nullptr);
    rows.fetch(tid, d, biased, q0, hi, nullptr);
    if (tid < kTile) {
      const size_t at = (size_t)h * d.n_nodes + min(q0 + tid, hi - 1);
      slse = a.lse_in[at];
      sdel = a.delta[at];
    }
  };
  TableFill<1, S::kThreads> fill;
  st.aim(tid, a.q, a.qs, a.go, a.gos, lo, q_first, step, D, [&](int) { return h; });
  prepare(0);
  fill.load(d, h);
  while (true) {
    fill.write(d, scale.inv, tbl);
    if (biased) {
      for (int i = lane; i < ne * 16; i += 64) reinterpret_cast<f4*>(my_cols)[i] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        due[i] = col0;
        ds[i] = 0.f;
      }
    }
    const auto stage = [&](int buf) {
      st.stage(tiles_of(buf));
      rows.stage(tid, rows_of(buf));
      if (tid < kTile) {
        stat_of(buf)[tid] = rows.live ? row_lse(slse) : INFINITY;   // past the end: p = 0
        stat_of(buf)[kTile + tid] = rows.live ? sdel : 0.f;
      }
    };
    __syncthreads();                       // the table
    walk<(KV > 1), S::kBufs>(n, prepare, stage, [&](int buf) {
      const float *pos = rows_of(buf), *stat = stat_of(buf);
      if (RowStager::valid(pos) == 0) return;     // past the end
      if (biased) {
        // the latency of the column sums is filled with the distances of this tile
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 8 * j + 4 * half;
          const f4 px = *reinterpret_cast<const f4*>(pos + r), py = *reinterpret_cast<const f4*>(pos + kTile + r),
                   pz = *reinterpret_cast<const f4*>(pos + 2 * kTile + r);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int i = 4 * j + e;
            const ColumnPair u(due[i], due[i + 1]);
            ent[i] = bk.address(x, y, z, px[e], py[e], pz[e]);
            ent[i + 1] = bk.address(x, y, z, px[e + 1], py[e + 1], pz[e + 1]);
            u.add(ds[i], ds[i + 1]);
            due[i] = 2 * ent[i] + col;
            due[i + 1] = 2 * ent[i + 1] + col;
          }
        }
      }
      const uint16_t* qt = tiles_of(buf);
      f16v s = scores<G, KS, true>(qt, K, ent, 0, lane);
      const f16v dp = product<G, KS, true>(qt + G::kElems, V, lane);
      if (some_dead) mask_scores(live ? 0xffffffffu : 0u, half, s);   // p = 0: nothing for the bias
      float p[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + 4 * half;
        const f4 le = *reinterpret_cast<const f4*>(stat + r), de = *reinterpret_cast<const f4*>(stat + kTile + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[4 * j + e] = __builtin_amdgcn_exp2f(fmaf(s[4 * j + e], scale.c, -le[e]));
          ds[4 * j + e] = p[4 * j + e] * (dp[4 * j + e] - de[e]);
        }
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Frag<P> pf, df;
        to_frag(p + 8 * kb, pf);
        to_frag(ds + 8 * kb, df);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          dV[mt] = mma(col_frag<G>(qt + G::kElems, mt, kb, lane), pf, dV[mt]);
          dK[mt] = mma(col_frag<G>(qt, mt, kb, lane), df, dK[mt]);
        }
      }
    });
    if (biased) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) ColumnPair(due[i], due[i + 1]).add(ds[i], ds[i + 1]);
    }
    const int done = h++;
    if (h < h_hi) {                        // the next head's first tile, while this one's sums are taken
      st.again(n, D);
      prepare(0);
      fill.load(d, h);
    }
    if (a.gbias) {
      // each wave sums its own columns, a lane per entry, 16 bytes at a time; lanes start at
      // different columns so that they read different banks
      wave_sync();
      float s = 0.f;
      if (lane < nb) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const f4 v = reinterpret_cast<const f4*>(my_cols)[16 * lane + ((j + lane) & 15)];
          s += (v[0] + v[1]) + (v[2] + v[3]);
        }
      }
      wave_sync();
      my_cols[lane] = s;
      __syncthreads();
      if ((int)threadIdx.x < nb) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += cols[(size_t)w * ne * 64 + lane];
        a.part[((size_t)done * gridDim.x + blockIdx.x) * nb + lane] = s;
      }
    }
    if (h == h_hi) break;
    __syncthreads();                       // this head's table and columns have been read
  }

  float* join = reinterpret_cast<float*>(lds) + (size_t)kv * QS * S::kPart + lane;
  if (QS > 1) {
    __syncthreads();
    park<MT>(join + qs * S::kPart, dK);
    park<MT>(join + qs * S::kPart + S::kPart / 2, dV);
    __syncthreads();
  }
  if (k >= hi) return;
  // gi: register groups of dK, then of dV
  const auto store = [&](int gi, float v[4]) {
    const bool is_v = gi >= 4 * MT;
    const int e = is_v ? gi - 4 * MT : gi;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = live ? (is_v ? v[j] : v[j] * d.scale) : 0.f;
    if (a.split)                           // [n_nodes][n_heads][2][D]
      store4<float>(a.kv_part, (int64_t)d.n_heads * 2 * D, k, 2 * h_lo + is_v, D, half, e / 4, e % 4, v);
    else if (is_v)
      store4<T>(a.gv, a.gvs, k, g, D, half, e / 4, e % 4, v);
    else
      store4<T>(a.gk, a.gks, k, g, D, half, e / 4, e % 4, v);
  };
  if (QS > 1) {
    for (int gi = qs; gi < 8 * MT; gi += QS) {
      float v[4];
      sum_parked<QS>(join, S::kPart, gi, nullptr, v);
      store(gi, v);
    }
  } else {
#pragma unroll
    for (int gi = 0; gi < 8 * MT; ++gi) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (gi < 4 * MT ? dK : dV)[gi / 4 % MT][gi % 4 * 4 + j];
      store(gi, v);
    }
  }
}

// grad_k, grad_v [n][g] = sum over the query heads of key head g, in their order
template <typename T>
__global__ void __launch_bounds__(256)
    k_attn_join_kv(AttnArgs a) {
  const int D = a.d.head_dim, rep = a.d.n_heads / a.d.n_kv_heads;
  const int per = a.d.n_kv_heads * 2 * (D / 4);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t node = i / per;
  if (node >= a.d.n_nodes) return;
  const int e = (int)(i % per), c = e % (D / 4), which = e / (D / 4) % 2, g = e / (D / 4) / 2;
  const float* p = a.kv_part + (((size_t)node * a.d.n_heads + g * rep) * 2 + which) * D + 4 * c;
  f4 s = *reinterpret_cast<const f4*>(p);
  for (int r = 1; r < rep; ++r) s += *reinterpret_cast<const f4*>(p + (size_t)r * 2 * D);
  T* o = which ? static_cast<T*>(a.gv) + (size_t)node * a.gvs : static_cast<T*>(a.gk) + (size_t)node * a.gks;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[(size_t)g * D + 4 * c + j] = (T)s[j];
}

// grad_bias[h][b] = sum over the tiles' parts, in a fixed order.
//
// Every row of ds sums to zero, so a head's buckets do too.  What they sum to instead is
// rounding, most of it in the buckets of most pairs: n additions to a sum that grows as
// sqrt(n) round off about n.  It is taken off in proportion to n^2, n by the squares
// of the parts (a bucket without pairs stays 0).  Two structures of 3,000 to 6,000 atoms,
// 2 heads, 32 buckets, float32, 93 % of the pairs in the last: 4.4e-6 off without, 3.6e-7 with.
constexpr int kJoinThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    k_attn_join_bias(const float* __restrict__ part, int n, int nb, T* __restrict__ out) {
  __shared__ float2 lds[kJoinThreads];
  const int h = blockIdx.x, b = threadIdx.x & 63, g = threadIdx.x >> 6;
  float2 s = make_float2(0.f, 0.f);
  if (b < nb) {
#pragma unroll 8
    for (int t = g; t < n; t += kJoinThreads / 64) {
      const float v = part[((size_t)h * n + t) * nb + b];
      s.x += v;
      s.y = fmaf(v, v, s.y);
    }
  }
  lds[threadIdx.x] = s;
#pragma unroll
  for (int m = kJoinThreads / 2; m >= 64; m >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < m) {
      lds[threadIdx.x].x += lds[threadIdx.x + m].x;
      lds[threadIdx.x].y += lds[threadIdx.x + m].y;
    }
  }
  if (g > 0) return;                       // one wave, a lane per bucket
  s = lds[b];
  float most = s.y;
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor(most, m, 64));
  const float share = s.y / most;
  float over = s.x, weight = share * share;
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) {
    over += __shfl_xor(over, m, 64);
    weight += __shfl_xor(weight, m, 64);
  }
  const float off = over * (share * share / weight);
  // not where values are not finite, or so small or large that their squares are not
  if (b < nb) out[(size_t)h * nb + b] = (T)(__builtin_isfinite(off) ? s.x - off : s.x);
}

template <typename T>
hipError_t join_bias(const AttnArgs& a, int parts) {
  hipLaunchKernelGGL(k_attn_join_bias<T>, dim3(a.d.n_heads), dim3(kJoinThreads), 0, a.stream, a.part, parts,
                     a.d.n_buckets, static_cast<T*>(a.gbias));
  return hipGetLastError();
}

// Query heads apart: where key heads are shared and one workgroup per 32 keys and key
// head would leave most of the chip idle.
bool split_heads(const tp_attn& d) {
  return d.n_heads > d.n_kv_heads && ((int64_t)d.n_nodes / kTile + d.n_segments) * d.n_kv_heads < 512;
}

template <typename T, int KS, int KV, int QS>
hipError_t launch(const AttnArgs& a) {
  using S = DkvShape<T, KS, KV, QS>;
  const int tiles = a.d.n_nodes / (kTile * KV) + a.d.n_segments;
  hipError_t e = launch_lds(k_attn_dkv<T, KS, KV, QS>, dim3(tiles, a.split ? a.d.n_heads : a.d.n_kv_heads), S::kThreads,
                            S::lds_bytes(a.d.n_buckets), a);
  if (e != hipSuccess || a.dry) return e;
  if (a.split) {
    const int64_t n = (int64_t)a.d.n_nodes * a.d.n_kv_heads * 2 * (a.d.head_dim / 4);
    hipLaunchKernelGGL(k_attn_join_kv<T>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, a.stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return a.gbias ? join_bias<T>(a, tiles) : hipSuccess;
}

// ---- which variant
// As the query side, but the columns of the bias gradient bound the waves of a workgroup:
// eight up to 32 buckets, four up to 64.  (us) 1,536 atoms, 5 heads of 64 (245 tiles),
// float32: 1x4 78, 2x2 110; 1,536 atoms, 8 heads of 32, bfloat16: 2x4 40,
// 2x2 58, 4x1 92; 4,096 atoms: 4x2 152, 2x4 169; 512 molecules of 62 atoms: 2x1 124, 2x2 215.
// Eight waves leave a wave 256 registers, and wide heads spill.  Where waves split the queries
// four or eight ways four waves then do better, whole backward, 8 to 20 buckets: 1,536 atoms,
// 8 heads, float32, of 64: 2x4 207, 2x2 184, of 40: 178, 169 (of 32: 102, 122; bfloat16 of 64: 79,
// 94); 1,100 atoms, 4 heads of 64, bfloat16: 1x8 51, 1x4 49 (of 48: 45, 47; float32 of 32: 57,
// 60).  4x2 stays ahead with 125 registers spilled: 4,096 atoms, 8 heads of 64, float32: 818,
// 2x2 881, 4x1 802; bfloat16: 291, 424, 401.
template <typename T, int KS>
hipError_t by_waves(const AttnArgs& a) {
  const Extent x(a.d, a.split ? a.d.n_heads : a.d.n_kv_heads);
  hipError_t e = hipSuccess;
  // launched where LDS holds its tiles and the columns; not built where it never does, nor
  // where a split over eight waves spills
  const auto fits = [&](auto kv, auto qs) {
    using S = DkvShape<T, KS, kv(), qs()>;
    constexpr bool kSpills = kv() * qs() == 8 && qs() > 2 && S::kRegs > 250;
    if constexpr (S::lds_bytes(1) <= kLdsMax && !kSpills) {
      if (S::lds_bytes(a.d.n_buckets) <= kLdsMax) {
        e = launch<T, KS, kv(), qs()>(a);
        return true;
      }
    }
    return false;
  };
  const std::integral_constant<int, 1> c1;
  const std::integral_constant<int, 2> c2;
  const std::integral_constant<int, 4> c4;
  const std::integral_constant<int, 8> c8;
  if (x.mean <= kTile) return launch<T, KS, 1, 1>(a);
  if (x.units <= kCUs && (fits(c1, c8) || fits(c1, c4))) return e;
  if (x.mean < 1024 && x.units >= 1024) return launch<T, KS, 2, 1>(a);
  if (x.units >= 1024 ? fits(c4, c2) : fits(c2, c4)) return e;
  return fits(c2, c2) ? e : launch<T, KS, 2, 1>(a);
}

template <typename T>
hipError_t by_width(const AttnArgs& a) {
  const int ks = (a.d.head_dim + 15) / 16;
  if (ks <= 1) return by_waves<T, 1>(a);
  if (ks <= 2) return by_waves<T, 2>(a);
  if (ks <= 3) return by_waves<T, 3>(a);
  if (ks <= 4) return by_waves<T, 4>(a);
  if (ks <= 6) return by_waves<T, 6>(a);
  return by_waves<T, 8>(a);
}

}  // namespace

hipError_t attn_backward(const AttnArgs& args) {
  AttnArgs a = args;
  a.split = split_heads(a.d);
  if (a.d.n_nodes == 0) return a.d.dtype == TP_F32 ? join_bias<float>(a, 0) : join_bias<bf16_t>(a, 0);
  // both grids are checked before the first launch; the query side leaves delta for the key side
  hipError_t e = hipSuccess;
  for (const bool dry : {true, false}) {
    a.dry = dry;
    if ((e = attn_backward_q(a)) != hipSuccess) return e;
    if ((e = a.d.dtype == TP_F32 ? by_width<float>(a) : by_width<bf16_t>(a)) != hipSuccess) return e;
  }
  return e;
}

AttnWorkspace attn_workspace(const tp_attn& d) {
  AttnWorkspace w;
  w.part = ((size_t)d.n_heads * d.n_nodes + 3) / 4 * 4;
  w.kv_part = w.part + (((size_t)d.n_nodes / kTile + d.n_segments) * d.n_heads * d.n_buckets + 3) / 4 * 4;
  w.floats = w.kv_part + (split_heads(d) ? (size_t)d.n_nodes * d.n_heads * 2 * d.head_dim : 0);
  return w;
}

}  // namespace tpc
