// Gated delta rule, backward (gfx950).  With dO, and dS' the gradient of the
// state leaving a chunk (S, dS here as [d_k, d_v]; q carries the scale):
//   dU  = (Q K^T o D)^T dO + diag(exp(G_63 - G)) K dS'
//   Y   = T^T dU                      (the token-by-token gradient of beta_t (..))
//   dV  = diag(beta) Y,   d beta_i = Y_i . U_i / beta_i
//   dS  = e_63 dS' + (diag(e) Q)^T dO - (diag(e beta) K)^T Y
// goes from the last chunk to the first, by columns (d_v) like the forward;
// then, chunk by chunk in parallel, with dP = dO U^T (j <= i) and
// dA = -Y U^T (j < i), M1 = dP o D, M2 = diag(beta) dA o D:
//   dQ  = diag(e) dO S^T + M1 K
//   dK  = M1^T Q + M2^T K + M2 K + diag(exp(G_63 - G)) U dS'^T - diag(e beta) Y S^T
// and the decay's gradient from the pairs each token's g stands between:
//   E_ij = dP_ij P_ij + dA_ij A_ij (j < i)
//   dG_i = sum_j E_ij - sum_j E_ji + q_i.(e dO S^T)_i - k_i.(e beta Y S^T)_i - k_i.(.. U dS'^T)_i
//   dg_t = sum_{i >= t} dG_i + sum_i k_i.(.. U dS'^T)_i + e_63 <dS', S>
#include "gdelta_launch.h"

namespace gdelta {

// ------------------------------------------------------------------ scale of dS and Y
// One workgroup per (batch row, head, chunk) reads dy once (168 MB in 53 us, short workgroups' latency).
template <Act A>
__global__ void __launch_bounds__(256) gdelta_dymax_kernel(const BwdArgs p) {
  __shared__ float s[4];
  const Dims& d = p.d;
  const int tid = threadIdx.x;
  const ChunkPlace at_ = chunk_place(blockIdx.x, static_cast<uint32_t>(d.H), static_cast<uint32_t>(d.nc));
  const int64_t c = at_.c, h = at_.h, b = at_.b, bh = b * d.H + h;
  const int64_t t0 = c * kC, left = d.T - t0;
  float m = 0.0f;
  // the chunk's 16-byte pieces (of bf16) in order, four loads in flight a thread; i / n by a factor exact for i < 64 n, n <= 64
  const uint32_t n = static_cast<uint32_t>(d.V / 8), inv = (1u << 20) / n + 1;
  const uint32_t end = static_cast<uint32_t>(left < kC ? left : kC) * n;
  for (uint32_t i0 = tid; i0 < end; i0 += 4 * 256) {
    float x[4][8];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t i = i0 + 256 * k, row = i * inv >> 20;
      load8<A>(p.dy, ((b * d.T + t0 + row) * d.H + h) * d.V + (i - row * n) * 8, i < end, x[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_finite(m, x[k][e]);
  }
  m = wave_max(m);
  if ((tid & 63) == 0) s[tid >> 6] = m;
  __syncthreads();
  if (tid == 0) p.dymax[bh * d.nc + c] = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

// One wave per head: the largest value of |ds| <= e_63 |ds'| + 64 scale max |dy| over the chunks, last to first.
__global__ void __launch_bounds__(64) gdelta_dscale_kernel(const BwdArgs p) {
  const Dims& d = p.d;
  const int lane = threadIdx.x;
  const int64_t bh = blockIdx.x;
  float M = 0.0f, top = 0.0f;
  for (int64_t c0 = (d.nc - 1) / 64 * 64; c0 >= 0; c0 -= 64) {
    const int64_t c = c0 + lane, ci = bh * d.nc + c;
    const bool ok = c < d.nc;
    const float m = ok ? p.dymax[ci] : 0.0f;
    const float e = ok ? p.w.hsc[ci * (kHeadSc * kC) + H_E * kC + kC - 1] : 1.0f;
    const float add = static_cast<float>(kC) * fabsf(d.scale) * m;
    top = fmaxf(top, m);
    for (int i = 63; i >= 0; --i) {
      const float a = __shfl(add, i, 64), el = __shfl(e, i, 64);
      top = fmaxf(top, M + a);
      M = fmaf(el, M, a);
    }
  }
  top = wave_max(top);
  if (lane == 0) p.so[bh] = pow2_below(top, 14);
}

// ------------------------------------------------------------------ pass from the last chunk to the first
// As the forward's pass: a wave holds 16 columns of dS^T and needs nothing of any other, but for the fragments that the
// tiles of a head share; they come a chunk ahead, to LDS for 16-bit inputs; f32 inputs have two planes, twice of which are
// more than it holds: each wave has the first in registers, the second in LDS.  Fragments of a chunk in the shared buffer,
// in this order:
template <int KP>
struct BwdRing {
  static constexpr int NF = KP / 8, KF = 0, PT = NF, TT = PT + 12, QF = TT + 12, N = QF + NF;
};

template <Act A, int KP, bool RING>
struct BackChain {
  static constexpr int NP = A == Act::F32 ? 2 : 1, MT = KP / 16, KS = KP / 32, NF = KP / 8;
  using Place = PassPlace<A>;
  using R = BwdRing<KP>;
  f32x4 dS[MT];
  h8 kf[RING ? 1 : NF], kt[RING ? 1 : NF], qt[RING ? 1 : NF], ph[RING ? 1 : 6], pl[RING ? 1 : 6], th[RING ? 1 : 6], tl[RING ? 1 : 6];
  float sc[4], el;
  uint32_t v[4][4];
  const uint16_t *ring, *ring_t;   // + this lane's place, plain and for a transpose
  uint16_t* low;   // f32: the second planes of KF, QT and KT
  // the parts of dS and Y through LDS to wide stores: 563 us against 603 for 8192 tokens of 80 heads of 128 x 128, 89
  // against 87 for 2048 tokens of 96 heads of 64 x 64
  static constexpr bool KEEP = RING && KP == 128;
  uint16_t* kept;   // [KS][high, low] fragments of the wave's own

  template <int N>
  __device__ __forceinline__ h8 get(const h8 (&x)[N], int base, int i) const {
    if constexpr (RING) return ld8(ring + (base + i) * kFrag);
    else return x[i];
  }
  template <int N>
  __device__ __forceinline__ h8 get_t(const h8 (&x)[N], int base, int i) const {
    if constexpr (RING) return ld_trans<KP>(ring_t + base * kFrag, i);
    else return x[i];
  }
  template <int N>
  __device__ __forceinline__ void load(h8 (&x)[N], const uint16_t* base, int lane) {
    if constexpr (!RING) load_frags(x, base, lane);
  }
  __device__ __forceinline__ int64_t group(const Place& w, int64_t c) const { return (w.bg * w.nc + c) * (NP * NF * kFrag); }
  __device__ __forceinline__ void load_p(const BwdArgs& p, const Place& w, int64_t c) {
    const uint16_t* x = p.w.PT + (w.bh * w.nc + c) * (12 * kFrag);
    load(ph, x, w.lane);
    load(pl, x + 6 * kFrag, w.lane);
  }
  __device__ __forceinline__ void load_t(const BwdArgs& p, const Place& w, int64_t c) {
    const uint16_t* x = p.w.TT + (w.bh * w.nc + c) * (12 * kFrag);
    load(th, x, w.lane);
    load(tl, x + 6 * kFrag, w.lane);
  }
  __device__ __forceinline__ void load_sc(const BwdArgs& p, const Place& w, int64_t c) {
    const float* x = p.w.hsc + (w.bh * w.nc + c) * (kHeadSc * kC);
    sc[0] = x[H_BETA * kC + w.lane];
    sc[1] = x[H_BK * kC + w.lane];
    sc[2] = x[H_DK * kC + w.lane];
    sc[3] = x[H_EQ * kC + w.lane];
    el = x[H_E * kC + kC - 1];
  }
  __device__ __forceinline__ void load_dy(const BwdArgs& p, const Place& w, int64_t c) {
    const int vcol = w.ok ? w.col : static_cast<int>(p.d.V) - 1;
    load_cols<typename Place::Raw>(v, static_cast<const char*>(p.dy) + w.at_chunk(c), w.row, vcol * Place::ES, w.T - c * kC, w.g);
  }
  __device__ __forceinline__ void init(const BwdArgs& p, const Place& w) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t c = w.nc - 1;
    load(kf, p.w.KF + group(w, c), w.lane);
    load_sc(p, w, c);
    load_dy(p, w, c);
    load_p(p, w, c);
    load_t(p, w, c);
    load(qt, p.w.QT + group(w, c), w.lane);
    load(kt, p.w.KT + group(w, c), w.lane);
    load_low(0, p.w.KF + group(w, c), w.lane);
    load_low(1, p.w.QT + group(w, c), w.lane);
    load_low(2, p.w.KT + group(w, c), w.lane);
  }
  __device__ __forceinline__ void load_low(int i, const uint16_t* base, int lane) {
    if constexpr (NP == 2) copy_low<NF>(low + i * (NF * kFrag), base + NF * kFrag, lane);
  }
  // One chunk.  soc: the head's scale, 0 in columns behind d_v; s: [4][64] floats of the wave.
  __device__ __forceinline__ void step(const BwdArgs& p, const Place& w, int64_t c, float soc, float rso, float rps, float (*s)[kC]) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t ci = w.bh * w.nc + c, next = c > 0 ? c - 1 : c;   // the first chunk loads its own again: no branch in the loop
    const int VP = p.d.VP, poff = (4 * w.g * VP + w.col) * 4;
    const uint16_t *KF = p.w.KF, *KT = p.w.KT, *QT = p.w.QT;
    mscan::wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][w.lane] = sc[i];
    mscan::wave_lds_sync();
    const float elc = el;
    load_sc(p, w, next);
    if constexpr (NP == 2) wait_low();
    f32x4 dU[4] = {zero, zero, zero, zero}, pd[4] = {zero, zero, zero, zero}, dO[4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag f = to_b(dS[2 * ks], dS[2 * ks + 1]);
      if constexpr (KEEP) keep_parts(kept + 2 * ks * kFrag, w.lane, f);
      else store_packed(p.DS + (ci * KP + 32 * ks) * VP, poff, f, VP);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) dU[mt] = mma(get(kf, R::KF, mt * KS + ks), f.hi, dU[mt]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) dU[mt] = mma(get(kf, R::KF, mt * KS + ks), f.lo, dU[mt]);
      if (NP == 2) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) dU[mt] = mma(ld8(low + (mt * KS + ks) * kFrag + w.lane * 8), f.hi, dU[mt]);
      }
    }
    load(kf, KF + group(w, next), w.lane);
    load_low(0, KF + group(w, next), w.lane);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) dO[mt][e] = IO<A>::cvt(v[mt][e]) * soc;
    load_dy(p, w, next);
    const Frag o0 = to_b(dO[0], dO[1]), o1 = to_b(dO[2], dO[3]);   // 16-bit input: the low parts are zero
#pragma unroll
    for (int f = 0; f < 6; ++f) pd[kUm[f]] = mma(get(ph, R::PT, f), (kUk[f] ? o1 : o0).hi, pd[kUm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) pd[kUm[f]] = mma(get(pl, R::PT + 6, f), (kUk[f] ? o1 : o0).hi, pd[kUm[f]]);
    if (NP == 2) {
#pragma unroll
      for (int f = 0; f < 6; ++f) pd[kUm[f]] = mma(get(ph, R::PT, f), (kUk[f] ? o1 : o0).lo, pd[kUm[f]]);
    }
    load_p(p, w, next);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 dk = *reinterpret_cast<const f32x4*>(s[2] + 16 * mt + 4 * w.g);
      dU[mt] = dU[mt] * dk + pd[mt] * rps;
      dO[mt] *= *reinterpret_cast<const f32x4*>(s[3] + 16 * mt + 4 * w.g);
    }
    const Frag u0 = to_b(dU[0], dU[1]), u1 = to_b(dU[2], dU[3]);
    f32x4 Y[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int f = 0; f < 6; ++f) Y[kUm[f]] = mma(get(th, R::TT, f), (kUk[f] ? u1 : u0).hi, Y[kUm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) Y[kUm[f]] = mma(get(th, R::TT, f), (kUk[f] ? u1 : u0).lo, Y[kUm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) Y[kUm[f]] = mma(get(tl, R::TT + 6, f), (kUk[f] ? u1 : u0).hi, Y[kUm[f]]);
    load_t(p, w, next);
    // the part of dS from dO does not wait for Y
    const Frag e0 = to_b(dO[0], dO[1]), e1 = to_b(dO[2], dO[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] *= elc;
    update(qt, R::QF, 1, e0, e1, w.lane);
    load(qt, QT + group(w, next), w.lane);
    load_low(1, QT + group(w, next), w.lane);
    if constexpr (KEEP) {
      const int off = store_off(w.lane, VP), v0 = w.col - w.r;
      mscan::wave_lds_sync();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) store_kept(p.DS + (ci * KP + 32 * ks) * VP + v0, off, kept + 2 * ks * kFrag, w.lane, VP);
      mscan::wave_lds_sync();
      keep_parts(kept, w.lane, to_b(Y[0], Y[1]));
      keep_parts(kept + 2 * kFrag, w.lane, to_b(Y[2], Y[3]));
      mscan::wave_lds_sync();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) store_kept(p.DU + (ci * kC + 32 * ks) * VP + v0, off, kept + 2 * ks * kFrag, w.lane, VP);
      mscan::wave_lds_sync();
    } else {
      store_packed(p.DU + ci * kC * VP, poff, to_b(Y[0], Y[1]), VP);
      store_packed(p.DU + (ci * kC + 32) * VP, poff, to_b(Y[2], Y[3]), VP);
    }
    f32x4 dv[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      dv[mt] = Y[mt] * *reinterpret_cast<const f32x4*>(s[0] + 16 * mt + 4 * w.g) * rso;
      Y[mt] *= -*reinterpret_cast<const f32x4*>(s[1] + 16 * mt + 4 * w.g);
    }
    update(kt, R::KF, 2, to_b(Y[0], Y[1]), to_b(Y[2], Y[3]), w.lane);
    load(kt, KT + group(w, next), w.lane);
    load_low(2, KT + group(w, next), w.lane);
    store_cols<A>(dv, static_cast<char*>(p.d_v) + w.at_chunk(c), w.row, w.col * Place::ES, w.T - c * kC, w.g, w.ok);
  }
  // dS += X^T (a, b): X's transposed fragments; f32 inputs have a second plane, `second` of `low`
  template <int N>
  __device__ __forceinline__ void update(const h8 (&x)[N], int base, int second, const Frag& a, const Frag& b, int lane) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(get_t(x, base, 2 * mt), a.hi, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(get_t(x, base, 2 * mt), a.lo, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(get_t(x, base, 2 * mt + 1), b.hi, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(get_t(x, base, 2 * mt + 1), b.lo, dS[mt]);
    if (NP == 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        dS[mt] = mma(ld8(low + (second * NF + 2 * mt) * kFrag + lane * 8), a.hi, dS[mt]);
        dS[mt] = mma(ld8(low + (second * NF + 2 * mt + 1) * kFrag + lane * 8), b.hi, dS[mt]);
      }
    }
  }
};

template <Act A, int KP>
__global__ void __launch_bounds__(64) gdelta_bwd_state_kernel(const BwdArgs p) {
  __shared__ __attribute__((aligned(16))) float s[4][kC];   // beta; beta e rk; exp(G_63 - G) rk; e rq
  const PassPlace<A> w(p.d);
  const float so = p.so[w.bh], rso = 1.0f / so, rps = 1.0f / p.d.pscale, soc = w.ok ? so : 0.0f;
  __shared__ __attribute__((aligned(16))) uint16_t low[3][KP / 8 * kFrag];
  BackChain<A, KP, false> ch;
  ch.low = low[0];
  ch.init(p, w);
  for (int64_t c = p.d.nc - 1; c >= 0; --c) ch.step(p, w, c, soc, rso, rps, s);
}

// TILES waves with a tile each and four that copy the fragments, as in the forward and bound by the same: 8192 tokens of 80
// heads of 128 x 128 take 570 us, 2 GB of HBM traffic at 3.5 TB/s, against 850 with the fragments in each wave's
// registers; 2048 tokens of 96 heads of 64 x 64 take 87 against 124.
template <Act A, int KP, int TILES>
__global__ void __launch_bounds__(64 * (TILES + kCopyWaves)) gdelta_bwd_ring_kernel(const BwdArgs p) {
  using R = BwdRing<KP>;
  constexpr int NF = R::NF;
  __shared__ __attribute__((aligned(16))) uint16_t ring[2][R::N * kFrag];
  __shared__ __attribute__((aligned(16))) float s[TILES][4][kC];
  __shared__ __attribute__((aligned(16))) uint16_t kept[TILES][BackChain<A, KP, true>::KEEP ? KP / 16 * kFrag : 1];
  static_assert(sizeof(ring) + sizeof(s) + sizeof(kept) <= mscan::kLdsBytes, "LDS");
  const Dims& d = p.d;
  const int wv = wave_id();
  const PassPlace<A> w(d, TILES, wv < TILES ? wv : 0);
  const int64_t last = d.nc - 1;
  if (wv >= TILES) {
    const int first = wv - TILES;
    auto copy = [&](int64_t c) {
      uint16_t* dst = ring[c & 1];
      const int64_t gi = (w.bg * d.nc + c) * (NF * kFrag), ci = (w.bh * d.nc + c) * (12 * kFrag);
      copy_frags<NF, kCopyWaves>(dst + R::KF * kFrag, p.w.KF + gi, first, w.lane);
      copy_frags<12, kCopyWaves>(dst + R::PT * kFrag, p.w.PT + ci, first, w.lane);
      copy_frags<12, kCopyWaves>(dst + R::TT * kFrag, p.w.TT + ci, first, w.lane);
      copy_frags<NF, kCopyWaves>(dst + R::QF * kFrag, p.w.QF + gi, first, w.lane);
      wait_copies();
    };
    copy(last);
    mscan::lds_barrier();
    for (int64_t c = last; c >= 0; --c) {
      if (c > 0) copy(c - 1);
      mscan::lds_barrier();   // chunk c - 1 is there, and chunk c's readers are done
    }
    return;
  }
  const float so = p.so[w.bh], rso = 1.0f / so, rps = 1.0f / d.pscale, soc = w.ok ? so : 0.0f;
  const bool live = w.col < d.VP;   // a head's last workgroup may have tiles behind its columns
  BackChain<A, KP, true> ch;
  ch.kept = kept[wv];
  if (live) ch.init(p, w);
  mscan::lds_barrier();
  for (int64_t c = last; c >= 0; --c) {
    if (live) {
      ch.ring = ring[c & 1] + w.lane * 8;
      ch.ring_t = ring[c & 1] + trans_lane(w.lane);
      ch.step(p, w, c, soc, rso, rps, s[wv]);
    }
    mscan::lds_barrier();
  }
}

// ------------------------------------------------------------------ the chunks' own gradients
// One workgroup per (batch row, query / key head, chunk), over the value heads that share it.  First all products
// with d_v contracted, in slabs of 32 columns: rows of dO, U and Y through LDS (the next slab's in flight), S and dS'
// from global memory straight into the fragments of the wave that owns their d_k rows.  Then the 64 x 64 gradients
// M1 and M2 (ten lower tiles over the waves), and their products with q and k.  Bound by HBM: per chunk and head 320 KB
// at d_k = d_v = 128, S, dS', U and Y being 192 of them (80 heads of 8192 tokens: 3.3 GB in 790 us, 4.2 TB/s, two
// workgroups a CU; eight waves of half the d_k rows each took 1257).
constexpr int kSlab = 32 + 8;

template <Act A>
struct ChunkLds {
  static constexpr int NP = A == Act::F32 ? 2 : 1;
  union {
    struct {
      uint16_t dO[NP][kC * kSlab], U[2][kC * kSlab], Y[2][kC * kSlab];
    } slab[2];
    uint16_t M[8][kC * kCol];   // high and low parts of M1, its transpose, M2, its transpose
  };
  double G[kC], rowE[10][16], colE[10][16];   // E's sums, by lower tile
  float beta[kC], e[kC], dec[kC], rk[kC], rq[kC], pk[kC], pq[kC], db[kC];
  float red[2][8];

  // four floats in the padding of row i of plane n: the waves' row sums
  __device__ __forceinline__ f32x4& pad(int n, int i) { return *reinterpret_cast<f32x4*>(M[n] + i * kCol + kC); }
};
enum { M_1 = 0, M_1T = 2, M_2 = 4, M_2T = 6 };

__device__ __forceinline__ u32x2 low_halves(u32x4 a) {   // of packed words: the high parts of four values
  return u32x2{__builtin_amdgcn_perm(a[1], a[0], 0x05040100), __builtin_amdgcn_perm(a[3], a[2], 0x05040100)};
}
__device__ __forceinline__ u32x2 high_halves(u32x4 a) {
  return u32x2{__builtin_amdgcn_perm(a[1], a[0], 0x07060302), __builtin_amdgcn_perm(a[3], a[2], 0x07060302)};
}
__device__ __forceinline__ h8 join(u32x2 a, u32x2 b) { return __builtin_bit_cast(h8, (u32x4{a[0], a[1], b[0], b[1]})); }

// lower tile number n of ten: row tile, column tile
__device__ __forceinline__ int lower_row(int n) { return n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3; }
__device__ __forceinline__ int lower_col(int n) { return n - lower_row(n) * (lower_row(n) + 1) / 2; }

template <Act A, int KP, bool SHARED>
__global__ void __launch_bounds__(256, SHARED && KP == 128 ? 1 : 2) gdelta_bwd_chunk_kernel(const BwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, KS = KP / 32, NF = KP / 8, NW = 4, NTHR = NW * 64, NT = KP / 64;   // NT tiles of 16 d_k rows to a wave
  constexpr int CPT = 64 * 32 / NTHR, SUB = CPT / 4, TILES = (10 + NW - 1) / NW;   // a thread's columns of a slab, in fours
  __shared__ __attribute__((aligned(16))) ChunkLds<A> s;
  static_assert(sizeof(s) <= mscan::kLdsBytes / 2, "two workgroups a CU");
  const Dims& d = p.d;
  int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wv = wave_id();
  const ChunkPlace at_ = chunk_place(blockIdx.x, static_cast<uint32_t>(d.G), static_cast<uint32_t>(d.nc));
  const int64_t c = at_.c, hk = at_.h, b = at_.b, bg = b * d.G + hk;
  const int64_t t0 = c * kC, left = d.T - t0, gi = bg * d.nc + c;
  const int share = SHARED ? static_cast<int>(d.H / d.G) : 1;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* gsc = p.w.gsc + gi * (kGroupSc * kC);
  f32x4 totQ[4][NT], totK[4][NT];
  h8 kt[NT][NP][2], qt[NT][NP][2];   // elements 0 .. 3: token rows 4 g + e of tile 2 ks, 4 .. 7: of tile 2 ks + 1
  auto elem = [](const h8 (&x)[NP][2], int mt, int e, float f, float acc) {   // acc + f x, of the parts as they are
    acc = fmaf(f, static_cast<float>(x[0][mt >> 1][(mt & 1) * 4 + e]), acc);
    if (NP == 2) acc = fmaf(f, static_cast<float>(x[NP - 1][mt >> 1][(mt & 1) * 4 + e]), acc);
    return acc;
  };

#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int n = 0; n < NT; ++n) totQ[mt][n] = totK[mt][n] = zero;
#pragma clang loop unroll(disable)
  for (int hi_ = 0; hi_ < share; ++hi_) {
    const int64_t h = hk * share + hi_, bh = b * d.H + h, ci = bh * d.nc + c;
    int64_t fo = gi * (NP * NF * kFrag);
    if (SHARED) {   // or the heads' loop keeps every fragment of k and q, and every lane's addresses, in registers
      asm volatile("" : "+s"(fo), "+v"(tid));
      lane = tid & 63;
      r = lane & 15;
      g = lane >> 4;
    }
    const uint16_t* KF = p.w.KF + fo;
    const uint16_t* QF = p.w.QF + fo;
    const uint16_t* KT = p.w.KT + fo;
    const uint16_t* QT = p.w.QT + fo;
    const float so = p.so[bh], rs1 = 1.0f / so, rs2 = 1.0f / p.w.sv[bh];   // two factors: their product may leave f32's range
    f32x4 aP[TILES], aA[TILES], aQ[4][NT], aKq[4][NT], aKs[4][NT];
#pragma unroll
    for (int i = 0; i < TILES; ++i) aP[i] = aA[i] = zero;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n) aQ[mt][n] = aKq[mt][n] = aKs[mt][n] = zero;
    float dot = 0.0f;   // <dS', S>
    const int t = tid / (32 / CPT), cc = tid % (32 / CPT) * CPT;
    u32x4 ru[SUB], ry[SUB], rs[NT][2], rd[NT][2];
    uint32_t ro[SUB][NP * 2];
    const Buf bu = buf_of(p.w.U + ci * kC * d.VP), by = buf_of(p.DU + ci * kC * d.VP);
    const Buf bs = buf_of(p.w.S + (ci * KP + 16 * NT * wv) * d.VP), bd = buf_of(p.DS + (ci * KP + 16 * NT * wv) * d.VP);
    const Buf bo = buf_of(static_cast<const char*>(p.dy) + ((b * d.T + t0) * d.H + h) * (d.V * (NP * 2)));
    const int uoff = (t * d.VP + cc) * 4, soff = (r * d.VP + 8 * g) * 4;
    const int ooff = (t * static_cast<int>(d.H) * d.V + cc) * (NP * 2);
    auto load_rows = [&](int v0) {
#pragma unroll
      for (int i = 0; i < SUB; ++i) {
        ru[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(bu, uoff + 16 * i, v0 * 4, 0));
        ry[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(by, uoff + 16 * i, v0 * 4, 0));
#pragma unroll
        for (int k = 0; k < NP * 2; ++k) ro[i][k] = 0u;
        if (t < left && v0 + cc + 4 * i < d.V) {
          const int at_ = ooff + i * NP * 8;
          if constexpr (NP == 2) {
            const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(bo, at_, v0 * 4, 0));
#pragma unroll
            for (int k = 0; k < 4; ++k) ro[i][k] = x[k];
          } else {
            const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(bo, at_, v0 * 2, 0));
            ro[i][0] = x[0];
            ro[i][1] = x[1];
          }
        }
      }
    };
    auto load_states = [&](int v0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          rs[n][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(bs, soff + 16 * i, (v0 + 16 * n * d.VP) * 4, 0));
          rd[n][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(bd, soff + 16 * i, (v0 + 16 * n * d.VP) * 4, 0));
        }
    };
    load_rows(0);
    load_states(0);
    if (tid < kC) {
      const float* sc = p.w.hsc + ci * (kHeadSc * kC);
      const double G = p.w.G[ci * kC + tid], Gl = p.w.G[ci * kC + kC - 1];
      s.G[tid] = G;
      s.beta[tid] = sc[H_BETA * kC + tid];
      s.e[tid] = sc[H_E * kC + tid];
      s.dec[tid] = exp2_fast(static_cast<float>(Gl - G));
      s.rk[tid] = gsc[G_RK * kC + tid];
      s.rq[tid] = gsc[G_RQ * kC + tid];
      s.pk[tid] = gsc[G_PK * kC + tid];
      s.pq[tid] = gsc[G_PQ * kC + tid];
    }
    // what the decay's gradient reads at the end
    const float rate = exp2_fast(p.a_log[h] * kLog2e), bias = p.dt_bias[h];
    const float a_raw = tid < kC && tid < left ? p.a_raw[(b * d.T + t0 + tid) * d.H + h] : 0.0f;
    for (int v0 = 0; v0 < d.VP; v0 += 32) {
      auto& sl = s.slab[(v0 >> 5) & 1];
#pragma unroll
      for (int i = 0; i < SUB; ++i) {
        const int at_ = t * kSlab + cc + 4 * i;
        *reinterpret_cast<u32x2*>(sl.U[0] + at_) = low_halves(ru[i]);
        *reinterpret_cast<u32x2*>(sl.U[1] + at_) = high_halves(ru[i]);
        *reinterpret_cast<u32x2*>(sl.Y[0] + at_) = low_halves(ry[i]);
        *reinterpret_cast<u32x2*>(sl.Y[1] + at_) = high_halves(ry[i]);
        u32x2 hi, lo;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x, y;
          if constexpr (NP == 2) {
            x = __builtin_bit_cast(float, ro[i][2 * e]);
            y = __builtin_bit_cast(float, ro[i][2 * e + 1]);
          } else {
            x = IO<A>::cvt(ro[i][e] & 0xffffu);
            y = IO<A>::cvt(ro[i][e] >> 16);
          }
          uint32_t a, bb;
          split2(x * so, y * so, a, bb);
          hi[e] = a;
          lo[e] = bb;
        }
        *reinterpret_cast<u32x2*>(sl.dO[0] + at_) = hi;
        if (NP == 2) *reinterpret_cast<u32x2*>(sl.dO[NP - 1] + at_) = lo;
      }
      h8 sh[NT], slo[NT], gh[NT], gl[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sh[n] = join(low_halves(rs[n][0]), low_halves(rs[n][1]));
        slo[n] = join(high_halves(rs[n][0]), high_halves(rs[n][1]));
        gh[n] = join(low_halves(rd[n][0]), low_halves(rd[n][1]));
        gl[n] = join(high_halves(rd[n][0]), high_halves(rd[n][1]));
      }
      const int next = v0 + 32 < d.VP ? v0 + 32 : v0;   // the last slab loads its own again: no branch
      load_rows(next);
      load_states(next);
      mscan::lds_barrier();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot = fmaf(static_cast<float>(sh[n][e]), static_cast<float>(gh[n][e]), dot);
          dot = fmaf(static_cast<float>(sh[n][e]), static_cast<float>(gl[n][e]), dot);
          dot = fmaf(static_cast<float>(slo[n][e]), static_cast<float>(gh[n][e]), dot);
        }
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const int a = (16 * mt + r) * kSlab + 8 * g;
        const h8 oh = ld8(sl.dO[0] + a), uh = ld8(sl.U[0] + a), ul = ld8(sl.U[1] + a);
        const h8 yh = ld8(sl.Y[0] + a), yl = ld8(sl.Y[1] + a);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          aQ[mt][n] = mma(oh, sh[n], aQ[mt][n]);
          aKq[mt][n] = mma(yh, sh[n], aKq[mt][n]);
          aKs[mt][n] = mma(uh, gh[n], aKs[mt][n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          aQ[mt][n] = mma(oh, slo[n], aQ[mt][n]);
          aKq[mt][n] = mma(yh, slo[n], aKq[mt][n]);
          aKs[mt][n] = mma(uh, gl[n], aKs[mt][n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (NP == 2) aQ[mt][n] = mma(ld8(sl.dO[NP - 1] + a), sh[n], aQ[mt][n]);
          aKq[mt][n] = mma(yl, sh[n], aKq[mt][n]);
          aKs[mt][n] = mma(ul, gh[n], aKs[mt][n]);
        }
      }
#pragma unroll
      for (int i = 0; i < TILES; ++i) {   // lower tiles wv, wv + NW, ..
        const int tl = min(wv + NW * i, 9);
        const int a = (16 * lower_row(tl) + r) * kSlab + 8 * g, bb = (16 * lower_col(tl) + r) * kSlab + 8 * g;
        const h8 oh = ld8(sl.dO[0] + a), yh = ld8(sl.Y[0] + a), yl = ld8(sl.Y[1] + a);
        const h8 uh = ld8(sl.U[0] + bb), ul = ld8(sl.U[1] + bb);
        aP[i] = mma(oh, uh, aP[i]);
        aA[i] = mma(yh, uh, aA[i]);
        aP[i] = mma(oh, ul, aP[i]);
        aA[i] = mma(yh, ul, aA[i]);
        if (NP == 2) aP[i] = mma(ld8(sl.dO[NP - 1] + a), uh, aP[i]);
        aA[i] = mma(yl, uh, aA[i]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int pl = 0; pl < NP; ++pl)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          kt[n][pl][ks] = at<h8>(KT + (pl * NF + 2 * (NT * wv + n) + ks) * kFrag, lane * 16);
          qt[n][pl][ks] = at<h8>(QT + (pl * NF + 2 * (NT * wv + n) + ks) * kFrag, lane * 16);
        }
    // this wave's tiles of the 64 x 64 gradients, and of E
    f32x4 m1[TILES], m2[TILES];
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      m1[i] = m2[i] = zero;
      const bool mine = wv + NW * i < 10;   // else the last tile again, for nothing: one path for all waves
      const int tl = mine ? wv + NW * i : 9;
      const int mt = lower_row(tl), nt = lower_col(tl), j = 16 * nt + r, i0 = 16 * mt + 4 * g;
      const f32x4 kq = frag_mm<NP, KS, NF>(QF + mt * KS * kFrag, KF + nt * KS * kFrag, lane, zero);
      const f32x4 kk = frag_mm<NP, KS, NF>(KF + mt * KS * kFrag, KF + nt * KS * kFrag, lane, zero);
      const f32x4 rq = *reinterpret_cast<const f32x4*>(s.rq + i0), rk = *reinterpret_cast<const f32x4*>(s.rk + i0);
      const f32x4 be = *reinterpret_cast<const f32x4*>(s.beta + i0);
      const float rkj = s.rk[j];
      const double Gj = s.G[j];
      float db = 0.0f;
      double ce = 0.0, re[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ti = i0 + e;
        const float D = j <= ti ? exp2_fast(static_cast<float>(s.G[ti] - Gj)) : 0.0f;
        const float dP = aP[i][e] * rs1 * rs2, yu = aA[i][e] * rs1 * rs2;
        float E = 0.0f;
        m1[i][e] = j <= ti ? dP * D : 0.0f;
        if (j < ti) {
          m2[i][e] = -yu * be[e] * D;
          E = m1[i][e] * (rq[e] * rkj * kq[e]) + m2[i][e] * (rk[e] * rkj * kk[e]);
        }
        db = ti == j ? yu * (1.0f - be[e]) : db;
        // the sums over rows and over columns cancel where a token's g stands between neither or both of a pair: in
        // f64 they do so to the last bit of E
        ce += static_cast<double>(E);
        re[e] = sum16(static_cast<double>(E));
        big = max_finite(big, fmaxf(fabsf(m1[i][e]), fabsf(m2[i][e])) * fmaxf(rkj, fmaxf(fabsf(rq[e]), rk[e])));
      }
      ce += __shfl_xor(ce, 16, 64);
      ce += __shfl_xor(ce, 32, 64);
      if (mine) {
        if (r == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s.rowE[tl][4 * g + e] = re[e];
        }
        if (g == 0) s.colE[tl][r] = ce;
        if (mt == nt && r >> 2 == g) s.db[j] = db;
      }
    }
    big = wave_max(big);
    dot = wave_sum(dot);
    if (lane == 0) {
      s.red[0][wv] = big;
      s.red[1][wv] = dot;
    }
    __syncthreads();   // the slabs are read, s.red written
    big = dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      big = fmaxf(big, s.red[0][i]);
      dot += s.red[1][i];
    }
    const float sm = pow2_below(big, 13), rsm = 1.0f / sm;
    if (tid < 256) {   // zeros in the tiles past the diagonal that a 32-wide step reads: (0, 1), (2, 3), and (1, 0), (3, 2) of the transposes
      const int pl = tid >> 7, tile = (tid >> 6) & 1, row = (tid >> 2) & 15, q = tid & 3;
      const int up = (32 * tile + row) * kCol + 32 * tile + 8 * q + 4, dn = (32 * tile + 16 + row) * kCol + 32 * tile + 8 * q;
      *reinterpret_cast<u32x2*>(s.M[M_1 + pl] + up) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(s.M[M_2 + pl] + up) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(s.M[M_1T + pl] + dn) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(s.M[M_2T + pl] + dn) = u32x2{0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int tl = wv + NW * i;
      if (tl >= 10) break;
      const int j = 16 * lower_col(tl) + r, i0 = 16 * lower_row(tl) + 4 * g;
      const float rkj = s.rk[j];
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const f32x4 m = (which ? m2[i] : m1[i]) * sm, ri = *reinterpret_cast<const f32x4*>((which ? s.rk : s.rq) + i0);
        uint16_t* hp = s.M[which ? M_2 : M_1] + i0 * kCol + place(j);
        uint16_t* tp = s.M[which ? M_2T : M_1T] + j * kCol + place(i0);
        u32x2 th, tlo;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          uint32_t hh, ll, x, y;
          split2(m[2 * o] * rkj, m[2 * o + 1] * rkj, hh, ll);
          split2(m[2 * o] * ri[2 * o], m[2 * o + 1] * ri[2 * o + 1], x, y);
          th[o] = x;
          tlo[o] = y;
          hp[(2 * o) * kCol] = static_cast<uint16_t>(hh);
          hp[(2 * o + 1) * kCol] = static_cast<uint16_t>(hh >> 16);
          hp[kC * kCol + (2 * o) * kCol] = static_cast<uint16_t>(ll);
          hp[kC * kCol + (2 * o + 1) * kCol] = static_cast<uint16_t>(ll >> 16);
        }
        *reinterpret_cast<u32x2*>(tp) = th;
        *reinterpret_cast<u32x2*>(tp + kC * kCol) = tlo;
      }
    }
    // the parts through the state, in true units, and their products with q and k for the decay's gradient
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const int i0 = 16 * mt + 4 * g;
      const f32x4 ev = *reinterpret_cast<const f32x4*>(s.e + i0), be = *reinterpret_cast<const f32x4*>(s.beta + i0);
      const f32x4 de = *reinterpret_cast<const f32x4*>(s.dec + i0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        aQ[mt][n] = aQ[mt][n] * (ev * rs1) * rs2;
        aKq[mt][n] = aKq[mt][n] * (ev * be * -rs1) * rs2;
        aKs[mt][n] = aKs[mt][n] * (de * rs1) * rs2;
      }
      f32x4 sums[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float wq = 0.0f, wkq = 0.0f, wks = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          wq = elem(qt[n], mt, e, aQ[mt][n][e], wq);
          wkq = elem(kt[n], mt, e, aKq[mt][n][e], wkq);
          wks = elem(kt[n], mt, e, aKs[mt][n][e], wks);
        }
        sums[e] = f32x4{sum16(wq), sum16(wkq), sum16(wks), 0.0f};
      }
      if (r == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s.pad(wv, i0 + e) = sums[e];
      }
    }
    mscan::lds_barrier();
    // the parts inside the chunk
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      f32x4 q[NT], k[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        q[n] = aQ[mt][n] * sm;
        k[n] = (aKq[mt][n] + aKs[mt][n]) * sm;
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int a = (16 * mt + r) * kCol + 8 * g + 32 * ks;
        if (ks == 0 || mt >= 2) {   // rows i, columns j <= i
          const h8 xh = ld8(s.M[M_1] + a), xl = ld8(s.M[M_1 + 1] + a), yh = ld8(s.M[M_2] + a), yl = ld8(s.M[M_2 + 1] + a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            q[n] = mma(xh, kt[n][0][ks], q[n]);
            k[n] = mma(yh, kt[n][0][ks], k[n]);
            q[n] = mma(xl, kt[n][0][ks], q[n]);
            k[n] = mma(yl, kt[n][0][ks], k[n]);
            if (NP == 2) {
              q[n] = mma(xh, kt[n][NP - 1][ks], q[n]);
              k[n] = mma(yh, kt[n][NP - 1][ks], k[n]);
            }
          }
        }
        if (ks == 1 || mt < 2) {    // rows j, columns i >= j
          const h8 xh = ld8(s.M[M_1T] + a), xl = ld8(s.M[M_1T + 1] + a), yh = ld8(s.M[M_2T] + a), yl = ld8(s.M[M_2T + 1] + a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            k[n] = mma(xh, qt[n][0][ks], k[n]);
            k[n] = mma(xl, qt[n][0][ks], k[n]);
            k[n] = mma(yh, kt[n][0][ks], k[n]);
            k[n] = mma(yl, kt[n][0][ks], k[n]);
            if (NP == 2) {
              k[n] = mma(xh, qt[n][NP - 1][ks], k[n]);
              k[n] = mma(yh, kt[n][NP - 1][ks], k[n]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        totQ[mt][n] = SHARED ? totQ[mt][n] + q[n] * rsm : q[n] * rsm;
        totK[mt][n] = SHARED ? totK[mt][n] + k[n] * rsm : k[n] * rsm;
      }
    }
    if (tid < kC) {   // dg and what comes of it
      float x = 0.0f, z = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const f32x4 v = s.pad(w, tid);
        x += v[0] * s.rq[tid] + v[1] * s.rk[tid];
        z += v[2] * s.rk[tid];
      }
      double E = 0.0;
#pragma unroll
      for (int n = 0; n < 10; ++n) {
        if (lower_row(n) == (tid >> 4)) E += s.rowE[n][tid & 15];
        if (lower_col(n) == (tid >> 4)) E -= s.colE[n][tid & 15];
      }
      double dg = E + static_cast<double>(x);   // summed over this and the later tokens
      float before = z;                         // and this over the earlier ones
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_down(dg, o, 64);
        const float dn = __shfl_up(before, o, 64);
        if (tid + o < 64) dg += up;
        if (tid >= o) before += dn;
      }
      float dgt = static_cast<float>(dg + static_cast<double>(before - z) + static_cast<double>(s.e[kC - 1] * (dot * rs1 * rs2)));
      if (!p.has_h0 && c == 0 && tid == 0) dgt = 0.0f;   // the first token's decay meets no state: exactly zero
      float pa = 0.0f, pb = 0.0f;
      if (tid < left) {
        const int64_t i = (b * d.T + t0 + tid) * d.H + h;
        const float z2 = a_raw + bias;
        const float da = -rate * mscan::sigmoid(z2) * dgt;
        p.d_a_raw[i] = da;
        p.d_b_raw[i] = s.db[tid];
        pa = -rate * mscan::softplus(z2) * dgt;
        pb = da;
      }
      pa = wave_sum(pa);
      pb = wave_sum(pb);
      if (tid == 0) {
        p.part[ci * 2] = pa;
        p.part[ci * 2 + 1] = pb;
      }
    }
    __syncthreads();   // M, its padding and the scalars are read
  }
  // unit length's adjoint: r (d - n (n . d))
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    f32x4 sums[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float wq = 0.0f, wk = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        wq = elem(qt[n], mt, e, totQ[mt][n][e], wq);
        wk = elem(kt[n], mt, e, totK[mt][n][e], wk);
      }
      sums[e] = f32x4{sum16(wq), sum16(wk), 0.0f, 0.0f};
    }
    if (r == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s.pad(wv, 16 * mt + 4 * g + e) = sums[e];
    }
  }
  __syncthreads();
  const float rscale = 1.0f / d.scale;
  const int64_t qk = ((b * d.T + t0) * d.G + hk) * d.K;
  const int row = static_cast<int>(d.G) * d.K;   // elements from token to token
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const int i0 = 16 * mt + 4 * g;
    const f32x4 pq = *reinterpret_cast<const f32x4*>(s.pq + i0), rq = *reinterpret_cast<const f32x4*>(s.rq + i0);
    const f32x4 pk = *reinterpret_cast<const f32x4*>(s.pk + i0), rk = *reinterpret_cast<const f32x4*>(s.rk + i0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f32x4 w = s.pad(0, i0 + e);
#pragma unroll
      for (int n = 1; n < NW; ++n) w += s.pad(n, i0 + e);
      const float un = rq[e] * rscale, fq = -w[0] * un * un, fk = -w[1] * rk[e] * rk[e];
      const bool in = i0 + e < left;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = 16 * (NT * wv + n) + r;
        const float vq = rq[e] * elem(qt[n], mt, e, fq, totQ[mt][n][e]) * pq[e];
        const float vk = rk[e] * elem(kt[n], mt, e, fk, totK[mt][n][e]) * pk[e];
        if (in && col < d.K) {
          const int64_t o = qk + (i0 + e) * row + col;
          IO<A>::st(p.d_q, o, vq);
          IO<A>::st(p.d_k, o, vk);
        }
      }
    }
  }
}

// d_a_log, d_dt_bias: one workgroup per head adds its chunks' terms in a fixed order
__global__ void __launch_bounds__(256) gdelta_params_kernel(const BwdArgs p) {
  __shared__ float s[2][4];
  const Dims& d = p.d;
  const int tid = threadIdx.x;
  const int64_t h = blockIdx.x;
  float a = 0.0f, b = 0.0f;
  for (int64_t i = tid; i < d.B * d.nc; i += 256) {
    const int64_t ci = ((i / d.nc) * d.H + h) * d.nc + i % d.nc;
    a += p.part[ci * 2];
    b += p.part[ci * 2 + 1];
  }
  a = wave_sum(a);
  b = wave_sum(b);
  if ((tid & 63) == 0) {
    s[0][tid >> 6] = a;
    s[1][tid >> 6] = b;
  }
  __syncthreads();
  if (tid == 0) {
    p.d_a_log[h] += (s[0][0] + s[0][1]) + (s[0][2] + s[0][3]);
    p.d_dt_bias[h] += (s[1][0] + s[1][1]) + (s[1][2] + s[1][3]);
  }
}

// ------------------------------------------------------------------ launches
namespace {

template <Act A, int KP>
hipError_t launch(const BwdArgs& a, hipStream_t st) {
  const Dims& d = a.d;
  const unsigned bh = static_cast<unsigned>(d.B * d.H), nc = static_cast<unsigned>(d.nc);
  hipLaunchKernelGGL((gdelta_dymax_kernel<A>), dim3(bh * nc), dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gdelta_dscale_kernel, dim3(bh), dim3(64), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned tiles = d.VP / 16;
  if constexpr (A == Act::F32) {   // two planes a family: a chunk's fragments twice are more than the LDS
    hipLaunchKernelGGL((gdelta_bwd_state_kernel<A, KP>), dim3(bh * tiles), dim3(64), 0, st, a);
  } else {
    ring_tiles<true>(bh, tiles, [&](auto n, unsigned grid) {
      constexpr int N = decltype(n)::value;
      hipLaunchKernelGGL((gdelta_bwd_ring_kernel<A, KP, N>), dim3(grid), dim3(64 * (N + kCopyWaves)), 0, st, a);
    });
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>(d.B * d.G) * nc);
  if (d.H == d.G) hipLaunchKernelGGL((gdelta_bwd_chunk_kernel<A, KP, false>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((gdelta_bwd_chunk_kernel<A, KP, true>), grid, dim3(256), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(gdelta_params_kernel, dim3(static_cast<unsigned>(d.H)), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <Act A>
hipError_t launch_kp(const BwdArgs& a, hipStream_t st) {
  return a.d.K <= 64 ? launch<A, 64>(a, st) : launch<A, 128>(a, st);
}

}  // namespace

hipError_t launch_bwd(Act act, const BwdArgs& a, hipStream_t st) {
  switch (act) {
    case Act::F32: return launch_kp<Act::F32>(a, st);
    case Act::BF16: return launch_kp<Act::BF16>(a, st);
    default: return launch_kp<Act::F16>(a, st);
  }
}

}  // namespace gdelta
