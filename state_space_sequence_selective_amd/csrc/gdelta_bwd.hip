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
#include <type_traits>

#include "gdelta_launch.h"

namespace gdelta {

// ------------------------------------------------------------------ scale of dS and Y
template <Act A>
__global__ void __launch_bounds__(256) gdelta_dymax_kernel(const BwdArgs p) {
  __shared__ float s[4];
  const Dims& d = p.d;
  const int tid = threadIdx.x;
  const int64_t c = blockIdx.x % d.nc, bh = blockIdx.x / d.nc, h = bh % d.H, b = bh / d.H;
  const int64_t t0 = c * kC, left = d.T - t0;
  const int nv = d.V / 8, rows = left < kC ? static_cast<int>(left) : kC;
  float m = 0.0f;
  for (int i = tid; i < rows * nv; i += 256) {
    float x[8];
    load8<A>(p.dy, ((b * d.T + t0 + i / nv) * d.H + h) * d.V + (i % nv) * 8, true, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_finite(m, x[e]);
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
// As the forward's pass: a wave holds 16 columns of dS^T and needs nothing of any other.
template <Act A, int KP>
__global__ void __launch_bounds__(64) gdelta_bwd_state_kernel(const BwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, MT = KP / 16, KS = KP / 32, NF = KP / 8;
  constexpr bool AHEAD = NP == 1;
  using Raw = std::conditional_t<A == Act::F32, uint32_t, uint16_t>;
  constexpr int ES = sizeof(Raw);
  __shared__ __attribute__((aligned(16))) float s[4][kC];   // beta; beta e rk; exp(G_63 - G) rk; e rq
  const Dims& d = p.d;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  uint32_t head, cb;
  xcd_head(blockIdx.x, d.VP / 16, static_cast<uint32_t>(d.B * d.H), head, cb);
  const uint32_t H = static_cast<uint32_t>(d.H), G = static_cast<uint32_t>(d.G);
  const int64_t bh = head, h = head % H, b = head / H, bg = b * G + (head % H) / (H / G);
  const int col = cb * 16 + r;
  const bool ok = col < d.V;
  const int vrow = static_cast<int>(d.H) * d.V * ES, vcol = (ok ? col : d.V - 1) * ES;
  const int poff = (4 * g * d.VP + col) * 4;
  const float so = p.so[bh], rso = 1.0f / so, rps = 1.0f / d.pscale, soc = ok ? so : 0.0f;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 dS[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) dS[mt] = zero;
  h8 kf[NF], kt[NF], qt[NF], ph[6], pl[6], th[6], tl[6];
  float sc[4], el;
  uint32_t v[4][4];
  auto KFp = [&](int64_t c) { return p.w.KF + (bg * d.nc + c) * (NP * NF * kFrag); };
  auto KTp = [&](int64_t c) { return p.w.KT + (bg * d.nc + c) * (NP * NF * kFrag); };
  auto QTp = [&](int64_t c) { return p.w.QT + (bg * d.nc + c) * (NP * NF * kFrag); };
  auto load_p = [&](int64_t c) {
    const uint16_t* x = p.w.PT + (bh * d.nc + c) * (12 * kFrag);
    load_frags(ph, x, lane);
    load_frags(pl, x + 6 * kFrag, lane);
  };
  auto load_t = [&](int64_t c) {
    const uint16_t* x = p.w.TT + (bh * d.nc + c) * (12 * kFrag);
    load_frags(th, x, lane);
    load_frags(tl, x + 6 * kFrag, lane);
  };
  auto load_sc = [&](int64_t c) {
    const float* x = p.w.hsc + (bh * d.nc + c) * (kHeadSc * kC);
    sc[0] = x[H_BETA * kC + lane];
    sc[1] = x[H_BK * kC + lane];
    sc[2] = x[H_DK * kC + lane];
    sc[3] = x[H_EQ * kC + lane];
    el = x[H_E * kC + kC - 1];
  };
  auto load_v = [&](int64_t c) {
    load_cols<Raw>(v, static_cast<const char*>(p.dy) + ((b * d.T + c * kC) * d.H + h) * (d.V * ES), vrow, vcol, d.T - c * kC, g);
  };
  if (AHEAD) {
    load_frags(kf, KFp(d.nc - 1), lane);
    load_p(d.nc - 1);
    load_t(d.nc - 1);
    load_frags(kt, KTp(d.nc - 1), lane);
    load_frags(qt, QTp(d.nc - 1), lane);
  }
  load_sc(d.nc - 1);
  load_v(d.nc - 1);
  for (int64_t c = d.nc - 1; c >= 0; --c) {
    const int64_t left = d.T - c * kC, ci = bh * d.nc + c;
    const bool more = AHEAD && c > 0;
    mscan::wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][lane] = sc[i];
    mscan::wave_lds_sync();
    const float elc = el;
    if (c > 0) load_sc(c - 1);
    if (!AHEAD) {
      load_frags(kf, KFp(c), lane);
      load_p(c);
    }
    f32x4 dU[4] = {zero, zero, zero, zero}, pd[4] = {zero, zero, zero, zero}, dO[4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag f = to_b(dS[2 * ks], dS[2 * ks + 1]);
      store_packed(p.DS + (ci * KP + 32 * ks) * d.VP, poff, f, d.VP);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) dU[mt] = mma(kf[mt * KS + ks], f.hi, dU[mt]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) dU[mt] = mma(kf[mt * KS + ks], f.lo, dU[mt]);
      if (NP == 2) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) dU[mt] = mma(at<h8>(KFp(c) + (NF + mt * KS + ks) * kFrag, lane * 16), f.hi, dU[mt]);
      }
    }
    if (more) load_frags(kf, KFp(c - 1), lane);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) dO[mt][e] = IO<A>::cvt(v[mt][e]) * soc;
    if (c > 0) load_v(c - 1);
    const Frag o0 = to_b(dO[0], dO[1]), o1 = to_b(dO[2], dO[3]);   // 16-bit input: the low parts are zero
#pragma unroll
    for (int f = 0; f < 6; ++f) pd[kUm[f]] = mma(ph[f], (kUk[f] ? o1 : o0).hi, pd[kUm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) pd[kUm[f]] = mma(pl[f], (kUk[f] ? o1 : o0).hi, pd[kUm[f]]);
    if (NP == 2) {
#pragma unroll
      for (int f = 0; f < 6; ++f) pd[kUm[f]] = mma(ph[f], (kUk[f] ? o1 : o0).lo, pd[kUm[f]]);
    }
    if (more) load_p(c - 1);
    if (!AHEAD) {
      load_t(c);
      load_frags(kt, KTp(c), lane);
      load_frags(qt, QTp(c), lane);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 dk = *reinterpret_cast<const f32x4*>(s[2] + 16 * mt + 4 * g), eq = *reinterpret_cast<const f32x4*>(s[3] + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dU[mt][e] = fmaf(dU[mt][e], dk[e], pd[mt][e] * rps);
        dO[mt][e] *= eq[e];
      }
    }
    const Frag u0 = to_b(dU[0], dU[1]), u1 = to_b(dU[2], dU[3]);
    f32x4 Y[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int f = 0; f < 6; ++f) Y[kUm[f]] = mma(th[f], (kUk[f] ? u1 : u0).hi, Y[kUm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) Y[kUm[f]] = mma(th[f], (kUk[f] ? u1 : u0).lo, Y[kUm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) Y[kUm[f]] = mma(tl[f], (kUk[f] ? u1 : u0).hi, Y[kUm[f]]);
    if (more) load_t(c - 1);
    // e0, e1 and the state's part of dS from dO do not wait for Y
    const Frag e0 = to_b(dO[0], dO[1]), e1 = to_b(dO[2], dO[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) dS[mt][e] *= elc;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(qt[2 * mt], e0.hi, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(qt[2 * mt], e0.lo, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(qt[2 * mt + 1], e1.hi, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(qt[2 * mt + 1], e1.lo, dS[mt]);
    if (NP == 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        dS[mt] = mma(at<h8>(QTp(c) + (NF + 2 * mt) * kFrag, lane * 16), e0.hi, dS[mt]);
        dS[mt] = mma(at<h8>(QTp(c) + (NF + 2 * mt + 1) * kFrag, lane * 16), e1.hi, dS[mt]);
      }
    }
    if (more) load_frags(qt, QTp(c - 1), lane);
    store_packed(p.DU + ci * kC * d.VP, poff, to_b(Y[0], Y[1]), d.VP);
    store_packed(p.DU + (ci * kC + 32) * d.VP, poff, to_b(Y[2], Y[3]), d.VP);
    f32x4 dv[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      dv[mt] = Y[mt] * *reinterpret_cast<const f32x4*>(s[0] + 16 * mt + 4 * g) * rso;
      Y[mt] *= -*reinterpret_cast<const f32x4*>(s[1] + 16 * mt + 4 * g);
    }
    store_cols<A>(dv, static_cast<char*>(p.d_v) + ((b * d.T + c * kC) * d.H + h) * (d.V * ES), vrow, col * ES, left, g, ok);
    const Frag y0 = to_b(Y[0], Y[1]), y1 = to_b(Y[2], Y[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(kt[2 * mt], y0.hi, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(kt[2 * mt], y0.lo, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(kt[2 * mt + 1], y1.hi, dS[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) dS[mt] = mma(kt[2 * mt + 1], y1.lo, dS[mt]);
    if (NP == 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        dS[mt] = mma(at<h8>(KTp(c) + (NF + 2 * mt) * kFrag, lane * 16), y0.hi, dS[mt]);
        dS[mt] = mma(at<h8>(KTp(c) + (NF + 2 * mt + 1) * kFrag, lane * 16), y1.hi, dS[mt]);
      }
    }
    if (more) load_frags(kt, KTp(c - 1), lane);
  }
}

// ------------------------------------------------------------------ the chunks' own gradients
// One workgroup per (batch row, query / key head, chunk), over the value heads that share it.  First all products
// with d_v contracted, in slabs of 32 columns: rows of dO, U and Y through LDS (the next slab's in flight), S and dS'
// from global memory straight into the fragments of the wave that owns their d_k rows.  Then the 64 x 64 gradients M1
// and M2 (ten lower tiles over the four waves), and their products with q and k.
constexpr int kSlab = 32 + 8;

template <Act A>
struct ChunkLds {
  static constexpr int NP = A == Act::F32 ? 2 : 1;
  union {
    struct {
      uint16_t dO[NP][kC * kSlab], U[2][kC * kSlab], Y[2][kC * kSlab];
    } slab[2];
    struct {
      uint16_t M1[2][kC * kCol], M1T[2][kC * kCol], M2[2][kC * kCol], M2T[2][kC * kCol];
    };
  };
  double G[kC];
  float beta[kC], e[kC], dec[kC], rk[kC], rq[kC], db[kC];
  float rowE[4][kC], colE[4][kC];   // by column tile, by row tile
  float rows[4][3][kC];             // by wave
  float red[8];
};

__device__ __forceinline__ void unpack8(u32x4 a, u32x4 b, h8& hi, h8& lo) {
  u32x4 h, l;
  h[0] = (a[0] & 0xffffu) | (a[1] << 16);
  h[1] = (a[2] & 0xffffu) | (a[3] << 16);
  h[2] = (b[0] & 0xffffu) | (b[1] << 16);
  h[3] = (b[2] & 0xffffu) | (b[3] << 16);
  l[0] = (a[0] >> 16) | (a[1] & 0xffff0000u);
  l[1] = (a[2] >> 16) | (a[3] & 0xffff0000u);
  l[2] = (b[0] >> 16) | (b[1] & 0xffff0000u);
  l[3] = (b[2] >> 16) | (b[3] & 0xffff0000u);
  hi = __builtin_bit_cast(h8, h);
  lo = __builtin_bit_cast(h8, l);
}

template <Act A, int KP, bool SHARED>
__global__ void __launch_bounds__(256, SHARED ? 1 : 2) gdelta_bwd_chunk_kernel(const BwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, NT = KP / 64, KS = KP / 32, NF = KP / 8;
  __shared__ __attribute__((aligned(16))) ChunkLds<A> s;
  static_assert(sizeof(s) <= mscan::kLdsBytes / 2, "two workgroups a CU");
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
  const int64_t c = blockIdx.x % d.nc, bg = blockIdx.x / d.nc, hk = bg % d.G, b = bg / d.G;
  const int64_t t0 = c * kC, left = d.T - t0, gi = bg * d.nc + c;
  const int share = SHARED ? static_cast<int>(d.H / d.G) : 1;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const int n0 = wv * NT;   // this wave's d_k tiles: n0 .. n0 + NT - 1
  const float* gsc = p.w.gsc + gi * (kGroupSc * kC);
  const uint16_t* KF = p.w.KF + gi * (NP * NF * kFrag);
  const uint16_t* QF = p.w.QF + gi * (NP * NF * kFrag);
  const uint16_t* KT = p.w.KT + gi * (NP * NF * kFrag);
  const uint16_t* QT = p.w.QT + gi * (NP * NF * kFrag);
  f32x4 totQ[4][NT], totK[4][NT];
  h8 kt[NP][NT][2], qt[NP][NT][2];   // elements 0 .. 3: token rows 4 g + e of tile 2 ks, 4 .. 7: of tile 2 ks + 1

  for (int hi_ = 0; hi_ < share; ++hi_) {
    const int64_t h = hk * share + hi_, bh = b * d.H + h, ci = bh * d.nc + c;
    const float so = p.so[bh], rso = 1.0f / so, rsv = 1.0f / p.w.sv[bh];
    f32x4 aP[3], aA[3], aQ[4][NT], aKq[4][NT], aKs[4][NT];
#pragma unroll
    for (int i = 0; i < 3; ++i) aP[i] = aA[i] = zero;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n) aQ[mt][n] = aKq[mt][n] = aKs[mt][n] = zero;
    float dot = 0.0f;   // <dS', S>
    // a thread's part of a slab: 8 columns of one token
    const int t = tid >> 2, cc = (tid & 3) * 8;
    u32x4 ru[2], ry[2], ro[NP], rs[NT][2], rd[NT][2];
    const uint32_t uoff = (t * d.VP + cc) * 4, soff = (r * d.VP + 8 * g) * 4;
    const char* dyb = static_cast<const char*>(p.dy) + ((b * d.T + t0) * d.H + h) * (d.V * (NP * 2));
    const uint32_t dyoff = (static_cast<uint32_t>(t) * static_cast<uint32_t>(d.H * d.V) + cc) * (NP * 2);
    auto load_rows = [&](int v0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ru[i] = at<u32x4>(p.w.U + ci * kC * d.VP + v0 + 4 * i, uoff);
        ry[i] = at<u32x4>(p.DU + ci * kC * d.VP + v0 + 4 * i, uoff);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        ro[i] = u32x4{0u, 0u, 0u, 0u};
        if (t < left && v0 + cc < d.V) ro[i] = at<u32x4>(dyb + v0 * (NP * 2) + 16 * i, dyoff);
      }
    };
    auto load_states = [&](int v0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          rs[n][i] = at<u32x4>(p.w.S + (ci * KP + 16 * (n0 + n)) * d.VP + v0 + 4 * i, soff);
          rd[n][i] = at<u32x4>(p.DS + (ci * KP + 16 * (n0 + n)) * d.VP + v0 + 4 * i, soff);
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
    }
    for (int v0 = 0; v0 < d.VP; v0 += 32) {
      auto& sl = s.slab[(v0 >> 5) & 1];
      {
        h8 ph, pl;
        unpack8(ru[0], ru[1], ph, pl);
        *reinterpret_cast<h8*>(sl.U[0] + t * kSlab + cc) = ph;
        *reinterpret_cast<h8*>(sl.U[1] + t * kSlab + cc) = pl;
        unpack8(ry[0], ry[1], ph, pl);
        *reinterpret_cast<h8*>(sl.Y[0] + t * kSlab + cc) = ph;
        *reinterpret_cast<h8*>(sl.Y[1] + t * kSlab + cc) = pl;
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x, y;
          if constexpr (NP == 2) {
            x = __builtin_bit_cast(float, static_cast<uint32_t>(ro[e >> 1][(e & 1) * 2]));
            y = __builtin_bit_cast(float, static_cast<uint32_t>(ro[e >> 1][(e & 1) * 2 + 1]));
          } else {
            x = IO<A>::cvt(ro[0][e] & 0xffffu);
            y = IO<A>::cvt(ro[0][e] >> 16);
          }
          uint32_t a, bb;
          split2(x * so, y * so, a, bb);
          hi[e] = a;
          lo[e] = bb;
        }
        *reinterpret_cast<u32x4*>(sl.dO[0] + t * kSlab + cc) = hi;
        if (NP == 2) *reinterpret_cast<u32x4*>(sl.dO[NP - 1] + t * kSlab + cc) = lo;
      }
      h8 sh[NT], slo[NT], gh[NT], gl[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        unpack8(rs[n][0], rs[n][1], sh[n], slo[n]);
        unpack8(rd[n][0], rd[n][1], gh[n], gl[n]);
      }
      if (v0 + 32 < d.VP) {
        load_rows(v0 + 32);
        load_states(v0 + 32);
      }
      mscan::lds_barrier();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dot = fmaf(static_cast<float>(sh[n][e]) + static_cast<float>(slo[n][e]),
                     static_cast<float>(gh[n][e]) + static_cast<float>(gl[n][e]), dot);
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
          aKq[mt][n] = mma(yl, sh[n], aKq[mt][n]);
          aKs[mt][n] = mma(ul, gh[n], aKs[mt][n]);
          if (NP == 2) aQ[mt][n] = mma(ld8(sl.dO[NP - 1] + a), sh[n], aQ[mt][n]);
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {   // lower tiles wv, wv + 4, wv + 8
        const int tl = wv + 4 * i;
        if (tl >= 10) break;
        const int mt = tl < 1 ? 0 : tl < 3 ? 1 : tl < 6 ? 2 : 3, nt = tl - mt * (mt + 1) / 2;
        const int a = (16 * mt + r) * kSlab + 8 * g, bb = (16 * nt + r) * kSlab + 8 * g;
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
    for (int pl = 0; pl < NP; ++pl)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          kt[pl][n][ks] = at<h8>(KT + (pl * NF + 2 * (n0 + n) + ks) * kFrag, lane * 16);
          qt[pl][n][ks] = at<h8>(QT + (pl * NF + 2 * (n0 + n) + ks) * kFrag, lane * 16);
        }
    // this wave's tiles of the 64 x 64 gradients, and of E
    f32x4 m1[3], m2[3];
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      m1[i] = m2[i] = zero;
      const int tl = wv + 4 * i;
      if (tl >= 10) break;
      const int mt = tl < 1 ? 0 : tl < 3 ? 1 : tl < 6 ? 2 : 3, nt = tl - mt * (mt + 1) / 2, j = 16 * nt + r;
      const f32x4 kq = frag_mm<NP, KS, NF>(QF + mt * KS * kFrag, KF + nt * KS * kFrag, lane, zero);
      const f32x4 kk = frag_mm<NP, KS, NF>(KF + mt * KS * kFrag, KF + nt * KS * kFrag, lane, zero);
      const float rkj = s.rk[j];
      const double Gj = s.G[j];
      float ce = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ti = 16 * mt + 4 * g + e;
        const float rq = s.rq[ti], rk = s.rk[ti], be = s.beta[ti];
        const float D = j <= ti ? exp2_fast(static_cast<float>(s.G[ti] - Gj)) : 0.0f;
        const float dP = aP[i][e] * rso * rsv, yu = aA[i][e] * rso * rsv;
        float E = 0.0f;
        m1[i][e] = j <= ti ? dP * D : 0.0f;
        if (j < ti) {
          m2[i][e] = -yu * be * D;
          E = m1[i][e] * (rq * rkj * kq[e]) + m2[i][e] * (rk * rkj * kk[e]);
        }
        if (ti == j) s.db[ti] = yu * (1.0f - be);
        ce += E;
        const float re = sum16(E);
        if (r == 0) s.rowE[nt][ti] = re;
        big = max_finite(big, fmaxf(fabsf(m1[i][e]), fabsf(m2[i][e])) * fmaxf(rkj, fmaxf(fabsf(rq), rk)));
      }
      ce += __shfl_xor(ce, 16, 64);
      ce += __shfl_xor(ce, 32, 64);
      if (g == 0) s.colE[mt][j] = ce;
    }
    big = wave_max(big);
    dot = wave_sum(dot);
    if (lane == 0) {
      s.red[wv] = big;
      s.red[4 + wv] = dot;
    }
    __syncthreads();   // the slabs are read, s.red written
    const float sm = pow2_below(fmaxf(fmaxf(s.red[0], s.red[1]), fmaxf(s.red[2], s.red[3])), 13), rsm = 1.0f / sm;
    dot = (s.red[4] + s.red[5]) + (s.red[6] + s.red[7]);
    {   // zeros in the tiles past the diagonal that a 32-wide step reads: (0, 1), (2, 3), and (1, 0), (3, 2) of the transposes
      const int pl = tid >> 7, tile = (tid >> 6) & 1, row = (tid >> 2) & 15, q = tid & 3;
      const int up = (32 * tile + row) * kCol + 32 * tile + 8 * q + 4, dn = (32 * tile + 16 + row) * kCol + 32 * tile + 8 * q;
      *reinterpret_cast<u32x2*>(s.M1[pl] + up) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(s.M2[pl] + up) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(s.M1T[pl] + dn) = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(s.M2T[pl] + dn) = u32x2{0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int tl = wv + 4 * i;
      if (tl >= 10) break;
      const int mt = tl < 1 ? 0 : tl < 3 ? 1 : tl < 6 ? 2 : 3, nt = tl - mt * (mt + 1) / 2, j = 16 * nt + r, i0 = 16 * mt + 4 * g;
      const float rkj = s.rk[j];
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const f32x4 m = which ? m2[i] : m1[i];
        const float* ri = (which ? s.rk : s.rq) + i0;
        const int a = i0 * kCol + place(j), at_ = j * kCol + place(i0);
        uint16_t* hp = which ? s.M2[0] : s.M1[0];
        uint16_t* lp = which ? s.M2[1] : s.M1[1];
        uint32_t th[2], tlo[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float x = m[2 * o] * sm, y = m[2 * o + 1] * sm;
          uint32_t hh, ll;
          split2(x * rkj, y * rkj, hh, ll);
          split2(x * ri[2 * o], y * ri[2 * o + 1], th[o], tlo[o]);
          hp[a + (2 * o) * kCol] = static_cast<uint16_t>(hh);
          hp[a + (2 * o + 1) * kCol] = static_cast<uint16_t>(hh >> 16);
          lp[a + (2 * o) * kCol] = static_cast<uint16_t>(ll);
          lp[a + (2 * o + 1) * kCol] = static_cast<uint16_t>(ll >> 16);
        }
        *reinterpret_cast<u32x2*>((which ? s.M2T[0] : s.M1T[0]) + at_) = u32x2{th[0], th[1]};
        *reinterpret_cast<u32x2*>((which ? s.M2T[1] : s.M1T[1]) + at_) = u32x2{tlo[0], tlo[1]};
      }
    }
    // the parts through the state, in true units, and their products with q and k for the decay's gradient
    auto elem = [&](const h8 (&x)[NP][NT][2], int n, int mt, int e) {
      float v = static_cast<float>(x[0][n][mt >> 1][(mt & 1) * 4 + e]);
      if (NP == 2) v += static_cast<float>(x[NP - 1][n][mt >> 1][(mt & 1) * 4 + e]);
      return v;
    };
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ti = 16 * mt + 4 * g + e;
        const float ev = s.e[ti], be = s.beta[ti], de = s.dec[ti];
        float wq = 0.0f, wkq = 0.0f, wks = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          aQ[mt][n][e] *= ev * rso * rsv;
          aKq[mt][n][e] *= -(ev * be) * rso * rsv;
          aKs[mt][n][e] *= de * rso * rsv;
          const float kv = elem(kt, n, mt, e);
          wq = fmaf(aQ[mt][n][e], elem(qt, n, mt, e), wq);
          wkq = fmaf(aKq[mt][n][e], kv, wkq);
          wks = fmaf(aKs[mt][n][e], kv, wks);
        }
        wq = sum16(wq);
        wkq = sum16(wkq);
        wks = sum16(wks);
        if (r == 0) {
          s.rows[wv][0][ti] = wq * s.rq[ti];
          s.rows[wv][1][ti] = wkq * s.rk[ti];
          s.rows[wv][2][ti] = wks * s.rk[ti];
        }
      }
    mscan::lds_barrier();
    // the parts inside the chunk
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      f32x4 q[NT], k[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[n][e] = aQ[mt][n][e] * sm;
          k[n][e] = (aKq[mt][n][e] + aKs[mt][n][e]) * sm;
        }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int a = (16 * mt + r) * kCol + 8 * g + 32 * ks;
        if (ks == 0 || mt >= 2) {   // rows i, columns j <= i
          const h8 xh = ld8(s.M1[0] + a), xl = ld8(s.M1[1] + a), yh = ld8(s.M2[0] + a), yl = ld8(s.M2[1] + a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            q[n] = mma(xh, kt[0][n][ks], q[n]);
            k[n] = mma(yh, kt[0][n][ks], k[n]);
            q[n] = mma(xl, kt[0][n][ks], q[n]);
            k[n] = mma(yl, kt[0][n][ks], k[n]);
            if (NP == 2) {
              q[n] = mma(xh, kt[NP - 1][n][ks], q[n]);
              k[n] = mma(yh, kt[NP - 1][n][ks], k[n]);
            }
          }
        }
        if (ks == 1 || mt < 2) {    // rows j, columns i >= j
          const h8 xh = ld8(s.M1T[0] + a), xl = ld8(s.M1T[1] + a), yh = ld8(s.M2T[0] + a), yl = ld8(s.M2T[1] + a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            k[n] = mma(xh, qt[0][n][ks], k[n]);
            k[n] = mma(xl, qt[0][n][ks], k[n]);
            k[n] = mma(yh, kt[0][n][ks], k[n]);
            k[n] = mma(yl, kt[0][n][ks], k[n]);
            if (NP == 2) {
              k[n] = mma(xh, qt[NP - 1][n][ks], k[n]);
              k[n] = mma(yh, kt[NP - 1][n][ks], k[n]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          totQ[mt][n][e] = (SHARED && hi_ ? totQ[mt][n][e] : 0.0f) + q[n][e] * rsm;
          totK[mt][n][e] = (SHARED && hi_ ? totK[mt][n][e] : 0.0f) + k[n][e] * rsm;
        }
    }
    if (tid < kC) {   // dg and what comes of it
      float x = 0.0f, z = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x += s.rows[w][0][tid] + s.rows[w][1][tid];
        z += s.rows[w][2][tid];
      }
      float E = 0.0f, C = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w <= (tid >> 4)) E += s.rowE[w][tid];
        if (w >= (tid >> 4)) C += s.colE[w][tid];
      }
      float dG = (E - C) + (x - z);
      // suffix sum over the chunk's tokens
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float up = __shfl_down(dG, o, 64);
        if (tid + o < 64) dG += up;
      }
      const float through = wave_sum(z) + s.e[kC - 1] * (dot * rso * rsv);
      float dg = dG + through;
      if (!p.has_h0 && c == 0 && tid == 0) dg = 0.0f;   // the first token's decay meets no state: exactly zero
      float pa = 0.0f, pb = 0.0f;
      if (tid < left) {
        const int64_t i = (b * d.T + t0 + tid) * d.H + h;
        const float rate = exp2_fast(p.a_log[h] * kLog2e), z2 = p.a_raw[i] + p.dt_bias[h];
        const float da = -rate * mscan::sigmoid(z2) * dg;
        p.d_a_raw[i] = da;
        p.d_b_raw[i] = s.db[tid];
        pa = -rate * mscan::softplus(z2) * dg;
        pb = da;
      }
      pa = wave_sum(pa);
      pb = wave_sum(pb);
      if (tid == 0) {
        p.part[ci * 2] = pa;
        p.part[ci * 2 + 1] = pb;
      }
    }
    __syncthreads();   // M, rows and the scalars are read
  }
  // unit length's adjoint: r (d - n (n . d))
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float wq = 0.0f, wk = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float kv = static_cast<float>(kt[0][n][mt >> 1][(mt & 1) * 4 + e]), qv = static_cast<float>(qt[0][n][mt >> 1][(mt & 1) * 4 + e]);
        if (NP == 2) {
          kv += static_cast<float>(kt[NP - 1][n][mt >> 1][(mt & 1) * 4 + e]);
          qv += static_cast<float>(qt[NP - 1][n][mt >> 1][(mt & 1) * 4 + e]);
        }
        wq = fmaf(totQ[mt][n][e], qv, wq);
        wk = fmaf(totK[mt][n][e], kv, wk);
      }
      wq = sum16(wq);
      wk = sum16(wk);
      if (r == 0) {
        s.rows[wv][0][16 * mt + 4 * g + e] = wq;
        s.rows[wv][1][16 * mt + 4 * g + e] = wk;
      }
    }
  __syncthreads();
  const float rscale = 1.0f / d.scale;
  const int64_t qk = ((b * d.T + t0) * d.G + hk) * d.K;
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * mt + 4 * g + e;
      if (i >= left) continue;
      const float pq = gsc[G_PQ * kC + i], rq = s.rq[i], pk = gsc[G_PK * kC + i], rk = s.rk[i];
      const float un = rq * rscale;
      const float wq = ((s.rows[0][0][i] + s.rows[1][0][i]) + (s.rows[2][0][i] + s.rows[3][0][i])) * un * un;
      const float wk = ((s.rows[0][1][i] + s.rows[1][1][i]) + (s.rows[2][1][i] + s.rows[3][1][i])) * rk * rk;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = 16 * (n0 + n) + r;
        if (col >= d.K) continue;
        float kv = static_cast<float>(kt[0][n][mt >> 1][(mt & 1) * 4 + e]), qv = static_cast<float>(qt[0][n][mt >> 1][(mt & 1) * 4 + e]);
        if (NP == 2) {
          kv += static_cast<float>(kt[NP - 1][n][mt >> 1][(mt & 1) * 4 + e]);
          qv += static_cast<float>(qt[NP - 1][n][mt >> 1][(mt & 1) * 4 + e]);
        }
        const int64_t o = qk + i * (d.G * d.K) + col;
        IO<A>::st(p.d_q, o, rq * (totQ[mt][n][e] - qv * wq) * pq);
        IO<A>::st(p.d_k, o, rk * (totK[mt][n][e] - kv * wk) * pk);
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
  hipLaunchKernelGGL((gdelta_bwd_state_kernel<A, KP>), dim3(bh * (d.VP / 16)), dim3(64), 0, st, a);
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
