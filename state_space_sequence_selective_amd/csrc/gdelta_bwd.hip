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
    const float e = ok ? p.w.sc[ci * (kSc * kC) + SC_E * kC + kC - 1] : 1.0f;
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
__device__ constexpr int kTTm[6] = {0, 0, 1, 1, 2, 3}, kTTk[6] = {0, 1, 0, 1, 1, 1};

template <Act A, int KP>
struct BwdLds {
  static constexpr int NP = A == Act::F32 ? 2 : 1;
  uint16_t k[NP * kC * kRow<KP>];
  uint16_t q[NP * kC * kRow<KP>];
  uint16_t kT[NP * KP * kCol];
  uint16_t qT[NP * KP * kCol];
  uint16_t PT[2 * kC * kCol];
};

template <Act A, int KP, int NW>
__global__ void __launch_bounds__(NW * 64) gdelta_bwd_state_kernel(const BwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, MT = KP / 16, KS = KP / 32;
  __shared__ __attribute__((aligned(16))) BwdLds<A, KP> s;
  static_assert(sizeof(s) <= mscan::kLdsBytes, "LDS");
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, r = lane & 15, g = lane >> 4;
  const int ncb = (d.VP / 16 + NW - 1) / NW;
  const int64_t bh = blockIdx.x / ncb, h = bh % d.H, b = bh / d.H, hk = h / (d.H / d.G);
  const int col = ((blockIdx.x % ncb) * NW + wv) * 16 + r;
  const bool ok = col < d.V, live = col < d.VP;
  const float so = p.so[bh], rso = 1.0f / so, rps = 1.0f / d.pscale;
  const uint32_t poff = (4 * g * d.VP + col) * 4;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 dS[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) dS[mt] = zero;
  for (int64_t c = d.nc - 1; c >= 0; --c) {
    const int64_t t0 = c * kC, left = d.T - t0, ci = bh * d.nc + c;
    const float* sc = p.w.sc + ci * (kSc * kC);
    const double* Gs = p.w.G + ci * kC;
    const double Gl = Gs[kC - 1];
    __syncthreads();
    const int64_t qk = ((b * d.T + t0) * d.G + hk) * d.K;
    stage_qk<A, KP, NW * 64>(p.k, p.q, qk, d.G * d.K, d.K, left, sc, s.k, s.q, s.kT, s.qT, tid);
    __syncthreads();
    // P^T: rows j, columns i; zeros in the tiles below its diagonal that a 32-wide step reads
    for (int i = wv; i < 12; i += NW) {
      const int mt = i < 4 ? 0 : i < 8 ? 1 : i < 10 ? 2 : 3, nt = i < 8 ? (i & 3) : 2 + (i & 1);
      f32x4 acc = zero;
      if (nt >= mt) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint16_t* pa = s.k + (16 * mt + r) * kRow<KP> + 32 * ks + 8 * g;
          const uint16_t* pb = s.q + (16 * nt + r) * kRow<KP> + 32 * ks + 8 * g;
          acc = mma(ld8(pa), ld8(pb), acc);
          if (NP == 2) {
            acc = mma(ld8(pa), ld8(pb + kC * kRow<KP>), acc);
            acc = mma(ld8(pa + kC * kRow<KP>), ld8(pb), acc);
          }
        }
      }
      const int ti = 16 * nt + r;
      const float rq = sc[SC_RQ * kC + ti] * d.pscale;
      const double Gi = Gs[ti];
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float v[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int tj = 16 * mt + 4 * g + e + o;
          v[o] = tj <= ti ? rq * sc[SC_RK * kC + tj] * acc[e + o] * exp2_fast(static_cast<float>(Gi - Gs[tj])) : 0.0f;
        }
        uint32_t hi, lo;
        split2(v[0], v[1], hi, lo);
        uint16_t* dst = s.PT + (16 * mt + 4 * g + e) * kCol + place(ti);
        dst[0] = static_cast<uint16_t>(hi);
        dst[kCol] = static_cast<uint16_t>(hi >> 16);
        dst[kC * kCol] = static_cast<uint16_t>(lo);
        dst[kC * kCol + kCol] = static_cast<uint16_t>(lo >> 16);
      }
    }
    __syncthreads();

    f32x4 dU[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag f = to_b(dS[2 * ks], dS[2 * ks + 1]);
      if (live) store_packed(p.DS + (ci * KP + 32 * ks) * d.VP, poff, f, d.VP);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
        dU[mt] = mma_split<NP>(s.k + (16 * mt + r) * kRow<KP> + 32 * ks + 8 * g, kC * kRow<KP>, f, dU[mt]);
    }
    f32x4 dO[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * mt + 4 * g + e;
        dO[mt][e] = ok && t < left ? IO<A>::ld(p.dy, ((b * d.T + t0 + t) * d.H + h) * d.V + col) * so : 0.0f;
        dU[mt][e] *= exp2_fast(static_cast<float>(Gl - Gs[t])) * sc[SC_RK * kC + t];
      }
    const Frag o0 = to_b(dO[0], dO[1]), o1 = to_b(dO[2], dO[3]);   // 16-bit input: the low parts are zero
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      f32x4 acc = zero;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (mt >= 2 && ks == 0) continue;
        const uint16_t* a = s.PT + (16 * mt + r) * kCol + 32 * ks + 8 * g;
        const Frag& o = ks ? o1 : o0;
        const h8 ah = ld8(a);
        acc = mma(ah, o.hi, acc);
        acc = mma(ld8(a + kC * kCol), o.hi, acc);
        if (NP == 2) acc = mma(ah, o.lo, acc);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) dU[mt][e] = fmaf(acc[e], rps, dU[mt][e]);
    }
    const Frag u0 = to_b(dU[0], dU[1]), u1 = to_b(dU[2], dU[3]);
    f32x4 Y[4] = {zero, zero, zero, zero};
    const uint16_t* T = p.w.TT + ci * (kTFrag * 512) + lane * 8;
#pragma unroll
    for (int f = 0; f < 6; ++f) {
      const Frag& x = kTTk[f] ? u1 : u0;
      const h8 th = ld8(T + f * 512), tl = ld8(T + (6 + f) * 512);
      f32x4 a = Y[kTTm[f]];
      a = mma(th, x.hi, a);
      a = mma(th, x.lo, a);
      Y[kTTm[f]] = mma(tl, x.hi, a);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[mt][e] *= 1.0f / kTScale;
    if (live) {
      store_packed(p.DU + ci * kC * d.VP, poff, to_b(Y[0], Y[1]), d.VP);
      store_packed(p.DU + (ci * kC + 32) * d.VP, poff, to_b(Y[2], Y[3]), d.VP);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * mt + 4 * g + e;
        const float be = sc[SC_BETA * kC + t], ev = sc[SC_E * kC + t];
        const float dv = be * Y[mt][e];
        if (ok && t < left) IO<A>::st(p.d_v, ((b * d.T + t0 + t) * d.H + h) * d.V + col, dv * rso);
        Y[mt][e] = -(ev * sc[SC_RK * kC + t]) * dv;
        dO[mt][e] *= ev * sc[SC_RQ * kC + t];
      }
    const Frag y0 = to_b(Y[0], Y[1]), y1 = to_b(Y[2], Y[3]), e0 = to_b(dO[0], dO[1]), e1 = to_b(dO[2], dO[3]);
    const float el = exp2_fast(static_cast<float>(Gl));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) dS[mt][e] *= el;
      const uint16_t* a = s.kT + (16 * mt + r) * kCol + 8 * g;
      const uint16_t* q = s.qT + (16 * mt + r) * kCol + 8 * g;
      dS[mt] = mma_split<NP>(a, KP * kCol, y0, dS[mt]);
      dS[mt] = mma_split<NP>(a + 32, KP * kCol, y1, dS[mt]);
      dS[mt] = mma_split<NP>(q, KP * kCol, e0, dS[mt]);
      dS[mt] = mma_split<NP>(q + 32, KP * kCol, e1, dS[mt]);
    }
  }
}

// ------------------------------------------------------------------ the chunks' own gradients
// One workgroup per (batch row, query / key head, chunk), over the value heads that share it.  First all products
// with d_v contracted, in slabs of 32 columns: rows of dO, U and Y through LDS, S and dS' from global memory straight
// into the fragments of the wave that owns their d_k rows.  Then the 64 x 64 gradients M1 and M2, and their products
// with q and k.
constexpr int kSlab = 32 + 8;

template <Act A, int KP>
struct ChunkLds {
  static constexpr int NP = A == Act::F32 ? 2 : 1;
  union {
    struct {
      uint16_t dO[NP * kC * kSlab], U[2 * kC * kSlab], Y[2 * kC * kSlab];
    };
    struct {
      uint16_t k[NP * kC * kRow<KP>], q[NP * kC * kRow<KP>];
    };
    struct {
      uint16_t kT[NP * KP * kCol], qT[NP * KP * kCol];
    };
  };
  uint16_t M1[2 * kC * kCol], M1T[2 * kC * kCol], M2[2 * kC * kCol], M2T[2 * kC * kCol];
  float rows[4][4][kC];   // per wave: row sums
  float colE[kC], db[kC], red[8];
  double G[kC];
};

__device__ __forceinline__ void unpack8(const uint32_t* p, h8& hi, h8& lo) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 4);
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

__device__ __forceinline__ f32x4 mma3(h8 ah, h8 al, h8 bh, h8 bl, f32x4 c) {
  c = mma(ah, bh, c);
  c = mma(ah, bl, c);
  return mma(al, bh, c);
}

template <Act A, int KP>
__global__ void __launch_bounds__(256) gdelta_bwd_chunk_kernel(const BwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, NT = KP / 64, KS = KP / 32;
  __shared__ __attribute__((aligned(16))) ChunkLds<A, KP> s;
  static_assert(sizeof(s) <= mscan::kLdsBytes, "LDS");
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, r = lane & 15, g = lane >> 4;
  const int64_t c = blockIdx.x % d.nc, bg = blockIdx.x / d.nc, hk = bg % d.G, b = bg / d.G;
  const int64_t t0 = c * kC, left = d.T - t0;
  const int share = static_cast<int>(d.H / d.G);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t qk = ((b * d.T + t0) * d.G + hk) * d.K;
  const int n0 = wv * (KP / 4);   // this wave's d_k columns: n0 + 16 n + r
  f32x4 totQ[4][NT], totK[4][NT];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int n = 0; n < NT; ++n) totQ[mt][n] = totK[mt][n] = zero;

  for (int hi_ = 0; hi_ < share; ++hi_) {
    const int64_t h = hk * share + hi_, bh = b * d.H + h, ci = bh * d.nc + c;
    const float* sc = p.w.sc + ci * (kSc * kC);
    const float so = p.so[bh], sv = p.w.sv[bh], rso = 1.0f / so, rsv = 1.0f / sv;
    f32x4 aP[4], aA[4], aQ[4][NT], aKq[4][NT], aKs[4][NT];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      aP[mt] = aA[mt] = zero;
#pragma unroll
      for (int n = 0; n < NT; ++n) aQ[mt][n] = aKq[mt][n] = aKs[mt][n] = zero;
    }
    float dot = 0.0f;   // <dS', S>
    for (int v0 = 0; v0 < d.VP; v0 += 32) {
      __syncthreads();
      {
        const int t = tid >> 2, cc = (tid & 3) * 8;
        float x[8];
        load8<A>(p.dy, ((b * d.T + t0 + t) * d.H + h) * d.V + v0 + cc, t < left && v0 + cc < d.V, x);
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a, bb;
          split2(x[2 * e] * so, x[2 * e + 1] * so, a, bb);
          hi[e] = a;
          lo[e] = bb;
        }
        *reinterpret_cast<u32x4*>(s.dO + t * kSlab + cc) = hi;
        if (NP == 2) *reinterpret_cast<u32x4*>(s.dO + kC * kSlab + t * kSlab + cc) = lo;
        h8 ph, pl;
        unpack8(p.w.U + (ci * kC + t) * d.VP + v0 + cc, ph, pl);
        *reinterpret_cast<h8*>(s.U + t * kSlab + cc) = ph;
        *reinterpret_cast<h8*>(s.U + kC * kSlab + t * kSlab + cc) = pl;
        unpack8(p.DU + (ci * kC + t) * d.VP + v0 + cc, ph, pl);
        *reinterpret_cast<h8*>(s.Y + t * kSlab + cc) = ph;
        *reinterpret_cast<h8*>(s.Y + kC * kSlab + t * kSlab + cc) = pl;
      }
      __syncthreads();
      h8 sh[NT], sl[NT], gh[NT], gl[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t at = (ci * KP + n0 + 16 * n + r) * d.VP + v0 + 8 * g;
        unpack8(p.w.S + at, sh[n], sl[n]);
        unpack8(p.DS + at, gh[n], gl[n]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dot = fmaf(static_cast<float>(sh[n][e]) + static_cast<float>(sl[n][e]),
                     static_cast<float>(gh[n][e]) + static_cast<float>(gl[n][e]), dot);
      }
      const int bt = (16 * wv + r) * kSlab + 8 * g;
      const h8 ubh = ld8(s.U + bt), ubl = ld8(s.U + kC * kSlab + bt);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const int at = (16 * mt + r) * kSlab + 8 * g;
        const h8 oh = ld8(s.dO + at), uh = ld8(s.U + at), ul = ld8(s.U + kC * kSlab + at);
        const h8 yh = ld8(s.Y + at), yl = ld8(s.Y + kC * kSlab + at);
        h8 ol = {};
        if (NP == 2) ol = ld8(s.dO + kC * kSlab + at);
        if (mt >= wv) {
          aP[mt] = mma(oh, ubh, aP[mt]);
          aP[mt] = mma(oh, ubl, aP[mt]);
          if (NP == 2) aP[mt] = mma(ol, ubh, aP[mt]);
          aA[mt] = mma3(yh, yl, ubh, ubl, aA[mt]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          aQ[mt][n] = mma(oh, sh[n], aQ[mt][n]);
          aQ[mt][n] = mma(oh, sl[n], aQ[mt][n]);
          if (NP == 2) aQ[mt][n] = mma(ol, sh[n], aQ[mt][n]);
          aKq[mt][n] = mma3(yh, yl, sh[n], sl[n], aKq[mt][n]);
          aKs[mt][n] = mma3(uh, ul, gh[n], gl[n], aKs[mt][n]);
        }
      }
    }
    __syncthreads();
    if (tid < kC) s.G[tid] = p.w.G[ci * kC + tid];
    stage_qk<A, KP, 256>(p.k, p.q, qk, d.G * d.K, d.K, left, sc, s.k, s.q, nullptr, nullptr, tid);
    __syncthreads();
    // this wave's columns j of the 64 x 64 gradients
    const int j = 16 * wv + r;
    const float rkj = sc[SC_RK * kC + j];
    f32x4 m1[4], m2[4];
    float ce = 0.0f, big = 0.0f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      m1[mt] = m2[mt] = zero;
      f32x4 kq = zero, kk = zero;
      if (mt >= wv) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int at = (16 * mt + r) * kRow<KP> + 32 * ks + 8 * g, bt = j * kRow<KP> + 32 * ks + 8 * g;
          const h8 bk = ld8(s.k + bt), aq = ld8(s.q + at), ak = ld8(s.k + at);
          kq = mma(aq, bk, kq);
          kk = mma(ak, bk, kk);
          if (NP == 2) {
            const h8 bl = ld8(s.k + kC * kRow<KP> + bt);
            kq = mma(aq, bl, kq);
            kk = mma(ak, bl, kk);
            kq = mma(ld8(s.q + kC * kRow<KP> + at), bk, kq);
            kk = mma(ld8(s.k + kC * kRow<KP> + at), bk, kk);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * mt + 4 * g + e;
        const float rq = sc[SC_RQ * kC + i], rk = sc[SC_RK * kC + i], be = sc[SC_BETA * kC + i];
        const float D = j <= i ? exp2_fast(static_cast<float>(s.G[i] - s.G[j])) : 0.0f;
        const float dP = aP[mt][e] * rso * rsv, yu = aA[mt][e] * rso * rsv;
        float E = 0.0f;
        m1[mt][e] = j <= i ? dP * D : 0.0f;
        if (j < i) {
          m2[mt][e] = -yu * be * D;
          E = m1[mt][e] * (rq * rkj * kq[e]) + m2[mt][e] * (rk * rkj * kk[e]);
        }
        if (i == j) s.db[i] = yu * (1.0f - be);
        ce += E;
        const float re = sum16(E);
        if (r == 0) s.rows[wv][0][i] = re;
        const float a = fmaxf(fabsf(m1[mt][e]), fabsf(m2[mt][e])) * fmaxf(rkj, fmaxf(fabsf(rq), rk));
        big = max_finite(big, a);
      }
    }
    ce += __shfl_xor(ce, 16, 64);
    ce += __shfl_xor(ce, 32, 64);
    if (g == 0) s.colE[j] = ce;
    big = wave_max(big);
    dot = wave_sum(dot);
    if (lane == 0) {
      s.red[wv] = big;
      s.red[4 + wv] = dot;
    }
    __syncthreads();   // k, q read; s.red written
    stage_qk<A, KP, 256>(p.k, p.q, qk, d.G * d.K, d.K, left, sc, nullptr, nullptr, s.kT, s.qT, tid);
    const float sm = pow2_below(fmaxf(fmaxf(s.red[0], s.red[1]), fmaxf(s.red[2], s.red[3])), 13), rsm = 1.0f / sm;
    dot = s.red[4] + s.red[5] + s.red[6] + s.red[7];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const int i0 = 16 * mt + 4 * g;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const f32x4 m = which ? m2[mt] : m1[mt];
        uint16_t* a = (which ? s.M2 : s.M1) + i0 * kCol + place(j);
        uint16_t* at = (which ? s.M2T : s.M1T) + j * kCol + place(i0);
        uint32_t h[2], l[2], th[2], tl[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float x = m[2 * o] * sm, y = m[2 * o + 1] * sm;
          const float* ri = sc + (which ? SC_RK : SC_RQ) * kC + i0 + 2 * o;
          split2(x * rkj, y * rkj, h[o], l[o]);
          split2(x * ri[0], y * ri[1], th[o], tl[o]);
          a[(2 * o) * kCol] = static_cast<uint16_t>(h[o]);
          a[(2 * o + 1) * kCol] = static_cast<uint16_t>(h[o] >> 16);
          a[kC * kCol + (2 * o) * kCol] = static_cast<uint16_t>(l[o]);
          a[kC * kCol + (2 * o + 1) * kCol] = static_cast<uint16_t>(l[o] >> 16);
        }
        *reinterpret_cast<u32x2*>(at) = u32x2{th[0], th[1]};
        *reinterpret_cast<u32x2*>(at + kC * kCol) = u32x2{tl[0], tl[1]};
      }
    }
    __syncthreads();
    // the parts through the state, in true units, and their products with q and k for the decay's gradient
    const double Gl = s.G[kC - 1];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const int i0 = 16 * mt + 4 * g;
      float wq[4] = {}, wkq[4] = {}, wks[4] = {};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int at = (n0 + 16 * n + r) * kCol + place(i0);
        f32x4 kv, qv;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kv[e] = static_cast<float>(reinterpret_cast<const h4*>(s.kT + at)[0][e]);
          qv[e] = static_cast<float>(reinterpret_cast<const h4*>(s.qT + at)[0][e]);
          if (NP == 2) {
            kv[e] += static_cast<float>(reinterpret_cast<const h4*>(s.kT + KP * kCol + at)[0][e]);
            qv[e] += static_cast<float>(reinterpret_cast<const h4*>(s.qT + KP * kCol + at)[0][e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e;
          const float ev = sc[SC_E * kC + i], be = sc[SC_BETA * kC + i];
          aQ[mt][n][e] *= ev * rso * rsv;
          aKq[mt][n][e] *= -(ev * be) * rso * rsv;
          aKs[mt][n][e] *= exp2_fast(static_cast<float>(Gl - s.G[i])) * rso * rsv;
          wq[e] = fmaf(aQ[mt][n][e], qv[e], wq[e]);
          wkq[e] = fmaf(aKq[mt][n][e], kv[e], wkq[e]);
          wks[e] = fmaf(aKs[mt][n][e], kv[e], wks[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = sum16(wq[e]), y = sum16(wkq[e]), z = sum16(wks[e]);
        if (r == 0) {
          const int i = i0 + e;
          s.rows[wv][1][i] = x * sc[SC_RQ * kC + i];
          s.rows[wv][2][i] = y * sc[SC_RK * kC + i];
          s.rows[wv][3][i] = z * sc[SC_RK * kC + i];
        }
      }
    }
    // the parts inside the chunk
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 q = aQ[mt][n], k = aKq[mt][n] + aKs[mt][n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[e] *= sm;
          k[e] *= sm;
        }
        const int nr = (n0 + 16 * n + r) * kCol + 8 * g, ar = (16 * mt + r) * kCol + 8 * g;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const h8 kh = ld8(s.kT + nr + 32 * ks), qh = ld8(s.qT + nr + 32 * ks);
          h8 kl = {}, ql = {};
          if (NP == 2) {
            kl = ld8(s.kT + KP * kCol + nr + 32 * ks);
            ql = ld8(s.qT + KP * kCol + nr + 32 * ks);
          }
          const int a = ar + 32 * ks;
          if (ks == 0 || mt >= 2) {   // rows i, columns j <= i
            const h8 x = ld8(s.M1 + a), y = ld8(s.M2 + a);
            q = mma(x, kh, q);
            q = mma(ld8(s.M1 + kC * kCol + a), kh, q);
            k = mma(y, kh, k);
            k = mma(ld8(s.M2 + kC * kCol + a), kh, k);
            if (NP == 2) {
              q = mma(x, kl, q);
              k = mma(y, kl, k);
            }
          }
          if (ks == 1 || mt < 2) {    // rows j, columns i >= j
            const h8 x = ld8(s.M1T + a), y = ld8(s.M2T + a);
            k = mma(x, qh, k);
            k = mma(ld8(s.M1T + kC * kCol + a), qh, k);
            k = mma(y, kh, k);
            k = mma(ld8(s.M2T + kC * kCol + a), kh, k);
            if (NP == 2) {
              k = mma(x, ql, k);
              k = mma(y, kl, k);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          totQ[mt][n][e] += q[e] * rsm;
          totK[mt][n][e] += k[e] * rsm;
        }
      }
    }
    __syncthreads();
    if (tid < kC) {   // dg and what comes of it
      const int t = tid;
      float x = 0.0f, z = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x += s.rows[w][1][t] + s.rows[w][2][t];
        z += s.rows[w][3][t];
      }
      float E = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (w <= (t >> 4)) E += s.rows[w][0][t];
      float dG = (E - s.colE[t]) + (x - z);
      // suffix sum over the chunk's tokens
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float up = __shfl_down(dG, o, 64);
        if (t + o < 64) dG += up;
      }
      const float through = wave_sum(z) + exp2_fast(static_cast<float>(Gl)) * (dot * rso * rsv);
      float dg = dG + through;
      if (!p.has_h0 && c == 0 && t == 0) dg = 0.0f;   // the first token's decay meets no state: exactly zero
      float pa = 0.0f, pb = 0.0f;
      if (t < left) {
        const int64_t i = (b * d.T + t0 + t) * d.H + h;
        const float rate = exp2_fast(p.a_log[h] * kLog2e), z2 = p.a_raw[i] + p.dt_bias[h];
        const float da = -rate * mscan::sigmoid(z2) * dg;
        p.d_a_raw[i] = da;
        p.d_b_raw[i] = s.db[t];
        pa = -rate * mscan::softplus(z2) * dg;
        pb = da;
      }
      pa = wave_sum(pa);
      pb = wave_sum(pb);
      if (t == 0) {
        p.part[ci * 2] = pa;
        p.part[ci * 2 + 1] = pb;
      }
    }
  }
  // unit length's adjoint: r (d - n (n . d)); rows of q and k in kT, qT still
  const int64_t ci = (b * d.H + hk * share) * d.nc + c;
  const float* sc = p.w.sc + ci * (kSc * kC);
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const int i0 = 16 * mt + 4 * g;
    float wq[4] = {}, wk[4] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int at = (n0 + 16 * n + r) * kCol + place(i0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float kv = static_cast<float>(reinterpret_cast<const h4*>(s.kT + at)[0][e]);
        float qv = static_cast<float>(reinterpret_cast<const h4*>(s.qT + at)[0][e]);
        if (NP == 2) {
          kv += static_cast<float>(reinterpret_cast<const h4*>(s.kT + KP * kCol + at)[0][e]);
          qv += static_cast<float>(reinterpret_cast<const h4*>(s.qT + KP * kCol + at)[0][e]);
        }
        wq[e] = fmaf(totQ[mt][n][e], qv, wq[e]);
        wk[e] = fmaf(totK[mt][n][e], kv, wk[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = sum16(wq[e]), y = sum16(wk[e]);
      if (r == 0) {
        s.rows[wv][0][i0 + e] = x;
        s.rows[wv][1][i0 + e] = y;
      }
    }
  }
  __syncthreads();
  const float rscale = 1.0f / d.scale;
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const int i0 = 16 * mt + 4 * g;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e;
      if (i >= left) continue;
      const float pq = sc[SC_PQ * kC + i], rq = sc[SC_RQ * kC + i], pk = sc[SC_PK * kC + i], rk = sc[SC_RK * kC + i];
      const float un = rq * rscale;
      const float wq = (s.rows[0][0][i] + s.rows[1][0][i] + s.rows[2][0][i] + s.rows[3][0][i]) * un * un;
      const float wk = (s.rows[0][1][i] + s.rows[1][1][i] + s.rows[2][1][i] + s.rows[3][1][i]) * rk * rk;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = n0 + 16 * n + r, at = col * kCol + place(i0);
        if (col >= d.K) continue;
        float kv = static_cast<float>(reinterpret_cast<const h4*>(s.kT + at)[0][e]);
        float qv = static_cast<float>(reinterpret_cast<const h4*>(s.qT + at)[0][e]);
        if (NP == 2) {
          kv += static_cast<float>(reinterpret_cast<const h4*>(s.kT + KP * kCol + at)[0][e]);
          qv += static_cast<float>(reinterpret_cast<const h4*>(s.qT + KP * kCol + at)[0][e]);
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
  constexpr int NW = 4;
  const Dims& d = a.d;
  const unsigned bh = static_cast<unsigned>(d.B * d.H), nc = static_cast<unsigned>(d.nc);
  hipLaunchKernelGGL((gdelta_dymax_kernel<A>), dim3(bh * nc), dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gdelta_dscale_kernel, dim3(bh), dim3(64), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int ncb = (d.VP / 16 + NW - 1) / NW;
  hipLaunchKernelGGL((gdelta_bwd_state_kernel<A, KP, NW>), dim3(bh * ncb), dim3(NW * 64), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((gdelta_bwd_chunk_kernel<A, KP>), dim3(static_cast<unsigned>(d.B * d.G) * nc), dim3(256), 0, st, a);
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
