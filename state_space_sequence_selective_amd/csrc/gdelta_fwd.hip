// Gated delta rule, forward: the chunks' operands, the per-chunk triangular
// inverse, the pass over the chunks, and the token-by-token step (gfx950).
// The algebra and the number format are in gdelta.h.
#include <type_traits>

#include "gdelta_launch.h"

namespace gdelta {

// ------------------------------------------------------------------ q and k as operands
// One workgroup per (batch row, query / key head, chunk): each row's power of two and unit scale, and its f16 parts as
// fragments, through LDS.
template <Act A, int KP>
__global__ void __launch_bounds__(256) gdelta_rows_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, EPT = KP / 4, ROW = KP + 8, KS = KP / 32;
  __shared__ __attribute__((aligned(16))) uint16_t s[2][NP][kC * ROW];
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
  const int64_t c = blockIdx.x % d.nc, bg = blockIdx.x / d.nc, hk = bg % d.G, b = bg / d.G;
  const int64_t t0 = c * kC, left = d.T - t0, ci = bg * d.nc + c;
  float* sc = p.w.gsc + ci * (kGroupSc * kC);
  const int row = tid >> 2, part = tid & 3;   // four threads a row
  const int64_t base = ((b * d.T + t0 + row) * d.G + hk) * d.K;
  float x[2][EPT];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int e = 0; e < EPT; e += 8) {
      const int col = part * EPT + e;
      load8<A>(which ? p.q : p.k, base + col, row < left && col < d.K, x[which] + e);
    }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float m = 0.0f, ss = 0.0f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) m = max_finite(m, x[which][e]);
    m = fmaxf(m, __shfl_xor(m, 1, 64));
    m = fmaxf(m, __shfl_xor(m, 2, 64));
    const float pw = pow2_below(m, 2);
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      x[which][e] *= pw;
      ss = fmaf(x[which][e], x[which][e], ss);
    }
    ss += __shfl_xor(ss, 1, 64);
    ss += __shfl_xor(ss, 2, 64);
    const float rs = unit_scale(ss, pw, d.eps);
    if (part == 0) {
      sc[(which ? G_PQ : G_PK) * kC + row] = pw;
      sc[(which ? G_RQ : G_RK) * kC + row] = which ? rs * d.scale : rs;
    }
#pragma unroll
    for (int e = 0; e < EPT; e += 8) {
      u32x4 hi, lo;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a, bb;
        split2(x[which][e + 2 * k], x[which][e + 2 * k + 1], a, bb);
        hi[k] = a;
        lo[k] = bb;
      }
      *reinterpret_cast<u32x4*>(s[which][0] + row * ROW + part * EPT + e) = hi;
      if (NP == 2) *reinterpret_cast<u32x4*>(s[which][NP - 1] + row * ROW + part * EPT + e) = lo;
    }
  }
  __syncthreads();
  constexpr int NF = KP / 8;   // fragments of a plane, of either family
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int pl = 0; pl < NP; ++pl) {
      const uint16_t* src = s[which][pl];
      uint16_t* F = (which ? p.w.QF : p.w.KF) + (ci * NP + pl) * (NF * kFrag);
#pragma unroll
      for (int i = 0; i < NF / 4; ++i) {
        const int f = i * 4 + wv, mt = f / KS, ks = f % KS;
        const uint16_t* a = src + (16 * mt + r) * ROW + 32 * ks + 4 * g;
        const u32x2 lo = *reinterpret_cast<const u32x2*>(a), hi = *reinterpret_cast<const u32x2*>(a + 16);
        at<u32x4>(F + f * kFrag, lane * 16) = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
      if (which && !p.w.QT) continue;
      uint16_t* Tr = (which ? p.w.QT : p.w.KT) + (ci * NP + pl) * (NF * kFrag);
#pragma unroll
      for (int i = 0; i < NF / 4; ++i) {
        const int f = i * 4 + wv, n = f / 2, ks = f % 2;
        const uint16_t* a = src + (32 * ks + 4 * g) * ROW + 16 * n + r;
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x0 = (e & 1) * 2 + (e >> 1) * 16;
          v[e] = a[x0 * ROW] | (static_cast<uint32_t>(a[(x0 + 1) * ROW]) << 16);
        }
        at<u32x4>(Tr + f * kFrag, lane * 16) = v;
      }
    }
}

// y is rounded to its type.  For bf16 (2^-9) one f16 part (2^-12) of P, u and the state is enough in it, and adds
// about 1% to its error; f16 and f32 take both.  What feeds the state or a gradient has both always.
template <Act A>
constexpr int kPPlanes = A == Act::BF16 ? 1 : 2;

// ------------------------------------------------------------------ chunk preparation
// One workgroup per (batch row, head, chunk): the tokens' gates; P = q.k^T D and its transpose, whose fragments are the
// result tiles of k.q^T and q.k^T as they stand; A = beta k.k^T D in LDS and its unit lower triangular inverse: four
// 16 x 16 diagonal blocks by substitution, then two levels of T21 = -T22 (A21 T11) on f32 matrix instructions
// (v_mfma_f32_16x16x4_f32; full f32, as an inverse amplifies roundings of A).
constexpr int kAS = kC + 4;

__device__ __forceinline__ f32x4 mma32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// acc += A[16 x 16] * B[16 x 16], both in LDS with row length kAS; the contraction runs over 4 g + s, so that a D tile
// can be the next product's B operand as it is
__device__ __forceinline__ f32x4 tile_mm(const float* a, const float* b, int r, int g, f32x4 acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mma32(a[r * kAS + 4 * g + s], b[(4 * g + s) * kAS + r], acc);
  return acc;
}

__device__ __forceinline__ f32x4 tile_mm(const float* a, f32x4 b, int r, int g, f32x4 acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mma32(a[r * kAS + 4 * g + s], b[s], acc);
  return acc;
}

template <Act A, int KP>
__global__ void __launch_bounds__(256) gdelta_prep_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, KS = KP / 32, NF = KP / 8;
  __shared__ __attribute__((aligned(16))) float sA[kC * kAS], sT[kC * kAS];
  __shared__ double sG[kC];
  __shared__ float sBeta[kC], sRk[kC], sRq[kC], sMax[4];
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
  const int64_t c = blockIdx.x % d.nc, bh = blockIdx.x / d.nc, h = bh % d.H, b = bh / d.H, hk = h / (d.H / d.G);
  const int64_t t0 = c * kC, left = d.T - t0, ci = bh * d.nc + c, gi = (b * d.G + hk) * d.nc + c;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  if (tid < kC) {
    const bool ok = tid < left;
    const int64_t i = (b * d.T + t0 + tid) * d.H + h;
    const float rate = exp2_fast(p.a_log[h] * kLog2e);
    double G = ok ? log2_decay(rate, p.a_raw[i], p.dt_bias[h]) : 0.0f;
    const float beta = ok ? mscan::sigmoid(p.b_raw[i]) : 0.0f;
    const float rk = p.w.gsc[gi * (kGroupSc * kC) + G_RK * kC + tid], rq = p.w.gsc[gi * (kGroupSc * kC) + G_RQ * kC + tid];
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const double o = __shfl_up(G, s, 64);
      if (lane >= s) G += o;
    }
    const double Gl = __shfl(G, 63, 64);
    sG[tid] = G;
    sBeta[tid] = beta;
    sRk[tid] = rk;
    sRq[tid] = rq * d.pscale;
    p.w.G[ci * kC + tid] = G;
    float* sc = p.w.hsc + ci * (kHeadSc * kC);
    const float e = exp2_fast(static_cast<float>(G));
    sc[H_BETA * kC + tid] = beta;
    sc[H_E * kC + tid] = e;
    sc[H_BK * kC + tid] = beta * e * rk;
    sc[H_DK * kC + tid] = exp2_fast(static_cast<float>(Gl - G)) * rk;
    sc[H_EQ * kC + tid] = e * rq;
  }
  // the largest |v|, and the initial state's bound sqrt(d_k) max |h0|
  float m = 0.0f;
  {
    const int nv = d.V / 8;
    const int rows = left < kC ? static_cast<int>(left) : kC;
    for (int i = tid; i < rows * nv; i += 256) {
      float x[8];
      load8<A>(p.v, ((b * d.T + t0 + i / nv) * d.H + h) * d.V + (i % nv) * 8, true, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_finite(m, x[e]);
    }
    if (c == 0 && p.h0) {
      float m0 = 0.0f;
      for (int i = tid; i < d.V * d.K; i += 256) m0 = max_finite(m0, p.h0[bh * d.V * d.K + i]);
      m = fmaxf(m, m0 * sqrtf(static_cast<float>(d.K)));
    }
    m = wave_max(m);
    if (lane == 0) sMax[wv] = m;
  }
  __syncthreads();
  if (tid == 0) p.w.vmax[ci] = fmaxf(fmaxf(sMax[0], sMax[1]), fmaxf(sMax[2], sMax[3]));
  const uint16_t* KF = p.w.KF + gi * (NP * NF * kFrag);
  const uint16_t* QF = p.w.QF + gi * (NP * NF * kFrag);
  {
    // wave w: tiles (rows j of tile n, columns i of tile w), n <= w
    const int i = 16 * wv + r;
    const float rki = sRk[i], rqi = sRq[i], be = sBeta[i];
    const double Gi = sG[i];
    f32x4 P[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      P[n] = zero;
      if (n > wv) continue;
      const f32x4 kk = frag_mm<NP, KS, NF>(KF + n * KS * kFrag, KF + wv * KS * kFrag, lane, zero);
      const f32x4 kq = frag_mm<NP, KS, NF>(KF + n * KS * kFrag, QF + wv * KS * kFrag, lane, zero);
      f32x4 a;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * n + 4 * g + e;
        const float w = j <= i ? sRk[j] * exp2_fast(static_cast<float>(Gi - sG[j])) : 0.0f;
        P[n][e] = rqi * w * kq[e];
        a[e] = j < i ? be * rki * w * kk[e] : 0.0f;
      }
      *reinterpret_cast<f32x4*>(sA + i * kAS + 16 * n + 4 * g) = a;
    }
    constexpr int PP = kPPlanes<A>;
    uint16_t* dst = p.w.P + ci * (PP * 6 * kFrag);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && wv < 2) continue;
      const int f = wv < 2 ? wv : 2 * wv - 2 + ks;
      const Frag x = to_b(P[2 * ks], P[2 * ks + 1]);
      at<h8>(dst + f * kFrag, lane * 16) = x.hi;
      if (PP == 2) at<h8>(dst + (6 + f) * kFrag, lane * 16) = x.lo;
    }
  }
  if (p.w.PT) {   // wave w: tiles (rows i of tile n, columns j of tile w), n >= w
    const int j = 16 * wv + r;
    const float rkj = sRk[j];
    const double Gj = sG[j];
    f32x4 P[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      P[n] = zero;
      if (n < wv) continue;
      const f32x4 qk = frag_mm<NP, KS, NF>(QF + n * KS * kFrag, KF + wv * KS * kFrag, lane, zero);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * n + 4 * g + e;
        P[n][e] = j <= i ? sRq[i] * rkj * exp2_fast(static_cast<float>(sG[i] - Gj)) * qk[e] : 0.0f;
      }
    }
    uint16_t* dst = p.w.PT + ci * (2 * 6 * kFrag);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 0 && wv >= 2) continue;
      const int f = wv < 2 ? 2 * wv + ks : 2 + wv;
      const Frag x = to_b(P[2 * ks], P[2 * ks + 1]);
      at<h8>(dst + f * kFrag, lane * 16) = x.hi;
      at<h8>(dst + (6 + f) * kFrag, lane * 16) = x.lo;
    }
  }
  __syncthreads();
  if (wv == 0) {   // the four diagonal blocks: a lane solves one column
    float t[16];
    const float* a = sA + (16 * g) * kAS + 16 * g;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == r ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-a[i * kAS + j], t[j], s);
      t[i] = s;
      sT[(16 * g + i) * kAS + 16 * g + r] = s;
    }
  }
  __syncthreads();
  if (wv < 2) {    // blocks (1, 0) and (3, 2)
    const int o = 32 * wv;
    const f32x4 x = tile_mm(sA + (o + 16) * kAS + o, sT + o * kAS + o, r, g, zero);
    const f32x4 y = tile_mm(sT + (o + 16) * kAS + o + 16, x, r, g, zero);
#pragma unroll
    for (int e = 0; e < 4; ++e) sT[(o + 16 + 4 * g + e) * kAS + o + r] = -y[e];
  }
  __syncthreads();
  if (wv < 2) {    // the lower left 32 x 32 block, one 16-column strip a wave
    f32x4 x[2];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      x[mi] = zero;
      for (int kk = wv; kk < 2; ++kk)
        x[mi] = tile_mm(sA + (32 + 16 * mi) * kAS + 16 * kk, sT + 16 * kk * kAS + 16 * wv, r, g, x[mi]);
    }
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      f32x4 y = zero;
#pragma unroll
      for (int kk = 0; kk <= mi; ++kk) y = tile_mm(sT + (32 + 16 * mi) * kAS + 32 + 16 * kk, x[kk], r, g, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) sT[(32 + 16 * mi + 4 * g + e) * kAS + 16 * wv + r] = -y[e];
    }
  }
  __syncthreads();
  uint16_t* T = p.w.T + ci * (12 * kFrag);
  uint16_t* TT = p.w.TT ? p.w.TT + ci * (12 * kFrag) : nullptr;
  for (int it = tid; it < 2 * 6 * 64; it += 256) {
    const bool tr = it >= 6 * 64;
    if (tr && !TT) break;
    const int f = (it >> 6) % 6, i = 16 * (tr ? kUm[f] : kLm[f]) + r, k0 = 32 * (tr ? kUk[f] : kLk[f]);
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int s = 2 * e + o, x = k0 + (s < 4 ? 4 * g + s : 16 + 4 * g + s - 4);
        v[o] = tr ? (x >= i ? sT[x * kAS + i] : 0.0f) : (x <= i ? sT[i * kAS + x] : 0.0f);
      }
      uint32_t a, bb;
      split2(v[0] * kTScale, v[1] * kTScale, a, bb);
      hi[e] = a;
      lo[e] = bb;
    }
    uint16_t* dst = (tr ? TT : T) + f * kFrag + lane * 8;
    *reinterpret_cast<u32x4*>(dst) = hi;
    *reinterpret_cast<u32x4*>(dst + 6 * kFrag) = lo;
  }
}

// ------------------------------------------------------------------ pass over the chunks
// A wave holds 16 columns of one head's S^T (rows: d_k) in registers, as the accumulators of the state update; they
// are at once the B operand of the products with k and q, and u is one for the update, so a wave needs nothing of any
// other: no LDS but for its tokens' scalars, no barrier.  The next chunk's fragments are loaded as soon as this one's
// are used.
template <Act A, int KP, bool SAVE>
__global__ void __launch_bounds__(64) gdelta_fwd_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, MT = KP / 16, KS = KP / 32, NF = KP / 8, PP = kPPlanes<A>;
  constexpr bool AHEAD = NP == 1;   // two planes do not fit the registers: loaded where they are used
  using Raw = std::conditional_t<A == Act::F32, uint32_t, uint16_t>;
  constexpr int ES = sizeof(Raw);
  __shared__ __attribute__((aligned(16))) float s[4][kC];   // beta; beta e rk; exp(G_63 - G) rk; e rq
  const Dims& d = p.d;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  int64_t bh;
  int cb;
  xcd_head(blockIdx.x, d.VP / 16, d.B * d.H, bh, cb);
  const int64_t h = bh % d.H, b = bh / d.H, hk = h / (d.H / d.G), bg = b * d.G + hk;
  const int col = cb * 16 + r;
  const bool ok = col < d.V;
  const uint32_t vrow = static_cast<uint32_t>(d.H) * d.V * ES;   // bytes of a token's v
  const uint32_t voff = vrow * 4 * g + (ok ? col : d.V - 1) * ES, yoff = vrow * 4 * g + col * ES;
  const uint32_t poff = (4 * g * d.VP + col) * 4;                // this lane's place in the packed S and U
  // the head's power of two: |s|, |v - S k| <= 2 sqrt(T + 1) max(|v|, |h0|) scaled below 2^15
  float m = 0.0f;
  for (int64_t i = lane; i < d.nc; i += 64) m = fmaxf(m, p.w.vmax[bh * d.nc + i]);
  const float sv = pow2_below(wave_max(m), 15 - static_cast<int>(ceilf(1.0f + 0.5f * log2f(static_cast<float>(d.T) + 1.0f))));
  const float rsv = 1.0f / sv, rps = 1.0f / d.pscale, svc = ok ? sv : 0.0f;
  if (SAVE && lane == 0 && cb == 0) p.w.sv[bh] = sv;

  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 S[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    S[mt] = zero;
    const int row = 16 * mt + 4 * g;
    if (p.h0 && ok && row < d.K) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p.h0 + (bh * d.V + col) * d.K + row);
#pragma unroll
      for (int e = 0; e < 4; ++e) S[mt][e] = x[e] * sv;
    }
  }
  h8 kf[NF], qf[NF], kt[NF], pf[6], th[6], tl[6];
  float sc[4], el;
  uint32_t v[4][4];
  auto frags = [&](h8* x, const uint16_t* base, int n) {
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = at<h8>(base + i * kFrag, lane * 16);
  };
  auto KFp = [&](int64_t c) { return p.w.KF + (bg * d.nc + c) * (NP * NF * kFrag); };
  auto QFp = [&](int64_t c) { return p.w.QF + (bg * d.nc + c) * (NP * NF * kFrag); };
  auto KTp = [&](int64_t c) { return p.w.KT + (bg * d.nc + c) * (NP * NF * kFrag); };
  auto Pp = [&](int64_t c) { return p.w.P + (bh * d.nc + c) * (PP * 6 * kFrag); };
  auto Tp = [&](int64_t c) { return p.w.T + (bh * d.nc + c) * (12 * kFrag); };
  auto load_t = [&](int64_t c) {
    frags(th, Tp(c), 6);
    frags(tl, Tp(c) + 6 * kFrag, 6);
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
    const int64_t left = d.T - c * kC;
    const char* base = static_cast<const char*>(p.v) + ((b * d.T + c * kC) * d.H + h) * (d.V * ES);
    const int64_t row = fresh(vrow);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[mt][e] = 0u;
        if (left >= kC || 16 * mt + 4 * g + e < left) v[mt][e] = at<Raw>(base + (16 * mt + e) * row, voff);
      }
  };
  if (AHEAD) {
    frags(kf, KFp(0), NF);
    frags(qf, QFp(0), NF);
    load_t(0);
    frags(kt, KTp(0), NF);
    frags(pf, Pp(0), 6);
  }
  load_sc(0);
  load_v(0);
  for (int64_t c = 0; c < d.nc; ++c) {
    const int64_t left = d.T - c * kC, ci = bh * d.nc + c;
    const bool more = AHEAD && c + 1 < d.nc;
    mscan::wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][lane] = sc[i];
    mscan::wave_lds_sync();
    const float elc = el;
    if (c + 1 < d.nc) load_sc(c + 1);
    if (!AHEAD) {
      frags(kf, KFp(c), NF);
      frags(qf, QFp(c), NF);
    }
    f32x4 ak[4], aq[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) ak[mt] = aq[mt] = zero;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag f = to_b(S[2 * ks], S[2 * ks + 1]);
      if (SAVE) store_packed(p.w.S + (ci * KP + 32 * ks) * d.VP, poff, f, d.VP);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) ak[mt] = mma(kf[mt * KS + ks], f.hi, ak[mt]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) ak[mt] = mma(kf[mt * KS + ks], f.lo, ak[mt]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) aq[mt] = mma(qf[mt * KS + ks], f.hi, aq[mt]);
      if (PP == 2) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) aq[mt] = mma(qf[mt * KS + ks], f.lo, aq[mt]);
      }
      if (NP == 2) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          ak[mt] = mma(at<h8>(KFp(c) + (NF + mt * KS + ks) * kFrag, lane * 16), f.hi, ak[mt]);
          aq[mt] = mma(at<h8>(QFp(c) + (NF + mt * KS + ks) * kFrag, lane * 16), f.hi, aq[mt]);
        }
      }
    }
    if (more) {
      frags(kf, KFp(c + 1), NF);
      frags(qf, QFp(c + 1), NF);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 be = *reinterpret_cast<const f32x4*>(s[0] + 16 * mt + 4 * g), bk = *reinterpret_cast<const f32x4*>(s[1] + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) ak[mt][e] = fmaf(be[e], IO<A>::cvt(v[mt][e]) * svc, -bk[e] * ak[mt][e]);
    }
    if (c + 1 < d.nc) load_v(c + 1);
    if (!AHEAD) {
      load_t(c);
      frags(kt, KTp(c), NF);
      frags(pf, Pp(c), 6);
    }
    const Frag x0 = to_b(ak[0], ak[1]), x1 = to_b(ak[2], ak[3]);
    f32x4 U[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int f = 0; f < 6; ++f) U[kLm[f]] = mma(th[f], (kLk[f] ? x1 : x0).hi, U[kLm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) U[kLm[f]] = mma(th[f], (kLk[f] ? x1 : x0).lo, U[kLm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) U[kLm[f]] = mma(tl[f], (kLk[f] ? x1 : x0).hi, U[kLm[f]]);
    if (more) load_t(c + 1);
    f32x4 D[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 dk = *reinterpret_cast<const f32x4*>(s[2] + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        U[mt][e] *= 1.0f / kTScale;
        D[mt][e] = U[mt][e] * dk[e];
      }
    }
    const Frag d0 = to_b(D[0], D[1]), d1 = to_b(D[2], D[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[mt][e] *= elc;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(kt[2 * mt], d0.hi, S[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(kt[2 * mt], d0.lo, S[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(kt[2 * mt + 1], d1.hi, S[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(kt[2 * mt + 1], d1.lo, S[mt]);
    if (NP == 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        S[mt] = mma(at<h8>(KTp(c) + (NF + 2 * mt) * kFrag, lane * 16), d0.hi, S[mt]);
        S[mt] = mma(at<h8>(KTp(c) + (NF + 2 * mt + 1) * kFrag, lane * 16), d1.hi, S[mt]);
      }
    }
    if (more) frags(kt, KTp(c + 1), NF);
    const Frag u0 = to_b(U[0], U[1]), u1 = to_b(U[2], U[3]);
    if (SAVE) {
      store_packed(p.w.U + ci * kC * d.VP, poff, u0, d.VP);
      store_packed(p.w.U + (ci * kC + 32) * d.VP, poff, u1, d.VP);
    }
    f32x4 y[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int f = 0; f < 6; ++f) y[kLm[f]] = mma(pf[f], (kLk[f] ? u1 : u0).hi, y[kLm[f]]);
    if (PP == 2) {
#pragma unroll
      for (int f = 0; f < 6; ++f) {
        y[kLm[f]] = mma(pf[f], (kLk[f] ? u1 : u0).lo, y[kLm[f]]);
        y[kLm[f]] = mma(at<h8>(Pp(c) + (6 + f) * kFrag, lane * 16), (kLk[f] ? u1 : u0).hi, y[kLm[f]]);
      }
    }
    if (more) frags(pf, Pp(c + 1), 6);
    char* out = static_cast<char*>(p.y) + ((b * d.T + c * kC) * d.H + h) * (d.V * ES);
    const int64_t yrow = fresh(vrow);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 eq = *reinterpret_cast<const f32x4*>(s[3] + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (ok && (left >= kC || 16 * mt + 4 * g + e < left))
          IO<A>::st(&at<char>(out + (16 * mt + e) * yrow, yoff), 0, fmaf(eq[e], aq[mt][e], y[mt][e] * rps) * rsv);
    }
  }
  if (p.h_last && ok) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = 16 * mt + 4 * g;
      if (row < d.K) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = S[mt][e] * rsv;
        *reinterpret_cast<f32x4*>(p.h_last + (bh * d.V + col) * d.K + row) = x;
      }
    }
  }
}

// ------------------------------------------------------------------ token by token
// Eight lanes share R rows of the state (16-byte pieces of 128-byte lines), all in registers over the call's tokens;
// both products of a token, S k and S q, are taken of the state before it: y = alpha S q + u (k . q).  Bound by
// reading and writing the state once.
__device__ __forceinline__ float sum8(float v) {   // over aligned groups of eight lanes
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true));    // lane ^ 1
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true));    // lane ^ 2
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true));   // 7 - lane
  return v;
}

__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true)));
  v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true)));
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true)));
}

template <Act A>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t i) {
  if constexpr (A == Act::F32) {
    return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
  } else {
    const u32x2 a = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
    return f32x4{IO<A>::cvt(a[0] & 0xffffu), IO<A>::cvt(a[0] >> 16), IO<A>::cvt(a[1] & 0xffffu), IO<A>::cvt(a[1] >> 16)};
  }
}

template <Act A, int R>
__global__ void __launch_bounds__(256) gdelta_step_kernel(const FwdArgs p) {
  constexpr int NV = 4;   // 16-byte pieces of a row per lane: d_k <= 128
  const Dims& d = p.d;
  const int l8 = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int nb = (d.V + 32 * R - 1) / (32 * R);
  const int64_t bh = blockIdx.x / nb, h = bh % d.H, b = bh / d.H, hk = h / (d.H / d.G);
  const int row0 = static_cast<int>(blockIdx.x % nb) * 32 * R + grp;
  f32x4 S[R][NV];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int row = row0 + 32 * i, col = 4 * (l8 + 8 * n);
      S[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (p.h0 && row < d.V && col < d.K) S[i][n] = *reinterpret_cast<const f32x4*>(p.h0 + (bh * d.V + row) * d.K + col);
    }
  const float rate = exp2_fast(p.a_log[h] * kLog2e), bias = p.dt_bias[h];
  for (int64_t t = 0; t < d.T; ++t) {
    const int64_t bt = b * d.T + t, qk = (bt * d.G + hk) * d.K;
    f32x4 k[NV], q[NV];
    float mk = 0.0f, mq = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int col = 4 * (l8 + 8 * n);
      k[n] = q[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (col < d.K) {
        k[n] = load4<A>(p.k, qk + col);
        q[n] = load4<A>(p.q, qk + col);
      }
    }
    const float alpha = exp2_fast(log2_decay(rate, p.a_raw[bt * d.H + h], bias)), beta = mscan::sigmoid(p.b_raw[bt * d.H + h]);
    float v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = row0 + 32 * i;
      v[i] = row < d.V ? IO<A>::ld(p.v, (bt * d.H + h) * d.V + row) : 0.0f;
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mk = max_finite(mk, k[n][e]);
        mq = max_finite(mq, q[n][e]);
      }
    const float pk = pow2_below(max8(mk), 2), pq = pow2_below(max8(mq), 2);
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[n][e] *= pk;
        q[n][e] *= pq;
        kk = fmaf(k[n][e], k[n][e], kk);
        qq = fmaf(q[n][e], q[n][e], qq);
        kq = fmaf(k[n][e], q[n][e], kq);
      }
    const float rk = unit_scale(sum8(kk), pk, d.eps), rq = unit_scale(sum8(qq), pq, d.eps) * d.scale;
    kq = sum8(kq) * rk * rq;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float sk = 0.0f, sq = 0.0f;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sk = fmaf(S[i][n][e], k[n][e], sk);
          sq = fmaf(S[i][n][e], q[n][e], sq);
        }
      sk = sum8(sk) * rk;
      sq = sum8(sq) * rq;
      const float u = beta * (v[i] - alpha * sk), uk = u * rk;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][n][e] = fmaf(uk, k[n][e], alpha * S[i][n][e]);
      const int row = row0 + 32 * i;
      if (l8 == 0 && row < d.V) IO<A>::st(p.y, (bt * d.H + h) * d.V + row, alpha * sq + u * kq);
    }
  }
  if (p.h_last) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int row = row0 + 32 * i, col = 4 * (l8 + 8 * n);
        if (row < d.V && col < d.K) *reinterpret_cast<f32x4*>(p.h_last + (bh * d.V + row) * d.K + col) = S[i][n];
      }
  }
}

// ------------------------------------------------------------------ launches
namespace {

template <Act A, int KP>
hipError_t launch_chunks(const FwdArgs& a, bool save, hipStream_t st) {
  const Dims& d = a.d;
  const unsigned bh = static_cast<unsigned>(d.B * d.H), nc = static_cast<unsigned>(d.nc);
  hipLaunchKernelGGL((gdelta_rows_kernel<A, KP>), dim3(static_cast<unsigned>(d.B * d.G) * nc), dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdelta_prep_kernel<A, KP>), dim3(bh * nc), dim3(256), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const dim3 grid(bh * (d.VP / 16));
  if (save) hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, true>), grid, dim3(64), 0, st, a);
  else hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, false>), grid, dim3(64), 0, st, a);
  return hipGetLastError();
}

template <Act A>
hipError_t launch_act(const FwdArgs& a, bool save, hipStream_t st) {
  return a.d.K <= 64 ? launch_chunks<A, 64>(a, save, st) : launch_chunks<A, 128>(a, save, st);
}

template <Act A>
hipError_t launch_step_act(const FwdArgs& a, hipStream_t st) {
  const int nb = (a.d.V + 31) / 32;
  hipLaunchKernelGGL((gdelta_step_kernel<A, 1>), dim3(static_cast<unsigned>(a.d.B * a.d.H * nb)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fwd(Act act, const FwdArgs& a, bool save, hipStream_t st) {
  switch (act) {
    case Act::F32: return launch_act<Act::F32>(a, save, st);
    case Act::BF16: return launch_act<Act::BF16>(a, save, st);
    default: return launch_act<Act::F16>(a, save, st);
  }
}

hipError_t launch_step(Act act, const FwdArgs& a, hipStream_t st) {
  switch (act) {
    case Act::F32: return launch_step_act<Act::F32>(a, st);
    case Act::BF16: return launch_step_act<Act::BF16>(a, st);
    default: return launch_step_act<Act::F16>(a, st);
  }
}

}  // namespace gdelta
