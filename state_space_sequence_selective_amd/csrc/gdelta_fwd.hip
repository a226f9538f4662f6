// Gated delta rule, forward: the chunks' operands, the per-chunk triangular
// inverse, the pass over the chunks, and the token-by-token step (gfx950).
// The algebra and the number format are in gdelta.h.
#include "gdelta_launch.h"

namespace gdelta {

// ------------------------------------------------------------------ q and k as operands
// One workgroup per (batch row, query / key head, chunk): each row's power of two and unit scale, and its f16 parts as
// fragments, through LDS.  Bound by HBM: q and k read once, three or (for a backward pass) four families of their size
// written (8192 tokens of 80 heads of 128 x 128: 1.03 GB in 184 us, 5.6 TB/s).
template <Act A, int KP>
__global__ void __launch_bounds__(256) gdelta_rows_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, EPT = KP / 4, ROW = KP + 8, KS = KP / 32;
  __shared__ __attribute__((aligned(16))) uint16_t s[2][NP][kC * ROW];
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
  const ChunkPlace at_ = chunk_place(blockIdx.x, static_cast<uint32_t>(d.G), static_cast<uint32_t>(d.nc));
  const int64_t c = at_.c, hk = at_.h, b = at_.b;
  const int64_t t0 = c * kC, left = d.T - t0, ci = (b * d.G + hk) * d.nc + c;
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
    // a row of zeros (those behind the sequence too) takes a power of two that keeps its scale, 1 / (sqrt(eps) pw), near 1:
    // what it multiplies has to stay inside f16 although it then meets zeros
    const float pw = m > 0.0f ? pow2_below(m, 2) : pow2_below(sqrtf(d.eps), 1);
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
// (v_mfma_f32_16x16x4_f32; full f32, as an inverse amplifies roundings of A).  Five workgroups a CU hide the solve's
// steps (271 -> 250 us), which leaves it to HBM: 8192 tokens of 80 heads of d_k = 128 are 1.33 GB, 5.3 TB/s.  f32 rows
// of 128 need the registers of four (a forward of 4096 tokens of 16 heads 808 -> 613 us).
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
__global__ void __launch_bounds__(256, A == Act::F32 && KP == 128 ? 4 : 5) gdelta_prep_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, KS = KP / 32, NF = KP / 8;
  __shared__ __attribute__((aligned(16))) float sA[kC * kAS];   // A, and block by block its place taken by T
  __shared__ double sG[kC];
  __shared__ __attribute__((aligned(16))) float sBeta[kC], sRk[kC], sRq[kC];
  __shared__ float sMax[4];
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
  const ChunkPlace at_ = chunk_place(blockIdx.x, static_cast<uint32_t>(d.H), static_cast<uint32_t>(d.nc));
  const int64_t c = at_.c, h = at_.h, b = at_.b, bh = b * d.H + h, hk = at_.h / (static_cast<uint32_t>(d.H) / static_cast<uint32_t>(d.G));
  const int64_t t0 = c * kC, left = d.T - t0, ci = bh * d.nc + c, gi = (b * d.G + hk) * d.nc + c;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* KF = p.w.KF + gi * (NP * NF * kFrag);
  const uint16_t* QF = p.w.QF + gi * (NP * NF * kFrag);
  // Wave w's operands: k of tiles 0 .. w, q of tiles w .. 3 (five tiles), and k and q of tile w, in flight while the gates
  // are made.  A slot s <= w gives the tile (rows j of s, columns i of w) of k.k^T and k.q^T, a later one (rows i of
  // s - 1, columns j of w) of q.k^T.  (All five tiles in flight would take 80 more registers, and two of five workgroups a
  // CU.)
  h8 bk[KS], bq[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    bk[ks] = at<h8>(KF + (wv * KS + ks) * kFrag, lane * 16);
    bq[ks] = at<h8>(QF + (wv * KS + ks) * kFrag, lane * 16);
  }
  if (tid < kC) {
    const bool ok = tid < left;
    const int64_t i = (b * d.T + t0 + tid) * d.H + h;
    const float rate = exp2_fast(p.a_log[h] * kLog2e);
    double G = ok ? log2_decay(rate, p.a_raw[i], p.dt_bias[h]) : 0.0f;
    const float beta = ok ? mscan::sigmoid(p.b_raw[i]) : 0.0f;
    const float rk = p.w.gsc[gi * (kGroupSc * kC) + G_RK * kC + tid], rq = p.w.gsc[gi * (kGroupSc * kC) + G_RQ * kC + tid];
    G = wave_scan(G);
    const uint64_t gb = __builtin_bit_cast(uint64_t, G);
    const uint64_t glo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(gb), 63));
    const uint64_t ghi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(gb >> 32), 63));
    const double Gl = __builtin_bit_cast(double, (ghi << 32) | glo);
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
    const int row = tid >> 2;   // four threads a row, four loads in flight
    for (int c0 = (tid & 3) * 8; c0 < d.V; c0 += 4 * 32) {
      float y[4][8];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        load8<A>(p.v, ((b * d.T + t0 + row) * d.H + h) * d.V + c0 + 32 * k, row < left && c0 + 32 * k < d.V, y[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_finite(m, y[k][e]);
    }
    if (c == 0 && p.h0) {
      float m0 = 0.0f;
      const float* h0 = p.h0 + bh * d.V * d.K;
      for (int i0 = tid * 4; i0 < d.V * d.K; i0 += 8 * 1024) {   // eight loads in flight: this workgroup would be the last
        f32x4 y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          y[k] = i0 + k * 1024 < d.V * d.K ? *reinterpret_cast<const f32x4*>(h0 + i0 + k * 1024) : zero;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) m0 = max_finite(m0, y[k][e]);
      }
      m = fmaxf(m, m0 * sqrtf(static_cast<float>(d.K)));
    }
    m = wave_max(m);
    if (lane == 0) sMax[wv] = m;
  }
  __syncthreads();
  if (tid == 0) p.w.vmax[ci] = fmaxf(fmaxf(sMax[0], sMax[1]), fmaxf(sMax[2], sMax[3]));
  {
    const int i = 16 * wv + r;
    const float rki = sRk[i], rqi = sRq[i], be = sBeta[i];
    const double Gi = sG[i];
    f32x4 P[4], PT[4];   // tile n of this wave's row of P's transpose, and of P
#pragma unroll
    for (int n = 0; n < 4; ++n) P[n] = PT[n] = zero;
#pragma unroll
    for (int s = 0; s < 5; ++s) {
      f32x4 xk = zero, xq = zero;
      const uint16_t* src = s <= wv ? KF + s * KS * kFrag : QF + (s - 1) * KS * kFrag;
      h8 x[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) x[ks] = at<h8>(src + ks * kFrag, lane * 16);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        xk = mma(x[ks], bk[ks], xk);
        xq = mma(x[ks], bq[ks], xq);
      }
      if (NP == 2) {   // the planes of low parts
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const h8 xl = at<h8>(src + (NF + ks) * kFrag, lane * 16);
          xk = mma(xl, bk[ks], xk);
          xq = mma(xl, bq[ks], xq);
          xk = mma(x[ks], at<h8>(KF + (NF + wv * KS + ks) * kFrag, lane * 16), xk);
          xq = mma(x[ks], at<h8>(QF + (NF + wv * KS + ks) * kFrag, lane * 16), xq);
        }
      }
      if (s <= wv) {   // rows j, column i
        const int j0 = 16 * s + 4 * g;
        const f32x4 rkj = *reinterpret_cast<const f32x4*>(sRk + j0);
        f32x4 a, q;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = j0 + e <= i ? rkj[e] * exp2_fast(static_cast<float>(Gi - sG[j0 + e])) : 0.0f;
          q[e] = rqi * w * xq[e];
          a[e] = j0 + e < i ? be * rki * w * xk[e] : 0.0f;
        }
        if (s < 4) P[s < 4 ? s : 3] = q;
        *reinterpret_cast<f32x4*>(sA + i * kAS + j0) = a;
      } else {         // rows i', column j = i
        const int i0 = 16 * (s - 1) + 4 * g;
        const f32x4 rq = *reinterpret_cast<const f32x4*>(sRq + i0);
        f32x4 q;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = i <= i0 + e ? rq[e] * rki * exp2_fast(static_cast<float>(sG[i0 + e] - Gi)) * xk[e] : 0.0f;
        PT[s > 0 ? s - 1 : 0] = q;
      }
    }
    constexpr int PP = kPPlanes<A>;
    uint16_t* dst = p.w.P + ci * (PP * 6 * kFrag);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && wv < 2) continue;
      const int f = wv < 2 ? wv : 2 * wv - 2 + ks;
      const Frag y = to_b(P[2 * ks], P[2 * ks + 1]);
      at<h8>(dst + f * kFrag, lane * 16) = y.hi;
      if (PP == 2) at<h8>(dst + (6 + f) * kFrag, lane * 16) = y.lo;
    }
    if (p.w.PT) {
      dst = p.w.PT + ci * (2 * 6 * kFrag);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks == 0 && wv >= 2) continue;
        const int f = wv < 2 ? 2 * wv + ks : 2 + wv;
        const Frag y = to_b(PT[2 * ks], PT[2 * ks + 1]);
        at<h8>(dst + f * kFrag, lane * 16) = y.hi;
        at<h8>(dst + (6 + f) * kFrag, lane * 16) = y.lo;
      }
    }
  }
  __syncthreads();
  if (wv == 0) {   // the four diagonal blocks: a lane solves one column
    float t[16];
    float* a = sA + (16 * g) * kAS + 16 * g;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[2] = {i == r ? 1.0f : 0.0f, 0.0f};   // two chains
#pragma unroll
      for (int j = 0; j < i; ++j) s[j & 1] = fmaf(-a[i * kAS + j], t[j], s[j & 1]);
      t[i] = s[0] + s[1];
    }
    mscan::wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i * kAS + r] = t[i];
  }
  __syncthreads();
  if (wv < 2) {    // blocks (1, 0) and (3, 2)
    const int o = 32 * wv;
    const f32x4 y = tile_mm(sA + (o + 16) * kAS + o + 16, tile_mm(sA + (o + 16) * kAS + o, sA + o * kAS + o, r, g, zero), r, g, zero);
    mscan::wave_lds_sync();
#pragma unroll
    for (int e = 0; e < 4; ++e) sA[(o + 16 + 4 * g + e) * kAS + o + r] = -y[e];
  }
  __syncthreads();
  f32x4 z[2];      // the lower left 32 x 32 block, one 16-column strip a wave
  if (wv < 2) {
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      z[mi] = zero;
      for (int kk = wv; kk < 2; ++kk)
        z[mi] = tile_mm(sA + (32 + 16 * mi) * kAS + 16 * kk, sA + 16 * kk * kAS + 16 * wv, r, g, z[mi]);
    }
  }
  __syncthreads();
  if (wv < 2) {
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      f32x4 y = zero;
#pragma unroll
      for (int kk = 0; kk <= mi; ++kk) y = tile_mm(sA + (32 + 16 * mi) * kAS + 32 + 16 * kk, z[kk], r, g, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) sA[(32 + 16 * mi + 4 * g + e) * kAS + 16 * wv + r] = -y[e];
    }
  }
  __syncthreads();
  uint16_t* T = p.w.T + ci * (12 * kFrag);
  for (int f = wv; f < 6; f += 4) {
    // rows of T: two runs of four columns; the second run of fragments 0 and 3 is above the diagonal
    const float* a = sA + (16 * kLm[f] + r) * kAS + 32 * kLk[f] + 4 * g;
    const f32x4 u = *reinterpret_cast<const f32x4*>(a), v = f == 0 || f == 3 ? zero : *reinterpret_cast<const f32x4*>(a + 16);
    const Frag y = to_b(u, v);
    at<h8>(T + f * kFrag, lane * 16) = y.hi;
    at<h8>(T + (6 + f) * kFrag, lane * 16) = y.lo;
  }
  if (p.w.TT) {
    T = p.w.TT + ci * (12 * kFrag);
    for (int f = wv; f < 6; f += 4) {
      // columns of T: the first run of fragments 2 (tile 1, step 0) and 5 (tile 3, step 1) is above the diagonal
      const float* a = sA + (32 * kUk[f] + 4 * g) * kAS + 16 * kUm[f] + r;
      f32x4 u = zero, v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (f != 2 && f != 5) u[e] = a[e * kAS];
        v[e] = a[(16 + e) * kAS];
      }
      const Frag y = to_b(u, v);
      at<h8>(T + f * kFrag, lane * 16) = y.hi;
      at<h8>(T + (6 + f) * kFrag, lane * 16) = y.lo;
    }
  }
}

// ------------------------------------------------------------------ pass over the chunks
// 16 columns of one head's S^T (rows: d_k) to a wave, or to two.  The chain from chunk to chunk (k S, T x, k^T u: 82
// matrix instructions of 16 cycles for d_k = 128) holds the state in registers, as the accumulators of its update; they
// are at once the B operand of its product with k, and u is one for the update, so it needs nothing of other lanes.  The
// output (y, and what a backward pass reads) takes the parts of S and u: of the same wave, or of the first wave through
// LDS, a chunk behind.  Two waves halve the chain's time a chunk where there are SIMDs for both; it is then bound by the
// chain: 16384 tokens of 32 heads of 128 x 128 take 560 us, 2.2 a chunk, of which 1.3 without any load.  Every family of
// fragments is loaded a chunk ahead, as soon as this chunk's are used; the last chunk loads its own again, so that the
// loop has no branch.
template <int KP>
struct PassBuf {
  h8 S[KP / 32][2][64], U[2][2][64];   // [step][high, low][lane]
};

// Fragments of a chunk in a shared buffer, in this order; 16-bit inputs only
template <Act A, int KP>
struct FwdRing {
  static constexpr int NF = KP / 8, KF = 0, QF = NF, T = 2 * NF, P = T + 12, N = P + 6 * kPPlanes<A>;
};

// RING: fragments come from the shared buffer instead of registers
template <Act A, int KP, bool RING>
struct Chain {
  static constexpr int NP = A == Act::F32 ? 2 : 1, MT = KP / 16, KS = KP / 32, NF = KP / 8;
  using Place = PassPlace<A>;
  using R = FwdRing<A, KP>;
  f32x4 S[MT];
  h8 kf[RING ? 1 : NF], kt[RING ? 1 : NF], th[RING ? 1 : 6], tl[RING ? 1 : 6];
  float sc[3], el;
  uint32_t v[4][4];
  const uint16_t *ring, *ring_t;   // + this lane's place, plain and for a transpose
  uint16_t* low;   // f32: the second planes of KF and KT

  template <int N>
  __device__ __forceinline__ h8 get(const h8 (&x)[N], int base, int i) const {
    if constexpr (RING) return ld8(ring + (base + i) * kFrag);
    else return x[i];
  }
  __device__ __forceinline__ h8 get_kt(int i) const {
    if constexpr (RING) return ld_trans<KP>(ring_t + R::KF * kFrag, i);
    else return kt[i];
  }
  template <int N>
  __device__ __forceinline__ void load(h8 (&x)[N], const uint16_t* base, int lane) {
    if constexpr (!RING) load_frags(x, base, lane);
  }
  __device__ __forceinline__ const uint16_t* KF(const FwdArgs& p, const Place& w, int64_t c) const { return p.w.KF + (w.bg * w.nc + c) * (NP * NF * kFrag); }
  __device__ __forceinline__ const uint16_t* KT(const FwdArgs& p, const Place& w, int64_t c) const { return p.w.KT + (w.bg * w.nc + c) * (NP * NF * kFrag); }
  __device__ __forceinline__ void load_t(const FwdArgs& p, const Place& w, int64_t c) {
    const uint16_t* x = p.w.T + (w.bh * w.nc + c) * (12 * kFrag);
    load(th, x, w.lane);
    load(tl, x + 6 * kFrag, w.lane);
  }
  __device__ __forceinline__ void load_sc(const FwdArgs& p, const Place& w, int64_t c, float sv) {
    const float* x = p.w.hsc + (w.bh * w.nc + c) * (kHeadSc * kC);
    sc[0] = x[H_BETA * kC + w.lane] * sv;
    sc[1] = x[H_BK * kC + w.lane];
    sc[2] = x[H_DK * kC + w.lane];
    el = x[H_E * kC + kC - 1];
  }
  __device__ __forceinline__ void load_v(const FwdArgs& p, const Place& w, int64_t c) {
    // columns behind d_v repeat the last one: whatever they hold meets zeros in the backward pass
    const int vcol = w.ok ? w.col : static_cast<int>(p.d.V) - 1;
    load_cols<typename Place::Raw>(v, static_cast<const char*>(p.v) + w.at_chunk(c), w.row, vcol * Place::ES, w.T - c * kC, w.g);
  }
  __device__ __forceinline__ void init(const FwdArgs& p, const Place& w, float sv) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      S[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      const int row = 16 * mt + 4 * w.g;
      if (p.h0 && w.ok && row < p.d.K) S[mt] = *reinterpret_cast<const f32x4*>(p.h0 + (w.bh * p.d.V + w.col) * p.d.K + row) * sv;
    }
    load(kf, KF(p, w, 0), w.lane);
    load_sc(p, w, 0, sv);
    load_t(p, w, 0);
    load_v(p, w, 0);
    load(kt, KT(p, w, 0), w.lane);
    load_low(0, KF(p, w, 0), w.lane);
    load_low(1, KT(p, w, 0), w.lane);
  }
  __device__ __forceinline__ void load_low(int i, const uint16_t* base, int lane) {
    if constexpr (NP == 2) copy_low<NF>(low + i * (NF * kFrag), base + NF * kFrag, lane);
  }
  // One chunk.  on_state(step, parts) for the entering state, on_u(parts, parts) for u.  s: [3][64] floats of the wave.
  template <class OnState, class OnU>
  __device__ __forceinline__ void step(const FwdArgs& p, const Place& w, int64_t c, float sv, float (*s)[kC], OnState on_state, OnU on_u) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t next = c + 1 < w.nc ? c + 1 : c;
    mscan::wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i][w.lane] = sc[i];
    mscan::wave_lds_sync();
    const float elc = el;
    load_sc(p, w, next, sv);
    if constexpr (NP == 2) wait_low();
    f32x4 x[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag f = to_b(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) x[mt] = mma(get(kf, R::KF, mt * KS + ks), f.hi, x[mt]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) x[mt] = mma(get(kf, R::KF, mt * KS + ks), f.lo, x[mt]);
      if (NP == 2) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) x[mt] = mma(ld8(low + (mt * KS + ks) * kFrag + w.lane * 8), f.hi, x[mt]);
      }
      on_state(ks, f);
    }
    load(kf, KF(p, w, next), w.lane);
    load_low(0, KF(p, w, next), w.lane);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 be = *reinterpret_cast<const f32x4*>(s[0] + 16 * mt + 4 * w.g), bk = *reinterpret_cast<const f32x4*>(s[1] + 16 * mt + 4 * w.g);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[mt][e] = fmaf(be[e], IO<A>::cvt(v[mt][e]), -bk[e] * x[mt][e]);
    }
    load_v(p, w, next);
    const Frag x0 = to_b(x[0], x[1]), x1 = to_b(x[2], x[3]);
    f32x4 U[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int f = 0; f < 6; ++f) U[kLm[f]] = mma(get(th, R::T, f), (kLk[f] ? x1 : x0).hi, U[kLm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) U[kLm[f]] = mma(get(th, R::T, f), (kLk[f] ? x1 : x0).lo, U[kLm[f]]);
#pragma unroll
    for (int f = 0; f < 6; ++f) U[kLm[f]] = mma(get(tl, R::T + 6, f), (kLk[f] ? x1 : x0).hi, U[kLm[f]]);
    load_t(p, w, next);
    f32x4 D[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) D[mt] = U[mt] * *reinterpret_cast<const f32x4*>(s[2] + 16 * mt + 4 * w.g);
    const Frag d0 = to_b(D[0], D[1]), d1 = to_b(D[2], D[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] *= elc;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(get_kt(2 * mt), d0.hi, S[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(get_kt(2 * mt), d0.lo, S[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(get_kt(2 * mt + 1), d1.hi, S[mt]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) S[mt] = mma(get_kt(2 * mt + 1), d1.lo, S[mt]);
    if (NP == 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        S[mt] = mma(ld8(low + (NF + 2 * mt) * kFrag + w.lane * 8), d0.hi, S[mt]);
        S[mt] = mma(ld8(low + (NF + 2 * mt + 1) * kFrag + w.lane * 8), d1.hi, S[mt]);
      }
    }
    load(kt, KT(p, w, next), w.lane);
    load_low(1, KT(p, w, next), w.lane);
    on_u(to_b(U[0], U[1]), to_b(U[2], U[3]));
  }
  __device__ __forceinline__ void finish(const FwdArgs& p, const Place& w, float rsv) const {
    if (!p.h_last || !w.ok) return;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = 16 * mt + 4 * w.g;
      if (row < p.d.K) *reinterpret_cast<f32x4*>(p.h_last + (w.bh * p.d.V + w.col) * p.d.K + row) = S[mt] * rsv;
    }
  }
};

template <Act A, int KP, bool SAVE, bool RING>
struct Output {
  static constexpr int NP = A == Act::F32 ? 2 : 1, KS = KP / 32, NF = KP / 8, PP = kPPlanes<A>;
  using Place = PassPlace<A>;
  using R = FwdRing<A, KP>;
  h8 qf[RING ? 1 : NF], pf[RING ? 1 : 6];
  float eq;
  f32x4 y[4];
  const uint16_t* ring;
  // the parts of S and u through LDS to wide stores: 2048 tokens of 96 heads of 64 x 64 take 94 us against 111; 8192 tokens
  // of 80 heads of 128 x 128 659 against 561
  static constexpr bool KEEP = SAVE && RING && KP == 64;
  uint16_t* kept;   // [KS][high, low] fragments of the wave's own
  uint16_t* low;    // f32: the second plane of QF

  template <int N>
  __device__ __forceinline__ h8 get(const h8 (&x)[N], int base, int i) const {
    if constexpr (RING) return ld8(ring + (base + i) * kFrag);
    else return x[i];
  }

  __device__ __forceinline__ const uint16_t* QF(const FwdArgs& p, const Place& w, int64_t c) const { return p.w.QF + (w.bg * w.nc + c) * (NP * NF * kFrag); }
  __device__ __forceinline__ const uint16_t* P(const FwdArgs& p, const Place& w, int64_t c) const { return p.w.P + (w.bh * w.nc + c) * (PP * 6 * kFrag); }
  __device__ __forceinline__ void load_q(const FwdArgs& p, const Place& w, int64_t c) {
    if constexpr (!RING) load_frags(qf, QF(p, w, c), w.lane);
    if constexpr (NP == 2) copy_low<NF>(low, QF(p, w, c) + NF * kFrag, w.lane);
    eq = p.w.hsc[(w.bh * w.nc + c) * (kHeadSc * kC) + H_EQ * kC + w.lane] * p.d.pscale;
  }
  __device__ __forceinline__ void load_p(const FwdArgs& p, const Place& w, int64_t c) {
    if constexpr (!RING) load_frags(pf, P(p, w, c), w.lane);
  }
  __device__ __forceinline__ void begin(const Place& w, float* s) {
    if constexpr (NP == 2) wait_low();
    mscan::wave_lds_sync();
    s[w.lane] = eq;
    mscan::wave_lds_sync();
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) y[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  __device__ __forceinline__ void state(const FwdArgs& p, const Place& w, int64_t c, int ks, const Frag& f) {
    if constexpr (KEEP) keep_parts(kept + 2 * ks * kFrag, w.lane, f);
    else if (SAVE) store_packed(p.w.S + ((w.bh * w.nc + c) * KP + 32 * ks) * p.d.VP, (4 * w.g * p.d.VP + w.col) * 4, f, p.d.VP);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) y[mt] = mma(get(qf, R::QF, mt * KS + ks), f.hi, y[mt]);
    if (PP == 2) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) y[mt] = mma(get(qf, R::QF, mt * KS + ks), f.lo, y[mt]);
    }
    if (NP == 2) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) y[mt] = mma(ld8(low + (mt * KS + ks) * kFrag + w.lane * 8), f.hi, y[mt]);
    }
  }
  __device__ __forceinline__ void u(const FwdArgs& p, const Place& w, int64_t c, float scale, const float* s, const Frag& u0, const Frag& u1) {
    const int64_t ci = w.bh * w.nc + c, next = c + 1 < w.nc ? c + 1 : c;
    load_q(p, w, next);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) y[mt] *= *reinterpret_cast<const f32x4*>(s + 16 * mt + 4 * w.g);
    if constexpr (KEEP) {
      const int off = store_off(w.lane, p.d.VP), v0 = w.col - w.r;
      mscan::wave_lds_sync();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) store_kept(p.w.S + (ci * KP + 32 * ks) * p.d.VP + v0, off, kept + 2 * ks * kFrag, w.lane, p.d.VP);
      mscan::wave_lds_sync();
      keep_parts(kept, w.lane, u0);
      keep_parts(kept + 2 * kFrag, w.lane, u1);
      mscan::wave_lds_sync();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) store_kept(p.w.U + (ci * kC + 32 * ks) * p.d.VP + v0, off, kept + 2 * ks * kFrag, w.lane, p.d.VP);
      mscan::wave_lds_sync();
    } else if (SAVE) {
      const int off = (4 * w.g * p.d.VP + w.col) * 4;
      store_packed(p.w.U + ci * kC * p.d.VP, off, u0, p.d.VP);
      store_packed(p.w.U + (ci * kC + 32) * p.d.VP, off, u1, p.d.VP);
    }
#pragma unroll
    for (int f = 0; f < 6; ++f) y[kLm[f]] = mma(get(pf, R::P, f), (kLk[f] ? u1 : u0).hi, y[kLm[f]]);
    if (PP == 2) {
#pragma unroll
      for (int f = 0; f < 6; ++f) {
        y[kLm[f]] = mma(get(pf, R::P, f), (kLk[f] ? u1 : u0).lo, y[kLm[f]]);
        y[kLm[f]] = mma(RING ? ld8(ring + (R::P + 6 + f) * kFrag) : at<h8>(P(p, w, c) + (6 + f) * kFrag, w.lane * 16), (kLk[f] ? u1 : u0).hi, y[kLm[f]]);
      }
    }
    load_p(p, w, next);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) y[mt] *= scale;
    store_cols<A>(y, static_cast<char*>(p.y) + w.at_chunk(c), w.row, w.col * Place::ES, w.T - c * kC, w.g, w.ok);
  }
};

// the head's power of two: |s|, |v - S k| <= 2 sqrt(T + 1) max(|v|, |h0|) scaled below 2^15
__device__ __forceinline__ float head_scale(const FwdArgs& p, int64_t bh, int lane) {
  float m = 0.0f;
  for (int64_t i = lane; i < p.d.nc; i += 64) m = fmaxf(m, p.w.vmax[bh * p.d.nc + i]);
  return pow2_below(wave_max(m), 15 - static_cast<int>(ceilf(1.0f + 0.5f * log2f(static_cast<float>(p.d.T) + 1.0f))));
}

template <Act A, int KP, bool SAVE, bool PAIR>
__global__ void __launch_bounds__(PAIR ? 128 : 64) gdelta_fwd_kernel(const FwdArgs p) {
  constexpr int KS = KP / 32;
  constexpr bool LOW = SAVE || kPPlanes<A> == 2;   // the output takes the low parts too
  __shared__ __attribute__((aligned(16))) float s[4][kC];   // beta sv; beta e rk; exp(G_63 - G) rk / e rq pscale
  const Dims& d = p.d;
  __shared__ __attribute__((aligned(16))) uint16_t low[3][A == Act::F32 ? KP / 8 * kFrag : 1];
  const PassPlace<A> w(d);
  const float sv = head_scale(p, w.bh, w.lane);
  const float rsv = 1.0f / sv, yscale = rsv / d.pscale;
  if (SAVE && threadIdx.x == 0 && w.col < 16) p.w.sv[w.bh] = sv;
  if constexpr (PAIR) {
    __shared__ __attribute__((aligned(16))) PassBuf<KP> buf[2];
    if (wave_id() == 0) {
      Chain<A, KP, false> ch;
      ch.low = low[0];
      ch.init(p, w, sv);
      for (int64_t c = 0; c < d.nc; ++c) {
        PassBuf<KP>& o = buf[c & 1];
        ch.step(p, w, c, sv, s,
                [&](int ks, const Frag& f) {
                  o.S[ks][0][w.lane] = f.hi;
                  if (LOW) o.S[ks][1][w.lane] = f.lo;
                },
                [&](const Frag& u0, const Frag& u1) {
                  o.U[0][0][w.lane] = u0.hi;
                  o.U[1][0][w.lane] = u1.hi;
                  if (LOW) {
                    o.U[0][1][w.lane] = u0.lo;
                    o.U[1][1][w.lane] = u1.lo;
                  }
                });
        mscan::lds_barrier();   // chunk c's parts are there, and the other wave is done with those of chunk c - 1
      }
      ch.finish(p, w, rsv);
    } else {
      Output<A, KP, SAVE, false> out;
      out.low = low[2];
      out.load_q(p, w, 0);
      out.load_p(p, w, 0);
      for (int64_t c = 0; c < d.nc; ++c) {
        const PassBuf<KP>& o = buf[c & 1];
        out.begin(w, s[3]);
        mscan::lds_barrier();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          Frag f;
          f.hi = o.S[ks][0][w.lane];
          if (LOW) f.lo = o.S[ks][1][w.lane];
          out.state(p, w, c, ks, f);
        }
        Frag u0, u1;
        u0.hi = o.U[0][0][w.lane];
        u1.hi = o.U[1][0][w.lane];
        if (LOW) {
          u0.lo = o.U[0][1][w.lane];
          u1.lo = o.U[1][1][w.lane];
        }
        out.u(p, w, c, yscale, s[3], u0, u1);
      }
    }
  } else {
    Chain<A, KP, false> ch;
    Output<A, KP, SAVE, false> out;
    ch.low = low[0];
    out.low = low[2];
    ch.init(p, w, sv);
    out.load_q(p, w, 0);
    out.load_p(p, w, 0);
    for (int64_t c = 0; c < d.nc; ++c) {
      out.begin(w, s[3]);
      ch.step(p, w, c, sv, s, [&](int ks, const Frag& f) { out.state(p, w, c, ks, f); },
              [&](const Frag& u0, const Frag& u1) { out.u(p, w, c, yscale, s[3], u0, u1); });
    }
    ch.finish(p, w, rsv);
  }
}

// The same for many tiles: TILES waves with a tile of one head each, and four that copy the chunk's fragments into LDS
// (50 KB for d_k = 128 and bf16, twice) a chunk ahead.  What bounds the kernel above, once it has several waves a CU, is
// every wave loading its own copy (12 bytes a clock and CU); this one the CU's path to memory, copies in and the parts of S
// and u out: 8192 tokens of 80 heads of 128 x 128 take 564 us, 2 GB of HBM traffic at 3.5 TB/s (the products alone 276),
// against 850 without sharing.  k's transpose is read out of k, which leaves a family less to copy (602 -> 564 us).
template <Act A, int KP, bool SAVE, int TILES>
__global__ void __launch_bounds__(64 * (TILES + kCopyWaves)) gdelta_fwd_ring_kernel(const FwdArgs p) {
  using R = FwdRing<A, KP>;
  constexpr int NF = R::NF;
  __shared__ __attribute__((aligned(16))) uint16_t ring[2][R::N * kFrag];
  __shared__ __attribute__((aligned(16))) float s[TILES][4][kC];
  __shared__ __attribute__((aligned(16))) uint16_t kept[TILES][Output<A, KP, SAVE, true>::KEEP ? KP / 16 * kFrag : 1];
  static_assert(sizeof(ring) + sizeof(s) + sizeof(kept) <= mscan::kLdsBytes, "LDS");
  const Dims& d = p.d;
  const int wv = wave_id();
  const PassPlace<A> w(d, TILES, wv < TILES ? wv : 0);
  if (wv >= TILES) {
    const int first = wv - TILES;
    auto copy = [&](int64_t c) {
      uint16_t* dst = ring[c & 1];
      const int64_t gi = w.bg * d.nc + c, ci = w.bh * d.nc + c;
      copy_frags<NF, kCopyWaves>(dst + R::KF * kFrag, p.w.KF + gi * (NF * kFrag), first, w.lane);
      copy_frags<NF, kCopyWaves>(dst + R::QF * kFrag, p.w.QF + gi * (NF * kFrag), first, w.lane);
      copy_frags<12, kCopyWaves>(dst + R::T * kFrag, p.w.T + ci * (12 * kFrag), first, w.lane);
      copy_frags<6 * kPPlanes<A>, kCopyWaves>(dst + R::P * kFrag, p.w.P + ci * (6 * kPPlanes<A> * kFrag), first, w.lane);
      wait_copies();
    };
    copy(0);
    mscan::lds_barrier();
    for (int64_t c = 0; c < d.nc; ++c) {
      if (c + 1 < d.nc) copy(c + 1);
      mscan::lds_barrier();   // chunk c + 1 is there, and chunk c's readers are done
    }
    return;
  }
  const float sv = head_scale(p, w.bh, w.lane);
  const float rsv = 1.0f / sv, yscale = rsv / d.pscale;
  if (SAVE && threadIdx.x == 0 && w.col < 16) p.w.sv[w.bh] = sv;
  Chain<A, KP, true> ch;
  Output<A, KP, SAVE, true> out;
  out.kept = kept[wv];
  const bool live = w.col < d.VP;   // a head's last workgroup may have tiles behind its columns
  if (live) {
    ch.init(p, w, sv);
    out.load_q(p, w, 0);
  }
  mscan::lds_barrier();
  for (int64_t c = 0; c < d.nc; ++c) {
    if (live) {
      ch.ring = out.ring = ring[c & 1] + w.lane * 8;
      ch.ring_t = ring[c & 1] + trans_lane(w.lane);
      out.begin(w, s[wv][3]);
      ch.step(p, w, c, sv, s[wv], [&](int ks, const Frag& f) { out.state(p, w, c, ks, f); },
              [&](const Frag& u0, const Frag& u1) { out.u(p, w, c, yscale, s[wv][3], u0, u1); });
    }
    mscan::lds_barrier();
  }
  if (live) ch.finish(p, w, rsv);
}

// ------------------------------------------------------------------ token by token
// Eight lanes share R rows of the state (16-byte pieces of 128-byte lines), all in registers over the call's tokens;
// both products of a token, S k and S q, are taken of the state before it: y = alpha S q + u (k . q).  Bound by
// reading and writing the state once, or by the latency of one load, the products and one store (5.8 us).
__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  return fmaxf(v, dpp<0x141>(v));
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

template <Act A, int R, bool STREAM>
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
      if (p.h0 && row < d.V && col < d.K) {
        const f32x4* src = reinterpret_cast<const f32x4*>(p.h0 + (bh * d.V + row) * d.K + col);
        if constexpr (STREAM) S[i][n] = __builtin_nontemporal_load(src);
        else S[i][n] = *src;
      }
    }
  const float rate = exp2_fast(p.a_log[h] * kLog2e), bias = p.dt_bias[h];
  for (int64_t t = 0; t < d.T; ++t) {
    const int64_t bt = b * d.T + t, qk = (bt * d.G + hk) * d.K;
    f32x4 k[NV], q[NV];
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
    float mk = 0.0f, mq = 0.0f;
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
        if (row < d.V && col < d.K) {
          f32x4* dst = reinterpret_cast<f32x4*>(p.h_last + (bh * d.V + row) * d.K + col);
          if constexpr (STREAM) __builtin_nontemporal_store(S[i][n], dst);
          else *dst = S[i][n];
        }
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
  const unsigned tiles = bh * (d.VP / 16);
  if (tiles <= (save && A != Act::F32 ? kPairTilesSave : kPairTiles)) {
    if (save) hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, true, true>), dim3(tiles), dim3(128), 0, st, a);
    else hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, false, true>), dim3(tiles), dim3(128), 0, st, a);
  } else if constexpr (A == Act::F32) {   // two planes a family: a chunk's fragments twice are more than the LDS
    if (save) hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, true, false>), dim3(tiles), dim3(64), 0, st, a);
    else hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, false, false>), dim3(tiles), dim3(64), 0, st, a);
  } else {
    ring_tiles<false>(bh, d.VP / 16, [&](auto n, unsigned grid) {
      constexpr int N = decltype(n)::value;
      if (save) hipLaunchKernelGGL((gdelta_fwd_ring_kernel<A, KP, true, N>), dim3(grid), dim3(64 * (N + kCopyWaves)), 0, st, a);
      else hipLaunchKernelGGL((gdelta_fwd_ring_kernel<A, KP, false, N>), dim3(grid), dim3(64 * (N + kCopyWaves)), 0, st, a);
    });
  }
  return hipGetLastError();
}

template <Act A>
hipError_t launch_act(const FwdArgs& a, bool save, hipStream_t st) {
  return a.d.K <= 64 ? launch_chunks<A, 64>(a, save, st) : launch_chunks<A, 128>(a, save, st);
}

// Up to this many blocks of 32 rows, two workgroups a CU, every group of lanes takes one row, the shorter way to the end
// (16 heads of one token: 6.1 us against 6.5).  Above, it takes two, so that twice the state is in flight, and the state
// passes the caches by: 256 sequences of 32 heads take 180 us (1.08 GB at 6.0 TB/s) against 204 through the caches and
// 242 with one row, 16 sequences 11.4 against 16.2.
constexpr int64_t kStepWide = 512;

template <Act A, int R, bool STREAM>
hipError_t launch_step_rows(const FwdArgs& a, hipStream_t st) {
  const int nb = (a.d.V + 32 * R - 1) / (32 * R);
  hipLaunchKernelGGL((gdelta_step_kernel<A, R, STREAM>), dim3(static_cast<unsigned>(a.d.B * a.d.H * nb)), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <Act A>
hipError_t launch_step_act(const FwdArgs& a, hipStream_t st) {
  return a.d.B * a.d.H * ((a.d.V + 31) / 32) <= kStepWide ? launch_step_rows<A, 1, false>(a, st)
                                                          : launch_step_rows<A, 2, true>(a, st);
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
