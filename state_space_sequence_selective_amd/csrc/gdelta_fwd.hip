// Gated delta rule, forward: the per-chunk triangular inverse, the pass over
// the chunks, and the token-by-token step (gfx950).  The algebra and the
// number format are in gdelta.h.
#include <type_traits>

#include "gdelta_launch.h"

namespace gdelta {

// ------------------------------------------------------------------ chunk preparation
// One workgroup per (batch row, head, chunk): the tokens' gates and unit scales, A = beta k.k^T D in LDS, and its
// unit lower triangular inverse: four 16 x 16 diagonal blocks by substitution, then two levels of
// T21 = -T22 (A21 T11) on f32 matrix instructions (v_mfma_f32_16x16x4_f32; full f32, as an inverse amplifies
// roundings of A).
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

// the (row tile, 32-column step) pairs of T and of T^T that hold anything but zeros
__device__ constexpr int kTm[6] = {0, 1, 2, 2, 3, 3}, kTk[6] = {0, 0, 0, 1, 0, 1};
__device__ constexpr int kTTm[6] = {0, 0, 1, 1, 2, 3}, kTTk[6] = {0, 1, 0, 1, 1, 1};

template <Act A, int KP>
__global__ void __launch_bounds__(256) gdelta_prep_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1;
  constexpr int EPT = KP / 4;   // elements of a row per thread
  __shared__ __attribute__((aligned(16))) uint16_t sK[NP * kC * kRow<KP>];
  __shared__ __attribute__((aligned(16))) float sA[kC * kAS], sT[kC * kAS];
  __shared__ double sG[kC];
  __shared__ float sBeta[kC], sRk[kC], sMax[4];
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, r = lane & 15, g = lane >> 4;
  const int64_t c = blockIdx.x % d.nc, bh = blockIdx.x / d.nc, h = bh % d.H, b = bh / d.H, hk = h / (d.H / d.G);
  const int64_t t0 = c * kC, left = d.T - t0;
  float* sc = p.w.sc + (bh * d.nc + c) * (kSc * kC);
  if (tid < kC) {
    const bool ok = tid < left;
    const int64_t i = (b * d.T + t0 + tid) * d.H + h;
    const float rate = exp2_fast(p.a_log[h] * kLog2e);
    double G = ok ? log2_decay(rate, p.a_raw[i], p.dt_bias[h]) : 0.0f;
    const float beta = ok ? mscan::sigmoid(p.b_raw[i]) : 0.0f;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const double o = __shfl_up(G, s, 64);
      if (lane >= s) G += o;
    }
    sG[tid] = G;
    sBeta[tid] = beta;
    p.w.G[(bh * d.nc + c) * kC + tid] = G;
    sc[SC_BETA * kC + tid] = beta;
    sc[SC_E * kC + tid] = exp2_fast(static_cast<float>(G));
  }
  {
    const int row = tid >> 2, part = tid & 3;
    float x[EPT];
    const int64_t base = ((b * d.T + t0 + row) * d.G + hk) * d.K;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const void* src = which ? p.q : p.k;
      float m = 0.0f, ss = 0.0f;
#pragma unroll
      for (int e = 0; e < EPT; e += 8) {
        const int col = part * EPT + e;
        load8<A>(src, base + col, row < left && col < d.K, x + e);
      }
#pragma unroll
      for (int e = 0; e < EPT; ++e) m = max_finite(m, x[e]);
      m = fmaxf(m, __shfl_xor(m, 1, 64));
      m = fmaxf(m, __shfl_xor(m, 2, 64));
      const float pw = pow2_below(m, 2);
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        x[e] *= pw;
        ss = fmaf(x[e], x[e], ss);
      }
      ss += __shfl_xor(ss, 1, 64);
      ss += __shfl_xor(ss, 2, 64);
      const float rs = unit_scale(ss, pw, d.eps);
      if (which == 0) {
#pragma unroll
        for (int e = 0; e < EPT; e += 8) {
          u32x4 hi, lo;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a, bb;
            split2(x[e + 2 * k], x[e + 2 * k + 1], a, bb);
            hi[k] = a;
            lo[k] = bb;
          }
          uint16_t* dst = sK + row * kRow<KP> + part * EPT + e;
          *reinterpret_cast<u32x4*>(dst) = hi;
          if (NP == 2) *reinterpret_cast<u32x4*>(dst + kC * kRow<KP>) = lo;
        }
      }
      if (part == 0) {
        if (which == 0) sRk[row] = rs;
        sc[(which ? SC_PQ : SC_PK) * kC + row] = pw;
        sc[(which ? SC_RQ : SC_RK) * kC + row] = which ? rs * d.scale : rs;
      }
    }
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
  if (tid == 0) p.w.vmax[bh * d.nc + c] = fmaxf(fmaxf(sMax[0], sMax[1]), fmaxf(sMax[2], sMax[3]));
  for (int nt = 0; nt <= wv; ++nt) {
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < KP / 32; ++ks) {
      const uint16_t* pa = sK + (16 * wv + r) * kRow<KP> + 32 * ks + 8 * g;
      const uint16_t* pb = sK + (16 * nt + r) * kRow<KP> + 32 * ks + 8 * g;
      acc = mma(ld8(pa), ld8(pb), acc);
      if (NP == 2) {
        acc = mma(ld8(pa), ld8(pb + kC * kRow<KP>), acc);
        acc = mma(ld8(pa + kC * kRow<KP>), ld8(pb), acc);
      }
    }
    const int j = 16 * nt + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * wv + 4 * g + e;
      sA[i * kAS + j] = j < i ? sBeta[i] * (sRk[i] * sRk[j]) * acc[e] * exp2_fast(static_cast<float>(sG[i] - sG[j])) : 0.0f;
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
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    x = tile_mm(sA + (o + 16) * kAS + o, sT + o * kAS + o, r, g, x);
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    y = tile_mm(sT + (o + 16) * kAS + o + 16, x, r, g, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) sT[(o + 16 + 4 * g + e) * kAS + o + r] = -y[e];
  }
  __syncthreads();
  if (wv < 2) {    // the lower left 32 x 32 block, one 16-column strip a wave
    f32x4 x[2];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      x[mi] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int kk = wv; kk < 2; ++kk)
        x[mi] = tile_mm(sA + (32 + 16 * mi) * kAS + 16 * kk, sT + 16 * kk * kAS + 16 * wv, r, g, x[mi]);
    }
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk <= mi; ++kk) y = tile_mm(sT + (32 + 16 * mi) * kAS + 32 + 16 * kk, x[kk], r, g, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) sT[(32 + 16 * mi + 4 * g + e) * kAS + 16 * wv + r] = -y[e];
    }
  }
  __syncthreads();
  uint16_t* T = p.w.T + (bh * d.nc + c) * (kTFrag * 512);
  uint16_t* TT = p.w.TT ? p.w.TT + (bh * d.nc + c) * (kTFrag * 512) : nullptr;
  for (int it = tid; it < 2 * 6 * 64; it += 256) {
    const bool tr = it >= 6 * 64;
    if (tr && !TT) break;
    const int f = (it >> 6) % 6, i = 16 * (tr ? kTTm[f] : kTm[f]) + r, k0 = 32 * (tr ? kTTk[f] : kTk[f]);
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
    uint16_t* dst = (tr ? TT : T) + (f * 64 + lane) * 8;
    *reinterpret_cast<u32x4*>(dst) = hi;
    *reinterpret_cast<u32x4*>(dst + 6 * 512) = lo;
  }
}

// ------------------------------------------------------------------ pass over the chunks
// A wave holds 16 columns of one head's S^T (rows: d_k) in registers, as the accumulators of the state update; they
// are at once the B operand of the products with k and q, and u is one for the update, so a wave's chain needs no
// exchange with other waves.  The workgroup's waves share k, q and the masked q.k^T in LDS.
template <Act A, int KP, int NW>
struct FwdLds {
  static constexpr int NP = A == Act::F32 ? 2 : 1;
  uint16_t k[NP * kC * kRow<KP>];
  uint16_t q[NP * kC * kRow<KP>];
  uint16_t kT[NP * KP * kCol];
  uint16_t P[2 * kC * kCol];
  double G[kC];
  float beta[kC], ek[kC], eq[kC], dk[kC], rk[kC], rq[kC];
};

template <Act A, int KP, int NW, bool SAVE>
__global__ void __launch_bounds__(NW * 64) gdelta_fwd_kernel(const FwdArgs p) {
  constexpr int NP = A == Act::F32 ? 2 : 1, MT = KP / 16, KS = KP / 32;
  __shared__ __attribute__((aligned(16))) FwdLds<A, KP, NW> s;
  static_assert(sizeof(s) <= mscan::kLdsBytes, "LDS");
  const Dims& d = p.d;
  const int tid = threadIdx.x, lane = tid & 63, wv = wave_id(), r = lane & 15, g = lane >> 4;
  const int ncb = (d.VP / 16 + NW - 1) / NW;
  const int64_t bh = blockIdx.x / ncb, h = bh % d.H, b = bh / d.H, hk = h / (d.H / d.G);
  const int col = ((blockIdx.x % ncb) * NW + wv) * 16 + r;
  const bool ok = col < d.V, live = col < d.VP;
  using Raw = std::conditional_t<A == Act::F32, uint32_t, uint16_t>;
  constexpr int ES = sizeof(Raw);
  const uint32_t vrow = static_cast<uint32_t>(d.H) * d.V * ES, vcol = ok ? col : d.V - 1;   // bytes of a token's v; a column to read
  const uint32_t poff = (4 * g * d.VP + col) * 4;   // this lane's place in the packed S and U
  // the head's power of two: |s|, |v - S k| <= 2 sqrt(T + 1) max(|v|, |h0|) scaled below 2^15
  float m = 0.0f;
  for (int64_t i = lane; i < d.nc; i += 64) m = fmaxf(m, p.w.vmax[bh * d.nc + i]);
  const float sv = pow2_below(wave_max(m), 15 - static_cast<int>(ceilf(1.0f + 0.5f * log2f(static_cast<float>(d.T) + 1.0f))));
  const float rsv = 1.0f / sv, rps = 1.0f / d.pscale, svc = ok ? sv : 0.0f;
  if (SAVE && tid == 0 && blockIdx.x % ncb == 0) p.w.sv[bh] = sv;

  f32x4 S[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    S[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int row = 16 * mt + 4 * g;
    if (p.h0 && ok && row < d.K) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p.h0 + (bh * d.V + col) * d.K + row);
#pragma unroll
      for (int e = 0; e < 4; ++e) S[mt][e] = x[e] * sv;
    }
  }
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // what the next chunk reads, in flight while this one computes
  QkRegs<A, KP, NW * 64> qk;
  h8 th[6], tl[6];
  float scal[4];       // beta, e, rk, rq of token `lane`
  double G, Gl;
  uint32_t v[4][4];
  auto load_chunk = [&](int64_t c) {
    const int64_t t0 = c * kC, ci = bh * d.nc + c;
    const float* sc = p.w.sc + ci * (kSc * kC);
    qk.load(p.k, p.q, ((b * d.T + t0) * d.G + hk) * d.K, d.G * d.K, d.K, d.T - t0, sc, tid);
    G = p.w.G[ci * kC + lane];
    Gl = p.w.G[ci * kC + kC - 1];
    scal[0] = sc[SC_BETA * kC + lane];
    scal[1] = sc[SC_E * kC + lane];
    scal[2] = sc[SC_RK * kC + lane];
    scal[3] = sc[SC_RQ * kC + lane];
  };
  auto load_t = [&](int64_t c) {
    const uint16_t* T = p.w.T + (bh * d.nc + c) * (kTFrag * 512);
#pragma unroll
    for (int f = 0; f < 6; ++f) {
      th[f] = at<h8>(T + f * 512, lane * 16);
      tl[f] = at<h8>(T + (6 + f) * 512, lane * 16);
    }
  };
  auto load_v = [&](int64_t c) {
    const int64_t left = d.T - c * kC;
    const char* base = static_cast<const char*>(p.v) + ((b * d.T + c * kC) * d.H + h) * (d.V * ES);
    const uint32_t off = vrow * 4 * g + vcol * ES;
    const int64_t row = fresh(vrow);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[mt][e] = 0u;
        if (left >= kC || 16 * mt + 4 * g + e < left) v[mt][e] = at<Raw>(base + (16 * mt + e) * row, off);
      }
  };
  load_chunk(0);
  load_t(0);
  load_v(0);
  for (int64_t c = 0; c < d.nc; ++c) {
    const int64_t t0 = c * kC, left = d.T - t0, ci = bh * d.nc + c;
    mscan::lds_barrier();   // the previous chunk's readers are done
    qk.store(s.k, s.q, s.kT, nullptr, tid);
    if (wv == 0) {
      s.G[lane] = G;
      s.beta[lane] = scal[0];
      s.ek[lane] = scal[1] * scal[2];
      s.eq[lane] = scal[1] * scal[3];
      s.dk[lane] = exp2_fast(static_cast<float>(Gl - G)) * scal[2];
      s.rk[lane] = scal[2];
      s.rq[lane] = scal[3] * d.pscale;
    }
    const float el = exp2_fast(static_cast<float>(Gl));
    if (c + 1 < d.nc) load_chunk(c + 1);
    mscan::lds_barrier();
    // P = q.k^T D on and below the diagonal, zeros in the two tiles above it that a 32-wide step reads
#pragma unroll
    for (int n = 0; n < (12 + NW - 1) / NW; ++n) {
      const int i = wv + n * NW;
      if (12 % NW && i >= 12) break;
      const int mt = i < 2 ? 0 : i < 4 ? 1 : i < 8 ? 2 : 3, nt = i - (i < 2 ? 0 : i < 4 ? 2 : i < 8 ? 4 : 8);
      f32x4 acc = zero;
      if (nt <= mt) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint16_t* pa = s.q + (16 * mt + r) * kRow<KP> + 32 * ks + 8 * g;
          const uint16_t* pb = s.k + (16 * nt + r) * kRow<KP> + 32 * ks + 8 * g;
          acc = mma(ld8(pa), ld8(pb), acc);
          if (NP == 2) {
            acc = mma(ld8(pa), ld8(pb + kC * kRow<KP>), acc);
            acc = mma(ld8(pa + kC * kRow<KP>), ld8(pb), acc);
          }
        }
      }
      const int j = 16 * nt + r;
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float x[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int row = 16 * mt + 4 * g + e + o;
          x[o] = j <= row ? s.rq[row] * s.rk[j] * acc[e + o] * exp2_fast(static_cast<float>(s.G[row] - s.G[j])) : 0.0f;
        }
        uint32_t hi, lo;
        split2(x[0], x[1], hi, lo);
        uint16_t* dst = s.P + (16 * mt + 4 * g + e) * kCol + place(j);
        dst[0] = static_cast<uint16_t>(hi);
        dst[kCol] = static_cast<uint16_t>(hi >> 16);
        dst[kC * kCol] = static_cast<uint16_t>(lo);
        dst[kC * kCol + kCol] = static_cast<uint16_t>(lo >> 16);
      }
    }

    f32x4 ak[4], aq[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) ak[mt] = aq[mt] = zero;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag f = to_b(S[2 * ks], S[2 * ks + 1]);
      if (SAVE && live) store_packed(p.w.S + (ci * KP + 32 * ks) * d.VP, poff, f, d.VP);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const int at = (16 * mt + r) * kRow<KP> + 32 * ks + 8 * g;
        ak[mt] = mma_split<NP>(s.k + at, kC * kRow<KP>, f, ak[mt]);
        aq[mt] = mma_split<NP>(s.q + at, kC * kRow<KP>, f, aq[mt]);
      }
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 be = *reinterpret_cast<const f32x4*>(s.beta + 16 * mt + 4 * g), ek = *reinterpret_cast<const f32x4*>(s.ek + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) ak[mt][e] = be[e] * (IO<A>::cvt(v[mt][e]) * svc - ek[e] * ak[mt][e]);
    }
    const Frag x0 = to_b(ak[0], ak[1]), x1 = to_b(ak[2], ak[3]);
    f32x4 U[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int f = 0; f < 6; ++f) {
      const Frag& x = kTk[f] ? x1 : x0;
      f32x4 a = U[kTm[f]];
      a = mma(th[f], x.hi, a);
      a = mma(th[f], x.lo, a);
      U[kTm[f]] = mma(tl[f], x.hi, a);
    }
    if (c + 1 < d.nc) {
      load_v(c + 1);
      load_t(c + 1);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) U[mt][e] *= 1.0f / kTScale;
    const Frag u0 = to_b(U[0], U[1]), u1 = to_b(U[2], U[3]);
    if (SAVE && live) {
      store_packed(p.w.U + ci * kC * d.VP, poff, u0, d.VP);
      store_packed(p.w.U + (ci * kC + 32) * d.VP, poff, u1, d.VP);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f32x4 dk = *reinterpret_cast<const f32x4*>(s.dk + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) U[mt][e] *= dk[e];
    }
    const Frag d0 = to_b(U[0], U[1]), d1 = to_b(U[2], U[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[mt][e] *= el;
      const uint16_t* a = s.kT + (16 * mt + r) * kCol + 8 * g;
      S[mt] = mma_split<NP>(a, KP * kCol, d0, S[mt]);
      S[mt] = mma_split<NP>(a + 32, KP * kCol, d1, S[mt]);
    }
    mscan::lds_barrier();   // all of P
    char* y = static_cast<char*>(p.y) + ((b * d.T + t0) * d.H + h) * (d.V * ES);
    const uint32_t yoff = vrow * 4 * g + col * ES;
    const int64_t yrow = fresh(vrow);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      f32x4 a = zero;
      a = mma_split<2>(s.P + (16 * mt + r) * kCol + 8 * g, kC * kCol, u0, a);
      if (mt >= 2) a = mma_split<2>(s.P + (16 * mt + r) * kCol + 32 + 8 * g, kC * kCol, u1, a);
      const f32x4 eq = *reinterpret_cast<const f32x4*>(s.eq + 16 * mt + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (ok && (left >= kC || 16 * mt + 4 * g + e < left))
          IO<A>::st(&at<char>(y + (16 * mt + e) * yrow, yoff), 0, (eq[e] * aq[mt][e] + a[e] * rps) * rsv);
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

template <Act A, int KP, bool SAVE>
hipError_t launch_chunks(const FwdArgs& a, hipStream_t st) {
  constexpr int NW = 4;
  const Dims& d = a.d;
  const int64_t bh = d.B * d.H;
  hipLaunchKernelGGL((gdelta_prep_kernel<A, KP>), dim3(static_cast<unsigned>(bh * d.nc)), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int ncb = (d.VP / 16 + NW - 1) / NW;
  hipLaunchKernelGGL((gdelta_fwd_kernel<A, KP, NW, SAVE>), dim3(static_cast<unsigned>(bh * ncb)), dim3(NW * 64), 0, st, a);
  return hipGetLastError();
}

template <Act A>
hipError_t launch_act(const FwdArgs& a, bool save, hipStream_t st) {
  if (a.d.K <= 64) return save ? launch_chunks<A, 64, true>(a, st) : launch_chunks<A, 64, false>(a, st);
  return save ? launch_chunks<A, 128, true>(a, st) : launch_chunks<A, 128, false>(a, st);
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
