// Gated delta rule: argument blocks, the chunk algebra and the device helpers
// shared by its kernels (gfx950).
//
// One head's state S [d_v, d_k] with unit-length keys and queries (scale
// folded into q below):
//   u_t = beta_t (v_t - alpha_t S_{t-1} k_t),  S_t = alpha_t S_{t-1} + u_t k_t^T,
//   y_t = S_t q_t,  alpha_t = exp(g_t)
// Over a chunk of 64 tokens with entering state S and G_i the sum of g up to
// and including token i of the chunk, D_ij = exp(G_i - G_j), e_i = exp(G_i):
//   A_ij = beta_i (k_i . k_j) D_ij  (j < i),   T = (I + A)^-1
//   U    = T diag(beta) (V - diag(e) K S^T)
//   Y    = diag(e) Q S^T + (Q K^T o D, j <= i) U
//   S'   = e_63 S + sum_j exp(G_63 - G_j) u_j k_j^T
// so everything but the 64 x 64 solve is a product of tiles.
//
// Number format of the products.  v_mfma_f32_16x16x32_f16 multiplies f16 and
// adds in f32.  A bf16 or f16 input row, brought to [2, 4) at its largest
// element by a power of two, is one f16 exactly (elements 2^-18 below the
// largest lose bits at 2^-26 of it); any f32 value is the sum of two f16 parts
// with 22 significant bits, and a product of two split values drops only
// lo * lo (2^-22).  The state, u and their gradients are scaled by one power
// of two per head, chosen from proven bounds on their growth, so that they
// stay inside f16's range: with |k| <= 1 and alpha, beta <= 1 a column s of
// S^T obeys |s_t|^2 <= |s_{t-1}|^2 + max |v|^2, and its gradient
// |ds_{t-1}| <= alpha_t (|ds_t| + scale max |dy|).
#pragma once

#include "scan_common.h"

namespace gdelta {

using mscan::Act;
using mscan::exp2_fast;
using mscan::IO;
using mscan::kLog2e;

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = 64;          // tokens per chunk
constexpr int kSc = 6;          // per-token scalars kept per chunk: see below
constexpr int kTFrag = 12;      // 1 KB fragments of T (6 of its 8 row tile / k step pairs, high and low parts)

// rows of the per-chunk scalar block sc[kSc][64]
enum { SC_BETA = 0, SC_PK = 1, SC_RK = 2, SC_PQ = 3, SC_RQ = 4, SC_E = 5 };
// k' = k * pk is what the products take, and k' * rk the unit-length key; q' = q * pq, and q' * rq the unit-length
// query times the scale; e = exp(G)

struct Dims {
  int64_t B, T, H, G, nc;   // G: query / key heads
  int K, V, VP;             // d_k, d_v, d_v rounded up to 32
  float scale, eps;
  float pscale;             // power of two that P = q.k^T D is kept times (|P| <= |scale|)
};

// T's entries are at most 1: its f16 parts are kept times this, as small ones would lose bits below 2^-24
constexpr float kTScale = 4096.0f;

// What the chunks keep for each other and for the backward pass, [B * H][nc] outermost
struct Kept {
  float* sc;        // [6][64]
  double* G;        // [64] log2 of the decay since the chunk's start
  uint16_t* T;      // [12][64][8] f16: T's fragments, high then low parts
  uint16_t* TT;     // the same of T^T
  float* vmax;      // largest finite |v| of the chunk (the first chunk's entry also holds the initial state's bound)
  float* sv;        // [B * H] the head's power of two for S and u
  uint32_t* S;      // [KP][VP] the state entering the chunk, f16 high | low << 16, times sv
  uint32_t* U;      // [64][VP] u, the same
};

struct FwdArgs {
  Dims d;
  const void *q, *k, *v;
  const float *a_raw, *b_raw, *a_log, *dt_bias, *h0;
  void* y;
  float* h_last;
  Kept w;
};

struct BwdArgs {
  Dims d;
  const void *q, *k, *v, *dy;
  const float *a_raw, *b_raw, *a_log, *dt_bias;
  bool has_h0;
  Kept w;
  float* dymax;     // [B * H][nc]
  float* so;        // [B * H] the head's power of two for dS and du
  uint32_t* DS;     // [B * H][nc][KP][VP] gradient of the state leaving the chunk, packed, times so
  uint32_t* DU;     // [B * H][nc][64][VP] gradient of u's token-by-token form (T^T dU), the same
  float* part;      // [B * H][nc][2] the chunk's terms of d_a_log and d_dt_bias
  void *d_q, *d_k, *d_v;
  float *d_a_raw, *d_b_raw, *d_a_log, *d_dt_bias;
};

// ------------------------------------------------------------------ helpers

// v_mfma_f32_16x16x32_f16: lane l holds A[l % 16][8 (l / 16) + e], B[8 (l / 16) + e][l % 16] (e < 8) and
// D[4 (l / 16) + e][l % 16] (e < 4).
__device__ __forceinline__ f32x4 mma(h8 a, h8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The order in which a contracted index is laid out.  Two stacked D tiles hold rows 4 g + e and 16 + 4 g + e of a
// column in lane group g; taken as B's elements 8 g .. 8 g + 7 they are a B operand without any exchange between
// lanes, if the A operand has its columns in the same order: column x of a block of 32 stands at place(x).
__device__ __forceinline__ constexpr int place(int x) {
  return (x & ~31) + ((x & 15) >> 2) * 8 + ((x >> 4) & 1) * 4 + (x & 3);
}

// f32 pair -> packed f16 high parts and packed f16 remainders (towards zero: the remainder is exact in f32)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
  hi = __builtin_bit_cast(uint32_t, h);
  lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a - static_cast<float>(h[0]), b - static_cast<float>(h[1])));
}

struct Frag {
  h8 hi, lo;
};

// An address as a wave-uniform base and a 32-bit byte offset of the lane (the saddr form: no 64-bit address registers)
template <class T>
__device__ __forceinline__ T& at(void* base, uint32_t off) {
  return *reinterpret_cast<T*>(static_cast<char*>(base) + off);
}
template <class T>
__device__ __forceinline__ const T& at(const void* base, uint32_t off) {
  return *reinterpret_cast<const T*>(static_cast<const char*>(base) + off);
}

// The value, as something the compiler cannot carry out of a loop: multiples of a row length are cheaper to make again
// than to keep, one pair of scalar registers each
__device__ __forceinline__ int64_t fresh(int64_t x) {
  int lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
  asm volatile("" : "+s"(lo));
  return lo;
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// two stacked D tiles as a split B operand
__device__ __forceinline__ Frag to_b(f32x4 a, f32x4 b) {
  u32x4 hi, lo;
  uint32_t x, y;
  split2(a[0], a[1], x, y); hi[0] = x; lo[0] = y;
  split2(a[2], a[3], x, y); hi[1] = x; lo[1] = y;
  split2(b[0], b[1], x, y); hi[2] = x; lo[2] = y;
  split2(b[2], b[3], x, y); hi[3] = x; lo[3] = y;
  return {__builtin_bit_cast(h8, hi), __builtin_bit_cast(h8, lo)};
}

// Stores a split operand's parts as f16 high | low << 16 words to its 4 + 4 rows 4 g + e, 16 + 4 g + e of `rows` words;
// off: the lane's byte offset in the first of them
__device__ __forceinline__ void store_packed(uint32_t* base, uint32_t off, const Frag& f, int64_t rows_) {
  const int64_t rows = fresh(rows_);
  const u32x4 hi = __builtin_bit_cast(u32x4, f.hi), lo = __builtin_bit_cast(u32x4, f.lo);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t* q = base + ((e >> 1) * 16 + (e & 1) * 2) * rows;
    at<uint32_t>(q, off) = (hi[e] & 0xffffu) | (lo[e] << 16);
    at<uint32_t>(q + rows, off) = (hi[e] >> 16) | (lo[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ h8 ld8(const uint16_t* p) { return *reinterpret_cast<const h8*>(p); }

__device__ __forceinline__ float max_finite(float m, float x) {
  const float a = fabsf(x);
  return a < 3.0e38f ? fmaxf(m, a) : m;   // false for NaN too
}

// largest power of two p with p * x < 2^e; 1 for x = 0
__device__ __forceinline__ float pow2_below(float x, int e) {
  if (!(x > 0.0f)) return 1.0f;
  int k;
  frexpf(x, &k);                       // x in [2^(k-1), 2^k)
  k = e - k;
  k = k > 120 ? 120 : (k < -120 ? -120 : k);
  return ldexpf(1.0f, k);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v = fmaxf(v, __shfl_xor(v, s, 64));
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s, 64);
  return v;
}

__device__ __forceinline__ float sum16(float v) {   // over the 16 lanes of one l / 16 group
  v += __shfl_xor(v, 1, 64);
  v += __shfl_xor(v, 2, 64);
  v += __shfl_xor(v, 4, 64);
  v += __shfl_xor(v, 8, 64);
  return v;
}

// 8 consecutive elements (16-byte aligned) as f32, zeros if !ok
template <Act A>
__device__ __forceinline__ void load8(const void* p, int64_t i, bool ok, float* out) {
  if (!ok) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = 0.0f;
    return;
  }
  if constexpr (A == Act::F32) {
    const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const f32x4 a = s[0], b = s[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[e] = a[e];
      out[4 + e] = b[e];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[2 * e] = IO<A>::cvt(a[e] & 0xffffu);
      out[2 * e + 1] = IO<A>::cvt(a[e] >> 16);
    }
  }
}

// log2 of the decay and the write strength of one token
__device__ __forceinline__ float log2_decay(float rate, float a_raw, float dt_bias) {
  return -rate * mscan::softplus(a_raw + dt_bias) * kLog2e;
}

// the scale of a row with largest element m and sum of squares ss of the SCALED row (eps scaled along)
__device__ __forceinline__ float unit_scale(float ss, float p, float eps) { return 1.0f / sqrtf(ss + eps * p * p); }

// LDS planes of one chunk: rows of KP (or 64) f16, 16 bytes of padding against bank conflicts
template <int KP>
constexpr int kRow = KP + 8;    // [64][kRow]: token rows, d_k in place() order
constexpr int kCol = kC + 8;    // [KP][kCol] and [64][kCol]: token columns in place() order

// A workgroup's share of a chunk's q and k rows on their way from global memory to LDS.  A unit is four token rows by
// eight columns; k's units come first, then q's, NU of them to each of NT threads.
template <Act A, int KP, int NT>
struct QkRegs {
  static constexpr int NG = KP / 8, UNITS = (kC / 4) * NG, NU = 2 * UNITS / NT;
  static constexpr int W = A == Act::F32 ? 2 : 1;
  static_assert(2 * UNITS % NT == 0 && UNITS % 64 == 0, "a wave's units are all of k or all of q");
  u32x4 x[NU][4][W];
  f32x4 pw[NU];

  // q, k: element 0 of the chunk's first row of the head; rows `stride` elements apart, `left` of them; K columns
  __device__ __forceinline__ void load(const void* k, const void* q, int64_t base, int64_t stride, int K, int64_t left,
                                       const float* sc, int tid) {
    const int w0 = wave_id() * 64;
    const bool full = left >= kC && K == KP;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int n = (tid + u * NT) % UNITS, c = (n % NG) * 8, t = (n / NG) * 4;
      const bool isq = w0 + u * NT >= UNITS;
      const char* src = static_cast<const char*>(isq ? q : k) + base * (W * 2);
      const uint32_t off = (static_cast<uint32_t>(t) * static_cast<uint32_t>(stride) + c) * (W * 2);
      pw[u] = at<f32x4>(sc + (isq ? SC_PQ : SC_PK) * kC, t * 4);
      if (full) {
        const int64_t row = fresh(stride * (W * 2));
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int w = 0; w < W; ++w) x[u][r][w] = at<u32x4>(src + r * row + 16 * w, off);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int w = 0; w < W; ++w) {
            x[u][r][w] = u32x4{0u, 0u, 0u, 0u};
            if (t + r < left && c < K) x[u][r][w] = at<u32x4>(src + r * stride * (W * 2) + 16 * w, off);
          }
      }
    }
  }

  // token rows to `rows` (the other of k's and q's plane sets), their transposes to `cols` (nullptr: not wanted)
  __device__ __forceinline__ void store(uint16_t* krows, uint16_t* qrows, uint16_t* kcols, uint16_t* qcols, int tid) const {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int n = (tid + u * NT) % UNITS, c = (n % NG) * 8, t = (n / NG) * 4;
      const bool isq = wave_id() * 64 + u * NT >= UNITS;
      uint16_t* rows = isq ? qrows : krows;
      uint16_t* cols = isq ? qcols : kcols;
      float f[4][8];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (A == Act::F32) f[r][e] = __builtin_bit_cast(float, static_cast<uint32_t>(x[u][r][e / 4][e % 4]));
          else f[r][e] = IO<A>::cvt((e & 1) ? x[u][r][0][e / 2] >> 16 : x[u][r][0][e / 2] & 0xffffu);
          f[r][e] *= pw[u][r];
        }
#pragma unroll
      for (int pl = 0; pl < W; ++pl) {
        uint32_t w[4][4];   // packed pairs along d_k
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = f[r][2 * e], b = f[r][2 * e + 1];
            const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
            w[r][e] = __builtin_bit_cast(uint32_t, h);
            if (W == 2 && pl == 0) {
              f[r][2 * e] = a - static_cast<float>(h[0]);
              f[r][2 * e + 1] = b - static_cast<float>(h[1]);
            }
          }
        if (rows) {
          uint16_t* p = rows + pl * kC * kRow<KP>;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            *reinterpret_cast<u32x2*>(p + (t + r) * kRow<KP> + place(c)) = u32x2{w[r][0], w[r][1]};
            *reinterpret_cast<u32x2*>(p + (t + r) * kRow<KP> + place(c + 4)) = u32x2{w[r][2], w[r][3]};
          }
        }
        if (cols) {
          uint16_t* p = cols + pl * KP * kCol;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a = w[0][e], b = w[1][e], cc = w[2][e], dd = w[3][e];
            *reinterpret_cast<u32x2*>(p + (c + 2 * e) * kCol + place(t)) =
                u32x2{(a & 0xffffu) | (b << 16), (cc & 0xffffu) | (dd << 16)};
            *reinterpret_cast<u32x2*>(p + (c + 2 * e + 1) * kCol + place(t)) =
                u32x2{(a >> 16) | (b & 0xffff0000u), (cc >> 16) | (dd & 0xffff0000u)};
          }
        }
      }
    }
  }
};

// Stages a chunk's q and k at once (no overlap with anything)
template <Act A, int KP, int NT>
__device__ __forceinline__ void stage_qk(const void* k, const void* q, int64_t base, int64_t stride, int K, int64_t left,
                                         const float* sc, uint16_t* krows, uint16_t* qrows, uint16_t* kcols, uint16_t* qcols,
                                         int tid) {
  QkRegs<A, KP, NT> x;
  x.load(k, q, base, stride, K, left, sc, tid);
  x.store(krows, qrows, kcols, qcols, tid);
}

// acc += A-rows (NA planes) times a split B operand: the products that matter at 22 bits
template <int NA>
__device__ __forceinline__ f32x4 mma_split(const uint16_t* a, int plane, const Frag& b, f32x4 acc) {
  const h8 ah = ld8(a);
  acc = mma(ah, b.hi, acc);
  acc = mma(ah, b.lo, acc);
  if (NA == 2) acc = mma(ld8(a + plane), b.hi, acc);
  return acc;
}


}  // namespace gdelta
