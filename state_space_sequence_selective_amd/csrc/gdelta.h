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

#include <type_traits>

#include "scan_common.h"
#include "wave_ops.h"

namespace gdelta {

using mscan::Act;
using mscan::exp2_fast;
using mscan::IO;
using mscan::kLog2e;
using waveops::dpp;
using waveops::sum8;
using waveops::sum16;
using waveops::wave_max;
using waveops::wave_scan;
using waveops::wave_sum;

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = 64;          // tokens per chunk
constexpr int kFrag = 512;      // u16 of one operand fragment: 64 lanes x 8
constexpr int kCopyWaves = 4;   // of a workgroup that shares its tiles' fragments in LDS

// per-token scalars of a chunk, per query / key head: k' = k pk is what the products take, k' rk the unit-length key;
// q' = q pq, and q' rq the unit-length query times the scale
enum { G_PK = 0, G_RK, G_PQ, G_RQ, kGroupSc };
// and per head: beta, e = exp(G), beta e rk, exp(G_63 - G) rk, e rq
enum { H_BETA = 0, H_E, H_BK, H_DK, H_EQ, kHeadSc };

struct Dims {
  int64_t B, T, H, G, nc;   // G: query / key heads
  int K, V, VP;             // d_k, d_v, d_v rounded up to 32
  float scale, eps;
  float pscale;             // power of two that P = q.k^T D is kept times (|P| <= |scale|)
};

// The (row tile, 32-column step) pairs of a lower triangular 64 x 64 matrix that hold anything but zeros, and those of
// its transpose: six fragments each
__device__ constexpr int kLm[6] = {0, 1, 2, 2, 3, 3}, kLk[6] = {0, 0, 0, 1, 0, 1};
__device__ constexpr int kUm[6] = {0, 0, 1, 1, 2, 3}, kUk[6] = {0, 1, 0, 1, 1, 1};

// What the kernels keep for each other.  Fragments are stored as a wave reads them: 1 KB, 16 bytes a lane, lane
// (r = l % 16, g = l / 16) holding elements (r, place order 8 g ..) of the operand, so the readers need neither LDS
// nor any rearranging.  f32 inputs have a second plane of every k and q family, with the low parts.
struct Kept {
  // [B * G][nc] outermost
  float* gsc;       // [kGroupSc][64]
  uint16_t* KF;     // [planes][4 token tiles][KP / 32] k', contracted over d_k
  uint16_t* KT;     // [planes][KP / 16][2] its transpose, contracted over tokens
  uint16_t* QF;     // the same of q'
  uint16_t* QT;     // only for a backward pass
  // [B * H][nc] outermost
  float* hsc;       // [kHeadSc][64]
  double* G;        // [64] log2 of the decay since the chunk's start
  uint16_t* P;      // [1 for bf16, else 2][6] lower triangle of q.k^T D, times pscale
  uint16_t* PT;     // [2][6] its transpose (backward)
  uint16_t* T;      // [2][6] the inverse (its diagonal is 1, so parts below f16's 2^-24 do not matter)
  uint16_t* TT;     // [2][6] its transpose (backward)
  float* vmax;      // largest finite |v| of the chunk (the first chunk's entry also holds the initial state's bound)
  float* sv;        // [B * H] the head's power of two for S and u
  uint32_t* S;      // [KP][VP] the state entering the chunk, f16 high | low << 16, times sv (backward)
  uint32_t* U;      // [64][VP] u, the same (backward)
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
  const void *dy;
  const float *a_raw, *a_log, *dt_bias;
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

// f32 pair -> packed f16 high parts and packed f16 remainders, both rounded to nearest (v_cvt_pk_f16_f32).  The
// remainder is exact in f32; v_fma_mix_f32 takes the f16 part as it is (a - h in one instruction).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), h2));
  float x, y;
  asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(x) : "v"(hi), "v"(a));
  asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(y) : "v"(hi), "v"(b));
  lo = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), h2));
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

// Buffer instructions: base in scalar registers, a 32-bit byte offset of the lane, one of the wave, and a constant.  Every
// access here is inside its array; the descriptor's own range check is not relied on.
using Buf = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Buf buf_of(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, 0x7fffffff, 0x00027000);
}
__device__ __forceinline__ h8 buf_h8(Buf b, int lane_off, int wave_off) {
  return __builtin_bit_cast(h8, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, wave_off, 0));
}
// n fragments of 1 KB from the buffer's base
template <int N>
__device__ __forceinline__ void load_frags(h8 (&x)[N], const void* base, int lane) {
  const Buf b = buf_of(base);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = buf_h8(b, lane * 16 + (i & 3) * 1024, (i >> 2) * 4096);
}

// Copies fragments `first`, first + STEP, .. of N from global memory into LDS, asynchronously and without registers
// (global_load_lds: 16 bytes a lane to consecutive places); wait_copies() ends it
template <int N, int STEP>
__device__ __forceinline__ void copy_frags(uint16_t* dst, const uint16_t* src, int first, int lane) {
#pragma unroll
  for (int i = 0; i < (N + STEP - 1) / STEP; ++i) {
    const int f = first + i * STEP;
    if (N % STEP == 0 || f < N)
      __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)(const_cast<uint16_t*>(src) + f * kFrag + lane * 8),
                                       (__attribute__((address_space(3))) void*)(dst + f * kFrag), 16, 0, 0);
  }
}
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt(0);
}

// A family's second plane (f32 inputs) into a wave's own LDS for its next chunk, once its reads of the last one are done;
// wait_low() ends it.  Loaded where they are used, these planes took 12 to 20 us a chunk of 128 x 128 in place of 4 to 7
// (4096 tokens of 16 heads: forward 614 -> 259 us).
template <int N>
__device__ __forceinline__ void copy_low(uint16_t* dst, const uint16_t* src, int lane) {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  copy_frags<N, 1>(dst, src, 0, lane);
}
__device__ __forceinline__ void wait_low() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Stores a split operand's parts as f16 high | low << 16 words to its 4 + 4 rows 4 g + e, 16 + 4 g + e of `words` words;
// off: the lane's byte offset in the first of them
__device__ __forceinline__ void store_packed(uint32_t* base, int off, const Frag& f, int words) {
  const u32x4 hi = __builtin_bit_cast(u32x4, f.hi), lo = __builtin_bit_cast(u32x4, f.lo);
  const Buf b = buf_of(base);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = (e >> 1) * 16 + (e & 1) * 2;
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_amdgcn_perm(lo[e], hi[e], 0x05040100), b, off, row * words * 4, 0);          // low halves
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_amdgcn_perm(lo[e], hi[e], 0x07060302), b, off, (row + 1) * words * 4, 0);    // high halves
  }
}

__device__ __forceinline__ h8 ld8(const uint16_t* p) { return *reinterpret_cast<const h8*>(p); }

// A fragment of a family's transpose out of the family's own fragments in LDS ([4 token tiles][KP / 32 steps of d_k]):
// ds_read_b64_tr_b16 takes four rows of 16 elements, 8 bytes a lane, and gives lane i their column i.  Here a row is a
// token's 16 d_k of tile mt, four lanes' pieces in a fragment.  f: the family + trans_lane(); i: 2 mt + step of 32 tokens.
__device__ __forceinline__ int trans_lane(int lane) { return ((lane & 3) * 16 + (lane >> 2)) * 8; }
__device__ __forceinline__ u32x2 read_trans(const uint16_t* a) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)a));
}
template <int KP>
__device__ __forceinline__ h8 ld_trans(const uint16_t* f, int i) {
  const uint16_t* a = f + (2 * (i & 1) * (KP / 32) + (i >> 2)) * kFrag + ((i >> 1) & 1) * 4;
  const u32x2 x = read_trans(a), y = read_trans(a + KP / 32 * kFrag);
  return __builtin_bit_cast(h8, (u32x4{x[0], x[1], y[0], y[1]}));
}

// The same from the parts in LDS (their 64 x 16 bytes each, high then low: keep_parts), read transposed so that a lane has
// four columns of a row: two stores of 16 bytes a lane in place of eight of 4.  base: the tile's first column; off:
// store_off().
__device__ __forceinline__ void keep_parts(uint16_t* lds, int lane, const Frag& f) {
  *reinterpret_cast<h8*>(lds + lane * 8) = f.hi;
  *reinterpret_cast<h8*>(lds + kFrag + lane * 8) = f.lo;
}
__device__ __forceinline__ int store_off(int lane, int words) { return ((lane & 15) * words + (lane >> 4) * 4) * 4; }
__device__ __forceinline__ void store_kept(uint32_t* base, int off, const uint16_t* lds, int lane, int words) {
  const Buf b = buf_of(base);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint16_t* a = lds + trans_lane(lane) + 4 * half;
    const u32x2 hi = read_trans(a), lo = read_trans(a + kFrag);
    const u32x4 x = {__builtin_amdgcn_perm(lo[0], hi[0], 0x05040100), __builtin_amdgcn_perm(lo[0], hi[0], 0x07060302),
                     __builtin_amdgcn_perm(lo[1], hi[1], 0x05040100), __builtin_amdgcn_perm(lo[1], hi[1], 0x07060302)};
    __builtin_amdgcn_raw_buffer_store_b128(x, b, off, 16 * half * words * 4, 0);
  }
}

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

constexpr int kCol = kC + 8;    // row length of a 64 x 64 f16 plane in LDS: 16 bytes of padding against bank conflicts

// Workgroup n of the kernels that take one chunk each -> batch row, chunk, head.  Chunks fastest: the other order, whose
// workgroups read whole rows of the [tokens][heads][..] tensors at one time, measured 4% more in the preparation.
struct ChunkPlace {
  uint32_t b, c, h;
};
__device__ __forceinline__ ChunkPlace chunk_place(uint32_t n, uint32_t heads, uint32_t nc) {
  const uint32_t m = n / nc;
  return {m / heads, n % nc, m % heads};
}

// rows times columns of two fragment rows (KS steps, NP planes NF fragments apart)
template <int NP, int KS, int NF>
__device__ __forceinline__ f32x4 frag_mm(const uint16_t* a, const uint16_t* b, int lane, f32x4 acc) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const h8 x = at<h8>(a + ks * kFrag, lane * 16), y = at<h8>(b + ks * kFrag, lane * 16);
    acc = mma(x, y, acc);
    if (NP == 2) {
      acc = mma(x, at<h8>(b + (NF + ks) * kFrag, lane * 16), acc);
      acc = mma(at<h8>(a + (NF + ks) * kFrag, lane * 16), y, acc);
    }
  }
  return acc;
}

// Workgroup n of `per` for each of `heads` heads -> (head, index): workgroups go to the eight XCDs (each with its own
// L2) in turn, so a head's are given numbers of one XCD, which then reads the head's operands from HBM once
__device__ __forceinline__ void xcd_head(uint32_t n, uint32_t per, uint32_t heads, uint32_t& head, uint32_t& idx) {
  if (heads % 8 == 0) {
    const uint32_t m = n >> 3;
    head = (m / per) * 8 + (n & 7);
    idx = m % per;
  } else {
    head = n / per;
    idx = n % per;
  }
}

template <Act A>
struct PassPlace {   // where a wave's columns are
  using Raw = std::conditional_t<A == Act::F32, uint32_t, uint16_t>;
  static constexpr int ES = sizeof(Raw);
  int lane, r, g, col, row;   // row: bytes from token to token
  bool ok;
  int64_t bh, h, b, bg, nc, T, HV;

  // `tiles` 16-column tiles to a workgroup, of which this wave has number `tile`
  __device__ __forceinline__ explicit PassPlace(const Dims& d, int tiles = 1, int tile = 0) {
    lane = threadIdx.x & 63;
    r = lane & 15;
    g = lane >> 4;
    uint32_t head, cb;
    xcd_head(blockIdx.x, (d.VP / 16 + tiles - 1) / tiles, static_cast<uint32_t>(d.B * d.H), head, cb);
    const uint32_t H = static_cast<uint32_t>(d.H), G = static_cast<uint32_t>(d.G);
    bh = head;
    h = head % H;
    b = head / H;
    bg = b * G + (head % H) / (H / G);
    col = (cb * tiles + tile) * 16 + r;
    ok = col < d.V;
    row = static_cast<int>(d.H) * d.V * ES;
    nc = d.nc;
    T = d.T;
    HV = h * d.V * ES;
  }
  __device__ __forceinline__ int64_t at_chunk(int64_t c) const { return (b * T + c * kC) * row + HV; }
};

// A wave's 16 columns of a chunk's [64][d_v] rows as raw bits: elements of rows 16 mt + 4 g + e.  Rows behind the sequence
// repeat its last one (what they hold meets zeros).  base: the chunk's first row of the head; row: bytes from token to
// token; col: the lane's byte offset in a row
template <class Raw>
__device__ __forceinline__ void load_cols(uint32_t (&v)[4][4], const char* base, int row, int col, int64_t left, int g) {
  const Buf b = buf_of(base);
  auto ld = [&](int lane_off, int wave_off) -> uint32_t {
    if constexpr (sizeof(Raw) == 2) return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(b, lane_off, wave_off, 0));
    else return __builtin_amdgcn_raw_buffer_load_b32(b, lane_off, wave_off, 0);
  };
  const int last = left < kC ? static_cast<int>(left) - 1 : kC - 1;   // one path for all chunks: no branch in the callers' loops
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 16 * mt + 4 * g + e;
      v[mt][e] = ld((t < last ? t : last) * row + col, 0);
    }
}

// Its counterpart: rounds and stores the wave's columns
template <Act A>
__device__ __forceinline__ void store_cols(const f32x4 (&x)[4], char* base, int row, int col, int64_t left, int g, bool ok) {
  const Buf b = buf_of(base);
  auto st = [&](float v, int lane_off, int wave_off) {
    if constexpr (A == Act::F32) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), b, lane_off, wave_off, 0);
    else if constexpr (A == Act::BF16)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v)), b, lane_off, wave_off, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<_Float16>(v)), b, lane_off, wave_off, 0);
  };
  if (!ok) return;
  const int off = 4 * g * row + col;
  if (left >= kC) {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) st(x[mt][e], off, (16 * mt + e) * row);
  } else {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (16 * mt + 4 * g + e < left) st(x[mt][e], off, (16 * mt + e) * row);
  }
}

}  // namespace gdelta
