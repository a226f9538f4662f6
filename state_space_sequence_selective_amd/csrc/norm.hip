// Layer norm, forward and backward (gfx950), and the entry points of
// include/mamba_norm.h.
//
// A team of 8 to 1024 lanes holds one row in registers, a 16-byte piece a lane
// and step, so a row is read once: the mean, the centred sum of squares and
// the output all come from registers.  The backward keeps the columns' sums
// for d_w and d_b in registers over the rows its workgroup walks (the next
// row's loads in flight), writes one partial row per workgroup, and a second
// launch adds the partials in a fixed order (no atomics).  Both are bound by
// HBM.
#include <cmath>
#include <string>

#include "mamba_norm.h"
#include "scan_common.h"
#include "wave_ops.h"

namespace mscan {
void set_last_error(const std::string& msg);   // abi.hip
}

namespace lnorm {

using mscan::Act;
using mscan::IO;

struct Args {
  int64_t rows;
  int dim;
  float eps;
  const void *x, *dy, *d_add;
  const float *w, *b;
  void *y, *dx;
  float *mean, *rstd;
  float* part;   // [blocks][2][dim]
  float *d_w, *d_b;
  int blocks;
};

// E elements of type A as they lie in memory
template <Act A, int E>
struct Piece {
  static constexpr int S = A == Act::F32 ? 4 : 2, W = E * S / 4;
  uint32_t w[W];

  // from element i on, the first n of them inside the row.  Rows of an odd length start at any element, so the vector
  // accesses claim no more than the element's own alignment.
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const char* src = static_cast<const char*>(p) + i * S;
    if (n >= E) {
      __builtin_memcpy(w, __builtin_assume_aligned(src, S), E * S);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = 0u;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < n) w[e * S / 4] |= IO<A>::ldraw(p, i + e) << (S == 2 && (e & 1) ? 16 : 0);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (S == 4) return __builtin_bit_cast(float, w[e]);
    else return IO<A>::cvt((e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu);
  }
};

template <Act A, int E>
__device__ __forceinline__ void store_piece(void* p, int64_t i, int n, const float* v) {
  constexpr int S = A == Act::F32 ? 4 : 2;
  if (n >= E) {
    uint32_t w[E * S / 4];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (A == Act::F32) {
        w[e] = __builtin_bit_cast(uint32_t, v[e]);
      } else {
        uint16_t h;
        if constexpr (A == Act::BF16) h = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[e]));
        else h = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[e]));
        w[e / 2] = (e & 1) ? w[e / 2] | (static_cast<uint32_t>(h) << 16) : h;
      }
    }
    __builtin_memcpy(__builtin_assume_aligned(static_cast<char*>(p) + i * S, S), w, E * S);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < n) IO<A>::st(p, i + e, v[e]);
  }
}

template <int E>
__device__ __forceinline__ void load_weight(const float* p, int i, int n, float fill, float* out) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = fill;
  } else {
    Piece<Act::F32, E> x;
    x.load(p, i, n);
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = x.get(e);
  }
}

// Sum over a team; every lane gets it.  `s`: one float per wave and slot.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* s) {
  if constexpr (TEAM == 8) return waveops::sum8(v);
  if constexpr (TEAM == 16) return waveops::sum16(v);
  v = waveops::wave_sum(v);
  if constexpr (TEAM > 64) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TEAM / 64; ++i) v += s[i];
  }
  return v;
}

// elements of a lane's piece: 16 bytes of the wider type
template <Act X, Act Y>
constexpr int kPiece = X == Act::F32 || Y == Act::F32 ? 4 : 8;

// A workgroup walks rows too: w and b stay in its registers (read again for every row they would be more than the row:
// 40 KB of 5120 columns against 20), and the next row's loads are in flight.  16384 x 5120, f32 to bf16: 93 us, 5.4 TB/s;
// one row: 3.5 us.
template <Act X, Act Y, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) norm_fwd_kernel(const Args p) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM, TEAMS = BLOCK / TEAM, E = kPiece<X, Y>;
  __shared__ float s[2][2][BLOCK / 64];
  const int lane = threadIdx.x % TEAM;
  const float inv = 1.0f / static_cast<float>(p.dim);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
  int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TEAM;
  Piece<X, E> raw[NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = E * (lane + i * TEAM);
      raw[i].load(p.x, r * p.dim + col, r < p.rows ? p.dim - col : 0);
    }
  };
  load(row);
  float w[NV][E], b[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = E * (lane + i * TEAM);
    load_weight<E>(p.w, col, p.dim - col, 1.0f, w[i]);
    load_weight<E>(p.b, col, p.dim - col, 0.0f, b[i]);
  }
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * TEAMS; row0 < p.rows; row0 += stride, row += stride) {
    const bool ok = row < p.rows;
    float x[NV][E];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[i][e] = raw[i].get(e);
        sum += x[i][e];
      }
    load(row + stride);
    const float mean = team_sum<TEAM>(sum, s[turn][0]) * inv;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = p.dim - E * (lane + i * TEAM);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[i][e] = e < n ? x[i][e] - mean : 0.0f;
        sq = fmaf(x[i][e], x[i][e], sq);
      }
    }
    const float rstd = 1.0f / sqrtf(team_sum<TEAM>(sq, s[turn][1]) * inv + p.eps);
    turn ^= 1;   // the next row's sums go to the other slots: a barrier lies between this row's reads and those
    if (!ok) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = E * (lane + i * TEAM), n = p.dim - col;
      if (n <= 0) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) x[i][e] = fmaf(x[i][e] * rstd, w[i][e], b[i][e]);
      store_piece<Y, E>(p.y, row * p.dim + col, n, x[i]);
    }
    if (lane == 0 && p.mean) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

// 16384 x 5120, f32 and bf16, with d_add: 217 us (1.17 GB at 5.4 TB/s) and 10 us for the partial rows; 196608 x 64 of f16
// 25 us (101 MB at 4.0 TB/s) and 5 us.
template <Act X, Act Y, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) norm_bwd_kernel(const Args p) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM, TEAMS = BLOCK / TEAM, E = kPiece<X, Y>;
  __shared__ float s[2][2][BLOCK / 64];
  __shared__ float cols[TEAMS > 1 ? 2 * TEAM * NV * E : 1];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  float dw[NV][E], db[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.0f;
  const float inv = 1.0f / static_cast<float>(p.dim);
  // the row at work and the next one, as they lie in memory
  Piece<X, E> rx[NV], ra[NV];
  Piece<Y, E> ry[NV];
  float rmean, rrstd;
  auto load = [&](int64_t row) {
    const bool ok = row < p.rows;
    rmean = ok ? p.mean[row] : 0.0f;
    rrstd = ok ? p.rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = E * (lane + i * TEAM), left = ok ? p.dim - col : 0;
      rx[i].load(p.x, row * p.dim + col, left);
      ry[i].load(p.dy, row * p.dim + col, left);
      if (p.d_add) ra[i].load(p.d_add, row * p.dim + col, left);
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * TEAMS;
  load(row0 + team);
  int turn = 0;
  for (; row0 < p.rows; row0 += stride) {
    const int64_t row = row0 + team;
    const bool ok = row < p.rows;
    const float mean = rmean, rstd = rrstd;
    float n[NV][E], dn[NV][E], add[NV][E];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = E * (lane + i * TEAM), left = ok ? p.dim - col : 0;
      float w[E];
      load_weight<E>(p.w, col, p.dim - col, 1.0f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        n[i][e] = e < left ? (rx[i].get(e) - mean) * rstd : 0.0f;
        dn[i][e] = ry[i].get(e);
        add[i][e] = p.d_add ? ra[i].get(e) : 0.0f;
        db[i][e] += dn[i][e];
        dw[i][e] = fmaf(dn[i][e], n[i][e], dw[i][e]);
        dn[i][e] *= w[e];
        s1 += dn[i][e];
        s2 = fmaf(dn[i][e], n[i][e], s2);
      }
    }
    load(row + stride);
    s1 = team_sum<TEAM>(s1, s[turn][0]) * inv;
    s2 = team_sum<TEAM>(s2, s[turn][1]) * inv;
    turn ^= 1;   // the next row's sums go to the other slots: a barrier lies between this row's reads and those
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = E * (lane + i * TEAM), left = ok ? p.dim - col : 0;
      if (left <= 0) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) n[i][e] = fmaf(rstd, dn[i][e] - s1 - n[i][e] * s2, add[i][e]);
      store_piece<X, E>(p.dx, row * p.dim + col, left, n[i]);
    }
  }
  if (!p.part) return;
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
  if constexpr (TEAMS > 1) {
    for (int k = 0; k < TEAMS; ++k) {
      if (team == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float* a = cols + (i * E + e) * TEAM + lane;
            a[0] = (k ? a[0] : 0.0f) + dw[i][e];
            a[NV * E * TEAM] = (k ? a[NV * E * TEAM] : 0.0f) + db[i][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.dim; c += BLOCK) {
      const int l = (c / E) % TEAM, i = (c / E) / TEAM, e = c % E;
      const float* a = cols + (i * E + e) * TEAM + l;
      part[c] = a[0];
      part[p.dim + c] = a[NV * E * TEAM];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = E * (lane + i * TEAM), n = p.dim - col;
      if (n <= 0) continue;
      store_piece<Act::F32, E>(part, col, n, dw[i]);
      store_piece<Act::F32, E>(part, p.dim + col, n, db[i]);
    }
  }
}

// d_w, d_b += the sum of the partial rows: 16 columns a workgroup, 64 strips of partials, then the strips in order
__global__ void __launch_bounds__(1024) norm_colsum_kernel(const Args p) {
  __shared__ float s[64][17];
  const int c = threadIdx.x & 15, strip = threadIdx.x >> 4;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c;
  const int64_t n = 2 * static_cast<int64_t>(p.dim);
  float acc = 0.0f;
  for (int r0 = strip; r0 < p.blocks; r0 += 64 * 8) {   // eight loads in flight
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = col < n && r0 + 64 * k < p.blocks ? p.part[(r0 + 64 * k) * n + col] : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc += v[k];
  }
  s[strip][c] = acc;
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (strip < o) s[strip][c] += s[strip + o][c];
    __syncthreads();
  }
  if (strip == 0 && col < n) {
    float* out = col < p.dim ? p.d_w : p.d_b;
    if (out) out[col < p.dim ? col : col - p.dim] += s[0][c];
  }
}

namespace {

thread_local const char* g_fn = "";

int fail(int code, const std::string& msg) {
  mscan::set_last_error(std::string(g_fn) + ": " + msg);
  return code;
}

int check_dims(const mamba_norm_dims_t* d) {
  if (!d) return fail(MAMBA_ERR_INVALID, "dims is NULL");
  if (d->rows < 1 || d->dim < 1) return fail(MAMBA_ERR_INVALID, "rows and dim must be >= 1");
  if (d->x < 0 || d->x > 2) return fail(MAMBA_ERR_INVALID, "x is not a mamba_dtype_t");
  if (d->y < 0 || d->y > 2) return fail(MAMBA_ERR_INVALID, "y is not a mamba_dtype_t");
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return fail(MAMBA_ERR_INVALID, "eps must be finite and > 0");
  if (d->dim > 16384) return fail(MAMBA_ERR_UNSUPPORTED, "dim must be at most 16384");
  if (d->rows > (int64_t(1) << 40) / d->dim) return fail(MAMBA_ERR_CAPACITY, "rows * dim exceeds 2^40");
  return MAMBA_OK;
}

int check_ptr(const char* name, const void* p, bool need, int align) {
  if (!p) return need ? fail(MAMBA_ERR_INVALID, std::string(name) + " is NULL") : MAMBA_OK;
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail(MAMBA_ERR_INVALID, std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
  return MAMBA_OK;
}

#define LN_TRY(expr)                 \
  do {                               \
    const int rc_ = (expr);          \
    if (rc_ != MAMBA_OK) return rc_; \
  } while (0)

#define LN_HIP(expr)                                                                                         \
  do {                                                                                                       \
    const hipError_t e_ = (expr);                                                                            \
    if (e_ != hipSuccess) return fail(MAMBA_ERR_HIP, std::string(#expr) + ": " + hipGetErrorString(e_)); \
  } while (0)

// How a row is laid over lanes: the smallest team that holds it in at most 32 (few rows: 8) elements a lane.
struct Shape {
  int team, nv;
};

Shape shape_of(const mamba_norm_dims_t& d) {
  const int e = d.x == MAMBA_F32 || d.y == MAMBA_F32 ? 4 : 8;
  const int pieces = static_cast<int>((d.dim + e - 1) / e);
  if (pieces <= 8) return {8, 1};
  if (pieces <= 16) return {16, 1};
  if (pieces <= 32) return {16, 2};
  if (pieces <= 64 * 2) return {64, (pieces + 63) / 64};
  if (pieces <= 64 * 4 && d.rows > 1024) return {64, 4};
  const int per = (pieces + 255) / 256;
  if (per * e <= 32) return {256, per == 7 ? 8 : per};
  return {1024, 16 / e};
}

// Workgroups that walk the rows: four steps each at least, if that leaves 256 of them.  At most two for each CU where a
// workgroup has one row (their registers fill a CU: 217 us the backward of 16384 x 5120, against 223 with 1024 and half
// the partial sums), four where it has several (26 us of 196608 x 64 against 30).  In the backward each has a partial row
// of d_w and d_b.
int walkers(const mamba_norm_dims_t& d) {
  const int team = shape_of(d).team, teams = team < 256 ? 256 / team : 1;
  const int64_t steps = (d.rows + teams - 1) / teams, quarter = (steps + 3) / 4, most = teams > 1 ? 1024 : 512;
  if (steps <= 256) return static_cast<int>(steps);
  return static_cast<int>(quarter < 256 ? 256 : quarter < most ? quarter : most);
}

size_t part_bytes(const mamba_norm_dims_t& d) { return static_cast<size_t>(walkers(d)) * 2 * d.dim * 4; }

template <Act X, Act Y, int TEAM, int NV, bool BWD>
hipError_t launch_team(const Args& a, hipStream_t st) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM;
  if (BWD) hipLaunchKernelGGL((norm_bwd_kernel<X, Y, TEAM, NV>), dim3(a.blocks), dim3(BLOCK), 0, st, a);
  else hipLaunchKernelGGL((norm_fwd_kernel<X, Y, TEAM, NV>), dim3(a.blocks), dim3(BLOCK), 0, st, a);
  return hipGetLastError();
}

template <Act X, Act Y, bool BWD>
hipError_t launch_xy(const Shape& s, const Args& a, hipStream_t st) {
  constexpr int E = kPiece<X, Y>;
  if (s.team == 8) return launch_team<X, Y, 8, 1, BWD>(a, st);
  if (s.team == 16) return s.nv == 1 ? launch_team<X, Y, 16, 1, BWD>(a, st) : launch_team<X, Y, 16, 2, BWD>(a, st);
  if (s.team == 64) {
    if (s.nv == 1) return launch_team<X, Y, 64, 1, BWD>(a, st);
    return s.nv == 2 ? launch_team<X, Y, 64, 2, BWD>(a, st) : launch_team<X, Y, 64, 4, BWD>(a, st);
  }
  if (s.team == 1024) return launch_team<X, Y, 1024, 16 / E, BWD>(a, st);
  switch (s.nv) {
    case 1: return launch_team<X, Y, 256, 1, BWD>(a, st);
    case 2: return launch_team<X, Y, 256, 2, BWD>(a, st);
    case 3: return launch_team<X, Y, 256, 3, BWD>(a, st);
    case 4: return launch_team<X, Y, 256, 4, BWD>(a, st);
    default: break;
  }
  if constexpr (E == 4) {
    if (s.nv == 5) return launch_team<X, Y, 256, 5, BWD>(a, st);
    if (s.nv == 6) return launch_team<X, Y, 256, 6, BWD>(a, st);
    return launch_team<X, Y, 256, 8, BWD>(a, st);
  }
  return hipErrorInvalidValue;
}

template <bool BWD>
hipError_t launch(const mamba_norm_dims_t& d, const Args& a, hipStream_t st) {
  const Shape s = shape_of(d);
  switch (d.x * 3 + d.y) {
    case 0: return launch_xy<Act::F32, Act::F32, BWD>(s, a, st);
    case 1: return launch_xy<Act::F32, Act::BF16, BWD>(s, a, st);
    case 2: return launch_xy<Act::F32, Act::F16, BWD>(s, a, st);
    case 3: return launch_xy<Act::BF16, Act::F32, BWD>(s, a, st);
    case 4: return launch_xy<Act::BF16, Act::BF16, BWD>(s, a, st);
    case 5: return launch_xy<Act::BF16, Act::F16, BWD>(s, a, st);
    case 6: return launch_xy<Act::F16, Act::F32, BWD>(s, a, st);
    case 7: return launch_xy<Act::F16, Act::BF16, BWD>(s, a, st);
    default: return launch_xy<Act::F16, Act::F16, BWD>(s, a, st);
  }
}

}  // namespace
}  // namespace lnorm

using namespace lnorm;

extern "C" {

int mamba_layernorm_workspace_bytes(const mamba_norm_dims_t* dims, size_t* bytes) {
  g_fn = "mamba_layernorm_workspace_bytes";
  LN_TRY(check_dims(dims));
  if (!bytes) return fail(MAMBA_ERR_INVALID, "bytes is NULL");
  *bytes = part_bytes(*dims);
  mscan::set_last_error("");
  return MAMBA_OK;
}

int mamba_layernorm_fwd(const mamba_norm_dims_t* dims, const void* x, const float* w, const float* b, void* y, float* mean,
                        float* rstd, void* stream) {
  g_fn = "mamba_layernorm_fwd";
  LN_TRY(check_dims(dims));
  LN_TRY(check_ptr("x", x, true, 16));
  LN_TRY(check_ptr("w", w, false, 16));
  LN_TRY(check_ptr("b", b, false, 16));
  LN_TRY(check_ptr("y", y, true, 16));
  LN_TRY(check_ptr("mean", mean, rstd != nullptr, 4));
  LN_TRY(check_ptr("rstd", rstd, mean != nullptr, 4));
  Args a{};
  a.rows = dims->rows;
  a.dim = static_cast<int>(dims->dim);
  a.eps = dims->eps;
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.blocks = walkers(*dims);
  LN_HIP(launch<false>(*dims, a, static_cast<hipStream_t>(stream)));
  mscan::set_last_error("");
  return MAMBA_OK;
}

int mamba_layernorm_bwd(const mamba_norm_dims_t* dims, const void* x, const float* w, const float* mean, const float* rstd,
                        const void* dy, const void* d_add, void* dx, float* d_w, float* d_b, void* workspace,
                        size_t workspace_bytes, void* stream) {
  g_fn = "mamba_layernorm_bwd";
  LN_TRY(check_dims(dims));
  LN_TRY(check_ptr("x", x, true, 16));
  LN_TRY(check_ptr("w", w, false, 16));
  LN_TRY(check_ptr("mean", mean, true, 4));
  LN_TRY(check_ptr("rstd", rstd, true, 4));
  LN_TRY(check_ptr("dy", dy, true, 16));
  LN_TRY(check_ptr("d_add", d_add, false, 16));
  LN_TRY(check_ptr("dx", dx, true, 16));
  LN_TRY(check_ptr("d_w", d_w, false, 16));
  LN_TRY(check_ptr("d_b", d_b, false, 16));
  const bool sums = d_w || d_b;
  LN_TRY(check_ptr("workspace", workspace, sums, 256));
  if (sums && workspace_bytes < part_bytes(*dims))
    return fail(MAMBA_ERR_CAPACITY, "workspace_bytes " + std::to_string(workspace_bytes) + " < " +
                                        std::to_string(part_bytes(*dims)) + " needed");
  Args a{};
  a.rows = dims->rows;
  a.dim = static_cast<int>(dims->dim);
  a.eps = dims->eps;
  a.x = x;
  a.w = w;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.d_add = d_add;
  a.dx = dx;
  a.d_w = d_w;
  a.d_b = d_b;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.blocks = walkers(*dims);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  LN_HIP(launch<true>(*dims, a, st));
  if (sums) {
    hipLaunchKernelGGL(norm_colsum_kernel, dim3(static_cast<unsigned>((2 * dims->dim + 15) / 16)), dim3(1024), 0, st, a);
    LN_HIP(hipGetLastError());
  }
  mscan::set_last_error("");
  return MAMBA_OK;
}

}  // extern "C"
