// Layer norm, forward and backward (gfx950), and the entry points of
// include/mamba_norm.h.
//
// A team of 16, 64, 256 or 1024 lanes holds one row in registers, eight
// elements a lane and step, so a row is read once: the mean, the centred sum
// of squares and the output all come from registers.  The backward keeps the
// columns' sums for d_w and d_b in registers over the rows its workgroup
// walks, writes one partial row per workgroup, and a second launch adds the
// partials in a fixed order (no atomics).  Both are bound by HBM.
#include <cmath>
#include <string>

#include "mamba_norm.h"
#include "scan_common.h"

namespace mscan {
void set_last_error(const std::string& msg);   // abi.hip
}

namespace lnorm {

using mscan::Act;
using mscan::IO;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

// Eight elements from index i, the first n of them inside the row.  Rows of an odd length start at any element, so
// the vector accesses claim no more than the element's own alignment.
template <Act A>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float* out) {
  constexpr int S = A == Act::F32 ? 4 : 2;
  const char* src = static_cast<const char*>(p) + i * S;
  if (n >= 8) {
    uint32_t w[2 * S];
    __builtin_memcpy(w, __builtin_assume_aligned(src, S), 8 * S);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (A == Act::F32) out[e] = __builtin_bit_cast(float, w[e]);
      else out[e] = IO<A>::cvt((e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = e < n ? IO<A>::ld(p, i + e) : 0.0f;
  }
}

__device__ __forceinline__ void load8w(const float* p, int i, int n, float fill, float* out) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = fill;
  } else {
    load8<Act::F32>(p, i, n, out);
  }
}

template <Act A>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float* v) {
  constexpr int S = A == Act::F32 ? 4 : 2;
  if (n >= 8) {
    uint32_t w[2 * S];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (A == Act::F32) {
        w[e] = __builtin_bit_cast(uint32_t, v[e]);
      } else {
        uint16_t h;
        if constexpr (A == Act::BF16) h = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[e]));
        else h = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[e]));
        w[e / 2] = (e & 1) ? w[e / 2] | (static_cast<uint32_t>(h) << 16) : h;
      }
    }
    __builtin_memcpy(__builtin_assume_aligned(static_cast<char*>(p) + i * S, S), w, 8 * S);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) IO<A>::st(p, i + e, v[e]);
  }
}

// Sum over a team; every lane gets it.  `s`: one float per wave and slot.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* s) {
  constexpr int W = TEAM < 64 ? TEAM : 64;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TEAM > 64) {
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) s[wv] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TEAM / 64; ++i) v += s[i];
  }
  return v;
}

template <Act X, Act Y, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) norm_fwd_kernel(const Args p) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM, TEAMS = BLOCK / TEAM;
  __shared__ float s[2][BLOCK / 64];
  const int lane = threadIdx.x % TEAM;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TEAM;
  if (TEAM < 64 || TEAM == 64) {
    if (row >= p.rows) return;   // whole teams; no barrier below for them
  }
  float x[NV][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (lane + i * TEAM);
    load8<X>(p.x, row * p.dim + col, p.dim - col, x[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += x[i][e];
  }
  const float inv = 1.0f / static_cast<float>(p.dim), mean = team_sum<TEAM>(sum, s[0]) * inv;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int n = p.dim - 8 * (lane + i * TEAM);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[i][e] = e < n ? x[i][e] - mean : 0.0f;
      sq = fmaf(x[i][e], x[i][e], sq);
    }
  }
  const float rstd = 1.0f / sqrtf(team_sum<TEAM>(sq, s[1]) * inv + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (lane + i * TEAM), n = p.dim - col;
    if (n <= 0) continue;
    float w[8], b[8];
    load8w(p.w, col, n, 1.0f, w);
    load8w(p.b, col, n, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = fmaf(x[i][e] * rstd, w[e], b[e]);
    store8<Y>(p.y, row * p.dim + col, n, x[i]);
  }
  if (lane == 0 && p.mean) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

template <Act X, Act Y, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) norm_bwd_kernel(const Args p) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM, TEAMS = BLOCK / TEAM;
  __shared__ float s[2][2][BLOCK / 64];
  __shared__ float cols[TEAMS > 1 ? 2 * TEAM * NV * 8 : 1];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
  const float inv = 1.0f / static_cast<float>(p.dim);
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * TEAMS; row0 < p.rows; row0 += static_cast<int64_t>(gridDim.x) * TEAMS) {
    const int64_t row = row0 + team;
    const bool ok = row < p.rows;
    const float mean = ok ? p.mean[row] : 0.0f, rstd = ok ? p.rstd[row] : 0.0f;
    float n[NV][8], dn[NV][8];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (lane + i * TEAM), left = ok ? p.dim - col : 0;
      load8<X>(p.x, row * p.dim + col, left, n[i]);
      load8<Y>(p.dy, row * p.dim + col, left, dn[i]);
      float w[8];
      load8w(p.w, col, p.dim - col, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[i][e] = e < left ? (n[i][e] - mean) * rstd : 0.0f;
        db[i][e] += dn[i][e];
        dw[i][e] = fmaf(dn[i][e], n[i][e], dw[i][e]);
        dn[i][e] *= w[e];
        s1 += dn[i][e];
        s2 = fmaf(dn[i][e], n[i][e], s2);
      }
    }
    s1 = team_sum<TEAM>(s1, s[turn][0]) * inv;
    s2 = team_sum<TEAM>(s2, s[turn][1]) * inv;
    turn ^= 1;   // the next row's sums go to the other slots: a barrier lies between this row's reads and those
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (lane + i * TEAM), left = ok ? p.dim - col : 0;
      if (left <= 0) continue;
      float add[8];
      if (p.d_add) load8<X>(p.d_add, row * p.dim + col, left, add);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = rstd * (dn[i][e] - s1 - n[i][e] * s2);
        n[i][e] = p.d_add ? v + add[e] : v;
      }
      store8<X>(p.dx, row * p.dim + col, left, n[i]);
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
          for (int e = 0; e < 8; ++e) {
            float* a = cols + (i * 8 + e) * TEAM + lane;
            a[0] = (k ? a[0] : 0.0f) + dw[i][e];
            a[NV * 8 * TEAM] = (k ? a[NV * 8 * TEAM] : 0.0f) + db[i][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.dim; c += BLOCK) {
      const int l = (c / 8) % TEAM, i = (c / 8) / TEAM, e = c % 8;
      const float* a = cols + (i * 8 + e) * TEAM + l;
      part[c] = a[0];
      part[p.dim + c] = a[NV * 8 * TEAM];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (lane + i * TEAM), n = p.dim - col;
      if (n <= 0) continue;
      store8<Act::F32>(part, col, n, dw[i]);
      store8<Act::F32>(part, p.dim + col, n, db[i]);
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
  if (col < n)
    for (int r = strip; r < p.blocks; r += 64) acc += p.part[r * n + col];
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

// rows a workgroup works on at once
int teams_of(int dim) { return dim <= 256 ? 16 : dim <= 2048 ? 4 : 1; }

// Workgroups of the backward: at most 1024 (four for each CU), each with a partial row of d_w and d_b.
int bwd_blocks(const mamba_norm_dims_t& d) {
  const int64_t n = (d.rows + teams_of(static_cast<int>(d.dim)) - 1) / teams_of(static_cast<int>(d.dim));
  return static_cast<int>(n < 1024 ? n : 1024);
}

size_t part_bytes(const mamba_norm_dims_t& d) { return static_cast<size_t>(bwd_blocks(d)) * 2 * d.dim * 4; }

template <Act X, Act Y, int TEAM, int NV, bool BWD>
hipError_t launch_team(const Args& a, hipStream_t st) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM, TEAMS = BLOCK / TEAM;
  if (BWD) hipLaunchKernelGGL((norm_bwd_kernel<X, Y, TEAM, NV>), dim3(a.blocks), dim3(BLOCK), 0, st, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<X, Y, TEAM, NV>), dim3(static_cast<unsigned>((a.rows + TEAMS - 1) / TEAMS)),
                       dim3(BLOCK), 0, st, a);
  return hipGetLastError();
}

template <Act X, Act Y, bool BWD>
hipError_t launch_xy(const Args& a, hipStream_t st) {
  if (a.dim <= 128) return launch_team<X, Y, 16, 1, BWD>(a, st);
  if (a.dim <= 256) return launch_team<X, Y, 16, 2, BWD>(a, st);
  if (a.dim <= 512) return launch_team<X, Y, 64, 1, BWD>(a, st);
  if (a.dim <= 1024) return launch_team<X, Y, 64, 2, BWD>(a, st);
  if (a.dim <= 2048) return launch_team<X, Y, 64, 4, BWD>(a, st);
  if (a.dim <= 4096) return launch_team<X, Y, 256, 2, BWD>(a, st);
  if (a.dim <= 8192) return launch_team<X, Y, 256, 4, BWD>(a, st);
  return launch_team<X, Y, 1024, 2, BWD>(a, st);
}

template <bool BWD>
hipError_t launch(int x, int y, const Args& a, hipStream_t st) {
  switch (x * 3 + y) {
    case 0: return launch_xy<Act::F32, Act::F32, BWD>(a, st);
    case 1: return launch_xy<Act::F32, Act::BF16, BWD>(a, st);
    case 2: return launch_xy<Act::F32, Act::F16, BWD>(a, st);
    case 3: return launch_xy<Act::BF16, Act::F32, BWD>(a, st);
    case 4: return launch_xy<Act::BF16, Act::BF16, BWD>(a, st);
    case 5: return launch_xy<Act::BF16, Act::F16, BWD>(a, st);
    case 6: return launch_xy<Act::F16, Act::F32, BWD>(a, st);
    case 7: return launch_xy<Act::F16, Act::BF16, BWD>(a, st);
    default: return launch_xy<Act::F16, Act::F16, BWD>(a, st);
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
  const int teams = teams_of(static_cast<int>(dims->dim));
  if ((dims->rows + teams - 1) / teams >= (int64_t(1) << (dims->dim > 8192 ? 22 : 24)))   // fewer than 2^32 threads
    return fail(MAMBA_ERR_CAPACITY, "too many rows for one launch");
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
  LN_HIP(launch<false>(dims->x, dims->y, a, static_cast<hipStream_t>(stream)));
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
  a.blocks = bwd_blocks(*dims);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  LN_HIP(launch<true>(dims->x, dims->y, a, st));
  if (sums) {
    hipLaunchKernelGGL(norm_colsum_kernel, dim3(static_cast<unsigned>((2 * dims->dim + 15) / 16)), dim3(1024), 0, st, a);
    LN_HIP(hipGetLastError());
  }
  mscan::set_last_error("");
  return MAMBA_OK;
}

}  // extern "C"
