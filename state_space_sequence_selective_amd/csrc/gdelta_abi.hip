// Entry points of include/mamba_gdelta.h: argument checks, buffer layout, launches.
#include <cmath>
#include <string>

#include "gdelta_launch.h"
#include "mamba_gdelta.h"

namespace mscan {
void set_last_error(const std::string& msg);   // abi.hip
}

namespace gdelta {
namespace {

// Sequences up to this long take the token-by-token kernel when nothing is kept for a backward pass: 8 tokens of 16 heads
// of 128 x 128 take 18 us in it against 21 in chunks, 34 against 39 with 16 sequences, 398 against 511 with 256 (15
// against 17, 23 against 28 and 246 against 305 with 24 heads of 64 x 64); 12 tokens 26 against 21, 49 against 39, 560
// against 512.
constexpr int64_t kStepMaxT = MAMBA_GDELTA_STEP_TOKENS;

thread_local const char* g_fn = "";

int fail(int code, const std::string& msg) {
  mscan::set_last_error(std::string(g_fn) + ": " + msg);
  return code;
}

int check_dims(const mamba_gdelta_dims_t* dd, Dims* d, Act* act) {
  if (!dd) return fail(MAMBA_ERR_INVALID, "dims is NULL");
  if (dd->batch < 1 || dd->seqlen < 1 || dd->heads < 1 || dd->groups < 1)
    return fail(MAMBA_ERR_INVALID, "batch, seqlen, heads and groups must be >= 1");
  if (dd->heads % dd->groups != 0) return fail(MAMBA_ERR_INVALID, "heads must be a multiple of groups");
  if (dd->act < 0 || dd->act > 2) return fail(MAMBA_ERR_INVALID, "act is not a mamba_dtype_t");
  if (dd->d_k < 1 || dd->d_v < 1) return fail(MAMBA_ERR_INVALID, "d_k and d_v must be >= 1");
  if (dd->d_k % 8 != 0 || dd->d_k > 128) return fail(MAMBA_ERR_UNSUPPORTED, "d_k must be a multiple of 8, at most 128");
  if (dd->d_v % 8 != 0 || dd->d_v > 512) return fail(MAMBA_ERR_UNSUPPORTED, "d_v must be a multiple of 8, at most 512");
  if (dd->scale != 0.0f && !(std::fabs(dd->scale) >= 1e-6f && std::fabs(dd->scale) <= 1e6f))
    return fail(MAMBA_ERR_INVALID, "scale must be 0 (the default) or of a size between 1e-6 and 1e6");
  if (!(dd->eps > 0.0f) || !std::isfinite(dd->eps)) return fail(MAMBA_ERR_INVALID, "eps must be finite and > 0");
  if (dd->seqlen > (int64_t(1) << 24)) return fail(MAMBA_ERR_CAPACITY, "seqlen must be at most 2^24");
  if (dd->batch > (int64_t(1) << 24) || dd->heads > (int64_t(1) << 16))
    return fail(MAMBA_ERR_CAPACITY, "batch must be at most 2^24, heads at most 2^16");
  if (dd->heads * dd->d_v >= (int64_t(1) << 23) || dd->groups * dd->d_k >= (int64_t(1) << 23))   // 64 rows in 32-bit bytes
    return fail(MAMBA_ERR_CAPACITY, "heads * d_v and groups * d_k must be below 2^23");
  const int64_t nc = (dd->seqlen + kC - 1) / kC, per = (dd->d_v + 31) / 32;
  if (dd->batch * dd->heads * (nc > per ? nc : per) >= (int64_t(1) << 23))   // workgroups of at most 512: fewer than 2^32 threads
    return fail(MAMBA_ERR_CAPACITY, "batch * heads * max(seqlen / 64, d_v / 32) must be below 2^23");
  d->B = dd->batch;
  d->T = dd->seqlen;
  d->H = dd->heads;
  d->G = dd->groups;
  d->nc = nc;
  d->K = static_cast<int>(dd->d_k);
  d->V = static_cast<int>(dd->d_v);
  d->VP = (d->V + 31) / 32 * 32;
  d->scale = dd->scale != 0.0f ? dd->scale : 1.0f / std::sqrt(static_cast<float>(dd->d_k));
  d->eps = dd->eps;
  int e;
  std::frexp(d->scale, &e);
  d->pscale = std::ldexp(1.0f, 12 - e);
  *act = static_cast<Act>(dd->act);
  return MAMBA_OK;
}

int check_ptr(const char* name, const void* p, bool need, int align) {
  if (!p) return need ? fail(MAMBA_ERR_INVALID, std::string(name) + " is NULL") : MAMBA_OK;
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail(MAMBA_ERR_INVALID, std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
  return MAMBA_OK;
}

#define GD_TRY(expr)                 \
  do {                               \
    const int rc_ = (expr);          \
    if (rc_ != MAMBA_OK) return rc_; \
  } while (0)

#define GD_HIP(expr)                                                                                         \
  do {                                                                                                       \
    const hipError_t e_ = (expr);                                                                            \
    if (e_ != hipSuccess) return fail(MAMBA_ERR_HIP, std::string(#expr) + ": " + hipGetErrorString(e_)); \
  } while (0)

struct Taker {
  char* base;
  size_t off = 0;
  template <class P>
  void take(P*& p, size_t bytes) {
    p = base ? reinterpret_cast<P*>(base + off) : nullptr;
    off += (bytes + 255) / 256 * 256;
  }
};

// k and q as operands, the chunks' scalars, P and T; and what only a backward pass reads
size_t layout_kept(const Dims& d, Act act, bool save, char* base, Kept* w) {
  const size_t chunks = d.B * d.H * d.nc, groups = d.B * d.G * d.nc, kp = d.K <= 64 ? 64 : 128;
  const size_t planes = act == Act::F32 ? 2 : 1, fam = groups * planes * (kp / 8) * kFrag * 2, tri = chunks * 6 * kFrag * 2;
  Taker t{base};
  *w = Kept{};
  t.take(w->gsc, groups * kGroupSc * kC * 4);
  t.take(w->KF, fam);
  t.take(w->KT, fam);
  t.take(w->QF, fam);
  t.take(w->hsc, chunks * kHeadSc * kC * 4);
  t.take(w->G, chunks * kC * 8);
  t.take(w->P, (act == Act::BF16 ? 1 : 2) * tri);
  t.take(w->T, 2 * tri);
  t.take(w->vmax, chunks * 4);
  t.take(w->sv, d.B * d.H * 4);
  if (save) {
    t.take(w->QT, fam);
    t.take(w->PT, 2 * tri);
    t.take(w->TT, 2 * tri);
    t.take(w->S, chunks * kp * d.VP * 4);
    t.take(w->U, chunks * kC * d.VP * 4);
  }
  return t.off;
}

// [dymax | so | part | DS | DU]
size_t layout_bwd(const Dims& d, char* base, BwdArgs* a) {
  const size_t chunks = d.B * d.H * d.nc, kp = d.K <= 64 ? 64 : 128;
  Taker t{base};
  t.take(a->dymax, chunks * 4);
  t.take(a->so, d.B * d.H * 4);
  t.take(a->part, chunks * 2 * 4);
  t.take(a->DS, chunks * kp * d.VP * 4);
  t.take(a->DU, chunks * kC * d.VP * 4);
  return t.off;
}

int need(const char* what, size_t have, size_t want) {
  if (have >= want) return MAMBA_OK;
  return fail(MAMBA_ERR_CAPACITY, std::string(what) + " " + std::to_string(have) + " < " + std::to_string(want) + " needed");
}

int check_inputs(const void* q, const void* k, const void* v, const float* a_raw, const float* b_raw, const float* a_log,
                 const float* dt_bias) {
  GD_TRY(check_ptr("q", q, true, 16));
  GD_TRY(check_ptr("k", k, true, 16));
  GD_TRY(check_ptr("v", v, true, 16));
  GD_TRY(check_ptr("a_raw", a_raw, true, 4));
  GD_TRY(check_ptr("b_raw", b_raw, true, 4));
  GD_TRY(check_ptr("a_log", a_log, true, 4));
  return check_ptr("dt_bias", dt_bias, true, 4);
}

}  // namespace
}  // namespace gdelta

using namespace gdelta;

extern "C" {

int mamba_gdelta_saved_bytes(const mamba_gdelta_dims_t* dims, size_t* bytes) {
  g_fn = "mamba_gdelta_saved_bytes";
  Dims d;
  Act act;
  GD_TRY(check_dims(dims, &d, &act));
  if (!bytes) return fail(MAMBA_ERR_INVALID, "bytes is NULL");
  Kept w;
  *bytes = layout_kept(d, act, true, nullptr, &w);
  mscan::set_last_error("");
  return MAMBA_OK;
}

int mamba_gdelta_workspace_bytes(const mamba_gdelta_dims_t* dims, size_t* bytes) {
  g_fn = "mamba_gdelta_workspace_bytes";
  Dims d;
  Act act;
  GD_TRY(check_dims(dims, &d, &act));
  if (!bytes) return fail(MAMBA_ERR_INVALID, "bytes is NULL");
  Kept w;
  BwdArgs a{};
  const size_t f = layout_kept(d, act, false, nullptr, &w), b = layout_bwd(d, nullptr, &a);
  *bytes = f > b ? f : b;
  mscan::set_last_error("");
  return MAMBA_OK;
}

int mamba_gdelta_fwd(const mamba_gdelta_dims_t* dims, const void* q, const void* k, const void* v, const float* a_raw,
                     const float* b_raw, const float* a_log, const float* dt_bias, const float* h0, void* y,
                     float* h_last, void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes,
                     void* stream) {
  g_fn = "mamba_gdelta_fwd";
  FwdArgs a{};
  Act act;
  GD_TRY(check_dims(dims, &a.d, &act));
  GD_TRY(check_inputs(q, k, v, a_raw, b_raw, a_log, dt_bias));
  GD_TRY(check_ptr("h0", h0, false, 16));
  GD_TRY(check_ptr("y", y, true, 16));
  GD_TRY(check_ptr("h_last", h_last, false, 16));
  GD_TRY(check_ptr("saved", saved, false, 256));
  GD_TRY(check_ptr("workspace", workspace, !saved && a.d.T > kStepMaxT, 256));
  a.q = q;
  a.k = k;
  a.v = v;
  a.a_raw = a_raw;
  a.b_raw = b_raw;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.h0 = h0;
  a.y = y;
  a.h_last = h_last;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (saved) {
    GD_TRY(need("saved_bytes", saved_bytes, layout_kept(a.d, act, true, static_cast<char*>(saved), &a.w)));
    GD_HIP(launch_fwd(act, a, true, st));
  } else if (a.d.T <= kStepMaxT) {
    GD_HIP(launch_step(act, a, st));
  } else {
    GD_TRY(need("workspace_bytes", workspace_bytes, layout_kept(a.d, act, false, static_cast<char*>(workspace), &a.w)));
    GD_HIP(launch_fwd(act, a, false, st));
  }
  mscan::set_last_error("");
  return MAMBA_OK;
}

int mamba_gdelta_bwd(const mamba_gdelta_dims_t* dims, const void* q, const void* k, const void* v, const float* a_raw,
                     const float* b_raw, const float* a_log, const float* dt_bias, int32_t has_h0, const void* saved,
                     size_t saved_bytes, const void* dy, void* d_q, void* d_k, void* d_v, float* d_a_raw,
                     float* d_b_raw, float* d_a_log, float* d_dt_bias, void* workspace, size_t workspace_bytes,
                     void* stream) {
  g_fn = "mamba_gdelta_bwd";
  BwdArgs a{};
  Act act;
  GD_TRY(check_dims(dims, &a.d, &act));
  GD_TRY(check_inputs(q, k, v, a_raw, b_raw, a_log, dt_bias));
  GD_TRY(check_ptr("saved", saved, true, 256));
  GD_TRY(check_ptr("dy", dy, true, 16));
  GD_TRY(check_ptr("d_q", d_q, true, 16));
  GD_TRY(check_ptr("d_k", d_k, true, 16));
  GD_TRY(check_ptr("d_v", d_v, true, 16));
  GD_TRY(check_ptr("d_a_raw", d_a_raw, true, 4));
  GD_TRY(check_ptr("d_b_raw", d_b_raw, true, 4));
  GD_TRY(check_ptr("d_a_log", d_a_log, true, 4));
  GD_TRY(check_ptr("d_dt_bias", d_dt_bias, true, 4));
  GD_TRY(check_ptr("workspace", workspace, true, 256));
  GD_TRY(need("saved_bytes", saved_bytes,
              layout_kept(a.d, act, true, const_cast<char*>(static_cast<const char*>(saved)), &a.w)));
  GD_TRY(need("workspace_bytes", workspace_bytes, layout_bwd(a.d, static_cast<char*>(workspace), &a)));
  a.dy = dy;
  a.a_raw = a_raw;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.has_h0 = has_h0 != 0;
  a.d_q = d_q;
  a.d_k = d_k;
  a.d_v = d_v;
  a.d_a_raw = d_a_raw;
  a.d_b_raw = d_b_raw;
  a.d_a_log = d_a_log;
  a.d_dt_bias = d_dt_bias;
  GD_HIP(launch_bwd(act, a, static_cast<hipStream_t>(stream)));
  mscan::set_last_error("");
  return MAMBA_OK;
}

int mamba_gdelta_step(const mamba_gdelta_dims_t* dims, const void* q, const void* k, const void* v, const float* a_raw,
                      const float* b_raw, const float* a_log, const float* dt_bias, float* state, void* y, void* stream) {
  g_fn = "mamba_gdelta_step";
  FwdArgs a{};
  Act act;
  GD_TRY(check_dims(dims, &a.d, &act));
  GD_TRY(check_inputs(q, k, v, a_raw, b_raw, a_log, dt_bias));
  GD_TRY(check_ptr("state", state, true, 16));
  GD_TRY(check_ptr("y", y, true, 16));
  a.q = q;
  a.k = k;
  a.v = v;
  a.a_raw = a_raw;
  a.b_raw = b_raw;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.h0 = state;
  a.h_last = state;
  a.y = y;
  GD_HIP(launch_step(act, a, static_cast<hipStream_t>(stream)));
  mscan::set_last_error("");
  return MAMBA_OK;
}

}  // extern "C"
