/* C ABI of the gated delta rule core on MI355X (gfx950): chunked forward and
 * backward for training and prompts, and a token-by-token step for decoding.
 *
 * What is computed, per batch row b and head h (head h reads query / key
 * group h / (heads / groups); S_t [d_v, d_k] f32, S_{-1} = h0 or zero):
 *   k^_t = k_t / sqrt(|k_t|^2 + eps),   q^_t = q_t / sqrt(|q_t|^2 + eps)
 *   g_t  = -exp(a_log_h) softplus(a_raw_t + dt_bias_h)
 *   beta_t = sigmoid(b_raw_t)
 *   u_t  = beta_t (v_t - exp(g_t) S_{t-1} k^_t)
 *   S_t  = exp(g_t) S_{t-1} + u_t k^_t^T
 *   y_t  = scale S_t q^_t
 * Longer sequences are evaluated in 64-token chunks (one unit lower
 * triangular solve per chunk, the rest products of tiles); the result equals
 * the token-by-token definition up to rounding.  Sums, states, gates and
 * their gradients are f32; a product's f32 operand is the sum of two f16
 * parts with 22 significant bits.
 *
 * Layouts (row-major, last index fastest): q, k, d_q, d_k
 * [B, T, groups, d_k]; v, y, dy, d_v [B, T, heads, d_v] (activation dtype);
 * a_raw, b_raw, d_a_raw, d_b_raw [B, T, heads] f32; a_log, dt_bias, d_a_log,
 * d_dt_bias [heads] f32; h0, h_last [B, heads, d_v, d_k] f32.
 *
 * Ownership and errors: every pointer is caller-owned device memory on the
 * current device; the library allocates nothing and enqueues on `stream` (a
 * hipStream_t, NULL for the default stream).  Arguments are checked before
 * anything is enqueued; a failure returns a mamba_status_t code and
 * mamba_last_error() names the entry point.  Inputs and outputs must not
 * overlap, except that h_last may be h0.  Activation pointers, h0 and h_last
 * must be 16-byte aligned, `saved` and `workspace` 256-byte; calls that may
 * run at the same time need buffers of their own.  Parameter gradients
 * (d_a_log, d_dt_bias) accumulate (+=); every other output is overwritten.
 * No gradient flows into h0, and none comes from h_last (truncated
 * backpropagation through time).
 *
 * A NaN or infinity in a token reaches its own chunk's outputs of that head
 * (that group's heads, for q and k) and all later ones, earlier tokens of the
 * same 64-token chunk among them.
 */
#ifndef MAMBA_GDELTA_H
#define MAMBA_GDELTA_H

#include <stddef.h>
#include <stdint.h>

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t batch;   /* >= 1; batch * heads * max(seqlen / 64, d_v / 32) below 2^23 */
  int64_t seqlen;  /* 1 .. 2^24 */
  int64_t heads;   /* >= 1, a multiple of groups; heads * d_v and groups * d_k below 2^23 */
  int64_t groups;  /* >= 1: query / key heads */
  int64_t d_k;     /* 8 .. 128, a multiple of 8 */
  int64_t d_v;     /* 8 .. 512, a multiple of 8 */
  int32_t act;     /* mamba_dtype_t of q, k, v, y and their gradients */
  float scale;     /* of y, 1e-6 .. 1e6 in size; 0 = 1 / sqrt(d_k) */
  float eps;       /* > 0: added to |q|^2 and |k|^2 */
} mamba_gdelta_dims_t;

/* Bytes of what the forward keeps for the backward (chunk states among it). */
int mamba_gdelta_saved_bytes(const mamba_gdelta_dims_t* dims, size_t* bytes);

/* Bytes of device workspace one call needs (the larger of the forward's
 * without `saved` and the backward's; one buffer of this size serves both). */
int mamba_gdelta_workspace_bytes(const mamba_gdelta_dims_t* dims, size_t* bytes);

/* A forward without `saved` takes up to this many tokens one by one, as
 * mamba_gdelta_step does, and needs no `workspace` for them. */
#define MAMBA_GDELTA_STEP_TOKENS 8

/* Forward.  h0: f32 or NULL (= zeros); h_last: f32 or NULL.  `saved` is what
 * the backward needs, NULL when none follows; without it `workspace` is used
 * (else it may be NULL). */
int mamba_gdelta_fwd(const mamba_gdelta_dims_t* dims, const void* q, const void* k, const void* v,
                     const float* a_raw, const float* b_raw, const float* a_log, const float* dt_bias,
                     const float* h0, void* y, float* h_last, void* saved, size_t saved_bytes,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Backward of sum(dy * y): every input's gradient.  `saved` is what the
 * forward wrote for the same inputs; has_h0 says whether it had an h0 (the
 * first token's decay has a gradient only then). */
int mamba_gdelta_bwd(const mamba_gdelta_dims_t* dims, const void* q, const void* k, const void* v,
                     const float* a_raw, const float* b_raw, const float* a_log, const float* dt_bias,
                     int32_t has_h0, const void* saved, size_t saved_bytes, const void* dy, void* d_q,
                     void* d_k, void* d_v, float* d_a_raw, float* d_b_raw, float* d_a_log,
                     float* d_dt_bias, void* workspace, size_t workspace_bytes, void* stream);

/* The forward token by token with the state in registers, for the tokens of
 * a decoding step (any seqlen; made for a few).  `state` in and out, f32, is
 * updated in place.  Needs no workspace. */
int mamba_gdelta_step(const mamba_gdelta_dims_t* dims, const void* q, const void* k, const void* v,
                      const float* a_raw, const float* b_raw, const float* a_log, const float* dt_bias,
                      float* state, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_GDELTA_H */
