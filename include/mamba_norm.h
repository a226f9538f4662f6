/* C ABI of layer norm on MI355X (gfx950), forward and backward.
 *
 * Per row x of `rows` rows with `dim` elements:
 *   mean = sum(x) / dim,   rstd = 1 / sqrt(sum((x - mean)^2) / dim + eps)
 *   n = (x - mean) rstd,   y = n w + b
 * and for dy:
 *   dn = dy w,   dx = rstd (dn - mean(dn) - n mean(dn n)) + d_add
 *   d_w += sum over rows of dy n,   d_b += sum over rows of dy
 * All sums and statistics are f32 (the variance from the centred row).
 *
 * Layouts: x, dx, d_add [rows, dim] of dims->x; y, dy [rows, dim] of
 * dims->y; w, b, d_w, d_b [dim] f32; mean, rstd [rows] f32.  Rows are dense.
 *
 * Ownership and errors are those of mamba_scan.h: caller-owned device memory
 * of the current device, nothing allocated, arguments checked before anything
 * is enqueued.  x, dx, d_add, y, dy, w, b, d_w and d_b must be 16-byte
 * aligned, mean and rstd 4-byte, workspace 256-byte.  Inputs and outputs must
 * not overlap, except that dx may be d_add.  d_w and d_b accumulate (+=), in
 * an order fixed by the sizes.
 */
#ifndef MAMBA_NORM_H
#define MAMBA_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t rows;  /* >= 1 */
  int64_t dim;   /* 1 .. 16384 */
  int32_t x;     /* mamba_dtype_t of x, dx and d_add */
  int32_t y;     /* mamba_dtype_t of y and dy */
  float eps;     /* > 0 */
} mamba_norm_dims_t;

/* Bytes of device workspace the backward needs (the forward needs none). */
int mamba_layernorm_workspace_bytes(const mamba_norm_dims_t* dims, size_t* bytes);

/* Forward.  w NULL = ones, b NULL = zeros; mean, rstd (both or neither): the
 * statistics the backward reads. */
int mamba_layernorm_fwd(const mamba_norm_dims_t* dims, const void* x, const float* w, const float* b,
                        void* y, float* mean, float* rstd, void* stream);

/* Backward.  d_add (NULL = none) is added to dx: the residual path's gradient
 * of a norm in front of a block.  d_w and d_b may be NULL (not wanted). */
int mamba_layernorm_bwd(const mamba_norm_dims_t* dims, const void* x, const float* w, const float* mean,
                        const float* rstd, const void* dy, const void* d_add, void* dx, float* d_w,
                        float* d_b, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_NORM_H */
