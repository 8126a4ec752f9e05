// norm_residual.cu -- the norms' backward with the gradient that reaches the
// norm's input past the norm: dx = the norm's own + dsum, in the same pass.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8gb.h"
#include "norm_backward.cuh"

using namespace fp8gb;

extern "C" fp8_status_t fp8_residual_norm_backward(const void *dy, int y_dtype, int64_t ld_dy, const void *x,
                                                   int64_t ld_x, const uint8_t *q, int64_t ld_q, const uint8_t *s,
                                                   int64_t ld_s, int fmt, const void *dsum, int64_t ld_dsum,
                                                   int64_t rows, int64_t cols, int kind, const float *mean,
                                                   const float *rstd, const void *weight, int w_dtype, void *dx,
                                                   int x_dtype, int64_t ld_dx, void *dweight, void *dbias,
                                                   void *workspace, int64_t workspace_bytes, void *stream)
{
    return norm_backward<true>(dy, y_dtype, ld_dy, x, ld_x, q, ld_q, s, ld_s, fmt, dsum, ld_dsum, rows, cols, kind,
                               mean, rstd, weight, w_dtype, dx, x_dtype, ld_dx, dweight, dbias, workspace,
                               workspace_bytes, stream);
}
