// ckpt.cu -- 8-bit activation checkpoints: store and restore of any matrix,
// the SwiGLU forward that stores its gate|up input in the same read, and the
// SwiGLU backward that reads it.  The block rule is ckpt.cuh's.
//
// All four are one pass over their tensors and bounded by HBM.
//
// One warp works on one block of 32 columns, a lane per element: every
// alignment, row stride and width is the same code, the block maximum is five
// shuffles, and a warp's accesses are consecutive.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"

namespace fp8gb {

constexpr int CK_THREADS = 256;
constexpr int CK_WARPS = CK_THREADS / 32;

struct CkArgs {
    void *x;  // store: input; restore: output
    int64_t ld_x;
    uint8_t *q, *s;
    int64_t ld_q, ld_s;
    int64_t rows, cols;
    int parts, fmt;
};

struct SwArgs {
    const __nv_bfloat16 *gate_up, *dh;
    int64_t ld, ld_dh;
    uint8_t *q, *s;
    int64_t ld_q, ld_s;
    int64_t rows, F;
    int fmt;
    __nv_bfloat16 *h, *d;
    int64_t ld_h, ld_d;
};

template <typename T>
__global__ void __launch_bounds__(CK_THREADS) checkpoint_kernel(CkArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t nb = ckpt_width(a.cols) / FP8_MX_BLOCK;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.ld_x;
        for (int p = 0; p < a.parts; p++)
            for (int64_t b = warp; b < nb; b += CK_WARPS) {
                const int64_t c = b * FP8_MX_BLOCK + lane;
                const float v = c < a.cols ? to_f32<T>(x[p * a.cols + c]) : 0.0f;
                ckpt_store_lane(v, a.fmt, a.q + r * a.ld_q + (p * nb + b) * FP8_MX_BLOCK,
                                a.s + r * a.ld_s + p * nb + b, lane);
            }
    }
}

template <typename T>
__global__ void __launch_bounds__(CK_THREADS) restore_kernel(CkArgs a)
{
    const int64_t nb = ckpt_width(a.cols) / FP8_MX_BLOCK;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        T *x = static_cast<T *>(a.x) + r * a.ld_x;
        for (int p = 0; p < a.parts; p++)
            for (int64_t c = threadIdx.x; c < a.cols; c += CK_THREADS)
                x[p * a.cols + c] = from_f32<T>(
                    ckpt_load_one(a.q + r * a.ld_q + p * nb * FP8_MX_BLOCK, a.s + r * a.ld_s + p * nb, c, a.fmt));
    }
}

__global__ void __launch_bounds__(CK_THREADS) swiglu_checkpoint_kernel(SwArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t nb = ckpt_width(a.F) / FP8_MX_BLOCK;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const __nv_bfloat16 *x = a.gate_up + r * a.ld;
        uint8_t *q = a.q + r * a.ld_q, *s = a.s + r * a.ld_s;
        for (int64_t b = warp; b < nb; b += CK_WARPS) {
            const int64_t c = b * FP8_MX_BLOCK + lane;
            const float g = c < a.F ? to_f32(x[c]) : 0.0f, u = c < a.F ? to_f32(x[a.F + c]) : 0.0f;
            if (c < a.F) a.h[r * a.ld_h + c] = from_f32<__nv_bfloat16>(swiglu1(g, u));
            ckpt_store_lane(g, a.fmt, q + b * FP8_MX_BLOCK, s + b, lane);
            ckpt_store_lane(u, a.fmt, q + (nb + b) * FP8_MX_BLOCK, s + nb + b, lane);
        }
    }
}

__global__ void __launch_bounds__(CK_THREADS) swiglu_backward_kernel(SwArgs a)
{
    const int64_t nb = ckpt_width(a.F) / FP8_MX_BLOCK;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint8_t *q = a.q + r * a.ld_q, *s = a.s + r * a.ld_s;
        for (int64_t c = threadIdx.x; c < a.F; c += CK_THREADS) {
            float g, u;
            if (a.gate_up) {
                g = to_f32(a.gate_up[r * a.ld + c]);
                u = to_f32(a.gate_up[r * a.ld + a.F + c]);
            } else {
                g = ckpt_load_one(q, s, c, a.fmt);
                u = ckpt_load_one(q + nb * FP8_MX_BLOCK, s + nb, c, a.fmt);
            }
            float dg, du;
            swiglu_grad1(g, u, to_f32(a.dh[r * a.ld_dh + c]), dg, du);
            a.d[r * a.ld_d + c] = from_f32<__nv_bfloat16>(dg);
            a.d[r * a.ld_d + a.F + c] = from_f32<__nv_bfloat16>(du);
            if (a.h) a.h[r * a.ld_h + c] = from_f32<__nv_bfloat16>(swiglu1(g, u));
        }
    }
}

// Blocks of a grid that covers `rows` rows, eight resident per SM.
static unsigned row_grid(int64_t rows)
{
    const int64_t cap = (int64_t)num_sms() * 8;
    return (unsigned)(rows < cap ? rows : cap);
}

static fp8_status_t check_format(int fmt)
{
    if (fmt == FP8_E4M3FNUZ || fmt == FP8_E5M2FNUZ) return FP8_ERR_UNSUPPORTED;
    return fmt == FP8_E4M3FN || fmt == FP8_E5M2 ? FP8_OK : FP8_ERR_INVALID_ARG;
}

// Codes and scales of a checkpoint with `parts` parts of `cols` columns.
static fp8_status_t check_codes(const void *q, int64_t ld_q, const void *s, int64_t ld_s, int64_t cols, int64_t parts)
{
    const int64_t w = parts * ckpt_width(cols);
    if (!q || !s || ld_q < w || ld_s < w / FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    return ld_q % FP8_MX_BLOCK != 0 || !aligned(q, FP8_MX_BLOCK) ? FP8_ERR_ALIGNMENT : FP8_OK;
}

static fp8_status_t check_ck(const CkArgs &a, int dtype)
{
    if (a.rows < 0 || a.cols < 1 || a.parts < 1 || a.rows > INT32_MAX || a.cols > INT32_MAX / a.parts - FP8_MX_BLOCK)
        return FP8_ERR_INVALID_ARG;
    if (dtype < FP8_DTYPE_BF16 || dtype > FP8_DTYPE_F32) return FP8_ERR_INVALID_ARG;
    const fp8_status_t f = check_format(a.fmt);
    if (f != FP8_OK || a.rows == 0) return f;
    if (!a.x || a.ld_x < a.parts * a.cols) return FP8_ERR_INVALID_ARG;
    if (!aligned(a.x, dtype == FP8_DTYPE_F32 ? 4 : 2)) return FP8_ERR_ALIGNMENT;
    return check_codes(a.q, a.ld_q, a.s, a.ld_s, a.cols, a.parts);
}

static fp8_status_t check_bf16(const void *p, int64_t ld, int64_t cols)
{
    if (!p || ld < cols) return FP8_ERR_INVALID_ARG;
    return aligned(p, 2) ? FP8_OK : FP8_ERR_ALIGNMENT;
}

}  // namespace fp8gb

using namespace fp8gb;

extern "C" fp8_status_t fp8_checkpoint(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, int parts,
                                       int fmt, uint8_t *q, int64_t ld_q, uint8_t *s, int64_t ld_s, void *stream)
{
    CkArgs a{const_cast<void *>(x), ld_x, q, s, ld_q, ld_s, rows, cols, parts, fmt};
    const fp8_status_t rc = check_ck(a, dtype);
    if (rc != FP8_OK || rows == 0) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = row_grid(rows);
    if (dtype == FP8_DTYPE_BF16) checkpoint_kernel<__nv_bfloat16><<<grid, CK_THREADS, 0, st>>>(a);
    else if (dtype == FP8_DTYPE_F16) checkpoint_kernel<__half><<<grid, CK_THREADS, 0, st>>>(a);
    else checkpoint_kernel<float><<<grid, CK_THREADS, 0, st>>>(a);
    return check_launch();
}

extern "C" fp8_status_t fp8_checkpoint_restore(const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                               int64_t rows, int64_t cols, int parts, void *x, int dtype,
                                               int64_t ld_x, void *stream)
{
    CkArgs a{x, ld_x, const_cast<uint8_t *>(q), const_cast<uint8_t *>(s), ld_q, ld_s, rows, cols, parts, fmt};
    const fp8_status_t rc = check_ck(a, dtype);
    if (rc != FP8_OK || rows == 0) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = row_grid(rows);
    if (dtype == FP8_DTYPE_BF16) restore_kernel<__nv_bfloat16><<<grid, CK_THREADS, 0, st>>>(a);
    else if (dtype == FP8_DTYPE_F16) restore_kernel<__half><<<grid, CK_THREADS, 0, st>>>(a);
    else restore_kernel<float><<<grid, CK_THREADS, 0, st>>>(a);
    return check_launch();
}

extern "C" fp8_status_t fp8_swiglu_checkpoint(const void *gate_up_bf16, int64_t rows, int64_t F, int64_t ld, int fmt,
                                              void *h_bf16, int64_t ld_h, uint8_t *q, int64_t ld_q, uint8_t *s,
                                              int64_t ld_s, void *stream)
{
    if (rows < 0 || F < 1 || rows > INT32_MAX || F > INT32_MAX / 2 - FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    fp8_status_t rc = check_format(fmt);
    if (rc != FP8_OK || rows == 0) return rc;
    if ((rc = check_bf16(gate_up_bf16, ld, 2 * F)) != FP8_OK) return rc;
    if ((rc = check_bf16(h_bf16, ld_h, F)) != FP8_OK) return rc;
    if ((rc = check_codes(q, ld_q, s, ld_s, F, 2)) != FP8_OK) return rc;
    SwArgs a{};
    a.gate_up = static_cast<const __nv_bfloat16 *>(gate_up_bf16);
    a.ld = ld;
    a.rows = rows;
    a.F = F;
    a.fmt = fmt;
    a.h = static_cast<__nv_bfloat16 *>(h_bf16);
    a.ld_h = ld_h;
    a.q = q;
    a.s = s;
    a.ld_q = ld_q;
    a.ld_s = ld_s;
    swiglu_checkpoint_kernel<<<row_grid(rows), CK_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return check_launch();
}

extern "C" fp8_status_t fp8_swiglu_backward(const void *dh_bf16, int64_t ld_dh, const void *gate_up_bf16, int64_t ld,
                                            const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                            int64_t rows, int64_t F, void *d_gate_up_bf16, int64_t ld_d,
                                            void *h_bf16, int64_t ld_h, void *stream)
{
    if (rows < 0 || F < 1 || rows > INT32_MAX || F > INT32_MAX / 2 - FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    if (gate_up_bf16 && (q || s)) return FP8_ERR_INVALID_ARG;
    fp8_status_t rc = gate_up_bf16 ? FP8_OK : check_format(fmt);
    if (rc != FP8_OK || rows == 0) return rc;
    if ((rc = check_bf16(dh_bf16, ld_dh, F)) != FP8_OK) return rc;
    if ((rc = check_bf16(d_gate_up_bf16, ld_d, 2 * F)) != FP8_OK) return rc;
    if (h_bf16 && (rc = check_bf16(h_bf16, ld_h, F)) != FP8_OK) return rc;
    rc = gate_up_bf16 ? check_bf16(gate_up_bf16, ld, 2 * F) : check_codes(q, ld_q, s, ld_s, F, 2);
    if (rc != FP8_OK) return rc;
    SwArgs a{};
    a.dh = static_cast<const __nv_bfloat16 *>(dh_bf16);
    a.ld_dh = ld_dh;
    a.gate_up = static_cast<const __nv_bfloat16 *>(gate_up_bf16);
    a.ld = ld;
    a.q = const_cast<uint8_t *>(q);
    a.s = const_cast<uint8_t *>(s);
    a.ld_q = ld_q;
    a.ld_s = ld_s;
    a.fmt = fmt;
    a.rows = rows;
    a.F = F;
    a.d = static_cast<__nv_bfloat16 *>(d_gate_up_bf16);
    a.ld_d = ld_d;
    a.h = static_cast<__nv_bfloat16 *>(h_bf16);
    a.ld_h = ld_h;
    swiglu_backward_kernel<<<row_grid(rows), CK_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return check_launch();
}
