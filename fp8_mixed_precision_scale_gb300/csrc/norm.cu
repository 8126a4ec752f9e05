// norm.cu -- layer norm and RMS norm, forward and backward, with the 8-bit
// checkpoint of the normalized rows that the backward can read instead of x.
//
//   mu = sum x / n (0 for RMS),  r = 1 / sqrt(sum (x - mu)^2 / n + eps)
//   xh = (x - mu) r,  y = xh w + b
//   g = dy w,  c1 = sum g / n (0 for RMS),  c2 = sum g xh / n
//   dx = r (g - c1 - xh c2),  dw = sum over rows of dy xh,  db = of dy
//
// The variance is the sum of squared differences from the mean, never
// E[x^2] - mu^2, which cancels for rows far from zero.  Every sum, statistic
// and product is fp32; y, dx, dw and db are rounded once.  The checkpoint
// keeps xh, not x: its 8 bits then resolve xh itself however large the mean
// is against the spread, and the backward needs no mean.
//
// The row kernels give a block one row at a time and sweep it once per sum
// (the later sweeps hit L1/L2); dw and db are column sums over row slices
// into the caller's workspace, added in a fixed order by a second kernel: no
// atomics, the same bits every time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"

namespace fp8gb {

constexpr int NM_THREADS = 256;
constexpr int NM_WARPS = NM_THREADS / 32;
constexpr int NM_COLS = 32;   // columns of a column-sum block
constexpr int NM_LANES = NM_THREADS / NM_COLS;  // its row lanes

struct NormArgs {
    const void *x, *dy;  // x: forward input; backward: NULL when the checkpoint is read
    int64_t ld_x, ld_dy;
    void *out;  // y / dx
    int64_t ld_out;
    uint8_t *q, *s;
    int64_t ld_q, ld_s;
    int fmt;
    int64_t rows, cols;
    int rms;
    float eps;
    const void *weight, *bias;
    int w_dtype;
    float *mean_out, *rstd_out;
    const float *mean, *rstd;
    float *part;  // [splits][2][cols] dw and db sums of row slices
    int splits;
    void *dweight, *dbias;
};

// Element i of a parameter vector; NULL gives `absent`.
__device__ __forceinline__ float param(const void *p, int dtype, int64_t i, float absent)
{
    if (!p) return absent;
    if (dtype == FP8_DTYPE_F32) return static_cast<const float *>(p)[i];
    if (dtype == FP8_DTYPE_F16) return to_f32(static_cast<const __half *>(p)[i]);
    return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void set_param(void *p, int dtype, int64_t i, float v)
{
    if (!p) return;
    if (dtype == FP8_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == FP8_DTYPE_F16) static_cast<__half *>(p)[i] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = from_f32<__nv_bfloat16>(v);
}

// Sum of a pair over the block; every thread gets it.
__device__ __forceinline__ float2 block_sum(float a, float b)
{
    __shared__ float2 part[NM_WARPS];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, d);
        b += __shfl_xor_sync(0xffffffffu, b, d);
    }
    __syncthreads();  // the previous call's readers are done
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = part[0];
#pragma unroll
    for (int w = 1; w < NM_WARPS; w++) {
        t.x += part[w].x;
        t.y += part[w].y;
    }
    return t;
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(NM_THREADS) norm_forward_kernel(NormArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float n = (float)a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + r * a.ld_x;
        TY *y = static_cast<TY *>(a.out) + r * a.ld_out;
        float mean = 0.0f;
        if (!a.rms) {
            float t = 0.0f;
            for (int64_t c = threadIdx.x; c < a.cols; c += NM_THREADS) t += to_f32(x[c]);
            mean = block_sum(t, 0.0f).x / n;
        }
        float t = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += NM_THREADS) {
            const float d = to_f32(x[c]) - mean;
            t = fmaf(d, d, t);
        }
        const float rstd = 1.0f / sqrtf(block_sum(t, 0.0f).x / n + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean_out) a.mean_out[r] = mean;
            if (a.rstd_out) a.rstd_out[r] = rstd;
        }
        for (int64_t b = warp; b * 32 < a.cols; b += NM_WARPS) {
            const int64_t c = b * 32 + lane;
            float xh = 0.0f;
            if (c < a.cols) {
                xh = (to_f32(x[c]) - mean) * rstd;
                y[c] = from_f32<TY>(
                    fmaf(xh, param(a.weight, a.w_dtype, c, 1.0f), param(a.bias, a.w_dtype, c, 0.0f)));
            }
            if (a.q) ckpt_store_lane(xh, a.fmt, a.q + r * a.ld_q + b * 32, a.s + r * a.ld_s + b, lane);
        }
    }
}

// xh of one element, from x or from the checkpoint.
template <typename TX>
__device__ __forceinline__ float norm_xhat(const NormArgs &a, int64_t r, int64_t c, float mean, float rstd)
{
    if (a.x) return (to_f32(static_cast<const TX *>(a.x)[r * a.ld_x + c]) - mean) * rstd;
    return ckpt_load_one(a.q + r * a.ld_q, a.s + r * a.ld_s, c, a.fmt);
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(NM_THREADS) norm_dx_kernel(NormArgs a)
{
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const TY *dy = static_cast<const TY *>(a.dy) + r * a.ld_dy;
        TX *dx = static_cast<TX *>(a.out) + r * a.ld_out;
        const float rstd = a.rstd[r], mean = a.x && !a.rms ? a.mean[r] : 0.0f;
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += NM_THREADS) {
            const float g = to_f32(dy[c]) * param(a.weight, a.w_dtype, c, 1.0f);
            s1 += g;
            s2 = fmaf(g, norm_xhat<TX>(a, r, c, mean, rstd), s2);
        }
        const float2 t = block_sum(s1, s2);
        const float c1 = a.rms ? 0.0f : t.x / (float)a.cols, c2 = t.y / (float)a.cols;
        for (int64_t c = threadIdx.x; c < a.cols; c += NM_THREADS) {
            const float g = to_f32(dy[c]) * param(a.weight, a.w_dtype, c, 1.0f);
            dx[c] = from_f32<TX>(rstd * (g - c1 - norm_xhat<TX>(a, r, c, mean, rstd) * c2));
        }
    }
}

// Column sums over the rows of slice blockIdx.y (rows blockIdx.y, + splits, ...
// in groups of NM_LANES).
template <typename TX, typename TY>
__global__ void __launch_bounds__(NM_THREADS) norm_dw_kernel(NormArgs a)
{
    __shared__ float2 part[NM_LANES][NM_COLS];
    const int tc = threadIdx.x % NM_COLS, tr = threadIdx.x / NM_COLS;
    const int64_t c = (int64_t)blockIdx.x * NM_COLS + tc;
    float dw = 0.0f, db = 0.0f;
    if (c < a.cols)
        for (int64_t r = (int64_t)blockIdx.y * NM_LANES + tr; r < a.rows; r += (int64_t)a.splits * NM_LANES) {
            const float dy = to_f32(static_cast<const TY *>(a.dy)[r * a.ld_dy + c]);
            const float mean = a.x && !a.rms ? a.mean[r] : 0.0f;
            dw = fmaf(dy, norm_xhat<TX>(a, r, c, mean, a.x ? a.rstd[r] : 1.0f), dw);
            db += dy;
        }
    part[tr][tc] = make_float2(dw, db);
    __syncthreads();
    if (tr == 0 && c < a.cols) {
        for (int i = 1; i < NM_LANES; i++) {
            dw += part[i][tc].x;
            db += part[i][tc].y;
        }
        a.part[((int64_t)blockIdx.y * 2) * a.cols + c] = dw;
        a.part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = db;
    }
}

__global__ void __launch_bounds__(NM_THREADS) norm_dw_sum_kernel(NormArgs a)
{
    const int64_t c = (int64_t)blockIdx.x * NM_THREADS + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (int i = 0; i < a.splits; i++) {
        dw += a.part[((int64_t)i * 2) * a.cols + c];
        db += a.part[((int64_t)i * 2 + 1) * a.cols + c];
    }
    set_param(a.dweight, a.w_dtype, c, dw);
    set_param(a.dbias, a.w_dtype, c, db);
}

// Row slices of the column sums: enough blocks for eight per SM, at least
// NM_LANES rows each.
static int norm_splits(int64_t rows, int64_t cols)
{
    const int64_t tiles = (cols + NM_COLS - 1) / NM_COLS;
    int64_t want = ((int64_t)num_sms() * 8 + tiles - 1) / tiles;
    const int64_t most = (rows + NM_LANES - 1) / NM_LANES;
    if (want > most) want = most;
    return want < 1 ? 1 : (int)want;
}

static unsigned row_grid(int64_t rows)
{
    const int64_t cap = (int64_t)num_sms() * 8;
    return (unsigned)(rows < cap ? rows : cap);
}

template <typename TX, typename TY>
static void launch_backward(const NormArgs &a, cudaStream_t st)
{
    if (a.rows > 0) norm_dx_kernel<TX, TY><<<row_grid(a.rows), NM_THREADS, 0, st>>>(a);
    if (!a.dweight && !a.dbias) return;
    const dim3 grid((unsigned)((a.cols + NM_COLS - 1) / NM_COLS), (unsigned)a.splits);
    norm_dw_kernel<TX, TY><<<grid, NM_THREADS, 0, st>>>(a);
    norm_dw_sum_kernel<<<(unsigned)((a.cols + NM_THREADS - 1) / NM_THREADS), NM_THREADS, 0, st>>>(a);
}

template <typename TX, typename TY>
static void launch_forward(const NormArgs &a, cudaStream_t st)
{
    norm_forward_kernel<TX, TY><<<row_grid(a.rows), NM_THREADS, 0, st>>>(a);
}

static bool good_dtype(int d) { return d >= FP8_DTYPE_BF16 && d <= FP8_DTYPE_F32; }

// A [rows][ld] tensor of the type: pointer, row stride and alignment.
static fp8_status_t check_tensor(const void *p, int dtype, int64_t ld, int64_t cols)
{
    if (!p || ld < cols) return FP8_ERR_INVALID_ARG;
    return aligned(p, dtype == FP8_DTYPE_F32 ? 4 : 2) ? FP8_OK : FP8_ERR_ALIGNMENT;
}

static fp8_status_t check_codes(const void *q, int64_t ld_q, const void *s, int64_t ld_s, int64_t cols)
{
    if (!q || !s || ld_q < ckpt_width(cols) || ld_s < ckpt_width(cols) / FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    return ld_q % FP8_MX_BLOCK != 0 || !aligned(q, FP8_MX_BLOCK) ? FP8_ERR_ALIGNMENT : FP8_OK;
}

// What forward and backward check alike: sizes, kind, types (x of type xt on
// one side of the norm, y of type yt on the other), parameter pointers.
static fp8_status_t check_common(int64_t rows, int64_t cols, int kind, int xt, int yt, int wt, const void *w,
                                 const void *b)
{
    if (rows < 0 || cols < 1 || rows > INT32_MAX || cols > INT32_MAX - FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    if (kind != FP8_NORM_LAYER && kind != FP8_NORM_RMS) return FP8_ERR_INVALID_ARG;
    if (!good_dtype(xt) || !good_dtype(yt) || !good_dtype(wt)) return FP8_ERR_INVALID_ARG;
    if (xt != yt && xt != FP8_DTYPE_F32) return FP8_ERR_UNSUPPORTED;
    const uintptr_t al = wt == FP8_DTYPE_F32 ? 4 : 2;
    return aligned(w, al) && aligned(b, al) ? FP8_OK : FP8_ERR_ALIGNMENT;
}

static fp8_status_t check_fmt(int fmt)
{
    if (fmt == FP8_E4M3FNUZ || fmt == FP8_E5M2FNUZ) return FP8_ERR_UNSUPPORTED;
    return fmt == FP8_E4M3FN || fmt == FP8_E5M2 ? FP8_OK : FP8_ERR_INVALID_ARG;
}

// The five pairs of types: equal ones, and an fp32 x with 16-bit y.
#define NORM_TYPES(FN, xt, yt, ...)                                                        \
    do {                                                                                   \
        if (xt == FP8_DTYPE_BF16) FN<__nv_bfloat16, __nv_bfloat16>(__VA_ARGS__);           \
        else if (xt == FP8_DTYPE_F16) FN<__half, __half>(__VA_ARGS__);                     \
        else if (yt == FP8_DTYPE_BF16) FN<float, __nv_bfloat16>(__VA_ARGS__);              \
        else if (yt == FP8_DTYPE_F16) FN<float, __half>(__VA_ARGS__);                      \
        else FN<float, float>(__VA_ARGS__);                                                \
    } while (0)

}  // namespace fp8gb

using namespace fp8gb;

extern "C" fp8_status_t fp8_norm_forward(const void *x, int x_dtype, int64_t ld_x, int64_t rows, int64_t cols,
                                         int kind, float eps, const void *weight, const void *bias, int w_dtype,
                                         void *y, int y_dtype, int64_t ld_y, float *mean, float *rstd, int fmt,
                                         uint8_t *q, int64_t ld_q, uint8_t *s, int64_t ld_s, void *stream)
{
    fp8_status_t rc = check_common(rows, cols, kind, x_dtype, y_dtype, w_dtype, weight, bias);
    if (rc != FP8_OK) return rc;
    if (!(eps >= 0.0f)) return FP8_ERR_INVALID_ARG;
    if ((q || s) && (rc = check_fmt(fmt)) != FP8_OK) return rc;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return FP8_ERR_ALIGNMENT;
    if (rows == 0) return FP8_OK;
    if ((rc = check_tensor(x, x_dtype, ld_x, cols)) != FP8_OK) return rc;
    if ((rc = check_tensor(y, y_dtype, ld_y, cols)) != FP8_OK) return rc;
    if ((q || s) && (rc = check_codes(q, ld_q, s, ld_s, cols)) != FP8_OK) return rc;
    NormArgs a{};
    a.x = x;
    a.ld_x = ld_x;
    a.out = y;
    a.ld_out = ld_y;
    a.q = q;
    a.s = s;
    a.ld_q = ld_q;
    a.ld_s = ld_s;
    a.fmt = fmt;
    a.rows = rows;
    a.cols = cols;
    a.rms = kind == FP8_NORM_RMS;
    a.eps = eps;
    a.weight = weight;
    a.bias = bias;
    a.w_dtype = w_dtype;
    a.mean_out = mean;
    a.rstd_out = rstd;
    NORM_TYPES(launch_forward, x_dtype, y_dtype, a, static_cast<cudaStream_t>(stream));
    return check_launch();
}

extern "C" int64_t fp8_norm_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || rows > INT32_MAX || cols > INT32_MAX - FP8_MX_BLOCK) return -1;
    return (int64_t)norm_splits(rows, cols) * 2 * cols * (int64_t)sizeof(float);
}

extern "C" fp8_status_t fp8_norm_backward(const void *dy, int y_dtype, int64_t ld_dy, const void *x, int64_t ld_x,
                                          const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                          int64_t rows, int64_t cols, int kind, const float *mean, const float *rstd,
                                          const void *weight, int w_dtype, void *dx, int x_dtype, int64_t ld_dx,
                                          void *dweight, void *dbias, void *workspace, int64_t workspace_bytes,
                                          void *stream)
{
    fp8_status_t rc = check_common(rows, cols, kind, x_dtype, y_dtype, w_dtype, weight, nullptr);
    if (rc != FP8_OK) return rc;
    if (x && (q || s)) return FP8_ERR_INVALID_ARG;
    if (!x && (rc = check_fmt(fmt)) != FP8_OK) return rc;
    const uintptr_t al = w_dtype == FP8_DTYPE_F32 ? 4 : 2;
    if (!aligned(dweight, al) || !aligned(dbias, al) || !aligned(mean, 4) || !aligned(rstd, 4))
        return FP8_ERR_ALIGNMENT;
    if (dweight || dbias) {
        if (!workspace || workspace_bytes < fp8_norm_workspace_bytes(rows, cols)) return FP8_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return FP8_ERR_ALIGNMENT;
    }
    if (rows > 0) {
        if ((rc = check_tensor(dy, y_dtype, ld_dy, cols)) != FP8_OK) return rc;
        if ((rc = check_tensor(dx, x_dtype, ld_dx, cols)) != FP8_OK) return rc;
        if (!rstd || (x && kind == FP8_NORM_LAYER && !mean)) return FP8_ERR_INVALID_ARG;
        rc = x ? check_tensor(x, x_dtype, ld_x, cols) : check_codes(q, ld_q, s, ld_s, cols);
        if (rc != FP8_OK) return rc;
    }
    NormArgs a{};
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.x = x;
    a.ld_x = ld_x;
    a.q = const_cast<uint8_t *>(q);
    a.s = const_cast<uint8_t *>(s);
    a.ld_q = ld_q;
    a.ld_s = ld_s;
    a.fmt = fmt;
    a.rows = rows;
    a.cols = cols;
    a.rms = kind == FP8_NORM_RMS;
    a.mean = mean;
    a.rstd = rstd;
    a.weight = weight;
    a.w_dtype = w_dtype;
    a.out = dx;
    a.ld_out = ld_dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = static_cast<float *>(workspace);
    a.splits = norm_splits(rows, cols);
    NORM_TYPES(launch_backward, x_dtype, y_dtype, a, static_cast<cudaStream_t>(stream));
    return check_launch();
}
