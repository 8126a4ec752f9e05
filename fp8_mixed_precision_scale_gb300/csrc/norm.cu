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
// A row stays in the registers of its group of threads, 16 consecutive columns (a
// chunk) per thread and step; the group is a part of a warp or several warps with
// a named barrier of their own.  One persistent block per SM holds as many groups
// as its registers allow and one fp32 copy of the parameters in shared memory.
// A group issues the loads of its next rows before it reduces the current ones.
// The backward accumulates dw and db of its columns in registers over all its
// rows.  A row wider than one block's registers is split over the blocks of a
// cluster (2, 4 or 8), which trade their sums through distributed shared memory.
//
// dw and db are left as column sums over row slices in the caller's workspace
// and added in a fixed order by a last kernel: no atomics, the same bits every
// time.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"
#include "norm_backward.cuh"

namespace fp8gb {

// A row in the registers of its group: thread t of G holds columns (k G + t) 16
// .. + 15 for k < CH.  Two chunks a thread halve what a row sum costs per element
// and leave room for the next row.  Bound by HBM for large fp32 rows ([32768,
// 7168] fp32 to bf16 203 us, 6.95 TB/s).  bf16 rows are bound by latency: with 14 to
// 16 warps an SM, half of the issue slots are used (12 instructions an element, 16
// with the checkpoint) and the rest goes to waits for dependent instructions,
// shuffles and the group's barrier ([32768, 4096] 88.6 us, 6.1 TB/s; with the
// checkpoint [32768, 7168] 196 us, 6.0 TB/s).
template <typename TX, typename TY, int CH, bool MULTI, bool ANY, bool CLUSTER>
__global__ void __launch_bounds__(NM_BLOCK, CH == 1 && !ANY ? 2 : 1) norm_forward_kernel(NormArgs a)
{
    extern __shared__ __align__(16) float shared[];  // weight, bias
    __shared__ __align__(16) float2 parts[MULTI ? NM_MAX_GROUPS * 4 * NM_GROUP_WARPS : 1];
    __shared__ float trade[2][NM_MAX_RANKS][4];
    const float inv_n = 1.0f / (float)a.cols;
    const int rank = CLUSTER ? (int)cluster_ctarank() : 0;
    const int64_t end = rows_end(a.ld_x, a.rows, a.cols) - (CLUSTER ? rank * a.part_cols : 0);
    if (CLUSTER) a.out = static_cast<TY *>(a.out) + rank * a.part_cols;
    const int cols = CLUSTER ? take_part<TX, TY>(a, rank) : (int)a.cols, G = a.G, chunks = CH * G;
    const Group g = group_of<MULTI>(G, parts);
    // one group of a block where the row has several
    const int groups = CLUSTER ? 1 : MULTI ? blockDim.x / G : blockDim.x >> (31 - __clz(G));
    const int64_t step = (int64_t)(CLUSTER ? gridDim.x / a.ranks : gridDim.x) * groups;
    int n[CH];  // columns of the row in each chunk, from 16 down to 0
#pragma unroll
    for (int k = 0; k < CH; k++) n[k] = max(0, min(16, cols - (k * G + g.t) * 16));

    // the threads of a group (of a warp, where it holds several) run the same
    // iterations: `first` is the row of the first group among them
    int64_t r = (int64_t)(CLUSTER ? blockIdx.x / a.ranks : blockIdx.x) * groups + g.id;
    int64_t first = MULTI ? r : r - (threadIdx.x & 31) / G;
    int64_t at = r * a.ld_x + g.t * 16;  // of the row to load next, in x
    const TX *x = static_cast<const TX *>(a.x) + at;
    TY *y = static_cast<TY *>(a.out) + r * a.ld_out + g.t * 16;
    Raw<TX, ANY> raw[CH];
#pragma unroll
    for (int k = 0; k < CH; k++)
        load_chunk<ANY>(x + k * G * 16, r < a.rows ? n[k] : 0, a.w32, at + k * G * 16, end, raw[k]);
    params_to_shared(shared, a.weight, a.w_dtype, cols, chunks, 1.0f);
    if (a.bias) params_to_shared(shared + chunks * 16, a.bias, a.w_dtype, cols, chunks, 0.0f);
    if (MULTI)
        for (int i = threadIdx.x; i < NM_MAX_GROUPS * 4 * NM_GROUP_WARPS; i += blockDim.x)
            parts[i] = make_float2(0.0f, 0.0f);
    __syncthreads();
    if constexpr (CLUSTER) cluster_sync();  // all its blocks run: cluster_sum may write to them

    int slot = 0;
    for (; first < a.rows; first += step, r += step) {
        float f[CH][16];
        float v = 0.0f;
        x += step * a.ld_x;
        at += step * a.ld_x;
#pragma unroll
        for (int k = 0; k < CH; k++) {
            unpack16(raw[k], f[k]);
            if (ANY) fill_from(f[k], n[k], 0.0f);
            v += sum16(f[k]);
            if (r + step < a.rows)
                load_chunk<ANY>(x + k * G * 16, n[k], a.w32, at + k * G * 16, end, raw[k]);
        }
        float mean = 0.0f;
        if (!a.rms) {
            float t[1] = {row_sum<MULTI>(v, G, g, slot)};
            if (CLUSTER) cluster_sum(t, trade, slot, rank, a.ranks);
            mean = t[0] * inv_n;
            slot ^= 1;
        }
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < CH; k++) {
            float2 acc[2] = {};
            fill_from(f[k], n[k], mean);  // what is past the row adds nothing
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float2 d = add2(make_float2(f[k][j], f[k][j + 1]), make_float2(-mean, -mean));
                acc[j / 2 % 2] = fma2(d, d, acc[j / 2 % 2]);
                f[k][j] = d.x, f[k][j + 1] = d.y;
            }
            v += (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
        }
        float t[1] = {row_sum<MULTI>(v, G, g, slot)};
        if (CLUSTER) cluster_sum(t, trade, slot, rank, a.ranks);
        slot ^= 1;
        const float rstd = 1.0f / sqrtf(t[0] * inv_n + a.eps);
        const bool live = r < a.rows;
        if (g.t == 0 && rank == 0 && live) {
            if (a.mean_out) a.mean_out[r] = mean;
            if (a.rstd_out) a.rstd_out[r] = rstd;
        }
#pragma unroll
        for (int k = 0; k < CH; k++) {
            const int i = k * G + g.t;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float2 d = mul2(make_float2(f[k][j], f[k][j + 1]), make_float2(rstd, rstd));
                f[k][j] = d.x, f[k][j + 1] = d.y;
            }
            if (a.q) {
                const uint32_t code = ckpt_code(block_amax16(f[k]), a.fmt);
                if (live && (i & ~1) * 16 < cols) {
                    const float inv = ckpt_inv_scale(code);
                    *reinterpret_cast<uint4 *>(a.q + r * a.ld_q + i * 16) =
                        a.fmt == FP8_E5M2 ? encode16<FP8_E5M2>(f[k], inv) : encode16<FP8_E4M3FN>(f[k], inv);
                    if (!(i & 1)) a.s[r * a.ld_s + (i >> 1)] = (uint8_t)code;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float4 w = param4(shared, chunks, i, q);
                float2 lo = make_float2(f[k][4 * q], f[k][4 * q + 1]);
                float2 hi = make_float2(f[k][4 * q + 2], f[k][4 * q + 3]);
                if (a.bias) {
                    const float4 b = param4(shared + chunks * 16, chunks, i, q);
                    lo = fma2(lo, make_float2(w.x, w.y), make_float2(b.x, b.y));
                    hi = fma2(hi, make_float2(w.z, w.w), make_float2(b.z, b.w));
                } else {
                    lo = mul2(lo, make_float2(w.x, w.y));
                    hi = mul2(hi, make_float2(w.z, w.w));
                }
                f[k][4 * q] = lo.x, f[k][4 * q + 1] = lo.y, f[k][4 * q + 2] = hi.x, f[k][4 * q + 3] = hi.y;
            }
            store_chunk<ANY>(y + k * G * 16, f[k], live ? cols - i * 16 : 0, a.w32, g.t, G);
        }
        y += step * a.ld_out;
    }
}

// Dynamic shared memory of a launch, and the most that any launch of the kernel
// takes: NM_BLOCK threads, of which a row of up to 32 threads' chunks needs the
// parameters of no more than these.
static constexpr int forward_shared(int chunks, int G, bool bias)
{
    return chunks * G * 16 * (int)sizeof(float) * (bias ? 2 : 1);
}

static constexpr int forward_shared_most(bool multi) { return forward_shared(2, multi ? NM_BLOCK : 32, true); }

// Blocks (of one to an SM) that run at once in clusters of `ranks`, in
// clusters.  The SMs of a GPC are no multiple of 4 or 8, so it is fewer than the
// SMs would give: a grid for all SMs leaves clusters for a second wave ([2048,
// 20480] backward: 137 us with 38 clusters, 82 with those that fit).  Asked once
// per device, with the largest launch a cluster makes.
int clusters_at_once(int ranks)
{
    constexpr int MAX_DEVICES = 64;
    static std::atomic<int> known[MAX_DEVICES][NM_MAX_RANKS + 1];
    const int most = num_sms() / ranks > 0 ? num_sms() / ranks : 1;
    int dev = 0;
    if (ranks == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return most;
    int n = known[dev][ranks].load(std::memory_order_relaxed);
    if (n > 0) return n;
    constexpr auto kernel = norm_backward_kernel<float, __nv_bfloat16, true, false, false, true>;
    constexpr int shared = backward_shared_most<float, __nv_bfloat16, false, false>(true);
    static_assert(shared >= backward_shared_most<float, float, false, false>(true) &&
                      shared >= backward_shared_most<__nv_bfloat16, __nv_bfloat16, false, false>(true) &&
                      shared >= backward_shared_most<float, __nv_bfloat16, true, false>(true) &&
                      shared >= backward_shared_most<float, float, true, false>(true) &&
                      shared >= forward_shared_most(true),
                  "the largest launch");
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ranks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(most * ranks));
    cfg.blockDim = dim3(NM_BLOCK);
    cfg.dynamicSmemBytes = shared;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (!allow_shared<kernel, shared>() || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1 ||
        n > most) {
        cudaGetLastError();
        n = most;
    }
    known[dev][ranks].store(n, std::memory_order_relaxed);
    return n;
}

template <typename TX, typename TY, bool ANY>
static fp8_status_t launch_forward_as(const NormArgs &a, cudaStream_t st)
{
    const Plan p = make_plan(a.rows, a.cols, 2, !ANY);
    const int smem = forward_shared(p.chunks, p.G, a.bias != nullptr);
    constexpr int narrow = forward_shared_most(false), wide = forward_shared_most(true);
    if (p.ranks > 1) return launch<norm_forward_kernel<TX, TY, 2, true, ANY, true>, wide>(p, smem, a, st);
    if (p.chunks == 1) return launch<norm_forward_kernel<TX, TY, 1, false, ANY, false>, narrow>(p, smem, a, st);
    if (!p.multi) return launch<norm_forward_kernel<TX, TY, 2, false, ANY, false>, narrow>(p, smem, a, st);
    return launch<norm_forward_kernel<TX, TY, 2, true, ANY, false>, wide>(p, smem, a, st);
}

template <typename TX, typename TY>
static fp8_status_t launch_forward(NormArgs a, cudaStream_t st)
{
    const auto all_aligned = [&](int al) {
        return rows_aligned(a.x, a.ld_x, sizeof(TX), al) && rows_aligned(a.out, a.ld_out, sizeof(TY), al);
    };
    a.w32 = all_aligned(32);
    return all_aligned(16) ? launch_forward_as<TX, TY, false>(a, st) : launch_forward_as<TX, TY, true>(a, st);
}

// The five pairs of types: equal ones, and an fp32 x with 16-bit y.
#define NORM_TYPES(FN, xt, yt, ...)                                                        \
    (xt == FP8_DTYPE_BF16   ? FN<__nv_bfloat16, __nv_bfloat16>(__VA_ARGS__)                \
     : xt == FP8_DTYPE_F16  ? FN<__half, __half>(__VA_ARGS__)                              \
     : yt == FP8_DTYPE_BF16 ? FN<float, __nv_bfloat16>(__VA_ARGS__)                        \
     : yt == FP8_DTYPE_F16  ? FN<float, __half>(__VA_ARGS__)                               \
                            : FN<float, float>(__VA_ARGS__))

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
    return NORM_TYPES(launch_forward, x_dtype, y_dtype, a, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t fp8_norm_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || rows > INT32_MAX || cols > NM_MAX_COLS) return -1;
    const int64_t most = rows > 0 ? make_plan(rows, cols, 1).slices : 1;
    return most * 2 * cols * (int64_t)sizeof(float);
}

extern "C" fp8_status_t fp8_norm_backward(const void *dy, int y_dtype, int64_t ld_dy, const void *x, int64_t ld_x,
                                          const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                          int64_t rows, int64_t cols, int kind, const float *mean, const float *rstd,
                                          const void *weight, int w_dtype, void *dx, int x_dtype, int64_t ld_dx,
                                          void *dweight, void *dbias, void *workspace, int64_t workspace_bytes,
                                          void *stream)
{
    return norm_backward<false>(dy, y_dtype, ld_dy, x, ld_x, q, ld_q, s, ld_s, fmt, nullptr, 0, rows, cols, kind,
                                mean, rstd, weight, w_dtype, dx, x_dtype, ld_dx, dweight, dbias, workspace,
                                workspace_bytes, stream);
}
