// normquant.cu -- the residual's addition, a layer or RMS norm and the quantize
// of its result in one read: sum = x + residual (rounded to the residual's type
// and stored), y = norm(sum) w + b as in norm.cu, q = fp8(y / X).
//
// y is never written: it goes from fp32 registers into 8 bits with the one
// rounding of that conversion.  The norm is of the sum as it is stored, since that
// is what the backward reads.  Recipes: MX blocks of 32 (either layout), one scale
// per row, or a stored scale with the amax beside it (either layout).
//
//   norm_quantize_rows  a row stays in the registers of its group of threads, as
//                       in the norm's forward: sum, statistics, the row layout.
//                       Bound by HBM: [8192, 4096] bf16, MX 38 us = 6.2 TB/s, [32768,
//                       7168] with an fp32 residual 414 us = 6.3 TB/s.
//   norm_quantize_cols  the transposed layout, whose blocks run over rows, from
//                       the stored sum and the rows' statistics: [8192, 4096] 21 us,
//                       [32768, 7168] fp32 165 us = 7.2 TB/s (some of it from L2).
// Two kernels, and the sum read once more: both layouts in one kernel, 32 rows in
// the shared memory of a cluster, took 70 to 79 us for [8192, 4096] against 64, and
// 920 against 613 for the fp32 one: 26 instructions an element instead of 13 + 11, and
// phases that two or three blocks an SM do not hide.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"
#include "norm.cuh"

namespace fp8gb {
namespace nq {

enum { MX = 0, ROWWISE = 1, DELAYED = 2 };

struct Args {
    const void *x, *res;
    void *sum;
    int64_t ld_x, ld_res, ld_sum;
    int64_t rows, cols;
    int rms;
    float eps;
    const void *weight, *bias;
    int w_dtype;
    float *mean, *rstd;
    int recipe, fmt, margin;
    const float *scale_in;
    float *amax_out, *scale_inv_row, *scale_inv_col;
    uint8_t *q_row, *s_row, *q_col, *s_col;
    int64_t ld_col, rs_row, rs_col;
    int c32;                  // q_col's rows start on 32-byte boundaries
    int G, ranks, part_cols;  // as in a norm's launch
    int w32;
    int64_t end_x, end_res;  // elements from their start to the end of their last row
};

__device__ __forceinline__ uint4 encode(const float (&v)[16], float inv, int fmt)
{
    return fmt == FP8_E5M2 ? encode16<FP8_E5M2>(v, inv) : encode16<FP8_E4M3FN>(v, inv);
}

__device__ __forceinline__ uint32_t mx_code_of(uint32_t amax_bits, int fmt)
{
    return fmt == FP8_E5M2 ? mx_code<FP8_E5M2>(amax_bits) : mx_code<FP8_E4M3FN>(amax_bits);
}

__device__ __forceinline__ uint32_t amax16(const float (&f)[16], uint32_t m)
{
#pragma unroll
    for (int j = 0; j < 16; j++) m = max(m, abs_bits(f[j]));
    return m;
}

// Largest of the fp32 bit patterns over the threads of a row group (a NaN's is
// above all others'), through the same shared slots as its sums.
template <bool MULTI>
__device__ __forceinline__ uint32_t row_max(uint32_t v, int G, const Group &g, int slot)
{
    if constexpr (!MULTI) {
        for (int d = G >> 1; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    } else {
        v = __reduce_max_sync(0xffffffffu, v);
        uint32_t *part = reinterpret_cast<uint32_t *>(g.part + slot * 2 * NM_GROUP_WARPS);
        if ((g.t & 31) == 0) part[g.t >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(G) : "memory");
        v = 0;
#pragma unroll
        for (int w = 0; w < NM_GROUP_WARPS; w++) v = max(v, part[w]);
        return v;
    }
}

__device__ __forceinline__ uint32_t cluster_max(uint32_t v, float (*trade)[NM_MAX_RANKS][4], int slot, int rank,
                                                int ranks)
{
    if (threadIdx.x < ranks)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(trade[slot][rank]), threadIdx.x)),
                     "r"(v)
                     : "memory");
    cluster_sync();
    v = 0;
    for (int k = 0; k < ranks; k++) v = max(v, __float_as_uint(trade[slot][k][0]));
    return v;
}

// Zeros in the scale bytes behind the data: rows R .. of every K tile, and the
// blocks behind KB of the last one.
__device__ __forceinline__ void pad_scales(uint8_t *s, int64_t R, int64_t KB, int64_t thread, int64_t threads)
{
    const int64_t R128 = round_up_128(R), KT = (KB + 3) / 4, extra = R128 - R;
    for (int64_t i = thread; i < extra * KT; i += threads) {
        const int64_t kt = i / extra;
        reinterpret_cast<uint32_t *>(s)[mx_scale_word(kt, R + i - kt * extra, R128)] = 0;
    }
    const int have = (int)(KB & 3);
    if (have)
        for (int64_t r = thread; r < R; r += threads)
            for (int b = have; b < 4; b++) s[4 * mx_scale_word(KT - 1, r, R128) + b] = 0;
}

// The rows: sum, statistics, row layout, amax.  Thread t of G holds columns
// (k G + t) 16 .. + 15 of its group's row for k < CH.
template <typename TX, typename TR, int CH, bool MULTI, bool ANY, bool CLUSTER>
__global__ void __launch_bounds__(NM_BLOCK) norm_quantize_rows(Args a)
{
    extern __shared__ __align__(16) float shared[];  // weight, bias
    __shared__ __align__(16) float2 parts[MULTI ? NM_MAX_GROUPS * 4 * NM_GROUP_WARPS : 1];
    __shared__ float trade[2][NM_MAX_RANKS][4];
    const float inv_n = 1.0f / (float)a.cols;
    const int rank = CLUSTER ? (int)cluster_ctarank() : 0, base = CLUSTER ? rank * a.part_cols : 0;
    const int cols = CLUSTER ? min(a.part_cols, (int)a.cols - base) : (int)a.cols, G = a.G, chunks = CH * G;
    const Group g = group_of<MULTI>(G, parts);
    const int groups = CLUSTER ? 1 : MULTI ? blockDim.x / G : blockDim.x >> (31 - __clz(G));
    const int64_t step = (int64_t)(CLUSTER ? gridDim.x / a.ranks : gridDim.x) * groups;
    int n[CH];  // columns of the row in each chunk, from 16 down to 0
#pragma unroll
    for (int k = 0; k < CH; k++) n[k] = max(0, min(16, cols - (k * G + g.t) * 16));

    // the threads of a group (of a warp, where it holds several) run the same
    // iterations: `first` is the row of the first group among them
    int64_t r = (int64_t)(CLUSTER ? blockIdx.x / a.ranks : blockIdx.x) * groups + g.id;
    int64_t first = MULTI ? r : r - (threadIdx.x & 31) / G;
    const int c0 = base + g.t * 16;
    Raw<TX, ANY> rx[CH];
    Raw<TR, ANY> rr[CH];
    const auto fetch = [&](int64_t row) {
        const bool live = row < a.rows;
        const int64_t ax = row * a.ld_x + c0, ar = row * a.ld_res + c0;
#pragma unroll
        for (int k = 0; k < CH; k++) {
            load_chunk<ANY>(static_cast<const TX *>(a.x) + ax + k * G * 16, live ? n[k] : 0, a.w32, ax + k * G * 16,
                            a.end_x, rx[k]);
            if (a.res)
                load_chunk<ANY>(static_cast<const TR *>(a.res) + ar + k * G * 16, live ? n[k] : 0, a.w32,
                                ar + k * G * 16, a.end_res, rr[k]);
        }
    };
    fetch(r);
    const char *w = static_cast<const char *>(a.weight), *b = static_cast<const char *>(a.bias);
    const int pb = base * (a.w_dtype == FP8_DTYPE_F32 ? 4 : 2);
    params_to_shared(shared, w ? w + pb : nullptr, a.w_dtype, cols, chunks, 1.0f);
    if (b) params_to_shared(shared + chunks * 16, b + pb, a.w_dtype, cols, chunks, 0.0f);
    if (MULTI)
        for (int i = threadIdx.x; i < NM_MAX_GROUPS * 4 * NM_GROUP_WARPS; i += blockDim.x)
            parts[i] = make_float2(0.0f, 0.0f);
    float scale = 1.0f;
    uint32_t amax = 0;
    if (a.recipe == DELAYED) {
        scale = __ldg(a.scale_in);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            const float inv = recip_rn(scale);
            if (a.scale_inv_row) a.scale_inv_row[0] = inv;
            if (a.scale_inv_col) a.scale_inv_col[0] = inv;
        }
    } else if (a.recipe == MX && a.s_row) {
        pad_scales(a.s_row, a.rows, a.cols / FP8_MX_BLOCK, blockIdx.x * (int64_t)blockDim.x + threadIdx.x,
                   gridDim.x * (int64_t)blockDim.x);
    }
    __syncthreads();
    if constexpr (CLUSTER) cluster_sync();  // all its blocks run: the sums may be written to them

    int slot = 0;
    for (; first < a.rows; first += step, r += step) {
        float f[CH][16];
        const bool live = r < a.rows;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < CH; k++) {
            unpack16(rx[k], f[k]);
            if (a.res) {
                float t[16];
                unpack16(rr[k], t);
#pragma unroll
                for (int j = 0; j < 16; j++) f[k][j] = to_f32(from_f32<TR>(f[k][j] + t[j]));  // as it is stored
                store_chunk<ANY>(static_cast<TR *>(a.sum) + r * a.ld_sum + c0 + k * G * 16, f[k],
                                 live ? cols - (k * G + g.t) * 16 : 0, a.w32, g.t, G);
            }
            fill_from(f[k], n[k], 0.0f);
            v += sum16(f[k]);
        }
        if (r + step < a.rows) fetch(r + step);
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
        if (g.t == 0 && rank == 0 && live) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < CH; k++) {
            const int i = k * G + g.t;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float4 pw = param4(shared, chunks, i, q);
                float2 lo = mul2(make_float2(f[k][4 * q], f[k][4 * q + 1]), make_float2(rstd, rstd));
                float2 hi = mul2(make_float2(f[k][4 * q + 2], f[k][4 * q + 3]), make_float2(rstd, rstd));
                if (b) {
                    const float4 pc = param4(shared + chunks * 16, chunks, i, q);
                    lo = fma2(lo, make_float2(pw.x, pw.y), make_float2(pc.x, pc.y));
                    hi = fma2(hi, make_float2(pw.z, pw.w), make_float2(pc.z, pc.w));
                } else {
                    lo = mul2(lo, make_float2(pw.x, pw.y));
                    hi = mul2(hi, make_float2(pw.z, pw.w));
                }
                f[k][4 * q] = lo.x, f[k][4 * q + 1] = lo.y, f[k][4 * q + 2] = hi.x, f[k][4 * q + 3] = hi.y;
            }
            if (a.recipe != MX && live && n[k] > 0) m = amax16(f[k], m);  // widths are multiples of 16
        }
        float inv = scale;
        if (a.recipe == ROWWISE) {
            m = row_max<MULTI>(m, G, g, slot);
            if (CLUSTER) m = cluster_max(m, trade, slot, rank, a.ranks);
            slot ^= 1;
            inv = scale_from_amax(__uint_as_float(m), fp8_max_of(a.fmt), a.margin);
            if (g.t == 0 && rank == 0 && live) a.scale_inv_row[r] = recip_rn(inv);
        } else if (a.recipe == DELAYED) {
            amax = max(amax, m);
        }
        if (a.q_row) {
#pragma unroll
            for (int k = 0; k < CH; k++) {
                const int i = k * G + g.t, c = base + i * 16;
                if (a.recipe == MX) {
                    const uint32_t code = mx_code_of(block_amax16(f[k]), a.fmt);
                    inv = mx_inv_scale(code);
                    if (live && n[k] > 0 && !(i & 1))
                        a.s_row[4 * mx_scale_word(c >> 7, r, a.rs_row) + (c >> 5 & 3)] = (uint8_t)code;
                }
                if (live && n[k] > 0)
                    *reinterpret_cast<uint4 *>(a.q_row + r * a.cols + c) = encode(f[k], inv, a.fmt);
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the columns' blocks may start
    if (a.recipe == DELAYED) {
        amax = __reduce_max_sync(0xffffffffu, amax);
        if ((threadIdx.x & 31) == 0 && amax) atomicMax(reinterpret_cast<unsigned int *>(a.amax_out), amax);
    }
}

// The transposed layout: tiles of 128 rows x 128 columns of the normalized rows
// through shared memory, in fp32; a thread then has 32 rows of a column, a block.
// Launched while the rows' kernel ends (programmatic dependent launch), and from
// the last rows on, which are still in L2.
constexpr int CR = 128, CC = 128, C_THREADS = 256;
constexpr int C_SMEM = CR * CC * (int)sizeof(float);

// Word of column c in its row: 16-byte unit u is kept at u ^ (u / 4 % 8), so that
// neither the writes (threads 64 bytes apart) nor the reads (consecutive columns)
// meet a bank twice (four times without: the kernel was bound by that).
__device__ __forceinline__ int tile_word(int c) { return c ^ (c >> 2 & 28); }

// The first n of 32 codes.  Out of line: only the last rows have fewer.
static __device__ __noinline__ void put_some(uint8_t *dst, uint4 lo, uint4 hi, int n)
{
    const uint64_t q[4] = {lo.x | (uint64_t)lo.y << 32, lo.z | (uint64_t)lo.w << 32, hi.x | (uint64_t)hi.y << 32,
                           hi.z | (uint64_t)hi.w << 32};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint64_t v = q[i];
#pragma unroll 1
        for (int j = 8 * i; j < n && j < 8 * i + 8; j++, v >>= 8) dst[j] = (uint8_t)v;
    }
}

// 16 elements that the kernel before wrote (zeros if not `have`).  This kernel starts
// before that one ends, so its loads are the coherent ones: not load_chunk's, which
// want data that nobody writes while the kernel lives.
template <typename T, bool ANY>
__device__ __forceinline__ void load_written(const T *p, bool have, bool w32, int64_t at, int64_t end, Raw<T, ANY> &raw)
{
    if constexpr (ANY) {
        if (have && well_inside(at, end)) {
            const uintptr_t from = reinterpret_cast<uintptr_t>(p);
            const uint4 *w = reinterpret_cast<const uint4 *>(from & ~(uintptr_t)15);
            raw.shift = (uint32_t)from & 15u;
#pragma unroll
            for (int j = 0; j <= (int)sizeof(T); j++) raw.v[j] = w[j];
        } else {
            load16(p, have ? 16 : 0, false, raw);  // element by element
        }
    } else {
        const uint4 *w = reinterpret_cast<const uint4 *>(p);
        if (!have) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j++) raw.v[j] = make_uint4(0, 0, 0, 0);
        } else if (w32) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j += 2) ld_32b(w + j, raw.v[j], raw.v[j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j++) raw.v[j] = w[j];
        }
    }
}

// Three blocks an SM; two of fp32, whose 64 registers of loads in flight would spill
// ([32768, 7168] 207 against 165 us).  A persistent block that loads its next tile
// under this one's columns took 27 us against 21 for [8192, 4096] bf16 (25 with two blocks).
template <typename T, bool ANY>
__global__ void __launch_bounds__(C_THREADS, sizeof(T) == 4 ? 2 : 3) norm_quantize_cols(Args a)
{
    extern __shared__ __align__(16) float tile[];  // [CR][CC] xhat
    const T *src = static_cast<const T *>(a.res ? a.sum : a.x);
    const int64_t ld = a.res ? a.ld_sum : a.ld_x, end = rows_end(ld, a.rows, a.cols);
    const uint32_t n_ct = (uint32_t)(a.rs_col / CC), n_rt = gridDim.x / n_ct;
    const uint32_t rt = blockIdx.x / n_ct, ct = blockIdx.x - rt * n_ct;
    const int64_t r0 = (int64_t)(n_rt - 1 - rt) * CR;
    const int col0 = (int)ct * CC;
    const int left = (int)(a.rows - r0 < CR ? a.rows - r0 : CR);
    constexpr int PER = CC / 16, UNITS = CR * PER / C_THREADS, STEP = C_THREADS / PER;  // of 16 columns
    const int lr = threadIdx.x / PER, lc = threadIdx.x % PER * 16;
    const bool in = col0 + lc < a.cols;  // widths are multiples of 16

    const int c = col0 + threadIdx.x % CC;
    const bool column = c < a.cols;
    const float w = column ? param(a.weight, a.w_dtype, c, 1.0f) : 0.0f;
    const float b = column ? param(a.bias, a.w_dtype, c, 0.0f) : 0.0f;
    const float scale = a.recipe == MX ? 1.0f : __ldg(a.scale_in);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the sum and the statistics are written

    Raw<T, ANY> raw[UNITS];
    float rs[UNITS], mm[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; i++) {
        const int k = lr + i * STEP;
        const int64_t at = (r0 + k) * ld + col0 + lc;
        const bool live = k < left;
        load_written<T, ANY>(src + at, live && in, a.w32, at, end, raw[i]);
        rs[i] = live ? a.rstd[r0 + k] : 0.0f;
        mm[i] = live && !a.rms ? -a.mean[r0 + k] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < UNITS; i++) {
        float f[16];
        unpack16(raw[i], f);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float2 u = mul2(add2(make_float2(f[j], f[j + 1]), make_float2(mm[i], mm[i])), make_float2(rs[i], rs[i]));
            const float2 v =
                mul2(add2(make_float2(f[j + 2], f[j + 3]), make_float2(mm[i], mm[i])), make_float2(rs[i], rs[i]));
            *reinterpret_cast<float4 *>(tile + (lr + i * STEP) * CC + tile_word(lc + j)) = make_float4(u.x, u.y, v.x, v.y);
        }
    }
    __syncthreads();
    uint8_t *s = a.recipe == MX ? a.s_col + 4 * mx_scale_word(r0 >> 7, c, a.rs_col) : nullptr;
#pragma unroll
    for (int i = 0; i < CR / 32 * CC / C_THREADS; i++) {
        const int rb = threadIdx.x / CC + i * (C_THREADS / CC), n = min(32, left - 32 * rb);
        const float *from = tile + 32 * rb * CC + tile_word(threadIdx.x % CC);
        float v[2][16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            // behind the last column w = b = 0: 0, or NaN beside a row whose statistics are not finite
            const float2 y = fma2(make_float2(from[j * CC], from[(j + 1) * CC]), make_float2(w, w),
                                  make_float2(b, b));
            v[j >> 4][j & 15] = y.x, v[j >> 4][(j & 15) + 1] = y.y;
        }
        float inv = scale;
        if (a.recipe == MX) {  // whole blocks of 32 rows; zeros behind the data, whatever stands there
            float m = 0.0f, o = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                m = max3_abs(m, v[0][j], v[0][j + 1]);
                o = max3_abs(o, v[1][j], v[1][j + 1]);
            }
            const uint32_t code = column && n > 0 ? mx_code_of(__float_as_uint(max_nan(m, o)), a.fmt) : 0u;
            inv = mx_inv_scale(code);
            s[rb] = (uint8_t)code;
        }
        if (!column || n <= 0) continue;
        uint8_t *dst = a.q_col + c * a.ld_col + r0 + 32 * rb;
        const uint4 lo = encode(v[0], inv, a.fmt), hi = encode(v[1], inv, a.fmt);
        if (n < 32) {
            put_some(dst, lo, hi, n);
        } else if (a.c32) {
            st_32b(dst, lo, hi);
        } else {
            *reinterpret_cast<uint4 *>(dst) = lo;
            *reinterpret_cast<uint4 *>(dst + 16) = hi;
        }
    }
}

static constexpr int rows_shared(int chunks, int G, bool bias)
{
    return chunks * G * 16 * (int)sizeof(float) * (bias ? 2 : 1);
}

template <auto KERNEL, int MOST>
static fp8_status_t launch_rows_kernel(const Plan &p, int smem, Args a, cudaStream_t st)
{
    a.G = p.G;
    a.ranks = p.ranks;
    a.part_cols = p.part_cols;
    if (smem > NM_SHARED_FREE && !allow_shared<KERNEL, MOST>()) return cuda_fail();
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)p.ranks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = p.ranks > 1;
    cudaLaunchKernelEx(&cfg, KERNEL, a);
    return check_launch();
}

template <typename TX, typename TR, bool ANY>
static fp8_status_t launch_rows(const Args &a, cudaStream_t st)
{
    constexpr int narrow = rows_shared(2, 32, true), wide = rows_shared(2, NM_BLOCK, true);
    // Unaligned fp32 rows take one chunk a thread: two need 42 registers more of words
    // in flight, which spill ([16384, 4096] 240 against 167 us, bf16 + fp32 167 against 151;
    // 16 bits do not spill).  Beyond what one chunk covers in a block they stay two: a
    // cluster costs more ([8192, 14336] bf16 + fp32 346 against 431 us).
    if constexpr (ANY && sizeof(TR) == 4) {
        if (a.cols <= NM_PART) {
            const Plan p = make_plan(a.rows, a.cols, 1);
            const int smem = rows_shared(1, p.G, a.bias != nullptr);
            if (p.multi) return launch_rows_kernel<norm_quantize_rows<TX, TR, 1, true, ANY, false>, wide>(p, smem, a, st);
            return launch_rows_kernel<norm_quantize_rows<TX, TR, 1, false, ANY, false>, narrow>(p, smem, a, st);
        }
    }
    const Plan p = make_plan(a.rows, a.cols, 2);
    const int smem = rows_shared(p.chunks, p.G, a.bias != nullptr);
    if (p.ranks > 1) return launch_rows_kernel<norm_quantize_rows<TX, TR, 2, true, ANY, true>, wide>(p, smem, a, st);
    if constexpr (!(ANY && sizeof(TR) == 4)) {  // those rows are wider than one warp here
        if (p.chunks == 1)
            return launch_rows_kernel<norm_quantize_rows<TX, TR, 1, false, ANY, false>, narrow>(p, smem, a, st);
        if (!p.multi)
            return launch_rows_kernel<norm_quantize_rows<TX, TR, 2, false, ANY, false>, narrow>(p, smem, a, st);
    }
    return launch_rows_kernel<norm_quantize_rows<TX, TR, 2, true, ANY, false>, wide>(p, smem, a, st);
}

template <typename T>
static fp8_status_t launch_cols(Args a, cudaStream_t st)
{
    const void *src = a.res ? a.sum : a.x;
    const int64_t ld = a.res ? a.ld_sum : a.ld_x;
    a.w32 = rows_aligned(src, ld, sizeof(T), 32);
    a.c32 = rows_aligned(a.q_col, a.ld_col, 1, 32);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.rows + CR - 1) / CR * (a.rs_col / CC)));
    cfg.blockDim = dim3(C_THREADS);
    cfg.dynamicSmemBytes = C_SMEM;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (rows_aligned(src, ld, sizeof(T), 16)) {
        if (!allow_shared<norm_quantize_cols<T, false>, C_SMEM>()) return cuda_fail();
        cudaLaunchKernelEx(&cfg, norm_quantize_cols<T, false>, a);
    } else {
        if (!allow_shared<norm_quantize_cols<T, true>, C_SMEM>()) return cuda_fail();
        cudaLaunchKernelEx(&cfg, norm_quantize_cols<T, true>, a);
    }
    return check_launch();
}

// x and the residual; without one TR is TX.
template <typename TX, typename TR>
static fp8_status_t launch(Args a, cudaStream_t st)
{
    const auto all_aligned = [&](int al) {
        return rows_aligned(a.x, a.ld_x, sizeof(TX), al) && rows_aligned(a.res, a.ld_res, sizeof(TR), al) &&
               rows_aligned(a.sum, a.ld_sum, sizeof(TR), al);
    };
    a.w32 = all_aligned(32);
    a.end_x = rows_end(a.ld_x, a.rows, a.cols);
    a.end_res = rows_end(a.ld_res, a.rows, a.cols);
    const fp8_status_t rc = all_aligned(16) ? launch_rows<TX, TR, false>(a, st) : launch_rows<TX, TR, true>(a, st);
    if (rc != FP8_OK || !a.q_col) return rc;
    return launch_cols<TR>(a, st);
}

#define NQ_TRY(x)                      \
    do {                               \
        const fp8_status_t rc_ = (x);  \
        if (rc_ != FP8_OK) return rc_; \
    } while (0)

// Checks both entry points share, and the launch.
static fp8_status_t run(Args a, int x_dtype, int r_dtype, int kind, int layouts, void *stream)
{
    const int64_t rows = a.rows, cols = a.cols;
    if (rows < 0 || cols < 1 || rows > INT32_MAX) return FP8_ERR_INVALID_ARG;
    if (cols > NM_MAX_COLS) return FP8_ERR_UNSUPPORTED;
    if (kind != FP8_NORM_LAYER && kind != FP8_NORM_RMS) return FP8_ERR_INVALID_ARG;
    if (!good_dtype(x_dtype) || !good_dtype(a.w_dtype)) return FP8_ERR_INVALID_ARG;
    if (a.fmt == FP8_E4M3FNUZ || a.fmt == FP8_E5M2FNUZ) return FP8_ERR_UNSUPPORTED;
    if (a.fmt != FP8_E4M3FN && a.fmt != FP8_E5M2) return FP8_ERR_INVALID_ARG;
    if (layouts < 1 || layouts > 3 || !(a.eps >= 0.0f)) return FP8_ERR_INVALID_ARG;
    if (!a.res) r_dtype = x_dtype;
    if (!good_dtype(r_dtype) || (!a.res && a.sum)) return FP8_ERR_INVALID_ARG;
    if (r_dtype != x_dtype && r_dtype != FP8_DTYPE_F32) return FP8_ERR_UNSUPPORTED;
    if (a.recipe == ROWWISE && (layouts & FP8_LAYOUT_COLT)) return FP8_ERR_UNSUPPORTED;
    const uintptr_t al = a.w_dtype == FP8_DTYPE_F32 ? 4 : 2;
    if (cols % (a.recipe == MX ? FP8_MX_BLOCK : 16) != 0 || !aligned(a.weight, al) || !aligned(a.bias, al))
        return FP8_ERR_ALIGNMENT;
    const bool col = layouts & FP8_LAYOUT_COLT;
    if (col && ((a.recipe == MX && rows % FP8_MX_BLOCK != 0) || a.ld_col % 16 != 0)) return FP8_ERR_ALIGNMENT;
    if (col && a.ld_col < rows) return FP8_ERR_INVALID_ARG;
    if (rows == 0) return FP8_OK;
    NQ_TRY(check_tensor(a.x, x_dtype, a.ld_x, cols));
    if (a.res) {
        NQ_TRY(check_tensor(a.res, r_dtype, a.ld_res, cols));
        NQ_TRY(check_tensor(a.sum, r_dtype, a.ld_sum, cols));
    }
    if (!aligned(a.mean, 4) || !aligned(a.rstd, 4)) return FP8_ERR_ALIGNMENT;
    if (layouts & FP8_LAYOUT_ROW) {
        if (!a.q_row || (a.recipe == MX ? !a.s_row : !a.scale_inv_row)) return FP8_ERR_INVALID_ARG;
        if (!aligned(a.q_row, 16) || !aligned(a.s_row, 4) || !aligned(a.scale_inv_row, 4)) return FP8_ERR_ALIGNMENT;
    } else {
        a.q_row = a.s_row = nullptr;
        a.scale_inv_row = nullptr;
    }
    if (col) {
        if (!a.q_col || (a.recipe == MX ? !a.s_col : !a.scale_inv_col)) return FP8_ERR_INVALID_ARG;
        if (!a.rstd || (kind == FP8_NORM_LAYER && !a.mean)) return FP8_ERR_INVALID_ARG;
        if (!aligned(a.q_col, 16) || !aligned(a.s_col, 4) || !aligned(a.scale_inv_col, 4)) return FP8_ERR_ALIGNMENT;
    } else {
        a.q_col = a.s_col = nullptr;
        a.scale_inv_col = nullptr;
    }
    if (a.recipe == DELAYED && (!a.scale_in || !a.amax_out)) return FP8_ERR_INVALID_ARG;
    if (!aligned(a.scale_in, 4) || !aligned(a.amax_out, 4)) return FP8_ERR_ALIGNMENT;
    if (a.res && starts_at_any(a.sum, {a.x, a.res, a.weight, a.bias, a.scale_in})) return FP8_ERR_INVALID_ARG;
    a.rms = kind == FP8_NORM_RMS;
    a.rs_row = round_up_128(rows);
    a.rs_col = round_up_128(cols);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_dtype == FP8_DTYPE_BF16)
        return r_dtype == FP8_DTYPE_F32 ? launch<__nv_bfloat16, float>(a, st)
                                        : launch<__nv_bfloat16, __nv_bfloat16>(a, st);
    if (x_dtype == FP8_DTYPE_F16)
        return r_dtype == FP8_DTYPE_F32 ? launch<__half, float>(a, st) : launch<__half, __half>(a, st);
    return launch<float, float>(a, st);
}

static Args args(const void *x, int64_t ld_x, const void *residual, int64_t ld_r, int64_t rows, int64_t cols,
                 float eps, const void *weight, const void *bias, int w_dtype, void *sum, int64_t ld_sum, float *mean,
                 float *rstd, int fmt, uint8_t *q_row, uint8_t *q_colT, int64_t ld_colT)
{
    Args a{};
    a.x = x;
    a.ld_x = ld_x;
    a.res = residual;
    a.ld_res = ld_r;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.weight = weight;
    a.bias = bias;
    a.w_dtype = w_dtype;
    a.sum = sum;
    a.ld_sum = ld_sum;
    a.mean = mean;
    a.rstd = rstd;
    a.fmt = fmt;
    a.q_row = q_row;
    a.q_col = q_colT;
    a.ld_col = ld_colT;
    return a;
}

}  // namespace nq
}  // namespace fp8gb

using namespace fp8gb;

extern "C" fp8_status_t fp8_norm_quantize(const void *x, int x_dtype, int64_t ld_x, const void *residual, int r_dtype,
                                          int64_t ld_r, int64_t rows, int64_t cols, int kind, float eps,
                                          const void *weight, const void *bias, int w_dtype, void *sum,
                                          int64_t ld_sum, float *mean, float *rstd, int fmt,
                                          const fp8_recipe_t *recipe, int layouts, const float *scale_in,
                                          float *amax_out, uint8_t *q_row, float *scale_inv_row, uint8_t *q_colT,
                                          int64_t ld_colT, float *scale_inv_col, void *stream)
{
    if (!recipe) return FP8_ERR_INVALID_ARG;
    if (recipe->kind == FP8_RECIPE_TENSORWISE) return FP8_ERR_UNSUPPORTED;
    if (recipe->kind != FP8_RECIPE_DELAYED && recipe->kind != FP8_RECIPE_ROWWISE) return FP8_ERR_INVALID_ARG;
    if (recipe->margin < 0 || recipe->margin > 64) return FP8_ERR_INVALID_ARG;
    nq::Args a = nq::args(x, ld_x, residual, ld_r, rows, cols, eps, weight, bias, w_dtype, sum, ld_sum, mean, rstd,
                          fmt, q_row, q_colT, ld_colT);
    a.recipe = recipe->kind == FP8_RECIPE_DELAYED ? nq::DELAYED : nq::ROWWISE;
    if (a.recipe == nq::ROWWISE && (scale_in || amax_out)) return FP8_ERR_INVALID_ARG;
    a.margin = recipe->margin;
    a.scale_in = scale_in;
    a.amax_out = amax_out;
    a.scale_inv_row = scale_inv_row;
    a.scale_inv_col = scale_inv_col;
    return nq::run(a, x_dtype, r_dtype, kind, layouts, stream);
}

extern "C" fp8_status_t fp8_mx_norm_quantize(const void *x, int x_dtype, int64_t ld_x, const void *residual,
                                             int r_dtype, int64_t ld_r, int64_t rows, int64_t cols, int kind,
                                             float eps, const void *weight, const void *bias, int w_dtype, void *sum,
                                             int64_t ld_sum, float *mean, float *rstd, int fmt, int layouts,
                                             uint8_t *q_row, uint8_t *s_row, uint8_t *q_colT, int64_t ld_colT,
                                             uint8_t *s_col, void *stream)
{
    nq::Args a = nq::args(x, ld_x, residual, ld_r, rows, cols, eps, weight, bias, w_dtype, sum, ld_sum, mean, rstd,
                          fmt, q_row, q_colT, ld_colT);
    a.recipe = nq::MX;
    a.s_row = s_row;
    a.s_col = s_col;
    return nq::run(a, x_dtype, r_dtype, kind, layouts, stream);
}
