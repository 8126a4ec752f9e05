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

namespace fp8gb {

constexpr int NM_COLS = 32;            // columns of a block of the last sums
constexpr int NM_BLOCK = 512;          // threads of a block at most: 128 registers each
constexpr int NM_MAX_GROUPS = NM_BLOCK / 64;  // row groups of two warps or more, a named barrier each
constexpr int NM_GROUP_WARPS = 16;     // warps of a row group at most
constexpr int NM_MAX_RANKS = 8;        // blocks of a cluster at most
constexpr int NM_PART = 16 * 32 * NM_GROUP_WARPS;  // columns one chunk a thread covers in a block
constexpr int64_t NM_MAX_COLS = (int64_t)NM_PART * NM_MAX_RANKS;

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
    int G;          // threads of a row group
    int ranks;      // blocks that share a row
    int part_cols;  // columns of each of them but the last
    int w32;        // every row of the tensors starts on a 32-byte boundary
    int64_t end_x, end_dy;  // elements from their start to the end of their last row
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

// Parameters c .. c + 15, `absent` past the row.
__device__ __forceinline__ void param16(const void *p, int dtype, int c, int cols, float absent, float (&f)[16])
{
    if (!p || c + 16 > cols || (reinterpret_cast<uintptr_t>(p) & 15)) {
#pragma unroll
        for (int j = 0; j < 16; j++) f[j] = c + j < cols ? param(p, dtype, c + j, absent) : absent;
    } else if (dtype == FP8_DTYPE_F32) {
        Raw16<float> r;
        load16(static_cast<const float *>(p) + c, 16, false, r);
        unpack16(r, f);
    } else if (dtype == FP8_DTYPE_F16) {
        Raw16<__half> r;
        load16(static_cast<const __half *>(p) + c, 16, false, r);
        unpack16(r, f);
    } else {
        Raw16<__nv_bfloat16> r;
        load16(static_cast<const __nv_bfloat16 *>(p) + c, 16, false, r);
        unpack16(r, f);
    }
}

// A parameter vector in shared memory as fp32, in the order the row threads
// read it: quad q of chunk i is at quad q * chunks + i, so the 16-byte reads of
// a warp are consecutive.
__device__ __forceinline__ void params_to_shared(float *dst, const void *p, int dtype, int cols, int chunks,
                                                 float absent)
{
    for (int i = threadIdx.x; i < chunks; i += blockDim.x) {
        float f[16];
        param16(p, dtype, i * 16, cols, absent, f);
#pragma unroll
        for (int q = 0; q < 4; q++)
            reinterpret_cast<float4 *>(dst)[q * chunks + i] =
                make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
    }
}

__device__ __forceinline__ float4 param4(const float *src, int chunks, int i, int q)
{
    return reinterpret_cast<const float4 *>(src)[q * chunks + i];
}

// Where a thread of a wide kernel stands: its row group in the block, its place
// in the group, and the group's shared slots for the sums.
struct Group {
    int id, t;
    float2 *part;  // [2][2][NM_GROUP_WARPS], zero beyond the group's warps
};

template <bool MULTI>
__device__ __forceinline__ Group group_of(int G, float2 *parts)
{
    Group g;
    if constexpr (MULTI) {
        g.id = threadIdx.x / G;
        g.t = threadIdx.x - g.id * G;
    } else {  // G is a power of two
        g.id = threadIdx.x >> (31 - __clz(G));
        g.t = threadIdx.x & (G - 1);
    }
    g.part = parts + g.id * 4 * NM_GROUP_WARPS;
    return g;
}

// Sum of a pair over the threads of a row group; every thread gets the same
// bits.  MULTI: through slot `slot` of the group's shared sums, one group
// barrier; two uses in a row take different slots.
template <bool MULTI>
__device__ __forceinline__ float2 row_sum(float2 v, int G, const Group &g, int slot)
{
    if constexpr (!MULTI) {
        for (int d = G >> 1; d > 0; d >>= 1)
            v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d)));
        return v;
    } else {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d)));
        float2 *part = g.part + slot * 2 * NM_GROUP_WARPS;
        if ((g.t & 31) == 0) part[g.t >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(G) : "memory");
        v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < NM_GROUP_WARPS; w += 2) {
            const float4 q = reinterpret_cast<const float4 *>(part)[w >> 1];
            v = add2(v, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
        }
        return v;
    }
}

template <bool MULTI>
__device__ __forceinline__ float row_sum(float v, int G, const Group &g, int slot)
{
    if constexpr (!MULTI) {
        for (int d = G >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    } else {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        float *part = reinterpret_cast<float *>(g.part + slot * 2 * NM_GROUP_WARPS);
        if ((g.t & 31) == 0) part[g.t >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(G) : "memory");
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < NM_GROUP_WARPS; w += 4) {  // all slots: a loop over the group's own took 25 % longer
            const float4 q = reinterpret_cast<const float4 *>(part)[w >> 2];
            s = add2(s, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
        }
        return s.x + s.y;
    }
}

// Sums of two rows' pairs.  In a whole warp the lanes trade values until each
// holds a part of one, so that six shuffles do instead of twenty, and every
// lane then adds up a share of the warps' sums.
template <bool MULTI>
__device__ __forceinline__ void row_sum(float2 (&v)[2], int G, const Group &g, int slot)
{
    if constexpr (!MULTI) {
        v[0] = row_sum<false>(v[0], G, g, slot);
        v[1] = row_sum<false>(v[1], G, g, slot);
    } else {
        const int lane = g.t & 31;
        const bool low = (lane & 16) == 0, even = (lane & 8) == 0;
        // lanes 0-15: row 0's pair, 16-31: row 1's
        float2 p = low ? v[0] : v[1], o = low ? v[1] : v[0];
        p = add2(p, make_float2(__shfl_xor_sync(0xffffffffu, o.x, 16), __shfl_xor_sync(0xffffffffu, o.y, 16)));
        float u = (even ? p.x : p.y) + __shfl_xor_sync(0xffffffffu, even ? p.y : p.x, 8);
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
        // value lane / 8 of the four, warp by warp
        float *part = reinterpret_cast<float *>(g.part) + slot * 4 * NM_GROUP_WARPS;
        if ((lane & 7) == 0) part[(lane >> 3) * NM_GROUP_WARPS + (g.t >> 5)] = u;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(G) : "memory");
        const float2 w = reinterpret_cast<const float2 *>(part)[lane];  // two warps' sums of value lane / 8
        u = w.x + w.y;
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
        v[0] = make_float2(__shfl_sync(0xffffffffu, u, 0), __shfl_sync(0xffffffffu, u, 8));
        v[1] = make_float2(__shfl_sync(0xffffffffu, u, 16), __shfl_sync(0xffffffffu, u, 24));
    }
}

template <bool MULTI>
__device__ __forceinline__ void row_sum(float2 (&v)[1], int G, const Group &g, int slot)
{
    v[0] = row_sum<MULTI>(v[0], G, g, slot);
}

// A block's columns of a row that a cluster shares: the arguments as if they
// were the whole row.
template <typename TX, typename TY>
__device__ __forceinline__ int take_part(NormArgs &a, int rank)
{
    const int base = rank * a.part_cols, cols = min(a.part_cols, (int)a.cols - base);
    const int pb = base * (a.w_dtype == FP8_DTYPE_F32 ? 4 : 2);
    if (a.x) a.x = static_cast<const TX *>(a.x) + base;
    if (a.weight) a.weight = static_cast<const char *>(a.weight) + pb;
    if (a.bias) a.bias = static_cast<const char *>(a.bias) + pb;
    if (a.q) {
        a.q += base;
        a.s += base / FP8_MX_BLOCK;
    }
    if (a.part) a.part += base;
    return cols;
}

// Sums of N values over the blocks of a cluster, in rank order; every thread
// gets the same bits.  Called by all threads of every block equally often,
// with alternating slots: a slot is written again only after every block has
// passed the barrier in between, and so has read it.  A kernel passes a cluster
// barrier before its first call, since a block that has not started has no shared
// memory to write to.
template <int N>
__device__ __forceinline__ void cluster_sum(float (&v)[N], float (*trade)[NM_MAX_RANKS][4], int slot, int rank,
                                            int ranks)
{
    if (threadIdx.x < ranks) {
        const uint32_t dst = mapa_shared(smem_u32(trade[slot][rank]), threadIdx.x);
#pragma unroll
        for (int i = 0; i < N; i++)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 4 * i), "f"(v[i]) : "memory");
    }
    cluster_sync();
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = 0.0f;
    for (int k = 0; k < ranks; k++)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += trade[slot][k][i];
}

__device__ __forceinline__ float sum16(const float (&f)[16])
{
    float2 t[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        t[j] = add2(make_float2(f[4 * j], f[4 * j + 1]), make_float2(f[4 * j + 2], f[4 * j + 3]));
    const float2 s = add2(add2(t[0], t[1]), add2(t[2], t[3]));
    return s.x + s.y;
}

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

// What a thread reads of a row in the backward: dy, and x or its checkpoint.
template <typename TX, typename TY, bool CKPT, bool ANY>
struct RawBackward {
    Raw<TY, ANY> dy;
    Raw<TX, ANY> x;
};

template <typename TX, typename TY, bool ANY>
struct RawBackward<TX, TY, true, ANY> {
    Raw<TY, ANY> dy;
    uint4 q;
    uint32_t s;
};

// Chunk i (n columns of it) of row r.
template <typename TX, typename TY, bool CKPT, bool ANY>
__device__ __forceinline__ void load_backward(const NormArgs &a, int64_t r, int i, int n,
                                              RawBackward<TX, TY, CKPT, ANY> &v)
{
    const int64_t at_dy = r * a.ld_dy + i * 16;
    load_chunk<ANY>(static_cast<const TY *>(a.dy) + at_dy, n, a.w32, at_dy, a.end_dy, v.dy);
    if constexpr (CKPT) {
        v.q = make_uint4(0, 0, 0, 0);
        v.s = 127;
        if (n > 0) {
            v.q = ld_stream_16b(a.q + r * a.ld_q + i * 16);
            v.s = __ldg(a.s + r * a.ld_s + (i >> 1));
        }
    } else {
        const int64_t at_x = r * a.ld_x + i * 16;
        load_chunk<ANY>(static_cast<const TX *>(a.x) + at_x, n, a.w32, at_x, a.end_x, v.x);
    }
}

template <typename TX, typename TY, bool CKPT, bool ANY>
__device__ __forceinline__ void dy16(const RawBackward<TX, TY, CKPT, ANY> &v, int n, float (&d)[16])
{
    unpack16(v.dy, d);
    if (ANY) fill_from(d, n, 0.0f);
}

// xh of a chunk; 0 past the row.
template <typename TX, typename TY, bool CKPT, bool ANY>
__device__ __forceinline__ void xhat16(const NormArgs &a, const RawBackward<TX, TY, CKPT, ANY> &v, int n, float mean,
                                       float rstd, float (&xh)[16])
{
    if constexpr (CKPT) {
        if (a.fmt == FP8_E5M2) decode16<FP8_E5M2>(v.q, ckpt_scale(v.s), xh);
        else decode16<FP8_E4M3FN>(v.q, ckpt_scale(v.s), xh);
    } else {
        unpack16(v.x, xh);
        fill_from(xh, n, mean);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float2 d = mul2(add2(make_float2(xh[j], xh[j + 1]), make_float2(-mean, -mean)),
                                  make_float2(rstd, rstd));
            xh[j] = d.x, xh[j + 1] = d.y;
        }
    }
}

// Rows ahead of the backward, in shared memory: each warp copies its own
// columns of dy and of x (or the codes) with cp.async into a ring, so the loads
// in flight cost no registers and no block barrier, and the registers hold two
// rows at a time, whose sums share one barrier and each other's latencies.
// A copy instruction takes 512 consecutive bytes (a thread's own 32 as two
// halves fetched every sector twice, 25 % slower than no ring); 16-byte unit u
// of a warp's part is kept at u ^ (u / 8 % SLOTS), so that reading a thread's own
// SLOTS units meets no bank twice.
template <typename TX, typename TY, bool CKPT>
struct Ring {
    static constexpr int dy_slots = sizeof(TY), x_slots = CKPT ? 1 : (int)sizeof(TX);  // of 16 bytes
    static constexpr int slots = dy_slots + x_slots;
    // rows a step, and steps in the ring: what 512 threads and the parameters of 8192 columns leave room for
    static constexpr int rows = slots <= 4 ? 2 : 1;
    static constexpr int stages = CKPT && rows == 1 ? 0 : rows == 2 || slots >= 8 ? 2 : 3;  // 0: no ring
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, int bytes)  // the rest of the 16: zeros
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A thread's place in the copies of its warp: `lane` of it, or where the warp
// holds several rows, place t of G in row `sub`.
struct CopyPlace {
    int t, G, sub;
};

// Bytes 0 .. valid - 1 of the warp's part of a row at `src` (zeros after).
template <int SLOTS, bool MULTI>
__device__ __forceinline__ void copy_ahead(uint32_t dst, const void *src, int valid, const CopyPlace &c,
                                           const void *anywhere)
{
    if (MULTI && valid >= SLOTS * 512) {  // all of the warp's columns: its units are 32 apart, the swizzle one
        const char *p = static_cast<const char *>(src) + c.t * 16;
        dst += (c.t ^ (c.t >> 3 & (SLOTS - 1))) * 16;
#pragma unroll
        for (int j = 0; j < SLOTS; j++) cp_async_16(dst + j * 512, p + j * 512, 16);
        return;
    }
#pragma unroll
    for (int j = 0; j < SLOTS; j++) {
        const int u = j * c.G + c.t, at = c.sub * SLOTS * c.G + u, bytes = max(0, min(16, valid - u * 16));
        cp_async_16(dst + (at ^ (at >> 3 & (SLOTS - 1))) * 16,
                    bytes ? static_cast<const char *>(src) + u * 16 : static_cast<const char *>(anywhere), bytes);
    }
}

// Unit j of a lane's SLOTS.
template <int SLOTS>
__device__ __forceinline__ uint4 copied(uint32_t src, int lane, int j)
{
    const int at = SLOTS * lane + j;
    return ld_shared_16b(src + (at ^ (at >> 3 & (SLOTS - 1))) * 16);
}

__device__ __forceinline__ int lane_id()
{
    int v;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(v));
    return v;
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// dx, and the block's share of dw and db: in registers until the last row, then
// added over the block's groups in shared memory (in group order) into the
// block's slice of the workspace.  One chunk a thread, since the accumulators
// and two rows fill its 128 registers: whatever spills is waited for, and each
// spill that went was worth 3 to 10 %.  Aligned bf16 rows have none (8 bytes in a
// cluster, from the checkpoint).  Forms with an fp16 dy spill up to 56 bytes, and
// fp16 rows take 1.2 to 1.5 times as long ([32768, 7168] 302 us from x, 322 from the
// checkpoint).  From x bound by HBM ([32768, 4096] 124 us, 6.5 TB/s; [32768, 7168],
// one group an SM, 222 us, 6.4 TB/s).  From the checkpoint bound by latency, as the
// forward is: 18 instructions an element in half of the issue slots ([32768, 7168]
// 215 us, 5.5 TB/s).
template <typename TX, typename TY, bool MULTI, bool CKPT, bool ANY, bool CLUSTER>
__global__ void __launch_bounds__(NM_BLOCK) norm_backward_kernel(NormArgs a)
{
    extern __shared__ __align__(16) float shared[];  // weight; at the end dw and db
    __shared__ __align__(16) float2 parts[MULTI ? NM_MAX_GROUPS * 4 * NM_GROUP_WARPS : 1];
    __shared__ float trade[2][NM_MAX_RANKS][4];
    const float inv_n = 1.0f / (float)a.cols;
    const int rank = CLUSTER ? (int)cluster_ctarank() : 0, row_cols = (int)a.cols;
    if (CLUSTER) {
        a.end_x -= rank * a.part_cols;
        a.end_dy -= rank * a.part_cols;
        a.dy = static_cast<const TY *>(a.dy) + rank * a.part_cols;
        a.out = static_cast<TX *>(a.out) + rank * a.part_cols;
    }
    const int cols = CLUSTER ? take_part<TX, TY>(a, rank) : (int)a.cols, G = a.G;
    const Group g = group_of<MULTI>(G, parts);
    const int groups = CLUSTER ? 1 : MULTI ? blockDim.x / G : blockDim.x >> (31 - __clz(G));
    const int block = CLUSTER ? blockIdx.x / a.ranks : blockIdx.x;  // of those that split the rows
    // rows are counted in 32 bits: fewer registers, and below 2^31 + a few steps
    const uint32_t rows = (uint32_t)a.rows, step = (CLUSTER ? gridDim.x / a.ranks : gridDim.x) * groups;
    const int n = max(0, min(16, cols - g.t * 16));  // columns of the row in this thread's chunk

    uint32_t r = block * groups + g.id;
    using R = Ring<TX, TY, CKPT>;
    constexpr int S = ANY ? 0 : R::stages;  // 0: one row ahead in registers
    constexpr int ROWS = S ? R::rows : 1, AHEAD = S ? S - 1 : 1;
    RawBackward<TX, TY, CKPT, ANY> raw[ROWS];
    // statistics of the steps ahead, the next one first.  Two rows in whole
    // warps: one register, lanes 4 i to 4 i + 3 holding rstd and mean of row 0
    // and of row 1 (a value that is spilled on arrival is waited for).  0 for rows
    // past the last: their dy is 0, but times what another row's statistics make
    // of x = 0 it would be NaN where mean * rstd overflows
    constexpr bool LANES = MULTI && ROWS == 2;
    float mean_q[AHEAD][ROWS] = {}, rstd_q[AHEAD][ROWS] = {}, stat = 0.0f;
    uint32_t scale = 127;
    // %laneid: read where it is wanted, it costs no register over the loop
    const int lane = lane_id(), col0 = MULTI ? (g.t >> 5) * 512 : 0;  // of the warp's part of the row
    const CopyPlace cp{MULTI ? lane : g.t, MULTI ? 32 : G, MULTI ? 0 : lane / G};
    constexpr int DY = R::dy_slots, X = R::x_slots;
    // a warp's part of a row: 32 lanes of DY units, then of X
    const uint32_t ring = smem_u32(shared + 2 * G * 16) + (threadIdx.x >> 5) * (R::slots * 512);
    const uint32_t row_bytes = blockDim.x * R::slots * 16;
    const auto fetch = [&](uint32_t row0, int stage) {
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
            const uint32_t row = row0 + i * step;
            const bool live = row < rows;
            if constexpr (S == 0) {
                load_backward(a, row, g.t, live ? n : 0, raw[0]);
            } else {
                const uint32_t at = ring + (stage * ROWS + i) * row_bytes;
                const int have = live ? cols - col0 : 0;
                copy_ahead<DY, MULTI>(at, static_cast<const TY *>(a.dy) + row * a.ld_dy + col0,
                                      have * (int)sizeof(TY), cp, a.dy);
                if constexpr (CKPT)  // whole chunks of codes: a checkpoint's rows end on one
                    copy_ahead<X, MULTI>(at + DY * 512, a.q + row * a.ld_q + col0,
                                         have > 0 ? (have + 15) & ~15 : 0, cp, a.q);
                else
                    copy_ahead<X, MULTI>(at + DY * 512, static_cast<const TX *>(a.x) + row * a.ld_x + col0,
                                         have * (int)sizeof(TX), cp, a.x);
            }
            if (!LANES) {
                rstd_q[AHEAD - 1][i] = mean_q[AHEAD - 1][i] = 0.0f;
                if (live) {
                    rstd_q[AHEAD - 1][i] = __ldg(a.rstd + row);
                    if (!CKPT && !a.rms) mean_q[AHEAD - 1][i] = __ldg(a.mean + row);
                }
            }
        }
        if (LANES) {
            const uint32_t row = row0 + (lane >> 1 & 1) * step;
            stat = 0.0f;
            if (row < rows) stat = __ldg((lane & 1 && !CKPT && !a.rms ? a.mean : a.rstd) + row);
        }
        if (CKPT && S > 0) {
            // the scale byte of a block's two lanes: the even lane's of row 0, the odd lane's of row 1
            // (also where the odd lane's own columns are past the row)
            const uint32_t row = row0 + (lane & 1) * step;
            if (row < rows && (g.t & ~1) * 16 < cols) scale = __ldg(a.s + row * a.ld_s + (g.t >> 1));
        }
        if constexpr (S > 0) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto advance = [&]() {
#pragma unroll
        for (int q = 0; q + 1 < AHEAD; q++)
#pragma unroll
            for (int i = 0; i < ROWS; i++) {
                mean_q[q][i] = mean_q[q + 1][i];
                rstd_q[q][i] = rstd_q[q + 1][i];
            }
    };
#pragma unroll
    for (int q = 0; q < AHEAD; q++) {
        if (q) advance();
        fetch(r + q * ROWS * step, q);
    }
    params_to_shared(shared, a.weight, a.w_dtype, cols, G, 1.0f);
    if (MULTI)
        for (int i = threadIdx.x; i < NM_MAX_GROUPS * 4 * NM_GROUP_WARPS; i += blockDim.x)
            parts[i] = make_float2(0.0f, 0.0f);
    __syncthreads();
    if constexpr (CLUSTER) cluster_sync();  // all its blocks run: cluster_sum may write to them

    float2 dw[8] = {}, db[8] = {};  // of this thread's columns, over all its rows
    int slot = 0, stage = 0;
    // the groups of a warp go on until the first of them is done
    for (; (MULTI ? r : r - cp.sub) < rows; r += ROWS * step) {
        float gr[ROWS][16], xh[ROWS][16], rstd[ROWS];
        if constexpr (S > 0) {
            cp_async_wait<(S > 0 ? S - 2 : 0)>();
            __syncwarp();  // every lane's copies of these rows have arrived
#pragma unroll
            for (int i = 0; i < ROWS; i++) {
                const uint32_t at = ring + (stage * ROWS + i) * row_bytes;
#pragma unroll
                for (int j = 0; j < DY; j++) raw[i].dy.v[j] = copied<DY>(at, lane, j);
                if constexpr (CKPT) {
                    raw[i].q = copied<X>(at + DY * 512, lane, 0);
                    const uint32_t s = __shfl_sync(0xffffffffu, scale, (lane & ~1) | i);
                    raw[i].s = r + i * step < rows ? s : 127u;
                } else {
#pragma unroll
                    for (int j = 0; j < X; j++) raw[i].x.v[j] = copied<X>(at + DY * 512, lane, j);
                }
            }
            __syncwarp();  // and are read before their place is taken, a step later
        }
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
            float mean = mean_q[0][i];
            rstd[i] = rstd_q[0][i];
            if (LANES) {
                rstd[i] = __shfl_sync(0xffffffffu, stat, 2 * i);
                mean = CKPT || a.rms ? 0.0f : __shfl_sync(0xffffffffu, stat, 2 * i + 1);
            }
            dy16(raw[i], n, gr[i]);
            xhat16(a, raw[i], n, mean, rstd[i], xh[i]);
        }
        advance();
        if (S > 0 || (MULTI ? r : r - cp.sub) + step < rows) {
            // into the place of the step before this one
            fetch(r + AHEAD * ROWS * step, stage == 0 ? S - 1 : stage - 1);
            if (S > 0) stage = stage + 1 == S ? 0 : stage + 1;
        }
        float2 sum[ROWS], s1[ROWS] = {}, s2[ROWS] = {};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float4 w = param4(shared, G, g.t, q);
#pragma unroll
            for (int i = 0; i < ROWS; i++) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int j = 4 * q + 2 * h;
                    const float2 d = make_float2(gr[i][j], gr[i][j + 1]), x2 = make_float2(xh[i][j], xh[i][j + 1]);
                    dw[j / 2] = fma2(d, x2, dw[j / 2]);
                    db[j / 2] = add2(db[j / 2], d);
                    const float2 p = mul2(d, h ? make_float2(w.z, w.w) : make_float2(w.x, w.y));
                    s1[i] = add2(s1[i], p);
                    s2[i] = fma2(p, x2, s2[i]);
                    gr[i][j] = p.x, gr[i][j + 1] = p.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; i++) sum[i] = make_float2(s1[i].x + s1[i].y, s2[i].x + s2[i].y);
        row_sum<MULTI>(sum, G, g, slot);
        if constexpr (CLUSTER) {
            float t[2 * ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; i++) t[2 * i] = sum[i].x, t[2 * i + 1] = sum[i].y;
            cluster_sum(t, trade, slot, rank, a.ranks);
#pragma unroll
            for (int i = 0; i < ROWS; i++) sum[i] = make_float2(t[2 * i], t[2 * i + 1]);
        }
        slot ^= 1;
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
            const uint32_t row = r + i * step;
            const float c1 = a.rms ? 0.0f : -sum[i].x * inv_n * rstd[i], c2 = -sum[i].y * inv_n * rstd[i];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                float2 o = fma2(make_float2(gr[i][j], gr[i][j + 1]), make_float2(rstd[i], rstd[i]),
                                make_float2(c1, c1));
                o = fma2(make_float2(xh[i][j], xh[i][j + 1]), make_float2(c2, c2), o);
                gr[i][j] = o.x, gr[i][j + 1] = o.y;
            }
            store_chunk<ANY>(static_cast<TX *>(a.out) + row * a.ld_out + g.t * 16, gr[i],
                             row < rows ? cols - g.t * 16 : 0, a.w32, g.t, G);
        }
    }
    cp_async_wait<0>();
    if (!a.part) return;
    const int lanes = MULTI ? 32 : G;  // lanes that hold different columns
    if (!MULTI)
        for (int d = 16; d >= G; d >>= 1)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                dw[j] = add2(dw[j], make_float2(__shfl_xor_sync(0xffffffffu, dw[j].x, d),
                                                __shfl_xor_sync(0xffffffffu, dw[j].y, d)));
                db[j] = add2(db[j], make_float2(__shfl_xor_sync(0xffffffffu, db[j].x, d),
                                                __shfl_xor_sync(0xffffffffu, db[j].y, d)));
            }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sums' blocks may start
    // turns: the groups, or the warps of groups already added up in lanes
    const int turns = MULTI ? groups : blockDim.x >> 5, mine = MULTI ? g.id : threadIdx.x >> 5;
    float2 *sw = reinterpret_cast<float2 *>(shared), *sb = sw + G * 8;
    for (int turn = 0; turn < turns; turn++) {
        __syncthreads();
        if (turn == mine && lane < lanes) {
#pragma unroll
            for (int j = 0; j < 8; j++) {  // pair j of every chunk together: no bank conflicts
                const int at = j * G + g.t;
                sw[at] = turn ? add2(sw[at], dw[j]) : dw[j];
                sb[at] = turn ? add2(sb[at], db[j]) : db[j];
            }
        }
    }
    __syncthreads();
    float *part = a.part + (int64_t)block * 2 * row_cols;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
        const int at = ((c >> 1 & 7) * G + (c >> 4)) * 2 + (c & 1);
        part[c] = shared[at];
        part[row_cols + c] = shared[G * 16 + at];
    }
}

// The slices' sums: 32 columns a block, 32 threads a column that each add every
// 32nd slice, so that a few loads are the whole chain.  Launched while the
// kernel that writes the slices may still run (programmatic dependent launch):
// it waits for that kernel's end before it reads them.
constexpr int NM_SUM_LANES = 32;

__global__ void __launch_bounds__(NM_COLS * NM_SUM_LANES) norm_dw_sum_kernel(NormArgs a)
{
    __shared__ float2 part[NM_SUM_LANES][NM_COLS + 1];
    const int tc = threadIdx.x % NM_COLS, tr = threadIdx.x / NM_COLS;
    const int64_t c = (int64_t)blockIdx.x * NM_COLS + tc;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float dw = 0.0f, db = 0.0f;
    if (c < a.cols) {
#pragma unroll 4
        for (int i = tr; i < a.splits; i += NM_SUM_LANES) {
            dw += a.part[((int64_t)i * 2) * a.cols + c];
            db += a.part[((int64_t)i * 2 + 1) * a.cols + c];
        }
    }
    part[tr][tc] = make_float2(dw, db);
    __syncthreads();
    // warp w adds up column w, its lanes the slices
    float2 v = part[tc][tr];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d)));
    const int64_t out = (int64_t)blockIdx.x * NM_COLS + tr;
    if (tc == 0 && out < a.cols) {
        set_param(a.dweight, a.w_dtype, out, v.x);
        set_param(a.dbias, a.w_dtype, out, v.y);
    }
}

static fp8_status_t launch_dw_sum(NormArgs a, int slices, cudaStream_t st)
{
    a.splits = slices;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.cols + NM_COLS - 1) / NM_COLS));
    cfg.blockDim = dim3(NM_COLS * NM_SUM_LANES);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, norm_dw_sum_kernel, a);
    return check_launch();
}

static bool rows_aligned(const void *p, int64_t ld, int size, int al)
{
    return !p || (aligned(p, al) && ld * size % al == 0);
}

// Row groups, blocks and clusters of a launch.
struct Plan {
    bool multi;      // groups of several warps
    int chunks, G;   // chunks a thread, threads a group
    int ranks;       // blocks that share a row
    int part_cols;   // columns of a block
    unsigned threads, grid;
    int slices;      // of the rows, one a block (or cluster): slices of the workspace too
};

// Dynamic shared memory of a launch, and the most that any launch of the kernel
// takes: NM_BLOCK threads, of which a row of up to 32 threads' chunks needs the
// parameters of no more than these.
static constexpr int forward_shared(int chunks, int G, bool bias)
{
    return chunks * G * 16 * (int)sizeof(float) * (bias ? 2 : 1);
}

static constexpr int forward_shared_most(bool multi) { return forward_shared(2, multi ? NM_BLOCK : 32, true); }

template <typename TX, typename TY, bool CKPT, bool ANY>
static constexpr int backward_shared(int G, int threads)
{
    using R = Ring<TX, TY, CKPT>;
    return 2 * G * 16 * (int)sizeof(float) + (ANY ? 0 : R::stages * R::rows * R::slots * 16 * threads);
}

template <typename TX, typename TY, bool CKPT, bool ANY>
static constexpr int backward_shared_most(bool multi)
{
    return backward_shared<TX, TY, CKPT, ANY>(multi ? NM_BLOCK : 32, NM_BLOCK);
}

// 48 KB without asking, the kernel's own few KB among them.
constexpr int NM_SHARED_FREE = 40 * 1024;

// Lets a kernel's launches take more than that.  The limit belongs to the kernel
// and device, not to a launch, and other host threads may be about to launch with
// it: it is set once, to the most that any launch takes, and never lowered.
template <auto KERNEL, int MOST>
static bool allow_shared()
{
    constexpr int MAX_DEVICES = 64;
    static std::atomic<bool> allowed[MAX_DEVICES];
    static_assert(MOST + 8 * 1024 <= 227 * 1024, "more than a block can have");
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < MAX_DEVICES && allowed[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST) != cudaSuccess) return false;
    if (dev < MAX_DEVICES) allowed[dev].store(true, std::memory_order_release);
    return true;
}

// Blocks (of one to an SM) that run at once in clusters of `ranks`, in
// clusters.  The SMs of a GPC are no multiple of 4 or 8, so it is fewer than the
// SMs would give: a grid for all SMs leaves clusters for a second wave ([2048,
// 20480] backward: 137 us with 38 clusters, 82 with those that fit).  Asked once
// per device, with the largest launch a cluster makes.
static int clusters_at_once(int ranks)
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

// `chunks` chunks a thread where a warp's lanes do not cover the row (one where
// they do).  Few rows are spread over the SMs before a second group joins a
// block.  `small`: a kernel of one chunk and part-warp groups takes 64 registers,
// two blocks an SM.
static Plan make_plan(int64_t rows, int64_t cols, int chunks, bool small = false)
{
    Plan p;
    p.ranks = 1;
    while ((int64_t)NM_PART * chunks * p.ranks < cols) p.ranks *= 2;
    // whole warps of columns, so that only the last block has fewer
    const int64_t share = (cols + p.ranks - 1) / p.ranks, whole = 512 * chunks;
    p.part_cols = (int)(p.ranks == 1 ? cols : (share + whole - 1) / whole * whole);
    const int need = (p.part_cols + 15) / 16;
    p.chunks = need > 32 ? chunks : 1;
    p.multi = need > 32 * p.chunks;
    int groups;
    if (p.multi) {
        p.G = (need + 32 * p.chunks - 1) / (32 * p.chunks) * 32;
        groups = NM_BLOCK / p.G;
    } else {
        p.G = 2;  // at least two lanes: a checkpoint block's halves
        while (p.G * p.chunks < need) p.G *= 2;
        groups = NM_BLOCK / p.G;
    }
    const int64_t per_sm = (rows + num_sms() - 1) / num_sms();
    if (groups > per_sm) groups = (int)per_sm;
    if (!p.multi) groups = (groups * p.G + 31) / 32 * 32 / p.G;  // whole warps
    if (groups < 1 || p.ranks > 1) groups = 1;
    p.threads = (unsigned)(groups * p.G);
    const int64_t most = (int64_t)clusters_at_once(p.ranks) * (small && p.chunks == 1 && !p.multi ? 2 : 1);
    const int64_t blocks = (rows + groups - 1) / groups;
    p.slices = (int)(blocks < most ? blocks : most);
    p.grid = (unsigned)(p.slices * p.ranks);
    return p;
}

template <auto KERNEL, int MOST>
static fp8_status_t launch(const Plan &p, int smem, NormArgs a, cudaStream_t st)
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

template <typename TX, typename TY, bool CKPT, bool ANY>
static fp8_status_t launch_backward_as(NormArgs a, cudaStream_t st)
{
    const Plan p = make_plan(a.rows, a.cols, 1);
    const int smem = backward_shared<TX, TY, CKPT, ANY>(p.G, (int)p.threads);
    constexpr int narrow = backward_shared_most<TX, TY, CKPT, ANY>(false);
    constexpr int wide = backward_shared_most<TX, TY, CKPT, ANY>(true);
    const bool grads = a.dweight || a.dbias;
    if (!grads) a.part = nullptr;
    fp8_status_t rc;
    if (p.ranks > 1) rc = launch<norm_backward_kernel<TX, TY, true, CKPT, ANY, true>, wide>(p, smem, a, st);
    else if (p.multi) rc = launch<norm_backward_kernel<TX, TY, true, CKPT, ANY, false>, wide>(p, smem, a, st);
    else rc = launch<norm_backward_kernel<TX, TY, false, CKPT, ANY, false>, narrow>(p, smem, a, st);
    return rc == FP8_OK && grads ? launch_dw_sum(a, p.slices, st) : rc;  // no sums of slices never written
}

template <typename TX, typename TY>
static fp8_status_t launch_backward(NormArgs a, cudaStream_t st)
{
    if (a.rows == 0)  // gradients of zero: no slices to add
        return a.dweight || a.dbias ? launch_dw_sum(a, 0, st) : FP8_OK;
    const auto all_aligned = [&](int al) {
        return rows_aligned(a.dy, a.ld_dy, sizeof(TY), al) && rows_aligned(a.out, a.ld_out, sizeof(TX), al) &&
               rows_aligned(a.x, a.ld_x, sizeof(TX), al);
    };
    a.w32 = all_aligned(32);
    a.end_dy = rows_end(a.ld_dy, a.rows, a.cols);
    a.end_x = rows_end(a.ld_x, a.rows, a.cols);
    const bool any = !all_aligned(16);
    if (a.x && any) return launch_backward_as<TX, TY, false, true>(a, st);
    if (a.x) return launch_backward_as<TX, TY, false, false>(a, st);
    if (any) return launch_backward_as<TX, TY, true, true>(a, st);
    return launch_backward_as<TX, TY, true, false>(a, st);
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
    if (rows < 0 || cols < 1 || rows > INT32_MAX) return FP8_ERR_INVALID_ARG;
    if (cols > NM_MAX_COLS) return FP8_ERR_UNSUPPORTED;
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
    return NORM_TYPES(launch_backward, x_dtype, y_dtype, a, static_cast<cudaStream_t>(stream));
}
