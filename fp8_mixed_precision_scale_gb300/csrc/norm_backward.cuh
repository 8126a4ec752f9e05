// norm_backward.cuh -- the norms' backward kernels and their launch, for the
// translation units that have them with and without the gradient past the norm.
#pragma once

#include "norm.cuh"

namespace fp8gb {

constexpr int NM_COLS = 32;            // columns of a block of the last sums

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
    const void *dsum;       // backward: gradient that reaches x past the norm, of x's type
    int64_t ld_dsum, end_dsum;
};

__device__ __forceinline__ void set_param(void *p, int dtype, int64_t i, float v)
{
    if (!p) return;
    if (dtype == FP8_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == FP8_DTYPE_F16) static_cast<__half *>(p)[i] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = from_f32<__nv_bfloat16>(v);
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
//
// RES adds dsum, the gradient of x that does not come through the norm.  The ring has
// no room for it and the registers none while the sums are made: its lines are
// fetched into L2 with the rows ahead and read once the sums are there.  Two rows of it
// beside two rows of gradients spill in the aligned forms of 16-bit dy (bf16 132 bytes
// stored and 144 loaded a thread, from the checkpoint 100 and 116, rows of one warp 140
// and 136, in a cluster up to 168 and 148; fp16 alike; fp32 sums from the checkpoint up
// to 336 and 240); so do unaligned fp32 sums (up to 284 and 180), aligned ones from x
// do not.  [8192, 4096] bf16 60 us from x, 58 from the checkpoint, against 40 and 38
// without dsum, 69 and 67 with a separate addition; [32768, 7168] 374 and 368 (222 and
// 215; 417 and 410).
template <typename TX, typename TY, bool MULTI, bool CKPT, bool ANY, bool CLUSTER, bool RES = false>
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
        if (RES) {
            a.end_dsum -= rank * a.part_cols;
            a.dsum = static_cast<const TX *>(a.dsum) + rank * a.part_cols;
        }
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
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < ROWS; i++)
                if (row0 + i * step < rows && n > 0)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const TX *>(a.dsum) +
                                                                  (row0 + i * step) * a.ld_dsum + g.t * 16));
        }
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
        Raw<TX, ANY> past[RES ? ROWS : 1];
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < ROWS; i++) {
                const uint32_t row = r + i * step;
                const int64_t at = (int64_t)row * a.ld_dsum + g.t * 16;
                load_chunk<ANY>(static_cast<const TX *>(a.dsum) + at, row < rows ? n : 0, a.w32, at, a.end_dsum,
                                past[i]);
            }
        }
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
            if constexpr (RES) {
                float t[16];
                unpack16(past[i], t);
#pragma unroll
                for (int j = 0; j < 16; j++) gr[i][j] += t[j];
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

static __global__ void __launch_bounds__(NM_COLS * NM_SUM_LANES) norm_dw_sum_kernel(NormArgs a)
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

template <typename TX, typename TY, bool CKPT, bool ANY, bool RES>
static fp8_status_t launch_backward_as(NormArgs a, cudaStream_t st)
{
    const Plan p = make_plan(a.rows, a.cols, 1);
    const int smem = backward_shared<TX, TY, CKPT, ANY>(p.G, (int)p.threads);
    constexpr int narrow = backward_shared_most<TX, TY, CKPT, ANY>(false);
    constexpr int wide = backward_shared_most<TX, TY, CKPT, ANY>(true);
    const bool grads = a.dweight || a.dbias;
    if (!grads) a.part = nullptr;
    fp8_status_t rc;
    if (p.ranks > 1) rc = launch<norm_backward_kernel<TX, TY, true, CKPT, ANY, true, RES>, wide>(p, smem, a, st);
    else if (p.multi) rc = launch<norm_backward_kernel<TX, TY, true, CKPT, ANY, false, RES>, wide>(p, smem, a, st);
    else rc = launch<norm_backward_kernel<TX, TY, false, CKPT, ANY, false, RES>, narrow>(p, smem, a, st);
    return rc == FP8_OK && grads ? launch_dw_sum(a, p.slices, st) : rc;  // no sums of slices never written
}

template <typename TX, typename TY, bool RES>
static fp8_status_t launch_backward(NormArgs a, cudaStream_t st)
{
    if (a.rows == 0)  // gradients of zero: no slices to add
        return a.dweight || a.dbias ? launch_dw_sum(a, 0, st) : FP8_OK;
    const auto all_aligned = [&](int al) {
        return rows_aligned(a.dy, a.ld_dy, sizeof(TY), al) && rows_aligned(a.out, a.ld_out, sizeof(TX), al) &&
               rows_aligned(a.x, a.ld_x, sizeof(TX), al) && rows_aligned(a.dsum, a.ld_dsum, sizeof(TX), al);
    };
    a.w32 = all_aligned(32);
    a.end_dy = rows_end(a.ld_dy, a.rows, a.cols);
    a.end_x = rows_end(a.ld_x, a.rows, a.cols);
    a.end_dsum = rows_end(a.ld_dsum, a.rows, a.cols);
    const bool any = !all_aligned(16);
    if (a.x && any) return launch_backward_as<TX, TY, false, true, RES>(a, st);
    if (a.x) return launch_backward_as<TX, TY, false, false, RES>(a, st);
    if (any) return launch_backward_as<TX, TY, true, true, RES>(a, st);
    return launch_backward_as<TX, TY, true, false, RES>(a, st);
}

inline fp8_status_t check_codes(const void *q, int64_t ld_q, const void *s, int64_t ld_s, int64_t cols)
{
    if (!q || !s || ld_q < ckpt_width(cols) || ld_s < ckpt_width(cols) / FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    return ld_q % FP8_MX_BLOCK != 0 || !aligned(q, FP8_MX_BLOCK) ? FP8_ERR_ALIGNMENT : FP8_OK;
}

// What forward and backward check alike: sizes, kind, types (x of type xt on
// one side of the norm, y of type yt on the other), parameter pointers.
inline fp8_status_t check_common(int64_t rows, int64_t cols, int kind, int xt, int yt, int wt, const void *w,
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

inline fp8_status_t check_fmt(int fmt)
{
    if (fmt == FP8_E4M3FNUZ || fmt == FP8_E5M2FNUZ) return FP8_ERR_UNSUPPORTED;
    return fmt == FP8_E4M3FN || fmt == FP8_E5M2 ? FP8_OK : FP8_ERR_INVALID_ARG;
}

// Checks and launch of the backward; RES: with dsum.
template <bool RES>
static fp8_status_t norm_backward(const void *dy, int y_dtype, int64_t ld_dy, const void *x, int64_t ld_x,
                                  const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                  const void *dsum, int64_t ld_dsum, int64_t rows, int64_t cols, int kind,
                                  const float *mean, const float *rstd, const void *weight, int w_dtype, void *dx,
                                  int x_dtype, int64_t ld_dx, void *dweight, void *dbias, void *workspace,
                                  int64_t workspace_bytes, void *stream)
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
        if (RES && (rc = check_tensor(dsum, x_dtype, ld_dsum, cols)) != FP8_OK) return rc;
        if (!rstd || (x && kind == FP8_NORM_LAYER && !mean)) return FP8_ERR_INVALID_ARG;
        rc = x ? check_tensor(x, x_dtype, ld_x, cols) : check_codes(q, ld_q, s, ld_s, cols);
        if (rc != FP8_OK) return rc;
        if (RES && starts_at_any(dx, {dy, x, q, s, dsum, mean, rstd, weight})) return FP8_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.x = x;
    a.ld_x = ld_x;
    a.dsum = dsum;
    a.ld_dsum = ld_dsum;
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
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_dtype == FP8_DTYPE_BF16) return launch_backward<__nv_bfloat16, __nv_bfloat16, RES>(a, st);
    if (x_dtype == FP8_DTYPE_F16) return launch_backward<__half, __half, RES>(a, st);
    if (y_dtype == FP8_DTYPE_BF16) return launch_backward<float, __nv_bfloat16, RES>(a, st);
    if (y_dtype == FP8_DTYPE_F16) return launch_backward<float, __half, RES>(a, st);
    return launch_backward<float, float, RES>(a, st);
}

}  // namespace fp8gb
