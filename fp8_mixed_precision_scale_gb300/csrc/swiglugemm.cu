// swiglugemm.cu -- the matrix products on either side of a SwiGLU with the
// SwiGLU (or its backward) in their epilogue.
//
//   forward   gate = A W_gate^T, up = A W_up^T,  h = silu(gate) up
//   backward  dh = A B^T,  d_gate = dh up (s + silu (1 - s)),  d_up = dh silu,
//             s = sigma(gate), with gate and up as the forward kept them
//
// FP8 operands with MX block scales (tcgen05.mma kind::mxf8f6f4, the scales in
// tensor memory) or per-tensor / per-row scales (kind::f8f6f4, applied in the
// epilogue); fp32 accumulation.  gate, up and dh live in the accumulators and in
// registers alone: what is written is h (d_gate | d_up) as the 8-bit operand of
// the next product, in either layout, or in bf16, and of gate | up what the
// backward needs, in 8 bits or bf16.
//
// Design (GB300, sm_103a): persistent, warp-specialised, one CTA of 384 threads
// per SM.
//   warp 0     TMA producer: a 128 x 128-byte tile of A and two of B (forward:
//              128 gate rows and the 128 up rows of the same columns of h) per
//              stage of a four-stage ring, and for MX their scale blocks.
//   warp 1     MMA issuer: M = 128, N = 256, K = 32; gate in accumulator columns
//              0 .. 127, up in 128 .. 255, so that one thread of the epilogue
//              finds both of an element of h in its own TMEM lane.
//   warp 2     MX: copies each stage's scale blocks into the stage's own TMEM
//              columns, ahead of the MMA thread.
//   warps 4-11 epilogue: warp w has TMEM lane quarter w % 4 (32 rows) and half of
//              the columns.  A thread has one row: blocks of 32 columns, their
//              maxima and codes need no other thread.  The transposed layout's
//              blocks are 32 rows of a column, a warp's rows exactly: they go
//              through the warp's shared-memory staging, 16 columns at a time.
// With per-row scales two accumulators overlap the epilogue and the next tile's
// main loop.  MX scales take part of TMEM, which leaves one accumulator: each
// epilogue thread first takes its 128 columns into registers and releases it.
// For that the epilogue's warps take registers from the others (setmaxnreg).
// Every mbarrier wait is bounded (about 2 s); a wait that gives up records the
// device error word, drains what is in flight, releases TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"

namespace fp8gb {
namespace sg {

constexpr int BM = 128;
constexpr int BB = 128;  // rows of one of a stage's two B tiles
constexpr int BK = 128;
constexpr int UMMA_K = 32;
constexpr int STAGES = 4;
constexpr int EPI_WARPS = 8;
constexpr int EPI_FIRST = 4;  // their first warp: a warpgroup of its own for the registers
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
// registers a thread at launch, and after the split: 128 * 56 + 256 * 224 = 384 * 168
constexpr int REGS = 168, REGS_OTHER = 56, REGS_EPI = 224;
static_assert(128 * REGS_OTHER + 32 * EPI_WARPS * REGS_EPI <= THREADS * REGS, "registers");
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = 2 * BB * BK;
constexpr int SF_BLOCK = 512;  // scale words of 128 rows in one K tile
constexpr uint32_t TMEM_COLS = 512;
// MX: one accumulator at column 0, per stage 4 columns of A's scales and 8 of B's
constexpr uint32_t SFA_COL = 256, SFB_COL = 288;
static_assert(SFA_COL + 4 * STAGES <= SFB_COL && SFB_COL + 8 * STAGES <= TMEM_COLS, "scale columns");
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;

// Staging of a warp: 32 rows x 16 columns of fp32, rows 20 words apart and the
// second 16 rows 16 words further, so that neither the row writes (16 bytes a
// thread) nor the column reads (two columns' halves a warp) meet a bank twice.
constexpr int STAGE_WORDS = 31 * 20 + 16 + 16;
__device__ __forceinline__ int stage_word(int row) { return row * 20 + (row & 16); }

struct Smem {
    static constexpr int a_off = 0;
    static constexpr int b_off = STAGES * A_BYTES;
    static constexpr int sfa_off = b_off + STAGES * B_BYTES;
    static constexpr int sfb_off = sfa_off + STAGES * SF_BLOCK;
    static constexpr int bar_off = sfb_off + STAGES * 2 * SF_BLOCK;
    static constexpr int n_bars = 3 * STAGES + 2 + 2 + 2;
    static constexpr int slot_off = bar_off + n_bars * 8;
    static constexpr int stage_off = (slot_off + 16 + 127) / 128 * 128;
    static constexpr int total = stage_off + EPI_WARPS * STAGE_WORDS * 4;
};
constexpr int SMEM_BYTES = 1024 + Smem::total;
static_assert(SMEM_BYTES + 1024 <= 227 * 1024, "smem");

struct Params {
    int64_t M, F;       // rows; columns of h
    int64_t K;          // contraction
    const float *sa, *sb;
    int sa_row, sb_row;  // per row, else one of the tensor
    const uint8_t *sA, *sB;
    int64_t rsA, rsB;    // scale rows of A's and B's layouts
    int32_t b1_row;      // forward: row of B where up starts
    int64_t b1_srow;     // ... and its scale row
    int num_m, num_n, num_k, m_fastest;
    int64_t tiles;
    // bf16: h (forward) or d_gate | d_up (backward), up at column F
    uint16_t *out;
    int64_t ld_out;
    int out32;  // its rows and halves start on 32-byte boundaries
    // gate | up in bf16 (up at column F) or as a checkpoint; written by the forward, read by the backward
    uint16_t *gate_up;
    int64_t ld_gu;
    int gu32;
    uint8_t *cq, *cs;
    int64_t ld_cq, ld_cs;
    int cfmt;
    int64_t W;  // columns of a part of the checkpoint
    // 8 bits
    int fmt;
    const float *scale_in;  // per-tensor recipe
    float *amax_out, *scale_inv;
    uint8_t *q_row, *s_row, *q_col, *s_col;
    int64_t ld_row, ld_col, rs_row, rs_col;
    int64_t Fr;  // columns of h that q_row has (backward: of each half; zeros from F on)
    int q32;     // q_row's rows and halves start on 32-byte boundaries
    unsigned int *err;
};

__device__ __forceinline__ uint4 encode(const float (&v)[16], float inv, int fmt)
{
    return fmt == FP8_E5M2 ? encode16<FP8_E5M2>(v, inv) : encode16<FP8_E4M3FN>(v, inv);
}

__device__ __forceinline__ uint32_t mx_code_of(uint32_t amax_bits, int fmt)
{
    return fmt == FP8_E5M2 ? mx_code<FP8_E5M2>(amax_bits) : mx_code<FP8_E4M3FN>(amax_bits);
}

__device__ __forceinline__ float amax16(const float (&v)[16], float m)  // NaN if any is
{
#pragma unroll
    for (int j = 0; j < 16; j++) m = max_nan(m, fabsf(v[j]));
    return m;
}

// n (0, 16 or 32) codes, or their first n.
__device__ __forceinline__ void put_codes(uint8_t *p, const uint4 &lo, const uint4 &hi, int n, int w32)
{
    if (n >= 32 && w32) {
        st_32b(p, lo, hi);
    } else {
        if (n > 0) *reinterpret_cast<uint4 *>(p) = lo;
        if (n > 16) *reinterpret_cast<uint4 *>(p + 16) = hi;
    }
}

__device__ __forceinline__ void put_bf16(uint16_t *p, const float (&v)[2][16], int n, int w32)
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (n <= 16 * i) break;
        uint4 w[2];
#pragma unroll
        for (int j = 0; j < 2; j++)
            w[j] = make_uint4(pack_bf16x2(v[i][8 * j], v[i][8 * j + 1]), pack_bf16x2(v[i][8 * j + 2], v[i][8 * j + 3]),
                              pack_bf16x2(v[i][8 * j + 4], v[i][8 * j + 5]),
                              pack_bf16x2(v[i][8 * j + 6], v[i][8 * j + 7]));
        if (w32) {
            st_32b(p + 16 * i, w[0], w[1]);
        } else {
            *reinterpret_cast<uint4 *>(p + 16 * i) = w[0];
            *reinterpret_cast<uint4 *>(p + 16 * i + 8) = w[1];
        }
    }
}

// 32 columns of an 8-bit result.  A thread has row `row` (of a warp's 32 from
// row0 on; `live`: inside the matrix; values outside the data are 0).
//   oc, n_row   first column in q_row and how many of the 32 it has (0, 16, 32)
//   cc, n_col   first row in q_col, likewise
// The scale bytes of rows and columns behind the data are the zeros that a
// zero block's code is, and lie inside the 128-row blocks of the scale layout.
// PAD: they are written for all 32 columns (where the layouts' padding is this
// tile's alone).
template <bool MX, bool PAD>
__device__ __forceinline__ void put_8bit(const Params &p, const float (&v)[2][16], int64_t row, bool live,
                                         int64_t row0, int64_t oc, int n_row, int64_t cc, int n_col, float scale,
                                         float *stage, int lane, float &amax)
{
    if (!MX) amax = amax16(v[1], amax16(v[0], amax));
    if (p.q_row && (PAD || n_row > 0)) {
        float inv = scale;
        if (MX) {
            const uint32_t code = mx_code_of(__float_as_uint(amax16(v[1], amax16(v[0], 0.0f))), p.fmt);
            p.s_row[4 * mx_scale_word(oc >> 7, row, p.rs_row) + (oc >> 5 & 3)] = (uint8_t)code;
            inv = mx_inv_scale(code);
        }
        if (live)
            put_codes(p.q_row + row * p.ld_row + oc, encode(v[0], inv, p.fmt), encode(v[1], inv, p.fmt), n_row, p.q32);
    }
    if (p.q_col && (PAD || n_col > 0)) {
        const int c = lane & 15, h = lane >> 4;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            float4 *w = reinterpret_cast<float4 *>(stage + stage_word(lane));
#pragma unroll
            for (int j = 0; j < 4; j++)
                w[j] = make_float4(v[i][4 * j], v[i][4 * j + 1], v[i][4 * j + 2], v[i][4 * j + 3]);
            __syncwarp();
            float t[16];
#pragma unroll
            for (int j = 0; j < 16; j++) t[j] = stage[stage_word(16 * h + j) + c];
            const bool have = 16 * i + c < n_col;
            float inv = scale;
            if (MX) {
                float m = amax16(t, 0.0f);
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
                const uint32_t code = mx_code_of(__float_as_uint(m), p.fmt);
                inv = mx_inv_scale(code);
                if (h == 0 && (PAD || have))
                    p.s_col[4 * mx_scale_word(row0 >> 7, cc + 16 * i + c, p.rs_col) + (row0 >> 5 & 3)] = (uint8_t)code;
            }
            const int64_t r = row0 + 16 * h;
            const uint4 q = encode(t, inv, p.fmt);
            if (have) {
                uint8_t *dst = p.q_col + (cc + 16 * i + c) * p.ld_col + r;
                if (r + 16 <= p.M) {
                    *reinterpret_cast<uint4 *>(dst) = q;
                } else if (!MX) {  // MX: whole blocks of 32 rows
                    const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (r + j < p.M) dst[j] = (uint8_t)(qw[j >> 2] >> (8 * (j & 3)));
                }
            }
            __syncwarp();
        }
    }
}

// 16 or 32 bf16 (n of them; zeros after) of a row.
__device__ __forceinline__ void get_bf16(const uint16_t *p, int n, float (&v)[2][16])
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        Raw16<__nv_bfloat16> r;
        r.v[0] = r.v[1] = make_uint4(0, 0, 0, 0);
        if (n > 16 * i) load16(reinterpret_cast<const __nv_bfloat16 *>(p) + 16 * i, 16, false, r);
        unpack16(r, v[i]);
    }
}

// The block of 32 from a checkpoint.
__device__ __forceinline__ void get_kept(const uint8_t *q, const uint8_t *s, bool live, int fmt, float (&v)[2][16])
{
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    uint32_t code = 127;
    if (live) {
        ld_stream_32b(q, lo, hi);
        code = __ldg(s);
    }
    const float x = ckpt_scale(code);
    if (fmt == FP8_E5M2) {
        decode16<FP8_E5M2>(lo, x, v[0]);
        decode16<FP8_E5M2>(hi, x, v[1]);
    } else {
        decode16<FP8_E4M3FN>(lo, x, v[0]);
        decode16<FP8_E4M3FN>(hi, x, v[1]);
    }
}

// 32 accumulator columns as fp32, with the operands' scales (`col`: of B, for
// its row of column j of the 32 at lane j) and 0 where there is no data.
template <bool MX>
__device__ __forceinline__ void from_acc(const uint32_t (&r)[32], float sa, float col, bool per_col, bool live, int n,
                                         float (&v)[2][16])
{
#pragma unroll
    for (int j = 0; j < 32; j++) {
        float f = __uint_as_float(r[j]);
        if (!MX) f = f * sa * (per_col ? __shfl_sync(0xffffffffu, col, j) : col);
        v[j >> 4][j & 15] = live && j < n ? f : 0.0f;
    }
}

// 32 columns of h from its gate and up (forward).
template <bool MX>
__device__ __forceinline__ void forward_unit(const Params &p, float (&g)[2][16], float (&u)[2][16], int64_t row,
                                             bool live, int64_t row0, int64_t c, int n, float scale, float *stage,
                                             int lane, float &amax)
{
    if (p.gate_up && live) {
        uint16_t *dst = p.gate_up + row * p.ld_gu + c;
        put_bf16(dst, g, n, p.gu32);
        put_bf16(dst + p.F, u, n, p.gu32);
    }
    if (p.cq && live && c < p.W) {
        const uint32_t a = ckpt_code(__float_as_uint(amax16(g[1], amax16(g[0], 0.0f))), p.cfmt);
        const uint32_t b = ckpt_code(__float_as_uint(amax16(u[1], amax16(u[0], 0.0f))), p.cfmt);
        const float ia = ckpt_inv_scale(a), ib = ckpt_inv_scale(b);
        uint8_t *q = p.cq + row * p.ld_cq + c, *s = p.cs + row * p.ld_cs + (c >> 5);
        st_32b(q, encode(g[0], ia, p.cfmt), encode(g[1], ia, p.cfmt));
        st_32b(q + p.W, encode(u[0], ib, p.cfmt), encode(u[1], ib, p.cfmt));
        s[0] = (uint8_t)a;
        s[p.W >> 5] = (uint8_t)b;
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float2 e, sg, si;
            silu2(make_float2(g[i][j], g[i][j + 1]), e, sg, si);
            si = mul2(si, make_float2(u[i][j], u[i][j + 1]));
            g[i][j] = si.x, g[i][j + 1] = si.y;
        }
    if (p.out && live) put_bf16(p.out + row * p.ld_out + c, g, n, p.out32);
    if (p.q_row || p.q_col)
        put_8bit<MX, MX>(p, g, row, live, row0, c, n, c, n, scale, stage, lane, amax);
}

// 32 columns of d_gate and d_up from dh (backward).
template <bool MX>
__device__ __forceinline__ void backward_unit(const Params &p, float (&d)[2][16], int64_t row, bool live,
                                              int64_t row0, int64_t c, int n, float scale, float *stage, int lane,
                                              float &amax)
{
    float g[2][16], u[2][16];
    if (p.gate_up) {
        const uint16_t *src = p.gate_up + row * p.ld_gu + c;
        get_bf16(src, live ? n : 0, g);
        get_bf16(src + p.F, live ? n : 0, u);
    } else {
        const uint8_t *q = p.cq + row * p.ld_cq + c, *s = p.cs + row * p.ld_cs + (c >> 5);
        const bool have = live && n > 0;
        get_kept(q, s, have, p.cfmt, g);
        get_kept(q + p.W, s + (p.W >> 5), have, p.cfmt, u);
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float2 dg, du, h;
            swiglu_grad2(make_float2(g[i][j], g[i][j + 1]), make_float2(u[i][j], u[i][j + 1]),
                         make_float2(d[i][j], d[i][j + 1]), dg, du, h);
            // columns behind the data: what stands in the checkpoint there is not read into the result
            const bool have = live && 16 * i + j < n;
            g[i][j] = have ? dg.x : 0.0f, g[i][j + 1] = have ? dg.y : 0.0f;
            u[i][j] = have ? du.x : 0.0f, u[i][j + 1] = have ? du.y : 0.0f;
        }
    if (p.out && live) {
        uint16_t *dst = p.out + row * p.ld_out + c;
        put_bf16(dst, g, n, p.out32);
        put_bf16(dst + p.F, u, n, p.out32);
    }
    if (p.q_row || p.q_col) {
        const int n_row = c < p.Fr ? (MX ? 32 : n) : 0;
        put_8bit<MX, false>(p, g, row, live, row0, c, n_row, c, n, scale, stage, lane, amax);
        put_8bit<MX, false>(p, u, row, live, row0, p.Fr + c, n_row, p.F + c, n, scale, stage, lane, amax);
    }
}

template <bool MX, bool BWD>
__global__ void __launch_bounds__(THREADS, 1)
    swiglu_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ Params p, uint32_t idesc)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem + Smem::a_off;
    uint8_t *sB = smem + Smem::b_off;
    uint8_t *sfa = smem + Smem::sfa_off;
    uint8_t *sfb = smem + Smem::sfb_off;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Smem::bar_off);
    uint64_t *full = bars;
    uint64_t *empty = bars + STAGES;
    uint64_t *sf_full = bars + 2 * STAGES;  // MX: the stage's scales are in TMEM
    uint64_t *tfull = bars + 3 * STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *done = tempty + 2;
    uint64_t *sf_done = done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Smem::slot_off);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int ACCS = MX ? 1 : 2;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sf_full[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], EPI_WARPS);
        }
        mbar_init(done, 1);
        mbar_init(sf_done, 1);
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const auto coords = [&](int64_t t, int &mb, int &nb) {
        const uint32_t tt = (uint32_t)t;  // tile counts are below 2^31
        if (p.m_fastest) {
            nb = (int)(tt / (uint32_t)p.num_m);
            mb = (int)(tt - (uint32_t)nb * (uint32_t)p.num_m);
        } else {
            mb = (int)(tt / (uint32_t)p.num_n);
            nb = (int)(tt - (uint32_t)mb * (uint32_t)p.num_n);
        }
    };
    const int last_steps = (int)((p.K - (int64_t)(p.num_k - 1) * BK + UMMA_K - 1) / UMMA_K);

    if (warp < EPI_FIRST) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (warp == 0 && lane == 0) {
            // ---------------- producer ----------------
            int stage = 0;
            uint32_t phase = 0, used = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                int mb, nb;
                coords(t, mb, nb);
                const int32_t b0 = nb * (BWD ? 2 * BB : BB), b1 = BWD ? b0 + BB : p.b1_row + b0;
                const int64_t s0 = b0, s1 = BWD ? b0 + BB : p.b1_srow + b0;
                // the last tile of an odd number of 128-row blocks has one
                const bool two = s1 < p.rsB;
                for (int kb = 0; kb < p.num_k; kb++) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1, WAIT_LIMIT_NS, p.err, ERR_PRODUCER_WAIT)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[stage], A_BYTES + B_BYTES + (MX ? (two ? 3 : 2) * SF_BLOCK : 0));
                    tma_load_2d(sA + stage * A_BYTES, &tmA, kb * BK, mb * BM, &full[stage]);
                    tma_load_2d(sB + stage * B_BYTES, &tmB, kb * BK, b0, &full[stage]);
                    tma_load_2d(sB + stage * B_BYTES + B_BYTES / 2, &tmB, kb * BK, b1, &full[stage]);
                    if (MX) {
                        bulk_load(sfa + stage * SF_BLOCK, p.sA + (kb * p.rsA + (int64_t)mb * BM) * 4, SF_BLOCK,
                                  &full[stage]);
                        bulk_load(sfb + stage * 2 * SF_BLOCK, p.sB + (kb * p.rsB + s0) * 4, SF_BLOCK, &full[stage]);
                        if (two)
                            bulk_load(sfb + stage * 2 * SF_BLOCK + SF_BLOCK, p.sB + (kb * p.rsB + s1) * 4, SF_BLOCK,
                                      &full[stage]);
                    }
                    used |= 1u << stage;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // copies in flight land before the block ends: the last of stage s is of
            // this round for the stages before `stage`, of the round before for the others
            for (int s = 0; s < STAGES; s++)
                if (used >> s & 1)
                    mbar_wait_bounded(&full[s], s < stage ? phase : phase ^ 1, WAIT_LIMIT_NS, p.err, ERR_TEARDOWN_WAIT);
        } else if (warp == 1 && lane == 0) {
            // ---------------- MMA issuer ----------------
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, WAIT_LIMIT_NS, p.err, ERR_MMA_WAIT)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc * 2 * BB);
                for (int kb = 0; kb < p.num_k; kb++) {
                    if (!mbar_wait_bounded(MX ? &sf_full[stage] : &full[stage], phase, WAIT_LIMIT_NS, p.err,
                                           ERR_MMA_WAIT)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(sA + stage * A_BYTES), b_addr = smem_u32(sB + stage * B_BYTES);
                    const int steps = kb == p.num_k - 1 ? last_steps : BK / UMMA_K;
                    for (int k = 0; k < steps; k++) {
                        const uint64_t ad = smem_desc_k128_sw128(a_addr + k * UMMA_K);
                        const uint64_t bd = smem_desc_k128_sw128(b_addr + k * UMMA_K);
                        if (MX)
                            mma_mxf8f6f4(d, ad, bd, idesc_sf_ids(idesc, (uint32_t)k, (uint32_t)k),
                                         tmem_base + SFA_COL + 4 * stage, tmem_base + SFB_COL + 8 * stage,
                                         (kb | k) != 0);
                        else
                            mma_f8f6f4(d, ad, bd, idesc, (kb | k) != 0);
                    }
                    mma_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                mma_commit(&tfull[acc]);
                if (++acc == ACCS) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
            mma_commit(done);  // all issued MMAs complete before TMEM is released
            mbar_wait_bounded(done, 0, WAIT_LIMIT_NS, p.err, ERR_TEARDOWN_WAIT);
        } else if (MX && warp == 2 && lane == 0) {
            // ---------------- scale copies ----------------
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                for (int kb = 0; kb < p.num_k; kb++) {
                    if (!mbar_wait_bounded(&full[stage], phase, WAIT_LIMIT_NS, p.err, ERR_MMA_WAIT)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ca = tmem_base + SFA_COL + 4 * stage, cb = tmem_base + SFB_COL + 8 * stage;
                    const uint32_t ra = smem_u32(sfa + stage * SF_BLOCK), rb = smem_u32(sfb + stage * 2 * SF_BLOCK);
                    tmem_cp_32x128b_x4(ca, smem_desc_sf(ra));
                    tmem_cp_32x128b_x4(cb, smem_desc_sf(rb));
                    tmem_cp_32x128b_x4(cb + 4, smem_desc_sf(rb + SF_BLOCK));
                    mma_commit(&sf_full[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            mma_commit(sf_done);  // every issued copy lands before TMEM is released
            mbar_wait_bounded(sf_done, 0, WAIT_LIMIT_NS, p.err, ERR_TEARDOWN_WAIT);
        }
    } else {
        // ---------------- epilogue ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        const int q = warp & 3, hb = (warp - EPI_FIRST) >> 2;
        float *stage = reinterpret_cast<float *>(smem + Smem::stage_off) + (warp - EPI_FIRST) * STAGE_WORDS;
        constexpr int UNITS = BWD ? 4 : 2;
        float scale = 1.0f, amax = 0.0f;
        if (!MX && p.scale_in) {
            scale = __ldg(p.scale_in);
            if (blockIdx.x == 0 && warp == EPI_FIRST && lane == 0) p.scale_inv[0] = recip_rn(scale);
        }
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x) {
            int mb, nb;
            coords(t, mb, nb);
            const int64_t row0 = (int64_t)mb * BM + q * 32, row = row0 + lane;
            const bool live = row < p.M;
            const int64_t c0 = (int64_t)nb * (BWD ? 2 * BB : BB) + hb * 32 * UNITS;  // this warp's columns of h
            float sa = 1.0f;
            if (!MX) sa = p.sa_row ? (live ? __ldg(p.sa + row) : 0.0f) : __ldg(p.sa);
            if (!mbar_wait_bounded(&tfull[acc], acc_phase, WAIT_LIMIT_NS, p.err, ERR_EPILOGUE_WAIT)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 2 * BB);
            // accumulator column of unit u's first (forward: gate's; up's is 128 further)
            const auto column = [&](int u) { return taddr + (uint32_t)(hb * 32 * UNITS + 32 * u); };
            const auto release = [&]() {
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[acc]);
            };
            uint32_t r[MX ? 4 : BWD ? 1 : 2][32];
            if constexpr (MX) {
#pragma unroll
                for (int u = 0; u < 4; u++)
                    tmem_ld_32x32b_x32(BWD ? column(u) : column(u & 1) + (u >> 1) * BB, r[u]);
                release();
            }
#pragma unroll
            for (int u = 0; u < UNITS; u++) {
                const int64_t c = c0 + 32 * u;
                const int n = (int)(p.F - c < 0 ? 0 : p.F - c < 32 ? p.F - c : 32);
                if constexpr (!MX) {
                    tmem_ld_32x32b_x32(column(u), r[0]);
                    if (!BWD) tmem_ld_32x32b_x32(column(u) + BB, r[BWD ? 0 : 1]);
                    if (u == UNITS - 1) release();
                    else tmem_ld_wait();
                }
                float g[2][16], up[2][16];
                float cg = 1.0f, cu = 1.0f;
                if (!MX) {
                    cg = cu = p.sb_row ? 0.0f : __ldg(p.sb);
                    if (p.sb_row && lane < n) {
                        cg = __ldg(p.sb + c + lane);
                        if (!BWD) cu = __ldg(p.sb + p.F + c + lane);
                    }
                }
                from_acc<MX>(r[MX ? u : 0], sa, cg, p.sb_row, live, n, g);
                if constexpr (BWD) {
                    backward_unit<MX>(p, g, row, live, row0, c, n, scale, stage, lane, amax);
                } else {
                    from_acc<MX>(r[MX ? 2 + u : 1], sa, cu, p.sb_row, live, n, up);
                    forward_unit<MX>(p, g, up, row, live, row0, c, n, scale, stage, lane, amax);
                }
            }
            if (MX && BWD && p.q_col && hb == 0 && nb == p.num_n - 1)  // scale rows behind the data
                for (int64_t i = 2 * p.F + lane; i < p.rs_col; i += 32)
                    p.s_col[4 * mx_scale_word(row0 >> 7, i, p.rs_col) + (row0 >> 5 & 3)] = 0;
            if (++acc == ACCS) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (!MX && p.amax_out) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
            if (lane == 0 && m) atomicMax(reinterpret_cast<unsigned int *>(p.amax_out), m);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

// 2D map over a row-major u8 matrix [rows][ld] of `cols` columns, box {128
// bytes, 128 rows}, 128-byte swizzle, zero fill out of bounds.
static bool make_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld)
{
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)BB};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// The limit of a kernel's dynamic shared memory, set once per device.
template <auto KERNEL>
static bool allow_shared()
{
    constexpr int MAX_DEVICES = 64;
    static std::atomic<bool> allowed[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < MAX_DEVICES && allowed[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess)
        return false;
    if (dev < MAX_DEVICES) allowed[dev].store(true, std::memory_order_release);
    return true;
}

template <bool MX, bool BWD>
static fp8_status_t launch(const void *A, int fa, int64_t lda, const void *B, int fb, int64_t ldb, int64_t b_rows,
                           Params p, void *stream)
{
    CUtensorMap ma, mb;
    if (!make_map(&ma, A, p.M, p.K, lda) || !make_map(&mb, B, b_rows, p.K, ldb)) return FP8_ERR_CUDA;
    constexpr auto kernel = swiglu_gemm_kernel<MX, BWD>;
    if (!allow_shared<kernel>()) return cuda_fail();
    constexpr int cols = BWD ? 2 * BB : BB;  // of h in a tile
    p.num_m = (int)((p.M + BM - 1) / BM);
    p.num_n = (int)((p.F + cols - 1) / cols);
    p.num_k = (int)((p.K + BK - 1) / BK);
    p.m_fastest = p.M <= b_rows;  // the smaller operand stays in L2
    p.tiles = (int64_t)p.num_m * p.num_n;
    if (p.tiles > INT32_MAX) return FP8_ERR_UNSUPPORTED;
    p.err = device_error_word();
    const uint32_t idesc = MX ? idesc_mxf8f6f4(fa, fb, BM, 2 * BB) : idesc_f8f6f4(fa, fb, BM, 2 * BB);
    const int64_t grid = p.tiles < num_sms() ? p.tiles : num_sms();
    kernel<<<(unsigned)grid, THREADS, SMEM_BYTES, static_cast<cudaStream_t>(stream)>>>(ma, mb, p, idesc);
    return check_launch();
}

static fp8_status_t check_format(int f)
{
    if (f == FP8_E4M3FNUZ || f == FP8_E5M2FNUZ) return FP8_ERR_UNSUPPORTED;
    return f == FP8_E4M3FN || f == FP8_E5M2 ? FP8_OK : FP8_ERR_INVALID_ARG;
}

static bool rows_of(const void *p, int64_t ld, int64_t half, int size, int al)
{
    return aligned(p, al) && ld * size % al == 0 && half * size % al == 0;
}

#define SG_TRY(x)                             \
    do {                                      \
        const fp8_status_t rc_ = (x);         \
        if (rc_ != FP8_OK) return rc_;        \
    } while (0)

// What all four entry points check of their operands and sizes; unit: of F and K.
static fp8_status_t check_operands(const void *A, int fa, int64_t lda, const void *B, int fb, int64_t ldb, int64_t M,
                                   int64_t F, int64_t K, int unit)
{
    if (M < 0 || F < 1 || K < 1 || M > INT32_MAX || K > INT32_MAX || F > INT32_MAX / 2 - 128)
        return FP8_ERR_INVALID_ARG;
    SG_TRY(check_format(fa));
    SG_TRY(check_format(fb));
    if (M > 0 && (!A || !B)) return FP8_ERR_INVALID_ARG;
    if (lda < K || ldb < K) return FP8_ERR_INVALID_ARG;
    if (F % unit != 0 || K % unit != 0 || lda % 16 != 0 || ldb % 16 != 0) return FP8_ERR_ALIGNMENT;
    return aligned(A, 16) && aligned(B, 16) ? FP8_OK : FP8_ERR_ALIGNMENT;
}

// bf16 [M][ld] of `halves` halves of F columns
static fp8_status_t set_bf16(const void *ptr, int64_t ld, int64_t F, int halves, uint16_t *&to, int64_t &ld_to,
                             int &wide)
{
    if (!ptr) return FP8_OK;
    if (ld < halves * F) return FP8_ERR_INVALID_ARG;
    if (ld % 8 != 0 || !aligned(ptr, 16)) return FP8_ERR_ALIGNMENT;
    to = static_cast<uint16_t *>(const_cast<void *>(ptr));
    ld_to = ld;
    wide = rows_of(ptr, ld, halves == 2 ? F : 0, 2, 32);
    return FP8_OK;
}

static fp8_status_t set_checkpoint(const void *q, int64_t ld_q, const void *s, int64_t ld_s, int fmt, Params &p)
{
    p.W = ckpt_width(p.F);
    if (!q && !s) return FP8_OK;
    if (!q || !s || ld_q < 2 * p.W || ld_s < 2 * p.W / FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    SG_TRY(check_format(fmt));
    if (ld_q % FP8_MX_BLOCK != 0 || !aligned(q, FP8_MX_BLOCK)) return FP8_ERR_ALIGNMENT;
    p.cq = static_cast<uint8_t *>(const_cast<void *>(q));
    p.cs = static_cast<uint8_t *>(const_cast<void *>(s));
    p.ld_cq = ld_q;
    p.ld_cs = ld_s;
    p.cfmt = fmt;
    return FP8_OK;
}

// The 8-bit outputs: rows of q_row are halves * Fr wide, q_colT has halves * F rows.
template <bool MX>
static fp8_status_t set_8bit(int fmt, int layouts, uint8_t *q_row, uint8_t *s_row, uint8_t *q_colT, int64_t ld_colT,
                             uint8_t *s_col, int halves, Params &p)
{
    if (layouts & ~(FP8_LAYOUT_ROW | FP8_LAYOUT_COLT)) return FP8_ERR_INVALID_ARG;
    p.Fr = MX && halves == 2 ? round_up_128(p.F) : p.F;
    p.rs_row = round_up_128(p.M);
    p.rs_col = round_up_128(halves * p.F);
    if (!layouts) return FP8_OK;
    SG_TRY(check_format(fmt));
    p.fmt = fmt;
    if (layouts & FP8_LAYOUT_ROW) {
        if (!q_row || (MX && !s_row)) return FP8_ERR_INVALID_ARG;
        if (!aligned(q_row, 16) || !aligned(s_row, 4)) return FP8_ERR_ALIGNMENT;
        p.q_row = q_row;
        p.s_row = s_row;
        p.ld_row = halves * p.Fr;
        p.q32 = rows_of(q_row, p.ld_row, halves == 2 ? p.Fr : 0, 1, 32);
    }
    if (layouts & FP8_LAYOUT_COLT) {
        if (!q_colT || (MX && !s_col) || ld_colT < p.M) return FP8_ERR_INVALID_ARG;
        if ((MX && p.M % FP8_MX_BLOCK != 0) || ld_colT % 16 != 0 || !aligned(q_colT, 16) || !aligned(s_col, 4))
            return FP8_ERR_ALIGNMENT;
        p.q_col = q_colT;
        p.s_col = s_col;
        p.ld_col = ld_colT;
    }
    return FP8_OK;
}

static fp8_status_t set_scales(const float *sa, int sa_mode, const float *sb, int sb_mode, Params &p)
{
    if (p.M > 0 && (!sa || !sb)) return FP8_ERR_INVALID_ARG;
    if ((sa_mode != FP8_SCALE_TENSOR && sa_mode != FP8_SCALE_PER_ROW) ||
        (sb_mode != FP8_SCALE_TENSOR && sb_mode != FP8_SCALE_PER_ROW))
        return FP8_ERR_INVALID_ARG;
    if (!aligned(sa, 4) || !aligned(sb, 4)) return FP8_ERR_ALIGNMENT;
    p.sa = sa;
    p.sb = sb;
    p.sa_row = sa_mode == FP8_SCALE_PER_ROW;
    p.sb_row = sb_mode == FP8_SCALE_PER_ROW;
    return FP8_OK;
}

static fp8_status_t set_delayed(int layouts, const float *scale_in, float *amax_out, float *scale_inv, Params &p)
{
    if (!layouts) return FP8_OK;
    if (!scale_in || !amax_out || !scale_inv) return FP8_ERR_INVALID_ARG;
    if (!aligned(scale_in, 4) || !aligned(amax_out, 4) || !aligned(scale_inv, 4)) return FP8_ERR_ALIGNMENT;
    p.scale_in = scale_in;
    p.amax_out = amax_out;
    p.scale_inv = scale_inv;
    return FP8_OK;
}

// MX operands: A's scale rows are M, B's `b_rows` (a multiple of 128).
static fp8_status_t set_mx(const uint8_t *sA, const uint8_t *sB, int64_t b_rows, Params &p)
{
    if (p.M > 0 && (!sA || !sB)) return FP8_ERR_INVALID_ARG;
    if (!aligned(sA, 16) || !aligned(sB, 16)) return FP8_ERR_ALIGNMENT;
    p.sA = sA;
    p.sB = sB;
    p.rsA = round_up_128(p.M);
    p.rsB = b_rows;
    return FP8_OK;
}

static Params sizes(int64_t M, int64_t F, int64_t K)
{
    Params p{};
    p.M = M;
    p.F = F;
    p.K = K;
    p.b1_row = (int32_t)F;
    p.b1_srow = round_up_128(F);
    return p;
}

}  // namespace sg
}  // namespace fp8gb

using namespace fp8gb;

extern "C" fp8_status_t fp8_swiglu_gemm(const uint8_t *A, int fa, int64_t lda, const uint8_t *W, int fw, int64_t ldw,
                                        int64_t M, int64_t F, int64_t K, const float *sa, int sa_mode,
                                        const float *sw, int sw_mode, int fmt, int layouts, const float *scale_in,
                                        float *amax_out, uint8_t *q_row, uint8_t *q_colT, int64_t ld_colT,
                                        float *scale_inv, void *h_bf16, int64_t ld_h, void *gate_up_bf16,
                                        int64_t ld_gu, int ckpt_fmt, uint8_t *q, int64_t ld_q, uint8_t *s,
                                        int64_t ld_s, void *stream)
{
    SG_TRY(sg::check_operands(A, fa, lda, W, fw, ldw, M, F, K, 16));
    sg::Params p = sg::sizes(M, F, K);
    SG_TRY(sg::set_scales(sa, sa_mode, sw, sw_mode, p));
    SG_TRY(sg::set_8bit<false>(fmt, layouts, q_row, nullptr, q_colT, ld_colT, nullptr, 1, p));
    SG_TRY(sg::set_delayed(layouts, scale_in, amax_out, scale_inv, p));
    SG_TRY(sg::set_bf16(h_bf16, ld_h, F, 1, p.out, p.ld_out, p.out32));
    SG_TRY(sg::set_bf16(gate_up_bf16, ld_gu, F, 2, p.gate_up, p.ld_gu, p.gu32));
    SG_TRY(sg::set_checkpoint(q, ld_q, s, ld_s, ckpt_fmt, p));
    if (!layouts && !p.out && !p.gate_up && !p.cq && M > 0) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch<false, false>(A, fa, lda, W, fw, ldw, 2 * F, p, stream);
}

extern "C" fp8_status_t fp8_mx_swiglu_gemm(const uint8_t *A, int fa, int64_t lda, const uint8_t *sA, const uint8_t *W,
                                           int fw, int64_t ldw, const uint8_t *sW, int64_t M, int64_t F, int64_t K,
                                           int fmt, int layouts, uint8_t *q_row, uint8_t *s_row, uint8_t *q_colT,
                                           int64_t ld_colT, uint8_t *s_col, void *h_bf16, int64_t ld_h,
                                           void *gate_up_bf16, int64_t ld_gu, int ckpt_fmt, uint8_t *q, int64_t ld_q,
                                           uint8_t *s, int64_t ld_s, void *stream)
{
    SG_TRY(sg::check_operands(A, fa, lda, W, fw, ldw, M, F, K, FP8_MX_BLOCK));
    sg::Params p = sg::sizes(M, F, K);
    SG_TRY(sg::set_mx(sA, sW, 2 * round_up_128(F), p));
    SG_TRY(sg::set_8bit<true>(fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, 1, p));
    SG_TRY(sg::set_bf16(h_bf16, ld_h, F, 1, p.out, p.ld_out, p.out32));
    SG_TRY(sg::set_bf16(gate_up_bf16, ld_gu, F, 2, p.gate_up, p.ld_gu, p.gu32));
    SG_TRY(sg::set_checkpoint(q, ld_q, s, ld_s, ckpt_fmt, p));
    if (!layouts && !p.out && !p.gate_up && !p.cq && M > 0) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch<true, false>(A, fa, lda, W, fw, ldw, 2 * F, p, stream);
}

extern "C" fp8_status_t fp8_swiglu_gemm_backward(const uint8_t *A, int fa, int64_t lda, const uint8_t *B, int fb,
                                                 int64_t ldb, int64_t M, int64_t F, int64_t K, const float *sa,
                                                 int sa_mode, const float *sb, int sb_mode, const void *gate_up_bf16,
                                                 int64_t ld_gu, const uint8_t *q, int64_t ld_q, const uint8_t *s,
                                                 int64_t ld_s, int ckpt_fmt, int fmt, int layouts,
                                                 const float *scale_in, float *amax_out, uint8_t *q_row,
                                                 uint8_t *q_colT, int64_t ld_colT, float *scale_inv,
                                                 void *d_gate_up_bf16, int64_t ld_d, void *stream)
{
    SG_TRY(sg::check_operands(A, fa, lda, B, fb, ldb, M, F, K, 16));
    sg::Params p = sg::sizes(M, F, K);
    SG_TRY(sg::set_scales(sa, sa_mode, sb, sb_mode, p));
    SG_TRY(sg::set_bf16(gate_up_bf16, ld_gu, F, 2, p.gate_up, p.ld_gu, p.gu32));
    SG_TRY(sg::set_checkpoint(q, ld_q, s, ld_s, ckpt_fmt, p));
    if (M > 0 && (p.gate_up != nullptr) == (p.cq != nullptr)) return FP8_ERR_INVALID_ARG;  // one of them
    SG_TRY(sg::set_8bit<false>(fmt, layouts, q_row, nullptr, q_colT, ld_colT, nullptr, 2, p));
    SG_TRY(sg::set_delayed(layouts, scale_in, amax_out, scale_inv, p));
    SG_TRY(sg::set_bf16(d_gate_up_bf16, ld_d, F, 2, p.out, p.ld_out, p.out32));
    if (!layouts && !p.out && M > 0) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch<false, true>(A, fa, lda, B, fb, ldb, F, p, stream);
}

extern "C" fp8_status_t fp8_mx_swiglu_gemm_backward(const uint8_t *A, int fa, int64_t lda, const uint8_t *sA,
                                                    const uint8_t *B, int fb, int64_t ldb, const uint8_t *sB,
                                                    int64_t M, int64_t F, int64_t K, const void *gate_up_bf16,
                                                    int64_t ld_gu, const uint8_t *q, int64_t ld_q, const uint8_t *s,
                                                    int64_t ld_s, int ckpt_fmt, int fmt, int layouts, uint8_t *q_row,
                                                    uint8_t *s_row, uint8_t *q_colT, int64_t ld_colT, uint8_t *s_col,
                                                    void *d_gate_up_bf16, int64_t ld_d, void *stream)
{
    SG_TRY(sg::check_operands(A, fa, lda, B, fb, ldb, M, F, K, FP8_MX_BLOCK));
    sg::Params p = sg::sizes(M, F, K);
    SG_TRY(sg::set_mx(sA, sB, round_up_128(F), p));
    SG_TRY(sg::set_bf16(gate_up_bf16, ld_gu, F, 2, p.gate_up, p.ld_gu, p.gu32));
    SG_TRY(sg::set_checkpoint(q, ld_q, s, ld_s, ckpt_fmt, p));
    if (M > 0 && (p.gate_up != nullptr) == (p.cq != nullptr)) return FP8_ERR_INVALID_ARG;  // one of them
    SG_TRY(sg::set_8bit<true>(fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, 2, p));
    SG_TRY(sg::set_bf16(d_gate_up_bf16, ld_d, F, 2, p.out, p.ld_out, p.out32));
    if (!layouts && !p.out && M > 0) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch<true, true>(A, fa, lda, B, fb, ldb, F, p, stream);
}
