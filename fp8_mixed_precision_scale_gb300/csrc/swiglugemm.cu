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
// Design (GB300, sm_103a): persistent, warp-specialised, one CTA of 384 threads per
// SM; from 129 rows on (and for some MX forwards of fewer, at the launch) CTA pairs
// with 256 x 256 tiles from 2-SM MMAs, each CTA staging
// its 128 rows of A and half of B (forward: the even one 128 gate rows, the odd one
// the 128 up rows of the same columns of h).
//   warp 0     TMA producer: the CTA's tiles of A and B, 128 bytes along K, per stage
//              of a five-stage ring (three with a single CTA, which stages both halves
//              of B; with half as many columns five again), and for MX their scale blocks.
//   warp 1     MMA issuer (the even CTA's): N = 256, K = 32; gate in accumulator
//              columns 0 .. 127, up in 128 .. 255, so that one thread of the epilogue
//              finds both of an element of h in its own TMEM lane.
//   warp 2     MX: copies each stage's scale blocks into the stage's own TMEM
//              columns, ahead of the MMA thread.
//   warps 4-11 epilogue: warp w has TMEM lane quarter w % 4 (32 rows) and half of
//              the columns, 32 at a time (a unit).  A thread has one row: blocks of 32
//              columns, their maxima and codes need no other thread.  The transposed
//              layout's blocks are 32 rows of a column, a warp's rows exactly: they go
//              through the warp's shared-memory staging.
// With per-row scales two accumulators overlap the epilogue and the next tile's
// main loop.  MX scales take part of TMEM, which leaves one accumulator: each
// epilogue thread first takes its 128 columns into registers and releases it.
// For that the epilogue's warps take registers from the others (setmaxnreg).
//
// 8192 rows, K = 4096, F = 14336, MX, times of single calls in us: forward with h in bf16
// 547 (3.52 PFLOP/s; the plain product of the same size 622), with both 8-bit layouts
// and the 8-bit gate | up 596; backward from the 8-bit gate | up to both layouts 443.
// The forward is bound by the tensor cores: a tile's MMAs take 11.0 us of 12.3.  The
// backward is bound by its epilogue and by what it shares with the MMAs, the shared
// memory's port: 14.1 us a tile by itself, 18.1 beside MMAs that take 11.4 by themselves.
// Its MX pairs spill, 60 bytes stored and 96 loaded a thread from the 8-bit gate | up, 88
// and 120 from bf16; no forward form does (12 bytes in one), nor does a backward with
// per-tensor or per-row scales.
// Steps that carried it: a loop over the units in place of four copies (instructions
// then stay in the cache: backward 1066 -> 549), no release at cluster scope when an
// accumulator is handed back (it waited for the stores of the tile before: forward
// 688 -> 599), the transposed layout 32 columns at once (backward 527 -> 452).
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
#include "swiglugemm.cuh"

namespace fp8gb {
namespace sg {

constexpr int BM = 128;  // rows of A a CTA stages, and of the result that it holds
constexpr int BK = 128;
constexpr int UMMA_K = 32;
constexpr int EPI_WARPS = 8;
constexpr int EPI_FIRST = 4;  // their first warp: a warpgroup of its own for the registers
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
// registers a thread at launch, and after the split: 128 * 40 + 256 * 232 = 384 * 168
constexpr int REGS = 168, REGS_OTHER = 40, REGS_EPI = 232;
static_assert(128 * REGS_OTHER + 32 * EPI_WARPS * REGS_EPI <= THREADS * REGS, "registers");
constexpr int A_BYTES = BM * BK;
constexpr int SF_BLOCK = 512;  // scale words of 128 rows in one K tile
constexpr uint32_t TMEM_COLS = 512;
// MX: one accumulator at column 0, per stage 4 columns of A's scales and 8 of B's
constexpr uint32_t SFA_COL = 256, SFB_COL = 288;
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;

// Staging of a warp: 32 rows x 32 columns of fp32.  Rows of 36 words: the row
// writes (16 bytes a thread) and the column reads meet no bank twice.
constexpr int STAGE_PITCH = 36;
constexpr int STAGE_WORDS = 32 * STAGE_PITCH;

// The three forms of a tile: CTA pairs, one CTA, and one CTA with half as many
// columns (not for the MX forward, whose gate and up rows would start inside their
// 128-row scale blocks).
enum { PAIR = 0, SINGLE = 1, NARROW = 2 };

template <int FORM>
struct Smem {
    static constexpr int half = FORM == NARROW ? 64 : 128;  // rows of one box of B, half a tile's columns of B
    static constexpr int stages = FORM == SINGLE ? 3 : 5;
    static constexpr int boxes = FORM == PAIR ? 1 : 2;      // of B a CTA stages
    static constexpr int b_bytes = boxes * half * BK;
    static constexpr int a_off = 0;
    static constexpr int b_off = stages * A_BYTES;
    static constexpr int sfa_off = b_off + stages * b_bytes;
    static constexpr int sfb_off = sfa_off + stages * SF_BLOCK;
    static constexpr int bar_off = sfb_off + stages * 2 * SF_BLOCK;
    static constexpr int n_bars = 3 * stages + 2 + 2 + 2;
    static constexpr int slot_off = bar_off + n_bars * 8;
    static constexpr int stage_off = (slot_off + 16 + 127) / 128 * 128;
    static constexpr int bytes = 1024 + stage_off + EPI_WARPS * STAGE_WORDS * 4;
    static_assert(SFA_COL + 4 * stages <= SFB_COL && SFB_COL + 8 * stages <= TMEM_COLS, "scale columns");
    static_assert(bytes + 1024 <= 227 * 1024, "smem");
};

enum { FORWARD = 0, BACKWARD_CKPT = 1, BACKWARD_BF16 = 2 };  // KIND: the backward's gate|up in 8 bits or bf16

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

// Where a thread of the epilogue stands in its tile.
struct Place {
    int64_t row, row0;  // its row, and its warp's first
    bool live;          // the row is inside the matrix
    int lane;
    float *stage;       // its warp's
};

// 32 columns of a result into the row layout; values outside the data are 0.
// oc, n: the first column in q_row, and how many of the 32 it has (0, 16, 32).
// MX: returns the block's scale code.
template <bool MX>
__device__ __forceinline__ uint32_t put_row(const Params &p, const float (&v)[2][16], const Place &t, int64_t oc,
                                            int n, float scale)
{
    uint32_t code = 0;
    float inv = scale;
    if (MX) {
        code = mx_code_of(__float_as_uint(amax32(v, 0.0f)), p.fmt);
        inv = mx_inv_scale(code);
    }
    if (t.live)
        put_codes(p.q_row + t.row * p.ld_row + oc, encode(v[0], inv, p.fmt), encode(v[1], inv, p.fmt), n, p.q32);
    return code;
}

// ... and into the transposed layout: cc, n the first row in q_col and how many of
// the 32 it has.  A lane takes a column.  PAD: the scale bytes of all 32 are
// written, zeros (a zero block's code) behind the data, where the layout's
// padding is this tile's alone.
template <bool MX, bool PAD>
__device__ __forceinline__ void put_col(const Params &p, const float (&v)[2][16], const Place &t, int64_t cc, int n,
                                        float scale)
{
    float4 *w = reinterpret_cast<float4 *>(t.stage + t.lane * STAGE_PITCH);
    __syncwarp();  // the columns before are read
#pragma unroll
    for (int j = 0; j < 8; j++)
        w[j] = make_float4(v[j >> 2][4 * j & 15], v[j >> 2][(4 * j & 15) + 1], v[j >> 2][(4 * j & 15) + 2],
                           v[j >> 2][(4 * j & 15) + 3]);
    __syncwarp();
    float x[2][16];
#pragma unroll
    for (int j = 0; j < 32; j++) x[j >> 4][j & 15] = t.stage[j * STAGE_PITCH + t.lane];
    const bool have = t.lane < n;
    const int64_t r = cc + t.lane;
    float inv = scale;
    if (MX) {
        const uint32_t code = mx_code_of(__float_as_uint(amax32(x, 0.0f)), p.fmt);
        inv = mx_inv_scale(code);
        if (PAD || have) p.s_col[4 * mx_scale_word(t.row0 >> 7, r, p.rs_col) + (t.row0 >> 5 & 3)] = (uint8_t)code;
    }
    if (have) {
        uint8_t *dst = p.q_col + r * p.ld_col + t.row0;
        const uint4 lo = encode(x[0], inv, p.fmt), hi = encode(x[1], inv, p.fmt);
        if (t.row0 + 32 <= p.M) {
            put_codes(dst, lo, hi, 32, p.c32);
        } else if (!MX) {  // MX: whole blocks of 32 rows
            const uint32_t qw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int j = 0; j < 32; j++)
                if (t.row0 + j < p.M) dst[j] = (uint8_t)(qw[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// What the backward reads of a unit of 32 columns of gate and of up.
template <int KIND>
struct Kept {
    uint4 q[4];  // codes: gate's, then up's
};
template <>
struct Kept<BACKWARD_BF16> {
    uint4 q[8];
};

// n: columns that the data has from c on (0, 16, 32); zeros after, and in rows
// outside the matrix.
template <int KIND>
__device__ __forceinline__ void get_kept(const Params &p, const Place &t, int64_t c, int n, Kept<KIND> &k)
{
    constexpr int N = sizeof(k.q) / sizeof(uint4) / 2;
    const bool have = t.live && n > 0;
#pragma unroll
    for (int i = 0; i < 2 * N; i++) k.q[i] = make_uint4(0, 0, 0, 0);
    if constexpr (KIND == BACKWARD_CKPT) {
        if (have) {
            const uint8_t *q = p.cq + t.row * p.ld_cq + c;
            ld_stream_32b(q, k.q[0], k.q[1]);
            ld_stream_32b(q + p.W, k.q[2], k.q[3]);
        }
    } else if (have) {
        const uint16_t *src = p.gate_up + t.row * p.ld_gu + c;
#pragma unroll
        for (int h = 0; h < 2; h++, src += p.F)
#pragma unroll
            for (int i = 0; i < N; i += 2)
                if (n > 8 * i) {
                    if (p.gu32) {
                        ld_stream_32b(src + 8 * i, k.q[N * h + i], k.q[N * h + i + 1]);
                    } else {
                        k.q[N * h + i] = ld_stream_16b(src + 8 * i);
                        k.q[N * h + i + 1] = ld_stream_16b(src + 8 * i + 8);
                    }
                }
    }
}

// Scale bytes of a warp's blocks of a checkpoint's part from column c on, for the row.
// Every row is a line of its own, whatever is read of it: a word at a time.
template <int UNITS>
__device__ __forceinline__ uint32_t kept_scales(const Params &p, const Place &t, int64_t c, int part)
{
    if (!t.live || c >= p.F) return 0;
    const uint8_t *s = p.cs + t.row * p.ld_cs + part * (p.W >> 5) + (c >> 5);
    if (p.cs4 && UNITS == 4) return __ldg(reinterpret_cast<const uint32_t *>(s));
    if (p.cs4 && UNITS == 2) return __ldg(reinterpret_cast<const uint16_t *>(s));
    uint32_t v = 0;
    for (int i = 0; i < UNITS && c + 32 * i < p.W; i++) v |= (uint32_t)__ldg(s + i) << (8 * i);
    return v;
}

// Half h (16 columns) of gate (w = 0) or up (w = 1); `scales`: their scale bytes.
template <int KIND>
__device__ __forceinline__ void kept16(const Params &p, const Kept<KIND> &k, const uint32_t (&scales)[2], int w, int h,
                                       float (&v)[16])
{
    if constexpr (KIND == BACKWARD_CKPT) {
        const float x = ckpt_scale(scales[w] & 0xFFu);
        if (p.cfmt == FP8_E5M2) decode16<FP8_E5M2>(k.q[2 * w + h], x, v);
        else decode16<FP8_E4M3FN>(k.q[2 * w + h], x, v);
    } else {
        Raw16<__nv_bfloat16> r;
        r.v[0] = k.q[4 * w + 2 * h], r.v[1] = k.q[4 * w + 2 * h + 1];
        unpack16(r, v);
    }
}

// 32 accumulator columns as fp32, with the operands' scales (`col`: lane j holds
// that of column j, or all the same one).
template <bool MX>
__device__ __forceinline__ void from_acc(const uint32_t (&r)[32], float sa, float col, bool per_col, float (&v)[2][16])
{
#pragma unroll
    for (int j = 0; j < 32; j++) {
        float f = __uint_as_float(r[j]);
        if (!MX) f = f * sa * (per_col ? __shfl_sync(0xffffffffu, col, j) : col);
        v[j >> 4][j & 15] = f;
    }
}

// Zeros where there is no data: rows outside the matrix, columns from n on.
__device__ __forceinline__ void mask32(float (&v)[2][16], bool live, int n)
{
#pragma unroll
    for (int j = 0; j < 32; j++) v[j >> 4][j & 15] = live && j < n ? v[j >> 4][j & 15] : 0.0f;
}

// What a unit of 32 columns of h leaves, from its gate and up (forward) or its dh
// and kept gate | up (backward).  Returns MX: its blocks' scale codes in the row
// layout (the backward's d_up in bits 8 to 15).  kept: the checkpoint's scale bytes
// (up's in bits 16 to 23).
template <bool MX>
__device__ __forceinline__ uint32_t forward_unit(const Params &p, float (&g)[2][16], float (&u)[2][16],
                                                 const Place &t, int64_t c, int n, float scale, float &amax,
                                                 uint32_t &kept)
{
    if (p.gate_up && t.live) {
        uint16_t *dst = p.gate_up + t.row * p.ld_gu + c;
        put_bf16(dst, g, n, p.gu32);
        put_bf16(dst + p.F, u, n, p.gu32);
    }
    if (p.cq && t.live && c < p.W) {
        const uint32_t a = ckpt_code(__float_as_uint(amax32(g, 0.0f)), p.cfmt);
        const uint32_t b = ckpt_code(__float_as_uint(amax32(u, 0.0f)), p.cfmt);
        const float ia = ckpt_inv_scale(a), ib = ckpt_inv_scale(b);
        uint8_t *q = p.cq + t.row * p.ld_cq + c;
        st_32b(q, encode(g[0], ia, p.cfmt), encode(g[1], ia, p.cfmt));
        st_32b(q + p.W, encode(u[0], ib, p.cfmt), encode(u[1], ib, p.cfmt));
        kept = a | b << 16;
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float2 e, sg, si;
            silu2_ftz(make_float2(g[i][j], g[i][j + 1]), e, sg, si);
            si = mul2(si, make_float2(u[i][j], u[i][j + 1]));
            g[i][j] = si.x, g[i][j + 1] = si.y;
        }
    if (p.out && t.live) put_bf16(p.out + t.row * p.ld_out + c, g, n, p.out32);
    if (!MX) amax = amax32(g, amax);
    uint32_t code = 0;
    if (p.q_row) code = put_row<MX>(p, g, t, c, n, scale);
    if (p.q_col && (MX || n > 0)) put_col<MX, MX>(p, g, t, c, n, scale);
    return code;
}

template <bool MX, int KIND>
__device__ __forceinline__ uint32_t backward_unit(const Params &p, float (&g)[2][16], const Kept<KIND> &kept,
                                                  const uint32_t (&scales)[2], const Place &t, int64_t c, int n, float scale, float &amax)
{
    float u[2][16];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        float kg[16], ku[16];
        kept16(p, kept, scales, 0, i, kg);
        kept16(p, kept, scales, 1, i, ku);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float2 e, sg, si;
            silu2_ftz(make_float2(kg[j], kg[j + 1]), e, sg, si);
            const float2 dh = make_float2(g[i][j], g[i][j + 1]);
            const float2 dg = mul2(mul2(dh, make_float2(ku[j], ku[j + 1])), fma2(si, mul2(e, sg), sg));
            const float2 du = mul2(dh, si);
            g[i][j] = dg.x, g[i][j + 1] = dg.y;
            u[i][j] = du.x, u[i][j + 1] = du.y;
        }
    }
    // what stands in the checkpoint behind the data is not read into the result
    if (n < 32 || t.row0 + 32 > p.M) {
        mask32(g, t.live, n);
        mask32(u, t.live, n);
    }
    if (p.out && t.live) {
        uint16_t *dst = p.out + t.row * p.ld_out + c;
        put_bf16(dst, g, n, p.out32);
        put_bf16(dst + p.F, u, n, p.out32);
    }
    if (!MX) amax = amax32(u, amax32(g, amax));
    uint32_t codes = 0;
    if (p.q_row) {
        const int m = c < p.Fr ? (MX ? 32 : n) : 0;
        codes = put_row<MX>(p, g, t, c, m, scale);
        codes |= put_row<MX>(p, u, t, p.Fr + c, m, scale) << 8;
    }
    if (p.q_col && n > 0) {
        put_col<MX, false>(p, g, t, c, n, scale);
        put_col<MX, false>(p, u, t, p.F + c, n, scale);
    }
    return codes;
}

template <bool MX, int FORM, int KIND>
__global__ void __launch_bounds__(THREADS, 1)
    swiglu_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                       const __grid_constant__ Params p, uint32_t idesc)
{
    using L = Smem<FORM>;
    constexpr int STAGES = L::stages, HALF = L::half;
    constexpr bool BWD = KIND != FORWARD, PAIRED = FORM == PAIR;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem + L::a_off;
    uint8_t *sB = smem + L::b_off;
    uint8_t *sfa = smem + L::sfa_off;
    uint8_t *sfb = smem + L::sfb_off;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bar_off);
    uint64_t *full = bars;
    uint64_t *empty = bars + STAGES;
    uint64_t *sf_full = bars + 2 * STAGES;  // MX: the stage's scales are in TMEM
    uint64_t *tfull = bars + 3 * STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *done = tempty + 2;
    uint64_t *sf_done = done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::slot_off);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIRED ? (int)cluster_ctarank() : 0;  // the even CTA leads
    const int64_t first = PAIRED ? blockIdx.x >> 1 : blockIdx.x, step = PAIRED ? gridDim.x >> 1 : gridDim.x;
    constexpr int ACCS = MX ? 1 : 2;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sf_full[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], (PAIRED ? 2 : 1) * EPI_WARPS);
        }
        mbar_init(done, 1);
        mbar_init(sf_done, 1);
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        if (MX) {
            prefetch_tensormap(&tmSA);
            prefetch_tensormap(&tmSB);
        }
    }
    if (warp == 1) {
        if (PAIRED) tmem_alloc_pair(tmem_slot, TMEM_COLS);
        else tmem_alloc(tmem_slot, TMEM_COLS);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIRED) cluster_sync();  // both CTAs' barriers are initialised before any remote use
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
        if (PAIRED) mb = 2 * mb + rank;  // this CTA's 128 rows
    };
    const int last_steps = (int)((p.K - (int64_t)(p.num_k - 1) * BK + UMMA_K - 1) / UMMA_K);

    if (warp < EPI_FIRST) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (warp == 0 && lane == 0) {
            // ---------------- producer (both CTAs) ----------------
            int stage = 0;
            uint32_t phase = 0, used = 0;
            bool ok = true;
            for (int64_t t = first; t < p.tiles && ok; t += step) {
                int mb, nb;
                coords(t, mb, nb);
                const int32_t y = mb * BM;
                // first rows of the tile's two boxes of B, and of their scales
                const int32_t b0 = nb * (BWD ? 2 * HALF : HALF), b1 = BWD ? b0 + HALF : p.b1_row + b0;
                const int32_t s1 = (BWD ? b0 + HALF : p.b1_srow + b0) & ~127;  // whole blocks (narrow: the first again)
                for (int kb = 0; kb < p.num_k; kb++) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1, WAIT_LIMIT_NS, p.err, ERR_PRODUCER_WAIT)) {
                        ok = false;
                        break;
                    }
                    constexpr uint32_t bytes = A_BYTES + L::b_bytes + (MX ? 3 * SF_BLOCK : 0);
                    uint8_t *a = sA + stage * A_BYTES, *b = sB + stage * L::b_bytes;
                    uint8_t *fa = sfa + stage * SF_BLOCK, *fb = sfb + stage * 2 * SF_BLOCK;
                    if constexpr (PAIRED) {  // both CTAs' copies count on the even one's barrier
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
                        const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
                        tma_load_2d_pair(a, &tmA, kb * BK, y, bar);
                        tma_load_2d_pair(b, &tmB, kb * BK, rank ? b1 : b0, bar);
                        if (MX) {
                            tma_load_2d_pair(fa, &tmSA, y, kb, bar);
                            tma_load_2d_pair(fb, &tmSB, b0, kb, bar);
                            tma_load_2d_pair(fb + SF_BLOCK, &tmSB, s1, kb, bar);
                        }
                    } else {
                        mbar_arrive_expect_tx(&full[stage], bytes);
                        tma_load_2d(a, &tmA, kb * BK, y, &full[stage]);
                        tma_load_2d(b, &tmB, kb * BK, b0, &full[stage]);
                        tma_load_2d(b + HALF * BK, &tmB, kb * BK, b1, &full[stage]);
                        if (MX) {
                            tma_load_2d(fa, &tmSA, y, kb, &full[stage]);
                            tma_load_2d(fb, &tmSB, b0, kb, &full[stage]);
                            tma_load_2d(fb + SF_BLOCK, &tmSB, s1, kb, &full[stage]);
                        }
                    }
                    used |= 1u << stage;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // copies in flight land before the block ends: the last of stage s is of
            // this turn of the ring for the stages before `stage`, of the one before for the others.
            // The even CTA's barriers count both CTAs' (the odd one waits at the end)
            if (rank == 0)
                for (int s = 0; s < STAGES; s++)
                    if (used >> s & 1)
                        mbar_wait_bounded(&full[s], s < stage ? phase : phase ^ 1, WAIT_LIMIT_NS, p.err,
                                          ERR_TEARDOWN_WAIT);
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ---------------- MMA issuer (even CTA) ----------------
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t t = first; t < p.tiles && ok; t += step) {
                if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, WAIT_LIMIT_NS, p.err, ERR_MMA_WAIT)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc * 2 * HALF);
                for (int kb = 0; kb < p.num_k; kb++) {
                    if (!mbar_wait_bounded(MX ? &sf_full[stage] : &full[stage], phase, WAIT_LIMIT_NS, p.err,
                                           ERR_MMA_WAIT)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_k128_sw128(smem_u32(sA + stage * A_BYTES));
                    const uint64_t bd = smem_desc_k128_sw128(smem_u32(sB + stage * L::b_bytes));
                    const uint32_t ca = tmem_base + SFA_COL + 4 * stage, cb = tmem_base + SFB_COL + 8 * stage;
                    const auto mma = [&](int k) {  // K = 32: the descriptors' addresses are in 16 bytes
                        const uint64_t a = ad + k * (UMMA_K >> 4), b = bd + k * (UMMA_K >> 4);
                        const uint32_t id = MX ? idesc_sf_ids(idesc, (uint32_t)k, (uint32_t)k) : idesc;
                        if constexpr (MX && PAIRED) mma_mxf8f6f4_pair(d, a, b, id, ca, cb, (kb | k) != 0);
                        else if constexpr (MX) mma_mxf8f6f4(d, a, b, id, ca, cb, (kb | k) != 0);
                        else if constexpr (PAIRED) mma_f8f6f4_pair(d, a, b, id, (kb | k) != 0);
                        else mma_f8f6f4(d, a, b, id, (kb | k) != 0);
                    };
                    if (kb < p.num_k - 1 || last_steps == BK / UMMA_K) {
#pragma unroll
                        for (int k = 0; k < BK / UMMA_K; k++) mma(k);
                    } else {
                        for (int k = 0; k < last_steps; k++) mma(k);
                    }
                    if (PAIRED) mma_commit_pair(&empty[stage], 0x3);
                    else mma_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (PAIRED) mma_commit_pair(&tfull[acc], 0x3);
                else mma_commit(&tfull[acc]);
                if (++acc == ACCS) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
            // all issued MMAs complete before TMEM is released
            if (PAIRED) mma_commit_pair_local(done);
            else mma_commit(done);
            mbar_wait_bounded(done, 0, WAIT_LIMIT_NS, p.err, ERR_TEARDOWN_WAIT);
        } else if (MX && warp == 2 && lane == 0 && rank == 0) {
            // ---------------- scale copies (even CTA) ----------------
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t t = first; t < p.tiles && ok; t += step) {
                for (int kb = 0; kb < p.num_k; kb++) {
                    if (!mbar_wait_bounded(&full[stage], phase, WAIT_LIMIT_NS, p.err, ERR_MMA_WAIT)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ca = tmem_base + SFA_COL + 4 * stage, cb = tmem_base + SFB_COL + 8 * stage;
                    const uint32_t ra = smem_u32(sfa + stage * SF_BLOCK), rb = smem_u32(sfb + stage * 2 * SF_BLOCK);
                    if constexpr (PAIRED) {
                        tmem_cp_32x128b_x4_pair(ca, smem_desc_sf(ra));
                        tmem_cp_32x128b_x4_pair(cb, smem_desc_sf(rb));
                        tmem_cp_32x128b_x4_pair(cb + 4, smem_desc_sf(rb + SF_BLOCK));
                        mma_commit_pair_local(&sf_full[stage]);
                    } else {
                        tmem_cp_32x128b_x4(ca, smem_desc_sf(ra));
                        tmem_cp_32x128b_x4(cb, smem_desc_sf(rb));
                        tmem_cp_32x128b_x4(cb + 4, smem_desc_sf(rb + SF_BLOCK));
                        mma_commit(&sf_full[stage]);
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // every issued copy lands before TMEM is released
            if (PAIRED) mma_commit_pair_local(sf_done);
            else mma_commit(sf_done);
            mbar_wait_bounded(sf_done, 0, WAIT_LIMIT_NS, p.err, ERR_TEARDOWN_WAIT);
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        const int q = warp & 3, hb = (warp - EPI_FIRST) >> 2;
        Place pl;
        pl.lane = lane;
        pl.stage = reinterpret_cast<float *>(smem + L::stage_off) + (warp - EPI_FIRST) * STAGE_WORDS;
        constexpr int UNITS = (BWD ? 2 * HALF : HALF) / 64;  // of 32 columns, a warp: it has half of the tile's
        float scale = 1.0f, amax = 0.0f;
        if (!MX && p.scale_in) {
            scale = __ldg(p.scale_in);
            if (blockIdx.x == 0 && warp == EPI_FIRST && lane == 0) p.scale_inv[0] = recip_rn(scale);
        }
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int64_t t = first; t < p.tiles; t += step) {
            int mb, nb;
            coords(t, mb, nb);
            pl.row0 = (int64_t)mb * BM + q * 32;
            pl.row = pl.row0 + lane;
            pl.live = pl.row < p.M;
            const int64_t c0 = (int64_t)nb * (BWD ? 2 * HALF : HALF) + hb * 32 * UNITS;  // this warp's columns of h
            const auto columns = [&](int u) {  // that the data has in unit u
                const int64_t n = p.F - c0 - 32 * u;
                return (int)(n < 0 ? 0 : n < 32 ? n : 32);
            };
            // a pair's second 128 rows may lie behind the padded rows too
            const int units = (int64_t)mb * BM < p.rs_row ? UNITS : 0;
            float sa = 1.0f;
            if (!MX) sa = p.sa_row ? (pl.live ? __ldg(p.sa + pl.row) : 0.0f) : __ldg(p.sa);
            Kept<KIND> kept;
            uint32_t scales[2] = {};
            if constexpr (BWD) get_kept<KIND>(p, pl, c0, columns(0), kept);
            if constexpr (KIND == BACKWARD_CKPT) {
                scales[0] = kept_scales<UNITS>(p, pl, c0, 0);
                scales[1] = kept_scales<UNITS>(p, pl, c0, 1);
            }
            if (!mbar_wait_bounded(&tfull[acc], acc_phase, WAIT_LIMIT_NS, p.err, ERR_EPILOGUE_WAIT)) break;
            tc_fence_after();
            // accumulator column of the warp's first unit (forward: gate's; up's is 128 further)
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 2 * HALF + hb * 32 * UNITS);
            const auto release = [&]() {
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    // only TMEM is handed over: a release at cluster scope would wait for the stores
                    // of the tile before (2 us a tile)
                    if (PAIRED)
                        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                                         mapa_shared(smem_u32(&tempty[acc]), 0))
                                     : "memory");
                    else mbar_arrive(&tempty[acc]);
                }
            };
            constexpr int R = MX ? (BWD ? UNITS : 2 * UNITS) : BWD ? 1 : 2;
            uint32_t r[R][32];  // forward: gate and up of a unit, then of the next
            if constexpr (MX) {
#pragma unroll
                for (int i = 0; i < R; i++)
                    tmem_ld_32x32b_x32(BWD ? taddr + 32 * i : taddr + 32 * (i >> 1) + (i & 1) * HALF, r[i]);
                release();
            }
            uint32_t codes = 0, codes_up = 0;
            // a loop, not copies of it: four units' instructions do not stay in the instruction cache
#pragma unroll 1
            for (int u = 0; u < UNITS; u++) {
                const int64_t c = c0 + 32 * u;
                const int n = columns(u);
                if constexpr (!MX) {
                    tmem_ld_32x32b_x32(taddr + 32 * u, r[0]);
                    if (!BWD) tmem_ld_32x32b_x32(taddr + 32 * u + HALF, r[BWD ? 0 : 1]);
                    if (u == UNITS - 1) release();
                    else tmem_ld_wait();
                }
                if (u < units) {
                    float cg = 1.0f, cu = 1.0f;
                    if (!MX) {
                        cg = cu = p.sb_row ? 0.0f : __ldg(p.sb);
                        if (p.sb_row && lane < n) {
                            cg = __ldg(p.sb + c + lane);
                            if (!BWD) cu = __ldg(p.sb + p.F + c + lane);
                        }
                    }
                    float v[2][16];
                    from_acc<MX>(r[0], sa, cg, p.sb_row, v);
                    uint32_t code;
                    if constexpr (BWD) {
                        const Kept<KIND> now = kept;
                        if (u + 1 < UNITS) get_kept<KIND>(p, pl, c + 32, columns(u + 1), kept);
                        code = backward_unit<MX, KIND>(p, v, now, scales, pl, c, n, scale, amax);
                        scales[0] >>= 8, scales[1] >>= 8;
                    } else {
                        float up[2][16];
                        from_acc<MX>(r[R > 1 ? 1 : 0], sa, cu, p.sb_row, up);
                        if (n < 32 || pl.row0 + 32 > p.M) {
                            mask32(v, pl.live, n);
                            mask32(up, pl.live, n);
                        }
                        uint32_t k = 0;
                        code = forward_unit<MX>(p, v, up, pl, c, n, scale, amax, k);
                        scales[0] |= k << (8 * u);
                    }
                    codes |= (code & 0xFFu) << (8 * u);
                    codes_up |= (code >> 8) << (8 * u);
                }
                if constexpr (MX) {  // the next unit's accumulators
#pragma unroll
                    for (int i = 0; i + (BWD ? 1 : 2) < R; i++)
#pragma unroll
                        for (int j = 0; j < 32; j++) r[i][j] = r[i + (BWD ? 1 : 2)][j];
                }
            }
            if (!BWD && p.cq && pl.live && units && c0 < p.W) {  // the units' scale bytes of gate, and of up
                uint8_t *s = p.cs + pl.row * p.ld_cs + (c0 >> 5);
                const bool two = UNITS == 2 && c0 + 32 < p.W;
#pragma unroll
                for (int i = 0; i < 2; i++, s += p.W >> 5) {
                    const uint32_t v = scales[0] >> (16 * i);
                    if (two && p.cs4) {
                        *reinterpret_cast<uint16_t *>(s) = (uint16_t)v;
                    } else {
                        s[0] = (uint8_t)v;
                        if (two) s[1] = (uint8_t)(v >> 8);
                    }
                }
            }
            if (MX && units && p.q_row && (!BWD || c0 < p.Fr)) {
                // the row's scale bytes of its columns: a word of the layout, or a part of one
                const int64_t at = 4 * mx_scale_word(c0 >> 7, pl.row, p.rs_row) + (c0 >> 5 & 3);
                const auto put = [&](uint8_t *dst, uint32_t v) {
                    if (UNITS == 4) *reinterpret_cast<uint32_t *>(dst) = v;
                    else if (UNITS == 2) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)v;
                    else *dst = (uint8_t)v;
                };
                put(p.s_row + at, codes);
                if (BWD) put(p.s_row + at + 4 * (p.Fr >> 7) * p.rs_row, codes_up);
            }
            if (MX && BWD && units && p.q_col && hb == 0 && nb == p.num_n - 1)  // scale rows behind the data
                for (int64_t i = 2 * p.F + lane; i < p.rs_col; i += 32)
                    p.s_col[4 * mx_scale_word(pl.row0 >> 7, i, p.rs_col) + (pl.row0 >> 5 & 3)] = 0;
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
    if (PAIRED) cluster_sync();  // no CTA leaves while its peer may still touch its shared memory or TMEM
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (PAIRED) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
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
// bytes, box_rows}, 128-byte swizzle, zero fill out of bounds.
static bool make_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 2D map over MX scales [kt][rows] of words (rows: of the padded layout), box 128
// words: one 128-row block of a K tile.
static bool make_scale_map(CUtensorMap *map, const void *base, int64_t kt, int64_t rows)
{
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)rows, (cuuint64_t)kt};
    cuuint64_t strides[1] = {(cuuint64_t)rows * 4};
    cuuint32_t box[2] = {(cuuint32_t)BM, 1};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Lets a kernel's launches take their shared memory, and gives the pairs (or
// blocks) that run at once; asked once per device.  0: it failed.
template <auto KERNEL, int FORM>
static int at_once()
{
    constexpr int MAX_DEVICES = 64;
    static std::atomic<int> known[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return 0;
    int n = known[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<FORM>::bytes) != cudaSuccess)
        return 0;
    n = num_sms();
    if (FORM == PAIR) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() / 2 * 2));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = Smem<FORM>::bytes;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = num_sms() / 2;
        }
    }
    known[dev].store(n, std::memory_order_release);
    return n;
}

template <bool MX, int FORM, int KIND>
static fp8_status_t launch_as(const Operands &o, Params p, cudaStream_t st)
{
    using L = Smem<FORM>;
    CUtensorMap ma, mb, msa = {}, msb = {};
    if (!make_map(&ma, o.A, p.M, p.K, o.lda, BM) || !make_map(&mb, o.B, o.b_rows, p.K, o.ldb, L::half))
        return FP8_ERR_CUDA;
    constexpr int rows = FORM == PAIR ? 2 * BM : BM, cols = KIND == FORWARD ? L::half : 2 * L::half;  // of a tile of h
    p.num_m = (int)((p.M + rows - 1) / rows);
    p.num_n = (int)((p.F + cols - 1) / cols);
    p.num_k = (int)((p.K + BK - 1) / BK);
    if (MX && (!make_scale_map(&msa, o.sA, p.num_k, o.rsA) || !make_scale_map(&msb, o.sB, p.num_k, o.rsB)))
        return FP8_ERR_CUDA;
    p.m_fastest = p.M <= o.b_rows;  // the smaller operand stays in L2
    p.tiles = (int64_t)p.num_m * p.num_n;
    if (p.tiles > INT32_MAX) return FP8_ERR_UNSUPPORTED;
    p.err = device_error_word();
    constexpr auto kernel = swiglu_gemm_kernel<MX, FORM, KIND>;
    const int most = at_once<kernel, FORM>();
    if (!most) return cuda_fail();
    constexpr int n = 2 * L::half;  // columns of an MMA
    const uint32_t idesc = MX ? idesc_mxf8f6f4(o.fa, o.fb, rows, n) : idesc_f8f6f4(o.fa, o.fb, rows, n);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.tiles < most ? p.tiles : most) * (FORM == PAIR ? 2 : 1)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = L::bytes;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = FORM == PAIR;
    cudaLaunchKernelEx(&cfg, kernel, ma, mb, msa, msb, p, idesc);
    return check_launch();
}

// Pairs from 129 rows on, as the plain products: MX forward, backward in us, pairs
// against single CTAs: F = 14336, K = 4096 at 160 rows 36.7, 33.0 against 45.5, 35.6, at
// 1024 rows 81.6, 72.5 against 110.2, 78.2; F = 2048, K = 7168 at 160 rows 27.2, 39.0
// against 31.4, 41.6.  Narrow tiles where all of them run at once: more SMs share the
// columns, and a tile's epilogue is half as long (F = 2048: backward of K = 128, 96 rows
// 15.4 against 9.7 us, K = 7168 37.4 against 26.6, 512 rows 39.5 against 32.7;
// forward with per-row scales, K = 128 7.7 against 5.6, K = 7168 23.1 against 21.0).
template <bool MX, int KIND>
static fp8_status_t launch(const Operands &o, const Params &p, void *stream)
{
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    fp8_status_t rc;
    if (KIND == FORWARD && few_rows(o, p, MX, st, rc)) return rc;
    if constexpr (!MX || KIND != FORWARD) {
        constexpr int cols = KIND == FORWARD ? 64 : 128;
        if ((p.M + BM - 1) / BM * ((p.F + cols - 1) / cols) <= num_sms()) return launch_as<MX, NARROW, KIND>(o, p, st);
    }
    // The MX forward of few rows: a pair's CTAs fetch half of B each, which a long
    // contraction is bound by, while twice the CTAs still run at once. One CTA a tile against
    // a pair, 96 rows, F = 2048, one layout: K = 7168 28.2 and 24.1 us, K = 4096 18.5 and
    // 16.9, K = 1024 9.2 and 9.2 (both layouts 10.8 and 11.3), K = 128 6.7 and 7.2. With 112
    // tiles (F = 14336, K = 4096, 16 rows), more than half of the SMs: 32.8 and 38.4.
    const bool halves = MX && KIND == FORWARD && p.K >= 2048 && (p.F + 127) / 128 <= num_sms() / 2;
    return p.M > BM || halves ? launch_as<MX, PAIR, KIND>(o, p, st) : launch_as<MX, SINGLE, KIND>(o, p, st);
}

template <bool MX>
static fp8_status_t launch_backward(const Operands &o, const Params &p, void *stream)
{
    return p.gate_up ? launch<MX, BACKWARD_BF16>(o, p, stream) : launch<MX, BACKWARD_CKPT>(o, p, stream);
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
    p.cs4 = aligned(s, 4) && ld_s % 4 == 0 && p.W % 128 == 0;
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
        if (p.M > 0 && (!q_row || (MX && !s_row))) return FP8_ERR_INVALID_ARG;
        if (!aligned(q_row, 16) || !aligned(s_row, 4)) return FP8_ERR_ALIGNMENT;
        p.q_row = q_row;
        p.s_row = s_row;
        p.ld_row = halves * p.Fr;
        p.q32 = rows_of(q_row, p.ld_row, halves == 2 ? p.Fr : 0, 1, 32);
    }
    if (layouts & FP8_LAYOUT_COLT) {
        if ((p.M > 0 && (!q_colT || (MX && !s_col))) || ld_colT < p.M) return FP8_ERR_INVALID_ARG;
        if ((MX && p.M % FP8_MX_BLOCK != 0) || ld_colT % 16 != 0 || !aligned(q_colT, 16) || !aligned(s_col, 4))
            return FP8_ERR_ALIGNMENT;
        p.q_col = q_colT;
        p.s_col = s_col;
        p.ld_col = ld_colT;
        p.c32 = rows_of(q_colT, ld_colT, 0, 1, 32);
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

// MX scales: A's have M rows, B's `b_rows` (a multiple of 128).
static fp8_status_t set_mx(const uint8_t *sA, const uint8_t *sB, int64_t b_rows, int64_t M, Operands &o)
{
    if (M > 0 && (!sA || !sB)) return FP8_ERR_INVALID_ARG;
    if (!aligned(sA, 16) || !aligned(sB, 16)) return FP8_ERR_ALIGNMENT;
    o.sA = sA;
    o.sB = sB;
    o.rsA = round_up_128(M);
    o.rsB = b_rows;
    return FP8_OK;
}

static Params sizes(int64_t M, int64_t F, int64_t K)
{
    Params p{};
    p.M = M;
    p.F = F;
    p.K = K;
    p.b1_row = (int32_t)F;
    p.b1_srow = (int32_t)round_up_128(F);
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
    return sg::launch<false, sg::FORWARD>({A, W, fa, fw, lda, ldw, 2 * F}, p, stream);
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
    sg::Operands o{A, W, fa, fw, lda, ldw, 2 * F};
    SG_TRY(sg::set_mx(sA, sW, 2 * round_up_128(F), M, o));
    SG_TRY(sg::set_8bit<true>(fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, 1, p));
    SG_TRY(sg::set_bf16(h_bf16, ld_h, F, 1, p.out, p.ld_out, p.out32));
    SG_TRY(sg::set_bf16(gate_up_bf16, ld_gu, F, 2, p.gate_up, p.ld_gu, p.gu32));
    SG_TRY(sg::set_checkpoint(q, ld_q, s, ld_s, ckpt_fmt, p));
    if (!layouts && !p.out && !p.gate_up && !p.cq && M > 0) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch<true, sg::FORWARD>(o, p, stream);
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
    if (M > 0 && starts_at_any(p.out, {A, B, sa, sb, p.gate_up, p.cq, p.cs, p.scale_in})) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch_backward<false>({A, B, fa, fb, lda, ldb, F}, p, stream);
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
    sg::Operands o{A, B, fa, fb, lda, ldb, F};
    SG_TRY(sg::set_mx(sA, sB, round_up_128(F), M, o));
    SG_TRY(sg::set_bf16(gate_up_bf16, ld_gu, F, 2, p.gate_up, p.ld_gu, p.gu32));
    SG_TRY(sg::set_checkpoint(q, ld_q, s, ld_s, ckpt_fmt, p));
    if (M > 0 && (p.gate_up != nullptr) == (p.cq != nullptr)) return FP8_ERR_INVALID_ARG;  // one of them
    SG_TRY(sg::set_8bit<true>(fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, 2, p));
    SG_TRY(sg::set_bf16(d_gate_up_bf16, ld_d, F, 2, p.out, p.ld_out, p.out32));
    if (!layouts && !p.out && M > 0) return FP8_ERR_INVALID_ARG;
    if (M > 0 && starts_at_any(p.out, {A, B, sA, sB, p.gate_up, p.cq, p.cs})) return FP8_ERR_INVALID_ARG;
    if (M == 0) return FP8_OK;
    return sg::launch_backward<true>(o, p, stream);
}
