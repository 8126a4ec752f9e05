// swiglurows.cu -- the SwiGLU product's forward for a few rows (a token at a time):
// gate = A W_gate^T, up = A W_up^T, h = silu(gate) up, with what swiglugemm.cu's
// epilogue leaves.
//
// With one row or two the weights are read once and little else is done, so HBM
// bounds the call from below: 2 F K bytes.  A 128-row tensor-core tile of 128
// columns gives few SMs work and reads 128-byte pieces of 256 rows; here a warp reads
// 512 consecutive bytes of a row and goes along it.  A block has 32 columns of h, the
// width of an MX block, and each of its eight warps four of them: eight rows of W at a
// time, a row's next step asked for when this one's has been taken.  A in fp32 with its
// block scales (exact), in shared memory; each W code is exact in fp16 and fp32; fp32
// sums, a W block's scale applied to the sum of 16 products.  A's scales go in as far as
// 2^-60 to 2^60 (16 products of E5M2 are below 2^36), the rest of one beyond that after
// W's: nothing leaves fp32 on the way that the result would not.
//
// MX, one row, in a graph: F = 14336, K = 4096 31.7 to 34 us = 3.6 TB/s; F = 2048, K =
// 7168 22.8 us; F = 1504, K = 4096 13.9 us.  Bound by the conversions of the codes as much as
// by memory: 4.2 instructions a weight in 45 % of the issue slots, of which 1.5 convert.
// Two rows, this against the tiles (F, K): scaled 32.8 and 36.9 (14336, 4096), 24.0 and
// 22.8 (2048, 7168), 13.8 and 16.4 (1504, 4096), 36.4 and 45.1 (8192, 8192); MX 38.5 and
// 35.5 to 37.4, 30.0 and 27.3, 16.5 and 18.6, 43.1 and 40.4 to 42.6: two rows of scaled
// operands come here, of MX operands one.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "swiglugemm.cuh"

namespace fp8gb {
namespace sg {

constexpr int FR_THREADS = 256, FR_WARPS = FR_THREADS / 32;
constexpr int FR_COLS = 32;                     // of h, a block
constexpr int FR_EACH = FR_COLS / FR_WARPS;     // a warp
constexpr int FR_ROWS = 2 * FR_EACH;            // rows of W a warp reads at once
constexpr int FR_STEP = 512;                    // of K
constexpr int FR_MOST = 2;                      // rows of A at most: their values stay in registers
constexpr int FR_SMEM = 96 * 1024;              // of A at most: two blocks an SM
constexpr int FR_BLOCKS = FR_SMEM / (int)sizeof(float) / FP8_MX_BLOCK;  // scales of A at most (MX: one row)
constexpr uint32_t FR_LOW = 127 - 60, FR_HIGH = 127 + 60;

struct RowArgs {
    const uint8_t *A, *B, *sA, *sB;
    int64_t lda, ldb, rsA, rsB;
    int fa, fb;
};

__device__ __forceinline__ void decode(const uint4 &q, int fmt, float (&f)[16])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 a = fmt == FP8_E5M2 ? fp8x2_to_float2<FP8_E5M2>(w[j] & 0xFFFFu)
                                         : fp8x2_to_float2<FP8_E4M3FN>(w[j] & 0xFFFFu);
        const float2 b = fmt == FP8_E5M2 ? fp8x2_to_float2<FP8_E5M2>(w[j] >> 16)
                                         : fp8x2_to_float2<FP8_E4M3FN>(w[j] >> 16);
        f[4 * j] = a.x, f[4 * j + 1] = a.y, f[4 * j + 2] = b.x, f[4 * j + 3] = b.y;
    }
}

__device__ __forceinline__ uint8_t code_of(float v, int fmt)
{
    return (uint8_t)(fmt == FP8_E5M2 ? cvt2<FP8_E5M2>(v, 0.0f) : cvt2<FP8_E4M3FN>(v, 0.0f));
}

template <bool MX, int MT>
__global__ void __launch_bounds__(FR_THREADS, 2) swiglu_rows_kernel(RowArgs o, Params p)
{
    // A: quad j of lane l's 16 values of a step at ((row steps + step) 4 + j) 32 + l
    extern __shared__ __align__(16) float4 xs[];
    __shared__ float sums[2][MT][FR_COLS];
    __shared__ uint8_t code[FR_MOST];
    __shared__ float rest[MX ? FR_BLOCKS : 1];  // of A's scales
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c0 = (int64_t)blockIdx.x * FR_COLS;
    const int M = (int)p.M, K = (int)p.K, steps = (K + FR_STEP - 1) / FR_STEP;
    const int n = (int)(p.F - c0 < 0 ? 0 : p.F - c0 < FR_COLS ? p.F - c0 : FR_COLS);  // columns there are

    // the warp's columns: their rows of W, gate's and up's in turn.  Consecutive rows
    // of a 32-row block are four words apart in the scale layout
    const int64_t cw = c0 + warp * FR_EACH;
    const uint8_t *gate = o.B + cw * o.ldb + lane * 16, *up = gate + p.b1_row * o.ldb;
    const uint8_t *sg = nullptr, *su = nullptr;
    if (MX) {
        sg = o.sB + 4 * mx_scale_word(lane >> 3, cw, o.rsB) + (lane >> 1 & 3);
        su = o.sB + 4 * mx_scale_word(lane >> 3, p.b1_srow + cw, o.rsB) + (lane >> 1 & 3);
    }
    const int64_t s_step = 16 * o.rsB;  // bytes of the scales of a step: four K tiles
    uint4 w[FR_ROWS];
    uint32_t s[FR_ROWS];
    const auto fetch = [&](int i, int step) {
        const int j = i >> 1;
        w[i] = make_uint4(0, 0, 0, 0);
        s[i] = 127;
        if (step * FR_STEP + lane * 16 < K && warp * FR_EACH + j < n) {
            w[i] = ld_stream_16b((i & 1 ? up : gate) + j * o.ldb + (int64_t)step * FR_STEP);
            if (MX) s[i] = __ldg((i & 1 ? su : sg) + 16 * j + step * s_step);
        }
    };
#pragma unroll
    for (int i = 0; i < FR_ROWS; i++) fetch(i, 0);
    for (int i = threadIdx.x; i < MT * steps * 32; i += FR_THREADS) {
        const int m = i / (steps * 32), at = i - m * steps * 32, l = at & 31, k = (at >> 5) * FR_STEP + l * 16;
        float f[16] = {}, past = 1.0f;
        if (m < M && k < K) {
            decode(*reinterpret_cast<const uint4 *>(o.A + m * o.lda + k), o.fa, f);
            if (MX) {
                const uint32_t e = o.sA[4 * mx_scale_word(k >> 7, m, o.rsA) + (k >> 5 & 3)];
                const uint32_t in = e == 255u ? e : min(max(e, FR_LOW), FR_HIGH);
                const float x = ckpt_scale(in);
                past = ckpt_scale(127u + e - in);
#pragma unroll
                for (int j = 0; j < 16; j++) f[j] *= x;
            }
        }
        if (MX && !(at & 1)) rest[at >> 1] = past;  // a block's first thread
#pragma unroll
        for (int j = 0; j < 4; j++)
            xs[((m * steps + (at >> 5)) * 4 + j) * 32 + l] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
    }
    __syncthreads();

    float acc[FR_ROWS][MT] = {};
    for (int step = 0; step < steps; step++) {
        float4 x[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int j = 0; j < 4; j++) x[m][j] = xs[((m * steps + step) * 4 + j) * 32 + lane];
        const float past = MX ? rest[step * 16 + (lane >> 1)] : 1.0f;
#pragma unroll
        for (int i = 0; i < FR_ROWS; i++) {
            float f[16];
            decode(w[i], o.fb, f);
            const float scale = ckpt_scale(s[i]);
            if (step + 1 < steps) fetch(i, step + 1);
#pragma unroll
            for (int m = 0; m < MT; m++) {
                float2 t = make_float2(0.0f, 0.0f), u = t;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    t = fma2(make_float2(f[4 * j], f[4 * j + 1]), make_float2(x[m][j].x, x[m][j].y), t);
                    u = fma2(make_float2(f[4 * j + 2], f[4 * j + 3]), make_float2(x[m][j].z, x[m][j].w), u);
                }
                t = add2(t, u);
                acc[i][m] = MX ? fmaf((t.x + t.y) * scale, past, acc[i][m]) : acc[i][m] + (t.x + t.y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < FR_ROWS; i++)
#pragma unroll
        for (int m = 0; m < MT; m++) {
            float v = acc[i][m];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            if (lane == 0) sums[i & 1][m][warp * FR_EACH + (i >> 1)] = v;
        }
    __syncthreads();

    // warp m has row m, a lane a column
    const int64_t c = c0 + lane;
    const bool have = lane < n;
    if (warp < MT && warp < M) {
        const int m = warp;
        float g = sums[0][m][lane], u = sums[1][m][lane];
        if (!MX && have) {
            const float sa = p.sa_row ? __ldg(p.sa + m) : __ldg(p.sa);
            g = g * sa * (p.sb_row ? __ldg(p.sb + c) : __ldg(p.sb));
            u = u * sa * (p.sb_row ? __ldg(p.sb + p.F + c) : __ldg(p.sb));
        }
        g = have ? g : 0.0f, u = have ? u : 0.0f;
        if (p.gate_up && have) {
            uint16_t *dst = p.gate_up + m * p.ld_gu + c;
            dst[0] = (uint16_t)pack_bf16x2(g, 0.0f);
            dst[p.F] = (uint16_t)pack_bf16x2(u, 0.0f);
        }
        if (p.cq && c0 < p.W) {
            const uint32_t a = ckpt_code(__reduce_max_sync(0xffffffffu, abs_bits(g)), p.cfmt);
            const uint32_t b = ckpt_code(__reduce_max_sync(0xffffffffu, abs_bits(u)), p.cfmt);
            uint8_t *dst = p.cq + m * p.ld_cq + c, *sc = p.cs + m * p.ld_cs + (c0 >> 5);
            dst[0] = code_of(g * ckpt_inv_scale(a), p.cfmt);
            dst[p.W] = code_of(u * ckpt_inv_scale(b), p.cfmt);
            if (lane == 0) {
                sc[0] = (uint8_t)a;
                sc[p.W >> 5] = (uint8_t)b;
            }
        }
        float2 e, sg, si;
        silu2(make_float2(g, g), e, sg, si);
        const float h = si.x * u;
        if (p.out && have) p.out[m * p.ld_out + c] = (uint16_t)pack_bf16x2(h, 0.0f);
        const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(h));
        float inv = 1.0f;
        if (MX) {
            const uint32_t k = mx_code_of(top, p.fmt);
            inv = mx_inv_scale(k);
            if (lane == 0) code[m] = (uint8_t)k;
        } else if (p.scale_in) {
            inv = __ldg(p.scale_in);
            if (lane == 0 && top) atomicMax(reinterpret_cast<unsigned int *>(p.amax_out), top);
            if (blockIdx.x == 0 && m == 0 && lane == 0) p.scale_inv[0] = recip_rn(inv);
        }
        if (have) {
            const uint8_t q = code_of(h * inv, p.fmt);
            if (p.q_row) p.q_row[m * p.ld_row + c] = q;
            if (!MX && p.q_col) p.q_col[c * p.ld_col + m] = q;
        }
    }
    if (MX && p.q_row) {  // the block's scale bytes of all 128 rows of the layout: zeros behind the data
        __syncthreads();
        if (threadIdx.x < 128)
            p.s_row[4 * mx_scale_word(c0 >> 7, threadIdx.x, p.rs_row) + (c0 >> 5 & 3)] =
                threadIdx.x < M && n > 0 ? code[threadIdx.x] : 0;
    }
}

template <auto KERNEL>
static fp8_status_t launch(const RowArgs &o, const Params &p, unsigned grid, int smem, cudaStream_t st)
{
    constexpr int MAX_DEVICES = 64;
    static std::atomic<bool> allowed[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cuda_fail();
    if (dev >= MAX_DEVICES || !allowed[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, FR_SMEM) != cudaSuccess)
            return cuda_fail();
        if (dev < MAX_DEVICES) allowed[dev].store(true, std::memory_order_release);
    }
    KERNEL<<<grid, FR_THREADS, smem, st>>>(o, p);
    return check_launch();
}

bool few_rows(const Operands &o, const Params &p, bool mx, cudaStream_t st, fp8_status_t &rc)
{
    if (p.M > (mx ? 1 : FR_MOST)) return false;
    const int mt = (int)p.M;
    const int64_t steps = (p.K + FR_STEP - 1) / FR_STEP, smem = mt * steps * FR_STEP * (int64_t)sizeof(float);
    // MX with the transposed layout has 32 rows at least
    if (smem > FR_SMEM) return false;
    const RowArgs r{static_cast<const uint8_t *>(o.A),  static_cast<const uint8_t *>(o.B),
                    static_cast<const uint8_t *>(o.sA), static_cast<const uint8_t *>(o.sB),
                    o.lda, o.ldb, o.rsA, o.rsB, o.fa, o.fb};
    // MX: the scale bytes of the columns up to whole K tiles of the next product too
    const unsigned grid = (unsigned)((mx ? round_up_128(p.F) : p.F + FR_COLS - 1) / FR_COLS);
    if (mx) rc = launch<swiglu_rows_kernel<true, 1>>(r, p, grid, (int)smem, st);
    else rc = mt == 1 ? launch<swiglu_rows_kernel<false, 1>>(r, p, grid, (int)smem, st)
                      : launch<swiglu_rows_kernel<false, 2>>(r, p, grid, (int)smem, st);
    return true;
}

}  // namespace sg
}  // namespace fp8gb
