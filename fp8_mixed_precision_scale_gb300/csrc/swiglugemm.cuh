// swiglugemm.cuh -- what the SwiGLU products' translation units share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"

namespace fp8gb {
namespace sg {

struct Params {
    int64_t M, F;       // rows; columns of h
    int64_t K;          // contraction
    const float *sa, *sb;
    int sa_row, sb_row;  // per row, else one of the tensor
    int32_t b1_row;      // forward: row of B where up starts
    int32_t b1_srow;     // ... and its scale row
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
    int cs4;    // its scale bytes of four blocks stand on word boundaries
    int64_t W;  // columns of a part of the checkpoint
    // 8 bits
    int fmt;
    const float *scale_in;  // per-tensor recipe
    float *amax_out, *scale_inv;
    uint8_t *q_row, *s_row, *q_col, *s_col;
    int64_t ld_row, ld_col, rs_row, rs_col;
    int64_t Fr;  // columns of h that q_row has (backward: of each half; zeros from F on)
    int q32;     // q_row's rows and halves start on 32-byte boundaries
    int c32;     // q_col's rows do
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

// Largest magnitude of 32 values and m, in four chains.
__device__ __forceinline__ float amax32(const float (&v)[2][16], float m)
{
    float a[4] = {m, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; j += 2)
        a[j / 2 & 3] = max3_abs(a[j / 2 & 3], v[j >> 4][j & 15], v[j >> 4][(j & 15) + 1]);
    return max_nan(max3_abs(a[0], a[1], a[2]), a[3]);
}

// sigma(g), e^-g and silu(g) of two gates as silu2 has them, with the exponential's
// result flushed to zero below 2^-126 (1 - sigma and sigma - 1 are below that then).
// As there e and sigma err by less than 2^-16: the exponent's rounding at |g| = 88, and
// 2 ulp each of the exponential and the reciprocal, far inside the 8-bit and bf16
// roundings of the results.
__device__ __forceinline__ void silu2_ftz(float2 g, float2 &e, float2 &sigma, float2 &silu)
{
    g = make_float2(max_nan(g.x, -88.0f), max_nan(g.y, -88.0f));
    const float2 x = mul2(g, make_float2(-1.44269504f, -1.44269504f));  // -log2 e
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
    const float2 d = add2(e, make_float2(1.0f, 1.0f));
    sigma = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    silu = mul2(g, sigma);
}

// The operands of a launch; sA, sB: MX scales, of rsA and rsB rows.
struct Operands {
    const void *A, *B;
    int fa, fb;
    int64_t lda, ldb, b_rows;
    const void *sA, *sB;
    int64_t rsA, rsB;
};

// The forward of a few rows without tensor cores (swiglurows.cu).  false: more
// rows, or a longer contraction, than it takes.
bool few_rows(const Operands &o, const Params &p, bool mx, cudaStream_t st, fp8_status_t &rc);

}  // namespace sg
}  // namespace fp8gb
