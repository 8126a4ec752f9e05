// ckpt.cuh -- 8-bit activation checkpoints: the block rule and element
// conversions shared by the checkpoint, SwiGLU and norm kernels.
//
// A row is cut into blocks of 32 columns (FP8_MX_BLOCK).  A block's scale is
// X = 2^e, e the smallest integer with amax <= fp8_max * 2^e, clamped to
// [-127, 127] and stored as the byte e + 127; each element is stored as
// rne_fp8(v / X).  Against the MX rule (e from floor(log2 amax) alone) this
// e is one larger when amax lies in the top eighth of its binade, where the
// MX rule clips to fp8_max: a checkpoint has no tensor core to please, so
// nothing is clipped and every normal element is within 2^-4 (E4M3) or 2^-3
// (E5M2) of itself.  The scales are powers of two, so scaling by them is
// exact both ways and the conversion to 8 bits is the only rounding.  An all-zero block
// has byte 0; a block with a NaN or Inf has byte 255 and restores as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fp8gb_device.cuh"

namespace fp8gb {

// Columns of a part rounded up to whole blocks.
__host__ __device__ __forceinline__ int64_t ckpt_width(int64_t cols)
{
    return (cols + FP8_MX_BLOCK - 1) / FP8_MX_BLOCK * FP8_MX_BLOCK;
}

// Scale byte of a block from the fp32 bits of its largest magnitude.
// fp8_max = 1.75 * 2^EF for both formats: amax = m 2^E needs e = E - EF, one
// more when m > 1.75.  An fp32-subnormal amax clamps to e = -127.
__device__ __forceinline__ uint32_t ckpt_code(uint32_t amax_bits, int fmt)
{
    const int EF = fmt == FP8_E5M2 ? 15 : 8;
    if (amax_bits >= 0x7F800000u) return 255u;
    const int code = (int)(amax_bits >> 23) - EF + ((amax_bits & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
    return code < 0 ? 0u : (uint32_t)code;  // at most 247
}

// 1 / X of a code that ckpt_code gives (0 .. 247: a normal fp32), NaN for 255.
__device__ __forceinline__ float ckpt_inv_scale(uint32_t code)
{
    return code == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - code) << 23);
}

// X = 2^(code - 127) of any scale byte (code 0: the subnormal 2^-127).
__device__ __forceinline__ float ckpt_scale(uint32_t code)
{
    return code == 255u ? __uint_as_float(0x7FC00000u) : code == 0u ? __uint_as_float(0x00400000u)
                                                                    : __uint_as_float(code << 23);
}

// Two codes (low byte first) -> two fp32, exact (fp16 holds every value of
// both formats).
template <int FMT>
__device__ __forceinline__ float2 fp8x2_to_float2(uint32_t codes)
{
    uint32_t h;
    if constexpr (FMT == FP8_E5M2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    else
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// Element types of the tensors around a checkpoint.
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

// One rounding to nearest-even into the tensor's type.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// fp32 bits of |v|; NaN patterns order above Inf, so an unsigned maximum
// carries them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Maximum over the `width` consecutive lanes a block is spread over.
template <int WIDTH>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
#pragma unroll
    for (int d = WIDTH / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// One element per lane, a block per warp: store code and scale byte, return
// what the checkpoint gives back for it.
__device__ __forceinline__ void ckpt_store_lane(float v, int fmt, uint8_t *q, uint8_t *s, int lane)
{
    const uint32_t code = ckpt_code(lanes_max<32>(abs_bits(v)), fmt);
    const float t = v * ckpt_inv_scale(code);
    q[lane] = (uint8_t)(fmt == FP8_E5M2 ? cvt2<FP8_E5M2>(t, 0.0f) : cvt2<FP8_E4M3FN>(t, 0.0f));
    if (lane == 0) *s = (uint8_t)code;
}

__device__ __forceinline__ float ckpt_load_one(const uint8_t *q, const uint8_t *s, int64_t col, int fmt)
{
    const float v = fmt == FP8_E5M2 ? fp8x2_to_float2<FP8_E5M2>(q[col]).x : fp8x2_to_float2<FP8_E4M3FN>(q[col]).x;
    return v * ckpt_scale(s[col / FP8_MX_BLOCK]);
}

// SwiGLU backward of one pair, sigma formed as in swiglu1 (t = e^-|g| never
// overflows; 1 - sigma is the other sign's sigma, so neither cancels):
//   dg = dh u sigma (1 + g (1 - sigma)),  du = dh g sigma.
// g = -Inf takes the limit 0 of both sigma and sigma g (t == 0).  The error
// of sigma and of its complement is a few fp32 ulps, so each gradient is
// within 2^-9 of itself or 2^-20 |dh u| before its rounding to bf16.
__device__ __forceinline__ void swiglu_grad1(float g, float u, float dh, float &dg, float &du)
{
    const float t = __expf(-fabsf(g));
    const float r = __fdividef(1.0f, 1.0f + t);
    const float near1 = r, near0 = t * r;  // sigma(|g|), sigma(-|g|)
    const float gc = t == 0.0f ? 0.0f : g * near0;              // g (1 - sigma) for g >= 0, g sigma for g < 0
    const float gs = g >= 0.0f ? g * near1 : gc;                // silu(g)
    const float slope = g >= 0.0f ? near1 * (1.0f + gc) : near0 + gc * near1;  // sigma + sigma g (1 - sigma)
    dg = dh * u * slope;
    du = dh * gs;
}

}  // namespace fp8gb
