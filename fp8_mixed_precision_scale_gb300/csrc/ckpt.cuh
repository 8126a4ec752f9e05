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
// exact both ways and the conversion to 8 bits is the only rounding.  That one
// can go up to the next power of two, which at the top of a type's range lies
// outside: fp16 takes it back (hold_65536), while bf16 and fp32 values from 1.9375 *
// 2^127 (E4M3) or 1.875 * 2^127 (E5M2) on restore as Inf, for 2^128 is what
// their code and scale stand for.  An all-zero block has byte 0; a block with a
// NaN or Inf has byte 255 and restores as NaN.
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

// ---------------------------------------------------------------------------
// Sixteen consecutive elements per thread, half a block: 32 bytes of a 16-bit
// type (one 32-byte access when everything is 32-byte aligned, `w32`, else
// two of 16), 64 of fp32, 16 bytes of codes.
// ---------------------------------------------------------------------------
template <typename T>
struct Raw16 {
    uint4 v[sizeof(T)];  // 16 * sizeof(T) bytes
};

__device__ __forceinline__ void ld_stream_32b(const void *p, uint4 &lo, uint4 &hi)
{
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
                 : "l"(p));
}

__device__ __forceinline__ uint4 ld_stream_16b(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The same of memory that another kernel may have written while this one was there
// (before its griddepcontrol.wait, which as asm volatile stays ahead of this).
__device__ __forceinline__ void ld_32b(const void *p, uint4 &lo, uint4 &hi)
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
                 : "l"(p));
}

__device__ __forceinline__ uint4 ld_shared_16b(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

__device__ __forceinline__ void st_32b(void *p, const uint4 &lo, const uint4 &hi)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(lo.x), "r"(lo.y),
                 "r"(lo.z), "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                 : "memory");
}

// Elements 0 .. n-1 from p (n >= 16: all of them by wide loads), zeros after.
template <typename T>
__device__ __forceinline__ void load16(const T *p, int n, bool w32, Raw16<T> &r)
{
    if (n >= 16) {
        if (w32) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j += 2) ld_stream_32b(p + j * (16 / sizeof(T)), r.v[j], r.v[j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j++) r.v[j] = ld_stream_16b(p + j * (16 / sizeof(T)));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < (int)sizeof(T); j++) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            constexpr int PER = 4 / sizeof(T);  // elements per word
            const int e = (4 * j + k) * PER;
            if constexpr (sizeof(T) == 4) {
                w[k] = e < n ? __float_as_uint(to_f32(p[e])) : 0u;
            } else {
                const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
                w[k] = (e < n ? (uint32_t)h[e] : 0u) | (e + 1 < n ? (uint32_t)h[e + 1] << 16 : 0u);
            }
        }
        r.v[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Two elements of a 32-bit word.
template <typename T>
__device__ __forceinline__ float2 word_to_float2(uint32_t w)
{
    if constexpr (sizeof(T) == 2) {
        if constexpr (__is_same(T, __half)) return __half22float2(*reinterpret_cast<__half2 *>(&w));
        return make_float2(bf16lo(w), bf16hi(w));
    }
    return make_float2(__uint_as_float(w), 0.0f);
}

template <typename T>
__device__ __forceinline__ uint32_t float2_to_word(float lo, float hi)
{
    if constexpr (__is_same(T, __half)) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    return pack_bf16x2(lo, hi);
}

template <typename T>
__device__ __forceinline__ void unpack16(const Raw16<T> &r, float (&f)[16])
{
#pragma unroll
    for (int j = 0; j < (int)sizeof(T); j++) {
        const uint32_t w[4] = {r.v[j].x, r.v[j].y, r.v[j].z, r.v[j].w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if constexpr (sizeof(T) == 4) {
                f[4 * j + k] = __uint_as_float(w[k]);
            } else {
                const float2 v = word_to_float2<T>(w[k]);
                f[8 * j + 2 * k] = v.x;
                f[8 * j + 2 * k + 1] = v.y;
            }
        }
    }
}

// Elements 0 .. n-1 to p.
template <typename T>
__device__ __forceinline__ void store16(T *p, const float (&f)[16], int n, bool w32)
{
    if (n >= 16) {
        uint4 v[sizeof(T)];
#pragma unroll
        for (int j = 0; j < (int)sizeof(T); j++) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(f[4 * j + k]);
                else w[k] = float2_to_word<T>(f[8 * j + 2 * k], f[8 * j + 2 * k + 1]);
            }
            v[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (w32) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j += 2) st_32b(p + j * (16 / sizeof(T)), v[j], v[j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); j++) *reinterpret_cast<uint4 *>(p + j * (16 / sizeof(T))) = v[j];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; j++)
        if (j < n) p[j] = from_f32<T>(f[j]);
}

// ---------------------------------------------------------------------------
// The same sixteen elements at any element alignment.  Every lane of a row's
// segment stands at the same offset from a 16-byte boundary, since lanes are 32
// (64) bytes apart.
//
// Load: the aligned 16-byte words that cover the elements, one more than
// aligned data takes, moved into place when they are used (realign16).  They
// reach up to 14 bytes past the elements on either side, so only a caller that
// knows these to lie inside the tensor says `inside`; the others load element
// by element.  Elements from n on are whatever lies there.
//
// Store: a lane shifts its elements and the first ones of the next lane into
// aligned words; what has no neighbour to do that with (a row's or a warp's
// ends) goes element by element.
// ---------------------------------------------------------------------------
template <typename T>
struct RawAny {
    uint4 v[sizeof(T) + 1];
    uint32_t shift;  // bytes from v to the first element
};

template <typename T>
__device__ __forceinline__ void load16(const T *p, int n, bool inside, RawAny<T> &r)
{
    r.shift = 0;
    if (n > 0 && inside) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const uint4 *w = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        r.shift = (uint32_t)at & 15u;
        // through L1: neighbouring lanes read the words between them twice
#pragma unroll
        for (int j = 0; j <= (int)sizeof(T); j++) r.v[j] = __ldg(w + j);
    } else {
        Raw16<T> e;
        const T *own = p;
        load16(own, n < 16 ? n : 15, false, e);
        if (n >= 16) {  // the last element by itself: load16 would take wide accesses for all sixteen
            if constexpr (sizeof(T) == 4) e.v[sizeof(T) - 1].w = __float_as_uint(to_f32(p[15]));
            else e.v[sizeof(T) - 1].w |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[15] << 16;
        }
#pragma unroll
        for (int j = 0; j < (int)sizeof(T); j++) r.v[j] = e.v[j];
        r.v[sizeof(T)] = make_uint4(0, 0, 0, 0);
    }
}

// Words a[0 ..] shifted down by `shift` bytes (0 .. 14, even), N of them.
template <int N>
__device__ __forceinline__ void shift_words(const uint32_t (&a)[N + 4], uint32_t shift, uint32_t (&out)[N])
{
    uint32_t b[N + 2], c[N + 1];
#pragma unroll
    for (int j = 0; j < N + 2; j++) b[j] = shift & 8u ? a[j + 2] : a[j];
#pragma unroll
    for (int j = 0; j < N + 1; j++) c[j] = shift & 4u ? b[j + 1] : b[j];
#pragma unroll
    for (int j = 0; j < N; j++) out[j] = __funnelshift_r(c[j], c[j + 1], (shift & 2u) * 8u);
}

template <typename T>
__device__ __forceinline__ void unpack16(const RawAny<T> &r, float (&f)[16])
{
    constexpr int N = 4 * sizeof(T);
    uint32_t a[N + 4], w[N];
#pragma unroll
    for (int j = 0; j <= (int)sizeof(T); j++) {
        a[4 * j] = r.v[j].x, a[4 * j + 1] = r.v[j].y, a[4 * j + 2] = r.v[j].z, a[4 * j + 3] = r.v[j].w;
    }
    shift_words<N>(a, r.shift, w);
    Raw16<T> e;
#pragma unroll
    for (int j = 0; j < (int)sizeof(T); j++) e.v[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    unpack16(e, f);
}

// Elements 0 .. min(16, rest) - 1 to p, `rest` being what the row has from
// here on (<= 0: nothing).  `first` / `last`: the lane before / after does not
// hold the row's elements before / after these.  All lanes of a warp call it.
template <typename T>
__device__ __forceinline__ void store16_any(T *p, const float (&f)[16], int rest, bool first, bool last)
{
    constexpr int N = 4 * sizeof(T), PER = 16 / sizeof(T);  // words of a lane, elements of a 16-byte word
    uint32_t a[N + 4], w[N];
#pragma unroll
    for (int j = 0; j < N; j++) {
        if constexpr (sizeof(T) == 4) a[j] = __float_as_uint(f[j]);
        else a[j] = float2_to_word<T>(f[2 * j], f[2 * j + 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) a[N + j] = __shfl_down_sync(0xffffffffu, a[j], 1);
    const uint32_t o = (16u - (uint32_t)reinterpret_cast<uintptr_t>(p)) & 15u;  // bytes to the first aligned word
    const int head = (int)(o / sizeof(T));
    shift_words<N>(a, o, w);
    int lo = 0, hi = 0;  // elements that go one by one
    if (rest >= 16) {
        uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<uintptr_t>(p) + o);
#pragma unroll
        for (int j = 0; j < (int)sizeof(T) - 1; j++)
            dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        if (head == 0 || (!last && rest - 16 >= head))
            dst[sizeof(T) - 1] = make_uint4(w[N - 4], w[N - 3], w[N - 2], w[N - 1]);
        else
            lo = head + 16 - PER, hi = 16;
        if (first) {
#pragma unroll
            for (int j = 0; j < PER - 1; j++)
                if (j < head) p[j] = from_f32<T>(f[j]);
        }
    } else if (rest > 0) {
        lo = !first && rest >= head ? head : 0, hi = rest;
    }
    if (lo < hi) {
#pragma unroll
        for (int j = 0; j < 16; j++)
            if (j >= lo && j < hi) p[j] = from_f32<T>(f[j]);
    }
}

// Either form of the loads and stores as a template parameter: ANY alignment,
// or multiples of 16 bytes.
template <typename T, bool ANY>
struct RawOf {
    using type = Raw16<T>;
};
template <typename T>
struct RawOf<T, true> {
    using type = RawAny<T>;
};
template <typename T, bool ANY>
using Raw = typename RawOf<T, ANY>::type;

// Whether the 16 elements from `at` on (counted from a tensor's first) have 16
// bytes of the tensor before and after them; `end`: elements of the tensor
// from its first to its last row's end.
__device__ __forceinline__ bool well_inside(int64_t at, int64_t end) { return at >= 8 && at + 24 <= end; }

__host__ __device__ __forceinline__ int64_t rows_end(int64_t ld, int64_t rows, int64_t width)
{
    return (rows - 1) * ld + width;
}

// min(n, 16) elements from p on; `at` and `end` as in well_inside.
template <bool ANY, typename T>
__device__ __forceinline__ void load_chunk(const T *p, int n, bool w32, int64_t at, int64_t end, Raw<T, ANY> &raw)
{
    if constexpr (ANY) load16(p, n, well_inside(at, end), raw);
    else load16(p, n, w32, raw);
}

// The first min(rest, 16) of f to p.  `t` is the thread's place among the
// `lanes` threads that hold consecutive chunks of the row.
template <bool ANY, typename T>
__device__ __forceinline__ void store_chunk(T *p, const float (&f)[16], int rest, bool w32, int t, int lanes)
{
    if constexpr (ANY)
        store16_any(p, f, rest, t == 0 || (threadIdx.x & 31) == 0, t == lanes - 1 || (threadIdx.x & 31) == 31);
    else
        store16(p, f, rest, w32);
}

// Elements from n on replaced (n >= 16: none).
__device__ __forceinline__ void fill_from(float (&f)[16], int n, float v)
{
    if (n < 16) {
#pragma unroll
        for (int j = 0; j < 16; j++) f[j] = j < n ? f[j] : v;
    }
}

// The largest magnitude of a block whose halves two neighbouring lanes hold.
__device__ __forceinline__ uint32_t block_amax16(const float (&f)[16])
{
    uint32_t m = abs_bits(f[0]);
#pragma unroll
    for (int j = 1; j < 16; j++) m = max(m, abs_bits(f[j]));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 1));
}

template <int FMT>
__device__ __forceinline__ uint4 encode16(const float (&f)[16], float inv)
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float a = f[4 * j], b = f[4 * j + 1], c = f[4 * j + 2], d = f[4 * j + 3];
        mul2_rn(a, b, inv, inv);
        mul2_rn(c, d, inv, inv);
        w[j] = cvt4<FMT>(a, b, c, d);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int FMT>
__device__ __forceinline__ void decode16(const uint4 &q, float scale, float (&f)[16])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 a = fp8x2_to_float2<FMT>(w[j] & 0xFFFFu), b = fp8x2_to_float2<FMT>(w[j] >> 16);
        f[4 * j] = a.x;
        f[4 * j + 1] = a.y;
        f[4 * j + 2] = b.x;
        f[4 * j + 3] = b.y;
        mul2_rn(f[4 * j], f[4 * j + 1], scale, scale);
        mul2_rn(f[4 * j + 2], f[4 * j + 3], scale, scale);
    }
}

// Restored fp16 values: +-65536 as +-65504.  The largest finite fp16 values
// (from 63488 on in E4M3, 61440 in E5M2) are kept as 65536, which fp16 would round
// to Inf; 65504 is nearer to them.  Anything larger was no finite fp16 value.
__device__ __forceinline__ void hold_65536(float (&f)[16])
{
#pragma unroll
    for (int j = 0; j < 16; j++) f[j] = fabsf(f[j]) == 65536.0f ? copysignf(65504.0f, f[j]) : f[j];
}

// Packed pairs of fp32, each operation rounded to nearest.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    mul2_rn(a.x, a.y, b.x, b.y);
    return a;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\t"
        "mov.b64 {%0, %1}, w;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)  // NaN if either is
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest magnitude of three; NaN if any is.
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float rcp_fast(float v)  // 1 ulp; 0 where 1 / v is subnormal
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// SiLU of two gates with what its derivative needs, from e = e^-gate:
//   sigma = 1 / (1 + e),  1 - sigma = e sigma (no cancellation),  silu = gate sigma.
// gate is held at -88 from below: e^88 is finite and its reciprocal flushes to
// zero, so sigma, silu and the slope are 0 there (they are below 2^-119), also
// for gate = -Inf, where the formula as written gives NaN.  NaN stays
// NaN.  __expf is documented to 2 + 1.173 |x| ulp, at most 2^-16.3 relative here, so
// e and sigma err by less than 2^-16, far inside the bf16 rounding of the results.
__device__ __forceinline__ void silu2(float2 g, float2 &e, float2 &sigma, float2 &silu)
{
    g = make_float2(max_nan(g.x, -88.0f), max_nan(g.y, -88.0f));
    e = make_float2(__expf(-g.x), __expf(-g.y));
    const float2 d = add2(e, make_float2(1.0f, 1.0f));
    sigma = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    silu = mul2(g, sigma);
}

// SwiGLU backward of two pairs (gate, up):
//   d_gate = dh up (sigma + silu (1 - sigma)),  d_up = dh silu,  h = silu up.
__device__ __forceinline__ void swiglu_grad2(float2 g, float2 u, float2 dh, float2 &dg, float2 &du, float2 &h)
{
    float2 e, s, silu;
    silu2(g, e, s, silu);
    const float2 slope = fma2(silu, mul2(e, s), s);
    dg = mul2(mul2(dh, u), slope);
    du = mul2(dh, silu);
    h = mul2(silu, u);
}

}  // namespace fp8gb
