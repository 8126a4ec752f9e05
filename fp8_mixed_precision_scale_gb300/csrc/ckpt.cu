// ckpt.cu -- 8-bit activation checkpoints: store and restore of any matrix,
// the SwiGLU forward that stores its gate|up input in the same read, and the
// SwiGLU backward that reads it.  The block rule is ckpt.cuh's.
//
// All four are one pass over their tensors and bounded by HBM: at [8192, 14336]
// store 51.7, restore 53.0, SwiGLU forward with checkpoint 139 and backward from
// it 143 us, 6.6 to 6.9 TB/s.
//
// A thread works on 16 consecutive columns, half a block: the bf16 side is one
// 32-byte access, the codes one of 16, and the block maximum one shuffle with the
// neighbour.  Checkpoint and restore issue the loads of four rows before they work
// on the first.
// The threads of a block cover 2^lg chunks of CK_THREADS >> lg rows, so no thread
// divides.  Rows that are no multiple of 16 bytes apart (ANY) are read and
// written in the aligned words that cover them, shifted into place.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"

namespace fp8gb {

constexpr int CK_THREADS = 256;

// How the blocks of a launch cover rows x chunks of 16 columns.
struct Geometry {
    int lg;             // a block is 2^lg chunks wide and CK_THREADS / 2^lg rows high, times UNROLL
    uint32_t n_tiles;   // blocks across a row
    uint32_t grid;
};

struct CkArgs {
    void *x;  // store: input; restore: output
    int64_t ld_x;
    uint8_t *q, *s;
    int64_t ld_q, ld_s;
    int64_t rows, cols;
    int parts, fmt;
    Geometry geo;
    int w32;  // x's rows and parts start on 32-byte boundaries
};

struct SwArgs {
    const __nv_bfloat16 *gate_up, *dh;
    int64_t ld, ld_dh;
    uint8_t *q, *s;
    int64_t ld_q, ld_s;
    int64_t rows, F;
    int fmt;
    __nv_bfloat16 *h, *d;
    int64_t ld_h, ld_d;
    Geometry geo;
    int w32;
};

// A thread's chunk and first row; its later rows are `ty` further each.
struct Place {
    int64_t chunk, row;
    int ty;
};

template <int UNROLL>
__device__ __forceinline__ Place place_of(const Geometry &g)
{
    const uint32_t rt = blockIdx.x / g.n_tiles, ct = blockIdx.x - rt * g.n_tiles;
    Place p;
    p.ty = CK_THREADS >> g.lg;
    p.chunk = ((int64_t)ct << g.lg) + (threadIdx.x & ((1 << g.lg) - 1));
    p.row = (int64_t)rt * p.ty * UNROLL + (threadIdx.x >> g.lg);
    return p;
}

// Columns of a part from column c on, and how many of them are in c's chunk.
__device__ __forceinline__ int chunk_rest(int64_t cols, int64_t c) { return (int)(cols - c); }
__device__ __forceinline__ int chunk_columns(int64_t cols, int64_t c) { return max(0, min(16, chunk_rest(cols, c))); }

constexpr int STORE_UNROLL = 4, RESTORE_UNROLL = 4;  // rows whose loads a thread issues first

template <typename T, int FMT, bool ANY>
__global__ void __launch_bounds__(CK_THREADS) checkpoint_kernel(CkArgs a)
{
    const Place p = place_of<STORE_UNROLL>(a.geo);
    const int64_t cpp = ckpt_width(a.cols) / 16;  // chunks of a part
    const bool in = p.chunk < a.parts * cpp;
    const int64_t part = a.parts == 1 ? 0 : p.chunk / cpp, c = (p.chunk - part * cpp) * 16;
    const int n = in ? chunk_columns(a.cols, c) : 0;
    const T *x = static_cast<const T *>(a.x);
    const int64_t end = rows_end(a.ld_x, a.rows, a.parts * a.cols);
    Raw<T, ANY> raw[STORE_UNROLL];
#pragma unroll
    for (int k = 0; k < STORE_UNROLL; k++) {
        const int64_t r = p.row + (int64_t)k * p.ty;
        const int64_t at = r * a.ld_x + part * a.cols + c;
        load_chunk<ANY>(x + at, r < a.rows ? n : 0, a.w32, at, end, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < STORE_UNROLL; k++) {
        const int64_t r = p.row + (int64_t)k * p.ty;
        float f[16];
        unpack16(raw[k], f);
        if (ANY) fill_from(f, n, 0.0f);
        const uint32_t code = ckpt_code(block_amax16(f), FMT);
        if (!in || r >= a.rows) continue;
        *reinterpret_cast<uint4 *>(a.q + r * a.ld_q + p.chunk * 16) = encode16<FMT>(f, ckpt_inv_scale(code));
        if (!(p.chunk & 1)) a.s[r * a.ld_s + (p.chunk >> 1)] = (uint8_t)code;
    }
}

template <typename T, int FMT, bool ANY>
__global__ void __launch_bounds__(CK_THREADS) restore_kernel(CkArgs a)
{
    const Place p = place_of<RESTORE_UNROLL>(a.geo);
    const int64_t cpp = ckpt_width(a.cols) / 16;
    const bool in = p.chunk < a.parts * cpp;
    const int64_t part = a.parts == 1 ? 0 : p.chunk / cpp, c = (p.chunk - part * cpp) * 16;
    const int rest = in ? chunk_rest(a.cols, c) : 0;
    // a part's first chunk has no neighbour before it, whatever the lane there holds
    const int lanes = 1 << a.geo.lg, t = threadIdx.x & (lanes - 1);
    T *x = static_cast<T *>(a.x) + part * a.cols + c;
    uint4 q[RESTORE_UNROLL];
    uint32_t s[RESTORE_UNROLL];
#pragma unroll
    for (int k = 0; k < RESTORE_UNROLL; k++) {
        const int64_t r = p.row + (int64_t)k * p.ty;
        q[k] = make_uint4(0, 0, 0, 0);
        s[k] = 0;
        if (rest <= 0 || r >= a.rows) continue;
        q[k] = ld_stream_16b(a.q + r * a.ld_q + p.chunk * 16);
        s[k] = __ldg(a.s + r * a.ld_s + (p.chunk >> 1));
    }
#pragma unroll
    for (int k = 0; k < RESTORE_UNROLL; k++) {
        const int64_t r = p.row + (int64_t)k * p.ty;
        float f[16];
        decode16<FMT>(q[k], ckpt_scale(s[k]), f);
        if constexpr (__is_same(T, __half)) hold_65536(f);
        store_chunk<ANY>(x + r * a.ld_x, f, r < a.rows ? rest : 0, a.w32, c == 0 ? 0 : t, lanes);
    }
}

// The SwiGLU kernels take one row a thread and four blocks an SM (64 registers):
// two rows and two blocks took 149 and 153 us where these take 140 and 142 (forward
// and backward of [8192, 14336]).
template <int FMT, bool ANY>
__global__ void __launch_bounds__(CK_THREADS, ANY ? 3 : 4) swiglu_checkpoint_kernel(SwArgs a)
{
    using T = __nv_bfloat16;
    const Place p = place_of<1>(a.geo);
    const int64_t cpp = ckpt_width(a.F) / 16, c = p.chunk * 16, r = p.row;
    const bool in = p.chunk < cpp && r < a.rows;
    const int n = in ? chunk_columns(a.F, c) : 0, rest = in ? chunk_rest(a.F, c) : 0;
    const int lanes = 1 << a.geo.lg, t = threadIdx.x & (lanes - 1);
    const int64_t at = r * a.ld + c, end = rows_end(a.ld, a.rows, 2 * a.F);
    Raw<T, ANY> gr, ur;
    load_chunk<ANY>(a.gate_up + at, n, a.w32, at, end, gr);
    load_chunk<ANY>(a.gate_up + at + a.F, n, a.w32, at + a.F, end, ur);
    float g[16], u[16], h[16];
    unpack16(gr, g);
    unpack16(ur, u);
    if (ANY) {
        fill_from(g, n, 0.0f);
        fill_from(u, n, 0.0f);
    }
    const uint32_t cg = ckpt_code(block_amax16(g), FMT), cu = ckpt_code(block_amax16(u), FMT);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        float2 e, sigma, silu;
        silu2(make_float2(g[j], g[j + 1]), e, sigma, silu);
        const float2 v = mul2(silu, make_float2(u[j], u[j + 1]));
        h[j] = v.x, h[j + 1] = v.y;
    }
    store_chunk<ANY>(a.h + r * a.ld_h + c, h, rest, a.w32, t, lanes);
    if (!in) return;
    uint8_t *q = a.q + r * a.ld_q + c;
    *reinterpret_cast<uint4 *>(q) = encode16<FMT>(g, ckpt_inv_scale(cg));
    *reinterpret_cast<uint4 *>(q + cpp * 16) = encode16<FMT>(u, ckpt_inv_scale(cu));
    if (!(p.chunk & 1)) {
        uint8_t *s = a.s + r * a.ld_s + (p.chunk >> 1);
        s[0] = (uint8_t)cg;
        s[cpp >> 1] = (uint8_t)cu;
    }
}

// CKPT: gate and up from the checkpoint, else from bf16.
template <int FMT, bool CKPT, bool ANY>
__global__ void __launch_bounds__(CK_THREADS, 4) swiglu_backward_kernel(SwArgs a)
{
    using T = __nv_bfloat16;
    const Place p = place_of<1>(a.geo);
    const int64_t cpp = ckpt_width(a.F) / 16, c = p.chunk * 16, r = p.row;
    const int n = r < a.rows ? chunk_columns(a.F, c) : 0, rest = r < a.rows ? chunk_rest(a.F, c) : 0;
    const int lanes = 1 << a.geo.lg, t = threadIdx.x & (lanes - 1);
    float g[16], u[16], d[16];
    Raw<T, ANY> dr;
    const int64_t at_dh = r * a.ld_dh + c;
    load_chunk<ANY>(a.dh + at_dh, n, a.w32, at_dh, rows_end(a.ld_dh, a.rows, a.F), dr);
    if constexpr (CKPT) {
        uint4 gq = make_uint4(0, 0, 0, 0), uq = gq;
        uint32_t gs = 0, us = 0;
        if (n > 0) {
            const uint8_t *q = a.q + r * a.ld_q + c, *s = a.s + r * a.ld_s + (p.chunk >> 1);
            gq = ld_stream_16b(q);
            uq = ld_stream_16b(q + cpp * 16);
            gs = __ldg(s);
            us = __ldg(s + (cpp >> 1));
        }
        decode16<FMT>(gq, ckpt_scale(gs), g);
        decode16<FMT>(uq, ckpt_scale(us), u);
    } else {
        Raw<T, ANY> gr, ur;
        const int64_t at = r * a.ld + c, end = rows_end(a.ld, a.rows, 2 * a.F);
        load_chunk<ANY>(a.gate_up + at, n, a.w32, at, end, gr);
        load_chunk<ANY>(a.gate_up + at + a.F, n, a.w32, at + a.F, end, ur);
        unpack16(gr, g);
        unpack16(ur, u);
    }
    unpack16(dr, d);
    // the gradients take the places of g and u, h that of dh
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        float2 dg, du, h;
        swiglu_grad2(make_float2(g[j], g[j + 1]), make_float2(u[j], u[j + 1]), make_float2(d[j], d[j + 1]), dg, du, h);
        g[j] = dg.x, g[j + 1] = dg.y;
        u[j] = du.x, u[j + 1] = du.y;
        d[j] = h.x, d[j + 1] = h.y;
    }
    T *out = a.d + r * a.ld_d + c;
    if (a.h) store_chunk<ANY>(a.h + r * a.ld_h + c, d, rest, a.w32, t, lanes);
    store_chunk<ANY>(out, g, rest, a.w32, t, lanes);
    store_chunk<ANY>(out + a.F, u, rest, a.w32, t, lanes);
}

// The widest block whose tiles cover a row of `chunks` with at most 1/16 of
// their threads idle (two chunks at least: a block's halves are neighbours).
static Geometry geometry(int64_t rows, int64_t chunks, int unroll)
{
    Geometry g;
    g.lg = 8;
    while (g.lg > 1) {
        const int64_t covered = ((chunks + (1LL << g.lg) - 1) >> g.lg) << g.lg;
        if ((covered - chunks) * 16 <= covered) break;
        g.lg--;
    }
    g.n_tiles = (uint32_t)((chunks + (1LL << g.lg) - 1) >> g.lg);
    const int64_t high = (int64_t)(CK_THREADS >> g.lg) * unroll;
    // below 2^31 for anything a device can hold: a block covers 2^12 elements at least
    g.grid = (uint32_t)((rows + high - 1) / high * g.n_tiles);
    return g;
}

// Whether every row (and part) of a tensor starts on an `a`-byte boundary.
static bool rows_aligned(const void *p, int64_t ld, int64_t offset, int size, int a)
{
    return aligned(p, a) && ld * size % a == 0 && offset * size % a == 0;
}

static fp8_status_t check_format(int fmt)
{
    if (fmt == FP8_E4M3FNUZ || fmt == FP8_E5M2FNUZ) return FP8_ERR_UNSUPPORTED;
    return fmt == FP8_E4M3FN || fmt == FP8_E5M2 ? FP8_OK : FP8_ERR_INVALID_ARG;
}

// Codes and scales of a checkpoint with `parts` parts of `cols` columns.
static fp8_status_t check_codes(const void *q, int64_t ld_q, const void *s, int64_t ld_s, int64_t cols, int64_t parts)
{
    const int64_t w = parts * ckpt_width(cols);
    if (!q || !s || ld_q < w || ld_s < w / FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    return ld_q % FP8_MX_BLOCK != 0 || !aligned(q, FP8_MX_BLOCK) ? FP8_ERR_ALIGNMENT : FP8_OK;
}

static fp8_status_t check_ck(const CkArgs &a, int dtype)
{
    if (a.rows < 0 || a.cols < 1 || a.parts < 1 || a.rows > INT32_MAX || a.cols > INT32_MAX / a.parts - FP8_MX_BLOCK)
        return FP8_ERR_INVALID_ARG;
    if (dtype < FP8_DTYPE_BF16 || dtype > FP8_DTYPE_F32) return FP8_ERR_INVALID_ARG;
    const fp8_status_t f = check_format(a.fmt);
    if (f != FP8_OK || a.rows == 0) return f;
    if (!a.x || a.ld_x < a.parts * a.cols) return FP8_ERR_INVALID_ARG;
    if (!aligned(a.x, dtype == FP8_DTYPE_F32 ? 4 : 2)) return FP8_ERR_ALIGNMENT;
    return check_codes(a.q, a.ld_q, a.s, a.ld_s, a.cols, a.parts);
}

static fp8_status_t check_bf16(const void *p, int64_t ld, int64_t cols)
{
    if (!p || ld < cols) return FP8_ERR_INVALID_ARG;
    return aligned(p, 2) ? FP8_OK : FP8_ERR_ALIGNMENT;
}

// Geometry and alignment of x; whether its rows and parts take 16-byte accesses.
template <typename T>
static bool plan(CkArgs &a, int unroll)
{
    const int64_t off = a.parts > 1 ? a.cols : 0;
    a.geo = geometry(a.rows, a.parts * (ckpt_width(a.cols) / 16), unroll);
    a.w32 = rows_aligned(a.x, a.ld_x, off, sizeof(T), 32);
    return rows_aligned(a.x, a.ld_x, off, sizeof(T), 16);
}

template <typename T, int FMT>
static void launch_checkpoint(CkArgs a, cudaStream_t st)
{
    if (plan<T>(a, STORE_UNROLL)) checkpoint_kernel<T, FMT, false><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
    else checkpoint_kernel<T, FMT, true><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
}

template <typename T, int FMT>
static void launch_restore(CkArgs a, cudaStream_t st)
{
    if (plan<T>(a, RESTORE_UNROLL)) restore_kernel<T, FMT, false><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
    else restore_kernel<T, FMT, true><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
}

// The element type and format of a call as template parameters.
#define CK_DISPATCH(FN, dtype, a, st)                                                                       \
    do {                                                                                                    \
        if (a.fmt == FP8_E5M2) {                                                                            \
            if (dtype == FP8_DTYPE_BF16) FN<__nv_bfloat16, FP8_E5M2>(a, st);                                \
            else if (dtype == FP8_DTYPE_F16) FN<__half, FP8_E5M2>(a, st);                                   \
            else FN<float, FP8_E5M2>(a, st);                                                                \
        } else {                                                                                            \
            if (dtype == FP8_DTYPE_BF16) FN<__nv_bfloat16, FP8_E4M3FN>(a, st);                              \
            else if (dtype == FP8_DTYPE_F16) FN<__half, FP8_E4M3FN>(a, st);                                 \
            else FN<float, FP8_E4M3FN>(a, st);                                                              \
        }                                                                                                   \
    } while (0)

template <int FMT>
static void launch_swiglu_checkpoint(SwArgs a, cudaStream_t st)
{
    const auto all_aligned = [&](int al) {
        return rows_aligned(a.gate_up, a.ld, a.F, 2, al) && rows_aligned(a.h, a.ld_h, 0, 2, al);
    };
    a.geo = geometry(a.rows, ckpt_width(a.F) / 16, 1);
    a.w32 = all_aligned(32);
    if (all_aligned(16)) swiglu_checkpoint_kernel<FMT, false><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
    else swiglu_checkpoint_kernel<FMT, true><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
}

template <int FMT, bool CKPT>
static void launch_swiglu_backward(SwArgs a, cudaStream_t st)
{
    const auto all_aligned = [&](int al) {
        return rows_aligned(a.dh, a.ld_dh, 0, 2, al) && rows_aligned(a.d, a.ld_d, a.F, 2, al) &&
               rows_aligned(a.h, a.h ? a.ld_h : 0, 0, 2, al) && (CKPT || rows_aligned(a.gate_up, a.ld, a.F, 2, al));
    };
    a.geo = geometry(a.rows, ckpt_width(a.F) / 16, 1);
    a.w32 = all_aligned(32);
    if (all_aligned(16)) swiglu_backward_kernel<FMT, CKPT, false><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
    else swiglu_backward_kernel<FMT, CKPT, true><<<a.geo.grid, CK_THREADS, 0, st>>>(a);
}

}  // namespace fp8gb

using namespace fp8gb;

extern "C" fp8_status_t fp8_checkpoint(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, int parts,
                                       int fmt, uint8_t *q, int64_t ld_q, uint8_t *s, int64_t ld_s, void *stream)
{
    CkArgs a{const_cast<void *>(x), ld_x, q, s, ld_q, ld_s, rows, cols, parts, fmt};
    const fp8_status_t rc = check_ck(a, dtype);
    if (rc != FP8_OK || rows == 0) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    CK_DISPATCH(launch_checkpoint, dtype, a, st);
    return check_launch();
}

extern "C" fp8_status_t fp8_checkpoint_restore(const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                               int64_t rows, int64_t cols, int parts, void *x, int dtype,
                                               int64_t ld_x, void *stream)
{
    CkArgs a{x, ld_x, const_cast<uint8_t *>(q), const_cast<uint8_t *>(s), ld_q, ld_s, rows, cols, parts, fmt};
    const fp8_status_t rc = check_ck(a, dtype);
    if (rc != FP8_OK || rows == 0) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    CK_DISPATCH(launch_restore, dtype, a, st);
    return check_launch();
}

extern "C" fp8_status_t fp8_swiglu_checkpoint(const void *gate_up_bf16, int64_t rows, int64_t F, int64_t ld, int fmt,
                                              void *h_bf16, int64_t ld_h, uint8_t *q, int64_t ld_q, uint8_t *s,
                                              int64_t ld_s, void *stream)
{
    if (rows < 0 || F < 1 || rows > INT32_MAX || F > INT32_MAX / 2 - FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    fp8_status_t rc = check_format(fmt);
    if (rc != FP8_OK || rows == 0) return rc;
    if ((rc = check_bf16(gate_up_bf16, ld, 2 * F)) != FP8_OK) return rc;
    if ((rc = check_bf16(h_bf16, ld_h, F)) != FP8_OK) return rc;
    if ((rc = check_codes(q, ld_q, s, ld_s, F, 2)) != FP8_OK) return rc;
    SwArgs a{};
    a.gate_up = static_cast<const __nv_bfloat16 *>(gate_up_bf16);
    a.ld = ld;
    a.rows = rows;
    a.F = F;
    a.fmt = fmt;
    a.h = static_cast<__nv_bfloat16 *>(h_bf16);
    a.ld_h = ld_h;
    a.q = q;
    a.s = s;
    a.ld_q = ld_q;
    a.ld_s = ld_s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (fmt == FP8_E5M2) launch_swiglu_checkpoint<FP8_E5M2>(a, st);
    else launch_swiglu_checkpoint<FP8_E4M3FN>(a, st);
    return check_launch();
}

extern "C" fp8_status_t fp8_swiglu_backward(const void *dh_bf16, int64_t ld_dh, const void *gate_up_bf16, int64_t ld,
                                            const uint8_t *q, int64_t ld_q, const uint8_t *s, int64_t ld_s, int fmt,
                                            int64_t rows, int64_t F, void *d_gate_up_bf16, int64_t ld_d,
                                            void *h_bf16, int64_t ld_h, void *stream)
{
    if (rows < 0 || F < 1 || rows > INT32_MAX || F > INT32_MAX / 2 - FP8_MX_BLOCK) return FP8_ERR_INVALID_ARG;
    if (gate_up_bf16 && (q || s)) return FP8_ERR_INVALID_ARG;
    fp8_status_t rc = gate_up_bf16 ? FP8_OK : check_format(fmt);
    if (rc != FP8_OK || rows == 0) return rc;
    if ((rc = check_bf16(dh_bf16, ld_dh, F)) != FP8_OK) return rc;
    if ((rc = check_bf16(d_gate_up_bf16, ld_d, 2 * F)) != FP8_OK) return rc;
    if (h_bf16 && (rc = check_bf16(h_bf16, ld_h, F)) != FP8_OK) return rc;
    rc = gate_up_bf16 ? check_bf16(gate_up_bf16, ld, 2 * F) : check_codes(q, ld_q, s, ld_s, F, 2);
    if (rc != FP8_OK) return rc;
    SwArgs a{};
    a.dh = static_cast<const __nv_bfloat16 *>(dh_bf16);
    a.ld_dh = ld_dh;
    a.gate_up = static_cast<const __nv_bfloat16 *>(gate_up_bf16);
    a.ld = ld;
    a.q = const_cast<uint8_t *>(q);
    a.s = const_cast<uint8_t *>(s);
    a.ld_q = ld_q;
    a.ld_s = ld_s;
    a.fmt = fmt;
    a.rows = rows;
    a.F = F;
    a.d = static_cast<__nv_bfloat16 *>(d_gate_up_bf16);
    a.ld_d = ld_d;
    a.h = static_cast<__nv_bfloat16 *>(h_bf16);
    a.ld_h = ld_h;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (gate_up_bf16) launch_swiglu_backward<FP8_E4M3FN, false>(a, st);
    else if (fmt == FP8_E5M2) launch_swiglu_backward<FP8_E5M2, true>(a, st);
    else launch_swiglu_backward<FP8_E4M3FN, true>(a, st);
    return check_launch();
}
