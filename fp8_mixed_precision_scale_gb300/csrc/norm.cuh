// norm.cuh -- what the norm kernels share: parameter vectors, the sums of a row
// over its threads and over a cluster, and the plan of a launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ckpt.cuh"
#include "fp8gb.h"
#include "fp8gb_device.cuh"
#include "fp8gb_host.h"

namespace fp8gb {

constexpr int NM_BLOCK = 512;          // threads of a block at most: 128 registers each
constexpr int NM_MAX_GROUPS = NM_BLOCK / 64;  // row groups of two warps or more, a named barrier each
constexpr int NM_GROUP_WARPS = 16;     // warps of a row group at most
constexpr int NM_MAX_RANKS = 8;        // blocks of a cluster at most
constexpr int NM_PART = 16 * 32 * NM_GROUP_WARPS;  // columns one chunk a thread covers in a block
constexpr int64_t NM_MAX_COLS = (int64_t)NM_PART * NM_MAX_RANKS;

// Element i of a parameter vector; NULL gives `absent`.
__device__ __forceinline__ float param(const void *p, int dtype, int64_t i, float absent)
{
    if (!p) return absent;
    if (dtype == FP8_DTYPE_F32) return static_cast<const float *>(p)[i];
    if (dtype == FP8_DTYPE_F16) return to_f32(static_cast<const __half *>(p)[i]);
    return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
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

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline bool rows_aligned(const void *p, int64_t ld, int size, int al)
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

// 48 KB without asking, the kernel's own few KB among them.
constexpr int NM_SHARED_FREE = 40 * 1024;

// Lets a kernel's launches take more than that.  The limit belongs to the kernel
// and device, not to a launch, and other host threads may be about to launch with
// it: it is set once, to the most that any launch takes, and never lowered.
template <auto KERNEL, int MOST>
inline bool allow_shared()
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

// Clusters of `ranks` blocks (of one to an SM) that run at once.
int clusters_at_once(int ranks);

// `chunks` chunks a thread where a warp's lanes do not cover the row (one where
// they do).  Few rows are spread over the SMs before a second group joins a
// block.  `small`: a kernel of one chunk and part-warp groups takes 64 registers,
// two blocks an SM.
inline Plan make_plan(int64_t rows, int64_t cols, int chunks, bool small = false)
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

inline bool good_dtype(int d) { return d >= FP8_DTYPE_BF16 && d <= FP8_DTYPE_F32; }

// A [rows][ld] tensor of the type: pointer, row stride and alignment.
inline fp8_status_t check_tensor(const void *p, int dtype, int64_t ld, int64_t cols)
{
    if (!p || ld < cols) return FP8_ERR_INVALID_ARG;
    return aligned(p, dtype == FP8_DTYPE_F32 ? 4 : 2) ? FP8_OK : FP8_ERR_ALIGNMENT;
}

}  // namespace fp8gb
