// bm_norm_kernel.cuh -- layer norm over rows, forward and backward, the final sum of
// partial column sums, and the activation recomputed from an MXFP8 checkpoint.
//
// All of them are bound by HBM: each input is read once and each output written once,
// in 16-byte vectors of the row held in registers between the passes over it.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "bm_act.cuh"
#include "bm_gemm_kernel.cuh"
#include "bm_ptx.cuh"
#include "bm_quant_kernel.cuh"

namespace bm {

// Eight consecutive elements of a row: one 16-byte word of bf16, two of fp32.
template <bool BF16>
struct Vec8 {
    uint4 w[BF16 ? 1 : 2];

    __device__ __forceinline__ void load(const void *row, int64_t i)
    {
        const uint4 *src = reinterpret_cast<const uint4 *>(row) + (BF16 ? i : 2 * i);
#pragma unroll
        for (int q = 0; q < (BF16 ? 1 : 2); ++q) w[q] = src[q];
    }

    // elements [8 i, n) of a row that ends inside the vector; zeros past it
    __device__ __forceinline__ void load_tail(const void *row, int64_t i, int64_t n)
    {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = 0.0f;
            if (8 * i + e < n)
                v[e] = BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(row)[8 * i + e]) << 16)
                            : static_cast<const float *>(row)[8 * i + e];
        }
        set(v);
    }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int q = 0; q < (BF16 ? 1 : 2); ++q) w[q] = make_uint4(0u, 0u, 0u, 0u);
    }

    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        if constexpr (BF16) {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                v[4 * q] = __uint_as_float(w[q].x);
                v[4 * q + 1] = __uint_as_float(w[q].y);
                v[4 * q + 2] = __uint_as_float(w[q].z);
                v[4 * q + 3] = __uint_as_float(w[q].w);
            }
        }
    }

    __device__ __forceinline__ void set(const float (&v)[8])
    {
        if constexpr (BF16) {
            __nv_bfloat162 h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            w[0] = *reinterpret_cast<const uint4 *>(h);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                w[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                  __float_as_uint(v[4 * q + 3]));
        }
    }

    __device__ __forceinline__ void store(void *row, int64_t i) const
    {
        uint4 *dst = reinterpret_cast<uint4 *>(row) + (BF16 ? i : 2 * i);
#pragma unroll
        for (int q = 0; q < (BF16 ? 1 : 2); ++q) dst[q] = w[q];
    }

    __device__ __forceinline__ void store_tail(void *row, int64_t i, int64_t n) const
    {
        float v[8];
        get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (8 * i + e >= n) continue;
            if constexpr (BF16) static_cast<__nv_bfloat16 *>(row)[8 * i + e] = __float2bfloat16_rn(v[e]);
            else static_cast<float *>(row)[8 * i + e] = v[e];
        }
    }
};

__device__ __forceinline__ const void *row_at(const void *base, int64_t row, int64_t ld, bool bf16)
{
    return static_cast<const char *>(base) + row * ld * (bf16 ? 2 : 4);
}

// One parameter vector (8 elements from 8 i; `fill` past n or for a null array).
__device__ __forceinline__ void load_params(const void *base, bool bf16, int64_t i, int64_t n, float fill, float (&v)[8])
{
    if (base == nullptr || 8 * i >= n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fill;
    } else if (bf16) {
        Vec8<true> t;
        if (8 * i + 8 <= n) t.load(base, i);
        else t.load_tail(base, i, n);
        t.get(v);
    } else {
        Vec8<false> t;
        if (8 * i + 8 <= n) t.load(base, i);
        else t.load_tail(base, i, n);
        t.get(v);
    }
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sum over the block (`buf`: one float per warp; two buffers used in turn need one
// barrier per sum).
__device__ __forceinline__ float block_sum(float x, float *buf)
{
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < (blockDim.x >> 5) ? buf[lane] : 0.0f);
}

// Eight elements as four packed pairs.
template <bool BF16>
__device__ __forceinline__ void get_pairs(const Vec8<BF16> &w, float2 (&v)[4])
{
    float t[8];
    w.get(t);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(t[2 * e], t[2 * e + 1]);
}

template <bool BF16>
__device__ __forceinline__ void set_pairs(Vec8<BF16> &w, const float2 (&v)[4])
{
    float t[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[2 * e] = v[e].x, t[2 * e + 1] = v[e].y;
    w.set(t);
}

__device__ __forceinline__ void param_pairs(const void *base, bool bf16, int64_t i, int64_t n, float fill, float2 (&v)[4])
{
    float t[8];
    load_params(base, bf16, i, n, fill, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(t[2 * e], t[2 * e + 1]);
}

__device__ __forceinline__ float2 sum_pairs(float2 s, const float2 (&v)[4])
{
    return add2(s, add2(add2(v[0], v[1]), add2(v[2], v[3])));
}

struct NormParams {
    int64_t rows, n;
    const void *X;
    int64_t ldx;
    const void *gamma, *beta;
    int params_bf16;
    float eps;
    void *Y;
    int64_t ldy;
    float *mean, *rstd;
    int stages;       // ring form: rows of the ring
    int *status;      // device status word (first error wins)
    uint64_t timeout_ns;
};

// Sum and centred sum of squares over this thread's V vectors (vector t + k * team).
template <bool XB, int V>
__device__ __forceinline__ float thread_sum(const Vec8<XB> (&w)[V])
{
    float2 s = both(0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        float2 v[4];
        get_pairs(w[k], v);
        s = sum_pairs(s, v);
    }
    return s.x + s.y;
}

template <bool XB, int V>
__device__ __forceinline__ float thread_squares(const Vec8<XB> (&w)[V], float mean, int t, int team, int64_t n)
{
    const float2 shift = both(-mean);
    float2 q = both(0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = t + k * team;
        float2 v[4];
        get_pairs(w[k], v);
        if (8 * i + 8 <= n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 d = add2(v[e], shift);
                q = fma2(d, d, q);
            }
        } else {  // the row ends inside (or before) this vector
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float c = 8 * i + 2 * e < n ? v[e].x - mean : 0.0f, d = 8 * i + 2 * e + 1 < n ? v[e].y - mean : 0.0f;
                q = fma2(make_float2(c, d), make_float2(c, d), q);
            }
        }
    }
    return q.x + q.y;
}

// Y of a row, and its statistics. `held`: the parameters of this thread's vectors, where
// it keeps them.
template <bool XB, bool YB, int V, bool HELD>
__device__ __forceinline__ void write_row(const NormParams &p, int64_t row, const Vec8<XB> (&w)[V], float mean, float rstd,
                                          int t, int team, const float2 (*g)[4], const float2 (*b)[4])
{
    const float2 shift = both(-mean), scale = both(rstd);
    void *y = const_cast<void *>(row_at(p.Y, row, p.ldy, YB));
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = t + k * team;
        if (8 * i >= p.n) continue;
        float2 v[4], gk[4], bk[4];
        get_pairs(w[k], v);
        if constexpr (!HELD) {
            param_pairs(p.gamma, p.params_bf16, i, p.n, 1.0f, gk);
            param_pairs(p.beta, p.params_bf16, i, p.n, 0.0f, bk);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = fma2(mul2(add2(v[e], shift), scale), HELD ? g[k][e] : gk[e], HELD ? b[k][e] : bk[e]);
        Vec8<YB> o;
        set_pairs(o, v);
        if (8 * i + 8 <= p.n) o.store(y, i);
        else o.store_tail(y, i, p.n);
    }
    if (t == 0) {
        if (p.mean != nullptr) p.mean[row] = mean;
        if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
}

template <bool XB, int V>
__device__ __forceinline__ void load_row(Vec8<XB> (&w)[V], const void *x, int t, int team, int64_t n)
{
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = t + k * team;
        if (8 * i + 8 <= n) w[k].load(x, i);
        else if (8 * i < n) w[k].load_tail(x, i, n);
        else w[k].clear();
    }
}

// Forward, many short rows (at most 1024 elements): a warp per row, no barriers, four
// vectors a lane at once (V of each of 4 / V rows), so that enough loads are in flight.
// The variance is a second pass over the registers, of x - mean, so rows far from zero
// lose nothing.
template <bool XB, bool YB, int V>
__global__ void __launch_bounds__(128, 5) bm_layernorm_warp_kernel(const NormParams p)
{
    constexpr int R = 4 / V;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * R;
    for (int64_t row = (blockIdx.x * static_cast<int64_t>(4) + (threadIdx.x >> 5)) * R; row < p.rows; row += step) {
        Vec8<XB> w[R][V];
#pragma unroll
        for (int q = 0; q < R; ++q)  // (a row past the last reads the last again)
            load_row<XB, V>(w[q], row_at(p.X, min(row + q, p.rows - 1), p.ldx, XB), lane, 32, p.n);
        float mean[R], rstd[R];
#pragma unroll
        for (int q = 0; q < R; ++q) mean[q] = warp_sum(thread_sum(w[q])) * inv_n;
#pragma unroll
        for (int q = 0; q < R; ++q) rstd[q] = rsqrtf(warp_sum(thread_squares(w[q], mean[q], lane, 32, p.n)) * inv_n + p.eps);
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (row + q < p.rows) write_row<XB, YB, V, false>(p, row + q, w[q], mean[q], rstd[q], lane, 32, nullptr, nullptr);
    }
}

// Copies `bytes` (a multiple of 16, both sides 16-byte aligned) into shared memory,
// counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

constexpr int NORM_MAX_STAGES = 4;  // rows of a ring; their mbarriers take the first 32 bytes of shared memory
constexpr int NORM_RING_THREADS = 640;

// Forward, many rows: a block per row, whose rows come by bulk copies into a ring, several
// ahead, so that the barrier a row costs is not also a wait for memory; the parameters
// stay in registers. One barrier: each warp takes the mean m_w and the centred sum of
// squares q_w of its own n_w elements, and the block's are
//   mean = sum n_w m_w / n,  squares = sum (q_w + n_w (m_w - mean)^2).
// Two rows at a time: the chains of shuffles of both run side by side. A row's last, partly
// filled vector is not copied (the copy would run past the row); its thread loads it from
// global memory.
//
// 16384 x 5120 BF16 60.1 us, 5.6 TB/s (one row at a time 65.3; a device copy of the same
// bytes 52.3). Tried against it: eight stages, 60.8; three blocks per SM in 64 registers,
// 79; register loads by a block per row, 82; a warp per row with the row in registers, 240
// (the compiler spills 80 row registers).
template <bool XB, bool YB, int V>
__global__ void __launch_bounds__(NORM_RING_THREADS) bm_layernorm_ring_kernel(const NormParams p)
{
    constexpr int R = 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 buf[2][R][32];
    const int t = threadIdx.x, team = blockDim.x, lane = t & 31, warp = t >> 5;
    // elements of warp w (lane w of the final sums; 0 past the block's warps)
    auto warp_count = [&](int w) {
        int count = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int first = (w * 32 + k * team) * 8;
            count += max(0, min(256, static_cast<int>(p.n) - first));
        }
        return w < team >> 5 ? static_cast<float>(count) : 0.0f;
    };
    const float own_count = warp_count(warp), lane_count = warp_count(lane);
    const float inv_own = own_count > 0.0f ? 1.0f / own_count : 0.0f;
    const int whole = static_cast<int>(p.n / 8);
    constexpr int XV = XB ? 16 : 32;  // bytes of a vector
    const uint32_t stage_bytes = static_cast<uint32_t>(whole) * XV;
    const uint32_t bar0 = smem_addr(smem), ring = bar0 + 8 * NORM_MAX_STAGES;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    if (t == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(bar0 + 8u * s, 1);
        fence_barrier_init();
    }
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();
    auto fill = [&](int64_t row, int s) {  // thread 0
        mbar_arrive_expect_tx(bar0 + 8u * s, stage_bytes);
        bulk_load(ring + static_cast<uint32_t>(s) * stage_bytes, row_at(p.X, row, p.ldx, XB), stage_bytes, bar0 + 8u * s);
    };
    if (t == 0) {
        int64_t row = blockIdx.x;
        for (int s = 0; s < p.stages && row < p.rows; ++s, row += gridDim.x) fill(row, s);
    }
    float2 g[V][4], b[V][4];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        param_pairs(p.gamma, p.params_bf16, t + k * team, p.n, 1.0f, g[k]);
        param_pairs(p.beta, p.params_bf16, t + k * team, p.n, 0.0f, b[k]);
    }
    int s = 0, turn = 0;
    uint32_t parity = 0;
    bool ok = true;
    const int64_t step = gridDim.x;
    for (int64_t row = blockIdx.x; row < p.rows && ok; row += R * step, turn ^= 1) {
        Vec8<XB> w[R][V];
        float warp_mean[R], warp_squares[R];
        int stage[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = row + q * step;
            stage[q] = s;
            if (r < p.rows) {
                ok = wait_one(bar0 + 8u * s, parity, nullptr, p.timeout_ns) && ok;
                const uint8_t *x = smem + 8 * NORM_MAX_STAGES + static_cast<uint32_t>(s) * stage_bytes;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int i = t + k * team;
                    if (i < whole) w[q][k].load(x, i);
                    else if (8 * i < p.n) w[q][k].load_tail(row_at(p.X, r, p.ldx, XB), i, p.n);
                    else w[q][k].clear();
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) w[q][k].clear();
            }
            if (++s == p.stages) {
                s = 0;
                parity ^= 1u;
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) warp_mean[q] = warp_sum(thread_sum(w[q])) * inv_own;
#pragma unroll
        for (int q = 0; q < R; ++q) warp_squares[q] = warp_sum(thread_squares(w[q], warp_mean[q], t, team, p.n));
        if (lane == 0) {
#pragma unroll
            for (int q = 0; q < R; ++q) buf[turn][q][warp] = make_float2(warp_mean[q], warp_squares[q]);
        }
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (t == 0) {  // the rows' stages are read: their next rows may come in
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t next = row + (q + p.stages) * step;
                if (next < p.rows) fill(next, stage[q]);
            }
        }
        float mean[R], rstd[R];
        float2 o[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            o[q] = lane_count > 0.0f ? buf[turn][q][lane] : make_float2(0.0f, 0.0f);
            mean[q] = warp_sum(lane_count * o[q].x) * inv_n;
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float d = o[q].x - mean[q];
            rstd[q] = rsqrtf(warp_sum(fmaf(lane_count * d, d, o[q].y)) * inv_n + p.eps);
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (row + q * step < p.rows) write_row<XB, YB, V, true>(p, row + q * step, w[q], mean[q], rstd[q], t, team, g, b);
    }
    if (!ok) {
        if (p.status != nullptr) atomicCAS(p.status, 0, DEV_ERR_TIMEOUT);
        spin_ns(100000);  // copies in flight land before shared memory is released
    }
}

// Forward, few rows: a block per row, so that one row's latency is short.
template <bool XB, bool YB, int V>
__global__ void __launch_bounds__(1024) bm_layernorm_kernel(const NormParams p)
{
    __shared__ float buf[2][32];
    griddep_launch_dependents();
    const float inv_n = 1.0f / static_cast<float>(p.n);
    griddep_wait();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        Vec8<XB> w[V];
        load_row<XB, V>(w, row_at(p.X, row, p.ldx, XB), threadIdx.x, blockDim.x, p.n);
        constexpr bool HELD = V <= 2;  // (loaded beside the row, not after the statistics)
        float2 g[HELD ? V : 1][4], b[HELD ? V : 1][4];
        if constexpr (HELD) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                param_pairs(p.gamma, p.params_bf16, threadIdx.x + k * blockDim.x, p.n, 1.0f, g[k]);
                param_pairs(p.beta, p.params_bf16, threadIdx.x + k * blockDim.x, p.n, 0.0f, b[k]);
            }
        }
        const float mean = block_sum(thread_sum(w), buf[0]) * inv_n;
        const float rstd =
            rsqrtf(block_sum(thread_squares(w, mean, threadIdx.x, blockDim.x, p.n), buf[1]) * inv_n + p.eps);
        write_row<XB, YB, V, HELD>(p, row, w, mean, rstd, threadIdx.x, blockDim.x, g, b);
    }
}

// Forward for rows longer than the register form holds: the block reads the row three
// times (it is then in L2).
template <bool XB, bool YB>
__global__ void __launch_bounds__(1024) bm_layernorm_long_kernel(const NormParams p)
{
    __shared__ float buf[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const float inv_n = 1.0f / static_cast<float>(p.n);
    const int64_t nvec = (p.n + 7) / 8;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const void *x = row_at(p.X, row, p.ldx, XB);
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x) {
            Vec8<XB> w;
            if (8 * i + 8 <= p.n) w.load(x, i);
            else w.load_tail(x, i, p.n);
            float v[8];
            w.get(v);
            s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        const float mean = block_sum(s, buf[0]) * inv_n;
        float q = 0.0f;
        for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x) {
            Vec8<XB> w;
            if (8 * i + 8 <= p.n) w.load(x, i);
            else w.load_tail(x, i, p.n);
            float v[8], d = 0.0f;
            w.get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = 8 * i + e < p.n ? v[e] - mean : 0.0f;
                d = fmaf(c, c, d);
            }
            q += d;
        }
        const float rstd = rsqrtf(block_sum(q, buf[1]) * inv_n + p.eps);
        void *y = const_cast<void *>(row_at(p.Y, row, p.ldy, YB));
        for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x) {
            Vec8<XB> w;
            if (8 * i + 8 <= p.n) w.load(x, i);
            else w.load_tail(x, i, p.n);
            float v[8], g[8], b[8];
            w.get(v);
            load_params(p.gamma, p.params_bf16, i, p.n, 1.0f, g);
            load_params(p.beta, p.params_bf16, i, p.n, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - mean) * rstd, g[e], b[e]);
            Vec8<YB> o;
            o.set(v);
            if (8 * i + 8 <= p.n) o.store(y, i);
            else o.store_tail(y, i, p.n);
        }
        if (threadIdx.x == 0) {
            if (p.mean != nullptr) p.mean[row] = mean;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
    }
}

struct NormBwdParams {
    int64_t rows, n;
    const void *dY;
    int64_t lddy;
    const void *X;
    int64_t ldx;
    const void *gamma;
    int params_bf16;
    const float *mean, *rstd;
    const void *dres;
    int64_t lddres;
    void *dX;
    int64_t lddx;
    float *partial;   // [2][gridDim.x][ld]: dgamma's and dbeta's sums of each block, or null
    int64_t ld, plane;
    int stages;       // rows of the ring
    int *status;      // device status word (first error wins)
    uint64_t timeout_ns;
};

// Backward. One block holds a row (V vectors of 8 columns per thread) and visits rows
// gridDim apart; each thread owns its columns throughout, so their sums stay in registers
// until the block's last row and go out once. The rows of X, dY and dres come by bulk
// copies into a ring of `stages` rows, several ahead, so that the one barrier a row costs
// is not also a wait for memory. 8192 x 5120 BF16 with dres: 62 us, 5.4 TB/s, of which the
// column sums are 6 (105 with register loads); 16384 rows 113 us, 5.9 TB/s.
//
// Shared memory: mbarriers (32 bytes), then per stage x, dy, dres (dres only when given),
// each ceil(n / 8) vectors. A row's last, partly filled vector is not copied (the copy
// would run past the row); its thread loads it from global memory.
//
// With two vectors a thread x and dy are read from the ring again for dX rather than held.
//
// The next kernel may start as blocks end, not as they begin: blocks of the column sums
// that came in at once held places of this kernel's own (with the sums, 16384 x 2048:
// 63 us so and 51 now, 32768 x 256: 38 and 30).
template <bool XB, bool YB, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : 1) bm_layernorm_backward_kernel(const NormBwdParams p)
{
    constexpr bool HELD = V == 1;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float buf[2][2][32];
    const int t = threadIdx.x, team = blockDim.x, lane = t & 31, warps = team >> 5;
    const int nvec = static_cast<int>((p.n + 7) / 8), whole = static_cast<int>(p.n / 8);
    constexpr int XV = XB ? 16 : 32, YV = YB ? 16 : 32;  // bytes of a vector
    const uint32_t x_bytes = static_cast<uint32_t>(nvec) * XV, y_bytes = static_cast<uint32_t>(nvec) * YV;
    const uint32_t stage_bytes = x_bytes * (p.dres != nullptr ? 2 : 1) + y_bytes;
    const uint32_t bar0 = smem_addr(smem), ring = bar0 + 8 * NORM_MAX_STAGES;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    if (t == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(bar0 + 8u * s, 1);
        fence_barrier_init();
    }
    __syncthreads();
    griddep_wait();

    // thread 0: the row's whole vectors into stage s
    auto fill = [&](int64_t row, int s) {
        if (whole == 0) return;
        const uint32_t dst = ring + static_cast<uint32_t>(s) * stage_bytes, bar = bar0 + 8u * s;
        const uint32_t xb = static_cast<uint32_t>(whole) * XV, yb = static_cast<uint32_t>(whole) * YV;
        mbar_arrive_expect_tx(bar, xb * (p.dres != nullptr ? 2u : 1u) + yb);
        bulk_load(dst, row_at(p.X, row, p.ldx, XB), xb, bar);
        bulk_load(dst + x_bytes, row_at(p.dY, row, p.lddy, YB), yb, bar);
        if (p.dres != nullptr) bulk_load(dst + x_bytes + y_bytes, row_at(p.dres, row, p.lddres, XB), xb, bar);
    };
    // vector i of x and dy
    auto load_xy = [&](int i, int64_t row, const uint8_t *x, const uint8_t *dy, float2 (&a)[4], float2 (&b)[4]) {
        Vec8<XB> wx;
        Vec8<YB> wy;
        if (i < whole) wx.load(x, i), wy.load(dy, i);
        else wx.load_tail(row_at(p.X, row, p.ldx, XB), i, p.n), wy.load_tail(row_at(p.dY, row, p.lddy, YB), i, p.n);
        get_pairs(wx, a);
        get_pairs(wy, b);
    };
    if (t == 0) {
        int64_t row = blockIdx.x;
        for (int s = 0; s < p.stages && row < p.rows; ++s, row += gridDim.x) fill(row, s);
    }
    float2 g[V][4], dg[V][4], db[V][4];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        param_pairs(p.gamma, p.params_bf16, t + k * team, p.n, 1.0f, g[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) dg[k][e] = db[k][e] = both(0.0f);
    }
    int turn = 0, s = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        if (whole > 0) ok = wait_one(bar0 + 8u * s, parity, nullptr, p.timeout_ns);
        const uint8_t *x = smem + 8 * NORM_MAX_STAGES + static_cast<uint32_t>(s) * stage_bytes, *dy = x + x_bytes,
                      *res = dy + y_bytes;
        const float2 shift = both(-mean), scale = both(rstd);
        float2 xh[HELD ? V : 1][4], u[HELD ? V : 1][4], s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = t + k * team;
            if (i >= nvec) continue;
            float2 d[4];
            float2 (&xk)[4] = xh[HELD ? k : 0], (&uk)[4] = u[HELD ? k : 0];
            load_xy(i, row, x, dy, xk, d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xk[e] = mul2(add2(xk[e], shift), scale);
                uk[e] = mul2(d[e], g[k][e]);  // (0 past the row's end, where dy is)
                s1 = add2(s1, uk[e]);
                s2 = fma2(uk[e], xk[e], s2);
                dg[k][e] = fma2(d[e], xk[e], dg[k][e]);
                db[k][e] = add2(db[k][e], d[e]);
            }
        }
        const float a1 = warp_sum(s1.x + s1.y), a2 = warp_sum(s2.x + s2.y);
        if (lane == 0) {
            buf[turn][0][t >> 5] = a1;
            buf[turn][1][t >> 5] = a2;
        }
        if (!__syncthreads_and(ok)) break;
        // every thread is past the previous row's stage: its next row may come in
        if (t == 0 && row != blockIdx.x) {
            const int64_t next = row + static_cast<int64_t>(p.stages - 1) * gridDim.x;
            if (next < p.rows) fill(next, s == 0 ? p.stages - 1 : s - 1);
        }
        const float2 m1 = both(-warp_sum(lane < warps ? buf[turn][0][lane] : 0.0f) * inv_n);
        const float2 m2 = both(-warp_sum(lane < warps ? buf[turn][1][lane] : 0.0f) * inv_n);
        void *dx = const_cast<void *>(row_at(p.dX, row, p.lddx, XB));
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = t + k * team;
            if (i >= nvec) continue;
            float2 r[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
            if (p.dres != nullptr) {
                Vec8<XB> wr;
                if (i < whole) wr.load(res, i);
                else wr.load_tail(row_at(p.dres, row, p.lddres, XB), i, p.n);
                get_pairs(wr, r);
            }
            float2 (&xk)[4] = xh[HELD ? k : 0], (&uk)[4] = u[HELD ? k : 0];
            if constexpr (!HELD) {
                load_xy(i, row, x, dy, xk, uk);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xk[e] = mul2(add2(xk[e], shift), scale);
                    uk[e] = mul2(uk[e], g[k][e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = fma2(scale, fma2(xk[e], m2, add2(uk[e], m1)), r[e]);
            Vec8<XB> o;
            set_pairs(o, r);
            if (i < whole) o.store(dx, i);
            else o.store_tail(dx, i, p.n);
        }
        if (++s == p.stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    if (!ok) {
        if (p.status != nullptr) atomicCAS(p.status, 0, DEV_ERR_TIMEOUT);
        spin_ns(100000);  // copies in flight land before shared memory is released
        return;
    }
    if (p.partial == nullptr) return;
    float *out = p.partial + blockIdx.x * p.ld;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int64_t i = t + k * team;
        if (i >= nvec) continue;
        // (ld is a multiple of 8: whole vectors, the columns past n are never read)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<float4 *>(out + 8 * i + 4 * h) =
                make_float4(dg[k][2 * h].x, dg[k][2 * h].y, dg[k][2 * h + 1].x, dg[k][2 * h + 1].y);
            *reinterpret_cast<float4 *>(out + p.plane + 8 * i + 4 * h) =
                make_float4(db[k][2 * h].x, db[k][2 * h].y, db[k][2 * h + 1].x, db[k][2 * h + 1].y);
        }
    }
}

// Rows longer than the register form holds: row sums first (the block reads the row
// twice), and the column sums by a kernel over column strips.
template <bool XB, bool YB>
__global__ void __launch_bounds__(1024) bm_layernorm_backward_long_kernel(const NormBwdParams p)
{
    __shared__ float buf[2][2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    const int64_t nvec = (p.n + 7) / 8;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const void *x = row_at(p.X, row, p.ldx, XB), *dy = row_at(p.dY, row, p.lddy, YB);
        void *dx = const_cast<void *>(row_at(p.dX, row, p.lddx, XB));
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x) {
                const bool full = 8 * i + 8 <= p.n;
                Vec8<XB> wx, wr;
                Vec8<YB> wy;
                if (full) wx.load(x, i), wy.load(dy, i);
                else wx.load_tail(x, i, p.n), wy.load_tail(dy, i, p.n);
                float v[8], d[8], g[8], r[8];
                wx.get(v);
                wy.get(d);
                load_params(p.gamma, p.params_bf16, i, p.n, 1.0f, g);
                if (pass == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float u = d[e] * g[e];
                        s1 += u;
                        s2 = fmaf(u, (v[e] - mean) * rstd, s2);
                    }
                    continue;
                }
                wr.clear();
                if (p.dres != nullptr) {
                    if (full) wr.load(row_at(p.dres, row, p.lddres, XB), i);
                    else wr.load_tail(row_at(p.dres, row, p.lddres, XB), i, p.n);
                }
                wr.get(r);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = fmaf(rstd, d[e] * g[e] - s1 - (v[e] - mean) * rstd * s2, r[e]);
                wr.set(r);
                if (full) wr.store(dx, i);
                else wr.store_tail(dx, i, p.n);
            }
            if (pass == 0) {
                s1 = warp_sum(s1);
                s2 = warp_sum(s2);
                if (lane == 0) {
                    buf[turn][0][threadIdx.x >> 5] = s1;
                    buf[turn][1][threadIdx.x >> 5] = s2;
                }
                __syncthreads();
                s1 = warp_sum(lane < warps ? buf[turn][0][lane] : 0.0f) * inv_n;
                s2 = warp_sum(lane < warps ? buf[turn][1][lane] : 0.0f) * inv_n;
            }
        }
    }
}

// Column sums of one strip of 8 * blockDim.x columns (blockIdx.x: rows may have more than
// 65535 strips) over the rows blockIdx.y, + gridDim.y, ...: for the long rows above. Runs
// before dX is written, since dX may be dY.
template <bool XB, bool YB>
__global__ void __launch_bounds__(256) bm_layernorm_columns_kernel(const NormBwdParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (8 * i >= p.n) return;
    float dg[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[e] = db[e] = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        Vec8<XB> wx;
        Vec8<YB> wy;
        const void *x = row_at(p.X, row, p.ldx, XB), *dy = row_at(p.dY, row, p.lddy, YB);
        if (8 * i + 8 <= p.n) wx.load(x, i), wy.load(dy, i);
        else wx.load_tail(x, i, p.n), wy.load_tail(dy, i, p.n);
        const float mean = p.mean[row], rstd = p.rstd[row];
        float v[8], d[8];
        wx.get(v);
        wy.get(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dg[e] = fmaf(d[e], (v[e] - mean) * rstd, dg[e]);
            db[e] += d[e];
        }
    }
    float *out = p.partial + blockIdx.y * p.ld + 8 * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        out[e] = dg[e];
        out[p.plane + e] = db[e];
    }
}

// ---------------------------------------------------------------- act(z~)
struct ActParams {
    int64_t rows, n;
    const uint8_t *Q;
    int64_t ldq;
    const uint8_t *S;
    int64_t katoms;
    int act;
    void *H;
    int64_t ldh;
};

// Thread (x, y) of a block takes 16 columns of every (gridDim.y * blockDim.y)-th row:
// one 16-byte load of codes, one scale byte, two (bf16) or four (fp32) 16-byte stores, the
// next row's codes loaded ahead of this row's arithmetic. GELU takes about 11 instructions
// an element beside the special functions, and arithmetic is what it waits for: of 8.5
// cycles between a warp's instructions 2.3 are for a math pipe that is busy, 2.3 for the
// scheduler, 1.2 for a result, 0.7 for loads. No pipe is full over the whole time (issue
// slots 68 % of active cycles, ALU 42, FMA 37, special functions 15). 4096 x 16384 to BF16
// takes 45.5 us (4.5 TB/s), decoding alone 36 (5.6). With scalar arithmetic (21
// instructions) and four rows at a time in 101 registers: 63.6 us, at 58 % of the slots.
template <bool HB>
__global__ void __launch_bounds__(256, 4) bm_act_mxfp8_kernel(const ActParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t c = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) * 16;
    if (c >= p.n) return;
    const int left = p.n - c < 16 ? static_cast<int>(p.n - c) : 16;
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.y;
    int64_t r = blockIdx.y * static_cast<int64_t>(blockDim.y) + threadIdx.y;
    if (r >= p.rows) return;
    const uint8_t *src = p.Q + r * p.ldq + c;
    char *dst = static_cast<char *>(p.H) + (r * p.ldh + c) * (HB ? 2 : 4);
    const int64_t src_step = step * p.ldq, dst_step = step * p.ldh * (HB ? 2 : 4);
    const uint8_t *scales = p.S + (c >> 7) * 512 + ((c >> 5) & 3);
    auto codes_at = [&](const uint8_t *at) {
        if (left == 16) return __ldcs(reinterpret_cast<const uint4 *>(at));
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < left) u[e >> 2] |= static_cast<uint32_t>(at[e]) << (8 * (e & 3));
        return make_uint4(u[0], u[1], u[2], u[3]);
    };
    auto scale_at = [&](int64_t row) {
        return static_cast<uint32_t>(scales[(row >> 7) * p.katoms * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4]);
    };
    uint4 next = codes_at(src);
    uint32_t next_scale = scale_at(r);
    while (true) {
        const uint4 q = next;
        const float2 scale = both(ue8m0_value(next_scale));
        r += step;
        src += src_step;
        const bool more = r < p.rows;
        if (more) {
            next = codes_at(src);
            next_scale = scale_at(r);
        }
        float v[16];
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float d[4];
            e4m3x4_values(u[e], d);
            const float2 a = mul2(make_float2(d[0], d[1]), scale), b = mul2(make_float2(d[2], d[3]), scale);
            v[4 * e] = a.x, v[4 * e + 1] = a.y, v[4 * e + 2] = b.x, v[4 * e + 3] = b.y;
        }
        with_act(p.act, [&](auto tag) { act_values<decltype(tag)::value, 16>(v); });
        if (left == 16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Vec8<HB> o;
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = v[8 * h + e];
                o.set(w);
                o.store(dst, h);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (e >= left) continue;
                if constexpr (HB) reinterpret_cast<__nv_bfloat16 *>(dst)[e] = __float2bfloat16_rn(v[e]);
                else reinterpret_cast<float *>(dst)[e] = v[e];
            }
        }
        if (!more) return;
        dst += dst_step;
    }
}

}  // namespace bm
