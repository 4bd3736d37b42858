// bm_norm_kernel.cuh -- layer norm over rows, forward and backward, the final sum of
// partial column sums, and the activation recomputed from an MXFP8 checkpoint.
//
// All of them are bound by HBM: each input is read once and each output written once,
// in 16-byte vectors of the row held in registers between the passes over it.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "bm_act.cuh"
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

// Sum over a row's team: a warp, or the whole block (`buf`: one float per warp, two
// buffers used in turn, so one barrier per sum is enough).
template <bool WARP>
__device__ __forceinline__ float team_sum(float x, float *buf)
{
    x = warp_sum(x);
    if constexpr (WARP) return x;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < warps ? buf[lane] : 0.0f);
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
};

// Forward. A team (a warp for short rows, else the block) holds a row as V vectors per
// thread and visits rows gridDim apart; the parameters stay in registers. The variance
// is a second pass over the registers, of x - mean, so rows far from zero lose nothing.
template <bool XB, bool YB, int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) bm_layernorm_kernel(const NormParams p)
{
    __shared__ float buf[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int team = WARP ? 32 : blockDim.x;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t teams = WARP ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
    const int64_t first = WARP ? blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    float g[V][8], b[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        load_params(p.gamma, p.params_bf16, t + k * team, p.n, 1.0f, g[k]);
        load_params(p.beta, p.params_bf16, t + k * team, p.n, 0.0f, b[k]);
    }
    for (int64_t row = first; row < p.rows; row += teams) {
        const void *x = row_at(p.X, row, p.ldx, XB);
        Vec8<XB> w[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t i = t + k * team;
            if (8 * i + 8 <= p.n) w[k].load(x, i);
            else if (8 * i < p.n) w[k].load_tail(x, i, p.n);
            else w[k].clear();
        }
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float v[8];
            w[k].get(v);
            s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        const float mean = team_sum<WARP>(s, buf[0]) * inv_n;
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t i = t + k * team;
            float v[8];
            w[k].get(v);
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = 8 * i + e < p.n ? v[e] - mean : 0.0f;
                d = fmaf(c, c, d);
            }
            q += d;
        }
        const float rstd = rsqrtf(team_sum<WARP>(q, buf[1]) * inv_n + p.eps);
        void *y = const_cast<void *>(row_at(p.Y, row, p.ldy, YB));
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t i = t + k * team;
            if (8 * i >= p.n) continue;
            float v[8];
            w[k].get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - mean) * rstd, g[k][e], b[k][e]);
            Vec8<YB> o;
            o.set(v);
            if (8 * i + 8 <= p.n) o.store(y, i);
            else o.store_tail(y, i, p.n);
        }
        if (t == 0) {
            if (p.mean != nullptr) p.mean[row] = mean;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
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
        const float mean = team_sum<false>(s, buf[0]) * inv_n;
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
        const float rstd = rsqrtf(team_sum<false>(q, buf[1]) * inv_n + p.eps);
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
};

// Backward. One block holds a row (V vectors of x, dy per thread) and visits rows gridDim
// apart; each thread owns its columns throughout, so their sums stay in registers until
// the block's last row and go out once.
template <bool XB, bool YB, int V>
__global__ void __launch_bounds__(1024) bm_layernorm_backward_kernel(const NormBwdParams p)
{
    __shared__ float buf[2][2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x, team = blockDim.x, lane = t & 31, warps = team >> 5;
    const float inv_n = 1.0f / static_cast<float>(p.n);
    float g[V][8], dg[V][8], db[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        load_params(p.gamma, p.params_bf16, t + k * team, p.n, 1.0f, g[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[k][e] = db[k][e] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const void *x = row_at(p.X, row, p.ldx, XB), *dy = row_at(p.dY, row, p.lddy, YB);
        Vec8<XB> wx[V];
        Vec8<YB> wy[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t i = t + k * team;
            if (8 * i + 8 <= p.n) {
                wx[k].load(x, i);
                wy[k].load(dy, i);
            } else if (8 * i < p.n) {
                wx[k].load_tail(x, i, p.n);
                wy[k].load_tail(dy, i, p.n);
            } else {
                wx[k].clear();
                wy[k].clear();
            }
        }
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (8 * (t + k * team) >= p.n) continue;
            float v[8], d[8];
            wx[k].get(v);
            wy[k].get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (v[e] - mean) * rstd, u = d[e] * g[k][e];  // (dy is 0 past n)
                s1 += u;
                s2 = fmaf(u, xh, s2);
                dg[k][e] = fmaf(d[e], xh, dg[k][e]);
                db[k][e] += d[e];
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) {
            buf[turn][0][t >> 5] = s1;
            buf[turn][1][t >> 5] = s2;
        }
        __syncthreads();
        s1 = warp_sum(lane < warps ? buf[turn][0][lane] : 0.0f) * inv_n;
        s2 = warp_sum(lane < warps ? buf[turn][1][lane] : 0.0f) * inv_n;
        void *dx = const_cast<void *>(row_at(p.dX, row, p.lddx, XB));
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t i = t + k * team;
            if (8 * i >= p.n) continue;
            float v[8], d[8], r[8];
            wx[k].get(v);
            wy[k].get(d);
            const bool full = 8 * i + 8 <= p.n;
            if (p.dres != nullptr) {
                Vec8<XB> wr;
                if (full) wr.load(row_at(p.dres, row, p.lddres, XB), i);
                else wr.load_tail(row_at(p.dres, row, p.lddres, XB), i, p.n);
                wr.get(r);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (v[e] - mean) * rstd, u = d[e] * g[k][e];
                r[e] = fmaf(rstd, u - s1 - xh * s2, r[e]);
            }
            Vec8<XB> o;
            o.set(r);
            if (full) o.store(dx, i);
            else o.store_tail(dx, i, p.n);
        }
    }
    if (p.partial == nullptr) return;
    float *out = p.partial + blockIdx.x * p.ld;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int64_t i = t + k * team;
        if (8 * i >= p.n) continue;
        // (ld is a multiple of 8: whole vectors, the columns past n are never read)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<float4 *>(out + 8 * i + 4 * h) =
                make_float4(dg[k][4 * h], dg[k][4 * h + 1], dg[k][4 * h + 2], dg[k][4 * h + 3]);
            *reinterpret_cast<float4 *>(out + p.plane + 8 * i + 4 * h) =
                make_float4(db[k][4 * h], db[k][4 * h + 1], db[k][4 * h + 2], db[k][4 * h + 3]);
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

// Column sums of one strip of 8 * blockDim.x columns (blockIdx.y) over the rows
// blockIdx.x, + gridDim.x, ...: for the long rows above. Runs before dX is written,
// since dX may be dY.
template <bool XB, bool YB>
__global__ void __launch_bounds__(256) bm_layernorm_columns_kernel(const NormBwdParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t i = blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (8 * i >= p.n) return;
    float dg[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[e] = db[e] = 0.0f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
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
    float *out = p.partial + blockIdx.x * p.ld + 8 * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        out[e] = dg[e];
        out[p.plane + e] = db[e];
    }
}

// out[j] (+)= sum over rows of partial[row][j]; blockIdx.y picks one of two planes. 32
// warps take the rows w, w + 32, ... of 32 columns; their sums are added in warp order.
__global__ void __launch_bounds__(1024)
    bm_column_sums_kernel(const float *partial, int64_t rows, int64_t ld, int64_t plane, int64_t n, float *out0,
                          float *out1, int accumulate);

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
// one 16-byte load of codes, one scale byte, two (bf16) or four (fp32) 16-byte stores.
// ROWS rows are loaded ahead of the arithmetic.
template <bool HB, int ROWS>
__global__ void __launch_bounds__(256) bm_act_mxfp8_kernel(const ActParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t c = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) * 16;
    if (c >= p.n) return;
    const bool full = c + 16 <= p.n;
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.y;
    for (int64_t r0 = blockIdx.y * static_cast<int64_t>(blockDim.y) + threadIdx.y; r0 < p.rows; r0 += step * ROWS) {
        uint4 q[ROWS];
        uint32_t s[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t r = r0 + k * step;
            q[k] = make_uint4(0u, 0u, 0u, 0u);
            s[k] = 0;
            if (r >= p.rows) continue;
            const uint8_t *src = p.Q + r * p.ldq + c;
            if (full) {
                q[k] = __ldcs(reinterpret_cast<const uint4 *>(src));
            } else {
                uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c + e < p.n) u[e >> 2] |= static_cast<uint32_t>(src[e]) << (8 * (e & 3));
                q[k] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            s[k] = p.S[scale_offset(r, c >> 5, 4 * p.katoms)];
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t r = r0 + k * step;
            if (r >= p.rows) continue;
            const float scale = ue8m0_value(s[k]);
            float v[16];
            const uint32_t u[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float d[4];
                e4m3x4_values(u[e], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * e + i] = d[i] * scale;
            }
            with_act(p.act, [&](auto tag) {
                constexpr int ACT = decltype(tag)::value;
                act_values<ACT, 16>(v);
            });
            char *dst = static_cast<char *>(p.H) + (r * p.ldh + c) * (HB ? 2 : 4);
            if (full) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    Vec8<HB> o;
                    float t[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = v[8 * h + e];
                    o.set(t);
                    o.store(dst, h);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (c + e >= p.n) continue;
                    if constexpr (HB) reinterpret_cast<__nv_bfloat16 *>(dst)[e] = __float2bfloat16_rn(v[e]);
                    else reinterpret_cast<float *>(dst)[e] = v[e];
                }
            }
        }
    }
}

}  // namespace bm
