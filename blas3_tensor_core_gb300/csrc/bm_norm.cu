// bm_norm.cu -- layer norm, its backward pass, and the activation recomputed from an
// MXFP8 checkpoint: host side (argument checks, launch shapes) and the column-sum kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "bm.h"
#include "bm_host.h"
#include "bm_norm_kernel.cuh"
#include "bm_ops.h"

using namespace bmh;

namespace bm {

__global__ void __launch_bounds__(1024)
    bm_column_sums_kernel(const float *partial, int64_t rows, int64_t ld, int64_t plane, int64_t n, float *out0,
                          float *out1, int accumulate)
{
    __shared__ float part[32][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = blockIdx.x * static_cast<int64_t>(32) + lane;
    const float *src = partial + blockIdx.y * plane + j;
    float s = 0.0f;
    if (j < n) {
        int64_t r = warp;
        for (; r + 96 < rows; r += 128) {
            const float a = __ldcg(src + r * ld), b = __ldcg(src + (r + 32) * ld);
            const float c = __ldcg(src + (r + 64) * ld), d = __ldcg(src + (r + 96) * ld);
            s += (a + b) + (c + d);
        }
        for (; r < rows; r += 32) s += __ldcg(src + r * ld);
    }
    part[warp][lane] = s;
    __syncthreads();
    // column `warp` of the block, over the 32 warps' sums
    const float total = warp_sum(part[lane][warp]);
    const int64_t out = blockIdx.x * static_cast<int64_t>(32) + warp;
    float *dst = blockIdx.y == 0 ? out0 : out1;
    if (lane == 0 && out < n) dst[out] = accumulate ? dst[out] + total : total;
}

}  // namespace bm

namespace {

bool type_ok(int t) { return t == BM_F32 || t == BM_BF16; }
int64_t esize(int t) { return t == BM_BF16 ? 2 : 4; }

bool ld_ok(int64_t ld, int64_t n) { return ld >= std::max<int64_t>(1, n); }
bool rows16(const void *p, int64_t ld, int t) { return aligned16(p) && (ld * esize(t)) % 16 == 0; }

// Vectors of 8 elements per thread of a row's team, and the team.
struct Team {
    int v;        // 0: the long form
    int threads;  // of the block
    bool warp;    // a warp per row (8 rows per block)
};

// Up to 1024 elements a warp holds a row (4 vectors a lane): no barriers. Longer rows
// take a block with 2 vectors a thread up to 8192 elements, then 4 up to 32768.
Team forward_team(int64_t n)
{
    const int64_t nvec = ceil_div(n, 8);
    if (nvec <= 32) return {1, 256, true};
    if (nvec <= 64) return {2, 256, true};
    if (nvec <= 128) return {4, 256, true};
    if (nvec <= 1024) return {2, static_cast<int>(ceil_div(ceil_div(nvec, 2), 32) * 32), false};
    if (nvec <= 4096) return {4, static_cast<int>(ceil_div(ceil_div(nvec, 4), 32) * 32), false};
    return {0, 1024, false};
}

Team backward_team(int64_t n)
{
    const int64_t nvec = ceil_div(n, 8);
    if (nvec <= 512) return {1, static_cast<int>(ceil_div(nvec, 32) * 32), false};
    if (nvec <= 2048) return {2, static_cast<int>(ceil_div(ceil_div(nvec, 2), 32) * 32), false};
    return {0, 1024, false};
}

// Blocks of the backward kernel: each keeps its own column sums, so the workspace and
// the final sum grow with them.
int64_t backward_blocks(int64_t rows, int64_t n, int sms)
{
    const Team t = backward_team(n);
    const int64_t per_sm = t.v == 0 ? 2 : std::max<int64_t>(1, std::min<int64_t>(8, 1024 / t.threads));
    return std::min<int64_t>(rows, per_sm * sms);
}

int64_t sums_ld(int64_t n) { return ceil_div(n, 8) * 8; }

template <bool XB, bool YB>
bm_status launch_forward(const bm::NormParams &p, int sms, cudaStream_t stream)
{
    const Team t = forward_team(p.n);
    const int64_t per_sm = std::max<int64_t>(1, 2048 / t.threads);
    const int64_t teams = t.warp ? ceil_div(p.rows, 8) : p.rows;
    PdlLaunch l(stream, static_cast<unsigned>(std::min<int64_t>(teams, per_sm * sms)), static_cast<unsigned>(t.threads));
    cudaError_t e;
    if (t.warp) {
        if (t.v == 1) e = cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 1, true>, p);
        else if (t.v == 2) e = cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 2, true>, p);
        else e = cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 4, true>, p);
    } else if (t.v == 2) {
        e = cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 2, false>, p);
    } else if (t.v == 4) {
        e = cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 4, false>, p);
    } else {
        e = cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_long_kernel<XB, YB>, p);
    }
    return launched(e);
}

template <bool XB, bool YB>
bm_status launch_backward(const bm::NormBwdParams &p, int64_t blocks, cudaStream_t stream)
{
    const Team t = backward_team(p.n);
    PdlLaunch l(stream, static_cast<unsigned>(blocks), static_cast<unsigned>(t.threads));
    if (t.v == 1) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_kernel<XB, YB, 1>, p));
    if (t.v == 2) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_kernel<XB, YB, 2>, p));
    if (p.partial != nullptr) {
        PdlLaunch c(stream, static_cast<unsigned>(blocks), 256);
        c.cfg.gridDim.y = static_cast<unsigned>(ceil_div(p.n, 8 * 256));
        const bm_status s = launched(cudaLaunchKernelEx(&c.cfg, bm::bm_layernorm_columns_kernel<XB, YB>, p));
        if (s != BM_OK) return s;
    }
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_long_kernel<XB, YB>, p));
}

template <bool HB>
bm_status launch_act(const bm::ActParams &p, int sms, cudaStream_t stream)
{
    constexpr int kRows = 4;
    const int64_t cols = ceil_div(p.n, 16);
    unsigned tx = 1;
    while (tx < 256 && tx < cols) tx *= 2;
    const unsigned ty = 256 / tx;
    const int64_t bx = ceil_div(cols, tx);
    const int64_t by = std::min<int64_t>(ceil_div(p.rows, ty), std::max<int64_t>(1, ceil_div(8 * static_cast<int64_t>(sms), bx)));
    PdlLaunch l(stream, static_cast<unsigned>(bx), tx);
    l.cfg.gridDim.y = static_cast<unsigned>(by);
    l.cfg.blockDim.y = ty;
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_act_mxfp8_kernel<HB, kRows>, p));
}

}  // namespace

namespace bmh {

bm_status launch_column_sums(const float *partial, int64_t rows, int64_t ld, int64_t plane, int64_t n, float *out0,
                             float *out1, int accumulate, cudaStream_t stream)
{
    PdlLaunch l(stream, static_cast<unsigned>(ceil_div(n, 32)), 1024);
    l.cfg.gridDim.y = out1 != nullptr ? 2u : 1u;
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_column_sums_kernel, partial, rows, ld, plane, n, out0, out1,
                                       accumulate));
}

}  // namespace bmh

extern "C" {

bm_status bm_layernorm(int64_t rows, int64_t n, const void *X, int64_t ldx, bm_dtype x_type, const void *gamma,
                       const void *beta, bm_dtype param_type, float eps, void *Y, int64_t ldy, bm_dtype y_type,
                       float *mean, float *rstd, bm_stream_t stream)
{
    if (rows < 0 || n < 0 || !fits_int32(rows) || !fits_int32(n) || !(eps >= 0.0f)) return BM_ERR_INVALID_VALUE;
    if (!type_ok(x_type) || !type_ok(y_type) || !type_ok(param_type)) return BM_ERR_INVALID_VALUE;
    if (!ld_ok(ldx, n) || !ld_ok(ldy, n)) return BM_ERR_INVALID_VALUE;
    if (rows == 0 || n == 0) return BM_OK;
    if (X == nullptr || Y == nullptr) return BM_ERR_INVALID_VALUE;
    if (!rows16(X, ldx, x_type) || !rows16(Y, ldy, y_type) || !aligned16(gamma) || !aligned16(beta) ||
        (reinterpret_cast<uintptr_t>(mean) & 3u) != 0 || (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0)
        return BM_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    const bm_status s = device_state(&st);
    if (s != BM_OK) return s;
    const bm::NormParams p = {rows, n, X, ldx, gamma, beta, param_type == BM_BF16, eps, Y, ldy, mean, rstd};
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (x_type == BM_BF16)
        return y_type == BM_BF16 ? launch_forward<true, true>(p, st->sm_count, cs)
                                 : launch_forward<true, false>(p, st->sm_count, cs);
    return y_type == BM_BF16 ? launch_forward<false, true>(p, st->sm_count, cs)
                             : launch_forward<false, false>(p, st->sm_count, cs);
}

size_t bm_layernorm_backward_workspace_size(int64_t rows, int64_t n)
{
    if (rows <= 0 || n <= 0) return 0;
    return static_cast<size_t>(2 * backward_blocks(rows, n, sm_count_or_default()) * sums_ld(n)) * sizeof(float);
}

bm_status bm_layernorm_backward(int64_t rows, int64_t n, const void *dY, int64_t lddy, bm_dtype y_type, const void *X,
                                int64_t ldx, bm_dtype x_type, const void *gamma, bm_dtype param_type,
                                const float *mean, const float *rstd, const void *dres, int64_t lddres, void *dX,
                                int64_t lddx, float *dgamma, float *dbeta, int accumulate, void *workspace,
                                size_t workspace_bytes, bm_stream_t stream)
{
    if (rows < 0 || n < 0 || !fits_int32(rows) || !fits_int32(n)) return BM_ERR_INVALID_VALUE;
    if (!type_ok(x_type) || !type_ok(y_type) || !type_ok(param_type)) return BM_ERR_INVALID_VALUE;
    if (!ld_ok(lddy, n) || !ld_ok(ldx, n) || !ld_ok(lddx, n) || (dres != nullptr && !ld_ok(lddres, n)))
        return BM_ERR_INVALID_VALUE;
    if ((dgamma == nullptr) != (dbeta == nullptr)) return BM_ERR_INVALID_VALUE;
    if (workspace_bytes > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return BM_ERR_WORKSPACE;
    if (n == 0 || (rows == 0 && (dgamma == nullptr || accumulate != 0))) return BM_OK;
    if (!aligned16(dgamma) || !aligned16(dbeta)) return BM_ERR_MISALIGNED;
    if (rows > 0) {
        if (dY == nullptr || X == nullptr || dX == nullptr || mean == nullptr || rstd == nullptr) return BM_ERR_INVALID_VALUE;
        if (!rows16(dY, lddy, y_type) || !rows16(X, ldx, x_type) || !rows16(dX, lddx, x_type) || !aligned16(gamma) ||
            (dres != nullptr && !rows16(dres, lddres, x_type)) || (reinterpret_cast<uintptr_t>(mean) & 3u) != 0 ||
            (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0)
            return BM_ERR_MISALIGNED;
        if (dgamma != nullptr && (workspace == nullptr || workspace_bytes < bm_layernorm_backward_workspace_size(rows, n)))
            return BM_ERR_WORKSPACE;
    }
    DeviceState *st = nullptr;
    bm_status s = device_state(&st);
    if (s != BM_OK) return s;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    float *partial = dgamma != nullptr ? static_cast<float *>(workspace) : nullptr;
    const int64_t blocks = backward_blocks(rows, n, st->sm_count), ld = sums_ld(n), plane = blocks * ld;
    if (rows > 0) {
        const bm::NormBwdParams p = {rows, n,    dY,   lddy,   X,  ldx,  gamma,   param_type == BM_BF16,
                                     mean, rstd, dres, lddres, dX, lddx, partial, ld,
                                     plane};
        if (x_type == BM_BF16)
            s = y_type == BM_BF16 ? launch_backward<true, true>(p, blocks, cs) : launch_backward<true, false>(p, blocks, cs);
        else
            s = y_type == BM_BF16 ? launch_backward<false, true>(p, blocks, cs) : launch_backward<false, false>(p, blocks, cs);
        if (s != BM_OK) return s;
    }
    if (dgamma == nullptr) return BM_OK;
    return launch_column_sums(partial, blocks, ld, plane, n, dgamma, dbeta, accumulate, cs);
}

bm_status bm_act_mxfp8(int64_t rows, int64_t n, const void *Q, int64_t ldq, const void *S, bm_act act, void *H,
                       int64_t ldh, bm_ctype h_type, bm_stream_t stream)
{
    if (rows < 0 || n < 0 || !fits_int32(rows) || !fits_int32(n) || !type_ok(h_type)) return BM_ERR_INVALID_VALUE;
    if (act < BM_ACT_NONE || act > BM_ACT_SILU || !ld_ok(ldq, n) || !ld_ok(ldh, n)) return BM_ERR_INVALID_VALUE;
    if (rows == 0 || n == 0) return BM_OK;
    if (Q == nullptr || S == nullptr || H == nullptr) return BM_ERR_INVALID_VALUE;
    if (!aligned16(Q) || !aligned16(S) || ldq % 16 != 0 || !rows16(H, ldh, h_type)) return BM_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    const bm_status s = device_state(&st);
    if (s != BM_OK) return s;
    const bm::ActParams p = {rows, n, static_cast<const uint8_t *>(Q), ldq, static_cast<const uint8_t *>(S),
                             ceil_div(n, 128), act, H, ldh};
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    return h_type == BM_BF16 ? launch_act<true>(p, st->sm_count, cs) : launch_act<false>(p, st->sm_count, cs);
}

}  // extern "C"
