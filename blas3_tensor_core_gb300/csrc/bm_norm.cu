// bm_norm.cu -- layer norm, its backward pass, and the activation recomputed from an
// MXFP8 checkpoint: host side (argument checks, launch shapes) and the column-sum kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "bm.h"
#include "bm_host.h"
#include "bm_norm_kernel.cuh"
#include "bm_ops.h"

using namespace bmh;

namespace bm {

constexpr int SUM_WARPS = 16, SUM_SPLIT = 8;

// out[j] (+)= sum over rows of partial[row][j]; blockIdx.y picks one of two planes. A
// cluster of `split` CTAs takes 128 columns, four per lane; of its split * 16 warps, warp
// w the rows w, w + 16 split, ...; the sums are added in that order, so they do not depend
// on timing. ld is a multiple of 4 and partial on 16 bytes. What bounds it is loads in
// flight, so few columns need several CTAs each; 12 MB of partial sums (from L2) take 8 us.
__global__ void __launch_bounds__(32 * SUM_WARPS)
    bm_column_sums_kernel(const float *partial, int64_t rows, int64_t ld, int64_t plane, int64_t n, float *out0,
                          float *out1, int accumulate, int split)
{
    __shared__ float4 part[SUM_WARPS][32];
    __shared__ float gathered[SUM_SPLIT][128];
    if (split > 1) cluster_arrive();
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, rank = static_cast<int>(blockIdx.x) % split;
    const int64_t first = blockIdx.x / split * static_cast<int64_t>(128);
    const int64_t step = static_cast<int64_t>(SUM_WARPS) * split;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (first + 4 * lane < n) {
        const float *src = partial + blockIdx.y * plane + first + 4 * lane;
        int64_t r = rank * SUM_WARPS + warp;
        auto add = [&](const float4 &v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
        for (; r + 3 * step < rows; r += 4 * step) {
            float4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = __ldcg(reinterpret_cast<const float4 *>(src + (r + q * step) * ld));
#pragma unroll
            for (int q = 0; q < 4; ++q) add(v[q]);
        }
        for (; r < rows; r += step) add(__ldcg(reinterpret_cast<const float4 *>(src + r * ld)));
    }
    part[warp][lane] = s;
    __syncthreads();
    float sum = 0.0f;
    if (t < 128) {
#pragma unroll
        for (int w = 0; w < SUM_WARPS; ++w) sum += reinterpret_cast<const float *>(part[w])[t];
    }
    if (split > 1) {
        cluster_wait();  // CTA 0 has started
        if (t < 128) st_cluster_f1(map_shared_to_rank(smem_addr(&gathered[rank][t]), 0), sum);
        cluster_sync();
        if (rank == 0 && t < 128) {
            sum = 0.0f;
            for (int w = 0; w < split; ++w) sum += gathered[w][t];
        }
    }
    const int64_t j = first + t;
    if (t >= 128 || rank != 0 || j >= n) return;
    float *dst = blockIdx.y == 0 ? out0 : out1;
    dst[j] = accumulate ? dst[j] + sum : sum;
}

}  // namespace bm

namespace {

bool type_ok(int t) { return t == BM_F32 || t == BM_BF16; }
int64_t esize(int t) { return t == BM_BF16 ? 2 : 4; }

bool ld_ok(int64_t ld, int64_t n) { return ld >= std::max<int64_t>(1, n); }
bool rows16(const void *p, int64_t ld, int t) { return aligned16(p) && (ld * esize(t)) % 16 == 0; }

constexpr size_t kRingBytes = 200u * 1024u;  // of an SM's shared memory, for all its blocks' rings

// Forward, many short rows: vectors of 8 elements per lane of a row's warp, 0 for rows
// over 1024 elements. "Many" is four rows per SM.
int warp_vectors(int64_t n)
{
    const int64_t per_lane = ceil_div(ceil_div(n, 8), 32);
    return per_lane <= 1 ? 1 : per_lane <= 2 ? 2 : per_lane <= 4 ? 4 : 0;
}

// Forward, a block per row: threads for 2 vectors each up to 16384 elements, 4 up to
// 32768; 0 (longer rows): the form that reads the row three times.
int block_vectors(int64_t n) { return n <= 16384 ? 2 : n <= 32768 ? 4 : 0; }

int block_threads(int64_t n, int vectors)
{
    return static_cast<int>(ceil_div(ceil_div(ceil_div(n, 8), vectors), 32) * 32);
}

// Backward: threads, vectors, ring and blocks per SM.
struct BackwardShape {
    int v = 0;  // 0: the form that reads the rows twice
    int threads = 0, stages = 0, per_sm = 1;
    size_t smem = 0;
};

// One vector a thread up to 512 columns, two up to 16384 (16384 x 1024: 46 us at one, 34
// at two; 32768 x 512: 50 and 52). Blocks share an SM's threads (1024 at one vector, 640
// at two: their registers) and 200 KB of its shared memory for their rings; a ring of
// fewer than two rows gives way to the long form. dres is counted whether or not it is given.
BackwardShape backward_shape(int64_t n, bool xb, bool yb)
{
    BackwardShape s;
    const int64_t nvec = ceil_div(n, 8);
    const size_t stage = static_cast<size_t>(nvec) * (xb ? 32 : 64) + static_cast<size_t>(nvec) * (yb ? 16 : 32);
    s.v = nvec <= 64 ? 1 : nvec <= 2048 ? 2 : 0;
    if (s.v == 0 || 2 * stage > kRingBytes) {
        s.v = 0;
        s.threads = 1024;
        s.per_sm = 2;
        return s;
    }
    s.threads = block_threads(n, s.v);
    s.per_sm = std::max(1, std::min(16, (s.v == 1 ? 1024 : 640) / s.threads));
    while (s.per_sm > 1 && 3 * stage > kRingBytes / s.per_sm) --s.per_sm;
    s.stages = static_cast<int>(std::min<size_t>(bm::NORM_MAX_STAGES, kRingBytes / s.per_sm / stage));
    s.smem = 8 * bm::NORM_MAX_STAGES + s.stages * stage;
    return s;
}

// Blocks of the backward kernel: each keeps its own column sums, so the workspace and
// the final sum grow with them.
int64_t backward_blocks(int64_t rows, const BackwardShape &s, int sms)
{
    return std::min<int64_t>(rows, static_cast<int64_t>(s.per_sm) * sms);
}

int64_t sums_ld(int64_t n) { return ceil_div(n, 8) * 8; }

template <bool XB, bool YB>
bm_status launch_forward(bm::NormParams p, int sms, cudaStream_t stream)
{
    const bool many = p.rows >= 4 * static_cast<int64_t>(sms);
    if (const int v = warp_vectors(p.n); many && v > 0) {
        const int64_t blocks = std::min<int64_t>(ceil_div(p.rows, 16 / v), 20 * static_cast<int64_t>(sms));  // four waves
        PdlLaunch l(stream, static_cast<unsigned>(blocks), 128);
        if (v == 1) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_warp_kernel<XB, YB, 1>, p));
        if (v == 2) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_warp_kernel<XB, YB, 2>, p));
        return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_warp_kernel<XB, YB, 4>, p));
    }
    // the ring form: two vectors a thread, blocks that share about 640 threads and 200 KB of an SM
    const int ring_threads = block_threads(p.n, 2);
    const size_t row_bytes = static_cast<size_t>(p.n / 8) * (XB ? 16 : 32);
    if (many && ring_threads <= bm::NORM_RING_THREADS && 3 * row_bytes <= kRingBytes) {
        const int per_sm = std::max(1, std::min(8, bm::NORM_RING_THREADS / ring_threads));
        p.stages = static_cast<int>(std::min<size_t>(bm::NORM_MAX_STAGES, kRingBytes / per_sm / row_bytes));
        PdlLaunch l(stream, static_cast<unsigned>(std::min<int64_t>(p.rows, per_sm * static_cast<int64_t>(sms))),
                    static_cast<unsigned>(ring_threads), 8 * bm::NORM_MAX_STAGES + p.stages * row_bytes);
        return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_ring_kernel<XB, YB, 2>, p));
    }
    const int v = block_vectors(p.n);
    const int threads = v == 0 ? 1024 : block_threads(p.n, v);
    PdlLaunch l(stream, static_cast<unsigned>(std::min<int64_t>(p.rows, std::max(1, 2048 / threads) * static_cast<int64_t>(sms))),
                static_cast<unsigned>(threads));
    if (v == 2) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 2>, p));
    if (v == 4) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_kernel<XB, YB, 4>, p));
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_long_kernel<XB, YB>, p));
}

std::mutex g_mutex;
bool g_attrs_set[kMaxDevices] = {};

// Once per device: the dynamic shared memory of the ring kernels.
bm_status norm_attrs(const DeviceState &st)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_attrs_set[st.device]) return BM_OK;
    const void *fns[] = {reinterpret_cast<const void *>(&bm::bm_layernorm_ring_kernel<false, false, 2>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_ring_kernel<false, true, 2>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_ring_kernel<true, false, 2>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_ring_kernel<true, true, 2>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<false, false, 1, 256>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<false, true, 1, 256>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<true, false, 1, 256>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<true, true, 1, 256>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<false, false, 2, 640>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<false, true, 2, 640>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<true, false, 2, 640>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<true, true, 2, 640>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<false, false, 2, 1024>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<false, true, 2, 1024>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<true, false, 2, 1024>),
                         reinterpret_cast<const void *>(&bm::bm_layernorm_backward_kernel<true, true, 2, 1024>)};
    for (const void *fn : fns)
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 201 * 1024) != cudaSuccess) {
            cudaGetLastError();
            return BM_ERR_CUDA;
        }
    g_attrs_set[st.device] = true;
    return BM_OK;
}

template <bool XB, bool YB>
bm_status launch_backward(bm::NormBwdParams p, const BackwardShape &s, int64_t blocks, cudaStream_t stream)
{
    p.stages = s.stages;
    PdlLaunch l(stream, static_cast<unsigned>(blocks), static_cast<unsigned>(s.threads), s.smem);
    if (s.v == 1) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_kernel<XB, YB, 1, 256>, p));
    if (s.v == 2 && s.threads <= 640)
        return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_kernel<XB, YB, 2, 640>, p));
    if (s.v == 2) return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_kernel<XB, YB, 2, 1024>, p));
    if (p.partial != nullptr) {
        PdlLaunch c(stream, static_cast<unsigned>(ceil_div(p.n, 8 * 256)), 256);
        c.cfg.gridDim.y = static_cast<unsigned>(blocks);
        const bm_status e = launched(cudaLaunchKernelEx(&c.cfg, bm::bm_layernorm_columns_kernel<XB, YB>, p));
        if (e != BM_OK) return e;
    }
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_layernorm_backward_long_kernel<XB, YB>, p));
}

template <bool HB>
bm_status launch_act(const bm::ActParams &p, int sms, cudaStream_t stream)
{
    const int64_t cols = ceil_div(p.n, 16);
    unsigned tx = 1;
    while (tx < 256 && tx < cols) tx *= 2;
    const unsigned ty = 256 / tx;
    const int64_t bx = ceil_div(cols, tx);
    const int64_t by = std::min<int64_t>(ceil_div(p.rows, ty), std::max<int64_t>(1, ceil_div(4 * static_cast<int64_t>(sms), bx)));
    PdlLaunch l(stream, static_cast<unsigned>(bx), tx);
    l.cfg.gridDim.y = static_cast<unsigned>(by);
    l.cfg.blockDim.y = ty;
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_act_mxfp8_kernel<HB>, p));
}

}  // namespace

namespace bmh {

bm_status launch_column_sums(const float *partial, int64_t rows, int64_t ld, int64_t plane, int64_t n, float *out0,
                             float *out1, int accumulate, cudaStream_t stream)
{
    // The split doubles while the CTAs stay at 320 or fewer, about two per SM, each with a
    // row at least for every warp. Layer norm backward with the sums at splits of 1, 2, 4 and
    // 8, us: 16384 x 1024 35.9, 31.7, 29.4, 28.1 (8 taken: 128 CTAs); 8192 x 5120 57.9, 57.5,
    // 57.2, 60.9 (4: 320); 8192 x 10240 117.1, 116.9, 119.7, 121.8 (2: 320); 1500 x 5120 17.7,
    // 17.5, 17.2, 19.8 (4). The tile products' bias gradient, 4096 x 16384 x 512: 129.6, 127.6,
    // 126.4, 129.6 (2: 256).
    const int64_t planes = out1 != nullptr ? 2 : 1, strips = ceil_div(n, 128);
    int split = 1;
    while (split < bm::SUM_SPLIT && split * strips * planes <= 160 && 2 * split * bm::SUM_WARPS <= rows) split *= 2;
    PdlLaunch l(stream, static_cast<unsigned>(strips * split), 32 * bm::SUM_WARPS, 0, split > 1 ? split : 0);
    l.cfg.gridDim.y = static_cast<unsigned>(planes);
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_column_sums_kernel, partial, rows, ld, plane, n, out0, out1,
                                       accumulate, split));
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
    if (const bm_status a = norm_attrs(*st); a != BM_OK) return a;
    const bm::NormParams p = {rows, n,  X,  ldx,  gamma, beta, param_type == BM_BF16, eps, Y,
                              ldy,  mean, rstd, 0, st->status, wait_timeout_ns()};
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
    int64_t blocks = 0;
    for (int types = 0; types < 4; ++types)
        blocks = std::max(blocks, backward_blocks(rows, backward_shape(n, types & 1, types & 2), sm_count_or_default()));
    return static_cast<size_t>(2 * blocks * sums_ld(n)) * sizeof(float);
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
    const BackwardShape shape = backward_shape(n, x_type == BM_BF16, y_type == BM_BF16);
    const int64_t blocks = backward_blocks(rows, shape, st->sm_count), ld = sums_ld(n), plane = blocks * ld;
    if (rows > 0) {
        s = norm_attrs(*st);
        if (s != BM_OK) return s;
        const bm::NormBwdParams p = {rows, n,      dY,   lddy, X,  ldx,   gamma, param_type == BM_BF16, mean,
                                     rstd, dres,   lddres, dX, lddx, partial, ld, plane, 0, st->status,
                                     wait_timeout_ns()};
        if (x_type == BM_BF16)
            s = y_type == BM_BF16 ? launch_backward<true, true>(p, shape, blocks, cs)
                                  : launch_backward<true, false>(p, shape, blocks, cs);
        else
            s = y_type == BM_BF16 ? launch_backward<false, true>(p, shape, blocks, cs)
                                  : launch_backward<false, false>(p, shape, blocks, cs);
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
