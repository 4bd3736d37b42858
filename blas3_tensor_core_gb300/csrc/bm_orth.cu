// bm_orth.cu -- an update made orthogonal by Newton-Schulz products
// (bm_orthogonalize_bf16): the scaling kernels, argument checks, plans, launches.
//
//   X0 = X / (|X|_F + eps);  A = X X^T,  B = b A + c A^2,  X' = a X + B X;  C = alpha X + beta C
//
// (X tall: A = X^T X and X' = a X + X B, so that A has the shorter side.)
//
// Numbers. The products take fp16 operands (11 bits, the tensor cores' full rate) and FP32
// accumulators. Each step multiplies a direction of small size by up to a = 3.4, so what is
// lost in X before the last step comes back a few hundred times larger in the directions
// that an averaged gradient has least of. What enters X' by the factor a therefore keeps 22
// bits: X is two fp16 halves, high + low, of which the products take the high one. (Elements of
// X below 2^-11, the usual ones from 2048 x 2048 on, keep fewer: the low half's last step is
// 2^-24 / 256. 21.8 bits of a typical element of 4096 x 4096, 20.8 of 16384 x 4096.) The
// diagonals of A and B, near 1 and -2.7 in the end while the rest is small, stay FP32 in
// vectors of their own: (B X)_i = diag(B)_i X_i + (B off its diagonal) X. X is held times
// 256, its high half away from fp16's subnormal values. Relative error of X after five steps (of norms,
// before the rounding to bf16, against 64 bits; square and wide matrices of 64 to 1024 rows
// with Gaussian entries, sizes falling as 1 / i and 1 / i^2, and few directions over noise):
// 1e-4 to 9e-4. With bf16 intermediates it is 1e-2 to 1.7e-1, with fp16 ones and no low
// half 6e-4 to 2e-2, with the diagonals in fp16 2e-4 to 1.8e-3.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "bm.h"
#include "bm_epi.h"
#include "bm_host.h"
#include "bm_ops.h"
#include "bm_orth_kernel.cuh"
#include "bm_symm_kernel.cuh"

using namespace bmh;

namespace {

std::mutex g_mutex;
bool g_attrs_set[kMaxDevices] = {};
int g_small_cluster[kMaxDevices];      // CTAs of the largest cluster of the one-kernel update (a power of two)
int g_split_clusters[kMaxDevices][2];  // clusters of two and of four of the split symmetric products at once
int g_small_grid[kMaxDevices];         // CTAs of the one-kernel update that a cooperative launch can have
std::atomic<int> g_cluster_limit{0}, g_grid_limit{0};  // bm_debug_limit_clusters, bm_debug_limit_grid

using SplitKernel = void (*)(CUtensorMap, CUtensorMap, bm::EpiParams);

template <int KIND>
SplitKernel split_kernel(int s)
{
    if (s == 4) return &bm::bm_symm_split_kernel<4, KIND>;
    return &bm::bm_symm_split_kernel<2, KIND>;
}

bm_status orth_attrs(const DeviceState &st)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_attrs_set[st.device]) return BM_OK;
    if (!epi_attrs<bm::KIND_GRAM>() || !epi_attrs<bm::KIND_POLY>() || !epi_attrs<bm::KIND_STEP>()) return BM_ERR_CUDA;
    if (cudaFuncSetAttribute(bm::bm_orth_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bm::SmallSmem::BYTES) !=
            cudaSuccess ||
        cudaFuncSetAttribute(bm::bm_orth_small_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();
        return BM_ERR_CUDA;
    }
    g_small_cluster[st.device] = 1;
    for (int c = 2; c <= bm::SMALL_MAX_CLUSTER; c *= 2) {
        PdlLaunch l(nullptr, static_cast<unsigned>(c), bm::SMALL_THREADS, bm::SmallSmem::BYTES, c);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, bm::bm_orth_small_kernel, &l.cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            break;
        }
        g_small_cluster[st.device] = c;
    }
    int cooperative = 0, per_sm = 0;
    if (cudaDeviceGetAttribute(&cooperative, cudaDevAttrCooperativeLaunch, st.device) != cudaSuccess || cooperative == 0 ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, bm::bm_orth_small_kernel, bm::SMALL_THREADS,
                                                      bm::SmallSmem::BYTES) != cudaSuccess) {
        cudaGetLastError();
        per_sm = 0;
    }
    g_small_grid[st.device] = per_sm * st.sm_count;
    for (int s : {2, 4}) {
        for (SplitKernel fn : {split_kernel<bm::KIND_GRAM>(s), split_kernel<bm::KIND_POLY>(s)})
            if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     bm::SymmCfg::BYTES) != cudaSuccess) {
                cudaGetLastError();
                return BM_ERR_CUDA;
            }
        PdlLaunch l(nullptr, static_cast<unsigned>(s * st.sm_count), bm::SYMM_THREADS, bm::SymmCfg::BYTES, s);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void *>(split_kernel<bm::KIND_POLY>(s)), &l.cfg) !=
            cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        g_split_clusters[st.device][s / 4] = n;
    }
    g_attrs_set[st.device] = true;
    return BM_OK;
}

constexpr int kMaxBlocks = 4096;  // of the square sums
// Blocks per SM at most: what its registers hold at once (4096 x 4096 BF16, both kernels: 33 us
// with 4, 39 with 8, 42 with 2).
constexpr int kNormBlocks = 4;
using bm::kMaxSteps;
constexpr float kDefaultStep[3] = {3.4445f, -4.7750f, 2.0315f};

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int64_t padded(int64_t cols) { return ceil_div(cols, 16) * 16; }  // rows of 32 bytes

// Whether a workspace's bytes, 8 to an element of X and at most as many to one of A, can be counted.
bool countable(int64_t m, int64_t n) { return m <= (int64_t{1} << 58) / padded(n); }

// The form in which one kernel does all steps: a shorter side of at most 128 and a CTA per 128
// lines of the longer one, all of them on the GPU at once. -1: none.
int small_mode(int64_t m, int64_t n, int device)
{
    if (std::min(m, n) > bm::SMALL || tile_override() != 0) return -1;
    const int64_t ctas = ceil_div(std::max(m, n), bm::SMALL);
    if (ctas == 1) return bm::SMALL_ONE;
    int64_t cluster = 1;  // the rows of A are shared out evenly
    while (cluster < ctas) cluster *= 2;
    const int limit = g_cluster_limit.load();
    if (cluster <= g_small_cluster[device] && (limit == 0 || cluster <= limit)) return bm::SMALL_CLUSTER;
    return ctas <= g_small_grid[device] ? bm::SMALL_GRID : -1;
}

// Workspace: X in two buffers of two halves, A and B off their diagonals, the diagonals, the
// square sums; or, shorter side at most 128, the CTAs' sums of A and its total, the square
// sums and a counter. Room for either, so that it does not depend on the device.
struct Layout {
    int64_t ldx, lds;
    size_t x, sq, diag, hi[2], lo[2], a, b, da, db, sums, count, total;
    Layout(int64_t m, int64_t n)
    {
        const int64_t s = std::min(m, n);
        ldx = padded(n);
        lds = padded(s);
        x = round256(static_cast<size_t>(m) * ldx * 2);
        sq = round256(static_cast<size_t>(s) * lds * 2);
        diag = round256(static_cast<size_t>(s) * 4);
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t here = at;
            at += bytes;
            return here;
        };
        for (int i = 0; i < 2; ++i) hi[i] = take(x), lo[i] = take(x);
        a = take(sq), b = take(sq), da = take(diag), db = take(diag);
        if (s <= bm::SMALL) at = std::max(at, static_cast<size_t>(ceil_div(std::max(m, n), bm::SMALL) + 1) * 65536);
        sums = take(kMaxBlocks * sizeof(double));
        count = take(256);
        total = at;
    }
};

// Tiles of a symmetric product: SM pairs when they fill half the GPU, as plan_syrk has it.
int symmetric_variant(int64_t s, int pair_clusters)
{
    const int64_t t = ceil_div(s, 256);
    const int forced = tile_override() - 1;
    if (forced >= 0) return forced == kPair256 && pair_clusters > 0 ? kPair256 : kSingle128;
    return pair_clusters > 0 && t * (t + 1) >= pair_clusters ? kPair256 : kSingle128;
}

struct Orth {
    DeviceState *st;
    cudaStream_t stream;
    int64_t m, n, s, len;  // s: the shorter side, len: the longer
    bool wide;
    char *ws;
    Layout l;

    char *at(size_t offset) const { return ws + offset; }

    bm::EpiParams params(int64_t rows, int64_t cols, int64_t k, float alpha) const
    {
        bm::EpiParams f;
        std::memset(&f, 0, sizeof(f));
        f.g = base_params(rows, cols, k, alpha, 0.0f, nullptr, 1, BM_BF16, st);
        return f;
    }

    // A symmetric product over [s, k] (mn: stored [k, s]) into `out` and a diagonal.
    template <int KIND>
    bm_status symmetric(bm::EpiParams &f, const void *X, int64_t ld, bool mn, int64_t k, size_t out, size_t diag) const
    {
        const int v = symmetric_variant(s, st->max_pair_clusters);
        const Plan pl = epi_plan(v, s, s, k, true, st->sm_count, st->max_pair_clusters);
        const int split = split_ways(v, pl);
        fill_params(f.g, pl);
        f.g.mode = bm::MODE_SYRK_LOWER;
        f.g.a_mn_major = f.g.b_mn_major = mn;
        EpiMaps t;
        epi_output(f, 0, at(out), l.lds);
        epi_output_maps(f, t, s, l.lds);
        if (!f.tma[0]) return BM_ERR_CUDA;
        f.diag_out = reinterpret_cast<float *>(at(diag));
        if (split > 1) {
            if (!encode_operand(&t.a, X, mn, s, k, ld, bm::CTA_M)) return BM_ERR_CUDA;
            PdlLaunch launch(stream, static_cast<unsigned>(pl.num_tiles * split), bm::SYMM_THREADS, bm::SymmCfg::BYTES, split);
            return launched(cudaLaunchKernelEx(&launch.cfg, split_kernel<KIND>(split), t.a, t.out[0], f));
        }
        // (both operands are X, in boxes of 128 rows)
        if (!epi_operand(&t.a, &f.g.a_box3, X, mn, s, k, ld, bm::CTA_M, kVariantStageKBlocks[v])) return BM_ERR_CUDA;
        t.b = t.a;
        f.g.b_box3 = f.g.a_box3;
        if (KIND == bm::KIND_POLY && !encode_box64(&t.in[0], f.in[0], BM_BF16, s, l.lds, f.ldin[0])) return BM_ERR_CUDA;
        return epi_launch<KIND>(pl, t, f, stream);
    }

    // CTAs that share a tile's K: four or two while their clusters fit on the GPU at once and
    // each has two k-blocks or more.
    int split_ways(int v, const Plan &pl) const
    {
        if (v != kSingle128 || tile_override() != 0) return 1;
        for (int w : {4, 2})
            if (pl.num_tiles <= g_split_clusters[st->device][w / 4] && pl.kb_total >= 2 * w) return w;
        return 1;
    }

    bm_status gram(int cur) const
    {
        bm::EpiParams f = params(s, s, len, 1.0f / (bm::kOrthScale * bm::kOrthScale));
        return symmetric<bm::KIND_GRAM>(f, at(l.hi[cur]), l.ldx, !wide, len, l.a, l.da);
    }

    bm_status poly(const float *c) const
    {
        bm::EpiParams f = params(s, s, s, 1.0f);
        f.in[0] = at(l.a);
        f.ldin[0] = f.in_cols = l.lds;
        f.diag = reinterpret_cast<const float *>(at(l.da));
        f.ca = c[0], f.cb = c[1], f.cc = c[2];
        return symmetric<bm::KIND_POLY>(f, at(l.a), l.lds, false, s, l.b, l.db);
    }

    // X' from buffer `cur` into the other one, or (C given) the result.
    bm_status step(int cur, void *C, int64_t ldc, float alpha, float beta) const
    {
        const int v = epi_variant(m, n, s, st->sm_count, st->max_pair_clusters);
        const Plan pl = epi_plan(v, m, n, s, false, st->sm_count, st->max_pair_clusters);
        bm::EpiParams f = params(m, n, s, alpha / bm::kOrthScale);
        fill_params(f.g, pl);
        f.in[0] = at(l.hi[cur]);
        f.in[1] = at(l.lo[cur]);
        f.ldin[0] = f.ldin[1] = l.ldx;
        f.diag = reinterpret_cast<const float *>(at(l.db));
        f.diag_cols = !wide;
        const int kps = kVariantStageKBlocks[v], rows_b = pl.bn / pl.pair;
        EpiMaps t;
        bool ok;
        if (wide) {  // B [s, s] times X [s, n]
            f.g.b_mn_major = 1;
            ok = epi_operand(&t.a, &f.g.a_box3, at(l.b), false, s, s, l.lds, bm::CTA_M, kps) &&
                 epi_operand(&t.b, &f.g.b_box3, at(l.hi[cur]), true, n, s, l.ldx, rows_b, kps);
        } else {  // X [m, s] times B [s, s], which is its own transpose
            ok = epi_operand(&t.a, &f.g.a_box3, at(l.hi[cur]), false, m, s, l.ldx, bm::CTA_M, kps) &&
                 epi_operand(&t.b, &f.g.b_box3, at(l.b), false, s, s, l.lds, rows_b, kps);
        }
        if (!ok || !encode_box64(&t.in[0], f.in[0], BM_BF16, m, n, l.ldx) || !encode_box64(&t.in[1], f.in[1], BM_BF16, m, n, l.ldx))
            return BM_ERR_CUDA;
        if (C != nullptr) {
            f.last = 1;
            f.beta = beta;
            epi_output(f, 0, C, ldc);
        } else {
            epi_output(f, 0, at(l.hi[1 - cur]), l.ldx);
            epi_output(f, 1, at(l.lo[1 - cur]), l.ldx);
        }
        // (C's columns end with n, those of X's buffers with their padded rows)
        epi_output_maps(f, t, m, C != nullptr ? n : l.ldx);
        return epi_launch<bm::KIND_STEP>(pl, t, f, stream);
    }

    bm::ScaleParams scale_params(const void *X, int64_t ldx, bm_dtype t, float eps) const
    {
        bm::ScaleParams p;
        std::memset(&p, 0, sizeof(p));
        p.X = X;
        p.ldx = ldx;
        p.m = m;
        p.n = n;
        p.x_bf16 = t == BM_BF16;
        p.partial = reinterpret_cast<double *>(at(l.sums));
        p.eps = eps;
        p.hi = reinterpret_cast<__half *>(at(l.hi[0]));
        p.lo = reinterpret_cast<__half *>(at(l.lo[0]));
        p.ld = l.ldx;
        const int64_t items = m * ceil_div(n, 512);
        p.blocks = static_cast<int>(std::min<int64_t>(
            ceil_div(items, bm::NORM_THREADS / 32), std::min<int64_t>(kMaxBlocks, kNormBlocks * static_cast<int64_t>(st->sm_count))));
        return p;
    }

    bm_status square_sums(const bm::ScaleParams &p) const
    {
        PdlLaunch a(stream, static_cast<unsigned>(p.blocks), bm::NORM_THREADS);
        return launched(cudaLaunchKernelEx(&a.cfg, bm::bm_square_sum_kernel, p));
    }

    bm_status scale(const bm::ScaleParams &p) const
    {
        const bm_status r = square_sums(p);
        if (r != BM_OK) return r;
        PdlLaunch b(stream, static_cast<unsigned>(p.blocks), bm::NORM_THREADS);
        return launched(cudaLaunchKernelEx(&b.cfg, bm::bm_orth_scale_kernel, p));
    }

    // All steps in one kernel. *refused: CUDA would not have the CTAs of a grid on the GPU at once
    // (a context with part of the SMs), nothing has been written but the workspace.
    bm_status small(int mode, const bm::ScaleParams &x, int steps, const float *coeffs, void *C, int64_t ldc, float alpha,
                    float beta, bool *refused) const
    {
        *refused = false;
        bm::SmallParams p;
        std::memset(&p, 0, sizeof(p));
        p.x = x;
        p.len = len;
        p.s = static_cast<int>(s);
        p.wide = wide;
        p.mode = mode;
        int ctas = static_cast<int>(ceil_div(len, bm::SMALL));
        if (mode == bm::SMALL_CLUSTER)
            while ((ctas & (ctas - 1)) != 0) ++ctas;
        p.ctas = ctas;
        p.steps = steps;
        for (int t = 0; t < steps; ++t)
            std::memcpy(p.coeffs + 3 * t, coeffs != nullptr ? coeffs + 3 * t : kDefaultStep, 3 * sizeof(float));
        p.C = C;
        p.ldc = ldc;
        p.alpha = alpha;
        p.beta = beta;
        p.sums = reinterpret_cast<float4 *>(ws);
        p.count = reinterpret_cast<unsigned int *>(at(l.count));
        p.status = st->status;
        p.timeout_ns = wait_timeout_ns();
        const bm::GemmParams g = base_params(1, 1, 1, 1.0f, 0.0f, nullptr, 1, BM_BF16, st);
        p.debug_stall = g.debug_stall;
        if (p.mode != bm::SMALL_GRID) {
            PdlLaunch one(stream, static_cast<unsigned>(ctas), bm::SMALL_THREADS, bm::SmallSmem::BYTES,
                          p.mode == bm::SMALL_CLUSTER ? ctas : 0);
            return launched(cudaLaunchKernelEx(&one.cfg, bm::bm_orth_small_kernel, p));
        }
        p.x.count = p.count;
        const bm_status r = square_sums(p.x);
        if (r != BM_OK) return r;
        // every CTA waits for the others: all of them on the GPU at once
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
        cfg.blockDim = dim3(bm::SMALL_THREADS, 1, 1);
        cfg.dynamicSmemBytes = bm::SmallSmem::BYTES;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const int limit = g_grid_limit.load();
        const cudaError_t e = limit != 0 && ctas > limit ? cudaErrorCooperativeLaunchTooLarge
                                                         : cudaLaunchKernelEx(&cfg, bm::bm_orth_small_kernel, p);
        *refused = e == cudaErrorCooperativeLaunchTooLarge;
        return launched(e);
    }
};

}  // namespace

extern "C" {

bm_status bm_orthogonalize_bf16(int64_t m, int64_t n, float alpha, const void *X, int64_t ldx, bm_dtype x_type, int steps,
                                const float *coeffs, float eps, float beta, void *C, int64_t ldc, void *workspace,
                                size_t workspace_bytes, bm_stream_t stream)
{
    if (m < 0 || n < 0 || !fits_int32(m) || !fits_int32(n)) return BM_ERR_INVALID_VALUE;
    if (x_type != BM_F32 && x_type != BM_BF16) return BM_ERR_INVALID_VALUE;
    if (ldx < std::max<int64_t>(1, n) || ldc < std::max<int64_t>(1, n)) return BM_ERR_INVALID_VALUE;
    if (steps < 1 || steps > kMaxSteps || !(eps >= 0.0f) || !std::isfinite(eps)) return BM_ERR_INVALID_VALUE;
    if (m == 0 || n == 0) return BM_OK;
    if (!countable(m, n)) return BM_ERR_INVALID_VALUE;
    if (X == nullptr || C == nullptr) return BM_ERR_INVALID_VALUE;
    const int64_t esz = x_type == BM_BF16 ? 2 : 4;
    if (!aligned16(X) || !aligned16(C) || (ldx * esz) % 16 != 0 || (ldc * 2) % 16 != 0) return BM_ERR_MISALIGNED;
    const Layout l(m, n);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < l.total)
        return BM_ERR_WORKSPACE;
    if (alpha == 0.0f)  // C = beta C
        return bm_gemm_bf16(m, n, 0, BM_OP_N, BM_OP_N, 0.0f, nullptr, 1, nullptr, n, beta, C, ldc, BM_BF16, nullptr, 0, stream);
    DeviceState *st = nullptr;
    bm_status s = device_state(&st);
    if (s != BM_OK) return s;
    s = orth_attrs(*st);
    if (s != BM_OK) return s;
    const Orth o = {st, reinterpret_cast<cudaStream_t>(stream), m, n, std::min(m, n), std::max(m, n), m <= n,
                    static_cast<char *>(workspace), l};
    const bm::ScaleParams x = o.scale_params(X, ldx, x_type, eps);
    const int mode = small_mode(m, n, st->device);
    if (mode >= 0) {
        bool refused;
        s = o.small(mode, x, steps, coeffs, C, ldc, alpha, beta, &refused);
        if (!refused) return s;
    }
    s = o.scale(x);
    for (int t = 0; t < steps && s == BM_OK; ++t) {
        const float *c = coeffs != nullptr ? coeffs + 3 * t : kDefaultStep;
        const bool last = t == steps - 1;
        s = o.gram(t & 1);
        if (s == BM_OK) s = o.poly(c);
        if (s == BM_OK) s = o.step(t & 1, last ? C : nullptr, ldc, alpha, beta);
    }
    return s;
}

void bm_debug_limit_clusters(int ctas) { g_cluster_limit.store(ctas > 0 ? ctas : 0); }
void bm_debug_limit_grid(int ctas) { g_grid_limit.store(ctas > 0 ? ctas : 0); }

size_t bm_orthogonalize_bf16_workspace_size(int64_t m, int64_t n)
{
    if (m <= 0 || n <= 0 || !fits_int32(m) || !fits_int32(n) || !countable(m, n)) return 0;
    return Layout(m, n).total;
}

}  // extern "C"
