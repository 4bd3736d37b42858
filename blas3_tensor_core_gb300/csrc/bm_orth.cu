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
// bits: X is two fp16 halves, high + low, of which the products take the high one. The
// diagonals of A and B, near 1 and -2.7 in the end while the rest is small, stay FP32 in
// vectors of their own: (B X)_i = diag(B)_i X_i + (B off its diagonal) X. X is held times
// 256, away from fp16's subnormal values. Relative error of X after five steps (of norms,
// before the rounding to bf16, against 64 bits; square and wide matrices of 64 to 1024 rows
// with Gaussian entries, sizes falling as 1 / i and 1 / i^2, and few directions over noise):
// 1e-4 to 9e-4. With bf16 intermediates it is 1e-2 to 1.7e-1, with fp16 ones and no low
// half 6e-4 to 2e-2, with the diagonals in fp16 2e-4 to 1.8e-3.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "bm.h"
#include "bm_epi.h"
#include "bm_host.h"
#include "bm_ops.h"

using namespace bmh;

namespace bm {

constexpr float kOrthScale = 256.0f;  // X is held times this
constexpr int NORM_THREADS = 256;

struct ScaleParams {
    const void *X;  // [m, n] fp32 or bf16
    int64_t ldx, m, n;
    int x_bf16;
    double *partial;  // sums of squares, one per block
    int blocks;
    double eps;
    __half *hi, *lo;  // [m, ld]
    int64_t ld;
};

// Eight columns of a row from column j on (zeros past n).
__device__ __forceinline__ void load_x8(const ScaleParams &s, int64_t i, int64_t j, float (&v)[8])
{
    if (s.x_bf16) {
        uint32_t w[4];
        load_row<8>(s.X, s.ldx, i, s.m, j, s.n, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = bf16_pair(w[e]);
            v[2 * e] = t.x, v[2 * e + 1] = t.y;
        }
    } else {
        const float *src = static_cast<const float *>(s.X) + i * s.ldx + j;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (j + 4 * h + 4 <= s.n) {
                const float4 t = *reinterpret_cast<const float4 *>(src + 4 * h);
                v[4 * h] = t.x, v[4 * h + 1] = t.y, v[4 * h + 2] = t.z, v[4 * h + 3] = t.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] = j + 4 * h + e < s.n ? src[4 * h + e] : 0.0f;
            }
        }
    }
}

// Sum over the block's threads in a fixed order (thread 0 gets it).
__device__ __forceinline__ double block_sum(double v, double (&part)[NORM_THREADS / 32])
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < NORM_THREADS / 32; ++w) t += part[w];
    return t;
}

// Items (256 columns of a row) it, it + warps, ...: row and first column of the next one
// without a division.
struct ItemWalk {
    int64_t i, j, di, dj, width;
    __device__ ItemWalk(int64_t n, int64_t first, int64_t warps)
    {
        const int64_t segments = (n + 255) / 256;
        width = segments * 256;
        i = first / segments;
        j = (first - i * segments) * 256;
        di = warps / segments;
        dj = (warps - di * segments) * 256;
    }
    __device__ __forceinline__ void next()
    {
        i += di;
        j += dj;
        if (j >= width) j -= width, ++i;
    }
};

// Sums of squares, one per block. A warp takes 256 columns of a row at a time and has four
// such loads in flight (one at a time took 78 us for 4096 x 4096 in BF16, 34 MB). Squares are
// added in FP32 over at most 64 of those pieces and in FP64 beyond. Eight values whose squares
// FP32 could not hold are squared in FP64; there are hardly ever any.
__global__ void __launch_bounds__(NORM_THREADS) bm_square_sum_kernel(const ScaleParams s)
{
    __shared__ double part[NORM_THREADS / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (NORM_THREADS / 32);
    ItemWalk at(s.n, blockIdx.x * static_cast<int64_t>(NORM_THREADS / 32) + (threadIdx.x >> 5), warps);
    double total = 0.0;
    float sum = 0.0f;
    for (int held = 0; at.i < s.m; ++held) {
        float v[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (at.i < s.m && at.j + lane * 8 < s.n) {
                load_x8(s, at.i, at.j + lane * 8, v[q]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] = 0.0f;
            }
            at.next();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float most = 0.0f, here = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                most = fmaxf(most, fabsf(v[q][e]));
                here = fmaf(v[q][e], v[q][e], here);
            }
            if (most > 1.0e15f || (most < 1.0e-15f && most > 0.0f)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) total += static_cast<double>(v[q][e]) * v[q][e];
            } else {
                sum += here;
            }
        }
        if ((held & 15) == 15) {
            total += sum;
            sum = 0.0f;
        }
    }
    const double t = block_sum(total + sum, part);
    if (threadIdx.x == 0) s.partial[blockIdx.x] = t;
}

// X0 = 256 X / (|X| + eps) in two halves. Each block adds the blocks' sums, in the same
// order. A norm that is not finite, or 0 with eps = 0, makes every element NaN.
__global__ void __launch_bounds__(NORM_THREADS) bm_orth_scale_kernel(const ScaleParams s)
{
    __shared__ double part[NORM_THREADS / 32];
    __shared__ double scale_at;
    griddep_launch_dependents();
    griddep_wait();
    double sum = 0.0;
    for (int b = threadIdx.x; b < s.blocks; b += NORM_THREADS) sum += s.partial[b];
    sum = block_sum(sum, part);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum) + s.eps;
        scale_at = norm > 0.0 && norm < 1.0e300 ? kOrthScale / norm : nan("");
    }
    __syncthreads();
    const double scale = scale_at;
    const float scale32 = static_cast<float>(scale);
    const bool in32 = !(scale > 1.0e37 || scale < 1.0e-37);  // (the NaN too)
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (NORM_THREADS / 32);
    ItemWalk at(s.n, blockIdx.x * static_cast<int64_t>(NORM_THREADS / 32) + (threadIdx.x >> 5), warps);
    while (at.i < s.m) {
        float v[2][8];
        int64_t row[2], col[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            row[q] = at.i;
            col[q] = at.j + lane * 8;
            if (row[q] < s.m && col[q] < s.n) load_x8(s, row[q], col[q], v[q]);
            at.next();
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (row[q] >= s.m || col[q] >= s.n) continue;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float a = v[q][e], b = v[q][e + 1];
                const float2 x = in32 ? make_float2(a * scale32, b * scale32)
                                      : make_float2(static_cast<float>(a * scale), static_cast<float>(b * scale));
                hi[e / 2] = pack_f16(x);
                const float2 h = f16_pair(hi[e / 2]);
                lo[e / 2] = pack_f16(make_float2(x.x - h.x, x.y - h.y));
            }
            // (rows are padded to whole vectors)
            const int64_t to = row[q] * s.ld + col[q];
            *reinterpret_cast<uint4 *>(s.hi + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(s.lo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

}  // namespace bm

namespace {

std::mutex g_mutex;
bool g_attrs_set[kMaxDevices] = {};

bm_status orth_attrs(const DeviceState &st)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_attrs_set[st.device]) return BM_OK;
    if (!epi_attrs<bm::KIND_GRAM>() || !epi_attrs<bm::KIND_POLY>() || !epi_attrs<bm::KIND_STEP>()) return BM_ERR_CUDA;
    g_attrs_set[st.device] = true;
    return BM_OK;
}

constexpr int kMaxBlocks = 4096;  // of the square sums
constexpr int kMaxSteps = 64;
constexpr float kDefaultStep[3] = {3.4445f, -4.7750f, 2.0315f};

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int64_t padded(int64_t cols) { return ceil_div(cols, 16) * 16; }  // rows of 32 bytes

// Workspace: X in two buffers of two halves, A and B off their diagonals, the diagonals,
// the square sums.
struct Layout {
    int64_t ldx, lds;
    size_t x, sq, diag, hi[2], lo[2], a, b, da, db, sums, total;
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
        sums = take(kMaxBlocks * sizeof(double));
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

int step_variant(int64_t m, int64_t n, int64_t k, int sms, int pair_clusters)
{
    const Plan whole = plan_gemm(m, n, k, 0, sms, pair_clusters);
    if (tile_override() == 0 && ceil_div(m, 128) * ceil_div(n, 128) <= sms) return kSingle128;
    return whole.variant;
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
        fill_params(f.g, pl);
        f.g.mode = bm::MODE_SYRK_LOWER;
        f.g.a_mn_major = f.g.b_mn_major = mn;
        EpiMaps t;
        // (both operands are X, in boxes of 128 rows)
        if (!epi_operand(&t.a, &f.g.a_box3, X, mn, s, k, ld, bm::CTA_M, kVariantStageKBlocks[v])) return BM_ERR_CUDA;
        t.b = t.a;
        f.g.b_box3 = f.g.a_box3;
        epi_output(f, t, 0, at(out), l.lds, s, l.lds);
        if (!f.tma[0]) return BM_ERR_CUDA;
        f.diag_out = reinterpret_cast<float *>(at(diag));
        return epi_launch<KIND>(pl, t, f, stream);
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
        const int v = step_variant(m, n, s, st->sm_count, st->max_pair_clusters);
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
            epi_output(f, t, 0, C, ldc, m, n);
        } else {
            epi_output(f, t, 0, at(l.hi[1 - cur]), l.ldx, m, l.ldx);
            epi_output(f, t, 1, at(l.lo[1 - cur]), l.ldx, m, l.ldx);
        }
        return epi_launch<bm::KIND_STEP>(pl, t, f, stream);
    }

    bm_status scale(const void *X, int64_t ldx, bm_dtype t, float eps) const
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
        const int64_t items = m * ceil_div(n, 256);
        p.blocks = static_cast<int>(std::min<int64_t>(
            ceil_div(items, bm::NORM_THREADS / 32), std::min<int64_t>(kMaxBlocks, 8 * static_cast<int64_t>(st->sm_count))));
        PdlLaunch a(stream, static_cast<unsigned>(p.blocks), bm::NORM_THREADS);
        const bm_status r = launched(cudaLaunchKernelEx(&a.cfg, bm::bm_square_sum_kernel, p));
        if (r != BM_OK) return r;
        PdlLaunch b(stream, static_cast<unsigned>(p.blocks), bm::NORM_THREADS);
        return launched(cudaLaunchKernelEx(&b.cfg, bm::bm_orth_scale_kernel, p));
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
    s = o.scale(X, ldx, x_type, eps);
    for (int t = 0; t < steps && s == BM_OK; ++t) {
        const float *c = coeffs != nullptr ? coeffs + 3 * t : kDefaultStep;
        const bool last = t == steps - 1;
        s = o.gram(t & 1);
        if (s == BM_OK) s = o.poly(c);
        if (s == BM_OK) s = o.step(t & 1, last ? C : nullptr, ldc, alpha, beta);
    }
    return s;
}

size_t bm_orthogonalize_bf16_workspace_size(int64_t m, int64_t n)
{
    if (m <= 0 || n <= 0) return 0;
    return Layout(m, n).total;
}

}  // extern "C"
