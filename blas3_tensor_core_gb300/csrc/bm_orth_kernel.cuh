// bm_orth_kernel.cuh -- kernels of the orthogonalised update (bm_orth.cu) beside its tiled
// products: the norm and the scaling of X, and the whole update of a matrix whose shorter
// side is at most 128.
#pragma once

#include <cuda_fp16.h>

#include "bm_epi_kernel.cuh"

namespace bm {

constexpr float kOrthScale = 256.0f;  // X is held times this
constexpr int NORM_THREADS = 256;

struct ScaleParams {
    const void *X;  // [m, n] fp32 or bf16
    int64_t ldx, m, n;
    int x_bf16;
    double *partial;  // sums of squares, one per block
    int blocks;
    unsigned int *count;  // set to 0 for a kernel that follows (may be null)
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

// Sum of the squares of eight values, in FP64 where FP32 could not hold one of them (there are
// hardly ever any).
__device__ __forceinline__ double square8(const float (&v)[8])
{
    float most = 0.0f, here = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        most = fmaxf(most, fabsf(v[e]));
        here = fmaf(v[e], v[e], here);
    }
    if (!(most > 1.0e15f || (most < 1.0e-15f && most > 0.0f))) return here;
    double wide = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) wide += static_cast<double>(v[e]) * v[e];
    return wide;
}

// 256 / (|X| + eps) from the sum of squares: NaN when the norm is not finite, or 0 with
// eps = 0. FP32 multiplies by it unless it is near FP32's ends.
__device__ __forceinline__ double orth_scale(double squares, double eps)
{
    const double norm = sqrt(squares) + eps;
    return norm > 0.0 && norm < 1.0e300 ? kOrthScale / norm : nan("");
}

__device__ __forceinline__ bool scale_in32(double scale) { return !(scale > 1.0e37 || scale < 1.0e-37); }

// Eight values of X0 in two halves.
__device__ __forceinline__ void split8(const float (&v)[8], double scale, float scale32, bool in32, uint32_t (&hi)[4],
                                       uint32_t (&lo)[4])
{
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float a = v[e], b = v[e + 1];
        const float2 x = in32 ? make_float2(a * scale32, b * scale32)
                              : make_float2(static_cast<float>(a * scale), static_cast<float>(b * scale));
        hi[e / 2] = pack_f16(x);
        const float2 h = f16_pair(hi[e / 2]);
        lo[e / 2] = pack_f16(make_float2(x.x - h.x, x.y - h.y));
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

// Items (512 columns of a row, two vectors of eight a lane) it, it + warps, ...: row and first
// column of the next one without a division.
struct ItemWalk {
    int64_t i, j, di, dj, width;
    __device__ ItemWalk(int64_t n, int64_t first, int64_t warps)
    {
        const int64_t segments = (n + 511) / 512;
        width = segments * 512;
        i = first / segments;
        j = (first - i * segments) * 512;
        di = warps / segments;
        dj = (warps - di * segments) * 512;
    }
    __device__ __forceinline__ void next()
    {
        i += di;
        j += dj;
        if (j >= width) j -= width, ++i;
    }
};

// Sums of squares, one per block. A warp has two items (four loads a lane) in flight. Squares
// are added in FP32 over 32 items and in FP64 beyond.
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
            const int64_t j = at.j + 256 * (q & 1) + lane * 8;
            if (at.i < s.m && j < s.n) {
                load_x8(s, at.i, j, v[q]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q][e] = 0.0f;
            }
            if (q & 1) at.next();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float most = 0.0f, here = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                most = fmaxf(most, fabsf(v[q][e]));
                here = fmaf(v[q][e], v[q][e], here);
            }
            if (most > 1.0e15f || (most < 1.0e-15f && most > 0.0f)) total += square8(v[q]);
            else sum += here;
        }
        if ((held & 15) == 15) {
            total += sum;
            sum = 0.0f;
        }
    }
    const double t = block_sum(total + sum, part);
    if (threadIdx.x == 0) {
        s.partial[blockIdx.x] = t;
        if (blockIdx.x == 0 && s.count != nullptr) *s.count = 0u;
    }
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
    if (threadIdx.x == 0) scale_at = orth_scale(sum, s.eps);
    __syncthreads();
    const double scale = scale_at;
    const float scale32 = static_cast<float>(scale);
    const bool in32 = scale_in32(scale);
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (NORM_THREADS / 32);
    ItemWalk at(s.n, blockIdx.x * static_cast<int64_t>(NORM_THREADS / 32) + (threadIdx.x >> 5), warps);
    for (; at.i < s.m; at.next()) {
        float v[2][8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t j = at.j + 256 * q + lane * 8;
            if (j < s.n) load_x8(s, at.i, j, v[q]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t j = at.j + 256 * q + lane * 8;
            if (j >= s.n) continue;
            uint32_t hi[4], lo[4];
            split8(v[q], scale, scale32, in32, hi, lo);
            // (rows are padded to whole vectors)
            const int64_t to = at.i * s.ld + j;
            *reinterpret_cast<uint4 *>(s.hi + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(s.lo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// ---------------------------------------------------------------- shorter side at most 128
// Every step in one kernel. A CTA holds 128 lines of X along its longer side (X seen as
// [length, shorter side]: line n, column i) as fp16 halves in shared memory for all steps, so
// that only A passes between CTAs:
//
//   A = X^T X         128 x 128 over this CTA's lines; the CTAs' sums are added
//   B = b A + c A^2   every CTA for itself
//   X' = X (a I + B)  its own lines
//
// hi is stored as rows n of 128 bytes (64 columns i, swizzled), two such chunks: K-major for
// the last product and, read along n, M/N-major for the first. Sums: one CTA needs none; up to
// sixteen are a cluster and exchange them through distributed shared memory (each CTA adds some
// rows, in rank order, and sends what A keeps of them to all, both counted in bytes on the
// receiver's barriers); more, or as many where such a cluster has no room, are a cooperative
// launch and go through the workspace, with a barrier over the grid before and after the adding.
//
// Bound by latency: a step is three products of 128^3 with their handshakes and epilogues, 1.25
// us each, and the exchange: 3 us in a cluster of eight, 5 to 6 over a grid. Five steps, from a
// graph: 128 x 128 26.5 us (98 as launches of tiled products), 128 x 1000 41 (59 with stores to
// each receiver and cluster barriers), 128 x 2000 45, 64 x 4096 55, 128 x 16384 60.
constexpr int SMALL = 128;
constexpr int SMALL_THREADS = 512;
constexpr int SMALL_BLOCK = SMALL * SMALL * 2;  // bytes of one fp16 block: two chunks of 128 rows x 128 bytes
constexpr int SMALL_MAX_CLUSTER = 16;  // (more than 8: where the GPU has room for one)
enum : int { SMALL_ONE = 0, SMALL_CLUSTER = 1, SMALL_GRID = 2 };
constexpr int kMaxSteps = 64;

struct SmallParams {
    ScaleParams x;   // X, its type, eps; partial sums of squares (SMALL_GRID)
    int64_t len;     // the longer side
    int s, wide;     // the shorter side; wide: X is [s, len]
    int mode, ctas, steps;
    float coeffs[3 * kMaxSteps];
    void *C;         // [m, n] bf16
    int64_t ldc;
    float alpha, beta;
    float4 *sums;         // SMALL_GRID: [CTA][4096], then A as its block lies in shared memory and its diagonal
    unsigned int *count;  // SMALL_GRID: arrivals, 0 at the start
    int *status;
    uint64_t timeout_ns;
    int debug_stall;
};

struct SmallSmem {
    static constexpr int HI = 0, LO = SMALL_BLOCK, A = 2 * SMALL_BLOCK, B = 3 * SMALL_BLOCK;
    static constexpr int RECV = 4 * SMALL_BLOCK;            // SMALL_CLUSTER: 64 KB of sums to add
    static constexpr int DIAG = RECV + SMALL * SMALL * 4;   // two vectors of 128 floats
    static constexpr int NORMS = DIAG + 2 * SMALL * 4;      // square sums of the cluster's CTAs
    static constexpr int PART = NORMS + 8 * SMALL_MAX_CLUSTER;
    static constexpr int BAR = PART + 8 * (SMALL_THREADS / 32);
    static constexpr int SCALE = BAR + 24 + 16;             // three barriers, tensor memory's address, abort flag; the scale
    static constexpr int BYTES = 1024 + SCALE + 8;
};
static_assert(SmallSmem::BYTES <= 227 * 1024, "shared memory");

// 16-byte unit `u` (0 .. 15) of row r of a block: unit u % 8 of chunk u / 8, swizzled.
__device__ __forceinline__ uint8_t *small_at(uint8_t *block, int r, int u)
{
    return block + (u >> 3) * (SMALL * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v)
{
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// A store to, and a copy of shared memory to, another CTA of the cluster, counted in bytes on a
// barrier of that CTA.
__device__ __forceinline__ void st_async_f4(uint32_t addr, float4 v, uint32_t cluster_bar)
{
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr), "f"(v.x),
        "f"(v.y), "f"(v.z), "f"(v.w), "r"(cluster_bar)
        : "memory");
}

__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t cluster_bar)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(cluster_bar)
                 : "memory");
}

// All CTAs have arrived `round` times; what they wrote before is visible. False when the wait
// ran out (once `ok` is false nothing is waited for).
__device__ __forceinline__ bool grid_barrier(const SmallParams &p, unsigned int round, bool ok, volatile int *abort_flag)
{
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.count) : "memory");
        const unsigned int target = round * static_cast<unsigned int>(p.ctas);
        const uint64_t t0 = global_timer_ns();
        for (;;) {
            unsigned int v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.count) : "memory");
            if (v >= target || *abort_flag != 0) break;
            if (global_timer_ns() - t0 > p.timeout_ns) {
                *abort_flag = 1;
                break;
            }
        }
    }
    __syncthreads();
    return ok && *abort_flag == 0;
}

__global__ void __launch_bounds__(SMALL_THREADS, 1) bm_orth_small_kernel(const __grid_constant__ SmallParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // the same offset in every CTA of a cluster
    uint8_t *smem = smem_raw + (base - raw);
    uint8_t *hi = smem + SmallSmem::HI, *lo = smem + SmallSmem::LO, *ba = smem + SmallSmem::A, *bb = smem + SmallSmem::B;
    float *diag_a = reinterpret_cast<float *>(smem + SmallSmem::DIAG), *diag_b = diag_a + SMALL;
    double *norms = reinterpret_cast<double *>(smem + SmallSmem::NORMS);
    double *part = reinterpret_cast<double *>(smem + SmallSmem::PART);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SmallSmem::BAR + 24);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    double *scale_at = reinterpret_cast<double *>(smem + SmallSmem::SCALE);
    const uint32_t bar = smem_addr(smem + SmallSmem::BAR), recv_bar = bar + 8u, all_bar = bar + 16u;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, quad = warp & 3, part4 = warp >> 2;
    const bool cluster = p.mode == SMALL_CLUSTER;
    const int rank = static_cast<int>(blockIdx.x);  // (a cluster is the whole grid)
    const int64_t n0 = static_cast<int64_t>(rank) * SMALL;

    if (t == 0) {
        mbar_init(bar, 1);       // a product is done
        mbar_init(recv_bar, 1);  // SMALL_CLUSTER: the others' sums of this CTA's rows
        mbar_init(all_bar, 1);   // and A from all of them
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_addr(tmem_slot), SMALL);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (cluster) cluster_arrive();
    griddep_launch_dependents();
    griddep_wait();

    // ---- X0 = 256 X / (|X| + eps): a thread takes eight values (of a line, X tall, or of eight
    // lines) of 2048 / 512 pieces, all loaded at once and kept until the norm is known. For X wide
    // the lanes of a warp take neighbouring columns i.
    constexpr int PIECES = 2048 / SMALL_THREADS;
    float x0[PIECES][8];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
        const int it = q * SMALL_THREADS + t, r = p.wide ? it & 127 : it >> 4, u = p.wide ? it >> 7 : it & 15;
        const int64_t i = p.wide ? r : n0 + r, j = p.wide ? n0 + 8 * u : 8 * u;
        if (i < p.x.m && j < p.x.n) {
            load_x8(p.x, i, j, x0[q]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x0[q][e] = 0.0f;
        }
    }
    double sum = 0.0;
    if (p.mode == SMALL_GRID) {
        for (int b = t; b < p.x.blocks; b += SMALL_THREADS) sum += p.x.partial[b];
    } else {
#pragma unroll
        for (int q = 0; q < PIECES; ++q) sum += square8(x0[q]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (cluster) {
        cluster_wait();  // every CTA has started: its shared memory may be written
        if (t < p.ctas) {
            double own = 0.0;
            for (int w = 0; w < SMALL_THREADS / 32; ++w) own += part[w];
            st_cluster_f64(map_shared_to_rank(smem_addr(norms + rank), static_cast<uint32_t>(t)), own);
        }
        __syncwarp();
        cluster_sync();
    }
    if (t == 0) {
        double all = 0.0;
        if (cluster) {
            for (int c = 0; c < p.ctas; ++c) all += norms[c];
        } else {
            for (int w = 0; w < SMALL_THREADS / 32; ++w) all += part[w];
        }
        *scale_at = orth_scale(all, p.x.eps);
    }
    __syncthreads();
    {
        const double scale = *scale_at;
        const float scale32 = static_cast<float>(scale);
        const bool in32 = scale_in32(scale);
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            const int it = q * SMALL_THREADS + t, r = p.wide ? it & 127 : it >> 4, u = p.wide ? it >> 7 : it & 15;
            uint32_t h[4], l[4];
            split8(x0[q], scale, scale32, in32, h, l);
            if (p.wide) {  // column r of lines 8 u .. 8 u + 7
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = (r & 7) * 2;
                    *reinterpret_cast<uint16_t *>(small_at(hi, 8 * u + e, r >> 3) + at) =
                        static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
                    *reinterpret_cast<uint16_t *>(small_at(lo, 8 * u + e, r >> 3) + at) =
                        static_cast<uint16_t>(l[e >> 1] >> (16 * (e & 1)));
                }
            } else {
                *reinterpret_cast<uint4 *>(small_at(hi, r, u)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(small_at(lo, r, u)) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    }

    // ---- steps
    const int row = quad * 32 + lane;  // this thread's accumulator row, and its 32 columns
    const int col = 32 * part4;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(col);
    uint32_t phase = 0;
    bool ok = true;
    // A product of two 128 x 128 blocks into tensor memory, once all threads have written their
    // parts of them (K over lines of hi: M/N-major; along rows: K-major).
    auto product = [&](uint8_t *x, uint8_t *y, bool lines, bool skip) {
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncthreads();
        if (t == 0 && ok && !skip) {
            tc_fence_after_sync();
            const uint64_t tpl = lines ? smem_desc_sw128(0u, SMALL * 128, 1024u) : smem_desc_sw128(0u, 16u, 1024u);
            const uint32_t idesc = idesc_f32acc(SMALL, SMALL, 0u, lines, lines);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t step = lines ? kk * 2048u : (kk >> 2) * (SMALL * 128u) + (kk & 3) * 32u;
                // (in a cluster the upper bits of a shared address hold the CTA's rank)
                umma_bf16(tmem, tpl + (((smem_addr(x) + step) & 0x3FFFFu) >> 4), tpl + (((smem_addr(y) + step) & 0x3FFFFu) >> 4),
                          idesc, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar);
        }
        ok = ok && wait_warp<false>(bar, phase, abort_flag, p.timeout_ns);
        if (!ok) *abort_flag = 1;  // (nothing more is issued or waited for; every barrier is still met)
        phase ^= 1u;
        tc_fence_after_sync();
    };
    // Four columns 4 q .. of row i of A from their sum: the halves off the diagonal, and the
    // diagonal's value where it is among them.
    auto entries = [&](const float4 &sum4, int i, int q, float &diag) {
        const float unit = 1.0f / (kOrthScale * kOrthScale);
        float a[4] = {sum4.x * unit, sum4.y * unit, sum4.z * unit, sum4.w * unit};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * q + e == i) {
                diag = a[e];
                a[e] = 0.0f;
            }
        return make_uint2(pack_f16(make_float2(a[0], a[1])), pack_f16(make_float2(a[2], a[3])));
    };
    auto block_offset = [](int i, int q) {  // bytes to columns 4 q .. of row i of a block
        return (q >> 4) * (SMALL * 128) + i * 128 + (((q >> 1) & 7) ^ (i & 7)) * 16 + (q & 1) * 8;
    };
    unsigned int round = 0, exchange = 0;  // of the grid's barriers, of the cluster's sums
    for (int step = 0; step < p.steps; ++step) {
        const float ca = p.coeffs[3 * step], cb = p.coeffs[3 * step + 1], cc = p.coeffs[3 * step + 2];
        product(hi, hi, true, p.debug_stall && step == 0);
        {
            float4 v[8];
            uint32_t r[32];
            tmem_load_32cols(taddr, r);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]), __uint_as_float(r[4 * e + 2]),
                                   __uint_as_float(r[4 * e + 3]));
            // The sum over the CTAs of columns 4 q .. of row i, 4096 such items.
            if (cluster) {
                // rows [rank R, ..) are this CTA's to add
                const int R = SMALL / p.ctas, owner = row / R, local = row - owner * R;
                const uint32_t recv = smem_addr(smem + SmallSmem::RECV) + static_cast<uint32_t>((rank * 32 * R + local) * 16);
                if (t == 0 && ok) {
                    mbar_arrive_expect_tx(recv_bar, static_cast<uint32_t>((p.ctas - 1) * 32 * R * 16));
                    mbar_arrive_expect_tx(all_bar, static_cast<uint32_t>((p.ctas - 1) * (2 * R * 128 + R * 4)));
                }
                const uint32_t to = map_shared_to_rank(recv, static_cast<uint32_t>(owner));
                const uint32_t to_bar = map_shared_to_rank(recv_bar, static_cast<uint32_t>(owner));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t at = static_cast<uint32_t>((8 * part4 + e) * R * 16);
                    if (owner == rank)
                        reinterpret_cast<float4 *>(smem + SmallSmem::RECV)[(rank * 32 + 8 * part4 + e) * R + local] = v[e];
                    else if (ok) st_async_f4(to + at, v[e], to_bar);
                }
                __syncthreads();
                ok = ok && wait_warp<true>(recv_bar, exchange & 1u, abort_flag, p.timeout_ns);
                if (!ok) *abort_flag = 1;
                const float4 *got = reinterpret_cast<const float4 *>(smem + SmallSmem::RECV);
                for (int k = t; k < 32 * R; k += SMALL_THREADS) {
                    float4 s4 = got[k];
                    for (int c = 1; c < p.ctas; ++c) {
                        const float4 x = got[c * 32 * R + k];
                        s4.x += x.x, s4.y += x.y, s4.z += x.z, s4.w += x.w;
                    }
                    const int q = k / R, i = rank * R + k - q * R;
                    float d = 0.0f;
                    *reinterpret_cast<uint2 *>(ba + block_offset(i, q)) = entries(s4, i, q, d);
                    if (i >> 2 == q) diag_a[i] = d;
                }
                // these rows of A to everybody: two runs of 128-byte rows and the diagonal's part
                fence_proxy_async_shared();
                __syncthreads();
                if (ok && t < p.ctas && t != rank) {
                    const uint32_t peer = static_cast<uint32_t>(t), bytes = static_cast<uint32_t>(R * 128);
                    const uint32_t peer_bar = map_shared_to_rank(all_bar, peer);
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = smem_addr(ba) + static_cast<uint32_t>(h * SMALL * 128 + rank * R * 128);
                        bulk_copy_cluster(map_shared_to_rank(at, peer), at, bytes, peer_bar);
                    }
                    const uint32_t at = smem_addr(diag_a + rank * R);
                    bulk_copy_cluster(map_shared_to_rank(at, peer), at, static_cast<uint32_t>(R * 4), peer_bar);
                }
                __syncwarp();
                ok = ok && wait_warp<true>(all_bar, exchange & 1u, abort_flag, p.timeout_ns);
                if (!ok) *abort_flag = 1;
                ++exchange;
            } else if (p.mode == SMALL_GRID) {
                float4 *own = p.sums + static_cast<int64_t>(rank) * 4096;
                uint8_t *total = reinterpret_cast<uint8_t *>(p.sums + static_cast<int64_t>(p.ctas) * 4096);
                float *total_diag = reinterpret_cast<float *>(total + SMALL_BLOCK);
#pragma unroll
                for (int e = 0; e < 8; ++e) own[128 * (8 * part4 + e) + row] = v[e];
                ok = grid_barrier(p, ++round, ok, abort_flag);
                // this CTA's share of the items: fewer than there are threads (9 CTAs or more), each by
                // `groups` threads, which take a run of the CTAs each and whose sums are added in order; or
                // a thread each, in passes (2 to 8 CTAs, where their cluster has no room)
                const int per = (4096 + p.ctas - 1) / p.ctas, groups = max(1, SMALL_THREADS / per);
                float4 *shared = reinterpret_cast<float4 *>(smem + SmallSmem::RECV);
                const int g = per < SMALL_THREADS ? t / per : 0;
                for (int k = t - g * per; k < per; k += SMALL_THREADS) {
                    const int item = rank * per + k;
                    if (g >= groups || item >= 4096) break;
                    const int run = (p.ctas + groups - 1) / groups, first = g * run, last = min(p.ctas, first + run);
                    const float4 *src = p.sums + item;
                    float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    int c = first;
                    for (; c + 8 <= last; c += 8) {
                        float4 x[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) x[q] = __ldcg(src + static_cast<int64_t>(c + q) * 4096);
#pragma unroll
                        for (int q = 0; q < 8; ++q) s4.x += x[q].x, s4.y += x[q].y, s4.z += x[q].z, s4.w += x[q].w;
                    }
                    for (; c < last; ++c) {
                        const float4 x = __ldcg(src + static_cast<int64_t>(c) * 4096);
                        s4.x += x.x, s4.y += x.y, s4.z += x.z, s4.w += x.w;
                    }
                    shared[g * per + k] = s4;
                }
                __syncthreads();
                if (g == 0) {
                    for (int k = t; k < per; k += SMALL_THREADS) {
                        const int item = rank * per + k;
                        if (item >= 4096) break;
                        float4 s4 = shared[k];
                        for (int q = 1; q < groups; ++q) {
                            const float4 x = shared[q * per + k];
                            s4.x += x.x, s4.y += x.y, s4.z += x.z, s4.w += x.w;
                        }
                        const int i = item & 127, q = item >> 7;
                        float d = 0.0f;
                        *reinterpret_cast<uint2 *>(total + block_offset(i, q)) = entries(s4, i, q, d);
                        if (i >> 2 == q) total_diag[i] = d;
                    }
                }
                ok = grid_barrier(p, ++round, ok, abort_flag);
                const uint4 *src = reinterpret_cast<const uint4 *>(total);
#pragma unroll
                for (int e = 0; e < SMALL_BLOCK / 16 / SMALL_THREADS; ++e)
                    reinterpret_cast<uint4 *>(ba)[e * SMALL_THREADS + t] = __ldcg(src + e * SMALL_THREADS + t);
                if (t < SMALL) diag_a[t] = __ldcg(total_diag + t);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int q = 8 * part4 + e;
                    float d = 0.0f;
                    *reinterpret_cast<uint2 *>(ba + block_offset(row, q)) = entries(v[e], row, q, d);
                    if (row >> 2 == q) diag_a[row] = d;
                }
            }
        }

        // B off its diagonal, and the diagonal of a I + B
        product(ba, ba, false, false);
        {
            uint32_t r[32];
            tmem_load_32cols(taddr, r);
            const float di = diag_a[row];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 aw = *reinterpret_cast<const uint4 *>(small_at(ba, row, (col >> 3) + u));
                const uint32_t o[4] = {aw.x, aw.y, aw.z, aw.w};
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = col + 8 * u + 2 * e;
                    const float2 a = f16_pair(o[e]), dj = *reinterpret_cast<const float2 *>(diag_a + j);
                    const float2 z = make_float2(__uint_as_float(r[8 * u + 2 * e]), __uint_as_float(r[8 * u + 2 * e + 1]));
                    float2 w = fma2(both(cc), fma2(add2(both(di), dj), a, z), mul2(both(cb), a));
                    if (j == (row & ~1)) {
                        diag_b[row] = ca + fmaf(cc, j == row ? z.x : z.y, fmaf(cc * di, di, cb * di));
                        if (j == row) w.x = 0.0f;
                        else w.y = 0.0f;
                    }
                    b[e] = pack_f16(w);
                }
                *reinterpret_cast<uint4 *>(small_at(bb, row, (col >> 3) + u)) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }

        // X' of line `row`, columns col ..
        product(hi, bb, false, false);
        const bool last = step == p.steps - 1;
        const int64_t n = n0 + row;
        const float alpha = p.alpha / kOrthScale;
        uint32_t r[32];
        tmem_load_32cols(taddr, r);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i0 = col + 8 * u;
            uint4 *at_hi = reinterpret_cast<uint4 *>(small_at(hi, row, i0 >> 3));
            uint4 *at_lo = reinterpret_cast<uint4 *>(small_at(lo, row, i0 >> 3));
            const uint4 xh = *at_hi, xl = *at_lo;
            const uint32_t h[4] = {xh.x, xh.y, xh.z, xh.w}, l[4] = {xl.x, xl.y, xl.z, xl.w};
            float2 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 d = *reinterpret_cast<const float2 *>(diag_b + i0 + 2 * e);
                v[e] = fma2(d, add2(f16_pair(h[e]), f16_pair(l[e])),
                            make_float2(__uint_as_float(r[8 * u + 2 * e]), __uint_as_float(r[8 * u + 2 * e + 1])));
            }
            if (!last) {
                uint32_t nh[4], nl[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    nh[e] = pack_f16(v[e]);
                    const float2 b = f16_pair(nh[e]);
                    nl[e] = pack_f16(make_float2(v[e].x - b.x, v[e].y - b.y));
                }
                *at_hi = make_uint4(nh[0], nh[1], nh[2], nh[3]);
                *at_lo = make_uint4(nl[0], nl[1], nl[2], nl[3]);
            } else if (ok && n < p.len && i0 < p.s) {
                __nv_bfloat16 *C = static_cast<__nv_bfloat16 *>(p.C);
                if (p.wide) {  // neighbouring lanes, neighbouring columns of C
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (i0 + e >= p.s) continue;
                        __nv_bfloat16 *at = C + static_cast<int64_t>(i0 + e) * p.ldc + n;
                        float x = alpha * (e & 1 ? v[e >> 1].y : v[e >> 1].x);
                        if (p.beta != 0.0f) x = fmaf(p.beta, __bfloat162float(*at), x);
                        *at = __float2bfloat16_rn(x);
                    }
                } else {
                    uint32_t old[4] = {0u, 0u, 0u, 0u}, w[4];
                    if (p.beta != 0.0f) load_row<8>(p.C, p.ldc, n, p.len, i0, p.s, old);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 x = mul2(v[e], both(alpha));
                        if (p.beta != 0.0f) x = fma2(both(p.beta), bf16_pair(old[e]), x);
                        w[e] = pack_bf16(x);
                    }
                    uint16_t *at = reinterpret_cast<uint16_t *>(C + n * p.ldc + i0);
                    if (i0 + 8 <= p.s) {
                        *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 7; ++e)
                            if (i0 + e < p.s) at[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
                    }
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (t == 0 && *abort_flag != 0) {
        if (p.status != nullptr) atomicCAS(p.status, 0, DEV_ERR_TIMEOUT);
        spin_ns(100000);  // products in flight finish before tensor memory is freed
    }
    __syncthreads();
    if (cluster) cluster_sync();  // no CTA leaves while another may still write to it
    if (warp == 0) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, SMALL);
    }
}

}  // namespace bm
