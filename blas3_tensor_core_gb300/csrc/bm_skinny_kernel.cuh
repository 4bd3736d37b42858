// bm_skinny_kernel.cuh -- the products of bm_fused_kernel.cuh for few rows (m <= 128:
// served tokens), where reading op(B) once is the work.
//
// The weights take the 128-row side of the MMA and the m rows its narrow side, N = 16,
// 32, 64 or 128 (D = op(B)^T op(A)^T, one tile of 128 columns of C per cluster), so no
// tensor-core row is spent on padding the batch and one CTA needs only 16 KB of weights
// plus N * 128 bytes of A per 64 of K in flight. K is split over the CTAs of a cluster:
// each keeps its own ring and accumulator and stores its sums of row i into the shared
// memory of CTA i % S; after a cluster barrier every CTA adds its rows' S sums in rank
// order and runs the epilogue on them. So there is one launch, no workspace, and
// nothing but A, B and the outputs moves through global memory. Bound by HBM (or L2,
// where the weights stay there between calls). (Reading the other CTAs' sums instead
// costs a remote load's latency per row: 128 x 256 x 256 took 14.1 us.)
//
// One CTA per SM with a ring of about 170 KB. (Two per SM with half the ring each divide
// the columns over the GPU more evenly, and took as long for one row and up to a quarter
// longer for 64: 37.3 us at 64 x 4096 x 16384, 29.5 here.) Accumulation in chunks of 512
// of K (256 when a checkpoint is kept), longer ones where a CTA's share has more than its
// TMEM columns hold (four at 128 rows, 32 at 16): each chunk has its own columns, and all
// are added in FP32 at the end. (With half the columns 100 x 4096 x 8192 took 19.4 us
// instead of 19.8, at a relative error of 9.9e-7 instead of 4.7e-7.)
//
// 24 x 5120 x 5120 with bias and residual 15.2 us (3.5 TB/s of weights that are not in L2),
// 1 x 4096 x 4096 10.2 us through the Python call and 9.8 from a graph, of which the bytes
// are 5: what is left is the latency of the launch, the ring's first loads, the cluster
// barrier and the epilogue.
//
// Eight warps: warp 0's first lane issues the copies, warp 1's first lane the MMAs, then
// all run the epilogue (two per 32 TMEM lanes, then one per row). Every wait is bounded.
#pragma once

#include "bm_fused_kernel.cuh"

namespace bm {

constexpr int SKINNY_WARPS = 8;
constexpr int SKINNY_THREADS = 32 * SKINNY_WARPS;
constexpr int SKINNY_TMEM_COLS = 512;   // at most: all of an SM's, which one CTA has to itself
constexpr int SKINNY_W_BYTES = 16384;   // 128 rows x 128 bytes of K

template <int NT>
struct SkinnyCfg {
    static constexpr int STAGES = NT == 16 ? 10 : NT == 32 ? 9 : NT == 64 ? 7 : 4;
    static constexpr int X_BYTES = NT * 128;
    static constexpr int STAGE_BYTES = SKINNY_W_BYTES + X_BYTES;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
    // the cluster's sums of this CTA's rows, [i / S][CTA][128]: ceil(NT / S) S <= NT + 7 of them
    static constexpr int SUMS_BYTES = (NT + 7) * 128 * 4;
    static constexpr int COLSUM_BYTES = 8 * SKINNY_WARPS * 128 * 4;  // column sums [CTA][warp][128], over the ring
    static constexpr int NUM_BARS = 2 * STAGES + 1;
    static constexpr int SMEM_BYTES = 1024 + RING_BYTES + SUMS_BYTES + 8 * NUM_BARS + 16;
    static_assert(COLSUM_BYTES <= RING_BYTES, "reuse of the ring");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct SkinnyParams {
    FusedParams f;
    int cluster;       // CTAs per cluster: K is split over them
    int chunk_kb;      // k-blocks per accumulator chunk
    int tmem_cols;     // power of two >= 32
    float *dbias;      // backward: column sums, or null
    int accumulate;
};

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

template <int NT, bool BWD>
__global__ void __launch_bounds__(SKINNY_THREADS, 1)
    bm_gemm_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                          const SkinnyParams sp)
{
    using Cfg = SkinnyCfg<NT>;
    constexpr int STAGES = Cfg::STAGES;
    const FusedParams &f = sp.f;
    const GemmParams &p = f.g;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;  // the same offset in every CTA of the cluster
    uint8_t *smem = smem_raw + (ring - raw);
    uint8_t *sums = smem + Cfg::RING_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sums + Cfg::SUMS_BYTES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Cfg::NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t bar0 = smem_addr(bars);
    const uint32_t done = bar0 + 8u * (2 * STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_cta_rank();
    const int64_t tile = cluster_index();
    const int32_t n0 = static_cast<int32_t>(tile * 128);
    // this CTA's k-blocks are r, r + S, ...: the cluster's copies walk along the rows of the
    // weights together, in pieces of S * 128 bytes
    const int S = sp.cluster, r = static_cast<int>(rank);
    const int count = (p.kb_total - r + S - 1) / S;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar0 + 8u * s, 1);
            mbar_init(bar0 + 8u * (STAGES + s), 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&tmW);
        tma_prefetch_map(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), static_cast<uint32_t>(sp.tmem_cols));
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    cluster_arrive();
    griddep_launch_dependents();
    // While the previous kernel finishes, the weights start towards L2 (a prefetch only
    // warms the cache, so it is safe even if that kernel writes them).
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < count && i < STAGES; ++i) {
            const int kb = r + S * i;
            if (p.b_mn_major) {
                tma_prefetch_2d(&tmW, n0, kb * TILE_K);
                tma_prefetch_2d(&tmW, n0 + 64, kb * TILE_K);
            } else {
                tma_prefetch_2d(&tmW, kb * TILE_K, n0);
            }
        }
    }
    griddep_wait();

    if (warp == 0 && lane == 0) {
        // ---- copies
        uint32_t armed = 0, armed_parity = 0, phase = 0;
        int stage = 0;
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            const int kb = r + S * i;
            if (!wait_one(bar0 + 8u * (STAGES + stage), phase ^ 1u, abort_flag, p.timeout_ns)) {
                ok = false;
                break;
            }
            const uint32_t full = bar0 + 8u * stage, w = ring + stage * Cfg::STAGE_BYTES, x = w + SKINNY_W_BYTES;
            mbar_arrive_expect_tx(full, Cfg::STAGE_BYTES);
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (!(p.debug_stall && i == 0)) {
                if (p.b_mn_major) {
                    tma_load_2d(w, &tmW, full, n0, kb * TILE_K);
                    tma_load_2d(w + 8192u, &tmW, full, n0 + 64, kb * TILE_K);
                } else {
                    tma_load_2d(w, &tmW, full, kb * TILE_K, n0);
                }
                if (p.a_mn_major) {
#pragma unroll
                    for (int c = 0; c < (NT + 63) / 64; ++c) tma_load_2d(x + c * 8192u, &tmX, full, 64 * c, kb * TILE_K);
                } else {
                    tma_load_2d(x, &tmX, full, kb * TILE_K, 0);
                }
            }
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {
            signal_timeout(p, abort_flag);
            for (int s = 0; s < STAGES; ++s)  // copies in flight land before shared memory is released
                if ((armed >> s) & 1u) wait_one(bar0 + 8u * s, (armed_parity >> s) & 1u, nullptr, p.timeout_ns);
        }
    } else if (warp == 1 && lane == 0) {
        // ---- MMAs: D[128 columns of C][NT rows] per chunk of K
        const uint64_t w_tpl = p.b_mn_major ? smem_desc_sw128(0u, 8192u, 1024u) : smem_desc_sw128(0u, 16u, 1024u);
        const uint64_t x_tpl = p.a_mn_major ? smem_desc_sw128(0u, 8192u, 1024u) : smem_desc_sw128(0u, 16u, 1024u);
        const uint32_t w_kk = p.b_mn_major ? 2048u / 16u : 32u / 16u, x_kk = p.a_mn_major ? 2048u / 16u : 32u / 16u;
        const uint32_t idesc = idesc_f32acc(128, NT, 1u, p.b_mn_major, p.a_mn_major);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true, issued = false;
        for (int i = 0; i < count; ++i) {
            if (!wait_one(bar0 + 8u * stage, phase, abort_flag, p.timeout_ns)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            // the descriptor's address field: the offset in this CTA's own shared memory (in a
            // cluster the upper bits of a shared address hold the CTA's rank)
            const uint32_t wd = ((ring + stage * Cfg::STAGE_BYTES) & 0x3FFFFu) >> 4;
            const int in_chunk = i % sp.chunk_kb;
            const uint32_t d = tmem_base + static_cast<uint32_t>(i / sp.chunk_kb * NT);
#pragma unroll
            for (int kk = 0; kk < TILE_K / UMMA_K; ++kk)
                umma_bf16(d, w_tpl + wd + w_kk * kk, x_tpl + wd + SKINNY_W_BYTES / 16 + x_kk * kk, idesc,
                          in_chunk > 0 || kk > 0 ? 1u : 0u);
            issued = true;
            umma_commit(bar0 + 8u * (STAGES + stage));
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) signal_timeout(p, abort_flag);
        if (ok || issued) umma_commit(done);
        if (!ok && issued) wait_one(done, 0u, nullptr, p.timeout_ns);  // before TMEM is freed
    }
    __syncwarp();

    // ---- this CTA's sums of row i to CTA i % S: [i / S][this CTA][column of the tile]
    const bool ok = wait_warp<false>(done, 0u, abort_flag, p.timeout_ns);
    if (!ok && lane == 0) signal_timeout(p, abort_flag);
    tc_fence_after_sync();
    const uint32_t sums_addr = smem_addr(sums);
    cluster_wait();  // every CTA has started: its shared memory may be written
    if (ok) {
        const int quad = warp & 3;  // TMEM lanes 32 quad ..; two warps share them, 16 rows in turn
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        const int chunks = (count + sp.chunk_kb - 1) / sp.chunk_kb;
        const int column = quad * 32 + lane;
#pragma unroll 1
        for (int t0 = (warp >> 2) * 16; t0 < NT && t0 < p.m; t0 += 32) {
            float v[16];
            for (int c = 0; c < chunks; ++c) {
                uint32_t q[16];
                tmem_load_16cols(taddr + static_cast<uint32_t>(c * NT + t0), q);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = c == 0 ? __uint_as_float(q[e]) : v[e] + __uint_as_float(q[e]);
            }
            int owner = t0 % S, slot = t0 / S;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (t0 + e < p.m)
                    st_cluster_f1(map_shared_to_rank(sums_addr + static_cast<uint32_t>(((slot * S + r) * 128 + column) * 4),
                                                     static_cast<uint32_t>(owner)),
                                  v[e]);
                if (++owner == S) owner = 0, ++slot;
            }
        }
    }
    tc_fence_before_sync();
    cluster_sync();  // every CTA's sums have arrived

    // ---- rows rank + S q, one warp per row: sum over the cluster in rank order, epilogue
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ok) {
        const int64_t j = n0 + lane * 4;
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (!BWD) load_bias4(f, j, b);
        const int rows = !BWD && f.Q != nullptr ? 128 : static_cast<int>(p.m);
        Row4 next = load_row4<BWD>(f, r + S * warp, j);
        for (int i = r + S * warp, slot = warp; i < rows; i += S * SKINNY_WARPS, slot += SKINNY_WARPS) {
            const Row4 now = next;
            next = load_row4<BWD>(f, i + S * SKINNY_WARPS, j);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (i < p.m) {
                const float4 *q = reinterpret_cast<const float4 *>(sums) + slot * S * 32 + lane;
                for (int c = 0; c < S; ++c) {
                    const float4 x = q[c * 32];
                    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                }
            }
            fused_row4<BWD>(f, i, j, v, b, now, sum, lane);
        }
    }
    if (BWD && sp.dbias != nullptr) {
        // the warps' column sums to CTA 0 (over its ring, which it has done with), which adds
        // them in (CTA, warp) order
        st_cluster_f4(map_shared_to_rank(ring + static_cast<uint32_t>(((r * SKINNY_WARPS + warp) * 128 + lane * 4) * 4), 0u),
                      make_float4(sum[0], sum[1], sum[2], sum[3]));
        cluster_sync();
        const int64_t j = n0 + static_cast<int64_t>(threadIdx.x);
        if (r == 0 && ok && threadIdx.x < 128 && j < p.n) {
            const float *all = reinterpret_cast<const float *>(smem);
            float s = 0.0f;
            for (int q = 0; q < SKINNY_WARPS * S; ++q) s += all[q * 128 + threadIdx.x];
            sp.dbias[j] = sp.accumulate ? sp.dbias[j] + s : s;
        }
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, static_cast<uint32_t>(sp.tmem_cols));
    }
}

}  // namespace bm
