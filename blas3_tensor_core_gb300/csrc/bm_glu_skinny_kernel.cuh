// bm_glu_skinny_kernel.cuh -- a gated MLP's products (bm_epi_kernel.cuh, GLU and DGLU) for
// few rows (m <= 128: served tokens), where reading the weights once is the work.
//
// The plan is that of bm_skinny_kernel.cuh: the weights take the 128-row side of the MMA, the
// m rows its narrow side, K is split over the CTAs of a cluster, and each row's sums meet in
// one CTA's shared memory, in rank order. A GLU tile is 64 columns of H: 64 rows of the gate's
// weights and the same 64 of the up projection's, so that a row's g and u of a column meet in
// one lane. Everything is rounded to BF16 on its way out, so K is accumulated in one piece.
//
// Bound by HBM. 1 x 4096 x 4096 (both weights, 67 MB: 9.9 us) 14.0 us, with the tile
// kernel's 128 x 64 tiles 35: 64 CTAs of them do not ask for enough at once.
#pragma once

#include "bm_epi_kernel.cuh"
#include "bm_skinny_kernel.cuh"

namespace bm {

struct GluSkinnyParams {
    EpiParams f;
    int cluster;  // CTAs per cluster: K is split over them
};

// Two values (j even) or four (j a multiple of 4) of row i from column j on, masked at the
// row's end.
__device__ __forceinline__ void store_2(void *X, int64_t ld, int64_t i, int64_t j, int64_t n, float2 v)
{
    uint16_t *dst = static_cast<uint16_t *>(X) + i * ld + j;
    const uint32_t w = pack_bf16(v);
    if (j + 2 <= n) *reinterpret_cast<uint32_t *>(dst) = w;
    else if (j < n) *dst = static_cast<uint16_t>(w);
}

__device__ __forceinline__ void store_4(void *X, int64_t ld, int64_t i, int64_t j, int64_t n, const float2 (&v)[2])
{
    uint16_t *dst = static_cast<uint16_t *>(X) + i * ld + j;
    const uint2 w = make_uint2(pack_bf16(v[0]), pack_bf16(v[1]));
    if (j + 4 <= n) {
        *reinterpret_cast<uint2 *>(dst) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (j + e < n) dst[e] = static_cast<uint16_t>((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
    }
}

__device__ __forceinline__ uint2 load_4(const void *X, int64_t ld, int64_t i, int64_t j, int64_t n)
{
    const uint16_t *src = static_cast<const uint16_t *>(X) + i * ld + j;
    if (j + 4 <= n) return *reinterpret_cast<const uint2 *>(src);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (j + e < n) w[e >> 1] |= static_cast<uint32_t>(src[e]) << (16 * (e & 1));
    return make_uint2(w[0], w[1]);
}

template <int NT, int KIND>
__global__ void __launch_bounds__(SKINNY_THREADS, 1)
    bm_glu_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
                         const __grid_constant__ CUtensorMap tmX, const GluSkinnyParams sp)
{
    using Cfg = SkinnyCfg<NT>;
    constexpr bool GLU = KIND == KIND_GLU;
    constexpr int STAGES = Cfg::STAGES;
    constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
    const EpiParams &f = sp.f;
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
    const int32_t n0 = static_cast<int32_t>(tile * (GLU ? 64 : 128));
    // this CTA's k-blocks are r, r + S, ...
    const int S = sp.cluster, r = static_cast<int>(rank);
    const int count = (p.kb_total - r + S - 1) / S;
    // The stage's 128 x 64 block of weights in two copies (one, K-major, for DGLU): gate and up,
    // or the two chunks of 64 columns.
    const CUtensorMap *second = GLU ? &tmW2 : &tmW;
    const int32_t n1 = GLU ? n0 : n0 + 64;
    const bool two = GLU || p.b_mn_major;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar0 + 8u * s, 1);
            mbar_init(bar0 + 8u * (STAGES + s), 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&tmW);
        if (GLU) tma_prefetch_map(&tmW2);
        tma_prefetch_map(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
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
            const int kx = (r + S * i) * TILE_K;
            if (p.b_mn_major) {
                tma_prefetch_2d(&tmW, n0, kx);
                tma_prefetch_2d(second, n1, kx);
            } else {
                tma_prefetch_2d(&tmW, kx, n0);
                if (two) tma_prefetch_2d(second, kx, n1);
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
            const int kx = (r + S * i) * TILE_K;
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
                    tma_load_2d(w, &tmW, full, n0, kx);
                    tma_load_2d(w + 8192u, second, full, n1, kx);
                } else {
                    tma_load_2d(w, &tmW, full, kx, n0);
                    if (two) tma_load_2d(w + 8192u, second, full, kx, n1);
                }
                if (p.a_mn_major) {
#pragma unroll
                    for (int c = 0; c < (NT + 63) / 64; ++c) tma_load_2d(x + c * 8192u, &tmX, full, 64 * c, kx);
                } else {
                    tma_load_2d(x, &tmX, full, kx, 0);
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
        // ---- MMAs: D[128 rows of weights][NT rows of A]
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
            // (in a cluster the upper bits of a shared address hold the CTA's rank)
            const uint32_t wd = ((ring + stage * Cfg::STAGE_BYTES) & 0x3FFFFu) >> 4;
#pragma unroll
            for (int kk = 0; kk < TILE_K / UMMA_K; ++kk)
                umma_bf16(tmem_base, w_tpl + wd + w_kk * kk, x_tpl + wd + SKINNY_W_BYTES / 16 + x_kk * kk, idesc,
                          i > 0 || kk > 0 ? 1u : 0u);
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

    // ---- this CTA's sums of row i to CTA i % S: [i / S][this CTA][row of the weights' block]
    const bool ok = wait_warp<false>(done, 0u, abort_flag, p.timeout_ns);
    if (!ok && lane == 0) signal_timeout(p, abort_flag);
    tc_fence_after_sync();
    const uint32_t sums_addr = smem_addr(sums);
    cluster_wait();  // every CTA has started: its shared memory may be written
    if (ok) {
        const int quad = warp & 3;  // TMEM lanes 32 quad ..; two warps share them, 16 rows in turn
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        const int column = quad * 32 + lane;
#pragma unroll 1
        for (int t0 = (warp >> 2) * 16; t0 < NT && t0 < p.m; t0 += 32) {
            uint32_t q[16];
            tmem_load_16cols(taddr + static_cast<uint32_t>(t0), q);
            int owner = t0 % S, slot = t0 / S;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (t0 + e < p.m)
                    st_cluster_f1(map_shared_to_rank(sums_addr + static_cast<uint32_t>(((slot * S + r) * 128 + column) * 4),
                                                     static_cast<uint32_t>(owner)),
                                  __uint_as_float(q[e]));
                if (++owner == S) owner = 0, ++slot;
            }
        }
    }
    tc_fence_before_sync();
    cluster_sync();  // every CTA's sums have arrived

    // ---- rows rank + S q, one warp per row: sum over the cluster in rank order, epilogue
    if (ok) {
        const float2 alpha = both(p.alpha);
        for (int i = r + S * warp, slot = warp; i < p.m; i += S * SKINNY_WARPS, slot += SKINNY_WARPS) {
            if constexpr (GLU) {
                const int64_t j = n0 + lane * 2;
                const float2 *q = reinterpret_cast<const float2 *>(sums) + slot * S * 64 + lane;
                float2 gate = make_float2(0.0f, 0.0f), up = gate;
                for (int c = 0; c < S; ++c) {
                    gate = add2(gate, q[c * 64]);
                    up = add2(up, q[c * 64 + 32]);
                }
                gate = mul2(gate, alpha);
                up = mul2(up, alpha);
                with_act(f.act, [&](auto tag) {
                    store_2(f.out[0], f.ldout[0], i, j, p.n, mul2(act_value2<decltype(tag)::value>(gate), up));
                });
                if (f.out[1] != nullptr) {
                    store_2(f.out[1], f.ldout[1], i, j, p.n, gate);
                    store_2(f.out[2], f.ldout[2], i, j, p.n, up);
                }
            } else {
                const int64_t j = n0 + lane * 4;
                if (j >= p.n) continue;
                const uint2 gw = load_4(f.in[0], f.ldin[0], i, j, p.n), uw = load_4(f.in[1], f.ldin[1], i, j, p.n);
                const float4 *q = reinterpret_cast<const float4 *>(sums) + slot * S * 32 + lane;
                float2 dh[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                for (int c = 0; c < S; ++c) {
                    const float4 v = q[c * 32];
                    dh[0] = add2(dh[0], make_float2(v.x, v.y));
                    dh[1] = add2(dh[1], make_float2(v.z, v.w));
                }
                float2 dg[2], du[2], h[2];
                with_act(f.act, [&](auto tag) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 d = mul2(dh[e], alpha), gate = bf16_pair(e == 0 ? gw.x : gw.y);
                        const float2 up = bf16_pair(e == 0 ? uw.x : uw.y);
                        const ActPair a = act_pair2<decltype(tag)::value>(gate);
                        dg[e] = mul2(mul2(d, up), a.slope);
                        du[e] = mul2(d, a.value);
                        h[e] = mul2(a.value, up);
                    }
                });
                store_4(f.out[0], f.ldout[0], i, j, p.n, dg);
                store_4(f.out[1], f.ldout[1], i, j, p.n, du);
                if (f.out[2] != nullptr) store_4(f.out[2], f.ldout[2], i, j, p.n, h);
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

}  // namespace bm
