// bm_symm_kernel.cuh -- the symmetric products of bm_epi_kernel.cuh (GRAM and POLY) where their
// tiles leave SMs over: K is split over the CTAs of a cluster.
//
// One 128 x 128 tile of the lower triangle per cluster of two or four. Each CTA multiplies its
// k-blocks into tensor memory and stores the sums of 128 / S rows to each CTA of the cluster;
// after a cluster barrier a CTA adds its rows' sums in rank order and runs the epilogue on
// them, 32 rows x 32 columns a warp.
//
// Bound by latency: launch, loads, exchange, epilogue. Five steps, from a graph: 1024 x 1024
// 166 us with whole tiles, 133 with these; 512 x 2048 172 and 119; 1000 x 2162 218 and 152 (FP32 X;
// 140, 130 and 160 as calls). (Sums counted in bytes on the receiver's barrier instead of a cluster
// barrier: 137 at 1024 x 1024.) At most four CTAs share a tile however long K is: 129 x 16384, three
// tiles, 201 us, 256 x 65536 620.
#pragma once

#include "bm_epi_kernel.cuh"

namespace bm {

constexpr int SYMM_WARPS = 8;
constexpr int SYMM_THREADS = 32 * SYMM_WARPS;
constexpr int SYMM_STAGES = 4;
constexpr int SYMM_STAGE_BYTES = 2 * 16384;  // 128 rows of each operand x 128 bytes of K

struct SymmCfg {
    static constexpr int SUMS = SYMM_STAGES * SYMM_STAGE_BYTES;         // [CTA][4 columns][row] of this CTA's rows
    static constexpr int STAGING = SUMS + 128 * 128 * 4;
    static constexpr int BARS = STAGING + SYMM_WARPS * FUSED_STAGE_BYTES;
    static constexpr int BYTES = 1024 + BARS + 8 * (2 * SYMM_STAGES + 1) + 16;
};
static_assert(SymmCfg::BYTES <= 227 * 1024, "shared memory");

template <int S, int KIND>
__global__ void __launch_bounds__(SYMM_THREADS, 1)
    bm_symm_split_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tm0, const EpiParams f)
{
    constexpr int ROWS = 128 / S;  // of a tile that one CTA finishes
    const GemmParams &p = f.g;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;  // the same offset in every CTA of the cluster
    uint8_t *smem = smem_raw + (ring - raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SymmCfg::BARS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * SYMM_STAGES + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t bar0 = smem_addr(bars), done = bar0 + 8u * (2 * SYMM_STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = static_cast<int>(cluster_cta_rank());
    int64_t tm, tn;
    syrk_tile_coords<128, 128>(MODE_SYRK_LOWER, p.tiles_m, p.tiles_n, cluster_index(), tm, tn);
    const int count = (p.kb_total - r + S - 1) / S;  // this CTA's k-blocks r, r + S, ...
    const bool mn = p.a_mn_major != 0, one = tm == tn;  // one: both operands are the same rows

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * SYMM_STAGES + 1; ++s) mbar_init(bar0 + 8u * s, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&tmX);
        tma_prefetch_map(&tm0);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 128);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    cluster_arrive();
    griddep_launch_dependents();
    griddep_wait();

    // The rows and columns that this warp finishes, and what they need.
    const int quad = S == 4 ? r : 2 * r + (warp >> 2), part = warp & 3;
    const bool finisher = S == 2 || warp < 4;
    const int64_t i0 = tm * 128 + quad * 32, j0 = tn * 128 + part * 32;
    const bool live = finisher && i0 < p.m && j0 < p.n;
    uint32_t x[16] = {};
    float di = 0.0f, dcol = 0.0f;
    if (KIND == KIND_POLY && live) {
        load_row<32>(f.in[0], f.ldin[0], i0 + lane, p.m, j0, f.in_cols, x);
        di = i0 + lane < p.m ? f.diag[i0 + lane] : 0.0f;
        dcol = j0 + lane < p.n ? f.diag[j0 + lane] : 0.0f;
    }

    if (warp == 0 && lane == 0) {
        // ---- copies
        uint32_t armed = 0, armed_parity = 0, phase = 0;
        int stage = 0;
        bool ok = true;
        auto load = [&](uint32_t dst, uint32_t full, int64_t row, int kx) {
            if (mn) {
                tma_load_2d(dst, &tmX, full, static_cast<int32_t>(row), kx);
                tma_load_2d(dst + 8192u, &tmX, full, static_cast<int32_t>(row + 64), kx);
            } else {
                tma_load_2d(dst, &tmX, full, kx, static_cast<int32_t>(row));
            }
        };
        for (int i = 0; i < count; ++i) {
            if (!wait_one(bar0 + 8u * (SYMM_STAGES + stage), phase ^ 1u, abort_flag, p.timeout_ns)) {
                ok = false;
                break;
            }
            const uint32_t full = bar0 + 8u * stage, st = ring + stage * SYMM_STAGE_BYTES;
            mbar_arrive_expect_tx(full, one ? 16384u : SYMM_STAGE_BYTES);
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (!(p.debug_stall && i == 0)) {
                const int kx = (r + S * i) * TILE_K;
                load(st, full, tm * 128, kx);
                if (!one) load(st + 16384u, full, tn * 128, kx);
            }
            if (++stage == SYMM_STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {
            signal_timeout(p, abort_flag);
            for (int s = 0; s < SYMM_STAGES; ++s)  // copies in flight land before shared memory is released
                if ((armed >> s) & 1u) wait_one(bar0 + 8u * s, (armed_parity >> s) & 1u, nullptr, p.timeout_ns);
        }
    } else if (warp == 1 && lane == 0) {
        // ---- products
        const uint64_t tpl = mn ? smem_desc_sw128(0u, 8192u, 1024u) : smem_desc_sw128(0u, 16u, 1024u);
        const uint32_t step = mn ? 2048u / 16u : 32u / 16u, second = one ? 0u : 16384u / 16u;
        const uint32_t idesc = idesc_f32acc(128, 128, 0u, mn, mn);
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
            const uint32_t at = ((ring + stage * SYMM_STAGE_BYTES) & 0x3FFFFu) >> 4;
#pragma unroll
            for (int kk = 0; kk < TILE_K / UMMA_K; ++kk)
                umma_bf16(tmem, tpl + at + step * kk, tpl + at + second + step * kk, idesc, i > 0 || kk > 0 ? 1u : 0u);
            issued = true;
            umma_commit(bar0 + 8u * (SYMM_STAGES + stage));
            if (++stage == SYMM_STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) signal_timeout(p, abort_flag);
        if (ok || issued) umma_commit(done);
        if (!ok && issued) wait_one(done, 0u, nullptr, p.timeout_ns);  // before TMEM is freed
    }
    __syncwarp();

    // ---- this CTA's sums of each row to the CTA that finishes it
    const bool ok = wait_warp<false>(done, 0u, abort_flag, p.timeout_ns);
    if (!ok && lane == 0) signal_timeout(p, abort_flag);
    tc_fence_after_sync();
    cluster_wait();  // every CTA has started: its shared memory may be written
    const uint32_t sums = smem_addr(smem + SymmCfg::SUMS);
    if (ok) {
        const int q = warp & 3, first = (warp >> 2) * 16;  // rows 32 q .., sets of four columns first ..
        const uint32_t owner = static_cast<uint32_t>(32 * q / ROWS);
        const int local = 32 * q % ROWS + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(4 * first);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_load_32cols(taddr + 32u * h, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                st_cluster_f4(map_shared_to_rank(
                                  sums + static_cast<uint32_t>(((r * 32 + first + 8 * h + e) * ROWS + local) * 16), owner),
                              make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                          __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3])));
        }
    }
    tc_fence_before_sync();
    cluster_sync();  // every CTA's sums have arrived

    if (ok && live) {
        const float4 *got = reinterpret_cast<const float4 *>(smem + SymmCfg::SUMS);
        const int local = (quad * 32) % ROWS + lane;
        uint8_t *block = smem + SymmCfg::STAGING + warp * FUSED_STAGE_BYTES;
        uint32_t t[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float z[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int set = part * 8 + 4 * h + e;
                float4 s4 = got[set * ROWS + local];
#pragma unroll
                for (int c = 1; c < S; ++c) {
                    const float4 y = got[(c * 32 + set) * ROWS + local];
                    s4.x += y.x, s4.y += y.y, s4.z += y.z, s4.w += y.w;
                }
                z[4 * e] = s4.x, z[4 * e + 1] = s4.y, z[4 * e + 2] = s4.z, z[4 * e + 3] = s4.w;
            }
            symmetric_half<KIND>(f, z, x + 8 * h, di, dcol, i0, j0, h, t + 8 * h, lane);
        }
        store_rows<32>(f, 0, &tm0, block, t, i0, j0, lane);
        if (!one) store_mirrored(&tm0, block, t, i0, j0, lane);
        if (lane == 0) bulk_wait_group0();  // shared memory must outlive the stores that read it
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, 128);
    }
}

}  // namespace bm
