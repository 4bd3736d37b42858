// bm_epi.h -- host-side parts shared by the products of bm_epi_kernel.cuh: tiles and
// launches. Included by the translation units that hold the kernel copies.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "bm_epi_kernel.cuh"
#include "bm_host.h"
#include "bm_ops.h"

namespace bmh {

// The maps of a launch: A, B, a second B; outputs; inputs of the outputs' shape.
struct EpiMaps {
    CUtensorMap a, b, b2, out[3], in[2];
    EpiMaps() { std::memset(this, 0, sizeof(*this)); }
};

using EpiKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap,
                           CUtensorMap, bm::EpiParams);

template <int KIND>
EpiKernel epi_kernel(int v)
{
    if (v == kSingle128) return &bm::bm_gemm_epi_kernel<128, 3, 1, 2, KIND>;
    if constexpr (!bm::kind_symmetric(KIND))
        if (v == kSingle256) return &bm::bm_gemm_epi_kernel<256, 4, 1, 1, KIND>;
    return &bm::bm_gemm_epi_kernel<256, 3, 2, 2, KIND>;
}

inline int epi_smem(int v)
{
    switch (v) {
    case kSingle256: return bm::FusedCfg<256, 4, 1, 1>::FUSED_SMEM;
    case kSingle128: return bm::FusedCfg<128, 3, 1, 2>::FUSED_SMEM;
    default: return bm::FusedCfg<256, 3, 2, 2>::FUSED_SMEM;
    }
}

// The dynamic shared-memory size of every copy of a kind (once per device, by the caller). The
// warps share out the registers that the launch gives a block: with fewer than the split adds
// up to the epilogue's increase would wait for ever, so such a build is refused here.
template <int KIND>
bool epi_attrs()
{
    for (int v : {kSingle256, kSingle128, kPair256}) {
        const void *fn = reinterpret_cast<const void *>(epi_kernel<KIND>(v));
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, fn) != cudaSuccess || a.numRegs < bm::FUSED_LAUNCH_REGS ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 epi_smem(bm::kind_symmetric(KIND) && v == kSingle256 ? kPair256 : v)) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
    }
    return true;
}

// The GEMM planner's tile for an m x n accumulator, but for three cases: 128 x 128 tiles where
// all of them run at once on single SMs, or K is short (the rules and figures of plan_fused);
// 128 x 256 tiles on single SMs where these make one wave and pairs more than one (1111 x 2048 x
// 1000, GLU: 11.2 us, 15.6 on pairs).
inline int epi_variant(int64_t m, int64_t n, int64_t k, int sms, int pair_clusters)
{
    const Plan whole = plan_gemm(m, n, k, 0, sms, pair_clusters);
    if (tile_override() != 0) return whole.variant;
    if (ceil_div(m, 128) * ceil_div(n, 128) <= sms) return kSingle128;
    if (whole.variant == kSingle256 && whole.num_tiles > sms) return kSingle128;
    if (whole.variant == kPair256 && whole.num_tiles > pair_clusters && ceil_div(m, 128) * ceil_div(n, 256) <= sms)
        return kSingle256;
    return whole.variant;
}

// Whole tiles of variant v over an m x n accumulator (GLU: n counts both projections'
// columns), or over its lower triangle.
inline Plan epi_plan(int v, int64_t m, int64_t n, int64_t k, bool triangle, int sms, int pair_clusters)
{
    Plan pl;
    pl.variant = v;
    pl.bn = kVariantBN[v];
    pl.stages = kVariantStages[v];
    pl.pair = kVariantPair[v];
    pl.tile_m = bm::CTA_M * pl.pair;
    pl.tiles_m = ceil_div(m, pl.tile_m);
    pl.tiles_n = ceil_div(n, pl.bn);
    pl.num_tiles = triangle ? pl.tiles_m * (pl.tiles_m + 1) / 2 : pl.tiles_m * pl.tiles_n;
    pl.full_tiles = pl.num_units = pl.num_tiles;
    pl.kb_total = pl.kb_per_split = static_cast<int>(ceil_div(std::max<int64_t>(k, 1), bm::TILE_K));
    // A last wave that is at most half full runs as halves of its tiles' columns, on twice as
    // many SM pairs (X' of 4096 x 4096: 256 tiles for 76 pairs, 98 us whole and 93 in halves).
    if (v == kPair256 && !triangle && pl.kb_total >= 8 && pair_clusters > 0) {
        const int64_t tail = pl.num_tiles % pair_clusters;
        if (tail > 0 && 2 * tail <= pair_clusters) {
            pl.n_split = 2;
            pl.full_tiles = pl.num_tiles - tail;
            pl.num_units = pl.num_tiles + tail;
        }
    }
    pl.ctas = static_cast<int>(pl.pair == 2 ? 2 * std::min<int64_t>(pl.num_units, pair_clusters)
                                            : std::min<int64_t>(pl.num_units, sms));
    return pl;
}

// An operand's map: its stage box where it has one (then *box3 is set), else boxes of a k-block.
inline bool epi_operand(CUtensorMap *map, int *box3, const void *X, bool mn_major, int64_t rows, int64_t k, int64_t ld,
                        int tile_rows, int kps)
{
    *box3 = encode_stage_box(map, X, bm::ELEM_BF16, mn_major, rows, k, ld, tile_rows, kps) ? 1 : 0;
    return *box3 != 0 || encode_operand(map, X, mn_major, rows, k, ld, static_cast<uint32_t>(tile_rows));
}

// Output i of a call.
inline void epi_output(bm::EpiParams &f, int i, void *X, int64_t ld)
{
    f.out[i] = X;
    f.ldout[i] = ld;
}

// The outputs' maps, where rows of n 16-bit values end on 16 bytes. (GLU on 128 x 128 tiles stores
// its groups of 16 columns by lane and leaves them unused.)
inline void epi_output_maps(bm::EpiParams &f, EpiMaps &t, int64_t m, int64_t n)
{
    for (int i = 0; i < 3; ++i)
        f.tma[i] = f.out[i] != nullptr && n % 8 == 0 && encode_box64(&t.out[i], f.out[i], BM_BF16, m, n, f.ldout[i]) ? 1 : 0;
}

template <int KIND>
bm_status epi_launch(const Plan &pl, const EpiMaps &t, const bm::EpiParams &f, cudaStream_t stream)
{
    PdlLaunch l(stream, static_cast<unsigned>(pl.ctas), bm::FUSED_THREADS, static_cast<size_t>(epi_smem(pl.variant)),
                pl.pair == 2 ? 2 : 0);
    return launched(cudaLaunchKernelEx(&l.cfg, epi_kernel<KIND>(pl.variant), t.a, t.b, t.b2, t.out[0], t.out[1], t.out[2],
                                       t.in[0], t.in[1], f));
}

}  // namespace bmh
