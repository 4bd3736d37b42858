// bm_fused_kernel.cuh -- BF16 products with an MLP's work in the epilogue.
//
//   forward    z = alpha op(A) op(B) + bias,  C = act(z) + R,  and on request z
//              kept in 8 bits (MXFP8 codes Q, scales S: the rule of bm_quant_kernel.cuh)
//   backward   C = (alpha op(A) op(B)) . act'(z~), z~ what Q and S stand for, and on
//              request the column sums of C (before its rounding)
//
// The mainloop is that of bm_gemm_kernel.cuh: its producer, its schedule, its ring.
// Two things differ.
//
// Accumulation in chunks of K. The tensor core adds each K = 16 step to its FP32
// accumulator by truncation, so the error grows with K (measured 1.1e-9 K, relative:
// 9e-6 at K = 8192). When an output is FP32 (C, or the column sums) the MMA warp hands
// over the accumulator every chunk of K; the epilogue warps add the chunks in
// registers, rounding to nearest, while the next chunk fills the other accumulator.
// With a BF16 C alone (rounded at 2^-8) one chunk holds all of K.
//
// The epilogue takes its whole share of the accumulator into registers first (32 rows
// x BN / 2 columns per warp: up to 128 values per lane, lane = row) and gives tensor
// memory back before it computes: the activation of one tile overlaps the next tile's
// products. A lane then holds whole groups of 32 columns of its row, which is what an
// MXFP8 scale spans, so the 8-bit checkpoint needs no exchange between lanes. R, and in
// the backward pass Q, come in by TMA into the warp's 4 KB staging block ahead of the
// accumulator; C leaves through the same block.
#pragma once

#include "bm_act.cuh"
#include "bm_gemm_kernel.cuh"
#include "bm_quant_kernel.cuh"

namespace bm {

struct FusedParams {
    GemmParams g;  // schedule, sizes, C, alpha, split slots; beta unused
    const void *bias;  // [n] fp32 or bf16, or null
    int bias_bf16;
    int act;           // ACT_*
    const void *R;     // forward: residual of C's type, or null
    int64_t ldr;
    uint8_t *Q;        // MXFP8 codes and scales: written (forward, may be null) or read (backward)
    int64_t ldq;
    uint8_t *S;
    int64_t katoms;    // scale atoms along n: ceil(n / 128)
    int tma_r;         // tmR maps R (forward), box 128 bytes x 32 rows, 128B swizzle
    int tma_q;         // tmR maps Q (backward), the same box
    float *colsum;     // backward: partial column sums [ceil(m / row_block)][ld_colsum], or null
    int64_t ld_colsum;
    int row_block;     // rows per partial column sum: 32 (tile kernel) or the reduce kernel's rows
    int chunk_kb;      // k-blocks per accumulator chunk, a multiple of the stage's
};

constexpr int FUSED_EXTRA_BARS = NUM_EPI_WARPS;  // one load barrier per epilogue warp

template <int BN, int STAGES, int PAIR, int KPS>
struct FusedCfg : KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS> {
    using Base = KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS>;
    static constexpr int FUSED_BARS = 2 * STAGES + 5 + FUSED_EXTRA_BARS;
    static constexpr int FUSED_SMEM = 1024 + Base::RING_BYTES + Base::EPI_BYTES + 8 * FUSED_BARS + 16;
    static_assert(FUSED_SMEM <= 227 * 1024, "shared memory");
};

// ---------------------------------------------------------------- MMA issue
// run_mma of bm_gemm_kernel.cuh for bf16, with an accumulator per chunk of K.
template <int BN, int STAGES, int PAIR, int KPS>
__device__ __forceinline__ void run_mma_chunked(const FusedParams &f, uint32_t ring, uint32_t bar0, uint32_t tmem_base,
                                                volatile int *abort_flag, int lane)
{
    using Cfg = KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS>;
    const GemmParams &p = f.g;
    const uint64_t a_tpl = p.a_mn_major ? smem_desc_sw128(0u, Cfg::CHUNK_BYTES, 1024u) : smem_desc_sw128(0u, 16u, 1024u);
    const uint64_t b_tpl = p.b_mn_major ? smem_desc_sw128(0u, Cfg::CHUNK_BYTES, 1024u) : smem_desc_sw128(0u, 16u, 1024u);
    const uint32_t a_kk = p.a_mn_major ? 2048u / 16u : 32u / 16u;
    const uint32_t b_kk = p.b_mn_major ? 2048u / 16u : 32u / 16u;
    const uint32_t a_sub = p.a_mn_major ? 8192u / 16u : static_cast<uint32_t>(Cfg::A_BYTES) / 16u;
    const uint32_t b_sub = p.b_mn_major ? 8192u / 16u : static_cast<uint32_t>(Cfg::B_BYTES) / 16u;
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued_any = false;
    for (int64_t u = first_unit<PAIR>(); u < p.num_units && ok; u += unit_stride<PAIR>()) {
        const Unit w = map_unit<Cfg::TILE_M, BN, false>(p, u);
        const uint32_t idesc =
            idesc_f32acc(Cfg::TILE_M, w.nh < 0 ? BN : BN / 2, 1u, p.a_mn_major, p.b_mn_major);
        const uint32_t b_nh =
            w.nh > 0 ? (p.b_mn_major ? static_cast<uint32_t>(Cfg::CHUNK_BYTES) : 64u * 128u) / 16u : 0u;
        for (int c0 = w.kb0; c0 < w.kb1 && ok; c0 += f.chunk_kb) {
            const int c1 = min(w.kb1, c0 + f.chunk_kb);
            if (!wait_one<PAIR == 2>(bar0 + 8u * (2 * STAGES + 2 + acc), acc_phase ^ 1u, abort_flag, p.timeout_ns)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
            for (int kb = c0; kb < c1; kb += KPS) {
                if (!wait_one(bar0 + 8u * stage, phase, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const int nkb = c1 - kb < KPS ? c1 - kb : KPS;
                const uint32_t st = ring + stage * Cfg::STAGE_BYTES;
                for (int sub = 0; sub < nkb; ++sub) {
                    const uint64_t a0 = a_tpl + (st >> 4) + a_sub * sub;
                    const uint64_t b0 = b_tpl + ((st + Cfg::B_OFFSET) >> 4) + b_sub * sub + b_nh;
#pragma unroll
                    for (int kk = 0; kk < TILE_K / UMMA_K; ++kk) {
                        const uint32_t accumulate = (kb > c0 || sub > 0 || kk > 0) ? 1u : 0u;
                        if (lane == 0) {
                            if constexpr (PAIR == 1) umma_bf16(d_tmem, a0 + a_kk * kk, b0 + b_kk * kk, idesc, accumulate);
                            else umma_bf16_pair(d_tmem, a0 + a_kk * kk, b0 + b_kk * kk, idesc, accumulate);
                        }
                    }
                }
                issued_any = true;
                if (lane == 0) {
                    if constexpr (PAIR == 1) umma_commit(bar0 + 8u * (STAGES + stage));
                    else umma_commit_pair(bar0 + 8u * (STAGES + stage), 0x3);
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if (lane == 0) {
                if constexpr (PAIR == 1) umma_commit(bar0 + 8u * (2 * STAGES + acc));
                else umma_commit_pair(bar0 + 8u * (2 * STAGES + acc), 0x3);
            }
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    if (!ok) {
        signal_timeout(p, abort_flag);
        if (issued_any) {  // MMAs in flight must finish before TMEM is freed
            const uint32_t drain = bar0 + 8u * (2 * STAGES + 4);
            if (lane == 0) {
                if constexpr (PAIR == 1) umma_commit(drain);
                else umma_commit_pair(drain, 0x1);
            }
            wait_one(drain, 0u, nullptr, p.timeout_ns);
        }
    }
}

// ---------------------------------------------------------------- epilogue math
// bias[j .. j + 31] (zeros past n); j is a multiple of 32.
__device__ __forceinline__ void load_bias32(const FusedParams &f, int64_t j, float (&b)[32])
{
    if (j + 32 <= f.g.n) {
        if (f.bias_bf16) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(f.bias) + j);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 w = __ldg(src + q);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    b[8 * q + 2 * e] = __uint_as_float(u[e] << 16);
                    b[8 * q + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
                }
            }
        } else {
            const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(f.bias) + j);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 w = __ldg(src + q);
                b[4 * q] = w.x;
                b[4 * q + 1] = w.y;
                b[4 * q + 2] = w.z;
                b[4 * q + 3] = w.w;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            b[e] = 0.0f;
            if (j + e < f.g.n)
                b[e] = f.bias_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(f.bias)[j + e])
                                                     << 16)
                                   : static_cast<const float *>(f.bias)[j + e];
        }
    }
}

// MXFP8 codes of a group of 32 values (zeros past the row's end): returns the scale code.
__device__ __forceinline__ uint32_t mx_group_codes(const float (&z)[32], uint32_t (&codes)[8])
{
    float amax = 0.0f;
    bool special = false;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        const float a = fabsf(z[e]);
        special |= !(a <= 3.402823466e38f);
        amax = fmaxf(amax, a);
    }
    if (special) {
#pragma unroll
        for (int q = 0; q < 8; ++q) codes[q] = 0x7F7F7F7Fu;
        return 255u;
    }
    const uint32_t code = ue8m0_code(amax);
    const float inv = __uint_as_float((254u - code) << 23);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        codes[q] = e4m3x4(z[4 * q] * inv, z[4 * q + 1] * inv, z[4 * q + 2] * inv, z[4 * q + 3] * inv);
    return code;
}

// Column sums of a warp's 32 rows x 32 columns (lane = row): lane j gets column j's.
// Each step halves the columns a lane carries and adds the other half's from the lane
// 2^s away, so the order of the sum is fixed.
__device__ __forceinline__ float column_sum32(const float (&v)[32], int lane)
{
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const bool up = lane & 16;
        const float keep = up ? v[16 + i] : v[i];
        const float send = up ? v[i] : v[16 + i];
        t[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? t[w + i] : t[i];
            const float send = up ? t[i] : t[w + i];
            t[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
    }
    return t[0];
}

// ---------------------------------------------------------------- epilogue
template <int BN, int STAGES, int PAIR, int KPS, bool BWD>
__device__ __forceinline__ void run_epilogue_fused(const CUtensorMap *tmC, const CUtensorMap *tmP,
                                                   const CUtensorMap *tmR, const FusedParams &f, uint32_t bar0,
                                                   uint32_t tmem_base, float *epi, uint32_t rank,
                                                   volatile int *abort_flag, int warp, int lane)
{
    using Cfg = KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS>;
    constexpr int HC = BN / 2;  // accumulator columns of one warp of a whole tile
    const GemmParams &p = f.g;
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    float *stage_buf = epi + (warp - 2) * EPI_WARP_FLOATS;
    const uint32_t stage_addr = smem_addr(stage_buf);
    uint4 *srow = reinterpret_cast<uint4 *>(stage_buf) + lane * 8;  // this lane's row of the staging block
    const uint32_t lbar = bar0 + 8u * (2 * STAGES + 5 + (warp - 2));
    uint32_t lphase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true, loading = false;
    for (int64_t u = first_unit<PAIR>(); u < p.num_units && ok; u += unit_stride<PAIR>()) {
        const Unit w = map_unit<Cfg::TILE_M, BN, false>(p, u);
        const bool to_slot = w.slot >= 0;
        const bool halved = PAIR == 2 && BN == 256 && w.nh >= 0;
        const int ncol = halved ? BN / 4 : HC;  // columns of this warp in this unit
        const int64_t row0 = w.tm * Cfg::TILE_M + rank * CTA_M + quad * 32;
        const int64_t xcol = halved ? w.tn * BN + half * (BN / 2) + w.nh * (BN / 4) : w.tn * BN + half * HC;
        const bool live = row0 < p.m && xcol < p.n;  // anything of this warp's block inside C
        // First load into the staging block: the first columns of R, or the codes of Q.
        const bool pre = live && !to_slot && (BWD ? f.tma_q != 0 : f.tma_r != 0);
        if (pre) {
            if (lane == 0) {
                bulk_wait_group_read0();  // the last unit's stores have read the block
                mbar_arrive_expect_tx(lbar, EPI_WARP_FLOATS * 4);
                tma_load_2d(stage_addr, tmR, lbar, static_cast<int32_t>(xcol), static_cast<int32_t>(row0));
            }
            loading = true;
        }
        float v[HC];
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * ncol);
        for (int c0 = w.kb0; c0 < w.kb1; c0 += f.chunk_kb) {
            if (!wait_warp<PAIR == 2>(bar0 + 8u * (2 * STAGES + acc), acc_phase, abort_flag, p.timeout_ns)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t taddr = lane_base + static_cast<uint32_t>(acc * BN);
#pragma unroll
            for (int g = 0; g < HC / 32; ++g) {
                if (g * 32 >= ncol) continue;
                uint32_t r[32];
                tmem_load_32cols(taddr + 32u * g, r);
                if (c0 == w.kb0) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[32 * g + e] = __uint_as_float(r[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[32 * g + e] += __uint_as_float(r[e]);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                const uint32_t acc_empty = bar0 + 8u * (2 * STAGES + 2 + acc);
                if constexpr (PAIR == 1) mbar_arrive(acc_empty);
                else mbar_arrive_remote(map_shared_to_rank(acc_empty, 0));
            }
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (!ok) break;

        if (to_slot) {  // fp32 partial of a split tile, 32 x 32 blocks
            const int64_t slot_row = w.slot * Cfg::TILE_M + rank * CTA_M + quad * 32;
#pragma unroll
            for (int g = 0; g < HC / 32; ++g) {
                if (g * 32 >= ncol) continue;
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    srow[j ^ (lane & 7)] =
                        make_uint4(__float_as_uint(v[32 * g + 4 * j]), __float_as_uint(v[32 * g + 4 * j + 1]),
                                   __float_as_uint(v[32 * g + 4 * j + 2]), __float_as_uint(v[32 * g + 4 * j + 3]));
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(tmP, stage_addr, half * HC + 32 * g, static_cast<int32_t>(slot_row));
                    bulk_commit_group();
                }
            }
            continue;
        }

        const int64_t row = row0 + lane;
        const bool row_in = row < p.m;
        const int64_t s_at = ((row >> 7) * f.katoms + (xcol >> 7)) * SF_ATOM_BYTES + (row & 31) * 16 + ((row & 127) >> 5) * 4;
        if constexpr (BWD) {
            // ---- C = alpha v . act'(z~)
            uint32_t scales = 0;  // codes of this row's groups, lowest byte first
            if (row_in && xcol < p.n) {
                if (ncol == 128) scales = *reinterpret_cast<const uint32_t *>(f.S + s_at);
                else scales = *reinterpret_cast<const uint16_t *>(f.S + s_at + ((xcol >> 5) & 3));
            }
            if (pre) {
                if (!wait_warp<false>(lbar, lphase, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                lphase ^= 1u;
                loading = false;
            }
#pragma unroll
            for (int g = 0; g < HC / 32; ++g) {
                if (g * 32 >= ncol) continue;
                const int64_t j0 = xcol + 32 * g;
                float (&vg)[32] = *reinterpret_cast<float (*)[32]>(&v[32 * g]);
                uint32_t codes[8];
                if (pre) {
                    const uint4 c0 = srow[(2 * g) ^ (lane & 7)], c1 = srow[(2 * g + 1) ^ (lane & 7)];
                    codes[0] = c0.x, codes[1] = c0.y, codes[2] = c0.z, codes[3] = c0.w;
                    codes[4] = c1.x, codes[5] = c1.y, codes[6] = c1.z, codes[7] = c1.w;
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) codes[q] = 0u;
                }
                const float scale = ue8m0_value((scales >> (8 * g)) & 0xFFu);
                // rows past m and columns past n: their accumulators may hold NaN (a zero
                // row of A times an infinity of B), which must not reach the sums
                const bool edge = !row_in || j0 + 32 > p.n;
                with_act(f.act, [&](auto tag) {
                    constexpr int ACT = decltype(tag)::value;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float d[4];
                        e4m3x4_values(codes[q], d);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            vg[4 * q + e] = (p.alpha * vg[4 * q + e]) * act_slope<ACT>(d[e] * scale);
                    }
                });
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!row_in || j0 + e >= p.n) vg[e] = 0.0f;
                }
                if (f.colsum != nullptr && row0 < p.m) {
                    const float sum = column_sum32(vg, lane);
                    if (j0 + lane < p.n) f.colsum[(row0 >> 5) * f.ld_colsum + j0 + lane] = sum;
                }
            }
            __syncwarp();  // every lane has read its codes: the block is free
        } else {
            // ---- z = alpha v + bias, the checkpoint of z, act(z)
            uint32_t scales = 0;
#pragma unroll
            for (int g = 0; g < HC / 32; ++g) {
                if (g * 32 >= ncol) continue;
                const int64_t j0 = xcol + 32 * g;
                float (&vg)[32] = *reinterpret_cast<float (*)[32]>(&v[32 * g]);
                if (f.bias != nullptr) {
                    float b[32];
                    load_bias32(f, j0, b);
#pragma unroll
                    for (int e = 0; e < 32; ++e) vg[e] = fmaf(p.alpha, vg[e], b[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) vg[e] *= p.alpha;
                }
                if (f.Q != nullptr && row_in && j0 < p.n) {
                    uint32_t codes[8];
                    if (j0 + 32 > p.n) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (j0 + e >= p.n) vg[e] = 0.0f;
                    }
                    scales |= mx_group_codes(vg, codes) << (8 * g);
                    uint8_t *dst = f.Q + row * f.ldq + j0;
                    if (j0 + 32 <= p.n) {
                        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (j0 + e < p.n) dst[e] = static_cast<uint8_t>(codes[e >> 2] >> (8 * (e & 3)));
                    }
                }
                with_act(f.act, [&](auto tag) {
                    constexpr int ACT = decltype(tag)::value;
#pragma unroll
                    for (int e = 0; e < 32; ++e) vg[e] = act_value<ACT>(vg[e]);
                });
            }
            // scale codes of this row's groups, padding rows and groups of the array as zeros
            if (f.Q != nullptr && (row0 & ~int64_t(127)) < p.m && (xcol & ~int64_t(127)) < p.n) {
                if (ncol == 128) *reinterpret_cast<uint32_t *>(f.S + s_at) = scales;
                else *reinterpret_cast<uint16_t *>(f.S + s_at + ((xcol >> 5) & 3)) = static_cast<uint16_t>(scales);
            }
        }
        if (!live) continue;

        // ---- C, in blocks of 128 bytes per row (64 bf16 or 32 fp32 columns) by TMA, or
        // (rows of C that do not end on a 16-byte boundary) in 32 x 32 blocks with masked stores
        const bool has_r = !BWD && f.R != nullptr;
        if (p.tma_c && (!has_r || f.tma_r)) {
            const bool bf16_out = p.c_bf16 != 0;
            const int cw = bf16_out ? 64 : 32;
#pragma unroll
            for (int b = 0; b < HC / 32; ++b) {
                const int c = b * cw;
                if (c >= ncol || c >= HC) continue;
                const int64_t x = xcol + c;
                if (x >= p.n) continue;
                if (has_r) {
                    if (b > 0 && lane == 0) {
                        bulk_wait_group_read0();
                        mbar_arrive_expect_tx(lbar, EPI_WARP_FLOATS * 4);
                        tma_load_2d(stage_addr, tmR, lbar, static_cast<int32_t>(x), static_cast<int32_t>(row0));
                    }
                    loading = true;
                    if (!wait_warp<false>(lbar, lphase, abort_flag, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    lphase ^= 1u;
                    loading = false;
                } else {
                    if (lane == 0) bulk_wait_group_read0();
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 *slot = srow + (j ^ (lane & 7));
                    uint4 q;
                    if (bf16_out) {
                        float t[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) t[e] = (64 * b + 8 * j + e < HC) ? v[(64 * b + 8 * j + e) % HC] : 0.0f;
                        if (has_r) {
                            const uint4 old = *slot;
                            const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                t[2 * e] += __uint_as_float(o[e] << 16);
                                t[2 * e + 1] += __uint_as_float(o[e] & 0xFFFF0000u);
                            }
                        }
                        __nv_bfloat162 h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(t[2 * e], t[2 * e + 1]);
                        q = *reinterpret_cast<const uint4 *>(h);
                    } else {
                        float t[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[e] = v[32 * b + 4 * j + e];
                        if (has_r) {
                            const uint4 old = *slot;
                            t[0] += __uint_as_float(old.x);
                            t[1] += __uint_as_float(old.y);
                            t[2] += __uint_as_float(old.z);
                            t[3] += __uint_as_float(old.w);
                        }
                        q = make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]),
                                       __float_as_uint(t[3]));
                    }
                    *slot = q;
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(tmC, stage_addr, static_cast<int32_t>(x), static_cast<int32_t>(row0));
                    bulk_commit_group();
                }
            }
            if (!ok) break;
        } else {
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
#pragma unroll
            for (int g = 0; g < HC / 32; ++g) {
                if (g * 32 >= ncol) continue;
                // Row `lane` into shared memory (16-byte unit c of row r at slot c ^ (r & 7)),
                // then 8 lanes per 32-column row segment, 4 rows per step.
                float4 *frow = reinterpret_cast<float4 *>(srow);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    frow[c ^ (lane & 7)] =
                        make_float4(v[32 * g + 4 * c], v[32 * g + 4 * c + 1], v[32 * g + 4 * c + 2], v[32 * g + 4 * c + 3]);
                __syncwarp();
                const int cc = lane & 7;
                const int64_t j = xcol + 32 * g + cc * 4;
#pragma unroll 1
                for (int step = 0; step < 8; ++step) {
                    const int rr = step * 4 + (lane >> 3);
                    const int64_t i = row0 + rr;
                    const float4 v4 = reinterpret_cast<const float4 *>(stage_buf + rr * 32)[cc ^ (rr & 7)];
                    float t[4] = {v4.x, v4.y, v4.z, v4.w};
                    if (i >= p.m) continue;
                    if (p.c_bf16) {
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.C) + i * p.ldc;
                        const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(f.R) + i * f.ldr;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j + e < p.n) dst[j + e] = __float2bfloat16_rn(has_r ? t[e] + __bfloat162float(res[j + e]) : t[e]);
                    } else {
                        float *dst = static_cast<float *>(p.C) + i * p.ldc;
                        const float *res = static_cast<const float *>(f.R) + i * f.ldr;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j + e < p.n) dst[j + e] = has_r ? t[e] + res[j + e] : t[e];
                    }
                }
                __syncwarp();
            }
        }
    }
    if (!ok && lane == 0) signal_timeout(p, abort_flag);
    if (!ok && loading) spin_ns(100000);  // a copy may still land in the block
    if (lane == 0) bulk_wait_group0();    // shared memory must outlive the stores that read it
}

// ---------------------------------------------------------------- kernels
template <int BN, int STAGES, int PAIR, int KPS, bool BWD>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    bm_gemm_fused_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmP,
                         const __grid_constant__ CUtensorMap tmR, const FusedParams f)
{
    using Cfg = FusedCfg<BN, STAGES, PAIR, KPS>;
    const GemmParams &p = f.g;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    uint8_t *smem = smem_raw + pad;
    const uint32_t ring = raw + pad;
    float *epi = reinterpret_cast<float *>(smem + Cfg::RING_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::RING_BYTES + Cfg::EPI_BYTES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Cfg::FUSED_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t bar0 = smem_addr(bars);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR == 2 ? cluster_cta_rank() : 0u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar0 + 8u * s, 1);             // full: CTA 0's expect_tx arrival (+ bytes)
            mbar_init(bar0 + 8u * (STAGES + s), 1);  // empty: one tcgen05.commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar0 + 8u * (2 * STAGES + b), 1);                         // accumulator full
            mbar_init(bar0 + 8u * (2 * STAGES + 2 + b), NUM_EPI_WARPS * PAIR);  // accumulator empty
        }
        mbar_init(bar0 + 8u * (2 * STAGES + 4), 1);  // drain (abort path only)
        for (int e = 0; e < FUSED_EXTRA_BARS; ++e) mbar_init(bar0 + 8u * (2 * STAGES + 5 + e), 1);  // R or Q load
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        if (p.tma_c) tma_prefetch_map(&tmC);
        if (f.tma_r || f.tma_q) tma_prefetch_map(&tmR);
    }
    if (warp == 1) {
        if constexpr (PAIR == 1) {
            tmem_alloc(smem_addr(tmem_slot), Cfg::TMEM_COLS);
            tmem_relinquish();
        } else {
            tmem_alloc_pair(smem_addr(tmem_slot), Cfg::TMEM_COLS);
            tmem_relinquish_pair();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR == 2) cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    // as in bm_gemm_tcgen05_kernel: nothing in global memory is read into the SM or
    // written before the previous kernel on the stream is complete
    griddep_launch_dependents();
    if (warp == 0 && lane == 0 && p.a_box3 && p.b_box3)
        prefetch_first_stages<BN, STAGES, PAIR, ELEM_BF16, KPS, EPI_STORE>(&tmA, &tmB, p, rank);
    griddep_wait();

    if (warp == 0) {
        if (lane == 0)
            run_producer<BN, STAGES, PAIR, ELEM_BF16, KPS, EPI_STORE>(&tmA, &tmB, &tmA, &tmB, p, ring, bar0, rank,
                                                                      abort_flag);
    } else if (warp == 1) {
        if (rank == 0) run_mma_chunked<BN, STAGES, PAIR, KPS>(f, ring, bar0, tmem_base, abort_flag, lane);
    } else {
        run_epilogue_fused<BN, STAGES, PAIR, KPS, BWD>(&tmC, &tmP, &tmR, f, bar0, tmem_base, epi, rank, abort_flag,
                                                       warp, lane);
    }

    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR == 2) cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        if constexpr (PAIR == 1) tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
        else tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

// The epilogue's work from fp32 partial slots (every tile split along K), or from
// nothing (alpha == 0 or k == 0: k_splits == 0). One warp takes row_block rows x 128
// columns, four columns per lane, so that 8 lanes hold one MXFP8 group of a row and a
// lane can sum its columns over the rows.
template <int TM, int BN, bool BWD>
__global__ void __launch_bounds__(256) bm_fused_reduce_kernel(const FusedParams f)
{
    griddep_launch_dependents();
    griddep_wait();
    const GemmParams &p = f.g;
    const int lane = threadIdx.x & 31;
    const int64_t col_blocks = (p.n + 127) / 128;
    // rows up to the end of the last 128-row scale atom when a checkpoint is written
    // (its padding entries are zeros)
    const int64_t rows = !BWD && f.Q != nullptr ? (p.m + 127) / 128 * 128 : p.m;
    const int64_t items = (rows + f.row_block - 1) / f.row_block * col_blocks;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    const int64_t slot_elems = static_cast<int64_t>(TM) * BN;
    for (int64_t it = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += warps) {
        const int64_t rb = it / col_blocks;
        const int64_t j = (it - rb * col_blocks) * 128 + lane * 4;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (!BWD && f.bias != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < p.n)
                    b[e] = f.bias_bf16
                               ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(f.bias)[j + e]) << 16)
                               : static_cast<const float *>(f.bias)[j + e];
        }
#pragma unroll 1
        for (int rr = 0; rr < f.row_block; ++rr) {
            const int64_t i = rb * f.row_block + rr;
            if (i >= rows) break;
            const bool in = i < p.m && j < p.n;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (in && p.k_splits > 0) {
                const int64_t tm = i / TM, tn = j / BN;
                // (tiles are visited in grouped-raster order; its inverse gives the slot)
                const int64_t first = tm / p.group_m * p.group_m;
                const int64_t group_rows = p.tiles_m - first < p.group_m ? p.tiles_m - first : p.group_m;
                const int64_t t = first * p.tiles_n + tn * group_rows + (tm - first);
                const float *src = p.partial + t * p.k_splits * slot_elems + (i - tm * TM) * BN + (j - tn * BN);
                float4 s = __ldcg(reinterpret_cast<const float4 *>(src));
                int sp = 1;
                for (; sp + 4 <= p.k_splits; sp += 4) {
                    float4 t4[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) t4[q] = __ldcg(reinterpret_cast<const float4 *>(src + (sp + q) * slot_elems));
#pragma unroll
                    for (int q = 0; q < 4; ++q) s.x += t4[q].x, s.y += t4[q].y, s.z += t4[q].z, s.w += t4[q].w;
                }
                for (; sp < p.k_splits; ++sp) {
                    const float4 t4 = __ldcg(reinterpret_cast<const float4 *>(src + sp * slot_elems));
                    s.x += t4.x, s.y += t4.y, s.z += t4.z, s.w += t4.w;
                }
                v[0] = p.alpha * s.x, v[1] = p.alpha * s.y, v[2] = p.alpha * s.z, v[3] = p.alpha * s.w;
            }
            const int64_t s_at = ((i >> 7) * f.katoms + (j >> 7)) * SF_ATOM_BYTES + (i & 31) * 16 + ((i & 127) >> 5) * 4 +
                                 ((j >> 5) & 3);
            if constexpr (BWD) {
                if (in) {
                    const float scale = ue8m0_value(f.S[s_at]);
                    uint32_t codes = 0;
                    const uint8_t *q = f.Q + i * f.ldq + j;
                    if (j + 4 <= p.n) codes = *reinterpret_cast<const uint32_t *>(q);
                    else
                        for (int e = 0; e < 4; ++e)
                            if (j + e < p.n) codes |= static_cast<uint32_t>(q[e]) << (8 * e);
                    float d[4];
                    e4m3x4_values(codes, d);
                    with_act(f.act, [&](auto tag) {
                        constexpr int ACT = decltype(tag)::value;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] *= act_slope<ACT>(d[e] * scale);
                    });
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < p.n) sum[e] += v[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = j + e < p.n ? v[e] + b[e] : 0.0f;
                if (f.Q != nullptr) {
                    // the group's largest magnitude over its 8 lanes; NaN and infinities as one flag
                    float amax = 0.0f;
                    bool special = false;
                    if (in) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = fabsf(v[e]);
                            special |= !(a <= 3.402823466e38f);
                            amax = fmaxf(amax, a);
                        }
                    }
                    if (special) amax = __uint_as_float(0x7F800000u);
#pragma unroll
                    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    special = amax > 3.402823466e38f;
                    const uint32_t code = special ? 255u : ue8m0_code(amax);
                    if ((lane & 7) == 0) f.S[s_at] = static_cast<uint8_t>(in ? code : 0u);
                    if (in) {
                        const float inv = __uint_as_float((254u - (special ? 0u : code)) << 23);
                        const uint32_t codes = special ? 0x7F7F7F7Fu : e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                        uint8_t *dst = f.Q + i * f.ldq + j;
                        if (j + 4 <= p.n) *reinterpret_cast<uint32_t *>(dst) = codes;
                        else
                            for (int e = 0; e < 4; ++e)
                                if (j + e < p.n) dst[e] = static_cast<uint8_t>(codes >> (8 * e));
                    }
                }
                with_act(f.act, [&](auto tag) {
                    constexpr int ACT = decltype(tag)::value;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = act_value<ACT>(v[e]);
                });
            }
            if (!in) continue;
            const bool has_r = !BWD && f.R != nullptr;
            if (p.c_bf16) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.C) + i * p.ldc + j;
                const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(f.R) + i * f.ldr + j;
                if (j + 4 <= p.n) {
                    if (has_r) {
                        const uint2 o = *reinterpret_cast<const uint2 *>(res);
                        v[0] += __uint_as_float(o.x << 16), v[1] += __uint_as_float(o.x & 0xFFFF0000u);
                        v[2] += __uint_as_float(o.y << 16), v[3] += __uint_as_float(o.y & 0xFFFF0000u);
                    }
                    const __nv_bfloat162 h0 = __floats2bfloat162_rn(v[0], v[1]), h1 = __floats2bfloat162_rn(v[2], v[3]);
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&h0),
                                                                 *reinterpret_cast<const uint32_t *>(&h1));
                } else {
                    for (int e = 0; e < 4; ++e)
                        if (j + e < p.n) dst[e] = __float2bfloat16_rn(has_r ? v[e] + __bfloat162float(res[e]) : v[e]);
                }
            } else {
                float *dst = static_cast<float *>(p.C) + i * p.ldc + j;
                const float *res = static_cast<const float *>(f.R) + i * f.ldr + j;
                if (j + 4 <= p.n) {
                    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (has_r) o = *reinterpret_cast<const float4 *>(res);
                    *reinterpret_cast<float4 *>(dst) =
                        has_r ? make_float4(v[0] + o.x, v[1] + o.y, v[2] + o.z, v[3] + o.w) : make_float4(v[0], v[1], v[2], v[3]);
                } else {
                    for (int e = 0; e < 4; ++e)
                        if (j + e < p.n) dst[e] = has_r ? v[e] + res[e] : v[e];
                }
            }
        }
        if (BWD && f.colsum != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < p.n) f.colsum[rb * f.ld_colsum + j + e] = sum[e];
        }
    }
}

}  // namespace bm
