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
// With a BF16 C alone (rounded at 2^-8) one chunk holds all of K. The two accumulators
// let the MMAs run two chunks ahead of a tile's epilogue, so a tile's first two chunks
// are the long ones (16 and 16 k-blocks of 64, then 8 each, at K = 4096; 12 and 12 beside a
// checkpoint).
//
// An epilogue warp takes 32 rows x BN / 4 columns (lane = row) in groups of 32 columns:
// with one chunk straight from tensor memory, with several from the sums in its registers,
// and tensor memory is given back before the arithmetic of the (last) group: it overlaps
// the next tile's products. A lane holds whole groups of 32 columns of its row, which is
// what an MXFP8 scale spans, so the 8-bit checkpoint needs no exchange between lanes. C and
// the codes leave through a 2 KB staging block per warp, which turns rows per lane into
// 64-byte pieces of rows; Q comes in the same way ahead of the accumulator, and R by TMA,
// a piece ahead. C goes from the block by TMA where its rows end on a 16-byte boundary
// (4096 x 16384 x 4096 without an activation: 333 us with loads from the block and plain
// stores, 315 by TMA).
//
// Sixteen epilogue warps: the arithmetic of 128 x 256 elements per SM and tile has to fit
// into the time of two chunks of 16 k-blocks (11 us), and it is bound by instruction issue
// and latency. With eight warps of 128 columns each, the backward epilogue took 29 us per
// tile at 26 % of the issue slots, spilling (4096 x 8192 x 2048, GELU, column sums: 200 us).
//
// Bound by the tensor cores, and on long runs by the power limit. 4096 x 16384 x 4096 in
// such a run, BF16 C: the product alone 310 us (1770 TFLOP/s); with bias and GELU 342, a
// residual 341, a GELU checkpoint 393; backward through GELU 342, with column sums 383 to
// 404; FP32 C 352. What the checkpoint, the column sums and FP32 pay for is the chunks: six
// or seven passes over the accumulators of a tile (in one piece the checkpoint's call takes
// 350 us and the column sums' 352).
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
    float *colsum;     // backward: partial column sums [ceil(m / row_block)][ld_colsum], or null
    int64_t ld_colsum;
    int row_block;     // rows per partial column sum: 32 (tile kernel) or the reduce kernel's rows
    // k-blocks per accumulator chunk (multiples of the stage's): of a unit's first two
    // chunks, which fill while the last tile's epilogue still runs, and of the others
    int chunk_first, chunk_rest;
};

constexpr int FUSED_EPI_WARPS = 16;
// Warps 0 and 1 are the producer and the MMA issuer, 2 and 3 idle: register counts are set
// per group of four warps. Where the epilogue keeps running sums, the launch's 640 x 96
// registers are shared out as 128 x 32 and 512 x 112 (fused_attrs checks that the
// compiler's count is the 96 that this adds up to).
constexpr int FUSED_FIRST_EPI_WARP = 4;
constexpr int FUSED_THREADS = 32 * (FUSED_FIRST_EPI_WARP + FUSED_EPI_WARPS);
constexpr int FUSED_LAUNCH_REGS = 96, FUSED_MAIN_REGS = 32, FUSED_EPI_REGS = 112;
static_assert(128 * FUSED_MAIN_REGS + 32 * FUSED_EPI_WARPS * FUSED_EPI_REGS <= FUSED_THREADS * FUSED_LAUNCH_REGS,
              "register split");
constexpr int FUSED_STAGE_BYTES = 32 * 64;  // one epilogue warp's staging block: 32 rows x 64 bytes

template <int BN, int STAGES, int PAIR, int KPS>
struct FusedCfg : KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS> {
    using Base = KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS>;
    static constexpr int FUSED_BARS = 2 * STAGES + 5 + FUSED_EPI_WARPS;  // one residual barrier per epilogue warp
    static constexpr int STAGING_BYTES = FUSED_EPI_WARPS * FUSED_STAGE_BYTES;
    static constexpr int FUSED_SMEM = 1024 + Base::RING_BYTES + STAGING_BYTES + 8 * FUSED_BARS + 16;
    static_assert(FUSED_SMEM <= 227 * 1024, "shared memory");
};

// ---------------------------------------------------------------- tensor memory
// 16 consecutive 32-bit columns of a lane.
__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

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
        int c1 = w.kb0;
        for (int c0 = w.kb0, i = 0; c0 < w.kb1 && ok; c0 = c1, ++i) {
            c1 = min(w.kb1, c0 + (i < 2 ? f.chunk_first : f.chunk_rest));
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
// z = alpha z + bias on columns j .. j + 31 of a row (bias taken as 0 past n); j is a
// multiple of 32. The bias loads are the same for all lanes. (Ordinary loads, not those of
// the read-only path: the kernel before this one may still be writing the bias when this
// one starts.)
__device__ __forceinline__ void scale_bias32(const FusedParams &f, int64_t j, float *z)
{
    const float2 alpha = both(f.g.alpha);
    if (f.bias == nullptr || j >= f.g.n) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float2 y = mul2(make_float2(z[e], z[e + 1]), alpha);
            z[e] = y.x;
            z[e + 1] = y.y;
        }
    } else if (j + 32 > f.g.n) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            float b = 0.0f;
            if (j + e < f.g.n)
                b = f.bias_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(f.bias)[j + e]) << 16)
                                : static_cast<const float *>(f.bias)[j + e];
            z[e] = fmaf(f.g.alpha, z[e], b);
        }
    } else if (f.bias_bf16) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(f.bias) + j);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 w = src[q];
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 8 * q + 2 * e;
                const float2 y = fma2(make_float2(z[i], z[i + 1]), alpha,
                                      make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u)));
                z[i] = y.x;
                z[i + 1] = y.y;
            }
        }
    } else {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(f.bias) + j);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float4 w = src[q];
            const float2 y0 = fma2(make_float2(z[4 * q], z[4 * q + 1]), alpha, make_float2(w.x, w.y));
            const float2 y1 = fma2(make_float2(z[4 * q + 2], z[4 * q + 3]), alpha, make_float2(w.z, w.w));
            z[4 * q] = y0.x, z[4 * q + 1] = y0.y;
            z[4 * q + 2] = y1.x, z[4 * q + 3] = y1.y;
        }
    }
}

// MXFP8 codes of a group of 32 values (zeros past the row's end); returns the scale code.
__device__ __forceinline__ uint32_t mx_group(const float *z, uint4 (&codes)[2])
{
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e) amax = max_nan(amax, fabsf(z[e]));
    const bool special = !(amax <= 3.402823466e38f);  // a NaN or an infinity in the group
    const uint32_t code = special ? 0u : ue8m0_code(amax);
    const float2 inv = both(__uint_as_float((254u - code) << 23));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = 16 * h + 4 * q;
            const float2 a = mul2(make_float2(z[i], z[i + 1]), inv), b = mul2(make_float2(z[i + 2], z[i + 3]), inv);
            c[q] = special ? 0x7F7F7F7Fu : e4m3x4(a.x, a.y, b.x, b.y);
        }
        codes[h] = make_uint4(c[0], c[1], c[2], c[3]);
    }
    return special ? 255u : code;
}

// The first `left` of 32 codes to dst (16-byte aligned).
__device__ __forceinline__ void store_codes(uint8_t *dst, const uint4 (&codes)[2], int64_t left)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (left >= 16 * (h + 1)) {
            reinterpret_cast<uint4 *>(dst)[h] = codes[h];
        } else {
            const uint32_t c[4] = {codes[h].x, codes[h].y, codes[h].z, codes[h].w};
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (16 * h + e < left) dst[16 * h + e] = static_cast<uint8_t>(c[e >> 2] >> (8 * (e & 3)));
        }
    }
}

// R[i][j .. j + 3] (zeros past the row's end); j is a multiple of 4.
__device__ __forceinline__ float4 load_res4(const FusedParams &f, int64_t i, int64_t j)
{
    const bool full = j + 4 <= f.g.n;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (f.g.c_bf16) {
        const uint16_t *src = static_cast<const uint16_t *>(f.R) + i * f.ldr + j;
        if (full) {
            const uint2 o = *reinterpret_cast<const uint2 *>(src);
            v[0] = __uint_as_float(o.x << 16), v[1] = __uint_as_float(o.x & 0xFFFF0000u);
            v[2] = __uint_as_float(o.y << 16), v[3] = __uint_as_float(o.y & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (j + e < f.g.n) v[e] = __uint_as_float(static_cast<uint32_t>(src[e]) << 16);
        }
    } else {
        const float *src = static_cast<const float *>(f.R) + i * f.ldr + j;
        if (full) return *reinterpret_cast<const float4 *>(src);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (j + e < f.g.n) v[e] = src[e];
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// C[i][j .. j + 3] = t, rounded; masked at the row's end.
__device__ __forceinline__ void store_row4(const FusedParams &f, int64_t i, int64_t j, float4 t)
{
    const GemmParams &p = f.g;
    const bool full = j + 4 <= p.n;
    const float v[3] = {t.x, t.y, t.z};
    if (p.c_bf16) {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.C) + i * p.ldc + j;
        if (full) {
            const __nv_bfloat162 h0 = __floats2bfloat162_rn(t.x, t.y), h1 = __floats2bfloat162_rn(t.z, t.w);
            *reinterpret_cast<uint2 *>(dst) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (j + e < p.n) dst[e] = __float2bfloat16_rn(v[e]);
        }
    } else {
        float *dst = static_cast<float *>(p.C) + i * p.ldc + j;
        if (full) {
            *reinterpret_cast<float4 *>(dst) = t;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (j + e < p.n) dst[e] = v[e];
        }
    }
}

// Column sums of a warp's 32 rows x 32 columns (lane = row): lane j gets column j's.
// Each step halves the columns a lane carries and adds the other half's from the lane
// 2^s away, so the order of the sum is fixed.
__device__ __forceinline__ float column_sum32(const float *v, int lane)
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
// A warp's staging block: 32 rows x 64 bytes, 16-byte unit u of row r at slot
// u ^ ((r / 2) & 3), so that both a lane per row and four lanes per row meet no bank
// conflicts. Values go in by row (the accumulator's layout) and out in 64-byte pieces of
// eight rows at a time.
__device__ __forceinline__ uint4 *block_at(uint8_t *block, int row, int unit)
{
    return reinterpret_cast<uint4 *>(block) + row * 4 + (unit ^ ((row >> 1) & 3));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 64 bytes per row from column byte x0 on: rows row0 .. row0 + 31 of a byte matrix whose
// rows hold `width` bytes, copied towards the block (bytes past a row's end and rows past
// `rows` are left as they are). Pointers, pitches and x0 are multiples of 16.
__device__ __forceinline__ void start_block_copy(uint8_t *block, const uint8_t *src, int64_t pitch, int64_t row0,
                                                 int64_t rows, int64_t x0, int64_t width, int lane)
{
    const int64_t x = x0 + (lane & 3) * 16;
#pragma unroll
    for (int step = 0; step < 4; ++step) {
        const int r = step * 8 + (lane >> 2);
        if (row0 + r >= rows || x >= width) continue;
        const uint8_t *at = src + (row0 + r) * pitch + x;
        if (x + 16 <= width) {
            cp_async16(smem_addr(block_at(block, r, lane & 3)), at);
        } else {  // (the bytes past the last column may lie outside the matrix)
            uint8_t *dst = reinterpret_cast<uint8_t *>(block_at(block, r, lane & 3));
            for (int e = 0; x + e < width; ++e) dst[e] = at[e];
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// The block's first UNITS units of every row out, the same way.
template <int UNITS = 4>
__device__ __forceinline__ void store_block(uint8_t *block, uint8_t *dst, int64_t pitch, int64_t row0, int64_t rows,
                                            int64_t x0, int64_t width, int lane)
{
    constexpr int ROWS = 32 / UNITS;  // per step
    const int unit = lane % UNITS;
    const int64_t x = x0 + unit * 16;
#pragma unroll
    for (int step = 0; step < UNITS; ++step) {
        const int r = step * ROWS + lane / UNITS;
        const uint4 q = *block_at(block, r, unit);
        if (row0 + r >= rows || x >= width) continue;
        uint8_t *at = dst + (row0 + r) * pitch + x;
        if (x + 16 <= width) {
            *reinterpret_cast<uint4 *>(at) = q;
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 15; ++e)
                if (x + e < width) at[e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
        }
    }
}

// The block has been read by the last TMA store from it; and a TMA store of the block to C
// at column j, row i (the map clips both), once every lane has written its row.
__device__ __forceinline__ void free_block(int lane)
{
    if (lane == 0) bulk_wait_group_read0();
    __syncwarp();
}

__device__ __forceinline__ void send_block(const CUtensorMap *tmC, uint8_t *block, int64_t j, int64_t i, int lane)
{
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(tmC, smem_addr(block), static_cast<int32_t>(j), static_cast<int32_t>(i));
        bulk_commit_group();
    }
}

// The next piece of R (64 bytes per row from column j on) into the block, counted on the
// warp's barrier, once the block is free.
__device__ __forceinline__ void fetch_residual(const FusedParams &f, const CUtensorMap *tmR, uint32_t lbar, uint8_t *block,
                                               int64_t row0, int64_t j, int lane)
{
    if (lane != 0) return;
    if (f.g.tma_c) bulk_wait_group_read0();
    mbar_arrive_expect_tx(lbar, FUSED_STAGE_BYTES);
    tma_load_2d(smem_addr(block), tmR, lbar, static_cast<int32_t>(j), static_cast<int32_t>(row0));
}

// A warp's residual pieces: the barrier, its phase, and whether a copy is under way.
struct Residual {
    uint32_t bar;
    uint32_t phase;
    bool on, loading;
};

// 32 columns of C from column j0 on, a row per lane, through the block: one piece of bf16,
// two of fp32. With a residual its piece lies in the block already: the sum is taken there,
// in FP32, and rounded once; then the next piece comes (columns below `end`). False when
// the wait for a piece ran out.
__device__ __forceinline__ bool store_group(const FusedParams &f, const CUtensorMap *tmC, const CUtensorMap *tmR,
                                            Residual &res, uint8_t *block, const float *v, int64_t row0, int64_t j0,
                                            int64_t end, volatile int *abort_flag, int lane)
{
    const GemmParams &p = f.g;
    const int pieces = p.c_bf16 ? 1 : 2, width = p.c_bf16 ? 32 : 16;
    const int64_t esz = p.c_bf16 ? 2 : 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int64_t j = j0 + b * width;
        if (b >= pieces || j >= end) break;
        if (res.on) {
            if (!wait_warp<false>(res.bar, res.phase, abort_flag, p.timeout_ns)) return false;
            res.phase ^= 1u;
            res.loading = false;
        } else if (p.tma_c) {
            free_block(lane);
        }
        if (p.c_bf16) {
            if (b == 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint4 *slot = block_at(block, lane, u);
                    float2 t[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = make_float2(v[8 * u + 2 * e], v[8 * u + 2 * e + 1]);
                    if (res.on) {
                        const uint4 old = *slot;
                        const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            t[e] = add2(t[e], make_float2(__uint_as_float(o[e] << 16), __uint_as_float(o[e] & 0xFFFF0000u)));
                    }
                    __nv_bfloat162 h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(t[e].x, t[e].y);
                    *slot = *reinterpret_cast<const uint4 *>(h);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float4 *slot = reinterpret_cast<float4 *>(block_at(block, lane, u));
                float4 t = make_float4(v[16 * b + 4 * u], v[16 * b + 4 * u + 1], v[16 * b + 4 * u + 2], v[16 * b + 4 * u + 3]);
                if (res.on) {
                    const float4 o = *slot;
                    t = make_float4(t.x + o.x, t.y + o.y, t.z + o.z, t.w + o.w);
                }
                *slot = t;
            }
        }
        if (p.tma_c) {
            send_block(tmC, block, j, row0, lane);
        } else {
            __syncwarp();
            store_block(block, static_cast<uint8_t *>(p.C), p.ldc * esz, row0, p.m, j * esz, p.n * esz, lane);
            // R's next piece comes by TMA into the block that the lanes have just written and
            // read: every lane orders its own accesses before that copy
            if (res.on) fence_proxy_async_shared();
            __syncwarp();
        }
        if (res.on && j + width < end) {
            fetch_residual(f, tmR, res.bar, block, row0, j + width, lane);
            res.loading = true;
        }
    }
    return true;
}

template <int BN, int STAGES, int PAIR, int KPS, bool BWD, bool CHUNKED>
__device__ __forceinline__ void run_epilogue_fused(const CUtensorMap *tmC, const CUtensorMap *tmR, const FusedParams &f, uint32_t bar0,
                                                   uint32_t tmem_base, uint8_t *staging, uint32_t rank,
                                                   volatile int *abort_flag, int warp, int lane)
{
    using Cfg = KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS>;
    constexpr int HC = BN / 4;  // accumulator columns of one warp of a whole tile
    const GemmParams &p = f.g;
    const int quad = warp & 3;          // TMEM lanes 32 quad .. are this warp's rows
    const int part = (warp - FUSED_FIRST_EPI_WARP) >> 2;  // its quarter of the columns
    uint8_t *block = staging + (warp - FUSED_FIRST_EPI_WARP) * FUSED_STAGE_BYTES;
    Residual res = {bar0 + 8u * (2 * STAGES + 5 + warp - FUSED_FIRST_EPI_WARP), 0u, false, false};
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int64_t u = first_unit<PAIR>(); u < p.num_units && ok; u += unit_stride<PAIR>()) {
        const Unit w = map_unit<Cfg::TILE_M, BN, false>(p, u);
        const bool to_slot = w.slot >= 0;
        const bool halved = PAIR == 2 && BN == 256 && w.nh >= 0;
        const int ncol = halved ? HC / 2 : HC;  // columns of this warp in this unit
        const int64_t row0 = w.tm * Cfg::TILE_M + rank * CTA_M + quad * 32;
        // (a half unit's accumulator columns 0-63 and 64-127 lie BN / 2 apart in the tile)
        const int64_t xcol = w.tn * BN + (halved ? (part >> 1) * (BN / 2) + w.nh * (BN / 4) + (part & 1) * ncol : part * ncol);
        const bool live = row0 < p.m && xcol < p.n;  // anything of this warp's block inside C
        const int64_t row = row0 + lane;
        const bool row_in = row < p.m;
        // scale codes of this row: one byte per 32 columns, this warp's from xcol / 32 on
        const int64_t s_at = ((row >> 7) * f.katoms + (xcol >> 7)) * SF_ATOM_BYTES + (row & 31) * 16 +
                             ((row & 127) >> 5) * 4 + ((xcol >> 5) & 3);
        uint32_t scales = 0;  // lowest byte first
        if (BWD && live && !to_slot) {  // the codes and scales of Q and S, ahead of the accumulator
            if (p.tma_c) free_block(lane);
            start_block_copy(block, f.Q, f.ldq, row0, p.m, xcol, p.n, lane);
            if (row_in) scales = ncol == 64 ? *reinterpret_cast<const uint16_t *>(f.S + s_at) : f.S[s_at];
        }
        // The residual's first piece ahead of the accumulator.
        const int64_t col_end = min(p.n, xcol + ncol);
        res.on = !BWD && f.R != nullptr && live && !to_slot;
        if (res.on) {
            fetch_residual(f, tmR, res.bar, block, row0, xcol, lane);
            res.loading = true;
        }
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(part * ncol);
        uint4 codes[BWD ? HC / 16 : 1] = {};  // this row's, once they have landed

        // One group: 32 columns from xcol + 32 g, z holding their sums.
        auto finish_group = [&](int g, float *z) {
            const int64_t j0 = xcol + 32 * g;
            if (to_slot) {  // fp32 partial of a split tile, whole rows of the slot
                uint8_t *slot = reinterpret_cast<uint8_t *>(
                    p.partial + (w.slot * Cfg::TILE_M + rank * CTA_M + quad * 32) * static_cast<int64_t>(BN) + part * HC);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4 *>(block_at(block, lane, j)) = make_float4(
                            z[16 * b + 4 * j], z[16 * b + 4 * j + 1], z[16 * b + 4 * j + 2], z[16 * b + 4 * j + 3]);
                    __syncwarp();
                    store_block(block, slot, BN * 4, 0, 32, 128 * g + 64 * b, HC * 4, lane);
                    __syncwarp();
                }
                return;
            }
            if constexpr (BWD) {
                // ---- C = alpha z . act'(z~)
                if (j0 >= p.n || !live) return;
                const float2 scale = both(ue8m0_value((scales >> (8 * g)) & 0xFFu)), alpha = both(p.alpha);
                const uint4 u0 = codes[0], u1 = codes[BWD ? 1 : 0];
                const uint32_t u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                with_act(f.act, [&](auto tag) {
                    constexpr int ACT = decltype(tag)::value;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float d[4];
                        e4m3x4_values(u[q], d);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 x = mul2(make_float2(z[4 * q + e], z[4 * q + e + 1]), alpha);
                            const float2 y = mul2(x, act_slope2<ACT>(mul2(make_float2(d[e], d[e + 1]), scale)));
                            z[4 * q + e] = y.x;
                            z[4 * q + e + 1] = y.y;
                        }
                    }
                });
                if (f.colsum != nullptr) {
                    // rows past m and columns past n hold whatever the block and the
                    // accumulator had there (a zero row of A times an infinity of B): not
                    // in the sums
                    if (!row_in || j0 + 32 > p.n) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!row_in || j0 + e >= p.n) z[e] = 0.0f;
                    }
                    const float sum = column_sum32(z, lane);
                    if (j0 + lane < p.n) f.colsum[(row0 >> 5) * f.ld_colsum + j0 + lane] = sum;
                }
                store_group(f, tmC, tmR, res, block, z, row0, j0, col_end, abort_flag, lane);
            } else {
                // ---- z = alpha z + bias, the checkpoint of z, C = act(z) + R
                if (j0 >= p.n || !live) return;
                scale_bias32(f, j0, z);
                if (f.Q != nullptr) {
                    if (j0 + 32 > p.n) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (j0 + e >= p.n) z[e] = 0.0f;
                    }
                    // (through the block, unless it holds the residual)
                    uint4 c[2];
                    const uint32_t code = mx_group(z, c);
                    scales |= (row_in ? code : 0u) << (8 * g);
                    if (res.on) {
                        if (row_in) store_codes(f.Q + row * f.ldq + j0, c, p.n - j0);
                    } else {
                        if (p.tma_c) free_block(lane);  // of the last group's C
                        *block_at(block, lane, 0) = c[0];
                        *block_at(block, lane, 1) = c[1];
                        __syncwarp();
                        store_block<2>(block, f.Q, f.ldq, row0, p.m, j0, p.n, lane);
                        __syncwarp();
                    }
                }
                with_act(f.act, [&](auto tag) { act_values<decltype(tag)::value, 32>(z); });
                ok = store_group(f, tmC, tmR, res, block, z, row0, j0, col_end, abort_flag, lane) && ok;
            }
        };
        auto take_codes = [&] {
            if constexpr (BWD) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();  // every lane's copies have landed
#pragma unroll
                for (int q = 0; q < HC / 16; ++q) codes[q] = *block_at(block, lane, q);
                __syncwarp();  // every lane has read its codes: the block is free
            }
        };
        auto release = [&] {  // this warp's part of the accumulator is read
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
        };

        if constexpr (!CHUNKED) {
            // One accumulator holds the unit's sums: group by group from tensor memory, which is
            // given back with the last group's load.
            ok = wait_warp<PAIR == 2>(bar0 + 8u * (2 * STAGES + acc), acc_phase, abort_flag, p.timeout_ns);
            take_codes();
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t taddr = lane_base + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
            for (int g = 0; 32 * g < ncol; ++g) {
                uint32_t r[32];
                tmem_load_32cols(taddr + 32u * g, r);
                if (32 * (g + 1) >= ncol) release();
                float z[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) z[e] = __uint_as_float(r[e]);
                finish_group(g, z);
                if constexpr (BWD && HC > 32) codes[0] = codes[HC / 16 - 2], codes[1] = codes[HC / 16 - 1];
            }
        } else {
            float v[HC];
            for (int c0 = w.kb0, i = 0; c0 < w.kb1; c0 += i < 2 ? f.chunk_first : f.chunk_rest, ++i) {
                if (!wait_warp<PAIR == 2>(bar0 + 8u * (2 * STAGES + acc), acc_phase, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t taddr = lane_base + static_cast<uint32_t>(acc * BN);
                // (16 columns at a time: with 32 beside the 64 sums the kernel spilled more, 124
                // loads per tile and lane from a first-level cache of a few KB. What is left in
                // the 256 x 256 copies is 116 bytes of spills a thread forward, 240 backward)
#pragma unroll
                for (int g = 0; g < HC / 16; ++g) {
                    if (g * 16 >= ncol) continue;
                    uint32_t r[16];
                    tmem_load_16cols(taddr + 16u * g, r);
                    if (c0 == w.kb0) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[16 * g + e] = __uint_as_float(r[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 s = add2(make_float2(v[16 * g + e], v[16 * g + e + 1]),
                                                  make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
                            v[16 * g + e] = s.x;
                            v[16 * g + e + 1] = s.y;
                        }
                    }
                }
                release();
            }
            take_codes();
            if (!ok) break;
            // (one copy of the code, for the instruction cache: 4096 x 16384 x 4096 with FP32 C 372 us
            // with two, 356 with one)
#pragma unroll 1
            for (int g = 0; 32 * g < ncol; ++g) {
                finish_group(g, v);
                if constexpr (HC > 32) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = v[HC - 32 + e];
                    if constexpr (BWD) codes[0] = codes[HC / 16 - 2], codes[1] = codes[HC / 16 - 1];
                }
            }
        }
        // scale codes of this row's groups, padding rows and groups of the array as zeros
        if (!BWD && f.Q != nullptr && !to_slot && (row0 & ~int64_t(127)) < p.m && (xcol & ~int64_t(127)) < p.n) {
            if (ncol == 64) *reinterpret_cast<uint16_t *>(f.S + s_at) = static_cast<uint16_t>(scales);
            else f.S[s_at] = static_cast<uint8_t>(scales);
        }
    }
    if (!ok && lane == 0) signal_timeout(p, abort_flag);
    if (!ok && res.loading) spin_ns(100000);  // a copy may still land in the block
    if (p.tma_c && lane == 0) bulk_wait_group0();  // shared memory must outlive the stores that read it
}

// ---------------------------------------------------------------- kernels
template <int BN, int STAGES, int PAIR, int KPS, bool BWD, bool CHUNKED>
__global__ void __launch_bounds__(FUSED_THREADS, 1)
    bm_gemm_fused_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR,
                         const FusedParams f)
{
    using Cfg = FusedCfg<BN, STAGES, PAIR, KPS>;
    const GemmParams &p = f.g;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    uint8_t *smem = smem_raw + pad;
    const uint32_t ring = raw + pad;
    uint8_t *staging = smem + Cfg::RING_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + Cfg::STAGING_BYTES);
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
            mbar_init(bar0 + 8u * (2 * STAGES + 2 + b), FUSED_EPI_WARPS * PAIR);  // accumulator empty
        }
        mbar_init(bar0 + 8u * (2 * STAGES + 4), 1);  // drain (abort path only)
        for (int e = 0; e < FUSED_EPI_WARPS; ++e) mbar_init(bar0 + 8u * (2 * STAGES + 5 + e), 1);  // residual pieces
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        if (p.tma_c) tma_prefetch_map(&tmC);
        if (f.R != nullptr) tma_prefetch_map(&tmR);
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

    if (warp < FUSED_FIRST_EPI_WARP) {
        if constexpr (CHUNKED) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FUSED_MAIN_REGS));
        if (warp == 0 && lane == 0)
            run_producer<BN, STAGES, PAIR, ELEM_BF16, KPS, EPI_STORE>(&tmA, &tmB, &tmA, &tmB, p, ring, bar0, rank,
                                                                      abort_flag);
        if (warp == 1 && rank == 0)
            run_mma_chunked<BN, STAGES, PAIR, KPS>(f, ring, bar0, tmem_base, abort_flag, lane);
    } else {
        if constexpr (CHUNKED) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FUSED_EPI_REGS));
        run_epilogue_fused<BN, STAGES, PAIR, KPS, BWD, CHUNKED>(&tmC, &tmR, f, bar0, tmem_base, staging, rank, abort_flag, warp, lane);
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

// ---------------------------------------------------------------- four columns of a row
// The same work on columns j .. j + 3 of row i (j = 4 lane within a 128-column block, so
// that 8 lanes hold one MXFP8 group): `v` holds the product's sums, `b` the bias. Called
// by whole warps, for the rows past m too where the checkpoint's padding entries are
// written. Adds C to `sum` (backward).
__device__ __forceinline__ void load_bias4(const FusedParams &f, int64_t j, float (&b)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        b[e] = 0.0f;
        if (f.bias != nullptr && j + e < f.g.n)
            b[e] = f.bias_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(f.bias)[j + e]) << 16)
                               : static_cast<const float *>(f.bias)[j + e];
    }
}

// What the epilogue reads for those four columns (zeros where there is nothing): loaded on
// its own so that a loop over rows can load the next row's ahead.
struct Row4 {
    float4 res;      // forward: R
    uint32_t codes;  // backward: Q's codes and the group's scale code
    uint32_t scale;
};

__device__ __forceinline__ int64_t scale_at(const FusedParams &f, int64_t i, int64_t j)
{
    return ((i >> 7) * f.katoms + (j >> 7)) * SF_ATOM_BYTES + (i & 31) * 16 + ((i & 127) >> 5) * 4 + ((j >> 5) & 3);
}

template <bool BWD>
__device__ __forceinline__ Row4 load_row4(const FusedParams &f, int64_t i, int64_t j)
{
    const GemmParams &p = f.g;
    Row4 o;
    o.res = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    o.codes = o.scale = 0u;
    if (i >= p.m || j >= p.n) return o;
    if constexpr (BWD) {
        o.scale = f.S[scale_at(f, i, j)];
        const uint8_t *q = f.Q + i * f.ldq + j;
        if (j + 4 <= p.n) {
            o.codes = *reinterpret_cast<const uint32_t *>(q);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (j + e < p.n) o.codes |= static_cast<uint32_t>(q[e]) << (8 * e);
        }
    } else if (f.R != nullptr) {
        o.res = load_res4(f, i, j);
    }
    return o;
}

template <bool BWD>
__device__ __forceinline__ void fused_row4(const FusedParams &f, int64_t i, int64_t j, float (&v)[4], const float (&b)[4],
                                           const Row4 &o, float (&sum)[4], int lane)
{
    const GemmParams &p = f.g;
    const bool in = i < p.m && j < p.n;
    if constexpr (BWD) {
        if (!in) return;
        const float scale = ue8m0_value(o.scale);
        float d[4];
        e4m3x4_values(o.codes, d);
        with_act(f.act, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float2 y = act_slope2<ACT>(make_float2(d[e] * scale, d[e + 1] * scale));
                v[e] = p.alpha * v[e] * y.x;
                v[e + 1] = p.alpha * v[e + 1] * y.y;
            }
        });
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < p.n) sum[e] += v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = j + e < p.n ? fmaf(p.alpha, v[e], b[e]) : 0.0f;
        if (f.Q != nullptr) {
            // the group's largest magnitude over its 8 lanes; a NaN counts as infinite
            float amax = 0.0f;
            if (in) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = fabsf(v[e]);
                    amax = a <= 3.402823466e38f ? fmaxf(amax, a) : __uint_as_float(0x7F800000u);
                }
            }
#pragma unroll
            for (int o2 = 4; o2 >= 1; o2 >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o2));
            const bool special = amax > 3.402823466e38f;
            const uint32_t code = special ? 255u : ue8m0_code(amax);
            if ((lane & 7) == 0 && (j & ~int64_t(127)) < p.n) f.S[scale_at(f, i, j)] = static_cast<uint8_t>(in ? code : 0u);
            if (in) {
                const float inv = __uint_as_float((254u - (special ? 0u : code)) << 23);
                const uint32_t codes = special ? 0x7F7F7F7Fu : e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                uint8_t *dst = f.Q + i * f.ldq + j;
                if (j + 4 <= p.n) {
                    *reinterpret_cast<uint32_t *>(dst) = codes;
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (j + e < p.n) dst[e] = static_cast<uint8_t>(codes >> (8 * e));
                }
            }
        }
        if (!in) return;
        with_act(f.act, [&](auto tag) { act_values<decltype(tag)::value, 4>(v); });
    }
    store_row4(f, i, j, make_float4(v[0] + o.res.x, v[1] + o.res.y, v[2] + o.res.z, v[3] + o.res.w));
}

// The epilogue's work from fp32 partial slots (every tile split along K), or from
// nothing (alpha == 0 or k == 0: k_splits == 0). One warp takes row_block rows x 128
// columns, four columns per lane, and sums its columns over its rows.
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
        if constexpr (!BWD) load_bias4(f, j, b);
#pragma unroll 1
        for (int rr = 0; rr < f.row_block; ++rr) {
            const int64_t i = rb * f.row_block + rr;
            if (i >= rows) break;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (i < p.m && j < p.n && p.k_splits > 0) {
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
                v[0] = s.x, v[1] = s.y, v[2] = s.z, v[3] = s.w;
            }
            fused_row4<BWD>(f, i, j, v, b, load_row4<BWD>(f, i, j), sum, lane);
        }
        if (BWD && f.colsum != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < p.n) f.colsum[rb * f.ld_colsum + j + e] = sum[e];
        }
    }
}

}  // namespace bm
