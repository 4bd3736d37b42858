// bm_epi_kernel.cuh -- tiled products whose epilogue is an operator of its own:
//
//   GLU   (bf16)  G = alpha op(A) Wg, U = alpha op(A) Wu;  H = act(G) . U, and G, U on request
//   DGLU  (bf16)  dH = alpha op(A) op(B);  dG = dH . U . act'(G), dU = dH . act(G), and
//                 H = act(G) . U on request
//   GRAM  (fp16)  A = alpha X X^T over one triangle, written to both: its diagonal to an FP32
//                 vector, the rest to fp16
//   POLY  (fp16)  B = b A + c A^2 the same way, from A's two parts
//   STEP  (fp16)  X' = (a + diag B) X + (B off its diagonal) X, X in two fp16 halves; the last
//                 one C = alpha X' + beta C in bf16
//
// The mainloop is that of bm_gemm_kernel.cuh (producer, ring, schedule, MMA issue), but that
// a GLU tile's B rows come half from Wg and half from Wu: columns [0, BN / 2) of an
// accumulator are the gate's and the others the up projection's for the same BN / 2 columns
// of H, so that both meet in one lane of the epilogue and neither projection goes through
// global memory unless it is asked for. On an SM pair each CTA stages BN / 2 rows of B:
// rank 0 the gate's, rank 1 the up projection's.
//
// Epilogue: 16 warps of 32 rows (lane = row) x BN / 4 columns in groups of 32 columns, from
// tensor memory to 16-bit values, which leave through a 2 KB staging block per warp (by TMA
// where a row ends on 16 bytes). What DGLU and STEP read comes through the same block, a
// matrix at a time. (Loads of a row per lane keep no more lines in flight than the first-level
// cache beside the ring holds, about 200: 4096 x 16384 x 4096 with H took 435 us with them,
// 391 with TMA boxes of 16 columns that hold both matrices, 383 with these; 8192 x 8192 x 1024
// 242, 191 and 195.)
//
// Bound by the tensor cores, on long runs by the power limit, and by shared memory, whose
// bandwidth a pair tile's operands take whole (64 bytes a clock in, 64 out): what the epilogue
// stages comes on top. 4096 x 16384 x 4096 on long runs, in brackets on short ones: GLU with G
// and U kept 660 us, 1665 TFLOP/s (576); DGLU with H 425 us, 1293 TFLOP/s (380). A step of 4096 x
// 4096: GRAM 49 us, POLY 51, STEP 92, where the plain product takes 79. At 104 registers three
// copies' epilogues spill (stores and loads, bytes a thread): GLU on pairs 36 and 44, DGLU on pairs
// 60 and 88, DGLU on 128 x 256 tiles 64 and 104.
#pragma once

#include <cuda_fp16.h>

#include "bm_act.cuh"
#include "bm_fused_kernel.cuh"
#include "bm_gemm_kernel.cuh"

namespace bm {

enum : int { KIND_GLU = 0, KIND_DGLU = 1, KIND_GRAM = 2, KIND_POLY = 3, KIND_STEP = 4 };
__host__ __device__ constexpr int kind_elem(int kind) { return kind >= KIND_GRAM ? ELEM_F16 : ELEM_BF16; }
__host__ __device__ constexpr bool kind_symmetric(int kind) { return kind == KIND_GRAM || kind == KIND_POLY; }

struct EpiParams {
    GemmParams g;  // schedule, sizes, alpha; C unused
    int act;       // ACT_*
    // 16-bit matrices of the output's shape. GLU: out H, G, U (G, U null: not kept).
    // DGLU: in G, U, out dG, dU, H (null: not wanted). GRAM: out A. POLY: in A, out B.
    // STEP: in X high, X low, out the same of X', or C alone (the last step).
    const void *in[2];
    int64_t ldin[2];
    void *out[3];
    int64_t ldout[3];
    int tma[3];        // out[i] has a tensor map
    int64_t in_cols;   // POLY over clusters: columns of `in` that may be read, the padded row
    // GRAM writes diag_out; POLY reads diag and writes diag_out; STEP reads diag
    const float *diag;
    float *diag_out;
    float ca, cb, cc;  // the step's coefficients
    int diag_cols;     // STEP: the diagonal scales columns (X tall) instead of rows
    int last;          // STEP: out[0] is C
    float beta;        // STEP, last: C = alpha X' + beta C
};

// The launch's 640 x 96 registers, shared out (as in bm_fused_kernel.cuh; the host checks the 96).
constexpr int EPI_MAIN_REGS = 64, EPI_EPI_REGS = 104;
static_assert(128 * EPI_MAIN_REGS + 32 * FUSED_EPI_WARPS * EPI_EPI_REGS <= FUSED_THREADS * FUSED_LAUNCH_REGS, "register split");
constexpr int SPARE_BLOCKS = 6;  // 2 KB blocks of the ring per epilogue warp in a CTA's last unit

// ---------------------------------------------------------------- producer of a GLU tile
// Copies of `ROWS` rows of one weight from row `row` into its half of a stage's B region:
// half `h` starts h ROWS rows (K-major) or h ROWS / 64 chunks (N-major) into it.
template <int PAIR, int KPS, int ROWS, int B_ROWS>
__device__ __forceinline__ void load_weight(uint32_t b, int h, const CUtensorMap *map, bool box3, bool mn_major,
                                            uint32_t bar, int32_t row, int kb)
{
    if (mn_major) {
        const uint32_t dst = b + static_cast<uint32_t>(h * (ROWS / 64) * KPS * 8192);
        if (box3) {
            load_box3<PAIR>(dst, map, bar, 0, kb * TILE_K, row / 64);
            return;
        }
#pragma unroll
        for (int sub = 0; sub < KPS; ++sub)
#pragma unroll
            for (int c = 0; c < ROWS / 64; ++c)
                load_box<PAIR>(dst + c * KPS * 8192 + sub * 8192, map, bar, row + 64 * c, (kb + sub) * TILE_K);
        return;
    }
    const uint32_t dst = b + static_cast<uint32_t>(h * ROWS * 128);
    if (box3 && ROWS == B_ROWS) {
        load_box3<PAIR>(dst, map, bar, 0, row, kb);
        return;
    }
#pragma unroll
    for (int sub = 0; sub < KPS; ++sub) load_box<PAIR>(dst + sub * B_ROWS * 128, map, bar, (kb + sub) * TILE_K, row);
}

// run_producer of bm_gemm_kernel.cuh with two B operands.
template <int BN, int STAGES, int PAIR, int KPS>
__device__ __forceinline__ void run_producer_glu(const CUtensorMap *tmA, const CUtensorMap *tmG, const CUtensorMap *tmU,
                                                 const GemmParams &p, uint32_t ring, uint32_t bar0, uint32_t rank,
                                                 volatile int *abort_flag)
{
    using Cfg = KernelCfg<BN, STAGES, PAIR, ELEM_BF16, KPS>;
    constexpr int HALF = PAIR == 2 ? Cfg::B_ROWS : Cfg::B_ROWS / 2;  // rows of one weight that this CTA stages
    int stage = 0;
    uint32_t phase = 0;
    uint32_t armed = 0, armed_parity = 0;
    bool ok = true, first = true, issued_any = false;
    for (int64_t u = first_unit<PAIR>(); u < p.num_units && ok; u += unit_stride<PAIR>()) {
        const Unit w = map_unit<Cfg::TILE_M, BN, false>(p, u);
        const int32_t row_a = static_cast<int32_t>(w.tm * Cfg::TILE_M + rank * CTA_M);
        const int32_t row_b = static_cast<int32_t>(w.tn * (BN / 2));
        for (int kb = w.kb0; kb < w.kb1; kb += KPS) {
            if (!wait_one<PAIR == 2>(bar0 + 8u * (STAGES + stage), phase ^ 1u, abort_flag, p.timeout_ns)) {
                ok = false;
                break;
            }
            const uint32_t full = bar0 + 8u * stage;
            if (rank == 0) {
                mbar_arrive_expect_tx(full, static_cast<uint32_t>(Cfg::STAGE_BYTES * PAIR));
                armed |= 1u << stage;
                armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            }
            if (!(p.debug_stall && first)) {
                issued_any = true;
                const uint32_t bar = PAIR == 2 ? map_shared_to_rank(full, 0) : full;
                const uint32_t sa = ring + stage * Cfg::STAGE_BYTES;
                load_operand<PAIR, KPS, CTA_M, TILE_K>(sa, tmA, tmA, p.a_box3 != 0, p.a_mn_major != 0, bar, row_a, kb, 0);
                if constexpr (PAIR == 2) {
                    load_weight<PAIR, KPS, HALF, Cfg::B_ROWS>(sa + Cfg::B_OFFSET, 0, rank == 0 ? tmG : tmU, p.b_box3 != 0,
                                                              p.b_mn_major != 0, bar, row_b, kb);
                } else {
                    load_weight<PAIR, KPS, HALF, Cfg::B_ROWS>(sa + Cfg::B_OFFSET, 0, tmG, p.b_box3 != 0,
                                                              p.b_mn_major != 0, bar, row_b, kb);
                    load_weight<PAIR, KPS, HALF, Cfg::B_ROWS>(sa + Cfg::B_OFFSET, 1, tmU, p.b_box3 != 0,
                                                              p.b_mn_major != 0, bar, row_b, kb);
                }
            }
            first = false;
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok) {
        signal_timeout(p, abort_flag);
        for (int s = 0; s < STAGES; ++s)  // copies in flight land before shared memory is released
            if ((armed >> s) & 1u) wait_one(bar0 + 8u * s, (armed_parity >> s) & 1u, nullptr, p.timeout_ns);
        if (PAIR == 2 && issued_any) spin_ns(100000);
    }
}

// ---------------------------------------------------------------- rows of 16-bit values
__device__ __forceinline__ float2 bf16_pair(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 f16_pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

__device__ __forceinline__ uint32_t pack_f16(float2 v)
{
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// W 16-bit values of row i from column j on, in pairs; zeros past `cols` and rows past m.
// Rows and j lie on 16 bytes.
template <int W>
__device__ __forceinline__ void load_row(const void *base, int64_t ld, int64_t i, int64_t m, int64_t j, int64_t cols,
                                         uint32_t (&w)[W / 2])
{
    const uint16_t *src = static_cast<const uint16_t *>(base) + i * ld + j;
#pragma unroll
    for (int q = 0; q < W / 8; ++q) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i < m && j + 8 * q + 8 <= cols) {
            v = *reinterpret_cast<const uint4 *>(src + 8 * q);
        } else if (i < m && j + 8 * q < cols) {
            uint32_t t[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (j + 8 * q + e < cols) t[e >> 1] |= static_cast<uint32_t>(src[8 * q + e]) << (16 * (e & 1));
            v = make_uint4(t[0], t[1], t[2], t[3]);
        }
        w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
    }
}

// A warp's 32 rows x W 16-bit values (this lane's row in w) to out[o] at (row0, j), through a
// staging block (`fresh`: no store from it is under way).
template <int W>
__device__ __forceinline__ void store_rows(const EpiParams &f, int o, const CUtensorMap *tm, uint8_t *block,
                                           const uint32_t (&w)[W / 2], int64_t row0, int64_t j, int lane, bool fresh = false)
{
    const bool by_tma = W == 32 && f.tma[o];
    if (by_tma && !fresh) free_block(lane);
#pragma unroll
    for (int u = 0; u < W / 8; ++u) *block_at(block, lane, u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    if (by_tma) {
        send_block(tm, block, j, row0, lane);
    } else {
        __syncwarp();
        store_block<W / 8>(block, static_cast<uint8_t *>(f.out[o]), f.ldout[o] * 2, row0, f.g.m, j * 2, f.g.n * 2, lane);
        __syncwarp();
    }
}

// The same block transposed: this lane's row of 32 values becomes column row0 + lane of rows
// j .. j + 31 (symmetric outputs, which always have a map).
__device__ __forceinline__ void store_mirrored(const CUtensorMap *tm, uint8_t *block, const uint32_t (&w)[16], int64_t row0,
                                               int64_t j, int lane, bool fresh = false)
{
    if (!fresh) free_block(lane);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        uint16_t *at = reinterpret_cast<uint16_t *>(block_at(block, e, lane >> 3)) + (lane & 7);
        *at = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
    send_block(tm, block, row0, j, lane);
}

// Half a group of a symmetric product: columns j0 + 16 half .. of row i0 + lane, z their sums, to
// the 16-bit values t. POLY: x holds A there (off its diagonal), di and dcol A's diagonal at this
// row and at column j0 + lane. The matrix's diagonal passes through the group whose rows and
// columns meet: it goes to diag_out.
template <int KIND>
__device__ __forceinline__ void symmetric_half(const EpiParams &f, const float (&z)[16], const uint32_t *x, float di, float dcol,
                                               int64_t i0, int64_t j0, int half, uint32_t *t, int lane)
{
    const float2 alpha = both(f.g.alpha);
    const int mine = i0 == j0 ? lane - 16 * half : -1;  // the diagonal's place among the 16, if it is there
    float own = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        float2 w = make_float2(z[e], z[e + 1]);
        if constexpr (KIND == KIND_GRAM) {
            w = mul2(w, alpha);
        } else {
            // A = D + O (D its diagonal): (A^2)_ij = (O^2)_ij + (D_i + D_j) O_ij, and on the diagonal
            // (O^2)_ii + D_i^2; O_ii = 0
            const float2 a = f16_pair(x[e / 2]);
            const float2 dj = make_float2(__shfl_sync(0xffffffffu, dcol, 16 * half + e),
                                          __shfl_sync(0xffffffffu, dcol, 16 * half + e + 1));
            w = fma2(both(f.cc), fma2(add2(both(di), dj), a, w), mul2(both(f.cb), a));
        }
        if (e == mine) {
            own = KIND == KIND_GRAM ? w.x : z[e];
            w.x = 0.0f;
        }
        if (e + 1 == mine) {
            own = KIND == KIND_GRAM ? w.y : z[e + 1];
            w.y = 0.0f;
        }
        t[e / 2] = pack_f16(w);
    }
    if (mine >= 0 && mine < 16 && i0 + lane < f.g.m)
        f.diag_out[i0 + lane] = KIND == KIND_GRAM ? own : f.ca + fmaf(f.cc, own, fmaf(f.cc * di, di, f.cb * di));
}

// ---------------------------------------------------------------- epilogue
template <int BN, int STAGES, int PAIR, int KPS, int KIND>
__device__ __forceinline__ void run_epilogue_kind(const CUtensorMap *tm0, const CUtensorMap *tm1, const CUtensorMap *tm2,
                                                  const CUtensorMap *tmI0, const CUtensorMap *tmI1, const EpiParams &f,
                                                  uint32_t bar0, uint32_t tmem_base, uint8_t *ring, uint8_t *staging,
                                                  uint32_t rank, volatile int *abort_flag, int warp, int lane)
{
    using Cfg = KernelCfg<BN, STAGES, PAIR, kind_elem(KIND), KPS>;
    constexpr bool GLU = KIND == KIND_GLU;
    constexpr bool TWO = KIND == KIND_DGLU || KIND == KIND_STEP;  // two inputs of the output's shape
    constexpr bool ONE = KIND == KIND_POLY;                       // one
    static_assert(Cfg::RING_BYTES >= FUSED_EPI_WARPS * SPARE_BLOCKS * FUSED_STAGE_BYTES, "spare blocks");
    constexpr int OUT_BN = GLU ? BN / 2 : BN;  // output columns of a tile
    constexpr int HC = OUT_BN / 4;             // of one warp
    constexpr int W = HC < 32 ? HC : 32;       // of a group
    constexpr int GROUPS = HC / W;
    static_assert(GROUPS <= 2, "a CTA's last unit has spare input blocks for one group after the first");
    const GemmParams &p = f.g;
    const int quad = warp & 3;
    const int part = (warp - FUSED_FIRST_EPI_WARP) >> 2;
    uint8_t *block = staging + (warp - FUSED_FIRST_EPI_WARP) * FUSED_STAGE_BYTES;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    // Inputs (DGLU, STEP; POLY's one): 32 rows x 32 columns by TMA into the warp's block. A unit's
    // first comes ahead of the accumulator, the second once the first is in registers; the next
    // group's (or unit's) first once the block's last output has left. In a CTA's last unit the
    // ring is free when the accumulator is full: each warp has SPARE_BLOCKS blocks of it, takes the
    // other group's inputs there at once and waits for no output. (That unit's epilogue is the one
    // that nothing hides: 777 x 1320 x 520 backward, from a graph, 12.5 us without, 11.7 with.)
    const uint32_t in_bar = bar0 + 8u * (2 * STAGES + 5 + warp - FUSED_FIRST_EPI_WARP);
    uint32_t in_phase = 0;
    bool in_flight = false;
    auto spare = [&](int i) { return ring + ((warp - FUSED_FIRST_EPI_WARP) * SPARE_BLOCKS + i) * FUSED_STAGE_BYTES; };
    auto fetch = [&](const CUtensorMap *map, uint8_t *to, int64_t i, int64_t j) {
        in_flight = true;
        if (lane != 0) return;
        mbar_arrive_expect_tx(in_bar, FUSED_STAGE_BYTES);
        tma_load_2d(smem_addr(to), map, in_bar, static_cast<int32_t>(j), static_cast<int32_t>(i));
    };
    auto landed = [&] {
        if (!wait_warp<false>(in_bar, in_phase, abort_flag, p.timeout_ns)) return false;
        in_phase ^= 1u;
        in_flight = false;
        return true;
    };
    auto read = [&](uint32_t (&x)[W / 2], uint8_t *from) {
#pragma unroll
        for (int q = 0; q < W / 8; ++q) {
            const uint4 v = *block_at(from, lane, q);
            x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
        }
    };
    auto take = [&](uint32_t (&x)[W / 2]) {
        if (!landed()) return false;
        read(x, block);
        fence_proxy_async_shared();  // these reads before the next copy's writes
        __syncwarp();
        return true;
    };
    // A unit's rows, columns and accumulator columns of this warp. A tile of a last wave may
    // run as two halves of its columns (256 x 256 pair tiles): of each CTA's rows of B the first
    // or the second 64. Then a warp has one group, and of a GLU tile's warps every other has.
    int64_t row0 = 0, col0 = 0;
    int acc_col = 0, groups = GROUPS;
    Unit w;
    auto place = [&](int64_t u) {
        if (u >= p.num_units) return false;
        w = map_unit<Cfg::TILE_M, BN, kind_symmetric(KIND)>(p, u);
        row0 = w.tm * Cfg::TILE_M + rank * CTA_M + quad * 32;
        if (PAIR == 2 && !kind_symmetric(KIND) && w.nh >= 0) {
            groups = 1;
            acc_col = part * 32;
            col0 = GLU ? (part < 2 ? w.tn * OUT_BN + w.nh * 64 + part * 32 : p.n)
                       : w.tn * OUT_BN + (part >> 1) * 128 + w.nh * 64 + (part & 1) * 32;
        } else {
            groups = GROUPS;
            acc_col = part * HC;
            col0 = w.tn * OUT_BN + part * HC;
        }
        return row0 < p.m && col0 < p.n;
    };
    bool here = place(first_unit<PAIR>());  // anything of the unit's in this warp's rows and columns
    if ((TWO || ONE) && here) fetch(tmI0, block, row0, col0);
    for (int64_t u = first_unit<PAIR>(); u < p.num_units && ok; u += unit_stride<PAIR>()) {
        const bool final_unit = u + unit_stride<PAIR>() >= p.num_units;
        const int64_t row = row0 + lane;
        const bool mirrored = kind_symmetric(KIND) && w.tm != w.tn;
        uint32_t x0[W / 2], x1[W / 2];
        if constexpr (ONE) {
            if (here && !take(x0)) {
                ok = false;
                break;
            }
        }
        // Diagonal entries: this row's, and of the group's columns column `lane`'s, which the
        // lanes pass round. (32 loads that all lanes share took 16 us of a 128 x 128 tile: each
        // waited for the bounds check of the next.)
        float di = 0.0f, dcol = 0.0f;
        auto load_diag = [&](int64_t j) { return j + lane < p.n ? f.diag[j + lane] : 0.0f; };
        if constexpr (KIND == KIND_POLY || KIND == KIND_STEP) {
            di = row < p.m && !f.diag_cols ? f.diag[row] : 0.0f;
            if (KIND == KIND_POLY || f.diag_cols) dcol = load_diag(col0);
        }
        if (!wait_warp<PAIR == 2>(bar0 + 8u * (2 * STAGES + acc), acc_phase, abort_flag, p.timeout_ns)) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        const uint32_t taddr =
            tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * BN + acc_col);
        const uint32_t up_col = GLU && PAIR == 2 && w.nh >= 0 ? BN / 4 : BN / 2;  // GLU: from gate to up
        const int count = groups;
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
#pragma unroll 1
        for (int g = 0; g < count; ++g) {
            const int64_t j0 = col0 + g * W, i0 = row0;
            const bool live = i0 < p.m && j0 < p.n, end = g == count - 1;  // live: any of the group inside the output
            const float2 alpha = both(p.alpha);
            if constexpr (TWO) {
                if (live) {
                    if (final_unit && g > 0) {
                        ok = landed();
                        read(x0, spare(0));
                        read(x1, spare(1));
                    } else if ((ok = take(x0))) {
                        fetch(tmI1, block, i0, j0);
                        ok = take(x1);
                    }
                    if (!ok) break;
                    if (final_unit && !end && j0 + W < p.n) {
                        in_flight = true;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(in_bar, 2 * FUSED_STAGE_BYTES);
                            tma_load_2d(smem_addr(spare(0)), tmI0, in_bar, static_cast<int32_t>(j0 + W), static_cast<int32_t>(i0));
                            tma_load_2d(smem_addr(spare(1)), tmI1, in_bar, static_cast<int32_t>(j0 + W), static_cast<int32_t>(i0));
                        }
                    }
                }
                uint32_t h[KIND == KIND_DGLU ? W / 2 : 1];
#pragma unroll
                for (int s = 0; s < 2; ++s) {  // (16 columns at a time, to spare registers)
                    uint32_t r[16];
                    tmem_load_16cols(taddr + static_cast<uint32_t>(W * g + 16 * s), r);
                    if (end && s == 1) release();
                    auto z = [&](int e) { return make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])); };
                    if constexpr (KIND == KIND_DGLU) {
                        with_act(f.act, [&](auto tag) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int q = 8 * s + e;
                                const float2 dh = mul2(z(e), alpha), gate = bf16_pair(x0[q]), up = bf16_pair(x1[q]);
                                const ActPair a = act_pair2<decltype(tag)::value>(gate);
                                x0[q] = pack_bf16(mul2(mul2(dh, up), a.slope));
                                x1[q] = pack_bf16(mul2(dh, a.value));
                                h[q] = pack_bf16(mul2(a.value, up));
                            }
                        });
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int q = 8 * s + e;
                            float2 d = both(di);
                            if (f.diag_cols)
                                d = make_float2(__shfl_sync(0xffffffffu, dcol, 2 * q), __shfl_sync(0xffffffffu, dcol, 2 * q + 1));
                            const float2 v = fma2(d, add2(f16_pair(x0[q]), f16_pair(x1[q])), z(e));
                            if (!f.last) {
                                x0[q] = pack_f16(v);
                                const float2 hi = f16_pair(x0[q]);
                                x1[q] = pack_f16(make_float2(v.x - hi.x, v.y - hi.y));
                            } else {  // (both halves of X' alpha, until C has been read)
                                const float2 c = mul2(v, alpha);
                                x0[q] = __float_as_uint(c.x);
                                x1[q] = __float_as_uint(c.y);
                            }
                        }
                    }
                }
                if (live) {
                    if constexpr (KIND == KIND_STEP) {
                        if (f.last) {
                            uint32_t c[W / 2];
                            if (f.beta != 0.0f) load_row<W>(f.out[0], f.ldout[0], row, p.m, j0, p.n, c);
#pragma unroll
                            for (int q = 0; q < W / 2; ++q) {
                                float2 v = make_float2(__uint_as_float(x0[q]), __uint_as_float(x1[q]));
                                if (f.beta != 0.0f) v = fma2(both(f.beta), bf16_pair(c[q]), v);
                                x0[q] = pack_bf16(v);
                            }
                        }
                    }
                    // (the block holds an input that has been read: nothing is under way from it)
                    store_rows<W>(f, 0, tm0, final_unit && g > 0 ? spare(0) : block, x0, i0, j0, lane, true);
                    if (f.out[1] != nullptr)
                        store_rows<W>(f, 1, tm1, final_unit ? spare(g > 0 ? 1 : 2) : block, x1, i0, j0, lane, final_unit);
                    if constexpr (KIND == KIND_DGLU) {
                        if (f.out[2] != nullptr)
                            store_rows<W>(f, 2, tm2, final_unit ? spare(g > 0 ? 4 : 3) : block, h, i0, j0, lane, final_unit);
                    }
                    if (!final_unit) {
                        fence_proxy_async_shared();  // (accesses by the lanes, where there is no map)
                        free_block(lane);
                    }
                }
                if (!end) {
                    if (!final_unit && i0 < p.m && j0 + W < p.n) fetch(tmI0, block, i0, j0 + W);
                    if (f.diag_cols) dcol = load_diag(j0 + W);
                } else if ((here = place(u + unit_stride<PAIR>()))) {
                    fetch(tmI0, block, row0, col0);
                }
                continue;
            }
            if constexpr (kind_symmetric(KIND)) {
                if constexpr (ONE) {
                    if (live && g > 0) {
                        if (final_unit) {
                            ok = landed();
                            read(x0, spare(0));
                        } else {
                            ok = take(x0);
                        }
                        if (!ok) break;
                    }
                    if (live && final_unit && !end && j0 + W < p.n) fetch(tmI0, spare(0), i0, j0 + W);
                }
                uint32_t t[16];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    uint32_t r[16];
                    float z[16];
                    tmem_load_16cols(taddr + static_cast<uint32_t>(W * g + 16 * s), r);
                    if (end && s == 1) release();
#pragma unroll
                    for (int e = 0; e < 16; ++e) z[e] = __uint_as_float(r[e]);
                    symmetric_half<KIND>(f, z, x0 + 8 * s, di, dcol, i0, j0, s, t + 8 * s, lane);
                }
                if (live) {
                    store_rows<32>(f, 0, tm0, final_unit && g > 0 ? spare(0) : block, t, i0, j0, lane,
                                   ONE || (final_unit && g > 0));
                    if (mirrored) store_mirrored(tm0, final_unit ? spare(g > 0 ? 2 : 1) : block, t, i0, j0, lane, final_unit);
                    if (ONE && !final_unit) free_block(lane);
                }
                if (end) here = place(u + unit_stride<PAIR>());
                if constexpr (ONE) {
                    if (!end) {
                        if (live && !final_unit && j0 + W < p.n) fetch(tmI0, block, i0, j0 + W);
                        dcol = load_diag(j0 + W);
                    } else if (here) {
                        fetch(tmI0, block, row0, col0);
                    }
                }
                continue;
            }
            uint32_t r[W], r2[GLU ? W : 1];
            if constexpr (W == 32) tmem_load_32cols(taddr + 32u * g, r);
            else tmem_load_16cols(taddr + 16u * g, r);
            if constexpr (GLU) {
                if constexpr (W == 32) tmem_load_32cols(taddr + up_col, r2);
                else tmem_load_16cols(taddr + up_col, r2);
            }
            if (end) {
                release();
                place(u + unit_stride<PAIR>());
            }
            if (!live) continue;
            auto z = [&](int e) { return make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])); };
            if constexpr (GLU) {
                uint32_t h[W / 2];
                with_act(f.act, [&](auto tag) {
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        const float2 gate = mul2(z(e), alpha);
                        const float2 up = mul2(make_float2(__uint_as_float(r2[e]), __uint_as_float(r2[e + 1])), alpha);
                        h[e / 2] = pack_bf16(mul2(act_value2<decltype(tag)::value>(gate), up));
                        r[e / 2] = pack_bf16(gate);
                        r2[e / 2] = pack_bf16(up);
                    }
                });
                store_rows<W>(f, 0, tm0, block, h, i0, j0, lane);
                if (f.out[1] != nullptr) {
#pragma unroll
                    for (int e = 0; e < W / 2; ++e) x0[e] = r[e], x1[e] = r2[e];
                    store_rows<W>(f, 1, tm1, final_unit ? spare(0) : block, x0, i0, j0, lane, final_unit);
                    store_rows<W>(f, 2, tm2, final_unit ? spare(1) : block, x1, i0, j0, lane, final_unit);
                }
            }
        }
    }
    if (!ok && lane == 0) signal_timeout(p, abort_flag);
    if (!ok && in_flight) spin_ns(100000);  // a copy may still land in the block
    if (lane == 0) bulk_wait_group0();      // shared memory must outlive the stores that read it
}

// ---------------------------------------------------------------- kernel
template <int BN, int STAGES, int PAIR, int KPS, int KIND>
__global__ void __launch_bounds__(FUSED_THREADS, 1)
    bm_gemm_epi_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tm0,
                       const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                       const __grid_constant__ CUtensorMap tmI0, const __grid_constant__ CUtensorMap tmI1, const EpiParams f)
{
    using Cfg = FusedCfg<BN, STAGES, PAIR, KPS>;
    constexpr int ELEM = kind_elem(KIND);
    constexpr int EPI = kind_symmetric(KIND) ? EPI_FULL : EPI_STORE;  // (which tile order run_mma has)
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
            mbar_init(bar0 + 8u * (2 * STAGES + b), 1);                           // accumulator full
            mbar_init(bar0 + 8u * (2 * STAGES + 2 + b), FUSED_EPI_WARPS * PAIR);  // accumulator empty
        }
        mbar_init(bar0 + 8u * (2 * STAGES + 4), 1);  // drain (abort path only)
        for (int e = 0; e < FUSED_EPI_WARPS; ++e) mbar_init(bar0 + 8u * (2 * STAGES + 5 + e), 1);  // a warp's inputs
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        if constexpr (KIND == KIND_GLU) tma_prefetch_map(&tmB2);
        if (f.tma[0]) tma_prefetch_map(&tm0);
        if (f.tma[1]) tma_prefetch_map(&tm1);
        if (f.tma[2]) tma_prefetch_map(&tm2);
        if constexpr (KIND == KIND_DGLU || KIND == KIND_STEP || KIND == KIND_POLY) tma_prefetch_map(&tmI0);
        if constexpr (KIND == KIND_DGLU || KIND == KIND_STEP) tma_prefetch_map(&tmI1);
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
    // as in bm_gemm_tcgen05_kernel: nothing in global memory is read or written before the
    // previous kernel on the stream is complete
    griddep_launch_dependents();
    griddep_wait();

    if (warp < FUSED_FIRST_EPI_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(EPI_MAIN_REGS));
        if (warp == 0 && lane == 0) {
            if constexpr (KIND == KIND_GLU)
                run_producer_glu<BN, STAGES, PAIR, KPS>(&tmA, &tmB, &tmB2, p, ring, bar0, rank, abort_flag);
            else
                run_producer<BN, STAGES, PAIR, ELEM, KPS, EPI>(&tmA, &tmB, &tmA, &tmB, p, ring, bar0, rank, abort_flag);
        }
        if (warp == 1 && rank == 0) run_mma<BN, STAGES, PAIR, ELEM, KPS, EPI>(p, ring, bar0, tmem_base, abort_flag, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_EPI_REGS));
        run_epilogue_kind<BN, STAGES, PAIR, KPS, KIND>(&tm0, &tm1, &tm2, &tmI0, &tmI1, f, bar0, tmem_base, smem, staging,
                                                       rank, abort_flag, warp, lane);
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

}  // namespace bm
