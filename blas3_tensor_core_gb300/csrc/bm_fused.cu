// bm_fused.cu -- host side of the products with an MLP's work in the epilogue
// (bm_gemm_bf16_bias_act, bm_gemm_bf16_dact): argument checks, plan, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "bm.h"
#include "bm_fused_kernel.cuh"
#include "bm_host.h"
#include "bm_ops.h"
#include "bm_skinny_kernel.cuh"

using namespace bmh;

namespace {

// Rows per partial column sum of the reduce kernel: its warps take this many rows.
constexpr int kReduceRows = 4;
constexpr int kTileRows = 32;  // the tile kernel's: one epilogue warp's rows

// Accumulator chunks when an output is FP32 or a checkpoint is kept. Relative error of
// the product in one piece: 1.1e-9 K (4.4e-6 at K = 4096), and of chunks of n_i k-blocks
// at most 7e-8 sqrt(sum n_i^3 / sum n_i). Two chunks of 16 and the rest of 8 keep it below
// 1e-6 from 48 k-blocks on and leave the epilogue 32 k-blocks of time; shorter K takes
// 12 and 12, then 8, and below 24 k-blocks equal parts of at most 12. A checkpoint's codes
// are nearest values, and the error decides how many fall on the other side of a tie. So
// beside a checkpoint long K too starts with 12 and 12 (4096 x 16384 x 4096: 343 us, and
// 337 with 16 and 16), and below 24 k-blocks the parts are of at most 6. Measured beside a
// checkpoint, and for an FP32 product of the same operands by a library: 2.3e-7 and 1.6e-7
// at K = 512, 3.3e-7 and 2.5e-7 at 1024, 7.3e-7 and 3.2e-7 at 1536 (parts of 8: 99 us for
// 4096 x 8192 there, and 94 with these), 6.7e-7 and 3.9e-7 at 2048, 5.8e-7 and 6.1e-7 at
// 4096, 5.4e-7 and 9.6e-7 at 8192. About 40 times the error is the share of codes that are
// a neighbour of the nearest value's: 2e-5 at K = 4096.
// Returns whether there is more than one.
bool set_chunks(bm::FusedParams &f, int kb, int stage_kb, bool precise, bool codes)
{
    int first = kb, rest = kb;
    if (precise && kb >= 24) {
        first = kb >= 48 && !codes ? 16 : 12;
        rest = 8;
    } else if (codes && kb > 2) {
        first = rest = std::min(6, (kb + 1) / 2);
    } else if (precise && kb > 12) {
        first = (kb + 1) / 2;
        rest = 8;
    }
    f.chunk_first = static_cast<int>(ceil_div(first, stage_kb)) * stage_kb;
    f.chunk_rest = static_cast<int>(ceil_div(rest, stage_kb)) * stage_kb;
    return f.chunk_first < kb;
}

using FusedKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, bm::FusedParams);

template <bool BWD, bool CHUNKED>
FusedKernel fused_kernel(int v)
{
    switch (v) {
    case kSingle256: return &bm::bm_gemm_fused_kernel<256, 4, 1, 1, BWD, CHUNKED>;
    case kSingle128: return &bm::bm_gemm_fused_kernel<128, 3, 1, 2, BWD, CHUNKED>;
    default: return &bm::bm_gemm_fused_kernel<256, 3, 2, 2, BWD, CHUNKED>;
    }
}

int fused_smem(int v)
{
    switch (v) {
    case kSingle256: return bm::FusedCfg<256, 4, 1, 1>::FUSED_SMEM;
    case kSingle128: return bm::FusedCfg<128, 3, 1, 2>::FUSED_SMEM;
    default: return bm::FusedCfg<256, 3, 2, 2>::FUSED_SMEM;
    }
}

// ---------------------------------------------------------------- few rows
// At most 128 rows; over 32 rows only while the columns leave SMs to split K over: with a
// tile of 128 columns for every other SM the tile kernel reads the weights as fast
// (64 x 16384 x 4096: 29.4 us, 31.3 here; 128 rows: 29.2 and 37.5; but 128 x 5120 x 5120:
// 28.6 and 18.4).
bool few_rows(int64_t m, int64_t n, int64_t k, int sms)
{
    return m <= 128 && k > 0 && tile_override() == 0 && (m <= 32 || 2 * ceil_div(n, 128) <= sms);
}

constexpr int kMaxCluster = 8;    // CTAs of a portable cluster

// The narrow side of the MMA: 16, 32, 64 or 128 rows. A stored [k, m] comes in 64-wide
// chunks of m.
int skinny_nt(int64_t m, bool a_mn)
{
    if (m <= 16 && !a_mn) return 16;
    if (m <= 32 && !a_mn) return 32;
    return m <= 64 ? 64 : 128;
}

template <bool BWD>
const void *skinny_kernel(int nt)
{
    switch (nt) {
    case 16: return reinterpret_cast<const void *>(&bm::bm_gemm_skinny_kernel<16, BWD>);
    case 32: return reinterpret_cast<const void *>(&bm::bm_gemm_skinny_kernel<32, BWD>);
    case 64: return reinterpret_cast<const void *>(&bm::bm_gemm_skinny_kernel<64, BWD>);
    default: return reinterpret_cast<const void *>(&bm::bm_gemm_skinny_kernel<128, BWD>);
    }
}

int skinny_smem(int nt)
{
    switch (nt) {
    case 16: return bm::SkinnyCfg<16>::SMEM_BYTES;
    case 32: return bm::SkinnyCfg<32>::SMEM_BYTES;
    case 64: return bm::SkinnyCfg<64>::SMEM_BYTES;
    default: return bm::SkinnyCfg<128>::SMEM_BYTES;
    }
}

// Clusters of S CTAs that fit on the device at once, per narrow side and S (written
// once per device, under the mutex).
struct SkinnyCapacity {
    int clusters[4][kMaxCluster + 1];
};
SkinnyCapacity g_skinny[kMaxDevices] = {};
int nt_index(int nt) { return nt == 16 ? 0 : nt == 32 ? 1 : nt == 64 ? 2 : 3; }

// K is split over as many CTAs (at most 8, a k-block each at least) as keep every cluster
// on the GPU at once; more columns than that take one CTA per 128 columns.
int skinny_cluster(const SkinnyCapacity &cap, int nt, int64_t tiles, int kb_total)
{
    for (int s = std::min(kMaxCluster, kb_total); s > 1; --s)
        if (tiles <= cap.clusters[nt_index(nt)][s]) return s;
    return 1;
}

std::mutex g_mutex;
bool g_attrs_set[kMaxDevices] = {};

// The chunked copies' warps share out the registers that the launch gave the block. With
// fewer than the split adds up to, the epilogue's increase would wait for ever: such a
// build is refused before its first launch.
bool register_split_fits(const void *fn)
{
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, fn) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.numRegs >= bm::FUSED_LAUNCH_REGS;
}

// Once per device: the dynamic shared-memory size of every kernel copy.
bm_status fused_attrs(const DeviceState &st)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_attrs_set[st.device]) return BM_OK;
    for (int v : {kSingle256, kSingle128, kPair256})
        for (FusedKernel fn :
             {fused_kernel<false, false>(v), fused_kernel<false, true>(v), fused_kernel<true, false>(v), fused_kernel<true, true>(v)})
            if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, fused_smem(v)) != cudaSuccess) {
                cudaGetLastError();
                return BM_ERR_CUDA;
            }
    for (int v : {kSingle256, kSingle128, kPair256})
        for (FusedKernel fn : {fused_kernel<false, true>(v), fused_kernel<true, true>(v)})
            if (!register_split_fits(reinterpret_cast<const void *>(fn))) return BM_ERR_CUDA;
    for (int nt : {16, 32, 64, 128}) {
        for (const void *fn : {skinny_kernel<false>(nt), skinny_kernel<true>(nt)})
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, skinny_smem(nt)) != cudaSuccess) {
                cudaGetLastError();
                return BM_ERR_CUDA;
            }
        for (int s = 1; s <= kMaxCluster; ++s) {
            PdlLaunch l(nullptr, static_cast<unsigned>(s * st.sm_count), bm::SKINNY_THREADS,
                        static_cast<size_t>(skinny_smem(nt)), s);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, skinny_kernel<true>(nt), &l.cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            g_skinny[st.device].clusters[nt_index(nt)][s] = n;
        }
    }
    g_attrs_set[st.device] = true;
    return BM_OK;
}

// The GEMM planner's tiles, but for three things that an epilogue changes.
// Tiles of a last wave run whole or as N halves: the epilogue needs whole sums, so they
// are not split along K.
// Where all 128 x 128 tiles run at once on single SMs, those: with one wave nothing hides a
// tile's epilogue, so a tile of half the columns ends sooner (777 x 1320 x 520, backward
// with column sums: 18.0 -> 12.6 us). Every tile is split along K only where that saves
// more than the partial sums cost, about 6 us and their bytes twice at 5 TB/s (with SiLU
// and a residual, split and not: 512 x 512 x 4096 17.4 and about 22 us, 1024 x 1024 x 2048
// 22.3 and 13.9, 256 x 4096 x 2048 23.5 and 13.9). A k-block takes about 0.22 us on a
// 128 x 128 tile and 0.3 on the wider ones.
// Short K in several waves takes 128 x 128 tiles too: the epilogue is the longer part
// (2048 x 5120 x 256: 22.6 -> 19.9 us, 300 x 16384 x 256: 15.6 -> 13.2).
Plan plan_fused(int64_t m, int64_t n, int64_t k, size_t ws_bytes, int sms, int pair_clusters)
{
    const Plan whole = plan_gemm(m, n, k, 0, sms, pair_clusters);
    const int64_t tiles128 = ceil_div(m, 128) * ceil_div(n, 128);
    const int64_t slots = whole.pair == 2 ? pair_clusters : sms;
    if (whole.num_tiles * 2 <= slots && ws_bytes > 0) {
        const Plan split = plan_gemm(m, n, k, ws_bytes, sms, pair_clusters);
        const double saved = 0.22 * split.kb_total - 0.3 * split.kb_per_split;
        const double cost = 6.0 + 8.0 * static_cast<double>(m) * static_cast<double>(n) * split.k_splits / 5e6;
        if (split.k_splits > 1 && (saved > cost || tile_override() != 0)) return split;
    }
    const bool several_waves = whole.variant == kSingle256 && whole.num_tiles > sms;
    return tiles128 <= sms || several_waves ? plan_gemm(m, n, k, 0, sms, pair_clusters, bm::ELEM_BF16, false, kSingle128)
                                            : whole;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

int64_t colsum_ld(int64_t n) { return (n + 3) / 4 * 4; }

size_t colsum_bytes(int64_t m, int64_t n, int rows)
{
    return round256(static_cast<size_t>(ceil_div(m, rows)) * colsum_ld(n) * sizeof(float));
}

// Reduce kernel: partial slots (or nothing) -> epilogue.
template <bool BWD>
bm_status launch_reduce(const Plan &pl, const bm::FusedParams &f, cudaStream_t stream, int sms)
{
    const int64_t rows = !BWD && f.Q != nullptr ? ceil_div(f.g.m, 128) * 128 : f.g.m;
    const int64_t items = ceil_div(rows, f.row_block) * ceil_div(f.g.n, 128);
    PdlLaunch l(stream, static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(items, 8), 8 * static_cast<int64_t>(sms)))), 256);
    cudaError_t e;
    if (pl.variant == kSingle128) e = cudaLaunchKernelEx(&l.cfg, bm::bm_fused_reduce_kernel<128, 128, BWD>, f);
    else if (pl.variant == kSingle256) e = cudaLaunchKernelEx(&l.cfg, bm::bm_fused_reduce_kernel<128, 256, BWD>, f);
    else e = cudaLaunchKernelEx(&l.cfg, bm::bm_fused_reduce_kernel<256, 256, BWD>, f);
    return launched(e);
}

struct Call {
    int64_t m, n, k;
    int ta, tb;
    float alpha;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    void *C;
    int64_t ldc;
    bm_ctype ct;
    int act;
    void *ws;
    size_t ws_bytes;
    cudaStream_t stream;
};

bm_status check_call(const Call &c, const void *Q, int64_t ldq, const void *S)
{
    const bm_status s = check_gemm_args(c.m, c.n, c.k, c.ta, c.tb, c.lda, c.ldb, c.ldc, c.ct);
    if (s != BM_OK) return s;
    if (c.act < BM_ACT_NONE || c.act > BM_ACT_SILU) return BM_ERR_INVALID_VALUE;
    if (ldq < 0 || (Q != nullptr && ldq < std::max<int64_t>(1, c.n))) return BM_ERR_INVALID_VALUE;
    if (c.ws_bytes > 0 && (c.ws == nullptr || (reinterpret_cast<uintptr_t>(c.ws) & 255u) != 0)) return BM_ERR_WORKSPACE;
    return BM_OK;
}

bm_status check_pointers(const Call &c, bool products, const void *Q, int64_t ldq, const void *S)
{
    if (c.C == nullptr || (products && (c.A == nullptr || c.B == nullptr))) return BM_ERR_INVALID_VALUE;
    if ((Q == nullptr) != (S == nullptr)) return BM_ERR_INVALID_VALUE;
    const int64_t esz = c.ct == BM_C_BF16 ? 2 : 4;
    if (!aligned16(c.C) || (c.ldc * esz) % 16 != 0) return BM_ERR_MISALIGNED;
    if (products && (!aligned16(c.A) || !aligned16(c.B) || (c.lda * 2) % 16 != 0 || (c.ldb * 2) % 16 != 0))
        return BM_ERR_MISALIGNED;
    if (Q != nullptr && (!aligned16(Q) || !aligned16(S) || ldq % 16 != 0)) return BM_ERR_MISALIGNED;
    return BM_OK;
}

// Few rows: one launch, everything in it (the column sums too).
template <bool BWD>
bm_status run_skinny(const Call &c, bm::FusedParams &f, DeviceState *st, float *dbias, int accumulate)
{
    bm::SkinnyParams sp;
    std::memset(&sp, 0, sizeof(sp));
    f.g = base_params(c.m, c.n, c.k, c.alpha, 0.0f, c.C, c.ldc, c.ct, st);
    f.katoms = ceil_div(c.n, 128);
    f.g.kb_total = static_cast<int>(ceil_div(c.k, bm::TILE_K));
    const bool a_mn = c.ta == BM_OP_T, b_mn = c.tb == BM_OP_N;
    f.g.a_mn_major = a_mn;
    f.g.b_mn_major = b_mn;
    const int nt = skinny_nt(c.m, a_mn);
    CUtensorMap tw, tx;
    if (!encode_operand(&tw, c.B, b_mn, c.n, c.k, c.ldb, 128)) return BM_ERR_CUDA;
    if (!encode_operand(&tx, c.A, a_mn, c.m, c.k, c.lda, static_cast<uint32_t>(nt))) return BM_ERR_CUDA;
    const int64_t tiles = ceil_div(c.n, 128);
    sp.f = f;
    sp.cluster = skinny_cluster(g_skinny[st->device], nt, tiles, f.g.kb_total);
    // (longer chunks where a CTA's share of K would not fit its TMEM columns)
    const int kb_cta = static_cast<int>(ceil_div(f.g.kb_total, sp.cluster)), most = bm::SKINNY_TMEM_COLS / nt;
    // (4 k-blocks for a checkpoint, as in set_chunks)
    sp.chunk_kb = std::max(f.Q != nullptr && !BWD ? 4 : 8, static_cast<int>(ceil_div(kb_cta, most)));
    sp.tmem_cols = 32;
    while (sp.tmem_cols < ceil_div(kb_cta, sp.chunk_kb) * nt) sp.tmem_cols *= 2;
    sp.dbias = dbias;
    sp.accumulate = accumulate;
    PdlLaunch l(c.stream, static_cast<unsigned>(tiles * sp.cluster), bm::SKINNY_THREADS,
                static_cast<size_t>(skinny_smem(nt)), sp.cluster);
    switch (nt) {
    case 16: return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_gemm_skinny_kernel<16, BWD>, tw, tx, sp));
    case 32: return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_gemm_skinny_kernel<32, BWD>, tw, tx, sp));
    case 64: return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_gemm_skinny_kernel<64, BWD>, tw, tx, sp));
    default: return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_gemm_skinny_kernel<128, BWD>, tw, tx, sp));
    }
}

// Plan, maps and launches of one call; f holds the epilogue's operands. `partial_ws`:
// where split slots may go.
template <bool BWD>
bm_status run(const Call &c, bm::FusedParams &f, DeviceState *st, bool products, void *slots_ws, size_t slots_bytes)
{
    const Plan pl = plan_fused(c.m, c.n, products ? c.k : 1, products ? slots_bytes : 0, st->sm_count, st->max_pair_clusters);
    f.g = base_params(c.m, c.n, c.k, c.alpha, 0.0f, c.C, c.ldc, c.ct, st);
    f.g.mode = bm::MODE_GEMM;
    fill_params(f.g, pl);
    f.katoms = ceil_div(c.n, 128);
    if (!products) {
        f.g.k_splits = 0;
        f.row_block = BWD && f.colsum != nullptr ? kTileRows : kReduceRows;
        return launch_reduce<BWD>(pl, f, c.stream, st->sm_count);
    }
    bm_status s = fused_attrs(*st);
    if (s != BM_OK) return s;
    CUtensorMap ta, tb;
    const bool a_mn = c.ta == BM_OP_T, b_mn = c.tb == BM_OP_N;
    if (!encode_operand(&ta, c.A, a_mn, c.m, c.k, c.lda, bm::CTA_M)) return BM_ERR_CUDA;
    if (!encode_operand(&tb, c.B, b_mn, c.n, c.k, c.ldb, static_cast<uint32_t>(pl.bn / pl.pair))) return BM_ERR_CUDA;
    f.g.a_mn_major = a_mn;
    f.g.b_mn_major = b_mn;
    const int kps = kVariantStageKBlocks[pl.variant];
    f.g.a_box3 = encode_stage_box(&ta, c.A, bm::ELEM_BF16, a_mn, c.m, c.k, c.lda, bm::CTA_M, kps);
    f.g.b_box3 = encode_stage_box(&tb, c.B, bm::ELEM_BF16, b_mn, c.n, c.k, c.ldb, pl.bn / pl.pair, kps);
    f.g.partial = pl.k_splits > 1 ? static_cast<float *>(slots_ws) : nullptr;
    // (a checkpoint beside a BF16 C in one piece: 343 us instead of 376 at 4096 x 16384 x 4096
    // with GELU, and five times as many codes on the other side of a tie)
    const bool codes = !BWD && f.Q != nullptr, precise = c.ct == BM_C_F32 || f.colsum != nullptr || codes;
    CUtensorMap tc, tr;
    std::memset(&tc, 0, sizeof(tc));
    std::memset(&tr, 0, sizeof(tr));
    f.g.tma_c = (c.n * (c.ct == BM_C_BF16 ? 2 : 4)) % 16 == 0 && encode_box64(&tc, c.C, c.ct, c.m, c.n, c.ldc);
    if (f.R != nullptr && !encode_box64(&tr, f.R, c.ct, c.m, c.n, f.ldr)) return BM_ERR_CUDA;
    const bool chunked = set_chunks(f, pl.k_splits > 1 ? pl.kb_per_split : pl.kb_total, kps, precise, codes);
    f.row_block = pl.k_splits > 1 ? kReduceRows : kTileRows;

    PdlLaunch l(c.stream, static_cast<unsigned>(pl.ctas), bm::FUSED_THREADS, static_cast<size_t>(fused_smem(pl.variant)),
                pl.pair == 2 ? 2 : 0);
    FusedKernel fn = chunked ? fused_kernel<BWD, true>(pl.variant) : fused_kernel<BWD, false>(pl.variant);
    s = launched(cudaLaunchKernelEx(&l.cfg, fn, ta, tb, tc, tr, f));
    if (s != BM_OK || pl.k_splits == 1) return s;
    return launch_reduce<BWD>(pl, f, c.stream, st->sm_count);
}

}  // namespace

extern "C" {

bm_status bm_gemm_bf16_bias_act(int64_t m, int64_t n, int64_t k, bm_op transA, bm_op transB, float alpha, const void *A,
                                int64_t lda, const void *B, int64_t ldb, const void *bias, bm_dtype bias_type,
                                bm_act act, const void *R, int64_t ldr, void *C, int64_t ldc, bm_ctype c_type, void *Q,
                                int64_t ldq, void *S, void *workspace, size_t workspace_bytes, bm_stream_t stream)
{
    const Call c = {m,  n,   k,      transA, transB,    alpha,           A, lda, B, ldb, C, ldc, c_type,
                    act, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream)};
    bm_status s = check_call(c, Q, ldq, S);
    if (s != BM_OK) return s;
    if (bias_type != BM_F32 && bias_type != BM_BF16) return BM_ERR_INVALID_VALUE;
    if (R != nullptr && ldr < std::max<int64_t>(1, n)) return BM_ERR_INVALID_VALUE;
    if (m == 0 || n == 0) return BM_OK;
    const bool products = alpha != 0.0f && k > 0;
    s = check_pointers(c, products, Q, ldq, S);
    if (s != BM_OK) return s;
    const int64_t esz = c_type == BM_C_BF16 ? 2 : 4;
    if (!aligned16(bias) || !aligned16(R) || (R != nullptr && (ldr * esz) % 16 != 0)) return BM_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    s = device_state(&st);
    if (s != BM_OK) return s;
    bm::FusedParams f;
    std::memset(&f, 0, sizeof(f));
    f.bias = bias;
    f.bias_bf16 = bias_type == BM_BF16;
    f.act = act;
    f.R = R;
    f.ldr = ldr;
    f.Q = static_cast<uint8_t *>(Q);
    f.ldq = ldq;
    f.S = static_cast<uint8_t *>(S);
    if (products && few_rows(m, n, k, st->sm_count)) {
        s = fused_attrs(*st);
        return s == BM_OK ? run_skinny<false>(c, f, st, nullptr, 0) : s;
    }
    return run<false>(c, f, st, products, workspace, workspace != nullptr ? workspace_bytes : 0);
}

size_t bm_gemm_bf16_bias_act_workspace_size(int64_t m, int64_t n, int64_t k)
{
    const int sms = sm_count_or_default();
    if (m <= 0 || n <= 0 || k <= 0 || few_rows(m, n, k, sms)) return 0;
    const Plan pl = plan_fused(m, n, k, SIZE_MAX, sms, pair_clusters_or_default(sms));
    return pl.k_splits > 1 ? pl.ws_bytes : 0;
}

bm_status bm_gemm_bf16_dact(int64_t m, int64_t n, int64_t k, bm_op transA, bm_op transB, float alpha, const void *A,
                            int64_t lda, const void *B, int64_t ldb, const void *Q, int64_t ldq, const void *S,
                            bm_act act, void *C, int64_t ldc, bm_ctype c_type, float *dbias, int accumulate,
                            void *workspace, size_t workspace_bytes, bm_stream_t stream)
{
    const Call c = {m,  n,   k,      transA, transB,    alpha,           A, lda, B, ldb, C, ldc, c_type,
                    act, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream)};
    bm_status s = check_call(c, Q, ldq, S);
    if (s != BM_OK) return s;
    if (n == 0 || (m == 0 && (dbias == nullptr || accumulate != 0))) return BM_OK;
    if (m > 0 && Q == nullptr) return BM_ERR_INVALID_VALUE;
    if (!aligned16(dbias)) return BM_ERR_MISALIGNED;
    const bool products = alpha != 0.0f && k > 0;
    if (m > 0) s = check_pointers(c, products, Q, ldq, S);
    if (s != BM_OK) return s;
    const size_t ws = workspace != nullptr ? workspace_bytes : 0;
    const size_t least = dbias != nullptr ? colsum_bytes(m, n, kTileRows) : 0;
    if (ws < least) return BM_ERR_WORKSPACE;
    DeviceState *st = nullptr;
    s = device_state(&st);
    if (s != BM_OK) return s;
    bm::FusedParams f;
    std::memset(&f, 0, sizeof(f));
    f.act = act;
    f.Q = static_cast<uint8_t *>(const_cast<void *>(Q));
    f.ldq = ldq;
    f.S = static_cast<uint8_t *>(const_cast<void *>(S));
    f.colsum = dbias != nullptr ? static_cast<float *>(workspace) : nullptr;
    f.ld_colsum = colsum_ld(n);
    if (m > 0 && products && few_rows(m, n, k, st->sm_count)) {
        s = fused_attrs(*st);
        return s == BM_OK ? run_skinny<true>(c, f, st, dbias, accumulate) : s;
    }
    if (m > 0) {
        // split slots go after the partial column sums of the split plan, where both fit
        const size_t sums = dbias != nullptr ? colsum_bytes(m, n, kReduceRows) : 0;
        s = run<true>(c, f, st, products, static_cast<char *>(workspace) + sums, ws > sums ? ws - sums : 0);
        if (s != BM_OK || dbias == nullptr) return s;
    } else {
        f.row_block = kTileRows;
    }
    return launch_column_sums(f.colsum, ceil_div(m, f.row_block), f.ld_colsum, 0, n, dbias, nullptr, accumulate,
                              c.stream);
}

size_t bm_gemm_bf16_dact_workspace_size(int64_t m, int64_t n, int64_t k, int dbias)
{
    if (m <= 0 || n <= 0) return 0;
    const int sms = sm_count_or_default();
    const Plan pl = plan_fused(m, n, std::max<int64_t>(k, 1), SIZE_MAX, sms, pair_clusters_or_default(sms));
    const size_t slots = k > 0 && pl.k_splits > 1 && !few_rows(m, n, k, sms) ? pl.ws_bytes : 0;
    if (!dbias) return slots;
    return slots > 0 ? colsum_bytes(m, n, kReduceRows) + slots : colsum_bytes(m, n, kTileRows);
}

}  // extern "C"
