// bm_glu.cu -- host side of a gated MLP's products (bm_gemm_bf16_glu, bm_gemm_bf16_dglu):
// argument checks, tiles, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "bm.h"
#include "bm_epi.h"
#include "bm_glu_skinny_kernel.cuh"
#include "bm_host.h"
#include "bm_ops.h"

using namespace bmh;

namespace bm {

// What the two products leave when they are 0 (alpha == 0 or k == 0): zeros, and DGLU's
// H = act(G) . U. Eight columns of a row per thread.
template <bool BWD>
__global__ void __launch_bounds__(256) bm_glu_zero_kernel(const EpiParams f)
{
    griddep_launch_dependents();
    griddep_wait();
    const GemmParams &p = f.g;
    const int64_t vecs = (p.n + 7) / 8, total = p.m * vecs, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; t < total; t += step) {
        const int64_t i = t / vecs, j = (t - i * vecs) * 8;
        uint32_t h[4] = {0u, 0u, 0u, 0u};
        if (BWD && f.out[2] != nullptr) {
            uint32_t g[4], u[4];
            load_row<8>(f.in[0], f.ldin[0], i, p.m, j, p.n, g);
            load_row<8>(f.in[1], f.ldin[1], i, p.m, j, p.n, u);
            with_act(f.act, [&](auto tag) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = pack_bf16(mul2(act_pair2<decltype(tag)::value>(bf16_pair(g[e])).value, bf16_pair(u[e])));
            });
        }
#pragma unroll
        for (int o = 0; o < 3; ++o) {
            if (f.out[o] == nullptr) continue;
            uint16_t *dst = static_cast<uint16_t *>(f.out[o]) + i * f.ldout[o] + j;
            const bool kept = BWD && o == 2;
            if (j + 8 <= p.n) {
                *reinterpret_cast<uint4 *>(dst) = kept ? make_uint4(h[0], h[1], h[2], h[3]) : make_uint4(0u, 0u, 0u, 0u);
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (j + e < p.n) dst[e] = kept ? static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1))) : uint16_t(0);
            }
        }
    }
}

}  // namespace bm

namespace {

// ---------------------------------------------------------------- few rows
constexpr int kMaxCluster = 8;  // CTAs of a portable cluster

using GluSkinny = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, bm::GluSkinnyParams);

template <int KIND>
GluSkinny skinny_kernel(int nt)
{
    switch (nt) {
    case 16: return &bm::bm_glu_skinny_kernel<16, KIND>;
    case 32: return &bm::bm_glu_skinny_kernel<32, KIND>;
    case 64: return &bm::bm_glu_skinny_kernel<64, KIND>;
    default: return &bm::bm_glu_skinny_kernel<128, KIND>;
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

// The narrow side of the MMA. A stored [k, m] comes in 64-wide chunks of m.
int skinny_nt(int64_t m, bool a_mn)
{
    if (m <= 16 && !a_mn) return 16;
    if (m <= 32 && !a_mn) return 32;
    return m <= 64 ? 64 : 128;
}

int nt_index(int nt) { return nt == 16 ? 0 : nt == 32 ? 1 : nt == 64 ? 2 : 3; }

// At most 128 rows while the tiles leave SMs to split K over; at most 32 while there is an SM
// for each tile, and for the backward product, whose tiles are as wide as the tile kernel's,
// whatever their number; at most 8 in any case. Few rows' kernel and tile kernel, us:
//   forward  128 x 4096 x 4096 20.2 and 22.4, 128 x 5120 x 4096 30.5 and 23.2; 32 x 9728 x 4096 29.0
//            and 29.5, 32 x 12288 x 4096 49.4 and 38.0, 8 x 12288 x 4096 46.6 and 56.0, 1 x 9728 x
//            4096 27.7 and 45.3, 1 x 16384 x 4096 48.0 and 61.0
//   backward 128 x 9728 x 4096 26.9 and 28.9, 128 x 12288 x 4096 40.9 and 31.0; 32 x 16384 x 4096 27.6
//            and 31.7, 1 x 16384 x 4096 24.0 and 45.8
bool few_rows(bool forward, int64_t m, int64_t tiles, int sms)
{
    if (tile_override() != 0) return false;
    return m <= 8 || (m <= 32 && (!forward || tiles <= sms)) || (m <= 128 && 2 * tiles <= sms);
}

std::mutex g_mutex;
bool g_attrs_set[kMaxDevices] = {};
int g_clusters[kMaxDevices][4][kMaxCluster + 1];  // clusters of S CTAs that fit at once, per narrow side and S

bm_status glu_attrs(const DeviceState &st)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_attrs_set[st.device]) return BM_OK;
    if (!epi_attrs<bm::KIND_GLU>() || !epi_attrs<bm::KIND_DGLU>()) return BM_ERR_CUDA;
    for (int nt : {16, 32, 64, 128}) {
        for (GluSkinny fn : {skinny_kernel<bm::KIND_GLU>(nt), skinny_kernel<bm::KIND_DGLU>(nt)})
            if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     skinny_smem(nt)) != cudaSuccess) {
                cudaGetLastError();
                return BM_ERR_CUDA;
            }
        for (int s = 1; s <= kMaxCluster; ++s) {
            PdlLaunch l(nullptr, static_cast<unsigned>(s * st.sm_count), bm::SKINNY_THREADS,
                        static_cast<size_t>(skinny_smem(nt)), s);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void *>(skinny_kernel<bm::KIND_DGLU>(nt)),
                                               &l.cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            g_clusters[st.device][nt_index(nt)][s] = n;
        }
    }
    g_attrs_set[st.device] = true;
    return BM_OK;
}

// K over as many CTAs (at most 8, a k-block each at least) as keep every cluster on the GPU
// at once.
template <int KIND>
bm_status run_skinny(bm::EpiParams &f, const void *A, bool a_mn, int64_t lda, const void *B, int64_t ldb, const void *B2,
                     int64_t ldb2, bool b_mn, const DeviceState &st, cudaStream_t stream)
{
    const int64_t m = f.g.m, n = f.g.n, k = f.g.k;
    const int nt = skinny_nt(m, a_mn), rows = KIND == bm::KIND_GLU ? 64 : 128;
    const int64_t tiles = ceil_div(n, rows);
    f.g.kb_total = static_cast<int>(ceil_div(k, bm::TILE_K));
    f.g.a_mn_major = a_mn;
    f.g.b_mn_major = b_mn;
    CUtensorMap tw, tw2, tx;
    if (!encode_operand(&tw, B, b_mn, n, k, ldb, static_cast<uint32_t>(rows)) ||
        !encode_operand(&tw2, B2, b_mn, n, k, ldb2, static_cast<uint32_t>(rows)) ||
        !encode_operand(&tx, A, a_mn, m, k, lda, static_cast<uint32_t>(nt)))
        return BM_ERR_CUDA;
    bm::GluSkinnyParams sp;
    sp.f = f;
    sp.cluster = 1;
    for (int s = std::min(kMaxCluster, f.g.kb_total); s > 1; --s)
        if (tiles <= g_clusters[st.device][nt_index(nt)][s]) {
            sp.cluster = s;
            break;
        }
    PdlLaunch l(stream, static_cast<unsigned>(tiles * sp.cluster), bm::SKINNY_THREADS, static_cast<size_t>(skinny_smem(nt)),
                sp.cluster);
    return launched(cudaLaunchKernelEx(&l.cfg, skinny_kernel<KIND>(nt), tw, tw2, tx, sp));
}

Plan plan_glu(int64_t m, int64_t n, int64_t k, const DeviceState &st)
{
    const int v = epi_variant(m, n, k, st.sm_count, st.max_pair_clusters);
    return epi_plan(v, m, n, k, false, st.sm_count, st.max_pair_clusters);
}

bool row_ok(const void *X, int64_t ld) { return aligned16(X) && (ld * 2) % 16 == 0; }

template <bool BWD>
bm_status launch_zero(const bm::EpiParams &f, cudaStream_t stream, int sms)
{
    const int64_t blocks = std::min<int64_t>(ceil_div(f.g.m * ceil_div(f.g.n, 8), 256), 8 * static_cast<int64_t>(sms));
    PdlLaunch l(stream, static_cast<unsigned>(blocks), 256);
    return launched(cudaLaunchKernelEx(&l.cfg, bm::bm_glu_zero_kernel<BWD>, f));
}

}  // namespace

extern "C" {

bm_status bm_gemm_bf16_glu(int64_t m, int64_t n, int64_t k, bm_op transA, bm_op transB, float alpha, const void *A,
                           int64_t lda, const void *BG, int64_t ldbg, const void *BU, int64_t ldbu, bm_act act, void *H,
                           int64_t ldh, void *G, int64_t ldg, void *U, int64_t ldu, bm_stream_t stream)
{
    bm_status s = check_gemm_args(m, n, k, transA, transB, lda, ldbg, ldh, BM_BF16);
    if (s != BM_OK) return s;
    const int64_t need_b = transB == BM_OP_N ? n : k;
    if (ldbu < std::max<int64_t>(1, need_b) || !fits_int32(2 * n)) return BM_ERR_INVALID_VALUE;
    if (act < BM_ACT_NONE || act > BM_ACT_SILU) return BM_ERR_INVALID_VALUE;
    if ((G == nullptr) != (U == nullptr)) return BM_ERR_INVALID_VALUE;
    if (G != nullptr && (ldg < std::max<int64_t>(1, n) || ldu < std::max<int64_t>(1, n))) return BM_ERR_INVALID_VALUE;
    if (m == 0 || n == 0) return BM_OK;
    const bool products = alpha != 0.0f && k > 0;
    if (H == nullptr || (products && (A == nullptr || BG == nullptr || BU == nullptr))) return BM_ERR_INVALID_VALUE;
    if (!row_ok(H, ldh) || (G != nullptr && (!row_ok(G, ldg) || !row_ok(U, ldu)))) return BM_ERR_MISALIGNED;
    if (products && (!row_ok(A, lda) || !row_ok(BG, ldbg) || !row_ok(BU, ldbu))) return BM_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    s = device_state(&st);
    if (s != BM_OK) return s;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    bm::EpiParams f;
    std::memset(&f, 0, sizeof(f));
    f.g = base_params(m, n, k, alpha, 0.0f, H, ldh, BM_BF16, st);
    f.act = act;
    epi_output(f, 0, H, ldh);
    epi_output(f, 1, G, ldg);
    epi_output(f, 2, U, ldu);
    if (!products) return launch_zero<false>(f, cs, st->sm_count);
    s = glu_attrs(*st);
    if (s != BM_OK) return s;
    const bool a_mn = transA == BM_OP_T, b_mn = transB == BM_OP_N;
    if (few_rows(true, m, ceil_div(n, 64), st->sm_count))
        return run_skinny<bm::KIND_GLU>(f, A, a_mn, lda, BG, ldbg, BU, ldbu, b_mn, *st, cs);
    const Plan pl = plan_glu(m, 2 * n, k, *st);
    fill_params(f.g, pl);
    f.g.a_mn_major = a_mn;
    f.g.b_mn_major = b_mn;
    EpiMaps t;
    epi_output_maps(f, t, m, n);
    // (a tile's columns follow those of H: the two weights have bn / 2 rows of it each)
    const int kps = kVariantStageKBlocks[pl.variant], rows = pl.bn / 2;
    if (!epi_operand(&t.a, &f.g.a_box3, A, a_mn, m, k, lda, bm::CTA_M, kps)) return BM_ERR_CUDA;
    // (a K-major stage box of several k-blocks holds one weight's rows only: SM pairs. Both
    // weights have one or neither)
    f.g.b_box3 = (b_mn || pl.pair == 2) && encode_stage_box(&t.b, BG, bm::ELEM_BF16, b_mn, n, k, ldbg, rows, kps) &&
                         encode_stage_box(&t.b2, BU, bm::ELEM_BF16, b_mn, n, k, ldbu, rows, kps)
                     ? 1
                     : 0;
    if (!f.g.b_box3 && (!encode_operand(&t.b, BG, b_mn, n, k, ldbg, static_cast<uint32_t>(rows)) ||
                        !encode_operand(&t.b2, BU, b_mn, n, k, ldbu, static_cast<uint32_t>(rows))))
        return BM_ERR_CUDA;
    return epi_launch<bm::KIND_GLU>(pl, t, f, cs);
}

bm_status bm_gemm_bf16_dglu(int64_t m, int64_t n, int64_t k, bm_op transA, bm_op transB, float alpha, const void *A,
                            int64_t lda, const void *B, int64_t ldb, const void *G, int64_t ldg, const void *U, int64_t ldu,
                            bm_act act, void *dG, int64_t lddg, void *dU, int64_t lddu, void *H, int64_t ldh,
                            bm_stream_t stream)
{
    bm_status s = check_gemm_args(m, n, k, transA, transB, lda, ldb, lddg, BM_BF16);
    if (s != BM_OK) return s;
    if (act < BM_ACT_NONE || act > BM_ACT_SILU) return BM_ERR_INVALID_VALUE;
    const int64_t least = std::max<int64_t>(1, n);
    if (ldg < least || ldu < least || lddu < least || (H != nullptr && ldh < least)) return BM_ERR_INVALID_VALUE;
    if (m == 0 || n == 0) return BM_OK;
    const bool products = alpha != 0.0f && k > 0;
    if (G == nullptr || U == nullptr || dG == nullptr || dU == nullptr) return BM_ERR_INVALID_VALUE;
    if (products && (A == nullptr || B == nullptr)) return BM_ERR_INVALID_VALUE;
    if (!row_ok(G, ldg) || !row_ok(U, ldu) || !row_ok(dG, lddg) || !row_ok(dU, lddu)) return BM_ERR_MISALIGNED;
    if (H != nullptr && !row_ok(H, ldh)) return BM_ERR_MISALIGNED;
    if (products && (!row_ok(A, lda) || !row_ok(B, ldb))) return BM_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    s = device_state(&st);
    if (s != BM_OK) return s;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    bm::EpiParams f;
    std::memset(&f, 0, sizeof(f));
    f.g = base_params(m, n, k, alpha, 0.0f, dG, lddg, BM_BF16, st);
    f.act = act;
    f.in[0] = G;
    f.ldin[0] = ldg;
    f.in[1] = U;
    f.ldin[1] = ldu;
    epi_output(f, 0, dG, lddg);
    epi_output(f, 1, dU, lddu);
    epi_output(f, 2, H, ldh);
    if (!products) return launch_zero<true>(f, cs, st->sm_count);
    s = glu_attrs(*st);
    if (s != BM_OK) return s;
    const bool a_mn = transA == BM_OP_T, b_mn = transB == BM_OP_N;
    if (few_rows(false, m, ceil_div(n, 128), st->sm_count))
        return run_skinny<bm::KIND_DGLU>(f, A, a_mn, lda, B, ldb, B, ldb, b_mn, *st, cs);
    const Plan pl = plan_glu(m, n, k, *st);
    fill_params(f.g, pl);
    f.g.a_mn_major = a_mn;
    f.g.b_mn_major = b_mn;
    EpiMaps t;
    epi_output_maps(f, t, m, n);
    const int kps = kVariantStageKBlocks[pl.variant];
    if (!epi_operand(&t.a, &f.g.a_box3, A, a_mn, m, k, lda, bm::CTA_M, kps) ||
        !epi_operand(&t.b, &f.g.b_box3, B, b_mn, n, k, ldb, pl.bn / pl.pair, kps) ||
        !encode_box64(&t.in[0], G, BM_BF16, m, n, ldg) || !encode_box64(&t.in[1], U, BM_BF16, m, n, ldu))
        return BM_ERR_CUDA;
    return epi_launch<bm::KIND_DGLU>(pl, t, f, cs);
}

}  // extern "C"
