// bm_host.h -- host-side parts shared by the library's translation units: the
// per-device state, the launch plan of the tiled products, the tensor-map
// encoders and small argument checks. Defined in bm_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "bm.h"
#include "bm_gemm_kernel.cuh"

namespace bmh {

constexpr int kMaxDevices = 64;
constexpr int kGroupM = 16;

// Kernel variants: output tile (rows x BN), ring depth, CTAs per tile, k-blocks per stage.
//   kSingle256: 128 x 256 per CTA, 4 stages of one k-block (48 KB)
//   kSingle128: 128 x 128 per CTA, 3 stages of two k-blocks (64 KB; narrow outputs)
//   kPair256:   256 x 256 per CTA pair (cta_group::2), 3 stages of two k-blocks (64 KB per CTA)
// MXFP8 (the scale factors take tensor-memory columns beside the accumulators):
//   kSingle128Mx: 128 x 128 per CTA, 5 stages of one k-block (33 KB with scales)
//   kPair128Mx:   256 x 128 per CTA pair, 3 stages of two k-blocks (50 KB per CTA)
//   kPair256Mx:   256 x 256 per CTA pair, 5 stages of one k-block (33.5 KB per CTA),
//                 one accumulator (two 256-column ones would fill the tensor memory)
enum Variant {
    kSingle256 = 0, kSingle128 = 1, kPair256 = 2, kSingle128Mx = 3, kPair128Mx = 4, kPair256Mx = 5, kNumVariants = 6
};
constexpr int kVariantBN[kNumVariants] = {256, 128, 256, 128, 128, 256};
constexpr int kVariantStages[kNumVariants] = {4, 3, 3, 5, 3, 5};
constexpr int kVariantStageKBlocks[kNumVariants] = {1, 2, 2, 1, 2, 1};
constexpr int kVariantPair[kNumVariants] = {1, 1, 2, 1, 2, 2};
inline bool variant_scaled(int v) { return v >= kSingle128Mx; }

struct DeviceState {
    bool ready = false;
    int sm_count = 0;
    int cc_major = 0, cc_minor = 0;
    int device = -1;
    int *status = nullptr;  // one int, allocated on first use
    bool attrs_set = false;
    int max_pair_clusters = 0;     // co-resident clusters of the pair kernel
    int max_pair_clusters_mx = 0;  // same for the MXFP8 pair kernels (the smaller of the two)
};

inline bool fits_int32(int64_t v) { return v >= 0 && v <= 0x7FFFFFFFLL; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Plan {
    int variant = kSingle256;
    int tile_m = bm::CTA_M, bn = 256, stages = 4, pair = 1;
    int64_t tiles_m = 0, tiles_n = 0, num_tiles = 0;
    int64_t full_tiles = 0, num_units = 0;  // whole tiles first; the rest are split k_splits ways
    int k_splits = 1, kb_per_split = 0, kb_total = 0;
    int n_split = 1;         // 2: the tiles after full_tiles run as two N halves each
    int ctas = 0;
    int fixup = 0;           // split tiles reduced inside the kernel (no reduce kernel)
    size_t slot_bytes = 0;   // partial slots at the start of the workspace; fixup counters follow
    size_t ws_bytes = 0;
};

// Current device, checked for compute capability 10.3, with the one-time set-up
// of its state. With `alloc_status` the device status word is allocated on first
// use; without it nothing is allocated and the word is used only if it exists.
bm_status device_state(DeviceState **out, bool alloc_status = true);

int sm_count_or_default();
int pair_clusters_or_default(int sms, bool mxfp8 = false);
int variant_smem(int v);
uint64_t wait_timeout_ns();  // bm_set_wait_timeout_ms's limit
int tile_override();  // bm_set_tile_override's variant, 0 = automatic

// Tensor maps (see the definitions).
bool encode_operand(CUtensorMap *map, const void *base, bool mn_major, int64_t rows, int64_t k, int64_t ld,
                    uint32_t tile_rows);
bool encode_stage_box(CUtensorMap *map, const void *base, int elem, bool mn_major, int64_t mn, int64_t k, int64_t ld,
                      int rows, int kps);
bool encode_box64(CUtensorMap *map, const void *X, bm_ctype t, int64_t m, int64_t n, int64_t ld);

Plan plan_gemm(int64_t m, int64_t n, int64_t k, size_t ws_bytes, int sms, int pair_clusters,
               int elem = bm::ELEM_BF16, bool beta_nonzero = false, int variant = -1);
void fill_params(bm::GemmParams &prm, const Plan &pl);
bm::GemmParams base_params(int64_t m, int64_t n, int64_t k, float alpha, float beta, void *C, int64_t ldc,
                           bm_ctype ct, DeviceState *st);
bm_status check_gemm_args(int64_t m, int64_t n, int64_t k, int transA, int transB, int64_t lda, int64_t ldb,
                          int64_t ldc, int ct);

}  // namespace bmh
