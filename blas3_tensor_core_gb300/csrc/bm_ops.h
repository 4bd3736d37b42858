// bm_ops.h -- host-side parts shared by the operators around the products: launches
// with programmatic dependent launch, and the final sum of partial column sums.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "bm.h"

namespace bmh {

// Launch configuration that lets a kernel's set-up overlap the previous kernel's tail
// (the kernels wait for it before they touch global memory). cluster > 0: CTAs per cluster.
struct PdlLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    PdlLaunch(cudaStream_t stream, unsigned blocks, unsigned threads, size_t smem = 0, int cluster = 0)
    {
        cfg.gridDim = dim3(blocks, 1, 1);
        cfg.blockDim = dim3(threads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
        if (cluster > 0) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
    }
    PdlLaunch(const PdlLaunch &) = delete;
};

inline bm_status launched(cudaError_t e)
{
    if (e == cudaSuccess) return BM_OK;
    cudaGetLastError();
    return BM_ERR_CUDA;
}

// out0[j] (+)= sum of partial[0 .. rows - 1][j], row stride ld; out1 (may be null) the
// same from partial + plane. In a fixed order. rows == 0 gives zeros.
bm_status launch_column_sums(const float *partial, int64_t rows, int64_t ld, int64_t plane, int64_t n, float *out0,
                             float *out1, int accumulate, cudaStream_t stream);

}  // namespace bmh
