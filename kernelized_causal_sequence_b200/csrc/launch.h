// launch.h — kernel launch helpers of the softmax operators' host code.
#pragma once
#include <cuda_runtime.h>

#include "errors.h"
#include "tc_launch.h"

namespace la {

// Launches kern on st, with programmatic stream serialisation when pdl is set
// (the kernel may start launching while the previous one in the stream ends;
// it must call pdl_wait before its first access to that kernel's memory), in
// clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
la_status launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl,
                         int cluster, const char *what, Args... args) {
    if (smem > 48 * 1024) {
        la_status s = cuda_check(what, cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (s != LA_OK) return s;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
    count_launches(1);
    if (err != cudaSuccess) return cuda_fail(what, err);
    return cuda_check(what, cudaGetLastError());
}

template <typename... KArgs, typename... Args>
la_status launch_kernel(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl,
                        const char *what, Args... args) {
    return launch_cluster(kern, grid, block, smem, st, pdl, 1, what, args...);
}

}  // namespace la
