// Host helpers of the launches of thread-block clusters (step tables, block-sparse decode).
#pragma once
#include <atomic>

#include "pa_common.cuh"

namespace pa {

// A launch of clusters of c CTAs, programmatic dependent launch allowed.
template <typename... KArgs, typename... Args>
static cudaError_t launch_cluster(void (*kern)(KArgs...), int64_t ctas, int c, int threads, size_t smem, cudaStream_t st,
                                  Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// How many clusters of 1 .. 16 CTAs of one kernel a device holds at once, asked of CUDA once per
// device and size (above 8, which not every device has room for, the kernel is first allowed them).  A cluster lies within one GPC, so this is less than the CTAs that fit, and it
// differs from chip to chip: 16 clusters of 8 CTAs, one per SM, are not always there at once.
struct ClusterRoom {
    static constexpr int kDevices = 64;
    static constexpr int kMost = 16;
    std::atomic<int> n[kDevices][kMost + 1] = {};  // 0: not asked yet

    // 0 where CUDA does not say.
    template <typename K>
    int64_t of(K *kern, int c, int threads, size_t smem) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return 0;
        if (dev < kDevices && n[dev][c].load() > 0) return n[dev][c].load();
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(c * 1024));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = c;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int got = 0;
        if ((c > 8 && cudaFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                           cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
            cudaOccupancyMaxActiveClusters(&got, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        if (dev < kDevices) n[dev][c].store(got);
        return got;
    }

    // The largest cluster up to `most` CTAs of which `items` are resident at once (a second, partial
    // wave costs more than idle slots), at least 1.
    template <typename K>
    int largest(K *kern, int64_t items, int64_t most, int threads, size_t smem) {
        int c = most < 1 ? 1 : most > 8 ? 8 : (int)most;
        while (c > 1 && of(kern, c, threads, smem) < items) --c;
        return c;
    }
};

}  // namespace pa
