// launch.cpp -- host-side plumbing that the launch code of the product, attention
// and cache kernels shares (see launch.h).
#include "launch.h"

#include <cstring>
#include <mutex>

#include "entro.h"

namespace entro {

static std::mutex g_launch_mu;

int allow_smem(const void *fn, int dev) {
    constexpr int kMost = 256;  // kernels x devices remembered; past that the attribute is set again
    static struct {
        const void *fn;
        int dev;
    } seen[kMost];
    static int n = 0;
    std::lock_guard<std::mutex> lk(g_launch_mu);
    for (int i = 0; i < n; i++)
        if (seen[i].fn == fn && seen[i].dev == dev) return ENTRO_OK;
    DeviceInfo di;
    const int r = device_info(dev, &di);
    if (r != ENTRO_OK) return r;
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, fn);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin - static_cast<int>(at.sharedSizeBytes));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    if (n < kMost) seen[n++] = {fn, dev};
    return ENTRO_OK;
}

int clusters_at_once(const void *fn, int dev, unsigned threads, size_t smem, int cluster, int *clusters) {
    constexpr int kMost = 256;  // kernels x devices x sizes remembered; past that they are asked for again
    static struct {
        const void *fn;
        int dev, cluster, clusters;
    } seen[kMost];
    static int n = 0;
    std::lock_guard<std::mutex> lk(g_launch_mu);
    for (int i = 0; i < n; i++)
        if (seen[i].fn == fn && seen[i].dev == dev && seen[i].cluster == cluster) return *clusters = seen[i].clusters, ENTRO_OK;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr;
    std::memset(&attr, 0, sizeof(attr));
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(clusters, fn, &cfg);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
    }
    if (n < kMost) seen[n++] = {fn, dev, cluster, *clusters};
    return ENTRO_OK;
}

cudaError_t launch_ex(const void *fn, dim3 grid, unsigned threads, size_t smem, cudaStream_t st, unsigned cluster, bool early,
                      void **args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    std::memset(attr, 0, sizeof(attr));
    cfg.attrs = attr;
    if (early) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        cfg.numAttrs++;
    }
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) cudaGetLastError();  // reported by the caller: not left for others to find
    return e;
}

int encode_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
               const uint64_t *strides, const uint32_t *box) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = nullptr;
    {
        std::lock_guard<std::mutex> lk(g_launch_mu);
        if (!encode) {
            void *p = nullptr;
            cudaDriverEntryPointQueryResult q;
            const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
            if (e != cudaSuccess) return cuda_fail(e, "cudaGetDriverEntryPointByVersion");
            if (q != cudaDriverEntryPointSuccess || !p) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled");
            encode = reinterpret_cast<Encode>(p);
        }
    }
    cuuint64_t d[5], s[5];
    cuuint32_t b[5], ones[5];
    for (int i = 0; i < rank; i++) {
        d[i] = dims[i];
        b[i] = box[i];
        ones[i] = 1;
        if (i + 1 < rank) s[i] = strides[i];
    }
    const CUresult r = encode(map, type, rank, const_cast<void *>(base), d, s, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ENTRO_OK : cuda_fail(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
}

}  // namespace entro
