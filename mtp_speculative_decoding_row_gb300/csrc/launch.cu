// launch.cu -- what the launch plans of the tree and step operators share (launch.h).
#include <mutex>
#include <vector>

#include "launch.h"

namespace mtp {
namespace {

constexpr uint32_t kMaxSmem = 232448;  // 227 KB per CTA

struct FuncInfo {
    int device;
    const void *func;
    uint32_t smem;
    int per_sm;  // resident CTAs per SM
};
struct DeviceInfo {
    int device, sms;
};
std::mutex g_mu;
std::vector<FuncInfo> g_funcs;
std::vector<DeviceInfo> g_devices;

}  // namespace

bool device_sms(int &dev, int &sms) {
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto &d : g_devices)
        if (d.device == dev) {
            sms = d.sms;
            return true;
        }
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    try {
        g_devices.push_back({dev, sms});
    } catch (...) {  // out of memory: asked again next time
    }
    return true;
}

// Resident CTAs per SM of a kernel, its shared-memory limit raised first.
int resident(int dev, const void *func, uint32_t smem, int threads) {
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto &f : g_funcs)
        if (f.device == dev && f.func == func && f.smem == smem) return f.per_sm;
    int n = 0;
    // the limit is the kernel's largest, not this call's size: calls of one
    // kernel differ in it
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, func) != cudaSuccess ||
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMaxSmem - at.sharedSizeBytes)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, func, threads, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    try {
        g_funcs.push_back({dev, func, smem, n});
    } catch (...) {
    }
    return n;
}

// Every kernel here waits for the launches before it itself
// (griddepcontrol.wait) before it touches memory, and lets the next one's CTAs
// be set up early, so all are launched programmatically.
int launch(const void *func, dim3 grid, int threads, uint32_t smem, const void *args, mtp_stream_t stream,
           const void *map1, const void *map2, int cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    void *kargs[] = {const_cast<void *>(args), const_cast<void *>(map1), const_cast<void *>(map2)};
    return cudaLaunchKernelExC(&cfg, func, kargs) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // namespace mtp
