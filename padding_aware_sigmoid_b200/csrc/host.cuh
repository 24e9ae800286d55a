// Host state shared by the files that implement the C ABI: per-device status
// word and attributes, the cache of encoded TMA tensor maps, argument checks
// and kernel launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>
#include <unordered_map>
#include <unordered_set>

#include "../../include/sigattn.h"
#include "sigmoid.cuh"

namespace sigattn {

constexpr int kMaxDevices = 64;

inline std::mutex g_mu;
inline int *g_status[kMaxDevices] = {};          // device status word per device (lazy, never freed)
inline int g_cc_major[kMaxDevices] = {};         // 0 = not queried yet
inline int g_sm_count[kMaxDevices] = {};         // multiprocessors per device (persistent grids)
inline std::atomic<int> g_sigmoid_mode{kSigmoidTanh};
inline std::atomic<uint64_t> g_timeout_ns{4000000000ull};
inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
inline std::atomic<int> g_last_cuda_error{0};

// Records the failing call's error (and clears the runtime's last error).
inline sigattn_status cuda_fail(cudaError_t e = cudaSuccess) {
    cudaError_t last = cudaGetLastError();
    g_last_cuda_error.store(static_cast<int>(e != cudaSuccess ? e : last));
    return SIGATTN_ERR_CUDA;
}

inline sigattn_status device_state(int *dev, int *cc_major, int **status) {
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (*dev < 0 || *dev >= kMaxDevices) return SIGATTN_ERR_UNSUPPORTED_DEVICE;
    // Makes the device's primary context current in the calling thread: the
    // tensor-map encoder is a driver call and needs one (a fresh thread, such
    // as PyTorch's autograd worker, may not have one yet).
    e = cudaSetDevice(*dev);
    if (e != cudaSuccess) return cuda_fail(e);
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_cc_major[*dev] == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess)
            return cuda_fail();
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
            return cuda_fail();
        g_sm_count[*dev] = sms;
        g_cc_major[*dev] = major * 10 + minor;
    }
    if (g_status[*dev] == nullptr) {
        int *s = nullptr;
        if (cudaMalloc(&s, 64) != cudaSuccess) return cuda_fail();
        if (cudaMemset(s, 0, 64) != cudaSuccess) return cuda_fail();
        g_status[*dev] = s;
    }
    *cc_major = g_cc_major[*dev];
    *status = g_status[*dev];
    return SIGATTN_OK;
}

inline sigattn_status get_encoder() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_encode != nullptr) return SIGATTN_OK;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
        return cuda_fail();
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return SIGATTN_OK;
}

// [Z][L][H][D] bf16 viewed as a 4-D tensor (D, H, L, Z), boxes of 64 x 1 x 128 x 1
// elements with 128-byte swizzle: one box is one [128 rows][64 cols] operand atom.
inline sigattn_status encode_bf16_map_uncached(CUtensorMap *m, const void *base, int Z, int L, int H,
                                        int D) {
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                          static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(Z)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2,
                             static_cast<cuuint64_t>(L) * H * D * 2};
    cuuint32_t box[4] = {64, 1, 128, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        g_last_cuda_error.store(10000 + static_cast<int>(r));
        return SIGATTN_ERR_CUDA;
    }
    return SIGATTN_OK;
}

// Encoded maps, keyed by everything that goes into one: a bf16 map is a pure
// function of (base address, Z, L, H, D), so a hit returns exactly what a new
// encoding would, and repeated calls on the same buffers skip the driver call.
// Bounded: the cache is emptied when it reaches kMaxCachedMaps entries.
struct MapKey {
    const void *base;
    int Z, L, H, D;
    bool operator==(const MapKey &o) const {
        return base == o.base && Z == o.Z && L == o.L && H == o.H && D == o.D;
    }
};
struct MapKeyHash {
    size_t operator()(const MapKey &k) const {
        size_t h = std::hash<const void *>()(k.base);
        for (int v : {k.Z, k.L, k.H, k.D}) h = h * 1000003u ^ static_cast<size_t>(v);
        return h;
    }
};
constexpr size_t kMaxCachedMaps = 1024;
inline std::mutex g_map_mu;
inline std::unordered_map<MapKey, CUtensorMap, MapKeyHash> g_maps;

inline sigattn_status encode_bf16_map(CUtensorMap *m, const void *base, int Z, int L, int H, int D) {
    const MapKey key{base, Z, L, H, D};
    {
        std::lock_guard<std::mutex> lk(g_map_mu);
        auto it = g_maps.find(key);
        if (it != g_maps.end()) {
            *m = it->second;
            return SIGATTN_OK;
        }
    }
    sigattn_status s = encode_bf16_map_uncached(m, base, Z, L, H, D);
    if (s != SIGATTN_OK) return s;
    std::lock_guard<std::mutex> lk(g_map_mu);
    if (g_maps.size() >= kMaxCachedMaps) g_maps.clear();
    g_maps.emplace(key, *m);
    return SIGATTN_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// (kernel, device) pairs whose dynamic shared-memory limit has been raised; a
// kernel always asks for the same amount, so once per device is enough.
struct FuncDev {
    const void *f;
    int dev;
    bool operator==(const FuncDev &o) const { return f == o.f && dev == o.dev; }
};
struct FuncDevHash {
    size_t operator()(const FuncDev &k) const {
        return std::hash<const void *>()(k.f) * 31u ^ static_cast<size_t>(k.dev);
    }
};
inline std::mutex g_attr_mu;
inline std::unordered_set<FuncDev, FuncDevHash> g_attr_set;

// smem_most: the most dynamic shared memory any call asks of this kernel.
// overlap: the kernel may start while the one before it on the stream still
// runs (programmatic dependent launch); it waits for it by itself.  cluster: blocks
// of a cluster, along x.
template <typename... KArgs, typename... Args>
sigattn_status launch_with(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem_most, size_t smem,
                           bool overlap, unsigned cluster, cudaStream_t stream, Args... args) {
    if (smem_most > 48 * 1024) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail(e);
        const FuncDev key{reinterpret_cast<const void *>(kernel), dev};
        std::lock_guard<std::mutex> lk(g_attr_mu);
        if (g_attr_set.count(key) == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem_most));
            if (e != cudaSuccess) return cuda_fail(e);
            g_attr_set.insert(key);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2] = {};
    cfg.attrs = attrs;
    if (overlap) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = cluster;
        attrs[cfg.numAttrs].val.clusterDim.y = 1;
        attrs[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return cuda_fail(e);
    return SIGATTN_OK;
}
template <typename... KArgs, typename... Args>
sigattn_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                      Args... args) {
    return launch_with(kernel, grid, block, smem, smem, false, 1u, stream, args...);
}

}  // namespace sigattn
