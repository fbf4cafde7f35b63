// host.h -- helpers shared by the host side of the C ABI (abi.cu, attn_abi.cu):
// status mapping, device attributes, the tensor-map encoder and a cache of
// encoded maps.
#pragma once

#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "common.cuh"

namespace moe {

// A failed launch's error is taken off the runtime's record, which the next call
// would report as its own.
inline moe_status_t cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;
};

inline DeviceInfo device_info() {
    static std::mutex mu;
    static DeviceInfo cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DeviceInfo{};
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].sms == 0) {
        DeviceInfo d;
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        cache[dev] = d;
    }
    return cache[dev];
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// The last few tensor-map sets built on this thread, keyed by everything
// that goes into them (pointers, sizes, boxes, layout): a call on the same
// buffers reuses them instead of encoding them again (each encoding is a
// host call on the path of every layer).  Keys are compared bytewise and
// built from zeroed memory.
template <typename Key, typename Val, int N = 4>
struct MapCache {
    Key key[N];
    Val val[N];
    bool used[N] = {};
    int next = 0;
    const Val* find(const Key& k) const {
        for (int i = 0; i < N; ++i)
            if (used[i] && std::memcmp(&key[i], &k, sizeof(Key)) == 0) return &val[i];
        return nullptr;
    }
    void put(const Key& k, const Val& v) {
        key[next] = k;
        val[next] = v;
        used[next] = true;
        next = (next + 1) % N;
    }
};

}  // namespace moe
