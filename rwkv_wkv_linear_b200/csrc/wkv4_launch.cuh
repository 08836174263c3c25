// Launch helpers shared by the library's translation units: per-device limits
// and attributes, the programmatic launch, and the checked builds' fault
// injection (one count of launches over all of them).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "../../include/wkv4.h"
#include "wkv4_device.cuh"
#include "wkv4_internal.h"

namespace wkv4 {

// A function attribute (the dynamic shared memory limit, say) is one per
// device: set once per device for each kernel instantiation.
struct DeviceFlags {
    std::atomic<bool> done[64];
};

template <typename Kern>
inline cudaError_t ensure_attr(DeviceFlags& f, Kern kern, cudaFuncAttribute attr, int value) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && f.done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, attr, value);
    if (e == cudaSuccess && dev >= 0 && dev < 64) f.done[dev].store(true, std::memory_order_release);
    return e;
}

template <typename Kern>
inline cudaError_t ensure_smem_attr(DeviceFlags& f, Kern kern, size_t smem) {
    return ensure_attr(f, kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

inline int env_int(const char* name, int dflt) {
    const char* e = std::getenv(name);
    return e ? std::atoi(e) : dflt;
}

constexpr int kMaxDevices = 64;

// Per-device limits the launch shapes are worked out from, queried once per
// device (the launchers run on every call; attribute queries are not free).
struct DeviceAttrs {
    int smem_per_sm = 233472, smem_reserved = 1024, reg_file = 65536, max_threads = 2048,
        max_blocks = 32, sms = 148;
};

inline const DeviceAttrs& device_attrs() {
    static DeviceAttrs attrs[kMaxDevices];
    static std::once_flag once[kMaxDevices];
    static DeviceAttrs fallback;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return fallback;
    }
    std::call_once(once[dev], [dev] {
        DeviceAttrs& a = attrs[dev];
        cudaDeviceGetAttribute(&a.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
        cudaDeviceGetAttribute(&a.smem_reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
        cudaDeviceGetAttribute(&a.reg_file, cudaDevAttrMaxRegistersPerMultiprocessor, dev);
        cudaDeviceGetAttribute(&a.max_threads, cudaDevAttrMaxThreadsPerMultiProcessor, dev);
        cudaDeviceGetAttribute(&a.max_blocks, cudaDevAttrMaxBlocksPerMultiprocessor, dev);
        cudaDeviceGetAttribute(&a.sms, cudaDevAttrMultiProcessorCount, dev);
        cudaGetLastError();
    });
    return attrs[dev];
}

// A launch that may begin while the kernel before it in the stream is
// finishing (programmatic stream serialization): every kernel of the library
// waits for the earlier grid before its first global access.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Limit of each bounded device-side wait, in rounds of about 1 ms.  Checked
// builds (WKV4_CHECKED) take WKV4_WAIT_ROUNDS from the environment, so that a
// test can make a wait run out quickly.
inline uint32_t wait_rounds() {
#ifdef WKV4_CHECKED
    static const int r = env_int("WKV4_WAIT_ROUNDS", 0);
    if (r > 0) return (uint32_t)r;
#endif
    return kWaitRounds;
}

// Fault injection, in checked builds only (WKV4_CHECKED), read once from
// WKV4_FAULT:
//   launch:N   the N-th kernel launch of the process (1-based) is made with an
//              empty grid, which the runtime rejects (cudaErrorInvalid-
//              Configuration) without running anything: the launch error path
//              of every entry point, with no GPU fault;
//   exchange   no scan CTA pushes its segment aggregate, so every CTA's
//              bounded wait for its peers' aggregates runs out (with a short
//              limit from WKV4_WAIT_ROUNDS): the expiry path of the exchange.
// Production builds compile none of it.
struct FaultPlan {
    long launch_at = 0;  // 0: none
    bool exchange = false;
};

inline const FaultPlan& fault_plan() {
    static const FaultPlan plan = [] {
        FaultPlan f;
#ifdef WKV4_CHECKED
        if (const char* e = std::getenv("WKV4_FAULT")) {
            if (std::strncmp(e, "launch:", 7) == 0) f.launch_at = std::atol(e + 7);
            if (std::strcmp(e, "exchange") == 0) f.exchange = true;
        }
#endif
        return f;
    }();
    return plan;
}

// The grid of a launch: `g`, or an empty grid for the launch fault injection
// picks (one count over every launcher of the process).
#ifdef WKV4_CHECKED
inline std::atomic<long> g_launches{0};
#endif
template <typename G>
inline G launch_grid(G g) {
#ifdef WKV4_CHECKED
    const long at = fault_plan().launch_at;
    if (at > 0 && g_launches.fetch_add(1) + 1 == at) return G(0);
#endif
    return g;
}

// The device error word of this translation unit (each has its own), on the
// current device; synchronises the device.
static inline cudaError_t read_error_word(unsigned* bits, bool reset) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(bits, g_device_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    if (reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(unsigned));
    }
    return e;
}

inline bool aligned(const void* ptr, size_t bytes) {
    return ptr == nullptr || ((uintptr_t)ptr % bytes) == 0;
}

}  // namespace wkv4
