// host_utils.h -- what the host sides of the gated and the serving libraries
// share: the device query, argument helpers and the status read-back.  Each
// library includes it into its one translation unit, so the state below is
// that library's own.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "device_utils.cuh"
#include "jamba_ssm.h"

namespace jssm_host {

inline thread_local int t_last_cuda_error = 0;

inline jamba_ssm_status cuda_fail(cudaError_t e) {
    t_last_cuda_error = static_cast<int>(e);
    return JAMBA_SSM_ERR_CUDA;
}

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool ready = false;
    bool usable = false;
    int sms = 0;
    int id = 0;
};

// The current device's info, or null with *st set.
inline const DeviceInfo *current_device(jamba_ssm_status *st) {
    static DeviceInfo devices[kMaxDevices];
    static std::mutex mutex;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        *st = e == cudaSuccess || e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver
                  ? JAMBA_SSM_ERR_NO_DEVICE
                  : cuda_fail(e);
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(mutex);
    DeviceInfo &info = devices[dev];
    if (!info.ready) {
        int major = 0, minor = 0, sms = 0;
        if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) {
            *st = cuda_fail(e);
            return nullptr;
        }
        info.usable = (major == 10 && minor == 0);  // built for sm_100a only
        info.sms = sms;
        info.id = dev;
        info.ready = true;
    }
    if (!info.usable) {
        *st = JAMBA_SSM_ERR_NO_DEVICE;
        return nullptr;
    }
    return &info;
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool overlaps(const void *a, size_t an, const void *b, size_t bn) {
    if (!a || !b || an == 0 || bn == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

struct Range {
    const void *p;
    size_t n;
};
// Whether an output overlaps an input or another output.
inline bool any_overlap(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
    }
    return false;
}

inline jamba_ssm_status check_workspace(const void *ws, size_t bytes) {
    if (!ws) return JAMBA_SSM_OK;
    if (!aligned(ws, 16)) return JAMBA_SSM_ERR_MISALIGNED;
    return bytes < JAMBA_SSM_STATUS_BYTES ? JAMBA_SSM_ERR_WORKSPACE : JAMBA_SSM_OK;
}

// Version 1 structs are the whole structs; a later version's caller may pass more.
template <typename P> inline bool read_params(const P *pin, P *p) {
    if (!pin || pin->struct_size < sizeof(P)) return false;
    std::memcpy(p, pin, sizeof(P));
    return true;
}

// Waits for the stream, then reads and clears a status word: the workspace's,
// or the library's own.
inline jamba_ssm_status read_status(void *workspace, void *stream) {
    jamba_ssm_status st;
    if (!current_device(&st)) return st;
    if (!aligned(workspace, 16)) return JAMBA_SSM_ERR_MISALIGNED;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    int word = 0;
    e = workspace ? cudaMemcpy(&word, workspace, sizeof(int), cudaMemcpyDeviceToHost)
                  : cudaMemcpyFromSymbol(&word, jssm::g_status_word, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e);
    if (word != 0) {
        const int zero = 0;
        e = workspace ? cudaMemcpy(workspace, &zero, sizeof(int), cudaMemcpyHostToDevice)
                      : cudaMemcpyToSymbol(jssm::g_status_word, &zero, sizeof(int));
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return static_cast<jamba_ssm_status>(word);
}

// After an enqueue: with JAMBA_SSM_SYNC_CHECK set (and not "0"), wait and
// return what the work recorded as the call's own status.
inline jamba_ssm_status finish_launch(void *stream, void *workspace) {
    static const bool sync_check = [] {
        const char *v = std::getenv("JAMBA_SSM_SYNC_CHECK");
        return v != nullptr && *v != '\0' && *v != '0';
    }();
    return sync_check ? read_status(workspace, stream) : JAMBA_SSM_OK;
}

// Launches `k`, its clusters `cs` CTAs along x.  `early`: it may begin while the
// work before it in the stream ends; such a kernel touches no memory before its
// griddepcontrol.wait (jssm::after_earlier_work), so only its own start -- the
// launch itself, barriers, TMEM -- overlaps.
inline jamba_ssm_status launch(const void *k, dim3 grid, unsigned threads, size_t smem, int cs, bool early,
                               void **args, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cs > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cs);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, k, args);
    return e == cudaSuccess ? JAMBA_SSM_OK : cuda_fail(e);
}

inline jamba_ssm_status launch_early(const void *k, dim3 grid, unsigned threads, size_t smem, int cs,
                                     void **args, void *stream) {
    return launch(k, grid, threads, smem, cs, true, args, stream);
}

}  // namespace jssm_host
