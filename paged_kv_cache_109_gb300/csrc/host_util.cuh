// host_util.cuh -- host-side helpers of the entry points: argument checks, launches,
// NVTX ranges.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <mutex>
#include <utility>

#include "decode_config.cuh"

namespace pa {
namespace {

bool desc_ok(const pa_cache_desc* c) {
    return c && c->num_blocks > 0 && c->block_size > 0 && c->num_kv_heads > 0 &&
           c->head_dim > 0 && (c->dtype == PA_F32 || c->dtype == PA_BF16);
}

int elem_bytes(const pa_cache_desc* c) { return c->dtype == PA_F32 ? 4 : 2; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---- launches ------------------------------------------------------------------

// Launch with programmatic stream serialization: the kernel may be scheduled
// while the previous kernel in the stream finishes; it waits for that kernel
// (griddepcontrol.wait) before reading any input.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PA_USE_PDL ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <typename Kern>
bool set_smem(Kern kern, size_t bytes) {
    if (bytes <= 48 * 1024) return true;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)bytes) == cudaSuccess;
}

// Lets `kern` use `bytes` of shared memory on the current device: asked for once
// per instance (its slot in `done`, a bit a device), with the most it ever uses.
template <typename Kern>
bool allow_smem(std::atomic<uint64_t>& done, Kern kern, size_t bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return set_smem(kern, bytes);
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (!set_smem(kern, bytes)) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

// An NVTX range over one library call (host side: argument checks and
// launches), so profilers can attribute the kernels to the call that made them.
struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

// ---- memory of the arguments ---------------------------------------------------

// A debug pass, whose host copies may throw: no exception leaves the library.
template <typename F>
pa_status debug_pass(F f) {
    try {
        return f();
    } catch (...) {
        return PA_ERR_CUDA;
    }
}

// Arrays of na and nb bytes share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

// The memory checks of one call, the current device asked for once.
struct CallDevice {
    int id = -1;
    CallDevice() {
        if (cudaGetDevice(&id) != cudaSuccess) {
            cudaGetLastError();
            id = -1;
        }
    }
    bool attributes(const void* p, cudaPointerAttributes& at) const {
        if (id >= 0 && cudaPointerGetAttributes(&at, p) == cudaSuccess) return true;
        cudaGetLastError();
        return false;
    }
    // Replaces p by the address that kernels of the current device use; false for memory
    // they may not touch (allowed: the device's own, managed or page-locked memory;
    // nullptr passes).
    template <typename T>
    bool map(T*& p) const {
        cudaPointerAttributes at;
        if (!p) return true;
        if (!attributes(p, at)) return false;
        if (at.type == cudaMemoryTypeDevice) return at.device == id;
        if (at.type == cudaMemoryTypeHost && at.devicePointer) {
            p = static_cast<T*>(at.devicePointer);
            return true;
        }
        return at.type == cudaMemoryTypeManaged;
    }
    // Device memory of the current device (or managed memory).
    bool memory(const void* p) const {
        cudaPointerAttributes at;
        return p && attributes(p, at) &&
               (at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == id));
    }
};

// CallDevice::memory for many pointers of one call (a model's layers): those inside
// an allocation that was already looked at are not looked up again.
struct CallMemory {
    const CallDevice& dev;
    uintptr_t lo = 0, hi = 0;       // the last allocation found to be the device's
    explicit CallMemory(const CallDevice& d) : dev(d) {}
    bool memory(const void* p) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(p);
        if (x >= lo && x < hi) return true;
        if (!dev.memory(p)) return false;
        static PFN_cuMemGetAddressRange_v3020 range = nullptr;
        static std::once_flag once;
        std::call_once(once, [] {
            void* f = nullptr;
            cudaDriverEntryPointQueryResult q;
            if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &f, 3020, cudaEnableDefault, &q) ==
                    cudaSuccess &&
                q == cudaDriverEntryPointSuccess)
                range = reinterpret_cast<PFN_cuMemGetAddressRange_v3020>(f);
        });
        CUdeviceptr base = 0;
        size_t bytes = 0;
        if (range && range(&base, &bytes, (CUdeviceptr)x) == CUDA_SUCCESS) {
            lo = (uintptr_t)base;
            hi = lo + bytes;
        }
        return true;
    }
};

}  // namespace
}  // namespace pa
