// Host-side helpers of the C entry points, shared by the library's translation
// units (each gets its own copy): checked size arithmetic, overlap and
// alignment tests, device selection, the tensor-map encoder and the status word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "evo_attn.h"

namespace evo {
// evo_blocks.cu: reads and clears the status word of its kernels on the
// current device, synchronising `stream`.  EVO_OK or EVO_ERR_CUDA.
int take_blocks_status(cudaStream_t stream, int* status);
}  // namespace evo

namespace {

constexpr int kMaxDevices = 64;

// Sets a kernel's dynamic shared-memory limit once per device.  Calls from
// several host threads may race on the first use; a mutex orders them and
// the flag is only set once the attribute call has succeeded.
struct AttrOnce {
    std::mutex mu;
    bool done[kMaxDevices] = {};
    template <typename K>
    bool ensure(int dev, K kernel, int smem_bytes) {
        std::lock_guard<std::mutex> lock(mu);
        if (done[dev]) return true;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) != cudaSuccess)
            return false;
        done[dev] = true;
        return true;
    }
};

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    if (a == nullptr || b == nullptr || abytes <= 0 || bbytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + uint64_t(bbytes) && b0 < a0 + uint64_t(abytes);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The device that owns `ptr`, or a negative status if it is not device memory.
int device_of(const void* ptr) {
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, ptr) != cudaSuccess) {
        cudaGetLastError();
        return EVO_ERR_INVALID_ARG;
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) return EVO_ERR_INVALID_ARG;
    return attr.device;
}

// Makes the device that owns the buffers current for the duration of one
// call and restores the caller's current device afterwards.
struct DeviceScope {
    int prev = -1;
    bool changed = false;
    ~DeviceScope() {
        if (changed) cudaSetDevice(prev);
    }
};

// Relaxed stream-capture mode for this thread during one call, so that the
// call's host-side queries (pointer attributes, function attributes, the
// driver entry point) are allowed while the caller captures a CUDA graph;
// the launches and copies themselves are captured as usual.
struct RelaxedCapture {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
    ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

int select_device_of(const void* ptr, DeviceScope& scope) {
    const int dev = device_of(ptr);
    if (dev < 0) return dev;
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) return EVO_ERR_CUDA;
    if (cur != dev) {
        if (cudaSetDevice(dev) != cudaSuccess) return EVO_ERR_CUDA;
        scope.prev = cur;
        scope.changed = true;
    }
    return dev;
}

// Reads a device status word of the current device into *v and clears it,
// synchronising `st`.
template <typename Word>
bool take_status_word(Word& word, cudaStream_t st, int* v) {
    *v = 0;
    if (cudaMemcpyFromSymbolAsync(v, word, sizeof(int), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return false;
    if (*v == 0) return true;
    const int zero = 0;
    return cudaMemcpyToSymbolAsync(word, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) == cudaSuccess &&
           cudaStreamSynchronize(st) == cudaSuccess;
}

}  // namespace
