// Host-side argument checks, error messages and launch helpers of the matrix
// state and norm entry points (delta.cu, group_norm.cu).  capi.cu keeps its
// own copies: it is hashed together with the kernels it launches, and its
// helpers are tied to its per-stream workspaces, which nothing here uses.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "wkv_b200.h"

namespace wkvb {
void set_last_error(const char *msg);  // capi.cu: the message wkv_last_error() returns
}

namespace {

inline wkv_status fail(wkv_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    wkvb::set_last_error(buf);
    return st;
}

inline wkv_status cuda_fail(cudaError_t e, const char *what) {
    return fail(WKV_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// ---- driver entry points (no link-time dependency on libcuda) --------------
struct Driver {
    PFN_cuTensorMapEncodeTiled_v12000 encode_tiled = nullptr;
    PFN_cuMemGetAddressRange_v3020 get_address_range = nullptr;
    PFN_cuPointerGetAttribute_v4000 get_attribute = nullptr;
};

inline const Driver &driver() {
    static Driver d;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            d.encode_tiled = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        p = nullptr;
        if (cudaGetDriverEntryPoint("cuMemGetAddressRange", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            d.get_address_range = reinterpret_cast<PFN_cuMemGetAddressRange_v3020>(p);
        p = nullptr;
        if (cudaGetDriverEntryPoint("cuPointerGetAttribute", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            d.get_attribute = reinterpret_cast<PFN_cuPointerGetAttribute_v4000>(p);
        cudaGetLastError();
    });
    return d;
}

// Whether an address lies in memory that its owner maps into an address range
// piece by piece (a growing segment of an allocator, say): neither cudaMalloc's
// (which older inter-process handles can share) nor a memory pool's.
inline bool mapped_by_pieces(const Driver &d, CUdeviceptr p) {
    if (d.get_attribute == nullptr) return false;
    int shareable = 1;
    CUmemoryPool pool = nullptr;
    return d.get_attribute(&shareable, CU_POINTER_ATTRIBUTE_IS_LEGACY_CUDA_IPC_CAPABLE, p) == CUDA_SUCCESS &&
           d.get_attribute(&pool, CU_POINTER_ATTRIBUTE_MEMPOOL_HANDLE, p) == CUDA_SUCCESS && shareable == 0 &&
           pool == nullptr;
}

// The first address behind p's allocation, 0 if it is not known.  Pieces that
// follow one another without a gap are one allocation, as far as `enough`.
inline uintptr_t allocation_end(const Driver &d, CUdeviceptr p, uintptr_t enough) {
    CUdeviceptr base = 0;
    size_t size = 0;
    if (d.get_address_range == nullptr || d.get_address_range(&base, &size, p) != CUDA_SUCCESS) return 0;
    uintptr_t end = static_cast<uintptr_t>(base) + size;
    while (end < enough && mapped_by_pieces(d, end - 1) &&
           d.get_address_range(&base, &size, end) == CUDA_SUCCESS && base == end && size > 0 &&
           mapped_by_pieces(d, end))
        end += size;
    return end;
}

// One pointer argument: its extent in bytes, whether it may be NULL, and
// whether the call writes it.
struct Buf {
    const char *name;
    const void *p;
    size_t bytes;
    size_t align;
    bool written;
    bool optional;
};

inline wkv_status check_buffer(const Buf &b, int dev) {
    if (b.p == nullptr) {
        if (b.optional) return WKV_OK;
        return fail(WKV_ERR_INVALID_ARG, "%s is NULL", b.name);
    }
    if (reinterpret_cast<uintptr_t>(b.p) % b.align != 0)
        return fail(WKV_ERR_ALIGNMENT, "%s is not %zu-byte aligned", b.name, b.align);
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, b.p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(WKV_ERR_INVALID_ARG, "%s: not a CUDA pointer (%s)", b.name,
                    cudaGetErrorName(e));
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
        return fail(WKV_ERR_INVALID_ARG, "%s is not device memory", b.name);
    if (attr.type == cudaMemoryTypeDevice && attr.device != dev)
        return fail(WKV_ERR_INVALID_ARG, "%s lives on device %d, current device is %d", b.name,
                    attr.device, dev);
    const uintptr_t p = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t end = allocation_end(driver(), p, p + b.bytes);
    if (end != 0 && p + b.bytes > end)
        return fail(WKV_ERR_INVALID_ARG, "%s: %zu bytes needed but its allocation ends %zu bytes after it", b.name,
                    b.bytes, static_cast<size_t>(end - p));
    return WKV_OK;
}

// Every buffer of a call: each one valid, no written one overlapping another.
// `in_place` names a pair that may be one and the same buffer.
template <int N>
wkv_status check_buffers(const Buf (&b)[N], int dev, int in_place_a = -1, int in_place_b = -1) {
    for (int i = 0; i < N; ++i) {
        const wkv_status st = check_buffer(b[i], dev);
        if (st != WKV_OK) return st;
    }
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j) {
            if (!b[i].written && !b[j].written) continue;
            if (b[i].p == nullptr || b[j].p == nullptr || !b[i].bytes || !b[j].bytes) continue;
            const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p);
            const uintptr_t y = reinterpret_cast<uintptr_t>(b[j].p);
            if (!(x < y + b[j].bytes && y < x + b[i].bytes)) continue;
            if (i == in_place_a && j == in_place_b && x == y) continue;
            return fail(WKV_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
        }
    return WKV_OK;
}

inline bool aligned(const void *p, size_t a) {
    return p == nullptr || reinterpret_cast<uintptr_t>(p) % a == 0;
}

inline wkv_status current_device(int *dev) {
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    return WKV_OK;
}

inline int sm_count(int dev) {
    static std::atomic<int> cache[64];
    if (dev >= 0 && dev < 64 && cache[dev].load() > 0) return cache[dev].load();
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = 148;
    }
    if (dev >= 0 && dev < 64) cache[dev].store(n);
    return n;
}

// dynamic shared memory beyond 48 KB, set once per kernel and device
template <typename K>
wkv_status allow_smem(K kern, size_t smem, int dev, std::atomic<uint64_t> &done) {
    if (dev < 64 && (done.load() & (1ull << dev))) return WKV_OK;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    if (dev < 64) done.fetch_or(1ull << dev);
    return WKV_OK;
}

inline wkv_status launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? WKV_OK : cuda_fail(e, "kernel launch");
}

}  // namespace
