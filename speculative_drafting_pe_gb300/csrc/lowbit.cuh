// Shared by the low-bit serving operators: conversions and products, and what
// their entry points ask of the device.
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace pe {

// four E4M3 codes, nearest, beyond +-448 saturated
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// c += a b, m16n8k16
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8-bit KV cache codes of 128-wide heads as [lines][128] bytes (16 lines per
// page and head); box = one page of one head, swizzled over the row's 128 bytes
int encode_tmap_codes(CUtensorMap* map, const void* codes, uint64_t lines);

// Multiprocessors of the current device. The driver is asked once per device:
// a call that is a launch of a few microseconds waits for such questions.
inline int current_device(int* dev, int* sms) {
    static std::atomic<int> known[64];
    PE_CUDA_TRY(cudaGetDevice(dev));
    const bool kept = *dev >= 0 && *dev < 64;
    *sms = kept ? known[*dev].load(std::memory_order_relaxed) : 0;
    if (*sms == 0) {
        PE_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev));
        if (kept) known[*dev].store(*sms, std::memory_order_relaxed);
    }
    return PE_OK;
}
// Lets a kernel have `bytes` of dynamic shared memory (the same in every call)
// on device dev; likewise.
template <auto kern>
int allow_smem(int dev, int bytes) {
    static std::atomic<bool> done[64];
    const bool kept = dev >= 0 && dev < 64;
    if (kept && done[dev].load(std::memory_order_relaxed)) return PE_OK;
    PE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (kept) done[dev].store(true, std::memory_order_relaxed);
    return PE_OK;
}

}  // namespace pe
