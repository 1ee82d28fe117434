// Shared by the two kernels of the attention over the 4-bit KV cache.
#pragma once

#include "attn_line.cuh"

namespace pe {
namespace kv4 {

using namespace line;

struct Kv4Params : LineParams {
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint32_t* k_params;   // scale (bf16) in the low half, base in the high one
    const uint32_t* v_params;
};

// The eight codes n of a word as n - 8 in fp16, exactly: pair x is (code x, code
// x + 4). Under fp16's exponent of 1024 a code stands as 1024 + n, one four bits
// further up as 1024 + 16 n.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&out)[4]) {
    constexpr uint32_t kMagic = 0x64006400u;
    const __half2 low = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));       // 1032
    const __half2 part = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));      // 1/16
    const __half2 high = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));      // -72
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = h == 0 ? w : w >> 8;
        const uint32_t a = (x & 0x000F000Fu) | kMagic, b = (x & 0x00F000F0u) | kMagic;
        const __half2 lo = __hsub2(*reinterpret_cast<const __half2*>(&a), low);
        const __half2 hi = __hfma2(*reinterpret_cast<const __half2*>(&b), part, high);
        out[2 * h] = *reinterpret_cast<const uint32_t*>(&lo);
        out[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
}
// An entry's value is scale * (n - 8) + mid; mid is NaN where one of its
// parameters is not finite.
__device__ __forceinline__ float scale_of(uint32_t par) { return __uint_as_float(par << 16); }
__device__ __forceinline__ float mid_of(uint32_t par) {
    const float mid = fmaf(8.f, scale_of(par), __uint_as_float(par & 0xFFFF0000u));
    return fmaf(mid, 0.f, mid);
}

// the tensor-memory kernel, for more rows: its plan and launch
int plan_umma(int B, int nkv, int hd, int max_pages, Plan* out);
int launch_umma(const Kv4Params& p, const Plan& a, int hd, cudaStream_t s);

}  // namespace kv4
}  // namespace pe
