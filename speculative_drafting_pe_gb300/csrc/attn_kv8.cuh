// Shared by the two kernels of the attention over the 8-bit KV cache.
#pragma once

#include "attn_line.cuh"

namespace pe {
namespace kv8 {

using namespace line;

struct Kv8Params : LineParams {
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* k_scale;
    const float* v_scale;
};

__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// bytes of w that are E4M3's NaN become 0; `any` collects whether there were some
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int& any) {
    const uint32_t other = ((w & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu) + 0x7F7F7F7Fu;   // bit 7 of a byte: not NaN
    const uint32_t nan = ~other & 0x80808080u;
    any |= nan != 0;
    return w & ~((nan >> 7) * 0xFFu);
}

// rows past which the tensor-memory kernel takes over, and its launch
int launch_umma(const Kv8Params& p, const Plan& a, int hd, cudaStream_t s);
constexpr int kUmmaPages = 4, kUmmaRows = 128, kUmmaUnits = 640;
// A share's positions at least (B=1 K=7, 2048 entries: 14.9 us, with 1 15.5, with 6 16.6), and the units' worth of a
// segment's end (B=128 K=11: 190 us, with 0 208; 64-wide heads 87 and 91; as all of these were then)
constexpr int kUmmaLeast = 3, kUmmaPad = 7;

}  // namespace kv8
}  // namespace pe
