// pa_q8.cuh -- the 8-bit cache format: e4m3 codes, and a power of two for each 16 tokens of a
// page and KV head.
//
// A code c under the scale byte b stands for c 2^(b - 127) (b = 255: NaN).  The scale is a power
// of two because a block's scale grows while its tokens come in: the codes of the tokens already
// there are then rounded to the new scale, which changes a power of two's exponent and nothing
// else (but for codes that fall below 2^-6, whose steps are absolute); any other factor would
// round each of them again.  It also makes every value exact in FP16 and BF16 products, so the
// attention multiplies codes and touches the scale once a tile.  Floating codes keep 4 bits
// of values 2^15 below the block's largest, so the scale being up to twice as large as needed costs
// nothing.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kQ8Tokens = 16;  // of a page, under one scale

// Two codes (the lower byte first) -> FP16 pair, exact; NaN codes give NaN.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t codes) {  // the lower 16 bits
    uint32_t r;
    asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(codes));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3_hi(uint32_t codes) {  // the upper 16 bits
    uint32_t r;
    asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;}" : "=r"(r) : "r"(codes));
    return r;
}

// Four floats -> codes, to nearest (ties to even), the first in the lowest byte; NaN gives 127.
// Beyond 448 saturates: the scale keeps values within it.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// 2^(b - 127) of a scale byte; NaN for 255.
__device__ __forceinline__ float q8_scale(uint32_t b) {
    return b == 0 ? 0x1p-127f : b == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

// Page of a slot (>= 0).  (A 64-bit division is a hundred instructions for every warp.)
__device__ __forceinline__ int64_t q8_page_of(int64_t slot, int block_size) {
    return slot >> 31 ? slot / block_size : (uint32_t)slot / (uint32_t)block_size;
}

}  // namespace pa
