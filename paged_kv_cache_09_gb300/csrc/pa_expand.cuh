// pa_expand.cuh -- what the expansions of the 4-bit and the 8-bit cache into FP16 operands of the
// prefill share: scaling by powers of two, and the queries.
//
// FP16 holds the values to 2^-11 (BF16 to 2^-8) but spans fewer binades, so each query row and
// each KV head of a sequence is scaled by the power of two that brings its largest magnitude
// to [2^14, 2^15).  Values down to 2^-28 of the largest keep 11 bits; smaller ones are off by up
// to 2^-39 of it.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Eight BF16 values as floats.
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// The power of two that brings magnitudes up to `top` below 2^15 (1 for 0 and non-finite).
__device__ __forceinline__ float scale_for(float top) {
    const int e = (int)(__float_as_uint(top) >> 23) & 255;
    if (e == 255 || top == 0.f) return 1.f;
    return __uint_as_float((uint32_t)min(254, max(1, 127 + 14 - (e - 127))) << 23);
}

// One query row, by a warp: FP16 and the factor that undoes its scaling.
__device__ __forceinline__ void expand_query(const ExpandArgs &a, int64_t row, int lane) {
    float x[8], top = 0.f;
    unpack8(__ldg(reinterpret_cast<const uint4 *>(a.q + row * kHeadDim) + lane), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = scale_for(top);
    reinterpret_cast<uint4 *>(a.q_out + row * kHeadDim)[lane] =
        make_uint4(pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f),
                   pack_f16x2(x[4] * f, x[5] * f), pack_f16x2(x[6] * f, x[7] * f));
    if (lane == 0) a.q_factor[row] = 1.f / f;
}

}  // namespace pa
