// pa_q4.cuh -- the 4-bit cache format: where a token's bytes lie, and the quantiser.
//
// A row (one token of one KV head, 256 BF16 values) is cut into 4 groups of 64 dims.
// Group g keeps lo = its minimum and a step s = bf16((max - lo) / 15), both BF16, and a
// code n = clamp(rint((x - lo) / s), 0, 15) per value (0 where s is 0); it stands for
// lo + s * n.  Uniform codes with two BF16 numbers per group factor out of both products
// of the attention:
//     q . khat  = sum_g  s_g (q_g . n_g) + lo_g sum(q_g)
//     sum_t p_t vhat_t = sum_t (p_t s_tg) n_t + sum_t p_t lo_tg
// so the kernels multiply codes, which are small integers and exact in FP16, and touch
// the steps once per token and group rather than once per value.  lo is a value of the
// group, so it is exact in BF16; a group of equal values has s = 0 and is kept exactly.
//
// Bytes: 128 of codes and 16 of (s, lo) pairs, 144 for 512 of BF16.  A page holds, for
// each KV head, block_size * 128 bytes of codes and then block_size * 16 bytes of pairs:
// one head's tokens are one contiguous run, which a plain bulk copy brings in.
//
// Order of the codes of a token.  "Unit" u (16 bytes, u = 0..7) holds for each group g one
// 32-bit word, the codes of dims 64g + 8u + j at bits 4j.  A lane of the decode kernel
// then finds the 16 dims that it owns of every group in two units (K: units 2c, 2c + 1 for
// column c of a tensor-core fragment; V: unit r for row r), as whole 16-byte loads.  Unit
// u of the token at offset o of its page is stored at place u ^ (o % 8), so that the
// eight lanes of a load phase, which read different tokens, hit different banks.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kQ4Groups = 4, kQ4GroupDims = kHeadDim / kQ4Groups;
constexpr int kQ4CodeBytes = kHeadDim / 2;         // codes of a token: 128
constexpr int kQ4PairBytes = kQ4Groups * 4;        // its (s, lo) pairs: 16
constexpr int kQ4RowBytes = kQ4CodeBytes + kQ4PairBytes;

// Byte offset, within a (page, head) run, of word g of unit u of the token at offset o.
__device__ __forceinline__ int q4_word_offset(int o, int u, int g) {
    return o * kQ4CodeBytes + ((u ^ (o & 7)) << 4) + g * 4;
}
// ... and of its pair of group g.
__device__ __forceinline__ int q4_pair_offset(int block_size, int o, int g) {
    return block_size * kQ4CodeBytes + o * kQ4PairBytes + g * 4;
}

__device__ __forceinline__ float q4_step(uint32_t pair) { return bf16_lo(pair); }
__device__ __forceinline__ float q4_low(uint32_t pair) { return bf16_hi(pair); }

// Quantises one row held by a warp, lane l holding dims 8l .. 8l + 7 (BF16 values as
// floats), and stores it at offset o of the (page, head) run `run`.  A lane's dims are
// word g = l / 8 of unit l % 8.
//
// Codes are those of exact arithmetic (ties to even): the quotient's rounding in fp32 can
// be one off at a border, so the remainder x - lo - n s is formed exactly (the difference
// and its rounding error; n s has 12 bits) and compared with half a step.
// A group with a NaN or an infinity, or whose range overflows fp32, gets s = NaN: all of
// it reads back as NaN.
__device__ __forceinline__ void q4_store_row(const float (&x)[8], int lane, uint8_t *run,
                                             int block_size, int o) {
    float lo = x[0], hi = x[0];
    bool bad = !(fabsf(x[0]) <= 3.4028235e38f);
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
        bad |= !(fabsf(x[j]) <= 3.4028235e38f);
    }
#pragma unroll
    for (int sh = 1; sh < 8; sh <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, sh));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, sh));
    }
    const unsigned bad_lanes = __ballot_sync(0xffffffffu, bad);
    const int g = lane >> 3, u = lane & 7;
    const float range = __fsub_rn(hi, lo);
    bad = ((bad_lanes >> (g * 8)) & 0xffu) != 0 || !(range <= 3.4028235e38f);
    const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(range, 15.f)));
    uint32_t word = 0;
    if (!bad && s > 0.f) {
        // Steps near the subnormals: the same quotients from values 2^64 times as large.
        const float up = s < 1e-30f ? 0x1p64f : 1.f;
        const float st = s * up, rcp = __frcp_rn(st), half = 0.5f * st, l = lo * up;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = x[j] * up;
            const float d = __fsub_rn(v, l);
            const float b = __fsub_rn(d, v);  // two-sum: v - l = d + e exactly
            const float e = __fadd_rn(__fsub_rn(v, __fsub_rn(d, b)), __fsub_rn(-l, b));
            float n = fminf(rintf(d * rcp), 15.f);
            const float r = __fmaf_rn(-n, st, d);
            const bool odd = (static_cast<int>(n) & 1) != 0;
            if (r > half || (r == half && (e > 0.f || (e == 0.f && odd))))
                n += 1.f;
            else if (r < -half || (r == -half && (e < 0.f || (e == 0.f && odd))))
                n -= 1.f;
            word |= static_cast<uint32_t>(fminf(n, 15.f)) << (4 * j);
        }
    }
    *reinterpret_cast<uint32_t *>(run + q4_word_offset(o, u, g)) = word;
    if (u == 0) {
        const uint32_t sb = bad ? 0x7fc0u : (__float_as_uint(s) >> 16);
        *reinterpret_cast<uint32_t *>(run + q4_pair_offset(block_size, o, g)) =
            sb | (__float_as_uint(lo) & 0xffff0000u);
    }
}

// Lane l's dims 8l .. 8l + 7 of the row at offset o of `run`, rounded to BF16: two per
// register.
__device__ __forceinline__ uint4 q4_load_row(const uint8_t *run, int block_size, int o, int lane) {
    const int g = lane >> 3, u = lane & 7;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(run + q4_word_offset(o, u, g)));
    const uint32_t pair =
        __ldg(reinterpret_cast<const uint32_t *>(run + q4_pair_offset(block_size, o, g)));
    const float s = q4_step(pair), lo = q4_low(pair);
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        r[j] = pack_bf16x2(fmaf(s, static_cast<float>((w >> (8 * j)) & 15u), lo),
                           fmaf(s, static_cast<float>((w >> (8 * j + 4)) & 15u), lo));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace pa
