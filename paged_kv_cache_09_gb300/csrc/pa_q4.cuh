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

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Quantises one row held by a warp, lane l holding dims 8l .. 8l + 7 (BF16 pairs), and stores it
// at offset o of the (page, head) run `run`.  A lane's dims are word g = l / 8 of unit l % 8.
//
// Codes are those of exact arithmetic (ties to even).  q = (x - lo) / s by a product with the
// reciprocal and one correction from the exact remainder: a quotient that is a tie k + 1/2 comes
// out exactly, and no other quotient reaches one (x - lo is a multiple of its last place, so the
// quotient keeps further from a tie than fp32 rounds).  x - lo itself can round only where x is
// tiny beside lo, and that matters only where the value 0 lies on a tie: then the sign of x
// decides.
// A group with a NaN or an infinity, or whose range overflows fp32, gets s = NaN: all of
// it reads back as NaN.
__device__ __forceinline__ void q4_store_row(const uint4 &row, int lane, uint8_t *run,
                                             int block_size, int o) {
    const uint32_t w[4] = {row.x, row.y, row.z, row.w};
    const int g = lane >> 3, u = lane & 7;
    // (minimum, -maximum) of the group: one register, one kind of minimum
    uint32_t lows = min_bf16x2(min_bf16x2(w[0], w[1]), min_bf16x2(w[2], w[3]));
    uint32_t highs = max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3]));
    highs ^= 0x80008000u;
    uint32_t ends = min_bf16x2(__byte_perm(lows, highs, 0x5410), __byte_perm(lows, highs, 0x7632));
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
#pragma unroll
    for (int sh = 1; sh < 8; sh <<= 1) ends = min_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, sh));
    float lo = bf16_lo(ends), range = __fsub_rn(-bf16_hi(ends), lo);
    bad = ((__ballot_sync(0xffffffffu, bad) >> (g * 8)) & 0xffu) != 0 || !(range <= 3.4028235e38f);
    const uint32_t lo_bits = ends & 0xffffu;
    const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(range, 15.f)));
    uint32_t codes = 0;
    if (!bad && s > 0.f) {
        // Steps near the subnormals: the same quotients from values 2^64 times as large.
        const float up = s < 1e-30f ? 0x1p64f : 1.f;
        const float st = s * up, rcp = __frcp_rn(st), l = lo * up;
        auto quotient = [&](float d) {
            const float t = d * rcp;
            return __fmaf_rn(__fmaf_rn(-t, st, d), rcp, t);
        };
        const float zero = quotient(-l);
        const bool tie = zero - floorf(zero) == 0.5f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = (j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1])) * up;
            const float d = __fsub_rn(x, l);
            // (adding 1.5 * 2^23 rounds to an integer, ties to even, in the low bits)
            uint32_t n = __float_as_uint(__fadd_rn(quotient(d), 12582912.f)) & 31u;
            if (tie && d == -l && x != 0.f) n = (uint32_t)floorf(zero) + (x > 0.f ? 1u : 0u);
            codes |= min(n, 15u) << (4 * j);
        }
    }
    *reinterpret_cast<uint32_t *>(run + q4_word_offset(o, u, g)) = codes;
    if (u == 0)
        *reinterpret_cast<uint32_t *>(run + q4_pair_offset(block_size, o, g)) =
            (bad ? 0x7fc0u : (__float_as_uint(s) >> 16)) | (lo_bits << 16);
}

// Page of a slot (>= 0).  (A 64-bit division is a hundred instructions for every warp.)
__device__ __forceinline__ int64_t page_of(int64_t slot, int block_size) {
    return slot >> 31 ? slot / block_size : (uint32_t)slot / (uint32_t)block_size;
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
