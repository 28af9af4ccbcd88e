// pa_rope.cu -- RMS norm of each query and key head, rotation by position, and the KV
// write, in one pass.
//
// Row x of one head (D dims) becomes, in fp32,
//     y = x / sqrt(mean(x^2) + eps) * (w + bias)
// and its first R dims are rotated in pairs by the token's angles (a table of cosines and
// sines by position): (a, b) -> (a cos - b sin, b cos + a sin), the pair being dims
// (i, i + R/2) or (2i, 2i + 1).  One rounding to BF16 at the end.  A key row goes to its
// slot of the cache, the value row beside it unchanged (BF16 cache), or both quantised
// (4-bit cache: the key's BF16 value, so that the result is that of the two calls).
//
// Every value is read once and written once; bound by memory for a prompt chunk, by launch
// and one round trip for a decode batch.  D / 8 lanes hold a row, 8 dims (16 bytes) a lane.
// Instructions come close to bounding it too, so the weights are multiplied into the angles once
// per token and kind of row,
//     out_j = inv (x_j A_j + x_p B_j),   A_j = w_j cos, B_j = +- w_p sin   (p: j's partner),
// the partners are exchanged as packed BF16, before any arithmetic, and the arithmetic is on pairs.
// 4096 tokens of 24 + 4 + 4 heads of 256, into a BF16 cache: 28.7 us, 4.8 TB/s (43 with the
// weights applied to every row, 29.6 with the rows summed one by one); into a 4-bit cache 33.6 us,
// without a cache 26.3.  32 + 8 + 8 heads 45.9 us, 16 + 4 + 4 24.8, 12 + 2 + 2 20.5 (4.5, 4.2 and
// 3.5 TB/s: warps with fewer rows of a token on their way).  16 warps an SM with 8 rows each on
// their way move more than 20 or 24 with fewer (33 and 40 us): a row on its way is registers.
// 16 tokens: 2.3 us.
#include <algorithm>

#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 6;  // query rows of a warp that are loaded a token ahead (24 heads over 4 warps)

// Pairs of fp32 in one register pair.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f32x2 pair_bf16(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ f32x2 mul(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack(f32x2 v) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return pack_bf16x2(lo, hi);
}

template <int kD, bool kNeighbours, int kCache>  // kCache: 0 none, 1 BF16, 2 4-bit
__global__ void __launch_bounds__(kWarps * 32, 4)
    qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kLanes = kD / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a warp
    static_assert(kCache != 2 || kD == kHeadDim, "the 4-bit cache holds rows of 256");
    const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
    const int step = gridDim.y * kWarps * kPer;                              // rows of all warps
    const int unit = (blockIdx.y * kWarps + (threadIdx.x >> 5)) * kPer + sub;  // this warp's first
    const int hq = a.num_q_heads, hkv = a.num_kv_heads;
    // Keys start where the queries' last round ends among the warps, values after them.
    // (A warp's rows stay together: the shifts, below step, are by whole warps.)
    int unit_k = unit - a.shift_k, unit_v = unit - a.shift_v;
    unit_k += unit_k < 0 ? step : 0;
    unit_v += unit_v < 0 ? step : 0;
    auto row_of = [&](const uint16_t *p, int r, int n) {
        return r < n ? *reinterpret_cast<const uint4 *>(p + r * kD + 8 * l) : make_uint4(0, 0, 0, 0);
    };
    pdl_wait();
    pdl_trigger();
    const int R = a.rotary_dim, half = R / 2;
    const bool turns = 8 * l < R, second = 8 * l >= half;  // (second: of a pair of halves)
    const int partner = turns && !kNeighbours ? (second ? l - R / 16 : l + R / 16) : l;
    // A CTA takes every gridDim.x-th token, and loads ahead: a token's first rows of each kind into
    // registers and its angles (this lane's, into shared memory) while the token before is worked
    // on, its position a token earlier still.  (A padding token's rows are read for nothing.)
    __shared__ float4 angles[kWarps][2][kNeighbours ? 2 : 4][32];
    uint4 raw[kBatch], raw_k, raw_v;  // each is loaded again as soon as its row is done
    int64_t slot_next;
    const uint16_t *q_at, *k_at, *v_at;  // of the token that is loaded
    auto at = [&](int64_t t) {
        q_at = a.q + t * a.q_stride;
        k_at = a.k + t * a.k_stride;
        if (kCache) v_at = a.v + t * a.v_stride;
    };
    auto angles_of = [&](int64_t t, int pos, int buf) {
        slot_next = kCache ? a.slot_mapping[t] : -1;
        if (turns && pos >= 0 && pos < a.max_position) {
            const float *row = a.cos_sin + (int64_t)pos * R +
                               (kNeighbours ? 4 * l : second ? 8 * l - half : 8 * l);
            constexpr int kN = kNeighbours ? 1 : 2;
#pragma unroll
            for (int e = 0; e < 2 * kN; ++e)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_u32(&angles[threadIdx.x >> 5][buf][e][lane])),
                             "l"(row + (e / kN) * half + (e % kN) * 4)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto position = [&](int64_t t) { return t < a.num_tokens ? a.positions[t] : -1; };
    const int64_t stride = gridDim.x;
    int pos = position(blockIdx.x), pos_next = position(blockIdx.x + stride), buf = 0;
    at(blockIdx.x);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) raw[b] = row_of(q_at, unit + b * step, hq);
    raw_k = row_of(k_at, unit_k, hkv);
    if (kCache) raw_v = row_of(v_at, unit_v, hkv);
    angles_of(blockIdx.x, pos, 0);
    for (int64_t t = blockIdx.x; t < a.num_tokens; t += stride, buf ^= 1) {
    const int pos_now = pos;
    const int64_t slot = slot_next;
    const bool more = t + stride < a.num_tokens;
    pos = pos_next;
    if (more) {
        at(t + stride);
        angles_of(t + stride, pos, buf ^ 1);
        pos_next = position(t + 2 * stride);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    const bool live = pos_now >= 0 && pos_now < a.max_position;  // otherwise its rows stay as they are
    if (pos_now >= a.max_position && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrPosition);
    int64_t run = -1;  // the slot's place in the caches (of head 0)
    int o = 0;
    if (kCache && live && slot >= 0) {
        const int64_t page = page_of(slot, a.block_size);
        o = (int)(slot - page * a.block_size);
        if (page < a.num_pages)
            run = kCache == 1 ? page * a.page_stride + (int64_t)o * hkv * kD : page * a.page_stride;
        else if (threadIdx.x == 0 && blockIdx.y == 0)
            atomicOr(a.err, kErrSlot);
    }
    // A and B of this lane's dims for rows with these weights.
    f32x2 A[4], B[4];
    auto factors = [&](const uint16_t *w) {
        float wo[8], wp[8], c[8], s[8];
        const uint4 own = __ldg(reinterpret_cast<const uint4 *>(w) + l);
        const uint4 other = __ldg(reinterpret_cast<const uint4 *>(w) + partner);
        const uint32_t x[4] = {own.x, own.y, own.z, own.w}, y[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wo[2 * i] = bf16_lo(x[i]) + a.weight_bias;
            wo[2 * i + 1] = bf16_hi(x[i]) + a.weight_bias;
            wp[2 * i + (kNeighbours ? 1 : 0)] = bf16_lo(y[i]) + a.weight_bias;
            wp[2 * i + (kNeighbours ? 0 : 1)] = bf16_hi(y[i]) + a.weight_bias;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
        }
        if (turns) {
            const float4 (*mine)[32] = angles[threadIdx.x >> 5][buf];
            if (kNeighbours) {
                const float4 cv = mine[0][lane], sv = mine[1][lane];
                c[0] = c[1] = cv.x; c[2] = c[3] = cv.y; c[4] = c[5] = cv.z; c[6] = c[7] = cv.w;
                s[1] = sv.x; s[3] = sv.y; s[5] = sv.z; s[7] = sv.w;
                s[0] = -sv.x; s[2] = -sv.y; s[4] = -sv.z; s[6] = -sv.w;
            } else {
                const float sign = second ? 1.f : -1.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 cv = mine[e][lane], sv = mine[2 + e][lane];
                    c[4 * e] = cv.x; c[4 * e + 1] = cv.y; c[4 * e + 2] = cv.z; c[4 * e + 3] = cv.w;
                    s[4 * e] = sign * sv.x; s[4 * e + 1] = sign * sv.y;
                    s[4 * e + 2] = sign * sv.z; s[4 * e + 3] = sign * sv.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            A[i] = pair(wo[2 * i] * c[2 * i], wo[2 * i + 1] * c[2 * i + 1]);
            B[i] = pair(wp[2 * i] * s[2 * i], wp[2 * i + 1] * s[2 * i + 1]);
        }
    };

    auto squares = [&](const uint4 &row) {  // of this lane's dims
        const uint32_t w[4] = {row.x, row.y, row.z, row.w};
        f32x2 ss = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 x = pair_bf16(w[i]);
            ss = fma(x, x, ss);
        }
        float even, odd;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(even), "=f"(odd) : "l"(ss));
        return even + odd;
    };
    auto inverse = [&](float sum) {  // (rsqrt: within 2 units in the last place of fp32)
        return rsqrtf(sum * (1.f / kD) + a.eps);
    };
    auto inverse_of = [&](const uint4 &row) {  // (all lanes of the warp)
        float sum = squares(row);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        return inverse(sum);
    };
    auto turned = [&](const uint4 &row, float inv) {  // (all lanes of the warp)
        const uint32_t w[4] = {row.x, row.y, row.z, row.w};
        const f32x2 inv2 = pair(inv, inv);
        uint32_t res[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t y = kNeighbours ? __byte_perm(w[i], 0, 0x1032)
                                           : __shfl_sync(0xffffffffu, w[i], sub * kLanes + partner);
            res[i] = pack(mul(inv2, fma(pair_bf16(y), B[i], mul(pair_bf16(w[i]), A[i]))));
        }
        return make_uint4(res[0], res[1], res[2], res[3]);
    };
    auto to_cache = [&](uint8_t *cache, int h, const uint4 &row) {
        if (run < 0) return;
        if (kCache == 1) {
            *reinterpret_cast<uint4 *>(cache + 2 * (run + h * kD + 8 * l)) = row;
        } else {  // one row a warp: warp-uniform
            q4_store_row(row, lane, cache + run + (int64_t)h * a.block_size * kQ4RowBytes, a.block_size, o);
        }
    };

    // The shuffles need whole warps, so a warp goes on while any of its rows is left.
    factors(a.q_weight);
    // A warp with several whole rows sums them together: each step of the reduction halves the
    // rows that a lane has (9 exchanges and 7 for the results, instead of 5 a row), and every
    // lane takes one row's root.
    const bool joint = kD == 256 && unit + step < hq;
    float inv[kBatch + 1];
    if (joint) {
        static_assert(kBatch + 1 <= 8, "eight sums a warp");
        float v[8];
#pragma unroll
        for (int b = 0; b < 8; ++b)
            v[b] = b < kBatch ? squares(raw[b]) : b == kBatch ? squares(raw_k) : 0.f;
#pragma unroll
        for (int n = 4, d = 16; n > 0; n >>= 1, d >>= 1)
#pragma unroll
            for (int b = 0; b < n; ++b) {
                const bool up = (lane & d) != 0;
                const float send = up ? v[b] : v[b + n], keep = up ? v[b + n] : v[b];
                v[b] = keep + __shfl_xor_sync(0xffffffffu, send, d);
            }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        const float mine = inverse(v[0]);
#pragma unroll
        for (int b = 0; b <= kBatch; ++b) inv[b] = __shfl_sync(0xffffffffu, mine, 4 * b);
    }
    uint16_t *q_out = a.q_out + t * a.q_out_stride + 8 * l;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const int r = unit + b * step;
        if (r - sub >= hq) break;  // warp-uniform
        const uint4 out = turned(raw[b], joint ? inv[b] : inverse_of(raw[b]));
        if (live && r < hq) *reinterpret_cast<uint4 *>(q_out + r * kD) = out;
        if (more) raw[b] = row_of(q_at, r, hq);
    }
    for (int r = unit + kBatch * step; r - sub < hq; r += step) {  // many heads
        const uint4 row = row_of(a.q + t * a.q_stride, r, hq), out = turned(row, inverse_of(row));
        if (live && r < hq) *reinterpret_cast<uint4 *>(q_out + r * kD) = out;
    }
    if (unit_k - sub < hkv) factors(a.k_weight);
    for (int r = unit_k; r - sub < hkv; r += step) {
        const uint4 row = r == unit_k ? raw_k : row_of(a.k + t * a.k_stride, r, hkv);
        const uint4 out = turned(row, joint && r == unit_k ? inv[kBatch] : inverse_of(row));
        if (live && r < hkv) {
            if (kCache == 0)
                *reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride + r * kD + 8 * l) = out;
            else
                to_cache(a.k_cache, r, out);
        }
    }
    if (kCache)
        for (int r = unit_v; r < hkv; r += step)
            to_cache(a.v_cache, r, r == unit_v ? raw_v : row_of(a.v + t * a.v_stride, r, hkv));
    if (more) {
        raw_k = row_of(k_at, unit_k, hkv);
        if (kCache) raw_v = row_of(v_at, unit_v, hkv);
    }
    }
}

template <int kD>
cudaError_t launch_dim(RopeArgs a, cudaStream_t stream) {
    constexpr int per = kWarps * (256 / kD);
    // A small call: a row a warp, as many CTAs a token as that takes.  A large one: a token over as
    // few CTAs as give each warp kBatch query rows, and four CTAs an SM that go from token to token.
    // Small is what is resident at once, with the rows of a call that writes the cache (so that the
    // calls with and without a cache sum a row in the same order).  24 + 4 + 4 heads of 256, 8 CTAs
    // a token, small and large: 16 tokens 2.3 and 2.9 us, 64 2.7 and 3.0, 128 4.5 and 2.9, 256 7.3
    // and 3.4, 512 14.3 and 5.5; 32 + 8 + 8 heads, 12 CTAs: 16 tokens 2.3 and 2.8, 64 4.2 and 2.8;
    // 16 + 4 + 4 of 64, 2 CTAs: 128 tokens 2.3 and 2.3, 384 4.0 and 2.8.
    const int y_small = (a.num_q_heads + 2 * a.num_kv_heads + per - 1) / per;
    const bool small = (int64_t)a.num_tokens * y_small <= 4 * a.num_sms;
    const int y = small ? y_small : (a.num_q_heads + per * kBatch - 1) / (per * kBatch);
    constexpr int one = 256 / kD;  // rows of a warp
    const int step = y * per;
    a.shift_k = (a.num_q_heads + one - 1) / one * one % step;
    a.shift_v = (a.shift_k + (a.num_kv_heads + one - 1) / one * one) % step;
    const int x = small ? a.num_tokens : std::min(a.num_tokens, std::max(1, 4 * a.num_sms / y));
    const dim3 grid(x, y), block(kWarps * 32);
    if (a.interleaved) {
        if (a.cache == 0) return launch_pdl(qk_norm_rope_kernel<kD, true, 0>, grid, block, 0, stream, a);
        if (a.cache == 1) return launch_pdl(qk_norm_rope_kernel<kD, true, 1>, grid, block, 0, stream, a);
        if constexpr (kD == kHeadDim)
            return launch_pdl(qk_norm_rope_kernel<kD, true, 2>, grid, block, 0, stream, a);
    } else {
        if (a.cache == 0) return launch_pdl(qk_norm_rope_kernel<kD, false, 0>, grid, block, 0, stream, a);
        if (a.cache == 1) return launch_pdl(qk_norm_rope_kernel<kD, false, 1>, grid, block, 0, stream, a);
        if constexpr (kD == kHeadDim)
            return launch_pdl(qk_norm_rope_kernel<kD, false, 2>, grid, block, 0, stream, a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, cudaStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch_dim<64>(a, stream);
        case 128: return launch_dim<128>(a, stream);
        default: return launch_dim<256>(a, stream);
    }
}

}  // namespace pa
