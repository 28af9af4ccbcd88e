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
// and one round trip for a decode batch.  D / 8 lanes hold a row, 8 dims (16 bytes) a lane:
// the sum of squares is a few shuffles, a half-rotation's partner is the same register of
// another lane.  A CTA works on one token, so that the warps' cosines and sines come
// through L1 and stay in registers from row to row.
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {

namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4;  // rows of a warp whose loads are in flight together

template <int kD, bool kNeighbours, int kCache>  // kCache: 0 none, 1 BF16, 2 4-bit
__global__ void __launch_bounds__(kWarps * 32)
    qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kLanes = kD / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a warp
    static_assert(kCache != 2 || kD == kHeadDim, "the 4-bit cache holds rows of 256");
    const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
    const int unit = (blockIdx.y * kWarps + (threadIdx.x >> 5)) * kPer + sub;
    const int step = gridDim.y * kWarps * kPer;
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int pos = a.positions[t];
    if (pos < 0) return;  // padding: the token's rows stay as they are
    if (pos >= a.max_position) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrPosition);
        return;
    }
    int64_t run = -1;  // the slot's place in the caches (of head 0)
    int o = 0;
    if (kCache) {
        const int64_t slot = a.slot_mapping[t];
        if (slot >= 0) {
            const int64_t page = slot / a.block_size;
            o = (int)(slot - page * a.block_size);
            if (page < a.num_pages)
                run = kCache == 1
                          ? page * a.page_stride + (int64_t)o * a.num_kv_heads * kD
                          : page * a.page_stride;
            else if (threadIdx.x == 0 && blockIdx.y == 0)
                atomicOr(a.err, kErrSlot);
        }
    }
    // This lane's angles: dims 8l .. 8l + 7.
    const int R = a.rotary_dim, half = R / 2;
    const bool turns = 8 * l < R;
    const bool second = 8 * l >= half;  // of a pair of halves
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        c[j] = 1.f;
        s[j] = 0.f;
    }
    if (turns) {
        const float *row = a.cos_sin + (int64_t)pos * R;
        if (kNeighbours) {
            const float4 cv = __ldg(reinterpret_cast<const float4 *>(row + 4 * l));
            const float4 sv = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * l));
            c[0] = c[1] = cv.x; c[2] = c[3] = cv.y; c[4] = c[5] = cv.z; c[6] = c[7] = cv.w;
            s[1] = sv.x; s[3] = sv.y; s[5] = sv.z; s[7] = sv.w;
            s[0] = -sv.x; s[2] = -sv.y; s[4] = -sv.z; s[6] = -sv.w;
        } else {
            const int i = second ? 8 * l - half : 8 * l;
            const float sign = second ? 1.f : -1.f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4 cv = __ldg(reinterpret_cast<const float4 *>(row + i) + v);
                const float4 sv = __ldg(reinterpret_cast<const float4 *>(row + half + i) + v);
                c[4 * v] = cv.x; c[4 * v + 1] = cv.y; c[4 * v + 2] = cv.z; c[4 * v + 3] = cv.w;
                s[4 * v] = sign * sv.x; s[4 * v + 1] = sign * sv.y;
                s[4 * v + 2] = sign * sv.z; s[4 * v + 3] = sign * sv.w;
            }
        }
    }
    const int partner = sub * kLanes + (second ? l - R / 16 : l + R / 16) % kLanes;

    const int rows = a.num_q_heads + (kCache ? 2 : 1) * a.num_kv_heads;
    // Rows of all warps of the token in steps; the shuffles need whole warps, so a warp
    // goes on while any of its rows is left.
    for (int r0 = unit - sub; r0 < rows; r0 += kBatch * step) {
        uint4 raw[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * step + sub;
            raw[b] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const uint16_t *src;
                if (r < a.num_q_heads)
                    src = a.q + t * a.q_stride + r * kD;
                else if (r < a.num_q_heads + a.num_kv_heads)
                    src = a.k + t * a.k_stride + (r - a.num_q_heads) * kD;
                else
                    src = a.v + t * a.v_stride + (r - a.num_q_heads - a.num_kv_heads) * kD;
                raw[b] = *(reinterpret_cast<const uint4 *>(src) + l);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * step + sub;
            if (r0 + b * step >= rows) break;  // warp-uniform
            const bool is_q = r < a.num_q_heads;
            const int h = is_q ? r : (r - a.num_q_heads) % a.num_kv_heads;
            const bool is_v = r >= a.num_q_heads + a.num_kv_heads;
            float x[8];
            {
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = bf16_lo(w[i]);
                    x[2 * i + 1] = bf16_hi(w[i]);
                }
            }
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            if (!is_v) {
                const float inv = 1.f / sqrtf(ss * (1.f / kD) + a.eps);
                const uint4 wr = __ldg(reinterpret_cast<const uint4 *>(is_q ? a.q_weight : a.k_weight) + l);
                const uint32_t w[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] *= inv * (bf16_lo(w[i]) + a.weight_bias);
                    x[2 * i + 1] *= inv * (bf16_hi(w[i]) + a.weight_bias);
                }
            }
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = kNeighbours ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner);
            if (!is_v && turns) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], c[j], y[j] * s[j]);
            }
            const uint4 out = is_v ? raw[b]
                                   : make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
            if (is_q) {
                if (r < rows)
                    *(reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + h * kD) + l) = out;
            } else if (kCache == 0) {
                if (r < rows)
                    *(reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride + h * kD) + l) = out;
            } else if (kCache == 1) {
                if (r < rows && run >= 0)
                    *(reinterpret_cast<uint4 *>((is_v ? a.v_cache : a.k_cache) + 2 * (run + h * kD)) + l) = out;
            } else if (run >= 0) {  // one row a warp: warp-uniform
                const uint32_t w[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = bf16_lo(w[i]);
                    x[2 * i + 1] = bf16_hi(w[i]);
                }
                q4_store_row(x, lane,
                             (is_v ? a.v_cache : a.k_cache) + run +
                                 (int64_t)h * a.block_size * kQ4RowBytes,
                             a.block_size, o);
            }
        }
    }
}

template <int kD>
cudaError_t launch_dim(const RopeArgs &a, cudaStream_t stream) {
    const int rows = a.num_q_heads + (a.cache ? 2 : 1) * a.num_kv_heads;
    constexpr int per = kWarps * (256 / kD);
    // A large call: the token's rows over one CTA, kBatch a warp.  A small one: more CTAs a
    // token, one row a warp.
    const int y = a.num_tokens >= 512 ? (rows + per * kBatch - 1) / (per * kBatch)
                                      : (rows + per - 1) / per;
    const dim3 grid(a.num_tokens, y), block(kWarps * 32);
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
