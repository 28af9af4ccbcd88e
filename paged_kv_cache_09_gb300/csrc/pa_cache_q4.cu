// pa_cache_q4.cu -- writes into and reads from the 4-bit cache (format: pa_q4.cuh).
//
// One warp per row (a token's 256 dims of one KV head), 8 dims a lane: a row is one
// 16-byte load per lane of BF16, one 4-byte word per lane of codes.  The kernels move bytes and
// are bound by memory (large calls) or by launch and one round trip (a decode batch's); the
// write also by its instructions (a group's bounds and 8 codes a lane, about 150).
// Measured with 4 KV heads: 4096 tokens written in 9.5 us and read back in 6.7 (2.3 and 3.2
// TB/s); 16 tokens written and read in 3.7 us together.
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {

namespace {

constexpr int kWarps = 8;  // rows in flight per CTA

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// KV write: warp per (token, head), K and V of it; the warps of a CTA on one head.
__global__ void __launch_bounds__(kWarps * 32) write_q4_kernel(const Q4WriteArgs a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (t >= a.num_tokens) return;
    const int64_t slot = a.slot_mapping[t];
    const uint4 k = __ldg(reinterpret_cast<const uint4 *>(a.key + t * a.key_stride + h * kHeadDim) + lane);
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(a.value + t * a.value_stride + h * kHeadDim) + lane);
    if (slot < 0) return;
    const int64_t page = page_of(slot, a.block_size);
    if (page >= a.num_pages) {
        if (lane == 0) atomicOr(a.err, kErrSlot);
        return;
    }
    const int o = (int)(slot - page * a.block_size);
    const int64_t run = page * a.page_stride + (int64_t)h * a.block_size * kQ4RowBytes;
    q4_store_row(k, lane, a.k_cache + run, a.block_size, o);
    q4_store_row(v, lane, a.v_cache + run, a.block_size, o);
}

// Read back by slots: warp per (token, head), K and V of it.
__global__ void __launch_bounds__(kWarps * 32) gather_q4_kernel(const Q4GatherArgs a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (t >= a.num_tokens) return;
    const int64_t slot = a.slot_mapping[t];
    uint4 k = make_uint4(0, 0, 0, 0), v = k;  // padding, and a slot outside the pool
    if (slot >= 0) {
        const int64_t page = page_of(slot, a.block_size);
        if (page < a.num_pages) {
            const int o = (int)(slot - page * a.block_size);
            const int64_t run = page * a.page_stride + (int64_t)h * a.block_size * kQ4RowBytes;
            k = q4_load_row(a.k_cache + run, a.block_size, o, lane);
            v = q4_load_row(a.v_cache + run, a.block_size, o, lane);
        } else if (lane == 0) {
            atomicOr(a.err, kErrSlot);
        }
    }
    const int64_t row = (t * a.num_kv_heads + h) * kHeadDim;
    reinterpret_cast<uint4 *>(a.k_out + row)[lane] = k;
    reinterpret_cast<uint4 *>(a.v_out + row)[lane] = v;
}

// ---- prefill: FP16 operands from the 4-bit cache and BF16 queries
//
// FP16 holds the values to 2^-11 (BF16 to 2^-8) but spans fewer binades, so each query row and
// each KV head of a sequence is scaled by the power of two that brings its largest magnitude
// to [2^14, 2^15).  Values down to 2^-28 of the largest keep 11 bits; smaller ones are off by up
// to 2^-39 of it.

// The power of two that brings magnitudes up to `top` below 2^15 (1 for 0 and non-finite).
__device__ __forceinline__ float scale_for(float top) {
    const int e = (int)(__float_as_uint(top) >> 23) & 255;
    if (e == 255 || top == 0.f) return 1.f;
    return __uint_as_float((uint32_t)min(254, max(1, 127 + 14 - (e - 127))) << 23);
}

// Blocks [0, num_ranges * num_kv_heads): bounds of |K| and |V| over kQ4RangeKeys keys of one
// head, from the groups' minima and steps alone.  The other blocks: kWarps rows of Q each.
// 13973 keys of 4 heads and 1685 x 24 query rows: 8.2 us (43 MB, nearly all of it the queries).
__global__ void __launch_bounds__(kWarps * 32)
    range_q4_kernel(const __grid_constant__ Q4ExpandArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int nr = a.num_ranges * a.num_kv_heads;
    if ((int)blockIdx.x >= nr) {
        const int64_t row = (int64_t)(blockIdx.x - nr) * kWarps + warp;
        if (row >= a.q_rows) return;
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
        return;
    }
    const int h = blockIdx.x / a.num_ranges, range = blockIdx.x - h * a.num_ranges;
    int b = 0;
    while (b + 1 < a.num_seqs && range >= a.seq[b + 1].range0) ++b;
    const Q4ExpandSeq s = a.seq[b];
    const int32_t *bt = a.block_table + (int64_t)s.bt_row * a.bt_stride;
    const int k0 = (range - s.range0) * kQ4RangeKeys;
    const int k1 = min(s.num_keys, k0 + kQ4RangeKeys);
    float top[2] = {0.f, 0.f};
    for (int k = k0 + threadIdx.x; k < k1; k += kWarps * 32) {
        const int lp = k / a.block_size, o = k - lp * a.block_size, page = bt[lp];
        if (page < 0 || page >= a.num_pages) continue;  // reported by the expansion
        const int64_t at = page * a.page_stride + (int64_t)h * a.block_size * kQ4RowBytes +
                           q4_pair_offset(a.block_size, o, 0);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4 p = __ldg(reinterpret_cast<const uint4 *>((kv ? a.v_cache : a.k_cache) + at));
            const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int g = 0; g < kQ4Groups; ++g) {
                const float lo = q4_low(w[g]), hi = fmaf(15.f, q4_step(w[g]), lo);
                const float m = fmaxf(fabsf(lo), fabsf(hi));
                if (m <= 3.4028235e38f) top[kv] = fmaxf(top[kv], m);
            }
        }
    }
    __shared__ float2 part[kWarps];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
    }
    if (lane == 0) part[warp] = make_float2(top[0], top[1]);
    __syncthreads();
    if (threadIdx.x == 0) {
        float2 t = part[0];
        for (int w = 1; w < kWarps; ++w) {
            t.x = fmaxf(t.x, part[w].x);
            t.y = fmaxf(t.y, part[w].y);
        }
        a.ranges[(int64_t)h * a.num_ranges + range] = t;
    }
}

// Eight codes of a word as FP16 pairs of (lo + s n), lo and s already scaled.
__device__ __forceinline__ uint4 widen_word(uint32_t w, float s, float lo) {
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        r[j] = pack_f16x2(fmaf(s, static_cast<float>((w >> (8 * j)) & 15u), lo),
                          fmaf(s, static_cast<float>((w >> (8 * j + 4)) & 15u), lo));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Warp per (key, head), the warps of a CTA on consecutive keys of one head, whose codes are
// one contiguous run; kWarps keys' loads in flight a round.  13973 keys of 4 heads: 15.6 us (16 MB
// read, 57 MB written: 4.7 TB/s).
__global__ void __launch_bounds__(kWarps * 32)
    expand_q4_kernel(const __grid_constant__ Q4ExpandArgs a) {
    constexpr int kRows = kQ4ExpandKeys / kWarps;  // keys of a warp
    __shared__ float2 part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    const int64_t key0 = (int64_t)blockIdx.x * kQ4ExpandKeys;  // of the stacked, page-padded keys
    int b = 0;
    while (b + 1 < a.num_seqs && key0 >= (int64_t)a.seq[b + 1].page0 * kQ4PrefillPage) ++b;
    const Q4ExpandSeq sq = a.seq[b];
    const int k0 = (int)(key0 - (int64_t)sq.page0 * kQ4PrefillPage);  // key of the sequence
    const int g = lane >> 3, u = lane & 7;
    pdl_wait();
    pdl_trigger();
    if (h == 0 && k0 % kQ4PrefillPage == 0 && threadIdx.x == 0)
        a.table_out[(int64_t)b * a.table_stride + k0 / kQ4PrefillPage] = sq.page0 + k0 / kQ4PrefillPage;
    // This warp's words and pairs, all loads in flight.
    const int32_t *bt = a.block_table + (int64_t)sq.bt_row * a.bt_stride;
    uint32_t kw[kRows], vw[kRows], kp[kRows], vp[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int k = k0 + i * kWarps + warp;
        kw[i] = vw[i] = kp[i] = vp[i] = 0;  // a page outside the pool reads as zeros
        if (k >= sq.num_keys) continue;
        const int lp = k / a.block_size, o = k - lp * a.block_size, page = bt[lp];
        if (page >= 0 && page < a.num_pages) {
            const int64_t run = page * a.page_stride + (int64_t)h * a.block_size * kQ4RowBytes;
            const int64_t cw = run + q4_word_offset(o, u, g), cp = run + q4_pair_offset(a.block_size, o, g);
            kw[i] = __ldg(reinterpret_cast<const uint32_t *>(a.k_cache + cw));
            vw[i] = __ldg(reinterpret_cast<const uint32_t *>(a.v_cache + cw));
            kp[i] = __ldg(reinterpret_cast<const uint32_t *>(a.k_cache + cp));
            vp[i] = __ldg(reinterpret_cast<const uint32_t *>(a.v_cache + cp));
        } else if (lane == 0) {
            atomicOr(a.err, kErrPage);
        }
    }
    // The head's scales, from all of its sequence's ranges.
    float2 top = make_float2(0.f, 0.f);
    const int nr = (sq.num_keys - 1) / kQ4RangeKeys + 1;
    for (int i = threadIdx.x; i < nr; i += kWarps * 32) {
        const float2 t = a.ranges[(int64_t)h * a.num_ranges + sq.range0 + i];
        top.x = fmaxf(top.x, t.x);
        top.y = fmaxf(top.y, t.y);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, d));
        top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, d));
    }
    if (lane == 0) part[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        top.x = fmaxf(top.x, part[w].x);
        top.y = fmaxf(top.y, part[w].y);
    }
    const float fk = scale_for(top.x), fv = scale_for(top.y);
    if (k0 == 0 && threadIdx.x == 0)
        a.kv_factor[b * a.num_kv_heads + h] = make_float2(1.f / fk, 1.f / fv);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int k = i * kWarps + warp;
        if (k0 + k >= sq.num_keys) return;
        const int64_t dst = ((key0 + k) * a.num_kv_heads + h) * kHeadDim;
        reinterpret_cast<uint4 *>(a.k_out + dst)[lane] =
            widen_word(kw[i], q4_step(kp[i]) * fk, q4_low(kp[i]) * fk);
        reinterpret_cast<uint4 *>(a.v_out + dst)[lane] =
            widen_word(vw[i], q4_step(vp[i]) * fv, q4_low(vp[i]) * fv);
    }
}

dim3 row_grid(int num_tokens, int num_kv_heads) {
    return dim3((unsigned)((num_tokens - 1) / kWarps + 1), num_kv_heads);
}

}  // namespace

cudaError_t launch_write_q4(const Q4WriteArgs &a, cudaStream_t stream) {
    return launch_pdl(write_q4_kernel, row_grid(a.num_tokens, a.num_kv_heads), dim3(kWarps * 32), 0,
                      stream, a);
}

cudaError_t launch_gather_q4(const Q4GatherArgs &a, cudaStream_t stream) {
    return launch_pdl(gather_q4_kernel, row_grid(a.num_tokens, a.num_kv_heads), dim3(kWarps * 32), 0,
                      stream, a);
}

cudaError_t launch_expand_q4(const Q4ExpandArgs &a, int64_t num_pages_out, cudaStream_t stream) {
    const int64_t blocks = (int64_t)a.num_ranges * a.num_kv_heads + (a.q_rows + kWarps - 1) / kWarps;
    cudaError_t e = launch_pdl(range_q4_kernel, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(expand_q4_kernel,
                      dim3((unsigned)(num_pages_out * (kQ4PrefillPage / kQ4ExpandKeys)),
                           a.num_kv_heads),
                      dim3(kWarps * 32), 0, stream, a);
}

}  // namespace pa
