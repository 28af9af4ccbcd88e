// pa_cache_q8.cu -- writes into and reads from the 8-bit cache (format: pa_q8.cuh), and the
// expansion that the prefill reads.
//
// Write.  For a block (16 tokens of a page) with the new rows W, old scale byte b and codes c:
//     need = the smallest byte with |x| <= 448 2^(need - 127) for every finite x of W (1 at least)
//     b'   = max(b, need)      (need alone where W has the block's first row, or b = 255)
//     rows of W: rne(x 2^(127 - b')); the others: rne(c 2^(b - b')) where b' > b
// The tokens of a block share its scale, so one warp has to see them all, wherever in the call
// they stand.  A CTA takes a range of tokens, notes which blocks they fall into (a bitmap by
// slot / 16 and a list), and looks through the slots of the whole call for further tokens of
// these blocks; of a block's tokens the first one's CTA writes it.  So the result does not depend
// on the order of tokens, no two CTAs touch one block, and of tokens that share a slot the last
// one counts.  The look through the slots costs 8 bytes of L2 a slot and CTA.
#include "pa_internal.h"
#include "pa_q8.cuh"

namespace pa {

namespace {

constexpr int kWarps = 8;
constexpr int kWriteWarps = 16;
constexpr int kMaxRange = 16;      // tokens of a CTA of the write
constexpr int kScan = 8;           // slots of a thread in flight
constexpr int kMapBits = 4096;

__device__ __forceinline__ uint32_t map_bit(long long slot) { return (uint32_t)(slot >> 4) % kMapBits; }

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7fff7fffu); }

// The largest of 16-bit magnitudes in the halves of every lane's word.
__device__ __forceinline__ uint32_t warp_top(uint32_t m) {
    return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
}

// A BF16 pair with infinities (and NaN) as NaN, or as 0.
template <bool kZero>
__device__ __forceinline__ uint32_t without_inf(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w = (w & 0xffff0000u) | (kZero ? 0u : 0x7fc0u);
    if ((w & 0x7f800000u) == 0x7f800000u) w = (w & 0xffffu) | (kZero ? 0u : 0x7fc00000u);
    return w;
}

// Eight BF16 values times f, as codes.
__device__ __forceinline__ uint2 codes_of(const uint4 &v, float f) {
    return make_uint2(e4m3x4(bf16_lo(v.x) * f, bf16_hi(v.x) * f, bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                      e4m3x4(bf16_lo(v.z) * f, bf16_hi(v.z) * f, bf16_lo(v.w) * f, bf16_hi(v.w) * f));
}

// Four codes times f (a power of two below 1), as codes.
__device__ __forceinline__ uint32_t codes_down(uint32_t c, float f) {
    const uint32_t lo = f16x2_of_e4m3(c), hi = f16x2_of_e4m3_hi(c);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// Two warps for each head of K and of V: the first and the last 8 rows of a block, 8 dims a lane.
__global__ void __launch_bounds__(kWriteWarps * 32, 2) write_q8_kernel(const Q8WriteArgs a) {
    constexpr int kThreads = kWriteWarps * 32, kHalf = kQ8Tokens / 2;
    __shared__ long long first[kMaxRange];  // a block's first slot
    __shared__ int rows[kMaxRange];         // its rows in the page (0: no block)
    __shared__ int lowest[kMaxRange];       // its first token
    __shared__ __align__(16) int token[kMaxRange][kQ8Tokens];
    __shared__ uint32_t map[kMapBits / 32];
    __shared__ uint32_t tops[2][kWriteWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * a.range, n = min(a.range, a.num_tokens - t0);
    const int h = blockIdx.y * (kWriteWarps / 4) + (warp >> 2);  // this warp's head
    const bool is_v = warp & 2;                                  // of K or of V
    const int r0 = (warp & 1) * kHalf;                           // its first row
    const uint16_t *x = (is_v ? a.value : a.key) + (int64_t)h * kHeadDim + 8 * lane;
    const int64_t x_stride = is_v ? a.value_stride : a.key_stride;
    pdl_wait();
    pdl_trigger();
    // The first slots of all, and the rows of this CTA's tokens, are on their way while the
    // blocks are found.
    long long s[kScan];
#pragma unroll
    for (int k = 0; k < kScan; ++k) {
        const int j = threadIdx.x + k * kThreads;
        s[k] = j < a.num_tokens ? a.slot_mapping[j] : -1;
    }
    const long long slot = warp == 0 && lane < n ? a.slot_mapping[t0 + lane] : -1;
    if (h < a.num_kv_heads)
        for (int i = (lane >> 2) + r0; i < n; i += kQ8Tokens)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(x + (int64_t)(t0 + i) * x_stride - 8 * lane + 64 * (lane & 3)));
    for (int i = threadIdx.x; i < kMapBits / 32; i += kThreads) map[i] = 0;
    for (int i = threadIdx.x; i < kMaxRange * kQ8Tokens; i += kThreads) (&token[0][0])[i] = -1;
    if (threadIdx.x < kMaxRange) {
        rows[threadIdx.x] = 0;
        lowest[threadIdx.x] = 0x7fffffff;
    }
    __syncthreads();
    if (warp == 0) {
        long long f = -1;
        int count = 0;
        if (slot >= 0) {
            const int64_t page = q8_page_of(slot, a.block_size);
            const int o = (int)(slot - page * a.block_size) & ~(kQ8Tokens - 1);
            if (page < a.num_pages) {
                f = page * a.block_size + o;
                count = min(kQ8Tokens, a.block_size - o);
            } else if (blockIdx.y == 0) {
                atomicOr(a.err, kErrSlot);
            }
        }
        const unsigned same = __match_any_sync(0xffffffffu, f);
        if (f >= 0 && __ffs(same) - 1 == lane) {
            first[lane] = f;
            rows[lane] = count;
            // (a block's slots may lie in two of the map's sixteens)
            for (const uint32_t bit : {map_bit(f), map_bit(f + count - 1)})
                atomicOr(&map[bit / 32], 1u << (bit % 32));
        }
    }
    __syncthreads();
    for (int j0 = 0; j0 < a.num_tokens; j0 += kScan * kThreads) {
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const int j = j0 + threadIdx.x + k * kThreads;
            if (j0 > 0) s[k] = j < a.num_tokens ? a.slot_mapping[j] : -1;
        }
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const uint32_t bit = map_bit(s[k]);
            if (map[bit / 32] >> (bit % 32) & 1)
                for (int e = 0; e < n; ++e) {
                    const unsigned long long at = (unsigned long long)(s[k] - first[e]);
                    if (rows[e] && at < (unsigned)rows[e]) {
                        const int j = j0 + threadIdx.x + k * kThreads;
                        atomicMax(&token[e][at], j);
                        atomicMin(&lowest[e], j);
                    }
                }
        }
    }
    __syncthreads();
    if (h >= a.num_kv_heads) return;
    const int64_t row_stride = (int64_t)a.num_kv_heads * kHeadDim;
    int turn = 0;
    for (int e = 0; e < n; ++e) {
        const int in_page = rows[e];
        if (in_page == 0 || lowest[e] < t0) continue;  // none, or another CTA's
        const long long f = first[e];
        const int64_t page = q8_page_of(f, a.block_size);
        const int o = (int)(f - page * a.block_size);
        uint8_t *scale = (is_v ? a.v_scales : a.k_scales) + page * a.scale_stride +
                         (int64_t)(o / kQ8Tokens) * a.num_kv_heads + h;
        const uint32_t old = *scale;
        const int4 at[2] = {*reinterpret_cast<const int4 *>(&token[e][r0]),
                            *reinterpret_cast<const int4 *>(&token[e][r0 + 4])};
        auto token_of = [&](int i) { return (&at[i / 4].x)[i % 4]; };
        uint4 v[kHalf];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (token_of(i) >= 0) v[i] = __ldg(reinterpret_cast<const uint4 *>(x + token_of(i) * x_stride));
        }
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
            top = abs_max2(abs_max2(abs_max2(abs_max2(top, v[i].x), v[i].y), v[i].z), v[i].w);
        uint32_t m = warp_top(top);
        if (m >= 0x7f80u) {  // infinities and NaN: codes of NaN, and no part in the scale
            top = 0;
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                top = abs_max2(abs_max2(top, without_inf<true>(v[i].x)), without_inf<true>(v[i].y));
                top = abs_max2(abs_max2(top, without_inf<true>(v[i].z)), without_inf<true>(v[i].w));
                v[i].x = without_inf<false>(v[i].x);
                v[i].y = without_inf<false>(v[i].y);
                v[i].z = without_inf<false>(v[i].z);
                v[i].w = without_inf<false>(v[i].w);
            }
            m = warp_top(top);
        }
        // The two warps meet; both have read the old byte by then.
        if (lane == 0) tops[turn][warp] = m;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
        m = max(m, tops[turn][warp ^ 1]);
        turn ^= 1;
        // m = 1.f 2^(E - 127) <= 448 2^(b - 127) = 1.75 2^8 2^(b - 127): b = E - 8, or one more
        // where f > .75
        const uint32_t need = (uint32_t)max(1, (int)(m >> 7) - 8 + ((m & 127u) > 96u ? 1 : 0));
        const bool anew = token[e][0] >= 0 || old == 255;
        const uint32_t b = anew ? need : max(old, need);
        const float up = b == 254 ? 0x1p-127f : __uint_as_float((254 - b) << 23);
        uint8_t *row = (is_v ? a.v_cache : a.k_cache) + page * a.page_stride +
                       ((int64_t)(o + r0) * a.num_kv_heads + h) * kHeadDim + 8 * lane;
        if (lane == 0 && r0 == 0 && b != old) *scale = (uint8_t)b;
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
            if (token_of(i) >= 0) *reinterpret_cast<uint2 *>(row + i * row_stride) = codes_of(v[i], up);
        if (!anew && b > old) {
            const float down = b - old > 126 ? 0.f : __uint_as_float((127 - (b - old)) << 23);
            uint2 c[kHalf];
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
                if (r0 + i < in_page && token_of(i) < 0) c[i] = *reinterpret_cast<const uint2 *>(row + i * row_stride);
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
                if (r0 + i < in_page && token_of(i) < 0)
                    *reinterpret_cast<uint2 *>(row + i * row_stride) =
                        make_uint2(codes_down(c[i].x, down), codes_down(c[i].y, down));
        }
    }
}

// Eight codes times f, rounded to BF16.
__device__ __forceinline__ uint4 widen8(const uint2 &c, float f) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? c.x : c.y, x = i & 1 ? f16x2_of_e4m3_hi(w) : f16x2_of_e4m3(w);
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&x));
        r[i] = pack_bf16x2(p.x * f, p.y * f);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Read back by slots: warp per (token, head), K and V of it, 8 dims a lane; the warps of a CTA
// on one head, kTok tokens each.
template <int kTok>
__global__ void __launch_bounds__(kWarps * 32) gather_q8_kernel(const Q8GatherArgs a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * (kWarps * kTok) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    int64_t slot[kTok];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
        const int64_t t = t0 + k * kWarps;
        slot[k] = t < a.num_tokens ? a.slot_mapping[t] : -1;
    }
    uint2 ck[kTok], cv[kTok];
    uint32_t bk[kTok], bv[kTok];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
        ck[k] = cv[k] = make_uint2(0, 0);  // padding, and a slot outside the pool
        bk[k] = bv[k] = 127;
        if (slot[k] < 0) continue;
        const int64_t page = q8_page_of(slot[k], a.block_size);
        if (page < a.num_pages) {
            const int o = (int)(slot[k] - page * a.block_size);
            const int64_t at = page * a.page_stride + ((int64_t)o * a.num_kv_heads + h) * kHeadDim;
            const int64_t sat = page * a.scale_stride + (int64_t)(o / kQ8Tokens) * a.num_kv_heads + h;
            ck[k] = __ldg(reinterpret_cast<const uint2 *>(a.k_cache + at) + lane);
            cv[k] = __ldg(reinterpret_cast<const uint2 *>(a.v_cache + at) + lane);
            bk[k] = __ldg(a.k_scales + sat);
            bv[k] = __ldg(a.v_scales + sat);
        } else if (lane == 0) {
            atomicOr(a.err, kErrSlot);
        }
    }
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
        const int64_t t = t0 + k * kWarps;
        if (t >= a.num_tokens) return;
        const int64_t row = (t * a.num_kv_heads + h) * kHeadDim;
        reinterpret_cast<uint4 *>(a.k_out + row)[lane] = widen8(ck[k], q8_scale(bk[k]));
        reinterpret_cast<uint4 *>(a.v_out + row)[lane] = widen8(cv[k], q8_scale(bv[k]));
    }
}

// ---- prefill: operands from the 8-bit cache
//
// K becomes BF16, which holds a code times a power of two exactly, so that the scores are those of
// the BF16 queries as they are.  V becomes FP16, which its products with FP16 weights need (a weight
// takes one FP16 part, but two BF16 ones): a head's codes times 2^(6 + b - its largest b), 2^15
// at most, exact while a block's scale is down to 2^-15 of the head's largest (and then for all codes
// but those near 2^-9).

// The largest scale byte of V (but 255) over kExpandRange keys of one head.
__global__ void __launch_bounds__(kWarps * 32) range_q8_kernel(const __grid_constant__ ExpandArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x / a.num_ranges, range = blockIdx.x - h * a.num_ranges;
    int b = 0;
    while (b + 1 < a.num_seqs && range >= a.seq[b + 1].range0) ++b;
    const ExpandSeq s = a.seq[b];
    const int32_t *bt = a.block_table + (int64_t)s.bt_row * a.bt_stride;
    const int k0 = (range - s.range0) * kExpandRange;
    const int k1 = min(s.num_keys, k0 + kExpandRange);
    uint32_t top = 0;
    // (a block counts with its first key in the range, which need not be its first row)
    for (int k = k0 + threadIdx.x; k < k1; k += kWarps * 32) {
        const int lp = k / a.block_size, o = k - lp * a.block_size;
        if (o % kQ8Tokens && k > k0) continue;
        const int page = bt[lp];
        if (page < 0 || page >= a.num_pages) continue;  // reported by the expansion
        const uint32_t vb = __ldg(a.v_scales + page * a.scale_stride + (int64_t)(o / kQ8Tokens) * a.num_kv_heads + h);
        if (vb != 255) top = max(top, vb);
    }
    __shared__ uint32_t part[kWarps];
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) part[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w) top = max(top, part[w]);
        a.ranges[(int64_t)h * a.num_ranges + range] = make_float2(0.f, (float)top);
    }
}

// An FP16 pair of 2^e, e <= 6: exact down to 2^-24.
__device__ __forceinline__ __half2 half2_pow2(int e) { return __float2half2_rn(__uint_as_float((uint32_t)(e + 127) << 23)); }

// Eight codes times 2^d as FP16.
__device__ __forceinline__ uint4 expand8(const uint2 &c, int d, bool nan) {
    const __half2 f = nan ? __float2half2_rn(__uint_as_float(0x7fc00000u)) : half2_pow2(max(d, -15));
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? c.x : c.y, x = i & 1 ? f16x2_of_e4m3_hi(w) : f16x2_of_e4m3(w);
        __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x), f);  // exact
        if (d < -15) y = __hmul2(y, half2_pow2(max(d + 15, -24)));
        r[i] = *reinterpret_cast<uint32_t *>(&y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Warp per (key, head), K and V of it, 8 dims a lane; the warps of a CTA on consecutive keys of one
// head, a warp's kExpandKeys / kWarps keys in flight together.
__global__ void __launch_bounds__(kWarps * 32) expand_q8_kernel(const __grid_constant__ ExpandArgs a) {
    constexpr int kRows = kExpandKeys / kWarps;  // keys of a warp
    __shared__ uint32_t part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    const int64_t key0 = (int64_t)blockIdx.x * kExpandKeys;  // of the stacked, page-padded keys
    int b = 0;
    while (b + 1 < a.num_seqs && key0 >= (int64_t)a.seq[b + 1].page0 * kExpandPage) ++b;
    const ExpandSeq sq = a.seq[b];
    const int k0 = (int)(key0 - (int64_t)sq.page0 * kExpandPage);  // key of the sequence
    pdl_wait();
    pdl_trigger();
    if (h == 0 && k0 % kExpandPage == 0 && threadIdx.x == 0)
        a.table_out[(int64_t)b * a.table_stride + k0 / kExpandPage] = sq.page0 + k0 / kExpandPage;
    const int32_t *bt = a.block_table + (int64_t)sq.bt_row * a.bt_stride;
    uint2 ck[kRows], cv[kRows];
    uint32_t bk[kRows], bv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int k = k0 + i * kWarps + warp;
        ck[i] = cv[i] = make_uint2(0, 0);  // a page outside the pool reads as zeros
        bk[i] = bv[i] = 0;
        if (k >= sq.num_keys) continue;
        const int lp = k / a.block_size, o = k - lp * a.block_size, page = bt[lp];
        if (page >= 0 && page < a.num_pages) {
            const int64_t at = page * a.page_stride + ((int64_t)o * a.num_kv_heads + h) * kHeadDim;
            const int64_t sat = page * a.scale_stride + (int64_t)(o / kQ8Tokens) * a.num_kv_heads + h;
            ck[i] = __ldg(reinterpret_cast<const uint2 *>(a.k_cache + at) + lane);
            cv[i] = __ldg(reinterpret_cast<const uint2 *>(a.v_cache + at) + lane);
            bk[i] = __ldg(a.k_scales + sat);
            bv[i] = __ldg(a.v_scales + sat);
        } else if (lane == 0) {
            atomicOr(a.err, kErrPage);
        }
    }
    // The head's largest scale of V, from all of its sequence's ranges.
    uint32_t top = 0;
    const int nr = (sq.num_keys - 1) / kExpandRange + 1;
    for (int i = threadIdx.x; i < nr; i += kWarps * 32)
        top = max(top, (uint32_t)a.ranges[(int64_t)h * a.num_ranges + sq.range0 + i].y);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) part[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, part[w]);
    if (k0 == 0 && threadIdx.x == 0)  // 2^(b - 133)
        a.kv_factor[b * a.num_kv_heads + h] = make_float2(1.f, q8_scale(top) * 0x1p-6f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int k = i * kWarps + warp;
        if (k0 + k >= sq.num_keys) return;
        const int64_t dst = ((key0 + k) * a.num_kv_heads + h) * kHeadDim;
        reinterpret_cast<uint4 *>(a.k_out + dst)[lane] = widen8(ck[i], q8_scale(bk[i]));
        reinterpret_cast<uint4 *>(a.v_out + dst)[lane] = expand8(cv[i], 6 + (int)bv[i] - (int)top, bv[i] == 255);
    }
}

}  // namespace

cudaError_t launch_write_q8(const Q8WriteArgs &args, cudaStream_t stream) {
    Q8WriteArgs a = args;
    a.range = a.num_tokens <= 1024 ? 1 : a.num_tokens <= 2048 ? 8 : kMaxRange;
    return launch_pdl(write_q8_kernel,
                      dim3((unsigned)((a.num_tokens - 1) / a.range + 1),
                           (a.num_kv_heads + kWriteWarps / 4 - 1) / (kWriteWarps / 4)),
                      dim3(kWriteWarps * 32), 0, stream, a);
}

cudaError_t launch_gather_q8(const Q8GatherArgs &a, cudaStream_t stream) {
    const int tok = a.num_tokens > 1024 ? 2 : 1;
    const dim3 grid((unsigned)((a.num_tokens - 1) / (kWarps * tok) + 1), a.num_kv_heads);
    return tok == 2 ? launch_pdl(gather_q8_kernel<2>, grid, dim3(kWarps * 32), 0, stream, a)
                    : launch_pdl(gather_q8_kernel<1>, grid, dim3(kWarps * 32), 0, stream, a);
}

cudaError_t launch_expand_q8(const ExpandArgs &a, int64_t num_pages_out, cudaStream_t stream) {
    cudaError_t e = launch_pdl(range_q8_kernel, dim3((unsigned)a.num_ranges * a.num_kv_heads), dim3(kWarps * 32),
                               0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(expand_q8_kernel,
                      dim3((unsigned)(num_pages_out * (kExpandPage / kExpandKeys)), a.num_kv_heads),
                      dim3(kWarps * 32), 0, stream, a);
}

}  // namespace pa
