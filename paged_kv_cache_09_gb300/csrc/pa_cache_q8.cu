// pa_cache_q8.cu -- writes into and reads from the 8-bit cache (format: pa_q8.cuh), and the
// expansion that the prefill reads.
//
// Write.  For a block (16 tokens of a page) with the new rows W, old scale byte b and codes c:
//     need = the smallest byte with |x| <= 448 2^(need - 127) for every finite x of W (1 at least)
//     b'   = max(b, need)      (need alone where W has the block's first row, or b = 255)
//     rows of W: rne(x 2^(127 - b')); the others: rne(c 2^(b - b')) where b' > b
// The tokens of a block share its scale, so one warp has to see them all, wherever in the call
// they stand.  A CTA takes a range of tokens, notes which blocks they fall into (a bitmap by
// slot / 16 and a hash table), and looks through the slots of the whole call for further tokens of
// these blocks; of a block's tokens the first one's CTA writes it.  So the result does not depend
// on the order of tokens, no two CTAs touch one block, and of tokens that share a slot the last
// one counts.  (Rows, codes and scales may come from the kernel before, whose end this one's start
// overlaps: they are read with ordinary loads or past L1, not through the read-only path.)  The look
// through the slots costs 8 bytes of L2 a slot and CTA: with two CTAs an SM 2.4 KB a token, beside the 1.5
// KB that a token's row of each KV head takes.  A CTA takes 256 tokens at most, so from 78000 tokens on (4
// heads; 39000 with 8) there are more CTAs, and the look grows as the square of the tokens: 32768 of 4 heads
// 43 us (4.7 TB/s), 131072 201 (4.0), 262144 519 (3.1).
//
// Measured, 4 KV heads unless said: 16 tokens written in 2.6 us and 256 read in 1.7 (launch and three
// round trips: slots, rows, stores); 4096 written in 6.3 us and read in 4.6 (4.0 and 5.4 TB/s); 8192 in 11.6
// and 8.4; 12 x 333 tokens of 8 heads in 12.0 and 8.4.  The write's warps hold a block's 16 rows at
// once (64 registers): 16 warps an SM, and a call's first instructions are a fifth of its time.  With two
// warps a block and the blocks found by every 16 tokens, 4096 tokens took 9.1 us and 32768, whose every
// CTA looks through all slots, 121 (now 40).  Its code runs once a warp, so that it is fetched as it runs: a
// loop over the slots that may be of the CTA's blocks, instead of what follows such a slot written out for
// each of a thread's 16, took 4096 tokens from 7.2 to 6.4 us.
#include <algorithm>

#include "pa_internal.h"
#include "pa_q8.cuh"

namespace pa {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxRange = 256;     // tokens of a CTA of the write (its threads at most)
constexpr int kTableBits = 9, kTable = 1 << kTableBits;  // places for their blocks
constexpr int kMaxCut = 4;         // CTAs that share a range's heads (8 heads, 3996 tokens: 1, 2, 4: 16.2, 12.1, 12.1 us)
constexpr int kExpandLook = 16384;  // keys whose scales every CTA of the expansion looks at
constexpr int kScan = 16;          // slots of a thread in flight
constexpr int kMapBits = 16384;

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
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // (a pair is one instruction)
        asm("{.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1]) : "f"(bf16_lo(w[i])), "f"(bf16_hi(w[i])), "f"(f));
    return make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
}

// Four codes times f (a power of two below 1), as codes.
__device__ __forceinline__ uint32_t codes_down(uint32_t c, float f) {
    const uint32_t lo = f16x2_of_e4m3(c), hi = f16x2_of_e4m3_hi(c);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

__device__ __forceinline__ uint32_t hash_of(long long first) {
    return ((uint32_t)(first >> 4) * 0x9E3779B1u) >> (32 - kTableBits);
}

// Where a slot's block starts, its row in it and the block's rows; false: outside the pool.
struct Place {
    long long first;
    int row, rows;
};
__device__ __forceinline__ bool block_of(const Q8WriteArgs &a, long long slot, Place *p) {
    const int64_t page = q8_page_of(slot, a.block_size);
    const int o = (int)(slot - page * a.block_size);
    p->row = o % kQ8Tokens;
    p->first = slot - p->row;
    p->rows = min(kQ8Tokens, a.block_size - o + p->row);
    return page < a.num_pages;
}

// A warp for each block and head of K and of V, 8 dims of its 16 rows a lane.
// kOne: the CTA's range is one token, so there is one block, which needs no table.
template <bool kOne>
__global__ void __launch_bounds__(kWarps * 32, 2) write_q8_kernel(const __grid_constant__ Q8WriteArgs a) {
    constexpr int kThreads = kWarps * 32, kPlaces = kOne ? 1 : kTable, kSlots = kOne ? 2 : kScan;
    __shared__ long long keys[kPlaces];                       // first slots of blocks (-1: none)
    __shared__ int lowest[kPlaces];                           // a block's first token
    __shared__ __align__(16) int token[kPlaces][kQ8Tokens];   // the token of each row (-1: none)
    __shared__ int list[kOne ? 1 : kMaxRange], count;         // the blocks' places
    __shared__ uint32_t map[kOne ? 1 : kMapBits / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * a.range;
    const int n = (int)min((int64_t)a.range, a.num_tokens - t0);
    const int kinds = 2 * a.num_kv_heads;  // (head, K or V)
    pdl_wait();
    pdl_trigger();
    // The first slots of all, and the rows of this CTA's tokens, are on their way while the
    // blocks are found.
    long long s[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
        const int j = threadIdx.x + k * kThreads;
        s[k] = j < a.num_tokens ? a.slot_mapping[j] : -1;
    }
    const long long slot = kOne ? a.slot_mapping[t0] : (int)threadIdx.x < n ? a.slot_mapping[t0 + threadIdx.x] : -1;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < n * kinds * 4; i += gridDim.y * kThreads) {
        const int t = i / (kinds * 4), line = i - t * (kinds * 4), half = a.num_kv_heads * 4;
        const uint16_t *row = line < half ? a.key + (t0 + t) * a.key_stride + line * 64
                                          : a.value + (t0 + t) * a.value_stride + (line - half) * 64;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
    }
    Place own = {-1, 0, 0};
    const bool live = slot >= 0 && block_of(a, slot, &own);
    if (slot >= 0 && !live && blockIdx.y == 0 && (!kOne || threadIdx.x == 0)) atomicOr(a.err, kErrSlot);
    if constexpr (kOne) {
        if (!live) return;
        if (threadIdx.x < kQ8Tokens) token[0][threadIdx.x] = -1;
        if (threadIdx.x == 0) {
            keys[0] = own.first;
            lowest[0] = 0x7fffffff;
            list[0] = 0;
            count = 1;
        }
    } else {
        for (int i = threadIdx.x; i < kMapBits / 32; i += kThreads) map[i] = 0;
        for (int i = threadIdx.x; i < kTable; i += kThreads) keys[i] = -1;
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        if (live) {
            uint32_t at = hash_of(own.first);
            long long was;
            while ((was = (long long)atomicCAS(reinterpret_cast<unsigned long long *>(&keys[at]), ~0ull,
                                               (unsigned long long)own.first)) != -1 && was != own.first)
                at = (at + 1) % kTable;
            if (was == -1) {  // a new block
                lowest[at] = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < kQ8Tokens / 4; ++i)
                    reinterpret_cast<int4 *>(token[at])[i] = make_int4(-1, -1, -1, -1);
                list[atomicAdd(&count, 1)] = (int)at;
                // (its slots may lie in two of the map's sixteens)
                for (const uint32_t bit : {map_bit(own.first), map_bit(own.first + own.rows - 1)})
                    atomicOr(&map[bit / 32], 1u << (bit % 32));
            }
        }
    }
    __syncthreads();
    for (int64_t j0 = 0; j0 < a.num_tokens; j0 += kSlots * kThreads) {
        if (j0 > 0)
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int64_t j = j0 + threadIdx.x + k * kThreads;
                s[k] = j < a.num_tokens ? a.slot_mapping[j] : -1;
            }
        uint32_t hits = 0;  // the slots that may be of these blocks
        if constexpr (!kOne) {
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const uint32_t bit = map_bit(s[k]);
                hits |= (s[k] >= 0 ? map[bit / 32] >> (bit % 32) & 1u : 0u) << k;
            }
        }
        if constexpr (kOne) {
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int j = (int)(j0 + threadIdx.x + k * kThreads);
                const unsigned long long r = (unsigned long long)(s[k] - own.first);
                if (r < (unsigned)own.rows) {
                    atomicMax(&token[0][(int)r], j);
                    atomicMin(&lowest[0], j);
                }
            }
        } else {
            for (; hits; hits &= hits - 1) {
                const int j = (int)(j0 + threadIdx.x + (__ffs(hits) - 1) * kThreads);
                Place p;
                block_of(a, a.slot_mapping[j], &p);
                int at = (int)hash_of(p.first);
                while (keys[at] != p.first && keys[at] != -1) at = (at + 1) % kTable;
                if (keys[at] == -1) continue;
                atomicMax(&token[at][p.row], j);
                atomicMin(&lowest[at], j);
            }
        }
    }
    __syncthreads();
    // (The CTAs of a range each have kinds of their own: their lists are in orders of their own.)
    const int per = (kinds - 1) / (int)gridDim.y + 1, kind0 = blockIdx.y * per;
    const int mine = min(per, kinds - kind0), jobs = mine > 0 ? count * mine : 0;
    const int64_t row_stride = (int64_t)a.num_kv_heads * kHeadDim;
    for (int job = warp; job < jobs; job += kWarps) {
        const int e = job / mine, kind = kind0 + job - e * mine, at = list[e];
        if (lowest[at] < t0) continue;  // another CTA's
        const int h = kind >> 1;
        const bool is_v = kind & 1;
        const long long f = keys[at];
        const int64_t page = q8_page_of(f, a.block_size);
        const int o = (int)(f - page * a.block_size);
        uint8_t *scale = (is_v ? a.v_scales : a.k_scales) + page * a.scale_stride +
                         (int64_t)(o / kQ8Tokens) * a.num_kv_heads + h;
        const uint32_t old = *scale;
        const uint16_t *x = (is_v ? a.value : a.key) + h * kHeadDim + 8 * lane;
        const int64_t x_stride = is_v ? a.value_stride : a.key_stride;
        uint4 v[kQ8Tokens];
#pragma unroll
        for (int q = 0; q < kQ8Tokens / 4; ++q) {
            const int4 t4 = reinterpret_cast<const int4 *>(token[at])[q];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = i == 0 ? t4.x : i == 1 ? t4.y : i == 2 ? t4.z : t4.w;
                v[4 * q + i] = make_uint4(0, 0, 0, 0);
                if (t >= 0) v[4 * q + i] = __ldcg(reinterpret_cast<const uint4 *>(x + t * x_stride));
            }
        }
        // Rows that are written.
        const uint32_t rows = __ballot_sync(0xffffffffu, lane < kQ8Tokens && token[at][lane & 15] >= 0);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kQ8Tokens; ++i)
            top = abs_max2(abs_max2(abs_max2(abs_max2(top, v[i].x), v[i].y), v[i].z), v[i].w);
        uint32_t m = warp_top(top);
        if (m >= 0x7f80u) {  // infinities and NaN: codes of NaN, and no part in the scale
            top = 0;
#pragma unroll
            for (int i = 0; i < kQ8Tokens; ++i) {
                top = abs_max2(abs_max2(top, without_inf<true>(v[i].x)), without_inf<true>(v[i].y));
                top = abs_max2(abs_max2(top, without_inf<true>(v[i].z)), without_inf<true>(v[i].w));
                v[i].x = without_inf<false>(v[i].x);
                v[i].y = without_inf<false>(v[i].y);
                v[i].z = without_inf<false>(v[i].z);
                v[i].w = without_inf<false>(v[i].w);
            }
            m = warp_top(top);
        }
        // m = 1.f 2^(E - 127) <= 448 2^(b - 127) = 1.75 2^8 2^(b - 127): b = E - 8, or one more
        // where f > .75
        const uint32_t need = (uint32_t)max(1, (int)(m >> 7) - 8 + ((m & 127u) > 96u ? 1 : 0));
        const bool anew = (rows & 1) || old == 255;
        const uint32_t b = anew ? need : max(old, need);
        const float up = b == 254 ? 0x1p-127f : __uint_as_float((254 - b) << 23);
        uint8_t *row = (is_v ? a.v_cache : a.k_cache) + page * a.page_stride +
                       ((int64_t)o * a.num_kv_heads + h) * kHeadDim + 8 * lane;
        if (lane == 0 && b != old) *scale = (uint8_t)b;
#pragma unroll
        for (int i = 0; i < kQ8Tokens; ++i)
            if (rows >> i & 1) *reinterpret_cast<uint2 *>(row + i * row_stride) = codes_of(v[i], up);
        const uint32_t others = ~rows & ((1u << min(kQ8Tokens, a.block_size - o)) - 1);
        if (!anew && b > old && others) {
            const float down = b - old > 126 ? 0.f : __uint_as_float((127 - (b - old)) << 23);
            uint2 c[kQ8Tokens];
#pragma unroll
            for (int i = 0; i < kQ8Tokens; ++i)
                if (others >> i & 1) c[i] = *reinterpret_cast<const uint2 *>(row + i * row_stride);
#pragma unroll
            for (int i = 0; i < kQ8Tokens; ++i)
                if (others >> i & 1)
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

// Read back by slots: warp per (token, head), K and V of it, 8 dims a lane, so that a store is a whole
// line (16 dims a lane: 8.5 us cold for 4096 tokens, 8 dims 7.4); the warps of a CTA on one head,
// kTok tokens each.
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
            ck[k] = __ldcg(reinterpret_cast<const uint2 *>(a.k_cache + at) + lane);
            cv[k] = __ldcg(reinterpret_cast<const uint2 *>(a.v_cache + at) + lane);
            bk[k] = a.k_scales[sat];
            bv[k] = a.v_scales[sat];
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
        const uint32_t vb = a.v_scales[page * a.scale_stride + (int64_t)(o / kQ8Tokens) * a.num_kv_heads + h];
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
// head, a warp's kExpandKeys / kWarps keys in flight together.  13973 keys of 4 heads: 15 us cold (29 MB
// read, 57 MB written: 5.7 TB/s; 21 us with 16 dims a lane, whose stores were half lines).
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
            ck[i] = __ldcg(reinterpret_cast<const uint2 *>(a.k_cache + at) + lane);
            cv[i] = __ldcg(reinterpret_cast<const uint2 *>(a.v_cache + at) + lane);
            bk[i] = a.k_scales[sat];
            bv[i] = a.v_scales[sat];
        } else if (lane == 0) {
            atomicOr(a.err, kErrPage);
        }
    }
    // The head's largest scale of V: over all of its sequence's blocks, or from their ranges.
    uint32_t top = 0;
    if (a.num_ranges == 0) {
        const int in_page = (a.block_size - 1) / kQ8Tokens + 1, full = sq.num_keys / a.block_size;
        const int blocks = full * in_page + (sq.num_keys - full * a.block_size + kQ8Tokens - 1) / kQ8Tokens;
#pragma unroll 4
        for (int i = threadIdx.x; i < blocks; i += kWarps * 32) {
            const int lp = i / in_page, page = bt[lp];
            if (page < 0 || page >= a.num_pages) continue;
            const uint32_t vb = a.v_scales[page * a.scale_stride + (int64_t)(i - lp * in_page) * a.num_kv_heads + h];
            if (vb != 255) top = max(top, vb);
        }
    } else {
        const int nr = (sq.num_keys - 1) / kExpandRange + 1;
        for (int i = threadIdx.x; i < nr; i += kWarps * 32)
            top = max(top, (uint32_t)a.ranges[(int64_t)h * a.num_ranges + sq.range0 + i].y);
    }
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
    // Two CTAs an SM.  A call of few tokens gives each a token; others first cut the heads, so that a
    // CTA's warps work on one block at a time, then the tokens.  Calls of up to about one job a warp cut
    // the heads once more, so that blocks are spread over more SMs.  With 4 heads, 8 and 4 kinds a CTA: 16
    // tokens 2.8 and 2.6 us, 1000 5.4 and 4.3, 4096 7.1 and 6.4, 6000 10.6 and 9.4; 8192 11.7 and 12.6, 32768 40 and
    // 41; with 8 heads 2000 6.3 and 6.2, 4096 11.0 and 12.2.
    const int ctas = 2 * a.num_sms, kinds = 2 * a.num_kv_heads;
    const int heads = (kinds - 1) / kWarps + 1, twice = (kinds - 1) / (kWarps / 2) + 1;
    const bool few = a.num_tokens <= ctas, small = (int64_t)a.num_tokens * kinds <= (int64_t)10 * kQ8Tokens * ctas;
    int y = std::min(small ? twice : heads, kMaxCut);
    if (few) y = (int64_t)a.num_tokens * twice <= ctas ? twice : std::min(heads, ctas / a.num_tokens);
    a.range = few ? 1 : std::min(kMaxRange, (a.num_tokens - 1) / (ctas / y) + 1);
    const int x = (a.num_tokens - 1) / a.range + 1;
    return launch_pdl(a.range == 1 ? write_q8_kernel<true> : write_q8_kernel<false>, dim3(x, y), dim3(kWarps * 32), 0,
                      stream, a);
}

cudaError_t launch_gather_q8(const Q8GatherArgs &a, cudaStream_t stream) {
    const int tok = a.num_tokens > 1024 ? 2 : 1;
    const dim3 grid((unsigned)((a.num_tokens - 1) / (kWarps * tok) + 1), a.num_kv_heads);
    return tok == 2 ? launch_pdl(gather_q8_kernel<2>, grid, dim3(kWarps * 32), 0, stream, a)
                    : launch_pdl(gather_q8_kernel<1>, grid, dim3(kWarps * 32), 0, stream, a);
}

cudaError_t launch_expand_q8(const ExpandArgs &args, int64_t num_pages_out, cudaStream_t stream) {
    ExpandArgs a = args;
    // Every CTA looks at all scales of V of its sequence and head while that takes it a few reads a
    // thread; longer sequences' are gone through beforehand.  (5 rows over 300 keys: 16.1 us a call and,
    // with the launch that goes through them, 18.4; 1685 rows over 12288 keys 344 either way.)
    int longest = 0;
    for (int b = 0; b < a.num_seqs; ++b) longest = std::max(longest, a.seq[b].num_keys);
    if (longest <= kExpandLook) {
        a.num_ranges = 0;
    } else {
        const cudaError_t e = launch_pdl(range_q8_kernel, dim3((unsigned)a.num_ranges * a.num_kv_heads),
                                         dim3(kWarps * 32), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(expand_q8_kernel,
                      dim3((unsigned)(num_pages_out * (kExpandPage / kExpandKeys)), a.num_kv_heads),
                      dim3(kWarps * 32), 0, stream, a);
}

}  // namespace pa
