// pa_decode_q4.cu -- q=1 decode over the 4-bit cache (format: pa_q4.cuh): split-context
// kernel; the splits are merged by the BF16 decode's combine kernel.
//
// For query head h of KV head g, over the sequence's tokens t < seq_len,
//     out = softmax_t(scale q . khat_t) . vhat_t,   khat, vhat = lo + s n per group of 64.
// Neither is ever formed.  With A_g = sum over the group of q_d n_td (codes on the tensor
// cores, exact in FP16),
//     score_t = sum_g s_tg A_g + lo_tg sum_{d in g} q_d,
//     out_d   = [ sum_t (p_t s_tg) n_td + sum_t p_t lo_tg ] / sum_t p_t   (d in group g),
// so a step costs a multiplication per (token, group, head), not per value.
//
// Bytes: 288 per token and KV head (1024 in BF16).  At the copy bandwidth an SM has to
// take a 16-token tile (4.6 KB) about every 100 ns, so besides HBM the instruction count per
// value matters; it goes to widening codes:
//   * a code becomes FP16 by one three-input logic operation: (w & 0x000f000f) | 0x6400..
//     is the pair (1024 + n, 1024 + n'), (w & 0x00f000f0) | 0x5400.. the pair 64 + n; one
//     shift by 8 serves the other two pairs of a word: 5 operations for 8 codes;
//   * K: pairs of the 1024 kind lose 1032 by a half2 addition (n - 8, exact); those of the
//     64 kind keep their offset, and the accumulators start from the constant
//     8 sum(q) - 72 sum(q of those dims), so that they end as sum q n.  At 64 the offset
//     costs 1e-6 of the score's scale; at 1024 it would cost 2e-5;
//   * V: pairs run along tokens, so two tokens' words are first interleaved by halves (two
//     byte permutations for 16 codes); every pair is brought to n - 8 exactly by a half2
//     addition, since an offset would be summed over all tokens and cancel at the end
//     against a sum thousands of times smaller than it.
// q becomes FP16 after scaling each head by a power of two (largest value in [2^13, 2^14)):
// exact for values down to 2^-30 of the head's largest, and below that off by less than
// 2^-38 of it.  The weights p s become FP16 (2^-12 relative): an eighth of the output's own
// rounding to BF16.
// So that they neither overflow nor vanish, the running reference M is the largest
// score + log2(largest step of the token), not the largest score: p_t = 2^(score_t - M + 15)
// is kept in fp32 and p_t s_tg <= 2^15, which leaves 29 binades of full precision below the
// largest weight (a group whose steps are that much smaller than another's still gets its
// own).  The step is taken within [2^-80, 2^80] for this.
//
// Work split: grid (splits, KV heads, sequences), four consumer warps and a producer warp a
// CTA, two CTAs an SM (one's prologue and merge behind the other's stream).  A ring stage
// is four 16-token tiles, one a consumer warp.  The producer's 16 lanes bring one run
// each (codes and pairs of K and of V of one tile) by bulk copies: contiguous, needing no
// tensor map, and never longer than the page's and the sequence's valid rows.
#include <math_constants.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {

namespace {

constexpr int kTile = kDecTile;                       // 16 tokens
constexpr int kC = 4;                                 // consumer warps = tiles per stage
constexpr int kStages = 5;
constexpr int kTileCodes = kTile * kQ4CodeBytes;      // 2 KB
constexpr int kTilePairs = kTile * kQ4PairBytes;      // 256 B
constexpr int kTileBytes = 2 * (kTileCodes + kTilePairs);  // K codes, V codes, K pairs, V pairs
constexpr int kStageBytes = kC * kTileBytes;          // 18 KB
constexpr int kRingBytes = kStages * kStageBytes;
constexpr int kThreads = (kC + 1) * 32;
constexpr int kMergeRow = kHeadDim + 4;
constexpr int kSmem = kRingBytes + 2 * kStages * 8 + 16;
constexpr float kHeadroom = 15.f;                     // log2 of the largest weight
static_assert(kC * kDecMaxGroup * (kMergeRow + 2) * 4 <= kRingBytes, "merge buffers reuse the ring");

struct Params {
    const uint16_t *q;
    const uint8_t *k_cache, *v_cache;
    int64_t page_stride, num_pages;
    const int32_t *block_table;
    int64_t bt_stride;
    const int32_t *seq_lens;
    int max_seq_len, num_q_heads, group, block_size, tiles_per_page, tiles_per_split, num_splits;
    float scale_log2;
    float *part_o;
    float2 *part_ml;
    unsigned *err;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// D += A (16x16, row) * B (16x8, col), FP16 in, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (a & b) | c in one operation.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
constexpr uint32_t kMinus1032 = 0xe408e408u;  // (-1032, -1032)
constexpr uint32_t kMinus72 = 0xd480d480u;    // (-72, -72)

// The four pairs (n_k, n_{k+4}) of a word's codes as FP16: k even as n - 8, k odd as
// 64 + n (keep64) or n - 8.
template <bool keep64>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&x)[4]) {
    const uint32_t w8 = w >> 8;
    x[0] = h2_add(and_or(w, 0x000f000fu, 0x64006400u), kMinus1032);
    x[1] = and_or(w, 0x00f000f0u, 0x54005400u);
    x[2] = h2_add(and_or(w8, 0x000f000fu, 0x64006400u), kMinus1032);
    x[3] = and_or(w8, 0x00f000f0u, 0x54005400u);
    if (!keep64) {
        x[1] = h2_add(x[1], kMinus72);
        x[3] = h2_add(x[3], kMinus72);
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int g) {
    return g == 0 ? v.x : g == 1 ? v.y : g == 2 ? v.z : v.w;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ int tiles_of(int len, int block_size, int tpp) {
    const int full = len / block_size;
    return full * tpp + (len - full * block_size + kTile - 1) / kTile;
}

__global__ void __launch_bounds__(kThreads, 2) decode_q4_split_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kRingBytes);
    uint64_t *empty = full + kStages;
    volatile int *abort = reinterpret_cast<volatile int *>(empty + kStages);
    const int split = blockIdx.x, g = blockIdx.y, seq = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kC);
        }
        *abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    const int tpp = p.tiles_per_page;
    const int t0 = split * p.tiles_per_split;
    const int32_t *bt = p.block_table + (int64_t)seq * p.bt_stride;
    // The producer's first table entry is read beside the length: tile t0 + lane / 4 lies
    // in the row when it is a tile of the longest allowed sequence.
    const int max_tiles = tiles_of(p.max_seq_len, p.block_size, tpp);
    int page = 0;
    if (warp == kC && lane < 4 * kC && t0 + (lane >> 2) < max_tiles) page = bt[(t0 + (lane >> 2)) / tpp];
    int seq_len = p.seq_lens[seq];
    if (seq_len < 0 || seq_len > p.max_seq_len) {
        if (threadIdx.x == 0 && split == 0 && g == 0) atomicOr(p.err, kErrSeqLen);
        seq_len = seq_len < 0 ? 0 : p.max_seq_len;
    }
    const int t1 = min(tiles_of(seq_len, p.block_size, tpp), t0 + p.tiles_per_split);
    const int64_t part0 = ((int64_t)seq * p.num_q_heads + g * p.group) * p.num_splits + split;
    if (t0 >= t1) {  // no tiles of this sequence: an empty partial, which the merge skips
        if (threadIdx.x < p.group)
            p.part_ml[part0 + (int64_t)threadIdx.x * p.num_splits] = make_float2(-CUDART_INF_F, 0.f);
        return;
    }
    const int n = t1 - t0, nst = (n + kC - 1) / kC;

    if (warp == kC) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_evict_first_policy();
        const int ti = lane >> 2, kind = lane & 3;  // the lane's tile of a stage, and its run
        const int64_t head = (int64_t)g * p.block_size * kQ4RowBytes;
        const uint8_t *base = ((kind & 1) ? p.v_cache : p.k_cache) + head +
                              (kind >= 2 ? (int64_t)p.block_size * kQ4CodeBytes : 0);
        const int row_bytes = kind >= 2 ? kQ4PairBytes : kQ4CodeBytes;
        const int dst_off = ti * kTileBytes + (kind >= 2 ? 2 * kTileCodes + (kind - 2) * kTilePairs
                                                         : kind * kTileCodes);
        int issued = 0;  // stages loaded
        for (int m = 0; m < nst; ++m) {
            const int s = m % kStages;
            const int j = t0 + m * kC + ti;
            const bool mine = lane < 4 * kC && j < t1;
            // The next stage's table entry is read before this stage's wait.
            const int jn = j + kC;
            const int page_next = lane < 4 * kC && jn < t1 ? bt[jn / tpp] : 0;
            if (m >= kStages &&
                !__all_sync(0xffffffffu,
                            mbar_wait_abort(&empty[s], ((m / kStages) - 1) & 1, p.err, abort)))
                break;
            int bytes = 0;
            const uint8_t *src = nullptr;
            uint8_t *dst = smem + s * kStageBytes + dst_off;
            if (mine) {
                const int lp = j / tpp, off = (j - lp * tpp) * kTile;
                const int rows = min(kTile, min(p.block_size - off, seq_len - (lp * p.block_size + off)));
                bytes = rows * row_bytes;
                if (page >= 0 && page < p.num_pages) {
                    src = base + page * p.page_stride + (int64_t)off * row_bytes;
                } else {
                    // Outside the pool: reported, and read as zeros (steps and minima of 0).
                    if (kind == 0) atomicOr(p.err, kErrPage);
                    if (kind >= 2)
                        for (int i = 0; i < bytes / 16; ++i)
                            reinterpret_cast<uint4 *>(dst)[i] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    bytes = 0;
                }
            }
            const int total = __reduce_add_sync(0xffffffffu, bytes);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[s], total);
            __syncwarp();
            if (bytes) bulk_load(dst, src, bytes, &full[s], pol);
            issued = m + 1;
            page = page_next;
        }
        // Every load lands before the ring is reused by the merge or left.
        for (int m = max(0, issued - kStages); m < issued; ++m)
            mbar_wait(&full[m % kStages], (m / kStages) & 1, p.err);
        __syncwarp();
        bar_sync(1, kThreads);
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int r = lane >> 2, c = lane & 3;
    // q as FP16 B fragments: lane (head r, column c) holds dims 64g + 8(2c + h) + j; MMA i
    // of word h takes the pairs (2i, 2i + 4) and (2i + 1, 2i + 5).
    uint32_t qf[4][2][4];
    float init0[4], init1[4], qs0[4], qs1[4], sc0, sc1;  // of heads 2c and 2c + 1
    {
        const bool hv = r < p.group;
        const uint4 *qrow = reinterpret_cast<const uint4 *>(
            p.q + ((int64_t)seq * p.num_q_heads + g * p.group + (hv ? r : 0)) * kHeadDim);
        uint4 raw[4][2];
        uint32_t amax = 0;
#pragma unroll
        for (int gg = 0; gg < 4; ++gg)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                raw[gg][h] = hv ? qrow[gg * 8 + 2 * c + h] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = word(raw[gg][h], i);
                    amax = max(amax, max((w << 16) & 0x7fff0000u, w & 0x7fff0000u));
                }
            }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // A power of two f that brings the head's largest value to [2^13, 2^14).
        const int e = (int)(amax >> 23);
        const float f = e == 255 ? 1.f : __uint_as_float((uint32_t)min(254, max(1, 267 - e)) << 23);
        const float sc = p.scale_log2 / f;
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
            float sum = 0.f, odd = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = bf16_lo(word(raw[gg][h], i)) * f;
                    v[2 * i + 1] = bf16_hi(word(raw[gg][h], i)) * f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qf[gg][h][i] = pack_f16x2(v[i], v[i + 4]);
                    const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&qf[gg][h][i]));
                    sum += back.x + back.y;
                    if (i & 1) odd += back.x + back.y;
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            odd += __shfl_xor_sync(0xffffffffu, odd, 1);
            odd += __shfl_xor_sync(0xffffffffu, odd, 2);
            const float in = 8.f * (sum - odd) - 64.f * odd;  // codes come as n - 8 and 64 + n
            init0[gg] = __shfl_sync(0xffffffffu, in, 8 * c);
            init1[gg] = __shfl_sync(0xffffffffu, in, 8 * c + 4);
            qs0[gg] = __shfl_sync(0xffffffffu, sum, 8 * c);
            qs1[gg] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
        }
        sc0 = __shfl_sync(0xffffffffu, sc, 8 * c);
        sc1 = __shfl_sync(0xffffffffu, sc, 8 * c + 4);
    }

    float o[4][4][4];  // [group][dim pair][(dim, head) of the pairs]
    float low0[4], low1[4];  // this lane's share of sum p lo'
#pragma unroll
    for (int gg = 0; gg < 4; ++gg) {
        low0[gg] = low1[gg] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[gg][i][0] = o[gg][i][1] = o[gg][i][2] = o[gg][i][3] = 0.f;
    }
    float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;

    for (int m = 0; m < nst; ++m) {
        const int i = m * kC + warp;
        if (i >= n) break;
        const int s = m % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait_abort(&full[s], (m / kStages) & 1, p.err, abort)))
            break;
        const int j = t0 + i, lp = j / tpp, off = (j - lp * tpp) * kTile;
        const int nvalid = min(kTile, min(p.block_size - off, seq_len - (lp * p.block_size + off)));
        const uint32_t kb = smem_u32(smem + s * kStageBytes + warp * kTileBytes);
        const uint32_t vb = kb + kTileCodes, kp = vb + kTileCodes, vp = kp + kTilePairs;
        const bool in0 = r < nvalid, in1 = r + 8 < nvalid;

        // ---- scores: tokens r and r + 8, heads 2c and 2c + 1
        float x00 = 0.f, x01 = 0.f, x10 = 0.f, x11 = 0.f;
        {
            const uint32_t a0 = kb + r * 128 + (((2 * c) ^ r) << 4);
            const uint4 k00 = lds128(a0), k01 = lds128(a0 ^ 16);
            const uint4 k10 = lds128(a0 + 1024), k11 = lds128((a0 ^ 16) + 1024);
            const uint4 pr0 = lds128(kp + r * 16), pr1 = lds128(kp + r * 16 + 128);
#pragma unroll
            for (int gg = 0; gg < 4; ++gg) {
                float a[4] = {init0[gg], init1[gg], init0[gg], init1[gg]};
                uint32_t x[4], y[4];
                widen<true>(word(k00, gg), x);
                widen<true>(word(k10, gg), y);
                mma_f16(a, x[0], y[0], x[1], y[1], qf[gg][0][0], qf[gg][0][1]);
                mma_f16(a, x[2], y[2], x[3], y[3], qf[gg][0][2], qf[gg][0][3]);
                widen<true>(word(k01, gg), x);
                widen<true>(word(k11, gg), y);
                mma_f16(a, x[0], y[0], x[1], y[1], qf[gg][1][0], qf[gg][1][1]);
                mma_f16(a, x[2], y[2], x[3], y[3], qf[gg][1][2], qf[gg][1][3]);
                const float s0 = q4_step(word(pr0, gg)), lo0 = q4_low(word(pr0, gg));
                const float s1 = q4_step(word(pr1, gg)), lo1 = q4_low(word(pr1, gg));
                x00 = fmaf(s0, a[0], fmaf(lo0, qs0[gg], x00));
                x01 = fmaf(s0, a[1], fmaf(lo0, qs1[gg], x01));
                x10 = fmaf(s1, a[2], fmaf(lo1, qs0[gg], x10));
                x11 = fmaf(s1, a[3], fmaf(lo1, qs1[gg], x11));
            }
        }
        x00 = in0 ? x00 * sc0 : -CUDART_INF_F;
        x01 = in0 ? x01 * sc1 : -CUDART_INF_F;
        x10 = in1 ? x10 * sc0 : -CUDART_INF_F;
        x11 = in1 ? x11 * sc1 : -CUDART_INF_F;

        // ---- online softmax against M = max(score + log2(largest step))
        uint4 pr0 = lds128(vp + r * 16), pr1 = lds128(vp + r * 16 + 128);
        if (!in0) pr0 = make_uint4(0, 0, 0, 0);  // what is masked may hold anything
        if (!in1) pr1 = make_uint4(0, 0, 0, 0);
        float big0 = 0x1p-80f, big1 = 0x1p-80f;
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
            big0 = fmaxf(big0, q4_step(word(pr0, gg)));
            big1 = fmaxf(big1, q4_step(word(pr1, gg)));
        }
        big0 = lg2_approx(fminf(big0, 0x1p80f));
        big1 = lg2_approx(fminf(big1, 0x1p80f));
        float mx0 = fmaxf(x00 + big0, x10 + big1), mx1 = fmaxf(x01 + big0, x11 + big1);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        const float mu0 = mn0 == -CUDART_INF_F ? 0.f : mn0 - kHeadroom;
        const float mu1 = mn1 == -CUDART_INF_F ? 0.f : mn1 - kHeadroom;
        const float p00 = ex2_approx(x00 - mu0), p01 = ex2_approx(x01 - mu1);
        const float p10 = ex2_approx(x10 - mu0), p11 = ex2_approx(x11 - mu1);
        if (__any_sync(0xffffffffu, mn0 != m0 || mn1 != m1)) {
            const float al0 = m0 == -CUDART_INF_F ? 0.f : ex2_approx(m0 - mn0);
            const float al1 = m1 == -CUDART_INF_F ? 0.f : ex2_approx(m1 - mn1);
            l0 *= al0;
            l1 *= al1;
#pragma unroll
            for (int gg = 0; gg < 4; ++gg) {
                low0[gg] *= al0;
                low1[gg] *= al1;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[gg][k][0] *= al0;
                    o[gg][k][1] *= al1;
                    o[gg][k][2] *= al0;
                    o[gg][k][3] *= al1;
                }
            }
            m0 = mn0;
            m1 = mn1;
        }
        l0 += p00 + p10;
        l1 += p01 + p11;

        // ---- O^T += V^T (p s)^T, two tokens' codes a register
        const uint32_t v0 = vb + 2 * c * 128 + ((r ^ (2 * c)) << 4);  // token 2c, unit r
        const uint4 va = lds128(v0), vc = lds128(v0 + 1024);           // tokens 2c, 2c + 8
        const uint32_t v1 = (v0 ^ 16) + 128;
        const uint4 vb1 = lds128(v1), vd = lds128(v1 + 1024);          // tokens 2c + 1, 2c + 9
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
            const float s0 = q4_step(word(pr0, gg)), s1 = q4_step(word(pr1, gg));
            // codes come as n - 8: their constant part joins the minimum
            const float lo0 = fmaf(8.f, s0, q4_low(word(pr0, gg)));
            const float lo1 = fmaf(8.f, s1, q4_low(word(pr1, gg)));
            low0[gg] = fmaf(p00, lo0, fmaf(p10, lo1, low0[gg]));
            low1[gg] = fmaf(p01, lo0, fmaf(p11, lo1, low1[gg]));
            const uint32_t b0 = movmatrix_t(pack_f16x2(p00 * s0, p01 * s0));
            const uint32_t b1 = movmatrix_t(pack_f16x2(p10 * s1, p11 * s1));
            uint32_t x[4], y[4];
            widen<false>(__byte_perm(word(va, gg), word(vb1, gg), 0x5410), x);
            widen<false>(__byte_perm(word(vc, gg), word(vd, gg), 0x5410), y);
            mma_f16(o[gg][0], x[0], x[1], y[0], y[1], b0, b1);
            mma_f16(o[gg][1], x[2], x[3], y[2], y[3], b0, b1);
            widen<false>(__byte_perm(word(va, gg), word(vb1, gg), 0x7632), x);
            widen<false>(__byte_perm(word(vc, gg), word(vd, gg), 0x7632), y);
            mma_f16(o[gg][2], x[0], x[1], y[0], y[1], b0, b1);
            mma_f16(o[gg][3], x[2], x[3], y[2], y[3], b0, b1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
    }

#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
        l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
            low0[gg] += __shfl_xor_sync(0xffffffffu, low0[gg], sh);
            low1[gg] += __shfl_xor_sync(0xffffffffu, low1[gg], sh);
        }
    }

    // ---------------------------------------------------------------- CTA merge
    bar_sync(1, kThreads);  // every tile consumed, no load in flight
    if (*abort) {
        if (threadIdx.x < p.group)
            p.part_ml[part0 + (int64_t)threadIdx.x * p.num_splits] = make_float2(-CUDART_INF_F, 0.f);
        return;
    }
    float *red_o = reinterpret_cast<float *>(smem);  // [warp][head][row]
    float *red_m = red_o + kC * kDecMaxGroup * kMergeRow;
    float *red_l = red_m + kC * kDecMaxGroup;
    if (lane < 4) {
        red_m[warp * kDecMaxGroup + 2 * c] = m0;
        red_m[warp * kDecMaxGroup + 2 * c + 1] = m1;
        red_l[warp * kDecMaxGroup + 2 * c] = l0;
        red_l[warp * kDecMaxGroup + 2 * c + 1] = l1;
    }
    {
        float *w0 = red_o + (warp * kDecMaxGroup + 2 * c) * kMergeRow + 8 * r;
#pragma unroll
        for (int gg = 0; gg < 4; ++gg)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                *reinterpret_cast<float4 *>(w0 + gg * 64 + k * 4) =
                    make_float4(o[gg][2 * k][0] + low0[gg], o[gg][2 * k][2] + low0[gg],
                                o[gg][2 * k + 1][0] + low0[gg], o[gg][2 * k + 1][2] + low0[gg]);
                *reinterpret_cast<float4 *>(w0 + kMergeRow + gg * 64 + k * 4) =
                    make_float4(o[gg][2 * k][1] + low1[gg], o[gg][2 * k][3] + low1[gg],
                                o[gg][2 * k + 1][1] + low1[gg], o[gg][2 * k + 1][3] + low1[gg]);
            }
    }
    bar_sync(2, kC * 32);
    for (int qd = threadIdx.x; qd < p.group * (kHeadDim / 4); qd += kC * 32) {
        const int h = qd / (kHeadDim / 4), d = (qd - h * (kHeadDim / 4)) * 4;
        float M = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < kC; ++w) M = fmaxf(M, red_m[w * kDecMaxGroup + h]);
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kC; ++w) {
            const float e = M == -CUDART_INF_F ? 0.f : ex2_approx(red_m[w * kDecMaxGroup + h] - M);
            const float4 v =
                *reinterpret_cast<const float4 *>(red_o + (w * kDecMaxGroup + h) * kMergeRow + d);
            L += e * red_l[w * kDecMaxGroup + h];
            O.x += e * v.x;
            O.y += e * v.y;
            O.z += e * v.z;
            O.w += e * v.w;
        }
        const int64_t pi = part0 + (int64_t)h * p.num_splits;
        *reinterpret_cast<float4 *>(p.part_o + pi * kHeadDim + d) = O;
        if (d == 0) p.part_ml[pi] = make_float2(M, L);
    }
}

}  // namespace

// Tiles per split: all CTAs resident at once (two an SM) when the longest allowed length
// gives each at least a stage, and never more than kDecMaxSplits splits.
DecodePlan plan_decode_q4(int num_seqs, int num_kv_heads, int block_size, int max_seq_len,
                          int num_sms) {
    DecodePlan pl;
    pl.tiles_per_page = (block_size + kTile - 1) / kTile;
    const int full = max_seq_len / block_size;
    pl.max_tiles = full * pl.tiles_per_page + (max_seq_len - full * block_size + kTile - 1) / kTile;
    const long long pairs = (long long)num_seqs * num_kv_heads;
    const long long want = std::max(1ll, (2ll * num_sms + pairs - 1) / pairs);
    int tps = (int)((pl.max_tiles + want - 1) / want);
    tps = std::max(tps, (pl.max_tiles + kDecMaxSplits - 1) / kDecMaxSplits);
    pl.tiles_per_split = (std::max(tps, 1) + kC - 1) / kC * kC;
    pl.num_splits = (pl.max_tiles + pl.tiles_per_split - 1) / pl.tiles_per_split;
    return pl;
}

cudaError_t launch_decode_q4(const DecodeQ4Args &a, const DecodePlan &plan, cudaStream_t stream) {
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(decode_q4_split_kernel), kSmem, 6);
    if (e != cudaSuccess) return e;
    Params p;
    p.q = a.q;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.page_stride = a.page_stride;
    p.num_pages = a.num_pages;
    p.block_table = a.block_table;
    p.bt_stride = a.bt_stride;
    p.seq_lens = a.seq_lens;
    p.max_seq_len = a.max_seq_len;
    p.num_q_heads = a.num_q_heads;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.block_size = a.block_size;
    p.tiles_per_page = plan.tiles_per_page;
    p.tiles_per_split = plan.tiles_per_split;
    p.num_splits = plan.num_splits;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    decode_ws_parts(a.workspace, a.num_seqs, a.num_q_heads, plan, &p.part_o, &p.part_ml);
    p.err = a.err;
    if (a.ev_start && (e = record_event(a.ev_start, stream)) != cudaSuccess) return e;
    e = launch_pdl(decode_q4_split_kernel, dim3(plan.num_splits, a.num_kv_heads, a.num_seqs),
                   dim3(kThreads), kSmem, stream, p);
    if (e != cudaSuccess) return e;
    if (a.ev_stop && (e = record_event(a.ev_stop, stream)) != cudaSuccess) return e;
    return launch_decode_combine(p.part_o, p.part_ml, a.num_seqs, a.num_q_heads, plan.num_splits,
                                 a.out, stream);
}

}  // namespace pa
