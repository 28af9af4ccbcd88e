// pa_decode_split.cuh -- the work split of the streaming decodes over the 4-bit and the 8-bit
// cache, and the kernel that merges the parts of sequences that it cut.
//
// The tiles (16 tokens of a page) of all (sequence, KV head) pairs stand in a row, cut evenly
// over the CTAs, so that uneven lengths leave no SM idle; each CTA finds its share from the
// lengths.  A pair also costs its beginning: it counts as kPairCost tiles more (half a share at
// most), ahead of its first, so that CTAs with many short pairs get fewer tiles; shares below twice
// kMinShare stay even.  A pair that one CTA holds whole is finished there; the others leave a
// part per CTA (sums relative to their reference).
#pragma once

#include <math_constants.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kTile = kDecTile;                       // 16 tokens

// Division of n < 2^31 by a constant of the launch.
struct FastDiv {
    uint32_t d, mul, shift;
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
    return f;
}

struct SplitParams {
    const uint16_t *q;
    int64_t num_pages;
    const int32_t *block_table;
    int64_t bt_stride;
    const int32_t *seq_lens;
    int num_seqs, max_seq_len, num_q_heads, num_kv_heads, group, block_size, tiles_per_page;
    int ctas;  // of the streaming kernel (for a merge with kShare)
    FastDiv by_block, by_tpp;
    float scale_log2;
    // Part i: fp32 sums [group, 256] and (reference, sum of weights) [group].  CTA b's part of
    // pair x is part b + x (one of the two grows from part to part, so no two are the same).
    float *part_o;
    float2 *part_ml;
    int2 *info;  // [pairs]: a pair's first part and how many (0: finished by one CTA)
    int64_t parts;
    uint16_t *out;
    unsigned *err;
};

__device__ __forceinline__ int tiles_of(const SplitParams &p, int len) {
    const int full = (int)p.by_block(len);
    return full * p.tiles_per_page + ((len - full * p.block_size + kTile - 1) >> 4);
}

// Tiles of sequence s (none past the last); lengths out of range are cut to it.  kEarly: read from L2
// alone, so that a read before earlier work has written the lengths leaves no stale copy in L1.
template <bool kEarly = false>
__device__ __forceinline__ int seq_tiles(const SplitParams &p, int s, int *len, bool report) {
    int L = s >= p.num_seqs ? 0 : kEarly ? __ldcg(p.seq_lens + s) : p.seq_lens[s];
    if (L < 0 || L > p.max_seq_len) {
        if (report) atomicOr(p.err, kErrSeqLen);
        L = L < 0 ? 0 : p.max_seq_len;
    }
    *len = L;
    return tiles_of(p, L);
}

constexpr uint32_t kMaxTiles = 0x7fffffffu;  // of all pairs, with their leads

// Places ahead of each of `pairs` pairs' tiles, when `tiles` (at most kMaxTiles) are cut over `ctas`
// shares: half a share at most, and none where they would not be numbered in 31 bits.
template <int kMinShare, int kPairCost>
__host__ __device__ __forceinline__ int pair_lead(uint32_t tiles, uint64_t pairs, uint32_t ctas) {
    if (tiles < (uint64_t)2 * kMinShare * ctas) return 0;
    const uint32_t half = tiles / (2 * ctas);
    const uint32_t lead = half < (uint32_t)kPairCost ? half : (uint32_t)kPairCost;
    return tiles + lead * pairs > kMaxTiles ? 0 : (int)lead;
}

// CTA b's first tile when `total` tiles are cut over `ctas`: the first r shares have one more.
struct Shares {
    uint32_t q, r;
    __device__ __forceinline__ uint32_t begin(uint32_t b) const { return b * q + min(b, r); }
    __device__ __forceinline__ uint32_t owner(uint32_t tile) const {
        const uint32_t big = r * (q + 1);
        return tile < big ? tile / (q + 1) : r + (tile - big) / q;
    }
};

// A CTA's share: the next place `at` in the row of all pairs, the share's end, the places ahead of
// each pair's tiles, and the segment that it begins with: place v0 of KV head g of sequence seq.
struct Start {
    Shares shares;
    uint32_t at, end;
    int lead, v0, seq, g, seq_len, tiles;
    int ctas_a_pair;  // kAlone: CTAs of each pair, cut by itself (0: the pairs are cut in a row)
};
// What was found; refused: more tiles than a share can be found of.
enum class Found { kNone, kShare, kRefused };

// Tiles and lengths of kBatches times 32 sequences, a lane's being 32 b + lane.
template <int kBatches>
struct Lengths {
    int tiles[kBatches], len[kBatches];
};

// Finds this CTA's share, with the first sequences' lengths given (every warp finds the same).
// kAlone: with one sequence, each of its pairs is cut by itself, so that no CTA works on two (their
// beginnings would follow one another).  kEarly: as for seq_tiles.
template <int kMinShare, int kPairCost, bool kAlone = false, bool kEarly = false, int kBatches = 1>
__device__ __forceinline__ Found find_start(const SplitParams &p, int lane, bool report,
                                            const Lengths<kBatches> &first, Start &st) {
    uint64_t all = 0, used = 0;
    auto count = [&](uint64_t t) {
        used += __popc(__ballot_sync(0xffffffffu, t > 0));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        all += t;
    };
#pragma unroll
    for (int b = 0; b < kBatches; ++b)
        if (b == 0 || 32 * b < p.num_seqs) count(first.tiles[b]);
    for (int s0 = 32 * kBatches; s0 < p.num_seqs; s0 += 32) {
        int len;
        count(seq_tiles<kEarly>(p, s0 + lane, &len, report));
    }
    all *= p.num_kv_heads;
    if (all == 0) return Found::kNone;  // padding entries only
    if (all > kMaxTiles) {
        return Found::kRefused;
    }
    if constexpr (kAlone) {
        st.ctas_a_pair = 0;
        if (p.num_seqs == 1 && gridDim.x >= (unsigned)p.num_kv_heads) {
            const uint32_t tiles = __shfl_sync(0xffffffffu, first.tiles[0], 0);
            const uint32_t n = min(gridDim.x / p.num_kv_heads, (tiles + kMinShare - 1) / kMinShare);
            const uint32_t pair = blockIdx.x / n, i = blockIdx.x - pair * n;
            if (pair >= (uint32_t)p.num_kv_heads) return Found::kNone;
            st.ctas_a_pair = (int)n;
            st.shares.q = tiles / n;
            st.shares.r = tiles - st.shares.q * n;
            st.lead = 0;
            st.seq = 0;
            st.g = (int)pair;
            st.tiles = (int)tiles;
            st.seq_len = __shfl_sync(0xffffffffu, first.len[0], 0);
            st.v0 = (int)st.shares.begin(i);
            st.at = pair * tiles + st.v0;
            st.end = pair * tiles + st.shares.begin(i + 1);
            return Found::kShare;
        }
    }
    const uint32_t ctas = min(gridDim.x, ((uint32_t)all + kMinShare - 1) / kMinShare);
    st.lead = pair_lead<kMinShare, kPairCost>((uint32_t)all, used * p.num_kv_heads, ctas);
    const uint32_t total = (uint32_t)(all + st.lead * used * p.num_kv_heads);
    if (blockIdx.x >= ctas) return Found::kNone;
    st.shares.q = total / ctas;
    st.shares.r = total - st.shares.q * ctas;
    st.at = st.shares.begin(blockIdx.x);
    st.end = st.shares.begin(blockIdx.x + 1);
    uint32_t before = 0;
    auto here = [&](int s0, int t, int len) {
        const uint32_t span = t > 0 ? t + st.lead : 0;  // a pair's places
        uint32_t sum = span;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, (before + sum) * p.num_kv_heads > st.at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            st.seq = s0 + l;
            st.seq_len = __shfl_sync(0xffffffffu, len, l);
            st.tiles = __shfl_sync(0xffffffffu, t, l);
            const uint32_t rem = st.at - (before + __shfl_sync(0xffffffffu, sum - span, l)) * p.num_kv_heads;
            st.g = (int)(rem / (uint32_t)(st.tiles + st.lead));
            st.v0 = (int)(rem - (uint32_t)st.g * (st.tiles + st.lead));
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        return false;
    };
#pragma unroll
    for (int b = 0; b < kBatches; ++b)
        if (b == 0 || 32 * b < p.num_seqs)
            if (here(32 * b, first.tiles[b], first.len[b])) return Found::kShare;
    for (int s0 = 32 * kBatches; s0 < p.num_seqs; s0 += 32) {
        int len;
        const int t = seq_tiles<kEarly>(p, s0 + lane, &len, false);
        if (here(s0, t, len)) return Found::kShare;
    }
    return Found::kNone;  // (not reached: at < total)
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
// The same from D = 0.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Merges a row's parts: sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) l_j, M = max m_j; an empty
// part has m = -inf.  All loads of a round (kRound parts a warp) are in flight together.
//   kSplit > 1: that many warps for each 64 dims of a row take its parts in turn, for the
//               latency of many parts
//   kSplit = 1: two warps a row (128 dims each), 4 rows a CTA
// The fewer the rows, the more parts each may have: 8 up to a row an SM, 4 up to 8 rows an SM, 1
// beyond.  A step's us with 8, 4 and 1 (6 query heads a KV head):
//   sequences of 1..4096 keys    24 rows 11.1 11.3 12.5   144 14.3 15.3 16.7   192 18.9 18.6 19.2
//     384 19.3 17.5 17.8   768 27.8 24.7 23.1   1200 39.8 35.1 31.9   1536 48.1 42.2 38.2
//   one of 32768, others to 200   192 17.5 20.4 24.9   384 18.7 21.0 24.4   768 22.0 22.7 24.8
//     1200 24.2 22.9 25.0   1536 27.1 23.6 26.0
// so between 2 and 8 rows an SM 4 loses up to 9% to 1 where lengths are alike, and gains as much
// where one is long.
// kShare: one sequence whose pairs were cut alone (find_start, kMinShare); the parts follow from its
// length, which stands before the streaming kernel ends: no look at p.info after the wait.
template <int kSplit, int kRound, int kShare = 0>
__global__ void __launch_bounds__(256) decode_merge_kernel(const __grid_constant__ SplitParams p) {
    constexpr bool kFew = kSplit > 1;
    constexpr int kWarps = kSplit;
    constexpr int kBlocks = 8 / kSplit;  // of 64 dims, in a CTA
    constexpr int kVec = kFew ? 1 : 2;  // float2 a lane
    const int lane = threadIdx.x & 31, all = threadIdx.x >> 5;
    const int warp = kFew ? all % kWarps : all, block = kFew ? all / kWarps : 0;
    const int64_t row = kFew ? blockIdx.x / (4 / kBlocks) : (int64_t)blockIdx.x * 4 + (warp >> 1);
    const int d0 = kFew ? (blockIdx.x % (4 / kBlocks) * kBlocks + block) * 64 : (warp & 1) * 128;
    int2 info;
    int len;
    if constexpr (kShare > 0) {
        const int pair = (int)row / p.group, tiles = seq_tiles<true>(p, 0, &len, false);
        const int n = min(p.ctas / p.num_kv_heads, (tiles + kShare - 1) / kShare);
        const bool cut = n > 1 && (uint64_t)tiles * p.num_kv_heads <= kMaxTiles;
        info = make_int2(pair * (n + 1), cut ? n : 0);
    }
    pdl_wait();
    pdl_trigger();
    if (row >= (int64_t)p.num_seqs * p.num_q_heads) return;  // (warp-uniform; kFew: never)
    const int seq = (int)(row / p.num_q_heads), h = (int)(row - (int64_t)seq * p.num_q_heads);
    if constexpr (kShare == 0) {
        len = p.seq_lens[seq];
        info = p.info[(int64_t)seq * p.num_kv_heads + h / p.group];
    }
    uint16_t *out = p.out + row * kHeadDim + d0;
    if (len <= 0) {
        if (kFew ? warp == 0 : true)
#pragma unroll
            for (int v = 0; v < kVec; ++v) reinterpret_cast<uint32_t *>(out)[v * 32 + lane] = 0;
        return;
    }
    const int count = info.y;
    if (count <= 0 || info.x < 0 || info.x + (int64_t)count > p.parts) return;
    const int64_t first = (int64_t)info.x * p.group + h % p.group;  // parts are p.group rows apart
    float M = -CUDART_INF_F, L = 0.f;
    float2 acc[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) acc[v] = make_float2(0.f, 0.f);
    for (int j0 = kFew ? warp : 0; j0 < count; j0 += kWarps * kRound) {
        float2 o[kRound][kVec], ml[kRound];
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            const int j = j0 + k * kWarps;
            const int64_t at = first + (int64_t)j * p.group;
            ml[k] = j < count ? ld_f2_ordered(p.part_ml + at) : make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
            for (int v = 0; v < kVec; ++v)
                o[k][v] = j < count ? ld_f2_ordered(reinterpret_cast<const float2 *>(
                                          p.part_o + at * kHeadDim + d0) + v * 32 + lane)
                                    : make_float2(0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < kRound; ++k) mn = fmaxf(mn, ml[k].x);
        const float f = M == -CUDART_INF_F ? 0.f : ex2_approx(M - mn);
        M = mn;
        L *= f;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            acc[v].x *= f;
            acc[v].y *= f;
        }
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            // (an empty part is zeros; one of weight 0 counts too: its sums may be NaN)
            const float e = ml[k].x == -CUDART_INF_F ? 0.f : ex2_approx(ml[k].x - M);
            L = fmaf(e, ml[k].y, L);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                acc[v].x = fmaf(e, o[k][v].x, acc[v].x);
                acc[v].y = fmaf(e, o[k][v].y, acc[v].y);
            }
        }
    }
    if (kFew) {
        __shared__ float2 sums[kBlocks][kWarps][32], refs[kBlocks][kWarps];
        float2 (*so)[32] = sums[block], *sml = refs[block];
        so[warp][lane] = acc[0];
        if (lane == 0) sml[warp] = make_float2(M, L);
        __syncthreads();
        if (warp) return;
        M = -CUDART_INF_F;
        L = 0.f;
        acc[0] = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float e = sml[w].x == -CUDART_INF_F ? 0.f : ex2_approx(sml[w].x - M);
            L = fmaf(e, sml[w].y, L);
            acc[0].x = fmaf(e, so[w][lane].x, acc[0].x);
            acc[0].y = fmaf(e, so[w][lane].y, acc[0].y);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v)
        reinterpret_cast<uint32_t *>(out)[v * 32 + lane] = pack_bf16x2(acc[v].x * inv, acc[v].y * inv);
}

// Workspace: the parts' sums, their (reference, sum) pairs, and the pairs' info, each
// 256-byte aligned.  A part is numbered CTA + pair, so there are at most CTAs + pairs.
struct WsLayout {
    int64_t parts;
    size_t o, ml, info;
};
inline WsLayout ws_layout(int num_seqs, int num_q_heads, int num_kv_heads, int num_sms) {
    WsLayout l;
    const int64_t pairs = (int64_t)num_seqs * num_kv_heads, group = num_q_heads / num_kv_heads;
    l.parts = pairs + 2 * num_sms;
    l.o = (size_t)l.parts * group * kHeadDim * 4;
    l.ml = ((size_t)l.parts * group * sizeof(float2) + 255) & ~size_t(255);
    l.info = ((size_t)pairs * sizeof(int2) + 255) & ~size_t(255);
    return l;
}

// The split's parameters that follow from the call's, and the workspace's parts.
template <typename Args>
void fill_split(SplitParams &p, const Args &a) {
    p.q = a.q;
    p.num_pages = a.num_pages;
    p.block_table = a.block_table;
    p.bt_stride = a.bt_stride;
    p.seq_lens = a.seq_lens;
    p.num_seqs = a.num_seqs;
    p.max_seq_len = a.max_seq_len;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.block_size = a.block_size;
    p.tiles_per_page = (a.block_size + kTile - 1) / kTile;
    p.by_block = fast_div(a.block_size);
    p.by_tpp = fast_div(p.tiles_per_page);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    const WsLayout l = ws_layout(a.num_seqs, a.num_q_heads, a.num_kv_heads, a.num_sms);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + l.o);
    p.info = reinterpret_cast<int2 *>(ws + l.o + l.ml);
    p.parts = l.parts;
    p.out = a.out;
    p.err = a.err;
    p.ctas = 0;
}

// CTAs of the streaming kernel: no more than the longest allowed lengths would use.
template <int kMinShare, bool kAlone = false, typename Args>
int split_grid(const SplitParams &p, const Args &a) {
    const int64_t tiles = (int64_t)(a.max_seq_len / a.block_size) * p.tiles_per_page +
                          (a.max_seq_len % a.block_size + kTile - 1) / kTile;
    const int64_t pairs = (int64_t)a.num_seqs * a.num_kv_heads, most = 2 * a.num_sms;
    const int64_t grid = kAlone && a.num_seqs == 1 ? pairs * ((tiles + kMinShare - 1) / kMinShare)
                                                   : (pairs * tiles + kMinShare - 1) / kMinShare;
    return (int)(grid < most ? grid : most);
}

template <int kFewRound, int kShare = 0>
cudaError_t launch_merge(const SplitParams &p, int num_sms, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.num_seqs * p.num_q_heads;
    if constexpr (kShare > 0)
        if (p.num_seqs == 1 && rows <= num_sms && p.ctas >= p.num_kv_heads) {
            // All parts in one round, and code for no more (it runs once): 1701 keys of 4 heads (27 parts) with 4 a
            // warp 6.9 us, with 10 7.1; 4000 (63) with 8 7.8, with 10 8.4.
            const int parts = p.ctas / p.num_kv_heads;
            const auto kernel = parts <= 32   ? decode_merge_kernel<8, 4, kShare>
                                : parts <= 64 ? decode_merge_kernel<8, 8, kShare>
                                              : decode_merge_kernel<8, 10, kShare>;
            return launch_pdl(kernel, dim3((unsigned)(rows * 4)), dim3(256), 0, stream, p);
        }
    if (rows <= num_sms)
        return launch_pdl(decode_merge_kernel<8, kFewRound>, dim3((unsigned)(rows * 4)), dim3(256), 0, stream, p);
    if (rows <= 8 * num_sms)
        return launch_pdl(decode_merge_kernel<4, 4>, dim3((unsigned)(rows * 2)), dim3(256), 0, stream, p);
    return launch_pdl(decode_merge_kernel<1, 4>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, p);
}

}  // namespace

}  // namespace pa
