// pa_decode_q4.cu -- q=1 decode over the 4-bit cache (format: pa_q4.cuh): a kernel that
// streams the cache, and one that merges the parts of sequences that it cut.
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
// take a 16-token tile (4.6 KB) about every 100 ns (200 cycles), so besides HBM the
// instructions count; most of them widen codes.
//   * Four bits in the low bits of an FP16 are the subnormal n 2^-24, and in bits 4 to 7 the
//     subnormal n 2^-20: a mask alone makes a pair of codes an exact operand of the tensor
//     cores; 5 operations widen 8 codes.  The 2^4 between the two kinds is put into q (K) and
//     taken out of the sums at the end (V).  (As FP8 operands codes would need 3 operations for
//     8, but FP8 operands of this MMA are converted to FP16 first: measured slower.)
//   * V's pairs run along tokens: two tokens' words are interleaved by halves first (two byte
//     permutations for 16 codes).
//   * The lo terms of the scores are one more BF16 product over (group, part of sum(q)) with
//     sum(q) in three BF16 parts: one MMA instead of 16 multiply-adds.
// q becomes FP16 after scaling each head by a power of two (largest value in [2^13, 2^14)):
// exact for values down to 2^-24 of the head's largest, and below that off by less than
// 2^-34 of it.
// The weights p s become FP16 (off by 2^-11 of them at most), scaled so that they neither
// overflow nor vanish: p = 2^(x - m - kLag), m the largest score and at most kLag behind, so p <=
// 1, and the p of a token that outweighs all others is a power of two, which leaves p s as exact
// as s; and p s F, F for each head and group, that leaves the group's largest weight at 1 at
// least, so that the smallest FP16 is 2^-24 of it, whatever the other groups and the tokens
// without weight hold.  (One reference for all groups, from the largest score and the largest
// step taken apart, left groups 2^24 apart 5% off.)  While steps are alike F comes from them
// alone, for all heads; where they are not, from the scores too.  It is a power of two but where
// it follows m over tokens that are not alike.  One vote a step finds whether anything moves: a
// score above m + kLag, or a step that could give a weight above 2^15.  s and F are applied to
// both heads of a lane by products of pairs (1% of the time less than one by one).  Against a
// form without F, all of this costs 2% of a long batch's time (16 sequences: 67.2 us) and 0.8 us
// of a short sequence's.
//
// Work split: the tiles of all (sequence, KV head) pairs in a row, cut evenly over two CTAs an
// SM, so that uneven lengths leave no SM idle; each CTA finds its share from the lengths.  A pair
// also costs its beginning (table, q, the first loads' way, the merge): it counts as kPairCost
// tiles, half a share at most, ahead of the pair's first, so that CTAs with many short pairs get
// fewer tiles (with 0, 4, 8, 16 and 28: 64 sequences of 1..2048 keys, 8 KV heads, 69, 65, 54, 44
// and 45 us; 16 of 1..4096, 4 KV heads, 29, 22, 18, 17 and 17; 64 of which one has 32768 and the
// others up to 200, 60, 38, 31, 26 and 26).  Shares below two rounds of the warps' tiles stay even:
// there a CTA's time is its rounds (one sequence of 1701 keys, shares of 8).  A pair
// that one CTA holds whole is finished there; the others leave a part per CTA (sums relative to
// their reference), which a second kernel merges.
// Within a CTA each warp streams pairs of 16-token tiles of its own (every kW-th pair) through a
// ring of its own: eight of its lanes bring one run each (codes and pairs of K and of V, of each
// tile) by bulk copies, which are contiguous, need no tensor map and are never longer than the
// page's and the sequence's valid rows.  Nothing is exchanged between warps before the merge.
// A warp keeps all 256 dims' sums (64 registers) and works on two tiles at once, whose MMA chains
// are interleaved: 8 such warps an SM ran faster than 12 with 168 registers each, or 16 in pairs
// that shared the dims (16 sequences of 4K..32K keys: 82, 96 and 104 us in an earlier form),
// because the extra warps cost instructions (spills, exchanges, loads), and issue is what bounds.
//
// Measured, calls one after another, 4 KV heads of 6 query heads unless said: 16 sequences of
// 4K..32K keys 68.8 us (streaming kernel 4.9 TB/s); 64 of 1..2048 keys, 8 KV heads of 4, pages of
// 16: 43.7 us; one of 32768 keys 17.3 us; one of 1701 keys 11.0 us.  The short ones are latency:
// finding the share 1.5 us, q 1.2, one step 2, the CTA's merge 1, and the second kernel.
#include "pa_decode_split.cuh"
#include "pa_q4.cuh"

namespace pa {

namespace {

constexpr int kW = 4, kThreads = kW * 32;             // warps of a CTA
constexpr int kDepth = 2;                             // pairs of tiles in a warp's ring
constexpr int kTileCodes = kTile * kQ4CodeBytes;      // 2 KB
constexpr int kTilePairs = kTile * kQ4PairBytes;      // 256 B
// A slot: K codes of both tiles, V codes, K pairs, V pairs.
constexpr int kSlotBytes = 4 * (kTileCodes + kTilePairs);
constexpr int kOffV = 2 * kTileCodes, kOffPairs = 4 * kTileCodes, kOffVPairs = kOffPairs + 2 * kTilePairs;
constexpr int kRingBytes = kW * kDepth * kSlotBytes;
constexpr int kMergeRow = kHeadDim + 4;
// Shared memory: rings; the merge's rows and (reference, sum) pairs; q's fragments (8 x 512
// bytes, and sums and scales); barriers and valid rows.
constexpr int kOffMerge = kRingBytes, kOffMl = kOffMerge + kW * kDecMaxGroup * kMergeRow * 4;
constexpr int kOffQ = kOffMl + kW * kDecMaxGroup * 8, kOffBars = kOffQ + 9 * 512;
constexpr int kSmem = kOffBars + kW * kDepth * 16 + 16;
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
constexpr int kMinShare = 2 * kW;                     // tiles of the smallest share
constexpr int kPairCost = 16;                         // of beginning a pair, in tiles
constexpr float kLag = 8.f;  // log2 units: a score may pass the reference by it
constexpr float kTop = 4.f;  // where F follows the scores, the largest weight is 2^(kTop - 1) .. 2^(kTop + 1)
constexpr int kSpare = 2;    // where it follows the steps, they may grow by 2^kSpare unexamined

struct Params : SplitParams {
    const uint8_t *k_cache, *v_cache;
    int64_t page_stride;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// The four pairs (codes k, k + 4) of a word as FP16 subnormals: k
// even as n 2^-24, k odd as n 2^-20.  The last comes from a subtraction (of (n2 + 16 n3) 2^-24 and
// n2 2^-24, exact): it runs beside the logic unit, which bounds this kernel.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&x)[4]) {
    const uint32_t high = __byte_perm(w, 0, 0x4341);  // the halves' upper bytes
    x[0] = w & 0x000f000fu;
    x[1] = w & 0x00f000f0u;
    x[2] = high & 0x000f000fu;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x[3]) : "r"(high), "r"(x[2]));
}

// 2^e of a whole number e <= 127; 0 below the normal range.
__device__ __forceinline__ float exp2_whole(float e) {
    return e < -126.f ? 0.f : __uint_as_float((uint32_t)((int)e + 127) << 23);
}
// floor(log2) of a positive number.
__device__ __forceinline__ float log2_whole(float f) {
    return (float)((int)(__float_as_uint(f) >> 23) - 127);
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

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

#ifdef PA_TEST_HOOKS
// Test build only: the pair of tiles (counted over each warp's run) whose loads are left out (-1:
// none), so that the warp's wait runs out.
__device__ int g_test_skip_pair = -1;
#endif

__global__ void __launch_bounds__(kThreads, 2) decode_q4_stream_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBars) + warp * kDepth;  // this warp's ring,
    int2 *rows_in = reinterpret_cast<int2 *>(smem + kOffBars + kW * kDepth * 8) + warp * kDepth;  // its valid rows
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffBars + kW * kDepth * 16);
    uint8_t *ring = smem + warp * kDepth * kSlotBytes;

    if (lane == 0) {
        for (int s = 0; s < kDepth; ++s) mbar_init(&full[s], 1);
        if (warp == 0) *abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share of all tiles, and the segment that it begins with: tile t0 of KV head
    // g of sequence seq (every warp finds the same)
    const int tpp = p.tiles_per_page;
    Start st;
    Shares &shares = st.shares;
    uint32_t &at = st.at, &end = st.end;
    int &lead = st.lead, &v0 = st.v0, &seq = st.seq, &g = st.g, &seq_len = st.seq_len, &tiles = st.tiles;
    int t0;  // the segment's first tile

    const int r = lane >> 2, c = lane & 3;
    const uint32_t q_frag = smem_u32(smem + kOffQ) + lane * 16;
    // Lanes 0 .. 7 load: lane = 4 x (tile of the pair) + run (K codes, V codes, K pairs, V pairs).
    const int l_tile = (lane >> 2) & 1, kind = lane & 3;
    const int l_bytes = kind >= 2 ? kQ4PairBytes : kQ4CodeBytes;
    uint8_t *l_dst = ring + (kind >= 2 ? kOffPairs + (2 * (kind - 2) + l_tile) * kTilePairs
                                       : (2 * kind + l_tile) * kTileCodes);
    const uint8_t *l_src;            // of the KV head's codes or pairs
    const int32_t *bt;
    int j_in, lp_in, tip_in, page_in, t1, n;
    uint32_t it = 0;  // the warp's steps: slots and phases go on from segment to segment
    bool gave_up;  // a wait ran out: this and the CTA's remaining segments contribute nothing

    // Starts a segment: tiles [t0, t1) of KV head g of sequence seq, at least one.
    auto begin_segment = [&]() {
        t0 = max(0, v0 - lead);
        t1 = (int)min((uint32_t)tiles, v0 + (end - at) - lead);
        n = !*abort && t0 + 2 * warp < t1 ? (t1 - t0 - 2 * warp + 2 * kW - 1) / (2 * kW) : 0;
        bt = p.block_table + (int64_t)seq * p.bt_stride;
        j_in = t0 + 2 * warp + l_tile;  // this lane's next tile
        lp_in = (int)p.by_tpp(j_in);
        tip_in = j_in - lp_in * tpp;
        page_in = j_in < t1 ? bt[lp_in] : 0;
        l_src = ((kind & 1) ? p.v_cache : p.k_cache) + (int64_t)g * p.block_size * kQ4RowBytes +
                (kind >= 2 ? (int64_t)p.block_size * kQ4CodeBytes : 0);
    };
    // Loads the warp's pair i, its next, into slot i % kDepth.
    auto load = [&](uint32_t i) {
        const uint32_t s = i % kDepth;
        const int page = page_in, off = tip_in * kTile;
        const int rows = j_in < t1 ? min(kTile, min(p.block_size - off,
                                                    seq_len - lp_in * p.block_size - off))
                                   : 0;
        const bool inside = page >= 0 && page < p.num_pages;
        uint8_t *dst = l_dst + s * kSlotBytes;
        const uint8_t *src = l_src + page * p.page_stride + (int64_t)off * l_bytes;
        if (lane == 0 || lane == 4) (&rows_in[s].x)[l_tile] = rows;
        // The next pair's table entry, read ahead of its use.
        j_in += 2 * kW;
        for (tip_in += 2 * kW; tip_in >= tpp; tip_in -= tpp) ++lp_in;
        if (j_in < t1) page_in = bt[lp_in];
        if (rows > 0 && !inside && lane < 8) {
            // Outside the pool: reported, and read as zeros (steps and minima of 0).
            if (kind == 0) atomicOr(p.err, kErrPage);
            if (kind >= 2)
                for (int k = 0; k < rows; ++k) reinterpret_cast<uint4 *>(dst)[k] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
        }
        // Two tiles that follow one another in a page come as one run (a copy's cost hardly
        // grows with its size): lanes 0 .. 3 then take both tiles' rows.
        int mine = inside ? rows : 0;
        const int other = __shfl_xor_sync(0xffffffffu, mine, 4);
        const int next = __shfl_xor_sync(0xffffffffu, off, 4);  // lanes 0 .. 3: tile 1's place
        const int total = mine + other;
        const bool joined = __shfl_sync(0xffffffffu, (int)(mine == kTile && other > 0 && next == off + kTile), 0);
        if (joined) mine = l_tile ? 0 : total;
        __syncwarp();  // zeros go before the arrival
#ifdef PA_TEST_HOOKS
        if ((int)i == *reinterpret_cast<volatile int *>(&g_test_skip_pair)) return;
#endif
        if (lane == 0) mbar_arrive_expect_tx(&full[s], total * 2 * kQ4RowBytes);
        __syncwarp();
        if (lane < 8 && mine) bulk_load(dst, src, mine * l_bytes, &full[s], l2_evict_first_policy());
    };
    int loaded = 0;
    auto first_loads = [&]() {
        for (loaded = 0; loaded < min(n, kDepth - 1); ++loaded) load(it + loaded);
    };
    // q as FP16 B fragments in shared memory: lane (head r, column c) holds dims 64g + 8(2c + h)
    // + j; MMA i of word h takes the pairs (2i, 2i + 4) and (2i + 1, 2i + 5), the latter 2^-4 as
    // large.  Each warp loads all of q (for the heads' largest values) and makes one group's.
    uint4 raw[8];
    auto load_q = [&]() {
        const uint4 *qrow = reinterpret_cast<const uint4 *>(
            p.q + ((int64_t)seq * p.num_q_heads + g * p.group + (r < p.group ? r : 0)) * kHeadDim);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            raw[k] = r < p.group ? qrow[(k >> 1) * 8 + 2 * c + (k & 1)] : make_uint4(0, 0, 0, 0);
    };
    auto make_q = [&]() {
        uint4 *own = reinterpret_cast<uint4 *>(smem + kOffQ) + lane;
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                amax = max(amax, max((word(raw[k], i) << 16) & 0x7fff0000u, word(raw[k], i) & 0x7fff0000u));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // A power of two f that brings the head's largest value to [2^13, 2^14).
        const int e = (int)(amax >> 23);
        const float f = e == 255 ? 1.f : __uint_as_float((uint32_t)min(254, max(1, 267 - e)) << 23);
        static_assert(kW == 4, "a warp a group");
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 mine = raw[h];
#pragma unroll
            for (int k = 1; k < 4; ++k)
                if (warp == k) mine = raw[2 * k + h];
            float v[8];
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(word(mine, i)) * f;
                v[2 * i + 1] = bf16_hi(word(mine, i)) * f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum += v[i] + v[i + 4];
                x[i] = i & 1 ? pack_f16x2(v[i] * 0x1p-4f, v[i + 4] * 0x1p-4f) : pack_f16x2(v[i], v[i + 4]);
            }
            own[(2 * warp + h) * 32] = make_uint4(x[0], x[1], x[2], x[3]);
        }
        // sum(q) 2^-24 of head r and group c in three BF16 parts, and the scales of the columns'
        // heads
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= 0x1p-24f;
        const float p1 = __bfloat162float(__float2bfloat16_rn(sum));
        const float p2 = __bfloat162float(__float2bfloat16_rn(sum - p1));
        const float sc = p.scale_log2 * 0x1p24f / f;
        const float sc0 = __shfl_sync(0xffffffffu, sc, 8 * c), sc1 = __shfl_sync(0xffffffffu, sc, 8 * c + 4);
        if (c == warp)
            own[8 * 32] = make_uint4(pack_bf16x2(p1, p2), pack_bf16x2(sum - p1 - p2, 0.f),
                                     __float_as_uint(sc0), __float_as_uint(sc1));
    };

    // With one sequence, its length is nearly always the longest allowed: the table entry and q are
    // then read beside the length instead of after it.
    Lengths<1> lens, most;
    lens.tiles[0] = seq_tiles(p, lane, &lens.len[0], blockIdx.x == 0 && warp == 0);
    bool guess = p.num_seqs == 1;
    Found found;
    for (;;) {
        if (guess) {
            most.tiles[0] = lane == 0 ? tiles_of(p, p.max_seq_len) : 0;
            most.len[0] = p.max_seq_len;
            found = find_start<kMinShare, kPairCost>(p, lane, false, most, st);
        } else {
            found = find_start<kMinShare, kPairCost>(p, lane, blockIdx.x == 0 && warp == 0, lens, st);
        }
        if (found == Found::kShare) {
            begin_segment();
            load_q();
        }
        if (!guess || __shfl_sync(0xffffffffu, lens.len[0], 0) == p.max_seq_len) break;
        guess = false;
    }
    if (found != Found::kShare) {
        if (found == Found::kRefused) {  // (not by a guess) tells the merge so: the pairs have no parts
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrSeqLen);
            const int64_t pairs = (int64_t)p.num_seqs * p.num_kv_heads;
            for (int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x; x < pairs; x += gridDim.x * kThreads)
                p.info[x] = make_int2(0, 0);
        }
        return;
    }
    first_loads();
    make_q();
    __syncthreads();  // q is ready
    for (;;) {
        // [group][dim pair][(dim, head) of the pairs], of even dims 2^24 and of odd dims 2^20
        // times too small
        float o[4][4][4];
        float low0[4], low1[4];  // this lane's share of sum p lo
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
            low0[gg] = low1[gg] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[gg][k][0] = o[gg][k][1] = o[gg][k][2] = o[gg][k][3] = 0.f;
        }
        // Running references of heads 2c and 2c + 1, and their groups' factors.
        float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
        float f0[4], f1[4];
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) f0[gg] = f1[gg] = 0x1p126f;
        uint32_t safe01 = 0, safe23 = 0;  // steps up to these (of groups 0, 1 and 2, 3) give at most 2^15

        for (int i = 0; i < n; ++i) {
            if (loaded < n) load(it + loaded++);  // into the slot that the previous pair has left
            const uint32_t s = (it + i) % kDepth;
            if (!__all_sync(0xffffffffu,
                            mbar_wait_abort(&full[s], ((it + i) / kDepth) & 1, p.err, abort)))
                break;
            const int2 nv = rows_in[s];
            const uint32_t base = smem_u32(ring) + s * kSlotBytes;

            // ---- scores of tokens r and r + 8 of each tile, heads 2c and 2c + 1: 8 accumulators
            // (tile, group) in turn
            float x[2][4];
            uint32_t big01 = 0, big23 = 0;  // the largest steps of V, of groups 0, 1 and 2, 3
            {
                const uint4 qa = lds128(q_frag + 8 * 512);  // sums of (head r, group c); scales
                const uint32_t ka = base + r * 128 + (((2 * c) ^ r) << 4);
                const uint32_t pa = base + kOffPairs + r * 16;
                float a[2][4][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 k0[2], k1[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        k0[t] = lds128((h ? ka ^ 16 : ka) + t * kTileCodes);
                        k1[t] = lds128((h ? ka ^ 16 : ka) + t * kTileCodes + 1024);
                    }
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) {
                        const uint4 q = lds128(q_frag + (2 * gg + h) * 512);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            uint32_t u[4], v[4];
                            widen(word(k0[t], gg), u);
                            widen(word(k1[t], gg), v);
                            if (h == 0)
                                mma_f16_zero(a[t][gg], u[0], v[0], u[1], v[1], q.x, q.y);
                            else
                                mma_f16(a[t][gg], u[0], v[0], u[1], v[1], q.x, q.y);
                            mma_f16(a[t][gg], u[2], v[2], u[3], v[3], q.z, q.w);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t kp = pa + t * kTilePairs;
                    const uint32_t lo0 = __byte_perm(lds32(kp + c * 4), 0, 0x3232);
                    const uint32_t lo1 = __byte_perm(lds32(kp + c * 4 + 128), 0, 0x3232);
                    const uint4 pr0 = lds128(kp), pr1 = lds128(kp + 128);
                    const uint4 vp0 = lds128(kp + 2 * kTilePairs), vp1 = lds128(kp + 2 * kTilePairs + 128);
                    uint32_t a01 = __byte_perm(vp0.x, vp0.y, 0x5410), a23 = __byte_perm(vp0.z, vp0.w, 0x5410);
                    uint32_t b01 = __byte_perm(vp1.x, vp1.y, 0x5410), b23 = __byte_perm(vp1.z, vp1.w, 0x5410);
                    x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
                    mma_bf16_16816(x[t], lo0, lo1, lo0, lo1, qa.x, qa.y);
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) {
                        const float s0 = q4_step(word(pr0, gg)), s1 = q4_step(word(pr1, gg));
                        x[t][0] = fmaf(s0, a[t][gg][0], x[t][0]);
                        x[t][1] = fmaf(s0, a[t][gg][1], x[t][1]);
                        x[t][2] = fmaf(s1, a[t][gg][2], x[t][2]);
                        x[t][3] = fmaf(s1, a[t][gg][3], x[t][3]);
                    }
                    x[t][0] *= __uint_as_float(qa.z);
                    x[t][1] *= __uint_as_float(qa.w);
                    x[t][2] *= __uint_as_float(qa.z);
                    x[t][3] *= __uint_as_float(qa.w);
                    const int nvalid = t ? nv.y : nv.x;
                    if (nvalid < kTile) {  // what lies behind the valid rows may be anything
                        if (r >= nvalid) {
                            x[t][0] = x[t][1] = -CUDART_INF_F;
                            a01 = a23 = 0;
                        }
                        if (r + 8 >= nvalid) {
                            x[t][2] = x[t][3] = -CUDART_INF_F;
                            b01 = b23 = 0;
                        }
                    }
                    big01 = max_bf16x2(big01, max_bf16x2(a01, b01));
                    big23 = max_bf16x2(big23, max_bf16x2(a23, b23));
                }
            }

            // The pairs of V of tokens r and r + 8 of tile t.
            auto v_pairs = [&](int t, uint4 &vp0, uint4 &vp1) {
                const uint32_t vp = base + kOffVPairs + t * kTilePairs + r * 16;
                vp0 = lds128(vp);
                vp1 = lds128(vp + 128);
                const int nvalid = t ? nv.y : nv.x;
                if (nvalid < kTile) {
                    if (r >= nvalid) vp0 = make_uint4(0, 0, 0, 0);
                    if (r + 8 >= nvalid) vp1 = make_uint4(0, 0, 0, 0);
                }
            };

            // ---- references: moved (in the first step always) when a score passes by more than
            // kLag, or when a step is large enough for a weight to pass 2^15
            float mx0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
            float mx1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
            const bool large = max_bf16x2(big01, safe01) != safe01 || max_bf16x2(big23, safe23) != safe23;
            if (__any_sync(0xffffffffu, mx0 > m0 + kLag || mx1 > m1 + kLag || large)) {
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
                }
                const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                const float d0 = n0 == m0 ? 0.f : n0 - m0, d1 = n1 == m1 ? 0.f : n1 - m1;
                m0 = n0;
                m1 = n1;
                const float al0 = ex2_approx(-d0), al1 = ex2_approx(-d1);
                float g0[4], g1[4];  // what the sums of each group are multiplied by
#pragma unroll
                for (int gg = 0; gg < 4; ++gg) {
                    g0[gg] = al0;
                    g1[gg] = al1;
                }
                if (i == 0) {  // room for steps 2^kSpare times the largest
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) {
                        big01 = max_bf16x2(big01, __shfl_xor_sync(0xffffffffu, big01, sh));
                        big23 = max_bf16x2(big23, __shfl_xor_sync(0xffffffffu, big23, sh));
                    }
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) {
                        const int e = ((gg < 2 ? big01 : big23) >> (gg & 1 ? 23 : 7)) & 255;
                        f0[gg] = f1[gg] = __uint_as_float(min(253, 2 * 127 + 14 - kSpare - e) << 23);
                    }
                }
                // While every step times F is 2^8 at least, the token that moved m (p = 2^-8) gives the
                // group a weight of 1 at least, and F can stay.
                uint32_t low01 = 0x7f807f80u, low23 = low01;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int nvalid = t ? nv.y : nv.x;
                    uint4 vp0, vp1;
                    v_pairs(t, vp0, vp1);
                    if (r < nvalid) {
                        low01 = min_bf16x2(low01, __byte_perm(vp0.x, vp0.y, 0x5410));
                        low23 = min_bf16x2(low23, __byte_perm(vp0.z, vp0.w, 0x5410));
                    }
                    if (r + 8 < nvalid) {
                        low01 = min_bf16x2(low01, __byte_perm(vp1.x, vp1.y, 0x5410));
                        low23 = min_bf16x2(low23, __byte_perm(vp1.z, vp1.w, 0x5410));
                    }
                }
                const bool even = bf16_lo(low01) * fminf(f0[0], f1[0]) >= 256.f &&
                                  bf16_hi(low01) * fminf(f0[1], f1[1]) >= 256.f &&
                                  bf16_lo(low23) * fminf(f0[2], f1[2]) >= 256.f &&
                                  bf16_hi(low23) * fminf(f0[3], f1[3]) >= 256.f;
                if (!__all_sync(0xffffffffu, even && (i == 0 || !large))) {
                    // The groups' largest x + floor(log2 s): their p s is 2^(t - m - kLag) to twice that.
                    float t0[4], t1[4];
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) t0[gg] = t1[gg] = -CUDART_INF_F;
#pragma unroll 1
                    for (int t = 0; t < 2; ++t) {
                        uint4 vp0, vp1;
                        v_pairs(t, vp0, vp1);
#pragma unroll
                        for (int gg = 0; gg < 4; ++gg) {
                            const float s0 = q4_step(word(vp0, gg)), s1 = q4_step(word(vp1, gg));
                            const float e0 = s0 > 0.f ? log2_whole(s0) : -CUDART_INF_F;
                            const float e1 = s1 > 0.f ? log2_whole(s1) : -CUDART_INF_F;
                            t0[gg] = fmaxf(t0[gg], fmaxf((t ? x[1][0] : x[0][0]) + e0,
                                                         (t ? x[1][2] : x[0][2]) + e1));
                            t1[gg] = fmaxf(t1[gg], fmaxf((t ? x[1][1] : x[0][1]) + e0,
                                                         (t ? x[1][3] : x[0][3]) + e1));
                        }
                    }
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) {
#pragma unroll 1
                        for (int sh = 4; sh < 32; sh <<= 1) {
                            t0[gg] = fmaxf(t0[gg], __shfl_xor_sync(0xffffffffu, t0[gg], sh));
                            t1[gg] = fmaxf(t1[gg], __shfl_xor_sync(0xffffffffu, t1[gg], sh));
                        }
                        // F goes up only to follow m (it need not be a power of two then), and down
                        // where this step's largest needs it.
                        auto moved = [&](float &f, float n, float d, float al, float top) {
                            const float keep = i == 0 ? 0x1p126f : f * ex2_approx(d);
                            const float e = floorf(n + kLag + kTop - 1.f - top);
                            const float to = fminf(keep, exp2_whole(fmaxf(-122.f, fminf(126.f, e))));
                            const float g = to == keep ? 1.f : al * fminf(to / f, 0x1p127f);
                            f = to;
                            return g;
                        };
                        g0[gg] = moved(f0[gg], n0, d0, al0, t0[gg]);
                        g1[gg] = moved(f1[gg], n1, d1, al1, t1[gg]);
                    }
                }
                // Steps that cannot give a weight above 2^15 (p is 1 at most) with this lane's heads.
                auto safe = [&](int gg) {
                    const uint32_t up = (__float_as_uint(fmaxf(f0[gg], f1[gg])) + 0x7fffff) >> 23;
                    return min(254u, 2 * 127 + 15 - up) << 7;
                };
                safe01 = safe(0) | safe(1) << 16;
                safe23 = safe(2) | safe(3) << 16;
                if (i > 0) {
                    l0 *= al0;
                    l1 *= al1;
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) {
                        low0[gg] *= al0;
                        low1[gg] *= al1;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            o[gg][k][0] *= g0[gg];
                            o[gg][k][1] *= g1[gg];
                            o[gg][k][2] *= g0[gg];
                            o[gg][k][3] *= g1[gg];
                        }
                    }
                }
            }
            const float mu0 = m0 == -CUDART_INF_F ? 0.f : m0 + kLag;
            const float mu1 = m1 == -CUDART_INF_F ? 0.f : m1 + kLag;

            // ---- O^T += V^T (p s)^T, two tokens' codes a register
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float p00 = ex2_approx(x[t][0] - mu0), p01 = ex2_approx(x[t][1] - mu1);
                const float p10 = ex2_approx(x[t][2] - mu0), p11 = ex2_approx(x[t][3] - mu1);
                l0 += p00 + p10;
                l1 += p01 + p11;
                const uint32_t vt = base + kOffV + t * kTileCodes;
                const uint32_t v0 = vt + 2 * c * 128 + ((r ^ (2 * c)) << 4), v1 = (v0 ^ 16) + 128;
                const uint4 va = lds128(v0), vb = lds128(v1);                // tokens 2c, 2c + 1
                const uint4 vc = lds128(v0 + 1024), vd = lds128(v1 + 1024);  // tokens 2c + 8, 2c + 9
                uint4 vp0, vp1;
                v_pairs(t, vp0, vp1);
#pragma unroll
                for (int gg = 0; gg < 4; ++gg) {
                    const float lo0 = q4_low(word(vp0, gg)), lo1 = q4_low(word(vp1, gg));
                    low0[gg] = fmaf(p00, lo0, fmaf(p10, lo1, low0[gg]));
                    low1[gg] = fmaf(p01, lo0, fmaf(p11, lo1, low1[gg]));
                    const float s0 = q4_step(word(vp0, gg)), s1 = q4_step(word(vp1, gg));
                    float a0, a1, c0, c1;  // (p s is in fp32's range whatever F is)
                    mul2(a0, a1, p00, p01, s0, s0);
                    mul2(c0, c1, p10, p11, s1, s1);
                    mul2(a0, a1, a0, a1, f0[gg], f1[gg]);
                    mul2(c0, c1, c0, c1, f0[gg], f1[gg]);
                    const uint32_t b0 = movmatrix_t(pack_f16x2(a0, a1));
                    const uint32_t b1 = movmatrix_t(pack_f16x2(c0, c1));
                    uint32_t u[4], v[4];
                    widen(__byte_perm(word(va, gg), word(vb, gg), 0x5410), u);
                    widen(__byte_perm(word(vc, gg), word(vd, gg), 0x5410), v);
                    mma_f16(o[gg][0], u[0], u[1], v[0], v[1], b0, b1);
                    mma_f16(o[gg][1], u[2], u[3], v[2], v[3], b0, b1);
                    widen(__byte_perm(word(va, gg), word(vb, gg), 0x7632), u);
                    widen(__byte_perm(word(vc, gg), word(vd, gg), 0x7632), v);
                    mma_f16(o[gg][2], u[0], u[1], v[0], v[1], b0, b1);
                    mma_f16(o[gg][3], u[2], u[3], v[2], v[3], b0, b1);
                }
            }
            __syncwarp();  // the slot is free
        }
        // Every load lands before its slot is loaded again or left (when a wait gave up).
        for (uint32_t i = it + max(0, loaded - kDepth); i < it + loaded; ++i)
            mbar_wait(&full[i % kDepth], (i / kDepth) & 1, p.err);
        it += n;
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

        // ---- the next segment's first loads and its q, before this one's merge
        const int64_t pair = (int64_t)seq * p.num_kv_heads + g, part = blockIdx.x + pair;
        const bool whole = t0 == 0 && t1 == tiles;
        if (threadIdx.x == 0 && t0 == 0)
            p.info[pair] = make_int2((int)part, whole ? 0 : (int)(shares.owner(at - v0 + lead + tiles - 1) - blockIdx.x) + 1);
        uint16_t *out_rows = p.out + ((int64_t)seq * p.num_q_heads + g * p.group) * kHeadDim;
        at += lead + t1 - v0;
        const bool more = end > at + lead;  // (a share that ends before the next pair's first tile is done)
        if (more) {
            v0 = 0;
            if (++g == p.num_kv_heads) {
                g = 0;
                do tiles = seq_tiles(p, ++seq, &seq_len, false);
                while (tiles == 0 && seq < p.num_seqs);
            }
            begin_segment();
            load_q();
            first_loads();
        }

        // ------------------------------------------------------------ merge of the warps
        float *red_o = reinterpret_cast<float *>(smem + kOffMerge);      // [warp][head][row]
        float2 *red_ml = reinterpret_cast<float2 *>(smem + kOffMl);      // [warp][head]
        if (lane < 4) {
            red_ml[warp * kDecMaxGroup + 2 * c] = make_float2(m0, l0);
            red_ml[warp * kDecMaxGroup + 2 * c + 1] = make_float2(m1, l1);
        }
        {
            float *row0 = red_o + (warp * kDecMaxGroup + 2 * c) * kMergeRow + 8 * r;
#pragma unroll
            for (int gg = 0; gg < 4; ++gg) {
                const float u0 = rcp_approx(f0[gg]), u1 = rcp_approx(f1[gg]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    auto row = [&](int h, float low, float u) {
                        return make_float4(fmaf(o[gg][2 * k][h] * 0x1p24f, u, low),
                                           fmaf(o[gg][2 * k][2 + h] * 0x1p20f, u, low),
                                           fmaf(o[gg][2 * k + 1][h] * 0x1p24f, u, low),
                                           fmaf(o[gg][2 * k + 1][2 + h] * 0x1p20f, u, low));
                    };
                    *reinterpret_cast<float4 *>(row0 + gg * 64 + k * 4) = row(0, low0[gg], u0);
                    *reinterpret_cast<float4 *>(row0 + kMergeRow + gg * 64 + k * 4) = row(1, low1[gg], u1);
                }
            }
        }
        __syncthreads();  // every warp's rows are there, and q is no longer read
        gave_up = *abort != 0;
        if (more) make_q();
        for (int qd = threadIdx.x; qd < p.group * (kHeadDim / 4); qd += kThreads) {
            const int h = qd / (kHeadDim / 4), d = (qd - h * (kHeadDim / 4)) * 4;
            float M = -CUDART_INF_F;
            float2 ml[kW];
#pragma unroll
            for (int v = 0; v < kW; ++v) {
                ml[v] = red_ml[v * kDecMaxGroup + h];
                M = fmaxf(M, ml[v].x);
            }
            float L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < kW; ++v) {
                const float e = M == -CUDART_INF_F ? 0.f : ex2_approx(ml[v].x - M);
                const float4 f = *reinterpret_cast<const float4 *>(red_o + (v * kDecMaxGroup + h) * kMergeRow + d);
                L += e * ml[v].y;
                O.x += e * f.x;
                O.y += e * f.y;
                O.z += e * f.z;
                O.w += e * f.w;
            }
            if (gave_up) {  // an empty part, or zeros
                O = make_float4(0.f, 0.f, 0.f, 0.f);
                M = -CUDART_INF_F;
                L = 0.f;
            }
            if (whole) {
                const float inv = L > 0.f ? 1.f / L : 0.f;
                *reinterpret_cast<uint2 *>(out_rows + h * kHeadDim + d) =
                    make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (part * p.group + h) * kHeadDim + d) = O;
                if (d == 0) p.part_ml[part * p.group + h] = make_float2(M, L);
            }
        }

        if (!more) return;
        __syncthreads();  // q is ready, and the merge's rows are free
    }
}

}  // namespace

size_t decode_q4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int num_sms) {
    const WsLayout l = ws_layout(num_seqs, num_q_heads, num_kv_heads, num_sms);
    return l.o + l.ml + l.info;
}

#ifdef PA_TEST_HOOKS
cudaError_t set_decode_q4_test_hook(int skip_pair) {
    return cudaMemcpyToSymbol(g_test_skip_pair, &skip_pair, sizeof skip_pair);
}
int decode_q4_pair_lead(uint32_t tiles, uint64_t pairs, uint32_t ctas) { return pair_lead<kMinShare, kPairCost>(tiles, pairs, ctas); }
#endif

cudaError_t launch_decode_q4(const DecodeQ4Args &a, cudaStream_t stream) {
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(decode_q4_stream_kernel), kSmem, 6);
    if (e != cudaSuccess) return e;
    Params p;
    fill_split(p, a);
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.page_stride = a.page_stride;
    const int grid = split_grid<kMinShare>(p, a);
    if (a.ev_start && (e = record_event(a.ev_start, stream)) != cudaSuccess) return e;
    e = launch_pdl(decode_q4_stream_kernel, dim3(grid), dim3(kThreads), kSmem, stream, p);
    if (e != cudaSuccess) return e;
    if (a.ev_stop && (e = record_event(a.ev_stop, stream)) != cudaSuccess) return e;
    return launch_merge<4>(p, a.num_sms, stream);
}

}  // namespace pa
