// pa_decode_q8.cu -- q=1 decode over the 8-bit cache (format: pa_q8.cuh): a kernel that streams the
// cache, and one that merges the parts of sequences that it cut (pa_decode_split.cuh).
//
// For query head h of KV head g, over the sequence's tokens t < seq_len,
//     out = softmax_t(scale q . k_t) . v_t,   k_t = c_t 2^ek, v_t = d_t 2^ev,
// with one ek and one ev for each 16-token tile of a page: the tile of the matrix products.  So
// the products are of codes, which are exact in FP16:
//     x_t = (scale log2(e) 2^ek) (q . c_t),   out = sum_t 2^(x_t + ev - M') d_t / (2^-M' sum_t 2^x_t)
// and the scales cost an addition and a product per (token, head).
//
// q becomes FP16 after scaling each head by a power of two (largest value in [2^13, 2^14)):
// exact for values down to 2^-24 of the head's largest, and below that off by less than 2^-34 of
// it.  The weights 2^(x + ev - M') become FP16 (off by 2^-11 of them at most); M' follows the
// largest x + ev, the reference m of the weights' sum the largest x, each at most kLag behind: a
// weight is 2^(kTop + kLag) at most, and those down to 2^(-14 - kTop) = 2^-20 of the largest keep
// all of FP16's bits, whatever the scales of tokens without weight are.
//
// Bytes: 8192 of codes and 2 of scales for a tile of K and V; at the copy bandwidth an SM has to take a
// tile about every 185 ns (370 cycles).  A warp's tile takes some 550 instructions (128 of them widen
// codes, two each; q's and the tile's fragments, 32 MMAs), so issue slots are 36% used and memory
// bounds long batches; short ones are bound by the chain of latencies.
//
// Long sequences: the tiles are cut evenly over two CTAs an SM (pa_decode_split.cuh).  Within a CTA each
// warp streams every kW-th tile through a ring of its own, a box of K and one of V a tile: two
// tiles ahead of the one it works on, so that 128 KB an SM are on their way.  A warp's loads do not stop
// at the end of a pair but go on into the next ones of the share.  Nothing is exchanged between
// warps before the CTA's merge, whose rows stand in the ring's slots that are free then.
// One sequence: each pair is cut by itself, so that no CTA begins two (1701 keys 9.7 -> 7.7 us).
// Short sequences: a cluster a pair, whose CTAs' parts are merged through their shared memory; no
// second kernel.  (A CTA waits at the cluster's barriers for the others, whose own waits are bounded.)
//
// Measured, calls one after another in a graph, 4 KV heads of 6 query heads unless said: 16 sequences of
// 4096..32768 keys 102 us, 6.7 TB/s; 64 of 1..2048, 8 KV heads of 4, pages of 16: 47.3 us (5.1 TB/s: begin, end and
// the slowest CTAs); one of 32768 keys 17.0 us, of 1701 7.0; 16 of 1..700 8.7 us, of 1..300 7.3.
#include "pa_decode_split.cuh"
#include "pa_q8.cuh"

namespace pa {

namespace {

constexpr int kW = 4, kThreads = kW * 32;             // warps of a CTA
constexpr int kDepth = 3;                             // tiles in a warp's ring
constexpr int kTileCodes = kTile * kHeadDim;          // 4 KB: [2 halves of the dims][16 tokens][128 bytes]
constexpr int kSlotBytes = 2 * kTileCodes;            // K, V
// Shared memory: rings (whose slots also take a warp's sums for the CTA's merge); q's fragments
// and scales; the warps' references; barriers and the slots of the sums.
constexpr int kOffQ = kW * kDepth * kSlotBytes, kOffMl = kOffQ + 9 * 512;
constexpr int kOffBars = kOffMl + kW * kDecMaxGroup * 8, kOffMisc = kOffBars + kW * kDepth * 8;
constexpr int kSmem = kOffMisc + 32 + 1024;           // (the rings start at a multiple of 1024)
constexpr int kOffPart = kOffMisc + 32;               // in a cluster, the CTA's part: sums, references
constexpr int kSmemCluster = kSmem + kSlotBytes + kDecMaxGroup * 8;
static_assert(kOffPart % 16 == 0, "loads of 16 bytes");
static_assert(kDecMaxGroup * kHeadDim * 4 == kSlotBytes, "a slot holds a warp's sums");
static_assert(2 * (kSmemCluster + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(kTile == kQ8Tokens, "a tile has one scale");
// Tiles of the smallest share.  One sequence of 1701 keys with 4, 8 and 16: 7.1, 7.7 and 9.4 us.
constexpr int kMinShare = kW;
// Of beginning a pair, in tiles.  64 sequences of 1..2048 keys (8 KV heads) with 2, 4, 8, 12 and 20: 65,
// 59, 51, 49 and 50 us; 200 of 1..1024: 109, 99, 89, 83 and 85; 32 of 1..4096 (4): 37, 35, 31, 31 and 31.
constexpr int kPairCost = 12;
// Of 32 sequences, whose lengths a warp keeps.  64 sequences with 1 and 4: 49.2 and 47.0 us; one
// sequence 0.1 us more.
constexpr int kBatches = 4;
// CTAs of a cluster, and the tiles that it may take a warp, of one sequence and of several.  Without and with
// a cluster: one sequence of 200 keys 6.4 and 5.5 us, of 900 6.9 and 6.8, of 1701 7.3 and 8.8; 16 of
// 1..700 16.5 and 8.7, 16 of 1500 16.0 and 13.1; 64 of 300 15.9 and 12.0; beyond 8 tiles even lengths still
// gain (16 of 3000 23.0 and 20.1) and uneven ones lose (16 of 1..3000 15.9 and 17.5).  Clusters of 16 start
// later: 4 sequences of 1000 keys 14.4 us, in clusters of 8 7.9, without 11.3.
constexpr int kMaxCluster = 8, kClusterSteps = 3, kClusterStepsMany = 8;
constexpr float kLag = 8.f;  // log2 units: a score may pass the reference by it
constexpr float kTop = 6.f;  // log2 of the weight at the reference M'

struct Params : SplitParams {
    const uint8_t *k_scales, *v_scales;
    int64_t scale_stride;
    int cluster;  // CTAs of a pair (kCluster)
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// All threads of the cluster's CTAs meet; what they wrote to shared memory is seen by the others.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// From the shared memory of CTA `rank` of the cluster, at this CTA's address `addr`.
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr, int rank) {
    float2 v;
    asm volatile("{.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [a];}"
                 : "=f"(v.x), "=f"(v.y) : "r"(addr), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, int rank) {
    float4 v;
    asm volatile("{.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
    return v;
}

#ifdef PA_TEST_HOOKS
// Test build only: the tile (counted over each warp's run) whose loads are left out (-1: none),
// so that the warp's wait runs out.
__device__ int g_test_skip_tile = -1;
#endif

// kCluster: short sequences.  A cluster of p.cluster CTAs takes a pair and cuts its tiles evenly; its
// parts are merged through the CTAs' shared memory, and no second kernel follows.
template <bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
    decode_q8_stream_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                            const __grid_constant__ Params p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t *smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBars) + warp * kDepth;  // this warp's ring
    volatile int *sum_slot = reinterpret_cast<volatile int *>(smem + kOffMisc);      // [warp]
    volatile int *abort = sum_slot + kW;
    uint8_t *ring = smem + warp * kDepth * kSlotBytes;

    if (lane == 0) {
        for (int s = 0; s < kDepth; ++s) mbar_init(&full[s], 1);
        if (warp == 0) {
            *abort = 0;
            tma_prefetch_desc(&k_map);
            tma_prefetch_desc(&v_map);
        }
        fence_mbar_init();
    }
    __syncthreads();

    // ---- this CTA's share of all tiles, and the segment that it begins with: tiles [t0, t1) of KV
    // head g of sequence seq
    const int tpp = p.tiles_per_page;
    Start st;
    int t0, t1, n;    // n: this warp's tiles of the segment
    uint32_t it = 0;  // the warp's tiles so far: slots and phases go on from segment to segment
    auto begin_segment = [&]() {
        t0 = max(0, st.v0 - st.lead);
        t1 = (int)min((uint32_t)st.tiles, st.v0 + (st.end - st.at) - st.lead);
        const bool stop = __any_sync(0xffffffffu, *abort != 0);  // (n is the warp's: its lanes wait together)
        n = !stop && t0 + warp < t1 ? (t1 - t0 - warp + kW - 1) / kW : 0;
    };
    // The next segment of the share, KV head after KV head, sequence after sequence.
    auto next_pair = [&](int &seq, int &g, int &seq_len, int &tiles) {
        if (++g == p.num_kv_heads) {
            g = 0;
            do tiles = seq_tiles<true>(p, ++seq, &seq_len, false);
            while (tiles == 0 && seq < p.num_seqs);
        }
    };

    // ---- the warp's loads, which run ahead of its work into the segments that follow
    const int r = lane >> 2, c = lane & 3;
    const uint32_t q_frag = smem_u32(smem + kOffQ) + lane * 16;
    struct {
        int seq, g, seq_len, tiles, t1;  // the segment
        uint32_t at;                     // the place of the row that it ends at
        int j, lp, tip, page;            // the warp's next tile
        uint32_t count;                  // loads issued
    } in;
    in.count = 0;
    auto load_pair = [&](int first) {
        in.j = first + warp;
        in.lp = (int)p.by_tpp(in.j);
        in.tip = in.j - in.lp * tpp;
        in.page = in.j < in.t1 ? __ldcg(p.block_table + (int64_t)in.seq * p.bt_stride + in.lp) : 0;
    };
    auto load_start = [&]() {
        in.seq = st.seq;
        in.g = st.g;
        in.seq_len = st.seq_len;
        in.tiles = st.tiles;
        in.t1 = t1;
        in.at = st.at + st.lead + t1 - st.v0;
        load_pair(t0);
    };
    // A tile's scale bytes, and its valid rows.
    struct Tile {
        uint32_t k_scale, v_scale;
        int rows;
    };
    // Loads the warp's next tile, if there is one, into slot in.count % kDepth.
    auto load = [&](Tile &t) {
        while (in.j >= in.t1) {
            if (st.end <= in.at + st.lead) return;
            next_pair(in.seq, in.g, in.seq_len, in.tiles);
            in.t1 = (int)min((uint32_t)in.tiles, st.end - in.at - st.lead);
            in.at += st.lead + in.t1;
            load_pair(0);
        }
        const uint32_t i = in.count++, s = i % kDepth;
        const int page = in.page, off = in.tip * kTile, g = in.g;
        t.rows = min(kTile, min(p.block_size - off, in.seq_len - in.lp * p.block_size - off));
        t.k_scale = t.v_scale = 127;
        // A page outside the pool is reported, and its box, which lies outside the map, reads as zeros.
        if (page >= 0 && page < p.num_pages) {
            const int64_t o = page * p.scale_stride + (int64_t)in.tip * p.num_kv_heads + g;
            t.k_scale = __ldcg(p.k_scales + o);
            t.v_scale = __ldcg(p.v_scales + o);
        } else if (lane == 0) {
            atomicOr(p.err, kErrPage);
        }
        // The next tile's table entry, read ahead of its use.
        in.j += kW;
        for (in.tip += kW; in.tip >= tpp; in.tip -= tpp) ++in.lp;
        if (in.j < in.t1) in.page = __ldcg(p.block_table + (int64_t)in.seq * p.bt_stride + in.lp);
#ifdef PA_TEST_HOOKS
        if ((int)i == *reinterpret_cast<volatile int *>(&g_test_skip_tile)) return;
#endif
        if (lane == 0) {
            uint8_t *dst = ring + s * kSlotBytes;
            const uint64_t policy = l2_evict_first_policy();
            mbar_arrive_expect_tx(&full[s], kSlotBytes);
            tma_load_5d_hint(dst, &k_map, &full[s], 0, off, 0, g, page, policy);
            tma_load_5d_hint(dst + kTileCodes, &v_map, &full[s], 0, off, 0, g, page, policy);
        }
    };
    Tile next0{}, next1{};  // of the next tiles
    static_assert(kDepth == 3, "two tiles ahead");
    // q as FP16 B fragments in shared memory: lane (head r, column c) holds dims 128a + 32c + 16b +
    // {0..15} (a, b = 0, 1) as two 16-byte words, word w of which are dims 4w and 4w + 1 (or + 2, + 3).
    // Each warp loads all of q (for the heads' largest values) and makes a quarter.
    uint4 raw[8];
    auto load_q = [&]() {
        const uint4 *qrow = reinterpret_cast<const uint4 *>(
            p.q + ((int64_t)st.seq * p.num_q_heads + st.g * p.group + (r < p.group ? r : 0)) * kHeadDim);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            raw[k] = r < p.group ? qrow[(k >> 2) * 16 + 4 * c + (k & 3)] : make_uint4(0, 0, 0, 0);
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
        static_assert(kW == 4, "a warp a quarter");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 mine = raw[h];
#pragma unroll
            for (int k = 1; k < 4; ++k)
                if (warp == k) mine = raw[2 * k + h];
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = pack_f16x2(bf16_lo(word(mine, i)) * f, bf16_hi(word(mine, i)) * f);
            own[(2 * warp + h) * 32] = make_uint4(x[0], x[1], x[2], x[3]);
        }
        const float sc = p.scale_log2 / f;
        const float sc0 = __shfl_sync(0xffffffffu, sc, 8 * c), sc1 = __shfl_sync(0xffffffffu, sc, 8 * c + 4);
        if (warp == 0) own[8 * 32] = make_uint4(__float_as_uint(sc0), __float_as_uint(sc1), 0, 0);
    };

    // The share is found before the wait for earlier work on the stream, from lengths that this work may
    // still write, and holds if they are the same after it; if not, and with more sequences than a warp
    // keeps, it is found again.  Meanwhile each warp's first tile comes into L2 (its table entry only
    // steers that).  What is read before the wait bypasses L1.  No tile, one, two and four: one
    // sequence of 32768 keys 18.6, 17.5, 17.5 and 18.5 us, 16 of 4096..32768 104.1, 101.3, 102.0 and 102.7.
    constexpr int kB = kCluster ? 1 : kBatches;
    const int pair_of_cluster = blockIdx.x / p.cluster, rank = blockIdx.x - pair_of_cluster * p.cluster;
    auto find = [&](const Lengths<kB> &lens, bool report) {
        if constexpr (!kCluster) {
            return find_start<kMinShare, kPairCost, true, true, kB>(p, lane, report, lens, st);
        } else {  // (every CTA takes part in its cluster's merge)
            st.ctas_a_pair = p.cluster;
            st.lead = 0;
            st.seq = pair_of_cluster / p.num_kv_heads;
            st.g = pair_of_cluster - st.seq * p.num_kv_heads;
            st.tiles = lens.tiles[0];
            st.seq_len = lens.len[0];
            st.shares.q = st.tiles / p.cluster;
            st.shares.r = st.tiles - st.shares.q * p.cluster;
            st.at = st.v0 = (int)st.shares.begin(rank);
            st.end = st.shares.begin(rank + 1);
            return Found::kShare;
        }
    };
    auto lengths = [&](bool report) {
        Lengths<kB> l;
#pragma unroll
        for (int b = 0; b < kB; ++b) {
            const int s = kCluster ? pair_of_cluster / p.num_kv_heads : 32 * b + lane;
            l.tiles[b] = seq_tiles<true>(p, s, &l.len[b], report);
        }
        return l;
    };
    const bool reports = (kCluster ? rank == 0 && pair_of_cluster % p.num_kv_heads == 0 : blockIdx.x == 0) && warp == 0;
    const bool early = kCluster || p.num_seqs <= 32 * kB;
    Lengths<kB> lens;
    Found found = Found::kNone;
    if (early) {
        lens = lengths(false);
        found = find(lens, false);
    }
    if (found == Found::kShare) {
        begin_segment();
        load_start();
        if (lane == 0 && in.j < in.t1 && in.page >= 0 && in.page < p.num_pages) {
            tma_prefetch_l2_5d_hint(&k_map, 0, in.tip * kTile, 0, in.g, in.page, l2_evict_first_policy());
            tma_prefetch_l2_5d_hint(&v_map, 0, in.tip * kTile, 0, in.g, in.page, l2_evict_first_policy());
        }
    }
    pdl_wait();
    pdl_trigger();
    const Lengths<kB> now = lengths(reports);
    if (found == Found::kShare) {
        load_q();
        load_pair(t0);  // (the table entry)
    }
    bool changed = !early;
#pragma unroll
    for (int b = 0; b < kB; ++b) changed |= early && now.len[b] != lens.len[b];
    if (__any_sync(0xffffffffu, changed)) {
        found = find(now, reports);
        if (found == Found::kShare) {
            begin_segment();
            load_start();
            load_q();
        }
    }
    if (found != Found::kShare) {
        if (found == Found::kRefused) {  // tells the merge so: the pairs have no parts
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrSeqLen);
            const int64_t pairs = (int64_t)p.num_seqs * p.num_kv_heads;
            for (int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x; x < pairs; x += gridDim.x * kThreads)
                p.info[x] = make_int2(0, 0);
        }
        return;
    }
    load(next0);
    load(next1);
    make_q();
    __syncthreads();  // q is ready
    for (;;) {
        float o[2][4][2][4];  // [half][word][dim pair][(dim, head) of the pairs], relative to M'
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int k = 0; k < 2; ++k) o[a][w][k][0] = o[a][w][k][1] = o[a][w][k][2] = o[a][w][k][3] = 0.f;
        // References of heads 2c and 2c + 1: m of the sums l, v (M') of o.
        float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
        float v_ref0 = -CUDART_INF_F, v_ref1 = -CUDART_INF_F;

        for (int i = 0; i < n; ++i) {
            const Tile now = next0;
            next0 = next1;
            load(next1);  // into the slot that the previous tile has left
            const uint32_t s = (it + i) % kDepth;
            if (!__all_sync(0xffffffffu, mbar_wait_abort(&full[s], ((it + i) / kDepth) & 1, p.err, abort))) break;
            const uint32_t base = smem_u32(ring) + s * kSlotBytes;

            // ---- scores of tokens r and r + 8, heads 2c and 2c + 1: 4 accumulators in turn
            float x[4];
            {
                const uint32_t ka = base + r * 128 + (((2 * c) ^ r) << 4);
                float acc[4][4];
#pragma unroll
                for (int ab = 0; ab < 4; ++ab) {  // (half a of the dims, unit b of the lane's two)
                    const uint32_t k_at = (ab & 1 ? ka ^ 16 : ka) + (ab >> 1) * 2048;
                    const uint4 k0 = lds128(k_at), k1 = lds128(k_at + 1024);
                    const uint4 qa = lds128(q_frag + 2 * ab * 512), qb = lds128(q_frag + (2 * ab + 1) * 512);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a0 = f16x2_of_e4m3(word(k0, w)), a1 = f16x2_of_e4m3(word(k1, w));
                        const uint32_t a2 = f16x2_of_e4m3_hi(word(k0, w)), a3 = f16x2_of_e4m3_hi(word(k1, w));
                        const uint4 &q = w < 2 ? qa : qb;
                        const uint32_t b0 = w & 1 ? q.z : q.x, b1 = w & 1 ? q.w : q.y;
                        if (w == 0)
                            mma_f16_zero(acc[ab], a0, a1, a2, a3, b0, b1);
                        else
                            mma_f16(acc[ab], a0, a1, a2, a3, b0, b1);
                    }
                }
                const uint4 sc = lds128(q_frag + 8 * 512);
                const float ek = q8_scale(now.k_scale);
                const float f0 = __uint_as_float(sc.x) * ek, f1 = __uint_as_float(sc.y) * ek;
                x[0] = ((acc[0][0] + acc[1][0]) + (acc[2][0] + acc[3][0])) * f0;
                x[1] = ((acc[0][1] + acc[1][1]) + (acc[2][1] + acc[3][1])) * f1;
                x[2] = ((acc[0][2] + acc[1][2]) + (acc[2][2] + acc[3][2])) * f0;
                x[3] = ((acc[0][3] + acc[1][3]) + (acc[2][3] + acc[3][3])) * f1;
                if (now.rows < kTile) {  // what lies behind the valid rows may be anything
                    if (r >= now.rows) x[0] = x[1] = -CUDART_INF_F;
                    if (r + 8 >= now.rows) x[2] = x[3] = -CUDART_INF_F;
                }
            }
            const float ev = now.v_scale == 255 ? CUDART_NAN_F : (float)((int)now.v_scale - 127);

            // ---- references, moved when a score passes one by more than kLag
            float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
            if (__any_sync(0xffffffffu, mx0 > m0 + kLag || mx1 > m1 + kLag || mx0 + ev > v_ref0 + kLag ||
                                            mx1 + ev > v_ref1 + kLag)) {
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
                }
                auto moved = [](float &ref, float to) {  // what sums relative to it are multiplied by
                    const float n = fmaxf(ref, to), f = n == ref ? 1.f : ex2_approx(ref - n);
                    ref = n;
                    return f;
                };
                l0 *= moved(m0, mx0);
                l1 *= moved(m1, mx1);
                const float g0 = moved(v_ref0, mx0 + ev), g1 = moved(v_ref1, mx1 + ev);
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            o[a][w][k][0] *= g0;
                            o[a][w][k][1] *= g1;
                            o[a][w][k][2] *= g0;
                            o[a][w][k][3] *= g1;
                        }
            }
            // (a reference is -inf while there has been no score above it: all of them NaN or -inf)
            const float mu0 = m0 == -CUDART_INF_F ? 0.f : m0, mu1 = m1 == -CUDART_INF_F ? 0.f : m1;
            const float ve0 = (v_ref0 == -CUDART_INF_F ? 0.f : v_ref0) - kTop;
            const float ve1 = (v_ref1 == -CUDART_INF_F ? 0.f : v_ref1) - kTop;
            l0 += ex2_approx(x[0] - mu0) + ex2_approx(x[2] - mu0);
            l1 += ex2_approx(x[1] - mu1) + ex2_approx(x[3] - mu1);
            const float e0 = ev - ve0, e1 = ev - ve1;
            const uint32_t b0 = movmatrix_t(pack_f16x2(ex2_approx(x[0] + e0), ex2_approx(x[1] + e1)));
            const uint32_t b1 = movmatrix_t(pack_f16x2(ex2_approx(x[2] + e0), ex2_approx(x[3] + e1)));

            // ---- O^T += V^T W^T: two tokens' codes of a dim a register
            const uint32_t va = base + kTileCodes + 2 * c * 128 + ((r ^ (2 * c)) << 4);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const uint32_t v_at = va + a * 2048, v_at1 = (v_at ^ 16) + 128;
                uint4 t0v = lds128(v_at), t1v = lds128(v_at1);                // tokens 2c, 2c + 1
                uint4 t8v = lds128(v_at + 1024), t9v = lds128(v_at1 + 1024);  // tokens 2c + 8, 2c + 9
                if (now.rows < kTile) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    if (2 * c >= now.rows) t0v = zero;
                    if (2 * c + 1 >= now.rows) t1v = zero;
                    if (2 * c + 8 >= now.rows) t8v = zero;
                    if (2 * c + 9 >= now.rows) t9v = zero;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t sel = k ? 0x7362 : 0x5140;
                        const uint32_t lo = __byte_perm(word(t0v, w), word(t1v, w), sel);
                        const uint32_t hi = __byte_perm(word(t8v, w), word(t9v, w), sel);
                        mma_f16(o[a][w][k], f16x2_of_e4m3(lo), f16x2_of_e4m3_hi(lo), f16x2_of_e4m3(hi),
                                f16x2_of_e4m3_hi(hi), b0, b1);
                    }
            }
            __syncwarp();  // the slot is free
        }
        it += n;
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
            l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
        }

        // ---- the next segment's q, before this one's merge
        const int64_t pair = (int64_t)st.seq * p.num_kv_heads + st.g, part = blockIdx.x + pair;
        const bool whole = t0 == 0 && t1 == st.tiles;
        if (!kCluster && threadIdx.x == 0 && t0 == 0) {
            int parts = st.ctas_a_pair;
            if (parts == 0) parts = (int)(st.shares.owner(st.at - st.v0 + st.lead + st.tiles - 1) - blockIdx.x) + 1;
            p.info[pair] = make_int2((int)part, whole ? 0 : parts);
        }
        uint16_t *out_rows = p.out + ((int64_t)st.seq * p.num_q_heads + st.g * p.group) * kHeadDim;
        st.at += st.lead + t1 - st.v0;
        const bool more = !kCluster && st.end > st.at + st.lead;  // (a share that ends before the next pair's first tile is done)
        const uint32_t spare = (it + kDepth - 1) % kDepth;  // the slot of the last tile: the others hold the next ones
        if (more) {
            st.v0 = 0;
            next_pair(st.seq, st.g, st.seq_len, st.tiles);
            begin_segment();
            load_q();
        }

        // ------------------------------------------------------------ merge of the warps
        // A warp's sums, relative to m, as rows of 64 units of 16 bytes, unit u of head h at place
        // u ^ (h / 2).
        float2 *red_ml = reinterpret_cast<float2 *>(smem + kOffMl);  // [warp][head]
        if (lane < 4) {
            red_ml[warp * kDecMaxGroup + 2 * c] = make_float2(m0, l0);
            red_ml[warp * kDecMaxGroup + 2 * c + 1] = make_float2(m1, l1);
        }
        if (lane == 0) sum_slot[warp] = (int)(warp * kDepth + spare);
        {
            float4 *rows = reinterpret_cast<float4 *>(ring + spare * kSlotBytes) + 2 * c * 64;
            // (without a score above -inf the sums are 0, or NaN)
            const float u0 = m0 == -CUDART_INF_F ? 0.f : ex2_approx(v_ref0 - kTop - m0);
            const float u1 = m1 == -CUDART_INF_F ? 0.f : ex2_approx(v_ref1 - kTop - m1);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int unit = (32 * a + 4 * r + w) ^ c;
                    const float(&x)[2][4] = o[a][w];
                    rows[unit] = make_float4(x[0][0] * u0, x[0][2] * u0, x[1][0] * u0, x[1][2] * u0);
                    rows[64 + unit] = make_float4(x[0][1] * u1, x[0][3] * u1, x[1][1] * u1, x[1][3] * u1);
                }
        }
        fence_proxy_async_smem();  // (the slot's next contents come by a bulk copy)
        __syncthreads();  // every warp's rows are there, and q is no longer read
        const bool gave_up = *abort != 0;  // a wait ran out: this and the CTA's remaining segments contribute nothing
        if (more) make_q();
        for (int qd = threadIdx.x; qd < p.group * (kHeadDim / 4); qd += kThreads) {
            const int h = qd / (kHeadDim / 4), u = qd - h * (kHeadDim / 4), d = u * 4;
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
                const float4 f = reinterpret_cast<const float4 *>(smem + sum_slot[v] * kSlotBytes)[h * 64 + (u ^ (h >> 1))];
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
            if constexpr (kCluster) {
                reinterpret_cast<float4 *>(smem + kOffPart)[qd] = O;
                if (d == 0) reinterpret_cast<float2 *>(smem + kOffPart + kSlotBytes)[h] = make_float2(M, L);
            } else if (whole) {
                const float inv = L > 0.f ? 1.f / L : 0.f;
                *reinterpret_cast<uint2 *>(out_rows + h * kHeadDim + d) =
                    make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (part * p.group + h) * kHeadDim + d) = O;
                if (d == 0) p.part_ml[part * p.group + h] = make_float2(M, L);
            }
        }

        if constexpr (kCluster) {
            cluster_sync();  // every CTA's part is there
            const int units = p.group * (kHeadDim / 4);
            for (int u = threadIdx.x * p.cluster + rank; u < units; u += kThreads * p.cluster) {
                const int h = u / (kHeadDim / 4);
                const uint32_t at_o = smem_u32(smem + kOffPart) + u * 16, at_ml = smem_u32(smem + kOffPart + kSlotBytes) + h * 8;
                float4 f[kMaxCluster];
                float2 ml[kMaxCluster];
#pragma unroll
                for (int v = 0; v < kMaxCluster; ++v) {
                    ml[v] = make_float2(-CUDART_INF_F, 0.f);
                    f[v] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (v < p.cluster) {
                        ml[v] = ld_cluster_f2(at_ml, v);
                        f[v] = ld_cluster_f4(at_o, v);
                    }
                }
                float M = -CUDART_INF_F, L = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int v = 0; v < kMaxCluster; ++v) M = fmaxf(M, ml[v].x);
#pragma unroll
                for (int v = 0; v < kMaxCluster; ++v) {
                    const float e = ml[v].x == -CUDART_INF_F ? 0.f : ex2_approx(ml[v].x - M);
                    L = fmaf(e, ml[v].y, L);
                    O.x = fmaf(e, f[v].x, O.x);
                    O.y = fmaf(e, f[v].y, O.y);
                    O.z = fmaf(e, f[v].z, O.z);
                    O.w = fmaf(e, f[v].w, O.w);
                }
                const float inv = L > 0.f ? 1.f / L : 0.f;
                *reinterpret_cast<uint2 *>(out_rows + u * 4) =
                    make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
            }
            cluster_sync();  // every part has been read
            break;
        }
        if (!more) break;
        __syncthreads();  // q is ready, and the merge's rows are free
    }
    // Every load lands before the CTA's memory is left (when a wait gave up).
    for (uint32_t i = in.count - min(in.count, (uint32_t)kDepth); i < in.count; ++i)
        mbar_wait(&full[i % kDepth], (i / kDepth) & 1, p.err);
}

}  // namespace

size_t decode_q8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int num_sms) {
    const WsLayout l = ws_layout(num_seqs, num_q_heads, num_kv_heads, num_sms);
    return l.o + l.ml + l.info;
}

#ifdef PA_TEST_HOOKS
cudaError_t set_decode_q8_test_hook(int skip_tile) {
    return cudaMemcpyToSymbol(g_test_skip_tile, &skip_tile, sizeof skip_tile);
}
#endif

// CTAs of a pair's cluster, if the longest allowed sequence is short enough for that; else 0.
static int cluster_of(const SplitParams &p, const DecodeQ8Args &a) {
    const int64_t tiles = (int64_t)(a.max_seq_len / a.block_size) * p.tiles_per_page +
                          (a.max_seq_len % a.block_size + kTile - 1) / kTile;
    const int64_t pairs = (int64_t)a.num_seqs * a.num_kv_heads;
    const int steps = a.num_seqs == 1 ? kClusterSteps : kClusterStepsMany;
    int n = 1;
    while (n < kMaxCluster && tiles > n * kW && pairs * (2 * n) <= 2 * a.num_sms) n *= 2;
    return pairs * n <= 2 * a.num_sms && tiles <= (int64_t)n * kW * steps ? n : 0;
}

cudaError_t launch_decode_q8(const CUtensorMap *tmaps, const DecodeQ8Args &a, cudaStream_t stream) {
    Params p;
    fill_split(p, a);
    p.k_scales = a.k_scales;
    p.v_scales = a.v_scales;
    p.scale_stride = a.scale_stride;
    p.cluster = cluster_of(p, a);
    const void *kernel = reinterpret_cast<const void *>(
        p.cluster ? decode_q8_stream_kernel<true> : decode_q8_stream_kernel<false>);
    cudaError_t e = set_smem_once(kernel, p.cluster ? kSmemCluster : kSmem, p.cluster ? 12 : 9);
    if (e != cudaSuccess) return e;
    if (a.ev_start && (e = record_event(a.ev_start, stream)) != cudaSuccess) return e;
    if (p.cluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(a.num_seqs * a.num_kv_heads * p.cluster));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemCluster;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = p.cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, decode_q8_stream_kernel<true>, tmaps[0], tmaps[1], p);
    } else {
        p.cluster = 1;
        p.ctas = split_grid<kMinShare, true>(p, a);
        e = launch_pdl(decode_q8_stream_kernel<false>, dim3(p.ctas), dim3(kThreads), kSmem, stream, tmaps[0],
                       tmaps[1], p);
    }
    if (e != cudaSuccess) return e;
    if (a.ev_stop && (e = record_event(a.ev_stop, stream)) != cudaSuccess) return e;
    return kernel == reinterpret_cast<const void *>(decode_q8_stream_kernel<true>)
               ? cudaSuccess
               : launch_merge<10, kMinShare>(p, a.num_sms, stream);
}

}  // namespace pa
