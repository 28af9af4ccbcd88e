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
// Instructions come close to bounding it too (issue slots 60% used), so the weights are multiplied into the
// angles once per token and kind of row,
//     out_j = inv (x_j A_j + x_p B_j),   A_j = w_j cos, B_j = +- w_p sin   (p: j's partner),
// from weights that a CTA keeps in shared memory as it needs them; the partners are exchanged as packed
// BF16, before any arithmetic, and the arithmetic is on pairs.
// 4096 tokens of 24 + 4 + 4 heads of 256, into a BF16 cache: 22.2 us, 6.0 TB/s.  With the weights made
// ready at each token 25.5; besides, with a warp's next rows in registers instead of shared memory, which
// are on their way for a shorter time, 28.1, with the rows summed one by one 29, and with the weights
// applied to every row 43.  Into a 4-bit cache 29.5 us, without a cache 20.0.  32 + 8 + 8 heads 35.4 us, 12 + 2
// + 2 16.2 (5.7 and 4.1 TB/s), 64 + 8 + 8 of 128 35.0 (4.8 TB/s).  16 tokens 2.2 us.  20 warps an SM instead of
// 16 (when that took 22.8 and 34.1): 23.1 us, and 64 + 8 + 8 heads of 128 33.3, but 512 tokens 5.0 instead of
// 4.5.  Copying rows ahead pays where a CTA has several tokens of several rows: calls of 200 to 1500 tokens
// with one or two rows a warp and token lose 0.1 to 0.3 us to it (400 tokens of 32 + 8 + 8 heads of 128 3.9 and
// 4.2 us).
//
// Positions on several axes (time, height, width of a token): frequency i takes its angle from the
// position on the axis that the caller gives it.  Only the fetch of the angles differs: fours of
// frequencies, each on one axis, come as 16-byte copies, as with one position, others one by one: 4096
// tokens 22.9 and 24.6 us (by one kernel that chose for each token a microsecond more).
#include <algorithm>
#include <type_traits>

#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 6;  // query rows of a warp at most, copied a token ahead (24 heads over 4 warps)

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

// The axes of the frequencies of a token's i-th four of angles (cosines before sines), two bits each.
__host__ __device__ __forceinline__ uint32_t axes_of_four(const RopeArgs &a, int i) {
    const int half = a.rotary_dim / 2, freq = 4 * i < half ? 4 * i : 4 * i - half;
    return a.axes[freq / 16] >> (2 * (freq % 16)) & 0xffu;
}
// Whether each four of frequencies is on one axis.
bool axes_by_fours(const RopeArgs &a) {
    bool same = true;
    for (int i = 0; i < a.rotary_dim / 8; ++i)
        same = same && axes_of_four(a, i) == (axes_of_four(a, i) & 3) * 0x55u;
    return same;
}

// kCache: 0 none, 1 BF16, 2 4-bit.  kAxes: 0 one position, 1 several, and each four of
// frequencies on one axis, 2 several.
template <int kD, bool kNeighbours, int kCache, int kAxes>
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
    // A CTA takes every gridDim.x-th token, and copies ahead into shared memory: a token's first rows of
    // each kind (a lane its own 16 bytes, which no other reads) and its angles (this lane's or, with
    // axes, this warp's) while the token before is worked on, its position a token earlier still.  (A
    // padding token's rows are read for nothing.)
    constexpr int kN = kNeighbours ? 1 : 2;  // fours of frequencies of a lane
    __shared__ float4 angles[kWarps][2][kD / 4];
    constexpr int kK = kBatch, kV = kBatch + (kCache ? 1 : 0);  // places of the first key and value row
    __shared__ uint4 staged[kWarps][2][kV + 1][32];
    uint4 (*rows)[kV + 1][32] = staged[threadIdx.x >> 5];
    int64_t slot_next;
    const uint16_t *q_at, *k_at, *v_at;  // of the token that is loaded
    auto at = [&](int64_t t) {
        q_at = a.q + t * a.q_stride;
        k_at = a.k + t * a.k_stride;
        if (kCache) v_at = a.v + t * a.v_stride;
    };
    // (A row that there is not is zeros, or not looked at.)
    auto stage = [&](uint4 *to, const uint16_t *p, int r, int n) {
        if (r - sub >= n) return;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to + lane)),
                     "l"(r < n ? p + r * kD + 8 * l : p), "r"(r < n ? 16 : 0)
                     : "memory");
    };
    auto stage_rows = [&](uint4 (*to)[32]) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) stage(to[b], q_at, unit + b * step, hq);
        stage(to[kK], k_at, unit_k, hkv);
        if (kCache) stage(to[kV], v_at, unit_v, hkv);
    };
    // The weights with their bias, those of a lane's dims and of their partners (these with the sign of
    // the sine that they meet), of query and key rows.
    __shared__ float4 weights[2][4][32];
    auto keep_weights = [&](const uint4 &own, const uint4 &other, float4 (*to)[32]) {
        const uint32_t x[4] = {own.x, own.y, own.z, own.w}, y[4] = {other.x, other.y, other.z, other.w};
        float wo[8], wp[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wo[2 * i] = bf16_lo(x[i]) + a.weight_bias;
            wo[2 * i + 1] = bf16_hi(x[i]) + a.weight_bias;
            const float lo = bf16_lo(y[i]) + a.weight_bias, hi = bf16_hi(y[i]) + a.weight_bias;
            wp[2 * i] = kNeighbours ? (turns ? -hi : hi) : second ? lo : -lo;
            wp[2 * i + 1] = kNeighbours ? lo : second ? hi : -hi;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            to[i][lane] = make_float4(wo[4 * i], wo[4 * i + 1], wo[4 * i + 2], wo[4 * i + 3]);
            to[2 + i][lane] = make_float4(wp[4 * i], wp[4 * i + 1], wp[4 * i + 2], wp[4 * i + 3]);
        }
    };
    // With one position, each lane brings its own angles: 2 kN fours of frequencies, cosines before
    // sines (lanes of the same angles bring them to one place, each for itself).  With axes, a warp
    // brings the R / 4 fours of the token, lane i fours i and i + 32: a four of several axes takes four
    // copies, and lanes that share angles need not make them again.  Pairs of halves take two fours a
    // lane, 2i and 2i + 1: the even fours lie before the odd ones, so that lanes read neighbouring ones.
    // (Before the rows were copied ahead, 4096 tokens: with axes 31.6 us when each lane brought its own,
    // 30.3 so; 1000 tokens of 32 + 8 + 8 heads of 128 with axes in turn 9.8 and 6.9; with one position
    // 28.3 and 29.4.)
    constexpr int kFours = (kD / 4 + 31) / 32, kOwn = kNeighbours ? kLanes : kLanes / 2;
    const int own = !kNeighbours && second ? l - R / 16 : l;  // the lane's place (where it turns)
    auto place = [&](int four) { return kNeighbours ? four : (four & 1) * (R / 8) + (four >> 1); };
    uint32_t axes[kFours] = {};  // of each four, two bits each
    if constexpr (kAxes > 0) {
#pragma unroll
        for (int i = 0; i < kFours; ++i)
            if (lane + 32 * i < R / 4) axes[i] = axes_of_four(a, lane + 32 * i);
    }
    // The position on axis lane % 4 (on axis 0 where there are fewer): each axis' on lanes 0 .. 3.
    const int own_axis = kAxes && (lane & 3) < a.num_axes ? lane & 3 : 0;
    const int32_t *positions = a.positions + (kAxes ? own_axis * a.position_stride : 0);
    auto position = [&](int64_t t) { return t < a.num_tokens ? positions[t] : -1; };
    // Whether a token is padding, and whether it lies in the table.
    auto placed = [&](int pos) { return kAxes ? !__any_sync(0xffffffffu, pos < 0) : pos >= 0; };
    auto inside = [&](int pos) {
        return kAxes ? __all_sync(0xffffffffu, pos < a.max_position) : pos < a.max_position;
    };
    auto copy16 = [&](float4 *dst, const float *src) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    };
    auto angles_of = [&](int64_t t, int pos, int buf) {
        slot_next = kCache ? a.slot_mapping[t] : -1;
        float4 *to = angles[threadIdx.x >> 5][buf];
        if constexpr (kAxes == 0) {
            if (turns && placed(pos) && inside(pos)) {
                const float *row = a.cos_sin + (int64_t)pos * R +
                                   (kNeighbours ? 4 * l : second ? 8 * l - half : 8 * l);
#pragma unroll
                for (int e = 0; e < 2 * kN; ++e) copy16(to + e * kOwn + own, row + (e / kN) * half + (e % kN) * 4);
            }
        } else if (placed(pos) && inside(pos)) {
#pragma unroll
            for (int i = 0; i < kFours; ++i) {
                const int four = lane + 32 * i;
                const float *column = a.cos_sin + 4 * four;
                if constexpr (kAxes == 1) {
                    const int row = __shfl_sync(0xffffffffu, pos, axes[i] & 3);
                    if (four < R / 4) copy16(to + place(four), column + (int64_t)row * R);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = __shfl_sync(0xffffffffu, pos, axes[i] >> (2 * j) & 3);
                        if (four < R / 4)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to + place(four)) + 4 * j),
                                         "l"(column + (int64_t)row * R + j)
                                         : "memory");
                    }
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int64_t stride = gridDim.x;
    int pos = position(blockIdx.x), pos_next = position(blockIdx.x + stride), buf = 0;
    at(blockIdx.x);
    stage_rows(rows[0]);
    uint4 w_own, w_other;  // (the first two warps': on their way before the position is waited for)
    if (threadIdx.x < 64) {
        const uint4 *w = reinterpret_cast<const uint4 *>(threadIdx.x < 32 ? a.q_weight : a.k_weight);
        w_own = w[l];
        w_other = w[partner];
    }
    angles_of(blockIdx.x, pos, 0);
    if (threadIdx.x < 64) keep_weights(w_own, w_other, weights[threadIdx.x >> 5]);
    __syncthreads();
    for (int64_t t = blockIdx.x; t < a.num_tokens; t += stride, buf ^= 1) {
    const int pos_now = pos;
    const int64_t slot = slot_next;
    const bool more = t + stride < a.num_tokens;
    pos = pos_next;
    __syncwarp();  // the angles of the token before are read
    if (more) {
        at(t + stride);
        stage_rows(rows[buf ^ 1]);
        angles_of(t + stride, pos, buf ^ 1);
        pos_next = position(t + 2 * stride);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if constexpr (kAxes) __syncwarp();  // every lane's angles are there
    // (a token that is not live: its rows stay as they are)
    const bool some = placed(pos_now), in = inside(pos_now), live = some && in;
    if (some && !in && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrPosition);
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
    auto factors = [&](const float4 (*w)[32]) {
        float4 c[2], sn[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            c[e] = make_float4(1.f, 1.f, 1.f, 1.f);
            sn[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (turns) {
            const float4 *mine = angles[threadIdx.x >> 5][buf] + own;
            if (kNeighbours) {
                const float4 cv = mine[0], sv = mine[kAxes ? R / 8 : kOwn];
                c[0] = make_float4(cv.x, cv.x, cv.y, cv.y);
                c[1] = make_float4(cv.z, cv.z, cv.w, cv.w);
                sn[0] = make_float4(sv.x, sv.x, sv.y, sv.y);
                sn[1] = make_float4(sv.z, sv.z, sv.w, sv.w);
            } else {
                const int next = kAxes ? R / 8 : kOwn, sines = kAxes ? R / 16 : 2 * kOwn;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    c[e] = mine[e * next];
                    sn[e] = mine[sines + e * next];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 wo = w[e][lane], wp = w[2 + e][lane];
            A[2 * e] = mul(pair(wo.x, wo.y), pair(c[e].x, c[e].y));
            A[2 * e + 1] = mul(pair(wo.z, wo.w), pair(c[e].z, c[e].w));
            B[2 * e] = mul(pair(wp.x, wp.y), pair(sn[e].x, sn[e].y));
            B[2 * e + 1] = mul(pair(wp.z, wp.w), pair(sn[e].z, sn[e].w));
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
    factors(weights[0]);
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
            v[b] = b <= kK ? squares(rows[buf][b][lane]) : 0.f;
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
        asm volatile("" ::: "memory");  // (else the compiler brings all rounds' rows ahead of the first test)
        const uint4 row = rows[buf][b][lane], out = turned(row, joint ? inv[b] : inverse_of(row));
        if (live && r < hq) *reinterpret_cast<uint4 *>(q_out + r * kD) = out;
    }
    auto key_row = [&](int r, const uint4 &row, float root) {
        const uint4 out = turned(row, root);
        if (live && r < hkv) {
            if (kCache == 0)
                *reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride + r * kD + 8 * l) = out;
            else
                to_cache(a.k_cache, r, out);
        }
    };
    if (unit_k - sub < hkv) {
        factors(weights[1]);
        const uint4 first = rows[buf][kK][lane];
        key_row(unit_k, first, joint ? inv[kK] : inverse_of(first));
        for (int r = unit_k + step; r - sub < hkv; r += step) {  // many heads
            const uint4 row = row_of(a.k + t * a.k_stride, r, hkv);
            key_row(r, row, inverse_of(row));
        }
    }
    if (kCache)
        for (int r = unit_v; r < hkv; r += step)
            to_cache(a.v_cache, r, r == unit_v ? rows[buf][kV][lane] : row_of(a.v + t * a.v_stride, r, hkv));
    }
}

template <int kD>
cudaError_t launch_dim(RopeArgs a, cudaStream_t stream) {
    constexpr int per = kWarps * (256 / kD);
    // A small call: a row a warp, as many CTAs a token as that takes.  A large one: a token over as
    // few CTAs as give each warp kBatch query rows, and four CTAs an SM that go from token to token.
    // Small is what is resident at once, with the rows of a call that writes the cache (so that the
    // calls with and without a cache sum a row in the same order).  24 + 4 + 4 heads of 256, 8 CTAs a
    // token and one: 16 tokens 2.2 and 2.8 us, 64 2.8 and 2.9, 100 4.0 and 2.9, 200 5.6 and 3.4; 32 + 8 + 8 of
    // 128, 6 CTAs and one: 16 tokens 2.1 and 2.8, 64 2.8 and 2.9, 150 4.1 and 2.9.
    const int y_small = (a.num_q_heads + 2 * a.num_kv_heads + per - 1) / per;
    const bool small = (int64_t)a.num_tokens * y_small <= 4 * a.num_sms;
    const int y = small ? y_small : (a.num_q_heads + per * kBatch - 1) / (per * kBatch);
    constexpr int one = 256 / kD;  // rows of a warp
    const int step = y * per;  // (kBatch rounds of it take all query heads, either way)
    a.shift_k = (a.num_q_heads + one - 1) / one * one % step;
    a.shift_v = (a.shift_k + (a.num_kv_heads + one - 1) / one * one) % step;
    const int x = small ? a.num_tokens : std::min(a.num_tokens, std::max(1, 4 * a.num_sms / y));
    const dim3 grid(x, y), block(kWarps * 32);
    auto launch = [&](auto neighbours, auto axes) {
        constexpr bool kN = decltype(neighbours)::value;
        constexpr int kA = decltype(axes)::value;
        if (a.cache == 0) return launch_pdl(qk_norm_rope_kernel<kD, kN, 0, kA>, grid, block, 0, stream, a);
        if (a.cache == 1) return launch_pdl(qk_norm_rope_kernel<kD, kN, 1, kA>, grid, block, 0, stream, a);
        if constexpr (kD == kHeadDim)
            return launch_pdl(qk_norm_rope_kernel<kD, kN, 2, kA>, grid, block, 0, stream, a);
        return cudaErrorInvalidValue;
    };
    auto launch_axes = [&](auto axes) {
        return a.interleaved ? launch(std::true_type(), axes) : launch(std::false_type(), axes);
    };
    if (a.num_axes == 0) return launch_axes(std::integral_constant<int, 0>());
    return axes_by_fours(a) ? launch_axes(std::integral_constant<int, 1>())
                            : launch_axes(std::integral_constant<int, 2>());
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
