// gdla_decode_paged.cu - GDLA decode over a paged KV cache in bf16 or e4m3, for sm_100a.
//
// One query token per sequence (position L_b - 1, the cache holding it) over the pages
// that the sequence's row of the block table names: all its keys, or a sliding window
// and, outside it, the first `sinks` keys. Per (sequence, KV head) the five query heads
// share one pass over the keys:
//     s = scale_K(page) * (q . k_code) / sqrt(192),  p = exp2(s log2(e) - m),
//     O = sum over pages of scale_V(page) * sum over the page's keys of p * v_code,
// with the running maximum m and sum l of a softmax, then D = H_S - lambda H_N and the
// sigmoid gate (aitrends.kr/articles/94908, GDLA paragraphs).
//
// HBM bounds it where there are keys enough: 320 B (e4m3) or 640 B (bf16) per key and KV head against 3,200
// flops, 10 per byte. Measured on one B200, alone or in a graph and, in brackets, as called: 64 sequences of 1,024 to
// 32,768 e4m3 tokens, 16 heads: 862 us, 6.8 TB/s (913 to 1,000 at the card's power cap; a copy runs at 6.5 TB/s, reads
// alone somewhat faster). Short or few sequences are bound by the chain of a warp's start (length, page, first rows:
// 2 us), blocks (1.0 to 1.4 us each, their loads under way meanwhile) and join (1 us in the CTA, 1.5 over a cluster):
// one sequence of 4,096 bf16 tokens 14.5 us (16.3), 64 with window 128 and 4 sinks 22.4 us (24.4); floors 6.5 and 14.0,
// and a fifth of the latter's traffic is rows of the copied blocks that nobody sees.
//
// Keys come in blocks of 16 that never straddle a page (pages are multiples of 16), so
// a block has one scale for K and one for V. The products are mma.sync m16n8k16 with the
// keys (S^T = K Q^T) and the value dims (O^T = V^T P^T) as rows and the five heads in the
// eight columns. e4m3 codes become f16 (exact) and meet f16 queries divided by a power of
// two per head (exact but for elements 2^-14 under the head's largest) and f16
// probabilities; O is held in fp32, in units of a page's V scale.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdla_internal.h"
#include "gdla_paged.cuh"
#include "gdla_pair.cuh"
#include "gdla_ptx.cuh"

namespace gdla {

namespace dp {
constexpr int DQK = 192, DV = 128, HEADS = 5;
constexpr int BLOCK = 16;       // keys per block
constexpr int MAX_CLUSTER = 8;  // CTAs that join one (sequence, KV head) over distributed shared memory
// A warp's O leaves its registers as [head][place], place 16 mt + 2 g8 + e for row g8 + 8 e of tile mt (rows of 132: the
// sixteen lanes of a 64-bit store then take different banks). Sums keep that order; dim_of undoes it at the output.
constexpr int RED_ROW = DV + 4;
template <bool E4M3>
__device__ __forceinline__ int dim_of(int place) {
    const int mt = place >> 4, g8 = (place >> 1) & 7, e = place & 1;
    return E4M3 ? 16 * g8 + 2 * mt + e : 16 * mt + g8 + 8 * e;
}
constexpr float kTrail = 4.f;  // a probability is at most 2^4: with the largest ratio and the bias 2^15, which f16 holds
constexpr float kScoreLog2 = 0.07216878364870322f * 1.4426950408889634f;  // log2(e) / sqrt(192)

// Warps per CTA: 4, or 8 for few items, or 2 for many of few keys each (then a warp's own start and end weigh more
// than its blocks). 14 to 16 warps per SM.
template <bool E4M3, int WARPS_>
struct Cfg {
    static constexpr int WARPS = WARPS_, THREADS = 32 * WARPS, CTAS_PER_SM = WARPS == 2 ? 7 : 16 / WARPS;
    static constexpr int ELT = E4M3 ? 1 : 2;
    static constexpr int K_BYTES = BLOCK * DQK * ELT, V_BYTES = BLOCK * DV * ELT;
    static constexpr int STAGE = K_BYTES + V_BYTES;  // 5 or 10 KB
    static constexpr int STAGES = E4M3 ? 2 : 1;  // blocks ahead: 10 KB in flight per warp either way
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int RED = WARPS * HEADS * RED_ROW * 4;  // fp32 [WARPS][5][132], over the ring once it is done
    static constexpr int OFF_CTA = RING > RED ? RING : RED;        // fp32 [5][128]: this CTA's sums
    static constexpr int OFF_ML = OFF_CTA + HEADS * DV * 4;        // fp32 [WARPS][8][2], then [5][2] of the CTA
    static constexpr int OFF_AUX = OFF_ML + (WARPS + 1) * 64;      // float4 per stage: position, page, scales
    static constexpr int SMEM_BYTES = OFF_AUX + WARPS * STAGES * 16;
    static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 233472 && SMEM_BYTES <= 232448, "shared memory per SM");
};

// Shared-memory places of a block's rows: 16-byte units, permuted so that the eight lanes of a
// quarter warp read eight different bank groups.
//   K bf16 (24 units a row): units 0-3 and 4-7, 8-11 and 12-15, .. swapped in odd rows
//   K e4m3 (12 units): as it is, the 192-byte rows already alternate
//   V bf16 (16 units): by the row, for eight-row transposing matrix loads
//   V e4m3 (8 units): by the row pair (row / 2) % 4, which is the reading lane's c
template <bool E4M3>
__device__ __forceinline__ uint32_t k_place(int row, int unit) {
    return E4M3 ? row * 192 + unit * 16 : row * 384 + ((unit ^ ((row & 1) << 2)) << 4);
}
template <bool E4M3>
__device__ __forceinline__ uint32_t v_place(int row, int unit) {
    return E4M3 ? row * 128 + ((unit ^ (row & 6)) << 4) : row * 256 + ((unit ^ (row & 7)) << 4);
}
}  // namespace dp

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// fp32 at the address that `addr` of this CTA's shared memory has in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}

// The dims of a step's K slots. An MMA may take the 192 dims in any order as long as keys
// and queries agree, so every lane reads its share of a key row in whole 16-byte units
// straight from the page's own layout, without a swizzle: lane c = lane % 4 holds
//   bf16: units c + 4 j (j < 6), dims 32 j + 8 c + 0..7, for steps 2 j and 2 j + 1;
//   e4m3: units c and c + 4, dims 64 j + 16 c + 0..15, for steps 4 j .. 4 j + 3, and the 8-byte
//         units at 128 + 8 c (steps 8, 9) and 160 + 8 c (steps 10, 11).
// Dims i and i + 32 of the rotary part are then in one lane, two steps apart. step_dim is the
// first of the four dims that lane c holds in a step (slots 2c, 2c+1, then 2c+8, 2c+9).
template <bool E4M3>
__device__ __forceinline__ constexpr int step_dim(int ks, int c) {
    if (!E4M3) return 32 * (ks >> 1) + 8 * c + 4 * (ks & 1);
    return ks < 8 ? 64 * (ks >> 2) + 16 * c + 4 * (ks & 3) : 128 + 32 * ((ks - 8) >> 1) + 8 * c + 4 * (ks & 1);
}

// This lane's queries, raw: head lane / 4 (zero from 5 on), step ks at x[ks].
template <bool E4M3>
__device__ __forceinline__ void load_queries(uint2 (&raw)[12], const __nv_bfloat16 *q_sig, const __nv_bfloat16 *q_noise,
                                             size_t bg, int lane) {
    using namespace dp;
    const int g8 = lane >> 2, c = lane & 3;
    const __nv_bfloat16 *row = g8 < 4 ? q_sig + (bg * 4 + g8) * DQK : q_noise + bg * DQK;
#pragma unroll
    for (int ks = 0; ks < 12; ++ks)
        raw[ks] = g8 < HEADS ? __ldg(reinterpret_cast<const uint2 *>(row + step_dim<E4M3>(ks, c))) : make_uint2(0u, 0u);
}
// As fragments, turned to the query's position where asked. bf16 keys need bf16 queries: a
// turned rotary part is no longer exact in bf16, so its remainder goes along as a second
// fragment (qlo) and the scores keep fp32's accuracy. e4m3 keys meet f16 queries, divided
// by a power of two per head. Returns the factor of this head's scores.
template <bool E4M3>
__device__ __forceinline__ float query_fragments(const uint2 (&raw)[12], uint32_t (&qf)[12][2], uint32_t (&qlo)[4][2],
                                                 int lane, bool rotate, int pos) {
    using namespace dp;
    const int c = lane & 3;
    float x[12][4];
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) {
        x[ks][0] = __uint_as_float(raw[ks].x << 16);
        x[ks][1] = __uint_as_float(raw[ks].x & 0xFFFF0000u);
        x[ks][2] = __uint_as_float(raw[ks].y << 16);
        x[ks][3] = __uint_as_float(raw[ks].y & 0xFFFF0000u);
    }
    if (rotate) {
        float cs, sn;  // pair `lane`; the lanes share them
        rotary_angle(pos, lane, cs, sn);
#pragma unroll
        for (int ks = 8; ks < 10; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = step_dim<E4M3>(ks, c) - 128 + e;
                const float ci = __shfl_sync(0xffffffffu, cs, i), si = __shfl_sync(0xffffffffu, sn, i);
                const float a = x[ks][e], b = x[ks + 2][e];
                x[ks][e] = a * ci - b * si;
                x[ks + 2][e] = a * si + b * ci;
            }
    }
    float factor = kScoreLog2;
    if constexpr (E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int ks = 0; ks < 12; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(x[ks][e]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        e = amax > 0.f ? max(-100, min(100, e)) : 0;
        const float inv = power_of_two(-e);
        factor *= power_of_two(e);
#pragma unroll
        for (int ks = 0; ks < 12; ++ks)
#pragma unroll
            for (int s = 0; s < 2; ++s) qf[ks][s] = pack_f16x2(x[ks][2 * s] * inv, x[ks][2 * s + 1] * inv);
    } else {
#pragma unroll
        for (int ks = 0; ks < 12; ++ks)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                qf[ks][s] = pack_bf16x2(x[ks][2 * s], x[ks][2 * s + 1]);
                if (ks >= 8)
                    qlo[ks - 8][s] = pack_bf16x2(x[ks][2 * s] - __uint_as_float(qf[ks][s] << 16),
                                                 x[ks][2 * s + 1] - __uint_as_float(qf[ks][s] & 0xFFFF0000u));
            }
    }
    return factor;
}

// out = sigmoid(gate) (H_S - lambda H_N) of one value dim and signal head, in bf16.
__device__ __forceinline__ __nv_bfloat16 paged_output(float hs, float hn, float lam, __nv_bfloat16 gate) {
    return __float2bfloat16_rn(__fdividef(hs - lam * hn, 1.f + __expf(-__bfloat162float(gate))));
}
// H = O / l; no key at all: zero; a NaN goes through.
__device__ __forceinline__ float paged_head(float O, float l) { return l == 0.f ? 0.f : O / l; }

// Work: (sequence, KV head) items, each cut into `splits` runs of its visible blocks, one CTA
// a run; `cluster` of an item's CTAs form a cluster. Inside a CTA warp w takes every WARPS-th
// block of the run through a ring of its own: the lanes copy the block's K rows and V rows
// (contiguous in the page) asynchronously, as two groups, STAGES blocks ahead, so a warp waits
// on its own copies alone and K of the next block is under way while V of this one is
// multiplied. The warps join in shared memory, the cluster's CTAs in distributed shared
// memory, where CTA r finishes a share of the value dims; where an item has several clusters
// their sums are left to the combine kernel.
template <bool E4M3, int WARPS>
__global__ void __launch_bounds__(dp::Cfg<E4M3, WARPS>::THREADS, dp::Cfg<E4M3, WARPS>::CTAS_PER_SM)
gdla_decode_paged_kernel(const __grid_constant__ PagedDecode p) {
    using namespace dp;
    using C = Cfg<E4M3, WARPS>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, c = lane & 3;
    const unsigned item = blockIdx.x / p.splits;
    const int split = blockIdx.x - item * p.splits;
    const int b = item / p.hkv, group = item - b * p.hkv;
    const size_t bg = item;

    const int len = __ldg(p.seqlens_k + b);
    uint2 q_raw[12];
    load_queries<E4M3>(q_raw, p.q_sig, p.q_noise, bg, lane);
    const VisibleBlocks vis = visible_blocks(len, p.max_seqlen_k, p.window, p.sinks);
    const int i0 = static_cast<int>(static_cast<long long>(vis.n) * split / p.splits);
    const int i1 = static_cast<int>(static_cast<long long>(vis.n) * (split + 1) / p.splits);
    const int mine = max(0, (i1 - i0 - warp + WARPS - 1) / WARPS);  // blocks of this warp
    const auto position = [&](int n) { return vis.block(i0 + warp + n * WARPS) * BLOCK; };

    // What a copy needs of block n of this warp, held by lane n % 32 for 32 blocks at a time and
    // read 32 blocks ahead: page and head as one number (-1: no such page) and the scales.
    const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const auto look_up = [&](int n0, int &at, float &ks, float &vs) {
        const int n = n0 + lane;
        at = -1;
        ks = vs = 1.f;
        if (n < mine) {
            const int id = __ldg(table + (position(n) >> p.page_shift));
            if (id >= 0 && id < p.num_pages) {
                at = id * p.hkv + group;
                if (E4M3) {
                    ks = __ldg(p.k_scale + at);
                    vs = __ldg(p.v_scale + at);
                }
            }
        }
    };
    int at_cur, at_next = -1;
    float ks_cur, vs_cur, ks_next = 1.f, vs_next = 1.f;
    look_up(0, at_cur, ks_cur, vs_cur);
    if (mine > 32) look_up(32, at_next, ks_next, vs_next);

    uint8_t *ring = smem + warp * STAGES * C::STAGE;
    const uint32_t ring_a = smem_u32(ring);
    float4 *aux = reinterpret_cast<float4 *>(smem + C::OFF_AUX) + warp * STAGES;
    // where this lane's 16-byte units of a K block go: unit 32 i + lane of the block (three units cover 4 bf16 rows)
    uint32_t k_dst[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) k_dst[i] = k_place<E4M3>((32 * i + lane) / (12 * C::ELT), (32 * i + lane) % (12 * C::ELT));
    const auto copy_k = [&](int n) {  // K of block n into its stage, one group (the whole warp calls)
        if (n < mine) {
            if (n > 0 && (n & 31) == 0) {
                at_cur = at_next, ks_cur = ks_next, vs_cur = vs_next;
                look_up(n + 32, at_next, ks_next, vs_next);
            }
            const int at = __shfl_sync(0xffffffffu, at_cur, n & 31);
            const int st = n % STAGES, pos0 = position(n);
            if (at >= 0) {
                const size_t row = (static_cast<size_t>(at) << p.page_shift) + (pos0 & (p.page_size - 1));
                const uint8_t *src = static_cast<const uint8_t *>(p.k_pages) + row * (DQK * C::ELT) + lane * 16;
                const uint32_t dst = ring_a + st * C::STAGE;
#pragma unroll
                for (int i = 0; i < C::K_BYTES / 512; ++i)
                    cp_async16(dst + (i / 3) * 1536 + k_dst[i % 3], src + 512 * i);
            }
        }
        cp_async_commit();
    };
    const auto copy_v = [&](int n) {  // V of block n, after copy_k(n)
        if (n < mine) {
            const int st = n % STAGES, pos0 = position(n);
            const int at = __shfl_sync(0xffffffffu, at_cur, n & 31);
            if (at >= 0) {
                const size_t row = (static_cast<size_t>(at) << p.page_shift) + (pos0 & (p.page_size - 1));
                const uint8_t *src = static_cast<const uint8_t *>(p.v_pages) + row * (DV * C::ELT) + lane * 16;
                const uint32_t dst = ring_a + st * C::STAGE + C::K_BYTES;
#pragma unroll
                for (int i = 0; i < C::V_BYTES / 512; ++i) {
                    const int unit = 32 * i + lane;
                    cp_async16(dst + v_place<E4M3>(unit / (8 * C::ELT), unit % (8 * C::ELT)), src + 512 * i);
                }
            }
            // the scales, whose loads the copies need not wait for
            const float ks = __shfl_sync(0xffffffffu, ks_cur, n & 31), vs = __shfl_sync(0xffffffffu, vs_cur, n & 31);
            if (lane == 0) aux[st] = make_float4(__int_as_float(pos0), __int_as_float(at), ks, vs);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int n = 0; n < STAGES; ++n) {
        copy_k(n);
        copy_v(n);
    }

    uint32_t qf[12][2], qlo[4][2];
    const float factor = query_fragments<E4M3>(q_raw, qf, qlo, lane, p.rotate, len - 1);
    // scores come out with heads 2c and 2c + 1 in this lane
    const float f0 = __shfl_sync(0xffffffffu, factor, (8 * c) & 31), f1 = __shfl_sync(0xffffffffu, factor, (8 * c + 4) & 31);

    float o[DV / 16][4];
#pragma unroll
    for (int mt = 0; mt < DV / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    // Running maxima of heads 2c, 2c+1 (log2 units) and their sums. The maxima may trail the true ones by
    // kTrail: then a block costs one vote, and no reduction over the keys and no rescaling.
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    // e4m3: O is held in units of 1 / kBias of some page's V scale, the first page's to begin with, and the probabilities
    // take kBias and the ratio of their own page's scale to that one, so that the products add straight onto O. Ratios
    // from 2^-4 to 2^2 leave an f16 probability its 11 bits down to 2^-19 of the running maximum, or further, and a step
    // of 2^-29 under that (p <= 2^kTrail, so 2^15 at most); a page further off changes the unit. Without the bias, and with
    // ratios from 2^-8 on, a key that took nearly all the weight left the others 2^-17 of it as step: up to a fifth
    // of the output where its own value was small. The unit goes down to 2^-75 of the largest one so far at most: O,
    // under 2^51 of those, stays finite, and a page whose scale is smaller yet (one of zeros has 2^-110) is lost beside
    // them. Held are 1 / unit (0: no page yet) and the least unit.
    constexpr float kBias = 512.f, kRatioMin = kBias / 16.f, kRatioMax = kBias * 4.f;
    constexpr float kUnitDrop = 2.6469779601696886e-23f;  // 2^-75
    float vs_inv = 0.f, vs_floor = 1e-35f;  // (kBias over a smaller unit would leave fp32)
    for (int n = 0; n < mine; ++n) {
        const int st = n % STAGES;
        const uint8_t *kb = ring + st * C::STAGE, *vb = kb + C::K_BYTES;
        cp_async_wait<2 * STAGES - 1>();  // this lane's share of K is there; behind the barrier everyone's
        __syncwarp();
        const float4 a = aux[st];
        const int pos0 = __float_as_int(a.x);
        const bool there = __float_as_int(a.y) >= 0;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products
        if (there) {
            if constexpr (E4M3) {
                const uint8_t *r0 = kb + g8 * DQK, *r1 = r0 + 8 * DQK;
                const auto step = [&](float (&d)[4], uint32_t x, uint32_t y, int ks) {
                    mma_f16(d, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y), e4m3x2_to_f16x2(x >> 16),
                            e4m3x2_to_f16x2(y >> 16), qf[ks][0], qf[ks][1]);
                };
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(r0 + 64 * j + 16 * c);
                    const uint4 y = *reinterpret_cast<const uint4 *>(r1 + 64 * j + 16 * c);
                    step(s, x.x, y.x, 4 * j);
                    step(t, x.y, y.y, 4 * j + 1);
                    step(s, x.z, y.z, 4 * j + 2);
                    step(t, x.w, y.w, 4 * j + 3);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(r0 + 128 + 32 * j + 8 * c);
                    const uint2 y = *reinterpret_cast<const uint2 *>(r1 + 128 + 32 * j + 8 * c);
                    step(s, x.x, y.x, 8 + 2 * j);
                    step(t, x.y, y.y, 9 + 2 * j);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 6; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kb + k_place<false>(g8, c + 4 * j));
                    const uint4 y = *reinterpret_cast<const uint4 *>(kb + k_place<false>(g8 + 8, c + 4 * j));
                    mma_bf16(s, x.x, y.x, x.y, y.y, qf[2 * j][0], qf[2 * j][1]);
                    mma_bf16(t, x.z, y.z, x.w, y.w, qf[2 * j + 1][0], qf[2 * j + 1][1]);
                    if (j >= 4 && p.rotate) {
                        mma_bf16(s, x.x, y.x, x.y, y.y, qlo[2 * j - 8][0], qlo[2 * j - 8][1]);
                        mma_bf16(t, x.z, y.z, x.w, y.w, qlo[2 * j - 7][0], qlo[2 * j - 7][1]);
                    }
                }
            }
        }
        __syncwarp();  // every lane has its keys in registers: the stage's K may be overwritten
        copy_k(n + STAGES);
        uint32_t ph0 = 0u, ph1 = 0u, pl0 = 0u, pl1 = 0u;
        const bool partial = vis.partial(pos0 / BLOCK);
        if (there) {
            const float k0 = f0 * a.z, k1 = f1 * a.z;
            s[0] = (s[0] + t[0]) * k0;
            s[1] = (s[1] + t[1]) * k1;
            s[2] = (s[2] + t[2]) * k0;
            s[3] = (s[3] + t[3]) * k1;
            if (partial) {
                if (!vis.sees(pos0 + g8)) s[0] = s[1] = -INFINITY;
                if (!vis.sees(pos0 + g8 + 8)) s[2] = s[3] = -INFINITY;
            }
            float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
            if (__any_sync(0xffffffffu, x0 > m0 + kTrail || x1 > m1 + kTrail)) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
                }
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float a0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
                const float a1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
                m0 = n0, m1 = n1;
                l0 *= a0, l1 *= a1;
#pragma unroll
                for (int mt = 0; mt < DV / 16; ++mt) o[mt][0] *= a0, o[mt][1] *= a1, o[mt][2] *= a0, o[mt][3] *= a1;
            }
            const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
            float p0 = fast_exp2(s[0] - b0), p1 = fast_exp2(s[1] - b1);
            float p2 = fast_exp2(s[2] - b0), p3 = fast_exp2(s[3] - b1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            if constexpr (E4M3) {
                float ratio = a.w * vs_inv;
                const float size = fabsf(a.w);
                if (!(fabsf(ratio) >= kRatioMin && fabsf(ratio) <= kRatioMax) && size > 0.f) {
                    const float unit = fmaxf(size, vs_floor), inv = kBias / unit, f = vs_inv > 0.f ? inv / vs_inv : 1.f;
#pragma unroll
                    for (int mt = 0; mt < DV / 16; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][e] *= f;
                    vs_inv = inv, vs_floor = fmaxf(vs_floor, unit * kUnitDrop), ratio = a.w * inv;
                }
                p0 *= ratio, p1 *= ratio, p2 *= ratio, p3 *= ratio;
            }
            // P^T as the second product's B operand. f16 rounds it by 2^-12; bf16's 2^-9 would show beside the
            // output's own rounding, so there the remainder goes along as a second product.
            if constexpr (E4M3) {
                ph0 = movmatrix_t(pack_f16x2(p0, p1));
                ph1 = movmatrix_t(pack_f16x2(p2, p3));
            } else {
                const uint32_t h0 = pack_bf16x2(p0, p1), h1 = pack_bf16x2(p2, p3);
                ph0 = movmatrix_t(h0);
                ph1 = movmatrix_t(h1);
                pl0 = movmatrix_t(pack_bf16x2(p0 - __uint_as_float(h0 << 16), p1 - __uint_as_float(h0 & 0xFFFF0000u)));
                pl1 = movmatrix_t(pack_bf16x2(p2 - __uint_as_float(h1 << 16), p3 - __uint_as_float(h1 & 0xFFFF0000u)));
            }
        }
        cp_async_wait<2 * STAGES - 1>();
        __syncwarp();
        if (there) {
            // V^T as the A operand; keys that are not seen count as zero, whatever the slot holds.
            if constexpr (E4M3) {
                // rows of keys 2c, 2c+1, 2c+8, 2c+9, dims 16 g8 .. 16 g8 + 15: rows g8 and g8 + 8 of tile mt are
                // dims 16 g8 + 2 mt and the next
                uint32_t v[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 2 * c + (e & 1) + 8 * (e >> 1);
                    const uint4 x = *reinterpret_cast<const uint4 *>(vb + v_place<true>(key, g8));
                    v[e][0] = x.x, v[e][1] = x.y, v[e][2] = x.z, v[e][3] = x.w;
                }
                if (partial) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!vis.sees(pos0 + 2 * c + (e & 1) + 8 * (e >> 1))) v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0u;
                }
#pragma unroll
                for (int mt = 0; mt < DV / 16; ++mt) {
                    const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
                    const uint32_t lo = __byte_perm(v[0][mt >> 1], v[1][mt >> 1], sel);
                    const uint32_t hi = __byte_perm(v[2][mt >> 1], v[3][mt >> 1], sel);
                    mma_f16(o[mt], e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi),
                            e4m3x2_to_f16x2(hi >> 16), ph0, ph1);
                }
            } else {
                // matrices (keys 0-7 | 8-15) x (dims 0-7 | 8-15) of each 16-dim tile, transposed on the way
                const uint32_t va = smem_u32(vb);
                const int key = (lane & 7) + 8 * (lane >> 4), unit = (lane >> 3) & 1;
                uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;  // keys 2c, 2c+1 and 2c+8, 2c+9 of a register
                if (partial) {
                    const auto pair = [&](int k) {
                        return (vis.sees(pos0 + k) ? 0xFFFFu : 0u) | (vis.sees(pos0 + k + 1) ? 0xFFFF0000u : 0u);
                    };
                    keep0 = pair(2 * c);
                    keep1 = pair(2 * c + 8);
                }
#pragma unroll
                for (int mt = 0; mt < DV / 16; ++mt) {
                    uint32_t v0, v1, v2, v3;
                    ldsm_x4_t(va + v_place<false>(key, 2 * mt + unit), v0, v1, v2, v3);
                    if (partial) v0 &= keep0, v1 &= keep0, v2 &= keep1, v3 &= keep1;
                    mma_bf16(o[mt], v0, v1, v2, v3, ph0, ph1);
                    mma_bf16(o[mt], v0, v1, v2, v3, pl0, pl1);
                }
            }
        }
        __syncwarp();
        copy_v(n + STAGES);
    }
    cp_async_wait<0>();

    // What this thread will need of gate and lambda, under way while the sums are joined: outputs (place, signal
    // head) i = thread, thread + THREADS, ..
    const int n_part = p.splits / p.cluster;
    const int share = DV / p.cluster, first = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) * share : 0;
    constexpr int MAX_OUT = 4 * DV / C::THREADS;
    __nv_bfloat16 gate_in[MAX_OUT];
    float lam_in[MAX_OUT];
    if (n_part == 1) {
#pragma unroll
        for (int j = 0; j < MAX_OUT; ++j) {
            const int i = threadIdx.x + j * C::THREADS;
            if (i < 4 * share) {
                const int h = p.cluster > 1 ? i / share : i / DV, at = p.cluster > 1 ? i - h * share : i % DV;
                const size_t row = bg * 4 + h;
                gate_in[j] = p.gate[row * DV + dim_of<E4M3>(first + at)];
                lam_in[j] = __ldg(p.lambda + row);
            }
        }
    }

    // the warps' sums, each brought to the heads' maxima over the warps, over the ring
    float *red = reinterpret_cast<float *>(smem), *ml = reinterpret_cast<float *>(smem + C::OFF_ML);
    float *cta = reinterpret_cast<float *>(smem + C::OFF_CTA), *cml = ml + WARPS * 16;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (g8 == 0) *reinterpret_cast<float4 *>(ml + (warp * 8 + 2 * c) * 2) = make_float4(m0, l0, m1, l1);
    __syncthreads();
    float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        M0 = fmaxf(M0, ml[(w * 8 + 2 * c) * 2]);
        M1 = fmaxf(M1, ml[(w * 8 + 2 * c + 1) * 2]);
    }
    float w0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - M0), w1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - M1);
    if constexpr (E4M3) {
        if (vs_inv > 0.f) w0 /= vs_inv, w1 /= vs_inv;
    }
#pragma unroll
    for (int mt = 0; mt < DV / 16; ++mt) {
        float *dst = red + (warp * HEADS + 2 * c) * RED_ROW + 16 * mt + 2 * g8;
        if (2 * c < HEADS) *reinterpret_cast<float2 *>(dst) = make_float2(o[mt][0] * w0, o[mt][2] * w0);
        if (2 * c + 1 < HEADS) *reinterpret_cast<float2 *>(dst + RED_ROW) = make_float2(o[mt][1] * w1, o[mt][3] * w1);
    }
    if (threadIdx.x < HEADS) {  // the heads' maxima and sums
        const int h = threadIdx.x;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[(w * 8 + h) * 2]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float mw = ml[(w * 8 + h) * 2];
            // (a maximum of -inf goes with a sum of zero, or of NaN, which stays)
            L += (mw == -INFINITY ? 0.f : fast_exp2(mw - M)) * ml[(w * 8 + h) * 2 + 1];
        }
        cml[2 * h] = M, cml[2 * h + 1] = L;
    }
    __syncthreads();
    const auto warps_sum = [&](int h, int d) {
        const float *src = red + h * RED_ROW + d;
        float O = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) O += src[w * HEADS * RED_ROW];
        return O;
    };
    if (p.cluster == 1) {
        // (THREADS divides 128 or is its multiple, so a thread's outputs are those of one place or two)
        constexpr int PLACES = MAX_OUT >= 4 ? MAX_OUT / 4 : 1;
#pragma unroll
        for (int q = 0; q < PLACES; ++q) {
            const int d = (threadIdx.x + q * C::THREADS) % DV;
            const float hn = paged_head(warps_sum(4, d), cml[9]);
#pragma unroll
            for (int j = q; j < MAX_OUT; j += PLACES) {
                const int h = (threadIdx.x + j * C::THREADS) / DV;
                p.out[(bg * 4 + h) * DV + dim_of<E4M3>(d)] =
                    paged_output(paged_head(warps_sum(h, d), cml[2 * h + 1]), hn, lam_in[j], gate_in[j]);
            }
        }
        return;
    }
    for (int i = threadIdx.x; i < HEADS * DV; i += C::THREADS) cta[i] = warps_sum(i / DV, i % DV);
    cluster_sync();
    // this CTA's share of the places, from every CTA of the cluster
    {
        for (int i = threadIdx.x; i < HEADS * share; i += C::THREADS) {
            const int h = i / share, d = first + i % share;
            const uint32_t a_o = smem_u32(cta + h * DV + d), a_ml = smem_u32(cml + 2 * h);
            float mr[MAX_CLUSTER], lr[MAX_CLUSTER], orr[MAX_CLUSTER], M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) {
                mr[r] = -INFINITY, lr[r] = orr[r] = 0.f;
                if (r < p.cluster) {
                    mr[r] = ld_cluster(a_ml, r);
                    lr[r] = ld_cluster(a_ml + 4, r);
                    orr[r] = ld_cluster(a_o, r);
                }
                M = fmaxf(M, mr[r]);
            }
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) {
                const float f = mr[r] == -INFINITY ? 0.f : fast_exp2(mr[r] - M);
                L += f * lr[r];
                O += f * orr[r];
            }
            if (n_part > 1) {
                const size_t slot = static_cast<size_t>(item) * n_part + split / p.cluster;
                p.ws[slot * (HEADS * DV) + h * DV + d] = O;
                float *wml = p.ws + static_cast<size_t>(p.hkv) * p.batch * n_part * (HEADS * DV) + slot * (2 * HEADS);
                if (d == 0) wml[2 * h] = M, wml[2 * h + 1] = L;  // (O by place)
            } else {
                red[h * DV + d] = paged_head(O, L);
            }
        }
        cluster_sync();  // everyone has read everyone's sums: the CTAs may leave
    }
    if (n_part > 1) return;
#pragma unroll
    for (int j = 0; j < MAX_OUT; ++j) {
        const int i = threadIdx.x + j * C::THREADS;
        if (i < 4 * share) {
            const int h = i / share, d = first + i % share;
            p.out[(bg * 4 + h) * DV + dim_of<E4M3>(d)] =
                paged_output(red[h * DV + d], red[4 * DV + d], lam_in[j], gate_in[j]);
        }
    }
}

// Several clusters per item: their sums joined, one block of 128 threads (one per place) per item.
template <bool E4M3>
__global__ void __launch_bounds__(dp::DV)
gdla_decode_paged_combine_kernel(const __grid_constant__ PagedDecode p) {
    using namespace dp;
    const int n_part = p.splits / p.cluster, d = threadIdx.x, dim = dim_of<E4M3>(d);
    const size_t slot0 = static_cast<size_t>(blockIdx.x) * n_part;
    const float *wml = p.ws + static_cast<size_t>(p.hkv) * p.batch * n_part * (HEADS * DV);
    float hv[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int s = 0; s < n_part; ++s) M = fmaxf(M, wml[(slot0 + s) * (2 * HEADS) + 2 * h]);
        for (int s = 0; s < n_part; ++s) {
            const float ms = wml[(slot0 + s) * (2 * HEADS) + 2 * h];
            const float f = ms == -INFINITY ? 0.f : fast_exp2(ms - M);
            L += f * wml[(slot0 + s) * (2 * HEADS) + 2 * h + 1];
            O += f * p.ws[((slot0 + s) * HEADS + h) * DV + d];
        }
        hv[h] = paged_head(O, L);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t r = static_cast<size_t>(blockIdx.x) * 4 + i;
        p.out[r * DV + dim] = paged_output(hv[i], hv[4], __ldg(p.lambda + r), p.gate[r * DV + dim]);
    }
}

// How an item is cut, by measurement (us a call, 64-token pages; "8 x 2": two clusters of 8 CTAs, joined by the
// combine kernel):
//  - up to 18 items: CTAs of 8 warps in clusters of 8, which then all run at once. batch 1, 16 heads, 4,096 tokens, bf16:
//    69.6 with one CTA of 4 warps per item, 15.5 with 8, 14.0 with 8 of 8 warps; 8 heads: 13.5 and 10.8; 3 x 16 heads: 25.9
//    and 30.2
//  - the combine kernel costs some 5 us, so parts come with 8,192 keys each and only up to one CTA per SM. 1 x 1 x 32,768:
//    42.9 (8), 20.8 (8 x 4); 1 x 2 x 8,192: 15.4 (8), 15.1 (8 x 4); 1 x 16 x 16,384: 35.3 (8), 39.9 (8 x 2)
//  - more items: clusters as long as two CTAs per SM are not there yet and each gets a block per warp.
//    4 x 16 x 4,096: 72 (1), 43 (2), 32.0 (4), 32.6 (8)
//  - many of few keys (windows): CTAs of 2 warps. 64 x 16, window 128 and 4 sinks, bf16: 28.4 with 4 warps, 22.4 with 2
//  - many: runs of 2,048 keys even out unequal lengths. 64 x 16 x 1,024 to 32,768 e4m3: 932 (2), 862 (4, 8);
//    16 x 16 x 2,048 bf16: 55.2 (1), 57.9 (2)
PagedSplit paged_split(int batch, int hkv, int max_seqlen_k, int window, int sinks) {
    const long long items = static_cast<long long>(batch) * hkv;
    const long long keys = window > 0 ? std::min<long long>(max_seqlen_k, static_cast<long long>(window) + sinks)
                                      : max_seqlen_k;
    const long long blocks = (keys + dp::BLOCK - 1) / dp::BLOCK;
    PagedSplit s{1, 1, 4};
    if (items * dp::MAX_CLUSTER <= kPlanSms && blocks >= 64) {
        s.warps = 8;
        s.cluster = dp::MAX_CLUSTER;
        s.parts = static_cast<int>(
            std::max<long long>(1, std::min(blocks / 512, kPlanSms / (items * dp::MAX_CLUSTER))));
        return s;
    }
    while (s.cluster < dp::MAX_CLUSTER && s.cluster * 2 <= blocks / 4 &&
           (items * s.cluster * 2 <= 2 * kPlanSms || s.cluster * 2 <= blocks / 128))
        s.cluster *= 2;
    if (s.cluster == 1 && blocks <= 32 && items > 4 * kPlanSms) s.warps = 2;
    return s;
}

size_t paged_workspace_bytes(int batch, int hkv, const PagedSplit &s) {
    return s.parts > 1 ? static_cast<size_t>(batch) * hkv * s.parts * dp::HEADS * (dp::DV + 2) * sizeof(float) : 0;
}

template <bool E4M3, int WARPS>
static cudaError_t launch_decode_paged_as(const PagedDecode &p, cudaStream_t stream) {
    using C = dp::Cfg<E4M3, WARPS>;
    static PerContextFlag attr_set;  // per device, for the context it was set in
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long ctx = current_context_id();
    if (!attr_set.is_set(dev, ctx)) {
        e = cudaFuncSetAttribute(gdla_decode_paged_kernel<E4M3, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        attr_set.set(dev, current_context_id());
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.hkv) * p.batch * p.splits);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, gdla_decode_paged_kernel<E4M3, WARPS>, p);
    if (e != cudaSuccess) return e;
    if (p.splits > p.cluster) {
        gdla_decode_paged_combine_kernel<E4M3><<<static_cast<unsigned>(p.hkv) * p.batch, dp::DV, 0, stream>>>(p);
        return cudaPeekAtLastError();
    }
    return cudaSuccess;
}

template <bool E4M3>
static cudaError_t launch_decode_paged_of(const PagedDecode &p, cudaStream_t stream) {
    switch (p.warps) {
        case 2: return launch_decode_paged_as<E4M3, 2>(p, stream);
        case 4: return launch_decode_paged_as<E4M3, 4>(p, stream);
        default: return launch_decode_paged_as<E4M3, 8>(p, stream);
    }
}

cudaError_t launch_decode_paged(const PagedDecode &p, bool e4m3, cudaStream_t stream) {
    return e4m3 ? launch_decode_paged_of<true>(p, stream) : launch_decode_paged_of<false>(p, stream);
}

}  // namespace gdla
