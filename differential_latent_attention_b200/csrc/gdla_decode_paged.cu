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
// Keys come in blocks of 16 that never straddle a page (pages are multiples of 16), so
// a block has one scale for K and one for V. The products are mma.sync m16n8k16 with the
// keys (S^T = K Q^T) and the value dims (O^T = V^T P^T) as rows and the five heads in the
// eight columns. e4m3 codes become f16 (exact) and meet f16 queries divided by a power of
// two per head (exact but for elements 2^-14 under the head's largest) and f16
// probabilities; O's block sum takes the page's V scale in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdla_internal.h"
#include "gdla_paged.cuh"
#include "gdla_ptx.cuh"

namespace gdla {

namespace dp {
constexpr int DQK = 192, DV = 128, HEADS = 5;
constexpr int WARPS = 4;
constexpr float kScoreLog2 = 0.07216878364870322f * 1.4426950408889634f;  // log2(e) / sqrt(192)
}  // namespace dp

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

// This lane's query fragments: head lane / 4 (zero from 5 on), for each 16-dim step the
// dims of the MMA's K slots 2c, 2c+1 and 2c+8, 2c+9 (c = lane % 4). e4m3 keys are read four
// codes at a time, so there slot pair s of a step is dims 4c + 2s, 4c + 2s + 1 on both sides.
// The rotary dims 128..191 are turned to the query's position first: dim 128 + i (steps 8, 9)
// and its partner 160 + i (steps 10, 11) sit in the same slots of one lane. Returns the
// factor of this head's scores (1/sqrt(192) in log2 units, times the power of two taken
// out of an f16 query).
template <bool E4M3>
__device__ __forceinline__ float load_queries(uint32_t (&qf)[12][2], const __nv_bfloat16 *q_sig,
                                              const __nv_bfloat16 *q_noise, size_t bg, int lane, bool rotate, int pos) {
    using namespace dp;
    const int g8 = lane >> 2, c = lane & 3;
    float x[12][4];
    const __nv_bfloat16 *row = g8 < 4 ? q_sig + (bg * 4 + g8) * DQK : q_noise + bg * DQK;
#pragma unroll
    for (int ks = 0; ks < 12; ++ks)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int d = 16 * ks + (E4M3 ? 4 * c + 2 * s : 2 * c + 8 * s);
            const uint32_t two = g8 < HEADS ? *reinterpret_cast<const uint32_t *>(row + d) : 0u;
            x[ks][2 * s] = __uint_as_float(two << 16);
            x[ks][2 * s + 1] = __uint_as_float(two & 0xFFFF0000u);
        }
    if (rotate) {
#pragma unroll
        for (int ks = 8; ks < 10; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * (ks - 8) + (E4M3 ? 4 * c + e : 2 * c + 8 * (e >> 1) + (e & 1));
                float cs, sn;
                rotary_angle(pos, i, cs, sn);
                const float a = x[ks][e], b = x[ks + 2][e];
                x[ks][e] = a * cs - b * sn;
                x[ks + 2][e] = a * sn + b * cs;
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
            for (int s = 0; s < 2; ++s) qf[ks][s] = pack_bf16x2(x[ks][2 * s], x[ks][2 * s + 1]);
    }
    return factor;
}

// One block of four warps per (KV head, sequence); each warp takes every fourth block of
// 16 keys, straight from global memory, and the block joins the warps at the end.
template <bool E4M3>
__global__ void __launch_bounds__(dp::WARPS * 32)
gdla_decode_paged_kernel(const PagedDecode p) {
    using namespace dp;
    __shared__ float red[WARPS][HEADS][DV];
    __shared__ float ml[WARPS][8][2];
    const int group = blockIdx.x % p.hkv, b = blockIdx.x / p.hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, c = lane & 3;
    const int len = p.seqlens_k[b];
    const VisibleBlocks vis = visible_blocks(len, p.max_seqlen_k, p.window, p.sinks);
    const size_t bg = static_cast<size_t>(b) * p.hkv + group;

    uint32_t qf[12][2];
    const float factor = load_queries<E4M3>(qf, p.q_sig, p.q_noise, bg, lane, p.rotate, len - 1);
    const float f0 = __shfl_sync(0xffffffffu, factor, (8 * c) & 31), f1 = __shfl_sync(0xffffffffu, factor, (8 * c + 4) & 31);

    float o[DV / 16][4];
#pragma unroll
    for (int mt = 0; mt < DV / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1

    for (int i = warp; i < vis.n; i += WARPS) {
        const int pos0 = vis.block(i) * 16;
        const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + pos0 / p.page_size];
        if (page < 0 || page >= p.num_pages) continue;  // such an entry holds no keys
        const size_t blk = static_cast<size_t>(page) * p.hkv + group;
        const size_t row0 = blk * p.page_size + pos0 % p.page_size;
        const float ks_ = E4M3 ? p.k_scale[blk] : 1.f, vs_ = E4M3 ? p.v_scale[blk] : 1.f;
        const bool seen0 = vis.sees(pos0 + g8), seen1 = vis.sees(pos0 + g8 + 8);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 12; ++ks) {
            if constexpr (E4M3) {
                const uint8_t *k = static_cast<const uint8_t *>(p.k_pages) + (row0 + g8) * DQK + 16 * ks + 4 * c;
                const uint32_t x = *reinterpret_cast<const uint32_t *>(k);
                const uint32_t y = *reinterpret_cast<const uint32_t *>(k + 8 * DQK);
                mma_f16(s, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y), e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16),
                        qf[ks][0], qf[ks][1]);
            } else {
                const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(p.k_pages) + (row0 + g8) * DQK + 16 * ks + 2 * c;
                const auto at = [&](int o_) { return *reinterpret_cast<const uint32_t *>(k + o_); };
                mma_bf16(s, at(0), at(8 * DQK), at(8), at(8 * DQK + 8), qf[ks][0], qf[ks][1]);
            }
        }
        s[0] = seen0 ? s[0] * (f0 * ks_) : -INFINITY;
        s[1] = seen0 ? s[1] * (f1 * ks_) : -INFINITY;
        s[2] = seen1 ? s[2] * (f0 * ks_) : -INFINITY;
        s[3] = seen1 ? s[3] * (f1 * ks_) : -INFINITY;
        float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
        }
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
        const float a0 = fast_exp2(m0 - b0), a1 = fast_exp2(m1 - b1);
        m0 = n0, m1 = n1;
        const float p0 = fast_exp2(s[0] - b0), p1 = fast_exp2(s[1] - b1);
        const float p2 = fast_exp2(s[2] - b0), p3 = fast_exp2(s[3] - b1);
        l0 = l0 * a0 + p0 + p2;
        l1 = l1 * a1 + p1 + p3;
        const uint32_t pb0 = movmatrix_t(E4M3 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1));
        const uint32_t pb1 = movmatrix_t(E4M3 ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3));
        // values of keys that are not seen count as zero, whatever the page holds there
        bool sv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sv[e] = vis.sees(pos0 + 2 * c + (e & 1) + 8 * (e >> 1));
#pragma unroll
        for (int mt = 0; mt < DV / 16; ++mt) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (E4M3) {
                const uint8_t *v = static_cast<const uint8_t *>(p.v_pages) + (row0 + 2 * c) * DV + 16 * mt + 2 * g8;
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = sv[e] ? *reinterpret_cast<const uint16_t *>(v + ((e & 1) + 8 * (e >> 1)) * DV) : 0u;
                const auto two = [&](int e, int odd) {
                    return e4m3x2_to_f16x2(((w[e] >> (8 * odd)) & 0xFFu) | (((w[e + 1] >> (8 * odd)) & 0xFFu) << 8));
                };
                mma_f16(acc, two(0, 0), two(0, 1), two(2, 0), two(2, 1), pb0, pb1);
            } else {
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_pages) + (row0 + 2 * c) * DV + 16 * mt + g8;
                const auto two = [&](int e, int o_) {
                    const uint32_t lo = sv[e] ? *reinterpret_cast<const uint16_t *>(v + 4 * e * DV + o_) : 0u;
                    const uint32_t hi = sv[e + 1] ? *reinterpret_cast<const uint16_t *>(v + (4 * e + 1) * DV + o_) : 0u;
                    return lo | (hi << 16);
                };
                mma_bf16(acc, two(0, 0), two(0, 8), two(2, 0), two(2, 8), pb0, pb1);
            }
            o[mt][0] = fmaf(o[mt][0], a0, acc[0] * vs_);
            o[mt][1] = fmaf(o[mt][1], a1, acc[1] * vs_);
            o[mt][2] = fmaf(o[mt][2], a0, acc[2] * vs_);
            o[mt][3] = fmaf(o[mt][3], a1, acc[3] * vs_);
        }
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (g8 == 0) {
        ml[warp][2 * c][0] = m0, ml[warp][2 * c][1] = l0;
        ml[warp][2 * c + 1][0] = m1, ml[warp][2 * c + 1][1] = l1;
    }
    // value dim of accumulator rows g8 and g8 + 8 of tile mt
#pragma unroll
    for (int mt = 0; mt < DV / 16; ++mt) {
        const int da = 16 * mt + (E4M3 ? 2 * g8 : g8), db = 16 * mt + (E4M3 ? 2 * g8 + 1 : g8 + 8);
        if (2 * c < HEADS) red[warp][2 * c][da] = o[mt][0], red[warp][2 * c][db] = o[mt][2];
        if (2 * c + 1 < HEADS) red[warp][2 * c + 1][da] = o[mt][1], red[warp][2 * c + 1][db] = o[mt][3];
    }
    __syncthreads();
    const int d = threadIdx.x;
    float hv[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        float M = -INFINITY;
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w][h][0]);
        float L = 0.f, O = 0.f;
        for (int w = 0; w < WARPS; ++w) {
            const float f = ml[w][h][0] == -INFINITY ? 0.f : fast_exp2(ml[w][h][0] - M);
            L += f * ml[w][h][1];
            O += f * red[w][h][d];
        }
        hv[h] = L == 0.f ? 0.f : O / L;  // no key at all: zero; a NaN goes through
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t r = bg * 4 + i;
        const float g = __bfloat162float(p.gate[r * DV + d]);
        p.out[r * DV + d] = __float2bfloat16_rn(__fdividef(hv[i] - p.lambda[r] * hv[4], 1.f + __expf(-g)));
    }
}

cudaError_t launch_decode_paged(const PagedDecode &p, bool e4m3, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.hkv) * static_cast<unsigned>(p.batch);
    if (e4m3)
        gdla_decode_paged_kernel<true><<<grid, dp::WARPS * 32, 0, stream>>>(p);
    else
        gdla_decode_paged_kernel<false><<<grid, dp::WARPS * 32, 0, stream>>>(p);
    return cudaPeekAtLastError();
}

}  // namespace gdla
