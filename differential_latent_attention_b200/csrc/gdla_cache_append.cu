// gdla_cache_append.cu - new keys and values into a paged KV cache, for sm_100a.
//
// Token n of the call belongs to sequence b (cu[b] <= n < cu[b+1]) and stands at
// position p = seqlens_k[b] - (cu[b+1] - cu[b]) + (n - cu[b]); it goes to slot
// p % P of page block_table[b][p / P]. Its key is [k_nope | R(p) k_rope], the
// 64-wide rotary key shared by every KV head and turned to p on the way (pairs i,
// i + 32, base 10000: the prologue's reading); in e4m3 pages the block of one page
// and KV head shares one power-of-two scale per tensor, the smallest 2^e with
// amax <= 448 * 2^e over the tokens that the page holds. A page that goes on
// keeps the larger of its scale and the new tokens' one; where it grows, the
// codes that the page held are divided by the growth, which is exact but for codes
// that fall under e4m3's subnormals.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdla_internal.h"
#include "gdla_paged.cuh"
#include "gdla_ptx.cuh"

namespace gdla {

// Units: the pages that the call touches, found without the host. Sequence b owns units
// cu[b] / P + 2 b .. cu[b + 1] / P + 2 (b + 1) - 1, which is room for the
// floor(n / P) + 2 pages that n tokens can touch; the units that it leaves over do nothing.
struct AppendUnit {
    bool live;
    int page;            // page of the pool
    int pos0;            // position of slot 0
    int slot0, slot1;    // slots that the call fills
    int tok0;            // token of slot0
};
__device__ __forceinline__ AppendUnit append_unit(const AppendPlan &p, int u) {
    AppendUnit a{};
    int b = 0, hi = p.batch;  // last b whose first unit is <= u
    while (hi - b > 1) {
        const int mid = (b + hi) / 2;
        if (p.cu_new[mid] / p.page_size + 2 * mid <= u)
            b = mid;
        else
            hi = mid;
    }
    const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1], len = p.seqlens_k[b];
    const int n = c1 - c0, before = len - n;
    if (c0 < 0 || n < 1 || c1 > p.num_tokens || before < 0 || len > p.max_pages * static_cast<long long>(p.page_size))
        return a;
    const int P = p.page_size;
    const int j = before / P + (u - (c0 / P + 2 * b));
    if (u < c0 / P + 2 * b || j > (len - 1) / P) return a;
    a.page = p.block_table[static_cast<size_t>(b) * p.max_pages + j];
    a.live = a.page >= 0 && a.page < p.num_pages;
    a.pos0 = j * P;
    a.slot0 = max(before, a.pos0) - a.pos0;
    a.slot1 = min(len, a.pos0 + P) - a.pos0;
    a.tok0 = c0 + a.pos0 + a.slot0 - before;
    return a;
}

__device__ __forceinline__ float block_max(float x, float *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    __syncthreads();
    if (lane == 0) red[warp] = x;
    __syncthreads();
    x = red[0];
    for (int i = 1; i < static_cast<int>(blockDim.x) / 32; ++i) x = fmaxf(x, red[i]);
    return x;
}

// One block per (unit, KV head); every value by itself.
template <bool E4M3>
__global__ void __launch_bounds__(256)
gdla_cache_append_kernel(const AppendPlan p) {
    __shared__ float red[8];
    const AppendUnit a = append_unit(p, blockIdx.x);
    if (!a.live) return;
    const int h = blockIdx.y, P = p.page_size, n = a.slot1 - a.slot0;
    const size_t blk = static_cast<size_t>(a.page) * p.hkv + h;
    const auto key = [&](int i, int d) {
        const size_t t = static_cast<size_t>(a.tok0 + i);
        if (d < 128) return __bfloat162float(p.k_nope[t * p.nope_token + static_cast<size_t>(h) * p.nope_head + d]);
        const __nv_bfloat16 *r = p.k_rope + t * p.rope_token;
        if (!p.rotate) return __bfloat162float(r[d - 128]);
        const int pair = (d - 128) & 31;
        float c, s;
        rotary_angle(a.pos0 + a.slot0 + i, pair, c, s);
        const float x0 = __bfloat162float(r[pair]), x1 = __bfloat162float(r[pair + 32]);
        return d < 160 ? x0 * c - x1 * s : x0 * s + x1 * c;
    };
    const auto value = [&](int i, int d) {
        return __bfloat162float(p.v[static_cast<size_t>(a.tok0 + i) * p.v_token + static_cast<size_t>(h) * p.v_head + d]);
    };
    const auto put = [&](auto get, void *pages, float *scale, int D) {
        if constexpr (!E4M3) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(pages) + (blk * P + a.slot0) * D;
            for (int i = threadIdx.x; i < n * D; i += blockDim.x) dst[i] = __float2bfloat16_rn(get(i / D, i % D));
        } else {
            float amax = 0.f;
            for (int i = threadIdx.x; i < n * D; i += blockDim.x) amax = fmaxf(amax, finite_abs(get(i / D, i % D)));
            int e = scale_exponent(block_max(amax, red));
            uint8_t *dst = static_cast<uint8_t *>(pages) + blk * P * D;
            if (a.slot0 > 0) {  // the page goes on: the larger scale of the two, older codes to it
                const int was = exponent_of_scale(scale[blk]);
                e = max(e, was);
                const float shrink = power_of_two(max(was - e, -126));
                if (was < e)
                    for (int i = threadIdx.x; i < a.slot0 * D / 2; i += blockDim.x) {
                        const uint32_t two = e4m3x2_to_f16x2(reinterpret_cast<uint16_t *>(dst)[i]);
                        const __half2 hv = *reinterpret_cast<const __half2 *>(&two);
                        reinterpret_cast<uint16_t *>(dst)[i] =
                            pack_e4m3x2(__low2float(hv) * shrink, __high2float(hv) * shrink);
                    }
            }
            const float inv = power_of_two(-e);
            for (int i = threadIdx.x; i < n * D / 2; i += blockDim.x) {
                const int t = 2 * i / D, d = 2 * i % D;
                reinterpret_cast<uint16_t *>(dst + a.slot0 * D)[i] =
                    pack_e4m3x2(finite_or_nan(get(t, d)) * inv, finite_or_nan(get(t, d + 1)) * inv);
            }
            __syncthreads();
            if (threadIdx.x == 0) scale[blk] = power_of_two(e);
        }
    };
    put(key, p.k_pages, p.k_scale, 192);
    put(value, p.v_pages, p.v_scale, 128);
}

cudaError_t launch_cache_append(const AppendPlan &p, bool e4m3, cudaStream_t stream) {
    const long long units = p.num_tokens / p.page_size + 2ll * p.batch;
    const dim3 grid(static_cast<unsigned>(units), p.hkv);
    if (e4m3)
        gdla_cache_append_kernel<true><<<grid, 256, 0, stream>>>(p);
    else
        gdla_cache_append_kernel<false><<<grid, 256, 0, stream>>>(p);
    return cudaPeekAtLastError();
}

}  // namespace gdla
