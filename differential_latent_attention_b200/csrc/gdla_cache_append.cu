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
// that fall under e4m3's subnormals. A power of two costs e4m3 no precision (it is a floating type: a
// scale moves only where its smallest numbers begin) and keeps those divisions exact.
//
// Bytes alone bound it: 8,320 read and 5,120 (e4m3, 16 heads) or 10,240 (bf16) written per token.
// Measured on one B200 (16 heads), in a graph and, in brackets, as called: 32,600 tokens into e4m3 pages of 64 82 us
// (84 to 88), 5.3 TB/s of 6.5 TB/s copied, held by the conversions beside the loads (59 % of the issue slots); a step
// of 64 sequences 4.5 us (6.2), of one 3.1 us (4.1), which is a launch and a chain of five dependent loads (sequence,
// lengths, page, scale, row). One launch takes steps and prompts together, each page by the rows that it gets: 63
// steps beside a chunk of 65 tokens 8.6 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gdla_internal.h"
#include "gdla_paged.cuh"
#include "gdla_ptx.cuh"

namespace gdla {

// Units: the pages that the call touches, found without the host. Sequence b owns units
// cu[b] / P + 2 b .. cu[b + 1] / P + 2 (b + 1) - 1, which is room for the
// floor(n / P) + 2 pages that n tokens can touch; the units that it leaves over do nothing.
// (Where cu descends the ranges overlap and a unit goes to one of their sequences: what it finds there is checked
// as ever, but another sequence's page may find no unit.)
struct AppendUnit {
    bool fits;           // the unit has tokens (its page is still to be checked)
    int page;            // page of the pool
    int pos0;            // position of slot 0
    int slot0, slot1;    // slots that the call fills
    int tok0;            // token of slot0
};
// The sequence of unit u, the last one whose first unit is <= u; the whole warp calls. The lanes look first at the
// 32 sequences around where u would be if all brought equally many tokens (`per_unit` sequences a unit), which finds
// steps and up to 32 sequences at once. Otherwise each round tries 32 places of what is left: 1,024 sequences take
// two more dependent loads.
__device__ __forceinline__ int append_sequence(const AppendPlan &p, int u, float per_unit) {
    const auto first = [&](int b) { return (p.cu_new[b] >> p.page_shift) + 2 * b; };
    const int lane = threadIdx.x & 31;
    const int near = max(0, min(static_cast<int>(static_cast<float>(u) * per_unit) - 16, p.batch - 32));
    const unsigned seen = __ballot_sync(0xffffffffu, near + lane < p.batch && first(near + lane) <= u);
    if ((near == 0 || (seen & 1u)) && (near + 32 >= p.batch || !(seen >> 31))) return near + max(__popc(seen) - 1, 0);
    int b = 0, left = p.batch;  // it is one of b .. b + left - 1
    while (left > 1) {
        const int step = (left + 31) / 32, mine = b + lane * step;
        const bool before = lane * step < left && first(mine) <= u;
        const int hits = __popc(__ballot_sync(0xffffffffu, before));
        const int skip = max(hits - 1, 0) * step;
        b += skip;
        left = min(step, left - skip);
    }
    return b;
}
__device__ __forceinline__ AppendUnit append_unit(const AppendPlan &p, int u, float per_unit) {
    AppendUnit a{};
    const int b = append_sequence(p, u, per_unit);
    const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1], len = p.seqlens_k[b];
    const int P = p.page_size;
    if (c0 < 0 || c1 <= c0 || c1 > p.num_tokens || len > p.max_pages * static_cast<long long>(P)) return a;
    const int n = c1 - c0;
    if (len < n) return a;  // (compared, not subtracted: a length of -2^31 would come back positive)
    const int before = len - n, first = (c0 >> p.page_shift) + 2 * b, page0 = before >> p.page_shift;
    if (u < first || u - first > ((len - 1) >> p.page_shift) - page0) return a;
    const int j = page0 + (u - first);
    a.fits = true;
    a.page = p.block_table[static_cast<size_t>(b) * p.max_pages + j];
    a.pos0 = j << p.page_shift;
    a.slot0 = max(before, a.pos0) - a.pos0;
    a.slot1 = min(len - a.pos0, P);
    a.tok0 = c0 + a.pos0 + a.slot0 - before;
    return a;
}
__device__ __forceinline__ bool in_pool(const AppendPlan &p, int page) { return page >= 0 && page < p.num_pages; }

// Largest |x| of eight bf16 as fp32 bits: integers order like the numbers, and what is not
// finite is 0x7F800000 or more.
__device__ __forceinline__ uint32_t max_bits(const uint4 &x) {
    const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
}
constexpr uint32_t kInfBits = 0x7F800000u;
// The same over the finite ones alone (the rare case).
__device__ __forceinline__ uint32_t finite_max_bits(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] << 16) & 0x7FFFFFFFu, hi = w[i] & 0x7FFF0000u;
        m = max(m, max(lo < kInfBits ? lo : 0u, hi < kInfBits ? hi : 0u));
    }
    return m;
}
// Eight values times inv as e4m3 codes; FINITE: there is no infinity or NaN among them.
template <bool FINITE>
__device__ __forceinline__ uint32_t pair_e4m3(float lo, float hi, float inv) {
    return FINITE ? pack_e4m3x2(lo * inv, hi * inv) : pack_e4m3x2(finite_or_nan(lo) * inv, finite_or_nan(hi) * inv);
}
template <bool FINITE>
__device__ __forceinline__ uint2 to_e4m3(const uint4 &x, float inv) {
    const auto two = [inv](uint32_t w) {
        return pair_e4m3<FINITE>(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u), inv);
    };
    return make_uint2(__byte_perm(two(x.x), two(x.y), 0x5410), __byte_perm(two(x.z), two(x.w), 0x5410));
}
template <bool FINITE>
__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8], float inv) {
    const auto two = [&](int i) { return pair_e4m3<FINITE>(x[i], x[i + 1], inv); };
    return make_uint2(__byte_perm(two(0), two(2), 0x5410), __byte_perm(two(4), two(6), 0x5410));
}
__device__ __forceinline__ uint4 to_bf16(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint32_t max_bits(const float (&x)[8], bool finite_only) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        m = max(m, finite_only && v >= kInfBits ? 0u : v);
    }
    return m;
}

// Rotary dims 8 q .. 8 q + 7 and their partners 32 + 8 q .. of one token, turned.
struct RopePart {
    float lo[8], hi[8];
};
__device__ __forceinline__ RopePart rope_part(const AppendPlan &p, int token, int pos, int q) {
    const __nv_bfloat16 *src = p.k_rope + static_cast<size_t>(token) * p.rope_token + 8 * q;
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src)), b = __ldg(reinterpret_cast<const uint4 *>(src + 32));
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
    RopePart r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r.lo[i] = __uint_as_float((i & 1) ? aw[i >> 1] & 0xFFFF0000u : aw[i >> 1] << 16);
        r.hi[i] = __uint_as_float((i & 1) ? bw[i >> 1] & 0xFFFF0000u : bw[i >> 1] << 16);
    }
    if (p.rotate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            double c, s;
            rotary_angle(pos, 8 * q + i, c, s);
            const double x = r.lo[i], y = r.hi[i];
            r.lo[i] = static_cast<float>(x * c - y * s);
            r.hi[i] = static_cast<float>(x * s + y * c);
        }
    }
    return r;
}

// Codes of `bytes` bytes (a multiple of 8, 8-byte aligned) times a power of two <= 1, in place,
// by `threads` threads of which this is `t`.
__device__ __forceinline__ void shrink_codes(uint8_t *codes, int bytes, float by, int t, int threads) {
    for (int i = t; i < bytes / 8; i += threads) {
        uint2 x = reinterpret_cast<uint2 *>(codes)[i];
        const auto two = [by](uint32_t c) {
            const uint32_t h = e4m3x2_to_f16x2(c);
            const __half2 v = *reinterpret_cast<const __half2 *>(&h);
            return pack_e4m3x2(__low2float(v) * by, __high2float(v) * by);
        };
        x.x = two(x.x & 0xFFFFu) | (two(x.x >> 16) << 16);
        x.y = two(x.y & 0xFFFFu) | (two(x.y >> 16) << 16);
        reinterpret_cast<uint2 *>(codes)[i] = x;
    }
}
// The block's exponent from its new tokens' largest |x|, the scale it had and whether it goes on.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits, bool goes_on, float had, float &shrink) {
    int e = scale_exponent(__uint_as_float(amax_bits));
    shrink = 1.f;
    if (goes_on) {
        const int was = exponent_of_scale(had);
        e = max(e, was);
        shrink = power_of_two(max(was - e, -126));
    }
    return e;
}

// Few rows (a decode step): one warp per head, every row in its registers; lanes 0..15 hold a row's K content,
// 16..31 its V, and lane i pair i of the rotary part as well.
constexpr int kFewRows = 4;
template <bool E4M3>
__device__ __forceinline__ void append_few(const AppendPlan &p, const AppendUnit &a, int h0, int h1) {
    const int n = a.slot1 - a.slot0, lane = threadIdx.x & 31;
    const bool is_k = lane < 16;
    float lo[kFewRows], hi[kFewRows];  // rotary pair `lane`
    float rope_max = 0.f;
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
        lo[r] = hi[r] = 0.f;
        if (r < n) {
            const __nv_bfloat16 *rope = p.k_rope + static_cast<size_t>(a.tok0 + r) * p.rope_token + lane;
            lo[r] = __bfloat162float(rope[0]);
            hi[r] = __bfloat162float(rope[32]);
        }
    }
    for (int h = h0 + (threadIdx.x >> 5); h < h1; h += 8) {
        const __nv_bfloat16 *src = is_k ? p.k_nope + static_cast<size_t>(a.tok0) * p.nope_token + h * p.nope_head + 8 * lane
                                        : p.v + static_cast<size_t>(a.tok0) * p.v_token + h * p.v_head + 8 * (lane - 16);
        const long long step = is_k ? p.nope_token : p.v_token;
        uint4 x[kFewRows];  // eight values of K's content or V
#pragma unroll
        for (int r = 0; r < kFewRows; ++r)
            x[r] = r < n ? __ldg(reinterpret_cast<const uint4 *>(src + r * step)) : make_uint4(0u, 0u, 0u, 0u);
        if (!in_pool(p, a.page)) return;
        const size_t blk = static_cast<size_t>(a.page) * p.hkv + h, slot = (blk << p.page_shift) + a.slot0;
        const bool goes_on = E4M3 && a.slot0 > 0;
        const float k_had = goes_on ? p.k_scale[blk] : 0.f, v_had = goes_on ? p.v_scale[blk] : 0.f;
        if (h < h0 + 8) {  // the warp's first head: turn the keys while the rows are under way
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                if (r < n && p.rotate) {
                    double c, s;
                    rotary_angle(a.pos0 + a.slot0 + r, lane, c, s);
                    const double y = lo[r], z = hi[r];
                    lo[r] = static_cast<float>(y * c - z * s);
                    hi[r] = static_cast<float>(y * s + z * c);
                }
                if (E4M3) rope_max = fmaxf(rope_max, fmaxf(finite_abs(lo[r]), finite_abs(hi[r])));
            }
        }
        if constexpr (!E4M3) {
            __nv_bfloat16 *kd = static_cast<__nv_bfloat16 *>(p.k_pages) + slot * 192;
            __nv_bfloat16 *vd = static_cast<__nv_bfloat16 *>(p.v_pages) + slot * 128;
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                if (r < n) {
                    *reinterpret_cast<uint4 *>(is_k ? kd + r * 192 + 8 * lane : vd + r * 128 + 8 * (lane - 16)) = x[r];
                    kd[r * 192 + 128 + lane] = __float2bfloat16_rn(lo[r]);
                    kd[r * 192 + 160 + lane] = __float2bfloat16_rn(hi[r]);
                }
            }
        } else {
            uint32_t mine = 0u;
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                const uint32_t raw = max_bits(x[r]);
                mine = max(mine, raw < kInfBits ? raw : finite_max_bits(x[r]));
            }
            const uint32_t km = __reduce_max_sync(0xffffffffu, max(is_k ? mine : 0u, __float_as_uint(rope_max)));
            const uint32_t vm = __reduce_max_sync(0xffffffffu, is_k ? 0u : mine);
            float k_shrink, v_shrink;
            const int ke = block_exponent(km, goes_on, k_had, k_shrink);
            const int ve = block_exponent(vm, goes_on, v_had, v_shrink);
            uint8_t *kd = static_cast<uint8_t *>(p.k_pages) + slot * 192;
            uint8_t *vd = static_cast<uint8_t *>(p.v_pages) + slot * 128;
            if (k_shrink < 1.f) shrink_codes(kd - a.slot0 * 192, a.slot0 * 192, k_shrink, lane, 32);
            if (v_shrink < 1.f) shrink_codes(vd - a.slot0 * 128, a.slot0 * 128, v_shrink, lane, 32);
            const float ki = power_of_two(-ke), vi = power_of_two(-ve);
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                if (r < n) {
                    uint8_t *dst = is_k ? kd + r * 192 + 8 * lane : vd + r * 128 + 8 * (lane - 16);
                    *reinterpret_cast<uint2 *>(dst) = to_e4m3<false>(x[r], is_k ? ki : vi);
                    const uint32_t two = pair_e4m3<false>(lo[r], hi[r], ki);
                    kd[r * 192 + 128 + lane] = static_cast<uint8_t>(two);
                    kd[r * 192 + 160 + lane] = static_cast<uint8_t>(two >> 8);
                }
            }
            if (lane == 0 && (k_had != power_of_two(ke) || v_had != power_of_two(ve)))
                p.k_scale[blk] = power_of_two(ke), p.v_scale[blk] = power_of_two(ve);
        }
    }
}

// One CTA per (unit, heads_per_cta heads); a unit of few rows goes to its warps, one head each. Otherwise a page
// and head's new values stay in registers between the search for the largest and the writing, so each input is
// read once; the turned rotary key is shared by the CTA's heads. NI = page_size / 16: 16-byte pieces of K's
// content (and of V) per thread.
template <bool E4M3, int NI>
__global__ void __launch_bounds__(256, NI <= 4 ? 3 : 2)
gdla_cache_append_kernel(const __grid_constant__ AppendPlan p, float per_unit) {
    constexpr int NR = NI <= 4 ? 1 : NI / 4;  // rotary pieces (8 pairs) per thread
    __shared__ uint32_t red[2][2][8];
    const int groups = (p.hkv + p.heads_per_cta - 1) / p.heads_per_cta;
    const int u = blockIdx.x / groups;
    const AppendUnit a = append_unit(p, u, per_unit);
    if (!a.fits) return;
    const int n = a.slot1 - a.slot0, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int h0 = (blockIdx.x - u * groups) * p.heads_per_cta, h1 = min(p.hkv, h0 + p.heads_per_cta);
    if (n <= kFewRows) {
        append_few<E4M3>(p, a, h0, h1);
        return;
    }
    const int row = t >> 4, col = t & 15;     // pieces (row + 16 i, col)
    const int rrow = t >> 2, rq = t & 3;      // rotary pieces (rrow + 64 i, rq)
    RopePart rope[NR];
    uint32_t rope_max = 0u;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = rrow + 64 * i;
        if (r < n) {
            rope[i] = rope_part(p, a.tok0 + r, a.pos0 + a.slot0 + r, rq);
            if (E4M3) rope_max = max(rope_max, max(max_bits(rope[i].lo, false), max_bits(rope[i].hi, false)));
        }
    }
    if (!in_pool(p, a.page)) return;
    const size_t tok = static_cast<size_t>(a.tok0 + row);
    const __nv_bfloat16 *k_src = p.k_nope + tok * p.nope_token + h0 * p.nope_head + 8 * col;
    const __nv_bfloat16 *v_src = p.v + tok * p.v_token + h0 * p.v_head + 8 * col;
    for (int h = h0; h < h1; ++h, k_src += p.nope_head, v_src += p.v_head) {
        const size_t blk = static_cast<size_t>(a.page) * p.hkv + h;
        uint4 k[NI], v[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row + 16 * i < n) {
                k[i] = __ldg(reinterpret_cast<const uint4 *>(k_src + 16 * i * p.nope_token));
                v[i] = __ldg(reinterpret_cast<const uint4 *>(v_src + 16 * i * p.v_token));
            }
        }
        const size_t slot = (blk << p.page_shift) + a.slot0;
        if constexpr (!E4M3) {
            __nv_bfloat16 *kd = static_cast<__nv_bfloat16 *>(p.k_pages) + slot * 192;
            __nv_bfloat16 *vd = static_cast<__nv_bfloat16 *>(p.v_pages) + slot * 128;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = row + 16 * i;
                if (r < n) {
                    *reinterpret_cast<uint4 *>(kd + r * 192 + 8 * col) = k[i];
                    *reinterpret_cast<uint4 *>(vd + r * 128 + 8 * col) = v[i];
                }
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = rrow + 64 * i;
                if (r < n) {
                    *reinterpret_cast<uint4 *>(kd + r * 192 + 128 + 8 * rq) = to_bf16(rope[i].lo);
                    *reinterpret_cast<uint4 *>(kd + r * 192 + 160 + 8 * rq) = to_bf16(rope[i].hi);
                }
            }
        } else {
            const bool goes_on = a.slot0 > 0;
            const float k_had = goes_on ? p.k_scale[blk] : 0.f, v_had = goes_on ? p.v_scale[blk] : 0.f;
            const auto over_block = [&](uint32_t km, uint32_t vm, uint32_t (&buf)[2][8]) {
                km = __reduce_max_sync(0xffffffffu, km);
                vm = __reduce_max_sync(0xffffffffu, vm);
                if (lane == 0) buf[0][warp] = km, buf[1][warp] = vm;
                __syncthreads();
                km = __reduce_max_sync(0xffffffffu, buf[0][lane & 7]);
                vm = __reduce_max_sync(0xffffffffu, buf[1][lane & 7]);
                return make_uint2(km, vm);
            };
            uint32_t km = rope_max, vm = 0u;
#pragma unroll
            for (int i = 0; i < NI; ++i) km = max(km, max_bits(k[i])), vm = max(vm, max_bits(v[i]));
            uint2 m = over_block(km, vm, red[h & 1]);
            const bool fine = m.x < kInfBits && m.y < kInfBits;
            if (!fine) {  // infinities or NaN among them: once more without
                km = vm = 0u;
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    if (rrow + 64 * i < n) km = max(km, max(max_bits(rope[i].lo, true), max_bits(rope[i].hi, true)));
#pragma unroll
                for (int i = 0; i < NI; ++i) km = max(km, finite_max_bits(k[i])), vm = max(vm, finite_max_bits(v[i]));
                __syncthreads();
                m = over_block(km, vm, red[h & 1]);
            }
            float k_shrink, v_shrink;
            const int ke = block_exponent(m.x, goes_on, k_had, k_shrink);
            const int ve = block_exponent(m.y, goes_on, v_had, v_shrink);
            uint8_t *kd = static_cast<uint8_t *>(p.k_pages) + slot * 192;
            uint8_t *vd = static_cast<uint8_t *>(p.v_pages) + slot * 128;
            if (k_shrink < 1.f) shrink_codes(kd - a.slot0 * 192, a.slot0 * 192, k_shrink, t, 256);
            if (v_shrink < 1.f) shrink_codes(vd - a.slot0 * 128, a.slot0 * 128, v_shrink, t, 256);
            const float ki = power_of_two(-ke), vi = power_of_two(-ve);
            const auto write = [&](auto finite) {
                constexpr bool FINITE = decltype(finite)::value;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int r = row + 16 * i;
                    if (r < n) {
                        *reinterpret_cast<uint2 *>(kd + r * 192 + 8 * col) = to_e4m3<FINITE>(k[i], ki);
                        *reinterpret_cast<uint2 *>(vd + r * 128 + 8 * col) = to_e4m3<FINITE>(v[i], vi);
                    }
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int r = rrow + 64 * i;
                    if (r < n) {
                        *reinterpret_cast<uint2 *>(kd + r * 192 + 128 + 8 * rq) = to_e4m3<FINITE>(rope[i].lo, ki);
                        *reinterpret_cast<uint2 *>(kd + r * 192 + 160 + 8 * rq) = to_e4m3<FINITE>(rope[i].hi, ki);
                    }
                }
            };
            if (fine)
                write(std::true_type());
            else
                write(std::false_type());
            // every thread has read the old scales (before the reduction's barrier)
            if (t == 0) p.k_scale[blk] = power_of_two(ke), p.v_scale[blk] = power_of_two(ve);
        }
    }
}

template <bool E4M3>
static void launch_append_pages(const AppendPlan &p, float per_unit, unsigned grid, cudaStream_t stream) {
    switch (p.page_size) {
        case 16: gdla_cache_append_kernel<E4M3, 1><<<grid, 256, 0, stream>>>(p, per_unit); break;
        case 32: gdla_cache_append_kernel<E4M3, 2><<<grid, 256, 0, stream>>>(p, per_unit); break;
        case 64: gdla_cache_append_kernel<E4M3, 4><<<grid, 256, 0, stream>>>(p, per_unit); break;
        default: gdla_cache_append_kernel<E4M3, 8><<<grid, 256, 0, stream>>>(p, per_unit); break;
    }
}

cudaError_t launch_cache_append(const AppendPlan &plan, bool e4m3, cudaStream_t stream) {
    AppendPlan p = plan;
    const long long units = p.num_tokens / p.page_size + 2ll * p.batch;
    // Heads of a CTA. Prompts: 128 rows' worth (fewer and the search and the turned keys weigh more, us at 1, 2, 4, 8
    // heads: 13 chunks of 400 tokens, 5 heads, bf16 pages of 16: 13.3, 11.2, 8.8, 7.6; 8,000 tokens, 16 heads, e4m3 pages
    // of 32: 40, 32, 30, 33), four at least in large calls (32,600 tokens, e4m3 pages of 64: 119, 91, 82, 83).
    // Steps of one token: a head per warp or, once those CTAs would not all run at once, two (us at 4, 8, 16 heads, bf16
    // pages of 64: 64 sequences 4.0, 3.7, 4.0; 256: 9.2, 6.8, 5.2). Between them four heads, or eight for many
    // short ones (us at 2, 4, 8 heads, e4m3 pages of 64: 63 steps beside a chunk of 65 9.2, 8.5, 11.5; 255 beside
    // 1,024 20.8, 20.8, 23.4; 64 x 4 tokens 8.7, 6.3, 6.8). In each as long as every SM gets a CTA.
    const long long pairs = units * p.hkv;
    long long heads = 128 / p.page_size;
    if (p.num_tokens <= p.batch)
        heads = std::max(8ll, pairs / (3 * kPlanSms));
    else if (pairs >= 32ll * kPlanSms || p.num_tokens <= 16ll * p.batch)
        heads = std::max(heads, 4ll);
    if (p.num_tokens > p.batch && p.num_tokens <= 4ll * p.batch)
        heads = std::max(heads, std::min(8ll, pairs / (6 * kPlanSms)));
    p.heads_per_cta = static_cast<int>(std::max(1ll, std::min(heads, std::min<long long>(p.hkv, pairs / kPlanSms))));
    const float per_unit = static_cast<float>(p.batch) / static_cast<float>(units);
    const unsigned grid = static_cast<unsigned>(units * ((p.hkv + p.heads_per_cta - 1) / p.heads_per_cta));
    if (e4m3)
        launch_append_pages<true>(p, per_unit, grid, stream);
    else
        launch_append_pages<false>(p, per_unit, grid, stream);
    return cudaPeekAtLastError();
}

}  // namespace gdla
