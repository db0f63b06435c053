// gdla_paged.cuh - what the paged-cache kernels share: rotary angles and e4m3 blocks.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdla_internal.h"
#include "gdla_ptx.cuh"

namespace gdla {

// 10000^(-i/32) / (2 pi): turns of pair i per position. A position times this, its
// whole turns taken off in fp64, is good to 2^-24 of a turn at positions up to 2^31
// (2^-35 at 2^20); an fp32 angle is off by 2^-24 of the position itself.
__constant__ double kRotaryTurns[32] = {
    0.15915494309189535, 0.11934937021124886, 0.08949940160889101, 0.06711508300522726,
    0.050329212104487035, 0.03774158471741977, 0.0283021958306234, 0.02122365276477766,
    0.015915494309189534, 0.011934937021124886, 0.008949940160889102, 0.006711508300522725,
    0.005032921210448704, 0.003774158471741977, 0.00283021958306234, 0.0021223652764777662,
    0.0015915494309189533, 0.0011934937021124885, 0.0008949940160889101, 0.0006711508300522725,
    0.0005032921210448703, 0.0003774158471741977, 0.00028302195830623395, 0.0002122365276477766,
    0.00015915494309189532, 0.00011934937021124885, 8.949940160889102e-05, 6.711508300522725e-05,
    5.0329212104487035e-05, 3.774158471741977e-05, 2.8302195830623396e-05, 2.122365276477766e-05,
};

// cos and sin of the rotary angle of pair i at a position. In fp64 for keys, which are rounded once, to the
// cache's type, after the turn: an fp32 cosine, off by 2^-24, takes one turned value in a million to the e4m3
// code beside its own. Queries, which meet f16 or split bf16 next, have it in fp32.
__device__ __forceinline__ void rotary_angle(int position, int pair, double &c, double &s) {
    const double turns = static_cast<double>(position) * kRotaryTurns[pair];
    sincospi(2.0 * (turns - rint(turns)), &s, &c);
}
__device__ __forceinline__ void rotary_angle(int position, int pair, float &c, float &s) {
    const double turns = static_cast<double>(position) * kRotaryTurns[pair];
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
}

// e4m3 blocks: a block's scale is 2^e, the smallest with amax <= 448 * 2^e. With
// 448 = 1.75 * 2^8 that is amax's own exponent - 8, or - 7 where its significand is
// over 1.75: two integer operations on the bits, exact. Zero and amax under 2^-102
// (and no finite value at all) give the least exponent, so that scale and
// 1 / scale stay normal numbers.
constexpr int kScaleMinExp = -110;
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e > kScaleMinExp ? e : kScaleMinExp;
}
// 2^e as fp32, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Exponent of a scale that this library wrote; anything else (zero, a sign, a
// NaN) is read by its exponent bits alone, inside the range of the ones written.
__device__ __forceinline__ int exponent_of_scale(float scale) {
    const int e = static_cast<int>((__float_as_uint(scale) >> 23) & 0xFFu) - 127;
    return e < kScaleMinExp ? kScaleMinExp : (e > 120 ? 120 : e);
}
// Two fp32 values as e4m3 codes (low byte the first), round to nearest even. Callers
// pass |x| <= 448 or a NaN, so nothing saturates.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;  // a NaN fails the comparison too
}
__device__ __forceinline__ float finite_or_nan(float x) {
    return fabsf(x) <= 3.402823466e38f ? x : __uint_as_float(0x7FFFFFFFu);
}

// The 16-key blocks of a sequence that its query (position len - 1) sees: the blocks of
// the sinks outside the window, then those from the window's first key on.
struct VisibleBlocks {
    int len, lo, sink_end;  // keys seen: pos in [lo, len) or pos < sink_end
    int n_sink, first, n;   // sink blocks; first block after them; blocks in all
    __device__ __forceinline__ int block(int i) const { return i < n_sink ? i : first + (i - n_sink); }
    __device__ __forceinline__ bool sees(int pos) const { return (pos >= lo && pos < len) || pos < sink_end; }
    __device__ __forceinline__ bool partial(int blk) const {  // some key of the block is not seen
        const int a = blk * 16, b = a + 16;
        return !((a >= lo && b <= len) || b <= sink_end);
    }
};
__device__ __forceinline__ VisibleBlocks visible_blocks(int len, int max_seqlen_k, int window, int sinks) {
    VisibleBlocks v;
    v.len = (len >= 1 && len <= max_seqlen_k) ? len : 0;
    v.lo = (window > 0) ? max(0, v.len - window) : 0;
    v.sink_end = min(sinks, v.lo);  // window <= 0 leaves lo = 0 and so none
    v.n_sink = (v.sink_end + 15) / 16;
    v.first = max(v.lo / 16, v.n_sink);
    v.n = v.n_sink + max(0, (v.len + 15) / 16 - v.first);
    return v;
}

}  // namespace gdla
