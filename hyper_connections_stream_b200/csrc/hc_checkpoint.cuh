// hc_checkpoint.cuh -- the 8-bit stream checkpoint: e4m3 codes with one power
// of two per block of 32 values along d.
//
// For a block with largest finite magnitude m the scale is 2^e, e the smallest
// exponent with m / 2^e <= 448 (the largest e4m3 value), at least -126; a code
// is e4m3(x / 2^e), rounded to nearest even. Scaling by a power of two is
// exact, so the only rounding is the code's own (half a step: 2^-4 of the
// value while it stays above 2^-14 of the block's scale range), no value
// saturates, and the kept value code * 2^e is exact in bf16 as well as in
// fp32 (all but one: values from 1.9375 * 2^127 up round to 2^128, which both
// types hold as infinity). The exponent is stored biased by 127 in one byte (E8M0), 1 .. 247.
// A value that is not finite is kept as NaN and leaves its block's scale alone.
//
// Rows: codes [rows][d]; exponents [rows][ck_scale_stride(d)], the rows padded
// to 16 bytes so that a token's exponents can be moved by one bulk copy (bytes
// past the last block are neither written nor read).
#pragma once

#include <cuda_fp16.h>

#include "hc_device.cuh"

namespace hc {

constexpr int kCkBlock = 32;

__host__ __device__ constexpr int64_t ck_blocks(int64_t d) { return (d + kCkBlock - 1) / kCkBlock; }
__host__ __device__ constexpr int64_t ck_scale_stride(int64_t d) { return (ck_blocks(d) + 15) / 16 * 16; }

// Biased exponent for a block whose largest finite |x| has these fp32 bits:
// 448 = 1.75 * 2^8, so the exponent of m less 8, one more when m's mantissa is
// above 0.75.
__device__ __forceinline__ uint32_t ck_exponent(uint32_t amax_bits) {
    const int e = (int)((amax_bits + 0x1fffffu) >> 23) - 8;
    return (uint32_t)(e > 1 ? e : 1);
}
__device__ __forceinline__ float ck_scale(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float ck_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Two codes (element 0 in the low byte) of values already divided by the
// scale; NaN becomes NaN, an infinity 448.
__device__ __forceinline__ uint32_t ck_encode2(float2 x) {
    uint16_t q;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(x.y), "f"(x.x));
    return q;
}
// The two values (before scaling) of the codes in the low 16 bits.
__device__ __forceinline__ float2 ck_decode2(uint32_t q) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)q));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// fp32 bits of |x|, 0 where x is not finite.
__device__ __forceinline__ uint32_t ck_finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}

// The codes of VP pairs of one thread. The 32 / (2 VP) neighbouring lanes that
// share a block exchange their maxima, so all lanes of the warp call this
// together (a lane past the row's end passes zeros); e receives the block's
// biased exponent. Word w of q holds elements 4 w .. 4 w + 3. The floating
// maximum passes over NaN; an infinity (or nothing but NaN) shows in it.
template <int VP>
__device__ __forceinline__ void ck_encode(const float2 (&v)[VP], uint32_t (&q)[(VP + 1) / 2], uint32_t &e) {
    float mf = fmaxf(fabsf(v[0].x), fabsf(v[0].y));
#pragma unroll
    for (int p = 1; p < VP; ++p) mf = fmaxf(mf, fmaxf(fabsf(v[p].x), fabsf(v[p].y)));
    uint32_t m = __float_as_uint(mf) & 0x7fffffffu;
    float2 w[VP];
#pragma unroll
    for (int p = 0; p < VP; ++p) w[p] = v[p];
    if (__any_sync(0xffffffffu, m >= 0x7f800000u)) {  // rare: infinities become NaN and leave the maximum
        m = 0;
#pragma unroll
        for (int p = 0; p < VP; ++p) {
            m = max(m, max(ck_finite_bits(v[p].x), ck_finite_bits(v[p].y)));
            w[p] = ffma2_rn(v[p], make_float2(0.0f, 0.0f), v[p]);  // x * 0 + x: x, or NaN for an infinity
        }
    }
#pragma unroll
    for (int o = kCkBlock / (4 * VP); o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    e = ck_exponent(m);
    const float inv = ck_inverse(e);
    const float2 i2 = make_float2(inv, inv);
#pragma unroll
    for (int p = 0; p < VP; p += 2) {
        q[p / 2] = ck_encode2(fmul2_rn(w[p], i2));
        if (p + 1 < VP) q[p / 2] |= ck_encode2(fmul2_rn(w[p + 1], i2)) << 16;
    }
}

// The kept values of VP pairs: codes in words as above, scale 2^(e - 127).
template <int VP>
__device__ __forceinline__ void ck_decode(const uint32_t (&q)[(VP + 1) / 2], float scale, float2 (&v)[VP]) {
    const float2 s2 = make_float2(scale, scale);
#pragma unroll
    for (int p = 0; p < VP; ++p) v[p] = fmul2_rn(ck_decode2(q[p / 2] >> (p % 2 * 16)), s2);
}

// One thread's V = 8 or 4 codes at p (aligned to V bytes).
template <int V>
__device__ __forceinline__ void ck_load(const uint8_t *p, uint32_t (&q)[V / 4]) {
    if constexpr (V == 8) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
        q[0] = w.x;
        q[1] = w.y;
    } else {
        q[0] = __ldcs(reinterpret_cast<const unsigned int *>(p));
    }
}
template <int V>
__device__ __forceinline__ void ck_store(uint8_t *p, const uint32_t (&q)[V / 4]) {
    if constexpr (V == 8) __stcs(reinterpret_cast<uint2 *>(p), make_uint2(q[0], q[1]));
    else __stcs(reinterpret_cast<unsigned int *>(p), q[0]);
}

// Keep VP pairs at column k of a row (codes at q, exponents at s), called by
// the whole warp; lanes past the row's end pass in = false.
template <int VP>
__device__ __forceinline__ void ck_keep(const float2 (&v)[VP], bool in, uint8_t *q, uint8_t *s, int64_t k, int lane) {
    float2 w[VP];
#pragma unroll
    for (int p = 0; p < VP; ++p) w[p] = in ? v[p] : make_float2(0.0f, 0.0f);
    uint32_t c[(VP + 1) / 2], e;
    ck_encode<VP>(w, c, e);
    if (in) {
        ck_store<2 * VP>(q + k, c);
        if (lane % (kCkBlock / (2 * VP)) == 0) s[k / kCkBlock] = (uint8_t)e;
    }
}

// Storage values as fp32 pairs: 16 bytes (V elements) to and from global memory.
__device__ __forceinline__ void ck_widen(uint4 q, float2 (&v)[4]) {
    widen_bf16x2(q.x, v[0].x, v[0].y);
    widen_bf16x2(q.y, v[1].x, v[1].y);
    widen_bf16x2(q.z, v[2].x, v[2].y);
    widen_bf16x2(q.w, v[3].x, v[3].y);
}
__device__ __forceinline__ void ck_widen(uint4 q, float2 (&v)[2]) {
    v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ uint4 ck_narrow(const float2 (&v)[4]) {
    return make_uint4(pack_bf16x2_rn(v[0].x, v[0].y), pack_bf16x2_rn(v[1].x, v[1].y),
                      pack_bf16x2_rn(v[2].x, v[2].y), pack_bf16x2_rn(v[3].x, v[3].y));
}
__device__ __forceinline__ uint4 ck_narrow(const float2 (&v)[2]) {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
}
template <int VP>
__device__ __forceinline__ void load_gain2(const float *g, int64_t k, float2 (&gv)[VP]) {
    if (g == nullptr) {
#pragma unroll
        for (int p = 0; p < VP; ++p) gv[p] = make_float2(1.0f, 1.0f);
        return;
    }
#pragma unroll
    for (int p = 0; p < VP; p += 2) {
        const float4 q = __ldg(reinterpret_cast<const float4 *>(g + k + 2 * p));
        gv[p] = make_float2(q.x, q.y);
        gv[p + 1] = make_float2(q.z, q.w);
    }
}

}  // namespace hc
