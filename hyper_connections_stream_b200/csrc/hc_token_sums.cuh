// hc_token_sums.cuh -- sums of many per-thread values over a warp, as trees in
// fp32; the kernels add the warps' sums in a fixed order. The order follows from
// the launch shape, so results are reproducible.
#pragma once

#include "hc_backward_common.cuh"

namespace hc {

// dst[v] = the warp's sum of v[v], for any number of values (32 an exchange).
template <int NV, int B = 0>
__device__ __forceinline__ void warp_sums_all(const float (&v)[NV], float *dst, int lane) {
    constexpr int M = NV - B < 32 ? NV - B : 32;
    float w[M];
#pragma unroll
    for (int m = 0; m < M; ++m) w[m] = v[B + m];
    bw_warp_sums_to<M>(w, dst + B, lane);
    if constexpr (B + M < NV) warp_sums_all<NV, B + M>(v, dst, lane);
}

// Warp sums of M values (at most 32); put(m, sum) is called for each by one
// lane. The exchange of bw_warp_sums_to with a free destination.
template <int M, typename Put>
__device__ __forceinline__ void warp_sums_put(const float (&v)[M], int lane, Put &&put) {
    static_assert(M <= 32, "at most 32 values per exchange");
    constexpr int P = bw_pow2_ceil(M);
    float w[P];
#pragma unroll
    for (int m = 0; m < P; ++m) w[m] = m < M ? v[m] : 0.0f;
    int o = 16;
#pragma unroll
    for (int h = P / 2; h >= 1; h /= 2) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int m = 0; m < h; ++m) {
            const float send = up ? w[m] : w[m + h];
            const float keep = up ? w[m + h] : w[m];
            w[m] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
        o >>= 1;
    }
    float s = w[0];
#pragma unroll
    for (; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    constexpr int span = 32 / P;
    const int idx = lane / span;
    if (lane % span == 0 && idx < M) put(idx, s);
}

// (m + eps)^(-1/2) of a mean square m; NaN where m is not finite (a row that
// holds an infinity, or whose squares overflow, has no norm: its inverse is not
// to pass for 0).
__device__ __forceinline__ float inv_norm(float m, float eps) {
    return m < INFINITY ? __frsqrt_rn(m + eps) : m - m;
}

// Sum of 16 floats in shared memory (16-byte aligned).
__device__ __forceinline__ float sum16(const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    const float4 c = *reinterpret_cast<const float4 *>(p + 8), e = *reinterpret_cast<const float4 *>(p + 12);
    return (((a.x + b.x) + (a.y + b.y)) + ((a.z + b.z) + (a.w + b.w))) +
           (((c.x + e.x) + (c.y + e.y)) + ((c.z + e.z) + (c.w + e.w)));
}

}  // namespace hc
