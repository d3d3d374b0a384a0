// hc_token_sums.cuh -- sums of many per-thread values over a CTA: warp trees
// in fp32, then the warps in order in fp64. The order is fixed by the launch
// shape, so results are reproducible.
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

}  // namespace hc
