// hc_checkpoint_backward.cu -- backward of the fused HC step from the 8-bit
// checkpoint of its H and y.
//
// The gradients of  H'_j = sum_i A_ij H_i + b_j y,  h = sum_j a_j H'_j,
// x = h r g,  r = (mean h^2 + eps)^(-1/2)  at the checkpoint's values, H' not
// rounded. With H' linear in H and y so is h, and everything that multiplies
// them can be summed before the token's statistic is known:
//   h    = sum_i c_i H_i + c_y y,      c_i = sum_j A_ij a_j, c_y = sum_j a_j b_j
//   u    = g dx,   dh = r u - k z,     z = r h,  k = r mean(u z)
//   P_i  = <dh, H_i> = r <u, H_i> - k (r <h, H_i>),   P_y likewise with y
//   dA_ij = <H_i, dH'_j> + a_j P_i     db_j = <y, dH'_j> + a_j P_y
//   da_j  = sum_i A_ij P_i + b_j P_y   dg = sum_t dx z
//   dH_i = sum_j A_ij dH'_j + c_i dh   dy = sum_j b_j dH'_j + c_y dh
// So the first pass over a token takes n^2 + 3n + 4 sums and the checkpoint is
// read there only; the second needs dH', dx and h. Against taking the sums
// after dh is known (H and y read and decoded twice, n^2 + n products each to
// rebuild H') this leaves about half the arithmetic.
//
// hc_ck_bwd_ring_kernel (hc_checkpoint_ring.cuh) takes long rows of up to four
// streams. hc_ck_bwd_kernel, here, takes the rest: a CTA takes a token at a
// time; threads own column slices of 16 bytes of dH'. dH' and dx are read again
// from L2 in the second pass, h is parked in shared memory (fp32; rebuilt from
// the checkpoint where a row does not fit). The gain gradient accumulates in the
// CTA's workspace row. All sums are fp32: a row whose squares overflow it has no
// norm, and NaN gradients (hc_checkpoint_ring.cuh).
//
// Measured: n = 8, T = 2048, d = 4096, bf16 in 181 us with the parameter kernels
// (152 us of its own under the profiler, 42 % of the issue slots at eight warps
// of 255 registers); n = 4, T = 16384, d = 7168 in 894 us, which the ring does in
// 695 (65 % of the copy rate). At n = 4 the direct kernel is held by latency: 14 warps of 128 registers on a multiprocessor at n = 4, 39 %
// of the issue slots and of the FMA pipes used, 99 instructions a column. What
// did not help there: staging slices with cp.async (930 to 995), dH' and dx kept
// in shared memory for the second pass (909), slices of half the width at 80
// registers and three CTAs (1054: half as many instructions again). The prefetch
// into L2 gains 16 % at n = 8, where one CTA has a multiprocessor to itself.
#include <atomic>

#include "hc_checkpoint_ring.cuh"
#include "hc_launch.h"

namespace hc {

namespace {

constexpr int kThreads = 256;
constexpr int kTB = 32;  // parameter slots per batch

// Ask for `bytes` at p to be brought into L2 (both multiples of 16).
__device__ __forceinline__ void prefetch_l2(const void *p, int64_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)bytes) : "memory");
}

template <int N, typename S, bool PARK>
__global__ void __launch_bounds__(kThreads, (N <= 4 ? 2 : 1))
hc_ck_bwd_kernel(CkBwParams bp) {
    const StepParams &p = bp.f;
    constexpr int V = StorageTraits<S>::V, VP = V / 2, NN = N * N;
    using Q = CkSums<N>;
    constexpr int NV = Q::COUNT, NW = kThreads / 32;
    __shared__ float sA[kTB * NN], sb[kTB * N], sa[kTB * N], sc[kTB * (N + 1)];
    // of alternate tokens: the warps' sums, and their two statistics side by side
    __shared__ float red[2][NW * NV];
    __shared__ __align__(16) float stat[2][2][8];
    __shared__ float fin[NV];
    static_assert(NW <= 8, "the statistics of eight warps");
    __shared__ float swork[NW * kGroupScratch];
    extern __shared__ __align__(16) float shp[];  // [d] parked h

    const int tid = threadIdx.x, NT = blockDim.x, nwarps = NT >> 5;
    const int lane = tid & 31, warp = tid >> 5;
    const int64_t G = gridDim.x;
    const int d = (int)p.d, ns = (int)bp.ns;  // columns and a token's rows fit 32 bits
    int TB = nwarps * Group<N>::TPW;
    TB = TB < kTB ? TB : kTB;
    const float inv_d = 1.0f / (float)d;
    const uint8_t *QH = static_cast<const uint8_t *>(p.H), *QY = static_cast<const uint8_t *>(p.y);
    const S *DX = static_cast<const S *>(bp.dx), *DHO = static_cast<const S *>(bp.dHout);
    S *DH = static_cast<S *>(bp.dH), *DY = static_cast<S *>(bp.dy);
    float *sdg = bp.dg_part ? bp.dg_part + (int64_t)blockIdx.x * d : nullptr;
    if (sdg)
        for (int k = tid * V; k < d; k += NT * V) {
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<float4 *>(sdg + k + e) = make_float4(0.f, 0.f, 0.f, 0.f);
        }

    if (tid < 32) (&stat[0][0][0])[tid] = 0.0f;
    int par = 0, turn = 0;
    for (int64_t m0 = 0;; m0 += TB) {
        const int64_t first = blockIdx.x + m0 * G;
        if (first >= p.T) break;
        __syncthreads();  // previous batch's parameters no longer read
        prepare_params<N, true, true>(p, first, G, TB, sA, sb, sa, swork);
        __syncthreads();
        for (int v = tid; v < TB * (N + 1); v += NT) {
            const int tt = v / (N + 1), i = v - tt * (N + 1);
            if (first + (int64_t)tt * G >= p.T) continue;
            float c = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j)
                c = __fmaf_rn(i < N ? sA[tt * NN + i * N + j] : sb[tt * N + j], sa[tt * N + j], c);
            sc[v] = c;
        }
        __syncthreads();
        for (int tt = 0; tt < TB; ++tt) {
            const int64_t t = first + (int64_t)tt * G;
            if (t >= p.T) break;  // uniform over the CTA
            const float *At = sA + tt * NN, *bt = sb + tt * N, *at = sa + tt * N, *ct = sc + tt * (N + 1);
            // the next token's rows into L2 while this one is worked on: the
            // first pass then waits for L2, not for DRAM
            if (tid == 0 && t + G < p.T && d % 16 == 0) {
                const int64_t u = t + G;
                if (DHO) prefetch_l2(DHO + u * N * d, N * d * (int64_t)sizeof(S));
                prefetch_l2(DX + u * d, d * (int64_t)sizeof(S));
                prefetch_l2(QH + u * N * d, N * d);
                prefetch_l2(QY + u * d, d);
                prefetch_l2(bp.sH + u * N * bp.ns, N * bp.ns);
                prefetch_l2(bp.sy + u * bp.ns, bp.ns);
            }

            const uint8_t *QHt = QH + t * N * d, *QYt = QY + t * d;
            const uint8_t *EHt = bp.sH + t * N * ns, *EYt = bp.sy + t * ns;
            const S *DHOt = DHO ? DHO + t * N * d : nullptr, *DXt = DX + t * d;
            S *DHt = DH + t * N * d, *DYt = DY + t * d;

            // the checkpoint's values of slice k: H rows, then y
            auto load_kept = [&](int k, float2 (&hv)[N + 1][VP]) {
                uint32_t q[N + 1][V / 4], e[N + 1];
#pragma unroll
                for (int i = 0; i <= N; ++i) {
                    ck_load<V>(i < N ? QHt + (i * d + k) : QYt + k, q[i]);
                    e[i] = __ldg(i < N ? EHt + (i * ns + k / kCkBlock) : EYt + k / kCkBlock);
                }
#pragma unroll
                for (int i = 0; i <= N; ++i) ck_decode<VP>(q[i], ck_scale(e[i]), hv[i]);
            };
            auto mix_h = [&](const float2 (&hv)[N + 1][VP], float2 (&h)[VP]) {
#pragma unroll
                for (int e = 0; e < VP; ++e) h[e] = fmul2_rn(make_float2(ct[0], ct[0]), hv[0][e]);
#pragma unroll
                for (int i = 1; i <= N; ++i)
#pragma unroll
                    for (int e = 0; e < VP; ++e) h[e] = ffma2_rn(make_float2(ct[i], ct[i]), hv[i][e], h[e]);
            };

            // ---- pass 1: the token's sums ----
            float acc[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] = 0.0f;
            for (int k = tid * V; k < d; k += NT * V) {
                float2 hv[N + 1][VP], h[VP], u[VP], gv[VP];
                load_kept(k, hv);
                ck_widen(__ldg(reinterpret_cast<const uint4 *>(DXt + k)), u);
                load_gain2<VP>(p.g, k, gv);
#pragma unroll
                for (int e = 0; e < VP; ++e) u[e] = fmul2_rn(u[e], gv[e]);
                mix_h(hv, h);
                if constexpr (PARK) {
#pragma unroll
                    for (int e = 0; e < VP; e += 2)
                        *reinterpret_cast<float4 *>(shp + k + 2 * e) =
                            make_float4(h[e].x, h[e].y, h[e + 1].x, h[e + 1].y);
                }
                // a slice's product is summed in pairs, then added to the thread's sum
                auto dot = [&](const float2 (&x)[VP], const float2 (&y)[VP], float &s) {
                    float2 z = fmul2_rn(x[0], y[0]);
#pragma unroll
                    for (int e = 1; e < VP; ++e) z = ffma2_rn(x[e], y[e], z);
                    s += z.x + z.y;
                };
#pragma unroll
                for (int i = 0; i <= N; ++i) {
                    dot(u, hv[i], acc[Q::U + i]);
                    dot(h, hv[i], acc[Q::H + i]);
                }
                dot(h, h, acc[Q::SS]);
                dot(u, h, acc[Q::SG]);
                if (DHO) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float2 gr[VP];
                        ck_widen(__ldg(reinterpret_cast<const uint4 *>(DHOt + (j * d + k))), gr);
#pragma unroll
                        for (int i = 0; i < N; ++i) dot(hv[i], gr, acc[i * N + j]);
                        dot(hv[N], gr, acc[Q::B + j]);
                    }
                }
            }
            ck_means<N>(acc, inv_d);
            warp_sums_all<NV>(acc, red[par] + warp * NV, lane);
            __syncwarp();
            if (lane < 2) stat[par][lane][warp] = red[par][warp * NV + Q::SS + lane];
            __syncthreads();
            float tot[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 f = *reinterpret_cast<const float4 *>(&stat[par][x][0]);
                const float4 h4 = *reinterpret_cast<const float4 *>(&stat[par][x][4]);
                tot[x] = ((f.x + h4.x) + (f.y + h4.y)) + ((f.z + h4.z) + (f.w + h4.w));
            }
            const CkStat sv = ck_stat(tot[0], tot[1], p.eps);

            // ---- pass 2: the gradients of H and y ----
            const float2 r2 = make_float2(sv.r, sv.r), nk2 = make_float2(-sv.k, -sv.k);
            for (int k = tid * V; k < d; k += NT * V) {
                float2 dx[VP], gv[VP], h[VP], dh[VP];
                ck_widen(__ldcs(reinterpret_cast<const uint4 *>(DXt + k)), dx);
                load_gain2<VP>(p.g, k, gv);
                if constexpr (PARK) {
#pragma unroll
                    for (int e = 0; e < VP; e += 2) {
                        const float4 f = *reinterpret_cast<const float4 *>(shp + k + 2 * e);
                        h[e] = make_float2(f.x, f.y);
                        h[e + 1] = make_float2(f.z, f.w);
                    }
                } else {
                    float2 hv[N + 1][VP];
                    load_kept(k, hv);
                    mix_h(hv, h);
                }
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    h[e] = fmul2_rn(r2, h[e]);  // z
                    dh[e] = ffma2_rn(nk2, h[e], fmul2_rn(r2, fmul2_rn(dx[e], gv[e])));
                }
                if (sdg) {
#pragma unroll
                    for (int e = 0; e < VP; e += 2) {
                        float4 *pd = reinterpret_cast<float4 *>(sdg + k + 2 * e);
                        const float4 f = *pd;
                        const float2 s0 = ffma2_rn(dx[e], h[e], make_float2(f.x, f.y));
                        const float2 s1 = ffma2_rn(dx[e + 1], h[e + 1], make_float2(f.z, f.w));
                        *pd = make_float4(s0.x, s0.y, s1.x, s1.y);
                    }
                }
                float2 o[N + 1][VP];
#pragma unroll
                for (int i = 0; i <= N; ++i)
#pragma unroll
                    for (int e = 0; e < VP; ++e) o[i][e] = fmul2_rn(make_float2(ct[i], ct[i]), dh[e]);
                if (DHO) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float2 gr[VP];
                        ck_widen(__ldcs(reinterpret_cast<const uint4 *>(DHOt + (j * d + k))), gr);
#pragma unroll
                        for (int i = 0; i <= N; ++i) {
                            const float w = i < N ? At[i * N + j] : bt[j];
#pragma unroll
                            for (int e = 0; e < VP; ++e) o[i][e] = ffma2_rn(make_float2(w, w), gr[e], o[i][e]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    __stcs(reinterpret_cast<uint4 *>(DHt + (i * d + k)), ck_narrow(o[i]));
                __stcs(reinterpret_cast<uint4 *>(DYt + k), ck_narrow(o[N]));
            }
            if (warp == turn) {  // one warp a token, in turn, writes the parameter gradients
                for (int v = lane; v < Q::SS; v += 32) {
                    float a = 0.0f;
                    for (int w = 0; w < nwarps; ++w) a += red[par][w * NV + v];
                    fin[v] = a;
                }
                __syncwarp();
                ck_write_params<N, false>(fin, sv, (float)d, At, bt, at, bp.gA, bp.gb, bp.ga, t, lane);
            }
            turn = turn + 1 == nwarps ? 0 : turn + 1;
            par ^= 1;
        }
    }
}

template <int N, typename S>
struct CkBw {
    static constexpr int V = StorageTraits<S>::V;
    // The ring takes rows from 640 slices up, where ten warps have two full
    // slices a thread. Direct -> ring, 268 MB of values a call, n = 4: bf16 d =
    // 2048 251 -> 287, 4096 228 -> 235, 5120 252 -> 216, 7168 261 -> 199 us; fp32
    // d = 2048 162 -> 174, 2560 203 -> 156, 3840 224 -> 140 us; n = 2 and 3 alike.
    // With one fp32 stream a row is too little for one CTA a multiprocessor
    // (82 -> 95 us at 2560, 86 -> 88 at 3200). Beyond n = 4 a thread's sums
    // alone fill the registers.
    static constexpr int64_t kRingFrom = 640 * V;
    static constexpr bool RINGS = N <= 4 && !(N == 1 && V == 4);
    // The ring's geometry for rows of d; no stages where the direct kernel takes them.
    static CkRingShape ring(int64_t d, int64_t &smem) {
        CkRingShape sh{};
        if (!RINGS || d % 16 != 0 || d < kRingFrom) return sh;
        const int64_t nvec = d / V;
        const int64_t slices = (nvec + 32 * kCkWarps - 1) / (32 * kCkWarps);
        if (slices > kCkSlices) return sh;
        sh.gw = (int)((nvec + 32 * slices - 1) / (32 * slices));
        sh.stage_bytes = (N + 1) * (d * (int64_t)sizeof(S) + d + ck_scale_stride(d));
        int64_t nst = (kSmemLimitLogits - ck_ring_fixed_bytes<N>(0)) / (sh.stage_bytes + 16);
        if (nst < 2) return sh;
        if (nst > 4) nst = 4;
        sh.nst = (int)nst;
        smem = nst * sh.stage_bytes + ck_ring_fixed_bytes<N>((int)nst);
        return sh;
    }
    // Dynamic shared memory opted in once per device, at its most.
    static hc_status configure_ring(const LaunchCtx &ctx) {
        if constexpr (RINGS) {
            static std::atomic<bool> done[64];
            if (ctx.device < 0 || ctx.device >= 64)
                return set_error(HC_ERR_UNSUPPORTED, "device ordinal %d >= 64", ctx.device);
            if (done[ctx.device].load()) return HC_OK;
            const cudaError_t e = cudaFuncSetAttribute(
                hc_ck_bwd_ring_kernel<N, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimitLogits);
            if (e != cudaSuccess)
                return set_error(HC_ERR_CUDA, "checkpoint backward smem attribute: %s", cudaGetErrorString(e));
            done[ctx.device].store(true);
        }
        return HC_OK;
    }
    // h parked up to 96 KB of d: two CTAs a multiprocessor at n <= 4
    static bool parked(int64_t d) { return d * 4 <= 96 * 1024; }
    static int threads(int64_t d) {
        const int64_t nvec = d / V;
        int64_t nt = nvec < kThreads ? (nvec + 31) / 32 * 32 : kThreads;
        // a size that divides the row's slices, when one is near the largest
        for (int64_t c = nt; c >= nt / 2 && c >= 32 && nvec >= kThreads; c -= 32)
            if (nvec % c == 0) return (int)c;
        return (int)nt;
    }
    // Shared memory opted in once per device.
    template <bool PARK>
    static hc_status configure(const LaunchCtx &ctx) {
        static std::atomic<bool> done[64];
        if (ctx.device < 0 || ctx.device >= 64)
            return set_error(HC_ERR_UNSUPPORTED, "device ordinal %d >= 64", ctx.device);
        if (done[ctx.device].load()) return HC_OK;
        const cudaError_t e = cudaFuncSetAttribute(hc_ck_bwd_kernel<N, S, PARK>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
        if (e != cudaSuccess)
            return set_error(HC_ERR_CUDA, "checkpoint backward smem attribute: %s", cudaGetErrorString(e));
        done[ctx.device].store(true);
        return HC_OK;
    }
    static hc_status grid(int64_t T, int64_t d, const LaunchCtx &ctx, int64_t &grid) {
        int64_t smem = 0;
        if (ring(d, smem).nst) {
            grid = ctx.sms < T ? ctx.sms : T;
            return configure_ring(ctx);
        }
        const bool park = parked(d);
        const hc_status s = park ? configure<true>(ctx) : configure<false>(ctx);
        if (s != HC_OK) return s;
        grid = T;
        if (T <= ctx.sms) return HC_OK;
        int per_sm = 0;
        const int NT = threads(d);
        const cudaError_t e =
            park ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, hc_ck_bwd_kernel<N, S, true>, NT, (size_t)d * 4)
                 : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, hc_ck_bwd_kernel<N, S, false>, NT, 0);
        if (e != cudaSuccess)
            return set_error(HC_ERR_CUDA, "checkpoint backward occupancy: %s", cudaGetErrorString(e));
        const int64_t most = (int64_t)ctx.sms * (per_sm < 1 ? 1 : per_sm);
        if (grid > most) grid = most;
        return HC_OK;
    }
    static hc_status launch(const BackwardArgs &a, const uint8_t *sH, const uint8_t *sy, int64_t g,
                            const LaunchCtx &ctx, cudaStream_t st) {
        CkBwParams bp{};
        bp.f = a.f;
        bp.sH = sH;
        bp.sy = sy;
        bp.ns = ck_scale_stride(a.f.d);
        bp.dHout = a.dHout;
        bp.dx = a.dx;
        bp.dH = a.dH;
        bp.dy = a.dy;
        bp.gA = a.dA;
        bp.gb = a.db;
        bp.ga = a.da;
        bp.dg_part = a.dg ? static_cast<float *>(a.workspace) : nullptr;
        if constexpr (RINGS) {
            int64_t smem = 0;
            const CkRingShape sh = ring(a.f.d, smem);
            if (sh.nst) {
                hc_ck_bwd_ring_kernel<N, S><<<(unsigned)g, 32 * (2 + kCkWarps), (size_t)smem, st>>>(bp, sh, ctx.fault);
                const cudaError_t e = cudaGetLastError();
                if (e != cudaSuccess)
                    return set_error(HC_ERR_CUDA, "hc_ck_bwd_ring_kernel launch: %s", cudaGetErrorString(e));
                return HC_OK;
            }
        }
        const int NT = threads(a.f.d);
        if (parked(a.f.d)) hc_ck_bwd_kernel<N, S, true><<<(unsigned)g, NT, (size_t)a.f.d * 4, st>>>(bp);
        else hc_ck_bwd_kernel<N, S, false><<<(unsigned)g, NT, 0, st>>>(bp);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "hc_ck_bwd_kernel launch: %s", cudaGetErrorString(e));
        return HC_OK;
    }
};

template <int N>
hc_status grid_n(hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx, int64_t &g) {
    return dt == HC_BF16 ? CkBw<N, __nv_bfloat16>::grid(T, d, ctx, g) : CkBw<N, float>::grid(T, d, ctx, g);
}
template <int N>
hc_status launch_n(const BackwardArgs &a, const uint8_t *sH, const uint8_t *sy, int64_t g,
                   const LaunchCtx &ctx, cudaStream_t st) {
    return a.dt == HC_BF16 ? CkBw<N, __nv_bfloat16>::launch(a, sH, sy, g, ctx, st)
                           : CkBw<N, float>::launch(a, sH, sy, g, ctx, st);
}

hc_status grid_of(int n, hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx, int64_t &g) {
    switch (n) {
        case 1: return grid_n<1>(dt, T, d, ctx, g);
        case 2: return grid_n<2>(dt, T, d, ctx, g);
        case 3: return grid_n<3>(dt, T, d, ctx, g);
        case 4: return grid_n<4>(dt, T, d, ctx, g);
        case 5: return grid_n<5>(dt, T, d, ctx, g);
        case 6: return grid_n<6>(dt, T, d, ctx, g);
        case 7: return grid_n<7>(dt, T, d, ctx, g);
        default: return grid_n<8>(dt, T, d, ctx, g);
    }
}

}  // namespace

hc_status checkpoint_backward_workspace_bytes(int n, hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx,
                                              size_t *bytes) {
    int64_t g = 0;
    const hc_status s = grid_of(n, dt, T, d, ctx, g);
    if (s != HC_OK) return s;
    *bytes = (size_t)g * (size_t)d * sizeof(float);
    return HC_OK;
}

hc_status launch_checkpoint_backward(const BackwardArgs &a, const uint8_t *sH, const uint8_t *sy,
                                     const LaunchCtx &ctx, cudaStream_t st) {
    hc_status s = check_param_backward(a);
    if (s != HC_OK) return s;
    int64_t g = 0;
    s = grid_of(a.n, a.dt, a.f.T, a.f.d, ctx, g);
    if (s != HC_OK) return s;
    const size_t need = (size_t)g * (size_t)a.f.d * sizeof(float);
    if (a.dg && a.workspace_bytes < need)
        return set_error(HC_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed for dg", a.workspace_bytes, need);
    switch (a.n) {
        case 1: s = launch_n<1>(a, sH, sy, g, ctx, st); break;
        case 2: s = launch_n<2>(a, sH, sy, g, ctx, st); break;
        case 3: s = launch_n<3>(a, sH, sy, g, ctx, st); break;
        case 4: s = launch_n<4>(a, sH, sy, g, ctx, st); break;
        case 5: s = launch_n<5>(a, sH, sy, g, ctx, st); break;
        case 6: s = launch_n<6>(a, sH, sy, g, ctx, st); break;
        case 7: s = launch_n<7>(a, sH, sy, g, ctx, st); break;
        default: s = launch_n<8>(a, sH, sy, g, ctx, st); break;
    }
    if (s != HC_OK) return s;
    return launch_backward_tail(a, g, ctx, st);
}

}  // namespace hc
