// hc_checkpoint_ring.cuh -- backward of the fused HC step from its 8-bit
// checkpoint, fed by bulk copies (the formulas are in
// hc_checkpoint_backward.cu), and the pieces it shares with the direct kernel.
//
// One CTA per SM: a producer lane moves whole tokens (the rows of dH', dx, and
// the checkpoint's codes and exponents: 109 KB at n = 4, d = 7168, bf16) into
// a ring of stages with one bulk copy a tensor, a warp prepares the tokens'
// parameters ahead, and up to ten consumer warps (with the other two, 168
// registers a thread: the n^2 + 3n + 4 sums and a slice of every row fit
// without spilling) take the CTA's tokens in turn. Both passes read the stage,
// so nothing is read from global memory twice, and the next token's copies are
// in flight all the while. A thread owns up to three slices of 16 bytes of dH';
// between the passes it keeps h in the slices' own code bytes (the codes of
// four rows are as many floats), which only it reads, or in registers where
// n < 3, and the gain gradient in registers. The two statistics of a token are
// exchanged first; the other sums follow behind that wait.
//
// Measured: n = 4, T = 16384, d = 7168, bf16, Sinkhorn in 695 us with the
// parameter kernels (65 % of the copy rate); bound by latency, half the issue
// slots used. Fourteen warps of 128 registers spilled and took 813 us where this
// split took 733 (timed in turn, before the groups of warps became one).
//
// Every wait is bounded (hc_sync.cuh): on time-out the CTA records a fault
// code, stops, drains the copies it issued and exits.
#pragma once

#include "hc_checkpoint.cuh"
#include "hc_pipe_kernels.cuh"
#include "hc_token_sums.cuh"

namespace hc {

struct CkBwParams {
    StepParams f;          // H and y hold the codes
    const uint8_t *sH, *sy;
    int64_t ns;            // exponent bytes per row
    const void *dHout, *dx;
    void *dH, *dy;
    float *gA, *gb, *ga;   // per-token sums (w.r.t. the matrix and the weights)
    float *dg_part;        // [gridDim.x][d] or null
};

// Sums of a token, in this order: dA [n][n], db [n], <u, H_i> and <u, y>
// [n + 1], <h, H_i> and <h, y> [n + 1], sum h^2, sum u h. The products with h
// leave a thread divided by d: a mean fits fp32 wherever a thread's own columns
// do (|h| to 1e18), the sum over a row would not.
template <int N> struct CkSums {
    static constexpr int B = N * N, U = B + N, H = U + N + 1, SS = H + N + 1, SG = SS + 1, COUNT = SG + 1;
};

template <int N>
__device__ __forceinline__ void ck_means(float (&acc)[CkSums<N>::COUNT], float inv_d) {
#pragma unroll
    for (int x = CkSums<N>::H; x < CkSums<N>::COUNT; ++x) acc[x] *= inv_d;
}

// A token's two statistics from mean h^2 and mean(u h): r = (mean h^2 +
// eps)^(-1/2) and k = r mean(u z) with z = r h, so that dh = r u - k z. z and u z
// are of ordinary size however far h is from 1; r^3, which dh = r u - (r^3
// mean(u h)) h would take, leaves fp32's range below |h| = 1e-13 and above 1e12.
struct CkStat {
    float r, k;
};
__device__ __forceinline__ CkStat ck_stat(float mean_hh, float mean_uh, float eps) {
    const float r = inv_norm(mean_hh, eps);
    return {r, r * (r * mean_uh)};
}

// The token's parameter gradients from its sums (one warp). TR: At holds A
// transposed.
template <int N, bool TR>
__device__ __forceinline__ void ck_write_params(const float *fin, CkStat st, float d, const float *At,
                                                const float *bt, const float *at, float *gA, float *gb, float *ga,
                                                int64_t t, int lane) {
    using Q = CkSums<N>;
    // <dh, row x>
    auto along = [&](int x) { return st.r * fin[Q::U + x] - st.k * (st.r * fin[Q::H + x] * d); };
    for (int e = lane; e < N * N; e += 32) {
        const int i = e / N, j = e - i * N;
        gA[t * (N * N) + e] = fin[e] + at[j] * along(i);
    }
    if (lane < N) {
        const float py = along(N);
        gb[t * N + lane] = fin[Q::B + lane] + at[lane] * py;
        float s = bt[lane] * py;
#pragma unroll
        for (int i = 0; i < N; ++i) s += At[TR ? lane * N + i : i * N + lane] * along(i);
        ga[t * N + lane] = s;
    }
    __syncwarp();
}

// Geometry: gw consumer warps of kCkWarps, nst stages.
struct CkRingShape {
    int gw, nst;
    int64_t stage_bytes;
};
constexpr int kCkWarps = 10;   // consumer warps at most
constexpr int kCkSlices = 3;   // slices a thread at most
constexpr int kCkStat = 16;    // the warps' statistics, padded
__host__ __device__ constexpr int ck_ring_slots(int n) {  // parameter slots, a power of two
    return 2 * pipe_param_batch(n) > 16 ? 2 * pipe_param_batch(n) : 16;
}
// Shared memory behind the stages: barriers, parameter slots, sums, abort flag
// and the parameter warp's scratch.
template <int N>
__host__ __device__ constexpr int64_t ck_ring_fixed_bytes(int stages) {
    return (int64_t)stages * 16 + ck_ring_slots(N) * 16 + 32                       // barriers
           + (ck_ring_slots(N) * (N * N + 2 * N) + 3) / 4 * 16                     // slots
           + (CkSums<N>::COUNT + 3) / 4 * 16                                       // a token's sums
           + 4 * kCkStat * 4                                                       // statistics
           + (kCkWarps * CkSums<N>::COUNT + 3) / 4 * 16                            // warps' sums
           + 16 + pipe_param_replicas(N) * kGroupScratch * 4;
}

// s += <x, y>, columns in order.
template <int VP>
__device__ __forceinline__ void ck_dot(float &s, const float2 (&x)[VP], const float2 (&y)[VP]) {
#pragma unroll
    for (int e = 0; e < VP; ++e) s = __fmaf_rn(x[e].y, y[e].y, __fmaf_rn(x[e].x, y[e].x, s));
}

// Warps kCkWarps and kCkWarps + 1 are the producer and the parameter warp.
template <int N, typename S>
__global__ void __launch_bounds__(32 * (2 + kCkWarps), 1)
hc_ck_bwd_ring_kernel(CkBwParams bp, CkRingShape sh, int *fault) {
    const StepParams &p = bp.f;
    constexpr int V = StorageTraits<S>::V, VP = V / 2, NN = N * N, CPT = kCkSlices, CW = kCkWarps;
    constexpr int PSG = ck_ring_slots(N), PSTRIDE = NN + 2 * N;
    constexpr bool IN_CODES = N >= 3;  // four rows of codes hold a slice's h
    using Q = CkSums<N>;
    constexpr int NV = Q::COUNT;
    const int64_t d = p.d;
    const int GW = sh.gw, nst = sh.nst;
    const bool grad = bp.dHout != nullptr;

    extern __shared__ __align__(128) unsigned char smem[];
    const int64_t rb = d * (int64_t)sizeof(S);  // bytes of a row of dH'
    const int64_t o_dx = N * rb, o_qh = o_dx + rb, o_qy = o_qh + N * d, o_sh = o_qy + d, o_sy = o_sh + N * bp.ns;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + nst * sh.stage_bytes);
    uint64_t *empty = full + nst;
    uint64_t *pfull = empty + nst;
    uint64_t *pempty = pfull + PSG;
    uint64_t *statbar = pempty + PSG;  // a token's statistics are all there
    uint64_t *sumbar = statbar + 1;   // its other sums are
    uint64_t *sumfree = sumbar + 1;    // and have been read
    float *params = reinterpret_cast<float *>(statbar + 4);
    float *fin = params + (PSG * PSTRIDE + 3) / 4 * 4;  // [NV]
    float *stat_all = fin + (NV + 3) / 4 * 4;           // [2][2][kCkStat]
    float *red = stat_all + 4 * kCkStat;                // [kCkWarps][NV]
    int *abort_word = reinterpret_cast<int *>(red + (kCkWarps * NV + 3) / 4 * 4);
    volatile int *abort_flag = abort_word;
    float *pscratch = reinterpret_cast<float *>(abort_word + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], GW);
        }
        for (int s = 0; s < PSG; ++s) {
            mbar_init(&pfull[s], 1);
            mbar_init(&pempty[s], GW);
        }
        mbar_init(statbar, GW);
        mbar_init(sumbar, GW);
        mbar_init(sumfree, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    for (int v = threadIdx.x; v < 4 * kCkStat; v += blockDim.x) stat_all[v] = 0.0f;
    __syncthreads();
    const int64_t G = gridDim.x;
    const int64_t M = (p.T > (int64_t)blockIdx.x) ? (p.T - 1 - blockIdx.x) / G + 1 : 0;

    if (warp == CW) {
        // ---------------- producer ----------------
        if (lane != 0) return;
        const uint8_t *QH = static_cast<const uint8_t *>(p.H), *QY = static_cast<const uint8_t *>(p.y);
        const S *DX = static_cast<const S *>(bp.dx), *DHO = static_cast<const S *>(bp.dHout);
        const uint32_t bytes = (uint32_t)(sh.stage_bytes - (grad ? 0 : N * rb));
        int64_t m = 0;
        int s = 0;
        uint32_t ph = 1;  // parity of the stage's previous release
        for (; m < M; ++m) {
            if (m >= nst && !mbar_wait_bounded(&empty[s], ph, abort_flag, fault, FAULT_WAIT_EMPTY)) break;
            const int64_t t = blockIdx.x + m * G;
            unsigned char *st = smem + s * sh.stage_bytes;
            mbar_arrive_expect_tx(&full[s], bytes);
            bulk_load(st + o_qh, QH + t * N * d, (uint32_t)(N * d), &full[s]);
            bulk_load(st + o_qy, QY + t * d, (uint32_t)d, &full[s]);
            bulk_load(st + o_sh, bp.sH + t * N * bp.ns, (uint32_t)(N * bp.ns), &full[s]);
            bulk_load(st + o_sy, bp.sy + t * bp.ns, (uint32_t)bp.ns, &full[s]);
            bulk_load(st + o_dx, DX + t * d, (uint32_t)rb, &full[s]);
            if (grad) bulk_load(st, DHO + t * N * d, (uint32_t)(N * rb), &full[s]);
            if (++s == nst) {
                s = 0;
                ph ^= 1u;
            }
        }
        // every issued copy lands before the CTA may exit (normally already done)
        for (int64_t q = (m > nst ? m - nst : 0); q < m; ++q)
            mbar_wait_drain(&full[(int)(q % nst)], (uint32_t)((q / nst) & 1), fault);
        return;
    }
    if (warp == CW + 1) {
        pipe_param_warp<N, true, true, 1, PSG>(p, M, G, params, pfull, pempty, pscratch, abort_flag, fault, lane);
        return;
    }

    // ---------------- consumers ----------------
    // offsets inside a stage and columns fit 32 bits (a stage is below 227 KB)
    const int gw = warp;
    if (gw >= GW) return;
    const int di = (int)d, nsi = (int)bp.ns, rbi = (int)rb;
    const int oq = (int)o_qh, os = (int)o_sh, odx = (int)o_dx;
    const int k0 = threadIdx.x * V, kstep = GW * 32 * V;  // first column, columns between a thread's slices
    S *DH = static_cast<S *>(bp.dH), *DY = static_cast<S *>(bp.dy);
    const float inv_d = 1.0f / (float)d;
    float2 dga[CPT][VP];
#pragma unroll
    for (int u = 0; u < CPT; ++u)
#pragma unroll
        for (int e = 0; e < VP; ++e) dga[u][e] = make_float2(0.0f, 0.0f);
    // the gains come from L2: asked for a slice ahead of their use
    float2 gv[VP];
    auto fetch_gain = [&](int u) {
        if (k0 + u * kstep < di) load_gain2<VP>(p.g, k0 + u * kstep, gv);
    };

    int s = 0, turn = 0;
    uint32_t ph = 0;  // stage and its parity
    for (int64_t m = 0; m < M; ++m) {
        const int64_t t = blockIdx.x + m * G;
        const int ps = (int)(m & (PSG - 1)), par = (int)(m & 1);
        fetch_gain(0);
        bool ok = mbar_wait_bounded(&pfull[ps], (uint32_t)((m / PSG) & 1), abort_flag, fault, FAULT_WAIT_PARAM);
        if (!__all_sync(0xffffffffu, ok)) break;
        // the slot holds A transposed (A[i][j] at j * N + i), then b, then a
        const float *P = params + ps * PSTRIDE, *bt = P + NN, *at = bt + N;
        float ct[N + 1];
#pragma unroll
        for (int x = 0; x <= N; ++x) {
            ct[x] = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) ct[x] = __fmaf_rn(x < N ? P[j * N + x] : bt[j], at[j], ct[x]);
        }
        ok = mbar_wait_bounded(&full[s], ph, abort_flag, fault, FAULT_WAIT_FULL);
        if (!__all_sync(0xffffffffu, ok)) break;
        unsigned char *st = smem + s * sh.stage_bytes;

        // ---- pass 1: the token's sums ----
        float acc[NV];
#pragma unroll
        for (int x = 0; x < NV; ++x) acc[x] = 0.0f;
        [[maybe_unused]] float2 hk[IN_CODES ? 1 : CPT][VP];
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int k = k0 + u * kstep;
            if (k < di) {
                float2 hv[N + 1][VP], h[VP], w[VP];
#pragma unroll
                for (int x = 0; x <= N; ++x) {  // y's codes and exponents follow H's
                    uint32_t q[V / 4];
                    if constexpr (V == 8) {
                        const uint2 c2 = *reinterpret_cast<const uint2 *>(st + oq + x * di + k);
                        q[0] = c2.x;
                        q[1] = c2.y;
                    } else {
                        q[0] = *reinterpret_cast<const uint32_t *>(st + oq + x * di + k);
                    }
                    ck_decode<VP>(q, ck_scale(st[os + x * nsi + k / kCkBlock]), hv[x]);
                }
#pragma unroll
                for (int x = 0; x <= N; ++x)
#pragma unroll
                    for (int e = 0; e < VP; ++e)
                        h[e] = x == 0 ? fmul2_rn(make_float2(ct[0], ct[0]), hv[0][e])
                                      : ffma2_rn(make_float2(ct[x], ct[x]), hv[x][e], h[e]);
                if constexpr (IN_CODES) {
                    if constexpr (V == 8) {
#pragma unroll
                        for (int e = 0; e < VP; ++e) *reinterpret_cast<float2 *>(st + oq + e * di + k) = h[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < VP; ++e) {
                            *reinterpret_cast<float *>(st + oq + 2 * e * di + k) = h[e].x;
                            *reinterpret_cast<float *>(st + oq + (2 * e + 1) * di + k) = h[e].y;
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VP; ++e) hk[u][e] = h[e];
                }
                ck_widen(*reinterpret_cast<const uint4 *>(st + odx + k * (int)sizeof(S)), w);
#pragma unroll
                for (int e = 0; e < VP; ++e) w[e] = fmul2_rn(w[e], gv[e]);
#pragma unroll
                for (int x = 0; x <= N; ++x) {
                    ck_dot<VP>(acc[Q::H + x], h, hv[x]);
                    ck_dot<VP>(acc[Q::U + x], w, hv[x]);
                }
                ck_dot<VP>(acc[Q::SS], h, h);
                ck_dot<VP>(acc[Q::SG], w, h);
                if (u + 1 < CPT) fetch_gain(u + 1);
                if (grad) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        ck_widen(*reinterpret_cast<const uint4 *>(st + j * rbi + k * (int)sizeof(S)), w);
#pragma unroll
                        for (int x = 0; x <= N; ++x) ck_dot<VP>(acc[x < N ? x * N + j : Q::B + j], hv[x], w);
                    }
                }
            }
        }
        fetch_gain(0);
        // h lies where the producer's next copy lands: order the proxies (here,
        // where no stores to global memory are outstanding)
        if constexpr (IN_CODES) fence_proxy_async_smem();
        ck_means<N>(acc, inv_d);
        // the two statistics first: the others' exchange overlaps the wait for them
        float *stat = stat_all + par * 2 * kCkStat;
        {
            float ss = acc[Q::SS], sg = acc[Q::SG];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                sg += __shfl_xor_sync(0xffffffffu, sg, o);
            }
            if (lane == 0) {
                stat[gw] = ss;
                stat[kCkStat + gw] = sg;
                mbar_arrive(statbar);
            }
        }
        if (m > 0) {  // the last token's sums have been read
            ok = mbar_wait_bounded(sumfree, (uint32_t)((m - 1) & 1), abort_flag, fault, FAULT_WAIT_REDUCE);
            if (!__all_sync(0xffffffffu, ok)) break;
        }
        {
            float v[Q::SS];
#pragma unroll
            for (int x = 0; x < Q::SS; ++x) v[x] = acc[x];
            warp_sums_all<Q::SS>(v, red + gw * NV, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sumbar);
        ok = mbar_wait_bounded(statbar, (uint32_t)(m & 1), abort_flag, fault, FAULT_WAIT_REDUCE);
        if (!__all_sync(0xffffffffu, ok)) break;
        float tot[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) tot[x] = sum16(stat + x * kCkStat);
        const CkStat sv = ck_stat(tot[0], tot[1], p.eps);

        // ---- pass 2: the gradients of H and y ----
        const float2 r2 = make_float2(sv.r, sv.r), nk2 = make_float2(-sv.k, -sv.k);
        S *DHt = DH + t * N * d, *DYt = DY + t * d;
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int k = k0 + u * kstep;
            if (k < di) {
                float2 dx[VP], h[VP], dh[VP];
                ck_widen(*reinterpret_cast<const uint4 *>(st + odx + k * (int)sizeof(S)), dx);
                if constexpr (IN_CODES) {
                    if constexpr (V == 8) {
#pragma unroll
                        for (int e = 0; e < VP; ++e) h[e] = *reinterpret_cast<const float2 *>(st + oq + e * di + k);
                    } else {
#pragma unroll
                        for (int e = 0; e < VP; ++e)
                            h[e] = make_float2(*reinterpret_cast<const float *>(st + oq + 2 * e * di + k),
                                               *reinterpret_cast<const float *>(st + oq + (2 * e + 1) * di + k));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VP; ++e) h[e] = hk[u][e];
                }
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    const float2 z = fmul2_rn(r2, h[e]);
                    dga[u][e] = ffma2_rn(dx[e], z, dga[u][e]);
                    dh[e] = ffma2_rn(nk2, z, fmul2_rn(r2, fmul2_rn(dx[e], gv[e])));
                }
                if (u + 1 < CPT) fetch_gain(u + 1);
                float2 o[N + 1][VP];
#pragma unroll
                for (int x = 0; x <= N; ++x)
#pragma unroll
                    for (int e = 0; e < VP; ++e) o[x][e] = fmul2_rn(make_float2(ct[x], ct[x]), dh[e]);
                if (grad) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float2 gr[VP];
                        ck_widen(*reinterpret_cast<const uint4 *>(st + j * rbi + k * (int)sizeof(S)), gr);
#pragma unroll
                        for (int x = 0; x <= N; ++x) {
                            const float w = x < N ? P[j * N + x] : bt[j];
#pragma unroll
                            for (int e = 0; e < VP; ++e) o[x][e] = ffma2_rn(make_float2(w, w), gr[e], o[x][e]);
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < N; ++x) __stcs(reinterpret_cast<uint4 *>(DHt + x * di + k), ck_narrow(o[x]));
                __stcs(reinterpret_cast<uint4 *>(DYt + k), ck_narrow(o[N]));
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        if (gw == turn) {  // one warp a token, in turn, writes the parameter gradients
            ok = mbar_wait_bounded(sumbar, (uint32_t)(m & 1), abort_flag, fault, FAULT_WAIT_REDUCE);
            if (!__all_sync(0xffffffffu, ok)) break;
            for (int v = lane; v < Q::SS; v += 32) {
                float a0 = 0.0f, a1 = 0.0f;
                for (int w = 0; w + 1 < GW; w += 2) {
                    a0 += red[w * NV + v];
                    a1 += red[(w + 1) * NV + v];
                }
                if (GW & 1) a0 += red[(GW - 1) * NV + v];
                fin[v] = a0 + a1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sumfree);
            ck_write_params<N, true>(fin, sv, (float)d, P, bt, at, bp.gA, bp.gb, bp.ga, t, lane);
        }
        if (lane == 0) mbar_arrive(&pempty[ps]);
        turn = turn + 1 == GW ? 0 : turn + 1;
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
    }
    if (bp.dg_part) {
        float *row = bp.dg_part + (int64_t)blockIdx.x * d;
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int k = k0 + u * kstep;
            if (k < di) {
#pragma unroll
                for (int e = 0; e < VP; e += 2)
                    *reinterpret_cast<float4 *>(row + k + 2 * e) =
                        make_float4(dga[u][e].x, dga[u][e].y, dga[u][e + 1].x, dga[u][e + 1].y);
            }
        }
    }
}

}  // namespace hc
