// hc_layernorm.cu -- the read with layer norm, and its gradients.
//
//   h = sum_i a_i H_i,  mu = mean h,  s = (mean (h - mu)^2 + eps)^(-1/2),
//   x = (h - mu) s g + beta
//   u = g dx, z = (h - mu) s:  dh = s (u - mean u - z mean(u z)),
//   dH_i = a_i dh,  da_i = <dh, H_i>,  dg = sum_t dx z,  dbeta = sum_t dx
// (then da through the read softmax). Bound by memory in principle: n + 1 rows
// of d in or out a token forward, 2 n + 1 backward, and few operations an
// element.
//
// Moments: every warp sums about its own mean, and the warps' sums are moved to
// the token's mean (Chan's formula), so a mean much larger than the deviation
// costs no accuracy and one exchange a token is enough; all in fp32, and the sum
// of squares leaves a thread divided by d, so that a row is NaN only where a
// thread's own overflow (inv_norm). A warp's mean is rounded like
// any fp32 sum of the raw values; its sum of h about itself is what that lost,
// and goes along. (The direct backward sums about a pivot in each thread, moves
// the sums to the row's first h and adds in fp64; adding in fp64 in the forward
// cost a fifth of its time.)
//
// hc_layernorm_kernel keeps a token's h in registers between the statistic and
// the store, so H is read once: T = 16384, n = 4, d = 4096, bf16 in 126 us, 82 %
// of the copy rate. hc_layernorm_bwd_ring_kernel, below, takes the rows that
// its warps cover (d from 896 to 7168 in bf16, from 520 to 3584 in fp32) and of
// which three whole tokens fit in shared memory: n = 1, T = 16384, d = 7168,
// bf16 in 198 us (55 % of the copy rate); n = 4 from a checkpoint, T = 8192, in
// 206 us (62 %). It is held by its instructions' latency: 14 warps with 128
// registers a thread, half the issue slots used, the shared memory's latency and
// the one exchange a token. More warps with fewer registers spilled (335 us),
// two tokens at a time in one thread too (293 us).
// hc_layernorm_bwd_kernel takes the rest, n = 4 at d = 7168 and n = 8 at d = 4096
// in full precision and wider rows among it: it parks h in shared memory (fp32),
// reads dx, and H for da, again from L2, and accumulates the gradients of g and
// beta in the CTA's workspace row (522 us for the first of these cases; n = 4,
// T = 8192, d = 7168 398 us, 41 % of the copy rate; n = 1, T = 16384, d = 8192 591
// us, 21 %).
// Either leaves one row of partial sums a CTA, which are summed in a fixed
// order.
#include <atomic>

#include "hc_checkpoint.cuh"
#include "hc_launch.h"
#include "hc_sync.cuh"
#include "hc_token_sums.cuh"

namespace hc {

namespace {

constexpr int kTB = 32;            // parameter slots per batch
constexpr int kFwdThreads = 512;   // largest CTA of the forward
constexpr int kBwdThreads = 256;

// Moments of one thread about its pivot.
struct Moments {
    float p = 0.0f, r = 0.0f, m2 = 0.0f;  // pivot, sum (h - p), sum (h - p)^2
    int count = 0;
    template <int VP>
    __device__ __forceinline__ void add(const float2 (&h)[VP]) {
        if (count == 0) p = h[0].x;
        const float2 np = make_float2(-p, -p);
        float2 rs = make_float2(0.0f, 0.0f), ms = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < VP; ++e) {
            const float2 t = fadd2_rn(h[e], np);
            rs = fadd2_rn(rs, t);
            ms = ffma2_rn(t, t, ms);
        }
        r += rs.x + rs.y;
        m2 += ms.x + ms.y;
        count += 2 * VP;
    }
    // Sums of h - c and of its square. c is near the row's values, like p: about
    // zero the squares would cancel when the mean is far (2^-53 of its square).
    __device__ __forceinline__ double sum(float c) const {
        return (double)count * ((double)p - (double)c) + (double)r;
    }
    __device__ __forceinline__ double squares(float c) const {
        const double q = (double)p - (double)c;
        return (double)m2 + q * (2.0 * (double)r + (double)count * q);
    }
};

// The sums of M fp64 values over the CTA, in all threads. buf: [2][warps][M],
// used alternately so that one barrier a call is enough.
template <int M>
__device__ __forceinline__ void cta_sums(double (&v)[M], double *buf, int parity, int nwarps, int lane, int warp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    double *b = buf + parity * nwarps * M;
    if (lane == 0) {
#pragma unroll
        for (int m = 0; m < M; ++m) b[warp * M + m] = v[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = 0.0;
    for (int w = 0; w < nwarps; ++w)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += b[w * M + m];
}

// Read weights of TB tokens into sa (weight 1 without a).
template <int N>
__device__ __forceinline__ void read_weights(const StepParams &p, int64_t first, int64_t G, int TB, float *sa,
                                             float *scratch) {
    if (p.a) {
        prepare_params<N, false, true>(p, first, G, TB, nullptr, nullptr, sa, scratch);
    } else {
        for (int v = threadIdx.x; v < TB * N; v += blockDim.x) sa[v] = 1.0f;
    }
}

template <int N, typename S, int CPT>
__global__ void __launch_bounds__(kFwdThreads)
hc_layernorm_kernel(StepParams p, const float *beta, float inv_d) {
    constexpr int V = StorageTraits<S>::V, VP = V / 2;
    __shared__ float sa[kTB * N];
    // of alternate tokens: the warps' means, and their sums of squares and of h
    // about them (the latter is what the mean's rounding left), over d
    __shared__ float sums[2][3][32];
    __shared__ float swork[kFwdThreads / 32 * kGroupScratch];
    const int tid = threadIdx.x, NT = blockDim.x, nwarps = NT >> 5;
    const int lane = tid & 31, warp = tid >> 5;
    const int64_t d = p.d, nvec = d / V, G = gridDim.x;
    auto warp_columns = [&](int w) {
        int64_t n = 0;
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int64_t left = d - ((int64_t)u * NT + w * 32) * V;
            n += left < 0 ? 0 : left < 32 * V ? left : 32 * V;
        }
        return (float)n;
    };
    const float n_own = warp_columns(warp), inv_n = n_own > 0.0f ? 1.0f / n_own : 0.0f;
    const float f_w = lane < nwarps ? warp_columns(lane) * inv_d : 0.0f;  // lane w: warp w's part of the row
    int TB = nwarps * Group<N>::TPW;
    TB = TB < kTB ? TB : kTB;
    const S *H = static_cast<const S *>(p.H);
    S *X = static_cast<S *>(p.x);
    int parity = 0;
    for (int64_t m0 = 0;; m0 += TB) {
        const int64_t first = blockIdx.x + m0 * G;
        if (first >= p.T) break;
        __syncthreads();  // previous batch's weights no longer read
        read_weights<N>(p, first, G, TB, sa, swork);
        __syncthreads();
        for (int tt = 0; tt < TB; ++tt) {
            const int64_t t = first + (int64_t)tt * G;
            if (t >= p.T) break;  // uniform over the CTA
            float2 h[CPT][VP];
            float wm = 0.0f;
#pragma unroll
            for (int u = 0; u < CPT; ++u) {
                const int64_t c = tid + (int64_t)u * NT;
                if (c < nvec) {
                    uint4 raw[N];
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        raw[i] = __ldcs(reinterpret_cast<const uint4 *>(H + (t * N + i) * d + c * V));
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        float2 v[VP];
                        ck_widen(raw[i], v);
                        const float2 ai = make_float2(sa[tt * N + i], sa[tt * N + i]);
#pragma unroll
                        for (int e = 0; e < VP; ++e) h[u][e] = i == 0 ? fmul2_rn(ai, v[e]) : ffma2_rn(ai, v[e], h[u][e]);
                    }
                    float2 z = h[u][0];
#pragma unroll
                    for (int e = 1; e < VP; ++e) z = fadd2_rn(z, h[u][e]);
                    wm += z.x + z.y;
                }
            }
            // the warp's mean, and h, its sum and squares about it
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) wm += __shfl_xor_sync(0xffffffffu, wm, o);
            wm *= inv_n;
            float2 q2 = make_float2(0.0f, 0.0f), l2 = q2;
            const float2 nm = make_float2(-wm, -wm);
#pragma unroll
            for (int u = 0; u < CPT; ++u) {
                if (tid + (int64_t)u * NT < nvec) {
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        h[u][e] = fadd2_rn(h[u][e], nm);
                        q2 = ffma2_rn(h[u][e], h[u][e], q2);
                        l2 = fadd2_rn(l2, h[u][e]);
                    }
                }
            }
            const float v[2] = {(q2.x + q2.y) * inv_d, (l2.x + l2.y) * inv_d};
            warp_sums_put<2>(v, lane, [&](int x, float sx) { sums[parity][1 + x][warp] = sx; });
            if (lane == 0) sums[parity][0][warp] = wm;
            __syncthreads();
            // moved to the mean of all: lane w takes warp w's
            const bool has = f_w > 0.0f;
            const float m0 = sums[parity][0][0], dm = has ? sums[parity][0][lane] - m0 : 0.0f;
            const float sl = has ? sums[parity][2][lane] : 0.0f, s2 = has ? sums[parity][1][lane] : 0.0f;
            parity ^= 1;
            float mu = __fmaf_rn(f_w, dm, sl);  // the mean less m0
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mu += __shfl_xor_sync(0xffffffffu, mu, o);
            const float del = dm - mu;
            float sq = __fmaf_rn(del, __fmaf_rn(f_w, del, 2.0f * sl), s2);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float rs = inv_norm(sq < 0.0f ? 0.0f : sq, p.eps);  // below 0: rounding only
            const float own = (wm - m0) - mu;  // the warp's mean less the token's
            const float2 nz = make_float2(own, own), r2 = make_float2(rs, rs);
#pragma unroll
            for (int u = 0; u < CPT; ++u) {
                const int64_t c = tid + (int64_t)u * NT;
                if (c < nvec) {
                    float2 gv[VP], bv[VP], x[VP];
                    load_gain2<VP>(p.g, c * V, gv);
                    if (beta) load_gain2<VP>(beta, c * V, bv);
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        const float2 z = fmul2_rn(fadd2_rn(h[u][e], nz), r2);
                        x[e] = beta ? ffma2_rn(z, gv[e], bv[e]) : fmul2_rn(z, gv[e]);
                    }
                    __stcs(reinterpret_cast<uint4 *>(X + t * d + c * V), ck_narrow(x));
                }
            }
        }
    }
}

struct LnBwParams {
    StepParams f;          // H: rows of S, or codes with exponents sH
    const uint8_t *sH;
    int64_t ns;
    const void *dx;
    void *dH;
    float *da;             // [T][N] or null
    float *part;           // [gridDim.x][2][d] partial dg, dbeta, or null
};

// PACKED: H holds a checkpoint's codes.
template <int N, typename S, bool PACKED>
__global__ void __launch_bounds__(kBwdThreads, 2)
hc_layernorm_bwd_kernel(LnBwParams bp) {
    const StepParams &p = bp.f;
    constexpr int V = StorageTraits<S>::V, VP = V / 2, NW = kBwdThreads / 32;
    __shared__ float sa[kTB * N], sn[kTB];
    __shared__ double sums[2 * NW * 4];
    __shared__ float red[NW * N];
    __shared__ float swork[NW * kGroupScratch];
    extern __shared__ __align__(16) float shp[];  // [d] parked h
    const int tid = threadIdx.x, NT = blockDim.x, nwarps = NT >> 5;
    const int lane = tid & 31, warp = tid >> 5;
    const int64_t d = p.d, nvec = d / V, G = gridDim.x;
    int TB = nwarps * Group<N>::TPW;
    TB = TB < kTB ? TB : kTB;
    const S *DX = static_cast<const S *>(bp.dx);
    S *DH = static_cast<S *>(bp.dH);
    float *sdg = bp.part ? bp.part + (int64_t)blockIdx.x * 2 * d : nullptr;
    if (sdg)
        for (int64_t k = (int64_t)tid * 4; k < 2 * d; k += (int64_t)NT * 4)
            *reinterpret_cast<float4 *>(sdg + k) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    // rows of H at slice k of token t, as fp32
    auto load_row = [&](int64_t row, int64_t k, float2 (&v)[VP]) {
        if constexpr (PACKED) {
            uint32_t q[V / 4];
            ck_load<V>(static_cast<const uint8_t *>(p.H) + row * d + k, q);
            ck_decode<VP>(q, ck_scale(__ldg(bp.sH + row * bp.ns + k / kCkBlock)), v);
        } else {
            ck_widen(__ldg(reinterpret_cast<const uint4 *>(static_cast<const S *>(p.H) + row * d + k)), v);
        }
    };
    int parity = 0;
    for (int64_t m0 = 0;; m0 += TB) {
        const int64_t first = blockIdx.x + m0 * G;
        if (first >= p.T) break;
        __syncthreads();  // previous batch's weights no longer read
        read_weights<N>(p, first, G, TB, sa, swork);
        __syncthreads();
        // the first h of every row of the batch: what its threads' sums are moved to
        if (tid < TB && first + (int64_t)tid * G < p.T) {
            float near = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 v[VP];
                load_row((first + (int64_t)tid * G) * N + i, 0, v);
                near = __fmaf_rn(sa[tid * N + i], v[0].x, near);
            }
            sn[tid] = near;
        }
        __syncthreads();
        for (int tt = 0; tt < TB; ++tt) {
            const int64_t t = first + (int64_t)tt * G;
            if (t >= p.T) break;  // uniform over the CTA
            const float *at = sa + tt * N;
            const float near = sn[tt];
            // ---- pass 1: moments of h, sums of u and u h ----
            Moments mo;
            float su = 0.0f, sud = 0.0f;  // sum u, sum u (h - p)
            for (int64_t c = tid; c < nvec; c += NT) {
                const int64_t k = c * V;
                float2 h[VP], u[VP], gv[VP];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float2 v[VP];
                    load_row(t * N + i, k, v);
                    const float2 ai = make_float2(at[i], at[i]);
#pragma unroll
                    for (int e = 0; e < VP; ++e) h[e] = i == 0 ? fmul2_rn(ai, v[e]) : ffma2_rn(ai, v[e], h[e]);
                }
                ck_widen(__ldg(reinterpret_cast<const uint4 *>(DX + t * d + k)), u);
                load_gain2<VP>(p.g, k, gv);
                mo.add<VP>(h);
                float2 a1 = make_float2(0.f, 0.f), a2 = a1;
                const float2 np = make_float2(-mo.p, -mo.p);
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    u[e] = fmul2_rn(u[e], gv[e]);
                    a1 = fadd2_rn(a1, u[e]);
                    a2 = ffma2_rn(u[e], fadd2_rn(h[e], np), a2);
                }
                su += a1.x + a1.y;
                sud += a2.x + a2.y;
#pragma unroll
                for (int e = 0; e < VP; e += 2)
                    *reinterpret_cast<float4 *>(shp + k + 2 * e) = make_float4(h[e].x, h[e].y, h[e + 1].x, h[e + 1].y);
            }
            double v[4] = {mo.sum(near), mo.squares(near), (double)su,
                           (double)sud + ((double)mo.p - (double)near) * (double)su};
            cta_sums<4>(v, sums, parity, nwarps, lane, warp);
            parity ^= 1;
            const double md = v[0] / (double)d, mu = (double)near + md;  // the mean less near, the mean
            double var = v[1] / (double)d - md * md;
            var = var < 0.0 ? 0.0 : var < INFINITY ? var : NAN;  // below 0: rounding only
            const double rsd = 1.0 / sqrt(var + (double)p.eps);
            const double c2d = rsd * (v[3] - md * v[2]) / (double)d;  // mean(u z)
            const float muf = (float)mu, mul = (float)(mu - (double)muf), rs = (float)rsd;
            const float c1 = (float)(v[2] / (double)d), c2 = (float)c2d;
            const float2 nm = make_float2(-muf, -muf), nl = make_float2(-mul, -mul), r2 = make_float2(rs, rs);
            const float2 n1 = make_float2(-c1, -c1), n2 = make_float2(-c2, -c2);
            // ---- pass 2 ----
            float dacc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) dacc[i] = 0.0f;
            for (int64_t c = tid; c < nvec; c += NT) {
                const int64_t k = c * V;
                float2 z[VP], dx[VP], gv[VP], dh[VP];
#pragma unroll
                for (int e = 0; e < VP; e += 2) {
                    const float4 f = *reinterpret_cast<const float4 *>(shp + k + 2 * e);
                    z[e] = make_float2(f.x, f.y);
                    z[e + 1] = make_float2(f.z, f.w);
                }
                ck_widen(__ldcs(reinterpret_cast<const uint4 *>(DX + t * d + k)), dx);
                load_gain2<VP>(p.g, k, gv);
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    z[e] = fmul2_rn(fadd2_rn(fadd2_rn(z[e], nm), nl), r2);
                    const float2 w = ffma2_rn(n2, z[e], fadd2_rn(fmul2_rn(dx[e], gv[e]), n1));
                    dh[e] = fmul2_rn(w, r2);
                }
                if (sdg) {
#pragma unroll
                    for (int e = 0; e < VP; e += 2) {
                        float4 *pg = reinterpret_cast<float4 *>(sdg + k + 2 * e);
                        float4 *pb = reinterpret_cast<float4 *>(sdg + d + k + 2 * e);
                        const float4 fg = *pg, fb = *pb;
                        const float2 g0 = ffma2_rn(dx[e], z[e], make_float2(fg.x, fg.y));
                        const float2 g1 = ffma2_rn(dx[e + 1], z[e + 1], make_float2(fg.z, fg.w));
                        const float2 b0 = fadd2_rn(dx[e], make_float2(fb.x, fb.y));
                        const float2 b1 = fadd2_rn(dx[e + 1], make_float2(fb.z, fb.w));
                        *pg = make_float4(g0.x, g0.y, g1.x, g1.y);
                        *pb = make_float4(b0.x, b0.y, b1.x, b1.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float2 o[VP];
                    const float2 ai = make_float2(at[i], at[i]);
#pragma unroll
                    for (int e = 0; e < VP; ++e) o[e] = fmul2_rn(ai, dh[e]);
                    __stcs(reinterpret_cast<uint4 *>(DH + (t * N + i) * d + k), ck_narrow(o));
                    if (bp.da) {
                        float2 hv[VP];
                        load_row(t * N + i, k, hv);
                        float2 s = fmul2_rn(dh[0], hv[0]);
#pragma unroll
                        for (int e = 1; e < VP; ++e) s = ffma2_rn(dh[e], hv[e], s);
                        dacc[i] += s.x + s.y;
                    }
                }
            }
            if (bp.da) {
                warp_sums_all<N>(dacc, red + warp * N, lane);
                __syncthreads();
                if (warp == 0) {
                    double s = 0.0;
                    if (lane < N)
                        for (int w = 0; w < nwarps; ++w) s += (double)red[w * N + lane];
                    if (p.read_logits) {  // through the softmax: a (da - sum a da)
                        const double w = lane < N ? (double)at[lane] : 0.0;
                        double dot = 0.0;
#pragma unroll
                        for (int i = 0; i < N; ++i) dot += __shfl_sync(0xffffffffu, w * s, i);
                        s = w * (s - dot);
                    }
                    if (lane < N) bp.da[t * N + lane] = (float)s;
                }
                // red is written again only after the next token's first barrier
            }
        }
    }
}

// ---- token ring ------------------------------------------------------------------
// A producer warp moves whole tokens (H's rows or codes and exponents, dx) into
// a ring of stages with bulk copies and leaves the token's read weights beside
// them; NG groups of gw warps take the CTA's tokens in turn. A thread owns up to
// kCPT slices of 16 bytes of dx, the same columns for every token, so the
// gradients of g and beta stay in its registers; they are added over the groups
// in shared memory at the end (in group order) and leave one row a CTA.
//
// A token takes one exchange: every warp sums about its own mean, and the
// statistic warp moves the warps' sums to the token's mean (Chan's formula; all
// terms are differences of means and what the warp's mean lost to rounding, its
// sum of h about itself, so a mean far from zero costs no accuracy, and no
// exchange is needed to find it first). While it does, the group runs
// the next token's first pass; the second pass of a token comes after that.
//
// Every wait is bounded (hc_sync.cuh); on time-out the fault code is recorded
// and the CTA runs to its end without waiting again (its results are void, its
// accesses stay in bounds).
constexpr int kRingWarps = 14;   // consumer warps at most (128 registers a thread)
constexpr int kCPT = 2;          // slices a thread at most

struct LnRingShape {
    int gw, ng, nst;
    int nw;  // tokens whose weights are kept
    int stage_bytes;
};

// Floats of a group's exchange: two tokens' sums [kLnRows][32 warps], [8]
// statistics, [n][32 warps] da sums. A warp's sums: of (h - m)^2, over d, of u,
// of u (h - m) and of h - m, with m its mean of h as rounded, then m itself.
// (Three of the eight rows are not used: with five the second token's lie at no
// power of two, and the addresses cost the kernel 4 %.)
constexpr int kLnRows = 8;
__host__ __device__ constexpr int ln_red_floats(int n) { return 2 * (kLnRows * 32 + 8 + n * 32); }
__host__ __device__ inline int64_t ln_ring_fixed_bytes(int n, int64_t d, int ng, int nst) {
    return d * 4 + (int64_t)ng * ln_red_floats(n) * 4             // g, exchanges
           + (int64_t)(nst + 2 * ng + 2) * kMaxStreams * 4        // weights
           + (int64_t)nst * 16 + (int64_t)ng * 32 + 16;           // barriers, abort flag
}

__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int N, typename S, bool PACKED>
__global__ void __launch_bounds__(32 * (kRingWarps + 2), 1)
hc_layernorm_bwd_ring_kernel(LnBwParams bp, LnRingShape sh, int *fault) {
    const StepParams &p = bp.f;
    constexpr int V = StorageTraits<S>::V, VP = V / 2;
    constexpr int RF = ln_red_floats(N), kStat = 2 * kLnRows * 32, kDa = kStat + 2 * 8;
    const int d = (int)p.d, ns = (int)bp.ns, nst = sh.nst, GW = sh.gw, NG = sh.ng;
    const int64_t G = gridDim.x;
    const int64_t M = (p.T > (int64_t)blockIdx.x) ? (p.T - 1 - blockIdx.x) / G + 1 : 0;
    const int rb = d * (int)sizeof(S), o_sc = N * d, o_dx = PACKED ? N * (d + ns) : N * rb;

    extern __shared__ __align__(128) unsigned char smem[];
    float *sg = reinterpret_cast<float *>(smem + (int64_t)nst * sh.stage_bytes);  // [d]
    float *red = sg + d;                                                           // [NG][RF]
    float *wts = red + NG * RF;                                                    // [nw][8]
    uint64_t *full = reinterpret_cast<uint64_t *>(wts + sh.nw * kMaxStreams);
    uint64_t *empty = full + nst;
    uint64_t *sums = empty + nst;    // [NG][2]: the warps' sums of a token are there
    uint64_t *stats = sums + 2 * NG;  // [NG][2]: its statistics are
    int *abort_word = reinterpret_cast<int *>(stats + 2 * NG);
    volatile int *abort_flag = abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], GW);
        }
        for (int s = 0; s < 2 * NG; ++s) {
            mbar_init(&sums[s], GW);
            mbar_init(&stats[s], 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    for (int k = threadIdx.x; k < d; k += blockDim.x) sg[k] = p.g ? p.g[k] : 1.0f;
    for (int k = threadIdx.x; k < NG * RF; k += blockDim.x) red[k] = 0.0f;  // a group may have fewer than 32 warps
    __syncthreads();
    const float inv_d = 1.0f / (float)d;
    // columns of warp w of a group
    auto warp_columns = [&](int w) {
        int n = 0;
#pragma unroll
        for (int u = 0; u < kCPT; ++u) {
            const int left = d - (w + u * GW) * 32 * V;
            n += left < 0 ? 0 : left < 32 * V ? left : 32 * V;
        }
        return n;
    };

    if (warp == NG * GW) {
        // ---------------- producer ----------------
        const S *DX = static_cast<const S *>(bp.dx);
        auto weight = [&](int64_t m) {
            return p.a && lane < N && m < M ? __ldg(p.a + (blockIdx.x + m * G) * p.a_s + lane) : 1.0f;
        };
        float next = weight(0);
        int s = 0, sw = 0;
        uint32_t ph = 1;  // parity of the stage's previous release
        int64_t m = 0;
        for (; m < M; ++m) {
            const int64_t t = blockIdx.x + m * G;
            bool ok = true;
            if (m >= nst) ok = mbar_wait_bounded(&empty[s], ph, abort_flag, fault, FAULT_WAIT_EMPTY);
            if (!__all_sync(0xffffffffu, ok)) break;
            unsigned char *st = smem + (int64_t)s * sh.stage_bytes;
            float w = next;
            next = weight(m + 1);
            if (p.read_logits) {  // softmax over the n logits, in index order
                float mx = __shfl_sync(0xffffffffu, w, 0);
#pragma unroll
                for (int x = 1; x < N; ++x) {
                    const float v = __shfl_sync(0xffffffffu, w, x);
                    if (v > mx) mx = v;
                }
                const float e = expf(__fsub_rn(w, mx));
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < N; ++x) sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, e, x));
                w = __fdiv_rn(e, sum);
            }
            if (lane < N) wts[sw * kMaxStreams + lane] = w;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], (uint32_t)sh.stage_bytes);
                if constexpr (PACKED) {
                    bulk_load(st, static_cast<const uint8_t *>(p.H) + t * N * d, (uint32_t)(N * d), &full[s]);
                    bulk_load(st + o_sc, bp.sH + t * N * ns, (uint32_t)(N * ns), &full[s]);
                } else {
                    bulk_load(st, static_cast<const S *>(p.H) + t * N * d, (uint32_t)(N * rb), &full[s]);
                }
                bulk_load(st + o_dx, DX + t * d, (uint32_t)rb, &full[s]);
            }
            if (++s == nst) {
                s = 0;
                ph ^= 1u;
            }
            if (++sw == sh.nw) sw = 0;
        }
        // every issued copy lands before the CTA may exit (normally already done)
        if (lane == 0)
            for (int64_t q = (m > nst ? m - nst : 0); q < m; ++q)
                mbar_wait_drain(&full[(int)(q % nst)], (uint32_t)((q / nst) & 1), fault);
        return;
    }

    if (warp == NG * GW + 1) {
        // ---------------- statistics ----------------
        const float f_w = lane < GW ? (float)warp_columns(lane) * inv_d : 0.0f;  // lane w: warp w's part of the row
        // da of the CTA's token m (of group gg), whose sums are in buffer par
        auto write_da = [&](int64_t m, int gg, int par, int place) {
            const float *dr = red + gg * RF + kDa + par * N * 32;
            float sum = 0.0f;
            if (lane < N) sum = sum16(dr + lane * 32) + sum16(dr + lane * 32 + 16);
            if (p.read_logits) {  // through the softmax: a (da - sum a da)
                const float w = lane < N ? wts[place * kMaxStreams + lane] : 0.0f;
                float dot = 0.0f;
#pragma unroll
                for (int x = 0; x < N; ++x) dot += __shfl_sync(0xffffffffu, w * sum, x);
                sum = w * (sum - dot);
            }
            if (lane < N) bp.da[(blockIdx.x + m * G) * N + lane] = sum;
        };
        int g = 0, par = 0, wo = 0;  // wo: place of the weights of the next da
        uint32_t ph = 0;
        for (int64_t m = 0; m < M; ++m) {
            float *rq = red + g * RF + par * kLnRows * 32, *so = red + g * RF + kStat + par * 8;
            mbar_wait_bounded(&sums[g * 2 + par], ph, abort_flag, fault, FAULT_WAIT_REDUCE);
            // lane w: warp w's sums about its mean, moved to the mean of all
            const float q = rq[lane], u = rq[32 + lane] * inv_d, z = rq[64 + lane] * inv_d;
            const float l = rq[96 + lane] * inv_d;
            const float m0 = rq[128], dm = f_w > 0.0f ? rq[128 + lane] - m0 : 0.0f;
            float mu = __fmaf_rn(f_w, dm, l), su = u;  // the mean less m0, mean u
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                mu += __shfl_xor_sync(0xffffffffu, mu, o);
                su += __shfl_xor_sync(0xffffffffu, su, o);
            }
            const float del = dm - mu;
            float sq = __fmaf_rn(del, __fmaf_rn(f_w, del, 2.0f * l), q), sz = __fmaf_rn(del, u, z);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sq += __shfl_xor_sync(0xffffffffu, sq, o);
                sz += __shfl_xor_sync(0xffffffffu, sz, o);
            }
            // dh = rs (u - c1 - c2 z), z = (h - mean) rs
            const float rs = inv_norm(sq < 0.0f ? 0.0f : sq, p.eps);  // below 0: rounding only
            const float c1 = su, c2 = rs * sz;
            if (bp.da && m >= 2 * NG) {
                write_da(m - 2 * NG, g, par, wo);
                if (++wo == sh.nw) wo = 0;
            }
            if (lane == 0) {
                *reinterpret_cast<float4 *>(so) = make_float4(m0, mu, rs, -rs * c1);
                so[4] = -rs * c2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&stats[g * 2 + par]);
            if (++g == NG) {
                g = 0;
                ph ^= (uint32_t)par;
                par ^= 1;
            }
        }
        if (bp.da)  // the last two tokens of every group, after the group's last arrival
            for (int64_t m = M > 2 * NG ? M - 2 * NG : 0; m < M; ++m) {
                const int gg = (int)(m % NG);
                const int64_t cnt = (M - 1 - gg) / NG + 1;  // the group's tokens; its last arrival is number cnt
                mbar_wait_bounded(&sums[gg * 2 + (int)(cnt & 1)], (uint32_t)((cnt >> 1) & 1), abort_flag, fault,
                                  FAULT_WAIT_REDUCE);
                write_da(m, gg, (int)((m / NG) & 1), (int)(m % sh.nw));
            }
        return;
    }

    // ---------------- consumers ----------------
    const int g = warp / GW, gw = warp - g * GW, GT = GW * 32;
    const int k0 = (gw * 32 + lane) * V, kstep = GT * V;  // this thread's columns
    float *rg = red + g * RF;
    S *DH = static_cast<S *>(bp.dH);
    float2 ag[kCPT][VP], ab[kCPT][VP];  // gradients of g and beta
#pragma unroll
    for (int u = 0; u < kCPT; ++u)
#pragma unroll
        for (int e = 0; e < VP; ++e) ag[u][e] = ab[u][e] = make_float2(0.0f, 0.0f);
    const float inv_n = 1.0f / (float)warp_columns(gw);

    auto load_row = [&](const unsigned char *st, int x, int k, float2 (&v)[VP]) {
        if constexpr (PACKED) {
            uint32_t q[V / 4];
            if constexpr (V == 8) {
                const uint2 c = *reinterpret_cast<const uint2 *>(st + x * d + k);
                q[0] = c.x;
                q[1] = c.y;
            } else {
                q[0] = *reinterpret_cast<const uint32_t *>(st + x * d + k);
            }
            ck_decode<VP>(q, ck_scale(st[o_sc + x * ns + k / kCkBlock]), v);
        } else {
            ck_widen(*reinterpret_cast<const uint4 *>(st + x * rb + k * (int)sizeof(S)), v);
        }
    };
    auto load_gains = [&](int k, float2 (&v)[VP]) {
#pragma unroll
        for (int e = 0; e < VP; e += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(sg + k + 2 * e);
            v[e] = make_float2(f.x, f.y);
            v[e + 1] = make_float2(f.z, f.w);
        }
    };

    int slot = g % nst, slot0 = slot;        // stages of the token of the first and of the second pass
    int ws = g % sh.nw, ws0 = ws;            // and places of their weights
    uint32_t ph = (uint32_t)((g / nst) & 1);
    const int64_t Mg = M > g ? (M - 1 - g) / NG + 1 : 0;
    float2 h[kCPT][VP];  // h of the second pass's token, less the warp's mean
    uint4 dxr[kCPT];
    float wm = 0.0f;
    for (int64_t i = 0; i <= Mg; ++i) {
        float2 h1[kCPT][VP];
        uint4 dx1[kCPT];
        float wm1 = 0.0f;
        if (i < Mg) {
            // ---- first pass of token i ----
            mbar_wait_bounded(&full[slot], ph, abort_flag, fault, FAULT_WAIT_FULL);
            const unsigned char *st = smem + (int64_t)slot * sh.stage_bytes;
            const float *at = wts + ws * kMaxStreams;
#pragma unroll
            for (int u = 0; u < kCPT; ++u) {
                const int k = k0 + u * kstep;
                if (k < d) {
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        float2 v[VP];
                        load_row(st, x, k, v);
                        const float2 ax = make_float2(at[x], at[x]);
#pragma unroll
                        for (int e = 0; e < VP; ++e)
                            h1[u][e] = x == 0 ? fmul2_rn(ax, v[e]) : ffma2_rn(ax, v[e], h1[u][e]);
                    }
                    dx1[u] = *reinterpret_cast<const uint4 *>(st + o_dx + k * (int)sizeof(S));
                    float2 z = h1[u][0];
#pragma unroll
                    for (int e = 1; e < VP; ++e) z = fadd2_rn(z, h1[u][e]);
                    wm1 += z.x + z.y;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) wm1 += __shfl_xor_sync(0xffffffffu, wm1, o);
            wm1 *= inv_n;
            float2 q[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) q[x] = make_float2(0.0f, 0.0f);
            const float2 nm = make_float2(-wm1, -wm1);
#pragma unroll
            for (int u = 0; u < kCPT; ++u) {
                const int k = k0 + u * kstep;
                if (k < d) {
                    float2 gv[VP], dx[VP];
                    load_gains(k, gv);
                    ck_widen(dx1[u], dx);
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        h1[u][e] = fadd2_rn(h1[u][e], nm);
                        const float2 w = fmul2_rn(dx[e], gv[e]);
                        q[0] = ffma2_rn(h1[u][e], h1[u][e], q[0]);
                        q[1] = fadd2_rn(q[1], w);
                        q[2] = ffma2_rn(w, h1[u][e], q[2]);
                        q[3] = fadd2_rn(q[3], h1[u][e]);
                    }
                }
            }
            const float v[4] = {(q[0].x + q[0].y) * inv_d, q[1].x + q[1].y, q[2].x + q[2].y, q[3].x + q[3].y};
            float *rq = rg + (int)(i & 1) * kLnRows * 32 + gw;
            warp_sums_put<4>(v, lane, [&](int x, float sx) { rq[x * 32] = sx; });
            if (lane == 0) rq[4 * 32] = wm1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sums[g * 2 + (int)(i & 1)]);
            for (slot += NG; slot >= nst; slot -= nst) ph ^= 1u;
            for (ws += NG; ws >= sh.nw; ws -= sh.nw) {}
        }
        if (i > 0) {
            // ---- second pass of token i - 1 ----
            const int par = (int)((i - 1) & 1);
            mbar_wait_bounded(&stats[g * 2 + par], (uint32_t)(((i - 1) >> 1) & 1), abort_flag, fault,
                              FAULT_WAIT_REDUCE);
            const unsigned char *st = smem + (int64_t)slot0 * sh.stage_bytes;
            const float *at = wts + ws0 * kMaxStreams;
            const float4 so = *reinterpret_cast<const float4 *>(rg + kStat + par * 8);
            const float k2 = rg[kStat + par * 8 + 4], own = (wm - so.x) - so.y;  // the warp's mean less the token's
            const float2 nz = make_float2(own, own), r2 = make_float2(so.z, so.z);
            const float2 n1 = make_float2(so.w, so.w), n2 = make_float2(k2, k2);
            S *DHt = DH + (blockIdx.x + (g + (i - 1) * NG) * G) * N * d;
            float dacc[N];
#pragma unroll
            for (int x = 0; x < N; ++x) dacc[x] = 0.0f;
#pragma unroll
            for (int u = 0; u < kCPT; ++u) {
                const int k = k0 + u * kstep;
                if (k < d) {
                    float2 dx[VP], dh[VP];
                    load_gains(k, dh);
                    ck_widen(dxr[u], dx);
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        const float2 z = fmul2_rn(fadd2_rn(h[u][e], nz), r2);
                        ag[u][e] = ffma2_rn(dx[e], z, ag[u][e]);
                        ab[u][e] = fadd2_rn(dx[e], ab[u][e]);
                        dh[e] = ffma2_rn(r2, fmul2_rn(dx[e], dh[e]), ffma2_rn(n2, z, n1));
                    }
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        float2 o[VP];
                        const float2 ax = make_float2(at[x], at[x]);
#pragma unroll
                        for (int e = 0; e < VP; ++e) o[e] = fmul2_rn(ax, dh[e]);
                        if (bp.da) {
                            float2 v[VP];
                            load_row(st, x, k, v);
                            float2 q = fmul2_rn(dh[0], v[0]);
#pragma unroll
                            for (int e = 1; e < VP; ++e) q = ffma2_rn(dh[e], v[e], q);
                            dacc[x] += q.x + q.y;
                        }
                        __stcs(reinterpret_cast<uint4 *>(DHt + x * d + k), ck_narrow(o));
                    }
                }
            }
            if (bp.da) {
                float *dr = rg + kDa + par * N * 32 + gw;
                warp_sums_put<N>(dacc, lane, [&](int x, float sx) { dr[x * 32] = sx; });
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot0]);
            for (slot0 += NG; slot0 >= nst; slot0 -= nst) {}
            for (ws0 += NG; ws0 >= sh.nw; ws0 -= sh.nw) {}
        }
#pragma unroll
        for (int u = 0; u < kCPT; ++u) {
#pragma unroll
            for (int e = 0; e < VP; ++e) h[u][e] = h1[u][e];
            dxr[u] = dx1[u];
        }
        wm = wm1;
    }
    if (lane == 0) mbar_arrive(&sums[g * 2 + (int)(Mg & 1)]);  // the last tokens' da sums are there
    if (bp.part) {
        // the groups' sums, added in group order over the stages (all consumed)
        float *acc = reinterpret_cast<float *>(smem);  // [2][d]
        for (int q = 0; q < NG; ++q) {
            group_sync(1, NG * GT);
            if (q == g) {
#pragma unroll
                for (int u = 0; u < kCPT; ++u) {
                    const int k = k0 + u * kstep;
                    if (k < d) {
#pragma unroll
                        for (int e = 0; e < VP; ++e) {
                            float2 *pg = reinterpret_cast<float2 *>(acc + k) + e;
                            float2 *pb = reinterpret_cast<float2 *>(acc + d + k) + e;
                            *pg = q == 0 ? ag[u][e] : fadd2_rn(*pg, ag[u][e]);
                            *pb = q == 0 ? ab[u][e] : fadd2_rn(*pb, ab[u][e]);
                        }
                    }
                }
            }
        }
        group_sync(1, NG * GT);
        float *row = bp.part + (int64_t)blockIdx.x * 2 * d;
        for (int c = threadIdx.x * 4; c < 2 * d; c += NG * GT * 4)
            *reinterpret_cast<float4 *>(row + c) = *reinterpret_cast<const float4 *>(acc + c);
    }
}

// Sums over the rows of part [rows][cols] (fp64, 8 row slices in order):
// columns below split to lo, the others to hi (either may be null).
constexpr int kCols = 32, kSlices = 8;
__global__ void __launch_bounds__(kCols * kSlices)
hc_colsum_kernel(const float *part, int rows, int64_t cols, int64_t split, float *lo, float *hi) {
    __shared__ double acc_s[kSlices][kCols];
    const int col = threadIdx.x % kCols, q = threadIdx.x / kCols;
    for (int64_t k0 = (int64_t)blockIdx.x * kCols; k0 < cols; k0 += (int64_t)gridDim.x * kCols) {
        const int64_t k = k0 + col;
        double acc = 0.0;
        if (k < cols)
            for (int r = q; r < rows; r += kSlices) acc += (double)part[(int64_t)r * cols + k];
        acc_s[q][col] = acc;
        __syncthreads();
        if (q == 0 && k < cols) {
            double tot = 0.0;
#pragma unroll
            for (int j = 0; j < kSlices; ++j) tot += acc_s[j][col];
            float *o = k < split ? lo : hi;
            if (o) o[k < split ? k : k - split] = (float)tot;
        }
        __syncthreads();
    }
}

template <int N, typename S>
struct LayerNorm {
    static constexpr int V = StorageTraits<S>::V;

    template <int CPT>
    static hc_status forward_cpt(const LayerNormArgs &a, int NT, const LaunchCtx &ctx, cudaStream_t st) {
        auto kern = hc_layernorm_kernel<N, S, CPT>;
        int64_t grid = a.f.T;
        cudaError_t e;
        if (grid > ctx.sms) {
            int per_sm = 0;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, NT, 0);
            if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "layer norm occupancy: %s", cudaGetErrorString(e));
            const int64_t most = (int64_t)ctx.sms * (per_sm < 1 ? 1 : per_sm);
            if (grid > most) grid = most;
        }
        kern<<<(unsigned)grid, NT, 0, st>>>(a.f, a.beta, 1.0f / (float)a.f.d);
        e = cudaGetLastError();
        if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "hc_layernorm_kernel launch: %s", cudaGetErrorString(e));
        return HC_OK;
    }
    // Threads and 16-byte slices per thread: the least idle slices, then the
    // fewest slices per thread.
    static hc_status forward(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
        const int64_t nvec = a.f.d / V;
        int64_t best = INT64_MAX;
        int NT = 0, CPT = 0;
        for (int cpt : {1, 2, 4, 8}) {
            const int64_t nt = ((nvec + cpt - 1) / cpt + 31) / 32 * 32;
            if (nt > kFwdThreads || (nt < 64 && cpt > 1)) continue;
            if (nt * cpt - nvec < best) {
                best = nt * cpt - nvec;
                NT = (int)nt;
                CPT = cpt;
            }
        }
        switch (CPT) {
            case 1: return forward_cpt<1>(a, NT, ctx, st);
            case 2: return forward_cpt<2>(a, NT, ctx, st);
            case 4: return forward_cpt<4>(a, NT, ctx, st);
            case 8: return forward_cpt<8>(a, NT, ctx, st);
        }
        return set_error(HC_ERR_UNSUPPORTED, "no launch shape for d = %lld", (long long)a.f.d);
    }

    static int threads(int64_t d) {
        const int64_t nvec = d / V;
        const int64_t nt = nvec < kBwdThreads ? (nvec + 31) / 32 * 32 : kBwdThreads;
        for (int64_t c = nt; c >= nt / 2 && c >= 32 && nvec >= kBwdThreads; c -= 32)
            if (nvec % c == 0) return (int)c;
        return (int)nt;
    }
    template <bool PACKED>
    static hc_status occupancy(int64_t d, const LaunchCtx &ctx, int &per_sm) {
        auto kern = hc_layernorm_bwd_kernel<N, S, PACKED>;
        static std::atomic<bool> done[64];
        const hc_status s = opt_in_smem(reinterpret_cast<const void *>(kern), 32768 * 4, done, ctx);
        if (s != HC_OK) return s;
        const cudaError_t e =
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads(d), (size_t)d * 4);
        if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "layer norm occupancy: %s", cudaGetErrorString(e));
        return HC_OK;
    }
    // The ring takes rows from here up, in slices of 16 bytes of dx: below, a
    // group of one or two warps pays a token's exchange for too few columns.
    // Direct : ring in us, 134 MB of values a call, n = 1, 4 and 8: bf16 64
    // slices 354 : 647, 199 : 326, 164 : 229 (268 MB); 96 217 : 233, 120 : 128,
    // 97 : 96; 112 232 : 204, 124 : 114, 99 : 85; 128 220 : 183, 118 : 103,
    // 93 : 81; 256 223 : 108, 120 : 69, 93 : 71. fp32, half the columns a slice:
    // 112 171 : 200, 101 : 112, 83 : 81; 128 155 : 177, 93 : 99, 79 : 75; 130
    // 203 : 177, 110 : 97, 89 : 75; 256 162 : 103, 97 : 65, 77 : 60. From a
    // checkpoint alike (fp32 at n = 8 crosses at 96 already).
    static constexpr int64_t kRingFrom = V == 8 ? 112 : 130;
    // The ring's geometry, or gw = 0 where it does not apply: a group's warps
    // must cover the row, two stages a group and one more
    // must fit (a group holds the tokens of both passes), and a checkpoint's
    // codes must start on 16 bytes.
    static LnRingShape ring(int64_t d, bool packed, int64_t &smem) {
        LnRingShape sh{};
        const int64_t nvec = d / V, gw = (nvec + 32 * kCPT - 1) / (32 * kCPT);
        if (nvec < kRingFrom || gw > kRingWarps || (packed && d % 16 != 0)) return sh;
        const int64_t stage = N * (packed ? d + ck_scale_stride(d) : d * (int64_t)sizeof(S)) + d * (int64_t)sizeof(S);
        for (int64_t ng = kRingWarps / gw; ng >= 1; --ng) {
            int64_t nst = (kSmemLimitLogits - ln_ring_fixed_bytes(N, d, (int)ng, 0)) / (stage + kMaxStreams * 4 + 16);
            if (nst < 2 * ng + 1) continue;
            if (nst > 3 * ng + 3) nst = 3 * ng + 3;
            if (nst * stage < 8 * d) continue;
            sh.gw = (int)gw;
            sh.ng = (int)ng;
            sh.nst = (int)nst;
            sh.nw = (int)(nst + 2 * ng + 2);
            sh.stage_bytes = (int)stage;
            smem = nst * stage + ln_ring_fixed_bytes(N, d, (int)ng, (int)nst);
            break;
        }
        return sh;
    }
    // The grid, which the workspace is sized by (for the larger of the two forms').
    static hc_status grid(int64_t T, int64_t d, bool packed, const LaunchCtx &ctx, int64_t &g) {
        int64_t smem = 0;
        int per_sm = 1;
        if (!ring(d, packed, smem).gw) {
            const hc_status s = packed ? occupancy<true>(d, ctx, per_sm) : occupancy<false>(d, ctx, per_sm);
            if (s != HC_OK) return s;
        }
        g = (int64_t)ctx.sms * (per_sm < 1 ? 1 : per_sm);
        if (g > T) g = T;
        return HC_OK;
    }
    static hc_status workspace(int64_t T, int64_t d, const LaunchCtx &ctx, size_t *bytes) {
        int64_t g0 = 0, g1 = 0;
        hc_status s = grid(T, d, false, ctx, g0);
        if (s == HC_OK) s = grid(T, d, true, ctx, g1);
        if (s == HC_OK) *bytes = (size_t)(g0 > g1 ? g0 : g1) * 2 * (size_t)d * sizeof(float);
        return s;
    }
    template <bool PACKED>
    static hc_status launch_backward(const LnBwParams &bp, int64_t g, const LaunchCtx &ctx, cudaStream_t st) {
        int64_t smem = 0;
        const LnRingShape sh = ring(bp.f.d, PACKED, smem);
        cudaError_t e;
        if (sh.gw) {
            auto kern = hc_layernorm_bwd_ring_kernel<N, S, PACKED>;
            static std::atomic<bool> done[64];
            const hc_status s = opt_in_smem(reinterpret_cast<const void *>(kern), kSmemLimitLogits, done, ctx);
            if (s != HC_OK) return s;
            kern<<<(unsigned)g, 32 * (2 + sh.ng * sh.gw), (size_t)smem, st>>>(bp, sh, ctx.fault);
        } else {
            hc_layernorm_bwd_kernel<N, S, PACKED><<<(unsigned)g, threads(bp.f.d), (size_t)bp.f.d * 4, st>>>(bp);
        }
        e = cudaGetLastError();
        if (e != cudaSuccess)
            return set_error(HC_ERR_CUDA, "layer norm backward launch: %s", cudaGetErrorString(e));
        return HC_OK;
    }
    static hc_status backward(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
        int64_t g = 0;
        hc_status s = grid(a.f.T, a.f.d, a.sH != nullptr, ctx, g);
        if (s != HC_OK) return s;
        const bool want = a.dg || a.dbeta;
        const size_t need = (size_t)g * 2 * (size_t)a.f.d * sizeof(float);
        if (want && a.workspace_bytes < need)
            return set_error(HC_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed for dg and dbeta",
                             a.workspace_bytes, need);
        LnBwParams bp{};
        bp.f = a.f;
        bp.sH = a.sH;
        bp.ns = ck_scale_stride(a.f.d);
        bp.dx = a.dx;
        bp.dH = a.dH;
        bp.da = a.da;
        bp.part = want ? static_cast<float *>(a.workspace) : nullptr;
        s = a.sH ? launch_backward<true>(bp, g, ctx, st) : launch_backward<false>(bp, g, ctx, st);
        if (s != HC_OK) return s;
        if (want) {
            const int64_t cols = 2 * a.f.d;
            hc_colsum_kernel<<<(unsigned)((cols + kCols - 1) / kCols), kCols * kSlices, 0, st>>>(
                static_cast<const float *>(a.workspace), (int)g, cols, a.f.d, a.dg, a.dbeta);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "hc_colsum_kernel launch: %s", cudaGetErrorString(e));
        }
        return HC_OK;
    }
};

template <int N>
hc_status forward_n(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
    return a.dt == HC_BF16 ? LayerNorm<N, __nv_bfloat16>::forward(a, ctx, st)
                           : LayerNorm<N, float>::forward(a, ctx, st);
}
template <int N>
hc_status backward_n(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
    return a.dt == HC_BF16 ? LayerNorm<N, __nv_bfloat16>::backward(a, ctx, st)
                           : LayerNorm<N, float>::backward(a, ctx, st);
}
template <int N>
hc_status workspace_n(hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx, size_t *bytes) {
    return dt == HC_BF16 ? LayerNorm<N, __nv_bfloat16>::workspace(T, d, ctx, bytes)
                         : LayerNorm<N, float>::workspace(T, d, ctx, bytes);
}

}  // namespace

hc_status launch_layernorm(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
    switch (a.n) {
        case 1: return forward_n<1>(a, ctx, st);
        case 2: return forward_n<2>(a, ctx, st);
        case 3: return forward_n<3>(a, ctx, st);
        case 4: return forward_n<4>(a, ctx, st);
        case 5: return forward_n<5>(a, ctx, st);
        case 6: return forward_n<6>(a, ctx, st);
        case 7: return forward_n<7>(a, ctx, st);
        default: return forward_n<8>(a, ctx, st);
    }
}

hc_status layernorm_backward_workspace_bytes(int n, hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx,
                                             size_t *bytes) {
    switch (n) {
        case 1: return workspace_n<1>(dt, T, d, ctx, bytes);
        case 2: return workspace_n<2>(dt, T, d, ctx, bytes);
        case 3: return workspace_n<3>(dt, T, d, ctx, bytes);
        case 4: return workspace_n<4>(dt, T, d, ctx, bytes);
        case 5: return workspace_n<5>(dt, T, d, ctx, bytes);
        case 6: return workspace_n<6>(dt, T, d, ctx, bytes);
        case 7: return workspace_n<7>(dt, T, d, ctx, bytes);
        default: return workspace_n<8>(dt, T, d, ctx, bytes);
    }
}

hc_status launch_layernorm_backward(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
    switch (a.n) {
        case 1: return backward_n<1>(a, ctx, st);
        case 2: return backward_n<2>(a, ctx, st);
        case 3: return backward_n<3>(a, ctx, st);
        case 4: return backward_n<4>(a, ctx, st);
        case 5: return backward_n<5>(a, ctx, st);
        case 6: return backward_n<6>(a, ctx, st);
        case 7: return backward_n<7>(a, ctx, st);
        default: return backward_n<8>(a, ctx, st);
    }
}

}  // namespace hc
