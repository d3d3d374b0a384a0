// hc_layernorm.cu -- the read with layer norm, and its gradients.
//
//   h = sum_i a_i H_i,  mu = mean h,  s = (mean (h - mu)^2 + eps)^(-1/2),
//   x = (h - mu) s g + beta
//   u = g dx, z = (h - mu) s:  dh = s (u - mean u - z mean(u z)),
//   dH_i = a_i dh,  da_i = <dh, H_i>,  dg = sum_t dx z,  dbeta = sum_t dx
// (then da through the read softmax). Bound by memory: n + 1 rows of d in or
// out a token forward, 2 n + 1 backward, and few operations an element.
//
// Moments: every thread takes its first element of h as pivot p and sums
// h - p and (h - p)^2 in fp32; the sums of h and h^2 (and of u h) follow in
// fp64, where they are added over the CTA. One pass and one exchange, and a
// mean much larger than the deviation costs no accuracy: the fp32 errors are
// relative to the deviations from p, not to p.
//
// hc_layernorm_kernel keeps a token's h in registers between the statistic and
// the store, so H is read once. hc_layernorm_bwd_kernel parks h in shared
// memory (fp32) and reads dx, and H for da, again from L2; the gradients of g
// and beta accumulate in the CTA's workspace row and are summed over the rows
// in a fixed order.
#include "hc_checkpoint.cuh"
#include "hc_launch.h"
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
    __device__ __forceinline__ double sum() const { return (double)count * (double)p + (double)r; }
    __device__ __forceinline__ double squares() const {
        return (double)m2 + (double)p * (2.0 * (double)r + (double)count * (double)p);
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
hc_layernorm_kernel(StepParams p, const float *beta) {
    constexpr int V = StorageTraits<S>::V, VP = V / 2;
    __shared__ float sa[kTB * N];
    __shared__ double sums[2 * (kFwdThreads / 32) * 2];
    __shared__ float swork[kFwdThreads / 32 * kGroupScratch];
    const int tid = threadIdx.x, NT = blockDim.x, nwarps = NT >> 5;
    const int lane = tid & 31, warp = tid >> 5;
    const int64_t d = p.d, nvec = d / V, G = gridDim.x;
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
            Moments mo;
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
                    mo.add<VP>(h[u]);
                }
            }
            double v[2] = {mo.sum(), mo.squares()};
            cta_sums<2>(v, sums, parity, nwarps, lane, warp);
            parity ^= 1;
            const double mu = v[0] / (double)d;
            double var = v[1] / (double)d - mu * mu;
            var = var < 0.0 ? 0.0 : var;  // rounding only (NaN stays)
            const float rs = __double2float_rn(1.0 / sqrt(var + (double)p.eps)), muf = (float)mu;
            // h - mu with mu's own rounding kept: two fp32 parts
            const float mul = (float)(mu - (double)muf);
            const float2 nm = make_float2(-muf, -muf), nl = make_float2(-mul, -mul), r2 = make_float2(rs, rs);
#pragma unroll
            for (int u = 0; u < CPT; ++u) {
                const int64_t c = tid + (int64_t)u * NT;
                if (c < nvec) {
                    float2 gv[VP], bv[VP], x[VP];
                    load_gain2<VP>(p.g, c * V, gv);
                    if (beta) load_gain2<VP>(beta, c * V, bv);
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        const float2 z = fmul2_rn(fadd2_rn(fadd2_rn(h[u][e], nm), nl), r2);
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
    __shared__ float sa[kTB * N];
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
        for (int tt = 0; tt < TB; ++tt) {
            const int64_t t = first + (int64_t)tt * G;
            if (t >= p.T) break;  // uniform over the CTA
            const float *at = sa + tt * N;
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
            double v[4] = {mo.sum(), mo.squares(), (double)su, (double)sud + (double)mo.p * (double)su};
            cta_sums<4>(v, sums, parity, nwarps, lane, warp);
            parity ^= 1;
            const double mu = v[0] / (double)d;
            double var = v[1] / (double)d - mu * mu;
            var = var < 0.0 ? 0.0 : var;  // rounding only (NaN stays)
            const double rsd = 1.0 / sqrt(var + (double)p.eps);
            const double c2d = rsd * (v[3] - mu * v[2]) / (double)d;  // mean(u z)
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
        int per_sm = 0;
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, NT, 0);
        if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "layer norm occupancy: %s", cudaGetErrorString(e));
        int64_t grid = (int64_t)ctx.sms * (per_sm < 1 ? 1 : per_sm);
        if (grid > a.f.T) grid = a.f.T;
        kern<<<(unsigned)grid, NT, 0, st>>>(a.f, a.beta);
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
    static hc_status occupancy(int64_t d, int &per_sm) {
        auto kern = hc_layernorm_bwd_kernel<N, S, PACKED>;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * 4);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads(d), (size_t)d * 4);
        if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "layer norm occupancy: %s", cudaGetErrorString(e));
        return HC_OK;
    }
    // The grid, which the workspace is sized by: the same whether H is packed.
    static hc_status grid(int64_t T, int64_t d, const LaunchCtx &ctx, int64_t &g) {
        int p0 = 0, p1 = 0;
        hc_status s = occupancy<false>(d, p0);
        if (s == HC_OK) s = occupancy<true>(d, p1);
        if (s != HC_OK) return s;
        const int per_sm = p0 < p1 ? p0 : p1;
        g = (int64_t)ctx.sms * (per_sm < 1 ? 1 : per_sm);
        if (g > T) g = T;
        return HC_OK;
    }
    static hc_status backward(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st) {
        int64_t g = 0;
        const hc_status s = grid(a.f.T, a.f.d, ctx, g);
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
        const int NT = threads(a.f.d);
        if (a.sH) hc_layernorm_bwd_kernel<N, S, true><<<(unsigned)g, NT, (size_t)a.f.d * 4, st>>>(bp);
        else hc_layernorm_bwd_kernel<N, S, false><<<(unsigned)g, NT, (size_t)a.f.d * 4, st>>>(bp);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return set_error(HC_ERR_CUDA, "hc_layernorm_bwd_kernel launch: %s", cudaGetErrorString(e));
        if (want) {
            const int64_t cols = 2 * a.f.d;
            hc_colsum_kernel<<<(unsigned)((cols + kCols - 1) / kCols), kCols * kSlices, 0, st>>>(
                static_cast<const float *>(a.workspace), (int)g, cols, a.f.d, a.dg, a.dbeta);
            e = cudaGetLastError();
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
hc_status grid_n(hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx, int64_t &g) {
    return dt == HC_BF16 ? LayerNorm<N, __nv_bfloat16>::grid(T, d, ctx, g) : LayerNorm<N, float>::grid(T, d, ctx, g);
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
    int64_t g = 0;
    hc_status s;
    switch (n) {
        case 1: s = grid_n<1>(dt, T, d, ctx, g); break;
        case 2: s = grid_n<2>(dt, T, d, ctx, g); break;
        case 3: s = grid_n<3>(dt, T, d, ctx, g); break;
        case 4: s = grid_n<4>(dt, T, d, ctx, g); break;
        case 5: s = grid_n<5>(dt, T, d, ctx, g); break;
        case 6: s = grid_n<6>(dt, T, d, ctx, g); break;
        case 7: s = grid_n<7>(dt, T, d, ctx, g); break;
        default: s = grid_n<8>(dt, T, d, ctx, g); break;
    }
    if (s != HC_OK) return s;
    *bytes = (size_t)g * 2 * (size_t)d * sizeof(float);
    return HC_OK;
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
