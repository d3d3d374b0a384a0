// hc_checkpoint.cu -- checkpoint of rows of d values: codes and exponents from
// stored rows, and stored rows from codes and exponents (hc_checkpoint.cuh has
// the format).
//
// Both are bound by memory: a value costs its own bytes and 1 + 1/32. Measured
// for T = 16384, n = 4, d = 7168, bf16 (1.42 GB each way): the pair 512 us, 85 %
// of the copy rate; packing 242 us of it, 92 %; unpacking, which writes twice
// what it reads, 309 us under the profiler, 72 %, and about 270 us in the pair. Two or
// eight chunks in flight a thread, plain instead of streaming stores, and eight
// times the CTAs were 1 to 18 % slower. A warp
// takes one chunk of a row at a time, 16 bytes of X a lane (256 elements in
// bf16, 128 in fp32; 8 or 4 codes a lane), so the 4 or 8 lanes of a block of 32
// are neighbours and the maximum is two or three shuffles; rows of any length
// end inside a chunk.
// Every thread has kUnroll chunks' loads in flight. The chunk's place is carried along
// (row, chunk) instead of divided out.
#include "hc_checkpoint.cuh"
#include "hc_launch.h"

namespace hc {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Place of a warp's chunk: row and first element, stepped by a fixed number of
// chunks without dividing.
struct ChunkWalk {
    int64_t row;
    int chunk, per_row;
    int64_t step_rows;
    int step_chunks;
    __device__ ChunkWalk(int64_t first, int64_t step, int per) : per_row(per) {
        row = first / per;
        chunk = (int)(first - row * per);
        step_rows = step / per;
        step_chunks = (int)(step - step_rows * per);
    }
    __device__ __forceinline__ void next() {
        row += step_rows;
        chunk += step_chunks;
        if (chunk >= per_row) {
            chunk -= per_row;
            ++row;
        }
    }
};

template <typename S>
__global__ void __launch_bounds__(kThreads)
hc_checkpoint_pack_kernel(const S *X, uint8_t *Q, uint8_t *E, int64_t rows, int64_t d, int64_t ns, int per_row) {
    constexpr int V = StorageTraits<S>::V, VP = V / 2, LB = kCkBlock / V;
    constexpr int CH = 32 * V;  // elements of a chunk
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    ChunkWalk w(warp, (int64_t)gridDim.x * (kThreads / 32), per_row);
    while (w.row < rows) {
        uint4 raw[kUnroll];
        int64_t row[kUnroll];
        int64_t col[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            row[u] = w.row;
            col[u] = (int64_t)w.chunk * CH + lane * V;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (row[u] < rows && col[u] < d) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(X + row[u] * d + col[u]));
            w.next();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float2 v[VP];
            ck_widen(raw[u], v);
            uint32_t q[V / 4], e;
            ck_encode<VP>(v, q, e);
            if (row[u] < rows && col[u] < d) {
                ck_store<V>(Q + row[u] * d + col[u], q);
                if (lane % LB == 0) E[row[u] * ns + col[u] / kCkBlock] = (uint8_t)e;
            }
        }
    }
}

template <typename S>
__global__ void __launch_bounds__(kThreads)
hc_checkpoint_unpack_kernel(const uint8_t *Q, const uint8_t *E, S *X, int64_t rows, int64_t d, int64_t ns,
                            int per_row) {
    constexpr int V = StorageTraits<S>::V, VP = V / 2;
    constexpr int CH = 32 * V;
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    ChunkWalk w(warp, (int64_t)gridDim.x * (kThreads / 32), per_row);
    while (w.row < rows) {
        uint32_t q[kUnroll][V / 4], e[kUnroll];
        int64_t row[kUnroll];
        int64_t col[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            row[u] = w.row;
            col[u] = (int64_t)w.chunk * CH + lane * V;
            e[u] = 1;
#pragma unroll
            for (int x = 0; x < V / 4; ++x) q[u][x] = 0;
            if (row[u] < rows && col[u] < d) {
                ck_load<V>(Q + row[u] * d + col[u], q[u]);
                e[u] = __ldg(E + row[u] * ns + col[u] / kCkBlock);
            }
            w.next();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float2 v[VP];
            ck_decode<VP>(q[u], ck_scale(e[u]), v);
            if (row[u] < rows && col[u] < d) __stcs(reinterpret_cast<uint4 *>(X + row[u] * d + col[u]), ck_narrow(v));
        }
    }
}

// CTAs: enough for every chunk once, at most eight a multiprocessor (four are
// resident at unpacking's 58 registers; fewer or more CTAs were not faster).
int64_t grid_for(int64_t rows, int per_row, const LaunchCtx &ctx) {
    const int64_t chunks = rows * per_row, per_cta = kThreads / 32;
    int64_t grid = (chunks + per_cta - 1) / per_cta;
    const int64_t most = (int64_t)ctx.sms * 8;
    return grid < most ? grid : most;
}

template <typename S>
hc_status launch_pack(const void *X, uint8_t *q, uint8_t *s, int64_t rows, int64_t d, const LaunchCtx &ctx,
                      cudaStream_t st) {
    const int per_row = (int)((d + 32 * StorageTraits<S>::V - 1) / (32 * StorageTraits<S>::V));
    hc_checkpoint_pack_kernel<S><<<(unsigned)grid_for(rows, per_row, ctx), kThreads, 0, st>>>(
        static_cast<const S *>(X), q, s, rows, d, ck_scale_stride(d), per_row);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(HC_ERR_CUDA, "hc_checkpoint_pack_kernel launch: %s", cudaGetErrorString(e));
    return HC_OK;
}

template <typename S>
hc_status launch_unpack(const uint8_t *q, const uint8_t *s, void *X, int64_t rows, int64_t d, const LaunchCtx &ctx,
                        cudaStream_t st) {
    const int per_row = (int)((d + 32 * StorageTraits<S>::V - 1) / (32 * StorageTraits<S>::V));
    hc_checkpoint_unpack_kernel<S><<<(unsigned)grid_for(rows, per_row, ctx), kThreads, 0, st>>>(
        q, s, static_cast<S *>(X), rows, d, ck_scale_stride(d), per_row);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return set_error(HC_ERR_CUDA, "hc_checkpoint_unpack_kernel launch: %s", cudaGetErrorString(e));
    return HC_OK;
}

}  // namespace

hc_status launch_checkpoint_pack(const void *X, hc_dtype dt, uint8_t *q, uint8_t *s, int64_t rows, int64_t d,
                                 const LaunchCtx &ctx, cudaStream_t st) {
    return dt == HC_BF16 ? launch_pack<__nv_bfloat16>(X, q, s, rows, d, ctx, st)
                         : launch_pack<float>(X, q, s, rows, d, ctx, st);
}

hc_status launch_checkpoint_unpack(const uint8_t *q, const uint8_t *s, void *X, hc_dtype dt, int64_t rows, int64_t d,
                                   const LaunchCtx &ctx, cudaStream_t st) {
    return dt == HC_BF16 ? launch_unpack<__nv_bfloat16>(q, s, X, rows, d, ctx, st)
                         : launch_unpack<float>(q, s, X, rows, d, ctx, st);
}

}  // namespace hc
