// hc_launch.h -- internal interface between the C-ABI host layer (hc_api.cu)
// and the kernel translation units (one per storage dtype and kernel kind).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "hc_api.h"
#include "hc_device.cuh"

namespace hc {

constexpr int kSmemLimitLogits = 232448;  // 227 KB opt-in dynamic shared memory per CTA

struct LaunchCtx {
    int device;  // current device ordinal
    int sms;     // SMs of the current device
    int *fault;  // device fault word of the current device
    int path;    // hc_path: 0 auto, 1 pipelined, 2 register-streaming
};

// Record the calling thread's error text and return st.
hc_status set_error(hc_status st, const char *fmt, ...);

// The result of a driver call, made again with the current device's context
// bound to this host thread if there was none (a thread may make its first call
// here; runtime calls bind the context themselves, driver calls do not).
template <typename Call>
CUresult with_context(Call &&call) {
    CUresult r = call();
    if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = call();
    }
    return r;
}

// Let `kern` be launched with up to `bytes` of dynamic shared memory on the
// current device, once per device (done: one flag a device, of this kernel).
// `bytes` is the most that any launch of it asks for, not this call's need: the
// setting is the process's, and a call on another host thread that lowered it
// between here and this call's launch would have the launch refused.
inline hc_status opt_in_smem(const void *kern, int bytes, std::atomic<bool> (&done)[64], const LaunchCtx &ctx) {
    if (ctx.device < 0 || ctx.device >= 64)
        return set_error(HC_ERR_UNSUPPORTED, "device ordinal %d >= 64", ctx.device);
    if (done[ctx.device].load(std::memory_order_acquire)) return HC_OK;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess)
        return set_error(HC_ERR_CUDA, "cudaFuncSetAttribute(%d B smem): %s", bytes, cudaGetErrorString(e));
    done[ctx.device].store(true, std::memory_order_release);
    return HC_OK;
}

// Launch one step kind (KIND_READ / KIND_WRITE / KIND_FUSED) for n streams.
template <typename S, int KIND>
hc_status launch_kind(int n, const StepParams &p, const LaunchCtx &ctx, cudaStream_t st);
// The kernel family launch_kind would take for p: 1 pipelined, 2 register-streaming.
template <typename S, int KIND>
int step_path(int n, const StepParams &p, const LaunchCtx &ctx);

// 2-D bf16 TMA tensor map over a row-major [outer][inner] array: 128-byte
// swizzle, zero fill out of bounds, box of box_outer rows x box_inner elements.
hc_status make_tma_map_bf16(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
                            uint32_t box_inner, uint32_t box_outer);

// Input-dependent mixing logits on the tensor cores (bf16 H and W).
hc_status launch_mix_logits(const void *H, const void *W, float *z, int64_t T, int n, int64_t d,
                            int P, float eps, const LaunchCtx &ctx, cudaStream_t st);

// The block's output projection fused with the write mix (bf16):
// y = X Wo^T on the tensor cores, H'_j = sum_i A[i][j] H_i + b_j y.
struct LinearWriteArgs {
    const void *X, *Wo, *H;
    void *Hout, *y;  // y may be null
    int64_t T, d, k;
    int n;
    const float *A;
    int64_t A_s;
    const float *b;
    int64_t b_s;
};
hc_status launch_linear_write(const LinearWriteArgs &a, const LaunchCtx &ctx, cudaStream_t st);

// Backward pass of the fused step (see hc_write_then_read_backward).
struct BackwardArgs {
    StepParams f;  // forward inputs: H, y, A, b, a, g, eps, K, modes, T, d
    int n;
    hc_dtype dt;
    const void *dHout;  // [T][n][d] or null
    const void *dx;     // [T][d]
    void *dH;           // [T][n][d]
    void *dy;           // [T][d]
    float *dA, *db, *da, *dg;
    void *workspace;
    size_t workspace_bytes;
};
// Workspace the backward needs for the gain gradient on the current device.
hc_status backward_workspace_bytes(int n, hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx,
                                   size_t *bytes);
hc_status launch_backward(const BackwardArgs &a, const LaunchCtx &ctx, cudaStream_t st);

// The part of a backward after the streams' kernel: refused (before any
// launch) when the Sinkhorn iterates do not fit; then the softmax and Sinkhorn
// backward in place on a.da and a.dA, and a.dg from `rows` rows of a.workspace.
hc_status check_param_backward(const BackwardArgs &a);
hc_status launch_backward_tail(const BackwardArgs &a, int64_t rows, const LaunchCtx &ctx, cudaStream_t st);

// 8-bit checkpoints (hc_checkpoint.cuh): rows of d values to codes and
// exponents and back, and the step's backward from those of H and y (a.f.H and
// a.f.y hold the codes).
hc_status launch_checkpoint_pack(const void *X, hc_dtype dt, uint8_t *q, uint8_t *s, int64_t rows, int64_t d,
                                 const LaunchCtx &ctx, cudaStream_t st);
hc_status launch_checkpoint_unpack(const uint8_t *q, const uint8_t *s, void *X, hc_dtype dt, int64_t rows, int64_t d,
                                   const LaunchCtx &ctx, cudaStream_t st);
hc_status checkpoint_backward_workspace_bytes(int n, hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx,
                                              size_t *bytes);
hc_status launch_checkpoint_backward(const BackwardArgs &a, const uint8_t *sH, const uint8_t *sy,
                                     const LaunchCtx &ctx, cudaStream_t st);

// The read with layer norm, and its gradients (see hc_read_layernorm).
struct LayerNormArgs {
    StepParams f;         // H (rows of dt, or codes), x, a (null: weight 1, n == 1), g, eps, T, d
    int n;
    hc_dtype dt;
    const float *beta;    // forward
    const uint8_t *sH;    // backward: exponents of a checkpoint, or null when H holds rows of dt
    const void *dx;
    void *dH;
    float *da, *dg, *dbeta;  // each may be null
    void *workspace;
    size_t workspace_bytes;
};
hc_status launch_layernorm(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st);
hc_status layernorm_backward_workspace_bytes(int n, hc_dtype dt, int64_t T, int64_t d, const LaunchCtx &ctx,
                                             size_t *bytes);
hc_status launch_layernorm_backward(const LayerNormArgs &a, const LaunchCtx &ctx, cudaStream_t st);

// The write mix fused with the tensor-parallel all-reduce of y, then the
// next layer's read (see hc_reduce_write_then_read).
constexpr int kMaxRanks = 8;
struct ReduceWriteArgs {
    StepParams f;                  // H, Hout, params, T (tokens of this call), d (f.y, f.x unused)
    const void *parts[kMaxRanks];  // the ranks' partial y, in rank order
    int R;
    int n;
    void *y_out;                   // reduced y [T][d] (this call's tokens), or null
    int64_t t0;                    // row of the partials and of x for this call's token 0
    void *xs[kMaxRanks];           // x_next destinations (rows t0 .. t0 + T - 1 of each)
    int nx;
};
hc_status launch_reduce_write(const ReduceWriteArgs &ra, hc_dtype dt, const LaunchCtx &ctx,
                              cudaStream_t st);
// Its pipelined (TMA-fed) form; local[r] marks partials in this GPU's memory
// (staged by bulk copies; the others are read with plain loads). Launches
// nothing and sets *fits = false when the ring does not fit shared memory.
template <typename S>
hc_status launch_reduce_pipe(const ReduceWriteArgs &ra, const bool *local, const LaunchCtx &ctx,
                             cudaStream_t st, bool *fits);

hc_status launch_selftest_wait(int limit_us, const LaunchCtx &ctx, cudaStream_t st);

hc_status launch_sinkhorn(const float *L, float *out, int64_t T, int n, int K,
                          const LaunchCtx &ctx, cudaStream_t st);

}  // namespace hc
