// Instantiation of the step launcher for storage dtype f32, the fused step that keeps a checkpoint.
#include "hc_kernels_impl.cuh"

template hc_status hc::launch_kind<float, hc::KIND_SAVE>(int, const hc::StepParams &, const hc::LaunchCtx &,
                                                       cudaStream_t);
