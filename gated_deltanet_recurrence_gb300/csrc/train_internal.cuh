// train_internal.cuh -- what the kernels of the training form share (not part of the ABI).
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

// Launches a kernel.  A failure is returned and not left in the runtime, where the launch check of the next call
// would take it for its own.
template <class... P, class... A>
cudaError_t launch_config(const cudaLaunchConfig_t& cfg, void (*kernel)(P...), A... args) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// Launches a kernel that begins with dependency_wait() behind the kernel before it on the stream: its
// launch overlaps that kernel's end, and what that kernel wrote is seen after the wait.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return launch_config(cfg, kernel, args...);
}
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- launchers (called from abi.cu after argument checks) -----------------------------------

// Gradients of the output norms: RMS norm (rms = 1, groups = 1, bias null) and group norm.
struct NormArgs {
    const void* y; gdn_dtype y_dtype; const float* z; const float* w; const float* b; float eps;
    void* out; gdn_dtype out_dtype;                                       // forward
    const void* dout; gdn_dtype dout_dtype; void* dy; float* dz; float* dw; float* db;  // backward
    long rows; int groups, size, rms; float* partial;
};
cudaError_t launch_groupnorm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s);
size_t norm_bwd_workspace_bytes(long rows, int groups, int size);

struct GatePrepBwdArgs {
    const float* a; const float* A_log; const float* dt_bias; const float* b;
    const float* dg; const float* dbeta; float* da; float* dA_log; float* ddt; float* db;
    long total_T; int H; float* partial;
};
cudaError_t launch_gate_prep_bwd(const GatePrepBwdArgs& a, cudaStream_t s);
size_t gate_prep_bwd_workspace_bytes(long total_T, int H);

// Gradients of the chunked form (chunk_bwd.cu).
struct ChunkBwdArgs {
    const void* q; const void* k; const void* v; const float* g; const float* beta;
    const int32_t* cu_seqlens; int num_seqs, total_T, H, Hk, d; gdn_dtype qkv_dtype;
    float scale; int use_l2; const float* initial_state;
    const void* dout; gdn_dtype dout_dtype; const float* dfinal_state;
    void* dq; void* dk; void* dv; float* dg; float* dbeta; float* dinitial_state;
    void* workspace; int* err;
};
size_t chunk_bwd_workspace_bytes(int num_seqs, int total_T, int H, int Hk, int d);
cudaError_t launch_chunk_bwd(const ChunkBwdArgs& a, cudaStream_t s);
cudaError_t launch_chunk_bwd_zero_outside(const ChunkBwdArgs& a, cudaStream_t s);

}  // namespace gdn
