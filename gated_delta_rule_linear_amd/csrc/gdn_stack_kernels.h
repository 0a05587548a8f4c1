// Host-side launchers of the kernels around the layer (include/gdn_stack.h).
// Sizes and alignment are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct QkNormLaunch {
    const void *x[2];    // queries, keys
    const void *dy[2];   // gradients of the outputs (backward)
    int64_t stride[2], out_stride[2];
    void* out[2];        // outputs, or the inputs' gradients
    const float* weight[2];
    float* d_weight[2];
    int32_t heads[2];
    int64_t T;
    int32_t d, norm;
    float eps;
    const int32_t* positions;
    const float* inv_freq;
    int32_t rotary;
    bool interleaved;
    float q_scale;
    bool bf16;
    void* workspace;
};
hipError_t launch_qk_norm(const QkNormLaunch& p, hipStream_t stream);
size_t qk_norm_backward_workspace_bytes(int64_t T, int32_t H, int32_t H_k, int32_t d);
hipError_t launch_qk_norm_backward(const QkNormLaunch& p, hipStream_t stream);

struct ScanLaunch {
    const void* x;
    const float* g;
    const int32_t* cu_seqlens;
    int32_t num_seqs;
    int64_t T;
    int32_t C;
    bool mix;
    const float* initial_state;
    float* final_state;
    void* h;
    float* checkpoints;
    const void* d_h;
    const float* d_final_state;
    void* dx;
    float *dg, *d_initial_state;
    bool bf16;
    void* workspace;
};
size_t scan_checkpoint_bytes(int64_t T, int32_t C);
size_t scan_workspace_bytes(int64_t T, int32_t C);
size_t scan_backward_workspace_bytes(int64_t T, int32_t C);
hipError_t launch_scan(const ScanLaunch& p, hipStream_t stream);
hipError_t launch_scan_backward(const ScanLaunch& p, hipStream_t stream);

struct ScanPoolLaunch {
    const void* x;
    const float* g;
    float* states;
    const int32_t *slots, *cu_seqlens, *commit;
    int32_t num_seqs;
    int64_t T;
    int32_t num_slots, C;
    bool mix;
    void* h;
    bool bf16;
};
hipError_t launch_scan_pool(const ScanPoolLaunch& p, hipStream_t stream);

}  // namespace gdn
