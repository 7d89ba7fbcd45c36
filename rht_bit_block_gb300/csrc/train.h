// Internal launch interface of the training-step operators between the GEMMs
// (residual RMS norm and gated activation with 8-bit checkpoints, vocabulary
// loss): between their C entry points (train_api.cu) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ufp4 {

// SM count of the current device, with every kernel of the library loaded (api.cu).
int current_num_sms();

// One matrix of 8-bit checkpoints (ckpt8.cuh): codes rows x cols bytes, scales
// rows x ceil(cols / 32) bytes.
struct Ckpt {
    uint8_t* codes;
    uint8_t* scales;
    int64_t codes_ld, scales_ld;
};

struct GluArgs {
    const void* gate;   // forward
    const void* up;
    int64_t ld_gate, ld_up;
    const void* dy;     // backward
    int64_t ld_dy;
    bool f32;           // type of gate and up, or of dy
    int act;
    int64_t rows, cols;
    Ckpt cg, cu;
    bool ckpt;          // forward: write the checkpoints
    void* y;            // bf16; may be null in the backward pass
    int64_t ldy;
    void* dgate;        // bf16
    void* dup;
    int64_t ld_dgate, ld_dup;
};
cudaError_t launch_glu(const GluArgs& a, cudaStream_t st);
cudaError_t launch_glu_backward(const GluArgs& a, cudaStream_t st);
cudaError_t preload_glu_kernels();

struct NormArgs {
    const void* x;         // forward: bf16 or fp32
    const void* residual;  // bf16 or null
    const void* dy;        // backward: bf16 or fp32
    const void* dtotal;    // bf16 or null
    int64_t ldx, ld_residual, ld_dy, ld_dtotal;
    bool f32;              // type of x or dy
    const void* gamma;
    bool gamma_f32;
    int64_t rows, cols;
    float eps;
    void* y;               // bf16; may be null in the backward pass
    int64_t ldy;
    void* total;           // bf16 or null
    int64_t ld_total;
    float* rstd;
    Ckpt ck;
    bool ckpt;             // forward: write the checkpoint
    void* dx;              // bf16
    int64_t ld_dx;
    float* dgamma;
    float* partials;       // norm_parts() x cols
};
constexpr int64_t kNormMaxCols = 32768;
// Row groups whose dgamma sums the backward pass writes apart.
int norm_parts(int64_t rows, int64_t cols, int num_sms);
cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_rms_norm_backward(const NormArgs& a, int num_sms, cudaStream_t st);
cudaError_t preload_norm_kernels();

struct HeadArgs {
    const void* h;  // bf16 [T x K]
    int64_t ldh;
    const void* w;  // bf16 [V x K]
    int64_t ldw;
    const int64_t* targets;
    int64_t T, V, K;
    float z;
    float* loss;    // forward
    float* lse;     // written by the forward pass, read by the backward pass
    const float* weight;
    const float* scale;
    void* dh;       // may be null
    int64_t ld_dh;
    bool dh_f32;
    void* dw;       // may be null
    int64_t ld_dw;
    bool dw_f32, accumulate;
    void* workspace;
};
size_t head_loss_bytes(int64_t T, int64_t V, int64_t K, int num_sms);
size_t head_loss_backward_bytes(int64_t T, int64_t V, int64_t K, int num_sms);
cudaError_t launch_head_loss(const HeadArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_head_loss_backward(const HeadArgs& a, int num_sms, cudaStream_t st);
cudaError_t head_error_read_clear(int* value);
// Polls of a stage's arrival before the products give up, up to their default.
cudaError_t set_head_wait_limit(uint32_t polls);
cudaError_t preload_head_kernels();

}  // namespace ufp4
