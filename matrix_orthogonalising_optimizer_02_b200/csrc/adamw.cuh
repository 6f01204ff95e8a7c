// Kernel-level interface of the global gradient norm and of AdamW.
#pragma once
#include <cuda_runtime.h>

namespace muon {

// One dense tensor of a launch; the norm reads G alone.
struct alignas(16) AdamItem {
    void* W;
    const void* G;
    float* m;
    float* v;
    long long n;
    long long chunk0;
    int w_dtype, g_dtype;
    int vec;        // bit 0: G, bit 1: m and v, bit 2: W are 16-byte aligned
};
struct AdamParams {
    float lr, beta1, beta2, omb1, omb2, eps, decay;   // omb: 1 - beta; decay: 1 - lr * weight decay
    float c1, c2;                                     // 1 / (1 - beta^t), unless `step` gives t
    double beta1_d, beta2_d;
    const long long* step;                            // device step count (nullable)
    const float* gscale;                              // device factor of G (nullable: 1)
};
constexpr int kAdamMaxItems = 256;
constexpr int kAdamChunk = 4096;
constexpr int kAdamCtasPerSm = 8;

// `partials` holds kAdamCtasPerSm * num_sms doubles for every kAdamMaxItems tensors begun.
cudaError_t grad_norm_launch(const AdamItem* items, int n, double* partials, float max_norm, float* out,
                             unsigned* status, int num_sms, cudaStream_t stream);
cudaError_t adamw_launch(const AdamItem* items, int n, const AdamParams& h, int num_sms, cudaStream_t stream);

}  // namespace muon
