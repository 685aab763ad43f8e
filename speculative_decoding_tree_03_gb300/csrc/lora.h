// lora.h -- one lora_proj call, shared by its two kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace svf {

struct LoraArgs {
    const void *x;       // [R, H] bf16, rows x_stride elements apart
    long long x_stride;
    const void *weight;  // [O, H] bf16
    const void *lora_a;  // [adapters, rank, H] bf16
    const void *lora_b;  // [adapters, O, rank] bf16
    const float *scales; // [adapters] or null
    const int32_t *ids;  // [R / rows_per_id]
    int rows_per_id, R, H, O, adapters, rank;
    void *y;             // [R, O] bf16, rows y_stride elements apart
    long long y_stride;
    void *workspace;     // t [2, R, rank] bf16: hi + lo
    int32_t *status;     // [R / rows_per_id]
};

// t = scale * x A^T of every row's own adapter, and the status words (lora_shrink.cu).
// wait_ns: the deadline of its wait.
cudaError_t launch_lora_shrink(const LoraArgs &a, unsigned long long wait_ns, cudaStream_t stream);

}  // namespace svf
