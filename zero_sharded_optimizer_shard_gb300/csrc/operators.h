// Launch descriptions of the vocabulary operators, shared by their C ABI
// (operators.cpp) and their kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/zero3.h"

namespace z3 {

struct EmbedArgs {
    const void* table;
    const void* ids;
    void* out;
    int64_t n, vocab, dim;
    int64_t table_stride, out_stride;
    float scale;
    int32_t table_dtype, out_dtype, id64;
};

struct EmbedGradArgs {
    const void* dout;
    const void* ids;
    void* grad;
    void* workspace;
    int64_t n, vocab, dim;
    int64_t dout_stride, grad_stride;
    float scale;
    int32_t dout_dtype, grad_dtype, id64, accumulate;
};

struct LogprobArgs {
    const void* x;
    const void* targets;
    float* logprob;
    float* lse;
    float* entropy;
    int32_t* top_ids;
    float* top_logprobs;
    int64_t n, stride;
    int32_t vocab, k;
    float scale;
    int32_t dtype, id64;
    int32_t cluster;   // blocks per row (set by the launch)
};

struct LogprobGradArgs {
    const void* x;
    const void* targets;
    const float* lse;
    const float* entropy;
    const float* dlogprob;
    const float* dentropy;
    void* dx;
    int64_t n, stride, dx_stride;
    int32_t vocab;
    float scale;
    int32_t dtype, id64;
    int32_t segments;  // blocks per row (set by the launch)
};

struct DistillArgs {
    const void* x;
    const void* teacher;
    const void* teacher_ids;
    const float* weight;   // row weights (gradient), or null: 1
    float* loss;
    float* lse;            // written by the forward pass, read by the backward pass
    void* dx;
    int64_t n, stride, teacher_stride, dx_stride;
    int32_t vocab, k;
    float scale;
    int32_t dtype, teacher_dtype, id64;
    int32_t cluster;       // blocks per row (set by the launch)
    int32_t map_bytes;     // of the map of listed tokens (set by the launch)
};

int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim);

cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t stream);
cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t stream);
cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream);
cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t stream);
cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream);
cudaError_t launch_distill_grad(const DistillArgs& a, cudaStream_t stream);

}  // namespace z3
