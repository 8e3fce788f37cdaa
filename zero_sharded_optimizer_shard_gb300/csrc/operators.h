// Launch descriptions of the vocabulary operators, the gradient lists and the
// verification of drafted tokens, shared by their C ABI (operators.cpp, clip.cpp)
// and their kernels.
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

// Gradient tensors, cut into blocks of `per` 8-element chunks; a launch takes
// up to MAXT of them.  Every tensor has a block at least, so that its norm is
// written; block0[i] is the first block of tensor i in the launch.
constexpr int kSmallList = 64, kLargeList = 1024;
template <int MAXT>
struct ListArgs {
    const void* x[MAXT];
    void* out[MAXT];       // clipping only
    int64_t numel[MAXT];
    uint32_t block0[MAXT + 1];
    int32_t count;
    int64_t per;
    double* partial;       // norms: a sum of squares per block, from this launch's first block on
    int32_t* start;        // norms: number of the first block of each tensor
    int32_t first;         // of this launch's blocks
    const float* scale;    // clipping: the factor
};

// Sums of squares -> norms and the clipping coefficient.
struct NormArgs {
    const double* partial;  // n sums of blocks
    int64_t n;
    const double* folded;   // the same in fewer numbers
    int64_t n_folded;
    const int32_t* start;   // first block of each tensor
    int64_t n_tensors;
    float* tensor_norms;
    double* square_sum;
    float* norm;
    float* coef;
    float max_norm;
    int32_t accumulate;     // *square_sum is added to
};
// Sums of more blocks than this are folded by a kernel of their own first.
constexpr int64_t kFoldAbove = 16384;
constexpr int kFoldBlocks = 1024;

// Blocks of one gradient tensor.
inline int64_t list_blocks(int64_t numel, int64_t per) {
    const int64_t b = (numel / 8 + per - 1) / per;
    return b < 1 ? 1 : b;
}

// An inverse temperature a as weights are formed with it: of x relative to the row's
// largest logit m, exp(a (x - m)) = 2^((x h - m h) (c + cl)), z = a / h; h is 1, or in a
// FarScale a power of two.
struct LogitScale {
    float c, cl, z;
};
struct FarScale : LogitScale {
    float h;
};

struct VerifyArgs {
    const void* x;
    const void* y;          // draft logits, or null: the draft is certain of its tokens
    const void* ids;
    const float* uniform;
    const float* noise;
    int32_t* accepted;
    int32_t* tokens;
    float* logprobs;
    int64_t n, stride, y_stride, noise_stride;
    int32_t vocab, k;
    float scale, y_scale;    // inverse temperatures
    int32_t dtype, y_dtype, id64;
    int32_t cluster, ahead;  // blocks per sequence, positions per round (set by the launch)
    float sum_error;         // relative, of a row's sum (set by the launch)
};

int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim);

cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t stream);
cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t stream);
cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream);
cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t stream);
cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream);
cudaError_t launch_distill_grad(const DistillArgs& a, cudaStream_t stream);
cudaError_t launch_list_norm(const ListArgs<kSmallList>& a, int dtype, cudaStream_t stream);
cudaError_t launch_list_norm(const ListArgs<kLargeList>& a, int dtype, cudaStream_t stream);
cudaError_t launch_list_scale(const ListArgs<kSmallList>& a, int dtype, int out_dtype, cudaStream_t stream);
cudaError_t launch_list_scale(const ListArgs<kLargeList>& a, int dtype, int out_dtype, cudaStream_t stream);
// Folds a.partial into `to` (kFoldBlocks numbers) if there are many, then
// writes the norms.
cudaError_t launch_norms(NormArgs a, double* to, cudaStream_t stream);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);

}  // namespace z3
