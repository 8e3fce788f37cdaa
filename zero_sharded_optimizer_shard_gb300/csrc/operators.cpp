// C ABI of the vocabulary operators: argument checks and launches.
#include <cmath>
#include <cstdint>

#include "operators.h"

namespace {

constexpr int64_t kMaxVocab = int64_t{1} << 30;   // token ids and row offsets are 32-bit
constexpr int64_t kMaxRows = int64_t{1} << 27;    // rows times blocks per row fit a grid
constexpr int64_t kMaxDim = int64_t{1} << 27;     // embedding columns are 32-bit
// rows times columns (4 TB of bf16); with kMaxRows this keeps the elementwise
// gradients' blocks, one per 4096 elements of a row, below 2^29 + 2^27
constexpr int64_t kMaxElems = int64_t{1} << 41;

zero3_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ZERO3_OK : ZERO3_ECUDA; }

bool dtype_ok(zero3_dtype t) { return t == ZERO3_BF16 || t == ZERO3_F32; }
bool itype_ok(zero3_itype t) { return t == ZERO3_I32 || t == ZERO3_I64; }

int64_t size_of(zero3_dtype t) { return t == ZERO3_F32 ? 4 : 2; }
int64_t size_of(zero3_itype t) { return t == ZERO3_I64 ? 8 : 4; }

// Present and aligned to its elements.
bool ptr_ok(const void* p, int64_t size) {
    return p && reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(size) == 0;
}
// Absent, or aligned to its elements.
bool opt_ok(const void* p, int64_t size) { return !p || ptr_ok(p, size); }

bool positive(float x) { return std::isfinite(x) && x > 0.0f; }

// n rows of `cols` elements, `stride` apart (the stride of a single row is
// not used).
bool rows_ok(int64_t n, int64_t cols, int64_t stride) {
    return n >= 0 && n <= INT32_MAX && cols >= 1 && stride >= cols &&
           (n == 0 || cols <= kMaxElems / n);
}

bool logits_ok(int64_t n, int64_t vocab, int64_t stride) {
    return n <= kMaxRows && vocab <= kMaxVocab && rows_ok(n, vocab, stride);
}

// Bytes of n rows of `cols` elements of `size` bytes, and whether two ranges have
// one in common.
struct Bytes {
    const void* at;
    unsigned __int128 size;
};
Bytes rows_bytes(const void* p, int64_t n, int64_t cols, int64_t stride, int64_t size) {
    if (!p || n <= 0) return Bytes{p, 0};
    return Bytes{p, (static_cast<unsigned __int128>(n - 1) * static_cast<uint64_t>(stride) +
                     static_cast<uint64_t>(cols)) * static_cast<uint64_t>(size)};
}
bool overlap(const Bytes& a, const Bytes& b) {
    const unsigned __int128 a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
    return a.size > 0 && b.size > 0 && a0 < b0 + b.size && b0 < a0 + a.size;
}

// An embedding's two matrices.
bool embedding_ok(int64_t vocab, int64_t dim, int64_t table_stride, int64_t n, int64_t row_stride) {
    return vocab >= 1 && vocab <= kMaxVocab && dim <= kMaxDim && rows_ok(vocab, dim, table_stride) &&
           rows_ok(n, dim, row_stride);
}

}  // namespace

extern "C" {

zero3_status zero3_embedding_forward(const void* table, zero3_dtype table_dtype, int64_t vocab,
                                     int64_t dim, int64_t table_stride, const void* ids,
                                     zero3_itype id_type, int64_t n, float scale, void* out,
                                     zero3_dtype out_dtype, int64_t out_stride,
                                     zero3_stream stream) {
    if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype) || !itype_ok(id_type)) return ZERO3_EINVAL;
    if (!embedding_ok(vocab, dim, table_stride, n, out_stride) || !std::isfinite(scale))
        return ZERO3_EINVAL;
    if (n == 0) return ZERO3_OK;
    if (!ptr_ok(table, size_of(table_dtype)) || !ptr_ok(ids, size_of(id_type)) ||
        !ptr_ok(out, size_of(out_dtype)))
        return ZERO3_EINVAL;
    z3::EmbedArgs a;
    a.table = table;
    a.ids = ids;
    a.out = out;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.table_stride = table_stride;
    a.out_stride = out_stride;
    a.scale = scale;
    a.table_dtype = table_dtype;
    a.out_dtype = out_dtype;
    a.id64 = id_type == ZERO3_I64;
    return cuda_status(z3::launch_embed(a, stream));
}

zero3_status zero3_embedding_workspace(int64_t n, int64_t vocab, int64_t dim, int64_t* bytes) {
    if (!bytes || !embedding_ok(vocab, dim, dim, n, dim)) return ZERO3_EINVAL;
    *bytes = z3::embed_grad_workspace(n, vocab, dim);
    return ZERO3_OK;
}

zero3_status zero3_embedding_backward(const void* dout, zero3_dtype dout_dtype, int64_t dout_stride,
                                      const void* ids, zero3_itype id_type, int64_t n, float scale,
                                      int32_t accumulate, void* grad, zero3_dtype grad_dtype,
                                      int64_t vocab, int64_t dim, int64_t grad_stride,
                                      void* workspace, int64_t workspace_bytes,
                                      zero3_stream stream) {
    if (!dtype_ok(dout_dtype) || !dtype_ok(grad_dtype) || !itype_ok(id_type)) return ZERO3_EINVAL;
    if (!embedding_ok(vocab, dim, grad_stride, n, dout_stride) || !std::isfinite(scale))
        return ZERO3_EINVAL;
    if (n == 0 && accumulate) return ZERO3_OK;
    if (!ptr_ok(grad, size_of(grad_dtype)) || !ptr_ok(workspace, 16) ||
        workspace_bytes < z3::embed_grad_workspace(n, vocab, dim))
        return ZERO3_EINVAL;
    if (n > 0 && (!ptr_ok(dout, size_of(dout_dtype)) || !ptr_ok(ids, size_of(id_type))))
        return ZERO3_EINVAL;
    z3::EmbedGradArgs a;
    a.dout = dout;
    a.ids = ids;
    a.grad = grad;
    a.workspace = workspace;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.dout_stride = dout_stride;
    a.grad_stride = grad_stride;
    a.scale = scale;
    a.dout_dtype = dout_dtype;
    a.grad_dtype = grad_dtype;
    a.id64 = id_type == ZERO3_I64;
    a.accumulate = accumulate ? 1 : 0;
    return cuda_status(z3::launch_embed_grad(a, stream));
}

zero3_status zero3_token_logprobs(const void* logits, zero3_dtype dtype, int64_t n, int64_t vocab,
                                  int64_t stride, const void* targets, zero3_itype id_type,
                                  float inv_temperature, int32_t k, float* logprob, float* lse,
                                  float* entropy, int32_t* top_ids, float* top_logprobs,
                                  zero3_stream stream) {
    if (!dtype_ok(dtype) || !itype_ok(id_type) || !logits_ok(n, vocab, stride) ||
        !positive(inv_temperature) || k < 0 || k > ZERO3_MAX_TOP || k > vocab)
        return ZERO3_EINVAL;
    if (n == 0) return ZERO3_OK;
    if (!ptr_ok(logits, size_of(dtype)) || !ptr_ok(targets, size_of(id_type)) ||
        !ptr_ok(logprob, 4) || !opt_ok(lse, 4) || !opt_ok(entropy, 4))
        return ZERO3_EINVAL;
    if (k > 0 && (!ptr_ok(top_ids, 4) || !ptr_ok(top_logprobs, 4))) return ZERO3_EINVAL;
    z3::LogprobArgs a;
    a.x = logits;
    a.targets = targets;
    a.logprob = logprob;
    a.lse = lse;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.n = n;
    a.stride = stride;
    a.vocab = static_cast<int32_t>(vocab);
    a.k = k;
    a.scale = inv_temperature;
    a.dtype = dtype;
    a.id64 = id_type == ZERO3_I64;
    a.cluster = 1;
    return cuda_status(z3::launch_logprobs(a, stream));
}

zero3_status zero3_token_logprobs_backward(const void* logits, zero3_dtype dtype, int64_t n,
                                           int64_t vocab, int64_t stride, const void* targets,
                                           zero3_itype id_type, float inv_temperature,
                                           const float* lse, const float* entropy,
                                           const float* dlogprob, const float* dentropy,
                                           void* dlogits, int64_t dlogits_stride,
                                           zero3_stream stream) {
    if (!dtype_ok(dtype) || !itype_ok(id_type) || !logits_ok(n, vocab, stride) ||
        !logits_ok(n, vocab, dlogits_stride) || !positive(inv_temperature))
        return ZERO3_EINVAL;
    if (n == 0) return ZERO3_OK;
    if (!ptr_ok(logits, size_of(dtype)) || !ptr_ok(targets, size_of(id_type)) || !ptr_ok(lse, 4) ||
        !opt_ok(entropy, 4) || !opt_ok(dlogprob, 4) || !opt_ok(dentropy, 4) ||
        !ptr_ok(dlogits, size_of(dtype)))
        return ZERO3_EINVAL;
    if ((!dlogprob && !dentropy) || (dentropy && !entropy)) return ZERO3_EINVAL;
    if (dlogits == logits && stride != dlogits_stride && n > 1) return ZERO3_EINVAL;
    z3::LogprobGradArgs a;
    a.x = logits;
    a.targets = targets;
    a.lse = lse;
    a.entropy = entropy;
    a.dlogprob = dlogprob;
    a.dentropy = dentropy;
    a.dx = dlogits;
    a.n = n;
    a.stride = stride;
    a.dx_stride = dlogits_stride;
    a.vocab = static_cast<int32_t>(vocab);
    a.scale = inv_temperature;
    a.dtype = dtype;
    a.id64 = id_type == ZERO3_I64;
    a.segments = 1;
    return cuda_status(z3::launch_logprobs_grad(a, stream));
}

namespace {

// Checks shared by the two distillation calls, and their common arguments.
bool distill_ok(const void* logits, zero3_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                zero3_dtype teacher_dtype, zero3_itype id_type, int32_t k, int64_t teacher_stride,
                float inv_temperature, const void* dlogits, int64_t dlogits_stride) {
    if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype) || !itype_ok(id_type) ||
        !logits_ok(n, vocab, stride) || !positive(inv_temperature) || k < 1 ||
        k > ZERO3_MAX_TEACHER || teacher_stride < k)
        return false;
    if (dlogits && !logits_ok(n, vocab, dlogits_stride)) return false;
    return !(dlogits == logits && stride != dlogits_stride && n > 1);
}

z3::DistillArgs distill_args(const void* logits, zero3_dtype dtype, int64_t n, int64_t vocab,
                             int64_t stride, const void* teacher, zero3_dtype teacher_dtype,
                             const void* teacher_ids, zero3_itype id_type, int32_t k,
                             int64_t teacher_stride, float inv_temperature, const float* weight,
                             void* dlogits, int64_t dlogits_stride) {
    z3::DistillArgs a;
    a.x = logits;
    a.teacher = teacher;
    a.teacher_ids = teacher_ids;
    a.weight = weight;
    a.loss = nullptr;
    a.lse = nullptr;
    a.dx = dlogits;
    a.n = n;
    a.stride = stride;
    a.teacher_stride = teacher_stride;
    a.dx_stride = dlogits_stride;
    a.vocab = static_cast<int32_t>(vocab);
    a.k = k;
    a.scale = inv_temperature;
    a.dtype = dtype;
    a.teacher_dtype = teacher_dtype;
    a.id64 = id_type == ZERO3_I64;
    a.cluster = 1;
    a.map_bytes = 0;
    return a;
}

}  // namespace

zero3_status zero3_distill_loss(const void* logits, zero3_dtype dtype, int64_t n, int64_t vocab,
                                int64_t stride, const void* teacher_logits,
                                zero3_dtype teacher_dtype, const void* teacher_ids,
                                zero3_itype id_type, int32_t k, int64_t teacher_stride,
                                float inv_temperature, const float* row_weight, float* loss,
                                float* lse, void* dlogits, int64_t dlogits_stride,
                                zero3_stream stream) {
    if (!distill_ok(logits, dtype, n, vocab, stride, teacher_dtype, id_type, k, teacher_stride,
                    inv_temperature, dlogits, dlogits_stride))
        return ZERO3_EINVAL;
    if (n == 0) return ZERO3_OK;
    if (!ptr_ok(logits, size_of(dtype)) || !ptr_ok(teacher_logits, size_of(teacher_dtype)) ||
        !ptr_ok(teacher_ids, size_of(id_type)) || !ptr_ok(loss, 4) || !opt_ok(lse, 4) ||
        !opt_ok(row_weight, 4) || !opt_ok(dlogits, size_of(dtype)))
        return ZERO3_EINVAL;
    z3::DistillArgs a = distill_args(logits, dtype, n, vocab, stride, teacher_logits, teacher_dtype,
                                     teacher_ids, id_type, k, teacher_stride, inv_temperature,
                                     row_weight, dlogits, dlogits_stride);
    a.loss = loss;
    a.lse = lse;
    return cuda_status(z3::launch_distill(a, stream));
}

zero3_status zero3_distill_backward(const void* logits, zero3_dtype dtype, int64_t n, int64_t vocab,
                                    int64_t stride, const void* teacher_logits,
                                    zero3_dtype teacher_dtype, const void* teacher_ids,
                                    zero3_itype id_type, int32_t k, int64_t teacher_stride,
                                    float inv_temperature, const float* lse, const float* dloss,
                                    void* dlogits, int64_t dlogits_stride, zero3_stream stream) {
    if (!distill_ok(logits, dtype, n, vocab, stride, teacher_dtype, id_type, k, teacher_stride,
                    inv_temperature, dlogits, dlogits_stride))
        return ZERO3_EINVAL;
    if (n == 0) return ZERO3_OK;
    if (!ptr_ok(logits, size_of(dtype)) || !ptr_ok(teacher_logits, size_of(teacher_dtype)) ||
        !ptr_ok(teacher_ids, size_of(id_type)) || !ptr_ok(lse, 4) || !opt_ok(dloss, 4) ||
        !ptr_ok(dlogits, size_of(dtype)))
        return ZERO3_EINVAL;
    z3::DistillArgs a = distill_args(logits, dtype, n, vocab, stride, teacher_logits, teacher_dtype,
                                     teacher_ids, id_type, k, teacher_stride, inv_temperature, dloss,
                                     dlogits, dlogits_stride);
    a.lse = const_cast<float*>(lse);
    return cuda_status(z3::launch_distill_grad(a, stream));
}

zero3_status zero3_verify_draft(const void* logits, zero3_dtype dtype, int64_t n, int32_t k,
                                int64_t vocab, int64_t stride, const void* draft_logits,
                                zero3_dtype draft_dtype, int64_t draft_stride,
                                const void* draft_ids, zero3_itype id_type, float inv_temperature,
                                float draft_inv_temperature, const float* uniform,
                                const float* noise, int64_t noise_stride, int32_t* accepted,
                                int32_t* tokens, float* logprobs, zero3_stream stream) {
    if (!dtype_ok(dtype) || !itype_ok(id_type) || k < 0 || k > ZERO3_MAX_DRAFT || n < 0 ||
        n > kMaxRows / (k + 1) || !logits_ok(n * (k + 1), vocab, stride) ||
        !positive(inv_temperature) || noise_stride < vocab)
        return ZERO3_EINVAL;
    const bool draft = k > 0 && draft_logits;
    if (draft && (!dtype_ok(draft_dtype) || !logits_ok(n * k, vocab, draft_stride) ||
                  !positive(draft_inv_temperature)))
        return ZERO3_EINVAL;
    if (n == 0) return ZERO3_OK;
    if (!ptr_ok(logits, size_of(dtype)) || !ptr_ok(noise, 4) || !ptr_ok(accepted, 4) ||
        !ptr_ok(tokens, 4) || !opt_ok(logprobs, 4))
        return ZERO3_EINVAL;
    if (draft && !ptr_ok(draft_logits, size_of(draft_dtype))) return ZERO3_EINVAL;
    if (k > 0 && (!ptr_ok(draft_ids, size_of(id_type)) || !ptr_ok(uniform, 4))) return ZERO3_EINVAL;
    // A sequence's blocks each read what decides and have to decide alike: no result
    // of another sequence may change it.
    const Bytes in[] = {rows_bytes(logits, n * (k + 1), vocab, stride, size_of(dtype)),
                        rows_bytes(draft ? draft_logits : nullptr, n * k, vocab, draft_stride,
                                   size_of(draft_dtype)),
                        rows_bytes(draft_ids, n, k, k, size_of(id_type)), rows_bytes(uniform, n, k, k, 4),
                        rows_bytes(noise, n, vocab, noise_stride, 4)};
    const Bytes out[] = {rows_bytes(accepted, n, 1, 1, 4), rows_bytes(tokens, n, k + 1, k + 1, 4),
                         rows_bytes(logprobs, n, k + 1, k + 1, 4)};
    for (const Bytes& o : out)
        for (const Bytes& i : in)
            if (overlap(o, i)) return ZERO3_EINVAL;
    z3::VerifyArgs a;
    a.x = logits;
    a.y = draft ? draft_logits : nullptr;
    a.ids = draft_ids;
    a.uniform = uniform;
    a.noise = noise;
    a.accepted = accepted;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.n = n;
    a.stride = stride;
    a.y_stride = draft_stride;
    a.noise_stride = noise_stride;
    a.vocab = static_cast<int32_t>(vocab);
    a.k = k;
    a.scale = inv_temperature;
    a.y_scale = draft ? draft_inv_temperature : 1.0f;
    a.dtype = dtype;
    a.y_dtype = draft ? draft_dtype : dtype;
    a.id64 = id_type == ZERO3_I64;
    a.cluster = 1;
    a.ahead = 1;
    return cuda_status(z3::launch_verify(a, stream));
}

}  // extern "C"
