// C ABI of the gradient norms and clipping over tensor lists: argument checks
// and launches.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <new>

#include "operators.h"

namespace {

zero3_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ZERO3_OK : ZERO3_ECUDA; }

bool dtype_ok(zero3_dtype t) { return t == ZERO3_BF16 || t == ZERO3_F32; }
uintptr_t size_of(zero3_dtype t) { return t == ZERO3_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

constexpr int64_t kMaxTensors = int64_t{1} << 24;
constexpr int64_t kMaxElems = int64_t{1} << 41;
// Chunks per block: a multiple of what 256 threads load at once; more where the
// blocks would be over this many.
constexpr int64_t kUnit = 1024;
constexpr int64_t kMostBlocks = 4864;  // 32 for each of 152 SMs

bool list_ok(const int64_t* numels, int64_t n, int64_t* per, int64_t* blocks) {
    if (n < 0 || n > kMaxTensors || (n > 0 && !numels)) return false;
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (numels[i] < 0 || numels[i] > kMaxElems - total) return false;
        total += numels[i];
    }
    const int64_t units = total / 8 / kUnit;
    *per = kUnit * (units / kMostBlocks + 1);
    *blocks = 0;
    for (int64_t i = 0; i < n; ++i) *blocks += z3::list_blocks(numels[i], *per);
    return true;
}

// Partial sums, folded sums, each tensor's first block.
int64_t workspace_bytes(int64_t blocks, int64_t n) {
    return ((blocks + z3::kFoldBlocks) * 8 + n * 4 + 15) / 16 * 16;
}

bool tensors_ok(const void* const* x, const int64_t* numels, int64_t n, zero3_dtype dtype) {
    if (n > 0 && !x) return false;
    for (int64_t i = 0; i < n; ++i)
        if (numels[i] > 0 && (!x[i] || !aligned(x[i], size_of(dtype)))) return false;
    return true;
}

// Launches over the list, at most MAXT tensors each.
template <int MAXT, typename Launch>
zero3_status for_tensors(const void* const* x, void* const* out, const int64_t* numels, int64_t n,
                         int64_t per, double* partial, int32_t* start, const float* scale,
                         bool backwards, Launch launch) {
    std::unique_ptr<z3::ListArgs<MAXT>> a(new (std::nothrow) z3::ListArgs<MAXT>);
    if (!a) return ZERO3_ENOMEM;
    const int64_t launches = (n + MAXT - 1) / MAXT;
    int64_t first = 0;
    for (int64_t l = 0; l < launches; ++l) {
        const int64_t t0 = (backwards ? launches - 1 - l : l) * MAXT;
        a->count = static_cast<int32_t>(n - t0 < MAXT ? n - t0 : MAXT);
        a->per = per;
        a->scale = scale;
        a->first = static_cast<int32_t>(first);
        a->partial = partial ? partial + first : nullptr;
        a->start = start ? start + t0 : nullptr;
        int64_t blocks = 0;
        for (int32_t i = 0; i < a->count; ++i) {
            a->x[i] = x[t0 + i];
            a->out[i] = out ? out[t0 + i] : nullptr;
            a->numel[i] = numels[t0 + i];
            a->block0[i] = static_cast<uint32_t>(blocks);
            blocks += z3::list_blocks(numels[t0 + i], per);
        }
        a->block0[a->count] = static_cast<uint32_t>(blocks);
        const zero3_status st = cuda_status(launch(*a));
        if (st != ZERO3_OK) return st;
        first += blocks;
    }
    return ZERO3_OK;
}

}  // namespace

extern "C" {

zero3_status zero3_grad_norm_workspace(const int64_t* numels, int64_t n_tensors, int64_t* bytes) {
    int64_t per, blocks;
    if (!bytes || !list_ok(numels, n_tensors, &per, &blocks)) return ZERO3_EINVAL;
    *bytes = workspace_bytes(blocks, n_tensors);
    return ZERO3_OK;
}

zero3_status zero3_grad_norm(const void* const* tensors, const int64_t* numels, int64_t n_tensors,
                             zero3_dtype dtype, float max_norm, float* tensor_norms,
                             double* square_sum, float* norm, float* coef, void* workspace,
                             int64_t bytes, zero3_stream stream) {
    int64_t per, blocks;
    if (!dtype_ok(dtype) || !list_ok(numels, n_tensors, &per, &blocks) ||
        !tensors_ok(tensors, numels, n_tensors, dtype) || !(max_norm > 0.0f))
        return ZERO3_EINVAL;
    if (!aligned(tensor_norms, 4) || !aligned(square_sum, 8) || !aligned(norm, 4) || !aligned(coef, 4) ||
        (!tensor_norms && !square_sum && !norm && !coef))
        return ZERO3_EINVAL;
    if (!workspace || !aligned(workspace, 16) || bytes < workspace_bytes(blocks, n_tensors))
        return ZERO3_EINVAL;
    double* partial = static_cast<double*>(workspace);
    double* folded = partial + blocks;
    int32_t* start = reinterpret_cast<int32_t*>(folded + z3::kFoldBlocks);
    zero3_status st;
    if (n_tensors <= z3::kSmallList)
        st = for_tensors<z3::kSmallList>(tensors, nullptr, numels, n_tensors, per, partial, start, nullptr,
                                         false, [&](const z3::ListArgs<z3::kSmallList>& a) {
                                             return z3::launch_list_norm(a, dtype, stream);
                                         });
    else
        st = for_tensors<z3::kLargeList>(tensors, nullptr, numels, n_tensors, per, partial, start, nullptr,
                                         false, [&](const z3::ListArgs<z3::kLargeList>& a) {
                                             return z3::launch_list_norm(a, dtype, stream);
                                         });
    if (st != ZERO3_OK) return st;
    z3::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.partial = partial;
    a.n = blocks;
    a.start = start;
    a.n_tensors = n_tensors;
    a.tensor_norms = n_tensors > 0 ? tensor_norms : nullptr;
    a.square_sum = square_sum;
    a.norm = norm;
    a.coef = coef;
    a.max_norm = max_norm;
    return cuda_status(z3::launch_norms(a, folded, stream));
}

zero3_status zero3_clip_coefficient(const double* square_sum, float max_norm, float* norm, float* coef,
                                    zero3_stream stream) {
    if (!square_sum || !aligned(square_sum, 8) || !(max_norm > 0.0f) || !aligned(norm, 4) ||
        !aligned(coef, 4) || (!norm && !coef))
        return ZERO3_EINVAL;
    z3::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.partial = square_sum;
    a.n = 1;
    a.norm = norm;
    a.coef = coef;
    a.max_norm = max_norm;
    return cuda_status(z3::launch_norms(a, nullptr, stream));
}

zero3_status zero3_clip_grads(const void* const* tensors, const int64_t* numels, int64_t n_tensors,
                              zero3_dtype dtype, const float* coef, void* const* out,
                              zero3_dtype out_dtype, zero3_stream stream) {
    int64_t per, blocks;
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype) || !list_ok(numels, n_tensors, &per, &blocks) ||
        !tensors_ok(tensors, numels, n_tensors, dtype) || !coef || !aligned(coef, 4))
        return ZERO3_EINVAL;
    if (!out) {  // in place
        if (dtype != out_dtype) return ZERO3_EINVAL;
        out = const_cast<void* const*>(tensors);
    }
    if (!tensors_ok(out, numels, n_tensors, out_dtype)) return ZERO3_EINVAL;
    for (int64_t i = 0; i < n_tensors; ++i)
        if (numels[i] > 0 && out[i] == tensors[i] && dtype != out_dtype) return ZERO3_EINVAL;
    if (n_tensors <= z3::kSmallList)
        return for_tensors<z3::kSmallList>(tensors, out, numels, n_tensors, per, nullptr, nullptr, coef, true,
                                           [&](const z3::ListArgs<z3::kSmallList>& a) {
                                               return z3::launch_list_scale(a, dtype, out_dtype, stream);
                                           });
    return for_tensors<z3::kLargeList>(tensors, out, numels, n_tensors, per, nullptr, nullptr, coef, true,
                                       [&](const z3::ListArgs<z3::kLargeList>& a) {
                                           return z3::launch_list_scale(a, dtype, out_dtype, stream);
                                       });
}

}  // extern "C"
