// Distillation from a teacher's top logits: loss, loss with gradient in one
// call, and gradient alone (sm_103a).
//
//   q = softmax over the row's valid teacher entries of t_k * scale
//   loss = sum_k q_k (log q_k - log p_{id_k}) / scale^2,  p = softmax(x * scale)
//   d loss / d x_j = (p_j - sum_{k: id_k = j} q_k) / scale
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {
namespace {

// A row's teacher list in shared memory.
struct Teacher {
    float q[ZERO3_MAX_TEACHER];        // probabilities; 0 where the entry does not count
    float x[ZERO3_MAX_TEACHER];        // the student's logits at its tokens
    alignas(16) int32_t id[ZERO3_MAX_TEACHER];  // tokens, -1 where the entry does not count
};

__device__ __forceinline__ float teacher_value(const DistillArgs& a, int64_t r, int k) {
    const int64_t i = r * a.teacher_stride + k;
    return a.teacher_dtype == ZERO3_F32 ? static_cast<const float*>(a.teacher)[i]
                                        : bf16_f32(static_cast<const uint16_t*>(a.teacher)[i]);
}

// Loads row r's list and the student's logits at its tokens, and returns the
// softmax statistics of the list (s = 0: no entry counts).  An entry counts
// if its token lies in the vocabulary and its logit is not -inf.  Leaves
// weights relative to the returned maximum in T.q.  Contains barriers.
template <typename T, int NT>
__device__ __forceinline__ Soft teacher_load(const DistillArgs& a, int64_t r, const T* row,
                                             Teacher& t, Soft* sh) {
    Soft s = soft_empty();
    for (int k = threadIdx.x; k < a.k; k += NT) {
        int32_t id = load_id(a.teacher_ids, a.id64, r * a.teacher_stride + k, a.vocab);
        const float v = teacher_value(a, r, k);
        if (v == neg_inf()) id = -1;
        t.id[k] = id;
        t.q[k] = v;
        t.x[k] = id >= 0 ? to_f32(row[id]) : 0.0f;
        if (id >= 0) s.m = fmaxf(s.m, v);
    }
    s.mz = __fmul_rn(s.m, a.scale);
    if (s.mz == neg_inf()) s.mz = 0.0f;
    for (int k = threadIdx.x; k < a.k; k += NT) {
        if (t.id[k] < 0) continue;
        s.s = __fadd_rn(s.s, exp2_approx(__fmul_rn(fmaf(t.q[k], a.scale, -s.mz), kLog2e)));
    }
    soft_block<false, NT>(s, sh);
    return s;
}

// Turns the list's logits into probabilities and returns this thread's part
// of sum_k q_k (log q_k - (x_k scale - mz - logs)).
template <int NT>
__device__ __forceinline__ float teacher_loss(const DistillArgs& a, Teacher& t, const Soft& s,
                                              float mz, float logs) {
    const float tlog = logf(s.s);
    float sum = 0.0f;
    for (int k = threadIdx.x; k < a.k; k += NT) {
        float q = 0.0f;
        if (t.id[k] >= 0) {
            const float d = fmaf(t.q[k], a.scale, -s.mz);
            q = __fdiv_rn(exp2_approx(__fmul_rn(d, kLog2e)), s.s);
            if (q != 0.0f) {
                const float lp = __fsub_rn(fmaf(t.x[k], a.scale, -mz), logs);
                sum = fmaf(q, __fsub_rn(__fsub_rn(d, tlog), lp), sum);
            }
        }
        t.q[k] = q;
    }
    return sum;
}

template <int NT>
__device__ __forceinline__ float block_sum(float x, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0f;
    for (int w = 0; w < NT / 32; ++w) x = __fadd_rn(x, sh[w]);
    return x;
}

// What a sweep over a row writes: dx_j = coef 2^((x_j scale - base) log2 e),
// less c q_k at the teacher's tokens.
struct Sweep {
    float scale, base, coef, c;
};

__device__ __forceinline__ float sweep_value(float x, const Sweep& w) {
    return __fmul_rn(exp2_approx(__fmul_rn(fmaf(x, w.scale, -w.base), kLog2e)), w.coef);
}

template <typename T>
__device__ __forceinline__ void sweep_chunk(const Chunk<T>& c, T* out, const Sweep& w) {
    const uint64_t sc = pk2(w.scale, w.scale), nb = pk2(-w.base, -w.base);
    const uint64_t l2 = pk2(kLog2e, kLog2e), co = pk2(w.coef, w.coef);
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float t0, t1;
        upk2(mul2(fma2(c.pair(k), sc, nb), l2), t0, t1);
        upk2(mul2(pk2(exp2_approx(t0), exp2_approx(t1)), co), f[2 * k], f[2 * k + 1]);
    }
    Chunk<T>::store(out, f);
}

// Elements of a part outside its whole chunks, [lo, first) and [last, hi):
// at most seven each.
template <typename T>
__device__ __forceinline__ void sweep_edges(const T* row, T* out, int32_t lo, int32_t first,
                                            int32_t last, int32_t hi, const Sweep& w) {
    if (threadIdx.x >= 16) return;
    const int32_t i = threadIdx.x < 8 ? lo + static_cast<int32_t>(threadIdx.x)
                                      : last + static_cast<int32_t>(threadIdx.x) - 8;
    if (threadIdx.x < 8 ? i < first : i < hi) out[i] = from_f32<T>(sweep_value(to_f32(row[i]), w));
}

// Writes the teacher's tokens in [lo, hi) over the sweep's values (after a
// barrier).  A token listed more than once is written by its first entry,
// which adds up the others' probabilities in list order.
template <typename T, int NT>
__device__ __forceinline__ void write_teacher(const DistillArgs& a, const Teacher& t, T* out,
                                              int64_t lo, int64_t hi, const Sweep& w) {
    for (int k = threadIdx.x; k < a.k; k += NT) {
        const int32_t id = t.id[k];
        if (id < lo || id >= hi) continue;
        float q = t.q[k];
        bool first = true;
        for (int j = 0; j < a.k; ++j) {
            if (t.id[j] != id || j == k) continue;
            if (j < k) {
                first = false;
                break;
            }
            q = __fadd_rn(q, t.q[j]);
        }
        if (first) out[id] = from_f32<T>(fmaf(-w.c, q, sweep_value(t.x[k], w)));
    }
}

__device__ __forceinline__ float row_coef(const DistillArgs& a, int64_t r) {
    const float w = a.weight ? a.weight[r] : 1.0f;
    return __fdiv_rn(w, a.scale);
}

// One row per cluster of a.cluster blocks: the row's statistics in one pass
// over HBM, and with GRAD a second pass (from L2) that writes the gradient.
template <typename T, bool GRAD, bool SAME, int NT, int U>
__global__ void __launch_bounds__(NT) distill_kernel(const __grid_constant__ DistillArgs a) {
    __shared__ Teacher t;
    __shared__ Soft sh_soft[NT / 32], sh_teacher[NT / 32];
    __shared__ Soft sh_part;
    __shared__ float sh_sum[NT / 32];
    wait_prior_grids();
    allow_next_grid();
    const int tid = threadIdx.x;
    const int C = a.cluster;
    const int64_t r = blockIdx.x / C;
    const int part = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    const RowCut<T> cut(row, a.vocab);
    const int32_t c0 = static_cast<int32_t>(static_cast<int64_t>(cut.chunks) * part / C);
    const int32_t c1 = static_cast<int32_t>(static_cast<int64_t>(cut.chunks) * (part + 1) / C);
    const bool head = part == 0, tail = part == C - 1;
    const bool teach = GRAD || part == 0;  // uniform in a block
    Soft ts = soft_empty();
    if (teach) ts = teacher_load<T, NT>(a, r, row, t, sh_teacher);
    Soft q = soft_empty();
    soft_stream<T, false, NT, U>(q, row, cut, c0, c1, head, tail, a.scale);
    soft_block<false, NT>(q, sh_soft);
    if (C > 1) {
        if (tid == 0) sh_part = q;
        cluster_sync();
        Soft o = soft_empty();
        if (teach) {
            const uint32_t lane = tid & 31;
            if (lane < static_cast<uint32_t>(C)) {
                o.mz = __uint_as_float(ld_cluster(&sh_part.mz, lane));
                o.s = __uint_as_float(ld_cluster(&sh_part.s, lane));
            }
            soft_lanes<false, 32>(o);
            q = o;
        }
        cluster_sync();  // every part's statistics have been read
        if (!teach) return;
    }
    const bool none = q.s == 0.0f;
    const bool dead = none || ts.s == 0.0f;
    const float logs = none ? 0.0f : logf(q.s);
    float loss = 0.0f;
    if (!dead) loss = teacher_loss<NT>(a, t, ts, q.mz, logs);
    loss = block_sum<NT>(loss, sh_sum);
    if (part == 0 && tid == 0) {
        a.loss[r] = __fdiv_rn(__fdiv_rn(loss, a.scale), a.scale);
        if (a.lse) a.lse[r] = none ? neg_inf() : __fadd_rn(q.mz, logs);
    }
    if (!GRAD) return;
    T* out = static_cast<T*>(a.dx) + r * a.dx_stride;
    const int32_t lo = head ? 0 : cut.head + 8 * c0;
    const int32_t hi = tail ? a.vocab : cut.head + 8 * c1;
    if (dead) {
        for (int32_t i = lo + tid; i < hi; i += NT) out[i] = from_f32<T>(0.0f);
        return;
    }
    Sweep w;
    w.scale = a.scale;
    w.base = q.mz;
    w.c = row_coef(a, r);
    w.coef = __fdiv_rn(w.c, q.s);
    if (isnan(ts.s)) w.coef = ts.s;
    if (SAME) {
        const T* p = row + cut.head;
        T* d = out + cut.head;
        int32_t i = c0 + tid;
        for (; i + (U - 1) * NT < c1; i += U * NT) {
            Chunk<T> c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) c[u].load_stream(p + 8 * static_cast<int64_t>(i + u * NT));
#pragma unroll
            for (int u = 0; u < U; ++u)
                sweep_chunk<T>(c[u], d + 8 * static_cast<int64_t>(i + u * NT), w);
        }
        for (; i < c1; i += NT) {
            Chunk<T> c;
            c.load_stream(p + 8 * static_cast<int64_t>(i));
            sweep_chunk<T>(c, d + 8 * static_cast<int64_t>(i), w);
        }
        sweep_edges<T>(row, out, lo, cut.head + 8 * c0, cut.head + 8 * c1, hi, w);
    } else {
        for (int32_t i = lo + tid; i < hi; i += NT)
            out[i] = from_f32<T>(sweep_value(to_f32(row[i]), w));
    }
    __syncthreads();
    write_teacher<T, NT>(a, t, out, lo, hi, w);
}

// The gradient from a saved lse.  A block takes 8 * NT * U consecutive
// elements of one row.
template <typename T, bool SAME, int NT, int U>
__global__ void __launch_bounds__(NT) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
    __shared__ Teacher t;
    __shared__ Soft sh_teacher[NT / 32];
    wait_prior_grids();
    allow_next_grid();
    const int64_t r = blockIdx.x / a.segments;
    const int32_t seg = static_cast<int32_t>(blockIdx.x - r * a.segments);
    const int tid = threadIdx.x;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    T* out = static_cast<T*>(a.dx) + r * a.dx_stride;
    const RowCut<T> cut(row, a.vocab);
    // chunks [c0, c1) and, for the first and last block, the row's edges
    const int32_t c0 = min(seg * NT * U, cut.chunks), c1 = min(c0 + NT * U, cut.chunks);
    const int32_t lo = seg == 0 ? 0 : cut.head + 8 * c0;
    const int32_t hi = seg == a.segments - 1 ? a.vocab : cut.head + 8 * c1;
    const float lse = a.lse[r];
    const Soft ts = teacher_load<T, NT>(a, r, row, t, sh_teacher);
    if (ts.s == 0.0f || lse == neg_inf()) {
        for (int32_t i = lo + tid; i < hi; i += NT) out[i] = from_f32<T>(0.0f);
        return;
    }
    for (int k = tid; k < a.k; k += NT) {
        const float d = fmaf(t.q[k], a.scale, -ts.mz);
        t.q[k] = t.id[k] >= 0 ? __fdiv_rn(exp2_approx(__fmul_rn(d, kLog2e)), ts.s) : 0.0f;
    }
    Sweep w;
    w.scale = a.scale;
    w.base = lse;
    w.c = row_coef(a, r);
    w.coef = isnan(ts.s) ? ts.s : w.c;
    __syncthreads();  // the row's logits at the teacher's tokens have been read
    if (SAME) {
        Chunk<T> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + tid + u * NT < c1)
                c[u].load_stream(row + cut.head + 8 * static_cast<int64_t>(c0 + tid + u * NT));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + tid + u * NT < c1)
                sweep_chunk<T>(c[u], out + cut.head + 8 * static_cast<int64_t>(c0 + tid + u * NT), w);
        sweep_edges<T>(row, out, lo, cut.head + 8 * c0, cut.head + 8 * c1, hi, w);
    } else {
        for (int32_t i = lo + tid; i < hi; i += NT)
            out[i] = from_f32<T>(sweep_value(to_f32(row[i]), w));
    }
    __syncthreads();
    write_teacher<T, NT>(a, t, out, lo, hi, w);
}

template <typename T>
bool same_phase(const DistillArgs& a) {
    const auto phase = [](const void* p) {
        return (reinterpret_cast<uintptr_t>(p) / sizeof(T)) % Chunk<T>::kPhase;
    };
    return phase(a.x) == phase(a.dx) &&
           (a.n == 1 || (a.stride - a.dx_stride) % Chunk<T>::kPhase == 0);
}

template <typename T>
cudaError_t launch_loss(DistillArgs a, cudaStream_t stream) {
    constexpr int NT = 256, U = 4;
    const int64_t chunks = a.vocab / 8;
    int C = 1;
    while (C < 8 && a.n * C < 304 && chunks / (2 * C) >= 2 * NT) C *= 2;
    a.cluster = C;
    if (!a.dx)
        return launch_vocab(distill_kernel<T, false, true, NT, U>, a.n * C, NT, 0, C, a, stream);
    return same_phase<T>(a)
               ? launch_vocab(distill_kernel<T, true, true, NT, U>, a.n * C, NT, 0, C, a, stream)
               : launch_vocab(distill_kernel<T, true, false, NT, U>, a.n * C, NT, 0, C, a, stream);
}

template <typename T>
cudaError_t launch_grad(DistillArgs a, cudaStream_t stream) {
    constexpr int NT = 256, U = 4;
    a.segments = (a.vocab + 8 * NT * U - 1) / (8 * NT * U);
    const int64_t grid = a.n * a.segments;
    return same_phase<T>(a)
               ? launch_vocab(distill_grad_kernel<T, true, NT, U>, grid, NT, 0, 1, a, stream)
               : launch_vocab(distill_grad_kernel<T, false, NT, U>, grid, NT, 0, 1, a, stream);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
    return a.dtype == ZERO3_F32 ? launch_loss<float>(a, stream) : launch_loss<uint16_t>(a, stream);
}

cudaError_t launch_distill_grad(const DistillArgs& a, cudaStream_t stream) {
    return a.dtype == ZERO3_F32 ? launch_grad<float>(a, stream) : launch_grad<uint16_t>(a, stream);
}

}  // namespace z3
