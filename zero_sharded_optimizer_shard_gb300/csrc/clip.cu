// Norms of gradient tensors and their clipping (sm_103a).
//
//   N = sqrt(sum_t sum_i g_ti^2),  coef = min(1, max_norm / (N + 1e-6)),
//   out = coef * g
//
// Bound by HBM: one fused multiply-add per element read.  A launch takes up to
// 1024 tensors of any size; they are cut into blocks, a block belongs to one
// tensor and writes one binary64 sum of squares, and one more small kernel joins
// the sums in their order (no atomics: the bits do not depend on timing).
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {

static_assert(sizeof(ListArgs<kLargeList>) <= 32764, "ListArgs exceeds the kernel parameter limit");

namespace {

// The tensor of the launch that a block belongs to.
template <int MAXT>
__device__ __forceinline__ int list_tensor(const ListArgs<MAXT>& a, uint32_t block) {
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.block0[mid] <= block)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ uint32_t bits_of(const Chunk<uint16_t>& c) {
    return (c.r.x | c.r.y | c.r.z | c.r.w) & 0x7fff7fffu;
}
__device__ __forceinline__ uint32_t bits_of(const Chunk<float>& c) {
    const uint32_t u = __float_as_uint(c.a.x) | __float_as_uint(c.a.y) | __float_as_uint(c.a.z) |
                       __float_as_uint(c.a.w) | __float_as_uint(c.b.x) | __float_as_uint(c.b.y) |
                       __float_as_uint(c.b.z) | __float_as_uint(c.b.w);
    return u & 0x7fffffffu;
}

// Squares over the whole range of binary32: three sums, of numbers above 2^50
// (times 2^-90), below 2^-40 (times 2^90) and between, of one chunk.
struct WideSquares {
    float big = 0.0f, mid = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float ax = fabsf(x);
        if (ax > 0x1p50f) {
            const float t = x * 0x1p-90f;
            big = fmaf(t, t, big);
        } else if (ax < 0x1p-40f) {
            const float t = x * 0x1p90f;
            small = fmaf(t, t, small);
        } else {  // a NaN too
            mid = fmaf(x, x, mid);
        }
    }
    __device__ __forceinline__ double value() const {
        return static_cast<double>(big) * 0x1p180 + static_cast<double>(mid) +
               static_cast<double>(small) * 0x1p-180;
    }
};

// Blocks of 256 threads with 64 bytes per thread on their way, 1024 chunks of 8 per
// block and more only where that would make over 4864 blocks (32 per SM), so that
// the blocks' sums stay few.  A thread's four binary32 sums are taken into a binary64 one
// every kFold batches, so that their rounding errors (one-sided for equal numbers) do not
// grow with the list: 64 squares of bf16 each, 32 of binary32.  GPT-2-small's 148 binary32
// tensors: 77 us, 498 MB at 82% of the DRAM peak; 2000 ragged bf16 tensors, 1.05 GB: 153
// us with the join (6.9 TB/s; 171 with one batch per turn of the loop, 188 with four).
template <typename T, int MAXT>
__global__ void __launch_bounds__(kThreads) list_norm_kernel(const __grid_constant__ ListArgs<MAXT> a) {
    constexpr int U = sizeof(T) == 2 ? 4 : 2;  // chunks in flight per thread: 64 bytes
    constexpr int kFold = 16;
    __shared__ double sh[kThreads / 32];
    wait_prior_grids();
    allow_next_grid();
    const int t = list_tensor(a, blockIdx.x);
    const T* x = static_cast<const T*>(a.x[t]);
    const int64_t n = a.numel[t];
    const uint32_t b = blockIdx.x - a.block0[t];
    const bool last = blockIdx.x + 1 == a.block0[t + 1];
    constexpr int P = Chunk<T>::kPhase;
    const int ph = static_cast<int>((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % P);
    const int64_t head = ph && n > 0 ? (P - ph < n ? P - ph : n) : 0;
    const int64_t chunks = (n - head) / 8;
    const int64_t tail = n - head - 8 * chunks;
    // the block's own chunks (fewer than 2^26: the list has 2^41 elements at most)
    const int64_t c0 = static_cast<int64_t>(b) * a.per;
    const int64_t left = chunks - c0 < a.per ? chunks - c0 : a.per;
    const int own = left > 0 ? static_cast<int>(left) : 0;
    const int tid = static_cast<int>(threadIdx.x);
    // the element at the tensor's ends that the thread has
    const T* edge = nullptr;
    if (b == 0 && tid < head) edge = x + tid;
    if (last && tid >= 8 && tid - 8 < tail) edge = x + head + 8 * chunks + (tid - 8);
    const T* p = x + head + 8 * c0;

    uint64_t acc[4] = {0, 0, 0, 0};
    uint32_t any = 0;
    double d = 0.0;
    const auto sum = [&]() {
        float s, s1;
        upk2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), s, s1);
        return __fadd_rn(s, s1);
    };
    int i = tid;
    while (i + (U - 1) * kThreads < own) {
        const int stop = i + kFold * U * kThreads < own ? i + kFold * U * kThreads : own;
#pragma unroll 2
        for (; i + (U - 1) * kThreads < stop; i += U * kThreads) {
            Chunk<T> c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) c[u].load(p + 8 * static_cast<int64_t>(i + u * kThreads));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                any |= bits_of(c[u]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t v = c[u].pair(k);
                    acc[k] = fma2(v, v, acc[k]);
                }
            }
        }
        if (stop < own) {
            d += static_cast<double>(sum());
            acc[0] = acc[1] = acc[2] = acc[3] = 0;
        }
    }
    for (; i < own; i += kThreads) {
        Chunk<T> c;
        c.load(p + 8 * static_cast<int64_t>(i));
        any |= bits_of(c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t v = c.pair(k);
            acc[k] = fma2(v, v, acc[k]);
        }
    }
    float s = sum();
    if (edge) {
        const float f = to_f32(*edge);
        s = fmaf(f, f, s);
        any |= __float_as_uint(f) & 0x7fffffffu;
    }
    d += static_cast<double>(s);
    // A sum near the ends of binary32's range (numbers beyond 2^60, or so small
    // that squares have lost bits): the thread's share is read again.
    const bool again = any && !(d >= 0x1p-90 && d <= 0x1p120);
    if (again) {
        d = 0.0;
        for (int j = tid; j < own; j += kThreads) {
            WideSquares w;
            for (int e = 0; e < 8; ++e) w.add(to_f32(p[8 * static_cast<int64_t>(j) + e]));
            d += w.value();
        }
        if (edge) {
            WideSquares w;
            w.add(to_f32(*edge));
            d += w.value();
        }
    }
    if (__any_sync(0xffffffffu, again || d != static_cast<double>(s))) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
        d = static_cast<double>(s);
    }
    if ((tid & 31) == 0) sh[tid >> 5] = d;
    __syncthreads();
    if (tid == 0) {
        double sum = sh[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) sum += sh[w];
        a.partial[blockIdx.x] = sum;
        if (b == 0) a.start[t] = a.first + static_cast<int32_t>(blockIdx.x);
    }
}

// Sum of the block's binary64 values (thread 0 has it).
template <int NT>
__device__ __forceinline__ double block_sum(double d, double* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x < 32) {
        d = threadIdx.x < NT / 32 ? sh[threadIdx.x] : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    }
    return d;
}

struct FoldArgs {
    const double* from;
    double* to;
    int64_t n, per;
};

// Many blocks' sums (the sharded step has one per 2048 elements) into 1024: 8 us with
// cold caches for 61 thousand.
__global__ void __launch_bounds__(kThreads) fold_kernel(const __grid_constant__ FoldArgs a) {
    __shared__ double sh[kThreads / 32];
    wait_prior_grids();
    allow_next_grid();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.per;
    const int64_t hi = lo + a.per < a.n ? lo + a.per : a.n;
    double d = 0.0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) d += a.from[i];
    d = block_sum<kThreads>(d, sh);
    if (threadIdx.x == 0) a.to[blockIdx.x] = d;
}

constexpr int kNormThreads = 512;

// Block 0: the total.  The others: a tensor's norm per warp.  A chain of latencies: 2
// to 3 us behind the sums (7 us with cold caches).
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ double sh[kNormThreads / 32];
    wait_prior_grids();
    allow_next_grid();
    if (blockIdx.x > 0) {
        const int lane = threadIdx.x & 31;
        const int64_t t = static_cast<int64_t>(blockIdx.x - 1) * (kNormThreads / 32) + (threadIdx.x >> 5);
        if (t >= a.n_tensors) return;
        const int64_t lo = a.start[t], hi = t + 1 < a.n_tensors ? a.start[t + 1] : a.n;
        double d = 0.0;
        for (int64_t i = lo + lane; i < hi; i += 32) d += a.partial[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (lane == 0) a.tensor_norms[t] = static_cast<float>(sqrt(d));
        return;
    }
    double d = 0.0;
    for (int64_t i = threadIdx.x; i < a.n_folded; i += kNormThreads) d += a.folded[i];
    d = block_sum<kNormThreads>(d, sh);
    if (threadIdx.x != 0) return;
    if (a.accumulate) d += *a.square_sum;
    if (a.square_sum) *a.square_sum = d;
    const double norm = sqrt(d);
    if (a.norm) *a.norm = static_cast<float>(norm);
    if (a.coef) {
        // an infinite max_norm clips nothing, an infinite norm clips to zero
        double c = 1.0;
        if (a.max_norm < __int_as_float(0x7f800000)) {
            c = static_cast<double>(a.max_norm) / (norm + 1e-6);
            if (c > 1.0) c = 1.0;  // keeps a NaN
        }
        *a.coef = static_cast<float>(c);
    }
}

// ------------------------------------------------------------------ clipping
// 8 elements of a tensor as binary32: aligned ones by 16-byte loads, bf16 ones at
// another phase by the two aligned blocks around them where both lie in the
// tensor (inside), others one by one.
__device__ __forceinline__ void load8(const uint16_t* p, int ph, bool inside, float* f) {
    if (ph == 0) {
        unpack8(*reinterpret_cast<const uint4*>(p), f);
    } else if (inside) {
        unpack8(ld8_window(p, ph), f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = bf16_f32(p[e]);
    }
}
__device__ __forceinline__ void load8(const float* p, int ph, bool, float* f) {
    if (ph == 0) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = p[e];
    }
}
__device__ __forceinline__ void store8(uint16_t* p, int ph, const float* f) {
    if (ph == 0) {
        stcs16(p, pack8(f));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = to_bf16(f[e]);
    }
}
__device__ __forceinline__ void store8(float* p, int ph, const float* f) {
    if (ph == 0) {
        Chunk<float>::store(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = f[e];
    }
}

template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
    constexpr int P = Chunk<T>::kPhase;
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % P);
}

// Bound by HBM: GPT-2-small's binary32 gradients into bf16, 498 MB read and 249
// written in 107 us, 83% of the DRAM peak.
//
// Chunks start where the output lies on 16 bytes, or where the bf16 side does
// if the types differ: the binary32 side, whose phase repeats every 4 elements,
// then does too wherever both tensors lie at one offset of their buffers.
template <typename TI, typename TO, int MAXT>
__global__ void __launch_bounds__(kThreads) list_scale_kernel(const __grid_constant__ ListArgs<MAXT> a) {
    constexpr int U = 2;
    wait_prior_grids();
    allow_next_grid();
    // the last tensors first: they are what the norm has left in L2
    const uint32_t block = gridDim.x - 1 - blockIdx.x;
    const int t = list_tensor(a, block);
    const TI* x = static_cast<const TI*>(a.x[t]);
    TO* out = static_cast<TO*>(a.out[t]);
    const int64_t n = a.numel[t];
    const float scale = *a.scale;
    if (scale == 1.0f && static_cast<const void*>(x) == static_cast<const void*>(out)) return;
    const uint32_t b = block - a.block0[t];
    const bool last = block + 1 == a.block0[t + 1];
    constexpr bool kByInput = sizeof(TI) < sizeof(TO);
    const int ph = kByInput ? phase_of(x) : phase_of(out);
    constexpr int P = kByInput ? Chunk<TI>::kPhase : Chunk<TO>::kPhase;
    const int64_t head = ph && n > 0 ? (P - ph < n ? P - ph : n) : 0;
    const int64_t chunks = (n - head) / 8;
    const int64_t tail = n - head - 8 * chunks;
    const int64_t c0 = static_cast<int64_t>(b) * a.per;
    const int64_t c1 = c0 + a.per < chunks ? c0 + a.per : chunks;
    const int tid = static_cast<int>(threadIdx.x);
    if (b == 0 && tid < head) out[tid] = from_f32<TO>(__fmul_rn(to_f32(x[tid]), scale));
    if (last && tid >= 8 && tid - 8 < tail) {
        const int64_t e = head + 8 * chunks + (tid - 8);
        out[e] = from_f32<TO>(__fmul_rn(to_f32(x[e]), scale));
    }
    const int xp = phase_of(x + head), op = phase_of(out + head);
    int64_t i = c0 + tid;
    for (; i + (U - 1) * kThreads < c1; i += U * kThreads) {
        float f[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t e = head + 8 * (i + u * kThreads);
            load8(x + e, xp, e >= 8 && e + 16 <= n, f[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[u][k] = __fmul_rn(f[u][k], scale);
            store8(out + head + 8 * (i + u * kThreads), op, f[u]);
        }
    }
    for (; i < c1; i += kThreads) {
        float f[8];
        const int64_t e = head + 8 * i;
        load8(x + e, xp, e >= 8 && e + 16 <= n, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(f[k], scale);
        store8(out + e, op, f);
    }
}

template <int MAXT>
cudaError_t norm_launch(const ListArgs<MAXT>& a, int dtype, cudaStream_t stream) {
    const int64_t grid = a.block0[a.count];
    return dtype == ZERO3_BF16 ? launch_vocab(list_norm_kernel<uint16_t, MAXT>, grid, kThreads, 0, 1, a, stream)
                               : launch_vocab(list_norm_kernel<float, MAXT>, grid, kThreads, 0, 1, a, stream);
}

template <int MAXT>
cudaError_t scale_launch(const ListArgs<MAXT>& a, int dtype, int out_dtype, cudaStream_t stream) {
    const int64_t grid = a.block0[a.count];
    if (dtype == ZERO3_BF16)
        return out_dtype == ZERO3_BF16
                   ? launch_vocab(list_scale_kernel<uint16_t, uint16_t, MAXT>, grid, kThreads, 0, 1, a, stream)
                   : launch_vocab(list_scale_kernel<uint16_t, float, MAXT>, grid, kThreads, 0, 1, a, stream);
    return out_dtype == ZERO3_BF16
               ? launch_vocab(list_scale_kernel<float, uint16_t, MAXT>, grid, kThreads, 0, 1, a, stream)
               : launch_vocab(list_scale_kernel<float, float, MAXT>, grid, kThreads, 0, 1, a, stream);
}

}  // namespace

cudaError_t launch_list_norm(const ListArgs<kSmallList>& a, int dtype, cudaStream_t stream) {
    return norm_launch(a, dtype, stream);
}
cudaError_t launch_list_norm(const ListArgs<kLargeList>& a, int dtype, cudaStream_t stream) {
    return norm_launch(a, dtype, stream);
}
cudaError_t launch_list_scale(const ListArgs<kSmallList>& a, int dtype, int out_dtype, cudaStream_t stream) {
    return scale_launch(a, dtype, out_dtype, stream);
}
cudaError_t launch_list_scale(const ListArgs<kLargeList>& a, int dtype, int out_dtype, cudaStream_t stream) {
    return scale_launch(a, dtype, out_dtype, stream);
}

cudaError_t launch_norms(NormArgs a, double* to, cudaStream_t stream) {
    a.folded = a.partial;
    a.n_folded = a.n;
    if (a.n > kFoldAbove) {
        FoldArgs f;
        f.from = a.partial;
        f.to = to;
        f.n = a.n;
        f.per = (a.n + kFoldBlocks - 1) / kFoldBlocks;
        const int64_t grid = (a.n + f.per - 1) / f.per;
        const cudaError_t e = launch_vocab(fold_kernel, grid, kThreads, 0, 1, f, stream);
        if (e != cudaSuccess) return e;
        a.folded = to;
        a.n_folded = grid;
    }
    int64_t grid = 1;
    if (a.tensor_norms) grid += (a.n_tensors + kNormThreads / 32 - 1) / (kNormThreads / 32);
    return launch_vocab(norm_kernel, grid, kNormThreads, 0, 1, a, stream);
}

}  // namespace z3
