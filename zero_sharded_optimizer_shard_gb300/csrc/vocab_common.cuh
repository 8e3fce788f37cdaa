// Device helpers of the vocabulary operators (embedding.cu, logprobs.cu,
// distill.cu): typed 8-element chunks of a row, packed binary32 arithmetic,
// the streaming softmax statistics of a row and their joins, launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "operators.h"

namespace z3 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// 2^x of the hardware's exponential unit (2 ulp, subnormal results are 0).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A logarithm of a weight that exp2_approx (of it, or of it times log2 e) has
// turned into 0: what is below, -inf above all, is raised to this, so that the
// product of the two is 0.  (Small, so that times a weight of up to 2^120 it stays
// finite.)
constexpr float kNoWeight = -128.0f;
// max that keeps a NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two binary32 values per 64-bit register; each lane rounds as the scalar
// instruction does.
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void upk2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ------------------------------------------------------------ typed chunks
// A chunk is 8 consecutive elements starting on a 16-byte boundary: one
// 16-byte access of bf16, two of binary32.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    static constexpr int kPhase = 8;  // elements per 16 bytes
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t* p) {
        r = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void load_stream(const uint16_t* p) { r = ldcs16(p); }
    // from 16-byte parts that lie `step` apart
    __device__ __forceinline__ void from_parts(const uint4* p, int) { r = *p; }
    // the largest element; NaNs are passed over
    __device__ __forceinline__ float max() const {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(r.x), "r"(r.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(r.z), "r"(r.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fmaxf(bf16_lo(a), bf16_hi(a));
    }
    __device__ __forceinline__ uint64_t pair(int k) const {
        const uint32_t w = k == 0 ? r.x : k == 1 ? r.y : k == 2 ? r.z : r.w;
        return pk2(bf16_lo(w), bf16_hi(w));
    }
    __device__ __forceinline__ void fill(float x) {
        const uint32_t w = pack_bf16x2(x, x);
        r = make_uint4(w, w, w, w);
    }
    __device__ __forceinline__ void set(int e, uint16_t h) {
        uint32_t* w = &r.x;
        const uint32_t sh = (e & 1) * 16u;
        w[e >> 1] = (w[e >> 1] & ~(0xffffu << sh)) | (static_cast<uint32_t>(h) << sh);
    }
    static __device__ __forceinline__ void store(uint16_t* p, const float* f) {
        stcs16(p, pack8(f));
    }
};
template <>
struct Chunk<float> {
    static constexpr int kPhase = 4;
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void load_stream(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    }
    __device__ __forceinline__ void from_parts(const uint4* p, int step) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + step);
    }
    __device__ __forceinline__ float max() const {
        return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)),
                     fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
    }
    __device__ __forceinline__ uint64_t pair(int k) const {
        return k == 0 ? pk2(a.x, a.y) : k == 1 ? pk2(a.z, a.w)
               : k == 2 ? pk2(b.x, b.y) : pk2(b.z, b.w);
    }
    __device__ __forceinline__ void fill(float x) {
        a = make_float4(x, x, x, x);
        b = a;
    }
    __device__ __forceinline__ void set(int e, float x) {
        float* f = e < 4 ? &a.x : &b.x;
        f[e & 3] = x;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(p + 4), make_float4(f[4], f[5], f[6], f[7]));
    }
};

__device__ __forceinline__ float to_f32(uint16_t h) { return bf16_f32(h); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float x) { return to_bf16(x); }
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

// Id i of an int32 or int64 list; anything outside [0, limit) becomes -1.
__device__ __forceinline__ int32_t load_id(const void* ids, int i64, int64_t i, int64_t limit) {
    const int64_t v = i64 ? static_cast<const int64_t*>(ids)[i]
                          : static_cast<int64_t>(static_cast<const int32_t*>(ids)[i]);
    return v >= 0 && v < limit ? static_cast<int32_t>(v) : -1;
}

// A row of V elements cut at 16-byte boundaries: `head` elements before the
// first one, `chunks` whole chunks, then `tail` elements.
template <typename T>
struct RowCut {
    int head, tail;
    int32_t chunks;
    __device__ __forceinline__ RowCut(const T* row, int32_t V) {
        constexpr int P = Chunk<T>::kPhase;
        const int ph = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % P);
        head = ph ? P - ph : 0;
        if (head > V) head = V;
        chunks = (V - head) / 8;
        tail = V - head - 8 * chunks;
    }
};

// ------------------------------------------------- streaming softmax of a row
// Running statistics of z = x * scale over the elements that a thread has
// seen: m the largest x, mz = rn(m * scale) (0 while that is -inf, so that
// no difference of two infinities is taken), s = sum 2^t and a = sum t 2^t
// with t = (z - mz) log2(e).  Products are exact inside the FMA: z is never
// rounded by itself.  A NaN element is passed over by m and turns s into NaN.
struct alignas(16) Soft {
    float m, mz, s, a;
};

template <typename T, bool ENT, int U>
__device__ __forceinline__ void soft_add(Soft& q, const Chunk<T> (&c)[U], float scale) {
    float bm = c[0].max();
#pragma unroll
    for (int u = 1; u < U; ++u) bm = fmaxf(bm, c[u].max());
    if (bm > q.m) {
        const float nz = __fmul_rn(bm, scale);
        const float nzf = nz == neg_inf() ? 0.0f : nz;
        if (q.s != 0.0f) {
            const float dt = __fmul_rn(__fsub_rn(q.mz, nzf), kLog2e);
            const float f = exp2_approx(dt);
            if (ENT) q.a = __fmul_rn(f, fmaf(q.s, max_nan(dt, kNoWeight), q.a));
            q.s = __fmul_rn(q.s, f);
        }
        q.m = bm;
        q.mz = nzf;
    }
    const uint64_t sc = pk2(scale, scale), nm = pk2(-q.mz, -q.mz), l2 = pk2(kLog2e, kLog2e);
    uint64_t s0 = 0, s1 = 0, a0 = 0, a1 = 0;  // packed +0
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint64_t t = mul2(fma2(c[u].pair(k), sc, nm), l2);
            float t0, t1;
            upk2(t, t0, t1);
            if (ENT) {  // t = -inf has weight 0: keep 0 * t finite
                t0 = max_nan(t0, kNoWeight);
                t1 = max_nan(t1, kNoWeight);
                t = pk2(t0, t1);
            }
            const uint64_t e = pk2(exp2_approx(t0), exp2_approx(t1));
            if (k & 1) {
                s1 = add2(s1, e);
                if (ENT) a1 = fma2(e, t, a1);
            } else {
                s0 = add2(s0, e);
                if (ENT) a0 = fma2(e, t, a0);
            }
        }
    }
    float x, y;
    upk2(add2(s0, s1), x, y);
    q.s = __fadd_rn(q.s, __fadd_rn(x, y));
    if (ENT) {
        upk2(add2(a0, a1), x, y);
        q.a = __fadd_rn(q.a, __fadd_rn(x, y));
    }
}

// Statistics taken to a common maximum `to` >= q.mz.
template <bool ENT>
__device__ __forceinline__ void soft_rebase(Soft& q, float to) {
    if (q.s != 0.0f) {
        const float dt = __fmul_rn(__fsub_rn(q.mz, to), kLog2e);
        const float f = exp2_approx(dt);
        if (ENT) q.a = __fmul_rn(f, fmaf(q.s, max_nan(dt, kNoWeight), q.a));
        q.s = __fmul_rn(q.s, f);
    }
    q.mz = to;
}

// The maximum that lanes with weight agree on; lanes without (s = 0) do not
// count (their mz is a placeholder) unless their maximum has overflowed.
__device__ __forceinline__ float soft_top(const Soft& q) {
    return q.s != 0.0f || q.mz == -neg_inf() ? q.mz : neg_inf();
}

// Joins the statistics of `width` lanes (a power of two); every lane gets
// the result.  The tree is fixed, so the result does not depend on timing.
template <bool ENT, int WIDTH>
__device__ __forceinline__ void soft_lanes(Soft& q) {
    float top = soft_top(q);
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == neg_inf()) top = 0.0f;
    soft_rebase<ENT>(q, top);
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) {
        q.s = __fadd_rn(q.s, __shfl_xor_sync(0xffffffffu, q.s, o));
        if (ENT) q.a = __fadd_rn(q.a, __shfl_xor_sync(0xffffffffu, q.a, o));
    }
    if (top == -neg_inf()) q.s = __int_as_float(0x7fffffff);
}

// Joins the statistics of a block of NT threads; every thread gets the
// result.  `sh` holds one entry per warp; the call contains one barrier, and
// the caller puts one between two uses of `sh`.
template <bool ENT, int NT>
__device__ __forceinline__ void soft_block(Soft& q, Soft* sh) {
    constexpr int W = NT / 32;
    soft_lanes<ENT, 32>(q);
    if (W == 1) return;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = q;
    __syncthreads();
    q = sh[(threadIdx.x & 31) % W];
    soft_lanes<ENT, W>(q);
}

// Thread tid's share, of NT, of a row's chunks [c0, c1): chunk c0 + tid, + NT,
// ... in batches of U loads; the head elements go to thread 0, the tail
// elements to the last thread, when `head` / `tail` say that they are the
// caller's.
template <typename T, bool ENT, int NT, int U>
__device__ __forceinline__ void soft_stream(Soft& q, const T* row, const RowCut<T>& cut,
                                            int32_t c0, int32_t c1, bool head, bool tail,
                                            float scale, int tid) {
    if ((tid == 0 && head && cut.head) || (tid == NT - 1 && tail && cut.tail)) {
        Chunk<T> c[1];
        const bool h = tid == 0 && head && cut.head;
        const T* p = h ? row : row + cut.head + 8 * static_cast<int64_t>(cut.chunks);
        const int n = h ? cut.head : cut.tail;
        c[0].fill(neg_inf());
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) c[0].set(e, p[e]);
        soft_add<T, ENT, 1>(q, c, scale);
    }
    const T* p = row + cut.head;
    int32_t i = c0 + tid;
    for (; i + (U - 1) * NT < c1; i += U * NT) {
        Chunk<T> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) c[u].load(p + 8 * static_cast<int64_t>(i + u * NT));
        soft_add<T, ENT, U>(q, c, scale);
    }
    for (; i < c1; i += NT) {
        Chunk<T> c[1];
        c[0].load(p + 8 * static_cast<int64_t>(i));
        soft_add<T, ENT, 1>(q, c, scale);
    }
}

__device__ __forceinline__ Soft soft_empty() { return Soft{neg_inf(), 0.0f, 0.0f, 0.0f}; }

// Chunks of a row on their way to a thread: its share (chunk tid, + NT, ... of
// n from `first` on), once or twice over, in batches of U through a ring of two
// batches in shared memory, filled by asynchronous 16-byte copies.  A thread
// reads what it copied itself, so no barrier orders them; bytes in flight cost
// no registers.
template <typename T, int NT>
struct RowRing {
    static constexpr int P = sizeof(T) / 2;  // 16-byte parts per chunk
    static constexpr int U = 4 / P;          // chunks per batch
    static constexpr int kBytes = 8 * 16 * NT;
    const uint4* ring;
    uint32_t at;
    const T* mine;
    int tid, n, full, per, all;  // full: batches without a gap; per pass, in all
    __device__ __forceinline__ RowRing(uint4* mem, const T* first, int n_, int tid_, int passes)
        : ring(mem + tid_),
          at(static_cast<uint32_t>(__cvta_generic_to_shared(mem + tid_))),
          mine(first + 8 * tid_),
          tid(tid_),
          n(n_),
          full(n_ / (U * NT)),
          per((n_ + U * NT - 1) / (U * NT)),
          all(passes * per) {}
    // Sends batch b.
    __device__ __forceinline__ void send(int b) const {
        if (b < all) {
            const int c = (b >= per ? b - per : b) * U * NT;  // chunks before the batch
            const T* from = mine + 8 * static_cast<int64_t>(c);
            const uint32_t to = at + static_cast<uint32_t>((b & 1) * (16 * U * P * NT));
            const bool gaps = c + U * NT > n;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (!gaps || c + u * NT + tid < n) {
#pragma unroll
                    for (int h = 0; h < P; ++h)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         to + 16 * NT * (u * P + h)),
                                     "l"(from + 8 * NT * u + h * (8 / P))
                                     : "memory");
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Takes batch b, of two that have been sent, out of the ring.
    __device__ __forceinline__ void take(int b, Chunk<T> (&c)[U]) const {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const uint4* from = ring + (b & 1) * (U * P * NT);
#pragma unroll
        for (int u = 0; u < U; ++u) c[u].from_parts(from + u * P * NT, NT);
    }
    // Whether the thread has chunk u of a batch that has gaps (batch `full` of
    // its pass).
    __device__ __forceinline__ bool has(int u) const { return (full * U + u) * NT + tid < n; }
};
__device__ __forceinline__ void drain_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Adds the first pass of a ring, two batches of which have been sent.
template <typename T, bool ENT, int NT>
__device__ __forceinline__ void soft_ring(Soft& q, const RowRing<T, NT>& g, float scale) {
    constexpr int U = RowRing<T, NT>::U;
#pragma unroll 1
    for (int b = 0; b < g.full; ++b) {
        Chunk<T> c[U];
        g.take(b, c);
        g.send(b + 2);
        soft_add<T, ENT, U>(q, c, scale);
    }
    if (g.full < g.per) {
        Chunk<T> c[U];
        g.take(g.full, c);
        g.send(g.full + 2);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g.has(u)) soft_add<T, ENT, 1>(q, reinterpret_cast<Chunk<T>(&)[1]>(c[u]), scale);
    }
}

// The element of a row's part outside its whole chunks ([lo, first) and
// [last, hi), at most seven each) that this thread has, or -1.
__device__ __forceinline__ int32_t edge_element(int32_t lo, int32_t first, int32_t last, int32_t hi) {
    const int tid = static_cast<int>(threadIdx.x);
    if (tid < 8) return lo + tid < first ? lo + tid : -1;
    if (tid < 16) return last + tid - 8 < hi ? last + tid - 8 : -1;
    return -1;
}
template <typename T, bool ENT>
__device__ __forceinline__ void soft_element(Soft& q, T x, float scale) {
    Chunk<T> c[1];
    c[0].fill(neg_inf());
    c[0].set(0, x);
    soft_add<T, ENT, 1>(q, c, scale);
}

// ----------------------------------------------------------------- clusters
// A cluster's blocks send their results to one another's shared memory: all
// arrive when they start (whoever has waited for that may write to the others),
// and once more when they have sent.  Not the .aligned forms, which are
// undefined in a warp whose lanes have not met again after a branch.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Writes to the shared variable at `p` of block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_address(const void* p, uint32_t rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void send_cluster(uint64_t* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_address(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void send_cluster(Soft* p, uint32_t rank, const Soft& v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_address(p, rank)),
                 "f"(v.m), "f"(v.mz), "f"(v.s), "f"(v.a)
                 : "memory");
}
constexpr int kMaxCluster = 8;

// The statistics that C blocks have sent to `parts`, joined (every lane).
template <bool ENT>
__device__ __forceinline__ Soft soft_parts(const Soft* parts, int C) {
    Soft o = soft_empty();
    const int i = threadIdx.x % kMaxCluster;
    if (i < C) o = parts[i];
    soft_lanes<ENT, kMaxCluster>(o);
    return o;
}

// Launch with programmatic stream serialization (see wait_prior_grids), with
// `cluster` blocks per cluster.  Returns what the launch itself returned: the
// thread's last error may be an earlier call's, which is not this one's failure.
template <typename Args>
cudaError_t launch_vocab(void (*kernel)(Args), int64_t grid, int threads, int smem, int cluster,
                         const Args& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
}  // namespace z3
