// Log probabilities of given tokens with entropy and top alternatives, and
// their gradient (sm_103a).
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {
namespace {

// ------------------------------------------------------- top alternatives
// Keys that order binary32 values as unsigned integers; -0 counts as +0.  A
// row's part with a NaN (its sum says so) never comes here: an addition's
// NaN has the key 0xffffffff, and a bound one above it would wrap to 0.  Key 0
// is below every value.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return b ^ (b & 0x80000000u ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
// A candidate: larger is better, equal values go to the lower index.
__device__ __forceinline__ uint64_t candidate(uint32_t key, int32_t index) {
    return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(index));
}

constexpr int kGroups = 128;     // groups of threads whose maxima bound the k-th value
constexpr int kCandidates = 640; // candidates a block ranks

struct TopShared {
    alignas(16) uint64_t cand[kCandidates];
    uint64_t list[kMaxCluster * ZERO3_MAX_TOP];  // what a cluster's blocks have sent
    alignas(16) uint32_t group[kGroups];
    uint16_t thread[512];
    uint32_t bound;
    int flagged, count, sum;
};

// One block's part of a row: elements [lo, hi) of the row, chunks [c0, c1).
template <typename T>
struct Part {
    const T* row;
    RowCut<T> cut;
    int32_t c0, c1, lo, hi;
};

template <typename T>
__device__ __forceinline__ float chunk_value(const Chunk<T>& c, int e) {
    float lo, hi;
    upk2(c.pair(e >> 1), lo, hi);
    return e & 1 ? hi : lo;
}

__device__ __forceinline__ void offer(TopShared& sh, uint32_t key, int32_t index) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCandidates) sh.cand[at] = candidate(key, index);
}

// Offers the elements of chunk c, which holds x, whose key is at least `bound`.
template <typename T>
__device__ __forceinline__ void offer_chunk(TopShared& sh, const Part<T>& p, int32_t c,
                                            const Chunk<T>& x, uint32_t bound) {
    if (key_of(x.max()) < bound) return;
    const int32_t at = p.cut.head + 8 * c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t key = key_of(chunk_value(x, e));
        if (key >= bound) offer(sh, key, at + e);
    }
}

// Offers the elements of the part that lie outside its whole chunks (at most
// 14) with keys of at least `bound`.
template <typename T>
__device__ __forceinline__ void offer_edges(TopShared& sh, const Part<T>& p, uint32_t bound) {
    const int32_t first = p.cut.head + 8 * p.c0, last = p.cut.head + 8 * p.c1;
    const int32_t i = threadIdx.x < 8 ? p.lo + static_cast<int32_t>(threadIdx.x)
                                      : last + static_cast<int32_t>(threadIdx.x) - 8;
    if (threadIdx.x < 16 && (threadIdx.x < 8 ? i < first : i < p.hi)) {
        const uint32_t key = key_of(to_f32(p.row[i]));
        if (key >= bound) offer(sh, key, i);
    }
}

// Offers every element of the part with a key of at least `bound`, and
// returns how many there are.
template <typename T, int NT>
__device__ int offer_all(TopShared& sh, const Part<T>& p, uint32_t bound) {
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    for (int32_t c = p.c0 + threadIdx.x; c < p.c1; c += NT) {
        Chunk<T> x;
        x.load(p.row + p.cut.head + 8 * c);
        offer_chunk(sh, p, c, x, bound);
    }
    offer_edges(sh, p, bound);
    __syncthreads();
    return sh.count;
}

// Number of elements of the part with a key of at least `bound`.
template <typename T, int NT>
__device__ int count_from(TopShared& sh, const Part<T>& p, uint32_t bound) {
    int n = 0;
    for (int32_t i = p.lo + threadIdx.x; i < p.hi; i += NT) n += key_of(to_f32(p.row[i])) >= bound;
    __syncthreads();
    if (threadIdx.x == 0) sh.sum = 0;
    __syncthreads();
    atomicAdd(&sh.sum, n);
    __syncthreads();
    return sh.sum;
}

// Adds to the candidates the first `need` elements, by index, whose key
// equals `key`.
template <typename T, int NT>
__device__ void offer_equal(TopShared& sh, const Part<T>& p, uint32_t key, int need) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int have = 0;  // the same in every thread
    for (int32_t base = p.lo; base < p.hi && have < need; base += NT) {
        const int32_t i = base + threadIdx.x;
        const bool eq = i < p.hi && key_of(to_f32(p.row[i])) == key;
        const uint32_t m = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) sh.group[warp] = __popc(m);
        __syncthreads();
        int before = have, all = 0;
        for (int w = 0; w < NT / 32; ++w) {
            const int c = static_cast<int>(sh.group[w]);
            if (w < warp) before += c;
            all += c;
        }
        before += __popc(m & ((1u << lane) - 1u));
        if (eq && before < need) offer(sh, key, i);
        have += all;
        __syncthreads();
    }
}

// Finds candidates for the part's k best elements, sh.cand, and returns their
// number: at least k unless the part has fewer elements.
//
// Every thread knows the largest element of its share (best; `any`: it has
// a share).  The k-th largest of the 128 groups' maxima is a lower bound of
// the part's k-th largest element, and only the threads whose own maximum
// reaches it hold candidates: about k to 1.5 k of them, whose shares are
// read again (from L2) by the whole block.  (Of a binary32 bound only the upper
// half is found, which admits a few candidates more.)  They are then ranked by
// counting.  Masses of equal values or shares that hold the top in a
// regular pattern overflow the candidate list; then the exact k-th value is
// found bit by bit, and equal ones are taken in index order.
template <typename T, int NT>
__device__ int find_top(TopShared& sh, const Part<T>& p, float best, bool any, int k) {
    const int tid = threadIdx.x;
    const uint32_t mine = any ? key_of(best) : 0u;
    uint32_t g = mine;
#pragma unroll
    for (int o = NT / kGroups / 2; o > 0; o >>= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (tid == 0) sh.flagged = sh.count = 0;
    if (tid % (NT / kGroups) == 0) sh.group[tid / (NT / kGroups)] = g;
    __syncthreads();
    // the bound, bit by bit from the top: 16 bits here, the others if it has to
    // be exact
    const int lane = tid & 31;
    uint32_t bound = 0;
    const auto settle = [&](int from, int to) {  // two bits at a time
        const uint4 x = *reinterpret_cast<const uint4*>(&sh.group[4 * lane]);
        for (int b = from - 1; b >= to; b -= 2) {
            int n[4];
#pragma unroll
            for (int t = 1; t < 4; ++t) {
                const uint32_t c = bound + (static_cast<uint32_t>(t) << b);
                n[t] = __reduce_add_sync(0xffffffffu,
                                         (x.x >= c) + (x.y >= c) + (x.z >= c) + (x.w >= c));
            }
            bound += static_cast<uint32_t>(n[3] >= k ? 3 : n[2] >= k ? 2 : n[1] >= k ? 1 : 0) << b;
        }
    };
    if (tid < 32) {
        settle(31, 16);
        if (sizeof(T) == 2 && !(bound >> 31)) bound |= 0xffffu;  // the key of a negative bf16
        if (tid == 0) sh.bound = bound;
    }
    __syncthreads();
    bound = sh.bound;
    const uint32_t reach = __ballot_sync(0xffffffffu, mine >= bound && any);
    if (reach) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.flagged, __popc(reach));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(reach & ((1u << lane) - 1u));
        if (reach >> lane & 1u) sh.thread[at] = static_cast<uint16_t>(tid);
    }
    __syncthreads();
    const int flagged = sh.flagged;
    const int share = (p.c1 - p.c0 + NT - 1) / NT;
    bool over = flagged > 4 * k + 32;
    if (!over) {
        // Chunks whose loads are in flight together: one / four, 8192 x 50257 bf16 with
        // 20 alternatives 172 / 163 us (4 rows 7.7 / 7.8); binary32 lacks the registers
        // (two: 8192 x 31999 191 us, not 187).
        constexpr int U = sizeof(T) == 2 ? 4 : 1;
        for (int i = tid; i < flagged * share; i += U * NT) {
            Chunk<T> x[U];
            int32_t c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = i + u * NT;
                c[u] = k < flagged * share ? p.c0 + sh.thread[k % flagged] + (k / flagged) * NT : p.c1;
                if (c[u] < p.c1) x[u].load(p.row + p.cut.head + 8 * c[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c[u] < p.c1) offer_chunk(sh, p, c[u], x[u], bound);
        }
        offer_edges(sh, p, bound);
        __syncthreads();
        over = sh.count > kCandidates;
    }
    if (over) {  // block-uniform
        if (sizeof(T) == 4) settle(15, 0);
        int above = offer_all<T, NT>(sh, p, bound + 1);
        if (above > kCandidates) {
            bound = 0;
            for (int b = 31; b >= 0; --b) {
                const uint32_t c = bound | (1u << b);
                if (count_from<T, NT>(sh, p, c) >= k) bound = c;
            }
            above = offer_all<T, NT>(sh, p, bound + 1);
        }
        if (above < k) offer_equal<T, NT>(sh, p, bound, k - above);
        __syncthreads();
    }
    return min(sh.count, kCandidates);
}

// put(rank, candidate) for the k best of n candidates: ranked by counting.
template <int NT, typename Put>
__device__ __forceinline__ void rank_top(const uint64_t* cand, int n, int k, const Put& put) {
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t me = cand[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += cand[j] > me;
        if (rank < k) put(rank, me);
    }
}

// The row's outputs but for the alternatives.  q.s > 0, 0 (no element with
// weight) or NaN; y: the target, whose logit is xy, or -1.
template <bool ENT>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t r, const Soft& q, float logs,
                                          int32_t y, float xy) {
    const bool none = q.s == 0.0f;
    a.logprob[r] = y < 0 ? 0.0f
                   : none ? neg_inf()
                          : __fsub_rn(fmaf(xy, a.scale, -q.mz), logs);
    if (a.lse) a.lse[r] = none ? neg_inf() : __fadd_rn(q.mz, logs);
    if (ENT) a.entropy[r] = none ? 0.0f : __fsub_rn(logs, __fdiv_rn(__fmul_rn(q.a, kLn2), q.s));
}

// One row per warp, for many short rows: nothing is joined across warps.
template <typename T, int U, bool ENT>
__global__ void __launch_bounds__(128) logprob_warp_kernel(const __grid_constant__ LogprobArgs a) {
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (r >= a.n) return;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    const RowCut<T> cut(row, a.vocab);
    int32_t y = -1;
    float xy = 0.0f;
    if (lane == 0) {
        y = load_id(a.targets, a.id64, r, a.vocab);
        if (y >= 0) xy = to_f32(row[y]);
    }
    Soft q = soft_empty();
    soft_stream<T, ENT, 32, U>(q, row, cut, 0, cut.chunks, true, true, a.scale, lane);
    soft_lanes<ENT, 32>(q);
    if (lane == 0) write_row<ENT>(a, r, q, q.s == 0.0f ? 0.0f : logf(q.s), y, xy);
}

// Threads an SM is to hold: bytes in flight and warps to hide the exponentials
// behind, against the registers of the loads.  8192 rows of 50257 bf16 take, at
// 1280 / 1536 / 2048 threads, 131 / 127 / 129 us with entropy and 128 / 123 / 120 us
// without; binary32 238 / 234 / 242 us.
template <typename T, bool ENT, bool TOP>
constexpr int resident() {
    return sizeof(T) == 4 && TOP ? 1024 : sizeof(T) == 2 && !ENT && !TOP ? 2048 : 1536;
}

// One row per cluster of a.cluster blocks (one block where rows abound).
// Bound by HBM: the row is read once, each thread keeping the running
// maximum, sum and weighted sum of its share in registers (8192 rows of 50257 bf16
// with entropy: 125 us, 6.6 TB/s; with 20 alternatives 163 us; 1021 of 31999 binary32
// with 5 alternatives 31 us).  With few rows bound by latency: 4 rows of 50257
// take 4.0 us without alternatives and 7.8 us with 20.
template <typename T, int NT, int U, bool ENT, bool TOP>
__global__ void __launch_bounds__(NT, resident<T, ENT, TOP>() / NT)
    logprob_kernel(const __grid_constant__ LogprobArgs a) {
    __shared__ Soft sh_soft[NT / 32];
    __shared__ Soft sh_parts[kMaxCluster];
    __shared__ TopShared sh_top;
    wait_prior_grids();
    allow_next_grid();
    const int tid = threadIdx.x;
    const int C = a.cluster;
    if (C > 1) cluster_arrive();
    const int64_t r = blockIdx.x / C;
    const int part = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    const RowCut<T> cut(row, a.vocab);
    const int32_t c0 = static_cast<int32_t>(static_cast<int64_t>(cut.chunks) * part / C);
    const int32_t c1 = static_cast<int32_t>(static_cast<int64_t>(cut.chunks) * (part + 1) / C);
    const bool head = part == 0, tail = part == C - 1;
    // the target's logit, wanted at the end
    int32_t y = -1;
    float xy = 0.0f;
    if (part == 0 && tid == 0) {
        y = load_id(a.targets, a.id64, r, a.vocab);
        if (y >= 0) xy = to_f32(row[y]);
    }
    Soft q = soft_empty();
    soft_stream<T, ENT, NT, U>(q, row, cut, c0, c1, head, tail, a.scale, tid);
    const float best = q.m;
    soft_block<ENT, NT>(q, sh_soft);
    int n = 0;  // candidates
    const uint64_t* cand = sh_top.cand;
    if (TOP && !isnan(q.s)) {  // the same in every thread
        const Part<T> p{row, cut, c0, c1, head ? 0 : cut.head + 8 * c0,
                        tail ? a.vocab : cut.head + 8 * c1};
        const bool any = c0 + tid < c1 || (tid == 0 && head && cut.head) ||
                         (tid == NT - 1 && tail && cut.tail);
        n = find_top<T, NT>(sh_top, p, best, any, a.k);
    }
    if (C > 1) {
        cluster_wait();  // the first block has started
        if (tid == 0) send_cluster(&sh_parts[part], 0, q);
        if (TOP) {  // the best k, or as many as there are and then zeros
            uint64_t* const to = &sh_top.list[part * a.k];
            rank_top<NT>(cand, n, a.k, [&](int i, uint64_t c) { send_cluster(to + i, 0, c); });
            if (tid < a.k && tid >= n) send_cluster(to + tid, 0, 0);
        }
        cluster_sync();
        if (part != 0) return;
        q = soft_parts<ENT>(sh_parts, C);
        cand = sh_top.list;
        n = C * a.k;
    }
    const bool none = q.s == 0.0f;
    const float logs = none ? 0.0f : logf(q.s);
    if (tid == 0) write_row<ENT>(a, r, q, logs, y, xy);
    if (!TOP) return;
    int32_t* const ids = a.top_ids + r * a.k;
    float* const lps = a.top_logprobs + r * a.k;
    if (isnan(q.s)) {
        if (tid < a.k) {
            ids[tid] = -1;
            lps[tid] = q.s;
        }
        return;
    }
    rank_top<NT>(cand, n, a.k, [&](int i, uint64_t c) {
        ids[i] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(c));
        const float x = value_of(static_cast<uint32_t>(c >> 32));
        lps[i] = none ? neg_inf() : __fsub_rn(fmaf(x, a.scale, -q.mz), logs);
    });
}

// ---------------------------------------------------------------- gradient
// dx_j = scale ([j = y] g - p_j (g + h (log p_j + H))), log p_j = z_j - lse.
struct GradRow {
    float scale, neg_lse;
    float c0, c1;  // dx_j = p_j (c0 + c1 (z_j - lse)) besides the target
    float hit;     // what the target gets on top
    int32_t y;
};

template <bool ENT>
__device__ __forceinline__ float grad_value(float x, const GradRow& g) {
    const float d = fmaf(x, g.scale, g.neg_lse);
    const float p = exp2_approx(__fmul_rn(d, kLog2e));
    if (!ENT) return __fmul_rn(p, g.c0);
    return __fmul_rn(p, fmaf(max_nan(d, kNoWeight), g.c1, g.c0));
}

template <typename T, bool ENT>
__device__ __forceinline__ void grad_chunk(const Chunk<T>& c, T* out, int32_t at, const GradRow& g) {
    const uint64_t sc = pk2(g.scale, g.scale), nl = pk2(g.neg_lse, g.neg_lse);
    const uint64_t l2 = pk2(kLog2e, kLog2e), c0 = pk2(g.c0, g.c0), c1 = pk2(g.c1, g.c1);
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint64_t d = fma2(c.pair(k), sc, nl);
        float t0, t1;
        upk2(mul2(d, l2), t0, t1);
        const uint64_t p = pk2(exp2_approx(t0), exp2_approx(t1));
        uint64_t w = c0;
        if (ENT) {  // d = -inf has weight 0: keep 0 * d finite
            upk2(d, t0, t1);
            w = fma2(pk2(max_nan(t0, kNoWeight), max_nan(t1, kNoWeight)), c1, c0);
        }
        upk2(mul2(p, w), f[2 * k], f[2 * k + 1]);
    }
    const uint32_t h = static_cast<uint32_t>(g.y - at);  // y < 0 never matches: at >= 0
    if (h < 8u) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (h == static_cast<uint32_t>(e)) f[e] = __fadd_rn(f[e], g.hit);
    }
    Chunk<T>::store(out + at, f);
}

// A block takes 8 * NT * U consecutive elements of one row.  Elementwise and
// bound by HBM (one read, one write; 8192 x 50257 bf16 with entropy 236 us, 7.0 TB/s); in-place is allowed, so every element
// is read by the thread that writes it.  SAME: row and gradient row start at
// the same distance from a 16-byte boundary, so one cut serves both.
template <typename T, bool ENT, bool SAME, int NT, int U>
__global__ void __launch_bounds__(NT)
    logprob_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
    wait_prior_grids();
    allow_next_grid();
    const int64_t r = blockIdx.x / a.segments;
    const int32_t seg = static_cast<int32_t>(blockIdx.x - r * a.segments);
    const int tid = threadIdx.x;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    T* out = static_cast<T*>(a.dx) + r * a.dx_stride;
    const RowCut<T> cut(row, a.vocab);
    const int32_t i0 = seg * NT * U + tid;
    Chunk<T> c[U];
    if (SAME) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * NT < cut.chunks)
                c[u].load_stream(row + cut.head + 8 * static_cast<int64_t>(i0 + u * NT));
    }
    GradRow g;
    const float lse = a.lse[r];
    g.y = load_id(a.targets, a.id64, r, a.vocab);
    const float gl = g.y >= 0 && a.dlogprob ? a.dlogprob[r] : 0.0f;
    g.scale = a.scale;
    g.neg_lse = -lse;
    g.hit = __fmul_rn(gl, a.scale);
    g.c0 = -g.hit;
    g.c1 = 0.0f;
    if (ENT) {
        const float h = __fmul_rn(a.dentropy[r], a.scale);
        g.c0 = -fmaf(h, a.entropy[r], g.hit);
        g.c1 = -h;
    }
    if (lse == neg_inf()) {  // nothing left in the row: no gradient
        g.neg_lse = 0.0f;
        g.scale = 0.0f;
        g.c0 = g.c1 = g.hit = 0.0f;
    }
    const bool none = lse == neg_inf();
    if (SAME) {
        if (none) {
#pragma unroll
            for (int u = 0; u < U; ++u) c[u].fill(0.0f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * NT < cut.chunks)
                grad_chunk<T, ENT>(c[u], out, cut.head + 8 * (i0 + u * NT), g);
        if (seg == 0 && tid < 16) {
            const int32_t i = tid < 8 ? tid : cut.head + 8 * cut.chunks + tid - 8;
            if (tid < 8 ? i < cut.head : i < a.vocab) {
                float v = none ? 0.0f : grad_value<ENT>(to_f32(row[i]), g);
                if (i == g.y) v = __fadd_rn(v, g.hit);
                out[i] = from_f32<T>(v);
            }
        }
    } else {
        const int64_t lo = static_cast<int64_t>(seg) * NT * U * 8;
#pragma unroll 8
        for (int u = 0; u < 8 * U; ++u) {
            const int64_t i = lo + u * NT + tid;
            if (i < a.vocab) {
                float v = none ? 0.0f : grad_value<ENT>(to_f32(row[i]), g);
                if (i == g.y) v = __fadd_rn(v, g.hit);
                out[i] = from_f32<T>(v);
            }
        }
    }
}

template <typename T, bool ENT, bool TOP, int NT>
cudaError_t launch_blocks(LogprobArgs a, cudaStream_t stream) {
    // Chunks in flight per thread: 64 bytes, but 128 of binary32 where registers
    // limit the warps anyway.  Two / four chunks: 8192 x 31999 binary32 148 / 194 us,
    // with alternatives 191 / 187; 8192 x 4000 bf16 19.0 / 17.6.
    constexpr int U = sizeof(T) == 2 || TOP ? 4 : 2;
    const int64_t chunks = a.vocab / 8;
    // Blocks per row, up to the SMs' number: 4 rows of 50257 take 4.0 us (one block per
    // row: 5.2), 64 8.0 (8.7; 12.3 with up to 304 blocks).
    int C = 1;
    while (C < 8 && a.n * C < 152 && chunks / (2 * C) >= 2 * NT) C *= 2;
    a.cluster = C;
    return launch_vocab(logprob_kernel<T, NT, U, ENT, TOP>, a.n * C, NT, 0, C, a, stream);
}

template <typename T, bool ENT, bool TOP>
cudaError_t launch_fwd(const LogprobArgs& a, cudaStream_t stream) {
    // Many short rows: one per warp (8192 rows of bf16, by warps / by
    // blocks: 8000 28 / 30 us, 4000 18 / 22).
    if (!TOP && a.vocab <= 8192 && a.n >= 608)
        return launch_vocab(logprob_warp_kernel<T, sizeof(T) == 2 ? 4 : 2, ENT>, (a.n + 3) / 4, 128, 0,
                            1, a, stream);
    // Smaller blocks where the rows are short, or neither long nor too few to
    // fill the SMs with them: the join and the alternatives of a row then hide
    // behind more other rows.  128 / 256 threads, with 20 alternatives: 4096 rows
    // of 16000 40 / 46 us, 1000 of 16000 18 / 16, 2048 of 50257 70 / 54.
    const bool small = a.vocab <= 8192 || (a.vocab <= 24576 && a.n >= 1824);
    return small ? launch_blocks<T, ENT, TOP, 128>(a, stream) : launch_blocks<T, ENT, TOP, 256>(a, stream);
}

template <typename T>
cudaError_t launch_fwd_type(const LogprobArgs& a, cudaStream_t stream) {
    if (a.entropy)
        return a.k ? launch_fwd<T, true, true>(a, stream) : launch_fwd<T, true, false>(a, stream);
    return a.k ? launch_fwd<T, false, true>(a, stream) : launch_fwd<T, false, false>(a, stream);
}

template <typename T, bool ENT>
cudaError_t launch_bwd(LogprobGradArgs a, cudaStream_t stream) {
    // 4096 elements per block: with 8192, 9624 rows of 1097 bf16 take 17.0 us, not
    // 11.6, and 8192 rows of 50257 239, not 236; with 2048 1097's take 10.8 and
    // 50257's 247
    constexpr int NT = 128, U = 4;
    a.segments = (a.vocab + 8 * NT * U - 1) / (8 * NT * U);
    const auto phase = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) / sizeof(T)) % Chunk<T>::kPhase; };
    const bool same = phase(a.x) == phase(a.dx) &&
                      (a.n == 1 || (a.stride - a.dx_stride) % Chunk<T>::kPhase == 0);
    const int64_t grid = a.n * a.segments;
    return same ? launch_vocab(logprob_grad_kernel<T, ENT, true, NT, U>, grid, NT, 0, 1, a, stream)
                : launch_vocab(logprob_grad_kernel<T, ENT, false, NT, U>, grid, NT, 0, 1, a, stream);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
    return a.dtype == ZERO3_F32 ? launch_fwd_type<float>(a, stream)
                                : launch_fwd_type<uint16_t>(a, stream);
}

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t stream) {
    if (a.dtype == ZERO3_F32)
        return a.dentropy ? launch_bwd<float, true>(a, stream) : launch_bwd<float, false>(a, stream);
    return a.dentropy ? launch_bwd<uint16_t, true>(a, stream)
                      : launch_bwd<uint16_t, false>(a, stream);
}

}  // namespace z3
