// Distillation from a teacher's top logits: loss, loss with gradient in one
// call, and gradient alone (sm_103a).
//
//   q = softmax over the row's valid teacher entries of t_k * scale
//   loss = sum_k q_k (log q_k - log p_{id_k}) / scale^2,  p = softmax(x * scale)
//   d loss / d x_j = (p_j - sum_{k: id_k = j} q_k) / scale
//
// A block has NT threads that stream logits and one more warp that works on
// the teacher's list meanwhile: a list costs several dependent loads (token,
// then the student's logit there) and a softmax of its own.  The gradient's
// elements at the teacher's tokens are written by the list's warp, after the
// streaming threads' stores.  Both roles meet at the same barrier statements: a
// role's work stands between them, no barrier inside a branch that only one role
// takes.
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {
namespace {

enum class Make { kLoss, kBoth, kGrad };

// ------------------------------------------------------------------- teacher
constexpr int kMapBits = 65536;

// A row's list in shared memory, k entries, and room to find repeated tokens.
struct Teacher {
    float* q;       // logits, then probabilities
    float* x;       // the student's logits at the tokens
    int32_t* id;    // tokens; -1 where the entry does not count or repeats a token
    uint32_t* map;  // a bit per token of the block's part, or list_merge's table
    int32_t map_bytes;
    __device__ __forceinline__ Teacher(void* p, const DistillArgs& a)
        : q(static_cast<float*>(p)), x(q + a.k), id(reinterpret_cast<int32_t*>(x + a.k)),
          map(reinterpret_cast<uint32_t*>(static_cast<char*>(p) + entry_bytes(a.k))),
          map_bytes(a.map_bytes) {}
    __host__ __device__ static constexpr int entry_bytes(int k) { return (12 * k + 15) / 16 * 16; }
    // slots of list_merge's table: a power of two, at most half full
    __host__ __device__ static constexpr int table(int k) {
        int t = 32;
        while (t < 2 * k) t *= 2;
        return t;
    }
    // of the map, for parts of up to `tokens`
    __host__ static int bytes_of_map(int k, int64_t tokens) {
        const int64_t bits = tokens < kMapBits ? tokens : kMapBits;
        const int64_t map = (bits + 127) / 128 * 16, both = 8 * table(k);
        return static_cast<int>(map > both ? map : both);
    }
};

// What the loss needs of a list: with r the largest student z among the
// tokens, sum q (log q - z + r).  loss = that + (lse - r).
struct ListSums {
    float cross, ref;
};

// What a list is as a whole.
enum ListKind : int { kListPlain, kListEmpty, kListNan };

// The list's warp, for row r, first step: its entries.  An entry counts if its
// token lies in the vocabulary and its logit is not -inf.  Returns the list's
// kind (in every lane): empty if no entry counts, NaN if the softmax of those
// that do is.
constexpr int kEntries = 4;  // entries per lane whose loads are in flight together
__device__ __forceinline__ ListKind list_entries(const DistillArgs& a, int64_t r, const Teacher& t) {
    const int lane = threadIdx.x & 31;
    const int64_t base = r * a.teacher_stride;
    bool some = false, nan = false;
    for (int b = lane; b < a.k; b += 32 * kEntries) {
        // loads without branches between them (a lane past the end takes the
        // last entry), so that all are in flight together
        uint32_t lo[kEntries], hi[kEntries];
        float v[kEntries];
        if (a.id64) {
#pragma unroll
            for (int u = 0; u < kEntries; ++u) {
                const uint2 x = static_cast<const uint2*>(a.teacher_ids)[base + min(b + 32 * u, a.k - 1)];
                lo[u] = x.x;
                hi[u] = x.y;
            }
        } else {
#pragma unroll
            for (int u = 0; u < kEntries; ++u) {
                lo[u] = static_cast<const uint32_t*>(a.teacher_ids)[base + min(b + 32 * u, a.k - 1)];
                hi[u] = 0;
            }
        }
        if (a.teacher_dtype == ZERO3_F32) {
#pragma unroll
            for (int u = 0; u < kEntries; ++u)
                v[u] = static_cast<const float*>(a.teacher)[base + min(b + 32 * u, a.k - 1)];
        } else {
#pragma unroll
            for (int u = 0; u < kEntries; ++u)
                v[u] = bf16_f32(static_cast<const uint16_t*>(a.teacher)[base + min(b + 32 * u, a.k - 1)]);
        }
#pragma unroll
        for (int u = 0; u < kEntries; ++u) {
            const int k = b + 32 * u;
            if (k >= a.k) break;
            const float z = __fmul_rn(v[u], a.scale);
            const bool counts = hi[u] == 0 && lo[u] < static_cast<uint32_t>(a.vocab) && z != neg_inf();
            t.id[k] = counts ? static_cast<int32_t>(lo[u]) : -1;
            t.q[k] = v[u];
            some = some || counts;
            nan = nan || (counts && !(z < -neg_inf()));
        }
    }
    return __any_sync(0xffffffffu, nan) ? kListNan
           : __any_sync(0xffffffffu, some) ? kListPlain
                                           : kListEmpty;
}

// Second step: the student's logits at its tokens in [lo, hi).
template <typename T>
__device__ __forceinline__ void list_logits(const DistillArgs& a, const T* row, int32_t lo, int32_t hi,
                                            const Teacher& t) {
    const int lane = threadIdx.x & 31;
    for (int b = lane; b < a.k; b += 32 * kEntries) {
        T x[kEntries];
#pragma unroll
        for (int u = 0; u < kEntries; ++u) {  // without branches, as above
            const int32_t id = t.id[min(b + 32 * u, a.k - 1)];
            x[u] = row[id >= lo && id < hi ? id : 0];
        }
#pragma unroll
        for (int u = 0; u < kEntries; ++u)
            if (b + 32 * u < a.k) t.x[b + 32 * u] = to_f32(x[u]);
    }
}

// Third step: the softmax; t.q turns from logits into probabilities.
__device__ __forceinline__ ListSums list_softmax(const DistillArgs& a, const Teacher& t) {
    const int lane = threadIdx.x & 31;
    float top = neg_inf(), ref = neg_inf();
    for (int k = lane; k < a.k; k += 32) {
        if (t.id[k] < 0) continue;
        top = fmaxf(top, t.q[k]);
        ref = fmaxf(ref, t.x[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    }
    top = __fmul_rn(top, a.scale);
    if (top == neg_inf()) top = 0.0f;  // a list that is empty
    ref = __fmul_rn(ref, a.scale);
    if (ref == neg_inf()) ref = 0.0f;
    float sum = 0.0f;
    for (int k = lane; k < a.k; k += 32) {
        if (t.id[k] < 0) continue;
        const float d = fmaf(t.q[k], a.scale, -top);
        sum = __fadd_rn(sum, exp2_approx(__fmul_rn(d, kLog2e)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    const float inv = __fdiv_rn(1.0f, sum), logs = logf(sum);
    float cross = 0.0f;
    for (int k = lane; k < a.k; k += 32) {
        if (t.id[k] < 0) continue;
        const float d = fmaf(t.q[k], a.scale, -top);
        const float q = __fmul_rn(exp2_approx(__fmul_rn(d, kLog2e)), inv);
        if (q != 0.0f)  // log q - (z - ref)
            cross = fmaf(q, __fsub_rn(__fsub_rn(d, logs), fmaf(t.x[k], a.scale, -ref)), cross);
        t.q[k] = q;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cross = __fadd_rn(cross, __shfl_xor_sync(0xffffffffu, cross, o));
    return ListSums{cross, ref};
}

// Whether a token in [lo, hi) may be listed twice (in every lane): a bit per
// token, shared by tokens kMapBits apart.  The map is Teacher::map.
__device__ __forceinline__ bool list_repeats(const DistillArgs& a, const Teacher& t, int32_t lo,
                                             int32_t hi) {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < t.map_bytes / 16; i += 32)
        reinterpret_cast<uint4*>(t.map)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
    bool twice = false;
    for (int k = lane; k < a.k; k += 32) {
        const int32_t id = t.id[k];
        if (id < lo || id >= hi) continue;
        const uint32_t bit = static_cast<uint32_t>(id - lo) & (kMapBits - 1);
        twice = twice || (atomicOr(t.map + bit / 32, 1u << (bit & 31)) >> (bit & 31) & 1u);
    }
    return __any_sync(0xffffffffu, twice);
}

// Leaves one entry per distinct token, which holds the sum of its entries'
// probabilities in list order (fixed, 32 entries at a time); the others' id
// turns -1.  A hash table over the map's memory finds the entry of a token.
// Slow (a chain of atomics): only where tokens repeat.
__device__ __forceinline__ void list_merge(int count, const Teacher& t) {
    const int lane = threadIdx.x & 31;
    const uint32_t slots = Teacher::table(count), mask = slots - 1u;
    int32_t* const key = reinterpret_cast<int32_t*>(t.map);  // tokens, and after them
    int32_t* const at = key + slots;                          // the entry that stands for each
    __syncwarp();
    for (uint32_t s = lane; s < slots; s += 32) key[s] = -1;
    for (int b = 0; b < count; b += 32) {
        __syncwarp();
        const int k = b + lane;
        int32_t id = k < count ? t.id[k] : -1;
        float q = id >= 0 ? t.q[k] : 0.0f;
        // entries of this 32 with the same token: the first adds up the others
        const uint32_t peers = __match_any_sync(0xffffffffu, id);
        const bool lead = id >= 0 && (peers & ((1u << lane) - 1u)) == 0;
        for (int l = 1; l < 32; ++l) {
            const float o = __shfl_sync(0xffffffffu, q, l);
            if (lead && l > lane && (peers >> l & 1u)) q = __fadd_rn(q, o);
        }
        // and stands in the table or adds to the entry that does
        if (lead) {
            uint32_t s = static_cast<uint32_t>(id) * 2654435761u >> 12 & mask;
            for (uint32_t tries = 0; tries <= mask; ++tries) {  // at most half are taken
                const int32_t there = atomicCAS(&key[s], -1, id);
                if (there == -1) {
                    at[s] = k;
                    t.q[k] = q;
                    break;
                }
                if (there == id) {
                    t.q[at[s]] = __fadd_rn(t.q[at[s]], q);
                    id = -1;
                    break;
                }
                s = (s + 1) & mask;
            }
        } else {
            id = -1;
        }
        if (k < count) t.id[k] = id;
    }
    __syncwarp();
}

// ------------------------------------------------------------------ gradient
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
// Writes the gradient at the teacher's tokens in [lo, hi): `threads` threads
// from `tid` on.
template <typename T>
__device__ __forceinline__ void write_teacher(const DistillArgs& a, const Teacher& t, T* out,
                                              int64_t lo, int64_t hi, const Sweep& w, int tid,
                                              int threads) {
    for (int k = tid; k < a.k; k += threads) {
        const int32_t id = t.id[k];
        if (id >= lo && id < hi) out[id] = from_f32<T>(fmaf(-w.c, t.q[k], sweep_value(t.x[k], w)));
    }
}

// Whether a row's gradient is zero: no entry counts, or no student token is left
// (none).  A list with a NaN makes it NaN, as it does the loss.
__device__ __forceinline__ bool no_gradient(ListKind kind, bool none) {
    return kind == kListEmpty || (kind == kListPlain && none);
}

__device__ __forceinline__ float row_coef(const DistillArgs& a, int64_t r) {
    const float w = a.weight ? a.weight[r] : 1.0f;
    return __fdiv_rn(w, a.scale);
}

// ---------------------------------------------------------------------- loss
// The row's statistics, joined over the block's W warps and a cluster's C
// blocks, which have arrived when they started.  `sh` has been filled and a
// barrier passed; every thread calls.
template <int W>
__device__ __forceinline__ Soft soft_all(const Soft* sh, Soft* parts, int C, int part) {
    Soft q = sh[(threadIdx.x & 31) % W];
    soft_lanes<false, W>(q);
    if (C == 1) return q;
    cluster_wait();  // every block has started
    if (threadIdx.x < static_cast<unsigned>(C)) send_cluster(parts + part, threadIdx.x, q);
    cluster_sync();
    return soft_parts<false>(parts, C);
}

__device__ __forceinline__ void write_loss(const DistillArgs& a, int64_t r, const Soft& q,
                                           const ListSums& l, ListKind kind, float logs) {
    const bool none = q.s == 0.0f;
    float loss = 0.0f;
    if (kind == kListNan)
        loss = __int_as_float(0x7fffffff);
    else if (!none && kind != kListEmpty)
        loss = __fadd_rn(l.cross, __fadd_rn(__fsub_rn(q.mz, l.ref), logs));
    a.loss[r] = __fdiv_rn(__fdiv_rn(loss, a.scale), a.scale);
    if (a.lse) a.lse[r] = none ? neg_inf() : __fadd_rn(q.mz, logs);
}

// A block's part of a row: `n` chunks from element `start` on, elements
// [lo, hi).
template <typename T>
struct RowPart {
    const T* row;
    int32_t start, n, lo, hi;
    __device__ __forceinline__ RowPart(const DistillArgs& a, int64_t r, int part) {
        row = static_cast<const T*>(a.x) + r * a.stride;
        const RowCut<T> cut(row, a.vocab);
        const int shift = 31 - __clz(a.cluster);
        const int32_t c0 = static_cast<int32_t>(static_cast<int64_t>(cut.chunks) * part >> shift);
        const int32_t c1 = static_cast<int32_t>(static_cast<int64_t>(cut.chunks) * (part + 1) >> shift);
        start = cut.head + 8 * c0;
        n = c1 - c0;
        lo = part == 0 ? 0 : start;
        hi = part + 1 == a.cluster ? a.vocab : start + 8 * n;
    }
};

// The gradient, with (kBoth) or without (kGrad) the loss, of logits whose
// gradient's rows are equally far from a 16-byte boundary.  One row per
// cluster of a.cluster blocks.
//
// Bound by HBM (each logit read once, its gradient written once); kBoth reads
// a row twice, the second time from L2, where the rows in flight (a few per
// SM) stay.  What it takes is bytes in flight and few instructions per chunk:
// the chunks of both passes come through one ring of two batches per thread
// in shared memory, filled by asynchronous 16-byte copies (each thread reads
// what it copied itself, so no barrier orders them), and the second pass's
// first chunks are on their way while the block joins the row's statistics.
// 8192 rows of 50257 bf16, 64 entries, loss and gradient: 272 us (1.65 GB, 6.1 TB/s; a
// tenth of the second pass misses L2); gradient alone, 4096 of 32000 with 100
// entries, 82 us (6.4 TB/s).  Where the rows in flight outgrow L2 the second pass reads
// HBM: 4096 of 50257 binary32, loss and gradient, 530 us (floor 247).
template <typename T, Make M, int NT>
__global__ void __launch_bounds__(NT + 32) distill_kernel(const __grid_constant__ DistillArgs a) {
    constexpr bool LOSS = M == Make::kBoth;
    constexpr int U = RowRing<T, NT>::U;
    extern __shared__ uint4 dyn[];
    __shared__ Soft sh[NT / 32];
    __shared__ Soft sh_parts[kMaxCluster];
    __shared__ ListKind sh_kind;
    wait_prior_grids();
    allow_next_grid();
    const int tid = threadIdx.x;
    const bool lister = tid >= NT;  // the list's warp
    const int C = a.cluster;
    if (LOSS && C > 1) cluster_arrive();
    const int64_t r = blockIdx.x / C;
    const int part = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const RowPart<T> p(a, r, part);
    T* const out = static_cast<T*>(a.dx) + r * a.dx_stride;
    const int32_t last = p.start + 8 * p.n;
    // (the gradient alone waits for these next to the list's entries)
    const float lse = LOSS ? 0.0f : a.lse[r], coef = LOSS ? 0.0f : row_coef(a, r);
    const Teacher t(dyn + RowRing<T, NT>::kBytes / 16, a);
    const RowRing<T, NT> ring(dyn, p.row + p.start, p.n, tid, LOSS ? 2 : 1);  // not the list's warp's
    // The others' writes wait for the list's logits only where they overwrite
    // them; the loss wants the logits at all tokens, from its first part.
    const bool early = LOSS || a.dx == a.x;
    const bool all = LOSS && part == 0;
    int32_t edge = -1;
    T edge_x = from_f32<T>(0.0f);
    ListSums l{0.0f, 0.0f};
    Soft q = soft_empty();
    if (lister) {
        const ListKind kind = list_entries(a, r, t);
        if (tid == NT) sh_kind = kind;
        if (early) list_logits<T>(a, p.row, all ? 0 : p.lo, all ? a.vocab : p.hi, t);
        if (LOSS) {
            l = list_softmax(a, t);
            if (list_repeats(a, t, p.lo, p.hi)) list_merge(a.k, t);
        }
    } else {
        ring.send(0);
        ring.send(1);
        edge = edge_element(p.lo, p.start, last, p.hi);
        if (edge >= 0) edge_x = p.row[edge];
        if (LOSS) {
            if (edge >= 0) soft_element<T, false>(q, edge_x, a.scale);
            soft_ring<T, false, NT>(q, ring, a.scale);
            soft_lanes<false, 32>(q);
            if ((tid & 31) == 0) sh[tid >> 5] = q;
        }
    }
    __syncthreads();
    const ListKind kind = sh_kind;
    if (LOSS) {
        q = soft_all<NT / 32>(sh, sh_parts, C, part);
        if (part == 0 && tid == NT) write_loss(a, r, q, l, kind, q.s == 0.0f ? 0.0f : logf(q.s));
    }
    T* to = out + p.start + 8 * tid;
    if (no_gradient(kind, LOSS ? q.s == 0.0f : lse == neg_inf())) {  // the same in every thread
        if (lister) return;
        const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        drain_copies();
        for (int32_t c = tid; c < p.n; c += NT, to += 8 * NT) Chunk<T>::store(to, zero);
        if (edge >= 0) out[edge] = from_f32<T>(0.0f);
        return;
    }
    Sweep w;
    w.scale = a.scale;
    w.base = LOSS ? q.mz : lse;
    w.c = LOSS ? row_coef(a, r) : coef;
    w.coef = LOSS ? __fdiv_rn(w.c, q.s) : w.c;
    if (kind == kListNan) w.coef = __int_as_float(0x7fffffff);
    if (lister) {
        if (!LOSS) {
            if (!early) list_logits<T>(a, p.row, p.lo, p.hi, t);
            list_softmax(a, t);
            if (list_repeats(a, t, p.lo, p.hi)) list_merge(a.k, t);
        }
    } else {
        const int b0 = LOSS ? ring.per : 0;
#pragma unroll 1
        for (int b = 0; b < ring.full; ++b, to += 8 * U * NT) {
            Chunk<T> c[U];
            ring.take(b0 + b, c);
            ring.send(b0 + b + 2);
#pragma unroll
            for (int u = 0; u < U; ++u) sweep_chunk<T>(c[u], to + 8 * NT * u, w);
        }
        if (ring.full < ring.per) {
            Chunk<T> c[U];
            ring.take(b0 + ring.full, c);
            ring.send(b0 + ring.full + 2);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (ring.has(u)) sweep_chunk<T>(c[u], to + 8 * NT * u, w);
        }
        if (edge >= 0) out[edge] = from_f32<T>(sweep_value(to_f32(edge_x), w));
        drain_copies();
    }
    __syncthreads();  // the others have written, before the list's warp does
    if (lister) write_teacher<T>(a, t, out, p.lo, p.hi, w, tid - NT, 32);
}

// The loss alone, and the gradient of rows that are not as far from a 16-byte
// boundary as the gradient's rows (never in place: equal rows are equally far):
// one row per cluster of a.cluster blocks, the gradient written by single
// elements.  Loss of 2047 rows of 32000 binary32,
// 32 entries: 40 us (6.5 TB/s).
template <typename T, Make M, int NT, int U>
__global__ void __launch_bounds__(NT + 32) distill_plain_kernel(const __grid_constant__ DistillArgs a) {
    constexpr bool GRAD = M != Make::kLoss, LOSS = M != Make::kGrad;
    extern __shared__ uint4 dyn[];
    __shared__ Soft sh[NT / 32];
    __shared__ Soft sh_parts[kMaxCluster];
    __shared__ ListSums sh_list;
    __shared__ ListKind sh_kind;
    wait_prior_grids();
    allow_next_grid();
    const Teacher t(dyn, a);
    const int tid = threadIdx.x;
    const int C = a.cluster;
    if (LOSS && C > 1) cluster_arrive();
    const int64_t r = blockIdx.x / C;
    const int part = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const RowPart<T> p(a, r, part);
    const RowCut<T> cut(p.row, a.vocab);
    const int32_t c0 = (p.start - cut.head) / 8;
    if (tid >= NT) {
        if (GRAD || part == 0) {
            const ListKind kind = list_entries(a, r, t);
            list_logits<T>(a, p.row, 0, a.vocab, t);
            const ListSums l = list_softmax(a, t);
            if (GRAD && list_repeats(a, t, p.lo, p.hi)) list_merge(a.k, t);
            if (tid == NT) {
                sh_kind = kind;
                sh_list = l;
            }
        }
    } else if (LOSS) {
        Soft q = soft_empty();
        soft_stream<T, false, NT, U>(q, p.row, cut, c0, c0 + p.n, part == 0, part == C - 1, a.scale,
                                      tid);
        soft_lanes<false, 32>(q);
        if ((tid & 31) == 0) sh[tid >> 5] = q;
    }
    __syncthreads();
    Soft q = soft_empty();
    if (LOSS) q = soft_all<NT / 32>(sh, sh_parts, C, part);
    if (LOSS && part == 0 && tid == 0)
        write_loss(a, r, q, sh_list, sh_kind, q.s == 0.0f ? 0.0f : logf(q.s));
    if (!GRAD) return;
    T* out = static_cast<T*>(a.dx) + r * a.dx_stride;
    const float lse = LOSS ? 0.0f : a.lse[r];
    if (no_gradient(sh_kind, LOSS ? q.s == 0.0f : lse == neg_inf())) {
        for (int32_t i = p.lo + tid; i < p.hi; i += NT + 32) out[i] = from_f32<T>(0.0f);
        return;
    }
    Sweep w;
    w.scale = a.scale;
    w.base = LOSS ? q.mz : lse;
    w.c = row_coef(a, r);
    w.coef = LOSS ? __fdiv_rn(w.c, q.s) : w.c;
    if (sh_kind == kListNan) w.coef = __int_as_float(0x7fffffff);
#pragma unroll 4
    for (int32_t i = p.lo + tid; i < p.hi; i += NT + 32)
        out[i] = from_f32<T>(sweep_value(to_f32(p.row[i]), w));
    __syncthreads();
    write_teacher<T>(a, t, out, p.lo, p.hi, w, tid, NT + 32);
}

// ------------------------------------------------------------------ launches
template <typename T>
bool same_phase(const DistillArgs& a) {
    const auto phase = [](const void* p) {
        return (reinterpret_cast<uintptr_t>(p) / sizeof(T)) % Chunk<T>::kPhase;
    };
    return phase(a.x) == phase(a.dx) &&
           (a.n == 1 || (a.stride - a.dx_stride) % Chunk<T>::kPhase == 0);
}

// Blocks per row: more than one where rows are few and long.  Loss and gradient of
// 4 rows of 50257 take 5.4 us (one block per row: 7.9), 64 6.9 (8.7), 200 12.8 (two per
// row: 13.7).
int row_blocks(int64_t n, int64_t chunks, int threads) {
    int C = 1;
    while (C < 8 && n * C < 152 && chunks / (2 * C) >= 2 * threads) C *= 2;
    return C;
}

template <typename T, Make M, int NT>
cudaError_t launch(DistillArgs a, cudaStream_t stream) {
    // chunks in flight per thread of the register loads: 64 bytes (2047 x 32000
    // binary32 40 us, 43 with 128 bytes)
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    const int64_t chunks = a.vocab / 8;
    a.cluster = row_blocks(a.n, chunks, NT);
    // a part has at most this many tokens: its chunks and 14 elements
    a.map_bytes = M == Make::kLoss ? 0 : Teacher::bytes_of_map(a.k, 8 * (chunks / a.cluster + 1) + 14);
    const int list = Teacher::entry_bytes(a.k) + a.map_bytes;
    if constexpr (M != Make::kLoss) {
        constexpr int kRing = RowRing<T, NT>::kBytes, kMost = 96 * 1024;
        if (same_phase<T>(a)) {
            if (kRing + list > 46 * 1024) {
                const cudaError_t e = cudaFuncSetAttribute(
                    distill_kernel<T, M, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
                if (e != cudaSuccess) return e;
            }
            return launch_vocab(distill_kernel<T, M, NT>, a.n * a.cluster, NT + 32, kRing + list,
                                a.cluster, a, stream);
        }
    }
    return launch_vocab(distill_plain_kernel<T, M, NT, U>, a.n * a.cluster, NT + 32, list, a.cluster,
                        a, stream);
}

template <typename T, Make M>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
    // Short rows: more and smaller blocks, to hide a row's chain of latencies
    // (list, join, second pass) behind other rows; long rows: fewer rows at a
    // time, whose second pass then finds them in L2.  Rows of bf16, loss with
    // gradient, at 64 / 128 / 256 threads: 8192 of 4000 38 / 45 / 73 us, 8192 of
    // 8000 59 / 66 / 88, 4096 of 16000 60 / 57 / 67, 4096 of 32000 - / 115 / 98.
    const int64_t bytes = a.vocab * static_cast<int64_t>(sizeof(T));
    if (bytes <= 16 * 1024) return launch<T, M, 64>(a, stream);
    return bytes <= 40 * 1024 ? launch<T, M, 128>(a, stream) : launch<T, M, 256>(a, stream);
}

template <typename T>
cudaError_t launch_loss(const DistillArgs& a, cudaStream_t stream) {
    return a.dx ? launch<T, Make::kBoth>(a, stream) : launch<T, Make::kLoss>(a, stream);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
    return a.dtype == ZERO3_F32 ? launch_loss<float>(a, stream) : launch_loss<uint16_t>(a, stream);
}

cudaError_t launch_distill_grad(const DistillArgs& a, cudaStream_t stream) {
    return a.dtype == ZERO3_F32 ? launch<float, Make::kGrad>(a, stream)
                                : launch<uint16_t, Make::kGrad>(a, stream);
}

}  // namespace z3
