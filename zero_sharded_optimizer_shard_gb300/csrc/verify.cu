// Verification of drafted tokens and the draw of the token after them (sm_103a).
//
// Position j of a sequence has the target's row p_j = softmax(a x_j) and the
// draft's q_j.  In order, token d_j is accepted iff u_j q_j(d_j) < p_j(d_j); after
// the first refusal the next token is the argmax over i of max(p(i) - q(i), 0) / e_i,
// after a whole draft of p(i) / e_i (an exponential race: a draw from
// the normalised residual).
//
// Rows behind the first refusal are not needed, so a sequence's blocks (a cluster of
// 1 to 8, as many as are resident) take its positions in rounds of `ahead` and stop
// there; in a round each warp has a share of one row.  The race reads the target's
// row again, mostly from L2, and the noise; of the draft's row only what may win.
//
// What bounds it: one sequence, a chain of latencies (12.3 us: a round's loads and its
// exchange, the verdicts, the race and its exchange).  Many, the sequences that run
// longest: 512 of five tokens (50257 bf16) move 550 MB in 126 us, 6.8 TB/s in
// the first round and less as sequences end (floor: the rows up to the refusal and
// the noise once, 443 MB, 65 us).  256 threads with 64 registers, four blocks per SM, at
// which the instances with a draft spill 148 to 188 bytes and those without 8 to 12; five or
// six blocks, with more of them, 512 threads, rows or noise through shared memory, the
// race in a launch of its own: equal or slower.  Without a draft (k = 0) a kernel of its
// own takes statistics and race in one pass.
//
// Weights are 2^((x - m) c), m the row's largest logit and c = a log2(e): of the
// difference of two logits, not of the difference of two products, whose rounding is
// many units where a x is large (finite masks, draws that are nearly greedy).
//
// Decisions.  Weights are binary32, with errors that are bounded as they are
// formed.  A test or a race closer than its bound is taken again by the same
// blocks with weights of 31 bits, row sums in 64-bit integers and scores in
// binary64 (about 1e-9 relative): the answer does not hang on binary32 rounding.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "race_cut.h"
#include "vocab_common.cuh"

namespace z3 {
namespace {

__device__ __forceinline__ float pos_inf() { return __int_as_float(0x7f800000); }

// 16 bytes to the shared variable at `p` of block `rank` of the cluster.
__device__ __forceinline__ void send16(uint4* p, uint32_t rank, const uint4& v) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_address(p, rank)),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

constexpr int kNT = 256, kWarps = kNT / 32;

// A launch's arguments; S: LogitScale, or FarScale.
template <typename S>
struct Args : VerifyArgs {
    S x_unit, y_unit;
};

// What decides about a drafted token.
enum Verdict : int { kAccept = 0, kRefuse = 1, kClose = 2, kBroken = 3, kEnd = 4 };

struct Position {
    float pm, ps, qm, qs;  // the two rows' m (0 without a token) and s (RowSum)
    float xd, yd;    // the drafted token's logits
    float u;
    int32_t token;
    int32_t verdict;
};

// The 4-byte word of global memory that holds element d of a row of V, on its way to
// shared memory, and the element from there.
__device__ __forceinline__ void copy_word(uint32_t* to, uintptr_t at) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(at)
                 : "memory");
}
__device__ __forceinline__ void send_word(uint32_t* to, const float* row, int32_t d, int32_t) {
    copy_word(to, reinterpret_cast<uintptr_t>(row + d));
}
__device__ __forceinline__ void send_word(uint32_t* to, const uint16_t* row, int32_t d, int32_t V) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + d);
    const bool upper = (at & 2) != 0;
    if (word_in_row(upper, d, V))
        copy_word(to, at & ~static_cast<uintptr_t>(3));
    else  // a row's first or last element: its other half may be no one's
        *to = static_cast<uint32_t>(row[d]) << (upper ? 16 : 0);
}
__device__ __forceinline__ float from_word(uint32_t w, const float*) { return __uint_as_float(w); }
__device__ __forceinline__ float from_word(uint32_t w, const uint16_t* p) {
    return reinterpret_cast<uintptr_t>(p) & 2 ? bf16_hi(w) : bf16_lo(w);
}
// Brings the line at p to L2.
__device__ __forceinline__ void prefetch_line(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

constexpr int kMaxPositions = kWarps;  // per round: a warp each

// Differences of logits.  h is 1 (LogitScale) but for inverse temperatures next to the ends
// of binary32 (FarScale), whose instances are compiled apart: products with h cost 1 to 4%
// of a call.
__device__ __forceinline__ float in_unit(const LogitScale&, float x) { return x; }
__device__ __forceinline__ float in_unit(const FarScale& u, float x) { return __fmul_rn(x, u.h); }
// x h - m
__device__ __forceinline__ float less(const LogitScale&, float x, float m) { return __fsub_rn(x, m); }
__device__ __forceinline__ float less(const FarScale& u, float x, float m) { return fmaf(x, u.h, -m); }
__device__ __forceinline__ uint64_t less2(const LogitScale&, uint64_t x, float m) {
    return add2(x, pk2(-m, -m));
}
__device__ __forceinline__ uint64_t less2(const FarScale& u, uint64_t x, float m) {
    return fma2(x, pk2(u.h, u.h), pk2(-m, -m));
}
// Its product with the inverse temperature.
template <typename S>
__device__ __forceinline__ float scaled(const S& u, float x, float m) {
    return __fmul_rn(less(u, x, m), u.z);
}

// Sum of weights 2^((x h - m) c) of the logits that a thread has seen, m the largest
// x h of them (the lowest finite number before any: no difference of two infinities is
// taken).  A NaN is passed over by m and turns s into NaN, as an infinite m does.
struct RowSum {
    float m, s;
};
__device__ __forceinline__ uint4 pack(const RowSum& q) {
    return make_uint4(__float_as_uint(q.m), __float_as_uint(q.s), 0u, 0u);
}
__device__ __forceinline__ RowSum unpack(const uint4& v) {
    return RowSum{__uint_as_float(v.x), __uint_as_float(v.y)};
}
__device__ __forceinline__ float lowest() { return __int_as_float(0xff7fffff); }

template <typename T, int U, typename S>
__device__ __forceinline__ void row_add(RowSum& q, const Chunk<T> (&c)[U], const S& u) {
    float bm = c[0].max();
#pragma unroll
    for (int i = 1; i < U; ++i) bm = fmaxf(bm, c[i].max());
    bm = in_unit(u, bm);
    if (bm > q.m) {  // (before any token: 0 times 0; another branch around it costs 2%)
        q.s = __fmul_rn(q.s, exp2_approx(__fmul_rn(__fsub_rn(q.m, bm), u.c)));
        q.m = bm;
    }
    const uint64_t cc = pk2(u.c, u.c);
    uint64_t s0 = 0, s1 = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float t0, t1;
            upk2(mul2(less2(u, c[i].pair(k), q.m), cc), t0, t1);
            const uint64_t e = pk2(exp2_approx(t0), exp2_approx(t1));
            if (k & 1)
                s1 = add2(s1, e);
            else
                s0 = add2(s0, e);
        }
    }
    float x, y;
    upk2(add2(s0, s1), x, y);
    q.s = __fadd_rn(q.s, __fadd_rn(x, y));
}

// Joins the sums of `WIDTH` lanes (a power of two); every lane gets the result, in a
// fixed order.
template <int WIDTH>
__device__ __forceinline__ void row_lanes(RowSum& q, float c) {
    float top = q.m;
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    q.s = __fmul_rn(q.s, exp2_approx(__fmul_rn(__fsub_rn(q.m, top), c)));
    q.m = top;
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) q.s = __fadd_rn(q.s, __shfl_xor_sync(0xffffffffu, q.s, o));
}

// A whole row's: a largest logit whose product with the inverse temperature overflows
// counts as infinite, which leaves a NaN above and no token below.
__device__ __forceinline__ RowSum whole_row(RowSum q, float z) {
    const float top = __fmul_rn(q.m, z);
    if (top == pos_inf()) q.s = __int_as_float(0x7fffffff);
    if (top == neg_inf() && q.s == q.s) q.s = 0.0f;
    return q;
}

// Thread `tid`'s share, of `nt` threads in each of C blocks, of a row.
template <typename T, typename S>
__device__ __forceinline__ void stream_row(RowSum& q, const T* row, int32_t V, int rank, int C,
                                           const S& u, int tid, int nt) {
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    const RowCut<T> cut(row, V);
    const int32_t per = (cut.chunks + C - 1) / C;
    const int32_t c0 = rank * per;
    const int32_t c1 = c0 + per < cut.chunks ? c0 + per : cut.chunks;
    const bool head = tid == 0 && rank == 0 && cut.head;
    const bool tail = tid == nt - 1 && rank == C - 1 && cut.tail;
    const T* p = row + cut.head;
    int32_t i = c0 + tid;
    if (i + (U - 1) * nt < c1) {  // the next batch is on its way while one is added
        Chunk<T> c[U];
#pragma unroll
        for (int k = 0; k < U; ++k) c[k].load(p + 8 * static_cast<int64_t>(i + k * nt));
        for (i += U * nt; i + (U - 1) * nt < c1; i += U * nt) {
            Chunk<T> d[U];
#pragma unroll
            for (int k = 0; k < U; ++k) d[k].load(p + 8 * static_cast<int64_t>(i + k * nt));
            row_add<T, U>(q, c, u);
#pragma unroll
            for (int k = 0; k < U; ++k) c[k] = d[k];
        }
        row_add<T, U>(q, c, u);
    }
    for (; i < c1; i += nt) {
        Chunk<T> c[1];
        c[0].load(p + 8 * static_cast<int64_t>(i));
        row_add<T, 1>(q, c, u);
    }
    if (head || tail) {
        const T* f = head ? row : p + 8 * static_cast<int64_t>(cut.chunks);
        const int n = head ? cut.head : cut.tail;
        Chunk<T> c[1];
        c[0].fill(neg_inf());
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) c[0].set(e, f[e]);
        row_add<T, 1>(q, c, u);
    }
}

// Element k of a chunk.
template <typename T>
__device__ __forceinline__ float chunk_element(const Chunk<T>& c, int k) {
    float lo, hi;
    upk2(c.pair(k >> 1), lo, hi);
    return k & 1 ? hi : lo;
}
// ------------------------------------------------- 31-bit weights, exact sums
// 2^(n + f), |f| <= 0.5002, as y / 2^31 * 2^n with 0.70 < y / 2^31 < 1.42, from the Taylor
// series of 2^f = e^(f ln 2), terms (f ln 2)^k / k!, k <= 9 (the next is below 8e-12),
// in fixed point.
// Below 2^kLeast31 there is none: y * 2^(n - 31) stays a normal binary64 number (2^-1022).
constexpr int kLeast31 = -960, kNoWeight31 = -2000;
struct Weight {
    uint32_t y;
    int32_t n;  // kNoWeight31: no weight
};

template <typename T, typename S>
__device__ __forceinline__ Weight weight31(T x, const S& u, float m) {
    const float z = in_unit(u, to_f32(x));
    // z - m as a sum of two numbers: the difference with its rounding error
    const float d = __fsub_rn(z, m);
    const float bb = __fsub_rn(d, z);
    const float dl = __fadd_rn(__fsub_rn(z, __fsub_rn(d, bb)), -__fadd_rn(m, bb));
    // times c + cl (the second part is 2^-23 of the first at most, and -960 < t here:
    // below 2^-12)
    const float t = __fmul_rn(d, u.c);
    const float tl = fmaf(d, u.c, -t) + fmaf(d, u.cl, __fmul_rn(dl, u.c));
    Weight w;
    if (!(t > static_cast<float>(kLeast31))) {  // masked tokens too
        w.y = 0;
        w.n = kNoWeight31;
        return w;
    }
    const float r = rintf(t);
    const int32_t h = __float2int_rn((t - r) * 2147483648.0f) + __float2int_rn(tl * 2147483648.0f);
    // f = h / 2^31; a high product brings f / 2, so the coefficients are those of
    // powers of f / 2, in 2^-30: (2 ln 2)^k / k!
    constexpr int32_t c[10] = {0, 1488522236, 1031764991, 476776663, 165238200, 45813757, 10585225, 2096320, 363265, 55955};
    int32_t a = c[9];
#pragma unroll
    for (int k = 8; k >= 1; --k) a = c[k] + __mulhi(a, h);
    w.y = 0x80000000u + static_cast<uint32_t>((static_cast<int64_t>(a) * h) >> 31);
    w.n = static_cast<int32_t>(r);
    return w;
}

__device__ __forceinline__ double weight64(const Weight& w) {
    if (w.n == kNoWeight31) return 0.0;
    return static_cast<double>(w.y) * __hiloint2double((1023 + w.n - 31) << 20, 0);
}

// Bits behind the point of a row's integer sum: V weights below 4 fit 64 bits.
__device__ __forceinline__ int sum_bits(int32_t V) { return 61 - (32 - __clz(V)); }

// Sums of the target's and the draft's rows, in every thread of the cluster.
struct Sums {
    double p, q;
};
// ------------------------------------------------------------------ the race
// Scores with bounds: the best lower bound, the two best upper bounds and the
// token of the best one.
struct Race {
    float low, up, second;
    int32_t token;
};
__device__ __forceinline__ void race_add(Race& r, float low, float up, int32_t token) {
    r.low = fmaxf(r.low, low);
    r.second = fmaxf(r.second, fminf(r.up, up));
    if (up > r.up) {
        r.up = up;
        r.token = token;
    }
}
__device__ __forceinline__ void race_join(Race& r, const Race& o) {
    r.low = fmaxf(r.low, o.low);
    r.second = fmaxf(fmaxf(r.second, o.second), fminf(r.up, o.up));
    if (o.up > r.up) {
        r.up = o.up;
        r.token = o.token;
    }
}
// Joins a warp's (the numbers are not negative: their bits are in their order).
__device__ __forceinline__ Race race_lanes(const Race& r) {
    const uint32_t up = __float_as_uint(r.up);
    const uint32_t most = __reduce_max_sync(0xffffffffu, up);
    const int who = __ffs(__ballot_sync(0xffffffffu, up == most)) - 1;
    const bool me = static_cast<int>(threadIdx.x & 31) == who;
    Race o;
    o.low = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r.low)));
    o.second = __uint_as_float(__reduce_max_sync(0xffffffffu, me ? __float_as_uint(r.second) : up));
    o.up = __uint_as_float(most);
    o.token = __shfl_sync(0xffffffffu, r.token, who);
    return o;
}

// A weight 2^t, t = (x h - m) c, and its relative error: the unit's two ulp, and three
// roundings of t (of the difference, of c and of the product: 3 ln2 2^-24 = 1.04 * 2^-23 of
// |t|).  Without weight below 2^-126.
template <typename T, typename S>
__device__ __forceinline__ float weight(T x, const S& u, float m, float& rel) {
    const float t = __fmul_rn(less(u, to_f32(x), m), u.c);
    rel = fmaf(fabsf(fmaxf(t, -128.0f)), 0x1.2p-23f, 0x1p-21f);
    return exp2_approx(t);
}

// 1 / e of the hardware's unit (1 ulp; infinite for subnormal e, 0 above 2^126).
__device__ __forceinline__ float reciprocal(float e) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e));
    return r;
}
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % Chunk<T>::kPhase);
}

// What one pass needs to know of its two rows.
template <typename TX, typename TY>
struct Rows {
    const TX* x;
    const TY* y;       // the draft's row, or null
    const float* e;
    float pm, qm;      // m
    float ratio;       // sum of the target's weights over the draft's
    float ratio_error; // relative
    int32_t without;   // this token is not drawn (a refused token without probabilities)
};

// How the exact race, which is not inlined, takes them: by value, without a place in memory
// (512 sequences of ten tokens without probabilities: 96 -> 93 us), but by reference beside a
// draft, where the kernel around the call then comes out worse (512 of five: 126 -> 139).
template <typename TX, typename TY, bool DRAFT>
using RowsOf = std::conditional_t<DRAFT, const Rows<TX, TY>&, Rows<TX, TY>>;

// Below this scores decide nothing: they, and their bounds, are next to the subnormal
// numbers, and 1 / e of huge noise is 0.
constexpr float kLeastScore = 0x1p-100f;

// Score of token i: (wp - ratio wq) / e, and how far it may be off.
template <typename TX, typename TY, typename S>
__device__ __forceinline__ void score(const Args<S>& a, const Rows<TX, TY>& r, TX x, TY y, float e,
                                      int32_t i, float& s, float& off) {
    float rel;
    const float wp = weight(x, a.x_unit, r.pm, rel);
    float v = wp;
    off = wp * rel;
    if (r.y) {
        const float wq = weight(y, a.y_unit, r.qm, rel) * r.ratio;
        v = wp - wq;
        off = fmaf(wq, rel + r.ratio_error, off);
    }
    const float inv = reciprocal(e);
    // rounding of the difference, of 1 / e and of the product
    off = fmaf(fabsf(v), 0x1p-21f, off) * inv;
    s = v * inv;
    if (!(e > 0.0f)) {  // nothing is drawn at e < 0 or NaN; 0 wins, and is decided in 64 bits
        s = 0.0f;
        off = e == 0.0f && wp > 0.0f ? pos_inf() : 0.0f;
    } else if (inv == pos_inf()) {
        s = 0.0f;
        off = wp > 0.0f ? pos_inf() : 0.0f;
    }
    if (i == r.without) s = off = 0.0f;
}

// How the race passes over tokens.  No score exceeds wp / e, whose logarithm has a
// bound without a special function: log2(1 / e) is at most what the bits of e say
// (a line between powers of two lies below log2, by 0.086 at most), and t with 14
// bits behind the point is the integer part of one multiply-add on 2^23.  In
// 2^-23:  bound = 512 T - bits(e) + bits(1).  Below the normal numbers (and at 0) the bits of e
// say too much; such noise is never passed over, as no low above 2^26 is asked for (T is at
// least -100, and log2(1 / e) over 126 there).
struct Sieve {
    float a, c;
    int32_t margin;
    static constexpr float kFloor = 8388608.0f + 27.0f * 16384.0f;  // t = -100, masked tokens too
    template <typename S>
    __device__ __forceinline__ Sieve(const S& u, float m) {
        const float unit = u.c * 16384.0f;
        a = in_unit(u, unit);
        c = fmaf(-m, unit, 8388608.0f + 127.0f * 16384.0f);
        // T is off by half a unit, by the rounding of u.c in at most 100 and by that of c;
        // where they overflow nothing is passed over
        const float off = 0x1p-13f + (fabsf(m * u.c) + 150.0f) * 0x1p-21f;
        margin = off < 64.0f && a < 0x1p100f ? static_cast<int32_t>(off * 8388608.0f) : 0x7fffffff;
    }
    // bits(e) - 512 T - bits(1): the bound with its sign turned.  Negative e are
    // never drawn and may come out anyhow.
    __device__ __forceinline__ int32_t of(float x, float e) const {
        const float f = fmaxf(fmaf(x, a, c), kFloor);
        return __float_as_int(e) - (__float_as_int(f) << 9);
    }
    // What is above this cannot reach a score of `low`.
    __device__ __forceinline__ int32_t limit(uint32_t low) const {
        const int32_t most = 0x4c800000;  // 2^26
        const int32_t l = static_cast<int32_t>(low) < most ? static_cast<int32_t>(low) : most;
        return low == 0u || margin == 0x7fffffff ? 0x7fffffff : 0x3f800000 - l + margin;
    }
};

// 8 elements of noise from an address whose place on 16 bytes is `ph`, by the aligned
// blocks that hold them (which lie in the row: race_cut).
struct Noise8 {
    float4 a, b, c;
    __device__ __forceinline__ void load(const float* p, int ph) {
        const float4* q = reinterpret_cast<const float4*>(p - ph);
        a = __ldg(q);
        b = __ldg(q + 1);
        c = b;
        if (ph) c = __ldg(q + 2);
    }
    template <int PH>
    __device__ __forceinline__ float get(int k) const {
        const float f[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
        return f[k + PH];
    }
};
template <typename T, int PH>
__device__ __forceinline__ int32_t sieve_chunk(const Sieve& sieve, const Chunk<T>& x, const Noise8& e) {
    int32_t least = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < 8; ++k) least = min(least, sieve.of(chunk_element(x, k), e.get<PH>(k)));
    return least;
}

struct Shared {
    uint4 parts[2][kWarps][kMaxCluster];  // 16 bytes of each warp of all blocks, by turns
    Position pos[kMaxPositions];
    uint32_t words[kMaxPositions][4];  // words that hold a position's two logits, and its uniform number
    int32_t ids[ZERO3_MAX_DRAFT];
    float z[ZERO3_MAX_DRAFT], sum[ZERO3_MAX_DRAFT];  // an accepted token's (x - m) a, its row's s
    uint32_t low[2];   // bits of the race's best lower bound, first and second pass
};

// All of a cluster's warps send 16 bytes to all of its blocks; `turn` numbers the
// exchanges.  Whoever has come back from exchange t has read what exchange t - 1
// brought, so two sets of places are enough.
__device__ __forceinline__ void exchange(Shared& sh, int turn, int C, uint32_t rank, const uint4& v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (C == 1) {
        if (lane == 0) sh.parts[turn & 1][warp][0] = v;
        __syncthreads();
    } else {
        if (lane < C) send16(&sh.parts[turn & 1][warp][rank], lane, v);
        cluster_sync();
    }
}

// Joins what the warps `row`, `row` + R, ... of all blocks have sent, each half of
// the calling warp for a row of its own; every lane of the half gets the result.
__device__ __forceinline__ RowSum join_rows(const Shared& sh, int turn, int row, int R, int C, float c) {
    const int n = (kWarps - row + R - 1) / R * C;
    const int lg = 31 - __clz(C);
    const auto part = [&](int i) { return unpack(sh.parts[turn & 1][row + (i >> lg) * R][i & (C - 1)]); };
    const int i0 = threadIdx.x & 15;
    RowSum p{lowest(), 0.0f};
    if (i0 < n) p = part(i0);
    float top = p.m;
    for (int i = i0 + 16; i < n; i += 16) top = fmaxf(top, part(i).m);
    __syncwarp();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    RowSum q{top, __fmul_rn(p.s, exp2_approx(__fmul_rn(__fsub_rn(p.m, top), c)))};
    for (int i = i0 + 16; i < n; i += 16) {
        p = part(i);
        q.s = __fadd_rn(q.s, __fmul_rn(p.s, exp2_approx(__fmul_rn(__fsub_rn(p.m, top), c))));
    }
    __syncwarp();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) q.s = __fadd_rn(q.s, __shfl_xor_sync(0xffffffffu, q.s, o));
    return q;
}

// This thread's share of the integer sum of a row's weights.
template <typename T, typename S>
__device__ __forceinline__ uint64_t exact_share(const T* row, int32_t V, const S& scale, float m,
                                                int rank, int C, int bits) {
    uint64_t s = 0;
    const int step = C * kNT;
    // four at a time, the next four on their way (few registers: what this holds, the
    // kernel around the call cannot)
    float x[4];
    const auto load = [&](int32_t i) {
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = i < V - u * step ? to_f32(row[i + u * step]) : neg_inf();
    };
    int32_t i = rank * kNT + static_cast<int>(threadIdx.x);
    load(i);
    while (i < V) {
        float now[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) now[u] = x[u];
        i = i < V - 4 * step ? i + 4 * step : V;
        load(i);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const Weight w = weight31(now[u], scale, m);
            const int shift = bits - 31 + w.n;  // y * 2^shift
            if (shift >= 0)
                s += static_cast<uint64_t>(w.y) << (shift < 32 ? shift : 32);
            else if (shift > -34)  // rounded: the errors of many small weights cancel
                s += (w.y + (uint64_t{1} << (-shift - 1))) >> -shift;
        }
    }
    return s;
}

template <typename TX, typename TY, typename S>
__device__ __noinline__ Sums exact_sums(Shared& sh, int turn, const Args<S>& a, const TX* xr, const TY* yr,
                                        float pm, float qm, int rank) {
    const int32_t V = a.vocab;
    const int C = a.cluster, bits = sum_bits(V);
    uint64_t s = exact_share(xr, V, a.x_unit, pm, rank, C, bits);
    uint64_t t = yr ? exact_share(yr, V, a.y_unit, qm, rank, C, bits) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    exchange(sh, turn, C, rank,
             make_uint4(static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), static_cast<uint32_t>(t),
                        static_cast<uint32_t>(t >> 32)));
    s = t = 0;
    for (int w = 0; w < kWarps; ++w)
        for (int c = 0; c < C; ++c) {
            const uint4 v = sh.parts[turn & 1][w][c];
            s += v.x | static_cast<uint64_t>(v.y) << 32;
            t += v.z | static_cast<uint64_t>(v.w) << 32;
        }
    const double unit = __hiloint2double((1023 - bits) << 20, 0);
    return Sums{static_cast<double>(s) * unit, static_cast<double>(t) * unit};
}

// One pass over the rows.  Only tokens that the sieve lets through are scored, and
// only for them the draft's row is read.  (The best lower bound of the block, by
// which it sieves, depends on the warps' timing; the winner does not: what is
// passed over lies below a lower bound of another token's score.)
template <typename TX, typename TY, typename S>
__device__ __forceinline__ Race race_pass(Shared& sh, int turn, const Args<S>& a, const Rows<TX, TY>& r,
                                          int rank, volatile uint32_t* shared_low) {
    const int32_t V = a.vocab;
    const int C = a.cluster;
    Race b{0.0f, 0.0f, 0.0f, -1};
    const RowCut<TX> row(r.x, V);
    const int ep = phase_of(r.e + row.head);
    const RaceCut cut = race_cut(row.head, row.chunks, ep, V);
    const int step = C * kNT, lane = threadIdx.x & 31;
    const TX* xs = r.x + cut.head;
    const float* es = r.e + cut.head;
    const Sieve sieve(a.x_unit, r.pm);
    const auto look = [&](TX x, float e, int32_t i) {
        float s, off;
        score(a, r, x, r.y ? r.y[i] : TY(0), e, i, s, off);
        race_add(b, s - off, s + off, i);
    };
    // a warp takes 32 chunks at a time, and loads the next ones meanwhile
    Chunk<TX> nx;
    Noise8 ne;
    int c = rank * kNT + static_cast<int>(threadIdx.x);
    if (c < cut.chunks) {
        nx.load(xs + 8 * c);
        ne.load(es + 8 * c, ep);
    }
    for (; c - lane < cut.chunks; c += step) {
        const Chunk<TX> x = nx;
        const Noise8 e = ne;
        if (c + step < cut.chunks) {
            nx.load(xs + 8 * (c + step));
            ne.load(es + 8 * (c + step), ep);
        }
        const uint32_t low = *shared_low;
        int32_t least = 0x7fffffff;
        switch (ep) {
            case 0: least = sieve_chunk<TX, 0>(sieve, x, e); break;
            case 1: least = sieve_chunk<TX, 1>(sieve, x, e); break;
            case 2: least = sieve_chunk<TX, 2>(sieve, x, e); break;
            default: least = sieve_chunk<TX, 3>(sieve, x, e); break;
        }
        unsigned let = __ballot_sync(0xffffffffu, c < cut.chunks && least <= sieve.limit(low));
        if (let == 0) continue;
        if (__popc(let) > 4) {  // the first chunks, mostly: all of them whole
            if (let >> lane & 1) {
                const int32_t i = cut.head + 8 * c;
#pragma unroll 4
                for (int k = 0; k < 8; ++k) look(r.x[i + k], r.e[i + k], i + k);
            }
        } else {  // eight lanes for each chunk
            int from = 0;
            bool any = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k == lane >> 3 && let) {
                    from = __ffs(let) - 1;
                    any = true;
                }
                let &= let - 1;
            }
            const int32_t i = __shfl_sync(0xffffffffu, cut.head + 8 * c, from) + (lane & 7);
            if (any) look(r.x[i], r.e[i], i);
        }
        __syncwarp();
        const uint32_t found = __reduce_max_sync(0xffffffffu, __float_as_uint(b.low));
        if (lane == 0 && found > low) atomicMax(const_cast<uint32_t*>(shared_low), found);
    }
    // the ends of the row
    if (rank == 0 && threadIdx.x < 32) {
        const int32_t i = end_token(lane, cut.head, cut.head + 8 * cut.chunks, V);
        if (i >= 0) look(r.x[i], r.e[i], i);
    }
    __syncwarp();
    b = race_lanes(b);
    exchange(sh, turn, C, rank,
             make_uint4(__float_as_uint(b.low), __float_as_uint(b.up), __float_as_uint(b.second),
                        static_cast<uint32_t>(b.token)));
    Race best{0.0f, 0.0f, 0.0f, -1};
    for (int j = threadIdx.x & 31; j < kWarps * C; j += 32) {
        const uint4 v = sh.parts[turn & 1][j / C][j % C];
        race_join(best, Race{__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                             static_cast<int32_t>(v.w)});
    }
    return race_lanes(best);
}

// The race among the tokens whose upper bound reaches `low`, with 31-bit weights
// and scores in binary64; ties to the lowest token, -1 if no score is positive.
template <typename TX, typename TY, bool DRAFT, typename S>
__device__ __noinline__ int32_t exact_race(Shared& sh, int turn, const Args<S>& a, RowsOf<TX, TY, DRAFT> r,
                                           const Sums sums, float low, int rank) {
    const int32_t V = a.vocab;
    const int C = a.cluster;
    double best = 0.0;
    int32_t token = 0x7fffffff;
    // several at a time through the sieve of the bound that the race has found; one
    // without a draft, where a close race is one in 10^5 and registers count
    constexpr int U = DRAFT ? 4 : 1;
    const Sieve sieve(a.x_unit, r.pm);
    const int32_t limit = sieve.limit(__float_as_uint(low));
    const int step = C * kNT;
    for (int32_t i0 = rank * kNT + static_cast<int>(threadIdx.x); i0 < V;
         i0 = i0 < V - U * step ? i0 + U * step : V) {
        unsigned let = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 < V - u * step && sieve.of(to_f32(r.x[i0 + u * step]), r.e[i0 + u * step]) <= limit)
                let |= 1u << u;
        for (; let; let &= let - 1) {
            const int32_t i = i0 + (__ffs(let) - 1) * step;
            const TX x = r.x[i];
            const TY y = r.y ? r.y[i] : TY(0);
            const float e = r.e[i];
            float s, off, rel;
            score(a, r, x, y, e, i, s, off);
            // a token below the range of binary32 weights is not drawn, even alone
            if (!(s + off >= low) || !(e >= 0.0f) || __float_as_int(e) < 0 || i == r.without ||
                weight(x, a.x_unit, r.pm, rel) == 0.0f)
                continue;
            double v = weight64(weight31(x, a.x_unit, r.pm));
            if (r.y) v = v / sums.p - weight64(weight31(y, a.y_unit, r.qm)) / sums.q;
            v = v / static_cast<double>(e);
            if (v > best) {  // tokens come in ascending order
                best = v;
                token = i;
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double v = __shfl_xor_sync(0xffffffffu, best, o);
        const int32_t t = __shfl_xor_sync(0xffffffffu, token, o);
        if (v > best || (v == best && t < token)) {
            best = v;
            token = t;
        }
    }
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(best));
    exchange(sh, turn, C, rank,
             make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32),
                        static_cast<uint32_t>(token), 0u));
    best = 0.0;
    token = 0x7fffffff;
    for (int w = 0; w < kWarps; ++w)
        for (int c = 0; c < C; ++c) {
            const uint4 v = sh.parts[turn & 1][w][c];
            const double d = __longlong_as_double(static_cast<int64_t>(v.x | static_cast<uint64_t>(v.y) << 32));
            const int32_t t = static_cast<int32_t>(v.z);
            if (d > best || (d == best && t < token)) {
                best = d;
                token = t;
            }
        }
    return best > 0.0 ? token : -1;
}

// ---------------------------------------------------------------- the kernel
// Exact decision about a close position.
template <typename TX, typename TY, bool DRAFT, typename S>
__device__ __noinline__ int decide(Shared& sh, int turn, const Args<S>& a, const Position& o, const TX* xr,
                                   const TY* yr, int rank) {
    const Sums m = exact_sums<TX, TY>(sh, turn, a, xr, yr, o.pm, o.qm, rank);
    const double wp = weight64(weight31(xr[o.token], a.x_unit, o.pm));
    double wq = 1.0, sq = 1.0;
    if (DRAFT) {
        wq = weight64(weight31(yr[o.token], a.y_unit, o.qm));
        sq = m.q;
    }
    bool less = static_cast<double>(o.u) * wq * m.p < wp * sq;
    if (wp == 0.0 || wq == 0.0) {  // too far below: by their logarithms
        const S &u = a.x_unit, &w = a.y_unit;
        const double xd = in_unit(u, o.xd), yd = in_unit(w, o.yd);
        const double lp = (xd - o.pm) * u.z - log(m.p);
        const double lq = DRAFT ? (yd - o.qm) * w.z - log(m.q) : 0.0;
        less = log(static_cast<double>(o.u)) + lq < lp;
    }
    return less ? kAccept : kRefuse;
}

// Position j, number g of the round, from the rows' sums (one warp).
template <typename TX, typename TY, bool DRAFT, typename S>
__device__ __forceinline__ void weigh(Shared& sh, int turn, const Args<S>& a, int R, int g, int j, bool drafted,
                                      const TX* xr, const TY* yr) {
    const int lane = threadIdx.x & 31;
    const int row = (DRAFT ? 2 * g : g) + (DRAFT && lane >= 16 && drafted);
    const bool of_draft = DRAFT && lane >= 16;
    const RowSum h = whole_row(join_rows(sh, turn, row, R, a.cluster, of_draft ? a.y_unit.c : a.x_unit.c),
                               of_draft ? a.y_unit.z : a.x_unit.z);
    Position o;
    o.pm = __shfl_sync(0xffffffffu, h.m, 0);
    o.ps = __shfl_sync(0xffffffffu, h.s, 0);
    o.qm = __shfl_sync(0xffffffffu, h.m, 16);
    o.qs = __shfl_sync(0xffffffffu, h.s, 16);
    o.verdict = o.ps != o.ps ? kBroken : kEnd;
    o.xd = o.yd = o.u = 0.0f;
    o.token = -1;
    if (drafted) {
        o.token = sh.ids[j];
        o.xd = from_word(sh.words[g][0], xr + o.token);
        o.u = __uint_as_float(sh.words[g][2]);
        bool q_nan = false, in_q = true;
        float rel, rel_q = 0.0f, wq = 1.0f, sq = 1.0f;
        const float wp = weight(o.xd, a.x_unit, o.pm, rel);
        if (DRAFT) {
            o.yd = from_word(sh.words[g][1], yr + o.token);
            q_nan = o.qs != o.qs;
            in_q = o.qs != 0.0f && __fmul_rn(o.yd, a.y_scale) != neg_inf();
            wq = weight(o.yd, a.y_unit, o.qm, rel_q);
            sq = o.qs;
        }
        if (lane == 0) {
            sh.z[j] = scaled(a.x_unit, o.xd, o.pm);
            sh.sum[j] = o.ps;
        }
        if (o.ps != o.ps || q_nan) {
            o.verdict = kBroken;
        } else if (!(o.u >= 0.0f) || o.ps == 0.0f || __fmul_rn(o.xd, a.scale) == neg_inf()) {
            o.verdict = kRefuse;
        } else if (!in_q || o.u == 0.0f) {
            o.verdict = kAccept;
        } else {
            // u q < p: u wq sp < wp sq, off by the sums' and the weights' errors and
            // a few roundings; what is small for binary32 is close
            const float l = o.u * (wq * o.ps), r = wp * sq;
            const float off = fmaf(2.0f, a.sum_error, rel + rel_q + 0x1p-21f) * (l + r);
            o.verdict = kClose;
            if (l + r > 0x1p-60f) {
                if (r - l > off) o.verdict = kAccept;
                if (l - r > off) o.verdict = kRefuse;
            }
        }
    }
    if (lane == 0) sh.pos[g] = o;
}

// The token after position o: the row of the target, the draft's, the noise.
template <typename TX, typename TY, bool DRAFT, typename S>
__device__ __forceinline__ int32_t draw(Shared& sh, int& turn, const Args<S>& a, const Position& o,
                                        int verdict, const TX* xr, const TY* yr, const float* noise, int rank) {
    Rows<TX, TY> r;
    r.x = xr;
    r.y = nullptr;
    r.e = noise;
    r.pm = o.pm;
    r.qm = o.qm;
    r.ratio = 0.0f;
    r.ratio_error = 0.0f;
    r.without = -1;
    if (verdict == kRefuse) {
        if (!DRAFT) {
            r.without = o.token;
        } else if (o.qs != 0.0f) {
            r.y = yr;
            r.ratio = __fmul_rn(o.ps, reciprocal(o.qs));
            r.ratio_error = 2.0f * a.sum_error + 0x1p-22f;
        }
    }
    int32_t token = -1;
    for (int pass = 0; pass < 2; ++pass) {
        Race b = race_pass<TX, TY>(sh, turn, a, r, rank, &sh.low[pass]);
        ++turn;
        if (b.low < kLeastScore) b.low = 0.0f;
        if (b.low > 0.0f && b.second < b.low) {
            token = b.token;
        } else {
            Sums m{1.0, 1.0};
            if (r.y) {
                m = exact_sums<TX, TY>(sh, turn, a, r.x, r.y, r.pm, r.qm, rank);
                ++turn;
            }
            token = exact_race<TX, TY, DRAFT>(sh, turn, a, r, m, b.low, rank);
            ++turn;
        }
        if (token >= 0 || (!r.y && r.without < 0)) break;
        r.y = nullptr;  // no residual: from the target itself
        r.without = -1;
    }
    return token;
}

template <typename TX, typename TY, bool DRAFT, typename S>
__global__ void __launch_bounds__(kNT, 4) verify_kernel(const __grid_constant__ Args<S> a) {
    __shared__ Shared sh;
    const int C = a.cluster;
    const uint32_t rank = C > 1 ? cluster_rank() : 0u;
    if (C > 1) cluster_arrive();
    const int64_t s = blockIdx.x / C;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int32_t V = a.vocab;
    const int K = a.k;
    const TX* x = static_cast<const TX*>(a.x) + s * (K + 1) * a.stride;
    const TY* y = DRAFT ? static_cast<const TY*>(a.y) + s * K * a.y_stride : nullptr;
    const float* noise = a.noise + s * a.noise_stride;
    int32_t* tokens = a.tokens + s * (K + 1);
    wait_prior_grids();
    allow_next_grid();
    if (tid < 2) sh.low[tid] = 0;  // seen by all after the first barrier
    // The block's part of the noise goes to L2: at once where all sequences' fits
    // there beside the rows, else when it is needed.
    const auto prefetch_noise = [&]() {
        const int per = (V + C - 1) / C;
        const int lo = rank * per, hi = lo + per < V ? lo + per : V;
        for (int i = lo + 32 * tid; i < hi; i += 32 * kNT) prefetch_line(noise + i);
    };
    const bool early = a.n * V <= (int64_t{1} << 22);  // 16 MB
    const int ahead = a.ahead;  // its rows and one more are kWarps at most
    if (early) prefetch_noise();
    int turn = 0, verdict = kAccept;
    // the draft's length: ids up to the first ignored one (every warp by itself)
    int L = K;
    for (int j = lane; j - lane < K; j += 32) {
        const int32_t id = j < K ? load_id(a.ids, a.id64, s * K + j, V) : -1;
        if (warp == 0 && j < K) sh.ids[j] = id;
        const unsigned none = __ballot_sync(0xffffffffu, id < 0 && j < K);
        if (none) {
            L = j - lane + __ffs(none) - 1;
            break;
        }
    }
    __syncwarp();  // warp 0 reads the ids that its lanes have written
    if (C > 1) cluster_wait();     // the others' shared memory is there
    int at = -1, j0 = 0;
    for (;; j0 += ahead) {
        // ---- the round's rows, and what the verdicts need beside them.  The row behind
        // the draft comes along with the last position.
        const int G = ahead < L - j0 ? ahead : L - j0;
        const bool whole = j0 + G == L;
        const int R = (DRAFT ? 2 * G : G) + whole;
        if (warp == 0) {
            if (lane < G) {
                const int j = j0 + lane, d = sh.ids[j];
                send_word(&sh.words[lane][0], x + j * a.stride, d, V);
                if (DRAFT) send_word(&sh.words[lane][1], y + j * a.y_stride, d, V);
                send_word(&sh.words[lane][2], a.uniform + s * K, j, K);
            }
        }
        {
            const int row = warp % R, nt = (kWarps - row + R - 1) / R * 32;
            const int tr = warp / R * 32 + lane;
            const int j = j0 + (DRAFT ? row >> 1 : row);
            RowSum q{lowest(), 0.0f};
            const bool of_draft = DRAFT && (row & 1);
            if (of_draft)
                stream_row<TY>(q, y + j * a.y_stride, V, rank, C, a.y_unit, tr, nt);
            else
                stream_row<TX>(q, x + j * a.stride, V, rank, C, a.x_unit, tr, nt);
            __syncwarp();
            row_lanes<32>(q, of_draft ? a.y_unit.c : a.x_unit.c);
            if (warp == 0) drain_copies();
            exchange(sh, turn, C, rank, pack(q));
        }
        if (warp < G + whole) {
            const int j = j0 + warp;
            weigh<TX, TY, DRAFT>(sh, turn, a, R, warp, j, warp < G, x + j * a.stride,
                                 DRAFT ? y + j * a.y_stride : nullptr);
        }
        ++turn;
        __syncthreads();
        // ---- the first position that does not accept
        for (int g = 0; g < G + whole; ++g) {
            verdict = sh.pos[g].verdict;
            if (verdict == kClose) {
                const int j = j0 + g;
                verdict = decide<TX, TY, DRAFT>(sh, turn, a, sh.pos[g], x + j * a.stride,
                                                DRAFT ? y + j * a.y_stride : nullptr, rank);
                ++turn;
            }
            if (verdict != kAccept) {
                at = g;
                break;
            }
        }
        if (at >= 0) break;
        // (the next round's barrier lies before the positions' next writing)
    }
    const int A = j0 + at;
    const Position& o = sh.pos[at];
    int32_t token = -1;
    float lp = __int_as_float(0x7fffffff);
    if (verdict != kBroken) {
        lp = neg_inf();
        if (o.ps != 0.0f) {
            if (!early) prefetch_noise();
            const TX* xr = x + A * a.stride;
            token = draw<TX, TY, DRAFT>(sh, turn, a, o, verdict, xr, DRAFT ? y + A * a.y_stride : nullptr, noise,
                                        rank);
            if (token >= 0 && rank == 0)
                lp = __fsub_rn(scaled(a.x_unit, to_f32(xr[token]), o.pm), logf(o.ps));
        }
    }
    if (rank == 0) {
        if (tid == 0) a.accepted[s] = A;
        for (int j = tid; j <= K; j += kNT) {
            tokens[j] = j < A ? sh.ids[j] : j == A ? token : -1;
            if (a.logprobs)
                a.logprobs[s * (K + 1) + j] =
                    j < A ? __fsub_rn(sh.z[j], logf(sh.sum[j])) : j == A ? lp : 0.0f;
        }
    }
}

// ------------------------------------------------------------ without a draft
// Sampling (k = 0): the winner does not hang on the row's sum, so statistics and race
// share one pass over row and noise and one exchange.  A warp's weights are relative
// to the largest x h that it has met, and are taken to the row's largest when the warps
// are joined; the sum's weights w sift the race too, as no token with w < low e can reach
// a score of `low`.  A race that is not certain goes to the general kernel's code.
//
// 128 sequences of 32000 masked binary32 logits: 10.1 us (statistics first and the race
// behind them: 16.7), 33 MB, a chain of latencies around four batches per warp; 512 of
// 50257 bf16: 32.1 us (49.7), 154 MB at 4.8 TB/s, bound by the loads in flight: one batch
// ahead is 48 bytes a thread, 41 KB per SM, and 59% of the warps' time is waiting for them
// (150 instructions per 256 elements take 43% of the issue slots; 512 blocks stand on 608
// places).  80 registers and two batches ahead: 45; five blocks per SM (spills): 40; lines
// brought to L2 further ahead: 34 to 36.

// Scores relative to `from` taken to `to`.  Bounds stay bounds: an upper one gets the
// least normal number on top, a lower one is given up where little is left.
__device__ __forceinline__ void race_rebase(Race& r, float from, float to, float c) {
    const float t = fmaxf(__fmul_rn(__fsub_rn(from, to), c), -1024.0f);
    const float f = exp2_approx(0.5f * t), err = fmaf(fabsf(t), 0x1p-22f, 0x1p-20f);
    r.low = t > -30.0f ? r.low * f * f * (1.0f - err) : 0.0f;
    if (r.up > 0.0f && r.up < pos_inf()) r.up = fmaf(r.up * f, f * (1.0f + err), 0x1p-126f);
    if (r.second > 0.0f && r.second < pos_inf()) r.second = fmaf(r.second * f, f * (1.0f + err), 0x1p-126f);
}

// Weights 2^((x h - ref) c) of a chunk and their sum.
template <typename T, typename S>
__device__ __forceinline__ float chunk_weights(const Chunk<T>& x, const S& u, float ref, float (&w)[8]) {
    const uint64_t cc = pk2(u.c, u.c);
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float t0, t1;
        upk2(mul2(less2(u, x.pair(k), ref), cc), t0, t1);
        w[2 * k] = exp2_approx(t0);
        w[2 * k + 1] = exp2_approx(t1);
        s[k & 1] = add2(s[k & 1], pk2(w[2 * k], w[2 * k + 1]));
    }
    float a, b;
    upk2(add2(s[0], s[1]), a, b);
    return __fadd_rn(a, b);
}
// A chunk's noise in its order.
__device__ __forceinline__ void in_order(const Noise8& e, int ph, float (&v)[8]) {
    switch (ph) {
        case 0:
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = e.get<0>(k);
            break;
        case 1:
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = e.get<1>(k);
            break;
        case 2:
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = e.get<2>(k);
            break;
        default:
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = e.get<3>(k);
    }
}

// A token's score w / e, from a weight 2^t.  Relative errors: |t| 1.04 * 2^-23 of t's three
// roundings, the units' two ulp and one, the product's; a lower bound counts if the weight
// is far from the end of the range.  Nothing is drawn at e < 0 or NaN; 0 wins, and is
// decided in 64 bits, as is a subnormal e.
__device__ __forceinline__ void race_token(Race& b, float w, float e, int32_t i) {
    const float inv = reciprocal(e);
    const float v = w * inv;
    const float off = v * (w > 0x1p-16f ? 0x1.8p-19f : 0x1p-15f);
    float low = w >= 0x1p-60f ? v - off : 0.0f, up = v + off;
    if (!(e > 0.0f && inv < pos_inf())) {
        low = 0.0f;
        up = e >= 0.0f && w > 0.0f ? pos_inf() : 0.0f;
    }
    race_add(b, low, up, i);
}

template <typename TX, typename S>
__device__ __noinline__ int32_t draw_again(Shared& sh, const Args<S>& a, float pm, float ps, const TX* xr,
                                           const float* noise, int rank) {
    Position o;
    o.pm = pm;
    o.ps = ps;
    o.qm = o.qs = o.xd = o.yd = o.u = 0.0f;
    o.token = -1;
    int turn = 1;
    return draw<TX, TX, false>(sh, turn, a, o, kEnd, xr, nullptr, noise, rank);
}

template <typename TX, typename S>
__global__ void __launch_bounds__(kNT, 4) sample_kernel(const __grid_constant__ Args<S> a) {
    __shared__ Shared sh;
    __shared__ uint4 more[kWarps][kMaxCluster];
    const int C = a.cluster;
    const uint32_t rank = C > 1 ? cluster_rank() : 0u;
    if (C > 1) cluster_arrive();
    const int64_t s = blockIdx.x / C;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int32_t V = a.vocab;
    const S& u = a.x_unit;
    const TX* x = static_cast<const TX*>(a.x) + s * a.stride;
    const float* noise = a.noise + s * a.noise_stride;
    wait_prior_grids();
    allow_next_grid();
    if (tid < 2) sh.low[tid] = 0;
    const RowCut<TX> row(x, V);
    const int ep = phase_of(noise + row.head);
    const RaceCut cut = race_cut(row.head, row.chunks, ep, V);
    const int step = C * kNT;
    const TX* xs = x + cut.head;
    const float* es = noise + cut.head;
    float sum = 0.0f;
    Race b{0.0f, 0.0f, 0.0f, -1};
    float ref = lowest();  // before any token above that, none of which is in the race
    // `low`: of a score that some token of the warp has; base: the reference of the oldest
    float low = 0.0f, base = lowest();
    // The lanes' largest x h: the warp's weights become relative to it (all lanes).
    const auto meet = [&](float z) {
        if (!__any_sync(0xffffffffu, z > ref)) return;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
        sum = __fmul_rn(sum, exp2_approx(__fmul_rn(__fsub_rn(ref, z), u.c)));
        race_rebase(b, ref, z, u.c);
        if (!((z - base) * u.c < 28.0f)) {
            b.low = 0.0f;
            base = z;
        }
        low = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b.low)));
        ref = z;
    };
    Chunk<TX> nx;
    Noise8 ne;
    int c = rank * kNT + tid;
    const auto load = [&](int32_t at) {
        if (at < cut.chunks) {
            nx.load(xs + 8 * at);
            ne.load(es + 8 * at, ep);
        } else {
            nx.fill(neg_inf());
        }
    };
    ne.a = ne.b = ne.c = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    load(c);
    for (; c - lane < cut.chunks; c += step) {
        const Chunk<TX> xc = nx;
        const Noise8 e = ne;
        load(c + step);
        __syncwarp();
        meet(in_unit(u, xc.max()));
        // (a NaN, which max passes over, goes into the sum)
        float w[8], ev[8];
        sum = __fadd_rn(sum, chunk_weights(xc, u, ref, w));
        in_order(e, ep, ev);
        if (low == 0.0f && ref != lowest()) {  // about what the warp's best token has
            float l = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (ev[k] > 0x1p-100f) l = fmaxf(l, w[k] * reciprocal(ev[k]));
            if (c >= cut.chunks) l = 0.0f;
            low = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(l)));
        }
        // Tokens whose w - low e is not below 0 may reach `low` (less 2^-14, which is more
        // than the weights' errors).  A NaN e is passed over, a negative one may come out.
        const float under = -low * (1.0f - 0x1p-14f);
        float d = fmaf(ev[0], under, w[0]);
#pragma unroll
        for (int k = 1; k < 8; ++k) d = fmaxf(d, fmaf(ev[k], under, w[k]));
        const bool pass = c < cut.chunks && ref != lowest() && d >= 0.0f;
        if (!__any_sync(0xffffffffu, pass)) continue;
        if (pass) {
            const int32_t i0 = cut.head + 8 * c;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (fmaf(ev[k], under, w[k]) >= 0.0f) race_token(b, w[k], ev[k], i0 + k);
        }
        __syncwarp();
        low = fmaxf(low, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b.low))));
    }
    // the ends of the row
    if (rank == 0 && warp == 0) {
        const int32_t i = end_token(lane, cut.head, cut.head + 8 * cut.chunks, V);
        Chunk<TX> xc;
        xc.fill(neg_inf());
        if (i >= 0) xc.set(0, x[i]);
        __syncwarp();
        meet(in_unit(u, xc.max()));
        float w[8];
        sum = __fadd_rn(sum, chunk_weights(xc, u, ref, w));
        if (i >= 0 && ref != lowest()) race_token(b, w[0], noise[i], i);
    }
    RowSum q{ref, sum};
    __syncwarp();
    row_lanes<32>(q, u.c);
    b = race_lanes(b);
    {
        const uint4 v = make_uint4(__float_as_uint(q.m), __float_as_uint(q.s), __float_as_uint(b.low),
                                   __float_as_uint(b.up));
        const uint4 w = make_uint4(__float_as_uint(b.second), static_cast<uint32_t>(b.token), 0u, 0u);
        if (C == 1) {
            if (lane == 0) {
                sh.parts[0][warp][0] = v;
                more[warp][0] = w;
            }
            __syncthreads();
        } else {
            cluster_wait();  // the others' shared memory is there
            if (lane < C) {
                send16(&sh.parts[0][warp][rank], lane, v);
                send16(&more[warp][rank], lane, w);
            }
            cluster_sync();
        }
    }
    // One warp joins all of them: lane i has the parts i and i + 32.
    if (warp == 0) {
        RowSum g{lowest(), 0.0f}, h = g;
        if (lane < kWarps * C) g = unpack(sh.parts[0][lane / C][lane % C]);
        if (lane + 32 < kWarps * C) h = unpack(sh.parts[0][(lane + 32) / C][(lane + 32) % C]);
        float top = fmaxf(g.m, h.m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        h.s = __fadd_rn(__fmul_rn(g.s, exp2_approx(__fmul_rn(__fsub_rn(g.m, top), u.c))),
                        __fmul_rn(h.s, exp2_approx(__fmul_rn(__fsub_rn(h.m, top), u.c))));
        h.m = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) h.s = __fadd_rn(h.s, __shfl_xor_sync(0xffffffffu, h.s, o));
        h = whole_row(h, u.z);
        Race best{0.0f, 0.0f, 0.0f, -1};
        for (int j = lane; j < kWarps * C; j += 32) {
            const uint4 v = sh.parts[0][j / C][j % C], w = more[j / C][j % C];
            Race o{__uint_as_float(v.z), __uint_as_float(v.w), __uint_as_float(w.x), static_cast<int32_t>(w.y)};
            race_rebase(o, __uint_as_float(v.x), h.m, u.c);
            race_join(best, o);
        }
        __syncwarp();
        best = race_lanes(best);
        if (lane == 0) {
            Position& o = sh.pos[0];
            o.pm = h.m;
            o.ps = h.s;
            // whether the answer is there: no sum, or a race that is certain
            o.verdict = !(h.s > 0.0f) || (best.low >= kLeastScore && best.second < best.low) ? kEnd : kClose;
            o.token = h.s > 0.0f ? best.token : -1;
        }
    }
    __syncthreads();
    const Position o = sh.pos[0];
    int32_t token = o.token;
    if (o.verdict == kClose) token = draw_again<TX>(sh, a, o.pm, o.ps, x, noise, rank);
    if (rank == 0 && tid == 0) {
        a.accepted[s] = 0;
        a.tokens[s] = token;
        if (a.logprobs)
            a.logprobs[s] = o.ps != o.ps ? __int_as_float(0x7fffffff)
                            : token < 0  ? neg_inf()
                                         : __fsub_rn(scaled(u, to_f32(x[token]), o.pm), logf(o.ps));
    }
}

template <typename TX, typename TY, typename S>
cudaError_t launch_types(const Args<S>& a, cudaStream_t stream) {
    const int64_t grid = a.n * a.cluster;
    if (a.k == 0) return launch_vocab(sample_kernel<TX, S>, grid, kNT, 0, a.cluster, a, stream);
    return a.y ? launch_vocab(verify_kernel<TX, TY, true, S>, grid, kNT, 0, a.cluster, a, stream)
               : launch_vocab(verify_kernel<TX, TX, false, S>, grid, kNT, 0, a.cluster, a, stream);
}

void set_scale(LogitScale& u, double scale) {
    const double c = scale * 1.4426950408889634;
    u.c = static_cast<float>(c);
    u.cl = static_cast<float>(c - static_cast<double>(u.c));
    u.z = static_cast<float>(scale);
}
bool far(float scale) { return scale > 0x1p100f || scale < 0x1p-100f; }
// h keeps differences of logits, and what they are multiplied by, inside binary32: where
// the inverse temperature is small they may be over 2^128, where it is large c may be.
void set_scale(FarScale& u, double scale) {
    const double h = scale > 0x1p100 ? 0x1p64 : scale < 0x1p-100 ? 0x1p-64 : 1.0;
    set_scale(static_cast<LogitScale&>(u), scale / h);
    u.h = static_cast<float>(h);
}

template <typename S>
cudaError_t launch_scaled(const VerifyArgs& args, cudaStream_t stream) {
    Args<S> a;
    static_cast<VerifyArgs&>(a) = args;
    set_scale(a.x_unit, a.scale);
    set_scale(a.y_unit, a.y_scale);
    if (a.dtype == ZERO3_BF16)
        return a.y_dtype == ZERO3_BF16 ? launch_types<uint16_t, uint16_t>(a, stream)
                                       : launch_types<uint16_t, float>(a, stream);
    return a.y_dtype == ZERO3_BF16 ? launch_types<float, uint16_t>(a, stream) : launch_types<float, float>(a, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& args, cudaStream_t stream) {
    VerifyArgs a = args;
    // As many blocks per sequence as are resident at once (four on each of 152 SMs),
    // and two at least where there are drafts: with one, an SM whose sequences are all
    // accepted far ends last (512 of 50257, ten tokens without probabilities: 130
    // us with one, 104 with two; five with: 123 and 126; no draft: 34 and 38).
    a.cluster = 1;
    while (a.cluster < kMaxCluster && a.n * a.cluster * 2 <= 608) a.cluster *= 2;
    if (a.k > 0 && a.cluster == 1) a.cluster = 2;
    // Positions per round, a row of which a warp has: all of them at once while
    // the chain of rounds is the time (48 sequences of ten: 45 us one by one, 23 by
    // seven), two where rows that turn out not to be needed are (512 of ten: 126 us by
    // seven, 104 by two; 256 of five drafts: 76 by three, 71 by two, 73 one by one).  Next to the
    // places of the rule, 50257 tokens: five drafts, 76 sequences 40.9 by three, 41.8 by two,
    // 100 42.2 and 41.1, 130 46.8 and 44.9; ten tokens, 150 44.0 by seven, 45.0 by two, 200
    // 56.2 and 58.1, 260 65.7 and 61.4.  It looks at the sequences alone, and is late for short
    // rows, of which more in vain would pay (8192 tokens: 180 of five drafts 21.4 by three,
    // 22.8 by two; 350 of ten tokens 26.9 by seven, 30.8 by two).
    a.ahead = a.y ? (a.n <= 100 ? 3 : 2) : (a.n <= 200 ? 7 : 2);
    const int g = a.ahead < a.k ? a.ahead : a.k, rows = (a.y ? 2 * g : g) + 1;
    // Relative error of a row's sum.  Its terms: the unit's two ulp (2^-22), and three
    // roundings of t, 1.04 * 2^-23 |t| on their average |t|, which is at most log2(V).  A thread's
    // chain of additions and the joins: its batches, then at most 32 more.  Changes of the
    // reference, two ulp and a product each: where logits rise, every batch may be one, and the
    // sum before it keeps nearly all of its weight; four chunks and ends, and two joins, on top;
    // the roundings of their differences 2^-21, as a sum with |t| that much lower counts that
    // much less.  (Rows that rise by 0.01 to 3000 were off by a quarter of what the additions
    // alone allow.)
    int bits = 1;
    while (a.vocab >> bits) ++bits;
    const int threads = 32 * a.cluster * (kWarps / rows);  // of a row
    const bool wide = a.dtype == ZERO3_F32 || (a.y && a.y_dtype == ZERO3_F32);
    const int batches = a.vocab / ((wide ? 16 : 32) * threads);
    a.sum_error = 0x1p-22f + 0x1p-21f + 1.2f * 0x1p-23f * static_cast<float>(bits) +
                  static_cast<float>(batches + 32) * 0x1p-24f +
                  static_cast<float>(batches + 6) * (0x1p-22f + 0x1p-24f);
    return far(a.scale) || far(a.y_scale) ? launch_scaled<FarScale>(a, stream) : launch_scaled<LogitScale>(a, stream);
}

}  // namespace z3
