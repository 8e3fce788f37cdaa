// Verification of drafted tokens and the draw of the token after them (sm_103a).
//
// Position j of a sequence has the target's row p_j = softmax(a x_j) and the
// draft's q_j.  In order, token d_j is accepted iff u_j q_j(d_j) < p_j(d_j); after
// the first refusal the next token is the argmax over i of max(p(i) - q(i), 0) / e_i,
// after a whole draft of p(i) / e_i (an exponential race: a draw from
// the normalised residual).
//
// Bound by HBM where there are many sequences: rows behind the first refusal are
// not needed, so a sequence's blocks (a cluster of 1 to 8) take its positions in
// rounds of `ahead` and stop there; the race reads the last round's two rows again
// from L2, and the noise.  With few sequences the chain of latencies bounds it, and
// all positions go in one round.
//
// Decisions.  Weights are binary32, with errors that are bounded as they are
// formed.  A test or a race closer than its bound is taken again by the same
// blocks with weights of 31 bits, row sums in 64-bit integers and scores in
// binary64 (about 1e-9 relative): the answer does not hang on binary32 rounding.
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {
namespace {

constexpr int kNT = 512;
constexpr int kWarps = kNT / 32;

__device__ __forceinline__ float pos_inf() { return __int_as_float(0x7f800000); }

// 16 bytes to the shared variable at `p` of block `rank` of the cluster.
__device__ __forceinline__ void send16(uint4* p, uint32_t rank, const uint4& v) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_address(p, rank)),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 pack(const Soft& s) {
    return make_uint4(__float_as_uint(s.m), __float_as_uint(s.mz), __float_as_uint(s.s), 0u);
}
__device__ __forceinline__ Soft unpack(const uint4& v) {
    return Soft{__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), 0.0f};
}

// What decides about a drafted token.
enum Verdict : int { kAccept = 0, kRefuse = 1, kClose = 2, kBroken = 3, kEnd = 4 };

struct Position {
    Soft p, q;       // statistics of the two rows
    float xd, yd;    // the drafted token's logits
    float u;
    int32_t token;
    int32_t verdict;
};

constexpr int kMaxRows = 16;  // rows per round

struct Shared {
    uint4 parts[2][kWarps][kMaxCluster];  // what the cluster's warps have sent, by turns
    Position pos[kMaxRows];
    int32_t ids[ZERO3_MAX_DRAFT];
    float lp[ZERO3_MAX_DRAFT];
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

// Thread `tid`'s share, of `nt` threads in each of C blocks, of a row.
template <typename T>
__device__ __forceinline__ void stream_row(Soft& q, const T* row, int32_t V, int rank, int C,
                                           float scale, int tid, int nt) {
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    const RowCut<T> cut(row, V);
    const int32_t per = (cut.chunks + C - 1) / C;
    const int32_t c0 = rank * per;
    const int32_t c1 = c0 + per < cut.chunks ? c0 + per : cut.chunks;
    const bool head = tid == 0 && rank == 0 && cut.head;
    const bool tail = tid == nt - 1 && rank == C - 1 && cut.tail;
    const T* p = row + cut.head;
    int32_t i = c0 + tid;
    for (; i + (U - 1) * nt < c1; i += U * nt) {
        Chunk<T> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) c[u].load(p + 8 * static_cast<int64_t>(i + u * nt));
        soft_add<T, false, U>(q, c, scale);
    }
    for (; i < c1; i += nt) {
        Chunk<T> c[1];
        c[0].load(p + 8 * static_cast<int64_t>(i));
        soft_add<T, false, 1>(q, c, scale);
    }
    if (head || tail) {
        const T* f = head ? row : p + 8 * static_cast<int64_t>(cut.chunks);
        const int n = head ? cut.head : cut.tail;
        Chunk<T> c[1];
        c[0].fill(neg_inf());
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) c[0].set(e, f[e]);
        soft_add<T, false, 1>(q, c, scale);
    }
}

// Joins the parts that warps [w0, w0 + nw) of all blocks have sent; every lane of
// the calling warp gets the result.
__device__ __forceinline__ Soft join_rows(const Shared& sh, int turn, int w0, int nw, int C) {
    const int lane = threadIdx.x & 31;
    Soft o = soft_empty();
    for (int i = lane; i < nw * C; i += 32) {
        Soft s = unpack(sh.parts[turn & 1][w0 + i / C][i % C]);
        float top = fmaxf(soft_top(o), soft_top(s));
        if (top == neg_inf()) top = 0.0f;
        soft_rebase<false>(o, top);
        soft_rebase<false>(s, top);
        o.s = __fadd_rn(o.s, s.s);
        if (top == pos_inf()) o.s = __int_as_float(0x7fffffff);
    }
    soft_lanes<false, 32>(o);
    return o;
}

// ------------------------------------------------- 31-bit weights, exact sums
// 2^F for F = n + f / 2^31: y / 2^31 with 0.70 < y / 2^31 < 1.42, from the Taylor
// series of 2^f = e^(f ln 2), terms (ln 2)^k / k!, k <= 9 (the next is below 8e-12 for
// |f| <= 1/2), in 31-bit fixed point.
struct Weight {
    uint32_t y;
    int32_t n;  // below -1000: no weight
};

template <typename T>
__device__ __forceinline__ Weight weight31(T x, float scale, float mz) {
    const float f = to_f32(x);
    // z - mz as a sum of two numbers: the product and the difference with
    // their rounding errors
    const float z = __fmul_rn(f, scale);
    const float zl = fmaf(f, scale, -z);
    const float d = __fsub_rn(z, mz);
    const float bb = __fsub_rn(d, z);
    const float dl = __fadd_rn(__fadd_rn(__fsub_rn(z, __fsub_rn(d, bb)), -__fadd_rn(mz, bb)), zl);
    // times log2(e) = hi + lo
    const float hi = 1.44269502162933349609375f, lo = 1.92596299112661746e-8f;
    const float t = __fmul_rn(d, hi);
    const float tl = fmaf(d, hi, -t) + fmaf(d, lo, __fmul_rn(dl, hi));
    Weight w;
    if (!(t > -1000.0f)) {  // masked tokens too
        w.y = 0;
        w.n = -2000;
        return w;
    }
    const float r = rintf(t);
    const int32_t F = __float2int_rn((t - r) * 2147483648.0f) + __float2int_rn(tl * 2147483648.0f);
    constexpr int64_t c[10] = {2147483648ll, 1488522236ll, 515882496ll, 119194166ll, 20654775ll,
                               2863360ll,    330788ll,     32755ll,     2838ll,      219ll};
    int64_t a = c[9];
#pragma unroll
    for (int k = 8; k >= 0; --k) a = c[k] + ((a * F) >> 31);
    w.y = static_cast<uint32_t>(a);
    w.n = static_cast<int32_t>(r);
    return w;
}

__device__ __forceinline__ double weight64(const Weight& w) {
    if (w.n < -1000) return 0.0;
    return static_cast<double>(w.y) * __hiloint2double((1023 + w.n - 31) << 20, 0);
}

// Bits behind the point of a row's integer sum: V weights below 4 fit 64 bits.
__device__ __forceinline__ int sum_bits(int32_t V) { return 61 - (32 - __clz(V)); }

// This thread's share of the integer sum of a row's weights.
template <typename T>
__device__ __forceinline__ uint64_t exact_share(const T* row, int32_t V, float scale, float mz, int rank,
                                                int C, int bits) {
    uint64_t s = 0;
    for (int64_t i = rank * kNT + threadIdx.x; i < V; i += static_cast<int64_t>(C) * kNT) {
        const Weight w = weight31(row[i], scale, mz);
        const int shift = bits - 31 + w.n;  // y * 2^shift
        if (shift >= 0)
            s += static_cast<uint64_t>(w.y) << (shift < 32 ? shift : 32);
        else if (shift > -34)  // rounded: the errors of many small weights cancel
            s += (w.y + (uint64_t{1} << (-shift - 1))) >> -shift;
    }
    return s;
}

// Sums of the target's and the draft's rows, in every thread of the cluster.
struct Sums {
    double p, q;
};
template <typename TX, typename TY>
__device__ __noinline__ Sums exact_sums(Shared& sh, int turn, const TX* xr, const TY* yr, int32_t V,
                                        float xs, float ys, float mzp, float mzq, int rank, int C) {
    const int bits = sum_bits(V);
    uint64_t s = exact_share(xr, V, xs, mzp, rank, C, bits);
    uint64_t t = yr ? exact_share(yr, V, ys, mzq, rank, C, bits) : 0;
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

// A weight 2^t, t = (x scale - mz) log2(e), and its relative error: the unit's two
// ulp, and three roundings of t.  Without weight below 2^-126.
template <typename T>
__device__ __forceinline__ float weight(T x, float scale, float mz, float& rel) {
    const float t = __fmul_rn(fmaf(to_f32(x), scale, -mz), kLog2e);
    rel = fmaf(fabsf(fmaxf(t, -128.0f)), 0x1p-23f, 0x1p-21f);
    return exp2_approx(t);
}

// What one pass needs to know of its two rows.
template <typename TX, typename TY>
struct Rows {
    const TX* x;
    const TY* y;       // the draft's row, or null
    const float* e;
    float xs, ys, mzp, mzq;
    float ratio;       // sum of the target's weights over the draft's
    float ratio_error; // relative
    int32_t without;   // this token is not drawn (a refused token without probabilities)
};

// Score of token i: (wp - ratio wq) / e, and how far it may be off.
template <typename TX, typename TY>
__device__ __forceinline__ void score(const Rows<TX, TY>& r, TX x, TY y, float e, int32_t i, float& s,
                                      float& off) {
    float rel;
    const float wp = weight(x, r.xs, r.mzp, rel);
    float v = wp;
    off = wp * rel;
    if (r.y) {
        const float wq = weight(y, r.ys, r.mzq, rel) * r.ratio;
        v = wp - wq;
        off = fmaf(wq, rel + r.ratio_error, off);
    }
    const float inv = __fdividef(1.0f, e);
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

template <typename TX, typename TY>
__device__ __forceinline__ Race race_pass(Shared& sh, int turn, const Rows<TX, TY>& r, int32_t V,
                                          int rank, int C) {
    constexpr int U = 4;
    Race b{0.0f, 0.0f, 0.0f, -1};
    const int64_t step = static_cast<int64_t>(C) * kNT;
    int64_t i = rank * kNT + threadIdx.x;
    for (; i + (U - 1) * step < V; i += U * step) {
        TX x[U];
        TY y[U];
        float e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = r.x[i + u * step];
            y[u] = r.y ? r.y[i + u * step] : TY(0);
            e[u] = __ldcs(r.e + i + u * step);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s, off;
            score(r, x[u], y[u], e[u], static_cast<int32_t>(i + u * step), s, off);
            race_add(b, s - off, s + off, static_cast<int32_t>(i + u * step));
        }
    }
    for (; i < V; i += step) {
        float s, off;
        score(r, r.x[i], r.y ? r.y[i] : TY(0), __ldcs(r.e + i), static_cast<int32_t>(i), s, off);
        race_add(b, s - off, s + off, static_cast<int32_t>(i));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Race t;
        t.low = __shfl_xor_sync(0xffffffffu, b.low, o);
        t.up = __shfl_xor_sync(0xffffffffu, b.up, o);
        t.second = __shfl_xor_sync(0xffffffffu, b.second, o);
        t.token = __shfl_xor_sync(0xffffffffu, b.token, o);
        race_join(b, t);
    }
    exchange(sh, turn, C, rank,
             make_uint4(__float_as_uint(b.low), __float_as_uint(b.up), __float_as_uint(b.second),
                        static_cast<uint32_t>(b.token)));
    Race best{0.0f, 0.0f, 0.0f, -1};
    for (int j = threadIdx.x & 31; j < kWarps * C; j += 32) {
        const uint4 v = sh.parts[turn & 1][j / C][j % C];
        race_join(best, Race{__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                             static_cast<int32_t>(v.w)});
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Race t;
        t.low = __shfl_xor_sync(0xffffffffu, best.low, o);
        t.up = __shfl_xor_sync(0xffffffffu, best.up, o);
        t.second = __shfl_xor_sync(0xffffffffu, best.second, o);
        t.token = __shfl_xor_sync(0xffffffffu, best.token, o);
        race_join(best, t);
    }
    return best;
}

// The race among the tokens whose upper bound reaches `low`, with 31-bit weights
// and scores in binary64; ties to the lowest token, -1 if no score is positive.
template <typename TX, typename TY>
__device__ __noinline__ int32_t exact_race(Shared& sh, int turn, const Rows<TX, TY>& r, const Sums& sums,
                                           float low, int32_t V, int rank, int C) {
    double best = 0.0;
    int32_t token = 0x7fffffff;
    for (int64_t i = rank * kNT + threadIdx.x; i < V; i += static_cast<int64_t>(C) * kNT) {
        const TX x = r.x[i];
        const TY y = r.y ? r.y[i] : TY(0);
        const float e = r.e[i];
        float s, off;
        score(r, x, y, e, static_cast<int32_t>(i), s, off);
        if (!(s + off >= low) || !(e >= 0.0f) || i == r.without) continue;
        double v = weight64(weight31(x, r.xs, r.mzp));
        if (r.y) v = v / sums.p - weight64(weight31(y, r.ys, r.mzq)) / sums.q;
        v = v / static_cast<double>(e);
        if (v > best) {  // tokens come in ascending order
            best = v;
            token = static_cast<int32_t>(i);
        }
    }
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
template <typename TX, typename TY, bool DRAFT>
__global__ void __launch_bounds__(kNT, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
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
    wait_prior_grids();
    allow_next_grid();
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
    if (C > 1) cluster_wait();  // the others' shared memory is there
    // relative error of a row's sum: terms off by less than 2^-18 on average, the
    // longest chain of additions
    const int G = a.ahead;
    const int R = DRAFT ? 2 * G : G;
    const int WR = kWarps / R;          // warps per row
    const float sum_error = 0x1p-17f + static_cast<float>(V / (8 * C * WR * 32) + 16) * 0x1p-24f;
    int turn = 0;
    int A = 0;
    int32_t token = -1;
    float token_lp = 0.0f;
    for (int j0 = 0;; j0 += G) {
        // ---- the round's rows
        {
            const int row = warp / WR, g = DRAFT ? row >> 1 : row;
            const bool of_draft = DRAFT && (row & 1);
            Soft q = soft_empty();
            const int j = j0 + g;
            const int tr = (warp % WR) * 32 + lane;
            if (of_draft) {
                if (j < L)
                    stream_row<TY>(q, y + j * a.y_stride, V, rank, C, a.y_scale, tr, WR * 32);
            } else if (j <= L) {
                stream_row<TX>(q, x + j * a.stride, V, rank, C, a.scale, tr, WR * 32);
            }
            soft_lanes<false, 32>(q);
            exchange(sh, turn, C, rank, pack(q));
        }
        // ---- verdicts, a warp each
        if (warp < G && j0 + warp <= L) {
            const int g = warp, j = j0 + g;
            Position o;
            o.p = join_rows(sh, turn, (DRAFT ? 2 * g : g) * WR, WR, C);
            o.q = DRAFT && j < L ? join_rows(sh, turn, (2 * g + 1) * WR, WR, C) : soft_empty();
            o.verdict = kEnd;
            o.token = -1;
            o.xd = o.yd = o.u = 0.0f;
            if (j < L) {
                o.token = sh.ids[j];
                const TX xd = x[j * a.stride + o.token];
                o.xd = to_f32(xd);
                o.u = a.uniform[s * K + j];
                // log2 p = tp - lsp, log2 q = tq - lq; a token that is there keeps its
                // place among the smallest where t leaves binary32's range
                float tq = 0.0f, lq = 0.0f;
                bool q_nan = false, in_q = true;
                if (DRAFT) {
                    const TY yd = y[j * a.y_stride + o.token];
                    o.yd = to_f32(yd);
                    tq = fmaxf(__fmul_rn(fmaf(o.yd, a.y_scale, -o.q.mz), kLog2e), -0x1p126f);
                    lq = log2f(o.q.s);
                    q_nan = o.q.s != o.q.s;
                    in_q = o.q.s != 0.0f && __fmul_rn(o.yd, a.y_scale) != neg_inf();
                }
                const float tp = fmaxf(__fmul_rn(fmaf(o.xd, a.scale, -o.p.mz), kLog2e), -0x1p126f);
                const float lsp = log2f(o.p.s);
                const float lu = log2f(o.u);
                if (lane == 0) sh.lp[j] = __fsub_rn(fmaf(o.xd, a.scale, -o.p.mz), logf(o.p.s));
                if (o.p.s != o.p.s || q_nan || o.u != o.u) {
                    o.verdict = o.u != o.u && o.p.s == o.p.s && !q_nan ? kRefuse : kBroken;
                } else if (o.p.s == 0.0f || __fmul_rn(o.xd, a.scale) == neg_inf()) {
                    o.verdict = kRefuse;
                } else if (!in_q || lu == neg_inf()) {
                    o.verdict = kAccept;
                } else {
                    const float diff = (tp - lsp) - (tq - lq) - lu;
                    const float off = 3.0f * sum_error +
                                      (fabsf(tp) + fabsf(tq) + fabsf(lsp) + fabsf(lq) + fabsf(lu)) * 0x1p-21f;
                    o.verdict = diff > off ? kAccept : diff < -off ? kRefuse : kClose;
                }
            } else if (o.p.s != o.p.s) {
                o.verdict = kBroken;
            }
            if (lane == 0) sh.pos[g] = o;
        }
        ++turn;
        __syncthreads();
        // ---- the first position that does not accept
        int at = -1, verdict = kAccept;
        for (int g = 0; g < G && j0 + g <= L; ++g) {
            verdict = sh.pos[g].verdict;
            if (verdict == kClose) {
                const Position o = sh.pos[g];
                const int j = j0 + g;
                const TX* xr = x + j * a.stride;
                const TY* yr = DRAFT ? y + j * a.y_stride : nullptr;
                const Sums m = exact_sums<TX, TY>(sh, turn, xr, yr, V, a.scale, a.y_scale, o.p.mz, o.q.mz,
                                                  rank, C);
                ++turn;
                const double wp = weight64(weight31(xr[o.token], a.scale, o.p.mz));
                double wq = 1.0, sq = 1.0;
                if (DRAFT) {
                    wq = weight64(weight31(yr[o.token], a.y_scale, o.q.mz));
                    sq = m.q;
                }
                bool less = static_cast<double>(o.u) * wq * m.p < wp * sq;
                if (wp == 0.0 || wq == 0.0) {  // both below 2^-1000: by their logarithms
                    const double lp = static_cast<double>(o.xd) * a.scale - o.p.mz - log(m.p);
                    const double lq = DRAFT ? static_cast<double>(o.yd) * a.y_scale - o.q.mz - log(m.q) : 0.0;
                    less = log(static_cast<double>(o.u)) + lq < lp;
                }
                verdict = less ? kAccept : kRefuse;
            }
            if (verdict != kAccept) {
                at = g;
                break;
            }
        }
        if (at < 0) continue;  // the next exchange's barrier lies before the positions' next writing
        // ---- the draw
        A = j0 + at;
        const Position o = sh.pos[at];
        if (verdict == kBroken) {
            token_lp = __int_as_float(0x7fffffff);
            break;
        }
        if (o.p.s == 0.0f) {
            token_lp = neg_inf();
            break;
        }
        Rows<TX, TY> r;
        r.x = x + A * a.stride;
        r.y = nullptr;
        r.e = noise;
        r.xs = a.scale;
        r.ys = a.y_scale;
        r.mzp = o.p.mz;
        r.mzq = o.q.mz;
        r.ratio = 0.0f;
        r.ratio_error = 0.0f;
        r.without = -1;
        if (verdict == kRefuse) {
            if (!DRAFT) {
                r.without = o.token;
            } else if (o.q.s != 0.0f) {
                r.y = y + A * a.y_stride;
                r.ratio = __fdiv_rn(o.p.s, o.q.s);
                r.ratio_error = 2.5f * sum_error;
            }
        }
        for (int pass = 0; pass < 2; ++pass) {
            const Race b = race_pass(sh, turn, r, V, rank, C);
            ++turn;
            if (b.low > 0.0f && b.second < b.low) {
                token = b.token;
            } else {
                Sums m{1.0, 1.0};
                if (r.y) {
                    m = exact_sums<TX, TY>(sh, turn, r.x, r.y, V, r.xs, r.ys, r.mzp, r.mzq, rank, C);
                    ++turn;
                }
                token = exact_race(sh, turn, r, m, b.low, V, rank, C);
                ++turn;
            }
            if (token >= 0 || (!r.y && r.without < 0)) break;
            r.y = nullptr;  // no residual: from the target itself
            r.without = -1;
        }
        token_lp = neg_inf();
        if (token >= 0)
            token_lp = __fsub_rn(fmaf(to_f32(r.x[token]), a.scale, -o.p.mz), logf(o.p.s));
        break;
    }
    if (rank == 0) {
        if (tid == 0) a.accepted[s] = A;
        for (int j = tid; j <= K; j += kNT) {
            a.tokens[s * (K + 1) + j] = j < A ? sh.ids[j] : j == A ? token : -1;
            if (a.logprobs) a.logprobs[s * (K + 1) + j] = j < A ? sh.lp[j] : j == A ? token_lp : 0.0f;
        }
    }
}

template <typename TX, typename TY>
cudaError_t launch_types(const VerifyArgs& a, cudaStream_t stream) {
    const int64_t grid = a.n * a.cluster;
    return a.y ? launch_vocab(verify_kernel<TX, TY, true>, grid, kNT, 0, a.cluster, a, stream)
               : launch_vocab(verify_kernel<TX, TX, false>, grid, kNT, 0, a.cluster, a, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& args, cudaStream_t stream) {
    VerifyArgs a = args;
    a.cluster = 1;
    while (a.cluster < kMaxCluster && a.n * a.cluster * 2 <= 304) a.cluster *= 2;
    const int most = a.y ? kMaxRows / 2 : kMaxRows;
    a.ahead = 1;
    // few sequences: their rows in one round, while latency costs more than rows
    // that turn out not to be needed
    if (a.n <= 19)
        while (a.ahead < most && a.ahead < a.k + 1) a.ahead *= 2;
    if (a.dtype == ZERO3_BF16)
        return a.y_dtype == ZERO3_BF16 ? launch_types<uint16_t, uint16_t>(a, stream)
                                       : launch_types<uint16_t, float>(a, stream);
    return a.y_dtype == ZERO3_BF16 ? launch_types<float, uint16_t>(a, stream)
                                   : launch_types<float, float>(a, stream);
}

}  // namespace z3
