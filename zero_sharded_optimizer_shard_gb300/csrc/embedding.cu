// Embedding lookup with scaling, and its gradient by sorted tokens (sm_103a).
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {
namespace {

// ------------------------------------------------------------------ lookup
// Eight elements at any alignment, by the two or three aligned 16-byte words that
// hold them, shifted into place.
template <typename T>
struct Shifted;
template <>
struct Shifted<uint16_t> {
    uint4 a, b;
    uint32_t off;
    __device__ __forceinline__ void load(const uint16_t* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const uint4* w = reinterpret_cast<const uint4*>(at & ~uintptr_t{15});
        off = static_cast<uint32_t>(at & 15u);
        a = w[0];
        b = w[off ? 1 : 0];
    }
    // chunk `i` of a row that starts at element `skip` of words in shared memory
    __device__ __forceinline__ void take(const uint4* w, int i, uint32_t skip) {
        off = 2 * skip;
        a = w[i];
        b = w[off ? i + 1 : i];
    }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t y[6], z[5];
#pragma unroll
        for (int i = 0; i < 6; ++i) y[i] = off & 8u ? x[i + 2] : x[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) z[i] = off & 4u ? y[i + 1] : y[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = __funnelshift_r(z[i], z[i + 1], (off & 2u) * 8u);
            f[2 * i] = bf16_lo(v);
            f[2 * i + 1] = bf16_hi(v);
        }
    }
};
template <>
struct Shifted<float> {
    float4 a, b, c;
    uint32_t off;
    __device__ __forceinline__ void load(const float* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const float4* w = reinterpret_cast<const float4*>(at & ~uintptr_t{15});
        off = static_cast<uint32_t>(at & 15u);
        a = w[0];
        b = w[1];
        c = w[off ? 2 : 1];
    }
    __device__ __forceinline__ void take(const uint4* m, int i, uint32_t skip) {
        const float4* w = reinterpret_cast<const float4*>(m) + 2 * i;
        off = 4 * skip;
        a = w[0];
        b = w[1];
        c = w[off ? 2 : 1];
    }
    __device__ __forceinline__ void get(float* f) const {
        const float x[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
        float y[9];
#pragma unroll
        for (int i = 0; i < 9; ++i) y[i] = off & 8u ? x[i + 2] : x[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = off & 4u ? y[i + 1] : y[i];
    }
};
// Whether Shifted::load(p) stays within a matrix [begin, end) of rows and the
// gaps between them.
template <typename T>
__device__ __forceinline__ bool inside(const T* p, const T* begin, const T* end) {
    constexpr int64_t W = 16 / sizeof(T);  // a word's elements
    return p - begin >= W && end - p >= 8 + W;
}

// out[i] = rne(scale * table[ids[i]]), zeros where the id lies outside the
// vocabulary.  A copy of n random rows: bound by HBM (the row reads, of
// which repeated tokens hit L2, and the writes).  A row's units are 8 columns
// each; the n rows' units are numbered consecutively, a block takes NT * U of
// them, a thread U, NT apart, with all of its row loads in flight before its
// first store.
//
// VEC: all rows start on 16-byte boundaries.  Otherwise a row's units are cut at
// the output row's 16-byte boundaries, one more than dim / 8 rounded up, and the
// table's elements are shifted into place; a unit that sticks out of its row, or
// whose words would lie outside the table, goes by single elements.
//
// 16384 rows of 4096 bf16 take 30.4 us (182 MB, 6.0 TB/s), 8192 of 2047 15.1 us, one
// row of 2048 1.4 us.
template <typename TT, typename TO, bool VEC, int NT, int U>
__global__ void __launch_bounds__(NT) embed_kernel(const __grid_constant__ EmbedArgs a) {
    wait_prior_grids();
    allow_next_grid();
    const uint32_t units = static_cast<uint32_t>(VEC ? a.dim / 8 : a.dim / 8 + 2);  // per row
    const uint64_t b0 = static_cast<uint64_t>(blockIdx.x) * (NT * U);
    const uint64_t row0 = b0 / units;
    const uint32_t rem = static_cast<uint32_t>(b0 - row0 * units) + threadIdx.x;
    uint64_t row[U];
    uint32_t at[U];
    int32_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t k = rem + u * NT;
        const uint32_t d = k / units;
        row[u] = row0 + d;
        at[u] = k - d * units;
        id[u] = row[u] < static_cast<uint64_t>(a.n)
                    ? load_id(a.ids, a.id64, static_cast<int64_t>(row[u]), a.vocab) : -1;
    }
    const TT* table = static_cast<const TT*>(a.table);
    TO* out = static_cast<TO*>(a.out);
    const uint64_t sc = pk2(a.scale, a.scale);
    if (VEC) {
        Chunk<TT> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u].fill(0.0f);
            if (id[u] >= 0) c[u].load(table + id[u] * a.table_stride + 8ll * at[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] >= static_cast<uint64_t>(a.n)) continue;
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                upk2(mul2(c[u].pair(k), sc), f[2 * k], f[2 * k + 1]);
                if (id[u] < 0) f[2 * k] = f[2 * k + 1] = 0.0f;
            }
            Chunk<TO>::store(out + row[u] * a.out_stride + 8ll * at[u], f);
        }
    } else {
        constexpr int P = Chunk<TO>::kPhase;
        const TT* const end = table + (a.vocab - 1) * a.table_stride + a.dim;
        float f[U][8];
        int64_t j[U];  // the unit's first column
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const TO* o = out + row[u] * a.out_stride;
            j[u] = 8ll * at[u] - static_cast<int64_t>((reinterpret_cast<uintptr_t>(o) / sizeof(TO)) % P);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[u][k] = 0.0f;
            if (id[u] < 0 || j[u] >= a.dim) continue;
            const TT* p = table + id[u] * a.table_stride + j[u];
            if (inside(p, table, end)) {
                Shifted<TT> x;
                x.load(p);
                x.get(f[u]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (j[u] + k >= 0 && j[u] + k < a.dim) f[u][k] = to_f32(p[k]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] >= static_cast<uint64_t>(a.n)) continue;
            TO* o = out + row[u] * a.out_stride + j[u];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[u][k] = id[u] >= 0 ? __fmul_rn(f[u][k], a.scale) : 0.0f;
            if (j[u] >= 0 && j[u] + 8 <= a.dim) {
                Chunk<TO>::store(o, f[u]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (j[u] + k >= 0 && j[u] + k < a.dim) o[k] = from_f32<TO>(f[u][k]);
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
// grad[v] = rne(base + scale * sum over the positions i of token v, in
// ascending order, of dout[i]), in two launches: a stable counting sort of
// the positions by token, and the rows' sums.  Sums are binary32 and their
// order depends on the tokens alone, so the result does not depend on timing.
// (Adding each position's row to its token's row with atomics would neither
// have a fixed order nor spread the frequent tokens' work.)
//
// Both launches: 8192 x 768 bf16 into 50257 rows, all written, 20.0 us; 32768 x 2048
// bf16 added to bf16 49.4 us (220 MB: 4.5 TB/s), to binary32 71 us, binary32 to
// binary32 123 us.
constexpr int kOwn = 512;          // tokens a sorting block owns at most
constexpr int kList = 512;         // own positions a sorting warp lists
// Shortest piece of a token that has several.  Short ones spread frequent tokens,
// long ones cost fewer partial sums: at 8 / 16 / 32, 2048 x 64 takes 10.3 / 11.1 / 13.8
// us, 32768 x 2048 53.4 / 51.0 / 50.4.
constexpr int kPiece = 16;
constexpr int kSumThreads = 128;
// Bytes of rows in flight per summing warp (4096: 2048 x 64 10.8 us, not 11.1, but
// binary32 rows are left with few).
constexpr int kRing = 8192;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kGroupCols = 256;    // columns of a warp: 8 per lane, times CU

// A sorted position: where it was, its token, the token's first sorted index
// and number of positions.
struct alignas(16) Sorted {
    int32_t pos, token, first, count;
};

struct Workspace {
    int32_t* off;      // [places + 1] first sorted index of the token at each place
    Sorted* sorted;    // [n] positions by token, ascending
    int32_t* arrived;  // [buckets * groups] pieces of a token that are done
    float* partial;    // [buckets * 2 * dim] pieces' sums
    int64_t buckets, groups, step, bytes;
};

// Tokens are dealt out to the sorting blocks like cards (token v to block
// v mod 2^shift), because in text the frequent ones are neighbours; `place`
// is where a token stands in the sorted order.
struct Deal {
    int32_t shift, own;  // blocks = 2^shift, tokens per block
    __host__ __device__ __forceinline__ int32_t place(int32_t v) const {
        return (v & ((1 << shift) - 1)) * own + (v >> shift);
    }
};

// Sorting blocks: a power of two, about the SMs' number, more where a block
// would own too many tokens.
inline Deal deal_of(int64_t vocab) {
    Deal d;
    d.shift = 7;
    while ((vocab + (int64_t{1} << d.shift) - 1) >> d.shift > kOwn) ++d.shift;
    d.own = static_cast<int32_t>((vocab + (int64_t{1} << d.shift) - 1) >> d.shift);
    return d;
}

__host__ __device__ inline int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }

inline Workspace workspace_of(void* base, int64_t n, int64_t vocab, int64_t dim) {
    const Deal d = deal_of(vocab);
    const int64_t places = static_cast<int64_t>(d.own) << d.shift;
    Workspace w;
    w.buckets = n / kPiece + 1;
    w.groups = (dim + kGroupCols - 1) / kGroupCols;
    w.step = (dim + 3) / 4 * 4;
    char* p = static_cast<char*>(base);
    int64_t o = 0;
    const auto take = [&](int64_t bytes) {
        char* at = p + o;
        o += up16(bytes);
        return at;
    };
    w.off = reinterpret_cast<int32_t*>(take(4 * (places + 1)));
    w.sorted = reinterpret_cast<Sorted*>(take(static_cast<int64_t>(sizeof(Sorted)) * n));
    w.arrived = reinterpret_cast<int32_t*>(take(4 * w.buckets * w.groups));
    w.partial = reinterpret_cast<float*>(take(8 * w.buckets * w.step));
    w.bytes = o;
    return w;
}

struct SortArgs {
    const void* ids;
    Workspace w;
    Deal deal;
    int64_t n;
    int32_t vocab, id64;
};

// Stable counting sort without communication between blocks: every block
// reads all ids, counts those of the blocks before it (which gives the first
// sorted index of its own) and lists, warp by warp and in order, those of its
// own tokens; the lists are counted by token, the counts summed up, and each
// warp places its positions in order.  A warp's list that overflows (a token
// that fills the batch) is read from the ids again.  Small batches are bound by
// latency: what counts is that a warp's loads are in flight together.  Large ones are
// bound by issue, every block testing every id (32768: 64% of the issue slots): what
// counts is that little is done per id that is not the block's.  By itself 6 us
// for 3001 ids, 8 for 8192, 13 for 32768.  (A radix sort over the grid needs a wait between its digits.)
template <int W>
struct SortShared {
    int32_t cnt[W][kOwn];
    uint32_t list[W][kList];  // token, position from the warp's first on
    int32_t first[kOwn], count[kOwn];
    int32_t sh[W], scan[W];
};
template <int W, int J>
__global__ void __launch_bounds__(32 * W) embed_sort_kernel(const __grid_constant__ SortArgs a) {
    constexpr int NT = 32 * W;
    extern __shared__ uint4 dyn[];
    SortShared<W>& s = *reinterpret_cast<SortShared<W>*>(dyn);
    auto& cnt = s.cnt;
    auto& list = s.list;
    wait_prior_grids();
    allow_next_grid();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int32_t me = blockIdx.x, mask = (1 << a.deal.shift) - 1, own = a.deal.own;
    const int64_t per = (a.n + NT - 1) / NT * 32;
    const int64_t i0 = per * warp, i1 = i0 + per < a.n ? i0 + per : a.n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * NT + tid; i < a.w.buckets * a.w.groups;
         i += static_cast<int64_t>(gridDim.x) * NT)
        a.w.arrived[i] = 0;
    for (int k = lane; k < own; k += 32) cnt[warp][k] = 0;
    __syncwarp();
    int32_t less = 0;
    int n = 0;  // own positions of the warp
    for (int64_t b = i0; b < i1; b += 32 * J) {
        // an id as two words: valid if the high one is 0 and the low one
        // below the vocabulary
        uint32_t lo[J], hi[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = b + 32 * j + lane;
            lo[j] = 0xffffffffu;
            hi[j] = 0;
            if (i < i1) {
                if (a.id64) {
                    const uint2 x = static_cast<const uint2*>(a.ids)[i];
                    lo[j] = x.x;
                    hi[j] = x.y;
                } else {
                    lo[j] = static_cast<const uint32_t*>(a.ids)[i];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool valid = hi[j] == 0 && lo[j] < static_cast<uint32_t>(a.vocab);
            const int32_t o = valid ? static_cast<int32_t>(lo[j]) & mask : 0x7fffffff;
            less += o < me;
            const bool in = o == me;
            const uint32_t m = __ballot_sync(0xffffffffu, in);
            if (!m) continue;
            if (in) {
                const int32_t k = static_cast<int32_t>(lo[j]) >> a.deal.shift;
                const int at = n + __popc(m & below);
                if (at < kList)
                    list[warp][at] = static_cast<uint32_t>(k) << 16 |
                                     static_cast<uint32_t>(b - i0 + 32 * j + lane);
                atomicAdd(&cnt[warp][k], 1);
            }
            n += __popc(m);
        }
    }
    for (int o = 16; o > 0; o >>= 1) less += __shfl_xor_sync(0xffffffffu, less, o);
    if (lane == 0) s.sh[warp] = less;
    __syncthreads();
    // exclusive scan over the own tokens' totals, kPer tokens per thread
    constexpr int kPer = (kOwn + NT - 1) / NT;
    int32_t total[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int k = tid * kPer + j;
        total[j] = 0;
        if (k < own) {
#pragma unroll 8
            for (int w = 0; w < W; ++w) total[j] += cnt[w][k];
        }
        sum += total[j];
    }
    int32_t incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s.scan[warp] = incl;
    __syncthreads();
    int32_t run = incl - sum;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        run += s.sh[w];
        if (w < warp) run += s.scan[w];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int k = tid * kPer + j;
        if (k >= own) break;
        a.w.off[me * own + k] = run;
        if (me == mask && k == own - 1) a.w.off[(mask + 1) * own] = run + total[j];
        s.first[k] = run;
        s.count[k] = total[j];
        if (total[j] == 0) continue;
        for (int w = 0; w < W; ++w) {
            const int32_t c = cnt[w][k];
            cnt[w][k] = run;
            run += c;
        }
    }
    __syncthreads();
    // places 32 positions i (those >= 0) of tokens k, in lane order
    const auto place = [&](int32_t i, int32_t k) {
        if (!__any_sync(0xffffffffu, i >= 0)) return;
        const uint32_t peers = __match_any_sync(0xffffffffu, k);
        const int rank = __popc(peers & below);
        if (i >= 0) {
            Sorted x;
            x.pos = i;
            x.token = (k << a.deal.shift) | me;
            x.first = s.first[k];
            x.count = s.count[k];
            *reinterpret_cast<int4*>(a.w.sorted + cnt[warp][k] + rank) =
                *reinterpret_cast<const int4*>(&x);
        }
        __syncwarp();
        if (i >= 0 && rank == 0) cnt[warp][k] += __popc(peers);
        __syncwarp();
    };
    if (n <= kList && per < 65536) {
        for (int b = 0; b < n; b += 32) {
            const bool in = b + lane < n;
            const uint32_t x = in ? list[warp][b + lane] : 0;
            place(in ? static_cast<int32_t>(i0 + (x & 0xffffu)) : -1, in ? static_cast<int32_t>(x >> 16) : -1);
        }
        return;
    }
    for (int64_t b = i0; b < i1; b += 32 * J) {
        int32_t id[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = b + 32 * j + lane;
            id[j] = i < i1 ? load_id(a.ids, a.id64, i, a.vocab) : -1;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = id[j] >= 0 && (id[j] & mask) == me;
            place(in ? static_cast<int32_t>(b + 32 * j + lane) : -1,
                  in ? id[j] >> a.deal.shift : -1);
        }
    }
}

struct SumArgs {
    EmbedGradArgs a;
    Workspace w;
    Deal deal;
    int32_t rows;   // sorted positions whose pieces a summing warp takes
    int32_t slabs, zero_tokens;
    int64_t sum_blocks;
};

// A lane's columns: CU groups of 8.  Group u starts at:
__device__ __forceinline__ int32_t column(int32_t c0, int lane, int u) {
    return c0 + kGroupCols * u + 8 * lane;
}

// A group of a piece's sum, in `partial`, whose rows have room up to a
// multiple of 4 columns.
__device__ __forceinline__ void store_part(float* row, int32_t at, int32_t dim, const uint64_t* acc) {
    float4 x;
    upk2(acc[0], x.x, x.y);
    upk2(acc[1], x.z, x.w);
    if (at < dim) *reinterpret_cast<float4*>(row + at) = x;
    upk2(acc[2], x.x, x.y);
    upk2(acc[3], x.z, x.w);
    if (at + 4 < dim) *reinterpret_cast<float4*>(row + at + 4) = x;
}
// (Another SM has written it during this launch: it comes from L2.)
__device__ __forceinline__ void load_part(Chunk<float>& c, const float* row, int32_t at, int32_t dim) {
    c.fill(0.0f);
    if (at < dim) c.a = __ldcg(reinterpret_cast<const float4*>(row + at));
    if (at + 4 < dim) c.b = __ldcg(reinterpret_cast<const float4*>(row + at + 4));
}

// Writes group u of token v's row.  VEC: from 16-byte boundaries on, on top of
// `old`.  Otherwise the warp's 256 sums change places in `swap`, so that it
// reads and writes consecutive single elements.
template <typename TG, bool VEC, bool ACC>
__device__ __forceinline__ void put_group(const SumArgs& p, int32_t v, int32_t c0, int u, int lane,
                                          const uint64_t* acc, const Chunk<TG>& old, float* swap) {
    const int32_t dim = static_cast<int32_t>(p.a.dim), at = column(c0, lane, u);
    TG* g = static_cast<TG*>(p.a.grad) + v * p.a.grad_stride;
    if (VEC) {
        const uint64_t sc = pk2(p.a.scale, p.a.scale);
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            upk2(ACC ? fma2(acc[k], sc, old.pair(k)) : mul2(acc[k], sc), f[2 * k], f[2 * k + 1]);
        if (at < dim) Chunk<TG>::store(g + at, f);
        return;
    }
    float4 lo, hi;
    upk2(acc[0], lo.x, lo.y);
    upk2(acc[1], lo.z, lo.w);
    upk2(acc[2], hi.x, hi.y);
    upk2(acc[3], hi.z, hi.w);
    g += at - 7 * lane;  // the group's first column, plus the lane
    const int32_t left = dim - (at - 7 * lane);
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = ACC && 32 * k < left ? to_f32(g[32 * k]) : 0.0f;
    __syncwarp();
    reinterpret_cast<float4*>(swap)[2 * lane] = lo;
    reinterpret_cast<float4*>(swap)[2 * lane + 1] = hi;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float s = swap[32 * k + lane];
        if (32 * k < left)
            g[32 * k] = from_f32<TG>(ACC ? fmaf(s, p.a.scale, x[k]) : __fmul_rn(s, p.a.scale));
    }
}

// Clears the rows of tokens without a position: a warp takes p.zero_tokens
// tokens and all columns.
template <typename TG>
__device__ __forceinline__ void clear_rows(const SumArgs& p, int64_t warp, int lane) {
    constexpr int E = Chunk<TG>::kPhase;
    const int64_t v0 = warp * p.zero_tokens, v = v0 + lane;
    bool empty = false;
    if (lane < p.zero_tokens && v < p.a.vocab) {
        const int32_t at = p.deal.place(static_cast<int32_t>(v));
        empty = p.w.off[at] == p.w.off[at + 1];
    }
    uint32_t m = __ballot_sync(0xffffffffu, empty);
    while (m) {
        TG* g = static_cast<TG*>(p.a.grad) + (v0 + __ffs(m) - 1) * p.a.grad_stride;
        m &= m - 1;
        const int32_t head = RowCut<TG>(g, static_cast<int32_t>(p.a.dim)).head;
        const int32_t words = (static_cast<int32_t>(p.a.dim) - head) / E, end = head + words * E;
        for (int32_t c = lane; c < words; c += 32)
            __stcs(reinterpret_cast<uint4*>(g + head) + c, make_uint4(0, 0, 0, 0));
        if (lane < head) g[lane] = from_f32<TG>(0.0f);
        if (lane < p.a.dim - end) g[end + lane] = from_f32<TG>(0.0f);
    }
}

// Positions of a piece: a token with up to 512 positions is cut every 16, longer
// ones every 32 or 64, and from 8193 positions on every 128.  One warp joins a
// token's pieces, 8 at a time, so a token that fills a large batch costs:
// 131072 positions of 768 columns take 84 us when the tokens are spread, 249 when
// 15 of 16 are one token's.
__device__ __forceinline__ int32_t piece_rows(int32_t count) {
    return count <= 32 * kPiece ? kPiece
           : count <= 128 * kPiece ? 2 * kPiece
           : count <= 512 * kPiece ? 4 * kPiece
                                   : 8 * kPiece;
}
// Row of `partial` for the piece that starts at sorted index `at`: the
// pieces of tokens with several start at least kPiece apart but where one
// token's last and the next one's first meet, so a bucket of kPiece indices
// holds at most one first piece and one later one.
__device__ __forceinline__ int64_t piece_slot(int32_t at, bool first) {
    return 2 * static_cast<int64_t>(at / kPiece) + (first ? 1 : 0);
}

// Adds up a token's pieces in order and writes its row.
template <typename TG, bool VEC, bool ACC, int CU>
__device__ __forceinline__ void join(const SumArgs& p, int32_t v, int32_t first, int32_t count,
                                     int32_t c0, int lane, float* swap) {
    const int32_t step = piece_rows(count), dim = static_cast<int32_t>(p.a.dim);
    const TG* g = static_cast<const TG*>(p.a.grad) + v * p.a.grad_stride;
    for (int u = 0; u < CU; ++u) {
        const int32_t at = column(c0, lane, u);
        Chunk<TG> old;
        old.fill(0.0f);
        if (VEC && ACC && at < dim) old.load_stream(g + at);
        uint64_t acc[4] = {0, 0, 0, 0};
        constexpr int R = 8;
        // unsigned: steps past a count near 2^31 do not wrap
        for (uint32_t b = 0; b < static_cast<uint32_t>(count); b += R * step) {
            Chunk<float> x[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (b + r * step < static_cast<uint32_t>(count))
                    load_part(x[r], p.w.partial + piece_slot(first + static_cast<int32_t>(b + r * step),
                                                             b + r == 0) * p.w.step, at, dim);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (b + r * step >= static_cast<uint32_t>(count)) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] = add2(acc[k], x[r].pair(k));
            }
        }
        put_group<TG, VEC, ACC>(p, v, c0, u, lane, acc, old, swap);
    }
}

// The pieces that a warp sums: those that start among `rows` consecutive
// sorted positions, which together are consecutive rows [a, e) of the sorted
// order (counted from j0).  Lane l knows position j0 + l.
struct Pieces {
    Sorted x;
    uint32_t starts;
    int32_t j0, a, e, count;
    __device__ __forceinline__ bool last(int l) const {  // of its piece
        return l == e - 1 || (l < 31 && (starts >> (l + 1) & 1u));
    }
    __device__ __forceinline__ int piece_of(int l) const {  // where row l's piece starts
        return 31 - __clz(l >= 31 ? starts : starts & ((2u << l) - 1u));
    }
};

// False if no piece starts there.
__device__ __forceinline__ bool find_pieces(const SumArgs& p, int64_t tile, int lane, Pieces& q) {
    const int64_t j = tile * p.rows;
    if (j >= p.a.n) return false;
    q.j0 = static_cast<int32_t>(j);
    q.x = Sorted{0, -1, 0, 0};
    if (j + lane < p.a.n)  // stale beyond the count, which arrives with it
        *reinterpret_cast<int4*>(&q.x) = *reinterpret_cast<const int4*>(p.w.sorted + j + lane);
    q.count = p.w.off[p.deal.own << p.deal.shift];  // ignored positions are not sorted
    // where in its token's positions the lane's lies (from j0 on, because j0 + 32
    // may pass 2^31)
    const uint32_t size = piece_rows(q.x.count);
    const uint32_t into = static_cast<uint32_t>(q.j0) + lane - static_cast<uint32_t>(q.x.first);
    q.starts = __ballot_sync(0xffffffffu, lane < p.rows && lane < q.count - q.j0 &&
                                              (into & (size - 1)) == 0);
    if (!q.starts) return false;
    q.a = __ffs(q.starts) - 1;
    const int32_t end = lane + static_cast<int32_t>(min(size, static_cast<uint32_t>(q.x.count) - into));
    q.e = __shfl_sync(0xffffffffu, end, 31 - __clz(q.starts));
    return true;
}

// Ends the piece that starts at lane `from`: the sum of a whole token is
// written as it is (on top of `old`); one of several goes to `partial`, and
// true is returned if it was the token's last to arrive.
template <typename TG, bool VEC, bool ACC, int CU>
__device__ __forceinline__ bool end_piece(const SumArgs& p, const Pieces& q, int from, int32_t slab,
                                          int lane, uint64_t (&acc)[CU][4],
                                          const Chunk<TG> (&old)[CU], float* swap) {
    const int32_t c0 = slab * (kGroupCols * CU);
    const int32_t v = __shfl_sync(0xffffffffu, q.x.token, from);
    const int32_t n = __shfl_sync(0xffffffffu, q.x.count, from);
    bool done = false;
    if (n <= kPiece) {
#pragma unroll
        for (int u = 0; u < CU; ++u)
            put_group<TG, VEC, ACC>(p, v, c0, u, lane, acc[u], old[u], swap);
    } else {
        const int32_t first = __shfl_sync(0xffffffffu, q.x.first, from);
        float* to = p.w.partial + piece_slot(q.j0 + from, q.j0 + from == first) * p.w.step;
#pragma unroll
        for (int u = 0; u < CU; ++u)
            store_part(to, column(c0, lane, u), static_cast<int32_t>(p.a.dim), acc[u]);
        __threadfence();
        __syncwarp();
        int all = 0;
        if (lane == 0)
            all = atomicAdd(p.w.arrived + static_cast<int64_t>(first / kPiece) * p.slabs + slab, 1) ==
                  (n - 1) / piece_rows(n);
        done = __shfl_sync(0xffffffffu, all, 0);
    }
#pragma unroll
    for (int u = 0; u < CU; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[u][k] = 0;  // packed +0
    return done;
}

template <typename TG, bool VEC, bool ACC, int CU>
__device__ __forceinline__ void join_pieces(const SumArgs& p, const Pieces& q, uint32_t joins,
                                            int32_t slab, int lane, float* swap) {
    while (joins) {
        __threadfence();
        const int from = __ffs(joins) - 1;
        joins &= joins - 1;
        join<TG, VEC, ACC, CU>(p, __shfl_sync(0xffffffffu, q.x.token, from),
                               __shfl_sync(0xffffffffu, q.x.first, from),
                               __shfl_sync(0xffffffffu, q.x.count, from),
                               slab * (kGroupCols * CU), lane, swap);
    }
}

// The sums.  The sorted positions are cut into pieces (all of a token's
// positions, or piece_rows of them), and a warp takes the pieces that start
// among `rows` consecutive positions, for CU groups of columns: the work
// is even however often a token occurs.  Pieces of one token are added up in
// order by whichever warp of the token comes last.  Bound by HBM once there
// are some thousand positions: each row is read once (32768 x 2048 added to bf16:
// 220 MB in about 37 us, 20 warps per SM; more blocks per SM by fewer registers
// spill, 61 us for 49 in all), by latency below.
//
// Rows on 16-byte boundaries pass through a ring of D slots per warp in
// shared memory, filled by asynchronous 16-byte copies (each lane reads what
// it copied itself, so there are no barriers); the row that a sum is added to
// takes a slot like the others, behind its piece's last row.
template <typename TD, typename TG, bool ACC, int CU>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ SumArgs p) {
    constexpr int PD = sizeof(TD) / 2, PG = sizeof(TG) / 2;  // 16-byte parts per group
    constexpr int P = CU * (ACC && PG > PD ? PG : PD);       // parts per slot
    constexpr int D = kRing / (512 * P);
    __shared__ __align__(16) uint4 ring[kSumWarps][D][P][32];
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= p.sum_blocks) {
        const int64_t b = blockIdx.x - p.sum_blocks;
        clear_rows<TG>(p, b * kSumWarps + warp, lane);
        return;
    }
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kSumWarps + warp;
    const int64_t tile = w / p.slabs;
    const int32_t slab = static_cast<int32_t>(w - tile * p.slabs);
    const int32_t c0 = slab * (kGroupCols * CU), dim = static_cast<int32_t>(p.a.dim);
    Pieces q;
    if (!find_pieces(p, tile, lane, q)) return;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&ring[warp][0][0][lane]));
    const auto copy = [&](const void* row, int parts, int bytes, int slot) {
#pragma unroll
        for (int u = 0; u < CU; ++u) {
            const int32_t at = column(c0, lane, u);
            if (at >= dim) continue;
            const char* from = static_cast<const char*>(row) + static_cast<int64_t>(at) * bytes;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (h < parts)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     to + static_cast<uint32_t>((slot * P + u * parts + h) * 512)),
                                 "l"(from + 16 * h)
                                 : "memory");
        }
    };
    int next = q.a, slot = 0;   // the next row to copy, and its slot
    bool base = false;          // first the row that the sum before it is added to
    int32_t pos = q.x.pos;
    const auto issue = [&] {
        if (ACC && base) {
            base = false;
            const int from = q.piece_of(next - 1);
            copy(static_cast<const TG*>(p.a.grad) +
                     __shfl_sync(0xffffffffu, q.x.token, from) * p.a.grad_stride,
                 PG, sizeof(TG), slot);
        } else if (next < q.e) {
            if (next >= 32 && (next & 31) == 0)
                pos = next + lane < q.count - q.j0 ? (p.w.sorted + q.j0)[next + lane].pos : 0;
            copy(static_cast<const TD*>(p.a.dout) +
                     __shfl_sync(0xffffffffu, pos, next & 31) * p.a.dout_stride,
                 PD, sizeof(TD), slot);
            base = ACC && q.last(next);
            ++next;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        slot = slot + 1 == D ? 0 : slot + 1;
    };
    const auto arrive = [&] { asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory"); };
#pragma unroll 1
    for (int i = 0; i < D; ++i) issue();
    uint64_t acc[CU][4];
#pragma unroll
    for (int u = 0; u < CU; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[u][k] = 0;  // packed +0
    uint32_t joins = 0;
#pragma unroll 1
    for (int l = q.a; l < q.e; ++l) {
        arrive();
#pragma unroll
        for (int u = 0; u < CU; ++u) {
            Chunk<TD> row;
            row.from_parts(&ring[warp][slot][u * PD][lane], 32);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[u][k] = add2(acc[u][k], row.pair(k));
        }
        issue();
        if (!q.last(l)) continue;
        Chunk<TG> old[CU];
        if (ACC) {
            arrive();
#pragma unroll
            for (int u = 0; u < CU; ++u) old[u].from_parts(&ring[warp][slot][u * PG][lane], 32);
            issue();
        }
        const int from = q.piece_of(l);
        if (end_piece<TG, true, ACC, CU>(p, q, from, slab, lane, acc, old, nullptr))
            joins |= 1u << from;
    }
    join_pieces<TG, true, ACC, CU>(p, q, joins, slab, lane, nullptr);
}

// The same for rows at any alignment: a slot holds the aligned 16-byte words
// that a row's 256 columns touch, which the lanes shift into place; a slot whose
// words might stick out of the matrix is copied by elements.  32768 x 2047 added to
// bf16: 76 us (131 by single elements).  (Columns past the row's end
// may hold another row's elements; their sums are not used.)
template <typename TD, typename TG, bool ACC>
__global__ void __launch_bounds__(kSumThreads)
    embed_sum_any_kernel(const __grid_constant__ SumArgs p) {
    constexpr int W = kGroupCols * sizeof(TD) / 16 + 1;  // words of a slot
    constexpr int E = 16 / sizeof(TD);                    // elements of a word
    constexpr int D = kRing / (16 * W);
    __shared__ __align__(16) uint4 ring[kSumWarps][D][W];
    __shared__ __align__(16) float swap[kSumWarps][kGroupCols];
    __shared__ uint32_t starts[kSumWarps][D];  // where in its first word a slot's row starts
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= p.sum_blocks) {
        const int64_t b = blockIdx.x - p.sum_blocks;
        clear_rows<TG>(p, b * kSumWarps + warp, lane);
        return;
    }
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kSumWarps + warp;
    const int64_t tile = w / p.slabs;
    const int32_t slab = static_cast<int32_t>(w - tile * p.slabs);
    const int32_t c0 = slab * kGroupCols, dim = static_cast<int32_t>(p.a.dim);
    const int32_t cols = min(kGroupCols, dim - c0);
    Pieces q;
    if (!find_pieces(p, tile, lane, q)) return;
    const TD* const dout = static_cast<const TD*>(p.a.dout);
    const TD* const end = dout + (p.a.n - 1) * p.a.dout_stride + dim;
    int next = q.a, slot = 0;  // the next row to copy, and its slot
    int32_t pos = q.x.pos;
    const auto issue = [&] {
        if (next < q.e) {
            if (next >= 32 && (next & 31) == 0)
                pos = next + lane < q.count - q.j0 ? (p.w.sorted + q.j0)[next + lane].pos : 0;
            const TD* row = dout + __shfl_sync(0xffffffffu, pos, next & 31) * p.a.dout_stride + c0;
            const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(TD));
            if (lane == 0) starts[warp][slot] = skip;
            uint4* const to = ring[warp][slot];
            const TD* from = row - skip;
            if (from - dout >= 0 && end - from >= W * E) {
                const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to + lane));
#pragma unroll
                for (int k = 0; k < W; k += 32)
                    if ((k + lane) * E < skip + cols)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 16 * k),
                                     "l"(from + (k + lane) * E)
                                     : "memory");
            } else {
                for (int k = lane; k < skip + cols; k += 32)
                    if (k >= skip) reinterpret_cast<TD*>(to)[k] = from[k];
            }
            if (ACC && q.last(next)) {  // the row that the sum is added to, soon
                const TG* g = static_cast<const TG*>(p.a.grad) + c0 +
                              __shfl_sync(0xffffffffu, q.x.token, q.piece_of(next)) * p.a.grad_stride;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(g + min(8 * lane, cols - 1)));
            }
            ++next;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        slot = slot + 1 == D ? 0 : slot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < D; ++i) issue();
    uint64_t acc[1][4] = {{0, 0, 0, 0}};  // packed +0
    uint32_t joins = 0;
#pragma unroll 1
    for (int l = q.a; l < q.e; ++l) {
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
        __syncwarp();
        Shifted<TD> x;
        x.take(ring[warp][slot], lane, starts[warp][slot]);
        __syncwarp();
        issue();
        float f[8];
        x.get(f);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[0][k] = add2(acc[0][k], pk2(f[2 * k], f[2 * k + 1]));
        if (!q.last(l)) continue;
        const int from = q.piece_of(l);
        Chunk<TG> none[1];
        if (end_piece<TG, false, ACC, 1>(p, q, from, slab, lane, acc, none, swap[warp]))
            joins |= 1u << from;
    }
    join_pieces<TG, false, ACC, 1>(p, q, joins, slab, lane, swap[warp]);
}

bool aligned_rows(const void* p, int64_t stride, int32_t dtype) {
    const int64_t size = dtype == ZERO3_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0;
}

template <typename TT, typename TO, bool VEC>
cudaError_t embed_typed(const EmbedArgs& a, cudaStream_t stream) {
    constexpr int NT = 256;
    const int64_t items = a.n * (VEC ? a.dim / 8 : a.dim / 8 + 2);
    // Few units: one per thread, so that they spread over the SMs (64 rows of
    // 4096 bf16 1.5 us, 1.8 at four per thread); many: several, for bytes in flight
    // (8192 x 2047 bf16 at 1 / 2 / 4 shifted units per thread: 15.7 / 15.1 / 16.7 us; by
    // single elements 40 us).
    if (items <= 152 * NT * 4)
        return launch_vocab(embed_kernel<TT, TO, VEC, NT, 1>, (items + NT - 1) / NT, NT, 0, 1, a, stream);
    constexpr int U = VEC ? 4 : 2;
    return launch_vocab(embed_kernel<TT, TO, VEC, NT, U>, (items + NT * U - 1) / (NT * U), NT, 0, 1,
                        a, stream);
}

template <typename TT, typename TO>
cudaError_t embed_vec(const EmbedArgs& a, cudaStream_t stream) {
    const bool vec = a.dim % 8 == 0 && aligned_rows(a.table, a.table_stride, a.table_dtype) &&
                     aligned_rows(a.out, a.out_stride, a.out_dtype);
    return vec ? embed_typed<TT, TO, true>(a, stream) : embed_typed<TT, TO, false>(a, stream);
}

template <typename TD, typename TG, bool VEC, bool ACC, int CU>
cudaError_t sum_launch(const EmbedGradArgs& a, const Workspace& w, cudaStream_t stream) {
    SumArgs p;
    p.a = a;
    p.w = w;
    p.deal = deal_of(a.vocab);
    p.slabs = static_cast<int32_t>((a.dim + kGroupCols * CU - 1) / (kGroupCols * CU));
    // More warps, or fewer with more rows of their own: 8 / 16 rows per warp, 32768 x
    // 2048 50.1 / 51.2 us, 65536 x 768 62.6 / 54.1; 2 / 8: 64 x 64 4.8 / 6.7 us, 512 x
    // 768 8.1 / 8.2, 8192 x 768 22.9 / 20.1.
    p.rows = a.n > 32768 ? 16 : a.n > 512 ? 8 : 2;
    p.sum_blocks = ((a.n + p.rows - 1) / p.rows * p.slabs + kSumWarps - 1) / kSumWarps;
    // Fewer tokens per clearing warp where that leaves SMs without one (1483 rows of
    // 2834 binary32: 6.4 us, 12.6 at 8).
    p.zero_tokens = 8;
    while (p.zero_tokens > 1 && a.vocab < p.zero_tokens * kSumWarps * 304) p.zero_tokens /= 2;
    const int64_t each = kSumWarps * p.zero_tokens;
    const int64_t grid = p.sum_blocks + (ACC ? 0 : (a.vocab + each - 1) / each);
    if constexpr (VEC)
        return launch_vocab(embed_sum_kernel<TD, TG, ACC, CU>, grid, kSumThreads, 0, 1, p, stream);
    else
        return launch_vocab(embed_sum_any_kernel<TD, TG, ACC>, grid, kSumThreads, 0, 1, p, stream);
}

template <typename TD, typename TG, bool VEC, bool ACC>
cudaError_t sum_typed(const EmbedGradArgs& a, const Workspace& w, cudaStream_t stream) {
    // Two groups of columns per lane halve the warps that find pieces and make
    // wider reads, where enough warps are left and few lanes idle: one / two groups,
    // 32768 x 2048 59.6 / 49.4 us, 8192 x 4096 31.7 / 27.9, 8192 x 512 14.9 / 16.7.
    // Binary32 rows are left with too short a ring: 8192 x 2048 41 / 48 us.
    if constexpr (VEC && sizeof(TD) == 2)
        if (a.n * a.dim >= 1 << 24 && (a.dim % (2 * kGroupCols) == 0 || a.dim >= 8 * kGroupCols))
            return sum_launch<TD, TG, VEC, ACC, 2>(a, w, stream);
    return sum_launch<TD, TG, VEC, ACC, 1>(a, w, stream);
}

template <typename TD, typename TG>
cudaError_t sum_vec(const EmbedGradArgs& a, const Workspace& w, cudaStream_t stream) {
    const bool vec = a.dim % 8 == 0 && aligned_rows(a.dout, a.dout_stride, a.dout_dtype) &&
                     aligned_rows(a.grad, a.grad_stride, a.grad_dtype);
    if (a.accumulate)
        return vec ? sum_typed<TD, TG, true, true>(a, w, stream)
                   : sum_typed<TD, TG, false, true>(a, w, stream);
    return vec ? sum_typed<TD, TG, true, false>(a, w, stream)
               : sum_typed<TD, TG, false, false>(a, w, stream);
}

template <int W, int J>
cudaError_t sort_launch(const SortArgs& s, int64_t grid, cudaStream_t stream) {
    constexpr int bytes = sizeof(SortShared<W>);
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel<W, J>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    return launch_vocab(embed_sort_kernel<W, J>, grid, 32 * W, bytes, 1, s, stream);
}

}  // namespace

int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim) {
    return workspace_of(nullptr, n, vocab, dim).bytes;
}

cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t stream) {
    if (a.table_dtype == ZERO3_F32)
        return a.out_dtype == ZERO3_F32 ? embed_vec<float, float>(a, stream)
                                        : embed_vec<float, uint16_t>(a, stream);
    return a.out_dtype == ZERO3_F32 ? embed_vec<uint16_t, float>(a, stream)
                                    : embed_vec<uint16_t, uint16_t>(a, stream);
}

cudaError_t launch_embed_grad(const EmbedGradArgs& a, cudaStream_t stream) {
    SortArgs s;
    s.ids = a.ids;
    s.w = workspace_of(a.workspace, a.n, a.vocab, a.dim);
    s.n = a.n;
    s.vocab = static_cast<int32_t>(a.vocab);
    s.id64 = a.id64;
    s.deal = deal_of(a.vocab);
    const int64_t grid = int64_t{1} << s.deal.shift;
    cudaError_t e;
    // Warps per block: each reads its part of all ids one batch after the other, but
    // every warp's counts are summed up.  8 / 16 warps: 512 tokens 8.3 / 8.9 us (768
    // columns), 4096 15.4 / 14.8 (64); 16 / 32: 2048 13.8 / 15.1 (64), 8192 22.5 / 20.7 (768).
    if (a.n <= 1024)
        e = sort_launch<8, 4>(s, grid, stream);
    else if (a.n <= 4096)
        e = sort_launch<16, 8>(s, grid, stream);
    else
        e = sort_launch<32, 8>(s, grid, stream);
    if (e != cudaSuccess) return e;
    if (a.dout_dtype == ZERO3_F32)
        return a.grad_dtype == ZERO3_F32 ? sum_vec<float, float>(a, s.w, stream)
                                         : sum_vec<float, uint16_t>(a, s.w, stream);
    return a.grad_dtype == ZERO3_F32 ? sum_vec<uint16_t, float>(a, s.w, stream)
                                     : sum_vec<uint16_t, uint16_t>(a, s.w, stream);
}

}  // namespace z3
