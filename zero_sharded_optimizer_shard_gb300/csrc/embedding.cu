// Embedding lookup with scaling, and its gradient by sorted tokens (sm_103a).
#include <cuda_runtime.h>

#include <cstdint>

#include "vocab_common.cuh"

namespace z3 {
namespace {

// ------------------------------------------------------------------ lookup
// out[i] = rne(scale * table[ids[i]]), zeros where the id lies outside the
// vocabulary.  A copy of n random rows: bound by HBM (the row reads, of
// which repeated tokens hit L2, and the writes).  The n rows' units (chunks of
// 8 columns, or single columns where rows are not 16-byte aligned) are
// numbered consecutively; a block takes NT * U of them, a thread U, NT apart,
// with all of its row loads in flight before its first store.
template <typename TT, typename TO, bool VEC, int NT, int U>
__global__ void __launch_bounds__(NT) embed_kernel(const __grid_constant__ EmbedArgs a) {
    wait_prior_grids();
    allow_next_grid();
    const uint32_t units = static_cast<uint32_t>(VEC ? a.dim / 8 : a.dim);  // per row
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
    if (VEC) {
        Chunk<TT> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u].fill(0.0f);
            if (id[u] >= 0) c[u].load(table + id[u] * a.table_stride + 8ll * at[u]);
        }
        const uint64_t sc = pk2(a.scale, a.scale);
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
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = id[u] >= 0 ? to_f32(table[id[u] * a.table_stride + at[u]]) : 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row[u] < static_cast<uint64_t>(a.n))
                out[row[u] * a.out_stride + at[u]] =
                    from_f32<TO>(id[u] >= 0 ? __fmul_rn(x[u], a.scale) : 0.0f);
    }
}

// ---------------------------------------------------------------- gradient
// grad[v] = rne(base + scale * sum over the positions i of token v, in
// ascending order, of dout[i]), in two launches: a stable counting sort of
// the positions by token, and the rows' sums.
//
// Sums are binary32 and their order depends on the tokens alone, so the
// result does not depend on timing.  A token with at most kLight positions is
// summed by one warp (per slab of columns).  One with more is cut into tiles
// of kTile positions, a block each, whose warps' sums are joined in shared
// memory in order; the tiles' sums are joined in order by whichever block
// comes last.  Tile t of the token whose positions start at sorted index s
// has slot ceil(s / kLight) + t: every slot j of a token lies inside the
// token's own range of sorted indices (64 j), so no two share one and a block
// finds its tile from the sorted index 64 j alone.
constexpr int kLight = 64;
constexpr int kTile = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kOwn = 352;  // tokens a sorting block owns at most
constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSlabMin = 256;  // narrowest slab of columns

struct Workspace {
    int32_t* off;      // [vocab + 1] first sorted index of each token
    int32_t* perm;     // [n] positions by token, ascending
    int32_t* arrived;  // [slots * slabs] tiles of a token that are done
    float* partial;    // [slots * dim] tile sums
    int64_t slots, arrivals, bytes;
};

__host__ __device__ inline int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }

__host__ __device__ inline Workspace workspace_of(void* base, int64_t n, int64_t vocab,
                                                  int64_t dim) {
    Workspace w;
    w.slots = n / kLight + 1;
    w.arrivals = w.slots * ((dim + kSlabMin - 1) / kSlabMin);
    char* p = static_cast<char*>(base);
    int64_t o = 0;
    w.off = reinterpret_cast<int32_t*>(p + o);
    o += up16(4 * (vocab + 1));
    w.perm = reinterpret_cast<int32_t*>(p + o);
    o += up16(4 * n);
    w.arrived = reinterpret_cast<int32_t*>(p + o);
    o += up16(4 * w.arrivals);
    w.partial = reinterpret_cast<float*>(p + o);
    o += 4 * w.slots * ((dim + 3) / 4 * 4);
    w.bytes = o;
    return w;
}

struct SortArgs {
    const void* ids;
    Workspace w;
    int64_t n;
    int32_t vocab, own, id64;
};

// Stable counting sort without communication between blocks: every block
// reads all ids, counts those below its own range of tokens (which gives the
// range's first sorted index) and, warp by warp, those of each own token;
// then each warp places its positions in order.
__global__ void __launch_bounds__(kSortThreads)
    embed_sort_kernel(const __grid_constant__ SortArgs a) {
    __shared__ int32_t cnt[kSortWarps][kOwn];
    __shared__ int32_t sh[kSortWarps], sh_scan[kSortWarps];
    wait_prior_grids();
    allow_next_grid();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t v0 = blockIdx.x * a.own;
    const int32_t own = min(a.own, a.vocab - v0);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; i < a.w.arrivals;
         i += static_cast<int64_t>(gridDim.x) * kSortThreads)
        a.w.arrived[i] = 0;
    for (int i = tid; i < kSortWarps * kOwn; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
    const int64_t per = (a.n + kSortThreads - 1) / kSortThreads * 32;
    const int64_t i0 = per * warp, i1 = i0 + per < a.n ? i0 + per : a.n;
    int32_t less = 0;
#pragma unroll 4
    for (int64_t i = i0 + lane; i < i1; i += 32) {
        const int32_t id = load_id(a.ids, a.id64, i, a.vocab);
        less += id >= 0 && id < v0;
        const int32_t k = id - v0;
        if (id >= v0 && k < own) atomicAdd(&cnt[warp][k], 1);
    }
    for (int o = 16; o > 0; o >>= 1) less += __shfl_xor_sync(0xffffffffu, less, o);
    if (lane == 0) sh[warp] = less;
    __syncthreads();
    // exclusive scan over the own tokens' totals, one token per thread
    int32_t total = 0;
    if (tid < own)
        for (int w = 0; w < kSortWarps; ++w) total += cnt[w][tid];
    int32_t incl = total;
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sh_scan[warp] = incl;
    __syncthreads();
    int32_t run = incl - total;
    for (int w = 0; w < kSortWarps; ++w) {
        run += sh[w];
        if (w < warp) run += sh_scan[w];
    }
    if (tid < own) {
        a.w.off[v0 + tid] = run;
        if (v0 + tid == a.vocab - 1) a.w.off[a.vocab] = run + total;
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = cnt[w][tid];
            cnt[w][tid] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int64_t b = i0; b < i1; b += 32) {
        const int64_t i = b + lane;
        const int32_t id = i < i1 ? load_id(a.ids, a.id64, i, a.vocab) : -1;
        const int32_t k = id - v0;
        const bool in = id >= v0 && k < own;
        if (!__any_sync(0xffffffffu, in)) continue;
        const uint32_t peers = __match_any_sync(0xffffffffu, in ? k : -1);
        const int rank = __popc(peers & ((1u << lane) - 1u));
        if (in) a.w.perm[cnt[warp][k] + rank] = static_cast<int32_t>(i);
        __syncwarp();
        if (in && rank == 0) cnt[warp][k] += __popc(peers);
        __syncwarp();
    }
}

struct SumArgs {
    EmbedGradArgs a;
    Workspace w;
    int32_t slabs;
    int64_t heavy_blocks;
};

// A lane's columns of a slab: CU chunks of 8, 32 chunks apart (VEC), or 8 CU
// single columns, 32 apart.
template <typename TD, bool VEC, int CU>
struct Columns {
    float acc[8 * CU];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < 8 * CU; ++k) acc[k] = 0.0f;
    }
    // column of acc[k]
    static __device__ __forceinline__ int32_t col(int32_t c0, int lane, int k) {
        return VEC ? c0 + 8 * (lane + 32 * (k / 8)) + k % 8 : c0 + lane + 32 * k;
    }
    // adds rows perm[s..e) in order
    __device__ __forceinline__ void add_rows(const SumArgs& p, int32_t s, int32_t e, int32_t c0,
                                             int lane) {
        const TD* dout = static_cast<const TD*>(p.a.dout);
        const int32_t dim = static_cast<int32_t>(p.a.dim);
        constexpr int R = VEC ? 2 : 4;  // rows in flight
        for (int32_t b = s; b < e; b += 32) {
            const int n = min(32, e - b);
            const int32_t mine = lane < n ? p.w.perm[b + lane] : 0;
            int j = 0;
            for (; j + R <= n; j += R) rows<R>(dout, p.a.dout_stride, mine, j, c0, lane, dim);
            for (; j < n; ++j) rows<1>(dout, p.a.dout_stride, mine, j, c0, lane, dim);
        }
    }
    template <int R>
    __device__ __forceinline__ void rows(const TD* dout, int64_t stride, int32_t mine, int j,
                                         int32_t c0, int lane, int32_t dim) {
        const TD* row[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            row[r] = dout + __shfl_sync(0xffffffffu, mine, j + r) * stride;
        if (VEC) {
            Chunk<TD> c[R][CU];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < CU; ++u) {
                    const int32_t at = c0 + 8 * (lane + 32 * u);
                    c[r][u].fill(0.0f);
                    if (at < dim) c[r][u].load_stream(row[r] + at);
                }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < CU; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x, y;
                        upk2(c[r][u].pair(k), x, y);
                        acc[8 * u + 2 * k] = __fadd_rn(acc[8 * u + 2 * k], x);
                        acc[8 * u + 2 * k + 1] = __fadd_rn(acc[8 * u + 2 * k + 1], y);
                    }
        } else {
            float x[R][8 * CU];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < 8 * CU; ++k) {
                    const int32_t at = c0 + lane + 32 * k;
                    x[r][k] = at < dim ? to_f32(row[r][at]) : 0.0f;
                }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < 8 * CU; ++k) acc[k] = __fadd_rn(acc[k], x[r][k]);
        }
    }
};

// grad[v][col] = rne(base + scale * x)
template <typename TG>
__device__ __forceinline__ void put(const SumArgs& p, int32_t v, int32_t col, float x) {
    if (col >= p.a.dim) return;
    TG* g = static_cast<TG*>(p.a.grad) + v * p.a.grad_stride + col;
    *g = from_f32<TG>(p.a.accumulate ? fmaf(x, p.a.scale, to_f32(*g)) : __fmul_rn(x, p.a.scale));
}

template <typename TD, typename TG, bool VEC, int CU>
__device__ __forceinline__ void put_row(const SumArgs& p, int32_t v, int32_t c0, int lane,
                                        const Columns<TD, VEC, CU>& s) {
    using Col = Columns<TD, VEC, CU>;
    if (!VEC) {
#pragma unroll
        for (int k = 0; k < 8 * CU; ++k) put<TG>(p, v, Col::col(c0, lane, k), s.acc[k]);
        return;
    }
    TG* g = static_cast<TG*>(p.a.grad) + v * p.a.grad_stride;
    Chunk<TG> old[CU];
    if (p.a.accumulate) {
#pragma unroll
        for (int u = 0; u < CU; ++u) {
            const int32_t at = c0 + 8 * (lane + 32 * u);
            if (at < p.a.dim) old[u].load_stream(g + at);
        }
    }
#pragma unroll
    for (int u = 0; u < CU; ++u) {
        const int32_t at = c0 + 8 * (lane + 32 * u);
        if (at >= p.a.dim) continue;
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float x = 0.0f, y = 0.0f;
            if (p.a.accumulate) {
                upk2(old[u].pair(k), x, y);
                f[2 * k] = fmaf(s.acc[8 * u + 2 * k], p.a.scale, x);
                f[2 * k + 1] = fmaf(s.acc[8 * u + 2 * k + 1], p.a.scale, y);
            } else {
                f[2 * k] = __fmul_rn(s.acc[8 * u + 2 * k], p.a.scale);
                f[2 * k + 1] = __fmul_rn(s.acc[8 * u + 2 * k + 1], p.a.scale);
            }
        }
        Chunk<TG>::store(g + at, f);
    }
}

template <typename TD, typename TG, bool VEC, int CU>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ SumArgs p) {
    constexpr int W = 256 * CU;  // columns of a slab
    __shared__ float sh[kSumWarps][W];
    __shared__ int sh_last;
    wait_prior_grids();
    allow_next_grid();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Columns<TD, VEC, CU> s;
    s.clear();
    const int32_t* off = p.w.off;
    if (blockIdx.x >= p.heavy_blocks) {  // one token per warp
        const int64_t b = blockIdx.x - p.heavy_blocks;
        const int64_t v = b / p.slabs * kSumWarps + warp;
        const int32_t c0 = static_cast<int32_t>(b % p.slabs) * W;
        if (v >= p.a.vocab) return;
        const int32_t s0 = off[v], e0 = off[v + 1];
        if (e0 - s0 > kLight || (e0 == s0 && p.a.accumulate)) return;
        s.add_rows(p, s0, e0, c0, lane);
        put_row<TD, TG, VEC, CU>(p, static_cast<int32_t>(v), c0, lane, s);
        return;
    }
    // one tile of a token with many positions
    const int32_t slot = static_cast<int32_t>(blockIdx.x / p.slabs);
    const int32_t slab = static_cast<int32_t>(blockIdx.x % p.slabs);
    const int32_t c0 = slab * W;
    const int64_t at = static_cast<int64_t>(slot) * kLight;
    if (at >= off[p.a.vocab]) return;
    const int32_t v = load_id(p.a.ids, p.a.id64, p.w.perm[at], p.a.vocab);
    const int32_t s0 = off[v], e0 = off[v + 1];
    const int32_t first = (s0 + kLight - 1) / kLight, tile = slot - first;
    const int32_t tiles = (e0 - s0 + kTile - 1) / kTile;
    if (e0 - s0 <= kLight || tile >= tiles) return;
    const int32_t t0 = s0 + tile * kTile, t1 = min(t0 + kTile, e0);
    constexpr int kRows = kTile / kSumWarps;
    const int32_t r0 = min(t0 + warp * kRows, t1), r1 = min(r0 + kRows, t1);
    s.add_rows(p, r0, r1, c0, lane);
#pragma unroll
    for (int k = 0; k < 8 * CU; ++k)
        sh[warp][Columns<TD, VEC, CU>::col(0, lane, k)] = s.acc[k];
    __syncthreads();
    float* part = p.w.partial + static_cast<int64_t>(slot) * ((p.a.dim + 3) / 4 * 4);
    for (int i = tid; i < W; i += kSumThreads) {
        float x = sh[0][i];
#pragma unroll
        for (int w = 1; w < kSumWarps; ++w) x = __fadd_rn(x, sh[w][i]);
        if (tiles == 1)
            put<TG>(p, v, c0 + i, x);
        else if (c0 + i < p.a.dim)
            part[c0 + i] = x;
    }
    if (tiles == 1) return;
    __threadfence();
    __syncthreads();
    if (tid == 0)
        sh_last = atomicAdd(&p.w.arrived[static_cast<int64_t>(first) * p.slabs + slab], 1) == tiles - 1;
    __syncthreads();
    if (!sh_last) return;
    __threadfence();
    const int64_t step = (p.a.dim + 3) / 4 * 4;
    const float* all = p.w.partial + static_cast<int64_t>(first) * step;
    for (int i = tid; i < W; i += kSumThreads) {
        if (c0 + i >= p.a.dim) continue;
        float x = 0.0f;
#pragma unroll 8
        for (int32_t t = 0; t < tiles; ++t) x = __fadd_rn(x, __ldcg(all + t * step + c0 + i));
        put<TG>(p, v, c0 + i, x);
    }
}

bool aligned_rows(const void* p, int64_t stride, int32_t dtype) {
    const int64_t size = dtype == ZERO3_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0;
}

template <typename TT, typename TO, bool VEC>
cudaError_t embed_typed(const EmbedArgs& a, cudaStream_t stream) {
    constexpr int NT = 256;
    const int64_t items = a.n * (VEC ? a.dim / 8 : a.dim);
    // few units: one per thread, so that they spread over the SMs
    if (items <= 152 * NT * 4)
        return launch_vocab(embed_kernel<TT, TO, VEC, NT, 1>, (items + NT - 1) / NT, NT, 0, 1, a, stream);
    constexpr int U = VEC ? 4 : 8;
    return launch_vocab(embed_kernel<TT, TO, VEC, NT, U>, (items + NT * U - 1) / (NT * U), NT, 0, 1,
                        a, stream);
}

template <typename TT, typename TO>
cudaError_t embed_vec(const EmbedArgs& a, cudaStream_t stream) {
    const bool vec = a.dim % 8 == 0 && aligned_rows(a.table, a.table_stride, a.table_dtype) &&
                     aligned_rows(a.out, a.out_stride, a.out_dtype);
    return vec ? embed_typed<TT, TO, true>(a, stream) : embed_typed<TT, TO, false>(a, stream);
}

template <typename TD, typename TG, bool VEC, int CU>
cudaError_t sum_typed(const EmbedGradArgs& a, const Workspace& w, cudaStream_t stream) {
    SumArgs p;
    p.a = a;
    p.w = w;
    p.slabs = static_cast<int32_t>((a.dim + 256 * CU - 1) / (256 * CU));
    p.heavy_blocks = a.n > kLight ? w.slots * p.slabs : 0;
    const int64_t grid = p.heavy_blocks + (a.vocab + kSumWarps - 1) / kSumWarps * p.slabs;
    return launch_vocab(embed_sum_kernel<TD, TG, VEC, CU>, grid, kSumThreads, 0, 1, p, stream);
}

template <typename TD, typename TG>
cudaError_t sum_vec(const EmbedGradArgs& a, const Workspace& w, cudaStream_t stream) {
    const bool vec = a.dim % 8 == 0 && aligned_rows(a.dout, a.dout_stride, a.dout_dtype) &&
                     aligned_rows(a.grad, a.grad_stride, a.grad_dtype);
    if (!vec) return sum_typed<TD, TG, false, 1>(a, w, stream);
    if (a.dim <= 256) return sum_typed<TD, TG, true, 1>(a, w, stream);
    if (a.dim <= 512) return sum_typed<TD, TG, true, 2>(a, w, stream);
    return sum_typed<TD, TG, true, 4>(a, w, stream);
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
    const int64_t each = (a.vocab + 151) / 152;
    s.own = static_cast<int32_t>(each < 32 ? 32 : each > kOwn ? kOwn : each);
    const int64_t grid = (a.vocab + s.own - 1) / s.own;
    const cudaError_t e = launch_vocab(embed_sort_kernel, grid, kSortThreads, 0, 1, s, stream);
    if (e != cudaSuccess) return e;
    if (a.dout_dtype == ZERO3_F32)
        return a.grad_dtype == ZERO3_F32 ? sum_vec<float, float>(a, s.w, stream)
                                         : sum_vec<float, uint16_t>(a, s.w, stream);
    return a.grad_dtype == ZERO3_F32 ? sum_vec<uint16_t, float>(a, s.w, stream)
                                     : sum_vec<uint16_t, uint16_t>(a, s.w, stream);
}

}  // namespace z3
