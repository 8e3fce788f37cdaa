// Device helpers shared by the streaming kernels (kernels.cu) and the piece
// kernel (pieces.cu): block size, programmatic dependent launch, bf16
// conversion and packing, streaming 16-byte accesses, the launch helper.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace z3 {
namespace {

constexpr int kThreads = 256;

// Programmatic dependent launch.  Every kernel of this library is launched with
// programmatic stream serialization, so it may be scheduled while the
// previous kernel of the stream drains.  Each thread therefore waits for the
// previous grids to complete (and their writes to become visible) before its
// first memory access, which keeps plain stream order for the data; what
// overlaps is the launch and block dispatch of this grid with the previous
// grid's tail.  Without a programmatic predecessor the wait returns at once.
__device__ __forceinline__ void wait_prior_grids() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next programmatic launch of the stream be scheduled.
__device__ __forceinline__ void allow_next_grid() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_f32(uint16_t h) {
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

// Two binary32 values -> packed bf16 pair, round to nearest even (hardware
// conversion); `lo` lands in bits 0..15.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint16_t to_bf16(float x) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
    return r;
}

// Streaming (evict-first) 16-byte accesses: every byte is touched once.
__device__ __forceinline__ uint4 ldcs16(const void* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void stcs16(void* p, uint4 x) { __stcs(reinterpret_cast<uint4*>(p), x); }

__device__ __forceinline__ void unpack8(const uint4& r, float* f) {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x);
    f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z);
    f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                      pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The 8 bf16 values at elements ph..ph+7 (1 <= ph <= 7) of the 16-element
// window formed by two consecutive aligned 16-byte blocks b0, b1 (window
// words w0..w7).  Branch-free, so the compiler keeps every rank's loads
// ahead of the first realignment: result word m is the funnel shift of
// words k+m and k+m+1 (k = ph / 2) right by 16 * (ph & 1) bits, the words
// picked by two rounds of selects (by 2 words, then by 1).
__device__ __forceinline__ uint4 realign8(const uint4& b0, const uint4& b1, int ph) {
    const bool by2 = (ph & 4) != 0, by1 = (ph & 2) != 0;
    const uint32_t sh = static_cast<uint32_t>(ph & 1) * 16u;
    const uint32_t t0 = by2 ? b0.z : b0.x, t1 = by2 ? b0.w : b0.y, t2 = by2 ? b1.x : b0.z;
    const uint32_t t3 = by2 ? b1.y : b0.w, t4 = by2 ? b1.z : b1.x, t5 = by2 ? b1.w : b1.y;
    const uint32_t v0 = by1 ? t1 : t0, v1 = by1 ? t2 : t1, v2 = by1 ? t3 : t2;
    const uint32_t v3 = by1 ? t4 : t3, v4 = by1 ? t5 : t4;
    return make_uint4(__funnelshift_r(v0, v1, sh), __funnelshift_r(v1, v2, sh),
                      __funnelshift_r(v2, v3, sh), __funnelshift_r(v3, v4, sh));
}

// 8 consecutive bf16 values at p, element phase ph != 0, read as the two
// aligned 16-byte blocks around them (through the read-only path, so the
// block a neighbouring thread also reads is served from L1).  The caller
// guarantees that both blocks lie inside the valid range: the 8 elements
// before p and the 16 from p on.
__device__ __forceinline__ uint4 ld8_window(const uint16_t* p, int ph) {
    const uint16_t* a = p - ph;
    const uint4 b0 = __ldg(reinterpret_cast<const uint4*>(a));
    const uint4 b1 = __ldg(reinterpret_cast<const uint4*>(a + 8));
    return realign8(b0, b1, ph);
}

// Launch with programmatic stream serialization (see wait_prior_grids).  What the
// launch itself returned is the call's result; the thread's last error may be an
// earlier call's.
template <typename Args>
cudaError_t launch_programmatic(void (*kernel)(Args), int grid, const Args& a,
                                cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
}  // namespace z3
