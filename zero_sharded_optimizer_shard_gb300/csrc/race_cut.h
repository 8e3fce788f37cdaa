// Which bytes a race's wide loads may touch: plain C++, so that every case of it can be
// checked without a GPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define Z3_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define Z3_HOST_DEVICE inline
#endif

namespace z3 {

// The tokens [head, head + 8 * chunks) of a row that a race takes in chunks of 8.
struct RaceCut {
    int32_t head, chunks;
};

// `head` and `chunks`: the row's cut at 16-byte boundaries of its logits.  The noise of
// token `head` lies `phase` elements (0 to 3) behind a 16-byte boundary, and a chunk's
// noise is read by the aligned blocks of 4 that hold it: `phase` elements before it
// and 4 - phase behind it come along.  A chunk whose blocks would reach outside the noise of
// the row, which may be all that the caller owns, is left to the ends: at most 15
// tokens on either side.
Z3_HOST_DEVICE RaceCut race_cut(int32_t head, int32_t chunks, int phase, int32_t vocab) {
    RaceCut c{head, chunks};
    if (phase == 0) return c;
    if (c.chunks > 0 && c.head < phase) {
        c.head += 8;
        --c.chunks;
    }
    if (c.chunks > 0 && vocab - c.head - 8 * c.chunks < 4 - phase) --c.chunks;
    return c;
}

// The token at the ends of the row, [0, first) and [last, vocab), that lane 0 to 31 has,
// or -1.
Z3_HOST_DEVICE int32_t end_token(int lane, int32_t first, int32_t last, int32_t vocab) {
    if (lane < 16) return lane < first ? lane : -1;
    return last + (lane - 16) < vocab ? last + (lane - 16) : -1;
}

// Whether the 4 bytes that hold a 16-bit logit lie in its row: `upper`, it is the upper
// half of them.
Z3_HOST_DEVICE bool word_in_row(bool upper, int32_t token, int32_t vocab) {
    return upper ? token > 0 : token + 1 < vocab;
}

}  // namespace z3
