// Where the simple layer norm kernels (norm.cu) read and write, for any sizes: plain integer
// functions that compile for the host too, so that a test can walk them at sizes whose offsets
// pass 32 bits.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DCN1D_HD __host__ __device__ __forceinline__
#else
#define DCN1D_HD inline
#endif

namespace dcn1d {

constexpr int kAnyThreads = 256;

// Lanes along the positions: a power of two up to 32.
DCN1D_HD int lanes_along(int64_t L) {
    int TL = 1;
    while (TL < 32 && TL < L)
        TL *= 2;
    return TL;
}

// A block takes TL consecutive positions of one b; thread i has position i % TL of them and
// channels i / TL, i / TL + rows, ...
struct AnyIndex {
    int64_t C, L, tiles;   // tiles: of one b
    int TL;
    DCN1D_HD AnyIndex(int64_t C_, int64_t L_, int TL_)
        : C(C_), L(L_), tiles((L_ + TL_ - 1) / TL_), TL(TL_) {}
    DCN1D_HD int rows() const { return kAnyThreads / TL; }
    DCN1D_HD int64_t b_of(int64_t tile) const { return tile / tiles; }
    DCN1D_HD int64_t l_of(int64_t tile, int thread) const {
        return (tile - tile / tiles * tiles) * TL + (thread & (TL - 1));
    }
    // of x, y, grad_y, grad_x and the codes
    DCN1D_HD int64_t value(int64_t b, int64_t c, int64_t l) const { return (b * C + c) * L + l; }
    // of mean and rstd
    DCN1D_HD int64_t stat(int64_t b, int64_t l) const { return b * L + l; }
    // of the checkpoint's steps: blocks of 32 along the positions, or the channels of L == 1
    DCN1D_HD int64_t step(int64_t b, int64_t c, int64_t l) const {
        return L == 1 ? b * ((C + 31) / 32) + c / 32 : (b * C + c) * ((L + 31) / 32) + l / 32;
    }
    // of a block's partial sums of grad_gamma; grad_beta's are C further on
    DCN1D_HD int64_t part(int64_t block) const { return block * 2 * C; }
};

}  // namespace dcn1d
