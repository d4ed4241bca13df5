// Packing a tensor into the 8-bit checkpoint of checkpoint.cuh, and reading one back.
//
// pack:   codes[row][i], scales[row][i / 32]  from x[row][i]
// unpack: out[b][c][l] = gamma[c] * (code * step) + beta[c], or code * step without them.
//
// Both only move bytes (1 + 1/32 for the checkpoint and 2 or 4 for the tensor, a value).  A
// thread works on kMany blocks of 32 values, spread over the grid, with all their loads in
// flight; where rows are aligned a block is 32 / V lanes of 16 bytes, else 32 lanes of one
// value.  The index type is 32 bits while the number of blocks allows: a 64-bit division a
// block costs more than the rest of the work.
#include "checkpoint.cuh"
#include "pairs.cuh"

namespace dcn1d {

namespace {

constexpr int kThreads = 256, kMany = 4;

// Blocks blockIdx.x * per_cta + ..., one for each group of `LANES` lanes, then a grid's
// further on, kMany of them.
template <class I, int LANES>
struct Blocks {
    I first, step;
    __device__ Blocks() {
        constexpr int PER_CTA = kThreads / LANES;
        first = (I)blockIdx.x * PER_CTA + threadIdx.x / LANES;
        step = (I)gridDim.x * PER_CTA;
    }
};

template <class T, class I, bool VEC>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T *__restrict__ x, int8_t *codes,
                                                        uint8_t *scales, I blocks, I nb,
                                                        int64_t n) {
    constexpr int V = VEC ? Vec<T>::V : 1, LANES = kCkBlock / V;
    const int part = threadIdx.x % LANES;
    const Blocks<I, LANES> at;
    // Whole warps walk together for the shuffles: the bound is the warp's first block.
    for (I j0 = at.first; j0 - (threadIdx.x % 32) / LANES < blocks; j0 += at.step * kMany) {
        uint4 u[kMany];
        float f[kMany];
        int64_t where[kMany];
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            const I j = j0 + q * at.step, row = j / nb;
            const int64_t i = (int64_t)(j - row * nb) * kCkBlock + part * V;
            where[q] = j < blocks && i < n ? (int64_t)row * n + i : -1;
            if constexpr (VEC)
                u[q] = where[q] >= 0 ? __ldcs(reinterpret_cast<const uint4 *>(x + where[q]))
                                     : make_uint4(0, 0, 0, 0);
            else
                f[q] = where[q] >= 0 ? ld_f32(x + where[q]) : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            const I j = j0 + q * at.step;
            if constexpr (VEC) {
                constexpr int H = Vec<T>::H;
                Pair p[H];
                chunk_to_pairs<T>(u[q], p);
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    const float2 a = halves(p[k]);
                    top = max(top, max(ck_abs_bits(a.x), ck_abs_bits(a.y)));
                }
#pragma unroll
                for (int o = 1; o < LANES; o <<= 1)
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const uint32_t s = ck_scale(top, ck_top<T>());
                const float inverse = ck_inverse(s);
                uint32_t w[V / 4];
                // a saturated block (within 0.4 % of the type's largest number) has values
                // past 127 steps
                const Pair inv = twice(inverse), magic = twice(kCkRound);
#pragma unroll
                for (int k = 0; k < H / 2; ++k) {
                    const float2 a = halves(fma2(p[2 * k], inv, magic)),
                                 b = halves(fma2(p[2 * k + 1], inv, magic));
                    auto keep = [](float v) {
                        return fminf(fmaxf(v, kCkRound - 127.0f), kCkRound + 127.0f);
                    };
                    w[k] = inverse == 0.0f ? 0u : ck_low_bytes(keep(a.x), keep(a.y), keep(b.x), keep(b.y));
                }
                if (where[q] >= 0) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2 *>(codes + where[q]) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint32_t *>(codes + where[q]) = w[0];
                    if (part == 0)
                        scales[j] = (uint8_t)s;
                }
            } else {
                const uint32_t s =
                    ck_scale(__reduce_max_sync(0xFFFFFFFFu, ck_abs_bits(f[q])), ck_top<T>());
                if (where[q] >= 0) {
                    codes[where[q]] = (int8_t)ck_code(f[q], ck_inverse(s));
                    if (part == 0)
                        scales[j] = (uint8_t)s;
                }
            }
        }
    }
}

template <class T, class I, bool VEC>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const int8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales,
                                                          const T *gamma, const T *beta, T *out,
                                                          I blocks, I nb, int64_t n, I C,
                                                          bool along_c) {
    constexpr int V = VEC ? Vec<T>::V : 1, LANES = kCkBlock / V;
    const int part = threadIdx.x % LANES;
    const Blocks<I, LANES> at;
    for (I j0 = at.first; j0 < blocks; j0 += at.step * kMany) {
        uint32_t w[kMany][2];
        float step[kMany];
        int64_t where[kMany], channel[kMany];
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            const I j = j0 + q * at.step, row = j / nb;
            const int64_t i = (int64_t)(j - row * nb) * kCkBlock + part * V;
            where[q] = j < blocks && i < n ? (int64_t)row * n + i : -1;
            channel[q] = gamma || beta ? (along_c ? i : (int64_t)(row % C)) : 0;
            w[q][0] = w[q][1] = 0;
            step[q] = 0.0f;
            if (where[q] >= 0) {
                step[q] = ck_step(__ldg(scales + j));
                const int8_t *p = codes + where[q];
                if constexpr (V == 8) {
                    const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p));
                    w[q][0] = u.x;
                    w[q][1] = u.y;
                } else if constexpr (V == 4) {
                    w[q][0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
                } else {
                    w[q][0] = (uint32_t)(int)*p;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            if (where[q] < 0)
                continue;
            float v[V];
            if constexpr (VEC) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    v[k] = (ck_biased(w[q][k / 4] ^ 0x80808080u, k % 4) - kCkBias) * step[q];
            } else {
                v[0] = (float)(int)w[q][0] * step[q];
            }
            if (gamma || beta)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int64_t c = channel[q] + (along_c ? k : 0);
                    if (gamma)
                        v[k] = __fmul_rn(v[k], ld_f32(gamma + c));
                    if (beta)
                        v[k] = __fadd_rn(v[k], ld_f32(beta + c));
                }
            if constexpr (VEC) {
                Pair p[V / 2];
#pragma unroll
                for (int k = 0; k < V / 2; ++k)
                    p[k] = pair(v[2 * k], v[2 * k + 1]);
                *reinterpret_cast<uint4 *>(out + where[q]) = pairs_to_chunk<T>(p);
            } else {
                out[where[q]] = from_f32<T>(v[0]);
            }
        }
    }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows, values and blocks of a row, and the blocks of a launch: eight per SM of 256 threads,
// fewer where there is less to do.
struct Shape {
    int64_t n, nb, blocks;
    explicit Shape(const CkProblem &P) {
        n = P.along_c() ? P.C : P.L;
        nb = ck_blocks(n);
        blocks = (P.along_c() ? P.B : P.B * P.C) * nb;
    }
    unsigned grid(int lanes) const {
        const int64_t want = (blocks * lanes + kThreads * kMany - 1) / (kThreads * kMany);
        const int64_t most = (int64_t)sm_count_or(148) * 8;
        return (unsigned)(want < 1 ? 1 : want < most ? want : most);
    }
    // 32-bit indices: also past the last block by a grid's worth
    bool narrow() const { return blocks < (1LL << 31); }
};

template <class T, class I>
void pack(const CkProblem &P, const Shape &s, cudaStream_t stream) {
    const bool vec = s.n % Vec<T>::V == 0 && aligned(P.in, 16) && aligned(P.codes, Vec<T>::V);
    auto kernel = vec ? pack_kernel<T, I, true> : pack_kernel<T, I, false>;
    kernel<<<s.grid(vec ? kCkBlock / Vec<T>::V : kCkBlock), kThreads, 0, stream>>>(
        static_cast<const T *>(P.in), static_cast<int8_t *>(P.codes),
        static_cast<uint8_t *>(P.scales), (I)s.blocks, (I)s.nb, s.n);
}

template <class T, class I>
void unpack(const CkProblem &P, const Shape &s, cudaStream_t stream) {
    const bool vec = s.n % Vec<T>::V == 0 && aligned(P.out, 16) && aligned(P.codes, Vec<T>::V);
    auto kernel = vec ? unpack_kernel<T, I, true> : unpack_kernel<T, I, false>;
    kernel<<<s.grid(vec ? kCkBlock / Vec<T>::V : kCkBlock), kThreads, 0, stream>>>(
        static_cast<const int8_t *>(P.codes), static_cast<const uint8_t *>(P.scales),
        static_cast<const T *>(P.gamma), static_cast<const T *>(P.beta), static_cast<T *>(P.out),
        (I)s.blocks, (I)s.nb, s.n, (I)P.C, P.along_c());
}

template <class T>
void pack_any(const CkProblem &P, cudaStream_t s) {
    const Shape shape(P);
    shape.narrow() ? pack<T, uint32_t>(P, shape, s) : pack<T, uint64_t>(P, shape, s);
}

template <class T>
void unpack_any(const CkProblem &P, cudaStream_t s) {
    const Shape shape(P);
    shape.narrow() ? unpack<T, uint32_t>(P, shape, s) : unpack<T, uint64_t>(P, shape, s);
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CkProblem &P, cudaStream_t s) {
    if (P.dtype == DCN1D_BF16)
        pack_any<__nv_bfloat16>(P, s);
    else if (P.dtype == DCN1D_F16)
        pack_any<__half>(P, s);
    else
        pack_any<float>(P, s);
    return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const CkProblem &P, cudaStream_t s) {
    if (P.dtype == DCN1D_BF16)
        unpack_any<__nv_bfloat16>(P, s);
    else if (P.dtype == DCN1D_F16)
        unpack_any<__half>(P, s);
    else
        unpack_any<float>(P, s);
    return cudaGetLastError();
}

}  // namespace dcn1d
