// Packing a tensor into the 8-bit checkpoint of checkpoint.cuh, and reading one back.
//
// pack:   codes[row][i], scales[row][i / 32]  from x[row][i]
// unpack: out[b][c][l] = gamma[c] * (code * step) + beta[c], or code * step without them.
//
// Both only move bytes (1 + 1/32 for the checkpoint and 2 or 4 for the tensor, a value).  A
// thread takes V neighbouring values (16 bytes of them; 4 values one by one where rows are
// not aligned) of kMany blocks of 32, spread over the grid, with all their loads in flight.
// The index type is 32 bits while the number of blocks allows: a 64-bit division a block
// costs more than the rest of the work.
//
// Measured (B200): [16, 256, 4096] bf16, 16.8 million values, pack 15 us and unpack 11 us =
// 3.4 and 4.6 TB/s of the bytes above; a value a thread with 64-bit indices took 68 and 48.
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

// Values of a thread's part of a block.
template <class T, bool VEC> constexpr int part_of() { return VEC ? Vec<T>::V : 4; }

template <class T, class I, bool VEC>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T *__restrict__ x, int8_t *codes,
                                                        uint8_t *scales, I blocks, I nb,
                                                        int64_t n) {
    constexpr int V = part_of<T, VEC>(), LANES = kCkBlock / V;
    const int part = threadIdx.x % LANES;
    const Blocks<I, LANES> at;
    // Whole warps walk together for the shuffles: the bound is the warp's first block.
    for (I j0 = at.first; j0 - (threadIdx.x % 32) / LANES < blocks; j0 += at.step * kMany) {
        __align__(16) T u[kMany][V];
        int64_t where[kMany];
        int live[kMany];                       // values of this part inside the row
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            const I j = j0 + q * at.step, row = j / nb;
            const int64_t i = (int64_t)(j - row * nb) * kCkBlock + part * V;
            where[q] = (int64_t)row * n + i;
            live[q] = j < blocks ? (int)max((int64_t)0, min((int64_t)V, n - i)) : 0;
            if constexpr (VEC) {
                const uint4 w = live[q] ? __ldcs(reinterpret_cast<const uint4 *>(x + where[q]))
                                        : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(u[q]) = w;
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    u[q][k] = k < live[q] ? __ldg(x + where[q] + k) : from_f32<T>(0.0f);
            }
        }
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            float v[V];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                v[k] = to_f32(u[q][k]);
                top = max(top, ck_abs_bits(v[k]));
            }
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1)
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const uint32_t s = ck_scale(top, ck_top<T>());
            const float inverse = ck_inverse(s);
            uint32_t w[V / 4];
#pragma unroll
            for (int k = 0; k < V; ++k)        // a saturated block has values past 127 steps
                v[k] = fminf(fmaxf(fmaf(v[k], inverse, kCkRound), kCkRound - 127.0f), kCkRound + 127.0f);
#pragma unroll
            for (int k = 0; k < V / 4; ++k)
                w[k] = inverse == 0.0f ? 0u : ck_low_bytes(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            if (live[q]) {
                if constexpr (!VEC) {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (k < live[q])
                            codes[where[q] + k] = (int8_t)(w[0] >> (8 * k));
                } else if constexpr (V == 8) {
                    *reinterpret_cast<uint2 *>(codes + where[q]) = make_uint2(w[0], w[V / 4 - 1]);
                } else {
                    *reinterpret_cast<uint32_t *>(codes + where[q]) = w[0];
                }
                if (part == 0)
                    scales[j0 + q * at.step] = (uint8_t)s;
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
    constexpr int V = part_of<T, VEC>(), LANES = kCkBlock / V;
    const int part = threadIdx.x % LANES;
    const Blocks<I, LANES> at;
    for (I j0 = at.first; j0 < blocks; j0 += at.step * kMany) {
        uint32_t w[kMany][V / 4];
        float step[kMany];
        int64_t where[kMany], channel[kMany];
        int live[kMany];
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            const I j = j0 + q * at.step, row = j / nb;
            const int64_t i = (int64_t)(j - row * nb) * kCkBlock + part * V;
            where[q] = (int64_t)row * n + i;
            live[q] = j < blocks ? (int)max((int64_t)0, min((int64_t)V, n - i)) : 0;
            channel[q] = gamma || beta ? (along_c ? i : (int64_t)(row % C)) : 0;
            step[q] = 0.0f;
#pragma unroll
            for (int k = 0; k < V / 4; ++k)
                w[q][k] = 0;
            if (live[q]) {
                step[q] = ck_step(__ldg(scales + j));
                const int8_t *p = codes + where[q];
                if constexpr (!VEC) {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (k < live[q])
                            w[q][0] |= (uint32_t)(uint8_t)__ldg(p + k) << (8 * k);
                } else if constexpr (V == 8) {
                    const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p));
                    w[q][0] = u.x;
                    w[q][V / 4 - 1] = u.y;
                } else {
                    w[q][0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            if (!live[q])
                continue;
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = (ck_biased(w[q][k / 4] ^ 0x80808080u, k % 4) - kCkBias) * step[q];
            if (gamma || beta)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (!VEC && k >= live[q])
                        continue;              // along_c: past the last channel
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
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k < live[q])
                        out[where[q] + k] = from_f32<T>(v[k]);
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
    kernel<<<s.grid(kCkBlock / (vec ? part_of<T, true>() : part_of<T, false>())), kThreads, 0, stream>>>(
        static_cast<const T *>(P.in), static_cast<int8_t *>(P.codes),
        static_cast<uint8_t *>(P.scales), (I)s.blocks, (I)s.nb, s.n);
}

template <class T, class I>
void unpack(const CkProblem &P, const Shape &s, cudaStream_t stream) {
    const bool vec = s.n % Vec<T>::V == 0 && aligned(P.out, 16) && aligned(P.codes, Vec<T>::V);
    auto kernel = vec ? unpack_kernel<T, I, true> : unpack_kernel<T, I, false>;
    kernel<<<s.grid(kCkBlock / (vec ? part_of<T, true>() : part_of<T, false>())), kThreads, 0, stream>>>(
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
