// Packing a tensor into the 8-bit checkpoint of checkpoint.cuh, and reading one back.
//
// pack:   codes[row][i], scales[row][i / 32]  from x[row][i]
// unpack: out[b][c][l] = gamma[c] * (code * step) + beta[c], or code * step without them.
//
// Both only move bytes (1 + 1/32 for the checkpoint and 2 or 4 for the tensor, a value).
#include "checkpoint.cuh"

namespace dcn1d {

namespace {

// One warp a block of 32 values, a value a lane.
template <class T>
__global__ void __launch_bounds__(256) pack_kernel(const T *__restrict__ x, int8_t *codes,
                                                   uint8_t *scales, int64_t blocks, int64_t nb,
                                                   int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t j = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; j < blocks; j += step) {
        const int64_t row = j / nb, i = (j - row * nb) * kCkBlock + lane;
        const float v = i < n ? ld_f32(x + row * n + i) : 0.0f;
        const uint32_t s = ck_scale(__reduce_max_sync(0xFFFFFFFFu, ck_abs_bits(v)), ck_top<T>());
        if (i < n)
            codes[row * n + i] = (int8_t)ck_code(v, ck_inverse(s));
        if (lane == 0)
            scales[j] = (uint8_t)s;
    }
}

// One thread a value; `channel` of row r, value i: r % C when rows run along L, else i.
template <class T>
__global__ void __launch_bounds__(256) unpack_kernel(const int8_t *__restrict__ codes,
                                                     const uint8_t *__restrict__ scales,
                                                     const T *gamma, const T *beta, T *out,
                                                     int64_t total, int64_t nb, int64_t n, int C,
                                                     bool along_c) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += step) {
        const int64_t row = t / n, i = t - row * n;
        float v = (float)codes[t] * ck_step(scales[row * nb + i / kCkBlock]);
        const int c = along_c ? (int)i : (int)(row % C);
        if (gamma)
            v = __fmul_rn(v, ld_f32(gamma + c));
        if (beta)
            v = __fadd_rn(v, ld_f32(beta + c));
        out[t] = from_f32<T>(v);
    }
}

unsigned grid_for(int64_t want) {
    const int64_t sms = sm_count_or(148);
    return (unsigned)(want < sms * 8 ? (want > 0 ? want : 1) : sms * 8);
}

template <class T>
void pack(const CkProblem &P, cudaStream_t s) {
    const int64_t n = P.along_c() ? P.C : P.L, nb = ck_blocks(n);
    const int64_t blocks = (P.along_c() ? P.B : P.B * P.C) * nb;
    pack_kernel<T><<<grid_for((blocks + 7) / 8), 256, 0, s>>>(
        static_cast<const T *>(P.in), static_cast<int8_t *>(P.codes),
        static_cast<uint8_t *>(P.scales), blocks, nb, n);
}

template <class T>
void unpack(const CkProblem &P, cudaStream_t s) {
    const int64_t n = P.along_c() ? P.C : P.L, nb = ck_blocks(n);
    const int64_t total = P.B * P.C * P.L;
    unpack_kernel<T><<<grid_for((total + 255) / 256), 256, 0, s>>>(
        static_cast<const int8_t *>(P.codes), static_cast<const uint8_t *>(P.scales),
        static_cast<const T *>(P.gamma), static_cast<const T *>(P.beta), static_cast<T *>(P.out),
        total, nb, n, (int)P.C, P.along_c());
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CkProblem &P, cudaStream_t s) {
    if (P.dtype == DCN1D_BF16)
        pack<__nv_bfloat16>(P, s);
    else if (P.dtype == DCN1D_F16)
        pack<__half>(P, s);
    else
        pack<float>(P, s);
    return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const CkProblem &P, cudaStream_t s) {
    if (P.dtype == DCN1D_BF16)
        unpack<__nv_bfloat16>(P, s);
    else if (P.dtype == DCN1D_F16)
        unpack<__half>(P, s);
    else
        unpack<float>(P, s);
    return cudaGetLastError();
}

}  // namespace dcn1d
