// Layer norm over the channels of x [B, C, L], forward and backward.
//
//   mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps),  v = (x - mean) rstd
//   y = gamma[c] v + beta[c]
// and with d = gamma[c] grad_y, A = sum_c d / C, S = sum_c d v / C:
//   grad_x = rstd (d - A - v S)
//   grad_gamma[c] = sum_{b,l} grad_y v,   grad_beta[c] = sum_{b,l} grad_y
//
// The normalised axis is strided by L in memory.  A block takes TL consecutive positions of
// one b (TL a power of two up to 32, at least L where L is shorter); its lanes run along
// them, so a warp covers 32 / TL channels, eight warps eight times that, and the block
// walks all C channels.  With L == 1 the lanes run along the channels.
#include "checkpoint.cuh"

namespace dcn1d {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Sums `v` over the lanes of a warp that hold the same position, then over the warps:
// every thread of the block gets the total of its own position.
__device__ __forceinline__ float sum_over_rows(float v, int TL, float (*part)[32]) {
    for (int o = TL; o < 32; o <<= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int lane = threadIdx.x & 31;
    __syncthreads();   // the last use of `part` is over
    part[threadIdx.x / 32][lane] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        t += part[w][lane];
    return t;
}

template <class T>
__global__ void __launch_bounds__(kThreads) norm_any_kernel(const NormProblem P, int TL) {
    __shared__ float part[kWarps][32];
    const int64_t tiles = (P.L + TL - 1) / TL;
    const int64_t b = blockIdx.x / tiles, l0 = (blockIdx.x - b * tiles) * TL;
    const int lane = threadIdx.x & 31, col = lane & (TL - 1);
    const int rows = kThreads / TL, row0 = threadIdx.x / TL;
    const int64_t l = l0 + col;
    const bool in = l < P.L;
    const T *x = static_cast<const T *>(P.x) + b * P.C * P.L + l;
    float s = 0.0f;
    for (int64_t c = row0; c < P.C; c += rows)
        s += in ? ld_f32(x + c * P.L) : 0.0f;
    const float mean = sum_over_rows(s, TL, part) / (float)P.C;
    s = 0.0f;
    for (int64_t c = row0; c < P.C; c += rows) {
        const float d = in ? ld_f32(x + c * P.L) - mean : 0.0f;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(sum_over_rows(s, TL, part) / (float)P.C + P.eps);
    if (in && row0 == 0) {
        if (P.mean)
            P.mean[b * P.L + l] = mean;
        if (P.rstd)
            P.rstd[b * P.L + l] = rstd;
    }
    T *y = static_cast<T *>(P.y) + b * P.C * P.L + l;
    const bool along_c = P.L == 1;
    const int64_t nb = ck_blocks(along_c ? P.C : P.L);
    // whole warps walk the rows together: the block maximum below is a warp reduction
    for (int64_t c0 = 0; c0 < P.C; c0 += rows) {
        const int64_t c = c0 + row0;
        const bool ok = in && c < P.C;
        const float v = ok ? (ld_f32(x + c * P.L) - mean) * rstd : 0.0f;
        if (ok) {
            float o = v;
            if (P.gamma)
                o = o * ld_f32(static_cast<const T *>(P.gamma) + c);
            if (P.beta)
                o = o + ld_f32(static_cast<const T *>(P.beta) + c);
            y[c * P.L] = from_f32<T>(o);
        }
        if (P.codes) {
            uint32_t m = ck_abs_bits(v);
            for (int o = along_c ? 16 : TL / 2; o > 0; o >>= 1)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const uint32_t e = ck_scale(m, ck_top<float>());
            if (ok) {
                P.codes[(b * P.C + c) * P.L + l] = (int8_t)ck_code(v, ck_inverse(e));
                if (along_c ? lane == 0 : col == 0)
                    P.scales[along_c ? b * nb + c / kCkBlock
                                     : (b * P.C + c) * nb + l / kCkBlock] = (uint8_t)e;
            }
        }
    }
}

// grad_x of the block's tiles, and the tiles' sums of grad_y v and grad_y over positions
// into the block's own rows of `part_g` [gridDim.x][2][C]: each of its entries is always
// the same thread's, so the sum has a fixed order.
template <class T, bool CK>
__global__ void __launch_bounds__(kThreads) norm_grad_any_kernel(const NormGrad P, int TL,
                                                                 int64_t ntiles, float *part_g) {
    __shared__ float part[kWarps][32];
    const int64_t tiles = (P.L + TL - 1) / TL;
    const int lane = threadIdx.x & 31, col = lane & (TL - 1);
    const int rows = kThreads / TL, row0 = threadIdx.x / TL;
    const bool along_c = P.L == 1;
    const int64_t nb = ck_blocks(along_c ? P.C : P.L);
    float *pg = part_g ? part_g + (int64_t)blockIdx.x * 2 * P.C : nullptr;
    for (int64_t tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
        const int64_t b = tile / tiles, l = (tile - b * tiles) * TL + col;
        const bool in = l < P.L;
        const float rstd = in ? P.rstd[b * P.L + l] : 0.0f;
        const float mean = !CK && in ? P.mean[b * P.L + l] : 0.0f;
        auto value = [&](int64_t c) {
            const int64_t at = (b * P.C + c) * P.L + l;
            if (CK)
                return (float)P.codes[at] *
                       ck_step(P.scales[along_c ? b * nb + c / kCkBlock
                                                : (b * P.C + c) * nb + l / kCkBlock]);
            return (ld_f32(static_cast<const T *>(P.x) + at) - mean) * rstd;
        };
        const T *gy = static_cast<const T *>(P.gy);
        float a = 0.0f, q = 0.0f;
        for (int64_t c0 = 0; c0 < P.C; c0 += rows) {
            const int64_t c = c0 + row0;
            float g = 0.0f, v = 0.0f;
            if (in && c < P.C) {
                g = ld_f32(gy + (b * P.C + c) * P.L + l);
                v = value(c);
                const float d = P.gamma ? g * ld_f32(static_cast<const T *>(P.gamma) + c) : g;
                a += d;
                q = fmaf(d, v, q);
            }
            if (pg) {
                float sg = g * v, sb = g;
                for (int o = TL / 2; o > 0; o >>= 1) {
                    sg += __shfl_xor_sync(0xFFFFFFFFu, sg, o);
                    sb += __shfl_xor_sync(0xFFFFFFFFu, sb, o);
                }
                if (col == 0 && c < P.C) {
                    const bool first = tile == blockIdx.x;
                    pg[c] = first ? sg : pg[c] + sg;
                    pg[P.C + c] = first ? sb : pg[P.C + c] + sb;
                }
            }
        }
        if (P.gx) {
            const float A = sum_over_rows(a, TL, part) / (float)P.C;
            const float S = sum_over_rows(q, TL, part) / (float)P.C;
            if (in)
                for (int64_t c = row0; c < P.C; c += rows) {
                    const float g = ld_f32(gy + (b * P.C + c) * P.L + l);
                    const float d = P.gamma ? g * ld_f32(static_cast<const T *>(P.gamma) + c) : g;
                    static_cast<T *>(P.gx)[(b * P.C + c) * P.L + l] =
                        from_f32<T>(rstd * (d - A - value(c) * S));
                }
        }
    }
}

// grad_gamma[c] and grad_beta[c]: the blocks' partial sums in block order.
template <class T>
__global__ void __launch_bounds__(256) norm_weight_grad_kernel(const float *part, int64_t n,
                                                               int64_t C, T *ggamma, T *gbeta) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * C)
        return;
    float s = 0.0f;
    for (int64_t j = 0; j < n; ++j)
        s += part[j * 2 * C + i];
    T *out = i < C ? ggamma : gbeta;
    if (out)
        out[i < C ? i : i - C] = from_f32<T>(s);
}

int lanes_along(int64_t L) {
    int TL = 1;
    while (TL < 32 && TL < L)
        TL *= 2;
    return TL;
}

int64_t grad_tiles(const NormGrad &P) {
    const int TL = lanes_along(P.L);
    return P.B * ((P.L + TL - 1) / TL);
}

int64_t grad_blocks(const NormGrad &P) {
    const int64_t most = (int64_t)sm_count_or(148) * 8, n = grad_tiles(P);
    return n < most ? n : most;
}

template <class T>
cudaError_t norm_grad(const NormGrad &P, void *ws, cudaStream_t s, int *launches) {
    const int64_t n = grad_tiles(P), blocks = grad_blocks(P);
    const bool weights = P.ggamma || P.gbeta;
    float *part = weights ? static_cast<float *>(ws) : nullptr;   // NULL for an empty input
    if (n > 0 && (P.gx || weights)) {
        const int TL = lanes_along(P.L);
        if (P.from_codes)
            norm_grad_any_kernel<T, true><<<(unsigned)blocks, kThreads, 0, s>>>(P, TL, n, part);
        else
            norm_grad_any_kernel<T, false><<<(unsigned)blocks, kThreads, 0, s>>>(P, TL, n, part);
        ++*launches;
    }
    if (weights) {
        norm_weight_grad_kernel<T><<<(unsigned)((2 * P.C + 255) / 256), 256, 0, s>>>(
            part, n > 0 ? blocks : 0, P.C, static_cast<T *>(P.ggamma), static_cast<T *>(P.gbeta));
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace

bool norm_grid_ok(int64_t B, int64_t L) {
    const int TL = lanes_along(L);
    return B * ((L + TL - 1) / TL) < (1LL << 31);
}

cudaError_t launch_norm(const NormProblem &P, cudaStream_t s) {
    const int TL = lanes_along(P.L);
    const unsigned grid = (unsigned)(P.B * ((P.L + TL - 1) / TL));
    if (P.dtype == DCN1D_BF16)
        norm_any_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(P, TL);
    else if (P.dtype == DCN1D_F16)
        norm_any_kernel<__half><<<grid, kThreads, 0, s>>>(P, TL);
    else
        norm_any_kernel<float><<<grid, kThreads, 0, s>>>(P, TL);
    return cudaGetLastError();
}

size_t norm_grad_workspace(const NormGrad &P) {
    return P.ggamma || P.gbeta ? (size_t)grad_blocks(P) * 2 * P.C * sizeof(float) : 0;
}

cudaError_t launch_norm_grad(const NormGrad &P, void *ws, cudaStream_t s, int *launches) {
    *launches = 0;
    if (P.dtype == DCN1D_BF16)
        return norm_grad<__nv_bfloat16>(P, ws, s, launches);
    if (P.dtype == DCN1D_F16)
        return norm_grad<__half>(P, ws, s, launches);
    return norm_grad<float>(P, ws, s, launches);
}

}  // namespace dcn1d
