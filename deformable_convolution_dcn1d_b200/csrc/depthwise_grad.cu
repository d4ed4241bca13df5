// Backward pass of the depthwise layer whose input is an 8-bit checkpoint, in one kernel.
//
// For groups == offset_groups == C_in == C_out a row (b, c) stands alone.  With dv =
// w[c, k] grad_out[b, c, l], v = (1-f) x[i0] + f x[i0+1] and m the mask (1 without one):
//   grad_offsets[b, c, l, k] = m (x[i0+1] - x[i0]) dv   (0 where the clamp moved the tap)
//   grad_mask[b, c, l, k]    = v dv
//   grad_x[b, c, i0]        += m (1-f) dv,  grad_x[b, c, i0+1] += m f dv
//   grad_weight[c, k]        = sum_{b,l} m v grad_out,  grad_bias[c] = sum_{b,l} grad_out
// No column buffer is needed: a block unpacks its row of x into shared memory (through the
// norm's weights where given, rounded to the layer's type as the forward's input was),
// gathers from it, adds grad_x up there in fp32, and writes every output once.  Both rows
// carry a zero at either end, so a tap next to the signal needs no bounds check of each
// neighbour; taps further out contribute nothing.  Order: grad_x is a sum of shared-memory
// atomic additions (its low bits may differ between calls); all other sums have a fixed
// order.
#include "checkpoint.cuh"
#include "sampler.cuh"
#include "sm100.cuh"

namespace dcn1d {

namespace {

constexpr int kMaxK = 9;                 // taps held in registers
constexpr int kSmemRow = 200 * 1024;     // most shared memory of a block

struct Args {
    CheckpointConv q;
    float *part;                         // [B * C][K + 1]: grad_weight and grad_bias of a row
    int wpr;                             // warps of a row
    int x_bytes;                         // of a row of x in shared memory, a multiple of 16
    int64_t rows, nb;
};

int row_bytes_x(const Problem &P) {
    const int es = P.dtype == DCN1D_F32 ? 4 : 2;
    return ((P.L_in + 2) * es + 15) / 16 * 16;
}
int row_bytes(const Problem &P) { return row_bytes_x(P) + ((P.L_in + 2) * 4 + 15) / 16 * 16; }

// Block of `blockDim.x / 32` warps, wpr of them a row.
template <class T, int K, bool MASK>
__global__ void __launch_bounds__(512) depthwise_grad_kernel(const Args a) {
    extern __shared__ uint4 raw4[];
    __shared__ float sums[16][kMaxK + 1];
    const Problem &P = a.q.P;
    const BackwardGrads &G = a.q.G;
    const int rpb = blockDim.x / 32 / a.wpr;               // rows of the block
    const int warp = threadIdx.x / 32, mine = warp / a.wpr;
    const int lanes = a.wpr * 32, lane = threadIdx.x - mine * lanes;
    const int64_t row = (int64_t)blockIdx.x * rpb + mine;
    const bool live = row < a.rows;
    const int L = P.L_in, Lo = P.L_out;
    const int stride_b = a.x_bytes + ((L + 2) * 4 + 15) / 16 * 16;
    char *smem = reinterpret_cast<char *>(raw4) + mine * stride_b;
    T *xs = reinterpret_cast<T *>(smem);                   // xs[p + 1] = x at p
    float *gs = reinterpret_cast<float *>(smem + a.x_bytes);
    const int c = live ? (int)(row % P.C_in) : 0;
    if (live) {
        const float g = a.q.gamma ? ld_f32(static_cast<const T *>(a.q.gamma) + c) : 1.0f;
        const float be = a.q.beta ? ld_f32(static_cast<const T *>(a.q.beta) + c) : 0.0f;
        const int8_t *codes = a.q.codes + row * L;
        const uint8_t *scales = a.q.scales + row * a.nb;
        for (int i = lane; i < L + 2; i += lanes) {
            float v = 0.0f;
            if (i > 0 && i <= L) {
                v = (float)codes[i - 1] * ck_step(scales[(i - 1) / kCkBlock]);
                if (a.q.gamma)
                    v = __fmul_rn(v, g);
                if (a.q.beta)
                    v = __fadd_rn(v, be);
            }
            xs[i] = from_f32<T>(v);
            gs[i] = 0.0f;
        }
    }
    __syncthreads();
    float gw[K], gb = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        gw[k] = 0.0f;
    if (live) {
        float w[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            w[k] = ld_f32(static_cast<const T *>(P.w) + c * K + k);
        const int span = P.dilation * (K - 1);
        const T *off = static_cast<const T *>(P.off) + row * Lo * K;
        const T *mask = static_cast<const T *>(P.mask) + (MASK ? row * Lo * K : 0);
        T *goff = static_cast<T *>(G.off) + (G.off ? row * Lo * K : 0);
        T *gmask = static_cast<T *>(G.mask) + (G.mask ? row * Lo * K : 0);
        const T *gout = static_cast<const T *>(G.gout) + row * Lo;
        for (int l = lane; l < Lo; l += lanes) {
            const float g = ld_f32(gout + l);
            gb += g;
            const int start = l * P.stride - P.padding;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float o = ld_f32(off + l * K + k);
                const float m = MASK ? ld_f32(mask + l * K + k) : 1.0f;
                const float at = __fadd_rn(__int2float_rn(start + k * P.dilation), o);
                const bool gate = P.unconstrained || (at >= __int2float_rn(start) &&
                                                      at <= __int2float_rn(start + span));
                const Tap tp = sample_tap(start, k, P.dilation, span, o, P.unconstrained);
                const float dv = w[k] * g;
                float slope = 0.0f, v = 0.0f;
                if (tp.i0 >= -1 && tp.i0 < L) {
                    const float x0 = to_f32(xs[tp.i0 + 1]), x1 = to_f32(xs[tp.i0 + 2]);
                    slope = x1 - x0;
                    v = __fadd_rn(__fmul_rn(__fsub_rn(1.0f, tp.f), x0), __fmul_rn(tp.f, x1));
                    gw[k] = fmaf(g, m * v, gw[k]);
                    if (G.x) {
                        atomicAdd(gs + tp.i0 + 1, m * (1.0f - tp.f) * dv);
                        atomicAdd(gs + tp.i0 + 2, m * tp.f * dv);
                    }
                }
                if (G.off)
                    goff[l * K + k] = from_f32<T>(gate ? m * slope * dv : 0.0f);
                if (MASK && G.mask)
                    gmask[l * K + k] = from_f32<T>(v * dv);
            }
        }
    }
    __syncthreads();
    if (live && G.x) {
        T *gx = static_cast<T *>(G.x) + row * L;
        for (int i = lane; i < L; i += lanes)
            gx[i] = from_f32<T>(gs[i + 1]);
    }
    if (!a.part)
        return;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        float v = k < K ? gw[k < K ? k : 0] : gb;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if ((threadIdx.x & 31) == 0)
            sums[warp][k] = v;
    }
    __syncthreads();
    if (live && lane <= K) {
        float v = 0.0f;
        for (int i = 0; i < a.wpr; ++i)
            v += sums[mine * a.wpr + i][lane];
        a.part[row * (K + 1) + lane] = v;
    }
}

// grad_weight[c, k] and grad_bias[c]: the rows' sums over the batch, in order.
template <class T>
__global__ void __launch_bounds__(256) depthwise_weight_grad_kernel(const float *part, int B, int C,
                                                                    int K, T *gw, T *gb) {
    const int i = blockIdx.x * 256 + threadIdx.x;      // c * (K + 1) + k
    if (i >= C * (K + 1))
        return;
    float s = 0.0f;
    for (int b = 0; b < B; ++b)
        s += part[(int64_t)b * C * (K + 1) + i];
    const int c = i / (K + 1), k = i - c * (K + 1);
    if (k < K) {
        if (gw)
            gw[c * K + k] = from_f32<T>(s);
    } else if (gb) {
        gb[c] = from_f32<T>(s);
    }
}

template <class T, int K>
cudaError_t run(const CheckpointConv &q, void *ws, cudaStream_t s, int *launches) {
    const Problem &P = q.P;
    const BackwardGrads &G = q.G;
    Args a;
    a.q = q;
    a.part = G.w || G.bias ? static_cast<float *>(ws) : nullptr;
    a.rows = (int64_t)P.B * P.C_in;
    a.nb = ck_blocks(P.L_in);
    a.x_bytes = row_bytes_x(P);
    // a warp for each 256 positions, up to the block; then as many rows as make a block of
    // 8 warps
    const int longest = P.L_out > P.L_in ? P.L_out : P.L_in;
    a.wpr = 1;
    while (a.wpr < 16 && a.wpr * 256 < longest)
        a.wpr *= 2;
    int rpb = a.wpr < 8 ? 8 / a.wpr : 1;
    while (rpb > 1 && rpb * row_bytes(P) > 48 * 1024)
        rpb /= 2;
    const size_t shared = (size_t)rpb * row_bytes(P);
    auto kernel = P.mask ? depthwise_grad_kernel<T, K, true> : depthwise_grad_kernel<T, K, false>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), (int)shared);
    if (e != cudaSuccess)
        return e;
    kernel<<<(unsigned)((a.rows + rpb - 1) / rpb), rpb * a.wpr * 32, shared, s>>>(a);
    ++*launches;
    if (a.part) {
        depthwise_weight_grad_kernel<T><<<(P.C_in * (K + 1) + 255) / 256, 256, 0, s>>>(
            a.part, P.B, P.C_in, K, static_cast<T *>(G.w), static_cast<T *>(G.bias));
        ++*launches;
    }
    return cudaGetLastError();
}

template <class T>
cudaError_t run_k(const CheckpointConv &q, void *ws, cudaStream_t s, int *launches) {
    switch (q.P.K) {
    case 1: return run<T, 1>(q, ws, s, launches);
    case 2: return run<T, 2>(q, ws, s, launches);
    case 3: return run<T, 3>(q, ws, s, launches);
    case 4: return run<T, 4>(q, ws, s, launches);
    case 5: return run<T, 5>(q, ws, s, launches);
    case 6: return run<T, 6>(q, ws, s, launches);
    case 7: return run<T, 7>(q, ws, s, launches);
    case 8: return run<T, 8>(q, ws, s, launches);
    case 9: return run<T, 9>(q, ws, s, launches);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

bool depthwise_grad_supported(const Problem &P) {
    return P.groups == P.C_in && P.C_out == P.C_in && P.offset_groups == P.C_in && P.K <= kMaxK &&
           P.B > 0 && row_bytes(P) <= kSmemRow;
}

size_t depthwise_grad_workspace(const Problem &P, const BackwardGrads &G) {
    return G.w || G.bias ? (size_t)P.B * P.C_in * (P.K + 1) * sizeof(float) : 0;
}

cudaError_t launch_depthwise_grad(const CheckpointConv &q, void *ws, cudaStream_t s,
                                  int *launches) {
    *launches = 0;
    if (!q.G.x && !q.G.off && !q.G.mask && !q.G.w && !q.G.bias)
        return cudaSuccess;
    if (q.P.dtype == DCN1D_BF16)
        return run_k<__nv_bfloat16>(q, ws, s, launches);
    if (q.P.dtype == DCN1D_F16)
        return run_k<__half>(q, ws, s, launches);
    return run_k<float>(q, ws, s, launches);
}

}  // namespace dcn1d
