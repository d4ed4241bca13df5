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
// gathers from it, adds grad_x up there, and writes every output once.  A site for the zero
// before the signal, one for the zero after it and one that far taps share make every tap
// the same code, without branches.
//
// grad_x is added up in fixed point by integer atomics: shared memory has no native fp32
// addition (a loop of compare-and-swap: 13 to 22 cycles a warp measured, more the more lanes
// meet at a site, against about 3 for an integer one), and integers make the sum exact and
// independent of the order.  With M the largest |m w grad_out| of the row (found first):
//  * 16-bit types: multiples of M 2^-22 in one word.  The unit is 2^-13 of what one
//    contribution of M 2^-9 rounds to in bf16.  A site may pass 2^31 only after more than
//    256 contributions of M; every addition looks at what it found, and a row where one
//    found 2^30 is added again in fp32.
//  * fp32: two words, hi 2^-s + lo 2^-(s+B) with |hi| <= 2^A, |lo| <= 2^(B-1).  With N =
//    L_out K < 2^n taps, A = 30 - n and B = 32 - n (at most 21 and 22) N additions overflow
//    neither, wherever they meet; the unit is M 2^-30 at 2^16 taps.
// A row whose M is not finite adds in fp32, so that NaN and infinities reach the sites they
// belong to.
//
// Measured (B200): [8, 512, 16000] bf16, 3 taps, 450 us for 1.11 GB = 2.5 TB/s, 0.38 of the
// copy bandwidth.  Bound by issue (84 % of the slots, 65 instructions a tap) and by the
// shared-memory pipe (79 %: the two additions of a tap collide about 4 ways, as offsets
// scatter the lanes).  Float atomics took 1194 us, two integers a sum 919, one position a
// lane 542.  512 threads and at most 64 registers for K <= 4: two blocks an SM, so that one
// unpacks or writes out while the other walks; more taps need the registers.
#include "checkpoint.cuh"
#include "pairs.cuh"
#include "sampler.cuh"
#include "sm100.cuh"

namespace dcn1d {

namespace {

constexpr int kMaxK = 9;                 // taps held in registers
constexpr int kMaxWarps = 16;
constexpr int kSmem = 224 * 1024;        // most dynamic shared memory of a block

struct Args {
    CheckpointConv q;
    float *part;                         // [B * C][K + 1]: grad_weight and grad_bias of a row
    int wpr;                             // warps of a row
    int x_words, sum_words;              // 4-byte words of a row's x and of each sum's array
    int a_bits, b_bits;                  // A and B above (16-bit types: A = 22)
    bool fixed;                          // they leave a fine enough unit
    bool wide;                           // offsets' gradients leave in 16-byte chunks
    bool even;                           // 16-bit types: two positions' values are whole words
    int64_t rows, nb;
};

// Sites of a row: -1, 0 .. L_in - 1, L_in, the far taps' two.  Position 0 is 16-byte aligned
// in each array: sites start one value before it.
template <class T> constexpr int lead() { return 16 / (int)sizeof(T) - 1; }
int words_of(const Problem &P, int size) {
    return (((P.L_in + 3) * size + 16 - size + 15) / 16) * 4;
}
int sums_of(const Problem &P) { return P.dtype == DCN1D_F32 ? 2 : 1; }
int row_words(const Problem &P) {
    return words_of(P, P.dtype == DCN1D_F32 ? 4 : 2) + sums_of(P) * words_of(P, 4);
}

constexpr int kGroup = 64;               // positions of a warp's step, two neighbours a lane

// Staging of a group's gradients of offsets (and mask).
int stage_bytes(const Problem &P) {
    return kGroup * P.K * (P.dtype == DCN1D_F32 ? 4 : 2) * (P.mask ? 2 : 1);
}

constexpr float kFarStart = 4194304.0f;  // 2^22, past every signal (fast_floor_ok)
constexpr float kRound = 12582912.0f;    // 1.5 * 2^23: adding it rounds to an integer
constexpr unsigned kRoundBits = 0x4B400000u;

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

// The `n` staged values of a group (fewer at the row's end) to global memory.
template <class T, int K>
__device__ __forceinline__ void unstage(const T *from, T *to, int n, bool wide) {
    constexpr int VE = 16 / (int)sizeof(T), CHUNKS = kGroup * K / VE;
    const int lane = threadIdx.x & 31;
    if (wide && n == kGroup * K) {
#pragma unroll
        for (int c = lane; c < (CHUNKS + 31) / 32 * 32; c += 32)
            if (c < CHUNKS)
                __stcs(reinterpret_cast<uint4 *>(to) + c, reinterpret_cast<const uint4 *>(from)[c]);
    } else {
        for (int i = lane; i < n; i += 32)
            to[i] = from[i];
    }
}

// Largest |value| of v[0 .. n) over the lanes of a row, as the bits of a float of its type
// (NaN above infinity above all others), a lane's part.
template <class T>
__device__ __forceinline__ uint32_t top_bits(const T *v, int64_t n, int lane, int lanes) {
    constexpr int VE = 16 / (int)sizeof(T);
    uint32_t top = 0;
    int64_t i = lane;
    if ((reinterpret_cast<uintptr_t>(v) & 15) == 0) {
        const uint4 *p = reinterpret_cast<const uint4 *>(v);
#pragma unroll 2
        for (int64_t c = lane; c < n / VE; c += lanes) {
            const uint4 u = __ldg(p + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4)
                    top = max(top, w[j] & 0x7FFFFFFFu);
                else
                    top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
            }
        }
        i += n / VE * VE;
    }
    if constexpr (sizeof(T) == 2)
        top = max(top >> 16, top & 0xFFFFu);
    for (; i < n; i += lanes) {
        if constexpr (sizeof(T) == 4)
            top = max(top, reinterpret_cast<const uint32_t *>(v)[i] & 0x7FFFFFFFu);
        else
            top = max(top, (uint32_t)(reinterpret_cast<const unsigned short *>(v)[i] & 0x7FFF));
    }
    return top;
}

template <class T>
__device__ __forceinline__ float bits_to_f32(uint32_t b) {
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(b);
    else if constexpr (std::is_same<T, __half>::value)
        return __half2float(__ushort_as_half((unsigned short)b));
    else
        return __uint_as_float(b << 16);
}

// Block of blockDim.x / 32 warps, wpr of them a row.  ALL: every gradient is wanted.
template <class T, int K, bool MASK, bool ALL>
__global__ void __launch_bounds__(512, K <= 4 ? 2 : 1) depthwise_grad_kernel(const Args a) {
    constexpr bool TWO = sizeof(T) == 4;                   // two words a sum
    extern __shared__ uint4 raw4[];
    __shared__ float sums[kMaxWarps][kMaxK + 1];
    __shared__ uint32_t tops[kMaxWarps][2];
    __shared__ int over[kMaxWarps];
    const Problem &P = a.q.P;
    const BackwardGrads &G = a.q.G;
    const int rpb = blockDim.x / 32 / a.wpr;               // rows of the block
    const int warp = threadIdx.x / 32, mine = warp / a.wpr, row_warp = warp - mine * a.wpr;
    const int me = threadIdx.x & 31;
    const int lanes = a.wpr * 32, lane = row_warp * 32 + me;
    const int64_t row = (int64_t)blockIdx.x * rpb + mine;
    const bool live = row < a.rows;
    const int L = P.L_in, Lo = P.L_out;
    const bool want_x = ALL || G.x, want_off = ALL || G.off, want_mask = MASK && (ALL || G.mask);
    // site s stands for position s - 1
    const int words = a.x_words + (TWO ? 2 : 1) * a.sum_words;
    uint32_t *base = reinterpret_cast<uint32_t *>(raw4) + (size_t)mine * words;
    T *xs = reinterpret_cast<T *>(base) + lead<T>();
    int *hi = reinterpret_cast<int *>(base + a.x_words) + 3, *lo = hi + a.sum_words;   // lo: TWO
    T *stage = reinterpret_cast<T *>(reinterpret_cast<uint32_t *>(raw4) + (size_t)rpb * words) +
               warp * kGroup * K * (MASK ? 2 : 1);
    const int c = live ? (int)(row % P.C_in) : 0;
    const int64_t out0 = row * Lo;
    const T *gout = static_cast<const T *>(G.gout) + out0;
    const T *mask = static_cast<const T *>(P.mask) + (MASK ? out0 * K : 0);
    float w[K];
    auto clear = [&]() {
        uint4 *p = reinterpret_cast<uint4 *>(base + a.x_words);
        for (int i = lane; i < (TWO ? 2 : 1) * a.sum_words / 4; i += lanes)
            p[i] = make_uint4(0, 0, 0, 0);
    };
    if (live) {
        const float g = a.q.gamma ? ld_f32(static_cast<const T *>(a.q.gamma) + c) : 1.0f;
        const float be = a.q.beta ? ld_f32(static_cast<const T *>(a.q.beta) + c) : 0.0f;
        const bool affine = a.q.gamma || a.q.beta;
        const int8_t *codes = a.q.codes + row * L;
        // a checkpoint of L == 1 has its blocks along the channels
        const uint8_t *scales = L == 1 ? a.q.scales + row / P.C_in * ck_blocks(P.C_in) + c / kCkBlock
                                       : a.q.scales + row * a.nb;
        // gamma v + beta, each rounded; 1 v + 0 changes no value but the sign of a zero
        auto through = [&](float v) {
            if (a.q.gamma)
                v = __fmul_rn(v, g);
            if (a.q.beta)
                v = __fadd_rn(v, be);
            return v;
        };
        if (L % 8 == 0 && (reinterpret_cast<uintptr_t>(a.q.codes) & 7) == 0) {
#pragma unroll 2
            for (int i = lane * 8; i < L; i += lanes * 8) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(codes + i));
                const float step = ck_step(__ldg(scales + i / kCkBlock));
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = (ck_biased((j < 4 ? u.x : u.y) ^ 0x80808080u, j % 4) - kCkBias) * step;
                    if (affine)
                        v[j] = through(v[j]);
                }
                constexpr int V = Vec<T>::V;
#pragma unroll
                for (int h = 0; h < 8 / V; ++h) {
                    Pair p[V / 2];
#pragma unroll
                    for (int j = 0; j < V / 2; ++j)
                        p[j] = pair(v[h * V + 2 * j], v[h * V + 2 * j + 1]);
                    *reinterpret_cast<uint4 *>(xs + 1 + i + h * V) = pairs_to_chunk<T>(p);
                }
            }
        } else {
            for (int i = lane; i < L; i += lanes)
                xs[1 + i] = from_f32<T>(through((float)codes[i] * ck_step(scales[i / kCkBlock])));
        }
        if (lane == 0)                                     // the zeros around the signal
            xs[0] = xs[L + 1] = xs[L + 2] = from_f32<T>(0.0f);
        clear();
#pragma unroll
        for (int k = 0; k < K; ++k)
            w[k] = ld_f32(static_cast<const T *>(P.w) + c * K + k);
        if (want_x) {
            const uint32_t tg = top_bits(gout, Lo, lane, lanes);
            const uint32_t tm = MASK ? top_bits(mask, (int64_t)Lo * K, lane, lanes) : 0u;
            const uint32_t wg = __reduce_max_sync(0xFFFFFFFFu, tg), wm = __reduce_max_sync(0xFFFFFFFFu, tm);
            if (me == 0) {
                tops[warp][0] = wg;
                tops[warp][1] = wm;
                over[warp] = 0;
            }
        }
    }
    __syncthreads();
    float to_hi = 0.0f;                                    // 2^s
    int s = 0;
    bool fixed = true;
    if (live && want_x) {
        uint32_t bg = 0, bm = 0;
        for (int i = 0; i < a.wpr; ++i) {
            bg = max(bg, tops[mine * a.wpr + i][0]);
            bm = max(bm, tops[mine * a.wpr + i][1]);
        }
        float tw = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            tw = w[k] == w[k] ? fmaxf(tw, fabsf(w[k])) : INFINITY;
        // M < 2^e; the product, associated as the contributions are, may round down twice
        const float tg = bits_to_f32<T>(bg), tm = MASK ? bits_to_f32<T>(bm) : 1.0f;
        const float M = tw * tg * tm;
        fixed = a.fixed && M < INFINITY && tg < INFINITY && tm < INFINITY && tw < INFINITY;   // not for NaN
        const int e = (int)((__float_as_uint(M) + 2u) >> 23) - 126;
        s = max(-126, min(126, a.a_bits - e));
        to_hi = two_to(s);
    }
    const float to_lo = two_to(a.b_bits);
    float gw[K], gb = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        gw[k] = 0.0f;
    const float span = (float)(P.dilation * (K - 1));
    const float from_start = P.unconstrained ? -INFINITY : 0.0f;
    const float to_end = P.unconstrained ? INFINITY : span;
    const T *off = static_cast<const T *>(P.off) + out0 * K;
    T *goff = static_cast<T *>(G.off) + (G.off ? out0 * K : 0);
    T *gmask = static_cast<T *>(G.mask) + (G.mask ? out0 * K : 0);
    // All taps of the row.  FIXED: grad_x in fixed point, and whether a site came near the
    // end of its range; AGAIN: grad_x alone, the rest has been written.
    auto walk = [&](auto fixed_tag, auto again_tag) {
        constexpr bool FIXED = decltype(fixed_tag)::value, AGAIN = decltype(again_tag)::value;
        constexpr int W = TWO ? 2 * K : K;                 // words of two positions' offsets
        uint32_t near_end = 0, o_next[W], m_next[MASK ? W : 1], g_next[TWO ? 2 : 1];
        auto two = [&](const T *from, uint32_t *to, int l, int per) {
            // `per` values of positions l and l + 1; past the end of the row: zeros
            const bool first = l < Lo, second = l + 1 < Lo;
            if (!TWO && a.even) {
                const uint32_t *p = reinterpret_cast<const uint32_t *>(from + l * per);
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k < per)
                        to[k] = first ? __ldg(p + k) : 0u;
                return;
            }
#pragma unroll
            for (int k = 0; k < 2 * K; ++k)
                if (k < 2 * per) {
                    const T *p = from + l * per + k;
                    const bool in = k < per ? first : second;
                    if constexpr (TWO)
                        to[k] = in ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
                    else {
                        const uint32_t v = in ? __ldg(reinterpret_cast<const unsigned short *>(p)) : 0u;
                        to[k / 2] = k % 2 == 0 ? v : to[k / 2] | v << 16;
                    }
                }
        };
        // value i of those words
        auto at = [](const uint32_t *w, int i) -> float {
            if constexpr (TWO)
                return __uint_as_float(w[i]);
            else if constexpr (std::is_same<T, __half>::value)
                return __half2float(__ushort_as_half((unsigned short)(i % 2 ? w[i / 2] >> 16 : w[i / 2])));
            else
                return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        };
        auto fetch = [&](int l0) {
            const int l = l0 + 2 * me;
            two(off, o_next, l, K);
            if (MASK)
                two(mask, m_next, l, K);
            two(gout, g_next, l, 1);
        };
        int l0 = row_warp * kGroup;
        if (l0 < Lo)
            fetch(l0);
        for (; l0 < Lo; l0 += 2 * lanes) {
            uint32_t o[W], m[MASK ? W : 1], gg[TWO ? 2 : 1];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                o[k] = o_next[k];
                if (MASK)
                    m[k] = m_next[k];
            }
            gg[0] = g_next[0];
            if (TWO)
                gg[TWO ? 1 : 0] = g_next[TWO ? 1 : 0];
            if (l0 + 2 * lanes < Lo)
                fetch(l0 + 2 * lanes);
            const float start0 = (float)((l0 + 2 * me) * P.stride - P.padding);
            float doff[2 * K], dmask[MASK ? 2 * K : 1];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float g = at(gg, u);
                if (!AGAIN)
                    gb += g;
                // Taps past the end of the row are far from the signal: with their zeros they
                // read zeros and add nothing, whatever x, the mask or the weight hold.
                const float start = l0 + 2 * me + u >= Lo ? kFarStart
                                    : u                   ? start0 + (float)P.stride
                                                          : start0;
                const float first = start + from_start, last = start + to_end;
                int found[2 * K];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float raw = __fadd_rn(start + (float)(k * P.dilation), at(o, u * K + k));
                    const float pos = fminf(fmaxf(raw, first), last);
                    // floor by one addition rounded down (sampler.cuh); positions too far for
                    // it give a site past the signal, like all that lie outside
                    const float t = __fadd_rd(pos, kFloorMagic);
                    const float f = __fsub_rn(pos, __fsub_rn(t, kFloorMagic));
                    const uint32_t site =
                        min(__float_as_uint(t) - (kFloorMagicBits - 1u), (uint32_t)L + 1u);
                    const float mk = MASK ? at(m, u * K + k) : 1.0f;
                    const float dv = w[k] * g, mdv = MASK ? mk * dv : dv;
                    if (!AGAIN) {
                        const float x0 = to_f32(xs[site]), x1 = to_f32(xs[site + 1]);
                        const float slope = x1 - x0, v = fmaf(f, slope, x0);
                        gw[k] = fmaf(MASK ? mk * g : g, v, gw[k]);
                        // no gradient where the clamp moved the tap
                        doff[u * K + k] = pos == raw ? slope * mdv : 0.0f;
                        if (MASK)
                            dmask[u * K + k] = v * dv;
                    }
                    if (want_x) {
                        const float d = site <= (uint32_t)L ? mdv : 0.0f;   // far taps add zeros
                        const float c1 = f * d, c0 = d - c1;
                        if constexpr (FIXED) {
                            const float h0 = fmaf(c0, to_hi, kRound), h1 = fmaf(c1, to_hi, kRound);
                            found[2 * k] = atomicAdd(hi + site, (int)(__float_as_uint(h0) - kRoundBits));
                            found[2 * k + 1] =
                                atomicAdd(hi + site + 1, (int)(__float_as_uint(h1) - kRoundBits));
                            if constexpr (TWO) {
                                const float r0 = fmaf(c0, to_hi, kRound - h0),
                                            r1 = fmaf(c1, to_hi, kRound - h1);
                                atomicAdd(lo + site,
                                          (int)(__float_as_uint(fmaf(r0, to_lo, kRound)) - kRoundBits));
                                atomicAdd(lo + site + 1,
                                          (int)(__float_as_uint(fmaf(r1, to_lo, kRound)) - kRoundBits));
                            }
                        } else {
                            atomicAdd(reinterpret_cast<float *>(hi) + site, c0);
                            atomicAdd(reinterpret_cast<float *>(hi) + site + 1, c1);
                        }
                    }
                }
                if constexpr (FIXED && !TWO) {
                    if (want_x) {
#pragma unroll
                        for (int k = 0; k < 2 * K; ++k)    // bit 31: 2^30 or more, either sign
                            near_end |= (uint32_t)found[k] + 0x40000000u;
                    }
                }
            }
            if constexpr (AGAIN)
                continue;
            const int n = min(kGroup, Lo - l0) * K;
            auto put = [&](T *to, const float (&d)[2 * K]) {
                if constexpr (TWO) {
#pragma unroll
                    for (int k = 0; k < 2 * K; ++k)
                        to[2 * K * me + k] = from_f32<T>(d[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const T q[2] = {from_f32<T>(d[2 * k]), from_f32<T>(d[2 * k + 1])};
                        reinterpret_cast<uint32_t *>(to)[K * me + k] = *reinterpret_cast<const uint32_t *>(q);
                    }
                }
            };
            if (want_off)
                put(stage, doff);
            if constexpr (MASK)
                if (want_mask)
                    put(stage + kGroup * K, dmask);
            __syncwarp();
            if (want_off)
                unstage<T, K>(stage, goff + l0 * K, n, a.wide);
            if (want_mask)
                unstage<T, K>(stage + kGroup * K, gmask + l0 * K, n, a.wide);
            __syncwarp();
        }
        return near_end >> 31;
    };
    if (live) {
        if (fixed) {
            if (walk(std::true_type(), std::false_type()))
                over[mine * a.wpr] = 1;
        } else {
            walk(std::false_type(), std::false_type());
        }
    }
    if constexpr (!TWO) {
        __syncthreads();
        const bool redo = live && want_x && fixed && over[mine * a.wpr];
        if (__syncthreads_or(redo)) {
            if (redo)
                clear();
            __syncthreads();
            if (redo) {
                fixed = false;
                walk(std::false_type(), std::true_type());
            }
        }
    }
    __syncthreads();
    if (live && want_x) {
        T *gx = static_cast<T *>(G.x) + row * L;
        const float from_hi = two_to(-s), from_lo = two_to(-a.b_bits);
        auto value = [&](int i) {
            const int h = hi[i + 1];
            if (!fixed)
                return __int_as_float(h);
            return (TWO ? fmaf((float)lo[i + 1], from_lo, (float)h) : (float)h) * from_hi;
        };
        if (sizeof(T) == 2 && L % 4 == 0 && (reinterpret_cast<uintptr_t>(G.x) & 7) == 0) {
            for (int i = lane * 4; i < L; i += lanes * 4) {
                const int4 h = *reinterpret_cast<const int4 *>(hi + 1 + i);
                auto one = [&](int v) { return fixed ? (float)v * from_hi : __int_as_float(v); };
                const T four[4] = {from_f32<T>(one(h.x)), from_f32<T>(one(h.y)), from_f32<T>(one(h.z)),
                                   from_f32<T>(one(h.w))};
                __stcs(reinterpret_cast<uint2 *>(gx + i), *reinterpret_cast<const uint2 *>(four));
            }
        } else {
            for (int i = lane; i < L; i += lanes)
                gx[i] = from_f32<T>(value(i));
        }
    }
    if (!a.part)
        return;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        float v = k < K ? gw[k < K ? k : 0] : gb;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (me == 0)
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

// Dynamic shared memory of a block of rpb rows of wpr warps.
size_t block_bytes(const Problem &P, int wpr, int rpb) {
    return (size_t)rpb * row_words(P) * 4 + (size_t)rpb * wpr * stage_bytes(P);
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
    a.x_words = words_of(P, sizeof(T));
    a.sum_words = words_of(P, 4);
    int n = 0;                                             // N < 2^n
    while ((1LL << n) <= (int64_t)P.L_out * K)
        ++n;
    a.a_bits = sizeof(T) == 2 ? 22 : 30 - n < 21 ? 30 - n : 21;
    a.b_bits = 32 - n < 22 ? 32 - n : 22;
    a.fixed = sizeof(T) == 2 || n <= 18;
    const int es = P.dtype == DCN1D_F32 ? 4 : 2;
    a.wide = (int64_t)P.L_out * K % (16 / es) == 0 &&
             ((reinterpret_cast<uintptr_t>(G.off) | reinterpret_cast<uintptr_t>(G.mask)) & 15) == 0;
    a.even = P.L_out % 2 == 0 && ((reinterpret_cast<uintptr_t>(P.off) | reinterpret_cast<uintptr_t>(P.mask) |
                                   reinterpret_cast<uintptr_t>(G.gout)) & 3) == 0;
    // a warp for each 64 positions, up to the block; then as many rows as make a block of
    // 8 warps
    const int longest = P.L_out > P.L_in ? P.L_out : P.L_in;
    a.wpr = 1;
    while (a.wpr < kMaxWarps && a.wpr * 64 < longest && block_bytes(P, 2 * a.wpr, 1) <= kSmem)
        a.wpr *= 2;
    int rpb = a.wpr < 8 ? 8 / a.wpr : 1;
    while (rpb > 1 && block_bytes(P, a.wpr, rpb) > 48 * 1024)
        rpb /= 2;
    const size_t shared = block_bytes(P, a.wpr, rpb);
    const bool all = G.x && G.off && (!P.mask || G.mask);
    auto kernel = P.mask ? (all ? depthwise_grad_kernel<T, K, true, true>
                                : depthwise_grad_kernel<T, K, true, false>)
                         : (all ? depthwise_grad_kernel<T, K, false, true>
                                : depthwise_grad_kernel<T, K, false, false>);
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
           P.B > 0 && block_bytes(P, 1, 1) <= kSmem && fast_floor_ok(P);
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
