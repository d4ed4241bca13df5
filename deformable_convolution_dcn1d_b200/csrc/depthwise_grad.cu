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
// independent of the order.  Every site has a unit of its own, so that quiet stretches of a
// row keep what fp32 additions would keep of them: a first walk takes the largest
// contribution of each site (atomic maxima of the bits), and each site gets four bits q,
// min(15, (E - e) / 4) for the row's largest exponent E and the site's e.  Its contributions
// are whole multiples of 2^(E - 4q - 26), at most 2^-22 of the largest one and below 2^26 of
// them: a contribution of at most 24 bits is off by at most 2^-23 of the site's largest,
// against 2^-24 of the sum an fp32 addition.  (Sites whose largest is under 2^-60 of the
// row's: by at most 2^-86 of that.)  A sum may pass 2^31 only after more than 16
// contributions of the largest kind; every addition looks at what it found, and a row where
// one found 2^30 is added again in fp32.  So is a row with a NaN or an infinity, so that
// they reach the sites they belong to, and a row too long for the bits q beside its sums.
//
// Measured (B200): [8, 512, 16000] bf16, 3 taps, 768 us for 1.11 GB = 1.45 TB/s, 0.22 of the
// copy bandwidth; fp32 1186 us.  Bound by issue (84 % of the slots, 112 instructions a tap
// over both walks) and by the shared-memory pipe (76 %: the two additions or maxima of a tap
// collide about 4 ways, as offsets scatter the lanes).  One unit for a whole row took 456 us
// and 65 instructions, and lost what lies far below the row's largest; fp32 additions
// run at 61 SM cycles a warp and tap where these take 51 (rows of 34000 to 37000, bf16).
// 512 threads and at most 64 registers for K <= 4: two blocks an SM, so that one
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
    int x_words, sum_words, code_words;  // 4-byte words of a row's x, its sums and the bits q
    bool fixed;                          // sums in fixed point: there is room for the bits q
    bool staged;                         // offsets' gradients go through shared memory
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
int code_words_of(const Problem &P) { return (words_of(P, 4) + 31) / 32 * 4; }   // 8 sites a word
int row_words(const Problem &P, bool fixed) {
    return words_of(P, P.dtype == DCN1D_F32 ? 4 : 2) + words_of(P, 4) + (fixed ? code_words_of(P) : 0);
}

constexpr int kGroup = 64;               // positions of a warp's step, two neighbours a lane

// Staging of a group's gradients of offsets, then of the mask.
int stage_bytes(const Problem &P) { return kGroup * P.K * (P.dtype == DCN1D_F32 ? 4 : 2); }

constexpr float kFarStart = 4194304.0f;  // 2^22, past every signal (fast_floor_ok)
constexpr int kBits = 26;                // of a site's largest contribution, in its units
// The least exponent (biased) of a row's largest contribution at which every unit is a normal
// number.  Rows below are taken times 2^100 (and at least this), sums and all.
constexpr int kLeastTop = kBits + 60;
constexpr float kUp = 0x1p100f, kDown = 0x1p-100f;

// What a walk over a row's taps does with grad_x; the first and the last write nothing else.
enum Walk { TOPS, FIXED, FLOAT, AGAIN };

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

// Block of blockDim.x / 32 warps, wpr of them a row.  ALL: every gradient is wanted.
template <class T, int K, bool MASK, bool ALL>
__global__ void __launch_bounds__(512, K <= (sizeof(T) == 4 ? 3 : 4) ? 2 : 1)
    depthwise_grad_kernel(const Args a) {
    constexpr bool F32 = sizeof(T) == 4;
    extern __shared__ uint4 raw4[];
    __shared__ float sums[kMaxWarps][kMaxK + 1];
    __shared__ uint32_t tops[kMaxWarps];
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
    const int words = a.x_words + a.sum_words + a.code_words;
    uint32_t *base = reinterpret_cast<uint32_t *>(raw4) + (size_t)mine * words;
    T *xs = reinterpret_cast<T *>(base) + lead<T>();
    int *sum = reinterpret_cast<int *>(base + a.x_words) + 3;
    uint32_t *qs = base + a.x_words + a.sum_words;         // q of sites 8 i - 3 .. 8 i + 4 in word i
    T *stage = reinterpret_cast<T *>(reinterpret_cast<uint32_t *>(raw4) + (size_t)rpb * words) +
               warp * kGroup * K;
    const int c = live ? (int)(row % P.C_in) : 0;
    const int64_t out0 = row * Lo;
    const T *gout = static_cast<const T *>(G.gout) + out0;
    const T *mask = static_cast<const T *>(P.mask) + (MASK ? out0 * K : 0);
    float w[K];
    auto clear = [&]() {
        uint4 *p = reinterpret_cast<uint4 *>(base + a.x_words);
        for (int i = lane; i < a.sum_words / 4; i += lanes)
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
        if (me == 0)
            over[warp] = 0;
    }
    __syncthreads();
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
    uint32_t unit_bits = 0;                                // 1 / the unit of q = 0, as a float
    float up = 1.0f;                                       // kUp in rows of tiny contributions
    // All taps of the row.  FIXED returns whether a site came near the end of its range.
    auto walk = [&](auto mode) {
        constexpr Walk MODE = decltype(mode)::value;
        constexpr bool REST = MODE == FIXED || MODE == FLOAT;   // all gradients, not grad_x alone
        constexpr int W = F32 ? 2 * K : K;                 // words of two positions' offsets
        uint32_t near_end = 0, o_next[W], m_next[MASK ? W : 1], g_next[F32 ? 2 : 1];
        auto two = [&](const T *from, uint32_t *to, int l, int per) {
            // `per` values of positions l and l + 1; past the end of the row: zeros
            const bool first = l < Lo, second = l + 1 < Lo;
            if (!F32 && a.even) {
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
                    if constexpr (F32)
                        to[k] = in ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
                    else {
                        const uint32_t v = in ? __ldg(reinterpret_cast<const unsigned short *>(p)) : 0u;
                        to[k / 2] = k % 2 == 0 ? v : to[k / 2] | v << 16;
                    }
                }
        };
        // value i of those words
        auto at = [](const uint32_t *w, int i) -> float {
            if constexpr (F32)
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
            uint32_t o[W], m[MASK ? W : 1], gg[F32 ? 2 : 1];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                o[k] = o_next[k];
                if (MASK)
                    m[k] = m_next[k];
            }
            gg[0] = g_next[0];
            if (F32)
                gg[F32 ? 1 : 0] = g_next[F32 ? 1 : 0];
            if (l0 + 2 * lanes < Lo)
                fetch(l0 + 2 * lanes);
            const float start0 = (float)((l0 + 2 * me) * P.stride - P.padding);
            float doff[2 * K], dmask[MASK ? 2 * K : 1];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float g = at(gg, u);
                if (REST)
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
                    if (REST) {
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
                        const float du = MODE == FIXED ? __fmul_rn(d, up) : d;
                        const float c1 = __fmul_rn(f, du), c0 = __fsub_rn(du, c1);
                        if constexpr (MODE == TOPS) {
                            atomicMax(sum + site, (int)(__float_as_uint(c0) & 0x7FFFFFFFu));
                            atomicMax(sum + site + 1, (int)(__float_as_uint(c1) & 0x7FFFFFFFu));
                        } else if constexpr (MODE == FIXED) {
                            auto in_units = [&](float c, uint32_t slot) {
                                const uint32_t q = qs[slot >> 3] >> (slot * 4 & 31u) & 15u;
                                return __float2int_rn(__fmul_rn(c, __uint_as_float(unit_bits + (q << 25))));
                            };
                            found[2 * k] = atomicAdd(sum + site, in_units(c0, site + 3));
                            found[2 * k + 1] = atomicAdd(sum + site + 1, in_units(c1, site + 4));
                        } else {
                            atomicAdd(reinterpret_cast<float *>(sum) + site, c0);
                            atomicAdd(reinterpret_cast<float *>(sum) + site + 1, c1);
                        }
                    }
                }
                if constexpr (MODE == FIXED) {
                    if (want_x) {
#pragma unroll
                        for (int k = 0; k < 2 * K; ++k)    // bit 31: 2^30 or more, either sign
                            near_end |= (uint32_t)found[k] + 0x40000000u;
                    }
                }
            }
            if constexpr (!REST)
                continue;
            const int n = min(kGroup, Lo - l0) * K;
            auto put = [&](T *to, const float (&d)[2 * K]) {
                if constexpr (F32) {
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
            if (a.staged) {
                if (want_off) {
                    put(stage, doff);
                    __syncwarp();
                    unstage<T, K>(stage, goff + l0 * K, n, a.wide);
                    __syncwarp();
                }
                if constexpr (MASK)
                    if (want_mask) {
                        put(stage, dmask);
                        __syncwarp();
                        unstage<T, K>(stage, gmask + l0 * K, n, a.wide);
                        __syncwarp();
                    }
            } else {
#pragma unroll
                for (int k = 0; k < 2 * K; ++k) {
                    const int i = 2 * K * me + k;
                    if (want_off && i < n)
                        goff[l0 * K + i] = from_f32<T>(doff[k]);
                    if constexpr (MASK)
                        if (want_mask && i < n)
                            gmask[l0 * K + i] = from_f32<T>(dmask[k]);
                }
            }
        }
        return near_end >> 31;
    };
    bool fixed = false;
    int top = 0;
    if (want_x && a.fixed) {                               // the same in every thread of the grid
        if (live)
            walk(std::integral_constant<Walk, TOPS>());
        __syncthreads();
        // the bits of the row's largest contribution (NaN above infinity above all others)
        uint4 *tp = reinterpret_cast<uint4 *>(base + a.x_words);
        uint32_t t = 0;
        if (live)
            for (int i = lane; i < a.sum_words / 4; i += lanes)
                t = max(t, max(max(tp[i].x, tp[i].y), max(tp[i].z, tp[i].w)));
        t = __reduce_max_sync(0xFFFFFFFFu, t);
        if (me == 0)
            tops[warp] = t;
        __syncthreads();
        t = 0;
        for (int i = 0; i < a.wpr; ++i)
            t = max(t, tops[mine * a.wpr + i]);
        fixed = t < 0x7F800000u;
        if ((int)(t >> 23) < kLeastTop)
            up = kUp;
        top = max((int)(__float_as_uint(__uint_as_float(t) * up) >> 23), kLeastTop);
        unit_bits = (uint32_t)(253 + kBits - top) << 23;
        if (live)
            for (int i = lane; i < a.code_words; i += lanes) {
                uint32_t q = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (2 * i + h < a.sum_words / 4) {
                        const uint4 u = tp[2 * i + h];
                        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = (int)(__float_as_uint(__uint_as_float(e[j]) * up) >> 23);
                            q |= (uint32_t)max(0, min(15, (top - at) >> 2)) << (16 * h + 4 * j);
                        }
                        tp[2 * i + h] = make_uint4(0, 0, 0, 0);
                    }
                qs[i] = q;
            }
        __syncthreads();
    }
    if (live) {
        if (fixed) {
            if (walk(std::integral_constant<Walk, FIXED>()))
                over[mine * a.wpr] = 1;
        } else {
            walk(std::integral_constant<Walk, FLOAT>());
        }
    }
    if (want_x && a.fixed) {
        __syncthreads();
        const bool redo = live && fixed && over[mine * a.wpr];
        if (__syncthreads_or(redo)) {
            if (redo)
                clear();
            __syncthreads();
            if (redo) {
                fixed = false;
                walk(std::integral_constant<Walk, AGAIN>());
            }
        }
    }
    __syncthreads();
    if (live && want_x) {
        T *gx = static_cast<T *>(G.x) + row * L;
        const uint32_t from_bits = (uint32_t)(top + 1 - kBits) << 23;   // the unit of q = 0
        const float down = up == 1.0f ? 1.0f : kDown;
        auto value = [&](int v, uint32_t q) {              // from a word of sums
            return fixed ? (float)v * __uint_as_float(from_bits - ((q & 15u) << 25)) * down
                         : __int_as_float(v);
        };
        auto q_of = [&](int slot) { return fixed ? qs[slot >> 3] >> (slot * 4 & 31) : 0u; };
        if (sizeof(T) == 2 && L % 4 == 0 && (reinterpret_cast<uintptr_t>(G.x) & 7) == 0) {
            for (int i = lane * 4; i < L; i += lanes * 4) {
                const int4 v = *reinterpret_cast<const int4 *>(sum + 1 + i);
                const uint32_t q = q_of(i + 4);            // four positions' are in one word
                const T four[4] = {from_f32<T>(value(v.x, q)), from_f32<T>(value(v.y, q >> 4)),
                                   from_f32<T>(value(v.z, q >> 8)), from_f32<T>(value(v.w, q >> 12))};
                __stcs(reinterpret_cast<uint2 *>(gx + i), *reinterpret_cast<const uint2 *>(four));
            }
        } else {
            for (int i = lane; i < L; i += lanes)
                gx[i] = from_f32<T>(value(sum[i + 1], q_of(i + 4)));
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
size_t block_bytes(const Problem &P, int wpr, int rpb, bool fixed, bool staged) {
    return (size_t)rpb * row_words(P, fixed) * 4 + (staged ? (size_t)rpb * wpr * stage_bytes(P) : 0);
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
    const int es = P.dtype == DCN1D_F32 ? 4 : 2;
    a.wide = (int64_t)P.L_out * K % (16 / es) == 0 &&
             ((reinterpret_cast<uintptr_t>(G.off) | reinterpret_cast<uintptr_t>(G.mask)) & 15) == 0;
    a.even = P.L_out % 2 == 0 && ((reinterpret_cast<uintptr_t>(P.off) | reinterpret_cast<uintptr_t>(P.mask) |
                                   reinterpret_cast<uintptr_t>(G.gout)) & 3) == 0;
    // a warp for each 64 positions, up to the block; then as many rows as make a block of
    // 8 warps
    const int longest = P.L_out > P.L_in ? P.L_out : P.L_in;
    a.wpr = 1;
    while (a.wpr < kMaxWarps && a.wpr * 64 < longest)
        a.wpr *= 2;
    // Rows near the limit give up the staging, and at last the bits q, before they give up
    // warps: [2, 148, 17900] fp32, 9 taps with a mask, takes 375 us, and took 978 with the few
    // warps that its staging left room for.
    a.fixed = block_bytes(P, a.wpr, 1, true, false) <= kSmem;
    a.staged = block_bytes(P, a.wpr, 1, a.fixed, true) <= kSmem;
    a.code_words = a.fixed ? code_words_of(P) : 0;
    int rpb = a.wpr < 8 ? 8 / a.wpr : 1;
    while (rpb > 1 && block_bytes(P, a.wpr, rpb, a.fixed, a.staged) > 48 * 1024)
        rpb /= 2;
    const size_t shared = block_bytes(P, a.wpr, rpb, a.fixed, a.staged);
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
           P.B > 0 && block_bytes(P, 1, 1, false, false) <= kSmem && fast_floor_ok(P);
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
