// Layer norm over the channels of x [B, C, L], forward and backward.
//
//   mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps),  v = (x - mean) rstd
//   y = gamma[c] v + beta[c]
// and with d = gamma[c] grad_y, A = sum_c d / C, S = sum_c d v / C:
//   grad_x = rstd (d - A - v S)
//   grad_gamma[c] = sum_{b,l} grad_y v,   grad_beta[c] = sum_{b,l} grad_y
//
// A few flops a value: the bytes bound all of it.  The normalised axis is strided by L in
// memory, so a block takes a tile of neighbouring positions x all channels (or, where they
// are many or tiles few, a cluster's block a slice of the channels): lanes of a warp lie
// along the positions, 16-byte chunks of V = 16 / sizeof(T) of them, and over channels.
// Sums over channels stay in registers, two fp32 values an instruction, until one exchange
// between lanes, warps and, in a cluster, distributed shared memory.
//  * Rows aligned for 16-byte accesses: the stream kernels below.
//  * Other rows: tiles staged in shared memory.
//  * Single tokens (L == 1): rows of C values in registers.
//  * Channels past what a cluster holds, unaligned single tokens: the simple kernels.
//
// The forward takes its sums about a k near the mean, s1 = sum (x - k) and s2 = sum (x -
// k)^2, a k for each warp, and joins groups of n_i values about a common k by
//   s1 = sum_i s1_i + n_i d_i,  s2 = sum_i s2_i + 2 d_i s1_i + n_i d_i^2,  d_i = k_i - k:
// one exchange instead of one for the mean and one for the variance, and no difference of
// large squares however far the mean is from zero (s1 carries what rounding k lost).  Where
// a few large channels put k far from the mean, s2 still cancels; a position at which the
// groups' s2 add up to more than three times what is left takes its sums again about the
// mean just found.  Rounding then costs the variance at most three times what it costs the
// sum of squares about the mean, everywhere, and ordinary values are walked once.
#include <cooperative_groups.h>

#include "checkpoint.cuh"
#include "norm_index.h"
#include "pairs.cuh"
#include "sm100.cuh"

namespace dcn1d {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
static_assert(kAnyThreads == kThreads && kCkBlock == 32, "norm_index.h");
constexpr int kTW = 32;                        // positions of a tile, at most; a block of codes
constexpr int kMaxSplit = 8;                   // blocks of a portable cluster

// How a launch cuts [B, C, L] into tiles.
struct Tiling {
    int tw, tw_log;    // positions of a tile, a power of two
    int lpr_log;       // log2 of the lanes of a row: tw / V
    int split;         // blocks that share the channels of a tile (a cluster)
    int slice;         // channels of a block, a multiple of the rows of its threads
    bool words, code_words;   // rows of T, and of codes, are whole 4-byte words
    int walk_b, walk_l;   // a walk's step over (b, tile of b): the number of clusters
    float inv_c;       // 1 / C
    int64_t tiles;     // tiles of one b
    int64_t total;     // tiles in all
};

template <class T>
__device__ __forceinline__ void chunk_to_f32(const uint4 &u, float (&f)[Vec<T>::V]) {
    const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int j = 0; j < Vec<T>::V; ++j)
        f[j] = to_f32(e[j]);
}

template <class T>
__device__ __forceinline__ uint4 f32_to_chunk(const float (&f)[Vec<T>::V]) {
    uint4 u;
    T *e = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int j = 0; j < Vec<T>::V; ++j)
        e[j] = from_f32<T>(f[j]);
    return u;
}

// Four bytes from global to shared memory without a register; zeros when !in (the source is
// then not read).
__device__ __forceinline__ void copy_async4(void *dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(in ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Where a thread stands in its block's tile.  Chunk k of a tile is row k / lpr, part k % lpr;
// a thread owns chunks threadIdx.x + j kThreads, j < n, so all its shared addresses are
// constants apart.  LPR_LOG < 0: from the tiling.
template <int LPR_LOG>
struct Place {
    int lpr_log, lane, sub, row, stride, n, warp_n;   // warp_n: the largest n of the warp
    __device__ Place(const Tiling &t, int nrow) {
        lpr_log = LPR_LOG >= 0 ? LPR_LOG : t.lpr_log;
        lane = threadIdx.x & 31;
        sub = lane & ((1 << lpr_log) - 1);
        row = (int)threadIdx.x >> lpr_log;
        stride = kThreads >> lpr_log;
        const int shift = __ffs(stride) - 1;
        n = max(0, (nrow - row + stride - 1) >> shift);
        warp_n = max(0, (nrow - ((int)(threadIdx.x & ~31u) >> lpr_log) + stride - 1) >> shift);
    }
};

// A block's rows of `E` values (T, or codes), tw a row, to shared memory: global rows start
// at src + row * L.  Lanes run along the values, each warp over the rows of its threads'
// chunks, and the warp meets afterwards; 4-byte values are copied asynchronously.
template <class E, int V>
__device__ __forceinline__ void load_rows(E *tile, const E *src, int64_t L, int64_t left, int nrow,
                                          const Tiling &t, const Place<-1> &p) {
    const int row0 = (int)(threadIdx.x & ~31u) >> p.lpr_log;   // the warp's first row
#pragma unroll 2
    for (int j = 0; j < p.warp_n; ++j) {
        E *to = tile + ((threadIdx.x & ~31u) + j * kThreads) * V;
        const E *from = src + (row0 + j * p.stride) * L;
        E v[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const int e = p.lane + 32 * q, r = e >> t.tw_log, col = e & (t.tw - 1);
            const bool in = row0 + j * p.stride + r < nrow && col < left;
            if constexpr (sizeof(E) == 4)
                copy_async4(to + e, in ? from + r * L + col : src, in);
            else
                v[q] = in ? from[r * L + col] : E(0.0f);
        }
        if constexpr (sizeof(E) < 4)
#pragma unroll
            for (int q = 0; q < V; ++q)
                to[p.lane + 32 * q] = v[q];
    }
}

// The same rows back to global memory, values along the lanes.
template <class E, int V>
__device__ __forceinline__ void store_rows(const E *tile, E *dst, int64_t L, int64_t left, int nrow,
                                           const Tiling &t, const Place<-1> &p) {
    const int row0 = (int)(threadIdx.x & ~31u) >> p.lpr_log;
#pragma unroll 2
    for (int j = 0; j < p.warp_n; ++j) {
        const E *from = tile + ((threadIdx.x & ~31u) + j * kThreads) * V;
        E *to = dst + (row0 + j * p.stride) * L;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const int e = p.lane + 32 * q, r = e >> t.tw_log, col = e & (t.tw - 1);
            if (row0 + j * p.stride + r < nrow && col < left)
                to[r * L + col] = from[e];
        }
    }
}

// max(|a|, |b|) but for the sign, NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The V codes of a chunk from its values and 1 / step (0: codes 0).  No value is past 127.5
// steps here: the step follows from the block's largest, and these are far from the end of
// the fp32 range.
template <int H>
__device__ __forceinline__ void code_pairs(const Pair (&v)[H], float inverse, uint32_t (&w)[H / 2]) {
    const Pair inv = twice(inverse), magic = twice(kCkRound);
#pragma unroll
    for (int j = 0; j < H / 2; ++j) {
        const float2 a = halves(fma2(v[2 * j], inv, magic)), b = halves(fma2(v[2 * j + 1], inv, magic));
        w[j] = inverse == 0.0f ? 0u : ck_low_bytes(a.x, a.y, b.x, b.y);
    }
}

// V codes as floats.
template <int H>
__device__ __forceinline__ void codes_to_pairs(const uint32_t (&w)[H / 2], Pair (&h)[H]) {
    const Pair bias = twice(-kCkBias);
#pragma unroll
    for (int j = 0; j < H / 2; ++j) {
        const uint32_t f = w[j] ^ 0x80808080u;
        h[2 * j] = add2(pair(ck_biased(f, 0), ck_biased(f, 1)), bias);
        h[2 * j + 1] = add2(pair(ck_biased(f, 2), ck_biased(f, 3)), bias);
    }
}

template <int V>
__device__ __forceinline__ void code_words(const int8_t *p, uint32_t (&w)[V / 4]) {
    if constexpr (V == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x;
        w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

template <int V>
__device__ __forceinline__ void put_code_words(int8_t *p, const uint32_t (&w)[V / 4]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(p) = w[0];
}

// v[i], i < 2H, summed over the lanes that hold the same positions, into part[2][TW] in
// shared memory: the first H for row 0, the others for row 1.  Full rows: by halving
// exchanges (a shuffle for each value that leaves), after which each lane has its share.
template <int H, int LPR_LOG, int TW = kTW>
__device__ __forceinline__ void put_row_sums(Pair (&v)[2 * H], float *part, int lpr_log, int lane,
                                             int sub) {
    constexpr int V = 2 * H;
    if constexpr (LPR_LOG >= 0) {
        // RL lanes hold the same positions; each ends with N = 2H / RL neighbouring sums
        constexpr int RL = 32 >> LPR_LOG, N = 2 * H / RL;
        static_assert(N >= 1 && N * RL == 2 * H, "whole sums a lane");
        const int rl = lane >> LPR_LOG;
#pragma unroll
        for (int m = RL / 2; m >= 1; m >>= 1) {
            const bool upper = rl & m;
#pragma unroll
            for (int j = 0; j < m * N; ++j) {
                const Pair send = upper ? v[j] : v[j + m * N], keep = upper ? v[j + m * N] : v[j];
                v[j] = add2(keep, __shfl_xor_sync(0xFFFFFFFFu, send, m << LPR_LOG));
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = rl * N + j;
            *reinterpret_cast<float2 *>(part + (i >= H ? TW : 0) + sub * V + 2 * (i & (H - 1))) =
                halves(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2 * H; ++j) {
            for (int o = 1 << lpr_log; o < 32; o <<= 1)
                v[j] = add2(v[j], __shfl_xor_sync(0xFFFFFFFFu, v[j], o));
            if (lane < (1 << lpr_log)) {
                const float2 f = halves(v[j]);
                float *to = part + (j >= H ? TW : 0) + sub * V + 2 * (j & (H - 1));
                to[0] = f.x;
                to[1] = f.y;
            }
        }
    }
}

// Sum over eight consecutive lanes.
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums of a group of n values about k; raw: the s2 of the groups it was joined from.
struct Moments {
    float k, s1, s2, raw;
};

// A group of n values a lane of eight (n may be 0, but not in the first lane), joined about
// their common mean, rounded; in every lane.
__device__ __forceinline__ Moments join8(Moments m, float n) {
    const float k0 = __shfl_sync(0xFFFFFFFFu, m.k, threadIdx.x & 24);
    const bool some = n > 0.0f;
    const float all = sum8(n), k = k0 + sum8(some ? fmaf(n, m.k - k0, m.s1) : 0.0f) / fmaxf(all, 1.0f);
    const float d = m.k - k;
    return Moments{k, sum8(some ? fmaf(n, d, m.s1) : 0.0f),
                   sum8(some ? fmaf(d, fmaf(n, d, 2.0f * m.s1), m.s2) : 0.0f),
                   sum8(some ? m.raw : 0.0f)};
}

// A walk of the clusters of a launch over the tiles.
struct Walk {
    int64_t b;
    unsigned lt;
    __device__ Walk(const Tiling &t, unsigned at) {
        b = at / (unsigned)t.tiles;
        lt = at - (unsigned)b * (unsigned)t.tiles;
    }
    __device__ void step(const Tiling &t) {
        b += t.walk_b;
        lt += t.walk_l;
        if (lt >= (unsigned)t.tiles) {
            lt -= (unsigned)t.tiles;
            ++b;
        }
    }
};

constexpr int kFirstRows = 4;   // rows of a lane that give its warp's k

// Rows of a warp of a block's `nrow`, as a float.
template <class P>
__device__ __forceinline__ float warp_rows(const P &p, int nrow) {
    const int rows = 32 >> p.lpr_log;
    int n = 0;
    for (int i = (int)(threadIdx.x & ~31u) >> p.lpr_log; i < nrow; i += p.stride)
        n += min(rows, nrow - i);
    return (float)n;
}

// (-mean, rstd) of C values from their sums, NaN kept (fmaxf drops it), and whether the
// variance cancelled too far (never for NaN and infinities).
__device__ __forceinline__ float2 finish(const Moments &m, const Tiling &t, float eps, bool *far) {
    const float off = m.s1 * t.inv_c, var = fmaxf(m.s2 * t.inv_c - off * off, 0.0f);
    *far = m.raw * t.inv_c > 3.0f * (var + eps) && m.raw < INFINITY && m.s2 == m.s2;
    return make_float2(-(m.k + off), 1.0f / sqrtf((m.s2 == m.s2 ? var : m.s2) + eps));
}

// ---------------------------------------------------------------- unaligned rows
//
// A tile of 32 positions (fewer when L is shorter) x the block's channels in shared memory,
// read and written with the lanes along the values, worked on in 16-byte chunks.  Bound by
// latency at the sizes tested: [3, 381, 1001] fp16 15 us forward and 16 us backward on the
// device (96 tiles, two blocks each).  At [8, 512, ~16000] bf16, where aligned rows take 63 us
// forward and 96 backward: rows of an even length, as 4-byte words, 120 and 211; odd rows,
// value by value, 159 and 279.

// The same in 4-byte words of `E` where rows hold whole words (t.words for T,
// t.code_words for codes): asynchronous copies, and fewer of them.
template <class E, int V>
__device__ __forceinline__ void load_tile(E *tile, const E *src, int64_t L, int64_t left, int nrow,
                                          const Tiling &t, const Place<-1> &p, bool words) {
    constexpr int N = 4 / (int)sizeof(E);
    if (N > 1 && words) {
        Tiling u = t;
        u.tw = t.tw / N;
        u.tw_log = t.tw_log - (N == 4 ? 2 : 1);
        load_rows<uint32_t, V / N>(reinterpret_cast<uint32_t *>(tile),
                                   reinterpret_cast<const uint32_t *>(src), L / N, (left + N - 1) / N,
                                   nrow, u, p);
    } else {
        load_rows<E, V>(tile, src, L, left, nrow, t, p);
    }
}

template <class E, int V>
__device__ __forceinline__ void store_tile(const E *tile, E *dst, int64_t L, int64_t left, int nrow,
                                           const Tiling &t, const Place<-1> &p, bool words) {
    constexpr int N = 4 / (int)sizeof(E);
    if (N > 1 && words) {
        Tiling u = t;
        u.tw = t.tw / N;
        u.tw_log = t.tw_log - (N == 4 ? 2 : 1);
        store_rows<uint32_t, V / N>(reinterpret_cast<const uint32_t *>(tile),
                                    reinterpret_cast<uint32_t *>(dst), L / N, (left + N - 1) / N, nrow,
                                    u, p);
    } else {
        store_rows<E, V>(tile, dst, L, left, nrow, t, p);
    }
}

template <class T, bool CK>
__global__ void __launch_bounds__(kThreads, 3) norm_tile_kernel(const NormProblem P,
                                                                const Tiling t) {
    constexpr int V = Vec<T>::V, H = Vec<T>::H;
    extern __shared__ uint4 tile4[];           // the tile, then its codes
    __shared__ __align__(8) float part[kWarps][2 * kTW];
    __shared__ float part_k[kWarps][kTW], count[kWarps];
    __shared__ Moments own[2][kTW];            // of the block's rows (cluster)
    __shared__ float2 stat[kTW];               // (-mean, rstd)
    const int rank = t.split > 1 ? blockIdx.x % t.split : 0;
    Walk w(t, t.split > 1 ? blockIdx.x / t.split : blockIdx.x);
    const int c0 = rank * t.slice;
    const int nrow = min(t.slice, (int)P.C - c0);   // may be 0 or less in the last blocks
    const Place<-1> p(t, nrow);
    T *tile = reinterpret_cast<T *>(tile4);
    int8_t *ctile = reinterpret_cast<int8_t *>(tile4 + (t.slice << p.lpr_log));
    uint4 *mine = tile4 + threadIdx.x;
    const int64_t nb = ck_blocks(P.L);
    const T *gamma = P.gamma ? static_cast<const T *>(P.gamma) + c0 + p.row : nullptr;
    const T *beta = P.beta ? static_cast<const T *>(P.beta) + c0 + p.row : nullptr;
    const float rows = warp_rows(p, nrow);
    if (p.lane == 0)
        count[threadIdx.x / 32] = rows;
    int turn = 0;
    bool far = false;                          // this thread's position takes its sums again
    for (; w.b < P.B; w.step(t), turn ^= 1) {
        const int64_t l0 = (int64_t)w.lt << t.tw_log;
        const int64_t left = P.L - l0;         // positions of this tile (tw or more: all)
        const int64_t base = (w.b * P.C + c0) * P.L + l0;
        load_tile<T, V>(tile, static_cast<const T *>(P.x) + base, P.L, left, nrow, t, p, t.words);
        copies_landed();
        __syncwarp();
        // k: the mean of the first rows of the warp's first lane of each position
        Pair f[H], k[H], s[2 * H];
        const int first = min(p.n, kFirstRows);
#pragma unroll
        for (int j = 0; j < H; ++j)
            k[j] = 0;
#pragma unroll
        for (int r = 0; r < kFirstRows; ++r)
            if (r < first) {
                chunk_to_pairs<T>(mine[r * kThreads], f);
#pragma unroll
                for (int j = 0; j < H; ++j)
                    k[j] = add2(k[j], f[j]);
            }
        const Pair over = twice(first > 0 ? -1.0f / (float)first : 0.0f);
#pragma unroll
        for (int j = 0; j < H; ++j)
            k[j] = __shfl_sync(0xFFFFFFFFu, mul2(k[j], over), p.sub);   // minus k
        // the sums about k, and once more about the mean where positions need it: those alone
        // take the second walk's result, so that none depends on its neighbours
        for (bool again = false;; again = true, turn ^= 1) {
#pragma unroll
            for (int j = 0; j < 2 * H; ++j)
                s[j] = 0;
#pragma unroll 4
            for (int r = 0; r < p.n; ++r) {
                chunk_to_pairs<T>(mine[r * kThreads], f);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const Pair d = add2(f[j], k[j]);
                    s[j] = add2(s[j], d);
                    s[H + j] = fma2(d, d, s[H + j]);
                }
            }
            put_row_sums<H, -1, kTW>(s, part[threadIdx.x / 32], p.lpr_log, p.lane, p.sub);
            if (p.lane < (1 << p.lpr_log))
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const float2 u = halves(k[j]);
                    part_k[threadIdx.x / 32][p.sub * V + 2 * j] = -u.x;
                    part_k[threadIdx.x / 32][p.sub * V + 2 * j + 1] = -u.y;
                }
            __syncthreads();
            // eight threads a position, one a warp's sums
            static_assert(kThreads == 8 * kTW && kWarps == 8, "a thread for each warp and position");
            const int col = threadIdx.x / 8, g = threadIdx.x % 8;
            const float s2 = part[g][kTW + col];
            Moments m = join8(Moments{part_k[g][col], part[g][col], s2, s2}, count[g]);
            if (t.split > 1) {
                cg::cluster_group cluster = cg::this_cluster();
                if (g == 0)
                    own[turn][col] = m;
                cluster.sync();
                // `own` alternates: a block writes one half while others may read the other,
                // and passes the next barrier only after its reads of this one
                static_assert(kMaxSplit == 8, "a thread for each block");
                if (g < t.split)
                    m = *cluster.map_shared_rank(&own[turn][col], g);
                m = join8(m, g < t.split ? (float)max(0, min(t.slice, (int)P.C - g * t.slice)) : 0.0f);
            }
            bool cancelled = false;
            if (g == 0 && col < min((int64_t)t.tw, left) && (!again || far)) {
                const float2 q = finish(m, t, P.eps, &cancelled);
                far = cancelled;
                stat[col] = q;
                if (rank == 0) {
                    if (P.mean)
                        P.mean[w.b * P.L + l0 + col] = -q.x;
                    if (P.rstd)
                        P.rstd[w.b * P.L + l0 + col] = q.y;
                }
            }
            // the same in every block of the cluster: they joined the same numbers
            if (!__syncthreads_or(cancelled && !again))
                break;
#pragma unroll
            for (int j = 0; j < H; ++j)
                k[j] = pair(stat[p.sub * V + 2 * j].x, stat[p.sub * V + 2 * j + 1].x);
        }
        Pair rstd[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const float2 u = stat[p.sub * V + 2 * j], v = stat[p.sub * V + 2 * j + 1];
            k[j] = pair(u.x, v.x);
            rstd[j] = pair(u.y, v.y);
        }
        uint8_t *scale = P.scales + (w.b * P.C + c0 + p.row) * nb + l0 / kCkBlock;
        // CK: whole warps walk together, for the block maximum's shuffles
        const int n = CK ? p.warp_n : p.n;
#pragma unroll 2
        for (int r = 0; r < n; ++r) {
            const bool row = !CK || r < p.n;
            Pair v[H];
            chunk_to_pairs<T>(mine[r * kThreads], v);   // rows past nrow: inside the tile, not used
            const Pair g = twice(gamma && row ? ld_f32(gamma + r * p.stride) : 1.0f);
            const Pair be = twice(beta && row ? ld_f32(beta + r * p.stride) : 0.0f);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                v[j] = mul2(add2(v[j], k[j]), rstd[j]);
                f[j] = fma2(v[j], g, be);
            }
            if (row)
                mine[r * kThreads] = pairs_to_chunk<T>(f);
            if constexpr (CK) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < H; ++j) {  // without the values past the row's end
                    float2 a = halves(v[j]);
                    a.x = p.sub * V + 2 * j < left ? a.x : 0.0f;
                    a.y = p.sub * V + 2 * j + 1 < left ? a.y : 0.0f;
                    v[j] = pair(a.x, a.y);
                    top = max_abs(max_abs(top, a.x), a.y);
                }
                uint32_t bits = row ? ck_abs_bits(top) : 0u;
                for (int o = 1; o < (1 << p.lpr_log); o <<= 1)   // a tile's row is a block of codes
                    bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
                const uint32_t e = ck_scale(bits, ck_top<float>());
                uint32_t q[V / 4];
                code_pairs<H>(v, ck_inverse(e), q);
                put_code_words<V>(ctile + (threadIdx.x + r * kThreads) * V, q);
                if (row && p.sub == 0)
                    scale[r * p.stride * nb] = (uint8_t)e;
            }
        }
        __syncwarp();
        store_tile<T, V>(tile, static_cast<T *>(P.y) + base, P.L, left, nrow, t, p, t.words);
        if constexpr (CK)
            store_tile<int8_t, V>(ctile, P.codes + base, P.L, left, nrow, t, p, t.code_words);
        __syncwarp();   // the next tile's values overwrite what the warp has read
    }
    if (t.split > 1)
        cg::this_cluster().sync();   // another block may still read this one's `own`
}

// Shared memory of the forward's tile kernel for a channel.
template <class T> constexpr int norm_row_bytes(int tw, bool ck) {
    return tw * ((int)sizeof(T) + (ck ? 1 : 0));
}

// The same of the gradient's: grad_y and x (or codes), each lane's sums of grad_y v and
// grad_y of its rows, and gamma with the step of the codes.
template <class T> constexpr int grad_row_bytes(int tw, bool ck) {
    return tw * ((int)sizeof(T) + (ck ? 1 : (int)sizeof(T))) + tw / Vec<T>::V * 8 + 8;
}

// A cluster of t.split blocks walks tiles cluster, cluster + n, ...; each lane's sums of
// grad_y v and grad_y over its rows and the walk stay in shared memory and are joined at
// the end into the cluster's rows of `part_g` [clusters][2][C]: a fixed order, no atomics.
template <class T, bool CK>
__global__ void __launch_bounds__(kThreads, 3) norm_grad_tile_kernel(const NormGrad P,
                                                                     const Tiling t,
                                                                     float *part_g) {
    constexpr int V = Vec<T>::V, H = Vec<T>::H;
    extern __shared__ uint4 tile4[];           // chunks of grad_y, then of x / codes
    __shared__ __align__(8) float part[kWarps][2 * kTW];
    __shared__ float2 own[2][kTW];
    __shared__ float2 stat[kTW];               // (-A, -S)
    const int rank = t.split > 1 ? blockIdx.x % t.split : 0;
    const unsigned cluster_at = t.split > 1 ? blockIdx.x / t.split : blockIdx.x;
    const int c0 = rank * t.slice;
    const int nrow = min(t.slice, (int)P.C - c0);
    const Place<-1> p(t, nrow);
    const int chunks = t.slice << p.lpr_log;
    T *gtile = reinterpret_cast<T *>(tile4);
    uint4 *after = tile4 + chunks;
    T *xtile = reinterpret_cast<T *>(after);
    int8_t *ctile = reinterpret_cast<int8_t *>(after);
    Pair *acc = reinterpret_cast<Pair *>(reinterpret_cast<unsigned char *>(after) +
                                         (size_t)chunks * V * (CK ? 1 : sizeof(T)));   // a chunk
    float2 *scaled = reinterpret_cast<float2 *>(acc + chunks);        // a row: gamma, step
    const int64_t nb = ck_blocks(P.L);
    const T *gamma = P.gamma ? static_cast<const T *>(P.gamma) + c0 : nullptr;
    for (int r = 0; r < p.n; ++r) {
        acc[threadIdx.x + r * kThreads] = 0;
        const int i = p.row + r * p.stride;
        if (p.sub == 0)
            scaled[i] = make_float2(gamma ? ld_f32(gamma + i) : 1.0f, 1.0f);
    }
    const uint4 *gmine = tile4 + threadIdx.x, *xmine = after + threadIdx.x;
    const int8_t *cmine = ctile + threadIdx.x * V;
    const float2 *smine = scaled + p.row;
    int turn = 0;
    for (Walk w(t, cluster_at); w.b < P.B; w.step(t), turn ^= 1) {
        const int64_t l0 = (int64_t)w.lt << t.tw_log;
        const int64_t left = P.L - l0;
        const int64_t base = (w.b * P.C + c0) * P.L + l0;
        load_tile<T, V>(gtile, static_cast<const T *>(P.gy) + base, P.L, left, nrow, t, p, t.words);
        if constexpr (CK) {
            load_tile<int8_t, V>(ctile, P.codes + base, P.L, left, nrow, t, p, t.code_words);
            const uint8_t *from = P.scales + (w.b * P.C + c0 + p.row) * nb + l0 / kCkBlock;
            if (p.sub == 0)
#pragma unroll 4
                for (int r = 0; r < p.n; ++r)
                    scaled[p.row + r * p.stride].y = ck_step(from[r * p.stride * nb]);
        } else {
            load_tile<T, V>(xtile, static_cast<const T *>(P.x) + base, P.L, left, nrow, t, p, t.words);
        }
        Pair rstd[H], neg[H];                  // neg: minus the mean
        const float *rs = P.rstd + w.b * P.L + l0 + p.sub * V, *me = nullptr;
        if constexpr (!CK)
            me = P.mean + w.b * P.L + l0 + p.sub * V;
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const bool u = p.sub * V + j < left, v = p.sub * V + j + 1 < left;
            rstd[j / 2] = pair(u ? __ldg(rs + j) : 0.0f, v ? __ldg(rs + j + 1) : 0.0f);
            neg[j / 2] = 0;
            if constexpr (!CK)
                neg[j / 2] = pair(u ? -__ldg(me + j) : 0.0f, v ? -__ldg(me + j + 1) : 0.0f);
        }
        copies_landed();
        __syncwarp();
        // v of a row's chunk, but for the step of its codes
        auto values = [&](int r, Pair (&h)[H]) {
            if constexpr (CK) {
                uint32_t words[V / 4];
                code_words<V>(cmine + r * kThreads * V, words);
                codes_to_pairs<H>(words, h);
            } else {
                chunk_to_pairs<T>(xmine[r * kThreads], h);
#pragma unroll
                for (int j = 0; j < H; ++j)
                    h[j] = mul2(add2(h[j], neg[j]), rstd[j]);
            }
        };
        // the checkpoint's v is h step, with one step a row: gamma gy v = (gy h) (gamma step)
        Pair s[2 * H];
#pragma unroll
        for (int j = 0; j < 2 * H; ++j)
            s[j] = 0;
#pragma unroll 2
        for (int r = 0; r < p.n; ++r) {
            Pair g[H], h[H], sg = 0, sb = 0;
            chunk_to_pairs<T>(gmine[r * kThreads], g);
            const float2 f = smine[r * p.stride];
            values(r, h);
            const Pair w2 = twice(f.x), ws = twice(CK ? f.x * f.y : f.x);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const Pair gh = mul2(g[j], h[j]);
                s[j] = fma2(g[j], w2, s[j]);
                s[H + j] = fma2(gh, ws, s[H + j]);
                sg = j ? add2(sg, gh) : gh;
                sb = j ? add2(sb, g[j]) : g[j];
            }
            if (part_g) {
                const float2 x = halves(sg), y = halves(sb);
                Pair *to = acc + threadIdx.x + r * kThreads;
                *to = add2(*to, pair(CK ? (x.x + x.y) * f.y : x.x + x.y, y.x + y.y));
            }
        }
        if (P.gx) {
            put_row_sums<H, -1, kTW>(s, part[threadIdx.x / 32], p.lpr_log, p.lane, p.sub);
            __syncthreads();
            {   // eight threads a position, one a warp's sums
                const int col = threadIdx.x / 8, g = threadIdx.x % 8;
                float2 sum = make_float2(sum8(part[g][col]), sum8(part[g][kTW + col]));
                if (t.split > 1) {
                    // `own` alternates: a block writes one half while others may read the
                    // other, and passes the next barrier only after its reads of this one
                    cg::cluster_group cluster = cg::this_cluster();
                    if (g == 0)
                        own[turn][col] = sum;
                    cluster.sync();
                    sum = make_float2(0.0f, 0.0f);
                    if (g < t.split)
                        sum = *cluster.map_shared_rank(&own[turn][col], g);
                    sum = make_float2(sum8(sum.x), sum8(sum.y));
                }
                if (g == 0)
                    stat[col] = make_float2(-sum.x * t.inv_c, -sum.y * t.inv_c);
            }
            __syncthreads();
            // grad_x = rstd gamma gy - rstd A - v rstd S
            Pair rA[H], rS[H];
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float2 u = stat[p.sub * V + 2 * j], v = stat[p.sub * V + 2 * j + 1];
                rA[j] = mul2(pair(u.x, v.x), rstd[j]);
                rS[j] = mul2(pair(u.y, v.y), rstd[j]);
            }
#pragma unroll 2
            for (int r = 0; r < p.n; ++r) {
                Pair g[H], h[H];
                chunk_to_pairs<T>(gmine[r * kThreads], g);
                const float2 f = smine[r * p.stride];
                values(r, h);
                const Pair w2 = twice(f.x), st = twice(f.y);   // st: 1 without a checkpoint
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    if constexpr (CK)
                        h[j] = mul2(h[j], st);
                    g[j] = fma2(h[j], rS[j], fma2(mul2(g[j], w2), rstd[j], rA[j]));
                }
                tile4[threadIdx.x + r * kThreads] = pairs_to_chunk<T>(g);
            }
            __syncwarp();
            store_tile<T, V>(gtile, static_cast<T *>(P.gx) + base, P.L, left, nrow, t, p, t.words);
        }
        __syncwarp();   // the next tile's values and steps overwrite what the warp has read
    }
    if (part_g) {
        float *out = part_g + (int64_t)cluster_at * 2 * P.C + c0;
        for (int r = 0; r < p.warp_n; ++r) {
            Pair v = r < p.n ? acc[threadIdx.x + r * kThreads] : 0;
            for (int o = 1; o < (1 << p.lpr_log); o <<= 1)
                v = add2(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            const int i = p.row + r * p.stride;
            if (r < p.n && p.sub == 0) {
                const float2 f = halves(v);
                out[i] = f.x;
                out[P.C + i] = f.y;
            }
        }
    }
    if (t.split > 1)
        cg::this_cluster().sync();   // another block may still read this one's `own`
}

// ---------------------------------------------------------------- aligned rows
//
// Where rows are aligned for 16-byte chunks nothing is staged: a block walks the channels of
// a tile of 64 positions (fp32: 32; 128 bytes of a row) twice, and the second walk finds the
// tile in the L1 or the L2 (a tile of 512 channels is 64 KB, of 1024 with grad_y and codes
// 192 KB).  That leaves the shared memory to the L1, needs no copies, takes any number of
// channels, and lets 16 to 32 warps an SM hide the latencies.
//
// Measured (B200, 1965 MHz): the forward of [8, 512, 16000] bf16 63.9 us = 4.1 TB/s, 0.63 of
// the copy bandwidth (79 us where channels lie far out and the sums are taken twice); the
// gradient from the checkpoint of [32, 1024, 8192] bf16 317 us = 4.3
// TB/s, 0.65.  DRAM moves only what it must; the loads' latency is the limit (6 of 13 cycles
// a warp between two instructions in the forward), and the gradient's 23 instructions a
// value next to it.  Tiles staged in shared memory with the next one's copies under way took
// 65 and 645 us (their exchange between warps is paid for half as many positions), a tile
// held in registers 75 us (too few warps), L2 prefetches of the next tile 72 and 460 us.

constexpr int kStreamTW = 64;
// Rows whose loads a thread has in flight.  Forward: 4 rows and 32 warps an SM 62.8 us, 2 rows
// 64.6, 8 rows and 16 warps 74.  Gradient: 8 rows and 16 warps 327 us, 4 rows and 24 warps 418.
constexpr int kRows = 4, kGradRows = 8;

// With the codes three blocks an SM: four leave too few registers (forward and gradient of
// [8, 512, 16000] bf16 181 us, with three 175).
template <class T, bool CK, int LPR_LOG>
__global__ void __launch_bounds__(kThreads, CK ? 3 : 4) norm_stream_kernel(const NormProblem P,
                                                                  const Tiling t) {
    constexpr int V = Vec<T>::V, H = Vec<T>::H;
    __shared__ __align__(8) float part[kWarps][2 * kStreamTW], part_k[kWarps][kStreamTW], count[kWarps];
    __shared__ Moments own[2][kStreamTW];      // of the block's rows (cluster), a walk's each
    __shared__ float2 stat[kStreamTW];         // (-mean, rstd)
    const int rank = t.split > 1 ? blockIdx.x % t.split : 0;
    const Walk w(t, t.split > 1 ? blockIdx.x / t.split : blockIdx.x);
    const int c0 = rank * t.slice;
    const int nrow = min(t.slice, (int)P.C - c0);   // may be 0 or less in the last blocks
    const Place<LPR_LOG> p(t, nrow);
    const int64_t l0 = (int64_t)w.lt << t.tw_log, left = P.L - l0;
    const int64_t base = (w.b * P.C + c0) * P.L + l0;
    const bool in = p.sub * V < left;
    // lanes past the end of the row, and of the slice, read the first values of b, for nothing
    const T *safe = static_cast<const T *>(P.x) + w.b * P.C * P.L;
    const T *x0 = in && p.n > 0 ? static_cast<const T *>(P.x) + base + p.row * P.L + p.sub * V : safe;
    const int64_t hop = p.stride * P.L, x_hop = in ? hop : 0;
    const float rows = warp_rows(p, nrow);
    if (p.lane == 0)
        count[threadIdx.x / 32] = rows;
    auto chunk = [](const T *at) { return __ldg(reinterpret_cast<const uint4 *>(at)); };
    // k: the mean of the first rows of the warp's first lane of each position
    Pair f[H], k[H], s[2 * H];
    const int first = min(p.n, kFirstRows);
#pragma unroll
    for (int j = 0; j < H; ++j)
        k[j] = 0;
#pragma unroll
    for (int r = 0; r < kFirstRows; ++r)
        if (r < first) {
            chunk_to_pairs<T>(chunk(x0 + r * x_hop), f);
#pragma unroll
            for (int j = 0; j < H; ++j)
                k[j] = add2(k[j], f[j]);
        }
    const Pair over = twice(first > 0 ? -1.0f / (float)first : 0.0f);
#pragma unroll
    for (int j = 0; j < H; ++j)
        k[j] = __shfl_sync(0xFFFFFFFFu, mul2(k[j], over), p.sub);   // minus k
    auto add_row = [&](const uint4 &u) {
        chunk_to_pairs<T>(u, f);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const Pair d = add2(f[j], k[j]);
            s[j] = add2(s[j], d);
            s[H + j] = fma2(d, d, s[H + j]);
        }
    };
    uint32_t far = 0;                          // bit i: this thread's i-th position, below
    // the sums about k, and once more about the mean where positions need it: those alone take
    // the second walk's result, so that none depends on its neighbours
    for (int again = 0;; again = 1) {
#pragma unroll
        for (int j = 0; j < 2 * H; ++j)
            s[j] = 0;
        const T *x = x0;
        int r = 0;
        for (; r + kRows <= p.n; r += kRows) {
            uint4 u[kRows];
#pragma unroll
            for (int q = 0; q < kRows; ++q, x += x_hop)
                u[q] = chunk(x);
#pragma unroll
            for (int q = 0; q < kRows; ++q)
                add_row(u[q]);
        }
        for (; r < p.n; ++r, x += x_hop)
            add_row(chunk(x));
        put_row_sums<H, LPR_LOG, kStreamTW>(s, part[threadIdx.x / 32], p.lpr_log, p.lane, p.sub);
        if (p.lane < (1 << p.lpr_log))
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float2 u = halves(k[j]);
                part_k[threadIdx.x / 32][p.sub * V + 2 * j] = -u.x;
                part_k[threadIdx.x / 32][p.sub * V + 2 * j + 1] = -u.y;
            }
        __syncthreads();
        // eight threads a position, one a warp's sums
        for (int c = threadIdx.x / 8; c < t.tw; c += kThreads / 8) {
            const int g = threadIdx.x % 8;
            const float s2 = part[g][kStreamTW + c];
            const Moments m = join8(Moments{part_k[g][c], part[g][c], s2, s2}, count[g]);
            if (g == 0)
                own[again][c] = m;
        }
        if (t.split > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
        uint32_t cancelled = 0, bit = 1;
        for (int c = threadIdx.x / 8; c < t.tw; c += kThreads / 8, bit <<= 1) {
            const int g = threadIdx.x % 8;
            Moments m = own[again][c];
            if (t.split > 1) {
                static_assert(kMaxSplit == 8, "a thread for each block");
                if (g < t.split)
                    m = *cg::this_cluster().map_shared_rank(&own[again][c], g);
                m = join8(m, g < t.split ? (float)max(0, min(t.slice, (int)P.C - g * t.slice)) : 0.0f);
            }
            if (g == 0 && c < left && (!again || (far & bit))) {
                bool more;
                const float2 q = finish(m, t, P.eps, &more);
                cancelled |= more ? bit : 0u;
                stat[c] = q;
                if (rank == 0) {
                    if (P.mean)
                        P.mean[w.b * P.L + l0 + c] = -q.x;
                    if (P.rstd)
                        P.rstd[w.b * P.L + l0 + c] = q.y;
                }
            }
        }
        far = cancelled;
        // the same in every block of the cluster: they joined the same numbers
        if (!__syncthreads_or(!again && cancelled))
            break;
#pragma unroll
        for (int j = 0; j < H; ++j)
            k[j] = pair(stat[p.sub * V + 2 * j].x, stat[p.sub * V + 2 * j + 1].x);
    }
    Pair rstd[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const float2 u = stat[p.sub * V + 2 * j], v = stat[p.sub * V + 2 * j + 1];
        k[j] = pair(u.x, v.x);
        rstd[j] = pair(u.y, v.y);
    }
    const int64_t nb = ck_blocks(P.L);
    const int lanes = min(kCkBlock / V, 1 << p.lpr_log);   // lanes of a block of 32 values
    const T *gamma = P.gamma ? static_cast<const T *>(P.gamma) + c0 + p.row : nullptr;
    const T *beta = P.beta ? static_cast<const T *>(P.beta) + c0 + p.row : nullptr;
    T *y = static_cast<T *>(P.y) + base + p.row * P.L + p.sub * V;
    int8_t *codes = P.codes + base + p.row * P.L + p.sub * V;
    uint8_t *scale = P.scales + (w.b * P.C + c0 + p.row) * nb + (l0 + p.sub * V) / kCkBlock;
    const int64_t scale_hop = p.stride * nb;
    auto put_row = [&](const uint4 &u, int at, bool row) {
        Pair v[H];
        chunk_to_pairs<T>(u, v);
        const Pair g = twice(gamma && row ? ld_f32(gamma + at * p.stride) : 1.0f);
        const Pair be = twice(beta && row ? ld_f32(beta + at * p.stride) : 0.0f);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            v[j] = mul2(add2(v[j], k[j]), rstd[j]);
            f[j] = fma2(v[j], g, be);
        }
        const uint4 o = pairs_to_chunk<T>(f);
        if (row && in)
            *reinterpret_cast<uint4 *>(y) = o;
        y += hop;
        if constexpr (CK) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float2 a = halves(v[j]);
                top = max_abs(max_abs(top, a.x), a.y);
            }
            uint32_t bits = row && in ? ck_abs_bits(top) : 0u;
            if constexpr (LPR_LOG >= 0) {
#pragma unroll
                for (int o2 = 1; o2 < kCkBlock / V; o2 <<= 1)
                    bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o2));
            } else {
                for (int o2 = 1; o2 < lanes; o2 <<= 1)
                    bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o2));
            }
            const uint32_t e = ck_scale(bits, ck_top<float>());
            uint32_t q[V / 4];
            code_pairs<H>(v, ck_inverse(e), q);
            if (row && in) {
                put_code_words<V>(codes, q);
                if ((p.sub & (lanes - 1)) == 0)
                    *scale = (uint8_t)e;
            }
            codes += hop;
            scale += scale_hop;
        }
    };
    const T *x = x0;
    int r = 0;
    const int full = CK ? __shfl_sync(0xFFFFFFFFu, p.n, 31) : p.n;   // the warp's smallest
    for (; r + kRows <= full; r += kRows) {
        uint4 u[kRows];
#pragma unroll
        for (int q = 0; q < kRows; ++q, x += x_hop)
            u[q] = chunk(x);
#pragma unroll
        for (int q = 0; q < kRows; ++q)
            put_row(u[q], r + q, true);
    }
    // CK: whole warps walk together, for the block maximum's shuffles
    for (; r < (CK ? p.warp_n : p.n); ++r, x += x_hop) {
        const bool row = r < p.n;
        put_row(chunk(row ? x : safe), r, row);
    }
    if (t.split > 1)
        cg::this_cluster().sync();   // another block may still read this one's `own`
}

// A cluster of t.split blocks walks tiles cluster, cluster + n, ...; the sums of grad_y v
// and grad_y over the walk stay in shared memory, a row of a warp's lanes each, and go to the
// cluster's rows of `part_g` [clusters][2][C] at the end: a fixed order, no atomics.
template <class T, bool CK, int LPR_LOG>
__global__ void __launch_bounds__(kThreads, 2) norm_grad_stream_kernel(const NormGrad P,
                                                                       const Tiling t,
                                                                       float *part_g) {
    constexpr int V = Vec<T>::V, H = Vec<T>::H;
    extern __shared__ uint4 tile4[];
    __shared__ __align__(8) float part[kWarps][2 * kStreamTW];
    __shared__ float2 own[2][kStreamTW];
    __shared__ float2 stat[kStreamTW];         // (-A, -S)
    const int rank = t.split > 1 ? blockIdx.x % t.split : 0;
    const unsigned cluster_at = t.split > 1 ? blockIdx.x / t.split : blockIdx.x;
    const int c0 = rank * t.slice;
    const int nrow = min(t.slice, (int)P.C - c0);
    const Place<LPR_LOG> p(t, nrow);
    Pair *acc = reinterpret_cast<Pair *>(tile4);               // [slice]: sums of a row
    float *gam = reinterpret_cast<float *>(acc + t.slice);     // [slice]
    const int64_t nb = ck_blocks(P.L);
    for (int i = threadIdx.x; i < nrow; i += kThreads) {
        acc[i] = 0;
        gam[i] = P.gamma ? ld_f32(static_cast<const T *>(P.gamma) + c0 + i) : 1.0f;
    }
    __syncthreads();
    const int64_t hop = p.stride * P.L, scale_hop = p.stride * nb;
    const int full = __shfl_sync(0xFFFFFFFFu, p.n, 31);        // the warp's smallest n
    int turn = 0;
    for (Walk w(t, cluster_at); w.b < P.B; w.step(t), turn ^= 1) {
        const int64_t l0 = (int64_t)w.lt << t.tw_log, left = P.L - l0;
        const int64_t base = (w.b * P.C + c0) * P.L + l0;
        const bool in = p.sub * V < left;
        // lanes past the end of the row, and of the slice, read the tile's first chunk
        const int64_t safe = w.b * P.C * P.L;
        const int64_t mine = in && p.n > 0 ? base + p.row * P.L + p.sub * V : safe;
        const int64_t v_hop = in ? hop : 0, e_hop = in ? scale_hop : 0;
        const T *g0 = static_cast<const T *>(P.gy) + mine;
        const T *x0 = static_cast<const T *>(P.x) + (CK ? 0 : mine);
        const int8_t *c0p = P.codes + (CK ? mine : 0);
        const uint8_t *e0 = P.scales;
        if (CK)
            e0 += in && p.n > 0 ? (w.b * P.C + c0 + p.row) * nb + (l0 + p.sub * V) / kCkBlock
                                : w.b * P.C * nb;
        Pair rstd[H], neg[H];                  // neg: minus the mean
        {
            const float *rs = P.rstd + w.b * P.L + (in ? l0 + p.sub * V : 0);
            const float *me = CK ? nullptr : P.mean + w.b * P.L + (in ? l0 + p.sub * V : 0);
#pragma unroll
            for (int j = 0; j < H; j += 2) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(rs) + j / 2);
                rstd[j] = in ? pair(u.x, u.y) : 0;
                rstd[j + 1] = in ? pair(u.z, u.w) : 0;
                neg[j] = neg[j + 1] = 0;
                if constexpr (!CK) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(me) + j / 2);
                    neg[j] = pair(-v.x, -v.y);
                    neg[j + 1] = pair(-v.z, -v.w);
                }
            }
        }
        // kGradRows rows' loads, then their use: a walk of this lane's rows
        struct Row {
            uint4 g, x;                        // CK: x.x, x.y the codes, x.w the step byte
        };
        auto fetch = [&](int r) {
            Row u;
            u.g = __ldg(reinterpret_cast<const uint4 *>(g0 + r * v_hop));
            if constexpr (CK) {
                uint32_t q[V / 4];
                code_words<V>(c0p + r * v_hop, q);
                u.x.x = q[0];
                u.x.y = q[V / 4 - 1];
                u.x.w = __ldg(e0 + r * e_hop);
            } else {
                u.x = __ldg(reinterpret_cast<const uint4 *>(x0 + r * v_hop));
            }
            return u;
        };
        auto open = [&](const Row &u, Pair (&g)[H], Pair (&h)[H]) {
            chunk_to_pairs<T>(u.g, g);
            if constexpr (CK) {
                uint32_t q[V / 4];
                q[0] = u.x.x;
                q[V / 4 - 1] = u.x.y;
                codes_to_pairs<H>(q, h);
            } else {
                chunk_to_pairs<T>(u.x, h);
#pragma unroll
                for (int j = 0; j < H; ++j)
                    h[j] = mul2(add2(h[j], neg[j]), rstd[j]);
            }
        };
        // the checkpoint's v is h step, with one step a chunk: gamma gy v = (gy h) (gamma step)
        Pair s[2 * H];
#pragma unroll
        for (int j = 0; j < 2 * H; ++j)
            s[j] = 0;
        auto add_row = [&](const Row &u, float w1) {   // returns (sum gy v, sum gy)
            Pair g[H], h[H], sg = 0, sb = 0;
            open(u, g, h);
            const float st = CK ? ck_step(u.x.w) : 1.0f;
            const Pair w2 = twice(w1), ws = twice(CK ? w1 * st : w1);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const Pair gh = mul2(g[j], h[j]);
                s[j] = fma2(g[j], w2, s[j]);
                s[H + j] = fma2(gh, ws, s[H + j]);
                sg = j ? add2(sg, gh) : gh;
                sb = j ? add2(sb, g[j]) : g[j];
            }
            const float2 a = halves(sg), b = halves(sb);
            return in ? pair(CK ? (a.x + a.y) * st : a.x + a.y, b.x + b.y) : Pair(0);
        };
        int r = 0;
        for (; r + kGradRows <= full; r += kGradRows) {
            Row u[kGradRows];
            Pair a[kGradRows];
#pragma unroll
            for (int q = 0; q < kGradRows; ++q)
                u[q] = fetch(r + q);
#pragma unroll
            for (int q = 0; q < kGradRows; ++q)
                a[q] = add_row(u[q], gam[p.row + (r + q) * p.stride]);
            if (part_g) {
                if constexpr (LPR_LOG == 3) {
                    // eight rows over eight lanes, by halving exchanges: lane sub has row sub
#pragma unroll
                    for (int m = 4; m >= 1; m >>= 1) {
                        const bool upper = p.sub & m;
#pragma unroll
                        for (int q = 0; q < m; ++q)
                            a[q] = add2(upper ? a[q + m] : a[q],
                                        __shfl_xor_sync(0xFFFFFFFFu, upper ? a[q] : a[q + m], m));
                    }
                    Pair *to = acc + p.row + (r + p.sub) * p.stride;
                    *to = add2(*to, a[0]);
                } else {
#pragma unroll
                    for (int q = 0; q < kGradRows; ++q) {
                        for (int o = 1; o < (1 << p.lpr_log); o <<= 1)
                            a[q] = add2(a[q], __shfl_xor_sync(0xFFFFFFFFu, a[q], o));
                        if (p.sub == 0) {
                            Pair *to = acc + p.row + (r + q) * p.stride;
                            *to = add2(*to, a[q]);
                        }
                    }
                }
            }
        }
        for (; r < p.warp_n; ++r) {
            const bool row = r < p.n;
            Pair a = row ? add_row(fetch(r), gam[p.row + r * p.stride]) : 0;
            if (part_g) {
                for (int o = 1; o < (1 << p.lpr_log); o <<= 1)
                    a = add2(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
                if (row && p.sub == 0) {
                    Pair *to = acc + p.row + r * p.stride;
                    *to = add2(*to, a);
                }
            }
        }
        if (!P.gx)
            continue;
        put_row_sums<H, LPR_LOG, kStreamTW>(s, part[threadIdx.x / 32], p.lpr_log, p.lane, p.sub);
        __syncthreads();
        for (int c = threadIdx.x / 8; c < t.tw; c += kThreads / 8) {
            const int q = threadIdx.x % 8;     // eight threads a position, one a warp's sums
            const float2 sum = make_float2(sum8(part[q][c]), sum8(part[q][kStreamTW + c]));
            if (q == 0)
                own[turn][c] = sum;
            if (t.split == 1 && q == 0)
                stat[c] = make_float2(-sum.x * t.inv_c, -sum.y * t.inv_c);
        }
        if (t.split > 1) {
            // `own` alternates: a block writes one half while others may read the other, and
            // passes the next barrier only after its reads of this one
            cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            for (int c = threadIdx.x / 8; c < t.tw; c += kThreads / 8) {
                const int q = threadIdx.x % 8;
                float2 sum = make_float2(0.0f, 0.0f);
                if (q < t.split)
                    sum = *cluster.map_shared_rank(&own[turn][c], q);
                sum = make_float2(sum8(sum.x), sum8(sum.y));
                if (q == 0)
                    stat[c] = make_float2(-sum.x * t.inv_c, -sum.y * t.inv_c);
            }
        }
        __syncthreads();
        // grad_x = rstd gamma gy - rstd A - v rstd S
        Pair rA[H], rS[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const float2 u = stat[p.sub * V + 2 * j], v = stat[p.sub * V + 2 * j + 1];
            rA[j] = mul2(pair(u.x, v.x), rstd[j]);
            rS[j] = mul2(pair(u.y, v.y), rstd[j]);
        }
        T *out = static_cast<T *>(P.gx) + base + p.row * P.L + p.sub * V;
        auto put_row = [&](const Row &u, int at) {
            Pair g[H], h[H];
            open(u, g, h);
            const Pair w2 = twice(gam[p.row + at * p.stride]);
            if constexpr (CK) {
                const Pair st = twice(ck_step(u.x.w));
#pragma unroll
                for (int j = 0; j < H; ++j)
                    h[j] = mul2(h[j], st);
            }
#pragma unroll
            for (int j = 0; j < H; ++j)
                g[j] = fma2(h[j], rS[j], fma2(mul2(g[j], w2), rstd[j], rA[j]));
            if (in)
                __stcs(reinterpret_cast<uint4 *>(out), pairs_to_chunk<T>(g));   // not to be kept
            out += hop;
        };
        r = 0;
        for (; r + kGradRows <= p.n; r += kGradRows) {
            Row u[kGradRows];
#pragma unroll
            for (int q = 0; q < kGradRows; ++q)
                u[q] = fetch(r + q);
#pragma unroll
            for (int q = 0; q < kGradRows; ++q)
                put_row(u[q], r + q);
        }
        for (; r < p.n; ++r)
            put_row(fetch(r), r);
    }
    if (part_g) {
        __syncthreads();
        float *out = part_g + (int64_t)cluster_at * 2 * P.C + c0;
        for (int i = threadIdx.x; i < nrow; i += kThreads) {
            const float2 f = halves(acc[i]);
            out[i] = f.x;
            out[P.C + i] = f.y;
        }
    }
    if (t.split > 1)
        cg::this_cluster().sync();   // another block may still read this one's `own`
}

// ---------------------------------------------------------------- rows of C values (L == 1)
//
// TPR threads (a warp, or the block) take a row and hold it in registers, NV 16-byte chunks
// a thread: every value is read once.  One token of 512 channels: 4.3 us on the device, the
// latency of a launch, one load and two reductions.  16384 rows of 1000 values in bf16: 16 us
// forward (host included), 28 backward (65 without the next row under way); of 4096, 64 and
// 100 us, 0.64 of the copy bandwidth.

// Sum over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (&part)[kWarps]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (TPR == kThreads) {
        __syncthreads();   // the last use of `part` is over
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += part[w];
    }
    return v;
}

template <class T, int TPR, int NV>
__global__ void __launch_bounds__(kThreads) norm_row_kernel(const NormProblem P) {
    constexpr int V = Vec<T>::V;
    __shared__ float part[kWarps];
    const int tid = threadIdx.x % TPR;
    const int64_t b = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    if (b >= P.B)   // whole warps, or (TPR == kThreads) never
        return;
    const int C = (int)P.C;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(P.x) + b * C);
    uint4 u[NV];
    float f[V], s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = k * TPR + tid;
        u[k] = i * V < C ? __ldg(x + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        chunk_to_f32<T>(u[k], f);
#pragma unroll
        for (int j = 0; j < V; ++j)
            s += f[j];
    }
    const float mean = row_sum<TPR>(s, part) / (float)C;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        chunk_to_f32<T>(u[k], f);
        if ((k * TPR + tid) * V < C)
#pragma unroll
            for (int j = 0; j < V; ++j)
                s = fmaf(f[j] - mean, f[j] - mean, s);
    }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, part) / (float)C + P.eps);
    if (tid == 0) {
        if (P.mean)
            P.mean[b] = mean;
        if (P.rstd)
            P.rstd[b] = rstd;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = k * TPR + tid;
        const bool in = i * V < C;
        float v[V], g[V], be[V];
        chunk_to_f32<T>(u[k], v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = in ? (v[j] - mean) * rstd : 0.0f;
            g[j] = 1.0f;
            be[j] = 0.0f;
        }
        if (in) {
            if (P.gamma)
                chunk_to_f32<T>(__ldg(static_cast<const uint4 *>(P.gamma) + i), g);
            if (P.beta)
                chunk_to_f32<T>(__ldg(static_cast<const uint4 *>(P.beta) + i), be);
#pragma unroll
            for (int j = 0; j < V; ++j)
                f[j] = fmaf(v[j], g[j], be[j]);
            reinterpret_cast<uint4 *>(static_cast<T *>(P.y) + b * C)[i] = f32_to_chunk<T>(f);
        }
        if (P.codes) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                top = max(top, ck_abs_bits(v[j]));
#pragma unroll
            for (int o = 1; o < kCkBlock / V; o <<= 1)
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const uint32_t e = ck_scale(top, ck_top<float>());
            typename CodeWord<V>::type word;
            int8_t *q = reinterpret_cast<int8_t *>(&word);
#pragma unroll
            for (int j = 0; j < V; ++j)
                q[j] = (int8_t)ck_code(v[j], ck_inverse(e));
            if (in) {
                reinterpret_cast<typename CodeWord<V>::type *>(P.codes + b * C)[i] = word;
                if (i * V % kCkBlock == 0)
                    P.scales[b * ck_blocks(C) + i * V / kCkBlock] = (uint8_t)e;
            }
        }
    }
}

// A thread keeps the weight gradients of its own channels over the block's rows; the row
// after the one in work is on its way.  The rows' groups of a block put theirs side by side
// in shared memory at the end and are added in order.
template <class T, int TPR, int NV, bool CK>
__global__ void __launch_bounds__(kThreads, NV == 4 ? 1 : 2) norm_grad_row_kernel(const NormGrad P,
                                                                                  float *part_g) {
    constexpr int V = Vec<T>::V, RPB = kThreads / TPR;
    extern __shared__ float sums[];   // [RPB][2][C] (TPR < kThreads)
    __shared__ float part[kWarps];
    const int tid = threadIdx.x % TPR;
    const int C = (int)P.C;
    const int64_t nb = ck_blocks(C), hop = (int64_t)gridDim.x * RPB;
    float ag[NV][V], ab[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j)
            ag[k][j] = ab[k][j] = 0.0f;
    struct Row {
        uint4 g[NV], x[NV];           // CK: x.x, x.y the codes, x.w the step byte
        float rstd, mean;
    };
    auto fetch = [&](int64_t b) {
        Row u;
        const uint4 *gy = reinterpret_cast<const uint4 *>(static_cast<const T *>(P.gy) + b * C);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * TPR + tid;
            u.g[k] = u.x[k] = make_uint4(0, 0, 0, 0);
            if (i * V < C) {
                u.g[k] = __ldg(gy + i);
                if constexpr (CK) {
                    uint32_t q[V / 4];
                    code_words<V>(P.codes + b * C + i * V, q);
                    u.x[k].x = q[0];
                    u.x[k].y = q[V / 4 - 1];
                    u.x[k].w = __ldg(P.scales + b * nb + i * V / kCkBlock);
                } else {
                    u.x[k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(P.x) + b * C) + i);
                }
            }
        }
        u.rstd = __ldg(P.rstd + b);
        u.mean = CK ? 0.0f : __ldg(P.mean + b);
        return u;
    };
    int64_t b = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    Row next;
    if (b < P.B)
        next = fetch(b);
    for (; b < P.B; b += hop) {
        const Row row = next;
        if (b + hop < P.B)
            next = fetch(b + hop);
        auto load = [&](int k, float (&g)[V], float (&v)[V], float (&d)[V]) {
            const int i = k * TPR + tid;
            const bool in = i * V < C;
            chunk_to_f32<T>(row.g[k], g);
            if constexpr (CK) {
                const float step = ck_step(row.x[k].w);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = (ck_biased((j < 4 ? row.x[k].x : row.x[k].y) ^ 0x80808080u, j % 4) - kCkBias) * step;
            } else {
                chunk_to_f32<T>(row.x[k], v);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = in ? (v[j] - row.mean) * row.rstd : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
                d[j] = 1.0f;
            if (P.gamma && in)
                chunk_to_f32<T>(__ldg(static_cast<const uint4 *>(P.gamma) + i), d);
#pragma unroll
            for (int j = 0; j < V; ++j)
                d[j] *= g[j];
        };
        float a = 0.0f, q = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float g[V], v[V], d[V];
            load(k, g, v, d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a += d[j];
                q = fmaf(d[j], v[j], q);
                ag[k][j] = fmaf(g[j], v[j], ag[k][j]);
                ab[k][j] += g[j];
            }
        }
        if (P.gx) {
            const float A = row_sum<TPR>(a, part) / (float)C;
            const float S = row_sum<TPR>(q, part) / (float)C;
            uint4 *gx = reinterpret_cast<uint4 *>(static_cast<T *>(P.gx) + b * C);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float g[V], v[V], d[V];
                load(k, g, v, d);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    d[j] = row.rstd * (d[j] - A - v[j] * S);
                if ((k * TPR + tid) * V < C)
                    gx[k * TPR + tid] = f32_to_chunk<T>(d);
            }
        }
    }
    if (!part_g)
        return;
    float *out = part_g + (int64_t)blockIdx.x * 2 * C;
    float *to = TPR == kThreads ? out : sums + (threadIdx.x / TPR) * 2 * C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = k * TPR + tid;
        if (i * V < C)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                to[i * V + j] = ag[k][j];
                to[C + i * V + j] = ab[k][j];
            }
    }
    if (TPR < kThreads) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * C; c += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int r = 0; r < RPB; ++r)
                v += sums[r * 2 * C + c];
            out[c] = v;
        }
    }
}

// ---------------------------------------------------------------- any sizes
//
// For channel counts past what a cluster holds, and unaligned rows of single tokens: the
// values are read again (from the L2) in each pass.  A block takes TL consecutive positions
// of one b, lanes along them, so a warp covers 32 / TL channels; with L == 1 the lanes run
// along the channels.

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
    const AnyIndex at(P.C, P.L, TL);
    const int64_t b = at.b_of(blockIdx.x), l = at.l_of(blockIdx.x, threadIdx.x);
    const int lane = threadIdx.x & 31, col = lane & (TL - 1);
    const int rows = at.rows(), row0 = threadIdx.x / TL;
    const bool in = l < P.L;
    const T *x = static_cast<const T *>(P.x);
    float s = 0.0f;
    for (int64_t c = row0; c < P.C; c += rows)
        s += in ? ld_f32(x + at.value(b, c, l)) : 0.0f;
    const float mean = sum_over_rows(s, TL, part) / (float)P.C;
    s = 0.0f;
    for (int64_t c = row0; c < P.C; c += rows) {
        const float d = in ? ld_f32(x + at.value(b, c, l)) - mean : 0.0f;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(sum_over_rows(s, TL, part) / (float)P.C + P.eps);
    if (in && row0 == 0) {
        if (P.mean)
            P.mean[at.stat(b, l)] = mean;
        if (P.rstd)
            P.rstd[at.stat(b, l)] = rstd;
    }
    const bool along_c = P.L == 1;
    // whole warps walk the rows together: the block maximum below is a warp reduction
    for (int64_t c0 = 0; c0 < P.C; c0 += rows) {
        const int64_t c = c0 + row0;
        const bool ok = in && c < P.C;
        const float v = ok ? (ld_f32(x + at.value(b, c, l)) - mean) * rstd : 0.0f;
        if (ok) {
            float o = v;
            if (P.gamma)
                o = o * ld_f32(static_cast<const T *>(P.gamma) + c);
            if (P.beta)
                o = o + ld_f32(static_cast<const T *>(P.beta) + c);
            static_cast<T *>(P.y)[at.value(b, c, l)] = from_f32<T>(o);
        }
        if (P.codes) {
            uint32_t m = ck_abs_bits(v);
            for (int o = along_c ? 16 : TL / 2; o > 0; o >>= 1)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const uint32_t e = ck_scale(m, ck_top<float>());
            if (ok) {
                P.codes[at.value(b, c, l)] = (int8_t)ck_code(v, ck_inverse(e));
                if (along_c ? lane == 0 : col == 0)
                    P.scales[at.step(b, c, l)] = (uint8_t)e;
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
    const AnyIndex at(P.C, P.L, TL);
    const int lane = threadIdx.x & 31, col = lane & (TL - 1);
    const int rows = at.rows(), row0 = threadIdx.x / TL;
    float *pg = part_g ? part_g + at.part(blockIdx.x) : nullptr;
    for (int64_t tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
        const int64_t b = at.b_of(tile), l = at.l_of(tile, threadIdx.x);
        const bool in = l < P.L;
        const float rstd = in ? P.rstd[at.stat(b, l)] : 0.0f;
        const float mean = !CK && in ? P.mean[at.stat(b, l)] : 0.0f;
        auto value = [&](int64_t c) {
            if (CK)
                return (float)P.codes[at.value(b, c, l)] * ck_step(P.scales[at.step(b, c, l)]);
            return (ld_f32(static_cast<const T *>(P.x) + at.value(b, c, l)) - mean) * rstd;
        };
        const T *gy = static_cast<const T *>(P.gy);
        float a = 0.0f, q = 0.0f;
        for (int64_t c0 = 0; c0 < P.C; c0 += rows) {
            const int64_t c = c0 + row0;
            float g = 0.0f, v = 0.0f;
            if (in && c < P.C) {
                g = ld_f32(gy + at.value(b, c, l));
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
                    const float g = ld_f32(gy + at.value(b, c, l));
                    const float d = P.gamma ? g * ld_f32(static_cast<const T *>(P.gamma) + c) : g;
                    static_cast<T *>(P.gx)[at.value(b, c, l)] = from_f32<T>(rstd * (d - A - value(c) * S));
                }
        }
    }
}

// grad_gamma[c] and grad_beta[c]: the blocks' partial sums.  A block takes 8 columns (a
// sector of each row) and 128 interleaved chains of rows, joined in a fixed order: few
// columns and short chains, so that a few hundred rows are a handful of loads deep.
template <class T>
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float *part, int64_t n,
                                                                int64_t C, T *ggamma, T *gbeta) {
    __shared__ float sums[32][8];
    // launched while the gradient's kernel still runs: wait for its partial sums
    cudaGridDependencySynchronize();
    const int col = threadIdx.x & 7, chain = threadIdx.x / 8, warp = threadIdx.x / 32;
    const int64_t i = (int64_t)blockIdx.x * 8 + col;
    float s = 0.0f;
    if (i < 2 * C)
#pragma unroll 4
        for (int64_t j = chain; j < n; j += 128)
            s += part[j * 2 * C + i];
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
    if ((threadIdx.x & 31) < 8)
        sums[warp][col] = s;
    __syncthreads();
    if (warp > 0)
        return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        s += sums[chain * 8 + k][col];         // chain is 0 to 3 here
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
    T *out = i < C ? ggamma : gbeta;
    if (chain == 0 && i < 2 * C && out)
        out[i < C ? i : i - C] = from_f32<T>(s);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Tiles of [B, C, L] for row_bytes(tw) bytes of shared memory a channel; false when a
// cluster cannot hold the channels of a tile.
//
// A block's share is at most a third of an SM's shared memory, so that three blocks are
// there to load, reduce and store at different times; channels past that are split over a
// cluster, and so are the channels of a tile where there are too few tiles for the SMs (at
// least as many channels a block as its threads have rows).
template <class Bytes>
bool make_tiling(int64_t B, int64_t C, int64_t L, int size, int most, Bytes row_bytes, Tiling *t) {
    const int V = 16 / size;
    if (L < 2)
        return false;
    t->tw = V;
    while (t->tw < most && t->tw < L)
        t->tw *= 2;
    t->tw_log = __builtin_ctz(t->tw);
    t->lpr_log = __builtin_ctz(t->tw / V);
    t->inv_c = 1.0f / (float)C;
    const int rows = kThreads >> t->lpr_log;   // rows of a block's threads
    t->tiles = (L + t->tw - 1) / t->tw;
    t->total = B * t->tiles;
    auto slice = [&](int split) { return ((C + split - 1) / split + rows - 1) / rows * rows; };
    auto shared = [&](int split) { return slice(split) * row_bytes(t->tw); };
    t->split = 1;
    while (t->split < kMaxSplit && shared(t->split) > 69 * 1024)
        t->split *= 2;
    if (shared(t->split) > 200 * 1024)
        return false;
    while (t->split < kMaxSplit && t->total * t->split < sm_count_or(148) &&
           slice(t->split) >= 2 * rows)
        t->split *= 2;
    t->slice = (int)slice(t->split);
    return true;
}

// Blocks of a tile kernel that one SM holds.
int blocks_per_sm(size_t shared) {
    const int n = (int)((227 * 1024) / (shared + 6 * 1024));   // 6 KB: static and reserved
    return n < 1 ? 1 : n > 3 ? 3 : n;   // 3: registers
}

// Clusters of a launch, `room` at most, and the step of their walks.
int64_t plan_walk(Tiling *t, int64_t room) {
    const int64_t n = t->total < room ? t->total : room;
    t->walk_b = (int)(n / t->tiles);
    t->walk_l = (int)(n % t->tiles);
    return n;
}

template <class... A>
cudaError_t launch_cluster(void (*kernel)(A...), unsigned grid, unsigned split, size_t shared,
                           cudaStream_t s, A... args) {
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), (int)shared);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Chunks a thread holds of a row of C values, for 32 and for kThreads threads a row: 1, 2
// or 4, else 0.
int row_chunks(int64_t C, int V, int threads) {
    const int64_t n = (C + (int64_t)threads * V - 1) / ((int64_t)threads * V);
    return n == 1 ? 1 : n == 2 ? 2 : n <= 4 ? 4 : 0;
}

template <class T>
cudaError_t norm(const NormProblem &P, cudaStream_t s) {
    constexpr int V = Vec<T>::V;
    const bool base = aligned(P.x, 16) && aligned(P.y, 16) && aligned(P.codes, V);
    if (P.L == 1 && base && P.C % V == 0 && aligned(P.gamma, 16) && aligned(P.beta, 16)) {
        const int warp = row_chunks(P.C, V, 32), block = row_chunks(P.C, V, kThreads);
        const unsigned gw = (unsigned)((P.B + kWarps - 1) / kWarps), gb = (unsigned)P.B;
        if (warp == 1)
            norm_row_kernel<T, 32, 1><<<gw, kThreads, 0, s>>>(P);
        else if (warp == 2)
            norm_row_kernel<T, 32, 2><<<gw, kThreads, 0, s>>>(P);
        else if (warp == 4)
            norm_row_kernel<T, 32, 4><<<gw, kThreads, 0, s>>>(P);
        else if (block == 1)
            norm_row_kernel<T, kThreads, 1><<<gb, kThreads, 0, s>>>(P);
        else if (block == 2)
            norm_row_kernel<T, kThreads, 2><<<gb, kThreads, 0, s>>>(P);
        else if (block == 4)
            norm_row_kernel<T, kThreads, 4><<<gb, kThreads, 0, s>>>(P);
        if (warp || block)
            return cudaGetLastError();
    }
    Tiling t;
    const bool vec = base && P.L % V == 0;
    constexpr int WIDE = 128 / (int)sizeof(T);
    if (vec && make_tiling(P.B, P.C, P.L, sizeof(T), WIDE, [](int) { return 0; }, &t)) {
        const bool full = t.tw == WIDE;
        auto kernel = P.codes ? (full ? norm_stream_kernel<T, true, 3> : norm_stream_kernel<T, true, -1>)
                              : (full ? norm_stream_kernel<T, false, 3>
                                      : norm_stream_kernel<T, false, -1>);
        return launch_cluster(kernel, (unsigned)(t.total * t.split), (unsigned)t.split, 0, s, P, t);
    }
    auto row_bytes = [&](int tw) { return norm_row_bytes<T>(tw, P.codes != nullptr); };
    if (!vec && make_tiling(P.B, P.C, P.L, sizeof(T), kTW, row_bytes, &t)) {
        t.words = P.L * sizeof(T) % 4 == 0 && aligned(P.x, 4) && aligned(P.y, 4);
        t.code_words = P.L % 4 == 0 && aligned(P.codes, 4);
        const size_t shared = (size_t)t.slice * row_bytes(t.tw);
        const unsigned grid = (unsigned)(plan_walk(&t, (int64_t)sm_count_or(148) *
                                                           blocks_per_sm(shared) / t.split) *
                                         t.split);
        return launch_cluster(P.codes ? norm_tile_kernel<T, true> : norm_tile_kernel<T, false>, grid,
                              (unsigned)t.split, shared, s, P, t);
    }
    const int TL = lanes_along(P.L);
    norm_any_kernel<T><<<(unsigned)(P.B * ((P.L + TL - 1) / TL)), kThreads, 0, s>>>(P, TL);
    return cudaGetLastError();
}

// How a backward runs: the kernel family, its blocks, and the rows of partial sums.
struct GradPlan {
    int kind;          // 0: any sizes, 1: tiles, 2: a warp a row, 3: a block a row, 4: streams
    int nv;
    Tiling t;
    size_t shared;
    int64_t blocks, rows;
};

template <class T>
GradPlan grad_plan(const NormGrad &P) {
    constexpr int V = Vec<T>::V;
    GradPlan g = {};
    const int sms = sm_count_or(148);
    const bool base = aligned(P.gy, 16) && aligned(P.gx, 16) &&
                      (P.from_codes ? aligned(P.codes, V) : aligned(P.x, 16)) &&
                      aligned(P.rstd, 16) && aligned(P.mean, 16);
    if (P.B == 0 || P.L == 0)
        return g;
    if (P.L == 1 && base && P.C % V == 0 && aligned(P.gamma, 16)) {
        const int warp = row_chunks(P.C, V, 32), block = row_chunks(P.C, V, kThreads);
        if (warp || block) {
            g.kind = warp ? 2 : 3;
            g.nv = warp ? warp : block;
            g.shared = warp ? kWarps * 2 * P.C * sizeof(float) : 0;
            const int64_t need = warp ? (P.B + kWarps - 1) / kWarps : P.B;
            const int64_t room = g.nv == 4 ? sms : 2 * sms;   // blocks that are there at once
            g.blocks = g.rows = need < room ? need : room;
            return g;
        }
    }
    const bool vec = base && P.L % V == 0;
    if (vec && make_tiling(P.B, P.C, P.L, sizeof(T), 128 / (int)sizeof(T),
                             [](int) { return (int)(sizeof(float) * 3); }, &g.t)) {
        g.kind = 4;
        g.shared = (size_t)g.t.slice * sizeof(float) * 3;
        const int64_t room = (int64_t)sms * 2 / g.t.split;
        g.rows = plan_walk(&g.t, room);
        g.blocks = g.rows * g.t.split;
        return g;
    }
    auto row_bytes = [&](int tw) { return grad_row_bytes<T>(tw, P.from_codes); };
    if (!vec && make_tiling(P.B, P.C, P.L, sizeof(T), kTW, row_bytes, &g.t)) {
        g.kind = 1;
        g.t.words = P.L * sizeof(T) % 4 == 0 && aligned(P.gy, 4) && aligned(P.gx, 4) && aligned(P.x, 4);
        g.t.code_words = P.L % 4 == 0 && aligned(P.codes, 4);
        g.shared = (size_t)g.t.slice * row_bytes(g.t.tw);
        g.rows = plan_walk(&g.t, (int64_t)sms * blocks_per_sm(g.shared) / g.t.split);
        g.blocks = g.rows * g.t.split;
        return g;
    }
    const int TL = lanes_along(P.L);
    const int64_t n = P.B * ((P.L + TL - 1) / TL), most = (int64_t)sms * 8;
    g.blocks = g.rows = n < most ? n : most;
    return g;
}

template <class T, bool CK>
cudaError_t run_norm_grad(const NormGrad &P, const GradPlan &g, float *part, cudaStream_t s) {
    const unsigned grid = (unsigned)g.blocks;
    if (g.kind == 4)
        return launch_cluster(g.t.tw == 128 / (int)sizeof(T) ? norm_grad_stream_kernel<T, CK, 3>
                                                             : norm_grad_stream_kernel<T, CK, -1>,
                              grid, (unsigned)g.t.split, g.shared, s, P, g.t, part);
    if (g.kind == 1)
        return launch_cluster(norm_grad_tile_kernel<T, CK>, grid, (unsigned)g.t.split, g.shared, s, P,
                              g.t, part);
    if (g.kind >= 2) {
        auto kernel = g.kind == 2 ? (g.nv == 1   ? norm_grad_row_kernel<T, 32, 1, CK>
                                     : g.nv == 2 ? norm_grad_row_kernel<T, 32, 2, CK>
                                                 : norm_grad_row_kernel<T, 32, 4, CK>)
                                  : (g.nv == 1   ? norm_grad_row_kernel<T, kThreads, 1, CK>
                                     : g.nv == 2 ? norm_grad_row_kernel<T, kThreads, 2, CK>
                                                 : norm_grad_row_kernel<T, kThreads, 4, CK>);
        return launch_cluster(kernel, grid, 1u, g.shared, s, P, part);
    }
    const int TL = lanes_along(P.L);
    norm_grad_any_kernel<T, CK>
        <<<grid, kThreads, 0, s>>>(P, TL, P.B * ((P.L + TL - 1) / TL), part);
    return cudaGetLastError();
}

template <class T>
cudaError_t norm_grad(const NormGrad &P, void *ws, cudaStream_t s, int *launches) {
    const GradPlan g = grad_plan<T>(P);
    const bool weights = P.ggamma || P.gbeta;
    float *part = weights ? static_cast<float *>(ws) : nullptr;   // NULL for an empty input
    if (g.blocks > 0 && (P.gx || weights)) {
        const cudaError_t e = P.from_codes ? run_norm_grad<T, true>(P, g, part, s)
                                           : run_norm_grad<T, false>(P, g, part, s);
        if (e != cudaSuccess)
            return e;
        ++*launches;
    }
    if (weights) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((2 * P.C + 7) / 8));
        cfg.blockDim = dim3(1024);
        cfg.stream = s;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_weight_grad_kernel<T>,
                                                 static_cast<const float *>(part), g.rows, P.C,
                                                 static_cast<T *>(P.ggamma), static_cast<T *>(P.gbeta));
        if (e != cudaSuccess)
            return e;
        ++*launches;
    }
    return cudaGetLastError();
}

// For any alignment of the tensors, so that a caller can keep the size of a shape.
template <class T>
size_t grad_workspace(NormGrad P) {
    P.gamma = P.x = P.gy = nullptr;   // aligned
    P.codes = nullptr;
    P.mean = P.rstd = nullptr;
    P.gx = nullptr;
    const int64_t a = grad_plan<T>(P).rows;
    P.gy = reinterpret_cast<const void *>((uintptr_t)1);
    const int64_t b = grad_plan<T>(P).rows;
    return (size_t)(a > b ? a : b) * 2 * P.C * sizeof(float);
}

}  // namespace

bool norm_grid_ok(int64_t B, int64_t L) {
    const int TL = lanes_along(L);
    return B * ((L + TL - 1) / TL) < (1LL << 31);
}

cudaError_t launch_norm(const NormProblem &P, cudaStream_t s) {
    if (P.dtype == DCN1D_BF16)
        return norm<__nv_bfloat16>(P, s);
    if (P.dtype == DCN1D_F16)
        return norm<__half>(P, s);
    return norm<float>(P, s);
}

size_t norm_grad_workspace(const NormGrad &P) {
    if (!P.ggamma && !P.gbeta)
        return 0;
    if (P.dtype == DCN1D_BF16)
        return grad_workspace<__nv_bfloat16>(P);
    if (P.dtype == DCN1D_F16)
        return grad_workspace<__half>(P);
    return grad_workspace<float>(P);
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
