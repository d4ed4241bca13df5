// Two fp32 values in one 64-bit register, and sm_100a's packed arithmetic on them (one
// instruction for two additions, products or fused multiply-adds), for kernels that memory
// should bound but single fp32 instructions would; and the 16-byte chunks of a tensor that
// such kernels move, as pairs.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace dcn1d {

using Pair = unsigned long long;

__device__ __forceinline__ Pair pair(float a, float b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ Pair twice(float a) { return pair(a, a); }
__device__ __forceinline__ float2 halves(Pair p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Values of a 16-byte chunk.
template <class T> struct Vec {
    static constexpr int V = 16 / (int)sizeof(T), H = V / 2;
};

template <class T>
__device__ __forceinline__ void chunk_to_pairs(const uint4 &u, Pair (&p)[Vec<T>::H]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) {
        p[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
        p[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                p[j] = pair(f.x, f.y);
            } else {
                p[j] = pair(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
            }
        }
    }
}

template <class T>
__device__ __forceinline__ uint4 pairs_to_chunk(const Pair (&p)[Vec<T>::H]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
        const float2 a = halves(p[0]), b = halves(p[1]);
        w[0] = __float_as_uint(a.x);
        w[1] = __float_as_uint(a.y);
        w[2] = __float_as_uint(b.x);
        w[3] = __float_as_uint(b.y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = halves(p[j]);
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The word of V codes that goes with a chunk.
template <int V> struct CodeWord;
template <> struct CodeWord<8> { using type = uint2; };
template <> struct CodeWord<4> { using type = uint32_t; };

}  // namespace dcn1d
