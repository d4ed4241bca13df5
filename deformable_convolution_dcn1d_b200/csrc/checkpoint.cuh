// The 8-bit checkpoint of an activation tensor [B, C, L].
//
// A row is the L positions of one (b, c), or, when L == 1, the C channels of one b (the
// contiguous axis).  A row is cut into blocks of 32 values (the last one may be shorter).
// Every value of a block is code * 2^(s - 127): an int8 code in [-127, 127] and one byte s
// a block, the biased exponent of the block's step.  With amax the block's largest
// magnitude, the step is the smallest power of two at which amax still rounds to a code of
// at most 127, and a code is the nearest integer to value / step (ties to even).
//
// A power of two rather than amax / 127: value / step and code * step are then exact in
// fp32 (and code * step in bf16), so codes do not depend on the rounding of a division,
// packing what was unpacked gives the same values back, and a block costs one byte.  The
// price is a step up to twice as wide (1.44 times on average).
//
// s = 255 marks a block that held a NaN or an infinity (its codes are 0): 0 * 2^128 reads
// back as NaN.  s is at least 1 (step 2^-126, the smallest normal number), and at most the
// input type's largest exponent less 6: a block within 0.4 % of the largest finite number
// saturates at code 127 rather than read back as infinity.
#pragma once

#include "common.cuh"

namespace dcn1d {

constexpr int kCkBlock = 32;

// Largest biased exponent of a finite value of the type that is packed.
template <class T> __host__ __device__ constexpr int ck_top() { return 254; }
template <> __host__ __device__ constexpr int ck_top<__half>() { return 142; }

__device__ __forceinline__ uint32_t ck_abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The step byte of a block from the fp32 bits of its largest magnitude (as an unsigned
// integer, in which NaN > infinity > every finite value).  amax has a significand in
// [64, 128) steps of 2^(E - 6); adding 2^16 carries into the exponent exactly when that
// is 127.5 or more, which would round to 128.
__device__ __forceinline__ uint32_t ck_scale(uint32_t amax_bits, int top) {
    if (amax_bits >= 0x7F800000u)
        return 255u;
    const int e = min((int)((amax_bits + 0x10000u) >> 23), top);
    return (uint32_t)max(e - 6, 1);
}

// 1 / step; 0 for s = 255, which makes every code of the block 0 (NaN converts to 0).
__device__ __forceinline__ float ck_inverse(uint32_t s) {
    return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

__device__ __forceinline__ int ck_code(float v, float inverse) {
    return max(-127, min(127, __float2int_rn(v * inverse)));
}

// The step itself; infinity for s = 255 (code 0 times infinity is NaN).
__device__ __forceinline__ float ck_step(uint32_t s) { return __uint_as_float(s << 23); }

// 1.5 * 2^23: a float near it steps by one, so v / step + kCkRound is v / step rounded to an
// integer (ties to even), whose low byte is the code.
constexpr float kCkRound = 12582912.0f;
// 2^23 + 128: the float with the bits 0x4B0000xx is 2^23 + xx, so with xx = code + 128 (the
// code's sign bit flipped) subtracting this gives the code.
constexpr float kCkBias = 8388736.0f;

// Four codes (a word whose sign bits are flipped) as 2^23 + 128 + code.
__device__ __forceinline__ float ck_biased(uint32_t flipped, int j) {
    return __uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7540 + j));
}

// The low bytes of four floats as one word.
__device__ __forceinline__ uint32_t ck_low_bytes(float a, float b, float c, float d) {
    return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                       __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

// Blocks of a row of n values.
__host__ __device__ __forceinline__ int64_t ck_blocks(int64_t n) {
    return (n + kCkBlock - 1) / kCkBlock;
}

}  // namespace dcn1d
