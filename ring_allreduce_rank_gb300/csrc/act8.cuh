// act8.cuh -- the 8-bit form of activations that act8.cu and experts.cu share.
//
// Blocks of 32 consecutive values of a row share a power of two 2^e, the least
// with |x| <= 127 2^e in the block, and a value is the nearest integer of
// x / 2^e (ties to even), a signed byte.  A power of two costs up to one bit of
// the step against largest / 127, and makes the stored value q 2^e a bf16
// number itself (seven bits and a sign), so that it enters a bf16 product
// without another rounding, and makes x / 2^e exact, so that the only error is
// the one rounding to an integer.  The block's byte is e + 127 (1 to 248); 255
// marks a block that held an infinity or a NaN and stands for 32 NaN.
#pragma once

#include "ccl_device.cuh"

namespace ccl {

constexpr uint32_t kActBlock = 32;
constexpr uint32_t kActNan = 255, kActLeast = 1, kActMost = 248;

// The block's byte from the bits of its largest magnitude.  Steps below 2^-126
// are not used (the values would not be normal bf16 numbers), nor one above
// 2^121 (64 * 2^122 is no bf16 number): values above 127 * 2^121 become that.
__device__ __forceinline__ uint32_t act8_byte(uint32_t largest)
{
    if (largest >= 0x7f800000u)
        return kActNan;
    const uint32_t e = largest >> 23, over = (largest & 0x7fffffu) > 0x7e0000u; // 127 = 1.984375 * 2^6
    const uint32_t b = e + over;
    return b < 6 + kActLeast ? kActLeast : b - 6 > kActMost ? kActMost : b - 6;
}

// 2^-e of a block that is not all NaN.
__device__ __forceinline__ float act8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^e; infinity for a block of NaN, whose codes are 0.
__device__ __forceinline__ float act8_step(uint32_t byte) { return __uint_as_float(byte << 23); }

// A value's code in the low byte: 1.5 * 2^23 + x / 2^e, rounded once, has the
// nearest integer in its last bits.  Only a block at the largest step can hold
// more than 127 of them.
__device__ __forceinline__ uint32_t act8_code(float x, float inverse) { return __float_as_uint(__fmaf_rn(x, inverse, 12582912.0f)); }

__device__ __forceinline__ float act8_clamp(float x) { return fminf(fmaxf(x, -0x1.fcp127f), 0x1.fcp127f); } // 127 * 2^121

// Codes of 32 values, four a word, and the block's byte.
__device__ __forceinline__ uint32_t act8_encode(const float *f, uint4 &lo, uint4 &hi)
{
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 32; ++i)
        m[i & 3] = max(m[i & 3], __float_as_uint(f[i]) & 0x7fffffffu);
    const uint32_t byte = act8_byte(max(max(m[0], m[1]), max(m[2], m[3])));
    uint32_t w[8];
    if (byte == kActNan) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = 0;
    } else {
        const float inverse = act8_inverse(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[4] = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
            if (byte == kActMost) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = act8_clamp(x[k]);
            }
            w[i] = __byte_perm(__byte_perm(act8_code(x[0], inverse), act8_code(x[1], inverse), 0x0040),
                               __byte_perm(act8_code(x[2], inverse), act8_code(x[3], inverse), 0x0040), 0x5410);
        }
    }
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
    return byte;
}

// Four codes as values: 2^23 + (q + 128) is a float whose last byte is q with
// its sign bit turned.
__device__ __forceinline__ void act8_decode4(uint32_t codes, float step, float *f)
{
    const uint32_t w = codes ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __fmul_rn(__fadd_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | i)), -8388736.0f), step);
}

__device__ __forceinline__ void act8_decode(const uint4 &lo, const uint4 &hi, float step, float *f)
{
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        act8_decode4(w[i], step, f + 4 * i);
}

} // namespace ccl
