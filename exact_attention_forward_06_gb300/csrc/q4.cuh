// q4.cuh -- the 4-bit cache block (one page of one KV head, keys and values):
// byte offsets, and the quantisation of a 32-channel group.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace attn {
namespace q4 {

constexpr int PAGE = 16;
constexpr int D = 128;
constexpr int BLOCK = 2560;
constexpr int V_CODES = 1024;
constexpr int K_SCALES = 2048;   // [token][group]
constexpr int K_CENTERS = 2176;  // [token][group]
constexpr int V_SCALES = 2304;   // [token][group]
constexpr int V_CENTERS = 2432;  // [group][token]

// Key codes of channels 8 w .. 8 w + 7 of token t: a 32-bit word.
__host__ __device__ constexpr int k_word(int t, int w) { return t * 64 + (w & 3) * 16 + (w >> 2) * 4; }
// Value codes of channels 32 g + 4 r .. + 3 of token t: a 16-bit half-word.
__host__ __device__ constexpr int v_half(int t, int g, int r) {
    return V_CODES + r * 128 + ((t & 7) >> 1) * 32 + (((t >> 3) ^ (r & 1)) << 4) + (t & 1) * 8 + g * 2;
}

// Largest of two bf16 pairs, half by half; NaN if either is.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Center and scale (bf16 bits) of a group with largest member hi and smallest
// lo (either not finite: some member is not).
struct GroupScale {
    uint16_t z, s;
};

__device__ __forceinline__ GroupScale group_scale(float hi, float lo) {
    if (!(fabsf(hi) < INFINITY && fabsf(lo) < INFINITY)) return GroupScale{0x7fff, 0x7fff};
    const float mid = __fadd_rn(__fmul_rn(0.5f, hi), __fmul_rn(0.5f, lo));
    const uint32_t z = ptx::pack_bf16x2(mid, 0.f) & 0xffffu;
    const float zf = __uint_as_float(z << 16);
    const float dev = fmaxf(__fsub_rn(hi, zf), __fsub_rn(zf, lo));
    const uint32_t s = ptx::pack_bf16x2(__fmul_rn(dev, (float)(2.0 / 15.0)), 0.f) & 0xffffu;
    return GroupScale{(uint16_t)z, (uint16_t)s};
}

// The codes of eight channels of one group as a word (channel j in bits 4 j ..).
// The definition's quotient (x - z) / s is a true division, and ties are common
// (x is z plus a whole number of steps for about one bf16 value in 150), so its
// rounding matters.  Within the range where nothing over- or underflows it comes
// from Markstein's correction: with r = 1/s correctly rounded, q = d r and the
// exact remainder d - q s (one fused operation), q + remainder * r is the
// correctly rounded quotient (s has eight significant bits, so the theorem's
// exception, a divisor of all ones, does not arise).  There the definition's clamp
// has nothing to do either: s is within 2^-8 of (largest |x - z|) * 2 / 15, so the
// sum lies within 0.03 of 0 .. 15.
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], GroupScale gs) {
    const float z = __uint_as_float((uint32_t)gs.z << 16), s = __uint_as_float((uint32_t)gs.s << 16);
    if (!(s > 0.f)) return 0;
    constexpr float MAGIC = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, in the low bits
    uint32_t word = 0;
    if (s > 7.8886090522101181e-31f && s < 1.2676506002282294e30f) {  // 2^-100, 2^100
        const float r1 = __frcp_rn(s);
        const float2 r = make_float2(r1, r1), minus_z = make_float2(-z, -z), minus_s = make_float2(-s, -s);
#pragma unroll
        for (int j = 6; j >= 0; j -= 2) {
            const float2 d = ptx::add2(make_float2(x[j], x[j + 1]), minus_z);
            const float2 q = ptx::mul2(d, r);
            const float2 exact = ptx::fma2(ptx::fma2(q, minus_s, d), r, q);
            const float2 t = ptx::add2(ptx::add2(exact, make_float2(7.5f, 7.5f)), make_float2(MAGIC, MAGIC));
            word = (word * 16 + (__float_as_uint(t.y) - 0x4B400000u)) * 16 + (__float_as_uint(t.x) - 0x4B400000u);
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i == j) d = __fsub_rn(x[i], z);
            const float t = __fadd_rn(__fdiv_rn(d, s), 7.5f);
            word |= (__float_as_uint(__fadd_rn(fminf(fmaxf(t, 0.f), 15.f), MAGIC)) - 0x4B400000u) << (4 * j);
        }
    }
    return word;
}

}  // namespace q4
}  // namespace attn
