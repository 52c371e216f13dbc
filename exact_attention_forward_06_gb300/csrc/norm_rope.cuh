// norm_rope.cuh -- norm and position rotation of one head vector by 16 lanes.
//
// A head row of 128 bf16 (256 B) belongs to a half-warp.  Lane l of it owns
// the four pairs 4 l .. 4 l + 3 of the plan and holds their eight channels, so
// a rotation needs no exchange:
//   pairs (2i, 2i+1):    channels 8 l .. 8 l + 7;
//   pairs (i, i + R/2):  channels 4 l .. + 3 and R/2 + 4 l .. + 3 (8-byte pieces).
// Lanes past the plan's pairs hold eight of the channels from R on, which only
// take the norm.  The norm's sum runs over the 16 lanes in a fixed order.
//
// The norm's weights are multiplied into the token's cosines and sines, once for
// all its rows; the root is applied to the rotated pair: with the weights u, w of a
// pair's channels, (a, b) -> r (a u cos - b w sin, a u sin + b w cos).
//
// Angles: position * turns modulo 2^64 is the exact fraction of a turn.  Its upper
// 32 bits, to the nearest quarter turn and the rest x in [-pi/4, pi/4], go to the
// Taylor series of sine (to x^9; the next term is below 2^-29) and cosine (to
// x^10; below 2^-33): half the instructions of a general sine and cosine of x.
#pragma once

#include <cstdint>

#include "cache_ops.h"
#include "common.cuh"

namespace attn {

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Where lane l (0..15)'s eight channels lie, and whether it rotates.
struct LanePieces {
    int a, b;      // first channel of each piece of four
    bool rotates;
};

template <bool INTER>
__device__ __forceinline__ LanePieces lane_pieces(int l, int R) {
    LanePieces p;
    p.rotates = 8 * l < R;
    if (INTER) {
        p.a = 8 * l;
        p.b = 8 * l + 4;
    } else {
        p.a = p.rotates ? 4 * l : 8 * l;
        p.b = p.rotates ? R / 2 + 4 * l : 8 * l + 4;
    }
    return p;
}

// cos and sin of the lane's four pairs for one token.
struct LaneTurn {
    float c[4], s[4];
};

// Sines and cosines of two angles, `frac` / 2^32 of a turn each.
__device__ __forceinline__ void sincos_turns(uint32_t frac0, uint32_t frac1, float (&s)[2], float (&c)[2]) {
    const auto all = [](float v) { return make_float2(v, v); };
    const uint32_t quarter[2] = {(frac0 + 0x20000000u) >> 30, (frac1 + 0x20000000u) >> 30};
    const float2 x = ptx::mul2(make_float2((float)(int32_t)(frac0 - (quarter[0] << 30)),
                                           (float)(int32_t)(frac1 - (quarter[1] << 30))),
                               all(1.4629180792671596e-09f));  // 2 pi / 2^32
    const float2 x2 = ptx::mul2(x, x);
    float2 sn = ptx::fma2(x2, all(2.7557319224e-06f), all(-1.9841269841e-04f));  // 1/9!, -1/7!
    sn = ptx::fma2(x2, sn, all(8.3333333333e-03f));                             // 1/5!
    sn = ptx::fma2(x2, sn, all(-1.6666666667e-01f));                            // -1/3!
    sn = ptx::fma2(ptx::mul2(x2, x), sn, x);
    float2 cs = ptx::fma2(x2, all(-2.7557319224e-07f), all(2.4801587302e-05f));  // -1/10!, 1/8!
    cs = ptx::fma2(x2, cs, all(-1.3888888889e-03f));                            // -1/6!
    cs = ptx::fma2(x2, cs, all(4.1666666667e-02f));                             // 1/4!
    cs = ptx::fma2(x2, cs, all(-0.5f));
    cs = ptx::fma2(x2, cs, all(1.f));
    const float sns[2] = {sn.x, sn.y}, css[2] = {cs.x, cs.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        // A quarter turn on: (sin, cos) -> (cos, -sin).
        const float a = quarter[j] & 1 ? css[j] : sns[j], b = quarter[j] & 1 ? sns[j] : css[j];
        s[j] = __uint_as_float(__float_as_uint(a) ^ (quarter[j] & 2) << 30);
        c[j] = __uint_as_float(__float_as_uint(b) ^ ((quarter[j] + 1) & 2) << 30);
    }
}

// pos_stride: tokens per axis in p.positions; `token` indexes them; without
// positions every axis has the position `pos0`.
__device__ __forceinline__ LaneTurn lane_turn(const RotateParams &p, int l, int64_t token, int64_t pos_stride,
                                              int pos0) {
    LaneTurn t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        t.c[j] = 1.f;
        t.s[j] = 0.f;
    }
    if (8 * l >= p.rotary_dim) return t;
    uint4 e[4];
    int pos[4];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = reinterpret_cast<const uint4 *>(p.rope)[4 * l + j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool known = e[j].z < (uint32_t)p.n_axes;
        bad = bad || !known;
        pos[j] = p.positions && known ? p.positions[(int64_t)e[j].z * pos_stride + token] : pos0;
        if (!known) e[j].x = e[j].y = 0;  // not rotated
    }
    if (bad) report_status(p.status, kStatusDeviceBounds, kSiteRopeAxis);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        uint32_t frac[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // The upper word of the 64-bit product, of a signed position.
            frac[i] = __umulhi((uint32_t)pos[j + i], e[j + i].x) + (uint32_t)pos[j + i] * e[j + i].y;
            if (pos[j + i] < 0) frac[i] -= e[j + i].x;
        }
        float s[2], c[2];
        sincos_turns(frac[0], frac[1], s, c);
        t.s[j] = s[0], t.s[j + 1] = s[1];
        t.c[j] = c[0], t.c[j + 1] = c[1];
    }
    return t;
}

// The lane's eight channels as two packed pieces.
struct LaneRow {
    uint2 a, b;
};

template <bool INTER>
__device__ __forceinline__ LaneRow load_row(const void *row, const LanePieces &lp) {
    LaneRow r;
    const uint16_t *x = static_cast<const uint16_t *>(row);
    if (INTER) {
        const uint4 v = *reinterpret_cast<const uint4 *>(x + lp.a);
        r.a = make_uint2(v.x, v.y);
        r.b = make_uint2(v.z, v.w);
    } else {
        r.a = *reinterpret_cast<const uint2 *>(x + lp.a);
        r.b = *reinterpret_cast<const uint2 *>(x + lp.b);
    }
    return r;
}

template <bool INTER>
__device__ __forceinline__ void store_row(void *row, const LanePieces &lp, const LaneRow &r) {
    uint16_t *x = static_cast<uint16_t *>(row);
    if (INTER) {
        *reinterpret_cast<uint4 *>(x + lp.a) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
    } else {
        *reinterpret_cast<uint2 *>(x + lp.a) = r.a;
        *reinterpret_cast<uint2 *>(x + lp.b) = r.b;
    }
}

// The lane's pairs (first, second channel) of a row, and back.
template <bool INTER>
__device__ __forceinline__ void unpack(const LaneRow &r, float (&a)[4], float (&b)[4]) {
    if (INTER) {
        const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = bf_lo(w[j]);
            b[j] = bf_hi(w[j]);
        }
    } else {
        a[0] = bf_lo(r.a.x), a[1] = bf_hi(r.a.x), a[2] = bf_lo(r.a.y), a[3] = bf_hi(r.a.y);
        b[0] = bf_lo(r.b.x), b[1] = bf_hi(r.b.x), b[2] = bf_lo(r.b.y), b[3] = bf_hi(r.b.y);
    }
}

template <bool INTER>
__device__ __forceinline__ LaneRow pack(const float (&a)[4], const float (&b)[4]) {
    LaneRow r;
    if (INTER) {
        r.a = make_uint2(ptx::pack_bf16x2(a[0], b[0]), ptx::pack_bf16x2(a[1], b[1]));
        r.b = make_uint2(ptx::pack_bf16x2(a[2], b[2]), ptx::pack_bf16x2(a[3], b[3]));
    } else {
        r.a = make_uint2(ptx::pack_bf16x2(a[0], a[1]), ptx::pack_bf16x2(a[2], a[3]));
        r.b = make_uint2(ptx::pack_bf16x2(b[0], b[1]), ptx::pack_bf16x2(b[2], b[3]));
    }
    return r;
}

// The factors of one tensor's rows at one token: weights times cosines and
// sines (a lane that does not rotate: the weights).
struct LaneFactors {
    float2 ac[2], bs[2], as[2], bc[2];  // bs: of the other sign
};

template <bool INTER>
__device__ __forceinline__ LaneFactors lane_factors(const LaneTurn &t, const void *weight, const LanePieces &lp) {
    float u[4] = {1.f, 1.f, 1.f, 1.f}, w[4] = {1.f, 1.f, 1.f, 1.f};
    if (weight) unpack<INTER>(load_row<INTER>(weight, lp), u, w);
    LaneFactors f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f.ac[j] = make_float2(u[2 * j] * t.c[2 * j], u[2 * j + 1] * t.c[2 * j + 1]);
        f.bs[j] = make_float2(-w[2 * j] * t.s[2 * j], -w[2 * j + 1] * t.s[2 * j + 1]);
        f.as[j] = make_float2(u[2 * j] * t.s[2 * j], u[2 * j + 1] * t.s[2 * j + 1]);
        f.bc[j] = make_float2(w[2 * j] * t.c[2 * j], w[2 * j + 1] * t.c[2 * j + 1]);
    }
    return f;
}

// Norm (when asked) and rotation of the lane's eight channels; the whole warp
// takes part (a mask of the half-warp's lanes, known only at run time, costs every
// shuffle a dozen instructions).
template <bool INTER>
__device__ __forceinline__ LaneRow norm_rotate(const LaneRow &in, bool norm, float eps, const LaneFactors &f,
                                               bool rotates) {
    float a[4], b[4], x[4], y[4];
    unpack<INTER>(in, a, b);
    const float2 a2[2] = {make_float2(a[0], a[1]), make_float2(a[2], a[3])};
    const float2 b2[2] = {make_float2(b[0], b[1]), make_float2(b[2], b[3])};
    float inv = 1.f;
    if (norm) {
        const float2 s2 = ptx::fma2(a2[0], a2[0], ptx::mul2(a2[1], a2[1]));
        const float2 t2 = ptx::fma2(b2[0], b2[0], ptx::mul2(b2[1], b2[1]));
        const float2 u2 = ptx::add2(s2, t2);
        float ss = u2.x + u2.y;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, 16);
        inv = rsqrtf(fmaf(ss, 1.f / 128.f, eps));
    }
    const float2 inv2 = make_float2(inv, inv);
    float2 x2[2], y2[2];
    if (rotates) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x2[j] = ptx::mul2(ptx::fma2(b2[j], f.bs[j], ptx::mul2(a2[j], f.ac[j])), inv2);
            y2[j] = ptx::mul2(ptx::fma2(b2[j], f.bc[j], ptx::mul2(a2[j], f.as[j])), inv2);
        }
    } else {
        // (not the general form with a sine of zero: infinities stay where they are)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x2[j] = ptx::mul2(ptx::mul2(a2[j], f.ac[j]), inv2);
            y2[j] = ptx::mul2(ptx::mul2(b2[j], f.bc[j]), inv2);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        x[2 * j] = x2[j].x;
        x[2 * j + 1] = x2[j].y;
        y[2 * j] = y2[j].x;
        y[2 * j + 1] = y2[j].y;
    }
    return pack<INTER>(x, y);
}

}  // namespace attn
