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
// Angles: position * turns modulo 2^64 is the exact fraction of a turn; its
// upper 32 bits as a signed number of half turns go to sincospi, whose argument
// in [-1, 1) needs no range reduction.
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
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 e = __ldg(reinterpret_cast<const uint4 *>(p.rope) + 4 * l + j);
        const uint64_t turns = (uint64_t)e.y << 32 | e.x;
        if (e.z >= (uint32_t)p.n_axes) {
            report_status(p.status, kStatusDeviceBounds, kSiteRopeAxis);
            continue;
        }
        const int pos = p.positions ? __ldg(p.positions + (int64_t)e.z * pos_stride + token) : pos0;
        const uint64_t frac = (uint64_t)(int64_t)pos * turns;
        // half turns in [-1, 1): the signed upper word over 2^31
        sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, &t.s[j], &t.c[j]);
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

// Norm (weight row w, or nullptr) and rotation of the lane's eight channels;
// all 16 lanes of `mask` take part.
template <bool INTER>
__device__ __forceinline__ LaneRow norm_rotate(const LaneRow &in, const LaneRow *w, float eps, const LaneTurn &t,
                                               bool rotates, unsigned mask) {
    float x[4] = {bf_lo(in.a.x), bf_hi(in.a.x), bf_lo(in.a.y), bf_hi(in.a.y)};
    float y[4] = {bf_lo(in.b.x), bf_hi(in.b.x), bf_lo(in.b.y), bf_hi(in.b.y)};
    if (w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(mask, ss, off, 16);
        const float inv = 1.f / sqrtf(fmaf(ss, 1.f / 128.f, eps));
        const float wa[4] = {bf_lo(w->a.x), bf_hi(w->a.x), bf_lo(w->a.y), bf_hi(w->a.y)};
        const float wb[4] = {bf_lo(w->b.x), bf_hi(w->b.x), bf_lo(w->b.y), bf_hi(w->b.y)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = x[j] * inv * wa[j];
            y[j] = y[j] * inv * wb[j];
        }
    }
    if (rotates) {
        if (INTER) {  // pairs 0, 1 in x, pairs 2, 3 in y
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = x[2 * j], b = x[2 * j + 1], c = y[2 * j], d = y[2 * j + 1];
                x[2 * j] = a * t.c[j] - b * t.s[j];
                x[2 * j + 1] = a * t.s[j] + b * t.c[j];
                y[2 * j] = c * t.c[2 + j] - d * t.s[2 + j];
                y[2 * j + 1] = c * t.s[2 + j] + d * t.c[2 + j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[j], b = y[j];
                x[j] = a * t.c[j] - b * t.s[j];
                y[j] = a * t.s[j] + b * t.c[j];
            }
        }
    }
    LaneRow r;
    r.a = make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
    r.b = make_uint2(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]));
    return r;
}

}  // namespace attn
