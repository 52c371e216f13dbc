// norm_rope.cu -- head norms with the position rotation: attn_qk_norm_rope, and
// on the way into the paged bf16 cache and the 4-bit cache (the appends).
//
// Every head row is read once and written once (512 B of traffic for about 60
// instructions of each of 16 lanes), so the bound is HBM bandwidth, and for a
// decode step's few tokens the latency of one launch.  A half-warp owns U head
// rows of one token (norm_rope.cuh has the lane layout): their loads are all in
// flight before the first is used, and the token's angles are computed once for
// the U rows.
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_ops.h"
#include "common.cuh"
#include "norm_rope.cuh"
#include "q4.cuh"

namespace attn {
namespace nr {

constexpr int D = 128;
constexpr int THREADS = 256;
constexpr int HALVES = THREADS / 16;  // half-warps, one token each

struct Place {
    int64_t token;  // this half-warp's token
    int row0;       // its first head row: q heads, then k heads (then v heads)
    int l;          // lane 0 .. 15
    unsigned mask;  // the half-warp's lanes
};

// blockIdx.x: token block x row chunk, the chunks of a token block adjacent.
__device__ __forceinline__ Place place(int chunks, int U) {
    Place p;
    const unsigned tb = blockIdx.x / (unsigned)chunks;
    p.token = (int64_t)tb * HALVES + (threadIdx.x >> 4);
    p.row0 = (int)(blockIdx.x - tb * (unsigned)chunks) * U;
    p.l = threadIdx.x & 15;
    p.mask = 0xffffu << (threadIdx.x & 16);
    return p;
}

template <bool INTER, int U>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const NormRopeParams p, int chunks) {
    const Place at = place(chunks, U);
    if (at.token >= (int64_t)p.B * p.S) return;
    const int b = (int)(at.token / p.S), s = (int)(at.token - (int64_t)b * p.S);
    const LanePieces lp = lane_pieces<INTER>(at.l, p.r.rotary_dim);
    const int rows = p.Hq + p.Hkv;
    const uint16_t *q = static_cast<const uint16_t *>(p.q) + b * p.q_stride[0] + s * p.q_stride[1];
    const uint16_t *k = static_cast<const uint16_t *>(p.k) + b * p.k_stride[0] + s * p.k_stride[1];
    LaneRow x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = at.row0 + u;
        if (r < rows) x[u] = load_row<INTER>(r < p.Hq ? q + r * p.q_stride[2] : k + (r - p.Hq) * p.k_stride[2], lp);
    }
    LaneRow wq, wk;
    if (p.r.q_weight) wq = load_row<INTER>(p.r.q_weight, lp);
    if (p.r.k_weight) wk = load_row<INTER>(p.r.k_weight, lp);
    const LaneTurn turn = lane_turn(p.r, at.l, at.token, (int64_t)p.B * p.S, s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = at.row0 + u;
        if (r >= rows) break;
        const bool is_q = r < p.Hq;
        const int h = is_q ? r : r - p.Hq, H = is_q ? p.Hq : p.Hkv;
        const LaneRow *w = is_q ? (p.r.q_weight ? &wq : nullptr) : (p.r.k_weight ? &wk : nullptr);
        const LaneRow y = norm_rotate<INTER>(x[u], w, p.r.eps, turn, lp.rotates, at.mask);
        const int64_t o = p.bhsd ? ((int64_t)b * H + h) * p.S + s : at.token * H + h;
        store_row<INTER>(static_cast<uint16_t *>(is_q ? p.q_out : p.k_out) + o * D, lp, y);
    }
}

// Where a new token goes: its sequence's position for it, and its page (-1: a
// bad table entry, already reported).  Returns false when the token belongs to
// no sequence or its sequence is malformed (reported).
__device__ __forceinline__ bool locate(const AppendParams &p, const Place &at, int *slot, int64_t *page) {
    const int t = (int)at.token;
    int b = t, begin = t, end = t + 1;
    if (p.cu) {
        // The last b with cu[b] <= t, by 16 probes a round.
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int step = (hi - lo + 15) >> 4;
            const int i = lo + (at.l + 1) * step;
            const bool le = i < hi && __ldg(p.cu + i) <= t;
            const int n = __popc(__ballot_sync(at.mask, le) & at.mask);
            lo += n * step;
            hi = min(hi, lo + step);
        }
        b = lo;
        begin = __ldg(p.cu + b);
        end = __ldg(p.cu + b + 1);
        if (t < begin || t >= end) {
            // Before the first or behind the last sequence: nobody's row.
            const bool nobody = t < __ldg(p.cu) || t >= __ldg(p.cu + p.B);
            if (!nobody && at.l == 0) report_status(p.r.status, kStatusDeviceBounds, kSiteAppendOffsets);
            return false;
        }
        if (begin < 0 || end > p.total) {
            if (at.l == 0) report_status(p.r.status, kStatusDeviceBounds, kSiteAppendOffsets);
            return false;
        }
    }
    const int L = __ldg(p.seqlens + b);
    if (L < end - begin || L > p.max_blocks * 16) {
        if (at.l == 0) report_status(p.r.status, kStatusDeviceBounds, kSiteAppendSlot);
        return false;
    }
    *slot = L - (end - t);
    const int pg = __ldg(p.block_table + (int64_t)b * p.max_blocks + *slot / 16);
    const bool ok = pg >= 0 && pg < p.num_pages;
    if (!ok && at.l == 0) report_status(p.r.status, kStatusDeviceBounds, kSiteAppendSlot);
    *page = ok ? pg : -1;
    return true;
}

// Eight consecutive channels 8 l .. 8 l + 7 of a row, as held for quantising.
__device__ __forceinline__ void quantise_store(uint8_t *block, int t, bool is_v, int l, uint4 v, unsigned mask) {
    float x[8] = {bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y), bf_lo(v.z), bf_hi(v.z), bf_lo(v.w), bf_hi(v.w)};
    float hi = x[0], lo = x[0];
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        hi = fmaxf(hi, x[j]);
        lo = fminf(lo, x[j]);
        finite = finite && fabsf(x[j]) < INFINITY;  // false for NaN
    }
    // A group is 32 channels: four lanes.
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(mask, hi, off, 16));
        lo = fminf(lo, __shfl_xor_sync(mask, lo, off, 16));
        finite = __shfl_xor_sync(mask, finite ? 1 : 0, off, 16) && finite;
    }
    const q4::GroupScale gs = q4::group_scale(hi, lo, finite);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) word |= q4::code_of(x[j], gs) << (4 * j);
    const int g = l >> 2;
    if (!is_v) {
        *reinterpret_cast<uint32_t *>(block + q4::k_word(t, l)) = word;
        if ((l & 3) == 0) {
            *reinterpret_cast<uint16_t *>(block + q4::K_SCALES + t * 8 + g * 2) = gs.s;
            *reinterpret_cast<uint16_t *>(block + q4::K_CENTERS + t * 8 + g * 2) = gs.z;
        }
    } else {
        const int r = 2 * (l & 3);
        *reinterpret_cast<uint16_t *>(block + q4::v_half(t, g, r)) = (uint16_t)word;
        *reinterpret_cast<uint16_t *>(block + q4::v_half(t, g, r + 1)) = (uint16_t)(word >> 16);
        if ((l & 3) == 0) {
            *reinterpret_cast<uint16_t *>(block + q4::V_SCALES + t * 8 + g * 2) = gs.s;
            *reinterpret_cast<uint16_t *>(block + q4::V_CENTERS + g * 32 + t * 2) = gs.z;
        }
    }
}

template <bool INTER, bool Q4, int U>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendParams p, int chunks) {
    // Q4: the lane layout of a rotated row goes to eight consecutive channels
    // a lane through shared memory, one row per half-warp.
    __shared__ __align__(16) uint16_t turn_row[Q4 && !INTER ? HALVES : 1][Q4 && !INTER ? D : 8];
    const Place at = place(chunks, U);
    if (at.token >= p.total) return;
    const LanePieces lp = lane_pieces<INTER>(at.l, p.r.rotary_dim);
    const int k0 = p.Hq, v0 = p.Hq + p.Hkv, rows = v0 + p.Hkv;
    const uint16_t *q = static_cast<const uint16_t *>(p.q) + at.token * p.q_stride;
    const uint16_t *k = static_cast<const uint16_t *>(p.k) + at.token * p.k_stride;
    const uint16_t *v = static_cast<const uint16_t *>(p.v) + at.token * p.v_stride;
    LaneRow x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = at.row0 + u;
        if (r < v0)
            x[u] = load_row<INTER>(r < k0 ? q + (int64_t)r * D : k + (int64_t)(r - k0) * D, lp);
        else if (r < rows)
            x[u] = load_row<true>(v + (int64_t)(r - v0) * D, lane_pieces<true>(at.l, 0));
    }
    LaneRow wq, wk;
    if (p.r.q_weight) wq = load_row<INTER>(p.r.q_weight, lp);
    if (p.r.k_weight) wk = load_row<INTER>(p.r.k_weight, lp);
    int slot = 0;
    int64_t page = -1;
    if (!locate(p, at, &slot, &page)) return;
    LaneTurn turn;
    if (at.row0 < v0) turn = lane_turn(p.r, at.l, at.token, p.total, slot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = at.row0 + u;
        if (r >= rows) break;
        if (r < k0) {
            const LaneRow y = norm_rotate<INTER>(x[u], p.r.q_weight ? &wq : nullptr, p.r.eps, turn, lp.rotates, at.mask);
            store_row<INTER>(static_cast<uint16_t *>(p.q_out) + (at.token * p.Hq + r) * D, lp, y);
            continue;
        }
        if (page < 0) break;
        const bool is_v = r >= v0;
        const int h = is_v ? r - v0 : r - k0;
        LaneRow y = x[u];
        if (!is_v) y = norm_rotate<INTER>(x[u], p.r.k_weight ? &wk : nullptr, p.r.eps, turn, lp.rotates, at.mask);
        if (!Q4) {
            uint16_t *to = static_cast<uint16_t *>(is_v ? p.v_pages : p.k_pages) +
                           ((page * 16 + (slot & 15)) * p.Hkv + h) * D;
            if (is_v)
                store_row<true>(to, lane_pieces<true>(at.l, 0), y);
            else
                store_row<INTER>(to, lp, y);
        } else {
            uint4 c = make_uint4(y.a.x, y.a.y, y.b.x, y.b.y);
            if (!INTER && !is_v) {
                uint16_t *mine = turn_row[threadIdx.x >> 4];
                __syncwarp(at.mask);  // the row before has been read
                store_row<false>(mine, lp, y);
                __syncwarp(at.mask);
                c = *reinterpret_cast<const uint4 *>(mine + 8 * at.l);
            }
            quantise_store(static_cast<uint8_t *>(p.cache) + (page * p.Hkv + h) * q4::BLOCK, slot & 15, is_v, at.l, c,
                           at.mask);
        }
    }
}

}  // namespace nr

namespace {

// Token blocks x row chunks; false when the grid does not fit.
bool row_grid(int64_t tokens, int rows, int U, int *chunks, unsigned *grid) {
    *chunks = (rows + U - 1) / U;
    const int64_t n = (tokens + nr::HALVES - 1) / nr::HALVES * *chunks;
    if (n > 0x7fffffff) return false;
    *grid = (unsigned)n;
    return true;
}

template <int U>
cudaError_t norm_rope_u(const NormRopeParams &p, cudaStream_t stream) {
    int chunks;
    unsigned grid;
    if (!row_grid((int64_t)p.B * p.S, p.Hq + p.Hkv, U, &chunks, &grid)) return cudaErrorInvalidValue;
    if (p.r.interleaved)
        nr::norm_rope_kernel<true, U><<<grid, nr::THREADS, 0, stream>>>(p, chunks);
    else
        nr::norm_rope_kernel<false, U><<<grid, nr::THREADS, 0, stream>>>(p, chunks);
    return cudaGetLastError();
}

template <int U>
cudaError_t append_u(const AppendParams &p, cudaStream_t stream) {
    int chunks;
    unsigned grid;
    if (!row_grid(p.total, p.Hq + 2 * p.Hkv, U, &chunks, &grid)) return cudaErrorInvalidValue;
    if (p.cache) {
        if (p.r.interleaved)
            nr::append_kernel<true, true, U><<<grid, nr::THREADS, 0, stream>>>(p, chunks);
        else
            nr::append_kernel<false, true, U><<<grid, nr::THREADS, 0, stream>>>(p, chunks);
    } else {
        if (p.r.interleaved)
            nr::append_kernel<true, false, U><<<grid, nr::THREADS, 0, stream>>>(p, chunks);
        else
            nr::append_kernel<false, false, U><<<grid, nr::THREADS, 0, stream>>>(p, chunks);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream) { return norm_rope_u<1>(p, stream); }

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream) { return append_u<1>(p, stream); }

}  // namespace attn
