// norm_rope.cu -- head norms with the position rotation: attn_qk_norm_rope, and
// on the way into the paged bf16 cache and the 4-bit cache (the appends).
//
// Every head row is read once and written once (512 B of traffic for about 60
// instructions of each of 16 lanes), so the bound is HBM bandwidth, and for a
// decode step's few tokens the latency of one launch.  A half-warp owns U head
// rows of one token (norm_rope.cuh has the lane layout): their loads are all in
// flight before the first is used, and the token's angles are computed once for
// the U rows.
//
// Measured on one GB300 (copy bandwidth 6781 GB/s): norm and rotation of 32760
// tokens, 12 + 12 heads (403 MB) 65 us, 0.91 of it; the append of 18 thousand
// tokens, 32 / 8 heads, into bf16 pages (464 MB) 70.5 us, 0.97.  Into the 4-bit cache
// the same tokens take 84 us: there the quantisation's instructions are the bound
// (3.0 of 4 issued per clock).  With 256 threads a block these took 71, 73 and 95 us.
// One token of each of 32 sequences: 3.4 us into bf16 pages and 6.1 into the 4-bit cache
// (in a graph), whose rows a half-warp quantises one after the other.
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_ops.h"
#include "common.cuh"
#include "norm_rope.cuh"
#include "q4.cuh"

namespace attn {
namespace nr {

constexpr int D = 128;
constexpr int THREADS = 128;
constexpr int HALVES = THREADS / 16;  // half-warps, one token each

// The rows of a token go to half-warps in chunks of one tensor's heads: `chunks`
// chunks of at most `rows` heads.
struct Chunks {
    int rows, chunks;
};

struct Place {
    int64_t token;  // this half-warp's token (the last one again for half-warps past it)
    bool there;     // whether the half-warp has a token of its own
    int chunk;      // of the token's chunks, the tensors' one after the other: the same in the whole block
    int l;          // lane 0 .. 15
};

// blockIdx.x: token block x chunk, the chunks of a token block adjacent.
__device__ __forceinline__ Place place(int chunks, int64_t tokens) {
    Place p;
    const unsigned tb = blockIdx.x / (unsigned)chunks;
    const int64_t t = (int64_t)tb * HALVES + (threadIdx.x >> 4);
    p.there = t < tokens;
    p.token = p.there ? t : tokens - 1;
    p.chunk = (int)(blockIdx.x - tb * (unsigned)chunks);
    p.l = threadIdx.x & 15;
    return p;
}

template <bool INTER, int U>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const NormRopeParams p, Chunks cq, Chunks ck) {
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    const Place at = place(cq.chunks + ck.chunks, (int64_t)p.B * p.S);
    const int b = (int)(at.token / p.S), s = (int)(at.token - (int64_t)b * p.S);
    const LanePieces lp = lane_pieces<INTER>(at.l, p.r.rotary_dim);
    const bool is_q = at.chunk < cq.chunks;
    const Chunks c = is_q ? cq : ck;
    const int H = is_q ? p.Hq : p.Hkv, h0 = (is_q ? at.chunk : at.chunk - cq.chunks) * c.rows;
    const int n = min(c.rows, H - h0);
    const int64_t step = is_q ? p.q_stride[2] : p.k_stride[2];
    const uint16_t *in = is_q ? static_cast<const uint16_t *>(p.q) + b * p.q_stride[0] + s * p.q_stride[1]
                              : static_cast<const uint16_t *>(p.k) + b * p.k_stride[0] + s * p.k_stride[1];
    in += h0 * step;
    LaneRow x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u < n) x[u] = load_row<INTER>(in + u * step, lp);
    const void *weight = is_q ? p.r.q_weight : p.r.k_weight;
    const LaneTurn turn = lane_turn(p.r, at.l, at.token, (int64_t)p.B * p.S, s);
    const LaneFactors f = lane_factors<INTER>(turn, weight, lp);
    uint16_t *out = static_cast<uint16_t *>(is_q ? p.q_out : p.k_out) +
                    (p.bhsd ? ((int64_t)b * H + h0) * p.S + s : at.token * H + h0) * D;
    const int64_t out_step = p.bhsd ? (int64_t)p.S * D : D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u >= n) break;
        const LaneRow y = norm_rotate<INTER>(x[u], weight != nullptr, p.r.eps, f, lp.rotates);
        if (at.there) store_row<INTER>(out + u * out_step, lp, y);
    }
}

// Looks all offsets over, in blocks of their own behind the rows' (the row of a token need
// not lead to the sequence whose offsets are wrong): in order, and within the rows.
constexpr int CHECKS = 8;  // sequences a thread
__device__ __forceinline__ void check_offsets(const AppendParams &p, unsigned block) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < CHECKS; ++i) {
        const int64_t b = ((int64_t)block * CHECKS + i) * THREADS + threadIdx.x;
        if (b < p.B) {
            const int begin = p.cu[b], end = p.cu[b + 1];
            bad = bad || begin < 0 || end < begin || end > p.total;
        }
    }
    if (bad) report_status(p.r.status, kStatusDeviceBounds, kSiteAppendOffsets);
}

// Where a new token goes: its sequence's position for it, and its page (-1: a
// bad table entry, already reported).  Returns false when the token belongs to
// no sequence, its row is idle or its sequence is malformed (reported).  The
// whole warp takes part.
__device__ __forceinline__ bool locate(const AppendParams &p, const Place &at, int *slot, int64_t *page) {
    const int t = (int)at.token;
    int b = t, begin = t, end = t + 1;
    *slot = 0;
    *page = -1;
    if (p.cu) {
        // The last b with cu[b] <= t, by 16 probes a round.
        int lo = 0;
        for (int len = p.B; len > 1;) {
            const int step = (len + 15) >> 4;
            const int i = lo + (at.l + 1) * step;
            const bool le = (at.l + 1) * step < len && i < p.B && p.cu[i] <= t;
            const unsigned votes = __ballot_sync(0xffffffffu, le) >> (threadIdx.x & 16);
            lo += __popc(votes & 0xffffu) * step;
            len = step;
        }
        b = lo;
        begin = p.cu[b];
        end = p.cu[b + 1];
        // A row of no sequence, or of malformed offsets (check_offsets reports them).
        if (t < begin || t >= end || begin < 0 || end > p.total) return false;
    }
    const int L = p.seqlens[b];
    if (L == 0 && !p.cu) return false;  // an idle row of a batch of single tokens
    if (L < end - begin || L > p.max_blocks * 16) {
        if (at.l == 0) report_status(p.r.status, kStatusDeviceBounds, kSiteAppendSlot);
        return false;
    }
    *slot = L - (end - t);
    const int pg = p.block_table[(int64_t)b * p.max_blocks + *slot / 16];
    if (pg >= 0 && pg < p.num_pages)
        *page = pg;
    else if (at.l == 0)
        report_status(p.r.status, kStatusDeviceBounds, kSiteAppendSlot);
    return true;
}

// Quantises a head row, eight consecutive channels 8 l .. 8 l + 7 a lane, into token
// t's place in its block (when `there`; the whole warp takes part).
__device__ __forceinline__ void quantise_store(uint8_t *block, int t, bool is_v, int l, uint4 v, bool there) {
    constexpr unsigned mask = 0xffffffffu;
    // The group's (four lanes') largest member and the largest of the negated ones,
    // as one bf16 pair.
    const uint32_t top = q4::max2(q4::max2(v.x, v.y), q4::max2(v.z, v.w));
    constexpr uint32_t SIGNS = 0x80008000u;
    const uint32_t neg = q4::max2(q4::max2(v.x ^ SIGNS, v.y ^ SIGNS), q4::max2(v.z ^ SIGNS, v.w ^ SIGNS));
    uint32_t both = q4::max2(__byte_perm(top, neg, 0x5410), __byte_perm(top, neg, 0x7632));
    both = q4::max2(both, __shfl_xor_sync(mask, both, 1, 16));
    both = q4::max2(both, __shfl_xor_sync(mask, both, 2, 16));
    const q4::GroupScale gs = q4::group_scale(bf_lo(both), -bf_hi(both));
    const float x[8] = {bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y), bf_lo(v.z), bf_hi(v.z), bf_lo(v.w), bf_hi(v.w)};
    const uint32_t word = q4::code_word(x, gs);
    const int g = l >> 2;
    if (!is_v) {
        if (!there) return;
        *reinterpret_cast<uint32_t *>(block + q4::k_word(t, l)) = word;
        if ((l & 3) == 0) {
            *reinterpret_cast<uint16_t *>(block + q4::K_SCALES + t * 8 + g * 2) = gs.s;
            *reinterpret_cast<uint16_t *>(block + q4::K_CENTERS + t * 8 + g * 2) = gs.z;
        }
    } else {
        // The word's halves are r = 2 (l % 4) and the next of group g.  Two exchanges
        // bring the four groups of one r together: lanes of even g take the even
        // r, those of odd g the odd one; then g = 0, 1 hold all eight bytes.
        const uint32_t w1 = __shfl_xor_sync(mask, word, 4, 16);
        const uint32_t two = g & 1 ? __byte_perm(w1, word, 0x7632) : __byte_perm(word, w1, 0x5410);
        const uint32_t rest = __shfl_xor_sync(mask, two, 8, 16);
        if (!there) return;
        if (g < 2)
            *reinterpret_cast<uint2 *>(block + q4::v_half(t, 0, 2 * (l & 3) + g)) = make_uint2(two, rest);
        if ((l & 3) == 0) {
            *reinterpret_cast<uint16_t *>(block + q4::V_SCALES + t * 8 + g * 2) = gs.s;
            *reinterpret_cast<uint16_t *>(block + q4::V_CENTERS + g * 32 + t * 2) = gs.z;
        }
    }
}

// Seven blocks an SM, eight for the 4-bit cache: its quantising branch would otherwise
// take 85 registers and leave the query rows, two thirds of the work, too few warps
// (with the read-back, 6, 7, 8 blocks: 148, 144, 141 us; the bf16 append, 7, 8: 69.9,
// 70.7).
template <bool INTER, bool Q4, int U>
__global__ void __launch_bounds__(THREADS, Q4 ? 8 : 7)
    append_kernel(const AppendParams p, Chunks cq, Chunks ckv, unsigned row_blocks) {
    // Q4: the lane layout of a rotated row goes to eight consecutive channels
    // a lane through shared memory, one row per half-warp.
    __shared__ __align__(16) uint16_t turn_row[Q4 && !INTER ? HALVES : 1][Q4 && !INTER ? D : 8];
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    if (blockIdx.x >= row_blocks) {
        check_offsets(p, blockIdx.x - row_blocks);
        return;
    }
    const Place at = place(cq.chunks + 2 * ckv.chunks, p.total);
    const bool is_q = at.chunk < cq.chunks, is_v = at.chunk >= cq.chunks + ckv.chunks;
    const Chunks c = is_q ? cq : ckv;
    const int H = is_q ? p.Hq : p.Hkv;
    const int h0 = (is_q ? at.chunk : at.chunk - cq.chunks - (is_v ? ckv.chunks : 0)) * c.rows;
    const int n = min(c.rows, H - h0);
    // Values are not rotated: eight consecutive channels a lane.
    const LanePieces lp = lane_pieces<INTER>(at.l, is_v ? 0 : p.r.rotary_dim);
    const uint16_t *in = is_q   ? static_cast<const uint16_t *>(p.q) + at.token * p.q_stride
                         : is_v ? static_cast<const uint16_t *>(p.v) + at.token * p.v_stride
                                : static_cast<const uint16_t *>(p.k) + at.token * p.k_stride;
    in += h0 * D;
    // Rows that are quantised go through a rolled loop, the next two rows' loads in
    // flight: unrolled, their code is eight times as long and spills.
    constexpr int AHEAD = 2;
    const bool rolled = Q4 && !is_q;
    LaneRow x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u < n && (u < AHEAD || !rolled)) x[u] = load_row<INTER>(in + u * D, lp);
    int slot = 0;
    int64_t page = -1;
    const bool owned = locate(p, at, &slot, &page) && at.there;
    const void *weight = is_q ? p.r.q_weight : is_v ? nullptr : p.r.k_weight;
    LaneFactors f;
    if (!is_v) f = lane_factors<INTER>(lane_turn(p.r, at.l, at.token, p.total, slot), weight, lp);
    const bool there = owned && (is_q || page >= 0);
    if (page < 0) page = 0;  // (nothing is written there)
    if (rolled) {
        uint8_t *block = static_cast<uint8_t *>(p.cache) + (page * p.Hkv + h0) * q4::BLOCK;
        LaneRow now = x[0], next = x[1];
#pragma unroll 1
        for (int u = 0; u < n; ++u) {
            LaneRow y = now;
            now = next;
            if (u + AHEAD < n) next = load_row<INTER>(in + (u + AHEAD) * D, lp);
            if (!is_v) y = norm_rotate<INTER>(y, weight != nullptr, p.r.eps, f, lp.rotates);
            uint4 v = make_uint4(y.a.x, y.a.y, y.b.x, y.b.y);
            if (!INTER && !is_v) {
                uint16_t *mine = turn_row[threadIdx.x >> 4];
                __syncwarp();  // the row before has been read
                store_row<false>(mine, lp, y);
                __syncwarp();
                v = *reinterpret_cast<const uint4 *>(mine + 8 * at.l);
            }
            quantise_store(block, slot & 15, is_v, at.l, v, there);
            block += q4::BLOCK;
        }
        return;
    }
    uint16_t *out = is_q ? static_cast<uint16_t *>(p.q_out) + (at.token * p.Hq + h0) * D
                         : static_cast<uint16_t *>(is_v ? p.v_pages : p.k_pages) +
                               ((page * 16 + (slot & 15)) * p.Hkv + h0) * D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u >= n) break;
        LaneRow y = x[u];
        if (!is_v) y = norm_rotate<INTER>(x[u], weight != nullptr, p.r.eps, f, lp.rotates);
        if (there) store_row<INTER>(out + u * D, lp, y);
    }
}

}  // namespace nr

namespace {

// H heads in as few chunks of at most U as go, of equal size.
nr::Chunks chunks_of(int H, int U) {
    const int chunks = (H + U - 1) / U;
    return {chunks ? (H + chunks - 1) / chunks : 0, chunks};
}

// Token blocks x chunks.
int64_t row_blocks(int64_t tokens, int64_t chunks) { return (tokens + nr::HALVES - 1) / nr::HALVES * chunks; }

// Blocks that look the offsets over.
int64_t check_blocks(const AppendParams &p) {
    constexpr int64_t per = nr::THREADS * nr::CHECKS;
    return p.cu ? (p.B + per - 1) / per : 0;
}

template <int U>
cudaError_t norm_rope_u(const NormRopeParams &p, cudaStream_t stream) {
    const nr::Chunks cq = chunks_of(p.Hq, U), ck = chunks_of(p.Hkv, U);
    const unsigned grid = (unsigned)row_blocks((int64_t)p.B * p.S, cq.chunks + ck.chunks);
    if (p.r.interleaved) return launch_dependent(nr::norm_rope_kernel<true, U>, grid, nr::THREADS, 0, stream, p, cq, ck);
    return launch_dependent(nr::norm_rope_kernel<false, U>, grid, nr::THREADS, 0, stream, p, cq, ck);
}

template <int U>
cudaError_t append_u(const AppendParams &p, cudaStream_t stream) {
    const nr::Chunks cq = chunks_of(p.Hq, U), ckv = chunks_of(p.Hkv, U);
    const unsigned rows = (unsigned)row_blocks(p.total, cq.chunks + 2 * ckv.chunks);
    const unsigned grid = rows + (unsigned)check_blocks(p);
    const auto kernel = p.cache ? (p.r.interleaved ? nr::append_kernel<true, true, U> : nr::append_kernel<false, true, U>)
                                : (p.r.interleaved ? nr::append_kernel<true, false, U> : nr::append_kernel<false, false, U>);
    return launch_dependent(kernel, grid, nr::THREADS, 0, stream, p, cq, ckv, rows);
}

}  // namespace

// Rows a half-warp takes: the unrolled row count U that covers the tensors' heads
// with the least work, a chunk's own (angles, factors, addresses) counting as three
// rows and the unrolled but unused rows in full.  Measured on 12 + 12 heads (32760
// tokens): U = 4 70 us, 6 64 us, 8 67 us; on 32 + 8 + 8 heads (about 18 thousand
// tokens): 79, 77 and 70 us.
static int rows_per_chunk(int Hq, int Hkv, int kv_tensors) {
    int best = 0, best_cost = 0;
    for (int U : {8, 6, 4}) {
        const int cost = (chunks_of(Hq, U).chunks + kv_tensors * chunks_of(Hkv, U).chunks) * (U + 3);
        if (best == 0 || cost < best_cost) {
            best = U;
            best_cost = cost;
        }
    }
    return best;
}

// The most heads that a token has; chunk counts are then far from overflowing.
constexpr int64_t MAX_HEADS = 65536;

bool norm_rope_fits(const NormRopeParams &p) {
    if ((int64_t)p.Hq + p.Hkv > MAX_HEADS) return false;
    const int U = rows_per_chunk(p.Hq, p.Hkv, 1);
    return row_blocks((int64_t)p.B * p.S, chunks_of(p.Hq, U).chunks + chunks_of(p.Hkv, U).chunks) <= 0x7fffffff;
}

bool append_fits(const AppendParams &p) {
    if (p.Hq + 2 * (int64_t)p.Hkv > MAX_HEADS) return false;
    const int U = rows_per_chunk(p.Hq, p.Hkv, 2);
    return row_blocks(p.total, chunks_of(p.Hq, U).chunks + 2 * chunks_of(p.Hkv, U).chunks) + check_blocks(p) <= 0x7fffffff;
}

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream) {
    switch (rows_per_chunk(p.Hq, p.Hkv, 1)) {
        case 8: return norm_rope_u<8>(p, stream);
        case 6: return norm_rope_u<6>(p, stream);
        default: return norm_rope_u<4>(p, stream);
    }
}

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream) {
    switch (rows_per_chunk(p.Hq, p.Hkv, 2)) {
        case 8: return append_u<8>(p, stream);
        case 6: return append_u<6>(p, stream);
        default: return append_u<4>(p, stream);
    }
}

}  // namespace attn
