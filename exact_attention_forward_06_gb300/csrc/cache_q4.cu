// cache_q4.cu -- reading a 4-bit cache: attn_gather_paged_q4 (back to packed
// bf16 keys and values), with given offsets or (for attn_fwd_paged_q4) its own.
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_ops.h"
#include "common.cuh"
#include "q4.cuh"

namespace attn {
namespace q4 {

constexpr int GWARPS = 8;

__device__ __forceinline__ float bf16_at(const uint8_t *p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}

// A word's eight values, rounded to bf16.  A code in bits 1..4 of a float whose other
// bits are those of 2^22 is 2^22 + n; the offset comes off exactly, s (n - 7.5) is exact
// in fp32 (8 + 5 bits), and the sum rounds to fp32 and then to bf16.
__device__ __forceinline__ uint4 unpack_word(uint32_t word, float s, float z) {
    uint32_t r[4];
    const float2 s2 = make_float2(s, s), z2 = make_float2(z, z), off = make_float2(-4194311.5f, -4194311.5f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = (j == 0 ? word << 1 : word >> (j == 0 ? 0 : 8 * j - 1)) & 0x1e, hi = word >> (8 * j + 3) & 0x1e;
        const float2 n = make_float2(__uint_as_float(0x4a800000u | lo), __uint_as_float(0x4a800000u | hi));
        const float2 v = ptx::fma2(s2, ptx::add2(n, off), z2);
        r[j] = ptx::pack_bf16x2(v.x, v.y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Where a warp's item lies: its sequence, the sequence's first row and length.
struct Found {
    int b, begin, L;
    bool ok;
};

// Whether a sequence's offsets and length are in order.
__device__ __forceinline__ bool in_order(const GatherQ4Params &p, int begin, int end, int L) {
    return begin >= 0 && end <= p.total_k && L >= 0 && L <= p.max_blocks * PAGE && (int64_t)end - begin == L;
}

// Looks all given offsets over, in blocks of their own behind the items' (with offsets out
// of order, no item need lead to a sequence).
constexpr int CHECKS = 8;  // sequences a thread
__device__ __forceinline__ void check_given(const GatherQ4Params &p, unsigned block) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < CHECKS; ++i) {
        const int64_t b = ((int64_t)block * CHECKS + i) * (GWARPS * 32) + threadIdx.x;
        if (b < p.B) bad = bad || !in_order(p, p.cu_k[b], p.cu_k[b + 1], p.seqlens[b]);
    }
    if (bad) report_status(p.status, kStatusDeviceBounds, kSiteQ4Offsets);
}

// The last sequence b with cu_k[b] / 16 + b <= j, from given offsets.
__device__ __forceinline__ Found find_given(const GatherQ4Params &p, int64_t j, int lane) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + (lane + 1) * step;
        const bool le = i < hi && (int64_t)p.cu_k[i] / PAGE + i <= j;
        lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
        hi = min(hi, lo + step);
    }
    const int begin = p.cu_k[lo], end = p.cu_k[lo + 1], L = p.seqlens[lo];
    return Found{lo, begin, L, in_order(p, begin, end, L)};
}

__device__ __forceinline__ int length_of(const GatherQ4Params &p, int b) {
    const int L = p.seqlens[b];
    return L < 0 || L > p.max_blocks * PAGE ? 0 : L;
}

// The same from the lengths alone, for offsets that begin at 0 and leave no gaps:
// a thread sums a run of sequences, the sums are scanned, and the warp looks for
// its item among the runs and then within one.  A length outside the table counts
// as 0; the sequences that go past total_k come last and are left out.  Block 0
// writes the offsets, and reports.
struct RunSums {
    int64_t start[GWARPS * 32];
    int64_t warp_sum[GWARPS];
    int last;
};

__device__ __forceinline__ Found find_own(const GatherQ4Params &p, int64_t j, int lane, RunSums &runs) {
    constexpr int THREADS = GWARPS * 32;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int b_lo = min(p.B, (int)threadIdx.x * per), b_hi = min(p.B, b_lo + per);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += length_of(p, b);
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    const int warp = threadIdx.x >> 5;
    if (lane == 31) runs.warp_sum[warp] = incl;
    if (threadIdx.x == 0) runs.last = 0;
    __syncthreads();
    int64_t before = incl - mine;
    for (int w = 0; w < warp; ++w) before += runs.warp_sum[w];
    runs.start[threadIdx.x] = before;
    if (blockIdx.x == 0) {
        int64_t end = before;
        int last = 0;  // the largest offset within the bound
        for (int b = b_lo; b < b_hi; ++b) {
            const int L = length_of(p, b);
            end += L;
            if (end <= p.total_k) last = (int)end;
            if (L != p.seqlens[b] || (end > p.total_k && L > 0))
                report_status(p.status, kStatusDeviceBounds, kSiteQ4Offsets);
        }
        atomicMax(&runs.last, last);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        int64_t end = before;
        if (threadIdx.x == 0) p.cu_out[0] = 0;
        for (int b = b_lo; b < b_hi; ++b) {
            end += length_of(p, b);
            p.cu_out[b + 1] = (int)min(end, (int64_t)runs.last);
        }
    }
    int n = 0;
    for (int r = lane; r < THREADS; r += 32)
        n += __popc(__ballot_sync(0xffffffffu, r * per < p.B && runs.start[r] / PAGE + r * per <= j));
    int b = (n - 1) * per;
    int64_t begin = runs.start[n - 1];
    Found f{b, 0, 0, false};
    for (int c = 0; c < per; c += 32) {
        const bool in = c + lane < per && b + c + lane < p.B;
        const int L = in ? length_of(p, b + c + lane) : 0;
        int64_t end = L;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, end, off);
            if (lane >= off) end += o;
        }
        const int64_t at = begin + end - L;
        const int k = __popc(__ballot_sync(0xffffffffu, in && at / PAGE + b + c + lane <= j));
        if (k == 0) break;
        f.b = b + c + k - 1;
        f.L = __shfl_sync(0xffffffffu, L, k - 1);
        const int64_t first = __shfl_sync(0xffffffffu, at, k - 1);
        f.ok = first + f.L <= p.total_k;
        f.begin = f.ok ? (int)first : 0;
        if (k < 32) break;
        begin += __shfl_sync(0xffffffffu, end, 31);
    }
    return f;
}

// One warp per page and KV head.  Item j of total_k / 16 + B candidate pages
// belongs to the last sequence b with cu_k[b] / 16 + b <= j, as its page
// j - (cu_k[b] / 16 + b): every sequence of L tokens gets at least ceil(L / 16)
// candidates whatever the other lengths, without a sum over the sequences'
// pages.  OWN: the offsets come from the lengths.  The block passes through shared
// memory, so that the loads are 16 bytes a lane and the stores whole rows of a
// head.  3.2 bytes are written for each one read; the bound is HBM: 68 thousand
// tokens of 8 heads (366 MB) take 57 us, 0.93 of the copy bandwidth.
template <bool OWN>
__global__ void __launch_bounds__(GWARPS * 32) gather_kernel(const GatherQ4Params p, unsigned item_blocks) {
    __shared__ __align__(16) uint8_t stage[GWARPS][BLOCK];
    __shared__ RunSums runs[1];
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    if (!OWN && blockIdx.x >= item_blocks) {
        check_given(p, blockIdx.x - item_blocks);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * GWARPS + warp;
    const int h = (int)(item % p.Hkv);
    const int64_t j = item / p.Hkv;
    const Found f = OWN ? find_own(p, j, lane, runs[0]) : find_given(p, j, lane);
    if (j >= (int64_t)p.total_k / PAGE + p.B) return;
    if (!f.ok) return;  // (reported by the blocks that look the offsets over)
    const int lo = f.b, begin = f.begin, L = f.L;
    const int64_t first = (int64_t)begin / PAGE + lo;
    const int64_t t0 = (j - first) * PAGE;
    if (j < first || t0 >= L) return;
    const int page = p.block_table[(int64_t)lo * p.max_blocks + (j - first)];
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && lane == 0) report_status(p.status, kStatusDeviceBounds, kSiteQ4Table);
    uint4 *to = reinterpret_cast<uint4 *>(stage[warp]);
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.cache) +
                                                        ((int64_t)page * p.Hkv + h) * BLOCK);
    uint4 part[BLOCK / 16 / 32];
#pragma unroll
    for (int i = 0; i < BLOCK / 16 / 32; ++i) part[i] = ok ? from[lane + 32 * i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < BLOCK / 16 / 32; ++i) to[lane + 32 * i] = part[i];
    __syncwarp();
    const uint8_t *blk = stage[warp];
    const int n = min(PAGE, L - (int)t0);
    // Two tokens a pass: lane = token x word of eight channels.
    const int w = lane & 15, g = w >> 2, r = 2 * (w & 3);
    for (int t = lane >> 4; t < n; t += 2) {
        const int64_t row = ((begin + t0 + t) * p.Hkv + h) * D + 8 * w;
        const uint32_t kw = *reinterpret_cast<const uint32_t *>(blk + k_word(t, w));
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.k_out) + row) =
            unpack_word(kw, bf16_at(blk + K_SCALES + t * 8 + g * 2), bf16_at(blk + K_CENTERS + t * 8 + g * 2));
        const uint32_t vw = (uint32_t)*reinterpret_cast<const uint16_t *>(blk + v_half(t, g, r)) |
                            (uint32_t)*reinterpret_cast<const uint16_t *>(blk + v_half(t, g, r + 1)) << 16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.v_out) + row) =
            unpack_word(vw, bf16_at(blk + V_SCALES + t * 8 + g * 2), bf16_at(blk + V_CENTERS + g * 32 + t * 2));
    }
}

}  // namespace q4

cudaError_t launch_gather_q4(const GatherQ4Params &p, cudaStream_t stream) {
    const int64_t items = ((int64_t)p.total_k / q4::PAGE + p.B) * p.Hkv;
    const int64_t blocks = (items + q4::GWARPS - 1) / q4::GWARPS;
    constexpr int64_t per = q4::GWARPS * 32 * q4::CHECKS;
    const int64_t grid = blocks + (p.cu_k ? (p.B + per - 1) / per : 0);
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(p.cu_k ? q4::gather_kernel<false> : q4::gather_kernel<true>, (unsigned)grid, q4::GWARPS * 32, 0,
                            stream, p, (unsigned)blocks);
}

}  // namespace attn
