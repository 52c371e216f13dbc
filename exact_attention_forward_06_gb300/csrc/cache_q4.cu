// cache_q4.cu -- reading a 4-bit cache: attn_gather_paged_q4 (back to packed
// bf16 keys and values) and the offsets of attn_fwd_paged_q4.
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_ops.h"
#include "common.cuh"
#include "q4.cuh"

namespace attn {
namespace q4 {

constexpr int GWARPS = 8;

// Value of channel 8 w + j's code in the word, given the group's scale and center.
__device__ __forceinline__ float value_of(uint32_t n, float s, float z) {
    // s (n - 7.5) is exact in fp32 (8 + 5 bits), the sum rounds once
    return fmaf(s, (float)n - 7.5f, z);
}

__device__ __forceinline__ float bf16_at(const uint8_t *p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}

// A word's eight values, rounded to bf16.
__device__ __forceinline__ uint4 unpack_word(uint32_t word, float s, float z) {
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        r[j] = ptx::pack_bf16x2(value_of(word >> (8 * j) & 15, s, z), value_of(word >> (8 * j + 4) & 15, s, z));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// One warp per page and KV head.  Item j of total_k / 16 + B candidate pages
// belongs to the last sequence b with cu_k[b] / 16 + b <= j, as its page
// j - (cu_k[b] / 16 + b): every sequence of L tokens gets at least ceil(L / 16)
// candidates whatever the other lengths, without a sum over the sequences.
__global__ void __launch_bounds__(GWARPS * 32) gather_kernel(const GatherQ4Params p) {
    __shared__ __align__(16) uint8_t stage[GWARPS][BLOCK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * GWARPS + warp;
    const int h = (int)(item % p.Hkv);
    const int64_t j = item / p.Hkv;
    if (j >= (int64_t)p.total_k / PAGE + p.B) return;
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + (lane + 1) * step;
        const bool le = i < hi && (int64_t)__ldg(p.cu_k + i) / PAGE + i <= j;
        lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
        hi = min(hi, lo + step);
    }
    const int begin = __ldg(p.cu_k + lo), end = __ldg(p.cu_k + lo + 1);
    const int L = __ldg(p.seqlens + lo);
    const int64_t first = (int64_t)begin / PAGE + lo;
    if (begin < 0 || end > p.total_k || L != end - begin || L < 0 || L > p.max_blocks * PAGE) {
        if (lane == 0) report_status(p.status, kStatusDeviceBounds, kSiteQ4Offsets);
        return;
    }
    const int64_t t0 = (j - first) * PAGE;
    if (j < first || t0 >= L) return;
    const int page = __ldg(p.block_table + (int64_t)lo * p.max_blocks + (j - first));
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && lane == 0) report_status(p.status, kStatusDeviceBounds, kSiteQ4Table);
    uint4 *to = reinterpret_cast<uint4 *>(stage[warp]);
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.cache) +
                                                        ((int64_t)page * p.Hkv + h) * BLOCK);
#pragma unroll
    for (int i = 0; i < BLOCK / 16 / 32; ++i)
        to[lane + 32 * i] = ok ? __ldg(from + lane + 32 * i) : make_uint4(0, 0, 0, 0);
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

// One CTA: offsets of the packed keys from the cache lengths.
constexpr int OFF_THREADS = 1024;
__global__ void __launch_bounds__(OFF_THREADS) offsets_kernel(const int32_t *seqlens, int32_t *cu_k,
                                                              int32_t *lens_out, int B, int max_blocks, int max_total,
                                                              unsigned *status) {
    __shared__ int64_t warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t base = 0;  // of this round of OFF_THREADS sequences
    if (threadIdx.x == 0) cu_k[0] = 0;
    for (int b0 = 0; b0 < B; b0 += OFF_THREADS) {
        const int b = b0 + threadIdx.x;
        int L = b < B ? seqlens[b] : 0;
        bool bad = L < 0 || L > max_blocks * PAGE;
        if (bad) L = 0;
        int64_t sum = L;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int64_t before = base, all = base;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) before += warp_sum[i];
            all += warp_sum[i];
        }
        // Past the bound: this sequence and those after it count as empty.
        const int64_t end = before + sum;
        if (end > max_total && L > 0) {
            bad = true;
            L = 0;
        }
        if (b < B) {
            cu_k[b + 1] = (int32_t)(end > max_total ? -1 : end);
            lens_out[b] = L;
            if (bad) report_status(status, kStatusDeviceBounds, kSiteQ4Offsets);
        }
        base = all;
        __syncthreads();
    }
    __syncthreads();
    // The offsets past the bound stay at the last one within it.
    if (base > max_total && threadIdx.x == 0) {
        for (int b = 0; b < B; ++b)
            if (cu_k[b + 1] < 0) cu_k[b + 1] = cu_k[b];
    }
}

}  // namespace q4

cudaError_t launch_gather_q4(const GatherQ4Params &p, cudaStream_t stream) {
    const int64_t items = ((int64_t)p.total_k / q4::PAGE + p.B) * p.Hkv;
    const int64_t grid = (items + q4::GWARPS - 1) / q4::GWARPS;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    q4::gather_kernel<<<(unsigned)grid, q4::GWARPS * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_q4_offsets(const int32_t *seqlens, int32_t *cu_k, int32_t *lens_out, int B, int max_blocks,
                              int max_total, unsigned *status, cudaStream_t stream) {
    q4::offsets_kernel<<<1, q4::OFF_THREADS, 0, stream>>>(seqlens, cu_k, lens_out, B, max_blocks, max_total, status);
    return cudaGetLastError();
}

}  // namespace attn
