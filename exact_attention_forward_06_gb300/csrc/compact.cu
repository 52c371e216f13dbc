// compact.cu -- the paged cache cut down to the accepted path of a tree of drafted
// tokens (attn_compact_paged).
//
// The tree's n tokens are the last of a sequence's cache of L; the accepted nodes
// path[0] < path[1] < ... move to the tree's first places: row L - n + path[j] of every
// layer, KV head, K and V goes to row L - n + j.  Nodes that are in their place (a path's
// beginning) are not touched.
//
// A thread owns 16 bytes of a row, in one tensor and layer, and takes the path in order,
// UNROLL rows at a time: all of them are loaded before the first is stored, and a later
// row's source lies behind every earlier row's place (path[j] >= j, ascending), so no
// row is overwritten before it has been read and threads need not wait for one another.
// Bound by HBM where there are many rows, by the chain of four dependent reads (offsets,
// path, block table, row) where there are few.  Measured on one GB300: all 32 layers of
// 32 sequences, 8 KV heads, paths of 3 to 10 nodes (40 MB) 8.4 us, 4.7 TB/s; one layer of
// one sequence 4.6 us.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn.h"
#include "cache_ops.h"
#include "common.cuh"
#include "speculate.h"

namespace attn {
namespace cp {

constexpr int THREADS = 128;
constexpr int UNROLL = 8;
constexpr int PAGE = 16;

// blockIdx.x: sequence x block of 16-byte columns (layer, K or V where they are two pools, byte
// of the row).
__global__ void __launch_bounds__(THREADS) compact_kernel(const CompactParams p, int blocks_per_seq, int64_t columns) {
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    __shared__ int from[ATTN_TREE_MAX], to[ATTN_TREE_MAX];  // row of the pool, -1: a page outside it
    __shared__ int first_move;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / blocks_per_seq, block = blockIdx.x - b * blocks_per_seq;
    const int begin = p.cu[b], end = p.cu[b + 1], L = p.seqlens[b], count = p.counts[b];
    const int n = end - begin;
    bool bad = begin < 0 || end < begin || end > p.total || L < n || L > p.max_blocks * PAGE;
    const bool bad_path = !bad && (n > p.width || count < 0 || count > n);
    const bool report = block == 0;
    if (report && tid == 0 && bad) report_status(p.status, kStatusDeviceBounds, kSiteCompactOffsets);
    const int *path = p.path + (int64_t)b * p.width;
    bool wrong = bad || bad_path;
    if (tid == 0) first_move = count;
    __syncthreads();
    if (!wrong) {
        for (int j = tid; j < count; j += THREADS) {
            const int node = path[j], before = j > 0 ? path[j - 1] : -1;
            if (node <= before || node >= n) {
                wrong = true;
                break;
            }
            if (node != j) {
                atomicMin(&first_move, j);
                int rows[2];
                for (int k = 0; k < 2; ++k) {
                    const int t = L - n + (k ? j : node);
                    const int page = p.block_table[(int64_t)b * p.max_blocks + t / PAGE];
                    const bool ok = page >= 0 && page < p.num_pages;
                    if (!ok && report) report_status(p.status, kStatusDeviceBounds, kSiteCompactTable);
                    rows[k] = ok ? page * PAGE + t % PAGE : -1;
                }
                from[j] = rows[0];
                to[j] = rows[1];
            }
        }
    }
    wrong = __syncthreads_or(wrong);
    if (wrong) {  // nothing moves, and the length stays
        if (report && tid == 0) {
            if (!bad) report_status(p.status, kStatusDeviceBounds, kSiteCompactPath);
            p.seqlens_out[b] = L;
        }
        return;
    }
    if (report && tid == 0) p.seqlens_out[b] = L - n + count;
    const int64_t column = (int64_t)block * THREADS + tid;
    if (column >= columns) return;
    const int row_columns = p.Hkv * 16;
    const int64_t part = column / row_columns;  // layer x tensor
    const int64_t layer = p.tensors == 2 ? part >> 1 : part;
    uint4 *pool = static_cast<uint4 *>(p.tensors == 2 && (part & 1) ? p.v_pages : p.k_pages) +
                  layer * p.num_pages * PAGE * row_columns + (column - part * row_columns);
    for (int j0 = first_move; j0 < count; j0 += UNROLL) {
        uint4 x[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k)
            if (j0 + k < count && (from[j0 + k] | to[j0 + k]) >= 0) x[k] = pool[(int64_t)from[j0 + k] * row_columns];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k)
            if (j0 + k < count && (from[j0 + k] | to[j0 + k]) >= 0) pool[(int64_t)to[j0 + k] * row_columns] = x[k];
    }
}

}  // namespace cp

cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream) {
    const int64_t columns = (int64_t)p.layers * p.tensors * p.Hkv * 16;
    const int blocks = (int)((columns + cp::THREADS - 1) / cp::THREADS);
    return launch_dependent(cp::compact_kernel, dim3((unsigned)(blocks * p.B)), dim3(cp::THREADS), 0, stream, p, blocks,
                            columns);
}

}  // namespace attn
