// cache_ops.h -- host-side interface of the kernels around the paged cache:
// head norms with the position rotation, the appends into the bf16 and the
// 4-bit cache, and the attention over the 4-bit cache.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "attn.h"

namespace attn {

// The rotation and norms shared by attn_qk_norm_rope and the appends.
struct RotateParams {
    const void *q_weight;  // bf16 [d] or nullptr
    const void *k_weight;
    float eps;
    const int32_t *positions;  // [n_axes][tokens] or nullptr
    int n_axes;
    const attn_rope_pair_t *rope;
    int rotary_dim;
    int interleaved;
    unsigned *status;
};

struct NormRopeParams {
    RotateParams r;
    const void *q, *k;  // k may be nullptr (Hkv 0)
    void *q_out, *k_out;
    int B, S, Hq, Hkv, bhsd;
    int64_t q_stride[3], k_stride[3];  // batch, position, head (elements)
};

struct AppendParams {
    RotateParams r;
    const void *q, *k, *v;  // q may be nullptr (Hq 0)
    void *q_out;
    void *k_pages, *v_pages;  // bf16 pools, or
    void *cache;              // the 4-bit cache
    const int32_t *block_table, *seqlens, *cu;  // cu nullptr: one token per sequence
    int B, total, Hq, Hkv, num_pages, max_blocks;
    int64_t q_stride, k_stride, v_stride;  // elements per token
};

struct GatherQ4Params {
    const void *cache;
    const int32_t *block_table, *seqlens;
    const int32_t *cu_k;  // offsets, or nullptr: made from seqlens and written to
    int32_t *cu_out;      // [B + 1]
    void *k_out, *v_out;
    int B, Hkv, total_k, num_pages, max_blocks;
    unsigned *status;
};

struct DecodeQ4Params {
    const void *q, *cache;
    const int32_t *block_table, *seqlens;
    void *out;
    float *lse;
    // Partial results of the shares that cut a sequence, for each CTA its first
    // and its last segment: normalised outputs and log2-sum-exp2 of its heads.
    float *o_part;    // [CTAs][2][heads][d]
    float *lse_part;  // [CTAs][2][heads]
    int4 *cuts;       // [CTAs][2]
    int B, Hq, Hkv, num_pages, max_blocks;
    float scale_log2;
    unsigned *status;
    uint64_t budget_ns;
    int inject;  // 1: the first two warps of each CTA issue no copy (fault-injection test)
};

// Launches a kernel as a programmatic dependent of the work before it on the
// stream: its blocks may be set up while that work finishes.  Such a kernel
// begins with ptx::wait_for_prior_work() (griddepcontrol.wait), before it reads
// or writes anything.  It reads with ordinary loads only: the work before may still
// be writing when its first blocks start, and the non-coherent loads of __ldg want
// data that nobody writes as long as the kernel runs.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Whether a launch's grid fits (the launches count on it).
bool norm_rope_fits(const NormRopeParams &p);
bool append_fits(const AppendParams &p);
cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream);
cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_gather_q4(const GatherQ4Params &p, cudaStream_t stream);
// Rows of o_part and lse_part, and CTAs, at most: a pure function of the shape,
// the workspace's size goes by them.
size_t decode_q4_partial_rows(int B, int Hq, int Hkv, int max_blocks, size_t *ctas);
cudaError_t launch_decode_q4(const DecodeQ4Params &p, int sm_count, cudaStream_t stream);

}  // namespace attn
