// speculate.h -- host-side interface of the kernels around a tree of drafted tokens:
// verification against the target's probabilities, and the cache cut down to the
// accepted path.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace attn {

struct VerifyParams {
    const void *logits, *draft;  // [total][V] bf16 or fp32; draft may be nullptr
    int64_t logits_stride, draft_stride, noise_stride;  // elements per row
    const int32_t *tokens, *parents, *cu;
    const float *temperature;  // [B] or nullptr: no drawing anywhere
    const float *uniforms;     // [total]
    const float *noise;        // [B][V]
    int32_t *path, *out_tokens, *counts;
    int B, total, V, width;
    int fp32;  // type of logits and draft
    // All rows summed up ahead of the walk, in `pieces` slices of `piece` tokens (0: a
    // row when the walk comes to it): maximum and sum, or the largest logit's key.
    int pieces, piece;
    float2 *sums;  // [target, draft][total][pieces]
    // Where every sequence's walk ended, kVerifyEndBytes each, and behind them a list of
    // `width` numbers each; nullptr where nothing is drawn.
    uint8_t *ends;
    unsigned *status;
};

struct CompactParams {
    void *k_pages, *v_pages;  // [layers][num_pages][16][Hkv][128] bf16
    const int32_t *block_table, *seqlens, *cu, *path, *counts;
    int32_t *seqlens_out;
    int B, layers, Hkv, total, width, num_pages, max_blocks;
    int tensors;  // 1: K and V are one pool, whose rows move once
    unsigned *status;
};

constexpr int kVerifyEndBytes = 64;
// The slices of a row that are summed up ahead: `rows` rows in all.
int verify_piece(int64_t rows, int vocab, int *pieces);
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream);

}  // namespace attn
