// api_speculate.cu -- the C ABI of the operators around a tree of drafted tokens:
// argument validation and launches of the verification and of the cache's
// compaction.  Nothing here allocates device memory.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "api_internal.h"
#include "attn.h"
#include "speculate.h"

namespace {

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A device pointer to 4-byte elements.
bool ok4(const void *p) { return p != nullptr && aligned(p, 4); }

}  // namespace

// Whether all rows are summed up ahead of the walk, and in what slices.  That reads rows
// that the walk may not come to, but all at once; the walk by itself waits for one row
// after the other, 2 to 4 us each, with draft 4 to 8.  us ahead against not, rows of 131072
// tokens in bf16 where nothing else is said:
//   with draft, chains: 16 of 8 rows 31 against 51, 64 of 5 58 against 95, 64 of 12 96 against
//     156; trees, up to 16 rows: 8 of 16 41 against 54, 16 of 16 61 against 57, 32 of 8 101
//     against 73, 64 of 5 164 against 119, 64 of 8 183 against 153, 64 of 16 220 against 155,
//     the same 64 in fp32 59 against 95, 76 against 97 and 117 against 129; more rows: one of
//     120 (60 MB) 49 against 56, 4 of 48 (96 MB) 45 against 29, 16 of 24 (192 MB) 72 against 55;
//   without, trees: 64 of 4 rows (64 MB) 40 against 47, 64 of 5 (80 MB) 44 against 47, 16 of 8
//     (32 MB) 27 against 25, 16 of 15 (60 MB) 31 against 32, 16 of 16 (64 MB) 33 against 24, one
//     of 24 (6 MB) 18 against 21, one of 64 (16 MB) 21 against 21; of 32000, 64 of 8 rows (31
//     MB) 27 against 34, 64 of 16 (62 MB) 33 against 37, 64 of 30 (117 MB) 46 against 35.
// So, with draft: up to 16 rows a sequence, or 64 MB in all; without: 16 MB, or 64 where a
// sequence has up to 16 rows.  The host does not see whether trees are chains: the rule is
// right for chains, which a draft model's tokens mostly are, and for fp32, and costs large
// batches of short drawn trees in bf16 up to 42% more time.
static bool verify_ahead(int B, int total, int vocab, int max_seqlen, int dtype, bool draft, int *piece, int *pieces) {
    const int64_t rows = std::min<int64_t>(total, (int64_t)B * max_seqlen), MB = 1 << 20;
    const int64_t bytes = rows * vocab * (dtype == ATTN_DTYPE_BF16 ? 2 : 4) * (draft ? 2 : 1);
    const bool few = rows <= 16 * (int64_t)B;
    *pieces = 0;
    if (draft ? !few && bytes > 64 * MB : bytes > (few ? 64 : 16) * MB) return false;
    *piece = attn::verify_piece(rows * (draft ? 2 : 1), vocab, pieces);
    if ((int64_t)B * std::min(max_seqlen, 16) * (draft ? 2 : 1) <= 0x7fffffff / *pieces) return true;
    *pieces = 0;  // (more blocks than a launch has)
    return false;
}

// The two parts of the workspace: where the walks end, and the sums ahead of them.
static void verify_workspace(int B, int total, int max_seqlen, bool draft, int pieces, size_t *ends, size_t *sums) {
    *ends = ((size_t)B * (attn::kVerifyEndBytes + (size_t)max_seqlen * 4) + 255) & ~(size_t)255;
    *sums = (size_t)total * (draft ? 2 : 1) * pieces * 8;
}

extern "C" {

size_t attn_verify_tree_workspace_bytes(int B, int total, int vocab, int max_seqlen, int dtype, int with_draft) {
    if (B < 1 || total < 1 || vocab < 1 || vocab > 1 << 28 || max_seqlen < 1 ||
        max_seqlen > ATTN_TREE_MAX)
        return 0;
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP32) return 0;
    int piece, pieces;
    size_t ends, sums;
    verify_ahead(B, total, vocab, max_seqlen, dtype, with_draft != 0, &piece, &pieces);
    verify_workspace(B, total, max_seqlen, with_draft != 0, pieces, &ends, &sums);
    return ends + sums;
}

attn_status_t attn_verify_tree(const void *logits, const void *draft_logits, int dtype, const int32_t *tokens,
                               const int32_t *parents, const int32_t *cu_seqlens, const float *temperature,
                               const float *uniforms, const float *noise, int32_t *path, int32_t *out_tokens,
                               int32_t *counts, int B, int total, int vocab, int max_seqlen, size_t logits_stride,
                               size_t draft_stride, size_t noise_stride, void *workspace, size_t workspace_bytes,
                               void *stream) {
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_FP32) return ATTN_ERR_INVALID_ARG;
    const uintptr_t size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
    if (!logits || !aligned(logits, size) || (draft_logits && !aligned(draft_logits, size)))
        return ATTN_ERR_INVALID_ARG;
    if (!ok4(tokens) || !ok4(parents) || !ok4(cu_seqlens) || !ok4(path) || !ok4(out_tokens) || !ok4(counts))
        return ATTN_ERR_INVALID_ARG;
    // Drawing wants random numbers; without it there is nothing to be said of a draft's distribution.
    if (temperature ? (!aligned(temperature, 4) || !ok4(uniforms) || !ok4(noise))
                    : (draft_logits || uniforms || noise))
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || total < 1 || vocab < 1 || vocab > 1 << 28 || max_seqlen < 1 || max_seqlen > ATTN_TREE_MAX)
        return ATTN_ERR_INVALID_ARG;
    // Blocks: a cluster a sequence, and in the race a slice of 2048 tokens.
    if (B > 0x7fffffff / 8 || (int64_t)B * (((int64_t)vocab + 2047) / 2048) > 0x7fffffff) return ATTN_ERR_INVALID_ARG;
    const size_t top = (size_t)1 << 40, V = (size_t)vocab;
    if (logits_stride < V || logits_stride > top || (draft_logits && (draft_stride < V || draft_stride > top)) ||
        (temperature && (noise_stride < V || noise_stride > top)))
        return ATTN_ERR_INVALID_ARG;
    attn::VerifyParams p = {};
    p.logits = logits;
    p.draft = draft_logits;
    p.logits_stride = (int64_t)logits_stride;
    p.draft_stride = (int64_t)draft_stride;
    p.noise_stride = (int64_t)noise_stride;
    p.tokens = tokens;
    p.parents = parents;
    p.cu = cu_seqlens;
    p.temperature = temperature;
    p.uniforms = uniforms;
    p.noise = noise;
    p.path = path;
    p.out_tokens = out_tokens;
    p.counts = counts;
    p.B = B;
    p.total = total;
    p.V = vocab;
    p.width = max_seqlen;
    p.fp32 = dtype == ATTN_DTYPE_FP32 ? 1 : 0;
    verify_ahead(B, total, vocab, max_seqlen, dtype, draft_logits != nullptr, &p.piece, &p.pieces);
    size_t ends, sums;
    verify_workspace(B, total, max_seqlen, draft_logits != nullptr, p.pieces, &ends, &sums);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ends + sums) return ATTN_ERR_WORKSPACE;
    // A sequence's CTAs read its rows and numbers, and other sequences' CTAs theirs, in any
    // order with what is written.
    const size_t ints = (size_t)B * 4, rows = (size_t)total * 4, kept = ints * max_seqlen;
    const size_t drawn = temperature ? 1 : 0, drafted = draft_logits ? 1 : 0;
    if (attn::writes_overlap({{path, kept}, {out_tokens, kept}, {counts, ints}, {workspace, ends + sums}},
                             {{logits, ((total - 1) * logits_stride + V) * size},
                              {draft_logits, drafted * ((total - 1) * draft_stride + V) * size},
                              {tokens, rows},
                              {parents, rows},
                              {cu_seqlens, ints + 4},
                              {temperature, drawn * ints},
                              {uniforms, drawn * rows},
                              {noise, drawn * ((B - 1) * noise_stride + V) * 4}}))
        return ATTN_ERR_INVALID_ARG;
    p.ends = temperature ? static_cast<uint8_t *>(workspace) : nullptr;
    p.sums = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + ends);
    int sms;
    uint64_t budget;
    const attn_status_t st = attn::device_state(&sms, &p.status, &budget);
    if (st != ATTN_OK) return st;
    return attn::launch_verify(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_compact_paged(void *k_pages, void *v_pages, const int32_t *block_table, const int32_t *seqlens_k,
                                 const int32_t *cu_seqlens, const int32_t *path, const int32_t *counts,
                                 int32_t *seqlens_out, int B, int layers, int Hkv, int total, int max_seqlen, int d,
                                 int page_size, int num_pages, int max_blocks_per_seq, void *stream) {
    if (!k_pages || !v_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16)) return ATTN_ERR_INVALID_ARG;
    if (!ok4(block_table) || !ok4(seqlens_k) || !ok4(cu_seqlens) || !ok4(path) || !ok4(counts) || !ok4(seqlens_out))
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || layers < 1 || Hkv < 1 || total < 1 || num_pages < 1 || max_blocks_per_seq < 1 || max_seqlen < 1 ||
        max_seqlen > ATTN_TREE_MAX)
        return ATTN_ERR_INVALID_ARG;
    if ((int64_t)num_pages * 16 > 0x7fffffff || (int64_t)max_blocks_per_seq * 16 > 0x7fffffff)
        return ATTN_ERR_INVALID_ARG;
    if (d != 128 || page_size != 16) return ATTN_ERR_UNSUPPORTED;
    // One block a sequence and 128 columns of 16 bytes.
    if ((int64_t)layers * 2 * Hkv > 0x7fffffff / 16 ||
        ((int64_t)layers * 2 * Hkv * 16 + 127) / 128 > (int64_t)0x7fffffff / B)
        return ATTN_ERR_INVALID_ARG;
    // Every block reads the lengths, offsets, paths and pages, in any order with the first
    // block's new lengths.
    const size_t ints = (size_t)B * 4, pool = (size_t)layers * num_pages * 16 * Hkv * 256;
    if (attn::writes_overlap({{seqlens_out, ints}},
                             {{seqlens_k, ints}, {counts, ints}, {cu_seqlens, ints + 4}, {path, ints * max_seqlen},
                              {block_table, ints * max_blocks_per_seq}, {k_pages, pool}, {v_pages, pool}}))
        return ATTN_ERR_INVALID_ARG;
    // A row's threads move it once: keys and values may be the same rows, and no others.
    if (k_pages != v_pages && attn::writes_overlap({{k_pages, pool}, {v_pages, pool}}, {})) return ATTN_ERR_INVALID_ARG;
    attn::CompactParams p = {};
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.block_table = block_table;
    p.seqlens = seqlens_k;
    p.cu = cu_seqlens;
    p.path = path;
    p.counts = counts;
    p.seqlens_out = seqlens_out;
    p.B = B;
    p.layers = layers;
    p.tensors = k_pages == v_pages ? 1 : 2;
    p.Hkv = Hkv;
    p.total = total;
    p.width = max_seqlen;
    p.num_pages = num_pages;
    p.max_blocks = max_blocks_per_seq;
    int sms;
    uint64_t budget;
    const attn_status_t st = attn::device_state(&sms, &p.status, &budget);
    if (st != ATTN_OK) return st;
    return attn::launch_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
