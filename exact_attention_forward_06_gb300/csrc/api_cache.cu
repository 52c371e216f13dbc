// api_cache.cu -- the C ABI of the operators around the paged cache: argument
// validation and launches for the norm and rotation, the appends, and the
// attention over the 4-bit cache.  Nothing here allocates device memory.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "api_internal.h"
#include "attn.h"
#include "cache_ops.h"
#include "prefill_tc.h"

namespace {

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// A stride in elements: a multiple of 8 (16-byte loads) that 64-bit indexing holds.
bool stride_ok(size_t s) { return s % 8 == 0 && s <= ((size_t)1 << 40); }

// The norm and rotation arguments; everything but the device's status word.
attn_status_t check_rotate(const void *q_weight, const void *k_weight, float eps, const int32_t *positions, int n_axes,
                           const attn_rope_pair_t *rope, int rotary_dim, int d, attn::RotateParams *r) {
    if (d != 128) return ATTN_ERR_UNSUPPORTED;
    if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16))) return ATTN_ERR_INVALID_ARG;
    if ((q_weight || k_weight) && !(std::isfinite(eps) && eps >= 0.f)) return ATTN_ERR_INVALID_ARG;
    if (positions && !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
    if (n_axes < 1 || n_axes > 4) return ATTN_ERR_INVALID_ARG;
    if (rotary_dim < 0 || rotary_dim > d || (rotary_dim > 0) != (rope != nullptr)) return ATTN_ERR_INVALID_ARG;
    if (rope && !aligned(rope, 16)) return ATTN_ERR_INVALID_ARG;
    if (rotary_dim % 8 != 0) return ATTN_ERR_UNSUPPORTED;
    r->q_weight = q_weight;
    r->k_weight = k_weight;
    r->eps = eps;
    r->positions = positions;
    r->n_axes = n_axes;
    r->rope = rope;
    r->rotary_dim = rotary_dim;
    return ATTN_OK;
}

// The paged-cache arguments that the appends and the gather share.
attn_status_t check_table(const int32_t *block_table, const int32_t *seqlens, int B, int Hkv, int d, int page_size,
                          int num_pages, int max_blocks) {
    if (!block_table || !seqlens || !aligned(block_table, 4) || !aligned(seqlens, 4)) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || Hkv < 1 || num_pages < 1 || max_blocks < 1) return ATTN_ERR_INVALID_ARG;
    if ((int64_t)num_pages * 16 > 0x7fffffff || (int64_t)max_blocks * 16 > 0x7fffffff) return ATTN_ERR_INVALID_ARG;
    if (d != 128 || page_size != 16) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

attn_status_t append_impl(const void *q, const void *k, const void *v, void *q_out, void *k_pages, void *v_pages,
                          void *cache, const int32_t *block_table, const int32_t *seqlens_k,
                          const int32_t *cu_seqlens, const void *q_weight, const void *k_weight, float eps,
                          const int32_t *positions, int n_axes, const attn_rope_pair_t *rope, int rotary_dim,
                          int interleaved, int B, int total, int Hq, int Hkv, int d, int page_size, int num_pages,
                          int max_blocks, size_t q_stride, size_t k_stride, size_t v_stride, void *stream) {
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_table(block_table, seqlens_k, B, Hkv, d, page_size, num_pages, max_blocks);
    if (st != ATTN_OK) return st;
    if (cu_seqlens ? !aligned(cu_seqlens, 4) : total != B) return ATTN_ERR_INVALID_ARG;
    if (total < 1 || !stride_ok(k_stride) || !stride_ok(v_stride) || k_stride < (size_t)Hkv * d ||
        v_stride < (size_t)Hkv * d)
        return ATTN_ERR_INVALID_ARG;
    if (q) {
        if (!q_out || !aligned(q, 16) || !aligned(q_out, 16) || Hq < 1) return ATTN_ERR_INVALID_ARG;
        if (!stride_ok(q_stride) || q_stride < (size_t)Hq * d) return ATTN_ERR_INVALID_ARG;
        if (q_out == q && q_stride != (size_t)Hq * d) return ATTN_ERR_INVALID_ARG;
    } else if (q_out) {
        return ATTN_ERR_INVALID_ARG;
    }
    attn::AppendParams p = {};
    st = check_rotate(q ? q_weight : nullptr, k_weight, eps, positions, n_axes, rope, rotary_dim, d, &p.r);
    if (st != ATTN_OK) return st;
    p.r.interleaved = interleaved ? 1 : 0;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.cache = cache;
    p.block_table = block_table;
    p.seqlens = seqlens_k;
    p.cu = cu_seqlens;
    p.B = B;
    p.total = total;
    p.Hq = q ? Hq : 0;
    p.Hkv = Hkv;
    p.num_pages = num_pages;
    p.max_blocks = max_blocks;
    p.q_stride = (int64_t)q_stride;
    p.k_stride = (int64_t)k_stride;
    p.v_stride = (int64_t)v_stride;
    if (!attn::append_fits(p)) return ATTN_ERR_INVALID_ARG;
    int sms;
    uint64_t budget;
    if ((st = attn::device_state(&sms, &p.r.status, &budget)) != ATTN_OK) return st;
    return attn::launch_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, const void *q_weight,
                                const void *k_weight, float eps, const int32_t *positions, int n_axes,
                                const attn_rope_pair_t *rope, int rotary_dim, int interleaved, int B, int S, int Hq,
                                int Hkv, int d, int layout, size_t q_stride_b, size_t q_stride_s, size_t q_stride_h,
                                size_t k_stride_b, size_t k_stride_s, size_t k_stride_h, void *stream) {
    if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return ATTN_ERR_INVALID_ARG;
    if (k ? (!k_out || !aligned(k, 16) || !aligned(k_out, 16) || Hkv < 1) : k_out != nullptr)
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || S < 1 || Hq < 1 || (int64_t)B * S > 0x7fffffff) return ATTN_ERR_INVALID_ARG;
    if (layout != ATTN_LAYOUT_BSHD && layout != ATTN_LAYOUT_BHSD) return ATTN_ERR_INVALID_ARG;
    if (!stride_ok(q_stride_b) || !stride_ok(q_stride_s) || !stride_ok(q_stride_h)) return ATTN_ERR_INVALID_ARG;
    if (k && (!stride_ok(k_stride_b) || !stride_ok(k_stride_s) || !stride_ok(k_stride_h)))
        return ATTN_ERR_INVALID_ARG;
    attn::NormRopeParams p = {};
    attn_status_t st =
        check_rotate(q_weight, k ? k_weight : nullptr, eps, positions, n_axes, rope, rotary_dim, d, &p.r);
    if (st != ATTN_OK) return st;
    p.r.interleaved = interleaved ? 1 : 0;
    p.bhsd = layout == ATTN_LAYOUT_BHSD ? 1 : 0;
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.B = B;
    p.S = S;
    p.Hq = Hq;
    p.Hkv = k ? Hkv : 0;
    // In place, a row must be read where it is written (a stride of an axis of
    // length one is never used).
    const auto dense = [&](int H, size_t sb, size_t ss, size_t sh) {
        const size_t ws = p.bhsd ? (size_t)d : (size_t)H * d, wh = p.bhsd ? (size_t)S * d : (size_t)d;
        return (B == 1 || sb == (size_t)S * H * d) && (S == 1 || ss == ws) && (H == 1 || sh == wh);
    };
    if (q_out == q && !dense(Hq, q_stride_b, q_stride_s, q_stride_h)) return ATTN_ERR_INVALID_ARG;
    if (k && k_out == k && !dense(Hkv, k_stride_b, k_stride_s, k_stride_h)) return ATTN_ERR_INVALID_ARG;
    if (!attn::norm_rope_fits(p)) return ATTN_ERR_INVALID_ARG;
    p.q_stride[0] = (int64_t)q_stride_b;
    p.q_stride[1] = (int64_t)q_stride_s;
    p.q_stride[2] = (int64_t)q_stride_h;
    p.k_stride[0] = (int64_t)k_stride_b;
    p.k_stride[1] = (int64_t)k_stride_s;
    p.k_stride[2] = (int64_t)k_stride_h;
    int sms;
    uint64_t budget;
    if ((st = attn::device_state(&sms, &p.r.status, &budget)) != ATTN_OK) return st;
    return attn::launch_norm_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_append_paged(const void *q, const void *k, const void *v, void *q_out, void *k_pages,
                                void *v_pages, const int32_t *block_table, const int32_t *seqlens_k,
                                const int32_t *cu_seqlens, const void *q_weight, const void *k_weight, float eps,
                                const int32_t *positions, int n_axes, const attn_rope_pair_t *rope, int rotary_dim,
                                int interleaved, int B, int total, int Hq, int Hkv, int d, int page_size,
                                int num_pages, int max_blocks_per_seq, size_t q_stride, size_t k_stride,
                                size_t v_stride, void *stream) {
    if (!k_pages || !v_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16)) return ATTN_ERR_INVALID_ARG;
    return append_impl(q, k, v, q_out, k_pages, v_pages, nullptr, block_table, seqlens_k, cu_seqlens, q_weight,
                       k_weight, eps, positions, n_axes, rope, rotary_dim, interleaved, B, total, Hq, Hkv, d,
                       page_size, num_pages, max_blocks_per_seq, q_stride, k_stride, v_stride, stream);
}

attn_status_t attn_append_paged_q4(const void *q, const void *k, const void *v, void *q_out, void *cache,
                                   const int32_t *block_table, const int32_t *seqlens_k, const int32_t *cu_seqlens,
                                   const void *q_weight, const void *k_weight, float eps, const int32_t *positions,
                                   int n_axes, const attn_rope_pair_t *rope, int rotary_dim, int interleaved, int B,
                                   int total, int Hq, int Hkv, int d, int page_size, int num_pages,
                                   int max_blocks_per_seq, size_t q_stride, size_t k_stride, size_t v_stride,
                                   void *stream) {
    if (!cache || !aligned(cache, 16)) return ATTN_ERR_INVALID_ARG;
    return append_impl(q, k, v, q_out, nullptr, nullptr, cache, block_table, seqlens_k, cu_seqlens, q_weight,
                       k_weight, eps, positions, n_axes, rope, rotary_dim, interleaved, B, total, Hq, Hkv, d,
                       page_size, num_pages, max_blocks_per_seq, q_stride, k_stride, v_stride, stream);
}

attn_status_t attn_gather_paged_q4(const void *cache, const int32_t *block_table, const int32_t *seqlens,
                                   const int32_t *cu_seqlens_k, void *k_out, void *v_out, int B, int Hkv, int total_k,
                                   int d, int page_size, int num_pages, int max_blocks_per_seq, void *stream) {
    if (!cache || !k_out || !v_out || !aligned(cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return ATTN_ERR_INVALID_ARG;
    if (!cu_seqlens_k || !aligned(cu_seqlens_k, 4) || total_k < 1) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_table(block_table, seqlens, B, Hkv, d, page_size, num_pages, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    if (((int64_t)total_k / 16 + B) * Hkv > 0x7fffffff) return ATTN_ERR_INVALID_ARG;
    attn::GatherQ4Params p = {cache, block_table, seqlens, cu_seqlens_k, nullptr, k_out, v_out,
                              B, Hkv, total_k, num_pages, max_blocks_per_seq, nullptr};
    int sms;
    uint64_t budget;
    if ((st = attn::device_state(&sms, &p.status, &budget)) != ATTN_OK) return st;
    return attn::launch_gather_q4(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_decode_q4_workspace_bytes(int B, int Hq, int Hkv, int d, int max_blocks_per_seq) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d != 128 || max_blocks_per_seq < 1) return 0;
    if ((int64_t)B * ((max_blocks_per_seq + (int64_t)1) / 2) > 0x7fffffff) return 0;
    // o_part [rows][d] fp32, lse_part [rows] fp32, cuts [CTAs][2] of 16 bytes, each 256-B aligned.
    size_t ctas = 0;
    const size_t rows = attn::decode_q4_partial_rows(B, Hq, Hkv, max_blocks_per_seq, &ctas);
    return align256(rows * d * 4) + align256(rows * 4) + align256(ctas * 32);
}

attn_status_t attn_decode_paged_q4(const void *q, const void *cache, const int32_t *block_table,
                                   const int32_t *seqlens, void *out, float *lse, int B, int Hq, int Hkv, int d,
                                   int page_size, int num_pages, int max_blocks_per_seq, float scale,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    attn_status_t st = attn::check_decode_args(q, cache, cache, block_table, seqlens, out, lse, B, Hq, Hkv, d,
                                               page_size, num_pages, max_blocks_per_seq, scale);
    if (st != ATTN_OK) return st;
    // The kernel's factor scale * log2 e * 2^33 (queries below 2^27) has to stay finite.
    if (!(scale < 0x1p94f)) return ATTN_ERR_INVALID_ARG;
    // Key positions, rows and the sum of all sequences' page pairs are 32-bit.
    if ((int64_t)max_blocks_per_seq * 16 > 0x7fffffff - 64 || (int64_t)B * Hq > 0x7fffffff ||
        (int64_t)B * (((int64_t)max_blocks_per_seq + 1) / 2) > 0x7fffffff)
        return ATTN_ERR_INVALID_ARG;
    const size_t need = attn_decode_q4_workspace_bytes(B, Hq, Hkv, d, max_blocks_per_seq);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    attn::DecodeQ4Params p = {};
    p.q = q;
    p.cache = cache;
    p.block_table = block_table;
    p.seqlens = seqlens;
    p.out = out;
    p.lse = lse;
    size_t ctas = 0;
    const size_t rows = attn::decode_q4_partial_rows(B, Hq, Hkv, max_blocks_per_seq, &ctas);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.o_part = reinterpret_cast<float *>(ws);
    p.lse_part = reinterpret_cast<float *>(ws + align256(rows * d * 4));
    p.cuts = reinterpret_cast<int4 *>(ws + align256(rows * d * 4) + align256(rows * 4));
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.num_pages = num_pages;
    p.max_blocks = max_blocks_per_seq;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    int sms;
    if ((st = attn::device_state(&sms, &p.status, &p.budget_ns)) != ATTN_OK) return st;
    p.inject = attn::take_inject(2);
    return attn::launch_decode_q4(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_fwd_paged_q4_workspace_bytes(int B, int Hkv, int d, int max_total_k) {
    if (B < 1 || Hkv < 1 || d != 128 || max_total_k < 1) return 0;
    // offsets [B + 1] int32, then k and v [max_total_k][Hkv][d] bf16.
    return align256(((size_t)B + 1) * 4) + 2 * align256((size_t)max_total_k * Hkv * d * 2);
}

attn_status_t attn_fwd_paged_q4(const void *q, const void *cache, const int32_t *block_table,
                                const int32_t *seqlens_k, const int32_t *cu_seqlens_q, void *out, float *lse, int B,
                                int Hq, int Hkv, int total_q, int max_seqlen_q, int d, int page_size, int num_pages,
                                int max_blocks_per_seq, int max_total_k, int causal, float scale, int round_mode,
                                void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !cache || !out || !aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) ||
        (lse && !aligned(lse, 4)) || !cu_seqlens_q || !aligned(cu_seqlens_q, 4))
        return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_table(block_table, seqlens_k, B, Hkv, d, page_size, num_pages, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    if (Hq < 1 || Hq % Hkv != 0 || total_q < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q || max_total_k < 1)
        return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || scale < 0.f) return ATTN_ERR_INVALID_ARG;
    if (round_mode != ATTN_ROUND_RTNE && round_mode != ATTN_ROUND_RTNA && round_mode != ATTN_ROUND_RTZ)
        return ATTN_ERR_INVALID_ARG;
    if ((int64_t)total_q * Hq > (int64_t)1 << 31 || (int64_t)max_total_k * Hkv > (int64_t)1 << 31 ||
        ((int64_t)max_total_k / 16 + B) * Hkv > 0x7fffffff ||
        (int64_t)B * Hq * (((int64_t)max_seqlen_q + 127) / 128) > 0x7fffffff)
        return ATTN_ERR_INVALID_ARG;
    const size_t need = attn_fwd_paged_q4_workspace_bytes(B, Hkv, d, max_total_k);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    int sms;
    unsigned *status;
    uint64_t budget;
    if ((st = attn::device_state(&sms, &status, &budget)) != ATTN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *cu_k = reinterpret_cast<int32_t *>(ws);
    uint8_t *k = ws + align256(((size_t)B + 1) * 4);
    uint8_t *v = k + align256((size_t)max_total_k * Hkv * d * 2);
    const attn::GatherQ4Params g = {cache, block_table, seqlens_k, nullptr, cu_k, k, v,
                                    B, Hkv, max_total_k, num_pages, max_blocks_per_seq, status};
    if (attn::launch_gather_q4(g, s) != cudaSuccess) return ATTN_ERR_CUDA;
    const int64_t longest = (int64_t)max_blocks_per_seq * 16;
    return attn_fwd_varlen(q, k, v, out, lse, cu_seqlens_q, cu_k, B, Hq, Hkv, total_q, max_total_k, max_seqlen_q,
                           longest < max_total_k ? (int)longest : max_total_k, d, causal, scale, round_mode, stream);
}

}  // extern "C"
