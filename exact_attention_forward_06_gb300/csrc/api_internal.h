// api_internal.h -- host-side helpers shared between the C-ABI translation
// units (not part of the public interface).
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "attn.h"

namespace attn {

// Checks every argument of a paged decode step except its workspace: null or
// misaligned pointers, shapes, Hq % Hkv, scale (ATTN_ERR_INVALID_ARG) and
// d / page_size (ATTN_ERR_UNSUPPORTED).  Touches no device state.
attn_status_t check_decode_args(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                                const int32_t *seqlens, const void *out, const float *lse, int B, int Hq, int Hkv,
                                int d, int page_size, int num_pages, int max_blocks_per_seq, float scale);

// The current device's status word and SM count, and the wait budget: the
// device is looked up once and must be one that the kernels are built for.
attn_status_t device_state(int *sm_count, unsigned **status, uint64_t *budget_ns);

// A range of memory that a call reads or writes (bytes 0: none).
struct MemRange {
    const void *at;
    size_t bytes;
};

// Whether a written range has a byte in common with another written one or with a read one.
inline bool writes_overlap(std::initializer_list<MemRange> written, std::initializer_list<MemRange> read) {
    const auto meet = [](const MemRange &a, const MemRange &b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
        return a.bytes != 0 && b.bytes != 0 && x < y + b.bytes && y < x + a.bytes;
    };
    for (const MemRange *w = written.begin(); w != written.end(); ++w) {
        for (const MemRange *o = w + 1; o != written.end(); ++o)
            if (meet(*w, *o)) return true;
        for (const MemRange &r : read)
            if (meet(*w, r)) return true;
    }
    return false;
}

// Whether attn_debug_inject has asked for this mode; the request is then cleared.
int take_inject(int mode);

}  // namespace attn
