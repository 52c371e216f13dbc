// decode_q4.cu -- attention of single tokens over the 4-bit cache
// (attn_decode_paged_q4): a key split and its log-sum-exp merge.
//
// A page of one KV head is one 2560-byte block, read once: 4096 codes and 256
// parameters for 4 flops a code and query head.  At the measured copy bandwidth
// its bytes take about 110 SM clocks, in which the SM's four schedulers issue at
// most 440 instructions, half of that to the integer pipe, so the arithmetic decides
// the form as much as the bytes do:
//
// - Codes go to the tensor cores without being turned into cache values.  A bf16
//   whose bits are those of a code n in its own place (bits 0..3 or 4..7) and zero
//   elsewhere is the number n 2^-133 or n 2^-129, subnormal or just above: a mask
//   makes the operand of two codes, a shift brings the other half of the word.  The
//   queries carry the powers of two, 2^k and 2^(k-4), k at most 100.
// - S^T = K Q^T (mma m16n8k16, the page's 16 tokens as rows, eight query heads of
//   the KV head as columns), a product for each group of 32 channels:
//       s_t += scale_tg * (sum_c q_c n_tc - 7.5 Q_g) + center_tg * Q_g,
//   with Q_g the sum of the group's q.  Both terms with Q_g are two more products
//   for all groups at once, Q_g and -7.5 Q_g cut into three bf16 parts (24 bits).
// - O^T += V^T P^T: value codes are f16 in their own places too, and become n - 7.5
//   (times 2^-9) by one packed multiply-add; a group's scale goes to the probability,
//   P'_t = P_t scale_tg; the centers' term is one product with the unscaled P.  (Masked
//   codes as they are, with 7.5 sum P' from four more products, took 152 us
//   where this takes 149: a product is dearer than eight packed multiply-adds.)
// - The byte order of the block (q4.cuh) is that of the fragments: every lane
//   reads its operands as 16-byte words without bank conflicts, and a value
//   pair of two tokens is one byte permutation.
// - Two pages a step share the wait, the vote on the running max and the loop.
//
// The work is cut into shares, one for each CTA that the GPU holds at once.  Where the
// batch is large the shares are equal: the page pairs of all sequences and KV heads in
// one row, CTA c taking the c-th part of it, a few segments (a run of one sequence's pages
// for one KV head).  Where it is small a share is one segment.  A segment that is a whole
// sequence is finished by its CTA, the parts of a cut one go to the workspace and are
// merged by log-sum-exp in the order of the keys.  Ragged lengths thus cost nothing: with
// a grid of fixed splits over the table's width an earlier page loop took 177 us instead
// of 168.
//
// In a segment each warp streams page pairs w, w + 4, .. through a ring of its own
// (bulk copies issued by one of its lanes as soon as a slot has been read): no producer
// warp and no barrier between warps until the four partial results meet at the
// segment's end.  Scores, sums and outputs are fp32.  P' is rounded to f16 (2^-11 of
// itself at most), P to bf16 for the centers; the row sum adds the fp32 values.
// With P' in bf16, as the bf16 decode's P, the output's error against 64 bits was
// 2.4e-3 (its own rounding alone makes 1.7e-3) instead of 1.8e-3, in 0.97 of the time.
//
// Measured on 64 sequences of 0 to 16384 tokens, 64 / 8 heads (758 MB): 146.4 us,
// 5.2 TB/s, 0.76 of the copy bandwidth; the copies alone take 120 us, the arithmetic
// alone 139.  On 32 sequences of 1024 to 8192 tokens, 32 / 8 heads (177 MB): 45.1 us,
// 0.58.  There the starts and ends of segments cost: a share's 76 pairs lie in two
// segments or three.  As many pairs with one run to a share (57 sequences of 2424) take
// 37.0 us on the GPU against 44.1, as long with 8 heads to a KV head as with 4; 2 us are
// the merge.  3 sequences of about 100 thousand tokens, 32 / 1 heads (55 MB): 38.7 us,
// the unpacking of two tiles' pages twice (with one tile a CTA, four times: 5 us more).
// With codes as 16 + n and n - 7.5, each by a shift and an and/or (and an addition),
// these took 167, 50 and 49 us.
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_ops.h"
#include "common.cuh"
#include "q4.cuh"

namespace attn {
namespace dq4 {

using q4::BLOCK;
using q4::D;
using q4::PAGE;

constexpr int NW = 4;  // warps = page streams, and groups of a head
constexpr int NT = NW * 32;
constexpr int STAGE = 2 * BLOCK;

// A CTA works for 8 * TILES query heads of a KV head, an MMA column each.  With more
// heads to a KV head than eight, two tiles share the unpacking of a page, which is
// two thirds of its instructions, at the price of registers: two CTAs an SM.
template <int TILES>
struct Shape {
    static constexpr int COLS = 8 * TILES;
    static constexpr int CTAS_PER_SM = TILES == 1 ? 3 : 2;
    static constexpr int MAX_CTAS = CTAS_PER_SM * 152;   // shares at most: the workspace's size goes by it
    static constexpr int NST = TILES == 1 ? 3 : 4;       // page pairs in flight per warp
    static constexpr int RING = NW * NST * STAGE;
    static constexpr int EXCHANGE = 36 * TILES * 32 * 4;  // one warp's partial result: 36 words a lane and tile
    static constexpr int Q_FRAGS = 4 * TILES * 32 * 16;   // a lane's query fragments, 16 bytes a group and tile
    static constexpr int BARRIERS = RING + 2 * EXCHANGE + Q_FRAGS;
    static constexpr int WORDS = BARRIERS + NW * NST * 8;
    static constexpr int SMEM = WORDS + 128;
    static_assert(CTAS_PER_SM * (SMEM + 1024) <= 233472, "CTAs per SM");
};
constexpr int MIN_PAIRS = 4;           // pairs a CTA takes at least, unless there is a KV head for each
constexpr int WHOLE_PAIRS = 16;        // a run of a table that holds no more is never cut
constexpr int SLACK_BITS = 8;          // a score this far (in log2) above the largest so far raises the reference
constexpr float SLACK = SLACK_BITS;
constexpr int ROOM = 8;  // bits of P given up for scales that grow, before their pages are checked one by one
constexpr float LN2 = 0.6931471805599453f;

// Codes J and J + 4 of a word as a bf16 pair: n 2^-133 (even J) or n 2^-129 (odd J).
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    return (J < 2 ? w : w >> 8) & (J & 1 ? 0x00f000f0u : 0x000f000fu);
}

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// The scale of group g in a token's four.
__device__ __forceinline__ float group_f(uint2 s, int g) {
    const uint32_t u = g < 2 ? s.x : s.y;
    return g & 1 ? hi_f(u) : lo_f(u);
}

// d = a b + c (mma m16n8k16, bf16 in, fp32 out), and the transpose of an 8x8
// matrix: plain functions of their operands, so that the compiler may interleave
// the two pages' chains.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{0f00000000, 0f00000000, 0f00000000, 0f00000000};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A pair's values (n - 7.5) 2^-9 as f16, exactly.  A code in bits 0..3 of an f16
// whose other bits are zero is the (subnormal) number n 2^-24, one in bits 4..7
// n 2^-20: for two of a half-word's four codes no shift, one multiply-add.
template <int J>
__device__ __forceinline__ uint32_t value_pair(uint32_t w) {
    uint32_t d;
    const uint32_t t = (J < 2 ? w : w >> 8) & (J & 1 ? 0x00f000f0u : 0x000f000fu);
    asm("fma.rn.f16x2 %0, %1, %2, %3;"
        : "=r"(d)
        : "r"(t), "r"(J & 1 ? 0x68006800u : 0x78007800u), "r"(0xa380a380u));  // 2^11 or 2^15, -7.5 * 2^-9
    return d;
}
constexpr float VALUE_STEPS = 512.f;  // 2^9

// mma with f16 operands.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Products of two bf16 pairs (exact by a power of two).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// One page's words in registers, as the lane's fragments take them.
struct KeyWords {
    uint4 ka, kb;    // codes of tokens r4 and r4 + 8, channels 32 g + 8 c4 ..
    uint2 ksa, ksb;  // scales of tokens r4 and r4 + 8, all groups
    uint2 kza, kzb;  // centers
};
struct ValueWords {
    uint4 va, vb;       // codes of tokens 2 c4, 2 c4 + 1 and those + 8
    uint2 vsa, vsb;     // scales of tokens r4 and r4 + 8, all groups
    uint32_t vza, vzb;  // centers of group r4 % 4, tokens 2 c4, 2 c4 + 1 and those + 8
};

__device__ __forceinline__ void load_keys(KeyWords &w, const uint8_t *blk, int r4, int c4) {
    w.ka = *reinterpret_cast<const uint4 *>(blk + r4 * 64 + c4 * 16);
    w.kb = *reinterpret_cast<const uint4 *>(blk + r4 * 64 + c4 * 16 + 512);
    const uint8_t *par = blk + r4 * 8;
    w.ksa = *reinterpret_cast<const uint2 *>(par + q4::K_SCALES);
    w.ksb = *reinterpret_cast<const uint2 *>(par + q4::K_SCALES + 64);
    w.kza = *reinterpret_cast<const uint2 *>(par + q4::K_CENTERS);
    w.kzb = *reinterpret_cast<const uint2 *>(par + q4::K_CENTERS + 64);
}

__device__ __forceinline__ void load_values(ValueWords &w, const uint8_t *blk, int r4, int c4) {
    const uint8_t *v = blk + r4 * 128 + c4 * 32;
    w.va = *reinterpret_cast<const uint4 *>(v + q4::V_CODES + ((r4 & 1) << 4));
    w.vb = *reinterpret_cast<const uint4 *>(v + q4::V_CODES + (((r4 & 1) ^ 1) << 4));
    w.vsa = *reinterpret_cast<const uint2 *>(blk + q4::V_SCALES + r4 * 8);
    w.vsb = *reinterpret_cast<const uint2 *>(blk + q4::V_SCALES + r4 * 8 + 64);
    const uint8_t *z = blk + q4::V_CENTERS + (r4 & 3) * 32 + c4 * 4;
    w.vza = *reinterpret_cast<const uint32_t *>(z);
    w.vzb = *reinterpret_cast<const uint32_t *>(z + 16);
}

// Page pairs of a sequence; 0 for a length outside the table.
__device__ __forceinline__ int pairs_of(int L, int max_blocks) {
    return L < 0 || L > max_blocks * PAGE ? 0 : (L + 2 * PAGE - 1) / (2 * PAGE);
}

// Whether the table's width alone says that no run is cut: then there is no merge to
// launch, which takes 2 to 3 us, as long as a CTA needs for the pairs that it saves.
// (8 sequences of 500 tokens, 64 / 8 heads: 8.9 us against 10.6 with runs in parts.)
__host__ __device__ __forceinline__ bool never_cut(int B, int Hkv, int max_blocks, int shares) {
    return (int64_t)B * Hkv <= shares && max_blocks <= 2 * WHOLE_PAIRS;
}

template <int TILES>
__global__ void __launch_bounds__(NT, Shape<TILES>::CTAS_PER_SM)
    share_kernel(const DecodeQ4Params p, int col_blocks) {
    using S = Shape<TILES>;
    constexpr int NST = S::NST, COLS = S::COLS;
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::wait_for_prior_work();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r4 = lane >> 2, c4 = lane & 3;
    uint8_t *ring = smem + warp * NST * STAGE;
    float *exchange = reinterpret_cast<float *>(smem + S::RING) + lane;                   // [half][word][lane]
    uint4 *q_frag = reinterpret_cast<uint4 *>(smem + S::RING + 2 * S::EXCHANGE) + lane;  // [(4 tile + g) * 32]
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::BARRIERS) + warp * NST;
    int *words = reinterpret_cast<int *>(smem + S::WORDS);
    volatile int *abort_flag = words;
    // words[1]: the share's first sequence; [2], [3]: which part of how many its run is of its
    // sequence (whole runs; else 0 and 0).  found: [0] total, [1] pairs before that
    // sequence, [2] shares, [3], [4] the share's first unit and the one behind its last.
    // words[14]: that sequence's length.
    int64_t *found = reinterpret_cast<int64_t *>(words + 4);
    int *scan = words + 16;  // [4][NW]

    // CTAs of one share that differ in the column block alone are neighbours, so
    // that their reads of the same pages meet in L2.
    const int blk = blockIdx.x % col_blocks, share = blockIdx.x / col_blocks;
    const int G = p.Hq / p.Hkv, col0 = blk * COLS;
    const int cols = min(COLS, G - col0);

    // All pairs, the sequences with any and the longest: a thread sums a run of
    // sequences, the sums are scanned; up to 32 sequences, each warp does all of it, a
    // lane a sequence, and waits for no other.
    const bool few = p.B <= 32;
    const int per = few ? 1 : (p.B + NT - 1) / NT;
    const int b_lo = min(p.B, (few ? lane : (int)threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
    int mine = 0, some = 0, longest = 0;  // pairs: at most 2^31, B * max_blocks / 2 is bounded by the caller
    int len = 0;                          // (few: of the lane's sequence)
    for (int b = b_lo; b < b_hi; ++b) {
        len = p.seqlens[b];
        const int np = pairs_of(len, p.max_blocks);
        mine += np;
        some += np > 0;
        longest = max(longest, np);
    }
    // The length of a sequence of this thread's run, read again only where there are several.
    const auto own_length = [&](int b) { return few ? len : p.seqlens[b]; };
    const auto inclusive = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += w;
        }
        return v;
    };
    const int incl = inclusive(mine);
    some = __reduce_add_sync(0xffffffffu, some);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
        for (int s = 0; s < NST; ++s) ptx::mbar_init(full + s, 1);
        if (warp == 0) *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    int64_t before = incl - mine, all = __shfl_sync(0xffffffffu, incl, 31);  // (before: of this thread's run)
    if (!few) {
        if (lane == 31) {
            scan[warp] = incl;
            scan[NW + warp] = some;
            scan[2 * NW + warp] = longest;
        }
        __syncthreads();
        all = some = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
            some += scan[NW + w];
            longest = max(longest, scan[2 * NW + w]);
        }
    }
    const int64_t total = all * p.Hkv, items = (int64_t)some * p.Hkv;
    const int ctas = gridDim.x / col_blocks;
    // Whole runs (a sequence and KV head), each cut into parts of at most `part` pairs, a CTA
    // a part, where the CTAs suffice for that and the longest part is not much longer than
    // an equal share: a share that takes parts of several runs pays for each the latency
    // of about 16 pairs.  Else equal shares, no more than there is work for and none
    // without a pair.  (16 sequences of 10 to 500 tokens, 32 / 8 heads: 9.8 us against 19 in
    // equal shares; 3 of about 100 thousand, 32 / 1 heads: 37.7 against 40.9.)
    uint32_t part = 0;
    if (items <= ctas && (longest <= MIN_PAIRS || never_cut(p.B, p.Hkv, p.max_blocks, ctas))) {
        part = max(1, longest);
    } else if (items <= ctas && total < 0x7fffffff) {
        const uint32_t units = (uint32_t)total, spare = (uint32_t)(ctas - (int)items);
        part = spare ? max((uint32_t)MIN_PAIRS, (units + spare - 1) / spare) : (uint32_t)longest;
        part = max(1u, min((uint32_t)longest, (part + NW - 1) / NW * NW));
        if (part > units / (uint32_t)ctas + 16) part = 0;
    }
    if (part) {
        const auto pieces_of = [&](int np) {
            return (uint32_t)np <= part ? (int)(np > 0) : (int)(((uint32_t)np + part - 1) / part);
        };
        int pieces = 0;
        for (int b = b_lo; b < b_hi; ++b) pieces += pieces_of(pairs_of(own_length(b), p.max_blocks));
        const int upto = inclusive(pieces);
        if (threadIdx.x == 0) found[3] = found[4] = 0;
        int behind = upto - pieces;  // (at most as many as there are CTAs)
        if (few) {
            __syncwarp();
        } else {
            if (lane == 31) scan[3 * NW + warp] = upto;
            __syncthreads();
            for (int w = 0; w < warp; ++w) behind += scan[3 * NW + w];
        }
        if ((!few || warp == 0) && share >= behind * p.Hkv && share < (behind + pieces) * p.Hkv) {
            int b = b_lo, L, np, n;
            for (;; ++b) {
                L = own_length(b);
                np = pairs_of(L, p.max_blocks);
                n = pieces_of(np);
                if (share < (behind + n) * p.Hkv) break;
                behind += n;
                before += np;
            }
            const uint32_t at = (uint32_t)(share - behind * p.Hkv);
            uint32_t head = at, piece = 0, each = np, more = 0;  // (the first `more` pieces have one more than `each`)
            if (n > 1) {
                head = at / (uint32_t)n;
                piece = at - head * n;
                each = (uint32_t)np / (uint32_t)n;
                more = np - each * n;
            }
            const int64_t run = before * p.Hkv + (int64_t)head * np + piece * each + min(piece, more);
            words[1] = b;
            words[14] = L;
            words[2] = (int)piece;
            words[3] = n;
            found[1] = before;
            found[3] = run;
            found[4] = run + each + (piece < more);
        }
    } else {
        const int64_t fill = (total + MIN_PAIRS - 1) / MIN_PAIRS;
        const int64_t shares = min(min((int64_t)ctas, total), max((int64_t)p.B * p.Hkv, fill));
        const int64_t lo = share < shares ? total * share / shares : total;
        if (threadIdx.x == 0) {
            words[3] = 0;
            found[0] = total;
            found[2] = shares;
            found[3] = lo;
            found[4] = share < shares ? total * (share + 1) / shares : total;
        }
        if ((!few || warp == 0) && share < shares && lo >= before * p.Hkv && lo < (before + mine) * p.Hkv) {
            int b = b_lo, L;
            for (;; ++b) {
                L = own_length(b);
                const int np = pairs_of(L, p.max_blocks);
                if (lo < (before + np) * p.Hkv) break;
                before += np;
            }
            words[1] = b;
            words[14] = L;
            found[1] = before;
        }
    }
    // Empty sequences (and lengths outside the table, which are reported) belong
    // to no share: their rows are written here.
    if (blk == 0) {
        for (int b = share; b < p.B; b += gridDim.x / col_blocks) {
            const int L = few ? __shfl_sync(0xffffffffu, len, b) : p.seqlens[b];
            if (pairs_of(L, p.max_blocks) > 0) continue;
            if (L != 0 && threadIdx.x == 0) report_status(p.status, kStatusDeviceBounds, kSiteQ4Seqlen);
            for (int i = threadIdx.x; i < p.Hq * (D / 8); i += NT)
                reinterpret_cast<uint4 *>(p.out)[(int64_t)b * p.Hq * (D / 8) + i] = make_uint4(0, 0, 0, 0);
            if (p.lse)
                for (int i = threadIdx.x; i < p.Hq; i += NT) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
        }
    }
    __syncthreads();
    const int64_t u0 = found[3], u1 = found[4];
    // For the merge: the cut run that the share goes on with, and the one it begins, as
    // first row, query heads, number of shares (0: none) and which of them this one is.
    if (threadIdx.x < 2) p.cuts[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
    const WaitCtx wc{abort_flag, p.status, p.budget_ns};
    const uint64_t pol = col_blocks == 1 ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    const int64_t page_step = (int64_t)p.Hkv * BLOCK;
    // The byte selector that doubles group c4's entry of four bf16.
    const uint32_t own = 0x1010u + 0x2222u * c4;
    int slot = 0;
    uint32_t parity = 0;

    int b = 0, h = 0, L = 0, seq_pairs = 0, first = 0;  // the segment: sequence, KV head, first pair
    if (u0 < u1) {
        b = words[1];
        L = words[14];
        seq_pairs = pairs_of(L, p.max_blocks);
        const int64_t rem = u0 - found[1] * p.Hkv;
        h = (int)(rem / seq_pairs);
        first = (int)(rem - (int64_t)h * seq_pairs);
    }
    for (int64_t u = u0; u < u1;) {
        const int count = (int)min((int64_t)(seq_pairs - first), u1 - u);  // this segment's pairs
        const int64_t row0 = (int64_t)b * p.Hq + h * G + col0;
        if (count < seq_pairs) {
            // The run lies in the shares of its first and last pairs and all between.
            if (threadIdx.x == (first == 0)) {
                int parts = words[3], index = words[2];
                if (parts == 0) {
                    const int64_t all_units = found[0], n_shares = found[2], unit = u - first;
                    const int begin = (int)(((unit + 1) * n_shares + all_units - 1) / all_units - 1);
                    parts = (int)(((unit + seq_pairs) * n_shares + all_units - 1) / all_units - 1) - begin + 1;
                    index = (int)(blockIdx.x / col_blocks) - begin;
                }
                p.cuts[2 * blockIdx.x + (first == 0)] = make_int4((int)row0, cols, parts, index);
            }
        }
        const uint8_t *cache = static_cast<const uint8_t *>(p.cache) + (int64_t)h * BLOCK;
        const int32_t *table = p.block_table + (int64_t)b * p.max_blocks;
        const int last_page = (L + PAGE - 1) / PAGE;
        const int n = warp < count ? (count - warp + NW - 1) / NW : 0;  // this warp's: first + warp + NW i

        // A batch of up to 32 pairs: lane j holds pair base + j's pages (-1: none,
        // or a bad entry) and their numbers of keys.
        int tab0, tab1, nv0, nv1;
        unsigned whole;
        auto load_table = [&](int base) {
            tab0 = tab1 = -1;
            nv0 = nv1 = 0;
            if (base + lane < n) {
                const int page = 2 * (first + warp + NW * (base + lane));
                tab0 = table[page];
                const bool two = page + 1 < last_page;
                if (two) tab1 = table[page + 1];
                const bool bad0 = tab0 < 0 || tab0 >= p.num_pages;
                const bool bad1 = two && (tab1 < 0 || tab1 >= p.num_pages);
                if (bad0 || bad1) report_status(p.status, kStatusDeviceBounds, kSiteQ4Table);
                if (bad0) tab0 = -1;
                if (bad1) tab1 = -1;
                const int left = L - page * PAGE;
                nv0 = bad0 ? 0 : min(PAGE, left);
                nv1 = tab1 < 0 ? 0 : min(PAGE, left - PAGE);
            }
            whole = __ballot_sync(0xffffffffu, nv0 == PAGE && nv1 == PAGE);
        };
        auto issue = [&](int i, int to) {  // pair i of the batch, by the lane that holds it
            if (lane == i && !(p.inject && warp < 2)) {  // (fault injection)
                uint8_t *dst = ring + to * STAGE;
                ptx::mbar_arrive_expect_tx(full + to, (tab0 >= 0 ? BLOCK : 0) + (tab1 >= 0 ? BLOCK : 0));
                if (tab0 >= 0) ptx::bulk_load(dst, cache + tab0 * page_step, BLOCK, full + to, pol);
                if (tab1 >= 0) ptx::bulk_load(dst + BLOCK, cache + tab1 * page_step, BLOCK, full + to, pol);
            }
        };
        auto issue_first = [&](int m) {  // the batch's first pairs, all slots being free
            int to = slot;
            for (int i = 0; i < min(m, NST); ++i) {
                issue(i, to);
                to = to + 1 == NST ? 0 : to + 1;
            }
        };
        // The queries' loads go out before the wait for the table's.
        uint4 q_words[TILES][4];
#pragma unroll
        for (int c = 0; c < TILES; ++c) {
            const uint4 *qrow =
                reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + (row0 + 8 * c + r4) * D);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                q_words[c][g] = 8 * c + r4 < cols ? qrow[4 * g + c4] : make_uint4(0, 0, 0, 0);
        }
        load_table(0);
        issue_first(min(n, 32));

        // Q^T as the B operand: head r4 (zero past the CTA's columns), the channels
        // 32 g + 8 c4 + (j, j + 4), j = 0..3, in the order of a key word's pairs.
        // qz, qo: B operands of the centers' and the scales' products, two each: at
        // k = 2 c4, 2 c4 + 1 (centers) and 2 c4 + 8, 2 c4 + 9 (scales) the first two
        // bf16 parts of group c4's Q_g and of -7.5 Q_g, then the third part.
        // The fragments are the same in every warp and stay in shared memory: one
        // 16-byte read a group and page is cheaper than 16 registers.
        // A head's all carry 2^k, k such that its largest q stays below 2^127: scores come
        // out times 2^(k - 133), which goes into the softmax's factor sl2.
        float sl2[TILES][2];
        uint32_t qz0[TILES], qz1[TILES], qo0[TILES], qo1[TILES];
#pragma unroll
        for (int c = 0; c < TILES; ++c) {
            const uint4(&v)[4] = q_words[c];
            uint32_t largest = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                constexpr uint32_t SIZE = 0x7fff7fffu;
                largest = __vmaxu2(largest, __vmaxu2(__vmaxu2(v[g].x & SIZE, v[g].y & SIZE),
                                                     __vmaxu2(v[g].z & SIZE, v[g].w & SIZE)));
            }
            largest = max(largest & 0xffffu, largest >> 16);
            largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
            largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
            const int k = max(7, min(100, 253 - (int)(largest >> 7)));
#pragma unroll
            for (int j = 0; j < 2; ++j)
                sl2[c][j] = p.scale_log2 * __uint_as_float((uint32_t)(260 - __shfl_sync(0xffffffffu, k, 4 * (2 * c4 + j)))
                                                           << 23);  // 2^(133 - k)
            const uint32_t even = (uint32_t)(k + 127) * 0x800080u, odd = (uint32_t)(k + 123) * 0x800080u;
            float x = 0.f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (warp == g)
                    q_frag[(4 * c + g) * 32] = make_uint4(mul_bf16x2(__byte_perm(v[g].x, v[g].z, 0x5410), even),
                                                          mul_bf16x2(__byte_perm(v[g].x, v[g].z, 0x7632), odd),
                                                          mul_bf16x2(__byte_perm(v[g].y, v[g].w, 0x5410), even),
                                                          mul_bf16x2(__byte_perm(v[g].y, v[g].w, 0x7632), odd));
                float s = ((lo_f(v[g].x) + hi_f(v[g].x)) + (lo_f(v[g].y) + hi_f(v[g].y))) +
                          ((lo_f(v[g].z) + hi_f(v[g].z)) + (lo_f(v[g].w) + hi_f(v[g].w)));
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                if (g == c4) x = s;
            }
            auto parts = [](float v, uint32_t &b0, uint32_t &b1) {
                const uint32_t h0 = ptx::pack_bf16x2(v, 0.f) & 0xffffu;
                const float v1 = v - lo_f(h0);
                const uint32_t h1 = ptx::pack_bf16x2(v1, 0.f) & 0xffffu;
                b0 = h0 | h1 << 16;
                b1 = ptx::pack_bf16x2(v1 - lo_f(h1), 0.f) & 0xffffu;
            };
            x *= __uint_as_float((uint32_t)(k - 6) << 23);  // 2^(k - 133)
            parts(x, qz0[c], qz1[c]);
            parts(-7.5f * x, qo0[c], qo1[c]);
        }
        __syncthreads();
        // Of each tile: running reference (log2 units, see below) and row sum of heads 2 c4, 2 c4 + 1;
        // acc[2 g + i]: channels 32 g + 4 r4 + 2 i (+ 1) times those heads; cen: the
        // centers' term of group r4 % 4.
        float m[TILES][2], lsum[TILES][2], acc[TILES][8][4], cen[TILES][4];
#pragma unroll
        for (int c = 0; c < TILES; ++c) {
            m[c][0] = m[c][1] = -INFINITY;
            lsum[c][0] = lsum[c][1] = 0.f;
            cen[c][0] = cen[c][1] = cen[c][2] = cen[c][3] = 0.f;
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[c][t][0] = acc[c][t][1] = acc[c][t][2] = acc[c][t][3] = 0.f;
        }

        // The values' range (see below): the common factor of their scales, a power of two
        // as a bf16 pair, the size (bf16 bits) from which a scale is too large (at first:
        // any), and how far above the running reference m a score may lie.
        constexpr uint32_t ONE = 0x3f803f80u;
        uint32_t vf = ONE, vf_limit = 1;
        float reach = SLACK;
        int room = 0;  // bits by which `reach` may still shrink
        int base = 0, left = n;
        while (left > 0) {
            const int batch = min(left, 32);
            int i = 0;
            for (; i < batch; ++i) {
                if (!warp_wait_bounded(full + slot, parity, wc, kSiteQ4Page)) break;
                const uint8_t *blk = ring + slot * STAGE;
                float s[2][TILES][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    KeyWords k;
                    load_keys(k, blk + u * BLOCK, r4, c4);
                    const uint32_t zs[4] = {
                        __byte_perm(k.kza.x, k.kza.y, own), __byte_perm(k.kzb.x, k.kzb.y, own),
                        __byte_perm(k.ksa.x, k.ksa.y, own), __byte_perm(k.ksb.x, k.ksb.y, own)};
#pragma unroll
                    for (int c = 0; c < TILES; ++c) {
                        mma_zero(s[u][c], zs, qz0[c], qo0[c]);
                        mma(s[u][c], zs, qz1[c], qo1[c]);
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t wa = g == 0 ? k.ka.x : g == 1 ? k.ka.y : g == 2 ? k.ka.z : k.ka.w;
                        const uint32_t wb = g == 0 ? k.kb.x : g == 1 ? k.kb.y : g == 2 ? k.kb.z : k.kb.w;
                        const uint32_t a0[4] = {code_pair<0>(wa), code_pair<0>(wb), code_pair<1>(wa), code_pair<1>(wb)};
                        const uint32_t a1[4] = {code_pair<2>(wa), code_pair<2>(wb), code_pair<3>(wa), code_pair<3>(wb)};
                        const float fa = group_f(k.ksa, g), fb = group_f(k.ksb, g);
#pragma unroll
                        for (int c = 0; c < TILES; ++c) {
                            const uint4 qb = q_frag[(4 * c + g) * 32];
                            float d[4];
                            mma_zero(d, a0, qb.x, qb.y);
                            mma(d, a1, qb.z, qb.w);
                            s[u][c][0] = fmaf(fa, d[0], s[u][c][0]);
                            s[u][c][1] = fmaf(fa, d[1], s[u][c][1]);
                            s[u][c][2] = fmaf(fb, d[2], s[u][c][2]);
                            s[u][c][3] = fmaf(fb, d[3], s[u][c][3]);
                        }
                    }
                }
                // s[u][c][0], [1]: token r4 of page u, heads 8 c + 2 c4, + 1; [2], [3]:
                // token r4 + 8.  x: over the reference m, in log2 units.
                float x[2][TILES][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < TILES; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[u][c][j] = fmaf(s[u][c][j], sl2[c][j & 1], -m[c][j & 1]);
                // The scales of one token's values for the check below: lane = page x token.
                const uint2 vs =
                    *reinterpret_cast<const uint2 *>(blk + (lane >> 4) * BLOCK + q4::V_SCALES + (lane & 15) * 8);
                uint32_t big = __vmaxu2(vs.x, vs.y);
                big = max(big & 0xffffu, big >> 16);
                const bool all = whole >> i & 1;
                if (!all) {
                    // Slots past the end hold arbitrary bits: their scores are replaced,
                    // and in shared memory the values' parameters.
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int nv = __shfl_sync(0xffffffffu, u ? nv1 : nv0, i);
#pragma unroll
                        for (int c = 0; c < TILES; ++c) {
                            if (r4 >= nv) x[u][c][0] = x[u][c][1] = -INFINITY;
                            if (r4 + 8 >= nv) x[u][c][2] = x[u][c][3] = -INFINITY;
                        }
                        if (u == lane >> 4 && (lane & 15) >= nv) {
                            big = 0;
                            uint8_t *mine = ring + slot * STAGE + u * BLOCK;
                            *reinterpret_cast<uint2 *>(mine + q4::V_SCALES + (lane & 15) * 8) = make_uint2(0, 0);
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                *reinterpret_cast<uint16_t *>(mine + q4::V_CENTERS + g * 32 + (lane & 15) * 2) = 0;
                        }
                    }
                    ptx::fence_proxy_async_smem();  // (the slot's next copy comes after these writes)
                    __syncwarp();
                }
                // Probability times scale goes to the product as f16 (11 bits: the values'
                // part of the output then loses nothing against its own rounding), so
                // it has to stay below 2^16 and, where it counts, above f16's last steps.
                // P is taken over a reference m of each head, below its largest score: what a
                // usual scale (2^e, found in the first pages) makes of the largest P then is
                // 2^5 or 2^6, and a token 2^19 times less likely still keeps 11 bits.  As
                // long as no score lies `reach` above m and no scale reaches vf_limit,
                // 2^15 over 2^reach, nothing can overflow and nothing is done.  Otherwise the
                // pages' products are bounded head by head, and m follows where it must: a
                // token that a head does not attend to takes no bits from it, whatever its
                // scale.  m follows a score SLACK bits late, so raises, with their shuffles
                // and rescaling, are rare instead of nearly every page.
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < TILES; ++c)
                        top = fmaxf(top, fmaxf(fmaxf(x[u][c][0], x[u][c][1]), fmaxf(x[u][c][2], x[u][c][3])));
                if (__any_sync(0xffffffffu, top > reach || big >= vf_limit)) {
                    uint32_t largest = 0;  // finite scale of this lane's token
                    if (big) {
                        const uint32_t h[4] = {vs.x & 0xffffu, vs.x >> 16, vs.y & 0xffffu, vs.y >> 16};
#pragma unroll
                        for (int g = 0; g < 4; ++g) largest = max(largest, h[g] < 0x7f80u ? h[g] : 0u);
                    }
                    const uint32_t most = __reduce_max_sync(0xffffffffu, largest);
                    const int e = (int)(most >> 7);  // exponent + 127
                    bool first_scales = false;
                    if (vf_limit == 1) {
                        first_scales = most != 0;
                        if (first_scales) {
                            // The tokens' mean exponent, or the largest where that is at most 3 more.
                            const unsigned some = __ballot_sync(0xffffffffu, largest != 0);
                            const int mean = (int)(__reduce_add_sync(0xffffffffu, largest >> 7) / __popc(some));
                            const int usual = min(e, mean + 3);
                            int factor = 127;  // of vf; 2^-10 .. 2^6 are taken as they are
                            if (usual >= 117 && usual < 134) {
                                reach = (float)(5 + SLACK_BITS + 127 - usual);
                                room = ROOM;
                            } else {
                                factor = max(1, min(259 - usual, 254));  // 2^(5 - exponent)
                            }
                            vf = (uint32_t)factor * 0x800080u;
                            vf_limit = (uint32_t)max(1, min(142 - (int)reach - (factor - 127), 255)) << 7;
                        }
                    } else if (most >= vf_limit) {
                        const int ev = (int)(vf >> 23) - 127;
                        if (e + ev >= 227) {
                            // 2^100 times too large: all start again from this scale.
                            const int factor = max(1, 259 - e);
                            const float ratio = __uint_as_float((uint32_t)factor << 23) / lo_f(vf);
                            vf = (uint32_t)factor * 0x800080u;
                            reach = SLACK;
                            room = 0;
                            vf_limit = (uint32_t)min(134 - (factor - 127), 255) << 7;
#pragma unroll
                            for (int c = 0; c < TILES; ++c)
#pragma unroll
                                for (int t = 0; t < 8; ++t)
#pragma unroll
                                    for (int j = 0; j < 4; ++j) acc[c][t][j] *= ratio;
                        } else {
                            // Larger than usual: the limit follows for a few bits.
                            const int up = min(e + 1 - (int)(vf_limit >> 7), room);
                            room -= up;
                            reach -= (float)up;
                            vf_limit += (uint32_t)up << 7;
                        }
                    }
                    const float lift = reach - SLACK;  // the largest score's distance from m
                    // A bound on log2 of the scales' size, of this lane's token; log2 vf.
                    const float size = largest ? (float)((int)(largest >> 7) - 126) : -INFINITY;
                    const float vf_log2 = (float)((int)(vf >> 23) - 127);
                    const float sizes[2][2] = {
                        {__shfl_sync(0xffffffffu, size, r4), __shfl_sync(0xffffffffu, size, r4 + 8)},
                        {__shfl_sync(0xffffffffu, size, r4 + 16), __shfl_sync(0xffffffffu, size, r4 + 24)}};
#pragma unroll
                    for (int c = 0; c < TILES; ++c) {
                        // The largest score, and the largest log2 of probability times scale.
                        float y[2] = {-INFINITY, -INFINITY}, z[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (x[u][c][j] != -INFINITY) {
                                    const float v = __fmul_rn(s[u][c][j], sl2[c][j & 1]);
                                    y[j & 1] = fmaxf(y[j & 1], v);
                                    z[j & 1] = fmaxf(z[j & 1], v + sizes[u][j >> 1]);
                                }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) {
                                y[j] = fmaxf(y[j], __shfl_xor_sync(0xffffffffu, y[j], o));
                                z[j] = fmaxf(z[j], __shfl_xor_sync(0xffffffffu, z[j], o));
                            }
                            z[j] += vf_log2;
                            // (with the first scales, m may go down: acc is still 0; products are
                            // rounded on their own here, or scores of 2^31, whose last step
                            // is above the exponential's range, would miss their own maximum)
                            float mx = first_scales ? m[c][j] - lift : m[c][j];
                            if (first_scales || y[j] - m[c][j] > reach || z[j] - m[c][j] > 15.f)
                                mx = fmaxf(mx, fmaxf(y[j] - lift, z[j] - 7.f));
                            const float a = m[c][j] == -INFINITY ? (mx == -INFINITY ? 1.f : 0.f) : ptx::ex2(m[c][j] - mx);
                            lsum[c][j] *= a;
                            cen[c][j] *= a;
#pragma unroll
                            for (int t = 0; t < 8; ++t) {
                                acc[c][t][j] *= a;
                                acc[c][t][2 + j] *= a;
                            }
                            m[c][j] = mx;
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (x[u][c][j] != -INFINITY)
                                    x[u][c][j] = __fsub_rn(__fmul_rn(s[u][c][j], sl2[c][j & 1]), m[c][j & 1]);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float p[TILES][4];
#pragma unroll
                    for (int c = 0; c < TILES; ++c) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[c][j] = ptx::ex2(x[u][c][j]);
                        lsum[c][0] += p[c][0] + p[c][2];
                        lsum[c][1] += p[c][1] + p[c][3];
                    }
                    ValueWords w;
                    load_values(w, blk + u * BLOCK, r4, c4);
                    if (u == 1) {
                        // The pair has been read: its slot goes back.
                        __syncwarp();
                        if (i + NST < batch) issue(i + NST, slot);
                    }
                    if (vf != ONE) {
                        w.vsa = make_uint2(mul_bf16x2(w.vsa.x, vf), mul_bf16x2(w.vsa.y, vf));
                        w.vsb = make_uint2(mul_bf16x2(w.vsb.x, vf), mul_bf16x2(w.vsb.y, vf));
                    }
                    {
                        const uint32_t a[4] = {w.vza, w.vza, w.vzb, w.vzb};
#pragma unroll
                        for (int c = 0; c < TILES; ++c)
                            mma(cen[c], a, transpose8(ptx::pack_bf16x2(p[c][0], p[c][1])),
                                transpose8(ptx::pack_bf16x2(p[c][2], p[c][3])));
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
                        const float fa = group_f(w.vsa, g), fb = group_f(w.vsb, g);
                        const uint32_t wa = __byte_perm(g < 2 ? w.va.x : w.va.y, g < 2 ? w.va.z : w.va.w, sel);
                        const uint32_t wb = __byte_perm(g < 2 ? w.vb.x : w.vb.y, g < 2 ? w.vb.z : w.vb.w, sel);
                        const uint32_t a0[4] = {value_pair<0>(wa), value_pair<1>(wa), value_pair<0>(wb), value_pair<1>(wb)};
                        const uint32_t a1[4] = {value_pair<2>(wa), value_pair<3>(wa), value_pair<2>(wb), value_pair<3>(wb)};
#pragma unroll
                        for (int c = 0; c < TILES; ++c) {
                            const uint32_t b0 = transpose8(pack_f16x2(p[c][0] * fa, p[c][1] * fa));
                            const uint32_t b1 = transpose8(pack_f16x2(p[c][2] * fb, p[c][3] * fb));
                            mma_f16(acc[c][2 * g], a0, b0, b1);
                            mma_f16(acc[c][2 * g + 1], a1, b0, b1);
                        }
                    }
                }
                if (++slot == NST) {
                    slot = 0;
                    parity ^= 1;
                }
            }
            if (i < batch) {
                // A wait gave up: let this warp's copies in flight land first.
                for (int j = i; j < min(batch, i + NST); ++j) {
                    drain_wait(full + slot, parity, wc);
                    if (++slot == NST) {
                        slot = 0;
                        parity ^= 1;
                    }
                }
                break;
            }
            left -= batch;
            base += batch;
            if (left > 0) {
                load_table(base);
                issue_first(min(left, 32));
            }
        }
        // The row sums over the tokens of the fragments (row groups r4), and each warp's
        // output, normalised, with the centers' term: its reference is then the
        // log-sum-exp, and warps need not agree on theirs or on the scales' factor.
        const float vf_back = 1.f / lo_f(vf);
#pragma unroll
        for (int c = 0; c < TILES; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) lsum[c][j] += __shfl_xor_sync(0xffffffffu, lsum[c][j], o);
                const bool any = lsum[c][j] != 0.f;  // NaN included
                const float inv = any ? 1.f / lsum[c][j] : 0.f;
                m[c][j] = any ? m[c][j] + ptx::lg2(lsum[c][j]) : -INFINITY;
                lsum[c][j] = any ? 1.f : 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float add = __shfl_sync(0xffffffffu, cen[c][j], 4 * g + c4) * inv;
#pragma unroll
                    for (int t = 2 * g; t < 2 * g + 2; ++t) {
                        acc[c][t][j] = fmaf(acc[c][t][j] * (inv * VALUE_STEPS), vf_back, add);
                        acc[c][t][2 + j] = fmaf(acc[c][t][2 + j] * (inv * VALUE_STEPS), vf_back, add);
                    }
                }
            }
        // The four warps' results meet in two rounds: 2 and 3 into 0 and 1, then 1
        // into 0, a lane's words with the same lane's.
        auto give = [&](int half) {
            float *x = exchange + half * (S::EXCHANGE / 4);
#pragma unroll
            for (int c = 0; c < TILES; ++c, x += 36 * 32) {
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[(4 * t + k) * 32] = acc[c][t][k];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[(32 + j) * 32] = m[c][j];
                    x[(34 + j) * 32] = lsum[c][j];
                }
            }
        };
        auto take = [&](int half) {
            const float *x = exchange + half * (S::EXCHANGE / 4);
#pragma unroll
            for (int c = 0; c < TILES; ++c, x += 36 * 32) {
                float fa[2], fb[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // (an empty side has zeros to add; a NaN stays one)
                    const float mo = x[(32 + j) * 32], mx = fmaxf(m[c][j], mo);
                    fa[j] = m[c][j] == -INFINITY ? 0.f : ptx::ex2(m[c][j] - mx);
                    fb[j] = mo == -INFINITY ? 0.f : ptx::ex2(mo - mx);
                    lsum[c][j] = lsum[c][j] * fa[j] + x[(34 + j) * 32] * fb[j];
                    m[c][j] = mx;
                }
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[c][t][k] = acc[c][t][k] * fa[k & 1] + x[(4 * t + k) * 32] * fb[k & 1];
            }
        };
        __syncthreads();  // the exchange of the segment before has been read
        if (warp >= 2) give(warp - 2);
        __syncthreads();
        if (*abort_flag) {  // a wait gave up: nothing more is written, or merged from here
            if (threadIdx.x < 2) p.cuts[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
            return;
        }
        if (warp < 2) take(warp);
        if (warp == 1) {
            __syncwarp();
            give(1);
        }
        __syncthreads();
        if (warp == 0) {
            take(1);
            const bool done = count == seq_pairs;  // the whole sequence: no merge
            const int64_t part = ((int64_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * COLS;
#pragma unroll
            for (int c = 0; c < TILES; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = 8 * c + 2 * c4 + j;
                    if (col >= cols) continue;
                    const bool any = lsum[c][j] != 0.f;  // NaN included
                    const float inv = any ? 1.f / lsum[c][j] : 0.f;
                    const float l2 = any ? m[c][j] + ptx::lg2(lsum[c][j]) : -INFINITY;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float o0 = any ? acc[c][2 * g][j] * inv : 0.f;
                        const float o1 = any ? acc[c][2 * g][2 + j] * inv : 0.f;
                        const float o2 = any ? acc[c][2 * g + 1][j] * inv : 0.f;
                        const float o3 = any ? acc[c][2 * g + 1][2 + j] * inv : 0.f;
                        const int64_t at = 32 * g + 4 * r4;
                        if (done)
                            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + (row0 + col) * D + at) =
                                make_uint2(ptx::pack_bf16x2(o0, o1), ptx::pack_bf16x2(o2, o3));
                        else
                            *reinterpret_cast<float4 *>(p.o_part + (part + col) * D + at) = make_float4(o0, o1, o2, o3);
                    }
                    if (r4 == 0) {
                        if (!done) p.lse_part[part + col] = l2;
                        else if (p.lse) p.lse[row0 + col] = l2 * LN2;
                    }
                }
        }
        u += count;
        first = 0;
        if (++h == p.Hkv && u < u1) {
            h = 0;
            do {
                L = p.seqlens[++b];
                seq_pairs = pairs_of(L, p.max_blocks);
            } while (seq_pairs == 0);
        }
    }
    ptx::allow_next_work();
}

// Merge of the cut runs.  A run of few parts is merged by the CTA of the share in which
// it begins, a warp a head; the heads of a longer one go to the CTAs of its shares in
// turn, each head to eight warps that take every eighth part.  Four channels a lane; the
// order is fixed.  It adds 2 to 5 us to the share kernel; with a CTA for each head of
// each run, 3 to 9 (3 sequences of 100 thousand tokens: 41.1 us in all against 44.8).
constexpr int MERGE_WARPS = 8;
constexpr int SHORT_RUN = 8;
constexpr int AHEAD = 4;  // parts in flight
__global__ void __launch_bounds__(MERGE_WARPS * 32)
    merge_kernel(const DecodeQ4Params p, int col_blocks, int cta_cols) {
    __shared__ __align__(16) float part[MERGE_WARPS][D];
    __shared__ float part_m[MERGE_WARPS], part_l[MERGE_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Launched as a programmatic dependent of the share kernel: its partials are
    // visible from here on.
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    const int4 cuts[2] = {p.cuts[2 * blockIdx.x], p.cuts[2 * blockIdx.x + 1]};
    float M, l;
    float4 o;
    // Adds up head c's parts sub, sub + each, .. of a run that begins in CTA `from`.  The first
    // part is its share's last one, the others are their shares' first.
    auto add_parts = [&](int from, int parts, int c, int sub, int each) {
        auto row_of = [&](int s) { return ((int64_t)(from + s * col_blocks) * 2 + (s == 0 ? 1 : 0)) * cta_cols + c; };
        M = -INFINITY, l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = sub; s0 < parts; s0 += AHEAD * each) {
            float x[AHEAD];
            float4 v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int s = s0 + i * each;
                x[i] = -INFINITY;
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s < parts) {
                    x[i] = p.lse_part[row_of(s)];
                    v[i] = reinterpret_cast<const float4 *>(p.o_part + row_of(s) * D)[lane];
                }
            }
            float mx = M;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) mx = fmaxf(mx, x[i]);
            const float f = M == -INFINITY ? 1.f : ptx::ex2(M - mx);  // (before a finite one: 0 or NaN, which stays)
            l *= f;
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            M = mx;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float w = x[i] == -INFINITY ? 0.f : ptx::ex2(x[i] - (M == -INFINITY ? 0.f : M));  // NaN stays
                l += w;
                o.x = fmaf(w, v[i].x, o.x);
                o.y = fmaf(w, v[i].y, o.y);
                o.z = fmaf(w, v[i].z, o.z);
                o.w = fmaf(w, v[i].w, o.w);
            }
        }
    };
    auto write_row = [&](int64_t r) {
        const bool any = l != 0.f;
        const float inv = any ? 1.f / l : 0.f;
        reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + r * D)[lane] =
            any ? make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv))
                : make_uint2(0, 0);
        if (p.lse && lane == 0) p.lse[r] = any ? (M + ptx::lg2(l)) * LN2 : -INFINITY;
    };
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int row0 = cuts[e].x, cols = cuts[e].y, parts = cuts[e].z, index = cuts[e].w;
        // (Always within this call's rows, unless a call that runs at the same time has been
        // given the same workspace: then nothing out of bounds is touched.)
        if ((unsigned)(parts - 1) >= gridDim.x || (unsigned)index >= (unsigned)parts || cols > cta_cols) continue;
        const int from = (int)blockIdx.x - index * col_blocks;
        if (from < 0 || from + (parts - 1) * col_blocks >= (int)gridDim.x || (unsigned)row0 > (unsigned)(p.B * p.Hq - cols))
            continue;
        if (parts <= SHORT_RUN) {
            if (index == 0)
                for (int c = warp; c < cols; c += MERGE_WARPS) {
                    add_parts(blockIdx.x, parts, c, 0, 1);
                    write_row((int64_t)row0 + c);
                }
            continue;
        }
        for (int c = index; c < cols; c += parts) {
            add_parts(from, parts, c, warp, MERGE_WARPS);
            reinterpret_cast<float4 *>(part[warp])[lane] = o;
            if (lane == 0) {
                part_m[warp] = M;
                part_l[warp] = l;
            }
            __syncthreads();
            if (warp == 0) {
                M = -INFINITY, l = 0.f;
                o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < MERGE_WARPS; ++w) M = fmaxf(M, part_m[w]);
#pragma unroll
                for (int w = 0; w < MERGE_WARPS; ++w) {
                    const float f = part_m[w] == -INFINITY ? 1.f : ptx::ex2(part_m[w] - M);  // no finite one: 0 or NaN
                    const float4 v = reinterpret_cast<const float4 *>(part[w])[lane];
                    l += part_l[w] * f;
                    o.x = fmaf(v.x, f, o.x);
                    o.y = fmaf(v.y, f, o.y);
                    o.z = fmaf(v.z, f, o.z);
                    o.w = fmaf(v.w, f, o.w);
                }
                write_row((int64_t)row0 + c);
            }
            __syncthreads();
        }
    }
}

// Column blocks of a KV head's G query heads, and CTAs: shares times those.
struct Grid {
    int tiles, cols, col_blocks, ctas;
};

Grid grid_of(int B, int Hq, int Hkv, int max_blocks, int sm_count) {
    const int G = Hq / Hkv;
    Grid g;
    g.tiles = G > 8 ? 2 : 1;
    g.cols = 8 * g.tiles;
    g.col_blocks = (G + g.cols - 1) / g.cols;
    const int per_sm = g.tiles == 2 ? Shape<2>::CTAS_PER_SM : Shape<1>::CTAS_PER_SM;
    const int most = g.tiles == 2 ? Shape<2>::MAX_CTAS : Shape<1>::MAX_CTAS;
    const int resident = sm_count > 0 && per_sm * sm_count < most ? per_sm * sm_count : most;
    const int64_t items = (int64_t)B * Hkv;
    const int64_t fill = (items * ((max_blocks + 1) / 2) + MIN_PAIRS - 1) / MIN_PAIRS;
    int64_t shares = resident / g.col_blocks;
    if (shares > (items > fill ? items : fill)) shares = items > fill ? items : fill;
    if (shares < 1) shares = 1;
    g.ctas = (int)shares * g.col_blocks;
    return g;
}

template <int TILES>
cudaError_t launch_shares(const DecodeQ4Params &p, const Grid &g, cudaStream_t stream) {
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device != dev) {
        e = cudaFuncSetAttribute(share_kernel<TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<TILES>::SMEM);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(share_kernel<TILES>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch_dependent(share_kernel<TILES>, g.ctas, NT, Shape<TILES>::SMEM, stream, p, g.col_blocks);
}

}  // namespace dq4

size_t decode_q4_partial_rows(int B, int Hq, int Hkv, int max_blocks, size_t *ctas) {
    const dq4::Grid g = dq4::grid_of(B, Hq, Hkv, max_blocks, 0);
    *ctas = (size_t)g.ctas;
    return (size_t)g.ctas * 2 * g.cols;
}

cudaError_t launch_decode_q4(const DecodeQ4Params &p, int sm_count, cudaStream_t stream) {
    const dq4::Grid g = dq4::grid_of(p.B, p.Hq, p.Hkv, p.max_blocks, sm_count);
    const cudaError_t e = g.tiles == 2 ? dq4::launch_shares<2>(p, g, stream) : dq4::launch_shares<1>(p, g, stream);
    // Nothing is cut either of one sequence with a share for each KV head.
    const int shares = g.ctas / g.col_blocks;
    if (e != cudaSuccess || (p.B == 1 && shares == p.Hkv) || dq4::never_cut(p.B, p.Hkv, p.max_blocks, shares)) return e;
    return launch_dependent(dq4::merge_kernel, g.ctas, dq4::MERGE_WARPS * 32, 0, stream, p, g.col_blocks, g.cols);
}

}  // namespace attn
