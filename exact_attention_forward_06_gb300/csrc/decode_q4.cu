// decode_q4.cu -- attention of single tokens over the 4-bit cache
// (attn_decode_paged_q4): a key split and its log-sum-exp merge.
//
// A page of one KV head is one 2560-byte block, read once: 4096 codes and 256
// parameters for 4 flops a code and query head, so HBM bandwidth is the bound
// as long as a page's arithmetic fits in the time its bytes take (about 110 SM
// clocks at the measured copy bandwidth).  That budget, about four instructions
// per eight codes, decides the form:
//
// - Codes go to the tensor cores without being turned into values.  A code n
//   moved to bits 3..6 of a bf16 whose other bits say 16.0 is the number 16 + n
//   exactly (one shift and one and/or per two codes); the offset to n - 7.5 is
//   -23.5 and is taken off after the product.
// - S^T = K Q^T (mma m16n8k16, the page's 16 tokens as rows, up to eight query
//   heads of the KV head as columns), group by group of 32 channels:
//       s_t += scale_tg * (sum_c q_c (16 + n_tc) - 23.5 Q_g) + center_tg * Q_g,
//   Q_g = sum of the group's q.  -23.5 Q_g is the product's initial accumulator;
//   the centers' term is one product for all groups, with Q_g cut into three
//   bf16 parts (24 bits).
// - O^T += V^T P^T: a group's scale goes to the probability, P'_t = P_t scale_tg
//   (rounded to bf16 as P is); the offset is one product per group with a
//   constant matrix of -23.5, so it takes off exactly what the rounded P' brought
//   in; the centers' term is one product with the unscaled P.
// - The byte order of the block (q4.cuh) is that of the fragments: every lane
//   reads its operands as 16-byte words without bank conflicts, and a value
//   pair of two tokens is one byte permutation.
//
// Each warp streams pages w, w + 4, .. of the CTA's split through a ring of its
// own (one bulk copy a page, issued by its lane 0 as soon as the page's words
// are in registers): no producer warp and no barrier between warps until the
// four partial results meet at the end.  Scores, sums and outputs are fp32; P and
// P' are rounded to bf16 for the product alone, the row sum adds the fp32 values.
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "cache_ops.h"
#include "common.cuh"
#include "q4.cuh"

namespace attn {
namespace dq4 {

using q4::BLOCK;
using q4::D;
using q4::PAGE;

constexpr int NW = 4;    // warps = page streams
constexpr int NST = 3;   // page pairs in flight per warp
constexpr int COLS = 8;  // query heads per CTA (MMA columns)
constexpr int NT = NW * 32;
constexpr int CTAS_PER_SM = 3;
constexpr int STAGE = 2 * BLOCK;
constexpr int RING = NW * NST * STAGE;
constexpr int SMEM = RING + NW * NST * 8 + 16;  // ring, barriers, abort flag
constexpr int MERGE_ROW = D + 2;
static_assert(NW * COLS * MERGE_ROW * 4 <= RING, "the merge reuses the ring");
static_assert(CTAS_PER_SM * (SMEM + 1024) <= 233472, "CTAs per SM");
constexpr int MAX_PAGES_PER_SPLIT = 64 * NW;  // a pair of table entries a lane
constexpr float RAISE = 8.f;  // a score this far (in log2) above the running max raises it
constexpr int TARGET_CTAS = 2048;
constexpr float LN2 = 0.6931471805599453f;
constexpr float LOG2E = 1.4426950408889634f;

// Codes j and j + 4 of a word as the bf16 pair (16 + n, 16 + n').
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    const uint32_t s = J == 0 ? w << 3 : w >> (4 * J - 3);
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x00780078, %2, 0xEA;" : "=r"(r) : "r"(s), "r"(0x41804180u));  // (s & mask) | 16.0
    return r;
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
    const uint8_t *par = blk + r4 * 8;
    w.vsa = *reinterpret_cast<const uint2 *>(par + q4::V_SCALES);
    w.vsb = *reinterpret_cast<const uint2 *>(par + q4::V_SCALES + 64);
    const uint8_t *z = blk + q4::V_CENTERS + (r4 & 3) * 32 + c4 * 4;
    w.vza = *reinterpret_cast<const uint32_t *>(z);
    w.vzb = *reinterpret_cast<const uint32_t *>(z + 16);
}

__global__ void __launch_bounds__(NT, CTAS_PER_SM) split_kernel(const DecodeQ4Params p, int col_blocks) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r4 = lane >> 2, c4 = lane & 3;
    uint8_t *ring = smem + warp * NST * STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + RING) + warp * NST;
    volatile int *abort_flag = reinterpret_cast<int *>(smem + RING + NW * NST * 8);

    const int G = p.Hq / p.Hkv;
    const int h = blockIdx.x / col_blocks, col0 = (blockIdx.x - h * col_blocks) * COLS;
    const int cols = min(COLS, G - col0);
    const int split = blockIdx.y, b = blockIdx.z;
    const int64_t row0 = (int64_t)b * p.Hq + h * G + col0;

    const int L_raw = __ldg(p.seqlens + b);
    const bool bad_len = L_raw < 0 || L_raw > p.max_blocks * PAGE;
    if (bad_len && threadIdx.x == 0 && split == 0 && blockIdx.x == 0)
        report_status(p.status, kStatusDeviceBounds, kSiteQ4Seqlen);
    const int L = bad_len ? 0 : L_raw;
    const int page0 = split * p.pages_per_split;
    const int np = min(p.pages_per_split, (L + PAGE - 1) / PAGE - page0);
    if (np <= 0) {
        // Nothing here; the merge does not read this split's partial.  With a
        // single split there is no merge, and the row is empty.
        if (p.nsplit == 1) {
            for (int i = threadIdx.x; i < cols * D / 2; i += NT)
                reinterpret_cast<uint32_t *>(p.out)[row0 * (D / 2) + i] = 0u;
            if (p.lse && threadIdx.x < cols) p.lse[row0 + threadIdx.x] = -INFINITY;
        }
        return;
    }
    // This warp's page pairs: pages page0 + 2 (warp + NW i) and the next, i < n.
    // Lane i holds pair i's pages (-1: none, or a bad entry) and their numbers
    // of keys.
    const int npairs = (np + 1) / 2;
    const int n = warp < npairs ? (npairs - warp + NW - 1) / NW : 0;
    int tab0 = -1, tab1 = -1, nv0 = 0, nv1 = 0;
    if (lane < n) {
        const int first = 2 * (warp + NW * lane);
        const int32_t *row = p.block_table + (int64_t)b * p.max_blocks + page0 + first;
        tab0 = __ldg(row);
        if (first + 1 < np) tab1 = __ldg(row + 1);
        const bool bad0 = tab0 < 0 || tab0 >= p.num_pages;
        const bool bad1 = first + 1 < np && (tab1 < 0 || tab1 >= p.num_pages);
        if (bad0 || bad1) report_status(p.status, kStatusDeviceBounds, kSiteQ4Table);
        if (bad0) tab0 = -1;
        if (bad1) tab1 = -1;
        const int left = L - (page0 + first) * PAGE;
        nv0 = bad0 ? 0 : min(PAGE, left);
        nv1 = tab1 < 0 ? 0 : min(PAGE, left - PAGE);
    }
    const unsigned whole = __ballot_sync(0xffffffffu, nv0 == PAGE && nv1 == PAGE);

    if (lane == 0) {
        for (int s = 0; s < NST; ++s) ptx::mbar_init(full + s, 1);
        if (warp == 0) *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const WaitCtx wc{abort_flag, p.status, p.budget_ns};

    const uint64_t pol = ptx::policy_evict_first();
    const uint8_t *cache = static_cast<const uint8_t *>(p.cache) + (int64_t)h * BLOCK;
    const int64_t page_step = (int64_t)p.Hkv * BLOCK;
    auto issue = [&](int i, int slot) {
        const int t0 = __shfl_sync(0xffffffffu, tab0, i), t1 = __shfl_sync(0xffffffffu, tab1, i);
        if (lane == 0) {
            uint8_t *dst = ring + slot * STAGE;
            ptx::mbar_arrive_expect_tx(full + slot, (t0 >= 0 ? BLOCK : 0) + (t1 >= 0 ? BLOCK : 0));
            if (t0 >= 0) ptx::bulk_load(dst, cache + t0 * page_step, BLOCK, full + slot, pol);
            if (t1 >= 0) ptx::bulk_load(dst + BLOCK, cache + t1 * page_step, BLOCK, full + slot, pol);
        }
    };
    const int ahead = min(n, NST);
    for (int i = 0; i < ahead; ++i) issue(i, i);

    // Q^T as the B operand: head r4 (zero past the CTA's columns), the channels
    // 32 g + 8 c4 + (j, j + 4), j = 0..3, in the order of a key word's pairs.
    // qz, qo: B operands of the centers' and the scales' products.  k = 2 c4,
    // 2 c4 + 1 and 2 c4 + 8 are group c4's Q_g (or -23.5 Q_g) in three bf16
    // parts, k = 2 c4 + 9 is zero.
    uint32_t qb[4][4], qz0, qz1, qo0, qo1;
    {
        const uint4 *qrow = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + (row0 + r4) * D);
        float x = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint4 v = r4 < cols ? __ldg(qrow + 4 * g + c4) : make_uint4(0, 0, 0, 0);
            qb[g][0] = __byte_perm(v.x, v.z, 0x5410);
            qb[g][1] = __byte_perm(v.x, v.z, 0x7632);
            qb[g][2] = __byte_perm(v.y, v.w, 0x5410);
            qb[g][3] = __byte_perm(v.y, v.w, 0x7632);
            float s = ((lo_f(v.x) + hi_f(v.x)) + (lo_f(v.y) + hi_f(v.y))) +
                      ((lo_f(v.z) + hi_f(v.z)) + (lo_f(v.w) + hi_f(v.w)));
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
        parts(x, qz0, qz1);
        parts(-23.5f * x, qo0, qo1);
    }
    // The byte selector that doubles group c4's entry of four bf16.
    const uint32_t own = 0x1010u + 0x2222u * c4;

    const float sl2 = p.scale_log2;
    // Running max (log2 units) and row sum of heads 2 c4, 2 c4 + 1.  acc[2 g + i]:
    // channels 32 g + 4 r4 + 2 i (+ 1) times those heads; off[g]: the group's
    // offset (the same in every row); cen: the centers' term of group r4 % 4.
    float m[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
    float acc[8][4], off[4][4], cen[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) off[g][0] = off[g][1] = off[g][2] = off[g][3] = 0.f;

    int slot = 0, i = 0;
    uint32_t parity = 0;
    for (; i < n; ++i) {
        if (!wait_bounded(full + slot, parity, wc, kSiteQ4Page)) break;
        const uint8_t *blk = ring + slot * STAGE;
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            KeyWords k;
            load_keys(k, blk + u * BLOCK, r4, c4);
            const uint32_t za = __byte_perm(k.kza.x, k.kza.y, own), zb = __byte_perm(k.kzb.x, k.kzb.y, own);
            const uint32_t sa = __byte_perm(k.ksa.x, k.ksa.y, own), sb = __byte_perm(k.ksb.x, k.ksb.y, own);
            const uint32_t az[4] = {za, zb, za, zb}, as[4] = {sa, sb, sa, sb};
            mma_zero(s[u], az, qz0, qz1);
            mma(s[u], as, qo0, qo1);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t wa = g == 0 ? k.ka.x : g == 1 ? k.ka.y : g == 2 ? k.ka.z : k.ka.w;
                const uint32_t wb = g == 0 ? k.kb.x : g == 1 ? k.kb.y : g == 2 ? k.kb.z : k.kb.w;
                float d[4];
                const uint32_t a0[4] = {code_pair<0>(wa), code_pair<0>(wb), code_pair<1>(wa), code_pair<1>(wb)};
                mma_zero(d, a0, qb[g][0], qb[g][1]);
                const uint32_t a1[4] = {code_pair<2>(wa), code_pair<2>(wb), code_pair<3>(wa), code_pair<3>(wb)};
                mma(d, a1, qb[g][2], qb[g][3]);
                const float fa = group_f(k.ksa, g), fb = group_f(k.ksb, g);
                s[u][0] = fmaf(fa, d[0], s[u][0]);
                s[u][1] = fmaf(fa, d[1], s[u][1]);
                s[u][2] = fmaf(fb, d[2], s[u][2]);
                s[u][3] = fmaf(fb, d[3], s[u][3]);
            }
        }
        // s[u][0], s[u][1]: token r4 of page u, heads 2 c4, 2 c4 + 1; [2], [3]:
        // token r4 + 8.  x: over the running max, in log2 units.
        float x[2][4];
        auto over = [&]() {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[u][j] = fmaf(s[u][j], sl2, -m[j & 1]);
        };
        over();
        const bool all = whole >> i & 1;
        if (!all) {
            // Slots past the end hold arbitrary bits: their scores are replaced
            // here, the values' parameters below.
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int nv = __shfl_sync(0xffffffffu, u ? nv1 : nv0, i);
                if (r4 >= nv) x[u][0] = x[u][1] = -INFINITY;
                if (r4 + 8 >= nv) x[u][2] = x[u][3] = -INFINITY;
            }
        }
        // The running max follows only when a score is RAISE above it (the first
        // keys are: the max is -inf): probabilities then stay below 2^RAISE,
        // which costs the sums nothing, and a raise, with its shuffles and the
        // rescaling, is rare instead of nearly every page.
        const float top0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
        const float top1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
        if (__any_sync(0xffffffffu, top0 > RAISE || top1 > RAISE)) {
            float y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                y0 = fmaxf(y0, fmaxf(x[u][0] == -INFINITY ? -INFINITY : s[u][0] * sl2,
                                     x[u][2] == -INFINITY ? -INFINITY : s[u][2] * sl2));
                y1 = fmaxf(y1, fmaxf(x[u][1] == -INFINITY ? -INFINITY : s[u][1] * sl2,
                                     x[u][3] == -INFINITY ? -INFINITY : s[u][3] * sl2));
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, o));
                y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, o));
            }
            const float m0 = fmaxf(m[0], y0), m1 = fmaxf(m[1], y1);
            const float a0 = m[0] == -INFINITY ? (m0 == -INFINITY ? 1.f : 0.f) : ptx::ex2(m[0] - m0);
            const float a1 = m[1] == -INFINITY ? (m1 == -INFINITY ? 1.f : 0.f) : ptx::ex2(m[1] - m1);
            lsum[0] *= a0;
            lsum[1] *= a1;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                acc[t][0] *= a0;
                acc[t][1] *= a1;
                acc[t][2] *= a0;
                acc[t][3] *= a1;
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                off[g][0] *= a0;
                off[g][1] *= a1;
            }
            cen[0] *= a0;
            cen[1] *= a1;
            m[0] = m0;
            m[1] = m1;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (x[u][j] != -INFINITY) x[u][j] = fmaf(s[u][j], sl2, -m[j & 1]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float p0 = ptx::ex2(x[u][0]), p1 = ptx::ex2(x[u][1]);
            const float p2 = ptx::ex2(x[u][2]), p3 = ptx::ex2(x[u][3]);
            lsum[0] += p0 + p2;
            lsum[1] += p1 + p3;
            ValueWords w;
            load_values(w, blk + u * BLOCK, r4, c4);
            if (u == 1) {
                // The pair has been read: its slot goes back.
                __syncwarp();
                if (i + NST < n) issue(i + NST, slot);
            }
            if (!all) {
                const int nv = __shfl_sync(0xffffffffu, u ? nv1 : nv0, i);
                if (r4 >= nv) w.vsa = make_uint2(0, 0);
                if (r4 + 8 >= nv) w.vsb = make_uint2(0, 0);
                w.vza &= (2 * c4 < nv ? 0x0000ffffu : 0u) | (2 * c4 + 1 < nv ? 0xffff0000u : 0u);
                w.vzb &= (2 * c4 + 8 < nv ? 0x0000ffffu : 0u) | (2 * c4 + 9 < nv ? 0xffff0000u : 0u);
            }
            {
                const uint32_t a[4] = {w.vza, w.vza, w.vzb, w.vzb};
                mma(cen, a, transpose8(ptx::pack_bf16x2(p0, p1)),
                                    transpose8(ptx::pack_bf16x2(p2, p3)));
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float fa = group_f(w.vsa, g), fb = group_f(w.vsb, g);
                // P'^T as the B operand: tokens 2 c4 (+ 1) and 2 c4 + 8 (+ 9), head r4.
                const uint32_t b0 = transpose8(ptx::pack_bf16x2(p0 * fa, p1 * fa));
                const uint32_t b1 = transpose8(ptx::pack_bf16x2(p2 * fb, p3 * fb));
                const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
                const uint32_t wa = __byte_perm(g < 2 ? w.va.x : w.va.y, g < 2 ? w.va.z : w.va.w, sel);
                const uint32_t wb = __byte_perm(g < 2 ? w.vb.x : w.vb.y, g < 2 ? w.vb.z : w.vb.w, sel);
                const uint32_t a0[4] = {code_pair<0>(wa), code_pair<1>(wa), code_pair<0>(wb), code_pair<1>(wb)};
                mma(acc[2 * g], a0, b0, b1);
                const uint32_t a1[4] = {code_pair<2>(wa), code_pair<3>(wa), code_pair<2>(wb), code_pair<3>(wb)};
                mma(acc[2 * g + 1], a1, b0, b1);
                const uint32_t a2[4] = {0xC1BCC1BCu, 0xC1BCC1BCu, 0xC1BCC1BCu, 0xC1BCC1BCu};  // -23.5
                mma(off[g], a2, b0, b1);
            }
        }
        if (++slot == NST) {
            slot = 0;
            parity ^= 1;
        }
    }
    // Row sums over the tokens of the fragments (row groups r4).
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        lsum[0] += __shfl_xor_sync(0xffffffffu, lsum[0], o);
        lsum[1] += __shfl_xor_sync(0xffffffffu, lsum[1], o);
    }
    // After a wait that gave up: let this warp's copies in flight land first.
    for (int j = i; j < min(n, i + NST); ++j) drain_wait(full + j % NST, (j / NST) & 1, wc);
    __syncthreads();  // every warp has read its pages: the ring becomes the merge's scratch
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (*abort_flag) return;
    float *merge = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int hc = 2 * c4 + j;
        float *dst = merge + (warp * COLS + hc) * MERGE_ROW;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float add = off[g][j] + __shfl_sync(0xffffffffu, cen[j], 4 * g + c4);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[32 * g + 4 * r4 + i] = acc[2 * g + i / 2][2 * (i & 1) + j] + add;
        }
        if (r4 == 0) {
            dst[D] = m[j];
            dst[D + 1] = lsum[j];
        }
    }
    __syncthreads();
    // Merge the page streams: thread = channel, loop over heads.
    const int e = threadIdx.x;
    for (int c = 0; c < cols; ++c) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, merge[(w * COLS + c) * MERGE_ROW + D]);
        float Ls = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float *src = merge + (w * COLS + c) * MERGE_ROW;
            // A stream without a finite score has only zeros, or NaN, to add.
            const float f = src[D] == -INFINITY ? 1.f : ptx::ex2(src[D] - M);
            Ls += src[D + 1] * f;
            o += src[e] * f;
        }
        const bool any = Ls != 0.f;  // NaN included
        o = any ? o / Ls : 0.f;
        const float lse = any ? (M + ptx::lg2(Ls)) * LN2 : -INFINITY;
        const int64_t r = row0 + c;
        if (p.nsplit == 1) {
            static_cast<uint16_t *>(p.out)[r * D + e] = (uint16_t)(ptx::pack_bf16x2(o, 0.f) & 0xffffu);
            if (p.lse && e == 0) p.lse[r] = lse;
        } else {
            p.o_part[(r * p.nsplit + split) * D + e] = o;
            if (e == 0) p.lse_part[r * p.nsplit + split] = lse;
        }
    }
}

// Merge of the splits that hold keys: one CTA per row, a warp takes every
// MERGE_WARPS-th split, four channels a lane; the order is fixed.
constexpr int MERGE_WARPS = 8;
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_kernel(const DecodeQ4Params p) {
    __shared__ float part[MERGE_WARPS][D];
    __shared__ float part_m[MERGE_WARPS], part_l[MERGE_WARPS];
    const int64_t r = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = __ldg(p.seqlens + r / p.Hq);
    const int pages = L < 0 || L > p.max_blocks * PAGE ? 0 : (L + PAGE - 1) / PAGE;
    const int used = (pages + p.pages_per_split - 1) / p.pages_per_split;
    // Launched as a programmatic dependent of the split kernel: its partials are
    // visible from here on.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *ls = p.lse_part + r * p.nsplit;
    const float4 *os = reinterpret_cast<const float4 *>(p.o_part + r * p.nsplit * D) + lane;
    float M = -INFINITY;
    for (int s = warp; s < used; s += MERGE_WARPS) M = fmaxf(M, ls[s]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = warp; s < used; s += MERGE_WARPS) {
        const float x = ls[s];
        const float w = x == -INFINITY ? 0.f : ptx::ex2((x - (M == -INFINITY ? 0.f : M)) * LOG2E);  // NaN stays
        const float4 v = os[s * (D / 4)];
        l += w;
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    }
    reinterpret_cast<float4 *>(part[warp])[lane] = o;
    if (lane == 0) {
        part_m[warp] = M;
        part_l[warp] = l;
    }
    __syncthreads();
    if (threadIdx.x >= D) return;
    float Mt = -INFINITY, Lt = 0.f, ot = 0.f;
#pragma unroll
    for (int w = 0; w < MERGE_WARPS; ++w) Mt = fmaxf(Mt, part_m[w]);
#pragma unroll
    for (int w = 0; w < MERGE_WARPS; ++w) {
        const float f = part_m[w] == -INFINITY ? 1.f : ptx::ex2((part_m[w] - Mt) * LOG2E);  // no finite one: 0 or NaN
        Lt += part_l[w] * f;
        ot += part[w][threadIdx.x] * f;
    }
    const bool any = Lt != 0.f;
    ot = any ? ot / Lt : 0.f;
    static_cast<uint16_t *>(p.out)[r * D + threadIdx.x] = (uint16_t)(ptx::pack_bf16x2(ot, 0.f) & 0xffffu);
    if (p.lse && threadIdx.x == 0) p.lse[r] = any ? Mt + ptx::lg2(Lt) * LN2 : -INFINITY;
}

}  // namespace dq4

// Key-split plan, a pure function of the shape: about TARGET_CTAS CTAs over
// the KV heads' column blocks, 16 .. 256 pages per split.
void decode_q4_split_plan(int B, int Hq, int Hkv, int max_blocks, int *nsplit, int *pages_per_split) {
    const int64_t groups = (int64_t)B * Hkv * ((Hq / Hkv + dq4::COLS - 1) / dq4::COLS);
    const int64_t want = (dq4::TARGET_CTAS + groups - 1) / groups;
    int64_t pps = (max_blocks + want - 1) / want;
    if (pps < 16) pps = 16;
    pps += pps & 1;  // whole pairs
    if (pps > dq4::MAX_PAGES_PER_SPLIT) pps = dq4::MAX_PAGES_PER_SPLIT;
    *pages_per_split = (int)pps;
    *nsplit = (int)((max_blocks + pps - 1) / pps);
}

cudaError_t launch_decode_q4(const DecodeQ4Params &p, cudaStream_t stream) {
    const int col_blocks = (p.Hq / p.Hkv + dq4::COLS - 1) / dq4::COLS;
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device != dev) {
        e = cudaFuncSetAttribute(dq4::split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dq4::SMEM);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(dq4::split_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    dq4::split_kernel<<<dim3(p.Hkv * col_blocks, p.nsplit, p.B), dq4::NT, dq4::SMEM, stream>>>(p, col_blocks);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.nsplit == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hq));
    cfg.blockDim = dim3(dq4::MERGE_WARPS * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dq4::merge_kernel, p);
}

}  // namespace attn
