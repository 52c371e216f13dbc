// verify.cu -- verification of drafted tokens against the target's probabilities
// (attn_verify_tree).
//
// The walk down a sequence's tree is a chain of decisions: node c's row of logits
// gives p = softmax(logits[c] / T), one of c's children is accepted (x its token, u
// its uniform number, q the draft's distribution or 1 for tokens that were not drawn)
//     u q(x) < p(x),  a rejected child leaving  p <- max(p - q, 0) / sum,
// and the walk goes on there, or none is and the last token is drawn from what is
// left of p as argmax_i p_i / e_i: of independent exponential numbers e_i / p_i the
// smallest is that of i with probability p_i.
//
// Three kernels.  sums_kernel (where trees are short or their rows few bytes: the rule
// is verify_ahead's) takes maximum and sum of the
// exponentials of all rows, which is what decisions need of a row besides the
// children's own logits; it reads rows that the walk may not come to, and draft rows of
// nodes without children, which nothing asks for, but all at once.
// verify_kernel walks, a cluster of CTAs a sequence, each on a slice of the vocabulary:
// where a row's sums are not there it takes them (one pass, an exchange through the
// cluster's shared memory), then every thread of every CTA decides by itself, from the
// same numbers in the same order.  race_kernel draws the last tokens.  The bound is the
// rows' bytes where there are many sequences, and the chain of row after row where
// there are few.  The kernels run through their code once, so it is kept short (rolled
// loops): with chunks of 32 elements unrolled, in one kernel, half the time went to
// fetching instructions.
// Measured on one GB300, 131072 tokens: 64 sequences of five rows with their draft's (168
// MB) 56 us, 31 of them the sums (5.4 TB/s); 16 trees of 40 to 64 rows, of which the walk
// comes to two to nine, 24 to 31 us (62 where they were drawn from a draft's distributions); five
// fp32 trees with 50001 tokens 18 us; one greedy chain of five rows of 32768 tokens 6 to 10 us.
#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "cache_ops.h"
#include "common.cuh"
#include "speculate.h"

namespace attn {
namespace vf {

// Of verify_kernel: 16 trees of 64 take 26 us with 512, 31 with 256 (fewer loads in flight),
// 27 with 768 and 28 with 1024 (slower barriers).
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int RACE_THREADS = 256;  // of race_kernel
constexpr int RACE_BLOCKS = 4;     // of it an SM
constexpr int SUM_THREADS = 128;  // of sums_kernel
constexpr int MAX_CLUSTER = 8;
constexpr int WALK_END_BYTES = kVerifyEndBytes;
constexpr unsigned ALL = 0xffffffffu;

// Eight consecutive elements of a row, as they are in memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void none() { w[0] = w[1] = w[2] = w[3] = 0xff80ff80u; }  // -inf
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
        if (vec) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        }
    }
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    // The largest element (NaN aside), or -inf.
    __device__ __forceinline__ float top() const {
        const auto h = [&](int i) { return *reinterpret_cast<const __nv_bfloat162 *>(w + i); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
        return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
    }
};
template <>
struct Chunk<float> {
    float2 w[4];
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_float2(-INFINITY, -INFINITY);
    }
    __device__ __forceinline__ void load(const float *p, bool vec) {
        if (vec) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            w[0] = make_float2(a.x, a.y), w[1] = make_float2(a.z, a.w);
            w[2] = make_float2(b.x, b.y), w[3] = make_float2(b.z, b.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = make_float2(p[2 * i], p[2 * i + 1]);
        }
    }
    __device__ __forceinline__ float2 pair(int i) const { return w[i]; }
    __device__ __forceinline__ float top() const {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = ptx::max3(m, w[i].x, w[i].y);
        return m;
    }
};

__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(float x) { return x; }

__device__ __forceinline__ bool vec_ok(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// (x - m) c of two logits, c = log2 e / T, with no overflow on the way.
__device__ __forceinline__ float odd_exponent(float x, float m, float c) {
    return (0.5f * fminf(x, FLT_MAX) - 0.5f * fminf(m, FLT_MAX)) * c * 2.f;
}

__device__ __noinline__ float odd_weight(float x, float m, float c);

// A row's largest logit m and r = m c, rounded.  Weights are taken relative to r, which
// the rounding leaves a little off m c: as every weight and every sum goes by the same r,
// or by the difference of two of them, that cancels, and a weight is one FFMA and one
// exponential.  r is off by half at most, up to 2^23: the largest weight is then up to
// sqrt(2).  Beyond (very low temperatures, a row that is masked with the type's lowest
// value) r is NaN, weights are relative to m c itself, and whatever does not come out as
// a number up to 2 goes the long way.
struct Top {
    float m, r;
    static constexpr float MOST = 8388608.f;
    __device__ __forceinline__ Top(float largest, float c) : m(fminf(largest, FLT_MAX)) {
        r = largest == -INFINITY ? 0.f : __fmul_rn(m, c);
        if (!(fabsf(r) <= MOST)) r = NAN;
    }
    __device__ __forceinline__ float weight(float x, float c) const {
        const float f = ptx::ex2(fmaf(x, c, -r));
        return f <= 2.f ? f : odd_weight(x, m, c);
    }
    // What a sum relative to another maximum, m2 (-inf: an empty sum), is multiplied with: by
    // its r, not by m2 c.
    __device__ __forceinline__ float step(float m2, float c) const {
        const float r2 = __fmul_rn(m2, c), f = ptx::ex2(r2 - r);
        return fabsf(r2) <= MOST || r2 == -INFINITY ? f : NAN;
    }
    static __device__ __forceinline__ bool is_weight(float f) { return f <= 2.f; }
};

// The weight of a logit x of a row whose largest is m, the long way: 0 for NaN and -inf (and
// where m is -inf: nothing is left), +inf counts as the largest finite number (as in m).
__device__ __noinline__ float odd_weight(float x, float m, float c) {
    if (!(x > -INFINITY) || m == -INFINITY) return 0.f;
    const Top t(m, c);
    return ptx::ex2(fminf(t.r == t.r ? fmaf(fminf(x, FLT_MAX), c, -t.r) : odd_exponent(x, m, c), 1.f));
}

// What a sum is multiplied with (see step) where one of the two maxima has no r, or neither.
__device__ __noinline__ float odd_step(float m2, float m, float c) {
    if (m2 == -INFINITY) return 0.f;
    const Top a(m2, c), b(m, c);
    const bool plain_a = a.r == a.r, plain_b = b.r == b.r;
    return ptx::ex2(plain_a ? (plain_b ? a.r - b.r : fmaf(-b.m, c, a.r))
                            : (plain_b ? fmaf(a.m, c, -b.r) : odd_exponent(a.m, b.m, c)));
}

// A maximum and a sum of weights relative to it.
struct Soft {
    float m = -INFINITY, s = 0.f;
    // One more logit.
    __device__ __forceinline__ void add(float x, float c) {
        const Top t(fmaxf(m, x), c);
        raise(t, c);
        s += t.weight(x, c);
    }
    __device__ __forceinline__ void raise(const Top &t, float c) {
        if (t.m > m) {
            const float f = t.step(m, c);
            s *= Top::is_weight(f) ? f : odd_step(m, t.m, c);
            m = t.m;
        }
    }
    // Another thread's or CTA's sum.
    __device__ __forceinline__ void add(float m2, float s2, float c) {
        const Top t(fmaxf(m, m2), c);
        raise(t, c);
        const float f = t.step(m2, c);
        s += s2 * (Top::is_weight(f) ? f : odd_step(m2, t.m, c));
    }
    template <typename T, int U>
    __device__ __forceinline__ void add(const Chunk<T> (&x)[U], float c);
};

// The slow way for a chunk with NaN or an infinity in it.
template <typename T>
__device__ __noinline__ float odd_sum(Chunk<T> x, float m, float c) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) all += odd_weight(x.pair(i).x, m, c) + odd_weight(x.pair(i).y, m, c);
    return all;
}

template <typename T, int U>
__device__ __forceinline__ void Soft::add(const Chunk<T> (&x)[U], float c) {
    float top = x[0].top();
#pragma unroll
    for (int u = 1; u < U; ++u) top = fmaxf(top, x[u].top());
    const Top t(fmaxf(m, top), c);
    raise(t, c);
    const float2 c2 = make_float2(c, c), r2 = make_float2(-t.r, -t.r);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) {
        const float2 e = ptx::fma2(x[i >> 2].pair(i & 3), c2, r2);
        sum[i & 1] = ptx::add2(sum[i & 1], make_float2(ptx::ex2(e.x), ptx::ex2(e.y)));
    }
    const float2 both = ptx::add2(sum[0], sum[1]);
    float all = both.x + both.y;
    if (!(all <= 16.f * U)) {
        all = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) all += odd_sum(x[u], t.m, c);
    }
    s += all;
}

// The largest value and its index, the lowest of equal ones: the value's order in the
// upper half of a word, the index from above in the lower (0: none).
__device__ __forceinline__ unsigned long long best_key(float v, int i) {
    const uint32_t u = __float_as_uint(v + 0.f);  // (-0 is 0)
    const uint32_t order = u & 0x80000000u ? ~u : u | 0x80000000u;
    return i < 0 ? 0ull : (unsigned long long)order << 32 | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ int best_index(unsigned long long k) {
    return k == 0 ? -1 : (int)(0xffffffffu - (uint32_t)k);
}

struct Shared {
    float4 warp[WARPS];
    float4 slot[2][MAX_CLUSTER];  // what each CTA of the cluster has, for even and odd exchanges
    int parent[ATTN_TREE_MAX], token[ATTN_TREE_MAX], path[ATTN_TREE_MAX];
    float u[ATTN_TREE_MAX], px[ATTN_TREE_MAX], qx[ATTN_TREE_MAX];
    float4 stat[ATTN_TREE_MAX];     // rows that were summed up ahead: maximum and sum of target and draft
    float inv_left[ATTN_TREE_MAX];  // 1 / what was left after each rejected sibling (0: nothing, p stays)
};

// Hands this CTA's number to the whole cluster and gives back everyone's.  The other
// parity's slots may still be read by a CTA that is behind; these may not: it passed
// the barrier of the exchange between.
__device__ __forceinline__ const float4 *exchange(Shared &sh, int &turn, uint32_t ctas, uint32_t rank, float4 mine) {
    float4 *slots = sh.slot[turn & 1];
    if (threadIdx.x < ctas) ptx::cluster_store(slots + rank, threadIdx.x, mine);
    ptx::cluster_sync();
    ++turn;
    return slots;
}

// The sums of a set of threads' weights in two rows, each relative to its own maximum,
// relative to the common ones: the maxima first, then one step each for the sums.
__device__ __forceinline__ float4 warp_soft(float4 x, float c) {
    float mp = x.x, mq = x.z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        mp = fmaxf(mp, __shfl_xor_sync(ALL, mp, o));
        mq = fmaxf(mq, __shfl_xor_sync(ALL, mq, o));
    }
    const Top p(mp, c), q(mq, c);
    float fp = p.step(x.x, c), fq = q.step(x.z, c);
    if (!(Top::is_weight(fp) && Top::is_weight(fq))) {
        fp = odd_step(x.x, mp, c);
        fq = odd_step(x.z, mq, c);
    }
    x = make_float4(mp, x.y * fp, mq, x.w * fq);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x.y += __shfl_xor_sync(ALL, x.y, o);
        x.w += __shfl_xor_sync(ALL, x.w, o);
    }
    return x;
}

// Numbers of all threads joined over each warp, the CTA and the cluster, always in the
// same order, so that every thread of the cluster has the same result.
struct Cluster {
    Shared &sh;
    uint32_t ctas, rank;
    int turn = 0;

    // After a warp's part is in x (in lane 0 at least): join(x) over the warps' parts in a
    // warp's first lanes.
    template <typename Join>
    __device__ __forceinline__ const float4 *share(float4 x, float4 none, Join join) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) sh.warp[threadIdx.x >> 5] = x;
        __syncthreads();
        if (threadIdx.x < 32) {
            x = lane < WARPS ? sh.warp[lane] : none;
            x = join(x);
        }
        return exchange(sh, turn, ctas, rank, x);
    }
    __device__ __forceinline__ void soft(Soft &p, Soft &q, float c) {
        float4 x = make_float4(p.m, p.s, q.m, q.s);
        x = warp_soft(x, c);
        const float4 *slots = share(x, make_float4(-INFINITY, 0.f, -INFINITY, 0.f), [c](float4 y) {
            return warp_soft(y, c);
        });
        const uint32_t lane = threadIdx.x & 31;
        x = warp_soft(lane < ctas ? slots[lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f), c);
        p.m = x.x, p.s = x.y, q.m = x.z, q.s = x.w;
    }
    __device__ __forceinline__ float sum(float v) {
        const auto over_warp = [](float4 x) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x.x += __shfl_xor_sync(ALL, x.x, o);
            return x;
        };
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 *slots = share(over_warp(make_float4(v, 0.f, 0.f, 0.f)), none, over_warp);
        float r = 0.f;
        for (uint32_t i = 0; i < ctas; ++i) r += slots[i].x;
        return r;
    }
    // The index that goes with the largest key.
    __device__ __forceinline__ int best(unsigned long long key) {
        const auto pack = [](unsigned long long k) {
            return make_float4(__uint_as_float((uint32_t)(k >> 32)), __uint_as_float((uint32_t)k), 0.f, 0.f);
        };
        const auto unpack = [](float4 x) {
            return (unsigned long long)__float_as_uint(x.x) << 32 | __float_as_uint(x.y);
        };
        const auto over_warp = [&](float4 x) {
            unsigned long long k = unpack(x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(ALL, k, o));
            return pack(k);
        };
        const float4 *slots = share(over_warp(pack(key)), pack(0), over_warp);
        unsigned long long r = 0;
        for (uint32_t i = 0; i < ctas; ++i) r = max(r, unpack(slots[i]));
        return best_index(r);
    }
};

// A slice [lo, hi) of a row of the vocabulary, or of two of the same type (b may be
// nullptr), in chunks of eight that begin on a's 16-byte boundaries, for NT threads.  Fewer
// than eight elements before the first and behind the last come by themselves.
template <typename T, int NT>
struct Slice {
    const T *a, *b;
    int lo, hi, first, chunks;
    bool vec;

    __device__ __forceinline__ Slice(const T *a_, const T *b_, int lo_, int hi_) : a(a_), b(b_), lo(lo_), hi(hi_) {
        const int head = (int)((-(reinterpret_cast<uintptr_t>(a + lo) / sizeof(T))) % (16 / sizeof(T)));
        first = lo + min(hi - lo, head);
        chunks = (hi - first) / 8;
        vec = b == nullptr || vec_ok(b + first);
    }
    // This thread's part, in ascending order: many(first element, chunks of a, of b, of e),
    // U chunks NT apart at a time (those behind the end hold -inf), one(element) for the
    // others.  The next DEPTH times' chunks are loaded before they are used; the loop stays
    // rolled, its code is fetched once.
    template <int U, int DEPTH, bool E, typename Many, typename One>
    __device__ __forceinline__ void each(const float *e, Many many, One one) const {
        const int tail = first + chunks * 8;
        const bool evec = E && vec_ok(e + first);
        if (lo + (int)threadIdx.x < first) one(lo + (int)threadIdx.x);
        Chunk<T> x[DEPTH + 1][U], y[DEPTH + 1][U];
        Chunk<float> z[DEPTH + 1][U];
        const auto fetch = [&](int d, int k0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * NT;
                if (k < chunks) {
                    const int at = first + k * 8;
                    x[d][u].load(a + at, true);
                    if (b != nullptr) y[d][u].load(b + at, vec);
                    if (E) z[d][u].load(e + at, evec);
                } else if (U > 1) {
                    x[d][u].none();
                    y[d][u].none();
                    if (E) z[d][u].none();
                }
            }
        };
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) fetch(d, threadIdx.x + d * U * NT);
#pragma unroll 1
        for (int k = threadIdx.x; k < chunks; k += U * NT) {
            fetch(DEPTH, k + DEPTH * U * NT);
            many(first + k * 8, x[0], y[0], z[0]);
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[d][u] = x[d + 1][u];
                    y[d][u] = y[d + 1][u];
                    if (E) z[d][u] = z[d + 1][u];
                }
        }
        if (tail + (int)threadIdx.x < hi) one(tail + (int)threadIdx.x);
    }
    // The thread to whose part the element belongs (-1: none of this slice's).
    __device__ __forceinline__ int owner(int at) const {
        const int tail = first + chunks * 8;
        if (at < lo || at >= hi) return -1;
        return at < first ? at - lo : at >= tail ? at - tail : (at - first) / 8 % NT;
    }
    // Brings it into L2, a line a thread at a time.
    static __device__ __forceinline__ void prefetch(const void *row, int lo, int hi, int size) {
        const char *p = static_cast<const char *>(row) + (int64_t)lo * size;
        const uint32_t bytes = (uint32_t)(hi - lo) * (uint32_t)size;  // (a row has 2^28 elements at most)
        for (uint32_t i = threadIdx.x * 128; i < bytes; i += NT * 128) ptx::prefetch_l2(p + i);
    }
};

// What a thread's part of a row's slice comes to: the largest logit's key where nothing
// is drawn, else maximum and sum.
template <int DEPTH, typename T, int NT>
__device__ __forceinline__ unsigned long long slice_best(const Slice<T, NT> &sl) {
    float top = -INFINITY;
    int where = -1;
    const auto take = [&](float v, int i) {
        if (v > top) {
            top = v;
            where = i;
        }
    };
    sl.template each<1, DEPTH, false>(
        nullptr,
        [&](int at, const Chunk<T>(&chunk)[1], const Chunk<T>(&)[1], const Chunk<float>(&)[1]) {
            const Chunk<T> &x = chunk[0];
            if (x.top() > top) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = x.pair(i);
                    take(v.x, at + 2 * i);
                    take(v.y, at + 2 * i + 1);
                }
            }
        },
        [&](int at) { take(value(sl.a[at]), at); });
    return best_key(top, where);
}
template <int U, int DEPTH, typename T, int NT>
__device__ __forceinline__ void slice_soft(const Slice<T, NT> &sl, Soft &p, Soft &q, float c) {
    sl.template each<U, DEPTH, false>(
        nullptr,
        [&](int, const Chunk<T>(&x)[U], const Chunk<T>(&y)[U], const Chunk<float>(&)[U]) {
            p.add(x, c);
            if (sl.b != nullptr) q.add(y, c);
        },
        [&](int at) {
            p.add(value(sl.a[at]), c);
            if (sl.b != nullptr) q.add(value(sl.b[at]), c);
        });
}

// A sequence's rows, and how its temperature is taken.
struct Sequence {
    int begin, n;
    bool bad, draws;
    float c;
    __device__ __forceinline__ Sequence(const VerifyParams &p, int b) {
        begin = p.cu[b];
        const int end = p.cu[b + 1];
        bad = begin < 0 || end < begin || end > p.total || end - begin > p.width;
        n = bad ? 0 : end - begin;
        const float temp = p.temperature != nullptr ? p.temperature[b] : 0.f;
        draws = temp > 0.f;  // (NaN: no)
        // (bounded: the largest logit's 0 times it has to be 0)
        c = draws ? fminf(1.4426950408889634f / temp, 1e30f) : 0.f;
    }
};

// Sums a slice of a row up for the walk.
template <typename T>
__device__ __forceinline__ void sum_slice(const VerifyParams &p, const Sequence &seq, int kind, int i, int piece,
                                          float4 (&warp)[SUM_THREADS / 32]) {
    constexpr int W = SUM_THREADS / 32;
    const int64_t row = seq.begin + i;
    const T *data = kind == 0 ? static_cast<const T *>(p.logits) + row * p.logits_stride
                              : static_cast<const T *>(p.draft) + row * p.draft_stride;
    const int lo = piece * p.piece, hi = min(p.V, lo + p.piece), lane = threadIdx.x & 31;
    const Slice<T, SUM_THREADS> sl(data, nullptr, lo, hi);
    float2 *out = p.sums + ((int64_t)kind * p.total + row) * p.pieces + piece;
    if (!seq.draws) {
        auto *keys = reinterpret_cast<unsigned long long *>(warp);
        unsigned long long k = slice_best<3>(sl);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(ALL, k, o));
        if (lane == 0) keys[threadIdx.x >> 5] = k;
        __syncthreads();
        if (threadIdx.x != 0) return;
#pragma unroll
        for (int j = 1; j < W; ++j) k = max(k, keys[j]);
        *reinterpret_cast<unsigned long long *>(out) = k;
        return;
    }
    Soft sp, none;
    slice_soft<4, 0>(sl, sp, none, seq.c);
    float4 v = make_float4(sp.m, sp.s, -INFINITY, 0.f);
    v = warp_soft(v, seq.c);
    if (lane == 0) warp[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x != 0) return;
    Soft all;
#pragma unroll
    for (int j = 0; j < W; ++j) all.add(warp[j].x, warp[j].y, seq.c);
    *out = make_float2(all.m, all.s);
}

// Sums all rows up ahead of the walk: a CTA a slice of a row (blockIdx.x: sequence, node,
// target or draft, slice).  Few threads with many elements each: what a thread does besides
// its elements (its row, the joining of sums) is worth a hundred.  MANY: `nodes` nodes of a
// sequence at once, and a CTA takes every so manyth (a form of its own: the loop takes
// registers, and a tenth of the time, from the other).
template <typename T, bool MANY>
__global__ void __launch_bounds__(SUM_THREADS) sums_kernel(const VerifyParams p, int nodes) {
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    __shared__ float4 warp[SUM_THREADS / 32];
    const unsigned kinds = p.draft != nullptr ? 2 : 1;
    const unsigned row_x = blockIdx.x / (unsigned)p.pieces, piece = blockIdx.x - row_x * (unsigned)p.pieces;
    const unsigned node = row_x / kinds, kind = row_x - node * kinds;
    const unsigned b = node / (unsigned)nodes;
    const Sequence seq(p, b);
    int i = (int)(node - b * (unsigned)nodes);
    if (i >= seq.n || (kind == 1 && !seq.draws)) return;
    sum_slice<T>(p, seq, kind, i, piece, warp);
    while (MANY && (i += nodes) < seq.n) {
        __syncthreads();  // (the row before has been joined)
        sum_slice<T>(p, seq, kind, i, piece, warp);
    }
}

// What is left of p where `stages` siblings were rejected, one after the other: p - q, no
// less than 0, times 1 / the sum of that (0: nothing was left, p stays); the sum of the last
// stage is open where stages > known, which the race does not mind.
__device__ __forceinline__ float rest(float pw, float qw, int stages, int known, const float *inv_left) {
    for (int k = 0; k < stages; ++k) {
        const float t = fmaxf(pw - qw, 0.f);
        if (k == known)
            pw = t;
        else if (inv_left[k] > 0.f)
            pw = t * inv_left[k];
    }
    return pw;
}

// The two distributions at a node, from the rows' maxima and sums.
struct Node {
    Top tp, tq;
    float ip, iq, c;
    bool plain;  // weights that are plain numbers need no second look (see Top)
    __device__ __forceinline__ Node(const Soft &p, const Soft &q, float c_)
        : tp(p.m, c_), tq(q.m, c_), ip(p.s > 0.f ? 1.f / p.s : 0.f), iq(q.s > 0.f ? 1.f / q.s : 0.f), c(c_) {
        plain = tp.m < FLT_MAX && tp.r == tp.r && tq.m < FLT_MAX && tq.r == tq.r;
    }
    // The weights of a token in plain rows (q's of a NaN: 0), and p - q.
    __device__ __forceinline__ float2 weights(float x, float y) const {
        const float q = ptx::ex2(fmaf(y, c, -tq.r));
        return make_float2(ptx::ex2(fmaf(x, c, -tp.r)), q <= 2.f ? q : 0.f);
    }
    __device__ __forceinline__ float difference(float x, float y) const {
        const float2 w = weights(x, y);
        return fmaf(w.x, ip, -w.y * iq);
    }
};

// The general case of what is left of a token's p, for a node's rows of any numbers.
__device__ __noinline__ float odd_rest(float x, float y, float pm, float qm, float ip, float iq, float c, int stages,
                                       int known, const float *inv_left) {
    const float w = odd_weight(x, pm, c);
    return stages == 0 ? w : rest(w * ip, odd_weight(y, qm, c) * iq, stages, known, inv_left);
}

// A token's p and q from its logits and the rows' maxima and sums (0 where there is none).
__device__ __forceinline__ void child_probability(float4 x, float c, float &p, float &q) {
    p = x.y > 0.f ? Top(x.x, c).weight(p, c) / x.y : 0.f;
    q = x.w > 0.f ? Top(x.z, c).weight(q, c) / x.w : 0.f;
}

// Where a sequence's walk has ended: what the race for its last token needs.
struct WalkEnd {
    int row;               // of logits (and draft); -1: nothing is drawn
    int place;             // of the token in out_tokens
    int rejected, known;   // children, and how many of them are in inv_left
    float pm, ps, qm, qs;  // the rows' maxima and sums
    float c;
    unsigned done;              // CTAs of the race that have arrived
    unsigned long long best;    // the largest key so far
};
static_assert(sizeof(WalkEnd) <= WALK_END_BYTES, "a sequence's place in the workspace");

// The walk down a sequence's tree, a cluster of CTAs each.  AHEAD: the rows' sums are there.
// KEEP: p and q of the slice's tokens stay in shared memory while a node's children are
// rejected one after another (there is room for them, keep_bytes).
template <typename T, bool AHEAD, bool KEEP>
__global__ void __launch_bounds__(THREADS, 1) verify_kernel(const VerifyParams p, int slice) {
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    ptx::cluster_arrive();
    using Part = Slice<T, THREADS>;
    __shared__ Shared sh;
    extern __shared__ float2 kept[];  // [place][THREADS]: p and q of this thread's tokens at a node
    const int tid = threadIdx.x;
    const uint32_t rank = ptx::cluster_rank(), ctas = (uint32_t)((p.V + slice - 1) / slice);
    const int b = blockIdx.x / ctas;
    const int lo = (int)rank * slice, hi = min(p.V, lo + slice);
    const Sequence seq(p, b);
    const int begin = seq.begin, n = seq.n;
    if (seq.bad && rank == 0 && tid == 0) report_status(p.status, kStatusDeviceBounds, kSiteVerifyOffsets);
    int32_t *path_out = p.path + (int64_t)b * p.width, *tokens_out = p.out_tokens + (int64_t)b * p.width;
    WalkEnd *walk_end = p.ends != nullptr ? reinterpret_cast<WalkEnd *>(p.ends + (int64_t)b * WALK_END_BYTES) : nullptr;
    ptx::cluster_wait();  // every CTA of the cluster runs: its shared memory may be written
    if (n == 0) {         // (the same in every CTA of the cluster)
        if (rank == 0) {
            for (int j = tid; j < p.width; j += THREADS) path_out[j] = tokens_out[j] = -1;
            if (tid == 0) p.counts[b] = 0;
            if (tid == 0 && walk_end != nullptr) walk_end->row = -1;
        }
        return;
    }
    const bool draws = seq.draws;
    const float c = seq.c;
    const T *logits = static_cast<const T *>(p.logits) + begin * p.logits_stride;
    const T *draft = draws && p.draft != nullptr ? static_cast<const T *>(p.draft) + begin * p.draft_stride : nullptr;
    // (the race reads it, whatever is accepted)
    if (draws) Part::prefetch(p.noise + (int64_t)b * p.noise_stride, lo, hi, sizeof(float));
    for (int i = tid; i < n; i += THREADS) {
        int up = p.parents[begin + i], token = p.tokens[begin + i];
        if (up < -1 || up >= i) {
            if (rank == 0) report_status(p.status, kStatusDeviceBounds, kSiteTreeParent);
            up = -1;
        }
        if (i > 0 && (token < 0 || token >= p.V)) {
            if (rank == 0) report_status(p.status, kStatusDeviceBounds, kSiteVerifyToken);
            token = -1;
        }
        sh.parent[i] = up;
        sh.token[i] = token;
        sh.u[i] = draws ? p.uniforms[begin + i] : 0.f;
        if (AHEAD && draws) {  // its logits in its parent's row
            const bool there = up >= 0 && token >= 0;
            sh.px[i] = there ? value(logits[up * p.logits_stride + token]) : -INFINITY;
            sh.qx[i] = there && draft != nullptr ? value(draft[up * p.draft_stride + token]) : -INFINITY;
        }
    }
    if (AHEAD) {
        // The rows' sums, a row a warp and a piece a lane.
        const int lane = tid & 31;
        for (int i = tid >> 5; i < n; i += WARPS) {
            if (draws) {
                const float2 *part = p.sums + (int64_t)(begin + i) * p.pieces;
                const float2 *dpart = part + (int64_t)p.total * p.pieces;
                Soft a, d;
                for (int k = lane; k < p.pieces; k += 32) {
                    a.add(part[k].x, part[k].y, c);
                    if (draft != nullptr) d.add(dpart[k].x, dpart[k].y, c);
                }
                float4 x = make_float4(a.m, a.s, d.m, d.s);
                x = warp_soft(x, c);
                if (lane == 0) sh.stat[i] = x;
            } else {
                const auto *part = reinterpret_cast<const unsigned long long *>(p.sums) + (int64_t)(begin + i) * p.pieces;
                unsigned long long k = 0;
                for (int j = lane; j < p.pieces; j += 32) k = max(k, part[j]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(ALL, k, o));
                if (lane == 0) sh.stat[i].x = __int_as_float(best_index(k));
            }
        }
        __syncthreads();
        for (int i = tid; draws && i < n; i += THREADS) {
            // A child's probabilities at its parent.
            const float4 x = sh.stat[max(sh.parent[i], 0)];
            child_probability(x, c, sh.px[i], sh.qx[i]);
        }
    }
    __syncthreads();

    Cluster all{sh, ctas, rank};
    int cur = 0, count = 1, last = -1, rejected = 0, known = 0;
    Soft sp, sq;
    for (;;) {
        const T *row = logits + cur * p.logits_stride;
        const T *drow = draft != nullptr ? draft + cur * p.draft_stride : nullptr;
        int next = -1;
        // The node's children in order: f(child) says whether it is accepted.  (No thread
        // writes to shared memory what another reads here without a barrier: a warp may
        // be a node ahead of another.)
        auto each_child = [&](auto f) {
            for (int i0 = (cur + 1) & ~31; i0 < n && next < 0; i0 += 32) {
                const int i = i0 + (tid & 31);
                for (unsigned m = __ballot_sync(ALL, i > cur && i < n && sh.parent[i < n ? i : 0] == cur); m != 0 && next < 0;
                     m &= m - 1) {
                    const int k = i0 + __ffs(m) - 1;
                    if (f(k)) next = k;
                }
            }
        };
        if (!draws) {
            if (AHEAD) {
                last = __float_as_int(sh.stat[cur].x);
            } else {
                Part::prefetch(row, lo, hi, sizeof(T));
                last = all.best(slice_best<0>(Part(row, nullptr, lo, hi)));
            }
            if (last >= 0) each_child([&](int k) { return sh.token[k] == last; });
        } else {
            const Part rows(row, drow, lo, hi);
            sp = sq = Soft();
            if (AHEAD) {
                const float4 st = sh.stat[cur];
                sp.m = st.x, sp.s = st.y, sq.m = st.z, sq.s = st.w;
            } else {
                Part::prefetch(row, lo, hi, sizeof(T));
                if (drow != nullptr) Part::prefetch(drow, lo, hi, sizeof(T));
                // The children's own logits, on their way during the pass.
                float px = -INFINITY, qx = -INFINITY;
                const bool child = tid < n && tid > cur && sh.parent[tid] == cur && sh.token[tid] >= 0;
                if (child) {
                    px = value(row[sh.token[tid]]);
                    if (drow != nullptr) qx = value(drow[sh.token[tid]]);
                }
                slice_soft<1, 0>(rows, sp, sq, c);
                all.soft(sp, sq, c);
                if (child) {
                    child_probability(make_float4(sp.m, sp.s, sq.m, sq.s), c, px, qx);
                    sh.px[tid] = px;
                    sh.qx[tid] = qx;
                }
                __syncthreads();
            }
            rejected = known = 0;
            int places = 0;    // tokens of this thread's in `kept`
            float left = 1.f;  // without draft: what is left of p
            each_child([&](int k) {
                const int token = sh.token[k];
                const float w = token >= 0 ? sh.px[k] : 0.f;
                if (draft == nullptr) {
                    bool again = false;  // the token of an earlier sibling, which has been rejected
                    if (rejected > 0)
                        for (int i0 = cur + 1; i0 < k; i0 += 32) {
                            const int i = i0 + (tid & 31);
                            again = again || __any_sync(ALL, i < k && sh.parent[i < k ? i : 0] == cur &&
                                                                 sh.token[i < k ? i : 0] == token);
                        }
                    const float mine = again ? 0.f : w;
                    if (sh.u[k] * left < mine) return true;
                    left = fmaxf(left - mine, 0.f);
                } else {
                    if (rejected > known) {  // the sum that the last rejection left
                        float sum = 0.f;
                        if (KEEP && known > 0) {
                            // (step by step what rest() does)
                            const float inv = sh.inv_left[known - 1];
                            for (int i = 0; i < places; ++i) {
                                float2 x = kept[i * THREADS + tid];
                                if (inv > 0.f) x.x = fmaxf(x.x - x.y, 0.f) * inv;
                                kept[i * THREADS + tid] = x;
                                sum += fmaxf(x.x - x.y, 0.f);
                            }
                        } else {
                            const Node node(sp, sq, c);
                            const bool simple = node.plain && rejected == 1;
                            const auto add = [&](float x, float y) {
                                if (KEEP) {
                                    const float2 w = simple ? node.weights(x, y)
                                                            : make_float2(odd_weight(x, sp.m, c), odd_weight(y, sq.m, c));
                                    const float2 pq = make_float2(w.x * node.ip, w.y * node.iq);
                                    kept[places++ * THREADS + tid] = pq;
                                    sum += fmaxf(pq.x - pq.y, 0.f);
                                } else {
                                    sum += simple ? fmaxf(node.difference(x, y), 0.f)
                                                  : odd_rest(x, y, sp.m, sq.m, node.ip, node.iq, c, rejected, known,
                                                             sh.inv_left);
                                }
                            };
                            rows.template each<1, 0, false>(
                                nullptr,
                                [&](int, const Chunk<T>(&x)[1], const Chunk<T>(&y)[1], const Chunk<float>(&)[1]) {
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float2 v = x[0].pair(i), q = y[0].pair(i);
                                        add(v.x, q.x);
                                        add(v.y, q.y);
                                    }
                                },
                                [&](int at) { add(value(row[at]), value(drow[at])); });
                        }
                        const float z = all.sum(sum);
                        if (tid == 0) sh.inv_left[known] = z > 0.f ? 1.f / z : 0.f;
                        __syncthreads();
                        ++known;
                    }
                    const float q = token >= 0 ? sh.qx[k] : 0.f;
                    if (sh.u[k] * q < rest(w, q, rejected, known, sh.inv_left)) return true;
                }
                ++rejected;
                return false;
            });
        }
        if (next < 0) break;
        if (tid == 0) sh.path[count] = next;
        ++count;
        cur = next;
    }
    // (No CTA writes into another's shared memory once that has left: the last exchange's
    // barrier was behind its stores.)
    __syncthreads();
    if (rank != 0) return;
    for (int j = tid; j < p.width; j += THREADS) {
        path_out[j] = j == 0 ? 0 : j < count ? sh.path[j] : -1;
        tokens_out[j] = j < count - 1 ? sh.token[sh.path[j + 1]] : j == count - 1 ? last : -1;
    }
    if (tid == 0) p.counts[b] = count;
    if (walk_end == nullptr) return;
    if (tid == 0)
        *walk_end = WalkEnd{draws ? begin + cur : -1, count - 1, rejected, known, sp.m, sp.s, sq.m, sq.s, c, 0u, 0ull};
    // The rejected children's tokens are out of the race (without draft), or the sums that
    // their rejections left.
    if (draws && rejected > 0) {
        auto *list = reinterpret_cast<float *>(p.ends + (int64_t)p.B * WALK_END_BYTES) + (int64_t)b * p.width;
        if (draft != nullptr) {
            for (int k = tid; k < known; k += THREADS) list[k] = sh.inv_left[k];
        } else if (tid < 32) {
            int k = 0;
            for (int i0 = (cur + 1) & ~31; i0 < n; i0 += 32) {
                const int i = i0 + tid;
                const bool mine = i > cur && i < n && sh.parent[i < n ? i : 0] == cur;
                const unsigned m = __ballot_sync(ALL, mine);
                if (mine) list[k + __popc(m & ((1u << tid) - 1u))] = __int_as_float(sh.token[i]);
                k += __popc(m);
            }
        }
    }
}

// The race for the last tokens: argmax of what is left of p over the noise.  A CTA a slice
// of a sequence's vocabulary; the largest key of all slices is found with atomics, whose
// order changes nothing in it, and the CTA that comes last writes the token.
template <typename T>
__global__ void __launch_bounds__(RACE_THREADS, RACE_BLOCKS) race_kernel(const VerifyParams p, int slice, int slices) {
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    constexpr int W = RACE_THREADS / 32;
    __shared__ unsigned long long keys[W];
    __shared__ float list[ATTN_TREE_MAX];  // the rejected tokens, or inv_left
    __shared__ int final;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / slices, piece = blockIdx.x - b * slices;
    WalkEnd *walk_end = reinterpret_cast<WalkEnd *>(p.ends + (int64_t)b * WALK_END_BYTES);
    const int at_row = walk_end->row;
    if (at_row < 0) return;
    const int place = walk_end->place, known = walk_end->known;
    int rejected = walk_end->rejected;
    Soft sp, sq;
    sp.m = walk_end->pm, sp.s = walk_end->ps, sq.m = walk_end->qm, sq.s = walk_end->qs;
    const float c = walk_end->c;
    const Node node(sp, sq, c);
    const T *row = static_cast<const T *>(p.logits) + at_row * p.logits_stride;
    const T *drow = p.draft != nullptr ? static_cast<const T *>(p.draft) + at_row * p.draft_stride : nullptr;
    const float *noise = p.noise + (int64_t)b * p.noise_stride;
    const bool drafted = p.draft != nullptr;
    {
        const auto *from = reinterpret_cast<const float *>(p.ends + (int64_t)p.B * WALK_END_BYTES) + (int64_t)b * p.width;
        for (int k = tid; k < (drafted ? known : rejected); k += RACE_THREADS) list[k] = from[k];
    }
    __syncthreads();
    int lo = piece * slice, hi = min(p.V, lo + slice);
    for (int attempt = 0;; ++attempt) {
        const bool subtract = drafted && rejected > 0;
        const Slice<T, RACE_THREADS> race(row, subtract ? drow : nullptr, lo, hi);
        // Without draft the rejected tokens, all the node's children's, are out: only the
        // threads that come to one look out for them.
        const int outs = drafted ? 0 : rejected;
        bool watch = false;
        for (int k = 0; k < outs; ++k) watch = watch || race.owner(__float_as_int(list[k])) == tid;
        float top = 0.f;
        int where = -1;
        const auto take = [&](float w, float e, int i) {
            const float v = w * ptx::rcp(e);
            // (no NaN: of 0 times infinity, or e's; e of 0 gives infinity, and where what is left
            // may be below 0, e below 0 a number above)
            if (v > top && e > 0.f) {
                bool out = false;
                if (watch)
                    for (int k = 0; k < outs; ++k) out = out || __float_as_int(list[k]) == i;
                if (!out) {
                    top = v;
                    where = i;
                }
            }
        };
        const auto run = [&](auto weight_of) {
            race.template each<1, 0, true>(
                noise,
                [&](int at, const Chunk<T>(&x)[1], const Chunk<T>(&y)[1], const Chunk<float>(&z)[1]) {
                    const Chunk<float> &e = z[0];
                    float w[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = x[0].pair(i), q = y[0].pair(i);
                        w[2 * i] = weight_of(v.x, q.x);
                        w[2 * i + 1] = weight_of(v.y, q.y);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) take(w[i], i & 1 ? e.pair(i >> 1).y : e.pair(i >> 1).x, at + i);
                },
                [&](int at) { take(weight_of(value(row[at]), subtract ? value(drow[at]) : 0.f), noise[at], at); });
        };
        if (node.plain && !subtract)
            run([&](float x, float) { return ptx::ex2(fmaf(x, c, -node.tp.r)); });
        else if (node.plain && rejected == 1 && known == 0)
            run([&](float x, float y) { return node.difference(x, y); });
        else
            run([&](float x, float y) {
                return odd_rest(x, y, sp.m, sq.m, node.ip, node.iq, c, subtract ? rejected : 0, known, list);
            });
        unsigned long long key = best_key(top, where);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(ALL, key, o));
        if ((tid & 31) == 0) keys[tid >> 5] = key;
        __syncthreads();
        if (tid == 0) {
#pragma unroll
            for (int k = 1; k < W; ++k) key = max(key, keys[k]);
            if (attempt == 0) {
                atomicMax(&walk_end->best, key);
                __threadfence();
                final = atomicAdd(&walk_end->done, 1u) == (unsigned)slices - 1;
                __threadfence();
                key = atomicMax(&walk_end->best, 0ull);
            }
            // Where the last rejection left nothing, of what was left before it (without
            // draft: of all tokens), the last CTA by itself: it takes rounding, or numbers
            // not below 1, to get here.
            if (final && (key != 0 || rejected == 0 || attempt > 0)) {
                p.out_tokens[(int64_t)b * p.width + place] = best_index(key);
                final = 0;
            }
        }
        __syncthreads();
        if (!final) return;
        rejected = drafted ? known : 0;
        lo = 0;
        hi = p.V;
    }
}

// The shared memory for a slice's p and q at a node: a thread has its chunks of eight, and two
// tokens at the ends.  With it (slices of up to KEEP_TOKENS) every sum after a node's first
// needs no row and no exponential: rows of 131072 tokens, drawn trees of 40 to 64 rows, 16 of
// them 62 us instead of 99; 32 of 8 to 16 rows of 32000 tokens 34 instead of 39.  Without it
// the rows are read again for every sum, from L2.
int64_t keep_bytes(int slice) {
    return (((slice + 7) / 8 + THREADS - 1) / THREADS * 8 + 2) * (int64_t)(THREADS * sizeof(float2));
}
constexpr int KEEP_TOKENS = 24576;
constexpr int KEEP_MOST = (KEEP_TOKENS / 8 / THREADS * 8 + 2) * THREADS * (int)sizeof(float2);
static_assert(KEEP_MOST + sizeof(Shared) <= 227 * 1024, "shared memory of a CTA");

template <typename T>
cudaError_t launch(const VerifyParams &p, cudaStream_t stream) {
    if (p.pieces > 0) {
        // Nodes of a sequence at once: as many as make 8192 blocks.  Under a bound that few
        // trees come near, most of the blocks would find nothing to do: 64 trees of 1 to 8
        // rows under a bound of 256 took 116 us with a block for every row, 28 like this.
        const int64_t each = (int64_t)p.B * (p.draft != nullptr ? 2 : 1) * p.pieces;
        const int nodes = (int)std::min<int64_t>(p.width, std::max<int64_t>(16, 8192 / each));
        const int64_t blocks = (int64_t)p.B * nodes * (p.draft != nullptr ? 2 : 1) * p.pieces;
        const cudaError_t e = launch_dependent(p.width > nodes ? sums_kernel<T, true> : sums_kernel<T, false>,
                                               dim3((unsigned)blocks), dim3(SUM_THREADS), 0, stream, p, nodes);
        if (e != cudaSuccess) return e;
    }
    // CTAs a sequence, with slices of 4096 tokens at least.  Walks that sum rows up: all eight as
    // long as they run at once; with more sequences a second wave of CTAs evens their lengths
    // out (131072 tokens, 40 rows: 64 sequences 58 us with four, 83 with the two that run at
    // once, 45 46 us with six, 50 with three; 25 36 us with six, 42 with eight).  Rows summed up
    // ahead: what a walk reads are the rows of rejected drawn children, most quickly in slices
    // that shared memory keeps (32000 tokens, 128 sequences of 8 rows: 76 us with two, 113 with
    // one, but chains of 131072, 100 of 5 rows, 85 against 79); a walk without temperature reads
    // nothing and needs one (16 of 5 rows 8.4 us, 10.2 with eight).  Up to eight sequences take
    // eight, more six (16 chains of 5 rows 26 us, 30 with eight).
    const int per = 152 / p.B;
    int want;
    if (p.pieces == 0) {
        want = per >= MAX_CLUSTER ? MAX_CLUSTER : std::min({6, 304 / p.B, (p.V + 8191) / 8192});
    } else if (p.draft != nullptr) {
        const int keeping = (p.V + KEEP_TOKENS - 1) / KEEP_TOKENS;
        want = std::max(keeping <= per ? keeping : 2, std::min(per, p.B > 8 ? 6 : MAX_CLUSTER));
    } else {
        want = p.temperature != nullptr ? per : 1;
    }
    int ctas = std::max(1, std::min({MAX_CLUSTER, (p.V + 4095) / 4096, want}));
    const int slice = ((p.V + ctas - 1) / ctas + 7) & ~7;
    ctas = (p.V + slice - 1) / slice;
    const int64_t bytes = keep_bytes(slice);
    const bool keep = p.draft != nullptr && bytes <= KEEP_MOST;
    const auto kernel = keep ? (p.pieces > 0 ? verify_kernel<T, true, true> : verify_kernel<T, false, true>)
                             : (p.pieces > 0 ? verify_kernel<T, true, false> : verify_kernel<T, false, false>);
    if (keep) {
        static thread_local int configured_device = -1;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && configured_device != dev) {
            for (auto k : {verify_kernel<T, true, true>, verify_kernel<T, false, true>})
                if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, KEEP_MOST);
            if (e == cudaSuccess) configured_device = dev;
        }
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B * ctas);
    cfg.dynamicSmemBytes = keep ? (size_t)bytes : 0;
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, slice);
    if (e != cudaSuccess || p.temperature == nullptr) return e;
    // The race: as many CTAs as all SMs hold at once, a slice of 2048 tokens at least.
    const int64_t each = std::max(1, RACE_BLOCKS * 152 / p.B), even = (p.V + each - 1) / each;
    const int part = (int)((std::min<int64_t>(p.V, std::max<int64_t>(even, 2048)) + 7) & ~(int64_t)7);
    const int slices = (p.V + part - 1) / part;
    return launch_dependent(race_kernel<T>, dim3((unsigned)p.B * slices), dim3(RACE_THREADS), 0, stream, p, part, slices);
}

}  // namespace vf

int verify_piece(int64_t rows, int vocab, int *pieces) {
    // Eight CTAs for every SM where that takes no slice below 4096 tokens, 16384 at most.
    const int64_t most = 16384, even = (rows * vocab + 1215) / 1216;
    int64_t piece = even < 4096 ? 4096 : even > most ? most : even;
    if (piece * 64 < vocab) piece = ((int64_t)vocab + 63) / 64;  // (64 a row at most)
    piece = (piece + 7) & ~(int64_t)7;
    *pieces = (int)((vocab + piece - 1) / piece);
    return (int)piece;
}

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
    return p.fp32 ? vf::launch<float>(p, stream) : vf::launch<__nv_bfloat16>(p, stream);
}

}  // namespace attn
