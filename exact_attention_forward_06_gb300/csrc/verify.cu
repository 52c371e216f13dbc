// verify.cu -- verification of drafted tokens against the target's probabilities
// (attn_verify_tree).
//
// The walk down a sequence's tree is a chain of decisions: node c's row of logits
// gives p = softmax(logits[c] / T), one of c's children is accepted (x its token, u
// its uniform number, q the draft's distribution or 1 for tokens that were not drawn)
//     u q(x) < p(x),  a rejected child leaving  p <- max(p - q, 0) / sum,
// and the walk goes on there, or none is and the last token is drawn from what is
// left of p as argmax_i p_i / e_i: of independent exponential numbers e_i / p_i the
// smallest is that of i with probability p_i.  Only rows on the path are read; the
// other nodes' rows, most of a tree, are not.
//
// A cluster of CTAs works on a sequence, each on a slice of the vocabulary.  A step
// of the walk is one pass over the node's row(s) for the maximum and the sum of the
// exponentials, kept per thread and joined once (the children's own logits are
// fetched meanwhile), an exchange through the cluster's shared memory, and the
// decision, which every thread of every CTA takes by itself from the same numbers
// in the same order.
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

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr unsigned ALL = 0xffffffffu;

// Eight consecutive elements of a row, as they are in memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
        if (vec) {
            w = *reinterpret_cast<const uint4 *>(p);
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
            w = make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                           h[6] | (uint32_t)h[7] << 16);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, bool vec) {
        if (vec) {
            a = reinterpret_cast<const float4 *>(p)[0];
            b = reinterpret_cast<const float4 *>(p)[1];
        } else {
            a = make_float4(p[0], p[1], p[2], p[3]);
            b = make_float4(p[4], p[5], p[6], p[7]);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(float x) { return x; }

__device__ __forceinline__ bool vec_ok(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The weight exp((x - m) / T) of a logit, c = log2 e / T: 0 for NaN and -inf (and where
// m is -inf: nothing is left), 1 for +inf (m is then the largest finite number).  x - m
// is taken before the scaling: with c folded in (one operation less) the rounding of m c
// would go into every weight.
__device__ __forceinline__ float weight(float x, float m, float c) {
    return ptx::ex2(fminf(fmaxf((x - m) * c, -INFINITY), 0.f));
}

// A running maximum and sum of weights.
struct Soft {
    float m = -INFINITY, s = 0.f;
    __device__ __forceinline__ void add(const float (&x)[8], float c) {
        float t = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = fmaxf(t, x[i]);
        t = fminf(t, FLT_MAX);
        if (t > m) {
            s *= weight(m, t, c);
            m = t;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += weight(x[i], m, c);
    }
    __device__ __forceinline__ void join(float m2, float s2, float c) {
        const float t = fmaxf(m, m2);
        s = s * weight(m, t, c) + s2 * weight(m2, t, c);
        m = t;
    }
};

// The largest value and its index, the lowest of equal ones (-1: none).
struct Best {
    float v;
    int i = -1;
    __device__ __forceinline__ void join(float v2, int i2) {
        if (i2 >= 0 && (i < 0 || v2 > v || (v2 == v && i2 < i))) {
            v = v2;
            i = i2;
        }
    }
};

struct Shared {
    float4 warp[WARPS];
    float4 slot[2][MAX_CLUSTER];  // what each CTA of the cluster has, for even and odd exchanges
    int parent[ATTN_TREE_MAX], token[ATTN_TREE_MAX], path[ATTN_TREE_MAX];
    float u[ATTN_TREE_MAX], px[ATTN_TREE_MAX], qx[ATTN_TREE_MAX];
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

// Joins a number over the CTA's threads and then the cluster, always in the same order.
template <typename Join>
__device__ __forceinline__ float4 reduce(Shared &sh, int &turn, uint32_t ctas, uint32_t rank, float4 x, Join join) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float4 y = make_float4(__shfl_xor_sync(ALL, x.x, o), __shfl_xor_sync(ALL, x.y, o),
                                     __shfl_xor_sync(ALL, x.z, o), __shfl_xor_sync(ALL, x.w, o));
        // the lower lane's number first, in both lanes
        x = (threadIdx.x & o) ? join(y, x) : join(x, y);
    }
    if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x < 32) {
        x = sh.warp[threadIdx.x % WARPS];
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1) {
            const float4 y = make_float4(__shfl_xor_sync(ALL, x.x, o), __shfl_xor_sync(ALL, x.y, o),
                                         __shfl_xor_sync(ALL, x.z, o), __shfl_xor_sync(ALL, x.w, o));
            x = (threadIdx.x & o) ? join(y, x) : join(x, y);
        }
    }
    const float4 *slots = exchange(sh, turn, ctas, rank, x);
    float4 r = slots[0];
    for (uint32_t i = 1; i < ctas; ++i) r = join(r, slots[i]);
    return r;
}

// A slice [lo, hi) of a row in chunks of eight that begin on 16-byte boundaries of the
// row, with single elements before and behind: body(first element, count, chunk of a,
// chunk of b), b another row of the same type or nullptr.  A thread's elements come in
// ascending order.
template <typename T, int U, typename Body>
__device__ __forceinline__ void each_chunk(const T *a, const T *b, int lo, int hi, Body body) {
    const int head = min(hi - lo, (int)((-(reinterpret_cast<uintptr_t>(a + lo) / sizeof(T))) % (16 / sizeof(T))));
    const int first = lo + head, chunks = (hi - first) / 8, tail = first + chunks * 8;
    const bool vec = b == nullptr || vec_ok(b + first);
    // fewer than eight before and eight behind
    auto one = [&](int at, bool there) {
        if (!there) return;
        float xs[8], ys[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) xs[i] = ys[i] = -INFINITY;
        xs[0] = value(a[at]);
        if (b != nullptr) ys[0] = value(b[at]);
        body(at, 1, xs, ys);
    };
    one(lo + (int)threadIdx.x, (int)threadIdx.x < head);
    for (int c0 = threadIdx.x; c0 < chunks; c0 += U * THREADS) {
        Chunk<T> x[U], y[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (c0 + i * THREADS < chunks) {
                const int at = first + (c0 + i * THREADS) * 8;
                x[i].load(a + at, true);
                if (b != nullptr) y[i].load(b + at, vec);
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (c0 + i * THREADS < chunks) {
                float xs[8], ys[8];
                x[i].get(xs);
                if (b != nullptr) y[i].get(ys);
                body(first + (c0 + i * THREADS) * 8, 8, xs, ys);
            }
    }
    one(tail + (int)threadIdx.x, (int)threadIdx.x < hi - tail);
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 2) verify_kernel(const VerifyParams p, int slice) {
    ptx::wait_for_prior_work();
    ptx::allow_next_work();
    constexpr int U = sizeof(T) == 2 ? 2 : 1;
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const uint32_t rank = ptx::cluster_rank(), ctas = (uint32_t)((p.V + slice - 1) / slice);
    const int b = blockIdx.x / ctas;
    const int lo = (int)rank * slice, hi = min(p.V, lo + slice);
    const int begin = p.cu[b], end = p.cu[b + 1];
    const bool bad = begin < 0 || end < begin || end > p.total || end - begin > p.width;
    if (bad && rank == 0 && tid == 0) report_status(p.status, kStatusDeviceBounds, kSiteVerifyOffsets);
    const int n = bad ? 0 : end - begin;
    int32_t *path_out = p.path + (int64_t)b * p.width, *tokens_out = p.out_tokens + (int64_t)b * p.width;
    if (n == 0) {  // (the same in every CTA of the cluster)
        if (rank == 0) {
            for (int j = tid; j < p.width; j += THREADS) path_out[j] = tokens_out[j] = -1;
            if (tid == 0) p.counts[b] = 0;
        }
        return;
    }
    const float temp = p.temperature != nullptr ? p.temperature[b] : 0.f;
    const bool draws = temp > 0.f;  // (NaN: no)
    // (bounded: the largest logit's 0 times it has to be 0)
    const float c = draws ? fminf(1.4426950408889634f / temp, 1e30f) : 0.f;
    const T *draft = draws ? static_cast<const T *>(p.draft) : nullptr;
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
    }
    __syncthreads();

    int turn = 0, cur = 0, count = 1, last = -1;
    for (;;) {
        const T *row = static_cast<const T *>(p.logits) + (int64_t)(begin + cur) * p.logits_stride;
        const T *drow = draft != nullptr ? draft + (int64_t)(begin + cur) * p.draft_stride : nullptr;
        // The children's own logits, on their way during the pass.
        float px = -INFINITY, qx = -INFINITY;
        const bool child = tid < n && tid > cur && sh.parent[tid] == cur && sh.token[tid] >= 0;
        if (child && draws) {
            px = value(row[sh.token[tid]]);
            if (drow != nullptr) qx = value(drow[sh.token[tid]]);
        }
        int next = -1;
        // The node's children in order: f(child) says whether it is accepted.
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
            Best best;
            best.v = -INFINITY;
            each_chunk<T, U>(row, static_cast<const T *>(nullptr), lo, hi,
                             [&](int at, int k, const float (&x)[8], const float (&)[8]) {
#pragma unroll
                                 for (int i = 0; i < 8; ++i)
                                     if (x[i] > best.v) {
                                         best.v = x[i];
                                         best.i = at + i;
                                     }
                             });
            const float4 r = reduce(sh, turn, ctas, rank, make_float4(best.v, __int_as_float(best.i), 0.f, 0.f),
                                    [](float4 x, float4 y) {
                                        Best q;
                                        q.v = x.x;
                                        q.i = __float_as_int(x.y);
                                        q.join(y.x, __float_as_int(y.y));
                                        return make_float4(q.v, __int_as_float(q.i), 0.f, 0.f);
                                    });
            last = __float_as_int(r.y);
            if (last >= 0) each_child([&](int k) { return sh.token[k] == last; });
        } else {
            Soft sp, sq;
            each_chunk<T, U>(row, drow, lo, hi, [&](int, int, const float (&x)[8], const float (&y)[8]) {
                sp.add(x, c);
                if (drow != nullptr) sq.add(y, c);
            });
            if (child) {
                sh.px[tid] = px;
                sh.qx[tid] = qx;
            }
            const float4 r = reduce(sh, turn, ctas, rank, make_float4(sp.m, sp.s, sq.m, sq.s), [c](float4 x, float4 y) {
                Soft a, d;
                a.m = x.x, a.s = x.y, d.m = x.z, d.s = x.w;
                a.join(y.x, y.y, c);
                d.join(y.z, y.w, c);
                return make_float4(a.m, a.s, d.m, d.s);
            });
            const float mp = r.x, mq = r.z, ip = r.y > 0.f ? 1.f / r.y : 0.f, iq = r.w > 0.f ? 1.f / r.w : 0.f;
            // Rejected siblings so far, and how many of them are in inv_left.
            int rejected = 0, known = 0;
            float left = r.y;  // without draft: what is left of the weights' sum
            // What is left of p where `stages` siblings are rejected, with the last one's
            // sum still open where stages > known.
            auto rest = [&](float pw, float qw, int stages) {
                for (int k = 0; k < stages; ++k) {
                    const float t = fmaxf(pw - qw, 0.f);
                    if (k == known)
                        pw = t;
                    else if (sh.inv_left[k] > 0.f)
                        pw = t * sh.inv_left[k];
                }
                return pw;
            };
            auto rejected_token = [&](int token) {  // of this node's rejected children: the first `rejected`
                int seen = 0;
                for (int i = cur + 1; i < n && seen < rejected; ++i)
                    if (sh.parent[i] == cur) {
                        ++seen;
                        if (sh.token[i] == token) return true;
                    }
                return false;
            };
            each_child([&](int k) {
                const float w = sh.token[k] >= 0 ? weight(sh.px[k], mp, c) : 0.f;
                if (draft == nullptr) {
                    const float mine = w > 0.f && rejected > 0 && rejected_token(sh.token[k]) ? 0.f : w;
                    if (sh.u[k] * left < mine) return true;
                    left = fmaxf(left - mine, 0.f);
                } else {
                    if (rejected > known) {  // the sum that the last rejection left
                        float sum = 0.f;
                        each_chunk<T, 1>(row, drow, lo, hi, [&](int, int, const float (&x)[8], const float (&y)[8]) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                sum += rest(weight(x[i], mp, c) * ip, weight(y[i], mq, c) * iq, rejected);
                        });
                        const float4 z = reduce(sh, turn, ctas, rank, make_float4(sum, 0.f, 0.f, 0.f),
                                                [](float4 x, float4 y) { return make_float4(x.x + y.x, 0.f, 0.f, 0.f); });
                        if (tid == 0) sh.inv_left[known] = z.x > 0.f ? 1.f / z.x : 0.f;
                        __syncthreads();
                        ++known;
                    }
                    const float q = sh.token[k] >= 0 ? weight(sh.qx[k], mq, c) * iq : 0.f;
                    if (sh.u[k] * q < rest(w * ip, q, rejected)) return true;
                }
                ++rejected;
                return false;
            });
            if (next < 0) {
                // The race.  Where the last rejection left nothing, of what was left before it
                // (without draft: of all tokens).
                const float *noise = p.noise + (int64_t)b * p.noise_stride;
                for (int attempt = 0; attempt < 2; ++attempt) {
                    Best best;
                    best.v = 0.f;
                    const bool subtract = draft != nullptr && rejected > 0;
                    each_chunk<T, 1>(row, subtract ? drow : static_cast<const T *>(nullptr), lo, hi,
                                     [&](int at, int k, const float (&x)[8], const float (&y)[8]) {
                                         Chunk<float> e8;
                                         float e[8];
                                         if (k == 8) {
                                             e8.load(noise + at, vec_ok(noise + at));
                                             e8.get(e);
                                         } else {
                                             e[0] = noise[at];
                                         }
#pragma unroll
                                         for (int i = 0; i < 8; ++i) {
                                             if (i >= k) break;
                                             float w = weight(x[i], mp, c);
                                             if (subtract) w = rest(w * ip, weight(y[i], mq, c) * iq, rejected);
                                             if (!(w > 0.f)) continue;
                                             const float v = __fdividef(w, e[i]);
                                             if (v > best.v && (draft != nullptr || rejected == 0 || !rejected_token(at + i))) {
                                                 best.v = v;
                                                 best.i = at + i;
                                             }
                                         }
                                     });
                    const float4 z = reduce(sh, turn, ctas, rank, make_float4(best.v, __int_as_float(best.i), 0.f, 0.f),
                                            [](float4 x, float4 y) {
                                                Best q;
                                                q.v = x.x;
                                                q.i = __float_as_int(x.y);
                                                q.join(y.x, __float_as_int(y.y));
                                                return make_float4(q.v, __int_as_float(q.i), 0.f, 0.f);
                                            });
                    last = __float_as_int(z.y);
                    if (last >= 0 || rejected == 0) break;
                    rejected = draft != nullptr ? known : 0;
                }
            }
        }
        if (next < 0) break;
        if (tid == 0) sh.path[count] = next;
        ++count;
        cur = next;
    }
    // No CTA may write into another's shared memory once that has left: the last exchange's
    // barrier was behind its stores.
    __syncthreads();
    if (rank != 0) return;
    for (int j = tid; j < p.width; j += THREADS) {
        path_out[j] = j == 0 ? 0 : j < count ? sh.path[j] : -1;
        tokens_out[j] = j < count - 1 ? sh.token[sh.path[j + 1]] : j == count - 1 ? last : -1;
    }
    if (tid == 0) p.counts[b] = count;
}

}  // namespace vf

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
    // CTAs a sequence: as many as keep two on every SM, a slice of 4096 tokens at least.
    int ctas = vf::MAX_CLUSTER;
    while (ctas > 1 && ((int64_t)p.B * ctas > 304 || (int64_t)(ctas - 1) * 4096 >= p.V)) ctas /= 2;
    int slice = ((p.V + ctas - 1) / ctas + 7) & ~7;
    ctas = (p.V + slice - 1) / slice;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B * ctas);
    cfg.blockDim = dim3(vf::THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, p.fp32 ? vf::verify_kernel<float> : vf::verify_kernel<__nv_bfloat16>, p, slice);
}

}  // namespace attn
