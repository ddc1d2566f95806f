// logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logit rows (Module gpu, module sampling: what a sampler
// reads beside the greedy argmax).  Per row x of n logits:
//   m = max x, s = sum e^(x - m), lse = m + log s
//   logprob = x[token] - lse,   entropy = lse - sum p x = log s - t / s,
//   t = sum e^(x - m) (x - m)   (terms of x = -inf count as 0)
//   top: the k largest (ties to the lowest index), as x - lse.
// One pass for (m, s, t) and each thread's largest value; then the k-th
// largest of the 128 quads' maxima bounds the k-th largest logit from below,
// and a second pass over the row (in L2 by then) collects the few values at or
// above that bound, which are ranked by counting.  Where a bound lets too many
// through (long ties, masked rows) the k largest are found one by one.
// HBM-bound on the row: a CTA a row when the rows fill the device; for fewer
// rows a cluster of up to 8 CTAs splits each row and joins through distributed
// shared memory, in one launch.
#include <cooperative_groups.h>

#include "gemv_launch.cuh"
#include "paged.cuh"

namespace q4 {
namespace dev {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 512;
constexpr int kLpQuads = kLpThreads / 4;
constexpr int kLpCand = 1024;  // candidates a CTA holds
constexpr int kLpTop = 32;     // largest k

// Order-preserving key of a logit: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t lp_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return x != x ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float lp_value(uint32_t k) {
    return k == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
// (key, index) as one word: larger value first, then the lower index
__device__ __forceinline__ unsigned long long lp_pair(uint32_t key, int i) {
    return ((unsigned long long)key << 32) | (0xFFFFFFFFu - (uint32_t)i);
}

// The elements [i0, i1) of row x: one(value, index) for those before a 16-byte
// boundary and after the last whole float4, and batch(float4 x 4, index of the
// first, step) for four float4 in flight a thread (their elements start at
// index + q * step); what is left of the vectors goes through one().
template <class One, class Batch>
__device__ __forceinline__ void lp_each(const float *x, int i0, int i1, int tid, One one, Batch batch) {
    const int head = min(i1 - i0, (int)((4u - (((uintptr_t)(x + i0) >> 2) & 3u)) & 3u));
    if (tid < head) one(x[i0 + tid], i0 + tid);
    const int v0 = i0 + head, nv = (i1 - v0) >> 2;
    const float4 *xv = reinterpret_cast<const float4 *>(x + v0);
    int j = tid;
    for (; j + 3 * kLpThreads < nv; j += 4 * kLpThreads) {
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = xv[j + q * kLpThreads];
        batch(v, v0 + 4 * j, 4 * kLpThreads);
    }
    for (; j < nv; j += kLpThreads) {
        const float4 v = xv[j];
        const int i = v0 + 4 * j;
        one(v.x, i);
        one(v.y, i + 1);
        one(v.z, i + 2);
        one(v.w, i + 3);
    }
    const int tail = v0 + 4 * nv + tid;
    if (tail < i1) one(x[tail], tail);
}
__device__ __forceinline__ float lp_at(const float4 &v, int e) { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; }

struct LpSums {
    float m, s, t;
};
__device__ __forceinline__ LpSums lp_join(const LpSums &a, const LpSums &b) {
    const float m = fmaxf(a.m, b.m), mu = m == -INFINITY ? 0.f : m;
    // a share without a finite maximum has nothing to scale; a difference below
    // -200 scales by e^-200 = 0 in fp32, and stays finite (0 * -inf is NaN)
    const float da = a.m == -INFINITY ? 0.f : fmaxf(a.m - mu, -200.f);
    const float db = b.m == -INFINITY ? 0.f : fmaxf(b.m - mu, -200.f);
    const float fa = __expf(da), fb = __expf(db);
    return {m, a.s * fa + b.s * fb, fa * fmaf(da, a.s, a.t) + fb * fmaf(db, b.s, b.t)};
}

constexpr int kLpMaxCluster = 8;

struct LpShared {
    // rank 0 of a cluster receives every CTA's sums and k best pairs (0: none)
    LpSums sums[kLpMaxCluster];
    unsigned long long top[kLpMaxCluster * kLpTop];
    unsigned long long mine[kLpTop];   // this CTA's
    unsigned long long cand[kLpCand];
    LpSums warp[kLpThreads / 32];
    __align__(16) uint32_t quad[kLpQuads];
    unsigned long long best[kLpThreads / 32];
    uint32_t bound;
    int ncand;
};

// v added to the running sums: a new maximum m rescales what came before.
__device__ __forceinline__ void lp_raise(LpSums &a, float m) {
    if (m > a.m) {
        const float d = fmaxf(a.m - m, -200.f), f = __expf(d);  // from -inf: the sums are zero
        a.t = f * fmaf(d, a.s, a.t);
        a.s *= f;
        a.m = m;
    }
}
__device__ __forceinline__ void lp_add(LpSums &a, float v, float mu) {
    const float d = v - mu, e = __expf(d);  // NaN stays; -inf: e = 0, and its term of t is 0
    a.s += e;
    a.t = fmaf(e, fmaxf(d, -200.f), a.t);
}

__global__ void __launch_bounds__(kLpThreads, 2) q4logprobs_kernel(const __grid_constant__ LogprobParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ LpShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int S = (int)cl.num_blocks(), rank = (int)cl.block_rank(), row = blockIdx.x / S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = ((p.n + S - 1) / S + 3) & ~3;
    const int i0 = min(p.n, rank * per), i1 = min(p.n, i0 + per);
    const float *x = p.logits + (size_t)row * p.n;
    const int k = p.k;
    // this CTA runs: the matching wait comes before the writes to rank 0
    if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (tid == 0) sh.ncand = 0;
    if (tid < kLpTop) sh.mine[tid] = 0ull;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    LpSums a = {-INFINITY, 0.f, 0.f};
    uint32_t kmax = 0u;
    lp_each(
        x, i0, i1, tid,
        [&](float v, int) {
            kmax = max(kmax, lp_key(v));
            lp_raise(a, v);
            lp_add(a, v, a.m == -INFINITY ? 0.f : a.m);
        },
        [&](const float4 (&v)[4], int, int) {
            float m = fmaxf(fmaxf(v[0].x, v[0].y), fmaxf(v[0].z, v[0].w));  // numbers before NaN
#pragma unroll
            for (int q = 1; q < 4; ++q) m = fmaxf(m, fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w)));
            kmax = max(kmax, lp_key(m));
            lp_raise(a, m);
            const float mu = a.m == -INFINITY ? 0.f : a.m;
            LpSums c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                c[q] = {0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) lp_add(c[q], lp_at(v[q], e), mu);
            }
            a.s += (c[0].s + c[1].s) + (c[2].s + c[3].s);
            a.t += (c[0].t + c[1].t) + (c[2].t + c[3].t);
        });
    uint32_t kq = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, 1));
    kq = max(kq, __shfl_xor_sync(0xffffffffu, kq, 2));
    if ((lane & 3) == 0) sh.quad[tid >> 2] = kq;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const LpSums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                          __shfl_xor_sync(0xffffffffu, a.t, o)};
        // the lower lane's share first: both lanes get the same sum
        a = (lane & o) ? lp_join(b, a) : lp_join(a, b);
    }
    if (lane == 0) sh.warp[warp] = a;
    __syncthreads();
    if (k > 0) {
        if (tid >= 32 && tid < 32 + kLpQuads) {  // warps 1..4: the k-th largest of the quads' maxima
            const int q = tid - 32;
            const uint32_t mine = sh.quad[q];
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < kLpQuads; j += 4) {
                const uint4 o = *reinterpret_cast<const uint4 *>(sh.quad + j);
                r += (o.x > mine || (o.x == mine && j < q)) + (o.y > mine || (o.y == mine && j + 1 < q)) +
                     (o.z > mine || (o.z == mine && j + 2 < q)) + (o.w > mine || (o.w == mine && j + 3 < q));
            }
            if (r == k - 1) sh.bound = mine;
        }
    }
    if (warp == 0) {  // meanwhile warp 0 joins the warps' sums
        a = lane < kLpThreads / 32 ? sh.warp[lane] : LpSums{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const LpSums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                              __shfl_xor_sync(0xffffffffu, a.t, o)};
            a = (lane & o) ? lp_join(b, a) : lp_join(a, b);
        }
    }
    if (k > 0) {
        __syncthreads();
        const uint32_t bound = sh.bound;
        const float bv = bound ? lp_value(bound) : 0.f;  // key 0: everything is a candidate
        auto take = [&](float v, int i) {
            if (v >= bv || bound == 0u) {
                const int at = atomicAdd(&sh.ncand, 1);
                if (at < kLpCand) sh.cand[at] = lp_pair(lp_key(v), i);
            }
        };
        lp_each(x, i0, i1, tid, take, [&](const float4 (&v)[4], int i, int step) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float m = fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w));
                if (m >= bv || bound == 0u) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) take(lp_at(v[q], e), i + q * step + e);
                }
            }
        });
        __syncthreads();
        const int nc = sh.ncand;
        if (nc <= kLpCand) {
            for (int c = tid; c < nc; c += kLpThreads) {
                const unsigned long long mine = sh.cand[c];
                int r = 0;
#pragma unroll 8
                for (int j = 0; j < nc; ++j) r += sh.cand[j] > mine;
                if (r < k) sh.mine[r] = mine;
            }
        } else {  // one by one: the best pair below the last one
            unsigned long long last = ~0ull;
            for (int q = 0; q < k; ++q) {
                unsigned long long best = 0ull;
                auto look = [&](float v, int i) {
                    const unsigned long long c = lp_pair(lp_key(v), i);
                    if (c < last && c > best) best = c;
                };
                lp_each(x, i0, i1, tid, look, [&](const float4 (&v)[4], int i, int step) {
#pragma unroll
                    for (int z = 0; z < 4; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e) look(lp_at(v[z], e), i + z * step + e);
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const unsigned long long c = __shfl_xor_sync(0xffffffffu, best, o);
                    best = c > best ? c : best;
                }
                if (lane == 0) sh.best[warp] = best;
                __syncthreads();
                best = sh.best[0];
#pragma unroll
                for (int w = 1; w < kLpThreads / 32; ++w) best = sh.best[w] > best ? sh.best[w] : best;
                if (tid == 0) sh.mine[q] = best;
                last = best;
                __syncthreads();
            }
        }
    }
    __syncthreads();
    // the sums and the best pairs to rank 0
    if (S > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    LpShared *root = cl.map_shared_rank(&sh, 0);
    if (tid == 0) root->sums[rank] = a;
    if (tid < k) root->top[rank * k + tid] = sh.mine[tid];
    if (S > 1)
        cl.sync();
    else
        __syncthreads();
    if (rank != 0) return;
    LpSums all = sh.sums[0];
    for (int r = 1; r < S; ++r) all = lp_join(all, sh.sums[r]);
    // a row whose logits are all -inf allows nothing: log probability -inf for
    // every token, entropy 0
    const bool empty = all.m == -INFINITY && all.s == 0.f;
    const float lse = empty ? 0.f : all.m + logf(all.s);
    if (tid == 0) {
        if (p.entropy) p.entropy[row] = empty ? 0.f : logf(all.s) - all.t / all.s;
        if (p.logprob) {
            const int tok = p.tokens[row];
            float lp = 0.f;  // a negative token: a row that is not scored
            if (tok >= p.n) {
                lp = __uint_as_float(0x7fffffffu);
                atomicExch(p.err, kErrPaged);
            } else if (tok >= 0) {
                lp = x[tok] - lse;
            }
            p.logprob[row] = lp;
        }
    }
    // the k best of the CTAs' lists, by rank (the pairs are all different)
    if (tid < S * k) {
        const unsigned long long mine = sh.top[tid];
        int at = 0;
#pragma unroll 8
        for (int j = 0; j < S * k; ++j) at += sh.top[j] > mine;
        if (mine != 0ull && at < k) {
            p.top_val[(size_t)row * k + at] = lp_value((uint32_t)(mine >> 32)) - lse;
            p.top_idx[(size_t)row * k + at] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
        }
    }
}

}  // namespace dev

int launch_logprobs(const LogprobParams &p, int sms, void *stream_) {
    cudaStream_t stream = (cudaStream_t)stream_;
    int S = 1;
    while (S < 8 && (long long)p.rows * S * 2 <= 2 * sms && p.n / (2 * S) >= 2 * dev::kLpThreads) S *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * S), 1, 1);
    cfg.blockDim = dim3(dev::kLpThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)S;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, dev::q4logprobs_kernel, p) == cudaSuccess ? 0 : -1;
}

}  // namespace q4
