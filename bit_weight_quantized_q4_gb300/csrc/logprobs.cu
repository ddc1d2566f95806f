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

// fn(value, index) for the elements [i0, i1) of row x: scalars up to a 16-byte
// boundary, then four 16-byte loads in flight a thread, then scalars.
template <class F>
__device__ __forceinline__ void lp_each(const float *x, int i0, int i1, int tid, F fn) {
    const int head = min(i1 - i0, (int)((4u - (((uintptr_t)(x + i0) >> 2) & 3u)) & 3u));
    if (tid < head) fn(x[i0 + tid], i0 + tid);
    const int v0 = i0 + head, nv = (i1 - v0) >> 2;
    const float4 *xv = reinterpret_cast<const float4 *>(x + v0);
    int j = tid;
    for (; j + 3 * kLpThreads < nv; j += 4 * kLpThreads) {
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = xv[j + q * kLpThreads];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = v0 + 4 * (j + q * kLpThreads);
            fn(v[q].x, i);
            fn(v[q].y, i + 1);
            fn(v[q].z, i + 2);
            fn(v[q].w, i + 3);
        }
    }
    for (; j < nv; j += kLpThreads) {
        const float4 v = xv[j];
        const int i = v0 + 4 * j;
        fn(v.x, i);
        fn(v.y, i + 1);
        fn(v.z, i + 2);
        fn(v.w, i + 3);
    }
    const int tail = v0 + 4 * nv + tid;
    if (tail < i1) fn(x[tail], tail);
}

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

struct LpShared {
    LpSums sums;                       // the CTA's, read by rank 0
    unsigned long long top[kLpTop];    // the CTA's k best pairs (0: none)
    unsigned long long cand[kLpCand];
    LpSums warp[kLpThreads / 32];
    uint32_t quad[kLpQuads];
    unsigned long long best[kLpThreads / 32];
    uint32_t bound;
    int ncand;
};

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
    if (tid == 0) sh.ncand = 0;
    if (tid < kLpTop) sh.top[tid] = 0ull;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    LpSums a = {-INFINITY, 0.f, 0.f};
    uint32_t kmax = 0u;
    lp_each(x, i0, i1, tid, [&](float v, int) {
        kmax = max(kmax, lp_key(v));
        if (v > a.m) {  // a new maximum: rescale what came before
            const float d = a.m == -INFINITY ? 0.f : fmaxf(a.m - v, -200.f), f = __expf(d);
            a.t = f * fmaf(d, a.s, a.t);
            a.s *= f;
            a.m = v;
        }
        const float d = a.m == -INFINITY && v == -INFINITY ? -200.f : fmaxf(v - a.m, -200.f);
        const float e = v != v ? v : __expf(d);
        a.s += e;
        a.t = fmaf(e, d, a.t);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const LpSums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                          __shfl_xor_sync(0xffffffffu, a.t, o)};
        // the lower lane's share first: both lanes get the same sum
        a = (lane & o) ? lp_join(b, a) : lp_join(a, b);
    }
    uint32_t kq = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, 1));
    kq = max(kq, __shfl_xor_sync(0xffffffffu, kq, 2));
    if ((lane & 3) == 0) sh.quad[tid >> 2] = kq;
    if (lane == 0) sh.warp[warp] = a;
    __syncthreads();
    if (warp == 0) {
        a = lane < kLpThreads / 32 ? sh.warp[lane] : LpSums{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const LpSums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                              __shfl_xor_sync(0xffffffffu, a.t, o)};
            a = (lane & o) ? lp_join(b, a) : lp_join(a, b);
        }
        if (lane == 0) sh.sums = a;
    }
    if (k > 0) {
        if (tid < kLpQuads) {  // the k-th largest of the quads' maxima
            const uint32_t mine = sh.quad[tid];
            int r = 0;
            for (int j = 0; j < kLpQuads; ++j) r += sh.quad[j] > mine || (sh.quad[j] == mine && j < tid);
            if (r == k - 1) sh.bound = mine;
        }
        __syncthreads();
        const uint32_t bound = sh.bound;
        lp_each(x, i0, i1, tid, [&](float v, int i) {
            const uint32_t key = lp_key(v);
            if (key >= bound) {
                const int at = atomicAdd(&sh.ncand, 1);
                if (at < kLpCand) sh.cand[at] = lp_pair(key, i);
            }
        });
        __syncthreads();
        const int nc = sh.ncand;
        if (nc <= kLpCand) {
            for (int c = tid; c < nc; c += kLpThreads) {
                const unsigned long long mine = sh.cand[c];
                int r = 0;
                for (int j = 0; j < nc; ++j) r += sh.cand[j] > mine;
                if (r < k) sh.top[r] = mine;
            }
        } else {  // one by one: the best pair below the last one
            unsigned long long last = ~0ull;
            for (int q = 0; q < k; ++q) {
                unsigned long long best = 0ull;
                lp_each(x, i0, i1, tid, [&](float v, int i) {
                    const unsigned long long c = lp_pair(lp_key(v), i);
                    if (c < last && c > best) best = c;
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
                if (tid == 0) sh.top[q] = best;
                last = best;
                __syncthreads();
            }
        }
    }
    if (S > 1)
        cl.sync();  // every CTA's sums and best pairs are there
    else
        __syncthreads();
    if (rank == 0) {
        LpSums all = sh.sums;
        for (int r = 1; r < S; ++r) all = lp_join(all, *cl.map_shared_rank(&sh.sums, r));
        // a row whose logits are all -inf allows nothing: log probability
        // -inf for every token, entropy 0
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
        // merge the CTAs' lists by rank: S * k pairs, all different
        if (k > 0 && tid < S * kLpTop && (tid & (kLpTop - 1)) < k) {
            const int r = tid / kLpTop, j = tid & (kLpTop - 1);
            const unsigned long long mine = cl.map_shared_rank(&sh, r)->top[j];
            if (mine != 0ull) {
                int at = j;
                for (int r2 = 0; r2 < S; ++r2) {
                    if (r2 == r) continue;
                    const unsigned long long *o = cl.map_shared_rank(&sh, r2)->top;
                    int c = 0;  // the lists are sorted: count the larger ones
                    while (c < k && o[c] > mine) ++c;
                    at += c;
                }
                if (at < k) {
                    p.top_val[(size_t)row * k + at] = lp_value((uint32_t)(mine >> 32)) - lse;
                    p.top_idx[(size_t)row * k + at] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
                }
            }
        }
    }
    if (S > 1) cl.sync();  // no CTA leaves while rank 0 reads it
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
