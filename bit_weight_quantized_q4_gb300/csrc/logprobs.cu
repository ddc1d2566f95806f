// logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logit rows (Module gpu, module sampling: what a sampler
// reads beside the greedy argmax).  Per row x of n logits:
//   m = max x, s = sum e^(x - m), lse = m + log s
//   logprob = x[token] - lse,   entropy = lse - sum p x = log s - t / s,
//   t = sum e^(x - m) (x - m)   (terms of x = -inf count as 0)
//   top: the k largest (ties to the lowest index), as x - lse.
// One pass for the sums and each thread's largest value; then the k-th largest
// of the 128 quads' maxima bounds the k-th largest logit from below, and a
// second look keeps the few values at or above that bound, which are ranked by
// counting.  The first pass leaves the largest value of every 16 in shared memory,
// so that the second reads again (from L2) only the 16s that reach the bound.
// Where a bound lets too many through (long ties; fewer finite logits than k, so that
// the bound is -inf) the k largest are found one by one: 512 rows of 65536 with 1 to 15
// tokens allowed and 20 asked for take 722 us.  (512 rows of 65536: 31 us; 34.5 with the whole row read again,
// 46 with candidates kept during the first pass from the bound of its first batch,
// 71 with slices staged in shared memory; 23.7 without the top.)
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
constexpr int kLpCand = 1024;  // candidates a CTA holds
constexpr int kLpTop = 32;     // largest k
constexpr int kLpSlots = 16;   // batches whose largest values are held apart

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

struct LpSums {
    float m, s, t;
};
// Joins the shares of a warp's lanes (of lanes l and l ^ o for o = width / 2, ..,
// 1; each lane ends with the same): the largest maximum first, then the sums
// scaled to it once and added, lower lanes first.
__device__ __forceinline__ LpSums lp_join(const LpSums &a, int width, int lane) {
    float m = a.m;
    for (int o = width / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // a share without a finite maximum has nothing to scale; a difference below
    // -200 scales by e^-200 = 0 in fp32, and stays finite (0 * -inf is NaN)
    const float d = a.m == -INFINITY ? 0.f : fmaxf(a.m - m, -200.f), f = __expf(d);
    float s = a.s * f, t = f * fmaf(d, a.s, a.t);
    for (int o = width / 2; o > 0; o >>= 1) {
        const float s2 = __shfl_xor_sync(0xffffffffu, s, o), t2 = __shfl_xor_sync(0xffffffffu, t, o);
        s = (lane & o) ? s2 + s : s + s2;
        t = (lane & o) ? t2 + t : t + t2;
    }
    return {m, s, t};
}

constexpr int kLpMaxCluster = 8;

struct LpShared {
    static constexpr int Quads = kLpThreads / 4, Quarter = Quads / 4;
    // rank 0 of a cluster receives every CTA's sums and k best pairs (0: none)
    LpSums sums[kLpMaxCluster];
    unsigned long long top[kLpMaxCluster * kLpTop];
    unsigned long long mine[kLpTop];   // this CTA's
    unsigned long long cand[kLpCand];
    LpSums warp[kLpThreads / 32];
    __align__(16) uint32_t quad[Quads + 12];  // quarters of it 4 words apart: their readers meet no bank twice
    unsigned long long best[kLpThreads / 32];
    float tops[kLpSlots][kLpThreads];  // a thread's largest value of each batch (of batches kLpSlots apart)
    uint32_t bound;
    int ncand;
    __device__ __forceinline__ uint32_t *quad_at(int q) { return quad + q + 4 * (q / Quarter); }
};

// The sums' reference m: raised (and what came before rescaled) when a logit is
// more than kLpSlack above it, so that few logits do, and at once from -inf.
constexpr float kLpSlack = 8.f;
__device__ __forceinline__ void lp_raise(LpSums &a, float m) {
    if (m > a.m + kLpSlack) {
        const float d = fmaxf(a.m - m, -200.f), f = __expf(d);  // from -inf: the sums are zero
        a.t = f * fmaf(d, a.s, a.t);
        a.s *= f;
        a.m = m;
    }
}
// Two logits into sums in log2 units, two at a time (mu: minus the reference):
// e = 2^y, y = (v - m) log2 e; NaN stays; -inf: e = 0, and its term of t is 0
__device__ __forceinline__ void lp_add2(uint64_t &s, uint64_t &t, float v0, float v1, uint64_t mu) {
    const uint64_t y = mul_f32x2(add_f32x2(pair_f32(v0, v1), mu), pair_f32(1.4426950408889634f, 1.4426950408889634f));
    const float y0 = lo_f32(y), y1 = hi_f32(y);
    const uint64_t e = pair_f32(ex2(y0), ex2(y1));
    s = add_f32x2(s, e);
    t = fma_f32x2(e, pair_f32(fmaxf(y0, -300.f), fmaxf(y1, -300.f)), t);
}

// The first n of v's values (at index i ..) whose key reaches the bound become
// candidates.  Not inlined: few values get here, and the kernel's own code,
// which a row runs through once, stays short.
__device__ __noinline__ void lp_take(LpShared &sh, float4 v, int i, int n, uint32_t bound) {
    for (int e = 0; e < n; ++e) {
        const uint32_t key = lp_key(v.x);
        if (key >= bound) {
            const int at = atomicAdd(&sh.ncand, 1);
            if (at < kLpCand) sh.cand[at] = lp_pair(key, i + e);
        }
        v = make_float4(v.y, v.z, v.w, v.x);
    }
}

__global__ void __launch_bounds__(kLpThreads, 2) q4logprobs_kernel(const __grid_constant__ LogprobParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int Batch = 16 * kLpThreads;  // logits: four float4 in flight a thread
    __shared__ LpShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int S = (int)cl.num_blocks(), rank = (int)cl.block_rank(), row = blockIdx.x / S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = ((p.n + S - 1) / S + 3) & ~3;
    const float *x = p.logits + (size_t)row * p.n;
    // this CTA's logits [i0, i1), whole batches of them from v0, a 16-byte boundary
    const int i0 = min(p.n, rank * per), i1 = min(p.n, i0 + per);
    const int v0 = min(i1, i0 + (int)((4u - (((uintptr_t)(x + i0) >> 2) & 3u)) & 3u));
    const int v1 = v0 + (i1 - v0) / Batch * Batch;
    const int k = p.k;
    // this CTA runs: the matching wait comes before the writes to rank 0
    if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (tid == 0) sh.ncand = 0;
    if (tid < kLpTop) sh.mine[tid] = 0ull;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    LpSums a = {-INFINITY, 0.f, 0.f};
    uint32_t kmax = 0u;
    auto add2 = [&](float v0, float v1) {
        const float mu = a.m == -INFINITY ? 0.f : -a.m;
        uint64_t s2 = 0ull, t2 = 0ull;
        lp_add2(s2, t2, v0, v1, pair_f32(mu, mu));
        a.s += lo_f32(s2) + hi_f32(s2);
        a.t = fmaf(lo_f32(t2) + hi_f32(t2), 0.69314718055994531f, a.t);
    };
    auto add4 = [&](const float4 (&v)[4]) {
        const float mu = a.m == -INFINITY ? 0.f : -a.m;
        uint64_t s2[2] = {0ull, 0ull}, t2[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            lp_add2(s2[0], t2[0], v[q].x, v[q].y, pair_f32(mu, mu));
            lp_add2(s2[1], t2[1], v[q].z, v[q].w, pair_f32(mu, mu));
        }
        s2[0] = add_f32x2(s2[0], s2[1]);
        t2[0] = add_f32x2(t2[0], t2[1]);
        a.s += lo_f32(s2[0]) + hi_f32(s2[0]);
        a.t = fmaf(lo_f32(t2[0]) + hi_f32(t2[0]), 0.69314718055994531f, a.t);
    };
    // The k-th largest of the quads' maxima (all threads; k > 0): the value
    // with fewer than k above it and at least k not below it, four threads a quad
    auto bound_of = [&]() {
        uint32_t kq = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, 1));
        kq = max(kq, __shfl_xor_sync(0xffffffffu, kq, 2));
        if ((lane & 3) == 0) *sh.quad_at(tid >> 2) = kq;
        if (tid == 0) sh.ncand = 0;
        __syncthreads();
        const uint32_t mine = *sh.quad_at(tid >> 2);
        int above = 0, below = 0;
#pragma unroll
        for (int j = 0; j < LpShared::Quarter; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4 *>(sh.quad_at((tid & 3) * LpShared::Quarter) + j);
            above += (int)(o.x > mine) + (int)(o.y > mine) + (int)(o.z > mine) + (int)(o.w > mine);
            below += (int)(o.x < mine) + (int)(o.y < mine) + (int)(o.z < mine) + (int)(o.w < mine);
        }
        int both = above | below << 16;
        both += __shfl_xor_sync(0xffffffffu, both, 1);
        both += __shfl_xor_sync(0xffffffffu, both, 2);
        if ((both & 0xffff) < k && LpShared::Quads - (both >> 16) >= k) sh.bound = mine;  // equal ones write the same
        __syncthreads();
    };
    // fn(value, index) for the logits [j0, j1), rolled: the ends, and slow paths
    auto each = [&](int j0, int j1, auto fn) {
#pragma unroll 4
        for (int i = j0 + tid; i < j1; i += kLpThreads) fn(x[i], i);
    };
    float4 v[4];
    float m[4];
    auto load = [&](int j) {
        const float4 *xv = reinterpret_cast<const float4 *>(x + j) + tid;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = xv[q * kLpThreads];
    };
    auto tops = [&]() {  // numbers before NaN
#pragma unroll
        for (int q = 0; q < 4; ++q) m[q] = fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w));
    };
    const int nbatch = (v1 - v0) / Batch;
#pragma unroll 2
    for (int b = 0; b < nbatch; ++b) {
        load(v0 + b * Batch);
        tops();
        const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        float &slot = sh.tops[b % kLpSlots][tid];
        slot = b < kLpSlots ? top : fmaxf(top, slot);
        kmax = max(kmax, lp_key(top));
        lp_raise(a, top);
        add4(v);
    }
    auto end = [&](float x1, int) {
        kmax = max(kmax, lp_key(x1));
        lp_raise(a, x1);
        add2(x1, -INFINITY);
    };
    each(i0, v0, end);
    each(v1, i1, end);
    a = lp_join(a, 32, lane);
    if (lane == 0) sh.warp[warp] = a;
    __syncthreads();
    if (warp == 0) {
        a = lane < kLpThreads / 32 ? sh.warp[lane] : LpSums{-INFINITY, 0.f, 0.f};
        a = lp_join(a, 32, lane);
    }
    if (k > 0) {
        bound_of();
        const uint32_t bound = sh.bound;
        const float bv = bound ? lp_value(bound) : -INFINITY;  // key 0: everything is a candidate
        auto take4 = [&](int j) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (m[q] >= bv || bound == 0u) lp_take(sh, v[q], j + 4 * (tid + q * kLpThreads), 4, bound);
        };
        if (nbatch == 1) {  // still in registers
            take4(v0);
        } else {
            unsigned hit = 0;
            for (int c = 0; c < min(nbatch, kLpSlots); ++c)
                if (sh.tops[c][tid] >= bv || bound == 0u) hit |= 1u << c;
            for (; hit; hit &= hit - 1)
                for (int b = __ffs(hit) - 1; b < nbatch; b += kLpSlots) {
                    load(v0 + b * Batch);
                    tops();
                    take4(v0 + b * Batch);
                }
        }
        auto take = [&](float x1, int i) {
            if (lp_key(x1) >= bound) lp_take(sh, make_float4(x1, 0.f, 0.f, 0.f), i, 1, bound);
        };
        each(i0, v0, take);
        each(v1, i1, take);
        __syncthreads();
        const int nc = sh.ncand;
        if (nc <= kLpCand) {
            for (int c = tid >> 1; c < nc; c += kLpThreads / 2) {  // two threads a candidate
                const unsigned long long mine = sh.cand[c];
                const int half = (nc + 1) / 2, j0 = (tid & 1) * half, j1 = min(nc, j0 + half);
                int r = 0;
#pragma unroll 8
                for (int j = j0; j < j1; ++j) r += sh.cand[j] > mine;
                r += __shfl_xor_sync(3u << (lane & ~1), r, 1);
                if ((tid & 1) == 0 && r < k) sh.mine[r] = mine;
            }
        } else {  // one by one: the best pair below the last one
            unsigned long long last = ~0ull;
            for (int q = 0; q < k; ++q) {
                unsigned long long best = 0ull;
                each(i0, i1, [&](float v, int i) {
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
    const LpSums all =
        S > 1 ? lp_join(lane < S ? sh.sums[lane] : LpSums{-INFINITY, 0.f, 0.f}, 32, lane) : sh.sums[0];
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
    if ((tid >> 1) < S * k) {  // two threads a pair, each half of the pairs
        const unsigned long long mine = sh.top[tid >> 1];
        const int half = (S * k + 1) / 2, j0 = (tid & 1) * half, j1 = min(S * k, j0 + half);
        int at = 0;
#pragma unroll 8
        for (int j = j0; j < j1; ++j) at += sh.top[j] > mine;
        at += __shfl_xor_sync(3u << (lane & ~1), at, 1);
        if ((tid & 1) == 0 && mine != 0ull && at < k) {
            p.top_val[(size_t)row * k + at] = lp_value((uint32_t)(mine >> 32)) - lse;
            p.top_idx[(size_t)row * k + at] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
        }
    }
}

}  // namespace dev

int launch_logprobs(const LogprobParams &p, int sms, void *stream_) {
    // a CTA a row, or a cluster for each row while those do not fill the device
    // (512 rows of 65536 by clusters of two: 48 us against 34.5 then)
    int S = 1;
    while (S < dev::kLpMaxCluster && (long long)p.rows * S * 2 <= 2 * sms && p.n / (2 * S) >= 2 * dev::kLpThreads) S *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * S), 1, 1);
    cfg.blockDim = dim3(dev::kLpThreads, 1, 1);
    cfg.stream = (cudaStream_t)stream_;
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
