// moe.cu -- a mixture-of-experts layer for up to 16 tokens, in two kernels:
//   xh = x / rms(x) gamma;  l = R xh;  the top_k experts of a token and their
//   weights w (softmax over the chosen, or over all);
//   h_e = silu(G_e Q(xh)) (U_e Q(xh));  y = r + sum_e w_e D_e Q(h_e)
// with Q the rounding to MXFP4 and G, U, D microscaled 4-bit weights.
//
// The time is the chosen experts' weights' from HBM.  On the block-scaled tensor
// core an instruction takes 16 columns at least, so every expert sees all tokens
// of the batch, and only a token's own experts' columns are used: nothing is
// gathered.
//   One token, 8 of 128 experts of 768 x 2048: 16.2 to 17.7 us over machines for 21 MB (floor
// 3.1); sixteen, which reach 83 experts: 49 to 50 for 208 MB (30.7); four tokens, 2 of 8 experts
// of 14336 x 4096, which reach five: 82 for 0.47 GB (69.0); sixteen, which reach all: 123 for
// 0.75 GB (110.4).  The fixed part is a chain of latencies: the logits' kernel 4 us, the choice
// 2.4, the grid's barrier 1.2, the first copies of each half, joining 2.  (One token's first half
// is 96 units: 56 SMs have none.)
#include <algorithm>

#include "mx_common.cuh"

namespace q4 {
namespace dev {

// ------------------------------------------------------------------ logits and codes

constexpr int kRouteSlices = 8;  // warps that share an expert's row

// Four consecutive values as they are stored.
template <typename T>
struct Raw4 {
    typename std::conditional<sizeof(T) == 4, uint4, uint2>::type w;
    __device__ __forceinline__ void load(const T *src) { w = *reinterpret_cast<const decltype(w) *>(src); }
    __device__ __forceinline__ void zero() { w = {}; }
    __device__ __forceinline__ float4 values() const {
        if constexpr (sizeof(T) == 4) {
            return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
        } else {
            const T *v = reinterpret_cast<const T *>(&w);
            return make_float4(to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3]));
        }
    }
};

// CTAs below E: an expert's logits, eight warps for each NT tokens, a warp every
// eighth 128 columns.  The others: a token's row each, its norm and its codes.
// Latency bounds it, of loads and of the code itself: the loads of 4096 (four tokens:
// 2048) columns of a warp's tokens go out before the first is used, and a warp has one token's or
// four tokens' sums (eight warps with sixteen tokens' straight code took 6 us longer; a
// token's loads at a time, 8).
template <typename T, int NT>
__global__ void __launch_bounds__(NT == 1 ? 256 : 1024) q4moe_route_kernel(const __grid_constant__ MoeParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float sums[NT == 1 ? 8 : 32][2 * NT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *x = (const T *)p.x;
    if ((int)blockIdx.x < p.E) {
        const int e = blockIdx.x, t0 = warp / kRouteSlices * NT;
        if (e == 0) {
            if (tid == 0) *p.barrier = 0u, *p.units = 0u;
            for (int i = tid; i < mx_rtiles(p.hidden); i += blockDim.x) p.count[i] = 0u;
        }
        // dots with the expert's row (below NT) and sums of squares, a token each
        float v[2 * NT] = {};
        const float *row = p.router + (size_t)e * p.hidden;
        constexpr int R = NT == 1 ? 4 : 2, Step = 128 * kRouteSlices;  // loads of a row under way
        for (int c0 = 128 * (warp % kRouteSlices) + 4 * lane; c0 < p.hidden; c0 += Step * R) {
            float4 w[R], g[R];
            Raw4<T> a[NT][R];
            auto in = [&](int i) { return i == 0 || c0 + Step * i < p.hidden; };
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (in(i)) {
                    const int c = c0 + Step * i;
                    w[i] = *reinterpret_cast<const float4 *>(row + c);
                    g[i] = p.gamma ? *reinterpret_cast<const float4 *>(p.gamma + c) : make_float4(1.f, 1.f, 1.f, 1.f);
                } else {
                    w[i] = g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    a[t][i].zero();
                    if (t0 + t < p.nb && in(i)) a[t][i].load(x + (t0 + t) * p.ldx + c0 + Step * i);
                }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                w[i] = make_float4(w[i].x * g[i].x, w[i].y * g[i].y, w[i].z * g[i].z, w[i].w * g[i].w);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float4 b = a[t][i].values();
                    v[t] = fmaf(b.x, w[i].x, fmaf(b.y, w[i].y, fmaf(b.z, w[i].z, fmaf(b.w, w[i].w, v[t]))));
                    v[NT + t] = fmaf(b.x, b.x, fmaf(b.y, b.y, fmaf(b.z, b.z, fmaf(b.w, b.w, v[NT + t]))));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            if (lane == 0) sums[warp][i] = v[i];
        }
        __syncthreads();
        if (tid < p.nb) {  // a token a thread
            float dot = 0.f, sq = 0.f;
#pragma unroll
            for (int w = 0; w < kRouteSlices; ++w) {
                dot += sums[tid / NT * kRouteSlices + w][tid % NT];
                sq += sums[tid / NT * kRouteSlices + w][NT + tid % NT];
            }
            p.logits[(size_t)tid * p.E + e] = p.gamma ? dot * rsqrtf(fmaf(sq, 1.f / (float)p.hidden, p.eps)) : dot;
        }
        return;
    }
    const int warps = blockDim.x / 32;
    const int t = blockIdx.x - p.E, KT = mx_ktiles(p.hidden);
    const T *src = x + t * p.ldx;
    float rstd = 1.f;
    auto load = [&](int kt, float (&v)[8]) {
        const int c = kt * kMxK + 8 * lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        if (c < p.hidden) {
            Raw4<T> lo, hi;
            lo.load(src + c);
            hi.load(src + c + 4);
            const float4 a = lo.values(), b = hi.values();
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
    };
    if (p.gamma) {
        float sum = 0.f;
        for (int kt = warp; kt < KT; kt += warps) {
            float v[8];
            load(kt, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sums[warp][0] = sum;
        __syncthreads();
        sum = 0.f;
        for (int i = 0; i < warps; ++i) sum += sums[i][0];
        rstd = rsqrtf(fmaf(sum, 1.f / (float)p.hidden, p.eps));
    }
    for (int kt = warp; kt < KT; kt += warps) {
        const int c = kt * kMxK + 8 * lane;
        float v[8];
        load(kt, v);
        if (p.gamma && c < p.hidden) {
            const float4 a = *reinterpret_cast<const float4 *>(p.gamma + c);
            const float4 b = *reinterpret_cast<const float4 *>(p.gamma + c + 4);
            const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * rstd * g[i];
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_abs(m, v[i]);
        m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float mul;
        const uint32_t sc = mx_block_scale<0>(m, MxGain{}, mul);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= mul;
        uint8_t *rec = p.xq + (size_t)kt * kMoeRec;
        *reinterpret_cast<uint32_t *>(rec + mx_code_off(t, 4 * lane)) = mul == 0.f ? 0u : e2m1x8(v);
        if (lane % 4 == 0) rec[2048 + (lane >> 4) * 512 + t * 16 + ((lane >> 2) & 3)] = (uint8_t)sc;
    }
}

// ------------------------------------------------------------------ experts

constexpr int kMoeThreads = 32 * kMaxNb;  // a warp a token to choose the experts; then six have roles
constexpr int kMoeStages = 6;  // (what waits in more of them only delays what is wanted first: nine took 1 to 3 % longer)
constexpr int kMoeStage = mx_rec(0) + kMoeRec;  // a record of weights, one of activations
constexpr int kMoeExch = 2 * 2 * 2 * 8 * 32 * 4;  // [turn][pair of warps][gate or up][token][row]
// what the choice of the experts leaves: the experts with a token in rising order,
// their tokens (a bit each) and the tokens' weights [expert][16]
constexpr int kMoeOffExch = kMoeStages * kMoeStage, kMoeOffIds = kMoeOffExch + kMoeExch,
              kMoeOffMask = kMoeOffIds + 4 * kMoeMaxActive, kMoeOffW = kMoeOffMask + 4 * kMoeMaxActive,
              kMoeOffBar = kMoeOffW + 64 * kMoeMaxActive, kMoeOffUnit = kMoeOffBar + 8 * (2 * kMoeStages + 5) + 16,
              kMoeSmem = kMoeOffUnit + 128;
static_assert(kMoeStage % 1024 == 0 && kMoeSmem <= (int)kSmemMax, "shared memory of the experts' kernel");
// while they are chosen, over the ring: the choices, an expert's tokens and its place
// in the list
constexpr int kMoeOffChosen = 0, kMoeOffChosenW = kMoeOffChosen + 4 * kMoeMaxActive, kMoeOffTok = kMoeOffChosenW + 4 * kMoeMaxActive,
              kMoeOffSlot = kMoeOffTok + 4 * kMoeMaxExperts;
static_assert(kMoeOffSlot + 4 * kMoeMaxExperts <= kMoeOffExch, "the ring's room");
constexpr int kMoeParts = 8;  // CTAs that share a tile of outputs, about (one token of 128 experts 16.2 us; 10: 17.5, 5: 16.7)

// Order of logits: larger first, NaN (1) behind every number (-inf: 0x7FFFFF).
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);  // (-0 is 0)
    return v != v ? 1u : (u >> 31) ? ~u : u | 0x80000000u;
}

// One token's choice by a warp: its experts and weights into idx and weight
// [top_k].  A lane keeps the logits of its experts (lane, lane + 32, ..: NL of them at
// most) and the best of those not chosen yet; a round takes the best of the lanes.
template <int NL>
__device__ __forceinline__ void moe_choose(const float *logits, int E, int top_k, bool renorm, int *idx, float *weight,
                                           int lane) {
    float v[NL];
    uint32_t key[NL];  // 0: none, or chosen
#pragma unroll
    for (int i = 0; i < NL; ++i) v[i] = 32 * i + lane < E ? __ldcg(logits + 32 * i + lane) : 0.f;
#pragma unroll
    for (int i = 0; i < NL; ++i) key[i] = 32 * i + lane < E ? logit_key(v[i]) : 0u;
    float top = 0.f, mine = 0.f;
    int at = 0;
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) best = max(best, key[i]);
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        int where = 0x7FFFFFFF;
        float bv = 0.f;
#pragma unroll
        for (int i = NL - 1; i >= 0; --i)
            if (key[i] == most) {
                where = 32 * i + lane;
                bv = v[i];
            }
        const int first = (int)__reduce_min_sync(0xffffffffu, (uint32_t)where);
        const float got = __shfl_sync(0xffffffffu, bv, first & 31);
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if (32 * i + lane == first) key[i] = 0u;
        if (j == 0) top = got;
        if (lane == j) {
            mine = got;
            at = first;
        }
    }
    // softmax with the largest logit as its reference (NaN where one is NaN)
    const float e = lane < top_k ? expf(mine - top) : 0.f;
    float sum = e;
    if (!renorm) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if (32 * i + lane < E) sum += expf(v[i] - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < top_k) {
        idx[lane] = at;
        weight[lane] = e / sum;
    }
}

// Named barrier `bar` of n threads (whole warps): whether `v` holds in all of them.
__device__ __forceinline__ bool bar_all(int bar, int n, bool v) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(bar), "r"(n), "r"((uint32_t)v)
        : "memory");
    return all != 0;
}

// Every CTA chooses the experts by itself (the logits are a few kilobytes), then two
// halves in one kernel: first every (expert with a token, 64 rows of gate and of up)
// unit, the next one to the CTA that is free first; then, behind a barrier of the grid, the down projections,
// whose stages (output tile, expert, k) form a line that the CTAs divide evenly: a
// stream needs all SMs (44 GB/s each; 6.3 of the 6.8 TB/s with all 152).  Parts of
// a tile are joined by the last of its CTAs to finish, in CTA order: nothing depends on
// scheduling.  The weights of the second half's first stages are on their way before
// the barrier.  warp 0 copies, warp 1 issues MMAs, warps 2-5 take the sums.
template <typename T>
__global__ void __launch_bounds__(kMoeThreads, 1) q4moe_experts_kernel(const __grid_constant__ MoeParams p) {
    constexpr int REC = mx_rec(0), S = kMoeStages;
    extern __shared__ __align__(1024) uint8_t sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t ring = smem_u32(sm), b_full = ring + kMoeOffBar, b_empty = b_full + 8 * S, b_acc = b_empty + 8 * S,
                   b_read = b_acc + 16, b_drain = b_read + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + kMoeOffBar + 8 * (2 * S + 5));
    volatile int *info = reinterpret_cast<volatile int *>(tslot + 1);  // experts with a token; tiles to join
    int *ids = reinterpret_cast<int *>(sm + kMoeOffIds);
    unsigned *masks = reinterpret_cast<unsigned *>(sm + kMoeOffMask);
    volatile int *unit_s = reinterpret_cast<volatile int *>(sm + kMoeOffUnit);  // this CTA's last 16 units,
    volatile int *more_s = unit_s + 16;                                         // and whether others followed
    float *wtab = reinterpret_cast<float *>(sm + kMoeOffW);
    if (warp == 0) {
        if (lane < S) {
            mbar_init(b_full + 8 * lane, 1);
            mbar_init(b_empty + 8 * lane, 1);
        }
        if (lane < 2) {
            mbar_init(b_acc + 8 * lane, 1);
            mbar_init(b_read + 8 * lane, 4);
        }
        if (lane == 0) mbar_init(b_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(tslot), 128);
        tc::tmem_relinquish();
        // after the allocation: a kernel that starts on this could hold the columns this one waits for
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    int *chosen = reinterpret_cast<int *>(sm + kMoeOffChosen);
    float *chosen_w = reinterpret_cast<float *>(sm + kMoeOffChosenW);
    unsigned *tokens = reinterpret_cast<unsigned *>(sm + kMoeOffTok);
    int *slot = reinterpret_cast<int *>(sm + kMoeOffSlot);
    for (int e = tid; e < p.E; e += kMoeThreads) tokens[e] = 0u;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp < p.nb) {
        const int t = warp;
        int *idx = chosen + t * p.top_k;
        float *w = chosen_w + t * p.top_k;
        if (p.positions && p.positions[t] < 0) {  // an idle row: no experts
            if (lane < p.top_k) {
                idx[lane] = -1;
                w[lane] = 0.f;
            }
        } else {
            const float *logits = p.logits + (size_t)t * p.E;
            if (p.E <= 256)
                moe_choose<8>(logits, p.E, p.top_k, p.renormalize != 0, idx, w, lane);
            else
                moe_choose<kMoeMaxExperts / 32>(logits, p.E, p.top_k, p.renormalize != 0, idx, w, lane);
        }
    }
    __syncthreads();
    const int pairs = p.nb * p.top_k;
    for (int i = tid; i < pairs; i += kMoeThreads) {
        const int e = chosen[i];
        if (e >= 0) atomicOr(&tokens[e], 1u << (i / p.top_k));
        if (blockIdx.x == 0) {
            p.idx[i] = e;
            p.weight[i] = chosen_w[i];
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int b = 0; b < p.E; b += 32) {
            const int e = b + lane;
            const unsigned has = e < p.E ? tokens[e] : 0u, hit = __ballot_sync(0xffffffffu, has != 0u);
            if (has) {
                const int s = n + __popc(hit & ((1u << lane) - 1u));
                slot[e] = s;
                ids[s] = e;
                masks[s] = has;
            }
            n += __popc(hit);
        }
        if (lane == 0) {
            info[0] = n;
            info[1] = info[2] = -1;
        }
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += kMoeThreads)
        if (chosen[i] >= 0) wtab[slot[chosen[i]] * 16 + i / p.top_k] = chosen_w[i];
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before copies into the same room
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;

    const int nA = info[0], KS1 = mx_ktiles(p.hidden), KS2 = mx_ktiles(p.inter);
    const int T1 = mx_rtiles(2 * p.inter), T2 = mx_rtiles(p.hidden);
    const int units = nA * T1, grid = gridDim.x, cta = blockIdx.x;
    // the second half's line: tile m's stages are [m line, (m + 1) line)
    const int line = nA * KS2, ctas2 = min(grid, T2 * min(kMoeParts, max(line, 1)));
    auto first_of = [&](int c) { return (long long)T2 * line * c / ctas2; };
    const long long g0 = cta < ctas2 ? first_of(cta) : 0, g1 = cta < ctas2 ? first_of(cta + 1) : 0;
    auto sharers = [&](int m, int &f, int &l) {  // the first and the last CTA with a part of tile m
        const long long all = (long long)T2 * line, s0 = (long long)m * line;
        f = (int)(((s0 + 1) * ctas2 - 1) / all);
        l = (int)(((s0 + line) * ctas2 - 1) / all);
    };
    // this CTA's segments: f(tile, first stage, end) until it says no
    auto walk = [&](auto f) {
        for (long long g = g0; g < g1;) {
            const int m = (int)(g / line), q0 = (int)(g - (long long)m * line), q1 = (int)min((long long)line, q0 + g1 - g);
            if (!f(m, q0, q1)) return;
            g += q1 - q0;
        }
    };
    const long long lim = p.wait_cycles;
    const size_t slot_floats = (size_t)p.nb * kMxRows;
    auto store = [&](int row, int t, float v) {
        if (row >= p.hidden) return;
        const size_t at = (size_t)t * p.hidden + row;
        ((T *)p.y)[at] = from_f32<T>(p.r ? v + to_f32(((const T *)p.r)[at]) : v);
    };

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        // (one thread's chain of instructions: what stages share is computed once, slots are counted)
        if (lane == 0) {
            uint32_t extra = (uint32_t)p.extra_tx;
            bool ok = true;
            struct Slot {  // the next slot to fill: of weights, of activations
                uint32_t dst, bar, par;
                __device__ __forceinline__ void next(uint32_t ring, uint32_t b_full) {
                    dst += kMoeStage, bar += 8;
                    if (bar == b_full + 8 * S) {
                        dst = ring;
                        bar = b_full;
                        par ^= 1;
                    }
                }
            } ws = {ring, b_full, 1}, as = {ring, b_full, 0};  // (a wait for the phase before the first passes)
            int issued = 0;
            // a stage's weights; its activations follow on the same barrier
            auto weights = [&](const uint8_t *src) {
                if (!mbar_wait(ws.bar + 8 * S, ws.par, lim)) return false;  // b_empty of this slot
                mbar_expect_tx(ws.bar, kMoeStage + extra);
                extra = 0;
                bulk_copy(ws.dst, src, REC, ws.bar);
                ws.next(ring, b_full);
                return true;
            };
            auto acts = [&](const uint8_t *src) {
                bulk_copy(as.dst + REC, src, kMoeRec, as.bar);
                as.next(ring, b_full);
                ++issued;
            };
            // units of the first half: this CTA's number, then the next that no CTA has.  A
            // unit's number is there before its first stage is complete, and whether it has a successor
            // before its last one is.  (The ring and the two accumulators hold fewer than 16 units.)
            for (int u = cta, count = 0; ok && u < units; ++count) {
                unit_s[count & 15] = u;
                const int next = units > grid ? grid + (int)atomicAdd(p.units, 1u) : units;
                const int a = u / T1, tile = u - a * T1;
                const uint8_t *w = p.gate_up + ((size_t)ids[a] * T1 + tile) * KS1 * REC, *x = p.xq;
                for (int ks = 0; ks < KS1; ++ks, w += REC, x += kMoeRec) {
                    if (ks + 1 == KS1) more_s[count & 15] = next < units;
                    ok = weights(w);
                    if (!ok) break;
                    acts(x);
                }
                u = next;
            }
            // the second half: a segment's weights run through the experts' matrices, a tile of KS2
            // records each
            int ahead = 0;  // stages with their weights on the way
            auto segment = [&](int m, int q0, int q1, auto f) {
                int a = q0 / KS2, k = q0 - a * KS2;
                const uint8_t *w = p.down + (((size_t)ids[a] * T2 + m) * KS2 + k) * REC;
                for (int q = q0; q < q1; ++q) {
                    if (!f(w, q)) return false;
                    w += REC;
                    if (++k == KS2 && q + 1 < q1) {
                        k = 0;
                        w = p.down + ((size_t)ids[++a] * T2 + m) * KS2 * REC;
                    }
                }
                return true;
            };
            if (ok && g0 < g1) {
                walk([&](int m, int q0, int q1) {
                    return segment(m, q0, q1, [&](const uint8_t *w, int) {
                        if (ahead == S) return false;
                        ok = weights(w);
                        ahead += ok;
                        return ok;
                    });
                });
                const unsigned target = (unsigned)grid + (unsigned)p.barrier_extra;
                for (long long n = 0; ok && ld_acquire_u32(p.barrier) < target; ++n) ok = n < p.barrier_polls;
                asm volatile("fence.proxy.async;" ::: "memory");  // what others wrote, for this thread's copies
            }
            int skip = ahead;
            if (ok)
                walk([&](int m, int q0, int q1) {
                    return segment(m, q0, q1, [&](const uint8_t *w, int q) {
                        if (skip > 0) {
                            --skip;
                        } else {
                            ok = weights(w);
                            if (!ok) return false;
                            ++ahead;
                        }
                        acts(p.h + (size_t)q * kMoeRec);
                        --ahead;
                        return true;
                    });
                });
            if (!ok) atomicExch(p.err, 4);
            // (after a failure: the stages that have their weights get some activations too, so
            // that their barriers complete)
            for (; ahead > 0; --ahead) acts(p.h);
            // what is in flight lands before the CTA ends
            for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(b_full + 8 * (i % S), (uint32_t)(i / S) & 1u, kWaitCycles);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        int slot = 0, seg = 0;
        uint32_t par = 0, sf_set = 0;
        bool ok = true;
        auto run = [&](int n) {  // n stages into the next accumulator
            const int buf = seg & 1;
            ok = ok && (seg < 2 || __all_sync(0xffffffffu, mbar_wait(b_read + 8 * buf, (uint32_t)(seg / 2 - 1) & 1u, lim)));
            tc::fence_after_sync();
            const uint32_t d = tmem + 16 * buf;
            for (int i = 0; ok && i < n; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait(b_full + 8 * slot, par, lim));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint32_t a = ring + slot * kMoeStage, b = a + REC;
                    const uint32_t ta = tmem + 32 + sf_set, tb = ta + 8;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        mx_copy_scales(ta + 4 * w, a + kMxCodes + 512 * w);
                        mx_copy_scales(tb + 4 * w, b + 2048 + 512 * w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mx_mma<0>(d, tc::desc_sw128(a + 32 * j, 0), tc::desc_sw128(b + 32 * j, 0),
                                  mx_idesc<0>(16, 2 * (j % 2)), ta + 4 * (j / 2), tb + 4 * (j / 2), i | j);
                    tc::commit(b_empty + 8 * slot);
                    if (i + 1 == n) tc::commit(b_acc + 8 * buf);
                }
                __syncwarp();
                sf_set ^= 16;
                if (++slot == S) {
                    slot = 0;
                    par ^= 1;
                }
            }
            ++seg;
            return ok;
        };
        bool more = cta < units;
        for (int count = 0; ok && more; ++count) {
            run(KS1);
            more = ok && more_s[count & 15] != 0;
        }
        if (ok)
            walk([&](int, int q0, int q1) {
                for (int q = q0; ok && q < q1;) {
                    const int e = min(q1, (q / KS2 + 1) * KS2);
                    run(e - q);
                    q = e;
                }
                return ok;
            });
        if (!ok && lane == 0) atomicExch(p.err, 4);
        if (tc::elect_one()) tc::commit(b_drain);
        __syncwarp();
        mbar_wait(b_drain, 0u, kWaitCycles);
    } else if (warp < 6) {
        // ------------------------------------------------------------ sums
        const int q = warp & 3, pair = q >> 1, up = q & 1, rl = 32 * q + lane;
        int seg = 0;
        bool ok = true;
        auto take = [&](float (&v)[16]) {  // the next accumulator's row of this lane
            const int buf = seg & 1;
            // (a wait that gave up: the barrier and the counts are kept up, what is stored is undefined)
            ok = ok && __all_sync(0xffffffffu, mbar_wait(b_acc + 8 * buf, (uint32_t)(seg / 2) & 1u, lim));
            tc::fence_after_sync();
            uint32_t w[16];
            tc::ld16(tmem + 16 * buf + ((uint32_t)(32 * q) << 16), w);
            tc::wait_ld16(w);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
            tc::fence_before_sync();
            __syncwarp();
            if (ok && lane == 0) bar_arrive(b_read + 8 * buf);  // (after a failure a phase could get too many)
            ++seg;
        };
        // a tile's rows: 32 of gate, 32 of up, twice: a warp has the gates or the ups of a
        // block of h.  The gates' warp takes tokens 0-7 of it, the ups' 8-15.
        float *exch = reinterpret_cast<float *>(sm + kMoeOffExch) + pair * 512;
        bool more = cta < units;
        for (int count = 0; more; ++count) {
            float v[16];
            take(v);
            float *buf = exch + (seg & 1) * 1024;
#pragma unroll
            for (int i = 0; i < 8; ++i) buf[(up * 8 + i) * 32 + lane] = up ? v[i] : v[8 + i];
            // (one warp's wait may give up just before the other's passes: both leave, or none)
            ok = bar_all(2 + pair, 64, ok);
            if (!ok) break;
            const int u = unit_s[count & 15];
            more = more_s[count & 15] != 0;
            const int a = u / T1, tile = u - a * T1, blk = 2 * tile + pair;
            const unsigned mask = masks[a];
            const bool in = blk * 32 < p.inter;
            uint8_t *rec = p.h + ((size_t)a * KS2 + blk / 8) * kMoeRec;
            // this block, and behind the last one the rest of its record as zeros
            const int end = 2 * tile + 2 >= p.inter / 32 && pair == 1 ? 8 : blk % 8 + 1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = up * 8 + i;
                if (!((mask >> t) & 1u)) continue;
                const float o = buf[((1 - up) * 8 + i) * 32 + lane];
                const float g = up ? o : v[i], w = up ? v[8 + i] : o;
                const float h = in ? mx_silu(g) * w : 0.f;
                float mul;
                const uint32_t sc = mx_block_scale<0>(
                    __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu)), MxGain{}, mul);
                uint32_t code = (mul == 0.f ? 0u : e2m1(h * mul)) << (4 * (lane & 7));
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) code |= __shfl_xor_sync(0xffffffffu, code, x);
                if (blk / 8 < KS2)
                    for (int b = blk % 8; b < end; ++b) {
                        const bool own = b == blk % 8;
                        if (lane % 8 == 0)
                            *reinterpret_cast<uint32_t *>(rec + mx_code_off(t, 16 * b + lane / 2)) = own ? code : 0u;
                        if (lane == 0) rec[2048 + (b >> 2) * 512 + t * 16 + (b & 3)] = own ? (uint8_t)sc : (uint8_t)0;
                    }
            }
        }
        asm volatile("fence.proxy.async;" ::: "memory");  // h, for the copies of other CTAs
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (warp == 2 && lane == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.barrier) : "memory");

        if (line == 0)  // only idle rows
            for (int m = cta; m < T2; m += grid)
                for (int t = 0; t < p.nb; ++t) store(m * kMxRows + rl, t, 0.f);
        int nseg = 0;
        walk([&](int m, int q0, int q1) {
            float sum[16] = {};
            for (int k = q0; k < q1;) {
                const int a = k / KS2;
                const unsigned mask = masks[a];
                float v[16];
                take(v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if ((mask >> i) & 1u) sum[i] = fmaf(wtab[a * 16 + i], v[i], sum[i]);
                k = min(q1, (a + 1) * KS2);
            }
            const int slot_of = nseg++ > 0;
            if (q1 - q0 == line) {
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t < p.nb) store(m * kMxRows + rl, t, sum[t]);
                return true;
            }
            float *mine = p.part + ((size_t)cta * 2 + slot_of) * slot_floats + rl;
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (t < p.nb) __stcg(mine + t * kMxRows, sum[t]);
            // the last of the tile's CTAs joins the parts, below
            int f, l;
            sharers(m, f, l);
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (warp == 2 && lane == 0) {
                unsigned before;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.count + m) : "memory");
                if ((int)before == l - f) info[1 + slot_of] = m;
            }
            return true;
        });
        if (!ok && lane == 0) atomicExch(p.err, 4);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 128);
    }
    // Tiles whose last part came from here: a thread a row and every fourth token, the
    // parts in CTA order, five of all its tokens at once.  (By the four warps of the sums, a
    // few loads at a time, 16 tokens took 13 us; a token after the other 7.)
    for (int j = 0; j < 2; ++j) {
        const int m = info[1 + j];
        if (m < 0) continue;
        int f, l;
        sharers(m, f, l);
        const int rl = tid & (kMxRows - 1);
        // CTA f's part is its second if it began in an earlier tile, the others' their first
        const float *part0 = p.part + ((size_t)f * 2 + (first_of(f) < (long long)m * line)) * slot_floats + rl;
        const float *parts = p.part + rl;
        constexpr int TT = kMaxNb * kMxRows / kMoeThreads, X = 5;  // a thread's tokens, parts at once
        const int t0 = tid / kMxRows;
        float v[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) v[i] = t0 + 4 * i < p.nb ? __ldcg(part0 + (t0 + 4 * i) * kMxRows) : 0.f;
        for (int x = f + 1; x <= l; x += X) {
            float o[X][TT];
#pragma unroll
            for (int j = 0; j < X; ++j)
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    o[j][i] = x + j <= l && t0 + 4 * i < p.nb ? __ldcg(parts + (size_t)(x + j) * 2 * slot_floats + (t0 + 4 * i) * kMxRows) : 0.f;
#pragma unroll
            for (int j = 0; j < X; ++j)
#pragma unroll
                for (int i = 0; i < TT; ++i) v[i] += o[j][i];
        }
#pragma unroll
        for (int i = 0; i < TT; ++i)
            if (t0 + 4 * i < p.nb) store(m * kMxRows + rl, t0 + 4 * i, v[i]);
    }
}

// Sixteen bytes of codes, or a word of scales, of a row a thread.  When a layer is made: 128
// experts of 768 x 2048 149 us (2.9 TB/s read and written).
__global__ void __launch_bounds__(256) q4moe_pack_kernel(const __grid_constant__ MoePackParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int KT = mx_ktiles(p.k), lane = threadIdx.x & 15;  // 16 threads a record's row
    const long long u = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / 16, units = 2ll * p.batch * p.rows * KT;
    if (u >= units) return;
    const int kt = (int)(u % KT);
    const long long row = u / KT, b = row / (2 * p.rows);
    const int ro = (int)(row - b * 2 * p.rows), ri = (ro / 64) * 32 + ro % 32;  // the output's row, its source's
    const uint8_t *src = (ro & 32 ? p.up : p.gate) + ((b * mx_rtiles(p.rows) + ri / kMxRows) * KT + kt) * mx_rec(0);
    uint8_t *dst = p.out + ((b * mx_rtiles(2 * p.rows) + ro / kMxRows) * KT + kt) * mx_rec(0);
    const int si = ri % kMxRows, so = ro % kMxRows;
    if (lane < 8)
        *reinterpret_cast<uint4 *>(dst + mx_code_off(so, 16 * lane)) = *reinterpret_cast<const uint4 *>(src + mx_code_off(si, 16 * lane));
    else if (lane < 10)
        *reinterpret_cast<uint32_t *>(dst + mx_scale_off(so, lane - 8)) = *reinterpret_cast<const uint32_t *>(src + mx_scale_off(si, lane - 8));
}

}  // namespace dev

constexpr int kMoeMaxCtas = 256;  // CTAs of the experts' kernel at most (its parts)

size_t moe_workspace(MoeParams &p, uint8_t *ws) {
    size_t at = 0;
    auto room = [&](size_t bytes) {
        uint8_t *x = ws ? ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return x;
    };
    uint8_t *ctl = room(256);
    p.barrier = (unsigned *)ctl;
    p.units = ws ? (unsigned *)(ctl + 128) : nullptr;
    p.count = (unsigned *)room(sizeof(unsigned) * mx_rtiles(p.hidden));
    p.logits = (float *)room(sizeof(float) * p.nb * p.E);
    p.xq = room((size_t)mx_ktiles(p.hidden) * kMoeRec);
    p.h = room((size_t)std::min(p.E, p.nb * p.top_k) * mx_ktiles(p.inter) * kMoeRec);
    p.part = (float *)room(sizeof(float) * kMoeMaxCtas * 2 * p.nb * kMxRows);
    return at;
}

template <typename T>
static int launch_route(const MoeParams &p, cudaStream_t stream) {
    auto kern = p.nb == 1 ? dev::q4moe_route_kernel<T, 1> : dev::q4moe_route_kernel<T, 4>;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)(p.E + p.nb), 32 * dev::kRouteSlices * ((p.nb + 3) / 4), 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

template <typename T>
static int launch_experts(const MoeParams &p, int sms, cudaStream_t stream) {
    auto kern = dev::q4moe_experts_kernel<T>;
    static size_t smem_set[64] = {0};
    if (!raise_smem(kern, dev::kMoeSmem, smem_set)) return -1;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config((unsigned)std::min(sms, kMoeMaxCtas), dev::kMoeThreads, dev::kMoeSmem, stream, attr);
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

int launch_moe(const MoeParams &p, int x_dtype, int y_dtype, int sms, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    const int rc = x_dtype == 0 ? launch_route<float>(p, s) : x_dtype == 1 ? launch_route<__half>(p, s) : launch_route<__nv_bfloat16>(p, s);
    if (rc != 0) return rc;
    return y_dtype == 0 ? launch_experts<float>(p, sms, s) : y_dtype == 1 ? launch_experts<__half>(p, sms, s) : launch_experts<__nv_bfloat16>(p, sms, s);
}

int launch_moe_pack(const MoePackParams &p, void *stream) {
    const long long threads = 16ll * 2 * p.batch * p.rows * mx_ktiles(p.k);
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)((threads + 255) / 256), 256, 0, (cudaStream_t)stream, &attr);
    return cudaLaunchKernelEx(&cfg, dev::q4moe_pack_kernel, p) == cudaSuccess ? 0 : -1;
}

}  // namespace q4
