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
#include <algorithm>
#include <atomic>

#include "mx_common.cuh"

namespace q4 {
namespace dev {

// ------------------------------------------------------------------ routing

constexpr int kRouteThreads = 256, kRouteWarps = kRouteThreads / 32;
constexpr int kRouteTok = 4;  // tokens of a warp

template <typename T>
__device__ __forceinline__ float4 load4(const T *src) {
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float4 *>(src);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(src);
        const T *v = reinterpret_cast<const T *>(&w);
        return make_float4(to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3]));
    }
}

// Order of logits: larger first, NaN behind every number.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);  // (-0 is 0)
    return v != v ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
}

// One token's choice by a warp: its experts into idx and weight [top_k].
__device__ __forceinline__ void route_token(const float *logits, int E, int top_k, bool renorm, int32_t *idx,
                                            float *weight, int lane) {
    constexpr int NL = kMoeMaxExperts / 32;
    uint32_t taken = 0;  // bit i: expert 32 i + lane is chosen
    float top = 0.f, mine = 0.f;
    int at = 0;
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = 0;
        int where = -1;
        float bv = 0.f;
        for (int i = 0; 32 * i < E; ++i) {
            const int e = 32 * i + lane;
            if (e >= E || ((taken >> i) & 1u)) continue;
            const float v = __ldcg(logits + e);
            const uint32_t key = logit_key(v);
            if (where < 0 || key > best) {
                best = key;
                where = e;
                bv = v;
            }
        }
        static_assert(NL <= 32, "a bit each");
        const uint32_t most = __reduce_max_sync(0xffffffffu, where < 0 ? 0u : best);
        const uint32_t first = __reduce_min_sync(0xffffffffu, where >= 0 && best == most ? (uint32_t)where : 0xFFFFFFFFu);
        const int from = (int)first & 31;
        const float v = __shfl_sync(0xffffffffu, bv, from);
        if (lane == from) taken |= 1u << (first >> 5);
        if (j == 0) top = v;
        if (lane == j) {
            mine = v;
            at = (int)first;
        }
    }
    // softmax with the largest logit as its reference (NaN where one is NaN)
    float p = lane < top_k ? expf(mine - top) : 0.f, sum = p;
    if (!renorm) {
        sum = 0.f;
        for (int e = lane; e < E; e += 32) sum += expf(__ldcg(logits + e) - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < top_k) {
        idx[lane] = at;
        weight[lane] = p / sum;
    }
}

// CTAs below `nl`: logits, a warp an expert and four tokens.  The others: a row of
// x each, its norm and its codes.  The last CTA to finish chooses the experts and
// lists those with a token.
template <typename T>
__global__ void __launch_bounds__(kRouteThreads) q4moe_route_kernel(const __grid_constant__ MoeParams p, const int nl) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float sums[kRouteWarps];
    __shared__ int is_last, count;
    __shared__ unsigned tokens[kMoeMaxExperts];
    __shared__ int slot[kMoeMaxExperts];
    __shared__ int32_t chosen[kMaxNb][kMoeMaxTop];
    __shared__ float weights[kMaxNb][kMoeMaxTop];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *x = (const T *)p.x;
    if ((int)blockIdx.x < nl) {
        const int groups = (p.nb + kRouteTok - 1) / kRouteTok, u = blockIdx.x * kRouteWarps + warp;
        const int e = u / groups, t0 = (u - e * groups) * kRouteTok;
        if (e < p.E) {
            float dot[kRouteTok] = {}, sq[kRouteTok] = {};
            const float *row = p.router + (size_t)e * p.hidden;
#pragma unroll 2
            for (int c = 4 * lane; c < p.hidden; c += 128) {
                float4 w = *reinterpret_cast<const float4 *>(row + c);
                if (p.gamma) {
                    const float4 g = *reinterpret_cast<const float4 *>(p.gamma + c);
                    w = make_float4(w.x * g.x, w.y * g.y, w.z * g.z, w.w * g.w);
                }
#pragma unroll
                for (int i = 0; i < kRouteTok; ++i) {
                    if (t0 + i >= p.nb) break;
                    const float4 v = load4(x + (t0 + i) * p.ldx + c);
                    dot[i] = fmaf(v.x, w.x, fmaf(v.y, w.y, fmaf(v.z, w.z, fmaf(v.w, w.w, dot[i]))));
                    sq[i] = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, sq[i]))));
                }
            }
#pragma unroll
            for (int i = 0; i < kRouteTok; ++i)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
                    sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
                }
#pragma unroll
            for (int i = 0; i < kRouteTok; ++i)
                if (lane == i && t0 + i < p.nb)
                    p.logits[(size_t)(t0 + i) * p.E + e] =
                        p.gamma ? dot[i] * (1.f / sqrtf(sq[i] / (float)p.hidden + p.eps)) : dot[i];
        }
    } else {
        const int t = blockIdx.x - nl, KT = mx_ktiles(p.hidden);
        const T *src = x + t * p.ldx;
        float rstd = 1.f;
        auto load = [&](int kt, float (&v)[8]) {
            const int c = kt * kMxK + 8 * lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
            if (c < p.hidden) {
                const float4 a = load4(src + c), b = load4(src + c + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            }
        };
        if (p.gamma) {
            float sum = 0.f;
            for (int kt = warp; kt < KT; kt += kRouteWarps) {
                float v[8];
                load(kt, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) sums[warp] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < kRouteWarps; ++i) sum += sums[i];
            rstd = 1.f / sqrtf(sum / (float)p.hidden + p.eps);
        }
        for (int kt = warp; kt < KT; kt += kRouteWarps) {
            const int c = kt * kMxK + 8 * lane;
            float v[8];
            load(kt, v);
            if (p.gamma && c < p.hidden) {
                const float4 a = *reinterpret_cast<const float4 *>(p.gamma + c);
                const float4 b = *reinterpret_cast<const float4 *>(p.gamma + c + 4);
                v[0] *= rstd, v[1] *= rstd, v[2] *= rstd, v[3] *= rstd;
                v[4] *= rstd, v[5] *= rstd, v[6] *= rstd, v[7] *= rstd;
                v[0] *= a.x, v[1] *= a.y, v[2] *= a.z, v[3] *= a.w;
                v[4] *= b.x, v[5] *= b.y, v[6] *= b.z, v[7] *= b.w;
            }
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            float mul;
            const uint32_t sc = mx_block_scale<0>(m, 1.f, 6.f, mul);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mx_scaled(v[i], mul);
            uint8_t *rec = p.xq + (size_t)kt * kMoeRec;
            *reinterpret_cast<uint32_t *>(rec + mx_code_off(t, 4 * lane)) = e2m1x8(v);
            if (lane % 4 == 0) rec[2048 + (lane >> 4) * 512 + t * 16 + ((lane >> 2) & 3)] = (uint8_t)sc;
        }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        unsigned before;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived) : "memory");
        is_last = before == gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    for (int e = tid; e < p.E; e += kRouteThreads) tokens[e] = 0u;
    for (int t = warp; t < p.nb; t += kRouteWarps) {
        if (p.positions && p.positions[t] < 0) {  // an idle row: no experts
            if (lane < p.top_k) {
                chosen[t][lane] = -1;
                weights[t][lane] = 0.f;
            }
        } else {
            route_token(p.logits + (size_t)t * p.E, p.E, p.top_k, p.renormalize != 0, chosen[t], weights[t], lane);
        }
    }
    __syncthreads();
    const int pairs = p.nb * p.top_k;
    for (int i = tid; i < pairs; i += kRouteThreads) {
        const int t = i / p.top_k, j = i - t * p.top_k, e = chosen[t][j];
        p.idx[i] = e;
        p.weight[i] = weights[t][j];
        if (e >= 0) atomicOr(&tokens[e], 1u << t);
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
                p.ids[s] = e;
                p.mask[s] = has;
            }
            n += __popc(hit);
        }
        if (lane == 0) {
            count = n;
            *p.active = n;
            *p.arrived = 0u;  // zero again for the next call
            *p.barrier = 0u;
        }
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += kRouteThreads) {
        const int t = i / p.top_k, e = chosen[t][i - t * p.top_k];
        if (e >= 0) p.wtab[slot[e] * 16 + t] = weights[t][i - t * p.top_k];
    }
}

// ------------------------------------------------------------------ experts

constexpr int kMoeThreads = 192;
constexpr int kMoeStages = 10;
constexpr int kMoeStage = mx_rec(0) + kMoeRec;  // a record of weights, one of activations
constexpr int kMoeSum = 12 * 1024;              // a cluster's parts of its columns: (16 + 8) 512 at most
constexpr int kMoeExch = 2 * 2 * 2 * 8 * 32 * 4;  // [turn][pair of warps][gate or up][token][row]
constexpr int kMoeOffSum = kMoeStages * kMoeStage, kMoeOffExch = kMoeOffSum + kMoeSum,
              kMoeOffBar = kMoeOffExch + kMoeExch, kMoeSmem = kMoeOffBar + 8 * (2 * kMoeStages + 5) + 16;
static_assert(kMoeStage % 1024 == 0 && kMoeSmem <= (int)kSmemMax, "shared memory of the experts' kernel");

// One kernel for both products: first every (expert with a token, 64 rows of gate
// and of up) unit, a CTA each in turn, then, behind a barrier of the grid, the down
// projections: a cluster of C CTAs a tile of 128 outputs, each CTA a part of the
// (expert, k) line.  The weights of the second half's first stages are on their way
// before the barrier.  warp 0 copies, warp 1 issues MMAs, warps 2-5 take the sums.
template <typename T>
__global__ void __launch_bounds__(kMoeThreads, 1) q4moe_experts_kernel(const __grid_constant__ MoeParams p, const int C) {
    constexpr int REC = mx_rec(0), S = kMoeStages;
    extern __shared__ __align__(1024) uint8_t sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t ring = smem_u32(sm), b_full = ring + kMoeOffBar, b_empty = b_full + 8 * S, b_acc = b_empty + 8 * S,
                   b_read = b_acc + 16, b_drain = b_read + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + kMoeOffBar + 8 * (2 * S + 5));
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
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;
    if (C > 1) cluster_sync();  // the cluster's CTAs run: their shared memory can be written
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int nA = *(const volatile int *)p.active;
    const int KS1 = mx_ktiles(p.hidden), KS2 = mx_ktiles(p.inter);
    const int T1 = mx_rtiles(2 * p.inter), T2 = mx_rtiles(p.hidden);
    const int units = nA * T1, grid = gridDim.x, cta = blockIdx.x;
    const int rank = C > 1 ? cta % C : 0, line = nA * KS2, q0 = (int)((long long)line * rank / C),
              q1 = (int)((long long)line * (rank + 1) / C);
    const long long lim = p.wait_cycles;

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            int it = 0;
            uint32_t extra = (uint32_t)p.extra_tx;
            bool ok = true;
            // the next slot's weights; its activations follow on the same barrier
            auto weights = [&](const uint8_t *src, int i) {
                const int s = i % S;
                if (i >= S && !mbar_wait(b_empty + 8 * s, (uint32_t)(i / S - 1) & 1u, lim)) return false;
                mbar_expect_tx(b_full + 8 * s, kMoeStage + extra);
                extra = 0;
                bulk_copy(ring + s * kMoeStage, src, REC, b_full + 8 * s);
                return true;
            };
            auto acts = [&](const uint8_t *src, int i) {
                bulk_copy(ring + (i % S) * kMoeStage + REC, src, kMoeRec, b_full + 8 * (i % S));
            };
            for (int u = cta; ok && u < units; u += grid) {
                const int a = u / T1, tile = u - a * T1;
                const uint8_t *w = p.gate_up + ((size_t)p.ids[a] * T1 + tile) * KS1 * REC;
                for (int ks = 0; ks < KS1; ++ks) {
                    ok = weights(w + (size_t)ks * REC, it);
                    if (!ok) break;
                    acts(p.xq + (size_t)ks * kMoeRec, it);
                    ++it;
                }
            }
            bool open = false;  // the first half is done in all CTAs
            int ahead = 0;      // stages with their weights on the way
            for (int m = cta / C; ok && m < T2; m += grid / C) {
                auto src = [&](int q) {
                    const int a = q / KS2;
                    return p.down + (((size_t)p.ids[a] * T2 + m) * KS2 + (q - a * KS2)) * REC;
                };
                if (!open) {
                    while (ahead < S && q0 + ahead < q1 && (ok = weights(src(q0 + ahead), it + ahead))) ++ahead;
                    const unsigned target = (unsigned)grid + (unsigned)p.barrier_extra;
                    for (long long n = 0; ok && ld_acquire_u32(p.barrier) < target; ++n) ok = n < p.barrier_polls;
                    asm volatile("fence.proxy.async;" ::: "memory");  // what others wrote, for this thread's copies
                    open = true;
                }
                for (int q = q0; ok && q < q1; ++q) {
                    if (ahead > 0)
                        --ahead;
                    else
                        ok = weights(src(q), it);
                    if (!ok) break;
                    acts(p.h + (size_t)q * kMoeRec, it);
                    ++it;
                }
            }
            if (!ok) atomicExch(p.err, 4);
            // (after a failure: the stages that have their weights get some activations too, so
            // that their barriers complete)
            for (; ahead > 0; --ahead, ++it) acts(p.h, it);
            // what is in flight lands before the CTA ends
            for (int i = max(0, it - S); i < it; ++i) mbar_wait(b_full + 8 * (i % S), (uint32_t)(i / S) & 1u, kWaitCycles);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        int it = 0, seg = 0;
        bool ok = true;
        auto run = [&](int n) {  // n stages into the next accumulator
            const int buf = seg & 1;
            ok = ok && (seg < 2 || __all_sync(0xffffffffu, mbar_wait(b_read + 8 * buf, (uint32_t)(seg / 2 - 1) & 1u, lim)));
            tc::fence_after_sync();
            const uint32_t d = tmem + 16 * buf;
            for (int i = 0; ok && i < n; ++i, ++it) {
                const int s = it % S;
                ok = __all_sync(0xffffffffu, mbar_wait(b_full + 8 * s, (uint32_t)(it / S) & 1u, lim));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint32_t a = ring + s * kMoeStage, b = a + REC;
                    const uint32_t ta = tmem + 32 + (it & 1) * 16, tb = ta + 8;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        mx_copy_scales(ta + 4 * w, a + kMxCodes + 512 * w);
                        mx_copy_scales(tb + 4 * w, b + 2048 + 512 * w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mx_mma<0>(d, tc::desc_sw128(a + 32 * j, 0), tc::desc_sw128(b + 32 * j, 0),
                                  mx_idesc<0>(16, 2 * (j % 2)), ta + 4 * (j / 2), tb + 4 * (j / 2), i | j);
                    tc::commit(b_empty + 8 * s);
                    if (i + 1 == n) tc::commit(b_acc + 8 * buf);
                }
                __syncwarp();
            }
            ++seg;
        };
        for (int u = cta; ok && u < units; u += grid) run(KS1);
        for (int m = cta / C; ok && m < T2; m += grid / C)
            for (int q = q0; ok && q < q1;) {
                const int e = min(q1, (q / KS2 + 1) * KS2);
                run(e - q);
                q = e;
            }
        if (!ok && lane == 0) atomicExch(p.err, 4);
        if (tc::elect_one()) tc::commit(b_drain);
        __syncwarp();
        mbar_wait(b_drain, 0u, kWaitCycles);
    } else {
        // ------------------------------------------------------------ sums
        const int q = warp & 3, pair = q >> 1, up = q & 1;
        int seg = 0;
        bool ok = true;
        auto take = [&](float (&v)[16]) {  // the next accumulator's row of this lane
            const int buf = seg & 1;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(b_acc + 8 * buf, (uint32_t)(seg / 2) & 1u, lim));
            tc::fence_after_sync();
            uint32_t w[16];
            tc::ld16(tmem + 16 * buf + ((uint32_t)(32 * q) << 16), w);
            tc::wait_ld16(w);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(b_read + 8 * buf);
            ++seg;
        };
        // a tile's rows: 32 of gate, 32 of up, twice: a warp has the gates or the ups of a
        // block of h.  The gates' warp takes tokens 0-7 of it, the ups' 8-15.
        float *exch = reinterpret_cast<float *>(sm + kMoeOffExch) + pair * 512;
        for (int u = cta; u < units; u += grid) {
            const int a = u / T1, tile = u - a * T1, blk = 2 * tile + pair;
            const unsigned mask = p.mask[a];
            float v[16];
            take(v);
            float *buf = exch + (seg & 1) * 1024;
#pragma unroll
            for (int i = 0; i < 8; ++i) buf[(up * 8 + i) * 32 + lane] = up ? v[i] : v[8 + i];
            asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory");
            const bool in = blk * 32 < p.inter;
            uint8_t *rec = p.h + ((size_t)a * KS2 + blk / 8) * kMoeRec;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = up * 8 + i;
                if (!((mask >> t) & 1u)) continue;
                const float o = buf[((1 - up) * 8 + i) * 32 + lane];
                const float g = up ? o : v[i], w = up ? v[8 + i] : o;
                const float h = in ? g / (1.f + __expf(-g)) * w : 0.f;
                float mul;
                const uint32_t sc = mx_block_scale<0>(
                    __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu), 1.f, 6.f, mul);
                uint32_t code = e2m1(mx_scaled(h, mul)) << (4 * (lane & 7));
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) code |= __shfl_xor_sync(0xffffffffu, code, x);
                // this block, and behind the last one the rest of its record as zeros
                const int last = blk % 8 + 1 < 8 && 2 * tile + 2 >= p.inter / 32 && pair == 1 ? 8 : blk % 8 + 1;
                if (blk / 8 < KS2)
                    for (int b = blk % 8; b < last; ++b) {
                        const uint32_t word = b == blk % 8 ? code : 0u;
                        if (lane % 8 == 0)
                            *reinterpret_cast<uint32_t *>(rec + mx_code_off(t, 16 * b + lane / 2)) = word;
                        if (lane == 0) rec[2048 + (b >> 2) * 512 + t * 16 + (b & 3)] = b == blk % 8 ? (uint8_t)sc : (uint8_t)0;
                    }
            }
        }
        __threadfence();
        asm volatile("fence.proxy.async;" ::: "memory");  // h, for the copies of other CTAs
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (warp == 2 && lane == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.barrier) : "memory");

        const int rl = 32 * q + lane;
        for (int m = cta / C; m < T2; m += grid / C) {
            float sum[16] = {};
            for (int k = q0; k < q1;) {
                const int a = k / KS2;
                const unsigned mask = p.mask[a];
                float4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(p.wtab + a * 16 + 4 * i);
                float v[16];
                take(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float wi = i % 4 == 0 ? w[i / 4].x : i % 4 == 1 ? w[i / 4].y : i % 4 == 2 ? w[i / 4].z : w[i / 4].w;
                    if ((mask >> i) & 1u) sum[i] = fmaf(wi, v[i], sum[i]);
                }
                k = min(q1, (a + 1) * KS2);
            }
            const int row = m * kMxRows + rl;
            if (C > 1) {
                // token t's sum to the CTA that adds it: ranks of `per` tokens each
                const int per = (16 + C - 1) / C;
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t < p.nb) {
                        const int to = t / per;
                        store_peer(ring + kMoeOffSum + 4 * ((rank * per + t - to * per) * kMxRows + rl), (uint32_t)to, sum[t]);
                    }
            } else if (row < p.hidden) {
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t < p.nb) {
                        const size_t at = (size_t)t * p.hidden + row;
                        ((T *)p.y)[at] = from_f32<T>(p.r ? sum[t] + to_f32(((const T *)p.r)[at]) : sum[t]);
                    }
            }
        }
        if (!ok && lane == 0) atomicExch(p.err, 4);
    }
    if (C > 1) {
        __syncwarp();
        cluster_sync();
        const int per = (16 + C - 1) / C, m = cta / C, rl = 32 * (warp & 3) + lane, row = m * kMxRows + rl;
        if (warp >= 2 && m < T2 && row < p.hidden) {
            const float *part = reinterpret_cast<const float *>(sm + kMoeOffSum) + rl;
            for (int i = 0; i < per && rank * per + i < p.nb; ++i) {
                const size_t at = (size_t)(rank * per + i) * p.hidden + row;
                float v = 0.f;
                for (int x = 0; x < C; ++x) v += part[(x * per + i) * kMxRows];
                ((T *)p.y)[at] = from_f32<T>(p.r ? v + to_f32(((const T *)p.r)[at]) : v);
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 128);
    }
}

// Sixteen bytes of codes, or a word of scales, of a row a thread.
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

size_t moe_workspace(MoeParams &p, uint8_t *ws) {
    size_t at = 0;
    auto room = [&](size_t bytes) {
        uint8_t *x = ws ? ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return x;
    };
    const size_t active = std::min(p.E, p.nb * p.top_k);
    uint8_t *ctl = room(256);
    p.arrived = (unsigned *)ctl;
    p.barrier = ws ? (unsigned *)(ctl + 64) : nullptr;
    p.active = ws ? (int *)(ctl + 128) : nullptr;
    p.logits = (float *)room(sizeof(float) * p.nb * p.E);
    p.ids = (int *)room(sizeof(int) * active);
    p.mask = (unsigned *)room(sizeof(unsigned) * active);
    p.wtab = (float *)room(sizeof(float) * 16 * active);
    p.xq = room((size_t)mx_ktiles(p.hidden) * kMoeRec);
    p.h = room(active * mx_ktiles(p.inter) * kMoeRec);
    return at;
}

template <typename T>
static int launch_route(const MoeParams &p, cudaStream_t stream) {
    const int warps = p.E * ((p.nb + dev::kRouteTok - 1) / dev::kRouteTok), nl = (warps + dev::kRouteWarps - 1) / dev::kRouteWarps;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)(nl + p.nb), dev::kRouteThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, dev::q4moe_route_kernel<T>, p, nl) == cudaSuccess ? 0 : -1;
}

template <typename T>
static int launch_experts(const MoeParams &p, int sms, cudaStream_t stream) {
    auto kern = dev::q4moe_experts_kernel<T>;
    static size_t smem_set[64] = {0};
    if (!raise_smem(kern, dev::kMoeSmem, smem_set)) return -1;
    // a cluster a tile of outputs, as wide as the device holds that many
    const int T2 = mx_rtiles(p.hidden);
    const int C = std::max(1, std::min(8, sms / T2));
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(dev::kMoeThreads, 1, 1);
    cfg.dynamicSmemBytes = dev::kMoeSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[3];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    attr[2].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[2].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // clusters of c CTAs that the device holds at once, 0: not asked yet
    static std::atomic<int> held[64][9];
    int dev_id = 0;
    if (cudaGetDevice(&dev_id) != cudaSuccess || dev_id < 0 || dev_id >= 64) return -1;
    for (int c = C; c >= 1; --c) {
        attr[0].val.clusterDim.x = (unsigned)c;
        int n = held[dev_id][c].load(std::memory_order_relaxed);
        if (n == 0) {
            cfg.gridDim = dim3((unsigned)(sms / c * c), 1, 1);
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) return -1;
            held[dev_id][c].store(n, std::memory_order_relaxed);
        }
        if (c > 1 && n < T2) continue;
        cfg.gridDim = dim3((unsigned)(std::min(n, sms / c) * c), 1, 1);
        cfg.numAttrs = 3;
        return cudaLaunchKernelEx(&cfg, kern, p, c) == cudaSuccess ? 0 : -1;
    }
    return -1;
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
