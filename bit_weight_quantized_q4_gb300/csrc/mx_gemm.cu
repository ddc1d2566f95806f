// mx_gemm.cu -- the product of two microscaled 4-bit matrices, y = alpha x w^T
// (+ r), w [n][k], x [nb][k], on the block-scaled tensor core: both operands go
// into tcgen05.mma as they are stored, so that no weight is ever dequantised.
//
// This file: up to 64 rows of x in one tile of columns (mx_pair.cu: more). w's rows are
// the instruction's 128 rows and x's its columns, for one token too: the columns that a few
// tokens leave empty (16 at least) cost the tensor core less time than the weights take to
// arrive.  A record of w is one bulk copy, scales and all; x's rows and scales come by bulk
// copies into the same stage; the scales go from shared to tensor memory (tcgen05.cp) in
// front of their MMAs.  Few row tiles: a cluster shares k, its sums meet in shared memory.
//   warp 0 copies, warp 1 issues MMAs, warps 2-5 write the results, while the
//   tensor core is at the next tile (two accumulators).
// The weights' stream bounds it: one row at 65536 x 8192 takes 42.9 us (6.7 TB/s), 64 rows
// 47; at 14336 x 4096 one row 7.8 (4.0 TB/s: 112 row tiles are 112 CTAs, so that 40 SMs have no
// part, and an SM draws 44 GB/s; a launch and the first copies' latency), at 4096 x 14336 8.8,
// at 4096 x 4096 4.8.
// A few rows that are not quantised yet are quantised here (QX): warps 6-9 write
// their codes and scales into the stages, while w's records arrive.
#include <algorithm>

#include "mx_rows.cuh"

namespace q4 {
namespace dev {

constexpr int kMxgThreads = 192, kMxgQuant = 128;  // and the threads that quantise
constexpr int kMxgMaxN = 64;        // columns of a tile
constexpr int kMxgMaxStages = 12;
constexpr int kMxgBars = (8 * (2 * kMxgMaxStages + 5) + 16 + 15) / 16 * 16;

template <int FMT, typename T, bool QX>
__global__ void __launch_bounds__(kMxgThreads + (QX ? kMxgQuant : 0), 2)
    q4mx_gemm_kernel(const __grid_constant__ MxGemmParams p) {
    constexpr int W = mx_words(FMT), REC = mx_rec(FMT);
    extern __shared__ __align__(1024) uint8_t sm[];  // the swizzle's pattern repeats every 1024 bytes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int S = p.stages, C = p.C, tiles = p.MT, rank = C > 1 ? blockIdx.x % C : 0;
    const int k0 = p.KS * rank / C, k1 = p.KS * (rank + 1) / C;  // this CTA's part of k
    constexpr uint32_t cols_tm = 256, sf_tm = 2 * kMxgMaxN;  // tensor memory: two accumulators, two sets of scales
    const uint32_t ring = smem_u32(sm), bars = ring + S * p.stage_bytes;
    // barriers: a stage has landed, a stage's MMAs are done; of an accumulator: it is
    // complete, it has been read; the last MMAs of all
    const uint32_t b_full = bars, b_empty = b_full + 8 * kMxgMaxStages, b_acc = b_empty + 8 * kMxgMaxStages,
                   b_read = b_acc + 16, b_drain = b_read + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + S * p.stage_bytes + 8 * (2 * kMxgMaxStages + 5));
    if (warp == 0) {
        if (lane < S) {
            mbar_init(b_full + 8 * lane, QX ? 2 : 1);
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
        tc::tmem_alloc(smem_u32(tslot), cols_tm);
        tc::tmem_relinquish();
        // after the allocation: a kernel that starts on this could hold the columns this one waits for
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;

    // this CTA's tiles: f(tile) until it says no
    auto walk = [&](auto f) {
        for (int t = blockIdx.x / C; t < tiles; t += gridDim.x / C)
            if (!f(t)) return;
    };
    const int N = p.NB;
    const long long lim = p.wait_cycles;

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        // (one thread's chain of instructions: what a tile's stages share is computed once,
        // and slots are counted, not divided; with that left to every stage the copies, not the
        // tensor core or the memory, set the pace)
        if (lane == 0) {
            uint32_t extra = (uint32_t)p.extra_tx;
            const int t0 = blockIdx.x / C;
            auto source = [&](int t) { return p.w + ((size_t)t * p.KS + k0) * REC; };
            const uint32_t bytes = QX ? REC : REC + N * 128 + 512 * W;
            int ahead = 0;  // stages with their copies of w, but not of x
            if (p.early && t0 < tiles) {
                // the first stages' weights before what is in front of this kernel is done
                const uint8_t *w = source(t0);
                for (; ahead < min(S, k1 - k0); ++ahead) {
                    mbar_expect_tx(b_full + 8 * ahead, bytes + extra);
                    extra = 0;
                    bulk_copy(ring + ahead * p.stage_bytes, w + (size_t)ahead * REC, REC, b_full + 8 * ahead);
                }
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int slot = 0, issued = 0;
            uint32_t par = 1, dst = ring, bar = b_full;  // (a wait for the phase before the first passes)
            walk([&](int t) {
                const uint8_t *w = source(t), *b = p.x + (size_t)k0 * REC, *sf = b + kMxCodes;
                const uint32_t len = N * 128, osf = REC + len;
                for (int ks = k0; ks < k1; ++ks) {
                    if (ahead > 0) {
                        --ahead;
                    } else {
                        if (!mbar_wait(bar + 8 * kMxgMaxStages, par, lim)) {  // b_empty of this slot
                            atomicExch(p.err, 4);
                            return false;
                        }
                        mbar_expect_tx(bar, bytes + extra);
                        extra = 0;
                        bulk_copy(dst, w, REC, bar);
                    }
                    if constexpr (!QX) {
                        bulk_copy(dst + REC, b, len, bar);
                        bulk_copy(dst + osf, sf, 512 * W, bar);
                    }
                    w += REC, b += REC, sf += REC;
                    ++issued;
                    dst += p.stage_bytes, bar += 8;
                    if (++slot == S) {
                        slot = 0;
                        par ^= 1;
                        dst = ring;
                        bar = b_full;
                    }
                }
                return true;
            });
            // what is in flight lands before the CTA ends
            for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(b_full + 8 * (i % S), (uint32_t)(i / S) & 1u, kWaitCycles);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        int slot = 0, seg = 0;
        uint32_t par = 0, sf_set = 0;
        bool ok = true;
        walk([&](int) {
            const int buf = seg & 1;
            ok = seg < 2 || __all_sync(0xffffffffu, mbar_wait(b_read + 8 * buf, (uint32_t)(seg / 2 - 1) & 1u, lim));
            tc::fence_after_sync();
            const uint32_t d = tmem + buf * kMxgMaxN;
            const uint32_t idesc0 = mx_idesc<FMT>(N, 0), idesc2 = mx_idesc<FMT>(N, FMT == 0 ? 2 : 0);
            for (int ks = k0; ok && ks < k1; ++ks) {
                ok = __all_sync(0xffffffffu, mbar_wait(b_full + 8 * slot, par, lim));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint32_t a = ring + slot * p.stage_bytes, b = a + REC, sb = b + N * 128;
                    const uint32_t ta = tmem + sf_tm + sf_set, tb = ta + 16;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        mx_copy_scales(ta + 4 * w, a + kMxCodes + 512 * w);
                        mx_copy_scales(tb + 4 * w, sb + 512 * w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int w = FMT == 0 ? j / 2 : j;
                        mx_mma<FMT>(d, tc::desc_sw128(a + 32 * j, 0), tc::desc_sw128(b + 32 * j, 0), j % 2 ? idesc2 : idesc0,
                                    ta + 4 * w, tb + 4 * w, (ks - k0) | j);
                    }
                    tc::commit(b_empty + 8 * slot);
                    if (ks + 1 == k1) tc::commit(b_acc + 8 * buf);
                }
                __syncwarp();
                sf_set ^= 64;
                if (++slot == S) {
                    slot = 0;
                    par ^= 1;
                }
            }
            ++seg;
            return ok;
        });
        if (!ok && lane == 0) atomicExch(p.err, 4);
        if (tc::elect_one()) tc::commit(b_drain);
        __syncwarp();
        mbar_wait(b_drain, 0u, kWaitCycles);
    } else if (QX && warp >= 6) {
        // ------------------------------------------------------------ rows of x into the stages
        // Every fourth stage a warp, two rows (a half warp each, sixteen values a lane) or two
        // such pairs at a time; D steps' loads are under way.  (All four warps on each stage, its
        // loads a stage ahead: 0.7 us a stage, the loads' latency.)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr int NQ = kMxgQuant / 32;
        const int w = warp - 6, half = lane >> 4, h = lane & 15, pairs = (p.nb + 1) / 2, len = k1 - k0;
        const MxGain gain{p.src.scale, p.src.six_g, p.src.inv};
        const T *x = (const T *)p.src.x, *up = (const T *)p.src.up;
        const int mine = (tiles - (int)blockIdx.x / C + (int)gridDim.x / C - 1) / ((int)gridDim.x / C);
        const int total = mine * len;  // tiles of this CTA, their stages
        bool ok = true;
        auto quantise = [&](auto glu) {
            constexpr bool GLU = decltype(glu)::value;
            constexpr int P = GLU ? 1 : 2;  // pairs of rows a step
            constexpr int D = (sizeof(T) == 2 ? 2 : 1) * (GLU ? 2 : 1);
            struct At {  // the stage and the first pair that a step loads, or stores
                int it, ks, pair;
            };
            auto next = [&](At &a) {
                a.pair += P;
                if (a.pair >= pairs) {
                    a.pair = 0;
                    a.it += NQ;
                    a.ks += NQ;
                    while (a.ks >= len) a.ks -= len;
                }
            };
            At in = {w, w % len, 0};
            Raw16<T> a[D][P], b[GLU ? D : 1][P];
            auto fetch = [&](int d) {
                const int c = (k0 + in.ks) * kMxK + 16 * h;
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const int row = 2 * (in.pair + q) + half;
                    a[d][q].zero();
                    if constexpr (GLU) b[d][q].zero();
                    if (in.it < total && row < p.nb && c < p.src.k) {
                        a[d][q].load(x + row * p.src.ld + c);
                        if constexpr (GLU) b[d][q].load(up + row * p.src.ld + c);
                    }
                }
                next(in);
            };
#pragma unroll
            for (int d = 0; d < D; ++d) fetch(d);
            At out = {w, w % len, 0};
            int slot = w;  // (a ring has more than four)
            uint32_t par = 1;
            while (ok && out.it < total) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (!ok || out.it >= total) break;
                    if (out.pair == 0) ok = __all_sync(0xffffffffu, mbar_wait(b_empty + 8 * slot, par, lim));
                    if (!ok) break;
                    uint64_t v[P][8];
#pragma unroll
                    for (int q = 0; q < P; ++q) a[d][q].pairs(v[q]);
                    if constexpr (GLU) {
                        uint64_t u[8];
                        b[d][0].pairs(u);
                        mx_glu(v[0], u);
                    }
                    fetch(d);
                    uint2 code[P];
                    uint32_t word[P];
#pragma unroll
                    for (int q = 0; q < P; ++q) mx_codes<FMT>(v[q], gain, code[q], word[q]);
                    uint8_t *rec = sm + slot * p.stage_bytes + REC;  // 16 rows of codes, then the scales
                    constexpr int L = 4 * mx_block(FMT) / 16;        // lanes of a word
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        const int row = 2 * (out.pair + q) + half;  // (below 16: P divides the pairs of 16 rows)
                        *reinterpret_cast<uint2 *>(rec + mx_code_off(row, 8 * h)) = code[q];
                        if (h % L == 0) *reinterpret_cast<uint32_t *>(rec + p.NB * 128 + h / L * 512 + row * 16) = word[q];
                    }
                    next(out);
                    if (out.pair == 0) {  // the stage is complete
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the codes, for the tensor core
                        __syncwarp();
                        if (lane == 0) bar_arrive(b_full + 8 * slot);
                        slot += NQ;
                        if (slot >= S) {
                            slot -= S;
                            par ^= 1;
                        }
                    }
                }
            }
        };
        if (up)
            quantise(std::true_type{});
        else
            quantise(std::false_type{});
        if (!ok && lane == 0) atomicExch(p.err, 4);
    } else {
        // ------------------------------------------------------------ results
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int q = warp & 3, rl = 32 * q + lane;
        int seg = 0;
        bool ok = true;
        T *y = (T *)p.y;
        const T *rs = (const T *)p.r;
        walk([&](int t) {
            const int row = t * kMxRows + rl, buf = seg & 1;
            const int live = row < p.n ? p.nb : 0;  // columns to write
            // the residual is under way before the sums are complete
            T add[kMxgMaxN / 16][16];
            auto fetch = [&](int s) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    add[s][i] = 16 * s + i < live ? rs[row + (size_t)(16 * s + i) * p.n] : from_f32<T>(0.f);
            };
            if (rs && C == 1)
#pragma unroll
                for (int s = 0; s < kMxgMaxN / 16; ++s) fetch(s);
            ok = ok && __all_sync(0xffffffffu, mbar_wait(b_acc + 8 * buf, (uint32_t)(seg / 2) & 1u, lim));
            tc::fence_after_sync();
            const uint32_t d = tmem + buf * kMxgMaxN + ((uint32_t)(32 * q) << 16);
            if (C == 1)
#pragma unroll
                for (int s = 0; s < kMxgMaxN / 16; ++s) {
                    const int c = 16 * s;
                    if (c >= N) break;
                    uint32_t w[16];
                    tc::ld16(d + c, w);
                    tc::wait_ld16(w);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < live) {
                            const float v = __uint_as_float(w[i]);
                            y[row + (size_t)(c + i) * p.n] = from_f32<T>(rs ? fmaf(v, p.alpha, to_f32(add[s][i])) : v * p.alpha);
                        }
                }
            tc::fence_before_sync();
            __syncwarp();
            if (ok && lane == 0) bar_arrive(b_read + 8 * buf);  // (after a failure a phase could get too many)
            ++seg;
            return true;
        });
        if (!ok && lane == 0) atomicExch(p.err, 4);
    }
    if (C > 1) {
        // the parts of k: each CTA sums its share of the columns, in the order of the ranks.
        // The rings are done in all CTAs behind the first barrier: their room takes the parts.
        __syncwarp();
        cluster_sync();
        const int per = (N + C - 1) / C, q = warp & 3, rl = 32 * q + lane, row = blockIdx.x / C * kMxRows + rl;
        if (warp >= 2 && warp < 6) {
            const uint32_t d = tmem + ((uint32_t)(32 * q) << 16);
            for (int c = 0; c < N; c += 16) {
                uint32_t w[16];
                tc::ld16(d + c, w);
                tc::wait_ld16(w);
                int to = c / per, left = c - to * per;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    store_peer(ring + 4 * ((rank * per + left) * kMxRows + rl), (uint32_t)to, __uint_as_float(w[i]));
                    if (++left == per) {
                        left = 0;
                        ++to;
                    }
                }
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 2 && warp < 6 && row < p.n) {
            const float *part = reinterpret_cast<const float *>(sm) + rl;
            const T *rs = (const T *)p.r;
            const int first = rank * per, live = min(per, p.nb - first);
            for (int i = 0; i < live; i += 4) {  // (one column at a time: up to 80 ns each)
                const size_t at = (size_t)(first + i) * p.n + row;
                float v[4], add[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = 0.f;
                    add[j] = rs && i + j < live ? to_f32(rs[at + j * (size_t)p.n]) : 0.f;
                }
                for (int x = 0; x < C; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i + j < live) v[j] += part[(x * per + i + j) * kMxRows];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (i + j < live)
                        ((T *)p.y)[at + j * (size_t)p.n] = from_f32<T>(rs ? fmaf(v[j], p.alpha, add[j]) : v[j] * p.alpha);
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, cols_tm);
    }
}

}  // namespace dev

int mx_gemm_plan(MxGemmParams &p, int fmt, int sms) {
    // Up to 64 rows of x: one tile of columns, whose k a cluster may share; or pairs of CTAs
    // (mx_pair.cu). By estimates in ns of what both took (MXFP4): a launch, its stages, the
    // results, a cluster's sum.  (us, a cluster / pairs: 64 rows at 4096 x 4096 7.1 / 6.3, at
    // 4096 x 14336 11.1 / 14.0, at 1024 x 14336 7.5 / 13.2.)
    const int pairs = sms / 2;
    p.MT = mx_rtiles(p.n);
    double best = 0.0;
    if (p.nb <= dev::kMxgMaxN) {
        p.NB = (p.nb + 15) / 16 * 16;
        for (int C = 1; C <= 8 && C <= p.KS; ++C) {
            // (Clusters have to find their SMs in one part of the GPU: with a CTA an SM 15 of eight
            // or seven can run at once, 23 of six, 28 of five, 36 of four, 46 of three.)
            if (C > 1 && 8 * p.MT * C > (C > 4 ? 6 : 7) * sms) break;
            const double stages = (double)((p.MT * C + sms - 1) / sms) * ((p.KS + C - 1) / C);
            const double cost = 3000.0 + 245.0 * stages + 150.0 * std::min(stages, 4.0) +
                                (C > 1 ? 300.0 + (22.0 + 36.0 / C) * p.NB : 8.0 * p.NB);
            if (best > 0.0 && cost >= best) continue;
            best = cost;
            p.C = C;
        }
    }
    if (p.nb > 16) {
        const int N = std::min(p.nb, kMxPairN), M2 = (p.MT + 1) / 2, CT = (p.nb + kMxPairN - 1) / kMxPairN;
        const int whole = M2 * CT, rest = whole % pairs;
        // The tiles of an incomplete last round are cut, as long as that keeps two thirds of the
        // pairs at most busy (us, whole / cut: 192 rows at 4096 x 14336, 16 tiles of 76 pairs, 16.3 / 14.4;
        // 128 at 8192 x 2048, 32 tiles, 5.4 / 5.8).
        int width = kMxPairN;
        for (const int to : {128, 64})
            if (3 * rest * ((N + to - 1) / to) <= 2 * pairs) width = to;
        const int last = rest ? std::min(width, N) : N;
        const double cost = 2500.0 + 6.0 * last + p.KS * (whole / pairs * (173 + 0.2 * N) + (rest ? 173 + 0.2 * last : 0.0));
        if (best == 0.0 || cost < best) {
            p.pair = 1;
            p.NB = kMxPairN;
            p.CT = CT;
            p.C = 1;
            p.whole = whole - rest;
            p.width = width;
            p.parts = (N + width - 1) / width;
            p.units = p.whole + rest * p.parts;
            return 2 * std::min(p.units, pairs);
        }
    }
    p.stage_bytes = (mx_rec(fmt) + p.NB * 128 + 512 * mx_words(fmt) + 1023) / 1024 * 1024;
    const bool two = p.MT * p.C > sms;  // two CTAs of an SM
    const int room = (two ? (int)kSmemMax / 2 - 1024 : (int)kSmemMax) - dev::kMxgBars;
    p.stages = std::min(dev::kMxgMaxStages, room / p.stage_bytes);
    return p.C > 1 ? p.MT * p.C : std::min(p.MT, two ? 2 * sms : sms);
}

bool mx_gemm_few(int nb, int dtype, bool norm, bool glu) {
    // Every CTA quantises the rows of its stages, while the weights arrive: up to this many
    // rows in less time than a kernel in front of the product takes (us at 14336 x 4096, MXFP4,
    // here / there: bf16 8.2 / 10.3 for one row, 9.7 / 10.6 for eight, 11.2 / 10.6 for ten; two
    // inputs 9.2 / 10.5 for four, 10.6 / 10.5 for six; float 9.5 / 10.1 for four, 11.1 / 10.1 for
    // six).  Behind a norm a CTA would read whole rows before its first stage: 10.1 / 10.1 for
    // one row, 10.8 / 10.1 for four.
    return !norm && nb <= (glu || dtype == 0 ? 4 : 8);
}

template <int FMT, typename T, bool QX>
static int launch_mx_gemm_t(const MxGemmParams &p, int ctas, cudaStream_t stream) {
    auto kern = dev::q4mx_gemm_kernel<FMT, T, QX>;
    static size_t smem_set[64] = {0};
    const size_t smem = (size_t)p.stages * p.stage_bytes + dev::kMxgBars;
    if (!raise_smem(kern, smem, smem_set)) return -1;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config((unsigned)ctas, dev::kMxgThreads + (QX ? dev::kMxgQuant : 0), smem, stream, attr);
    if (p.C > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)p.C;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}
template <int FMT, typename T>
static int launch_mx_gemm_x(const MxGemmParams &p, int ctas, cudaStream_t stream) {
    return p.src.x ? launch_mx_gemm_t<FMT, T, true>(p, ctas, stream) : launch_mx_gemm_t<FMT, T, false>(p, ctas, stream);
}

int launch_mx_gemm(const MxGemmParams &p, int fmt, int dtype, int ctas, void *stream_) {
    if (p.pair) return launch_mx_pair(p, fmt, dtype, ctas, stream_);
    cudaStream_t s = (cudaStream_t)stream_;
    switch (2 * dtype + fmt) {
        case 0: return launch_mx_gemm_x<0, float>(p, ctas, s);
        case 1: return launch_mx_gemm_x<1, float>(p, ctas, s);
        case 2: return launch_mx_gemm_x<0, __half>(p, ctas, s);
        case 3: return launch_mx_gemm_x<1, __half>(p, ctas, s);
        case 4: return launch_mx_gemm_x<0, __nv_bfloat16>(p, ctas, s);
        case 5: return launch_mx_gemm_x<1, __nv_bfloat16>(p, ctas, s);
    }
    return -1;
}

}  // namespace q4
