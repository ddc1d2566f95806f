// mx_pair.cu -- the product of mx_gemm.cu for many rows of x: a pair of CTAs on two
// SMs works on one tile (tcgen05 cta_group::2), 256 rows of w by 192 of x.
//
// A stage (256 of k) of a 128 x 192 tile is 44 KB that one SM has to bring from L2 and
// read from shared memory for 355 cycles of tensor work; the pair shares x's rows, so
// that each SM brings and reads 31 KB for as much.  Each CTA holds its half of w's rows
// and of x's; the first CTA of the pair issues the MMAs, whose completion is signalled in
// both.  x's scales are in both CTAs, of all columns: each tensor core needs them.  (Four
// warps of each CTA that wrote the scales to tensor memory, instead of the copies that
// the first CTA issues for both, took 0.8 us a stage.)
//
// What bounds it: a stage takes 430 cycles, 355 of them MMAs (of K = 64); the rest are the
// copies of the scales in front of each stage's MMAs (NVFP4 has twice as many) and stages that are
// not there yet: 74 bytes a cycle reach an SM from L2, whose queues are at 60 % on average.
// The results' stores and loads come on top.  8191 x 4096 x 14336 MXFP4 125 us (7.7 PFLOP/s;
// to 135 on other machines and clocks), 8192^3 146 (7.5; to 155), NVFP4 162 (6.8; to 171); 4096 x
// 14336 x 4096 NVFP4 81 (5.9; to 92), with a residual 92 (to 97).  (Scales copied a stage ahead,
// or two stages waited for together: a tenth slower; narrower tiles: w's records take as long to
// arrive.)
//
//   warps 0, 10 and 11 copy, warp 1 issues MMAs (first CTA) or tells the first CTA of stages
//   that have landed (second), warps 2-9 write the results (half of the columns each four).
#include <algorithm>
#include <type_traits>

#include "mx_common.cuh"

namespace q4 {
namespace dev {

constexpr int kPairThreads = 384;
constexpr int kPairN = kMxPairN, kPairHalf = kPairN / 2;
template <int FMT>
struct PairCfg {
    static constexpr int W = mx_words(FMT), REC = mx_rec(FMT);
    static constexpr int OffB = REC, OffSf = OffB + kPairHalf * 128, Stage = OffSf + 2 * 512 * W;
    static constexpr int S = FMT == 0 ? 7 : 6;
    static constexpr int OffBar = S * Stage, Smem = OffBar + 8 * (2 * S + 5) + 16;
    static_assert(Stage % 1024 == 0 && Smem <= (int)kSmemMax, "shared memory of a pair's CTA");
};

// An arrival on the first CTA's barrier at this offset, and a wait for arrivals that may be
// the other CTA's: both of cluster scope (they are of their own CTA's where they do not say
// more).  The arrival is relaxed.  It tells of two things, neither of them a store of its
// thread that a release would have to make visible:
//  - a stage's bytes in the second CTA's shared memory.  They came by bulk copies, whose
//    completion the telling thread has waited for, and there is no other copy of that memory
//    that the second SM's tensor core could read;
//  - an accumulator that has been read: tcgen05.ld, complete by tcgen05.wait::ld, in front of
//    tcgen05.fence::before_thread_sync, which orders it before the arrival, as
//    fence::after_thread_sync orders the MMAs behind the wait.
// (With a release at cluster scope for every stage 8191 x 4096 x 14336 took 492 us, not 126.)
__device__ __forceinline__ void arrive_first(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ bool mbar_wait_pair(uint32_t bar, uint32_t parity, long long limit) {
    long long t0 = 0;
    for (int it = 0;; ++it) {
        uint32_t done;
        asm volatile(
            "{ .reg .pred P; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2; selp.b32 %0, 1, 0, P; }"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if (it == 0) {
            t0 = clock64();
        } else if (clock64() - t0 > limit) {
            return false;
        }
    }
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
template <int FMT>
__device__ __forceinline__ void mx_mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                            uint32_t acc) {
    if constexpr (FMT == 0)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "n"(tc::kSw128Hi)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "n"(tc::kSw128Hi)
            : "memory");
}
// mx_copy_scales in both CTAs, each from its own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint32_t saddr) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(tc::smem_desc(saddr, 128, 128))
                 : "memory");
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kPairThreads, 1) q4mx_pair_kernel(const __grid_constant__ MxGemmParams p) {
    using Cf = PairCfg<FMT>;
    constexpr int W = Cf::W, REC = Cf::REC, S = Cf::S;
    extern __shared__ __align__(1024) uint8_t sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = blockIdx.x & 1, KS = p.KS, M2 = (p.MT + 1) / 2;
    const uint32_t ring = smem_u32(sm);
    // barriers: a stage has landed here (the first CTA's: in both), a stage's MMAs are done; of an
    // accumulator: it is complete, both CTAs have read it (the first CTA's); the last MMAs of all
    const uint32_t b_full = ring + Cf::OffBar, b_empty = b_full + 8 * S, b_acc = b_empty + 8 * S, b_read = b_acc + 16,
                   b_drain = b_read + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Cf::OffBar + 8 * (2 * S + 5));
    if (warp == 0) {
        if (lane < S) {
            mbar_init(b_full + 8 * lane, rank == 0 ? 4 : 3);  // the three copying warps, the second CTA
            mbar_init(b_empty + 8 * lane, 1);
        }
        if (lane < 2) {
            mbar_init(b_acc + 8 * lane, 1);
            mbar_init(b_read + 8 * lane, 16);
        }
        if (lane == 0) mbar_init(b_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tslot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        // after the allocation: a kernel that starts on this could hold the columns this one waits for
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // the barriers of both CTAs
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;

    // unit u of the work: a pair of row tiles of w, the first column and how many (whole 32s).
    // The tiles of the last, incomplete round may be cut. (A part begins at a multiple of 64
    // columns: its scales' column in tensor memory has to be even.)
    auto unit = [&](int u, int &mt, int &c0, int &N) {
        int t = u, part = 0, width = kPairN;
        if (u >= p.whole) {
            t = p.whole + (u - p.whole) / p.parts;
            part = (u - p.whole) % p.parts;
            width = p.width;
        }
        // the larger matrix is read once, the smaller one again and again (from L2)
        mt = M2 > p.CT ? t / p.CT : t % M2;
        const int first = (M2 > p.CT ? t % p.CT : t / M2) * kPairN;
        c0 = first + part * width;
        N = min(min(width, first + kPairN - c0), (p.nb - c0 + 31) & ~31);
        return N > 0;  // (a ragged tile's columns may end before its parts do)
    };
    // this pair's tiles: f(row tiles, first column, columns) until it says no
    auto walk = [&](auto f) {
        for (int u = blockIdx.x >> 1; u < p.units; u += gridDim.x >> 1) {
            int mt, c0, N;
            if (unit(u, mt, c0, N) && !f(mt, c0, N)) return;
        }
    };
    const long long lim = p.wait_cycles;

    if (warp == 0 || warp >= 10) {
        // ------------------------------------------------------------ copies
        // Three warps, one thread each, each with its own share of every stage's bytes: warp 0
        // w's record, warp 10 x's codes, warp 11 x's scales.  (One thread for all took 560
        // cycles a stage to issue them.)  What a tile's stages share is computed once.
        if (tc::elect_one()) {
            int slot = 0, issued = 0, ahead = 0;
            uint32_t par = 1, extra = warp == 0 ? (uint32_t)p.extra_tx : 0u;  // (a wait for the phase before the first passes)
            auto source = [&](int mt) {
                // (behind an odd number of row tiles the last one again: its results are not stored)
                return p.w + (size_t)min(2 * mt + rank, p.MT - 1) * KS * REC;
            };
            // a tile's stages: one or two copies each, KS times, a record further each time
            auto stages = [&](uint32_t at, const uint8_t *src, uint32_t len, uint32_t at2, const uint8_t *src2, uint32_t len2) {
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t st = ring + slot * Cf::Stage, bar = b_full + 8 * slot;
                    if (ahead > 0) {
                        --ahead;
                    } else {
                        if (!mbar_wait_pair(b_empty + 8 * slot, par, lim)) {
                            atomicExch(p.err, 4);
                            return false;
                        }
                        mbar_expect_tx(bar, len + len2 + extra);
                        extra = 0;
                        bulk_copy(st + at, src, len, bar);
                        if (len2) bulk_copy(st + at2, src2, len2, bar);
                    }
                    src += REC, src2 += REC;
                    ++issued;
                    if (++slot == S) {
                        slot = 0;
                        par ^= 1;
                    }
                }
                return true;
            };
            int mt0, first, N0;
            if (warp == 0 && p.early && unit(blockIdx.x >> 1, mt0, first, N0)) {
                // the first stages' weights before what is in front of this kernel is done
                const uint8_t *w = source(mt0);
                for (; ahead < min(S, KS); ++ahead, w += REC) {
                    mbar_expect_tx(b_full + 8 * ahead, REC + extra);
                    extra = 0;
                    bulk_copy(ring + ahead * Cf::Stage, w, REC, b_full + 8 * ahead);
                }
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            walk([&](int mt, int c0, int N) {
                if (warp == 0) return stages(0, source(mt), REC, 0, nullptr, 0);
                const size_t step = (size_t)KS * REC;  // a row tile of x
                if (warp == 10) {
                    const int r0 = c0 + rank * (N / 2), off = r0 & 127, n0 = min(N / 2, 128 - off);
                    const uint8_t *b = p.x + (r0 >> 7) * step;
                    return stages(Cf::OffB, b + off * 128, n0 * 128, Cf::OffB + n0 * 128, b + step, (N / 2 - n0) * 128);
                }
                const uint8_t *sf = p.x + (c0 >> 7) * step + kMxCodes;
                return stages(Cf::OffSf, sf, 512 * W, Cf::OffSf + 512 * W, sf + step, (c0 & 127) + N > 128 ? 512 * W : 0);
            });
            // what is in flight lands before the CTA ends
            for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(b_full + 8 * (i % S), (uint32_t)(i / S) & 1u, kWaitCycles);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        int slot = 0;
        uint32_t par = 0;
        auto next = [&]() {
            if (++slot == S) {
                slot = 0;
                par ^= 1;
            }
        };
        if (rank == 0) {
            // (a stage has one barrier; with one for each CTA's bytes it took 80 cycles more)
            int seg = 0;
            uint32_t sf_set = 0;
            bool ok = true;
            walk([&](int, int c0, int N) {
                const int buf = seg & 1;
                ok = seg < 2 || __all_sync(0xffffffffu, mbar_wait_pair(b_read + 8 * buf, (uint32_t)(seg / 2 - 1) & 1u, lim));
                const uint32_t d = tmem + buf * kPairN, skip = (uint32_t)(c0 & 127) / 32;
                const bool two = (c0 & 127) + N > 128;
                // (M = 256 is bit 28, M = 128 bit 27)
                const uint32_t idesc0 = mx_idesc<FMT>(N, 0) + (1u << 27), idesc2 = mx_idesc<FMT>(N, FMT == 0 ? 2 : 0) + (1u << 27);
                for (int ks = 0; ok && ks < KS; ++ks) {
                    ok = __all_sync(0xffffffffu, mbar_wait_pair(b_full + 8 * slot, par, lim));
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        const uint32_t a = ring + slot * Cf::Stage, b = a + Cf::OffB, sb = a + Cf::OffSf;
                        const uint32_t ta = tmem + 2 * kPairN + sf_set, tb = ta + 16;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            copy_scales_pair(ta + 4 * w, a + kMxCodes + 512 * w);
                            copy_scales_pair(tb + 8 * w, sb + 512 * w);
                            if (two) copy_scales_pair(tb + 8 * w + 4, sb + 512 * (W + w));
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int w = FMT == 0 ? j / 2 : j;
                            mx_mma_pair<FMT>(d, tc::desc_sw128(a + 32 * j, 0), tc::desc_sw128(b + 32 * j, 0), j % 2 ? idesc2 : idesc0,
                                             ta + 4 * w, tb + 8 * w + skip, ks | j);
                        }
                        commit_pair(b_empty + 8 * slot);
                        if (ks + 1 == KS) commit_pair(b_acc + 8 * buf);
                    }
                    __syncwarp();
                    sf_set ^= 64;
                    next();
                }
                ++seg;
                return ok;
            });
            if (!ok && lane == 0) atomicExch(p.err, 4);
            if (tc::elect_one()) commit_pair(b_drain);
            __syncwarp();
        } else if (lane == 0) {
            walk([&](int, int, int) {
                for (int ks = 0; ks < KS; ++ks, next()) {
                    if (!mbar_wait(b_full + 8 * slot, par, lim)) {
                        atomicExch(p.err, 4);
                        return false;
                    }
                    arrive_first(b_full + 8 * slot);
                }
                return true;
            });
        }
        __syncwarp();
        mbar_wait_pair(b_drain, 0u, kWaitCycles);
    } else {
        // ------------------------------------------------------------ results
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // Two types of 16 bits: a lane takes two rows (n) of every second column, its
        // neighbour the same rows of the others, so that each reads and writes 4 bytes.  (2
        // bytes a lane: 8500 cycles a tile with a residual, longer than its MMAs.)
        const int q = warp & 3, part = (warp - 2) / 4;
        bool ok = true;
        const size_t n = p.n;
        auto results = [&](auto two_rows) {
            constexpr bool P2 = decltype(two_rows)::value;
            using V = std::conditional_t<P2, uint32_t, T>;  // what a lane reads and writes at once
            constexpr int CW = P2 ? 2 : 1, WIN = P2 ? kPairHalf : 64;  // columns of a V of two lanes; of the residual held
            const int odd = P2 ? lane & 1 : 0, rl = 32 * q + lane - odd;
            int seg = 0;
            walk([&](int mt, int c0, int N) {
                const int row = (2 * mt + rank) * kMxRows + rl, buf = seg & 1;
                c0 += part * (N / 2);
                N /= 2;
                const int live = (row < p.n ? min(N, p.nb - c0) : 0) - odd;  // columns to read and write, from this lane's first
                const size_t at = (size_t)(c0 + odd) * n + row;
                T *y = (T *)p.y + at;
                V add[WIN / CW];  // the residual, before the sums are there
                auto fetch = [&](int c) {  // 16 columns
                    const T *src = (const T *)p.r + at + c * n;
#pragma unroll
                    for (int i = 0; i < 16 / CW; ++i, src += CW * n) {
                        V v{};
                        if (c + CW * i < live) v = *reinterpret_cast<const V *>(src);
                        add[c % WIN / CW + i] = v;
                    }
                };
                if (p.r)
#pragma unroll
                    for (int c = 0; c < WIN; c += 16) fetch(c);
                ok = ok && __all_sync(0xffffffffu, mbar_wait_pair(b_acc + 8 * buf, (uint32_t)(seg / 2) & 1u, lim));
                tc::fence_after_sync();
                const uint32_t d = tmem + buf * kPairN + part * N + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int c = 0; c < kPairHalf; c += 16) {
                    if (c >= N) break;
                    uint32_t w[16];
                    tc::ld16(d + c, w);
                    tc::wait_ld16(w);
                    if (c + 16 >= N) {  // the accumulator has been read
                        tc::fence_before_sync();
                        __syncwarp();
                        if (ok && lane == 0) arrive_first(b_read + 8 * buf);  // (after a failure a phase could get too many)
                    }
                    T *dst = y + c * n;
#pragma unroll
                    for (int i = 0; i < 16 / CW; ++i, dst += CW * n) {
                        float v[CW];
                        if constexpr (P2) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[2 * i] : w[2 * i + 1], 1);
                            v[0] = __uint_as_float(odd ? got : w[2 * i]), v[1] = __uint_as_float(odd ? w[2 * i + 1] : got);
                        } else {
                            v[0] = __uint_as_float(w[i]);
                        }
                        if (p.r) {
                            const T *r = reinterpret_cast<const T *>(&add[c % WIN / CW + i]);
#pragma unroll
                            for (int e = 0; e < CW; ++e) v[e] = fmaf(v[e], p.alpha, to_f32(r[e]));
                        } else {
#pragma unroll
                            for (int e = 0; e < CW; ++e) v[e] *= p.alpha;
                        }
                        if (c + CW * i < live) {
                            if constexpr (P2)
                                *reinterpret_cast<V *>(dst) = pack2<T>(v[0], v[1]);
                            else
                                *dst = from_f32<T>(v[0]);
                        }
                    }
                    if (p.r && c + WIN < N) fetch(c + WIN);
                }
                ++seg;
                return true;
            });
        };
        if constexpr (sizeof(T) == 2) {
            if (p.n % 2 == 0)
                results(std::true_type{});
            else
                results(std::false_type{});
        } else {
            results(std::false_type{});
        }
        if (!ok && lane == 0) atomicExch(p.err, 4);
    }
    __syncwarp();
    tc::fence_before_sync();
    cluster_sync();  // neither CTA's memory is in use any more
    if (warp == 1) {
        tc::fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace dev

template <int FMT, typename T>
static int launch_mx_pair_t(const MxGemmParams &p, int ctas, cudaStream_t stream) {
    auto kern = dev::q4mx_pair_kernel<FMT, T>;
    static size_t smem_set[64] = {0};
    const size_t smem = dev::PairCfg<FMT>::Smem;
    if (!raise_smem(kern, smem, smem_set)) return -1;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config((unsigned)ctas, dev::kPairThreads, smem, stream, attr);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

int launch_mx_pair(const MxGemmParams &p, int fmt, int dtype, int ctas, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    switch (2 * dtype + fmt) {
        case 0: return launch_mx_pair_t<0, float>(p, ctas, s);
        case 1: return launch_mx_pair_t<1, float>(p, ctas, s);
        case 2: return launch_mx_pair_t<0, __half>(p, ctas, s);
        case 3: return launch_mx_pair_t<1, __half>(p, ctas, s);
        case 4: return launch_mx_pair_t<0, __nv_bfloat16>(p, ctas, s);
        case 5: return launch_mx_pair_t<1, __nv_bfloat16>(p, ctas, s);
    }
    return -1;
}

}  // namespace q4
