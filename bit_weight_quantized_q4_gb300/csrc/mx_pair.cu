// mx_pair.cu -- the product of mx_gemm.cu for many rows of x: a pair of CTAs on two
// SMs works on one tile (tcgen05 cta_group::2), 256 rows of w by 192 of x.
//
// A stage (256 of k) of a 128 x 192 tile is 44 KB that one SM has to bring from L2 and
// read from shared memory for 364 cycles of tensor work; the pair shares x's rows, so
// that each SM brings and reads 31 KB for as much.  Each CTA holds its half of w's rows
// and of x's; the first CTA of the pair issues the MMAs, whose completion is signalled in
// both.  x's scales are in both CTAs, of all columns: each tensor core needs them.  (Four
// warps of each CTA that wrote the scales to tensor memory, instead of the copies that
// the first CTA issues for both, took 0.8 us a stage.)
//   warp 0 copies, warp 1 issues MMAs (first CTA) or tells the first CTA of stages that
//   have landed (second), warps 2-9 write the results (half of the columns each four).
#include <algorithm>

#include "mx_common.cuh"

namespace q4 {
namespace dev {

constexpr int kPairThreads = 320;
constexpr int kPairN = 192, kPairHalf = kPairN / 2;
template <int FMT>
struct PairCfg {
    static constexpr int W = mx_words(FMT), REC = mx_rec(FMT);
    static constexpr int OffB = REC, OffSf = OffB + kPairHalf * 128, Stage = OffSf + 2 * 512 * W;
    static constexpr int S = FMT == 0 ? 7 : 6;
    static constexpr int OffBar = S * Stage, Smem = OffBar + 8 * (3 * S + 5) + 16;
    static_assert(Stage % 1024 == 0 && Smem <= (int)kSmemMax, "shared memory of a pair's CTA");
};

// An arrival on the first CTA's barrier at this offset.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
        : "memory");
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
    const int rank = blockIdx.x & 1, KS = p.KS, M2 = (p.MT + 1) / 2, tiles = M2 * p.CT;
    const uint32_t ring = smem_u32(sm);
    // barriers: a stage has landed here, a stage has landed in the second CTA (the first
    // CTA's), a stage's MMAs are done; of an accumulator: it is complete, both CTAs have read it (the
    // first CTA's); the last MMAs of all
    const uint32_t b_full = ring + Cf::OffBar, b_ready = b_full + 8 * S, b_empty = b_ready + 8 * S, b_acc = b_empty + 8 * S,
                   b_read = b_acc + 16, b_drain = b_read + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Cf::OffBar + 8 * (3 * S + 5));
    if (warp == 0) {
        if (lane < S) {
            mbar_init(b_full + 8 * lane, 1);
            mbar_init(b_ready + 8 * lane, 1);
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
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // the barriers of both CTAs
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;

    // this pair's tiles: f(tile) until it says no
    auto walk = [&](auto f) {
        for (int t = blockIdx.x >> 1; t < tiles; t += gridDim.x >> 1)
            if (!f(t)) return;
    };
    // a tile's columns: the first and how many (whole 32s); the row tile of w
    auto cols = [&](int ct, int &c0, int &N) {
        c0 = ct * kPairN;
        N = min(kPairN, (p.nb - c0 + 31) & ~31);
    };
    const long long lim = p.wait_cycles;

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        // (one thread's chain of instructions: what a tile's stages share is computed once)
        if (lane == 0) {
            uint32_t extra = (uint32_t)p.extra_tx;
            // the first stages' weights before what is in front of this kernel is done
            const int t0 = blockIdx.x >> 1;
            int ahead = 0;
            auto source = [&](int t) {
                // (behind an odd number of row tiles the last one again: its results are not stored)
                return p.w + (size_t)min(2 * (t % M2) + rank, p.MT - 1) * KS * REC;
            };
            auto bytes_of = [&](int c0, int N) {
                return (uint32_t)(REC + N / 2 * 128 + ((c0 & 127) + N > 128 ? 2 : 1) * 512 * W);
            };
            if (p.early && t0 < tiles) {
                int c0, N;
                cols(t0 / M2, c0, N);
                const uint8_t *w = source(t0);
                for (; ahead < min(S, KS); ++ahead) {
                    mbar_expect_tx(b_full + 8 * ahead, bytes_of(c0, N) + extra);
                    extra = 0;
                    bulk_copy(ring + ahead * Cf::Stage, w + (size_t)ahead * REC, REC, b_full + 8 * ahead);
                }
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int slot = 0, issued = 0;
            uint32_t par = 1, dst = ring, bar = b_full;  // (a wait for the phase before the first passes)
            walk([&](int t) {
                int c0, N;
                cols(t / M2, c0, N);
                const int r0 = c0 + rank * (N / 2), off = r0 & 127, n0 = min(N / 2, 128 - off);
                const size_t step = (size_t)KS * REC;  // a row tile of x
                const uint8_t *w = source(t), *b = p.x + (r0 >> 7) * step + off * 128, *b2 = p.x + ((r0 >> 7) + 1) * step;
                const uint8_t *sf = p.x + (c0 >> 7) * step + kMxCodes, *sf2 = sf + step;
                const uint32_t bytes = bytes_of(c0, N), len = n0 * 128, len2 = (N / 2 - n0) * 128;
                const bool two = (c0 & 127) + N > 128;
                for (int ks = 0; ks < KS; ++ks) {
                    if (ahead > 0) {
                        --ahead;
                    } else {
                        if (!mbar_wait(bar + 8 * 2 * S, par, lim)) {  // b_empty of this slot
                            atomicExch(p.err, 4);
                            return false;
                        }
                        mbar_expect_tx(bar, bytes + extra);
                        extra = 0;
                        bulk_copy(dst, w, REC, bar);
                    }
                    bulk_copy(dst + Cf::OffB, b, len, bar);
                    if (len2) bulk_copy(dst + Cf::OffB + len, b2, len2, bar);
                    bulk_copy(dst + Cf::OffSf, sf, 512 * W, bar);
                    if (two) bulk_copy(dst + Cf::OffSf + 512 * W, sf2, 512 * W, bar);
                    w += REC, b += REC, b2 += REC, sf += REC, sf2 += REC;
                    ++issued;
                    dst += Cf::Stage, bar += 8;
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
        int slot = 0;
        uint32_t par = 0;
        auto next = [&]() {
            if (++slot == S) {
                slot = 0;
                par ^= 1;
            }
        };
        if (rank == 0) {
            int seg = 0;
            uint32_t sf_set = 0;
            bool ok = true;
            walk([&](int t) {
                int c0, N;
                cols(t / M2, c0, N);
                const int buf = seg & 1;
                ok = seg < 2 || __all_sync(0xffffffffu, mbar_wait(b_read + 8 * buf, (uint32_t)(seg / 2 - 1) & 1u, lim));
                tc::fence_after_sync();
                const uint32_t d = tmem + buf * kPairN, skip = (uint32_t)(c0 & 127) / 32;
                const bool two = (c0 & 127) + N > 128;
                // (M = 256 is bit 28, M = 128 bit 27)
                const uint32_t idesc0 = mx_idesc<FMT>(N, 0) + (1u << 27), idesc2 = mx_idesc<FMT>(N, FMT == 0 ? 2 : 0) + (1u << 27);
                for (int ks = 0; ok && ks < KS; ++ks) {
                    ok = __all_sync(0xffffffffu, mbar_wait(b_full + 8 * slot, par, lim) && mbar_wait(b_ready + 8 * slot, par, lim));
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
            walk([&](int) {
                for (int ks = 0; ks < KS; ++ks, next()) {
                    if (!mbar_wait(b_full + 8 * slot, par, lim)) {
                        atomicExch(p.err, 4);
                        return false;
                    }
                    arrive_first(b_ready + 8 * slot);
                }
                return true;
            });
        }
        __syncwarp();
        mbar_wait(b_drain, 0u, kWaitCycles);
    } else {
        // ------------------------------------------------------------ results
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int q = warp & 3, rl = 32 * q + lane, part = (warp - 2) / 4;
        int seg = 0;
        bool ok = true;
        const size_t n = p.n;
        walk([&](int t) {
            const int row = (2 * (t % M2) + rank) * kMxRows + rl, buf = seg & 1;
            int c0, N;
            cols(t / M2, c0, N);
            c0 += part * (N / 2);
            N /= 2;
            const int live = row < p.n ? min(N, p.nb - c0) : 0;  // columns to write
            T *y = (T *)p.y + c0 * n + row;
            const T *rs = (const T *)p.r + c0 * n + row;
            T add[4][16];  // the residual, 64 columns ahead (mx_gemm.cu)
            auto fetch = [&](int s, int c) {
                const T *src = rs + c * n;
#pragma unroll
                for (int i = 0; i < 16; ++i, src += n) add[s][i] = c + i < live ? *src : from_f32<T>(0.f);
            };
            if (p.r)
#pragma unroll
                for (int s = 0; s < 4; ++s) fetch(s, 16 * s);
            ok = ok && __all_sync(0xffffffffu, mbar_wait(b_acc + 8 * buf, (uint32_t)(seg / 2) & 1u, lim));
            tc::fence_after_sync();
            const uint32_t d = tmem + buf * kPairN + part * N + ((uint32_t)(32 * q) << 16);
            for (int cb = 0; cb < N; cb += 64)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int c = cb + 16 * s;
                    if (c >= N) break;
                    uint32_t w[16];
                    tc::ld16(d + c, w);
                    tc::wait_ld16(w);
                    T *dst = y + c * n;
#pragma unroll
                    for (int i = 0; i < 16; ++i, dst += n)
                        if (c + i < live) {
                            const float v = __uint_as_float(w[i]);
                            *dst = from_f32<T>(p.r ? fmaf(v, p.alpha, to_f32(add[s][i])) : v * p.alpha);
                        }
                    if (p.r) fetch(s, c + 64);
                }
            tc::fence_before_sync();
            __syncwarp();
            if (ok && lane == 0) arrive_first(b_read + 8 * buf);  // (after a failure a phase could get too many)
            ++seg;
            return true;
        });
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
