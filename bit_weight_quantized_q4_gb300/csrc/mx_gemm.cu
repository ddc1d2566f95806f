// mx_gemm.cu -- the product of two microscaled 4-bit matrices, y = alpha x w^T
// (+ r), w [n][k], x [nb][k], on the block-scaled tensor core: both operands go
// into tcgen05.mma as they are stored, so that no weight is ever dequantised.
//
// w's rows are the instruction's 128 rows and x's its columns, for one token as
// for thousands: the columns that a few tokens leave empty (16 at least) cost the
// tensor core less time than the weights take to arrive.  A record of w is one bulk
// copy, scales and all; x's rows and scales come by bulk copies into the same
// stage; the scales go from shared to tensor memory (tcgen05.cp) in front of their
// MMAs.
//   warp 0 copies, warp 1 issues MMAs, warps 2-5 write the results, while the
//   tensor core is at the next tile (two accumulators).
#include <algorithm>

#include "mx_common.cuh"

namespace q4 {
namespace dev {

constexpr int kMxgThreads = 192;
constexpr int kMxgMaxN = 192;      // columns of a tile
constexpr int kMxgMaxStages = 12;
constexpr int kMxgSf = 2 * kMxgMaxN;  // tensor memory: two accumulators, then two sets of scales
constexpr int kMxgBars = 8 * (2 * kMxgMaxStages + 5) + 16;

// CTA c's share of the stages of all tiles, [mx_first(c), mx_first(c + 1)); and
// the CTA that has unit u.
__device__ __forceinline__ int mx_first(int c, int units, int ctas) { return (int)((long long)units * c / ctas); }
__device__ __forceinline__ int mx_cta_of(int u, int units, int ctas) {
    return (int)((((long long)u + 1) * ctas - 1) / units);
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kMxgThreads, 1) q4mx_gemm_kernel(const __grid_constant__ MxGemmParams p) {
    constexpr int W = mx_words(FMT), REC = mx_rec(FMT);
    extern __shared__ __align__(1024) uint8_t sm[];  // the swizzle's pattern repeats every 1024 bytes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int S = p.stages, KS = p.KS, tiles = p.MT * p.CT, ctas = gridDim.x, cta = blockIdx.x;
    const uint32_t ring = smem_u32(sm), bars = ring + S * p.stage_bytes;
    // barriers: a stage has landed, a stage's MMAs are done; of an accumulator: it is
    // complete, it has been read; the last MMAs of all
    const uint32_t b_full = bars, b_empty = b_full + 8 * kMxgMaxStages, b_acc = b_empty + 8 * kMxgMaxStages,
                   b_read = b_acc + 16, b_drain = b_read + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + S * p.stage_bytes + 8 * (2 * kMxgMaxStages + 5));
    volatile int *last = reinterpret_cast<volatile int *>(tslot + 1);
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
        tc::tmem_alloc(smem_u32(tslot), 512);
        tc::tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;

    const int units = tiles * KS, u0 = mx_first(cta, units, ctas), u1 = mx_first(cta + 1, units, ctas);
    // this CTA's segments (tile, first and last stage): f(tile, k0, k1) until it says no
    auto walk = [&](auto f) {
        if (!p.split) {
            for (int t = cta; t < tiles; t += ctas)
                if (!f(t, 0, KS)) return;
        } else {
            for (int u = u0; u < u1;) {
                const int t = u / KS, k0 = u - t * KS, k1 = min(KS, k0 + u1 - u);
                if (!f(t, k0, k1)) return;
                u += k1 - k0;
            }
        }
    };
    // a tile's columns: the first, how many (whole 16s), and how many of them lie in
    // the first of the (two at most) row tiles of x that it covers
    auto cols = [&](int ct, int &c0, int &N, int &n0) {
        c0 = ct * p.NB;
        N = min(p.NB, (p.nb - c0 + 15) & ~15);
        n0 = min(N, kMxRows - (c0 & (kMxRows - 1)));
    };
    const long long lim = p.wait_cycles;

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            int it = 0, issued = 0;  // stages with their copies of x, with those of w
            uint32_t extra = (uint32_t)p.extra_tx;
            auto bytes_of = [&](int ct) {
                int c0, N, n0;
                cols(ct, c0, N, n0);
                return (uint32_t)(REC + N * 128 + (N > n0 ? 2 : 1) * 512 * W);
            };
            auto copy_w = [&](int slot, int mt, int ct, int ks) {
                const uint32_t bar = b_full + 8 * slot;
                mbar_expect_tx(bar, bytes_of(ct) + extra);
                extra = 0;
                bulk_copy(ring + slot * p.stage_bytes, p.w + ((size_t)mt * KS + ks) * REC, REC, bar);
            };
            if (p.early) {
                // the first stages' weights before what is in front of this kernel is done
                walk([&](int t, int k0, int k1) {
                    const int ct = t / p.MT, mt = t - ct * p.MT;
                    for (int ks = k0; ks < k1 && issued < S; ++ks) copy_w(issued++, mt, ct, ks);
                    return issued < S;
                });
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            walk([&](int t, int k0, int k1) {
                const int ct = t / p.MT, mt = t - ct * p.MT;
                int c0, N, n0;
                cols(ct, c0, N, n0);
                const uint8_t *x0 = p.x + (size_t)(c0 / kMxRows) * KS * REC, *x1 = x0 + (size_t)KS * REC;
                for (int ks = k0; ks < k1; ++ks, ++it) {
                    const int slot = it % S;
                    if (it >= issued) {
                        if (it >= S && !mbar_wait(b_empty + 8 * slot, (uint32_t)(it / S - 1) & 1u, lim)) {
                            atomicExch(p.err, 4);
                            return false;
                        }
                        copy_w(slot, mt, ct, ks);
                    }
                    const uint32_t dst = ring + slot * p.stage_bytes + REC, bar = b_full + 8 * slot;
                    const uint32_t sf = dst + p.NB * 128;
                    const uint8_t *a = x0 + (size_t)ks * REC;
                    bulk_copy(dst, a + (c0 & (kMxRows - 1)) * 128, n0 * 128, bar);
                    bulk_copy(sf, a + kMxCodes, 512 * W, bar);
                    if (N > n0) {
                        const uint8_t *b = x1 + (size_t)ks * REC;
                        bulk_copy(dst + n0 * 128, b, (N - n0) * 128, bar);
                        bulk_copy(sf + 512 * W, b + kMxCodes, 512 * W, bar);
                    }
                }
                return true;
            });
            // what is in flight lands before the CTA ends
            for (int i = max(0, it - S); i < it; ++i) mbar_wait(b_full + 8 * (i % S), (uint32_t)(i / S) & 1u, kWaitCycles);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        int it = 0, seg = 0;
        bool ok = true;
        walk([&](int t, int k0, int k1) {
            int c0, N, n0;
            cols(t / p.MT, c0, N, n0);
            const int buf = seg & 1;
            ok = seg < 2 || __all_sync(0xffffffffu, mbar_wait(b_read + 8 * buf, (uint32_t)(seg / 2 - 1) & 1u, lim));
            tc::fence_after_sync();
            const uint32_t d = tmem + buf * kMxgMaxN, skip = (uint32_t)(c0 & (kMxRows - 1)) / 32;
            const bool two = N > n0;
            for (int ks = k0; ok && ks < k1; ++ks, ++it) {
                const int slot = it % S;
                ok = __all_sync(0xffffffffu, mbar_wait(b_full + 8 * slot, (uint32_t)(it / S) & 1u, lim));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint32_t a = ring + slot * p.stage_bytes, b = a + REC, sb = b + p.NB * 128;
                    const uint32_t ta = tmem + kMxgSf + (it & 1) * 64, tb = ta + 16;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        mx_copy_scales(ta + 4 * w, a + kMxCodes + 512 * w);
                        mx_copy_scales(tb + 8 * w, sb + 512 * w);
                        if (two) mx_copy_scales(tb + 8 * w + 4, sb + 512 * (W + w));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int w = FMT == 0 ? j / 2 : j, id = FMT == 0 ? 2 * (j % 2) : 0;
                        mx_mma<FMT>(d, tc::desc_sw128(a + 32 * j, 0), tc::desc_sw128(b + 32 * j, 0), mx_idesc<FMT>(N, id),
                                    ta + 4 * w, tb + 8 * w + skip, (ks - k0) | j);
                    }
                    tc::commit(b_empty + 8 * slot);
                    if (ks + 1 == k1) tc::commit(b_acc + 8 * buf);
                }
                __syncwarp();
            }
            ++seg;
            return ok;
        });
        if (!ok && lane == 0) atomicExch(p.err, 4);
        if (tc::elect_one()) tc::commit(b_drain);
        __syncwarp();
        mbar_wait(b_drain, 0u, kWaitCycles);
    } else {
        // ------------------------------------------------------------ results
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int q = warp & 3, rl = 32 * q + lane;
        int seg = 0;
        bool ok = true;
        T *y = (T *)p.y;
        const T *rs = (const T *)p.r;
        // Columns c .. c + 15 of the tile: v alpha + r.
        auto store = [&](int row, int col0, const float (&v)[16]) {
            if (row >= p.n) return;
            float add[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                add[i] = rs && col0 + i < p.nb ? to_f32(rs[(size_t)(col0 + i) * p.n + row]) : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (col0 + i < p.nb) y[(size_t)(col0 + i) * p.n + row] = from_f32<T>(fmaf(v[i], p.alpha, add[i]));
        };
        walk([&](int t, int k0, int k1) {
            const int ct = t / p.MT, row = (t - ct * p.MT) * kMxRows + rl, buf = seg & 1;
            int c0, N, n0;
            cols(ct, c0, N, n0);
            // (a wait that gave up: the counters are kept up, what is stored is undefined)
            ok = ok && __all_sync(0xffffffffu, mbar_wait(b_acc + 8 * buf, (uint32_t)(seg / 2) & 1u, lim));
            tc::fence_after_sync();
            const uint32_t d = tmem + buf * kMxgMaxN + ((uint32_t)(32 * q) << 16);
            const bool whole = k0 == 0 && k1 == KS;
            float *mine = p.part + ((size_t)cta * 2 + (seg > 0)) * (p.NB * kMxRows) + rl;
            for (int c = 0; c < N; c += 16) {
                uint32_t w[16];
                tc::ld16(d + c, w);
                tc::wait_ld16(w);
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
                if (whole) {
                    store(row, c0 + c, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) __stcg(mine + (c + i) * kMxRows, v[i]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(b_read + 8 * buf);
            if (!whole) {
                // the last of the tile's CTAs to finish adds their shares in CTA order
                const int s0 = t * KS, f = mx_cta_of(s0, units, ctas), l = mx_cta_of(s0 + KS - 1, units, ctas);
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (warp == 2 && lane == 0) {
                    int before;
                    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.count + t) : "memory");
                    *last = before == l - f;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (*last) {
                    const size_t slot = (size_t)p.NB * kMxRows;
                    const float *first = p.part + ((size_t)f * 2 + (mx_first(f, units, ctas) < s0)) * slot + rl;
                    for (int c = 0; c < N; c += 16) {
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __ldcg(first + (c + i) * kMxRows);
                        for (int x = f + 1; x <= l; ++x) {
                            const float *other = p.part + (size_t)x * 2 * slot + rl;
                            float o[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __ldcg(other + (c + i) * kMxRows);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] += o[i];
                        }
                        store(row, c0 + c, v);
                    }
                    if (warp == 2 && lane == 0) p.count[t] = 0;  // zero again for the next call
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");  // the flag is read before the next tile's
            }
            ++seg;
            return true;
        });
        if (!ok && lane == 0) atomicExch(p.err, 4);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

}  // namespace dev

int mx_gemm_plan(MxGemmParams &p, int fmt, int sms) {
    p.MT = mx_rtiles(p.n);
    // one tile of columns up to 192 rows of x, else tiles of 192 or 128: whichever pads less
    if (p.nb <= dev::kMxgMaxN) {
        p.NB = (p.nb + 15) / 16 * 16;
    } else {
        const int a = (p.nb + 191) / 192 * 192, b = (p.nb + 127) / 128 * 128;
        p.NB = b < a - a / 16 ? 128 : 192;
    }
    p.CT = (p.nb + p.NB - 1) / p.NB;
    const int W = mx_words(fmt), blocks = p.NB > 128 || p.CT > 1 ? 2 : 1;
    p.stage_bytes = mx_rec(fmt) + p.NB * 128 + blocks * 512 * W;
    p.stage_bytes = (p.stage_bytes + 1023) / 1024 * 1024;
    p.stages = std::min<int>(dev::kMxgMaxStages, ((int)kSmemMax - dev::kMxgBars) / p.stage_bytes);
    const long long tiles = (long long)p.MT * p.CT;
    // whole tiles where the last wave of them is nearly full, else the stages evenly
    const long long waves = (tiles + sms - 1) / sms;
    p.split = tiles <= kMxMaxTiles && tiles * 8 < waves * sms * 7;
    const long long units = tiles * p.KS;
    return (int)std::min<long long>(p.split ? units : tiles, sms);
}
size_t mx_gemm_part_bytes(const MxGemmParams &p, int ctas) {
    return p.split ? (size_t)ctas * 2 * p.NB * kMxRows * sizeof(float) : 0;
}

template <int FMT, typename T>
static int launch_mx_gemm_t(const MxGemmParams &p, int ctas, cudaStream_t stream) {
    auto kern = dev::q4mx_gemm_kernel<FMT, T>;
    static size_t smem_set[64] = {0};
    const size_t smem = (size_t)p.stages * p.stage_bytes + dev::kMxgBars;
    if (!raise_smem(kern, smem, smem_set)) return -1;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)ctas, dev::kMxgThreads, smem, stream, &attr);
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

int launch_mx_gemm(const MxGemmParams &p, int fmt, int dtype, int ctas, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    switch (2 * dtype + fmt) {
        case 0: return launch_mx_gemm_t<0, float>(p, ctas, s);
        case 1: return launch_mx_gemm_t<1, float>(p, ctas, s);
        case 2: return launch_mx_gemm_t<0, __half>(p, ctas, s);
        case 3: return launch_mx_gemm_t<1, __half>(p, ctas, s);
        case 4: return launch_mx_gemm_t<0, __nv_bfloat16>(p, ctas, s);
        case 5: return launch_mx_gemm_t<1, __nv_bfloat16>(p, ctas, s);
    }
    return -1;
}

}  // namespace q4
