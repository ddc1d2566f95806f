// mx_quant.cu -- rows into the microscaled 4-bit forms and back: quantising,
// optionally behind an RMSNorm (x / rms(x) gamma) or a SwiGLU (silu(x) up);
// dequantising; codes and scales from and into plain rows.
//
// Pure streams: HBM bounds the float forms, the arithmetic of scales and codes the 16-bit
// ones.  14336 x 4096 float 39.7 us (6.7 TB/s), bf16 26.2 (5.6); 8191 x 4096 bf16 behind a
// norm 19.4 (4.4); 8191 x 14336 fp16 SwiGLU 82.9 (6.4); back into bf16, 14336 x 4096, 24.3
// (6.1).  When a model is loaded: codes and scales of 14336 x 4096 from plain rows 27.6 (2.3
// TB/s: a record's rows in words of 4 bytes a lane, its scales in single bytes), into them 29.8.
// A lane takes sixteen consecutive values, half a record row a half warp: a block of 32
// (16) is two lanes (one), a row's codes of a record one whole 128-byte line.  (Eight values
// a lane: half the time of the 16-bit forms was the arithmetic of scales and addresses.)
#include <algorithm>

#include "mx_rows.cuh"

namespace q4 {
namespace dev {

constexpr int kMxThreads = 256, kMxWarps = kMxThreads / 32;

// The sixteen values v from column c of row `row` into the matrix at `out`; all
// lanes of a warp, those of a row of a record (16 of them) in order.
template <int FMT>
__device__ __forceinline__ void mx_store(uint8_t *out, bool live, int row, int c, int KT, const uint64_t (&v)[8],
                                         const MxGain &gain) {
    uint2 code;
    uint32_t word;
    mx_codes<FMT>(v, gain, code, word);
    if (!live) return;
    constexpr int L = 4 * mx_block(FMT) / 16;  // lanes of a word
    const int r = row % kMxRows, h = (c % kMxK) / 16;  // h: which sixteen of the record's row
    uint8_t *rec = out + ((size_t)(row / kMxRows) * KT + c / kMxK) * mx_rec(FMT);
    *reinterpret_cast<uint2 *>(rec + mx_code_off(r, 8 * h)) = code;
    if (h % L == 0) *reinterpret_cast<uint32_t *>(rec + mx_scale_off(r, h / L)) = word;
}

// A warp's units: two rows (of the whole batch) and a column tile, a half warp each.
struct MxUnit {
    int pair, kt;
    __device__ __forceinline__ MxUnit(long long u, int KT) : pair((int)(u / KT)), kt((int)(u - (long long)pair * KT)) {}
    __device__ __forceinline__ void next(int KT) {
        if (++kt == KT) {
            kt = 0;
            ++pair;
        }
    }
};

// Values as they are, or a SwiGLU of two rows: a warp takes AH units, their loads
// issued together.
template <typename T, int FMT, bool GLU, int AH>
__global__ void __launch_bounds__(kMxThreads) q4mx_quant_kernel(const __grid_constant__ MxQuantParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // after the wait: a kernel that starts on this may read what was complete before
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, half = lane >> 4, KT = mx_ktiles(p.k), rows = p.batch * p.rows;
    const long long mat = (long long)mx_rtiles(p.rows) * KT * mx_rec(FMT);
    const MxUnit first((((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * AH), KT);
    const MxGain gain{p.scale, p.six_g, p.inv};
    Raw16<T> x[AH], y[GLU ? AH : 1];
    MxUnit u = first;
#pragma unroll
    for (int i = 0; i < AH; ++i, u.next(KT)) {
        const int c = u.kt * kMxK + 16 * (lane & 15);
        const long long row = 2ll * u.pair + half;
        x[i].zero();
        if constexpr (GLU) y[i].zero();
        if (row < rows && c < p.k) {
            x[i].load((const T *)p.x + row * p.ld + c);
            if constexpr (GLU) y[i].load((const T *)p.up + row * p.ld + c);
        }
    }
    u = first;
#pragma unroll
    for (int i = 0; i < AH; ++i, u.next(KT)) {
        if (2ll * u.pair >= rows) break;
        uint64_t v[8];
        x[i].pairs(v);
        if constexpr (GLU) {
            uint64_t w[8];
            y[i].pairs(w);
            mx_glu(v, w);
        }
        const int row = 2 * u.pair + half, b = p.batch == 1 ? 0 : row / p.rows;
        mx_store<FMT>(p.out + b * mat, row < rows, row - b * p.rows, u.kt * kMxK + 16 * (lane & 15), KT, v, gain);
    }
}

// Behind an RMSNorm: WPR warps a row, which keep up to R sixteens a lane of it in
// registers (what a longer row has beyond is read again once its sum of squares is
// known).  As many CTAs as are resident take every grid-th rows each, the loads of the
// next DP rows under way.  Its arithmetic and the latencies that 16 warps leave uncovered bound
// it, not the memory: 8191 x 4096 bf16 takes 19 us with four warps a row and two CTAs of an
// SM (three, whose registers spill: 26); with eight, three CTAs and two rows under way 22 (a
// CTA a row: 30; more CTAs than are resident: 25; four, which spill: 26).
template <int R>
constexpr int mx_norm_ctas() { return R == 1 ? 3 : 2; }
template <typename T, int FMT, int WPR, int R>
__global__ void __launch_bounds__(kMxThreads, mx_norm_ctas<R>()) q4mx_quant_norm_kernel(const __grid_constant__ MxQuantParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float sums[2][kMxWarps];
    constexpr int RPC = kMxWarps / WPR;  // rows of a CTA
    constexpr int DP = sizeof(T) == 2 && R == 1 ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, KT = mx_ktiles(p.k);
    const int at = 16 * (32 * (warp % WPR) + lane), step = 512 * WPR, kpad = KT * kMxK;
    const int rows = p.batch * p.rows, ahead = gridDim.x * RPC;
    const long long mat = (long long)mx_rtiles(p.rows) * KT * mx_rec(FMT);
    const MxGain gain{p.scale, p.six_g, p.inv};
    const float inv_k = 1.f / (float)p.k;
    // the lane's columns are the same in every row
    uint64_t gm[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) gm[i][e] = 0;
        if (at + i * step < p.k) mx_factors(gm[i], p.gamma + at + i * step);
    }
    Raw16<T> next[DP][R];
    auto fetch = [&](int d, int row) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            next[d][i].zero();
            if (row < rows && at + i * step < p.k) next[d][i].load((const T *)p.x + row * p.ld + at + i * step);
        }
    };
    auto one = [&](const Raw16<T> (&x)[R], int row, int turn) {
        const bool live = row < rows;
        const T *src = (const T *)p.x + (live ? row : 0) * p.ld;
        uint64_t s2 = 0;
        auto squares = [&](const Raw16<T> &a) {
            uint64_t v[8];
            a.pairs(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s2 = fma_f32x2(v[e], v[e], s2);
        };
#pragma unroll
        for (int i = 0; i < R; ++i) squares(x[i]);
        for (int c = at + R * step; c < p.k; c += step) {
            Raw16<T> a;
            a.load(src + c);
            squares(a);
        }
        float sum = lo_f32(s2) + hi_f32(s2);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if constexpr (WPR > 1) {
            if (lane == 0) sums[turn][warp] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) sum += sums[turn][warp / WPR * WPR + i];
        }
        const float rstd = mx_rstd(sum, inv_k, p.eps);
        const int b = p.batch == 1 ? 0 : row / p.rows;
        auto put = [&](const Raw16<T> &a, const uint64_t (&gv)[8], int c) {
            uint64_t v[8];
            a.pairs(v);
            // (columns behind k are zeros even where rstd is infinite or NaN)
            const float f = c < p.k ? rstd : 1.f;
            const uint64_t by = pair_f32(f, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = mul_f32x2(mul_f32x2(v[e], by), gv[e]);
            mx_store<FMT>(p.out + b * mat, live && c < kpad, row - b * p.rows, c, KT, v, gain);
        };
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (at - 16 * lane + i * step < kpad) put(x[i], gm[i], at + i * step);
        for (int c = at + R * step; c - 16 * lane < kpad; c += step) {
            Raw16<T> a;
            uint64_t gv[8] = {};
            a.zero();
            if (c < p.k) {
                a.load(src + c);
                mx_factors(gv, p.gamma + c);
            }
            put(a, gv, c);
        }
    };
    int row = blockIdx.x * RPC + warp / WPR, turn = 0;
#pragma unroll
    for (int d = 0; d < DP; ++d) fetch(d, row + d * ahead);
    while (row - warp / WPR < rows) {
#pragma unroll
        for (int d = 0; d < DP; ++d) {
            if (row - warp / WPR >= rows) break;
            Raw16<T> x[R];
#pragma unroll
            for (int i = 0; i < R; ++i) x[i] = next[d][i];
            fetch(d, row + DP * ahead);
            one(x, row, turn);
            row += ahead;
            turn ^= 1;
        }
    }
}

// Back into values: g s e in fp32, rounded to T.  A warp a record's row, eight values a
// lane: its stores are whole lines (sixteen a lane: 16 -> 19 us for 8191 x 4096).
constexpr int kMxAhead = 4;  // units (row, column tile) of a warp
template <typename T, int FMT>
__global__ void __launch_bounds__(kMxThreads) q4mx_dequant_kernel(const __grid_constant__ MxCopyParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int L = mx_block(FMT) / 8;
    const int lane = threadIdx.x & 31, KT = mx_ktiles(p.k), rows = p.batch * p.rows;
    const long long mat = (long long)mx_rtiles(p.rows) * KT * mx_rec(FMT);
    const long long u0 = ((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * kMxAhead;
    const int row0 = (int)(u0 / KT), kt0 = (int)(u0 - (long long)row0 * KT);
    uint32_t code[kMxAhead], sc[kMxAhead];
    int row = row0, kt = kt0;
    auto next = [&]() {
        if (++kt == KT) {
            kt = 0;
            ++row;
        }
    };
#pragma unroll
    for (int i = 0; i < kMxAhead; ++i, next()) {
        code[i] = sc[i] = 0u;
        if (row < rows) {
            const int b = p.batch == 1 ? 0 : row / p.rows, rr = row - b * p.rows, r = rr % kMxRows;
            const uint8_t *rec = p.mx + b * mat + ((size_t)(rr / kMxRows) * KT + kt) * mx_rec(FMT);
            code[i] = *reinterpret_cast<const uint32_t *>(rec + mx_code_off(r, 4 * lane));
            sc[i] = rec[mx_scale_off(r, lane / (4 * L)) + (lane / L) % 4];
        }
    }
    row = row0;
    kt = kt0;
#pragma unroll
    for (int i = 0; i < kMxAhead; ++i, next()) {
        const int c = kt * kMxK + 8 * lane;
        if (row >= rows || c >= p.k) continue;
        const float s = mx_scale_value<FMT>(sc[i]);
        float v[8];
        e2m1_values(code[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = FMT == 0 ? v[e] * s : v[e] * s * p.scale;
        T *dst = (T *)p.out + (size_t)row * p.k + c;
        if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4 *>(dst), make_float4(v[0], v[1], v[2], v[3]));
            __stcs(reinterpret_cast<float4 *>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                              pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])));
        }
    }
}

// Codes and scales between plain rows and records; UNPACK: out of the records.
template <int FMT, bool UNPACK>
__global__ void __launch_bounds__(kMxThreads) q4mx_pack_kernel(const __grid_constant__ MxCopyParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int L = mx_block(FMT) / 8;
    const int lane = threadIdx.x & 31, KT = mx_ktiles(p.k);
    const long long units = (long long)p.batch * p.rows * KT;
    const long long mat = (long long)mx_rtiles(p.rows) * KT * mx_rec(FMT);
    const long long u0 = ((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * kMxAhead;
#pragma unroll
    for (int i = 0; i < kMxAhead; ++i) {
        const long long u = u0 + i;
        if (u >= units) break;
        const long long row = u / KT, b = p.batch == 1 ? 0 : row / p.rows;
        const int kt = (int)(u - row * KT), rr = (int)(row - b * p.rows), r = rr % kMxRows, c = kt * kMxK + 8 * lane;
        uint8_t *rec = p.mx + b * mat + ((size_t)(rr / kMxRows) * KT + kt) * mx_rec(FMT);
        uint32_t *code = reinterpret_cast<uint32_t *>(rec + mx_code_off(r, 4 * lane));
        uint8_t *sc = rec + mx_scale_off(r, lane / (4 * L)) + (lane / L) % 4;
        uint32_t *pc = reinterpret_cast<uint32_t *>(p.codes + (row * p.k + c) / 2);
        uint8_t *ps = p.scales + (row * p.k + c) / mx_block(FMT);
        const bool in = c < p.k;
        if constexpr (UNPACK) {
            if (in) *pc = *code;
            if (in && lane % L == 0) *ps = *sc;
        } else {
            *code = in ? *pc : 0u;
            if (lane % L == 0) *sc = in ? *ps : (uint8_t)0;
        }
    }
}

}  // namespace dev

namespace {
// CTAs of a launch over `units` of which a warp takes `ahead`
unsigned mx_grid(long long units, int ahead) {
    const long long per = (long long)dev::kMxWarps * ahead;
    return (unsigned)((units + per - 1) / per);
}
// units of two rows and a column tile
long long mx_pairs(int batch, int rows, int k) { return ((long long)batch * rows + 1) / 2 * mx_ktiles(k); }

template <typename Kern, typename P>
int mx_launch(Kern kern, unsigned grid, const P &p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config(grid, dev::kMxThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

template <typename T, int FMT, int WPR, int R>
int launch_mx_norm(const MxQuantParams &p, int sms, cudaStream_t stream) {
    const long long ctas = ((long long)p.batch * p.rows * WPR + dev::kMxWarps - 1) / dev::kMxWarps;
    return mx_launch(dev::q4mx_quant_norm_kernel<T, FMT, WPR, R>, (unsigned)std::min<long long>(ctas, (long long)dev::mx_norm_ctas<R>() * sms), p, stream);
}
template <typename T, int FMT, bool GLU>
int launch_mx_values(const MxQuantParams &p, int sms, cudaStream_t stream) {
    // 16-bit types: two units a warp once there are many (us, one / two: 16 x 4096 bf16 1.5 / 1.9,
    // 8191 x 14336 53.5 / 48.9, SwiGLU 86 / 83); float has as many bytes under way with one
    const long long units = mx_pairs(p.batch, p.rows, p.k);
    if constexpr (sizeof(T) == 2)
        if (units > 64 * sms) return mx_launch(dev::q4mx_quant_kernel<T, FMT, GLU, 2>, mx_grid(units, 2), p, stream);
    return mx_launch(dev::q4mx_quant_kernel<T, FMT, GLU, 1>, mx_grid(units, 1), p, stream);
}
template <typename T, int FMT>
int launch_mx_quant_t(const MxQuantParams &p, int sms, cudaStream_t stream) {
    if (p.gamma) {
        // as many warps a row as it has 512s, up to eight; from about a round of the SMs on and for
        // 16-bit types half as many, of whose work a row's sum is a smaller part (us, 4096 columns of
        // bf16, eight warps / four: 152 rows 2.1 / 2.4, 304 3.0 / 2.7, 8191 21.9 / 18.8; float
        // 26.3 / 26.8)
        if (p.k <= 512) return launch_mx_norm<T, FMT, 1, 1>(p, sms, stream);
        if constexpr (sizeof(T) == 2) {
            if ((long long)p.batch * p.rows * p.k >= 1 << 20) {
                if (p.k <= 1024) return launch_mx_norm<T, FMT, 1, 2>(p, sms, stream);
                if (p.k <= 2048) return launch_mx_norm<T, FMT, 2, 2>(p, sms, stream);
                if (p.k <= 4096) return launch_mx_norm<T, FMT, 4, 2>(p, sms, stream);
            }
        }
        if (p.k <= 1024) return launch_mx_norm<T, FMT, 2, 1>(p, sms, stream);
        if (p.k <= 2048) return launch_mx_norm<T, FMT, 4, 1>(p, sms, stream);
        if (p.k <= 4096) return launch_mx_norm<T, FMT, 8, 1>(p, sms, stream);
        return launch_mx_norm<T, FMT, 8, 2>(p, sms, stream);
    }
    if (p.up) return launch_mx_values<T, FMT, true>(p, sms, stream);
    return launch_mx_values<T, FMT, false>(p, sms, stream);
}
}  // namespace

int launch_mx_quant(const MxQuantParams &params, int fmt, int dtype, int sms, void *stream_) {
    MxQuantParams p = params;
    p.set_gain();
    cudaStream_t s = (cudaStream_t)stream_;
    switch (2 * dtype + fmt) {
        case 0: return launch_mx_quant_t<float, 0>(p, sms, s);
        case 1: return launch_mx_quant_t<float, 1>(p, sms, s);
        case 2: return launch_mx_quant_t<__half, 0>(p, sms, s);
        case 3: return launch_mx_quant_t<__half, 1>(p, sms, s);
        case 4: return launch_mx_quant_t<__nv_bfloat16, 0>(p, sms, s);
        case 5: return launch_mx_quant_t<__nv_bfloat16, 1>(p, sms, s);
    }
    return -1;
}

int launch_mx_dequant(const MxCopyParams &p, int fmt, int dtype, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    const unsigned grid = mx_grid((long long)p.batch * p.rows * mx_ktiles(p.k), dev::kMxAhead);
    switch (2 * dtype + fmt) {
        case 0: return mx_launch(dev::q4mx_dequant_kernel<float, 0>, grid, p, s);
        case 1: return mx_launch(dev::q4mx_dequant_kernel<float, 1>, grid, p, s);
        case 2: return mx_launch(dev::q4mx_dequant_kernel<__half, 0>, grid, p, s);
        case 3: return mx_launch(dev::q4mx_dequant_kernel<__half, 1>, grid, p, s);
        case 4: return mx_launch(dev::q4mx_dequant_kernel<__nv_bfloat16, 0>, grid, p, s);
        case 5: return mx_launch(dev::q4mx_dequant_kernel<__nv_bfloat16, 1>, grid, p, s);
    }
    return -1;
}

int launch_mx_pack(const MxCopyParams &p, int fmt, bool unpack, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    const unsigned grid = mx_grid((long long)p.batch * p.rows * mx_ktiles(p.k), dev::kMxAhead);
    if (fmt == 0) return unpack ? mx_launch(dev::q4mx_pack_kernel<0, true>, grid, p, s) : mx_launch(dev::q4mx_pack_kernel<0, false>, grid, p, s);
    return unpack ? mx_launch(dev::q4mx_pack_kernel<1, true>, grid, p, s) : mx_launch(dev::q4mx_pack_kernel<1, false>, grid, p, s);
}

}  // namespace q4
