// mx_quant.cu -- rows into the microscaled 4-bit forms and back: quantising,
// optionally behind an RMSNorm (x / rms(x) gamma) or a SwiGLU (silu(x) up);
// dequantising; codes and scales from and into plain rows.
//
// Pure streams.  A warp takes 256 columns of a row, one record row: a lane eight
// consecutive values, so that a block of 32 (16) is four (two) lanes, its largest
// magnitude two (one) shuffles, and the warp's codes are one whole 128-byte line.
#include <algorithm>

#include "mx_common.cuh"

namespace q4 {
namespace dev {

constexpr int kMxThreads = 256, kMxWarps = kMxThreads / 32;

// Eight consecutive values in 16-byte words of T.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w_of(w[i / 4], i % 4));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = w_of(w[0], i);
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                } else {
                    v[2 * i] = __uint_as_float(x << 16);
                    v[2 * i + 1] = __uint_as_float(x & 0xFFFF0000u);
                }
            }
        }
    }
};

__device__ __forceinline__ float mx_silu(float g) { return g / (1.f + __expf(-g)); }

// A warp's 256 values (lane: 8 of them) of row `row`, column tile kt, into the
// matrix at `out`.
template <int FMT>
__device__ __forceinline__ void mx_store(uint8_t *out, int row, int kt, int KT, const float (&v)[8], float g, float six_g,
                                         int lane) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < mx_block(FMT) / 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    float mul;
    const uint32_t sc = mx_block_scale<FMT>(a, g, six_g, mul);
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = mx_scaled(v[i], mul);
    uint8_t *rec = out + ((size_t)(row / kMxRows) * KT + kt) * mx_rec(FMT);
    const int r = row % kMxRows;
    *reinterpret_cast<uint32_t *>(rec + mx_code_off(r, 4 * lane)) = e2m1x8(u);
    // four blocks' scales a word: lanes 0, 16 (MXFP4) or 0, 8, 16, 24 (NVFP4)
    constexpr int L = mx_block(FMT) / 8;  // lanes of a block
    uint32_t word = sc;
    word |= __shfl_down_sync(0xffffffffu, word, L) << 8;
    word |= __shfl_down_sync(0xffffffffu, word, 2 * L) << 16;
    if (lane % (4 * L) == 0) *reinterpret_cast<uint32_t *>(rec + mx_scale_off(r, lane / (4 * L))) = word;
}

// Values as they are, or a SwiGLU of two rows: a warp takes kMxAhead units (row,
// column tile), their loads issued together.
constexpr int kMxAhead = 4;
template <typename T, int FMT, bool GLU>
__global__ void __launch_bounds__(kMxThreads) q4mx_quant_kernel(const __grid_constant__ MxQuantParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // after the wait: a kernel that starts on this may read what was complete before
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, KT = mx_ktiles(p.k);
    const long long units = (long long)p.batch * p.rows * KT;
    const long long u0 = ((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * kMxAhead;
    const long long mat = (long long)mx_rtiles(p.rows) * KT * mx_rec(FMT);
    const float six_g = 6.f * p.scale;
    Raw8<T> x[kMxAhead], y[GLU ? kMxAhead : 1];
    long long row = u0 / KT;  // over the batch
    int kt = (int)(u0 - row * KT);
    const long long row0 = row;
    const int kt0 = kt;
    auto next = [&]() {
        if (++kt == KT) {
            kt = 0;
            ++row;
        }
    };
#pragma unroll
    for (int i = 0; i < kMxAhead; ++i, next()) {
        const int c = kt * kMxK + 8 * lane;
        x[i].zero();
        if constexpr (GLU) y[i].zero();
        if (u0 + i < units && c < p.k) {
            x[i].load((const T *)p.x + row * p.ld + c);
            if constexpr (GLU) y[i].load((const T *)p.up + row * p.ld + c);
        }
    }
    row = row0;
    kt = kt0;
#pragma unroll
    for (int i = 0; i < kMxAhead; ++i, next()) {
        if (u0 + i >= units) break;
        float v[8];
        x[i].values(v);
        if constexpr (GLU) {
            float w[8];
            y[i].values(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = mx_silu(v[e]) * w[e];
        }
        const long long b = p.batch == 1 ? 0 : row / p.rows;
        mx_store<FMT>(p.out + b * mat, (int)(row - b * p.rows), kt, KT, v, p.scale, six_g, lane);
    }
}

// Behind an RMSNorm: WPR warps a row (1 or all eight of the CTA), which keep up to
// R column tiles each in registers; what a longer row has beyond them is read
// again after the sum of squares is known.
template <typename T, int FMT, int WPR, int R>
__global__ void __launch_bounds__(kMxThreads) q4mx_quant_norm_kernel(const __grid_constant__ MxQuantParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float sums[kMxWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, KT = mx_ktiles(p.k);
    const int w = warp % WPR;
    const long long row = (long long)blockIdx.x * (kMxWarps / WPR) + warp / WPR, rows = (long long)p.batch * p.rows;
    const bool live = row < rows;
    const T *src = (const T *)p.x + (live ? row : 0) * p.ld;
    const float six_g = 6.f * p.scale;
    Raw8<T> x[R];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (w + i * WPR) * kMxK + 8 * lane;
        x[i].zero();
        if (live && c < p.k) x[i].load(src + c);
    }
    auto squares = [&](const Raw8<T> &a) {
        float v[8];
        a.values(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
    };
#pragma unroll
    for (int i = 0; i < R; ++i) squares(x[i]);
    for (int t = w + R * WPR; t < KT; t += WPR) {
        const int c = t * kMxK + 8 * lane;
        Raw8<T> a;
        a.zero();
        if (live && c < p.k) a.load(src + c);
        squares(a);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (WPR > 1) {
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMxWarps; ++i) sum += sums[i];
    }
    if (!live) return;
    const float rstd = 1.f / sqrtf(sum / (float)p.k + p.eps);
    const long long b = p.batch == 1 ? 0 : row / p.rows;
    uint8_t *out = p.out + b * ((long long)mx_rtiles(p.rows) * KT * mx_rec(FMT));
    const int r = (int)(row - b * p.rows);
    auto put = [&](const Raw8<T> &a, int t) {
        const int c = t * kMxK + 8 * lane;
        float v[8], gm[8] = {};
        a.values(v);
        if (c < p.k) {
            const float4 g0 = *reinterpret_cast<const float4 *>(p.gamma + c);
            const float4 g1 = *reinterpret_cast<const float4 *>(p.gamma + c + 4);
            gm[0] = g0.x, gm[1] = g0.y, gm[2] = g0.z, gm[3] = g0.w;
            gm[4] = g1.x, gm[5] = g1.y, gm[6] = g1.z, gm[7] = g1.w;
        }
        // (columns behind k are zeros even where rstd is infinite or NaN)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c < p.k ? v[e] * rstd * gm[e] : 0.f;
        mx_store<FMT>(out, r, t, KT, v, p.scale, six_g, lane);
    };
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (w + i * WPR < KT) put(x[i], w + i * WPR);
    for (int t = w + R * WPR; t < KT; t += WPR) {
        const int c = t * kMxK + 8 * lane;
        Raw8<T> a;
        a.zero();
        if (c < p.k) a.load(src + c);
        put(a, t);
    }
}

// Back into values: g s e, rounded once to T.
template <typename T, int FMT>
__global__ void __launch_bounds__(kMxThreads) q4mx_dequant_kernel(const __grid_constant__ MxCopyParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, KT = mx_ktiles(p.k);
    const long long units = (long long)p.batch * p.rows * KT;
    const long long mat = (long long)mx_rtiles(p.rows) * KT * mx_rec(FMT);
    const long long u0 = ((long long)blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * kMxAhead;
    uint32_t code[kMxAhead], sc[kMxAhead];
    long long row = u0 / KT;
    int kt = (int)(u0 - row * KT);
    const long long row0 = row;
    const int kt0 = kt;
    auto next = [&]() {
        if (++kt == KT) {
            kt = 0;
            ++row;
        }
    };
    constexpr int L = mx_block(FMT) / 8;
#pragma unroll
    for (int i = 0; i < kMxAhead; ++i, next()) {
        code[i] = sc[i] = 0u;
        if (u0 + i < units) {
            const long long b = p.batch == 1 ? 0 : row / p.rows;
            const int rr = (int)(row - b * p.rows), r = rr % kMxRows;
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
        if (u0 + i >= units || c >= p.k) continue;
        const float s = mx_scale_value<FMT>(sc[i]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e2m1_value((code[i] >> (4 * e)) & 15u) * s * p.scale;
        T *dst = (T *)p.out + row * p.k + c;
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
// CTAs of a launch over `units` warps' work
unsigned mx_grid(long long units) {
    const long long per = (long long)dev::kMxWarps * dev::kMxAhead;
    return (unsigned)((units + per - 1) / per);
}
template <typename Kern, typename P>
int mx_launch(Kern kern, unsigned grid, const P &p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config(grid, dev::kMxThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

template <typename T, int FMT>
int launch_mx_quant_t(const MxQuantParams &p, cudaStream_t stream) {
    const int KT = mx_ktiles(p.k);
    const long long rows = (long long)p.batch * p.rows;
    if (p.gamma) {
        // a warp a row up to 2048 columns where there are rows for all SMs, else a CTA a row
        if (KT <= 2 || (KT <= 8 && rows >= 2048)) {
            const unsigned grid = (unsigned)((rows + dev::kMxWarps - 1) / dev::kMxWarps);
            if (KT <= 2) return mx_launch(dev::q4mx_quant_norm_kernel<T, FMT, 1, 2>, grid, p, stream);
            return mx_launch(dev::q4mx_quant_norm_kernel<T, FMT, 1, 8>, grid, p, stream);
        }
        if (KT <= 8) return mx_launch(dev::q4mx_quant_norm_kernel<T, FMT, 8, 1>, (unsigned)rows, p, stream);
        if (KT <= 16) return mx_launch(dev::q4mx_quant_norm_kernel<T, FMT, 8, 2>, (unsigned)rows, p, stream);
        return mx_launch(dev::q4mx_quant_norm_kernel<T, FMT, 8, 8>, (unsigned)rows, p, stream);
    }
    const unsigned grid = mx_grid(rows * KT);
    if (p.up) return mx_launch(dev::q4mx_quant_kernel<T, FMT, true>, grid, p, stream);
    return mx_launch(dev::q4mx_quant_kernel<T, FMT, false>, grid, p, stream);
}
}  // namespace

int launch_mx_quant(const MxQuantParams &p, int fmt, int dtype, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    switch (2 * dtype + fmt) {
        case 0: return launch_mx_quant_t<float, 0>(p, s);
        case 1: return launch_mx_quant_t<float, 1>(p, s);
        case 2: return launch_mx_quant_t<__half, 0>(p, s);
        case 3: return launch_mx_quant_t<__half, 1>(p, s);
        case 4: return launch_mx_quant_t<__nv_bfloat16, 0>(p, s);
        case 5: return launch_mx_quant_t<__nv_bfloat16, 1>(p, s);
    }
    return -1;
}

int launch_mx_dequant(const MxCopyParams &p, int fmt, int dtype, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    const unsigned grid = mx_grid((long long)p.batch * p.rows * mx_ktiles(p.k));
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
    const unsigned grid = mx_grid((long long)p.batch * p.rows * mx_ktiles(p.k));
    if (fmt == 0) return unpack ? mx_launch(dev::q4mx_pack_kernel<0, true>, grid, p, s) : mx_launch(dev::q4mx_pack_kernel<0, false>, grid, p, s);
    return unpack ? mx_launch(dev::q4mx_pack_kernel<1, true>, grid, p, s) : mx_launch(dev::q4mx_pack_kernel<1, false>, grid, p, s);
}

}  // namespace q4
