// mx_rows.cuh -- rows of values into microscaled 4-bit codes, sixteen values a lane
// (mx_quant.cu, mx_gemm.cu).
#pragma once
#include "mx_common.cuh"

namespace q4 {
namespace dev {

// Sixteen consecutive values as they are stored.
template <typename T>
struct Raw16 {
    static constexpr int N = (int)sizeof(T);
    uint4 w[N];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // values 2 i and 2 i + 1 as a pair
    __device__ __forceinline__ void pairs(uint64_t (&v)[8]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = pair_u32(w_of(w[i / 2], 2 * (i % 2)), w_of(w[i / 2], 2 * (i % 2) + 1));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = w_of(w[i / 4], i % 4);
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                    v[i] = pair_f32(f.x, f.y);
                } else {
                    v[i] = pair_u32(x << 16, x & 0xFFFF0000u);
                }
            }
        }
    }
};

// v silu(g) of sixteen values each.
__device__ __forceinline__ void mx_glu(uint64_t (&v)[8], const uint64_t (&up)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul_f32x2(pair_f32(mx_silu(lo_f32(v[i])), mx_silu(hi_f32(v[i]))), up[i]);
}
// Sixteen consecutive factors.
__device__ __forceinline__ void mx_factors(uint64_t (&v)[8], const float *src) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 g = *reinterpret_cast<const float4 *>(src + 4 * i);
        v[2 * i] = pair_f32(g.x, g.y);
        v[2 * i + 1] = pair_f32(g.z, g.w);
    }
}
// 1 / sqrt(mean of squares + eps) of a row, from its sum (inv_k = 1 / k).
__device__ __forceinline__ float mx_rstd(float sum, float inv_k, float eps) { return rsqrtf(fmaf(sum, inv_k, eps)); }

// The codes of the sixteen values v of each lane, and in the first lane of four
// blocks their scales' word; all lanes of a warp, those of a row in order.  (A row's
// factor is in v already: its product with a block's, 2^127 for a block of zeros, may
// be infinite.)
template <int FMT>
__device__ __forceinline__ void mx_codes(const uint64_t (&v)[8], const MxGain &gain, uint2 &code, uint32_t &word) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = max_abs(lo_f32(v[i]), hi_f32(v[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max_abs(m[i], m[4 + i]);
    float a = max_abs(max_abs(m[0], m[1]), max_abs(m[2], m[3]));
    if constexpr (FMT == 0) a = max_abs(a, __shfl_xor_sync(0xffffffffu, a, 1));
    float mul;
    const uint32_t sc = mx_block_scale<FMT>(a, gain, mul);
    const uint64_t by = pair_f32(mul, mul);
    uint64_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = mul_f32x2(v[i], by);
    const uint64_t lo[4] = {u[0], u[1], u[2], u[3]}, hi[4] = {u[4], u[5], u[6], u[7]};
    code = mul == 0.f ? make_uint2(0u, 0u) : make_uint2(e2m1x8(lo), e2m1x8(hi));
    constexpr int L = mx_block(FMT) / 16;  // lanes of a block
    word = sc;
    word |= __shfl_down_sync(0xffffffffu, word, L) << 8;
    word |= __shfl_down_sync(0xffffffffu, word, 2 * L) << 16;
}

}  // namespace dev
}  // namespace q4
