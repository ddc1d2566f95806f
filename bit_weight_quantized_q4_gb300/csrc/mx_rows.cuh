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
    __device__ __forceinline__ void values(float (&v)[16]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w_of(w[i / 4], i % 4));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = w_of(w[i / 4], i % 4);
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

// The codes of the sixteen values v f of each lane, and in the first lane of four
// blocks their scales' word; all lanes of a warp, those of a row in order.
template <int FMT>
__device__ __forceinline__ void mx_codes(const float (&v)[16], float f, const MxGain &gain, uint2 &code, uint32_t &word) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = max_abs(v[i], v[8 + i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max_abs(m[i], m[4 + i]);
    float a = max_abs(max_abs(m[0], m[1]), max_abs(m[2], m[3]));
    if constexpr (FMT == 0) a = max_abs(a, __shfl_xor_sync(0xffffffffu, a, 1));
    float mul;
    const uint32_t sc = mx_block_scale<FMT>(a * f, gain, mul);
    const float by = f * mul;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = v[i] * by;
        hi[i] = v[8 + i] * by;
    }
    code = mul == 0.f ? make_uint2(0u, 0u) : make_uint2(e2m1x8(lo), e2m1x8(hi));
    constexpr int L = mx_block(FMT) / 16;  // lanes of a block
    word = sc;
    word |= __shfl_down_sync(0xffffffffu, word, L) << 8;
    word |= __shfl_down_sync(0xffffffffu, word, 2 * L) << 16;
}

}  // namespace dev
}  // namespace q4
