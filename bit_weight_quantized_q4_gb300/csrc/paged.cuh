// paged.cuh -- what the kernels over a paged KV cache share: the cache's
// device view, the cache element types and RoPE row lookups.
//
// A page holds page_size consecutive positions of every kv head:
// [kv_heads][page_size][D] of f32, f16 or bf16; position p of sequence b lies
// in page table[b][p / page_size], slot p % page_size.  A table entry outside
// 0 .. num_pages - 1 is never followed.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q4_internal.h"

namespace q4 {
namespace dev {

constexpr int kErrPaged = 5;  // error word: a position, page or token out of range

// Table column of position p (p / page), without a division.
__device__ __forceinline__ int page_col(const PagedKv &kv, int p) {
    return kv.page == 1 ? p : (int)(__umulhi((unsigned)p, kv.page_mul) >> kv.page_shift);
}
// Page id of table column `i` of sequence b, or -1 where the table's entry
// (or the column) is out of range.
__device__ __forceinline__ int page_at(const PagedKv &kv, int b, int i) {
    if ((unsigned)i >= (unsigned)kv.width) return -1;
    const int id = kv.table[(size_t)b * kv.width + i];
    return (unsigned)id < (unsigned)kv.num_pages ? id : -1;
}
// The same in two steps, for a lookup ahead of its use: the raw entry (a load
// whose result nothing needs yet), and its check.
__device__ __forceinline__ int page_raw(const PagedKv &kv, int b, int i) {
    return (unsigned)i < (unsigned)kv.width ? kv.table[(size_t)b * kv.width + i] : -1;
}
__device__ __forceinline__ int page_ok(const PagedKv &kv, int id) {
    return (unsigned)id < (unsigned)kv.num_pages ? id : -1;
}
// Element offset of (page, kv head, slot, dim 0).
__device__ __forceinline__ size_t row_off(const PagedKv &kv, int page, int hk, int slot, int D) {
    return (((size_t)page * kv.hkv + hk) * kv.page + slot) * (size_t)D;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two floats as one word of a 16-bit type, `a` in the low half (nearest even).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Four consecutive values rounded to T and stored (16-byte aligned for f32,
// 8-byte for the 16-bit types).
template <typename T>
__device__ __forceinline__ void store4(T *dst, float4 v) {
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4 *>(dst) = v;
    else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
}

// (a, b) -> (a c - b s, b c + a s) for four pairs.
__device__ __forceinline__ void rotate4(float4 &a, float4 &b, const float4 &c, const float4 &s) {
    const float4 x = a, y = b;
    a = make_float4(x.x * c.x - y.x * s.x, x.y * c.y - y.y * s.y, x.z * c.z - y.z * s.z, x.w * c.w - y.w * s.w);
    b = make_float4(y.x * c.x + x.x * s.x, y.y * c.y + x.y * s.y, y.z * c.z + x.z * s.z, y.w * c.w + x.w * s.w);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Word i of four, i a constant after unrolling.
__device__ __forceinline__ uint32_t w_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Two fp32 values in one 64-bit register, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pair_u32(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
    return pair_u32(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ float lo_f32(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_f32(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace dev
}  // namespace q4
