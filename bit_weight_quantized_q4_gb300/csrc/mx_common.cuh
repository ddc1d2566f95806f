// mx_common.cuh -- what the kernels of the microscaled 4-bit formats share: the
// stored forms, and the block-scaled tensor core (tcgen05 kind::mxf4 and
// kind::mxf4nvf4).
//
// A code is E2M1: 0, .5, 1, 1.5, 2, 3, 4, 6 and a sign.  MXFP4: blocks of 32
// share an E8M0 power of two (255: NaN).  NVFP4: blocks of 16 share an E4M3
// factor (127: NaN), the matrix an fp32 one.
#pragma once
#include "gemv_launch.cuh"
#include "paged.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace q4 {
namespace dev {

constexpr uint32_t kInfBits = 0x7F800000u;

// Offset in a record of byte `c` (of 128) of row r's codes, and of row r's scale
// word w.
__device__ __forceinline__ uint32_t mx_code_off(int r, int c) {
    return (uint32_t)(r * 128 + (((c >> 4) ^ (r & 7)) << 4) + (c & 15));
}
__device__ __forceinline__ uint32_t mx_scale_off(int r, int w) {
    return (uint32_t)(kMxCodes + w * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4);
}

// Eight values as codes, value i in bits 4 i .. (to nearest, ties to the even
// code, within 6).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t (&p)[4]) {
    const float v[8] = {lo_f32(p[0]), hi_f32(p[0]), lo_f32(p[1]), hi_f32(p[1]), lo_f32(p[2]), hi_f32(p[2]), lo_f32(p[3]), hi_f32(p[3])};
    return e2m1x8(v);
}
__device__ __forceinline__ uint32_t e2m1(float v) {
    uint16_t w;
    asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.u16.u8 %0, a;\n\t}"
        : "=h"(w)
        : "f"(v), "f"(0.f));
    return w & 15u;
}
// The values of a word's eight codes.
__device__ __forceinline__ void e2m1_values(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b & 255u));
    return __half2float(__ushort_as_half((unsigned short)h));
}
// 2^(E - 127); E = 255: NaN.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
    return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23);
}
template <int FMT>
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
    return FMT == 0 ? e8m0_value(b) : e4m3_value(b);
}

// The larger magnitude, with any sign; NaN where one is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float m;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// silu(g), g / (1 + exp(-g)): off by about 4 + 1.17 |g| units in the last place (the fast
// exponential by 2 + 1.17 |g|, the fast quotient by 2), 27 of them at g = -20; zero below -87.3,
// where the denominator passes 2^126 (the value: -1e-36); -inf: NaN, as the formula has it.
__device__ __forceinline__ float mx_silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

// NVFP4's factor g of the whole matrix, 6 g, and 1 / (6 g) to the nearest fp32.
struct MxGain {
    float g = 1.f, six_g = 6.f, inv = 0.f;
};

// The scale byte of a block whose largest magnitude is |a|, and the factor its
// values are multiplied with before they are rounded to codes.
//   MXFP4: the smallest power of two s with |a| <= 6 s = 1.5 * 2^2 s, 2^-127 at least.
//   NVFP4: |a| / (6 g) to the nearest E4M3, 448 at most.  The quotient is the nearest
//   fp32 one, by Markstein's method (IBM J. Res. Dev. 34, 1990): from the nearest 1 / b,
//   q + (a - q b) (1 / b) with an exact remainder is the nearest fp32 to a / b once q is
//   within a unit in the last place of it, which one such step ensures.  1 / (s g): one
//   such step from the hardware's estimate, which is within a unit already; the method
//   leaves out significands of ones alone, and values beside every border of codes are tested
//   with those too.  (Divisions of the language took as long as the rest of the kernel.)
// A block with an infinity or NaN: a NaN scale, and a factor of 0: its codes are zeros.
template <int FMT>
__device__ __forceinline__ uint32_t mx_block_scale(float a, const MxGain &gain, float &mul) {
    const uint32_t bits = __float_as_uint(a) & 0x7FFFFFFFu;
    if constexpr (FMT == 0) {
        const int E = max((int)(bits >> 23) - ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 2), 0);
        mul = bits < kInfBits ? __uint_as_float((uint32_t)(254 - E) << 23) : 0.f;
        return bits < kInfBits ? (uint32_t)E : 255u;
    } else {
        const float x = __uint_as_float(bits);
        const float q = x * gain.inv;
        float t = fmaf(fmaf(-q, gain.six_g, x), gain.inv, q);
        t = fmaf(fmaf(-t, gain.six_g, x), gain.inv, t);
        t = q < 500.f ? fminf(t, 448.f) : 448.f;  // (beyond, the remainder may overflow)
        uint16_t b;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(t));
        const uint32_t sc = b & 255u;
        const float sg = e4m3_value(sc) * gain.g;
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sg));
        r = fmaf(r, fmaf(-sg, r, 1.f), r);
        mul = sc != 0u && bits < kInfBits ? r : 0.f;
        return bits < kInfBits ? sc : 127u;
    }
}

// ------------------------------------------------------------------ tensor core

// D[tmem] (+)= sum over blocks of sA sB A B^T, M = 128, N, K = 64, one thread.
// a, b: lower words of the operands' descriptors (128-byte swizzle, K-major); sa,
// sb: the scale factors' tensor-memory addresses.  Descriptor of the instruction:
// bits 4-5 and 29-30 the byte of sb's and sa's word where the blocks' factors
// begin, 7-9 and 10-11 the types (1: E2M1), 17-22 N / 8, 23 the factors' type (1:
// E8M0, 0: E4M3), 27-28 M / 128.
template <int FMT>
__device__ __forceinline__ constexpr uint32_t mx_idesc(int N, int id) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (FMT == 0 ? 1u << 23 : 0u) | (1u << 27) |
           ((uint32_t)id << 4) | ((uint32_t)id << 29);
}
template <int FMT>
__device__ __forceinline__ void mx_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t acc) {
    if constexpr (FMT == 0)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "n"(tc::kSw128Hi)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "n"(tc::kSw128Hi)
            : "memory");
}
// One word of 128 rows' scales (512 bytes of shared memory) into four columns of
// tensor memory, the same in all four quarters of the lanes.  The descriptor: no
// swizzle, groups of 8 rows of 16 bytes 128 bytes apart.
__device__ __forceinline__ void mx_copy_scales(uint32_t taddr, uint32_t saddr) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(tc::smem_desc(saddr, 128, 128))
                 : "memory");
}

// global -> shared bulk copy without a cache hint.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// All threads of the cluster's CTAs (whole warps).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A value into the shared memory (offset as here) of the cluster's CTA `rank`.
__device__ __forceinline__ void store_peer(uint32_t saddr, uint32_t rank, float v) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f32 [a], %2;\n\t}" ::"r"(saddr),
        "r"(rank), "f"(v)
        : "memory");
}

}  // namespace dev
}  // namespace q4
