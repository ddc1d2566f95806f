// attn_row.cuh -- one row and head of attention by the definition, for results
// that are not finite: only attended positions are touched, and no value enters
// as a product with zero that the formula does not have.
//
// A warp walks the positions 32 at a time with a running softmax, a position a
// lane for the scores, a dim a lane for the sums (a position at a time took
// seven times as long: its five shuffles and two loads waited for each other).
#pragma once
#include "paged.cuh"

namespace q4 {
namespace dev {

// The running softmax of a warp: lane l has dims l, l + 32, .. of the sums and its
// own positions' share of l.
template <int D>
struct RowSum {
    float m = -INFINITY, l = 0.f, acc[D / 32] = {};
    bool seen = false;  // a position had a page
};

// Positions k0 .. k0 + 31, none behind pos.  q: dims lane, lane + 32, .. in log2
// units.  Positions on pages out of range are skipped, and recorded.
template <typename T, int D>
__device__ __forceinline__ void attn_span(RowSum<D> &a, const PagedKv &kv, const float (&q)[D / 32], int seq, int hk,
                                          int k0, int pos, int lane, int *err) {
    constexpr int DL = D / 32, V = 16 / (int)sizeof(T);
    const int key = k0 + lane, col = page_col(kv, key);
    const int page = key <= pos ? page_at(kv, seq, col) : -1;
    if (key <= pos && page < 0) atomicExch(err, kErrPaged);
    const size_t off = page < 0 ? 0 : row_off(kv, page, hk, key - col * kv.page, D);
    const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
    a.seen = a.seen || have != 0u;
    float s = 0.f;
    // (two loads at a time: as many registers as the loads of a whole row make the
    // kernels that call this spill around the call)
#pragma unroll
    for (int i = 0; i < DL; ++i)
#pragma unroll 2
        for (int x = 0; x < 32; x += V) {
            T k[V];
            *reinterpret_cast<uint4 *>(k) =
                page < 0 ? make_uint4(0u, 0u, 0u, 0u)
                         : __ldcg(reinterpret_cast<const uint4 *>((const T *)kv.k + off + 32 * i + x));
#pragma unroll
            for (int e = 0; e < V; ++e) s = fmaf(__shfl_sync(0xffffffffu, q[i], x + e), to_f32(k[e]), s);
        }
    if (page < 0) s = -INFINITY;
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(a.m, mx), mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2(a.m - mu), w = ex2(s - mu);
    a.m = mn;
    a.l = fmaf(a.l, alpha, w);
#pragma unroll
    for (int i = 0; i < DL; ++i) a.acc[i] *= alpha;
#pragma unroll 1
    for (int j = 0; j < 32; j += 8) {
        float v[8][DL];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const size_t at = __shfl_sync(0xffffffffu, off, j + y);
#pragma unroll
            for (int i = 0; i < DL; ++i)
                v[y][i] = (have >> (j + y)) & 1u ? to_f32(__ldcg((const T *)kv.v + at + lane + 32 * i)) : 0.f;
        }
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const float wy = __shfl_sync(0xffffffffu, w, j + y);
#pragma unroll
            for (int i = 0; i < DL; ++i) a.acc[i] = fmaf(wy, v[y][i], a.acc[i]);
        }
    }
}

// Whether every output is NaN already (a score was NaN or +inf).
template <int D>
__device__ __forceinline__ bool all_nan(const RowSum<D> &a) {
    return __any_sync(0xffffffffu, a.l != a.l);
}

// out = sum_j p_j v_j over j in (pos - window, pos], p = softmax of scale q . k_j of
// a packed prompt row (one warp).  No position with a page: zeros; scores that are
// all -inf: 0 / 0.
template <typename T, int D>
__device__ __noinline__ void attn_row(const PrefillParams &p, int row, int head, int seq, int pos, int lane) {
    constexpr int DL = D / 32;
    const size_t at = ((size_t)row * p.H + head) * D + lane;
    float q[DL];
#pragma unroll
    for (int i = 0; i < DL; ++i) q[i] = to_f32(((const T *)p.q)[at + 32 * i]) * (p.scale * 1.4426950408889634f);
    RowSum<D> a;
    const int lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    for (int k0 = lo; k0 <= pos && !all_nan(a); k0 += 32)
        attn_span<T, D>(a, p.kv, q, seq, head / (p.H / p.kv.hkv), k0, pos, lane, p.err);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.l += __shfl_xor_sync(0xffffffffu, a.l, o);
#pragma unroll
    for (int i = 0; i < DL; ++i) ((T *)p.out)[at + 32 * i] = from_f32<T>(a.seen ? a.acc[i] / a.l : 0.f);
}

}  // namespace dev
}  // namespace q4
