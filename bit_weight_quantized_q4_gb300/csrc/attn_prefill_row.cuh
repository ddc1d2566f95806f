// attn_prefill_row.cuh -- one packed prompt row and head by the definition:
// one warp walks the attended positions in order with a running softmax.
#pragma once
#include "paged.cuh"

namespace q4 {
namespace dev {

// out = sum_j p_j v_j over j in (pos - window, pos], p = softmax of scale q . k_j;
// lane l holds dims l, l + 32, ...; positions on pages out of range are skipped (all
// of them: zeros).  Scores that are all -inf are 0 / 0.
template <typename T, int D>
__device__ __noinline__ void attn_row(const PrefillParams &p, int row, int head, int seq, int pos, int lane) {
    constexpr int DL = D / 32;
    const int hk = head / (p.H / p.kv.hkv);
    const T *q = (const T *)p.q + ((size_t)row * p.H + head) * D;
    float qv[DL], acc[DL];
#pragma unroll
    for (int i = 0; i < DL; ++i) {
        qv[i] = to_f32(q[lane + 32 * i]) * (p.scale * 1.4426950408889634f);
        acc[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    int page = -1, col = -1;
    bool seen = false;
    for (int j = lo; j <= pos; ++j) {
        if (j / p.kv.page != col) {
            col = j / p.kv.page;
            page = page_at(p.kv, seq, col);
            if (page < 0 && lane == 0) atomicExch(p.err, kErrPaged);
        }
        if (page < 0) continue;
        seen = true;
        const size_t off = row_off(p.kv, page, hk, j - col * p.kv.page, D);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < DL; ++i) s = fmaf(qv[i], to_f32(((const T *)p.kv.k)[off + lane + 32 * i]), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m - mu), e = ex2(s - mu);
        m = mn;
        l = fmaf(l, alpha, e);
#pragma unroll
        for (int i = 0; i < DL; ++i) acc[i] = fmaf(e, to_f32(((const T *)p.kv.v)[off + lane + 32 * i]), acc[i] * alpha);
    }
    T *out = (T *)p.out + ((size_t)row * p.H + head) * D;
#pragma unroll
    for (int i = 0; i < DL; ++i) out[lane + 32 * i] = from_f32<T>(seen ? acc[i] / l : 0.f);
}

}  // namespace dev
}  // namespace q4
