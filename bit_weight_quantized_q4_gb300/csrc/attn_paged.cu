// attn_paged.cu -- attention of one new token per sequence over a paged KV
// cache (honeycrisp/mod.rs: gpu_attention and the fused RoPE + KV-append +
// SDPA dispatch of forward_decode_fused_layers, for a batch of sequences):
// RoPE of q and the new k, append of k and v at the sequence's position, then
// out_h = sum_t p_t v_t, p = softmax over the attended t of scale q_h . k_t.
//
// The work is HBM-bound on the cache rows, whatever the cache's type: a kv
// head's G query heads share each row, so the arithmetic runs on the tensor
// cores (mma.sync m16n8k16: the batch of 8 columns is the group's heads) and
// costs a fraction of the row's load time.  A warp takes 16 positions per
// step, entirely in registers:
//   S^T [16 positions][heads] = K Q^T   A = K rows as loaded (16 bytes of a row
//        per lane; the k order inside a 32-dim block is permuted, and Q's
//        fragments carry the same permutation),
//   O^T [dims][heads] += V^T P^T        A = V rows, pairs of positions packed,
//        rows of the m tiles permuted so that a lane's 16 bytes of a V row are
//        rows of its own tiles; P goes through movmatrix.
// Nothing goes through shared memory but Q's fragments and the final merge.
//
// Precision: q and p stay fp32-like.  f16 caches: q (scaled per head by a
// power of two) and p enter as two f16 parts (22 bits); bf16 caches: as three
// bf16 parts (24 bits); f32 caches: K and V as three bf16 parts too, with the
// six products of order >= 2^-16.  The cache's values themselves are exact.
//
// Split: the 128-position units of all (sequence, kv head) pairs form one
// line that the CTAs divide evenly, whatever the lengths; lengths are read on
// the device, so a captured launch follows them.  A pair cut by a boundary is
// joined by the last of its CTAs to finish, in CTA order: the result does not
// depend on scheduling.
#include <algorithm>

#include "gemv_launch.cuh"
#include "paged.cuh"

namespace q4 {
namespace dev {

constexpr int kPagedWarps = 8;
constexpr int kPagedUnit = 16 * kPagedWarps;  // positions of one unit

template <typename T>
struct PagedT;
template <>
struct PagedT<__half> {
    using M = __half;
    static constexpr int KP = 1, QP = 2;  // parts of a cache value, of q and p
    static constexpr bool SCALED = true;
    static constexpr float PEXP = 14.f;  // p reaches 2^14: its low part stays a normal f16
};
template <>
struct PagedT<__nv_bfloat16> {
    using M = __nv_bfloat16;
    static constexpr int KP = 1, QP = 3;
    static constexpr bool SCALED = false;
    static constexpr float PEXP = 0.f;
};
template <>
struct PagedT<float> {
    using M = __nv_bfloat16;
    static constexpr int KP = 3, QP = 3;
    static constexpr bool SCALED = false;
    static constexpr float PEXP = 0.f;
};

// (a, b) as N words of the 16-bit type M whose values add up to a and b
// (each part the nearest M to what the parts before it leave).
template <typename M, int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = pack2<M>(a, b);
        if (i + 1 < N) {
            if constexpr (std::is_same<M, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                a -= f.x;
                b -= f.y;
            } else {
                a -= __uint_as_float(w[i] << 16);
                b -= __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
}

template <typename M>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<M, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float f_of(const uint4 &v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
}
__device__ __forceinline__ uint32_t w_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Shared memory of a CTA: the prefix of units over the sequences, Q's
// fragments and factors, the warps' maxima and sums, the fold's sums, a flag,
// then the warps' outputs [warps][G][D] (also the fold's weights).
template <typename T, int D, int NT>
struct PagedSmem {
    static constexpr int Prefix = 0;
    static constexpr int Qf = Prefix + 8 * (kMaxSeqs + 2);
    static constexpr int Qs = Qf + PagedT<T>::QP * NT * (D / 16) * 32 * 8;
    static constexpr int Wm = Qs + 4 * 8 * NT;
    static constexpr int Wl = Wm + 4 * kPagedWarps * 8 * NT;
    static constexpr int Fl = Wl + 4 * kPagedWarps * 8 * NT;  // [8 NT] fold sums
    static constexpr int Flag = Fl + 4 * 8 * NT;
    static constexpr int Red = (Flag + 16 + 15) / 16 * 16;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kPagedWarps, (sizeof(T) == 4 && D == 128) || NT == 2 ? 1 : 2)
    q4attn_paged_kernel(const __grid_constant__ PagedAttnParams p) {
    using C = PagedT<T>;
    using M = typename C::M;
    using S = PagedSmem<T, D, NT>;
    constexpr int KP = C::KP, QP = C::QP, NW = kPagedWarps, KS = D / 16, KB = D / 32, VB = D / 64;
    constexpr int LV = sizeof(T) == 4 ? 2 : 1;  // 16-byte loads per 8 values
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int hkv = p.kv.hkv, G = p.H / hkv, nseq = p.kv.nseq;
    long long *prefix = reinterpret_cast<long long *>(smem + S::Prefix);
    uint2 *qf = reinterpret_cast<uint2 *>(smem + S::Qf);
    float *qs = reinterpret_cast<float *>(smem + S::Qs);
    float *wm = reinterpret_cast<float *>(smem + S::Wm), *wl = reinterpret_cast<float *>(smem + S::Wl);
    float *fl = reinterpret_cast<float *>(smem + S::Fl);
    int *flag = reinterpret_cast<int *>(smem + S::Flag);
    float *red = reinterpret_cast<float *>(smem + S::Red);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const long long cap = (long long)p.kv.width * p.kv.page;
    auto lo_of = [&](int pos) { return p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0; };
    // units of one kv head of sequence b: 0 for an idle row (or a position
    // the cache or the RoPE tables do not have)
    auto units_of = [&](int pos) -> int {
        if (pos < 0 || pos >= cap || (p.rope_cos && pos >= p.rope_rows)) return 0;
        const int lo = lo_of(pos) & ~15;
        return (pos - lo) / kPagedUnit + 1;
    };
    {  // prefix[b] = units of sequences before b (all kv heads): four sequences a thread
        int pos[4];
        long long n[4], own = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = 4 * tid + i;
            pos[i] = b < nseq ? p.positions[b] : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            n[i] = (long long)units_of(pos[i]) * hkv;
            own += n[i];
        }
        long long inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        long long *wsum = reinterpret_cast<long long *>(red);
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        long long base = inc - own;
        for (int w = 0; w < warp; ++w) base += wsum[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = 4 * tid + i;
            if (b <= nseq) prefix[b] = base;
            base += n[i];
        }
        if (tid == 255 && nseq == kMaxSeqs) prefix[nseq] = base;
        __syncthreads();
    }
    // idle rows: zeros
    for (int b = blockIdx.x; b < nseq; b += gridDim.x)
        if (prefix[b + 1] == prefix[b]) {
            for (int i = tid; i < p.H * D; i += 32 * NW) p.out[(size_t)b * p.H * D + i] = 0.f;
            if (tid == 0 && p.positions[b] >= 0) atomicExch(p.err, kErrPaged);
        }
    const long long W = prefix[nseq];
    // CTAs with work: never more than units, so that none of a pair's CTAs is
    // without a share (each adds to the pair's count)
    const int N = W < gridDim.x ? (int)W : (int)gridDim.x, cta = blockIdx.x;
    if (cta >= N) return;
    const long long u0 = W * cta / N, u1 = W * (cta + 1) / N;
    int b = 0;
    {  // the last b with prefix[b] <= u0 that has units
        int hi = nseq;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (prefix[mid] <= u0)
                b = mid;
            else
                hi = mid;
        }
    }
    const float qscale = p.scale * 1.4426950408889634f;
    const size_t slot_floats = (size_t)G * (D + 2);

    for (long long u = u0; u < u1;) {
        while (prefix[b + 1] <= u) ++b;
        const int pos = p.positions[b], lo = lo_of(pos), base16 = lo & ~15;
        const int cs = units_of(pos);
        const long long rem = u - prefix[b];
        const int hk = (int)(rem / cs), st = (int)(rem - (long long)hk * cs);
        const long long s0 = prefix[b] + (long long)hk * cs, s1 = s0 + cs;  // the pair's units
        const long long ue = s1 < u1 ? s1 : u1;
        const int n_units = (int)(ue - u);
        const bool owner = ue == s1;  // this segment ends with the new token
        const float *cosr = p.rope_cos ? p.rope_cos + (size_t)pos * (D / 2) : nullptr;
        const float *sinr = p.rope_cos ? p.rope_sin + (size_t)pos * (D / 2) : nullptr;

        // the group's query heads: rotated, scaled (log2 units), in parts, as
        // B fragments; lane j < D / 8 holds dims 4j.. and D/2 + 4j..
        for (int h = warp; h < 8 * NT; h += NW) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
            if (h < G && lane < D / 8) {
                const float *src = p.q + ((size_t)b * p.H + hk * G + h) * D + 4 * lane;
                a = *reinterpret_cast<const float4 *>(src);
                c = *reinterpret_cast<const float4 *>(src + D / 2);
                if (cosr)
                    rotate4(a, c, *reinterpret_cast<const float4 *>(cosr + 4 * lane),
                            *reinterpret_cast<const float4 *>(sinr + 4 * lane));
            }
            float f = qscale;
            if constexpr (C::SCALED) {
                float mx = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                                 fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(c.z), fabsf(c.w))));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                // mx = f 2^e: f = 2^(14 - e) puts it in [2^13, 2^14)
                f = 1.f;
                float back = qscale;
                if (mx > 0.f && mx < INFINITY) {
                    int e;
                    frexpf(mx, &e);
                    const int se = min(max(14 - e, -126), 126);
                    f = ldexpf(1.f, se);
                    back = ldexpf(qscale, -se);
                }
                if (lane == 0) qs[h] = back;
            }
            if (lane < D / 8) {
                const int nt = h >> 3, gg = h & 7;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float4 v = half ? c : a;
                    const int d = 4 * lane + half * (D / 2), kb = d >> 5, r = d & 31;
                    const int ks = 2 * kb + ((r >> 2) & 1), ln = gg * 4 + (r >> 3);
                    uint32_t w0[QP], w1[QP];
                    split2<M, QP>(v.x * f, v.y * f, w0);
                    split2<M, QP>(v.z * f, v.w * f, w1);
#pragma unroll
                    for (int i = 0; i < QP; ++i) qf[((i * NT + nt) * KS + ks) * 32 + ln] = make_uint2(w0[i], w1[i]);
                }
            }
        }
        if (owner && warp < 2) {  // append: warp 0 the new k (rotated), warp 1 the new v
            const int page = page_at(p.kv, b, pos / p.kv.page);
            if (page < 0) {
                if (lane == 0) atomicExch(p.err, kErrPaged);
            } else if (lane < D / 8) {
                const float *src = (warp == 0 ? p.k_new : p.v_new) + ((size_t)b * hkv + hk) * D + 4 * lane;
                float4 a = *reinterpret_cast<const float4 *>(src), c = *reinterpret_cast<const float4 *>(src + D / 2);
                if (warp == 0 && cosr)
                    rotate4(a, c, *reinterpret_cast<const float4 *>(cosr + 4 * lane),
                            *reinterpret_cast<const float4 *>(sinr + 4 * lane));
                T *dst = (T *)(warp == 0 ? p.kv.k : p.kv.v) + row_off(p.kv, page, hk, pos % p.kv.page, D) + 4 * lane;
                store4(dst, a);
                store4(dst + D / 2, c);
            }
        }
        __syncthreads();  // Q's fragments; the appended rows, for this CTA's loads

        float m[NT][2], l[NT][2], qi[NT][2], acc[NT][KS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nt][i] = -INFINITY;
                l[nt][i] = 0.f;
                qi[nt][i] = C::SCALED ? qs[8 * nt + 2 * t + i] : 1.f;
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][j][i] = 0.f;

        uint4 kr[KB][2][LV], vr[VB][4][LV];
        const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
        // a step's first position, its first row's element offset (or none)
        // and the attended rows [r0, r1) of its 16
        struct Step {
            size_t off;
            int r0, r1;
        };
        auto step_of = [&](int s) {
            Step x;
            const int key0 = base16 + 16 * s;
            x.r0 = max(lo - key0, 0);
            x.r1 = min(pos - key0 + 1, 16);
            x.off = 0;
            if (x.r1 > x.r0) {
                const int col = key0 / p.kv.page, page = page_at(p.kv, b, col);
                if (page < 0) {
                    x.r1 = 0;
                    if (lane == 0) atomicExch(p.err, kErrPaged);
                } else {
                    x.off = row_off(p.kv, page, hk, key0 - col * p.kv.page, D);
                }
            }
            return x;
        };
        auto load_k = [&](const Step &x) {
            const T *base = (const T *)p.kv.k + x.off;
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int r = g + 8 * rr;
                const bool ok = r >= x.r0 && r < x.r1;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < LV; ++i)
                        kr[kb][rr][i] =
                            ok ? __ldcg(reinterpret_cast<const uint4 *>(base + (size_t)r * D + 32 * kb + 8 * t) + i)
                               : zero4;
            }
        };
        auto load_v = [&](const Step &x) {
            const T *base = (const T *)p.kv.v + x.off;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int r = 2 * t + (kk & 1) + 8 * (kk >> 1);
                const bool ok = r >= x.r0 && r < x.r1;
#pragma unroll
                for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                    for (int i = 0; i < LV; ++i)
                        vr[vb][kk][i] =
                            ok ? __ldcg(reinterpret_cast<const uint4 *>(base + (size_t)r * D + 64 * vb + 8 * g) + i)
                               : zero4;
            }
        };

        const int first = st * NW, last = (st + n_units) * NW;  // 16-position steps of this segment
        Step cur = step_of(first + warp);
        load_k(cur);
        for (int s = first + warp; s < last; s += NW) {
            load_v(cur);
            Step nxt = cur;
            if (s + NW < last) nxt = step_of(s + NW);
            // scores: rows g and g + 8, heads 2t and 2t + 1
            float sc[NT][QP][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < QP; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[nt][i][e] = 0.f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int hs = 0; hs < 2; ++hs) {
                    uint32_t a[KP][4];
                    if constexpr (KP == 1) {
                        a[0][0] = w_of(kr[kb][0][0], 2 * hs);
                        a[0][1] = w_of(kr[kb][1][0], 2 * hs);
                        a[0][2] = w_of(kr[kb][0][0], 2 * hs + 1);
                        a[0][3] = w_of(kr[kb][1][0], 2 * hs + 1);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 &x = kr[kb][e & 1][LV == 2 ? hs : 0];
                            uint32_t w[KP];
                            split2<M, KP>(f_of(x, 2 * (e >> 1)), f_of(x, 2 * (e >> 1) + 1), w);
#pragma unroll
                            for (int i = 0; i < KP; ++i) a[i][e] = w[i];
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < QP; ++i) {
                            const uint2 bq = qf[((i * NT + nt) * KS + 2 * kb + hs) * 32 + lane];
#pragma unroll
                            for (int j = 0; j < KP; ++j)
                                if (i + j < QP) mma16816<M>(sc[nt][i], a[j], bq.x, bq.y);
                        }
                }
            if (s + NW < last) load_k(nxt);
            const bool ok0 = g >= cur.r0 && g < cur.r1, ok1 = g + 8 >= cur.r0 && g + 8 < cur.r1;
            uint32_t pw[NT][2][QP];  // P as B fragments: positions 2t.. and 2t + 8.., head g
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = sc[nt][QP - 1][e];
#pragma unroll
                    for (int i = QP - 2; i >= 0; --i) v += sc[nt][i][e];
                    x[e] = (e < 2 ? ok0 : ok1) ? v * qi[nt][e & 1] : -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = fmaxf(x[i], x[2 + i]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float mn = fmaxf(m[nt][i], mx);
                    const float mu = mn == -INFINITY ? 0.f : mn;  // nothing attended yet
                    const float alpha = ex2(m[nt][i] - mu);
                    m[nt][i] = mn;
                    x[i] = ex2(x[i] - mu + C::PEXP);
                    x[2 + i] = ex2(x[2 + i] - mu + C::PEXP);
                    l[nt][i] = fmaf(l[nt][i], alpha, x[i] + x[2 + i]);
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        acc[nt][j][i] *= alpha;
                        acc[nt][j][2 + i] *= alpha;
                    }
                }
                uint32_t w0[QP], w1[QP];
                split2<M, QP>(x[0], x[1], w0);
                split2<M, QP>(x[2], x[3], w1);
#pragma unroll
                for (int i = 0; i < QP; ++i) {
                    pw[nt][0][i] = transpose8x8(w0[i]);
                    pw[nt][1][i] = transpose8x8(w1[i]);
                }
            }
            // outputs: m tile (vb, j) has rows dim 64 vb + 8 g + j and + 4
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a[KP][4];
                    if constexpr (KP == 1) {
                        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
#pragma unroll
                        for (int e = 0; e < 4; ++e)  // e & 1: + 4 dims; e >> 1: + 8 positions
                            a[0][e] = __byte_perm(w_of(vr[vb][2 * (e >> 1)][0], (j >> 1) + 2 * (e & 1)),
                                                  w_of(vr[vb][2 * (e >> 1) + 1][0], (j >> 1) + 2 * (e & 1)), sel);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[KP];
                            split2<M, KP>(f_of(vr[vb][2 * (e >> 1)][LV == 2 ? (e & 1) : 0], j),
                                          f_of(vr[vb][2 * (e >> 1) + 1][LV == 2 ? (e & 1) : 0], j), w);
#pragma unroll
                            for (int i = 0; i < KP; ++i) a[i][e] = w[i];
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = QP - 1; i >= 0; --i)
#pragma unroll
                            for (int jj = KP - 1; jj >= 0; --jj)
                                if (i + jj < QP) mma16816<M>(acc[nt][4 * vb + j], a[jj], pw[nt][0][i], pw[nt][1][i]);
                }
            cur = nxt;
        }

        // merge the warps in warp order: M = max_w m_w, l = sum l_w 2^(m_w - M), ...
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s = l[nt][i];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                const int h = 8 * nt + 2 * t + i;
                if (g == 0) {
                    wm[warp * 8 * NT + h] = m[nt][i];
                    wl[warp * 8 * NT + h] = s;
                }
                if (h < G) {
                    float *dst = red + ((size_t)warp * G + h) * D + 8 * g;
#pragma unroll
                    for (int vb = 0; vb < VB; ++vb) {
                        *reinterpret_cast<float4 *>(dst + 64 * vb) = make_float4(
                            acc[nt][4 * vb][i], acc[nt][4 * vb + 1][i], acc[nt][4 * vb + 2][i], acc[nt][4 * vb + 3][i]);
                        *reinterpret_cast<float4 *>(dst + 64 * vb + 4) =
                            make_float4(acc[nt][4 * vb][2 + i], acc[nt][4 * vb + 1][2 + i], acc[nt][4 * vb + 2][2 + i],
                                        acc[nt][4 * vb + 3][2 + i]);
                    }
                }
            }
        __syncthreads();
        const bool whole = u == s0 && ue == s1;
        float *mine = p.part + ((size_t)cta * 2 + (u == u0 ? 0 : 1)) * slot_floats;
        for (int idx = tid; idx < G * D; idx += 32 * NW) {
            const int h = idx / D;
            float Mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w) Mx = fmaxf(Mx, wm[w * 8 * NT + h]);
            const float mu = Mx == -INFINITY ? 0.f : Mx;
            float o = 0.f, L = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = ex2(wm[w * 8 * NT + h] - mu);
                o = fmaf(red[(size_t)w * G * D + idx], f, o);
                L = fmaf(wl[w * 8 * NT + h], f, L);
            }
            if (whole) {
                p.out[((size_t)b * p.H + hk * G) * D + idx] = L == 0.f ? 0.f : o / L;
            } else {
                mine[idx] = o;
                if (idx - h * D == 0) {
                    mine[G * D + h] = Mx;
                    mine[G * D + G + h] = L;
                }
            }
        }
        if (!whole) {
            // the last of the pair's CTAs to finish folds their shares in CTA order
            const long long c0 = ((s0 + 1) * N - 1) / W, c1 = (s1 * N - 1) / W;  // first and last CTA
            const int nc = (int)(c1 - c0) + 1;
            __threadfence();
            __syncthreads();
            if (tid == 0) *flag = atomicAdd(p.count + (size_t)b * hkv + hk, 1) == nc - 1;
            __syncthreads();
            if (*flag) {
                __threadfence();
                // CTA c0 + i's slot: its first segment, except a first CTA whose
                // range starts before the pair
                auto slot_of = [&](int i) {
                    const int sl = i == 0 && W * c0 / N != s0 ? 1 : 0;
                    return p.part + ((size_t)(c0 + i) * 2 + sl) * slot_floats;
                };
                float *wts = red;  // [nc][G]
                for (int h = warp; h < G; h += NW) {
                    float Mx = -INFINITY;
                    for (int i = lane; i < nc; i += 32) Mx = fmaxf(Mx, __ldcg(slot_of(i) + G * D + h));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
                    const float mu = Mx == -INFINITY ? 0.f : Mx;
                    float L = 0.f;
                    for (int i = lane; i < nc; i += 32) {
                        const float f = ex2(__ldcg(slot_of(i) + G * D + h) - mu);
                        wts[i * G + h] = f;
                        L = fmaf(__ldcg(slot_of(i) + G * D + G + h), f, L);
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
                    if (lane == 0) fl[h] = L;
                }
                __syncthreads();
                for (int idx = tid; idx < G * D; idx += 32 * NW) {
                    const int h = idx / D;
                    float o = 0.f;
#pragma unroll 8
                    for (int i = 0; i < nc; ++i) o = fmaf(__ldcg(slot_of(i) + idx), wts[i * G + h], o);
                    p.out[((size_t)b * p.H + hk * G) * D + idx] = fl[h] == 0.f ? 0.f : o / fl[h];
                }
                if (tid == 0) p.count[(size_t)b * hkv + hk] = 0;  // zero again for the next call
            }
        }
        __syncthreads();  // the shared memory is free for the next segment
        u = ue;
    }
}

}  // namespace dev

namespace {
// grid slots of one SM: two CTAs, one where the registers allow no more
int paged_occ(int dtype, int D, int G) { return (dtype == 0 && D == 128) || G > 8 ? 1 : 2; }
}  // namespace

int paged_attn_ctas(int dtype, int D, int G, int sms) { return paged_occ(dtype, D, G) * sms; }
size_t paged_attn_slot_floats(int D, int G) { return (size_t)G * (D + 2); }

template <typename T, int D, int NT>
static int launch_paged_t(const PagedAttnParams &p, int ctas, cudaStream_t stream) {
    auto kern = dev::q4attn_paged_kernel<T, D, NT>;
    static size_t smem_set[64] = {0};
    const int G = p.H / p.kv.hkv;
    // the merge area also holds the fold's weights, one per CTA and head
    const size_t merge = sizeof(float) * G * (size_t)std::max(dev::kPagedWarps * D, ctas);
    const size_t smem = dev::PagedSmem<T, D, NT>::Red + merge;
    if (!raise_smem(kern, smem, smem_set)) return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(32 * dev::kPagedWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

template <typename T>
static int launch_paged_d(const PagedAttnParams &p, int ctas, cudaStream_t stream) {
    const bool wide = p.H / p.kv.hkv > 8;
    if (p.D == 64) return wide ? launch_paged_t<T, 64, 2>(p, ctas, stream) : launch_paged_t<T, 64, 1>(p, ctas, stream);
    return wide ? launch_paged_t<T, 128, 2>(p, ctas, stream) : launch_paged_t<T, 128, 1>(p, ctas, stream);
}

int launch_paged_attn(const PagedAttnParams &p, int dtype, int ctas, void *stream_) {
    cudaStream_t stream = (cudaStream_t)stream_;
    switch (dtype) {
        case 0: return launch_paged_d<float>(p, ctas, stream);
        case 1: return launch_paged_d<__half>(p, ctas, stream);
        case 2: return launch_paged_d<__nv_bfloat16>(p, ctas, stream);
    }
    return -1;
}

}  // namespace q4
