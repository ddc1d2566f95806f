// attn_paged.cu -- attention of one new token per sequence over a paged KV
// cache (honeycrisp/mod.rs: gpu_attention and the fused RoPE + KV-append +
// SDPA dispatch of forward_decode_fused_layers, for a batch of sequences):
// RoPE of q and the new k, append of k and v at the sequence's position, then
// out_h = sum_t p_t v_t, p = softmax over the attended t of scale q_h . k_t.
//
// The work is HBM-bound on the cache rows, whatever the cache's type: a kv
// head's G query heads share each row, so the arithmetic runs on the tensor
// cores (mma.sync m16n8k16: the 8 columns are the group's heads; a wider
// instruction would leave most of its rows empty) and costs a fraction of the
// row's load time.  Each of a CTA's four warps brings its own tiles of 16
// positions by TMA into a ring of its own and waits for nobody else:
//   S^T [16 positions][heads] = K Q^T   A = K rows (16-bit: ldmatrix of swizzled
//        rows; fp32: 16 bytes of a row per lane, the k order inside a 32-dim
//        block permuted, and Q's fragments with it),
//   O^T [dims][heads] += V^T P^T        A = V rows (16-bit: transposing ldmatrix;
//        fp32: pairs of positions packed, rows of the m tiles permuted so that a
//        lane's 32 bytes of a V row are rows of its own tiles); P goes through
//        movmatrix.
// 64 ragged bf16 contexts up to 8191 (1.03 GB): 174 us, 5.9 TB/s; one of 32768
// (134 MB): 31 us, 4.3 TB/s, whether from HBM or partly from L2, of which about 5 us
// are the scan, Q, the warps' merge and the joining of the CTAs' shares.
//
// Precision: q and p stay fp32-like.  f16 caches: q (scaled per head by a
// power of two) and p enter as two f16 parts (22 bits); bf16 caches: as three
// bf16 parts (24 bits); f32 caches: K and V as three bf16 parts too, with the
// six products of order >= 2^-16.  The cache's values themselves are exact.  Outputs
// that are not finite are taken again by the definition (paged_again).
//
// Split: the units (64 or 128 positions) of all (sequence, kv head) pairs form
// one line that the CTAs (two an SM) divide evenly, whatever the lengths; lengths are read on
// the device, so a captured launch follows them.  A pair cut by a boundary is
// joined by the last of its CTAs to finish, in CTA order: the result does not
// depend on scheduling.
#include <algorithm>

#include "attn_row.cuh"
#include "gemv_launch.cuh"
#include "tensor_map.h"

namespace q4 {
namespace dev {

constexpr int kPagedWarps = 4;
constexpr int kPagedThreads = 32 * kPagedWarps;
constexpr int kPagedBatch = 8;  // shares a joining thread has in flight
constexpr int kPagedOcc = 2;  // CTAs of an SM: eight warps with up to 255 registers each

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

// Four 8 x 8 matrices of 16-bit values from shared memory (lane l gives a row's
// address), as A fragments; and transposed.
__device__ __forceinline__ void ldsm4(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ float f_of(const uint4 &v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
}

// A warp's step and its ring.  A step takes MT tiles of 16 positions (two share
// each Q fragment; one where two would leave no room to look ahead), so a unit
// of the split is 64 MT positions.  A ring item is the K, or the V, of one step;
// the rings hold about 190 KB of an SM.
template <typename T, int D>
struct PagedCfg {
    static constexpr int Tile = 16 * D * (int)sizeof(T);
    static constexpr int MT = Tile <= 4096 ? 2 : 1;
    static constexpr int Step = 16 * MT, Unit = Step * kPagedWarps;
    static constexpr int Item = MT * Tile;
    static constexpr int NI = 24 * 1024 / Item;
    static_assert(NI >= 3, "two items in flight while one is read");
};

// Shared memory of a CTA: the prefix of units over the sequences (per kv head)
// and their positions, Q's fragments (more than 8 heads: else they live in
// registers after their preparation) and factors, the warps' maxima and sums, a
// flag, then the rings; over them, when a segment's loop is done, the warps'
// outputs [warps][G][D], or the joining's.
template <typename T, int D, int NT>
struct PagedSmem {
    static constexpr int Prefix = 0;
    static constexpr int Pos = Prefix + 4 * (kMaxSeqs + 4);
    static constexpr int Qf = Pos + 4 * kMaxSeqs;
    static constexpr int Qs = Qf + PagedT<T>::QP * NT * (D / 16) * 32 * 8;
    static constexpr int Wm = Qs + 4 * 8 * NT;
    static constexpr int Wl = Wm + 4 * kPagedWarps * 8 * NT;
    static constexpr int Flag = Wl + 4 * kPagedWarps * 8 * NT;
    static constexpr int New = (Flag + 16 + 15) / 16 * 16;    // the new k and v in the cache's type [2][D]
    static constexpr int Bars = New + 2 * D * (int)sizeof(T);
    static constexpr int Red = (Bars + 8 * kPagedWarps * PagedCfg<T, D>::NI + 1023) / 1024 * 1024;
};

// A partial result: G outputs of D, G maxima, G sums, in whole 16 bytes.
Q4_HD constexpr size_t paged_slot_floats(int G, int D) { return ((size_t)G * (D + 2) + 3) / 4 * 4; }

// The heads of (sequence b, kv head hk) whose outputs are not finite, again by the
// definition, by the whole CTA: a product's parts (of p, and of fp32 values) can be
// zero or negative, so an attended infinity comes out as NaN.  The outputs, and the new
// token's row of the pages, are visible to this CTA.  room: kPagedWarps (D + 3) floats.
template <typename T, int D>
__device__ __noinline__ void paged_again(const PagedAttnParams &p, int b, int hk, int pos, float *room) {
    constexpr int DL = D / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.H / p.kv.hkv;
    const int lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    float *stat = room + kPagedWarps * D;  // per warp: maximum, sum, whether a position had a page
    for (int h = 0; h < G; ++h) {
        const size_t at = ((size_t)b * p.H + hk * G + h) * D;
        bool bad = false;
        for (int d = tid; d < D; d += kPagedThreads) bad = bad || !(fabsf(p.out[at + d]) < INFINITY);
        if (!__syncthreads_or(bad)) continue;  // (and the room is free again)
        float q[DL];
#pragma unroll
        for (int i = 0; i < DL; ++i) q[i] = p.q[at + lane + 32 * i];
#pragma unroll
        for (int i = 0; i < DL / 2; ++i) {
            const float x = q[i], y = q[i + DL / 2];
            const float c = p.rope_cos ? p.rope_cos[(size_t)pos * (D / 2) + lane + 32 * i] : 1.f;
            const float s = p.rope_cos ? p.rope_sin[(size_t)pos * (D / 2) + lane + 32 * i] : 0.f;
            if (p.rope_cos) {
                q[i] = x * c - y * s;
                q[i + DL / 2] = y * c + x * s;
            }
        }
#pragma unroll
        for (int i = 0; i < DL; ++i) q[i] *= p.scale * 1.4426950408889634f;
        RowSum<D> a;
        for (int k0 = lo + 32 * warp; k0 <= pos && !all_nan(a); k0 += 32 * kPagedWarps)
            attn_span<T, D>(a, p.kv, q, b, hk, k0, pos, lane, p.err);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a.l += __shfl_xor_sync(0xffffffffu, a.l, o);
#pragma unroll
        for (int i = 0; i < DL; ++i) room[warp * D + lane + 32 * i] = a.acc[i];
        if (lane == 0) {
            stat[3 * warp] = a.m;
            stat[3 * warp + 1] = a.l;
            stat[3 * warp + 2] = a.seen ? 1.f : 0.f;
        }
        __syncthreads();
        for (int d = tid; d < D; d += kPagedThreads) {
            float M = -INFINITY, o = 0.f, L = 0.f, seen = 0.f;
            for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, stat[3 * w]);
            const float mu = M == -INFINITY ? 0.f : M;
            for (int w = 0; w < kPagedWarps; ++w) {
                const float f = ex2(stat[3 * w] - mu);
                if (stat[3 * w + 2] == 0.f) continue;
                o = fmaf(room[w * D + d], f, o);
                L = fmaf(stat[3 * w + 1], f, L);
                seen = 1.f;
            }
            p.out[at + d] = seen == 0.f ? 0.f : o / L;
        }
    }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kPagedThreads, kPagedOcc)
    q4attn_paged_kernel(const __grid_constant__ PagedAttnParams p, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv) {
    using C = PagedT<T>;
    using M = typename C::M;
    using S = PagedSmem<T, D, NT>;
    using Cfg = PagedCfg<T, D>;
    constexpr int KP = C::KP, QP = C::QP, NW = kPagedWarps, KS = D / 16, VB = D / 64;
    constexpr bool H16 = sizeof(T) == 2;
    constexpr int MT = Cfg::MT, Step = Cfg::Step, NI = Cfg::NI, Item = Cfg::Item, Tile = Cfg::Tile;
    constexpr bool QReg = NT == 1;
    extern __shared__ __align__(1024) uint8_t psm[];  // the swizzle's pattern repeats every 1024 bytes
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int hkv = p.kv.hkv, G = p.H / hkv, nseq = p.kv.nseq;
    int *prefix = reinterpret_cast<int *>(psm + S::Prefix), *pos_s = reinterpret_cast<int *>(psm + S::Pos);
    uint2 *qf = reinterpret_cast<uint2 *>(psm + S::Qf);
    float *qs = reinterpret_cast<float *>(psm + S::Qs);
    float *wm = reinterpret_cast<float *>(psm + S::Wm), *wl = reinterpret_cast<float *>(psm + S::Wl);
    int *flag = reinterpret_cast<int *>(psm + S::Flag);
    float *red = reinterpret_cast<float *>(psm + S::Red);
    T *fresh = reinterpret_cast<T *>(psm + S::New);
    const uint32_t bars = smem_u32(psm + S::Bars) + 8 * NI * warp;
    const uint32_t ring = smem_u32(red) + (uint32_t)(warp * NI * Item);
    uint8_t *ring_p = reinterpret_cast<uint8_t *>(red) + warp * NI * Item;
    if (lane == 0) {
        for (int i = 0; i < NI; ++i) mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const long long cap = (long long)p.kv.width * p.kv.page;
    auto lo_of = [&](int pos) { return p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0; };
    // units of one kv head of sequence b: 0 for an idle row (or a position
    // the cache or the RoPE tables do not have)
    auto units_of = [&](int pos) -> int {
        if (pos < 0 || pos >= cap || (p.rope_cos && pos >= p.rope_rows)) return 0;
        const int lo = lo_of(pos) & ~15;
        return (pos - lo) / Cfg::Unit + 1;
    };
    // prefix[b] = units of a kv head of the sequences before b (the host bounds
    // the sum over all heads to 31 bits).  Up to 32 sequences: every warp scans
    // them for itself and writes the same words, no barrier; else a thread each.
    int Wh = 0;
    if (nseq <= 32) {
        const int pos = lane < nseq ? p.positions[lane] : -1, n = units_of(pos);
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        Wh = __shfl_sync(0xffffffffu, inc, 31);
        if (lane < nseq) {
            prefix[lane] = inc - n;
            pos_s[lane] = pos;
        }
        if (lane == 0) prefix[nseq] = Wh;
        __syncwarp();
    }
    for (int b0 = 0; nseq > 32 && b0 < nseq; b0 += kPagedThreads) {
        const int b = b0 + tid;
        const int pos = b < nseq ? p.positions[b] : -1;
        int inc = units_of(pos);
        const int n = inc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        int *wsum = reinterpret_cast<int *>(red) + ((b0 / kPagedThreads) & 1) * NW;
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int before = Wh;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += wsum[w];
            Wh += wsum[w];
        }
        if (b < nseq) {
            prefix[b] = before + inc - n;
            pos_s[b] = pos;
        }
    }
    if (nseq > 32) {
        if (tid == 0) prefix[nseq] = Wh;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the scan's room is the rings'
        __syncthreads();
    }
    // idle rows: zeros
    for (int b = blockIdx.x; b < nseq; b += gridDim.x)
        if (prefix[b + 1] == prefix[b]) {
            for (int i = tid; i < p.H * D; i += kPagedThreads) p.out[(size_t)b * p.H * D + i] = 0.f;
            if (tid == 0 && pos_s[b] >= 0) atomicExch(p.err, kErrPaged);
        }
    // CTAs with work: never more than units, so that none of a pair's CTAs is
    // without a share (each adds to the pair's count)
    const int W = Wh * hkv, N = min(W, (int)gridDim.x), cta = blockIdx.x;
    if (cta >= N) return;
    // CTA c's units start at floor(W c / N), the larger shares spread over the
    // CTAs (all in front, the SMs that get two of them end last: 34 -> 38 us for
    // one context of 32768)
    const int each = W / N, more = W - each * N;
    // (more c < 2^17 is exact in fp32, and the quotient's estimate off by one at most)
    const float per_n = 1.f / (float)N, per_w = (float)N / (float)W;
    auto start_of = [&](int c) {
        const int x = more * c, q = (int)((float)x * per_n), r = x - q * N;
        return each * c + q + (r >= N) - (r < 0);
    };
    auto cta_of = [&](int u) {  // the CTA of unit u: an estimate, then the exact one
        int c = min(N - 1, (int)((float)u * per_w));
        while (start_of(c) > u) --c;
        while (start_of(c + 1) <= u) ++c;
        return c;
    };
    const int u0 = start_of(cta), u1 = start_of(cta + 1);
    int b = 0;
    {  // the last b with prefix[b] <= u0 that has units
        int hi = nseq;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (prefix[mid] * hkv <= u0)
                b = mid;
            else
                hi = mid;
        }
    }
    const float qscale = p.scale * 1.4426950408889634f;
    const size_t slot_floats = paged_slot_floats(G, D);
    // the ring's state, carried over the segments: the slot (and its phase) of
    // the next item to issue and to read
    int fill_slot = 0, slot = 0;
    uint32_t phase = 0;
    int out = 0;                     // items in flight
    bool ok = true;                  // no wait of this warp gave up
    const uint64_t pol = evict_first_policy();
    uint32_t extra = p.extra_tx;     // testing the give-up path only

    for (int u = u0; u < u1;) {
        while (prefix[b + 1] * hkv <= u) ++b;
        const int pos = pos_s[b], lo = lo_of(pos), base16 = lo & ~15;
        const int cs = units_of(pos);
        const int sb = prefix[b] * hkv, hk = (u - sb) / cs, st = u - sb - hk * cs;
        const int s0 = sb + hk * cs, s1 = s0 + cs;  // the pair's units
        const int ue = min(s1, u1);
        const int n_units = ue - u;
        const bool owner = ue == s1;  // this segment ends with the new token

        // Q's heads (warp, warp + NW, ..; lane j < D / 8 holds dims 4 j .. and D / 2 +
        // 4 j ..) and the position's rotation, loaded before the copies go out
        constexpr int HW = 8 * NT / NW;
        const bool ql = lane < D / 8;
        float4 qa[HW], qb[HW], cr = make_float4(1.f, 1.f, 1.f, 1.f), sr = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < HW; ++x) {
            const int h = warp + NW * x;
            qa[x] = qb[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (h < G && ql) {
                const float *src = p.q + ((size_t)b * p.H + hk * G + h) * D + 4 * lane;
                qa[x] = *reinterpret_cast<const float4 *>(src);
                qb[x] = *reinterpret_cast<const float4 *>(src + D / 2);
            }
        }
        if (p.rope_cos && ql) {
            cr = *reinterpret_cast<const float4 *>(p.rope_cos + (size_t)pos * (D / 2) + 4 * lane);
            sr = *reinterpret_cast<const float4 *>(p.rope_sin + (size_t)pos * (D / 2) + 4 * lane);
        }
        float4 na = make_float4(0.f, 0.f, 0.f, 0.f), nb = na;  // warp 0: the new k, warp 1: the new v
        if (owner && warp < 2 && ql) {
            const float *src = (warp == 0 ? p.k_new : p.v_new) + ((size_t)b * hkv + hk) * D + 4 * lane;
            na = *reinterpret_cast<const float4 *>(src);
            nb = *reinterpret_cast<const float4 *>(src + D / 2);
        }

        // this warp's steps: first + warp, first + warp + NW, .. below last.  Their
        // K and V tiles come through the warp's own ring in shared memory by TMA
        // (16-bit: 16 rows x 64 values a box, swizzled; fp32: whole rows), each
        // slot on its mbarrier: item 2 i is the K of its i-th step, 2 i + 1 the V.
        // (16-byte copies by the lanes themselves measured the same 4.5 TB/s as
        // loads into registers: the load path, not the room, was full.)
        const int new_step = (pos - base16) / Step;  // the step of the new token, the last of all
        const int first = st * NW + warp, last = min((st + n_units) * NW, new_step + 1);
        const int count = first < last ? (last - first + NW - 1) / NW : 0;
        int fill_n = 0;                    // items issued
        uint32_t bad = 0;                  // bit (i MT + m) % 32: that tile's page is out of range
        int page_next[MT], page[MT], slot0[MT];  // table entries of the next step to issue, loaded ahead; this one's
        auto pages_of = [&](int i) {       // load the i-th step's
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int key = base16 + Step * (first + NW * i) + 16 * m;
                page_next[m] = i < count && key <= pos ? page_raw(p.kv, b, page_col(p.kv, key)) : -1;
            }
        };
        auto issue = [&]() {
            const int i = fill_n >> 1;
            if (i >= count || !ok) return;
            const int key0 = base16 + Step * (first + NW * i);
            if ((fill_n & 1) == 0) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int key = key0 + 16 * m;
                    const uint32_t bit = 1u << ((i * MT + m) & 31);
                    page[m] = page_ok(p.kv, page_next[m]);
                    slot0[m] = key - page_col(p.kv, key) * p.kv.page;
                    bad = page[m] < 0 ? bad | bit : bad & ~bit;
                    if (page[m] < 0 && key <= pos && lane == 0) atomicExch(p.err, kErrPaged);
                }
                pages_of(i + 1);
            }
            const bool isv = (fill_n & 1) != 0;
            const uint32_t dst = ring + (uint32_t)(fill_slot * Item), bar = bars + 8 * fill_slot;
            __syncwarp();  // every lane has read what the slot held
            if constexpr (H16) {
                if (lane == 0) mbar_expect_tx(bar, Item + extra);
                __syncwarp();
                if (lane < MT * VB) {  // box: tile m, 64-value block; a page out of range is copied as zeros
                    const int m = lane / VB, blk = lane - m * VB;
                    int pg = page[0], sl = slot0[0];
#pragma unroll
                    for (int x = 1; x < MT; ++x)
                        if (m == x) {
                            pg = page[x];
                            sl = slot0[x];
                        }
                    tma_page(dst + m * Tile + blk * 2048, isv ? &mv : &mk, 64 * blk, sl, hk, pg, bar);
                }
            } else if (lane == 0) {  // the attended rows of each tile
                uint32_t bytes = 0;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int key = key0 + 16 * m, r0 = max(lo - key, 0), r1 = page[m] < 0 ? 0 : min(pos - key + 1, 16);
                    if (r1 > r0) bytes += (uint32_t)(r1 - r0) * D * 4;
                }
                mbar_expect_tx(bar, bytes + extra);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int key = key0 + 16 * m, r0 = max(lo - key, 0), r1 = page[m] < 0 ? 0 : min(pos - key + 1, 16);
                    if (r1 > r0)
                        bulk_g2s(dst + m * Tile + r0 * D * 4,
                                 (const T *)(isv ? p.kv.v : p.kv.k) + row_off(p.kv, page[m], hk, slot0[m] + r0, D),
                                 (uint32_t)(r1 - r0) * D * 4, bar, pol);
                }
            }
            extra = 0;
            ++out;
            ++fill_n;
            fill_slot = fill_slot + 1 == NI ? 0 : fill_slot + 1;
        };
        // the next item has landed (false: a wait gave up)
        auto landed = [&]() {
            if (ok && !__all_sync(0xffffffffu, mbar_wait(bars + 8 * slot, phase, p.wait_cycles))) {
                ok = false;
                if (lane == 0) atomicExch(p.err, 7);
            }
            return ok;
        };
        auto advance = [&]() {
            --out;
            if (++slot == NI) {
                slot = 0;
                phase ^= 1;
            }
        };
        // byte offset of 16 bytes of a tile row (dims 16 / size x ..)
        auto at_of = [&](int m, int r, int x) {
            if constexpr (H16) return m * Tile + (x >> 3) * 2048 + r * 128 + (((x & 7) ^ (r & 7)) << 4);
            return m * Tile + r * D * 4 + x * 16;
        };
        // a step at an end of the range: the new token's row (its copy may have
        // come before the append), zeros in V's rows that are not attended
        auto mend = [&](int i, bool isv) {
            const int key0 = base16 + Step * (first + NW * i);
            constexpr int XR = D * (int)sizeof(T) / 16;  // 16-byte parts of a row
            uint8_t *it = ring_p + slot * Item;
            for (int y = lane; y < Step * XR; y += 32) {
                const int r = y / XR, x = y - r * XR, key = key0 + r, m = r >> 4;
                uint4 *dst = reinterpret_cast<uint4 *>(it + at_of(m, r & 15, x));
                const bool none = (bad >> ((i * MT + m) & 31)) & 1u;
                if (key == pos && !none)
                    *dst = *(reinterpret_cast<const uint4 *>(fresh + (isv ? D : 0)) + x);
                else if (isv && (key < lo || key > pos || none))
                    *dst = make_uint4(0u, 0u, 0u, 0u);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the slot's next copy
            __syncwarp();
        };
        pages_of(0);
        // the first items now, under Q's preparation
        for (int i = 0; i < NI - 1; ++i) issue();

        // the group's query heads: rotated, scaled (log2 units), in parts, as
        // B fragments
#pragma unroll
        for (int y = 0; y < HW; ++y) {
            const int h = warp + NW * y;
            float4 a = qa[y], c = qb[y];
            if (p.rope_cos) rotate4(a, c, cr, sr);
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
            if (ql) {
                const int nt = h >> 3, gg = h & 7;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float4 v = half ? c : a;
                    const int d = 4 * lane + half * (D / 2);
                    uint32_t w0[QP], w1[QP];
                    split2<M, QP>(v.x * f, v.y * f, w0);
                    split2<M, QP>(v.z * f, v.w * f, w1);
                    if constexpr (H16) {
                        // k16 step d / 16: word (d % 16) / 8 of lanes t = (d % 8) / 2 and t + 1
                        const int ks = d >> 4, ln = gg * 4 + ((d & 7) >> 1), wd = (d >> 3) & 1;
#pragma unroll
                        for (int i = 0; i < QP; ++i) {
                            uint32_t *at = reinterpret_cast<uint32_t *>(qf + ((i * NT + nt) * KS + ks) * 32 + ln) + wd;
                            at[0] = w0[i];
                            at[2] = w1[i];
                        }
                    } else {
                        // fp32: a lane's 32 bytes of a row are its k pairs of two steps
                        const int kb = d >> 5, r = d & 31, ks = 2 * kb + ((r >> 2) & 1), ln = gg * 4 + (r >> 3);
#pragma unroll
                        for (int i = 0; i < QP; ++i) qf[((i * NT + nt) * KS + ks) * 32 + ln] = make_uint2(w0[i], w1[i]);
                    }
                }
            }
        }
        if (owner && warp < 2) {  // append: warp 0 the new k (rotated), warp 1 the new v
            const int col = page_col(p.kv, pos), page = page_at(p.kv, b, col);
            if (page < 0) {
                if (lane == 0) atomicExch(p.err, kErrPaged);
            } else if (ql) {
                float4 a = na, c = nb;
                if (warp == 0 && p.rope_cos) rotate4(a, c, cr, sr);
                T *dst = (T *)(warp == 0 ? p.kv.k : p.kv.v) + row_off(p.kv, page, hk, pos - col * p.kv.page, D) + 4 * lane;
                store4(dst, a);
                store4(dst + D / 2, c);
                store4(fresh + warp * D + 4 * lane, a);
                store4(fresh + warp * D + 4 * lane + D / 2, c);
            }
        }
        __syncthreads();  // Q's fragments, the new row

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
        uint2 qr[QReg ? QP * KS : 1];
        if constexpr (QReg)
#pragma unroll
            for (int x = 0; x < QP * KS; ++x) qr[x] = qf[x * 32 + lane];

        for (int i = 0; i < count; ++i) {
            const int key0 = base16 + Step * (first + NW * i);
            const bool whole_step = key0 >= lo && key0 + Step - 1 < pos && ((bad >> ((i * MT) & 31)) & ((1u << MT) - 1u)) == 0;
            if (!landed()) break;
            if (!whole_step) mend(i, false);
            // scores: rows g and g + 8 of tile mt, heads 2t and 2t + 1, a sum for the
            // products of each order (parts x of Q and y of K: x + y), so that the
            // accumulation's truncation meets the largest ones D / 16 times only
            float sc[MT][NT][QP][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < QP; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[mt][nt][x][e] = 0.f;
            const uint32_t kt = ring + slot * Item;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[MT][KP][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (H16) {
                        // matrices: rows 0-7 and 8-15, k 0-7 then 8-15
                        ldsm4(a[mt][0], kt + at_of(mt, lane & 15, 2 * ks + (lane >> 4)));
                    } else {
                        // the lane's k pairs of this step: four of its eight values of a 32-value block
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const uint4 v = lds128_at<0>(kt + at_of(mt, g + 8 * rr, 8 * (ks >> 1) + 2 * t + (ks & 1)));
                            uint32_t w0[KP], w1[KP];
                            split2<M, KP>(f_of(v, 0), f_of(v, 1), w0);
                            split2<M, KP>(f_of(v, 2), f_of(v, 3), w1);
#pragma unroll
                            for (int y = 0; y < KP; ++y) {
                                a[mt][y][rr] = w0[y];
                                a[mt][y][2 + rr] = w1[y];
                            }
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < QP; ++x) {
                        const int at = (x * NT + nt) * KS + ks;
                        const uint2 bq = QReg ? qr[QReg ? at : 0] : qf[at * 32 + lane];
#pragma unroll
                        for (int y = 0; y < KP; ++y)
                            if (x + y < QP)
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt) mma16816<M>(sc[mt][nt][x + y], a[mt][y], bq.x, bq.y);
                    }
            }
            advance();
            issue();  // into the slot of the item read before this one
            uint32_t pw[MT][NT][2][QP];  // P as B fragments: positions 2t.. and 2t + 8.., head g
            float alpha[NT][2];          // what the outputs so far are rescaled by
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = sc[mt][nt][QP - 1][e];
#pragma unroll
                        for (int y = QP - 2; y >= 0; --y) v += sc[mt][nt][y][e];
                        x[mt][e] = v * qi[nt][e & 1];
                    }
                if (!whole_step) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const bool none = (bad >> ((i * MT + mt) & 31)) & 1u;
                        const int key = key0 + 16 * mt;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int at = key + g + 8 * (e >> 1);
                            if (none || at < lo || at > pos) x[mt][e] = -INFINITY;
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mx = fmaxf(x[0][h], x[0][2 + h]);
#pragma unroll
                    for (int mt = 1; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(x[mt][h], x[mt][2 + h]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float mn = fmaxf(m[nt][h], mx);
                    const float mu = mn == -INFINITY ? 0.f : mn;  // nothing attended yet
                    alpha[nt][h] = ex2(m[nt][h] - mu);
                    m[nt][h] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        x[mt][h] = ex2(x[mt][h] - mu + C::PEXP);
                        x[mt][2 + h] = ex2(x[mt][2 + h] - mu + C::PEXP);
                        sum += x[mt][h] + x[mt][2 + h];
                    }
                    l[nt][h] = fmaf(l[nt][h], alpha[nt][h], sum);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t w0[QP], w1[QP];
                    split2<M, QP>(x[mt][0], x[mt][1], w0);
                    split2<M, QP>(x[mt][2], x[mt][3], w1);
#pragma unroll
                    for (int y = 0; y < QP; ++y) {
                        pw[mt][nt][0][y] = transpose8x8(w0[y]);
                        pw[mt][nt][1][y] = transpose8x8(w1[y]);
                    }
                }
            }
            if (!landed()) break;
            if (!whole_step) mend(i, true);
            const uint32_t vt = ring + slot * Item;
            // outputs: 16-bit, m tile j: dims 16 j + g and + 8; fp32, m tile 4 vb + j:
            // dims 64 vb + 8 g + j and + 4 (a lane's 32 bytes of a V row are rows of its own tiles)
            // Each step's products are summed by themselves and added to the outputs
            // in fp32: the tensor core's own accumulation truncates, and over a long
            // context that bias would show (2e-6 after 1000 positions a warp).
            if constexpr (H16) {
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    float d[NT][4] = {};
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        // matrices: dims 0-7 and 8-15 of positions 0-7, then of 8-15
                        ldsm4t(a, vt + at_of(mt, (lane & 7) + 8 * (lane >> 4), 2 * j + ((lane >> 3) & 1)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = QP - 1; x >= 0; --x) mma16816<M>(d[nt], a, pw[mt][nt][0][x], pw[mt][nt][1][x]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[nt][j][e] = fmaf(acc[nt][j][e], alpha[nt][e & 1], d[nt][e]);
                }
            } else {
#pragma unroll
                for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint4 vr[4][2];
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                vr[kk][x] = lds128_at<0>(vt + at_of(mt, 2 * t + (kk & 1) + 8 * (kk >> 1), 16 * vb + 2 * g + x));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t a[KP][4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {  // e & 1: + 4 dims; e >> 1: + 8 positions
                                uint32_t w[KP];
                                split2<M, KP>(f_of(vr[2 * (e >> 1)][e & 1], j), f_of(vr[2 * (e >> 1) + 1][e & 1], j), w);
#pragma unroll
                                for (int y = 0; y < KP; ++y) a[y][e] = w[y];
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float d[4] = {};
#pragma unroll
                                for (int s = QP - 1; s >= 0; --s)  // the smallest products first
#pragma unroll
                                    for (int x = 0; x <= s; ++x) mma16816<M>(d, a[s - x], pw[mt][nt][0][x], pw[mt][nt][1][x]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[nt][4 * vb + j][e] = fmaf(acc[nt][4 * vb + j][e], mt == 0 ? alpha[nt][e & 1] : 1.f, d[e]);
                            }
                        }
                    }
            }
            advance();
            issue();
        }
        // a wait gave up: what is in flight lands before the room is used again
        for (; out > 0; --out) {
            mbar_wait(bars + 8 * slot, phase, kWaitCycles);
            if (++slot == NI) {
                slot = 0;
                phase ^= 1;
            }
        }
        __syncthreads();  // the rings are done: their room holds the merge

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
                    float *dst = red + ((size_t)warp * G + h) * D;
                    if constexpr (H16) {
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            dst[16 * j + g] = acc[nt][j][i];
                            dst[16 * j + 8 + g] = acc[nt][j][2 + i];
                        }
                    } else {
#pragma unroll
                        for (int vb = 0; vb < VB; ++vb) {
                            *reinterpret_cast<float4 *>(dst + 64 * vb + 8 * g) =
                                make_float4(acc[nt][4 * vb][i], acc[nt][4 * vb + 1][i], acc[nt][4 * vb + 2][i],
                                            acc[nt][4 * vb + 3][i]);
                            *reinterpret_cast<float4 *>(dst + 64 * vb + 8 * g + 4) =
                                make_float4(acc[nt][4 * vb][2 + i], acc[nt][4 * vb + 1][2 + i], acc[nt][4 * vb + 2][2 + i],
                                            acc[nt][4 * vb + 3][2 + i]);
                        }
                    }
                }
            }
        __syncthreads();
        const bool whole = u == s0 && ue == s1;
        // an output that is not finite (or without a weight: 0 / 0 here) is looked at again
        bool again = false;
        auto result = [&](float o, float L) {
            const float x = o / L;
            again = again || !(fabsf(x) < INFINITY);
            return x;
        };
        float *mine = p.part + ((size_t)cta * 2 + (u == u0 ? 0 : 1)) * slot_floats;
        for (int idx = tid; idx < G * D; idx += kPagedThreads) {
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
                p.out[((size_t)b * p.H + hk * G) * D + idx] = result(o, L);
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
            const int c0 = cta_of(s0), nc = cta_of(s1 - 1) - c0 + 1;  // first CTA, CTAs
            __syncthreads();
            if (tid == 0) {  // the CTA's share (the barrier orders it before), then the count; the others' after it
                int before;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                             : "=r"(before)
                             : "l"(p.count + (size_t)b * hkv + hk)
                             : "memory");
                *flag = before == nc - 1;
            }
            __syncthreads();
            if (*flag) {
                // CTA c0 + i's slot: its first segment, except a first CTA whose
                // range starts before the pair
                const float *part0 = p.part + ((size_t)c0 * 2 + (start_of(c0) != s0 ? 1 : 0)) * slot_floats;
                const float *part1 = p.part + (size_t)c0 * 2 * slot_floats;
                auto slot_of = [&](int i) { return i == 0 ? part0 : part1 + (size_t)i * 2 * slot_floats; };
                // A thread a float4 of the outputs (with threads to spare, groups of them
                // that take every NG-th share): eight shares at once, so that their latencies
                // overlap, joined like the softmax's own steps.  (A warp's lanes
                // on 128 outputs, one pass for the weights and another for the sums, took
                // the last CTA of 38 9 us.)
                const int T4 = G * D / 4, NG = T4 < kPagedThreads ? kPagedThreads / T4 : 1;
                const int grp = NG > 1 ? tid / T4 : 0;
                float *dst = p.out + ((size_t)b * p.H + hk * G) * D;
                for (int e = tid - grp * T4; grp < NG && e < T4; e += kPagedThreads) {
                    const int idx = 4 * e, h = idx / D;
                    float Mx = -INFINITY, L = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i0 = grp; i0 < nc; i0 += NG * kPagedBatch) {
                        float4 v[kPagedBatch];
                        float mi[kPagedBatch], li[kPagedBatch];
#pragma unroll
                        for (int y = 0; y < kPagedBatch; ++y) {
                            const int i = i0 + NG * y;
                            mi[y] = -INFINITY;
                            li[y] = 0.f;
                            v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (i < nc) {
                                const float *sl = slot_of(i);
                                v[y] = __ldcg(reinterpret_cast<const float4 *>(sl + idx));
                                mi[y] = __ldcg(sl + G * D + h);
                                li[y] = __ldcg(sl + G * D + G + h);
                            }
                        }
                        float mn = Mx;
#pragma unroll
                        for (int y = 0; y < kPagedBatch; ++y) mn = fmaxf(mn, mi[y]);
                        const float mu = mn == -INFINITY ? 0.f : mn, a = ex2(Mx - mu);
                        o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
                        L *= a;
#pragma unroll
                        for (int y = 0; y < kPagedBatch; ++y) {
                            const float f = ex2(mi[y] - mu);
                            o = make_float4(fmaf(v[y].x, f, o.x), fmaf(v[y].y, f, o.y), fmaf(v[y].z, f, o.z),
                                            fmaf(v[y].w, f, o.w));
                            L = fmaf(li[y], f, L);
                        }
                        Mx = mn;
                    }
                    if (NG == 1) {
                        const float r = 1.f / L;
                        const float4 x = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
                        again = again || !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY &&
                                           fabsf(x.w) < INFINITY);
                        *reinterpret_cast<float4 *>(dst + idx) = x;
                    } else {
                        *reinterpret_cast<float4 *>(red + (size_t)grp * G * D + idx) = o;
                        if (idx == h * D) {
                            wm[grp * G + h] = Mx;
                            wl[grp * G + h] = L;
                        }
                    }
                }
                if (NG > 1) {
                    __syncthreads();
                    for (int idx = tid; idx < G * D; idx += kPagedThreads) {
                        const int h = idx / D;
                        float Mx = -INFINITY, o = 0.f, L = 0.f;
                        for (int y = 0; y < NG; ++y) Mx = fmaxf(Mx, wm[y * G + h]);
                        const float mu = Mx == -INFINITY ? 0.f : Mx;
                        for (int y = 0; y < NG; ++y) {
                            const float f = ex2(wm[y * G + h] - mu);
                            o = fmaf(red[(size_t)y * G * D + idx], f, o);
                            L = fmaf(wl[y * G + h], f, L);
                        }
                        dst[idx] = result(o, L);
                    }
                }
                if (tid == 0) p.count[(size_t)b * hkv + hk] = 0;  // zero again for the next call
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the merge's writes, before the next copies
        if (__syncthreads_or(again)) {  // the shared memory is free for the next segment
            paged_again<T, D>(p, b, hk, pos, red);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
        }
        u = ue;
    }
}

}  // namespace dev

// above 8 heads a kv head Q's fragments leave room for one CTA of an SM
int paged_attn_ctas(int G, int sms) { return (G > 8 ? 1 : dev::kPagedOcc) * sms; }
size_t paged_attn_slot_floats(int D, int G) { return dev::paged_slot_floats(G, D); }

template <typename T, int D, int NT>
static int launch_paged_t(const PagedAttnParams &p, int ctas, cudaStream_t stream) {
    auto kern = dev::q4attn_paged_kernel<T, D, NT>;
    static size_t smem_set[64] = {0};
    const int G = p.H / p.kv.hkv;
    using Cfg = dev::PagedCfg<T, D>;
    // the rings; over them the merge (or the joining, of 512 floats at most)
    const size_t merge = sizeof(float) * std::max(G * dev::kPagedWarps * D, 512);
    const size_t smem = dev::PagedSmem<T, D, NT>::Red + std::max(merge, (size_t)dev::kPagedWarps * Cfg::NI * Cfg::Item);
    if (!raise_smem(kern, smem, smem_set)) return -1;
    CUtensorMap mk{}, mv{};
    if (sizeof(T) == 2) {
        const bool bf = std::is_same<T, __nv_bfloat16>::value;
        const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.kv.page, (cuuint64_t)p.kv.hkv, (cuuint64_t)p.kv.num_pages};
        const cuuint32_t box[4] = {64, 16, 1, 1};
        if (!make_map(&mk, bf, p.kv.k, 4, dims, box) || !make_map(&mv, bf, p.kv.v, 4, dims, box)) return -1;
    }
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)ctas, dev::kPagedThreads, smem, stream, &attr);
    return cudaLaunchKernelEx(&cfg, kern, p, mk, mv) == cudaSuccess ? 0 : -1;
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
