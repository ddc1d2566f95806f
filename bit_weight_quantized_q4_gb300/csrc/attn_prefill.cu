// attn_prefill.cu -- causal attention of packed prompt rows over the pages of
// their sequences (honeycrisp/mod.rs, gpu_attention, for a prompt).
//
// A CTA (q4attn_prefill_tc_kernel) takes up to NT tiles of up to 128 rows of one
// kv head's group -- floor(128 / G) consecutive tokens by G query heads, so the
// group shares every K and V tile -- and walks the key tiles of KT positions with
// a running softmax:
//   S = Q K^T          tcgen05.mma, 128 x KT fp32 in tensor memory
//   P = 2^(c S - m)    64 columns a thread; P (16-bit) over S's columns, or in
//                      shared memory
//   O += P V           tcgen05.mma
// Q, K and V tiles come by tensor-map copies (TMA, 128-byte swizzle) straight
// from the packed rows and the pages; V is the MN-major operand, so nothing is
// transposed.  Up to sixteen softmax warps, two that issue MMAs, one that copies,
// one for rows taken by the definition (below).
// While some tiles' softmax runs, the tensor core works on the others'
// products: a tile's own chain (scores, weights, product) takes several times
// its tensor work.  16-bit at head size 64: four tiles, key tiles of 64 positions
// (4 x (S 64 + O 64) columns fill the tensor memory), a thread a row.  Else two
// tiles (one for fp32 at head size 128, whose parts fill the shared memory), key
// tiles of 128 positions, two warps a row that exchange its maximum.
// An MMA of 128 rows takes about 60 cycles per K = 16 at N = 64 as at N = 128
// (measured by its issue), so at head size 64 the product runs at half the
// tensor rate whatever the tiling: 8192 rows took 277 us with two tiles of 128
// positions, P beside S and S a key tile ahead, and 277 with four of 64 (249 now:
// 1100 TFLOP/s, the tensor core busy over 90 % of the loop).  At head size 128 (nine
// ragged prompts, 93 GFLOP: 86 us, 1080 TFLOP/s) a key tile of two row tiles takes 2900
// cycles, 1920 of them tensor work.  What takes the rest is not settled: over the
// launch the tensor pipe is busy 53 % of the active cycles, and of shared memory's
// wavefronts the tensor core's operands take 48 % and the warps' accesses 21 %, so
// no unit is full; the chain scores - weights - product and the ends of items are
// the likely cause.  (P over its S spares a third of the operands' traffic, but the
// next scores then wait for the product: 89 us.  The halves' maxima joined a key tile
// late, with bf16's exponents: 87; a warp a row: 89.)  fp32 (2048 rows: 76 us): three
// products each, of which 4300 cycles a key tile are tensor work, and about 14 us to
// write the operands' parts; the longest item has 16 key tiles.
// O is rescaled in tensor memory only when a row's maximum grew by more than 2^8
// (the sums stay exact: the reference maximum is the row's own, and its factor
// cancels).
//
// Masked positions: scores are replaced before the maximum; V rows behind the
// sequence's end are zeroed in shared memory.  A non-finite value at a position
// that some rows of a tile see and others do not would still enter as 0 * NaN:
// a row whose result is not finite is therefore taken again by the definition
// (attn_row), which never touches what it does not attend; and so is one whose weights
// are all zero.
#include <algorithm>
#include <limits>

#include "attn_row.cuh"
#include "gemv_launch.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace q4 {
namespace dev {

constexpr int kPfBlk = 128 * 128;           // bytes of 128 rows x 64 16-bit values (a block of a Q tile)
constexpr int kPfItems = 4;                 // work items of a CTA that are known and not done
constexpr float kPfUsual = 0.0078125f;      // the usual factor back of a position of K or V, 2^-7
constexpr float kPfGrow = 8.f;              // log2 growth of a maximum that rescales O

// What enters the products of a cache type: 16-bit values as they are (one
// part); fp32 values as two f16 parts hi + lo (22 bits) after a power-of-two
// scale, three products each (lo lo, of 2^-22, is left out).  The 16-bit types'
// weights are rounded to the type too: a second part for them would be another P V,
// half of the tensor work again, against an error of 1.3 times the output's own rounding.
//
// The scales of fp32: every row of Q and every position of K and of V has its own,
// so that no value's bits depend on another's size -- another sequence's, a later
// token's, or a stale one's.  A position's factors back (K's and V's, powers of two)
// multiply its column of S, and its weight: a row's scaled weights are brought to
// f16's range by one more power of two a key tile, found from their own largest, which
// goes into the sum beside O.  So does the reference of a key tile's weights, its own
// maximum: the row's so far would leave the weights of a later key tile few bits, which
// large values there would show.
// Factors of their own cost twice the time, so the scales of K and V are steps of 2^12:
// a key tile whose positions have the same ones takes them as one factor, and a call
// whose attended positions all have the usual one (rows whose largest value is in
// [2^-5, 2^7), or zeros) never looks at them (2048 rows: 76 us; 84 where a position of
// the call has another one, 165 where every key tile mixes them).  A row's bits are the
// same by each way.
template <typename T>
struct PfT {
    using M = T;
    static constexpr int Parts = 1;
    static constexpr float PExp = 0.f;
};
template <>
struct PfT<__half> {
    using M = __half;
    static constexpr int Parts = 1;
    static constexpr float PExp = 6.f;  // weights reach 2^(6 + kPfGrow), and stay normal down to 2^-20 of the largest
};
template <>
struct PfT<float> {
    using M = __half;
    static constexpr int Parts = 2;
    static constexpr float PExp = 13.f;  // weights reach 2^13 in each key tile: its own maximum is their reference
};

template <int D, int Parts>
struct PfCfg {
    static constexpr int KT = D == 64 && Parts == 1 ? 64 : 128;  // positions of a key tile
    // warps that share a row, CW columns each
    static constexpr int HF = KT / 64;
    static constexpr int CW = KT / HF;
    static constexpr int NT = KT == 64 ? 4 : D * Parts == 256 ? 1 : 2;  // row tiles of a CTA at most
    // softmax warps (row tiles x columns x 4 row quarters), two that issue MMAs, the
    // copy warp, the warp of the rows taken by the definition
    static constexpr int Soft = 4 * HF * NT, Mma = Soft, Copy = Soft + 2, Rows = Soft + 3, Threads = 32 * (Soft + 4);
    static constexpr int NB = D / 64;                  // 64-value blocks of a row
    static constexpr int KBlk = KT * 128;              // a block of a K or V tile
    static constexpr int Tile = NB * KBlk;             // one part of a K or V tile
    static constexpr int QPart = NB * kPfBlk, QTile = Parts * QPart;
    // P in shared memory (blocks like Q's) instead of over its S: S is free as soon as
    // it is in registers, and the next key tile's can be under way
    static constexpr bool PS = D == 128 && Parts == 1;
    // ring stages: per key tile K's parts, then V's (P in shared memory: K a tile ahead)
    static constexpr int NS = KT == 64 ? 12 : D == 64 ? 9 : PS ? 3 : 5;
    static constexpr int OffQ = 0, OffP = NT * QTile, PTile = PS ? (KT / 64) * kPfBlk : 0;
    static constexpr int OffRing = OffP + NT * PTile, OffBar = OffRing + NS * Tile;
    // tensor memory columns: S of tile i from KT i, O of tile i from ColO + D i; P
    // lies over its S (two parts: each column half's over its own, 16 columns of hi
    // and 16 of lo per 32 positions)
    static constexpr int ColO = NT * KT, ColSum = ColO + NT * D;
    static constexpr int OffX = OffBar + 608 + (20 + 4 * 16) * kPfItems;  // values the column halves exchange [tile][half][row]
    // fp32: the factors back of a key tile's positions (bf16, K's in the upper half),
    // and the one that all share, if so; of as many key tiles as the ring can be ahead of
    // the weights: the slot that a key tile's first copy waits for held V of the tile NF
    // before, whose weights are written
    static constexpr int NF = Parts == 2 ? (NS + 2 * Parts - 1) / (2 * Parts) : 0;
    static constexpr int OffF = OffX + (HF == 2 ? NT * 2 * 128 * 4 : 0);
    static constexpr int FacBytes = KT * 4 + 16;
    static constexpr int OffWide = OffF + NF * FacBytes;  // fp32: whether factors are looked at at all
    static constexpr int Smem = OffWide + (Parts == 2 ? 16 : 0);
    static_assert(Parts == 1 || (NS % (2 * Parts) == 1 && HF == 2), "NF; the weights' exchange");
    static_assert(Smem <= (int)kSmemMax, "prefill shared memory");
    static_assert(ColO + NT * D * Parts <= 512, "tensor memory");
    static_assert(Soft <= 16, "a barrier of the exchange for each pair of warps; masks");
    static_assert(16 * NS + 48 * NT + 24 * kPfItems + 88 + (PS ? 16 * NT : 0) + 8 * NF <= 576, "barriers before the tensor-memory address");
    // P's column of 16 positions (step ks), part 0
    static constexpr int p_col(int ks) {
        return Parts == 1 ? 8 * ks : 64 * (ks / 4) + 32 * ((ks % 4) / 2) + 8 * (ks % 2);
    }
};

__device__ __forceinline__ void pf_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void tma5(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w, int v,
                                     uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
        "[%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
        : "memory");
}

// Transposes 16-byte parts among eight lanes: lane l's part x becomes lane x's part l.
__device__ __forceinline__ void pf_transpose8(uint32_t (&w)[8][4], int lane) {
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) {
        const bool up = (lane & k) != 0;
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if ((x & k) == 0)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[x][e] : w[x | k][e], k);
                    if (up)
                        w[x][e] = got;
                    else
                        w[x | k][e] = got;
                }
    }
}

// A work item: sequence, its first token (row of the packed batch and position),
// its tokens, and the kv head.  Tiles of a sequence are numbered from its end: the
// longest first.
struct PfTile {
    int seq, row0, pos0, tokens, hk;
};
// Item number `item` of tiles of tpc tokens; called by one warp.  seq = -1 when
// there is no such item (nor one of a higher number).
__device__ __forceinline__ PfTile pf_find(const PrefillParams &p, int item, int tpc, int lane) {
    const int idx = item / p.kv.hkv;
    PfTile t = {-1, 0, 0, 0, item - idx * p.kv.hkv};
    long long before = 0;
    for (int b0 = 0; b0 < p.kv.nseq; b0 += 32) {
        const int b = b0 + lane;
        int begin = 0, rows = 0;
        if (b < p.kv.nseq) {
            begin = min(max(p.cu[b], 0), p.rows);
            rows = max(min(p.cu[b + 1], p.rows) - begin, 0);
        }
        const int first = b < p.kv.nseq && p.start ? p.start[b] : 0;
        const long long cap = (long long)p.kv.width * p.kv.page;
        if (rows > 0 && (first < 0 || (long long)first + rows > cap)) {
            atomicExch(p.err, kErrPaged);
            rows = first < 0 || first >= cap ? 0 : (int)(cap - first);
        }
        const int n = (rows + tpc - 1) / tpc;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > idx);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int nb = __shfl_sync(0xffffffffu, n, l);
            const int at = (int)(idx - (before + __shfl_sync(0xffffffffu, inc, l) - nb));  // 0: the last tile
            const int tok = (nb - 1 - at) * tpc;
            t.seq = b0 + l;
            t.row0 = __shfl_sync(0xffffffffu, begin, l) + tok;
            t.pos0 = __shfl_sync(0xffffffffu, first, l) + tok;
            t.tokens = min(tpc, __shfl_sync(0xffffffffu, rows, l) - tok);
            return t;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return t;
}

// Work items (a kv head's tiles of one CTA) are CTAs of the grid; a CTA that has
// one goes on with the next that has not been launched yet (it cancels that
// launch and takes its number), so the copies and first scores of an item run
// under the softmax and the epilogue of the one before it: a CTA an item took
// 11 us beside its key tiles (8192 rows: 272 us, nine ragged prompts: 117).
// Asks for the next item: the answer comes to `resp` (16 bytes) on `bar`.
__device__ __forceinline__ void pf_ask_next(uint32_t resp, uint32_t bar) {
    mbar_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(resp),
        "r"(bar)
        : "memory");
}
// The answer: a CTA's number, or -1 when there is none (and none may be asked for).
__device__ __forceinline__ int pf_next(uint32_t resp) {
    int x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tmov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=r"(x)
        : "r"(resp)
        : "memory");
    return x;
}

template <typename T, int D>
__global__ void __launch_bounds__(PfCfg<D, PfT<T>::Parts>::Threads, 1)
    q4attn_prefill_tc_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap mq,
                             const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                             const int box_rows, const int row_tiles, const bool more) {
    using M = typename PfT<T>::M;
    constexpr int NP = PfT<T>::Parts;
    using Cf = PfCfg<D, NP>;
    constexpr bool BF = std::is_same<M, __nv_bfloat16>::value;
    constexpr int NB = Cf::NB, NS = Cf::NS, NT = Cf::NT, KT = Cf::KT, HF = Cf::HF, CW = Cf::CW;
    extern __shared__ __align__(1024) uint8_t sm[];  // the swizzle's pattern repeats every 1024 bytes
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // barriers.  Of the ring: a stage's copies have landed, both MMA warps are
    // done with it.  Of row tile i: Q has landed, Q is free, a key tile's S is
    // complete, its P is written, O is complete, O is free (P in shared memory: S has
    // been read, P has been used).  Of the factors (fp32): a key tile's are written.  Of
    // the work items: slot's tile is known, every warp has read it, the answer to pf_ask_next.
    const uint32_t bars = sb + Cf::OffBar;
    const uint32_t b_full = bars, b_empty = b_full + 8 * NS, b_q = b_empty + 8 * NS, b_qe = b_q + 8 * NT,
                   b_s = b_qe + 8 * NT, b_p = b_s + 8 * NT, b_o = b_p + 8 * NT, b_oe = b_o + 8 * NT,
                   b_known = b_oe + 8 * NT, b_read = b_known + 8 * kPfItems, b_mask = b_read + 8 * kPfItems,
                   b_next = b_mask + 8 * kPfItems, b_drain = b_next + 8, b_x = b_drain + 16,
                   b_sr = b_x + 64, b_pe = b_sr + 8 * NT, b_f = b_sr + (Cf::PS ? 16 * NT : 0);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Cf::OffBar + 576);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Cf::OffBar + 580);
    volatile int *slow = reinterpret_cast<volatile int *>(sm + Cf::OffBar + 584);  // a row is being taken by the definition
    volatile int *progress = reinterpret_cast<volatile int *>(sm + Cf::OffBar + 588);  // key tiles copied
    const uint32_t resp = bars + 592;
    PfTile *tile_s = reinterpret_cast<PfTile *>(sm + Cf::OffBar + 608);  // [kPfItems]
    unsigned *mask_s = reinterpret_cast<unsigned *>(sm + Cf::OffBar + 608 + 20 * kPfItems);  // [kPfItems][Cf::Soft]: rows to take again
    const long long lim = p.wait_cycles;
    const int G = p.H / p.kv.hkv, TQ = 128 / G;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        auto init = [&](uint32_t bar, int n, uint32_t count) {  // n consecutive barriers, one a lane
            if (lane < n) mbar_init(bar + 8 * lane, count);
        };
        init(b_full, NS, 1);
        init(b_empty, NS, 2);  // one for each MMA warp
        init(b_q, 3 * NT, 1);  // Q, free Q, S
        init(b_p, NT, 4 * HF);
        init(b_o, NT, 1);
        init(b_oe, NT, 4 * HF);
        init(b_known, kPfItems, 1);
        init(b_read, kPfItems, Cf::Soft + 3);
        init(b_mask, kPfItems, Cf::Soft);
        init(b_next, 3, 1);  // and b_drain
        init(b_x, 8, 2);
        if constexpr (Cf::PS) {
            init(b_sr, NT, 4 * HF);
            init(b_pe, NT, 1);
        }
        if constexpr (NP == 2) init(b_f, Cf::NF, 1);
        if (lane == 0) {
            *abort_flag = 0;
            *slow = 0;
            *progress = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == Cf::Mma) {
        tc::tmem_alloc(smem_u32(tslot), 512);
        tc::tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == Cf::Copy) {
        const PfTile t = pf_find(p, (int)blockIdx.x, row_tiles * TQ, lane);
        if (lane == 0) tile_s[0] = t;
    }
    if (NP == 2 && warp == Cf::Rows) {  // a CTA of the staging met another factor than the usual one
        uint32_t met = 0u;
        for (int x = lane; x < p.nmet; x += 32) met |= __ldcg(p.met + x);
        met = __reduce_or_sync(0xffffffffu, met);
        if (lane == 0) *reinterpret_cast<uint32_t *>(sm + Cf::OffWide) = met;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t taddr = *tslot;
    bool wide = false;
    if constexpr (NP == 2) wide = *reinterpret_cast<const uint32_t *>(sm + Cf::OffWide) != 0u;
    if (tile_s[0].seq < 0) {  // no item of this number
        __syncthreads();
        if (warp == Cf::Mma) tc::tmem_dealloc(taddr, 512);
        return;
    }
    auto fail = [&]() {
        *abort_flag = 1;
        atomicExch(p.err, 6);
    };
    // A wait of a whole warp
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, lim)) != 0; };
    // one that ends too when another warp has given up (of the copies, so that none
    // follow; the others run dry and end by themselves)
    auto wait_go = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, lim) && *abort_flag == 0) != 0;
    };
    // and one that may last a whole item: it gives up when, for the limit, no copy
    // has gone out and no rows were being taken by the definition, nor had been since
    // (slow: odd while they are, so that the moment between two items' is seen)
    auto wait_item = [&](uint32_t bar, uint32_t parity) {
        int seen = __shfl_sync(0xffffffffu, *progress + *slow, 0);
        while (!wait(bar, parity)) {
            const int was = __shfl_sync(0xffffffffu, *slow, 0), now = __shfl_sync(0xffffffffu, *progress, 0) + was;
            if ((now == seen && (was & 1) == 0) || __any_sync(0xffffffffu, *abort_flag != 0)) return false;
            seen = now;
        }
        return true;
    };
    // key tiles of an item: the first position, how many, the last one's positions
    auto keys_of = [&](const PfTile &t, int &k_first, int &nk, int &tail) {
        const int key_end = t.pos0 + t.tokens;
        const int key_lo = p.window > 0 && t.pos0 + 1 > p.window ? t.pos0 + 1 - p.window : 0;
        k_first = key_lo & ~(KT - 1);
        nk = (key_end - k_first + KT - 1) / KT;
        tail = key_end - (k_first + (nk - 1) * KT);
        return key_lo;
    };
    // item n, as the copy warp published it (seq < 0: no more)
    auto tile_of = [&](int n, PfTile &t) {
        const bool ok = wait_item(b_known + 8 * (n % kPfItems), (uint32_t)(n / kPfItems) & 1u);
        t = tile_s[n % kPfItems];
        return ok;
    };
    auto tile_read = [&](int n) {
        __syncwarp();
        if (lane == 0) pf_arrive(b_read + 8 * (n % kPfItems));
    };

    if (warp == Cf::Copy) {
        // ------------------------------------------------------------ copies
        // lane = 64-value block bl, box r of a tile (at most 16 boxes)
        const int boxes = KT / box_rows, bl = lane / boxes, r = lane - bl * boxes;
        bool ok = true, asked = false;  // asked: an answer is outstanding, in this phase
        uint32_t nph = 0;
        auto ask = [&]() {
            if (lane == 0) pf_ask_next(resp, b_next);
            asked = true;
        };
        auto answer = [&]() {  // the next item's number, -1: none
            if (!asked) return -1;
            ok = wait(b_next, nph);
            if (!ok) return -1;
            asked = false;
            nph ^= 1u;
            const int at = pf_next(resp);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next answer
            __syncwarp();
            return at;
        };
        int issued = 0, st = 0;  // ring tiles issued, the next one's stage
        int n_tile = 0;          // key tiles
        uint32_t ph = 1;         // an empty slot's phase: the first pass finds them free
        uint32_t qph = ~0u, q_out = 0;  // bit i: the phase of tile i's free Q; Q copies issued and perhaps in flight
        PfTile t = tile_s[0];
        if (lane == 0) pf_arrive(b_known);
        for (int n = 0; ok && t.seq >= 0; ++n) {
            int k_first, nk, tail;
            const int key_lo = keys_of(t, k_first, nk, tail), key_end = t.pos0 + t.tokens;
            const int nt = (t.tokens + TQ - 1) / TQ;
            PfTile next = {-1, 0, 0, 0, 0};
            // the next key tile's pages are looked up while this one's copies go out:
            // looked up in place they held the ring back (a tile every 1400 cycles)
            auto lookup = [&](int j, int &page, int &slot) {
                const int key = k_first + j * KT + r * box_rows, col = page_col(p.kv, key);
                slot = key - col * p.kv.page;
                page = bl < NB && key < key_end ? page_raw(p.kv, t.seq, col) : -1;
            };
            int page1, slot1, v_live = 0, v_page = -1, v_slot = 0;
            lookup(0, page1, slot1);
            // the factors of a key tile, four positions a lane (0 where nothing is attended)
            auto factors = [&](int j) {
                uint4 f = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (NP == 2) {
                    const int box = 4 * lane / box_rows, left = key_end - (k_first + j * KT + 4 * lane);
                    const int page = page_ok(p.kv, __shfl_sync(0xffffffffu, page1, box));
                    const int slot = __shfl_sync(0xffffffffu, slot1, box) + 4 * lane - box * box_rows;
                    if (page >= 0 && left > 0)
                        f = __ldcg(reinterpret_cast<const uint4 *>(
                            p.fac + ((size_t)page * p.kv.hkv + t.hk) * p.fac_stride + slot));
                    if (left < 4) f.w = 0u;
                    if (left < 3) f.z = 0u;
                    if (left < 2) f.y = 0u;
                }
                return f;
            };
            uint4 fac = make_uint4(0u, 0u, 0u, 0u);
            if (wide) fac = factors(0);
            for (int j = 0; ok && j < nk; ++j) {
                const int page = page_ok(p.kv, page1), slot = slot1;
                // a page out of range is copied as zeros (its coordinate is out of
                // the map's range); below the window it may be gone
                const int key = k_first + j * KT + r * box_rows;
                if (page < 0 && bl < NB && key < key_end && key + box_rows > key_lo) atomicExch(p.err, kErrPaged);
                const int live = min(boxes, (key_end - k_first - j * KT + box_rows - 1) / box_rows);  // boxes with attended positions
                if (j + 1 < nk) {
                    lookup(j + 1, page1, slot1);
                } else if (more) {  // no sooner, or the CTAs with the longest items would have all the others too
                    ask();
                }
                auto put = [&](int kv, int live, int page, int slot) {  // K's parts (kv < NP), V's parts
                    ok = ok && wait_go(b_empty + 8 * st, ph);
                    if (!ok) return;
                    if constexpr (NP == 2)
                        if (wide && kv == 0) {
                            uint8_t *at = sm + Cf::OffF + (n_tile % Cf::NF) * Cf::FacBytes;
                            *reinterpret_cast<uint4 *>(at + 16 * lane) = fac;
                            // the largest and the smallest of each half (0, of a row of zeros, goes with any)
                            uint32_t k1 = 0u, k0 = 0xffffu, v1 = 0u, v0 = 0xffffu;
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint32_t k = w_of(fac, x) >> 16, v = w_of(fac, x) & 0xffffu;
                                k1 = max(k1, k);
                                v1 = max(v1, v);
                                k0 = min(k0, k ? k : 0xffffu);
                                v0 = min(v0, v ? v : 0xffffu);
                            }
                            k1 = __reduce_max_sync(0xffffffffu, k1);
                            v1 = __reduce_max_sync(0xffffffffu, v1);
                            k0 = __reduce_min_sync(0xffffffffu, k0);
                            v0 = __reduce_min_sync(0xffffffffu, v0);
                            if (lane == 0)
                                *reinterpret_cast<uint2 *>(at + 4 * KT) =
                                    make_uint2(k1 << 16 | v1, (k1 == k0 || k1 == 0u) && (v1 == v0 || v1 == 0u));
                            __syncwarp();
                            if (lane == 0) pf_arrive(b_f + 8 * (n_tile % Cf::NF));
                        }
                    if (lane == 0) mbar_expect_tx(b_full + 8 * st, (uint32_t)(live * box_rows) * 128u * NB);
                    __syncwarp();
                    if (bl < NB && r < live)
                        tma5(sb + Cf::OffRing + st * Cf::Tile + bl * Cf::KBlk + r * box_rows * 128, kv >= NP ? &mv : &mk,
                             64 * bl, slot, t.hk, page, kv % NP, b_full + 8 * st);
                    ++issued;
                    if (++st == NS) {
                        st = 0;
                        ph ^= 1;
                    }
                };
                for (int kv = 0; kv < NP; ++kv) put(kv, live, page, slot);
                if (j == 0)
                    for (int i = 0; ok && i < nt; ++i) {
                        ok = wait_go(b_qe + 8 * i, (qph >> i) & 1u);
                        if (ok) {
                            if (lane == 0) {
                                const uint32_t bytes = (uint32_t)(NP * NB) * 128u * (uint32_t)(G * TQ);
                                mbar_expect_tx(b_q + 8 * i, bytes + (n == 0 && i == 0 ? (uint32_t)p.extra_tx : 0u));
                                for (int b = 0; b < NP * NB; ++b)
                                    tma4(sb + Cf::OffQ + i * Cf::QTile + b * kPfBlk, &mq, 64 * (b % NB), t.hk * G,
                                         t.row0 + i * TQ, b / NB, b_q + 8 * i);
                            }
                            __syncwarp();
                            qph ^= 1u << i;
                            q_out |= 1u << i;
                        }
                    }
                if constexpr (Cf::PS) {  // V follows the next key tile's K
                    if (j > 0) put(NP, v_live, v_page, v_slot);
                    v_live = live;
                    v_page = page;
                    v_slot = slot;
                    if (j + 1 == nk) put(NP, live, page, slot);
                } else {
                    for (int kv = NP; kv < 2 * NP; ++kv) put(kv, live, page, slot);
                }
                if (lane == 0) *progress = issued;
                ++n_tile;
                if (wide && j + 1 < nk) fac = factors(j + 1);  // the lookup has come back by now
                if (ok && j + 1 == nk) {  // the ring is full: time to find the next item
                    int at = answer();
                    if (at >= 0) next = pf_find(p, at, row_tiles * TQ, lane);
                    while (ok && at >= 0 && next.seq < 0) {  // the numbers behind it have no item either: nothing launches them
                        ask();
                        at = answer();
                    }
                    if (ok) ok = wait_item(b_read + 8 * ((n + 1) % kPfItems), ((uint32_t)((n + 1) / kPfItems) & 1u) ^ 1u);
                    if (ok && lane == 0) {
                        tile_s[(n + 1) % kPfItems] = next;
                        pf_arrive(b_known + 8 * ((n + 1) % kPfItems));
                    }
                    __syncwarp();
                }
            }
            if (ok) t = next;
        }
        if (!ok && lane == 0) fail();
        // what is in flight lands before the CTA ends (it has, unless a wait gave up)
        if (lane == 0) {
            for (int n = max(0, issued - NS); n < issued; ++n)
                mbar_wait(b_full + 8 * (n % NS), (uint32_t)(n / NS) & 1u, kWaitCycles);
            if (!ok) {
                for (int i = 0; i < NT; ++i)
                    if ((q_out >> i) & 1u) mbar_wait(b_q + 8 * i, (qph >> i) & 1u, kWaitCycles);
                if (asked) mbar_wait(b_next, nph, kWaitCycles);
            }
        }
        __syncwarp();
    } else if (warp == Cf::Mma || warp == Cf::Mma + 1) {
        // ------------------------------------------------------------ MMA issue
        // warp w: row tiles w and w + 2, so that tiles seldom wait for each other's
        // softmax (one warp for two tiles: 315 us against 277 at 8192 rows, head
        // size 64, two tiles a CTA)
        const int w = warp - Cf::Mma;
        const bool leader = tc::elect_one();
        const uint32_t id_s = tc::idesc_16(128, KT, BF, false), id_o = tc::idesc_16(128, D, BF, true);
        const uint32_t q0 = tc::desc_sw128(sb + Cf::OffQ, 16), k0 = tc::desc_sw128(sb + Cf::OffRing, 16);
        const uint32_t v0 = tc::desc_sw128(sb + Cf::OffRing, Cf::KBlk), p0 = tc::desc_sw128(sb + Cf::OffP, 16);
        int st = 0;  // the ring: key tile j's K parts, then its V parts
        uint32_t ph = 0;
        uint32_t qph = 0, pph = 0, oph = ~0u, rph = ~0u;  // bit i: phases of tile i's Q, P, free O and read S
        auto next = [&]() {
            if (++st == NS) {
                st = 0;
                ph ^= 1;
            }
        };
        auto landed = [&](int s0, uint32_t p0) {  // the NP stages from s0 on
            bool all = true;
#pragma unroll
            for (int y = 0; y < NP; ++y) {
                const int at = s0 + y < NS ? s0 + y : s0 + y - NS;
                all = all && wait(b_full + 8 * at, s0 + y < NS ? p0 : p0 ^ 1u);
            }
            return all;
        };
        bool ok = true;
        PfTile t;
        for (int n = 0; ok; ++n) {
            ok = tile_of(n, t);
            if (!ok || t.seq < 0) break;
            tile_read(n);
            int k_first, nk, tail;
            keys_of(t, k_first, nk, tail);
            const int nt = (t.tokens + TQ - 1) / TQ;
            if (w >= nt) {  // the other warp frees the stages
                for (int x = 0; x < 2 * NP * nk; ++x) next();
                continue;
            }
            const int last = w + 2 < nt ? w + 2 : w;  // this warp's last tile
            // both warps free a ring stage after their last tile; a warp alone does it twice
            auto release = [&](int s) {
                tc::commit(b_empty + 8 * s);
                if (nt == 1) tc::commit(b_empty + 8 * s);
            };
            // S_i = Q_i K^T of the NP ring stages from s0 on, which have landed
            auto scores = [&](int i, int s0, bool final) {
                if (leader) {
                    const uint32_t ts = taddr + (uint32_t)(KT * i);
                    const uint32_t qd = q0 + (uint32_t)((i * Cf::QTile) >> 4);
#pragma unroll
                    for (int y = NP - 1; y >= 0; --y) {  // the small products first
                        const int sk = s0 + y < NS ? s0 + y : s0 + y - NS;
                        const uint32_t kd = k0 + (uint32_t)((sk * Cf::Tile) >> 4);
#pragma unroll
                        for (int x = NP - 1 - y; x >= 0; --x)  // Q's part x by K's part y
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks)
                                tc::mma_sw128(ts,
                                              qd + (uint32_t)((x * Cf::QPart + (ks / 4) * kPfBlk + (ks % 4) * 32) >> 4),
                                              kd + (uint32_t)(((ks / 4) * Cf::KBlk + (ks % 4) * 32) >> 4), id_s,
                                              !(y == NP - 1 && x == 0 && ks == 0));
                        if (y == 0) tc::commit(b_s + 8 * i);
                        if (y == 0 && final) tc::commit(b_qe + 8 * i);
                        if (i == last) release(sk);
                    }
                }
                __syncwarp();
            };
            auto s_read = [&](int i) {  // the tile's S before has been read
                if constexpr (Cf::PS) {
                    ok = ok && wait(b_sr + 8 * i, (rph >> i) & 1u);
                    rph ^= 1u << i;
                }
            };
            ok = landed(st, ph);
            for (int i = w; ok && i < nt; i += 2) {
                ok = wait(b_q + 8 * i, (qph >> i) & 1u);
                qph ^= 1u << i;
                s_read(i);
                tc::fence_after_sync();
                if (ok) scores(i, st, nk == 1);
            }
            for (int y = 0; y < NP; ++y) next();
            for (int j = 0; ok && j < nk; ++j) {
                if constexpr (Cf::PS)
                    if (j + 1 < nk) {  // the next scores, as soon as S has been read
                        ok = landed(st, ph);
                        s_read(w);
                        tc::fence_after_sync();
                        if (ok) scores(w, st, j + 2 == nk);
                        next();
                    }
                const int sv = st;  // V's stages
                const uint32_t phv = ph;
                for (int y = 0; y < NP; ++y) next();
                const int sk = st;  // the next K's
                const uint32_t phk = ph;
                ok = ok && landed(sv, phv);
                if (j + 1 < nk) {
                    if constexpr (!Cf::PS) {
                        for (int y = 0; y < NP; ++y) next();
                        ok = ok && landed(sk, phk);
                    }
                } else if (ok && tail < KT) {
                    // V rows behind the last position: zeros, whatever the page holds
                    // (each MMA warp writes them: nobody waits)
#pragma unroll
                    for (int y = 0; y < NP; ++y) {
                        uint8_t *v = sm + Cf::OffRing + (sv + y < NS ? sv + y : sv + y - NS) * Cf::Tile;
                        for (int x = tail * 8 + lane; x < KT * 8; x += 32)
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                *reinterpret_cast<uint4 *>(v + b * Cf::KBlk + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                for (int i = w; ok && i < nt; i += 2) {
                    ok = wait(b_p + 8 * i, (pph >> i) & 1u);
                    pph ^= 1u << i;
                    if (j == 0) {  // the item before has left O
                        ok = ok && wait(b_oe + 8 * i, (oph >> i) & 1u);
                        oph ^= 1u << i;
                    }
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (leader) {  // O_i += P_i V
                        const uint32_t to = taddr + (uint32_t)(Cf::ColO + D * i), tp = taddr + (uint32_t)(KT * i);
                        const bool fresh = NP == 2 || j == 0;
#pragma unroll
                        for (int y = NP - 1; y >= 0; --y) {
                            const int at = sv + y < NS ? sv + y : sv + y - NS;
                            const uint32_t vd = v0 + (uint32_t)((at * Cf::Tile) >> 4);
#pragma unroll
                            for (int x = NP - 1 - y; x >= 0; --x)  // P's part x by V's part y
#pragma unroll
                                for (int ks = 0; ks < KT / 16; ++ks)
                                    if constexpr (Cf::PS)
                                        tc::mma_sw128(to,
                                                      p0 + (uint32_t)((i * Cf::PTile + (ks / 4) * kPfBlk + (ks % 4) * 32) >> 4),
                                                      vd + (uint32_t)((ks * 2048) >> 4), id_o, !(fresh && ks == 0));
                                    else
                                        tc::mma_ta_sw128(to, tp + Cf::p_col(ks) + 16 * x, vd + (uint32_t)((ks * 2048) >> 4),
                                                     id_o, !(fresh && y == NP - 1 && x == 0 && ks == 0));
                            if (y == 0 && j + 1 == nk) tc::commit(b_o + 8 * i);
                            if (Cf::PS) tc::commit(b_pe + 8 * i);
                            if (i == last) release(at);
                        }
                    }
                    __syncwarp();
                    if constexpr (!Cf::PS)
                        if (j + 1 < nk) scores(i, sk, j + 2 == nk);
                }
            }
        }
        if (!ok && leader) fail();
        if (leader) {  // nothing is in flight when the CTA ends
            tc::commit(b_drain + 8 * w);
            mbar_wait(b_drain + 8 * w, 0u, kWaitCycles);
        }
        __syncwarp();
    } else if (warp == Cf::Rows) {
        // ------------------------------------------------------------ rows by the definition
        bool ok = true;
        PfTile t;
        for (int n = 0; ok; ++n) {
            ok = tile_of(n, t);
            if (!ok || t.seq < 0) break;
            ok = wait_item(b_mask + 8 * (n % kPfItems), (uint32_t)(n / kPfItems) & 1u);
            if (!ok) break;
            const unsigned rows = lane < Cf::Soft ? mask_s[(n % kPfItems) * Cf::Soft + lane] : 0u;
            unsigned warps = __ballot_sync(0xffffffffu, rows != 0u);
            if (warps) {
                if (lane == 0) *slow = *slow + 1;
                for (; warps; warps &= warps - 1) {
                    const int w = __ffs(warps) - 1;
                    for (unsigned left = __shfl_sync(0xffffffffu, rows, w); left; left &= left - 1) {
                        const int r = 32 * (w & 3) + __ffs(left) - 1, tok = (w >> 2) / HF * TQ + r / G;
                        attn_row<T, D>(p, t.row0 + tok, t.hk * G + r % G, t.seq, t.pos0 + tok, lane);
                    }
                }
                __syncwarp();
                if (lane == 0) *slow = *slow + 1;
            }
            tile_read(n);
        }
        if (!ok && lane == 0) fail();
    } else {
        // ------------------------------------------------------------ softmax
        auto softmax = [&](auto wide_t) {
            constexpr bool Wide = decltype(wide_t)::value;
            // tile i, columns 64 hf .. of every key tile, row r
            const int i = (warp >> 2) / HF, hf = (warp >> 2) % HF, r = 32 * (warp & 3) + lane;
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t ts = taddr + lanes + KT * i, to = taddr + lanes + Cf::ColO + D * i;
            const uint32_t tsum = taddr + lanes + Cf::ColSum + D * i;  // fp32: the sum of the O before
            constexpr int QO = D / (16 * HF);  // 16-column parts of O
            const uint32_t bx = b_x + 8 * (4 * (i & 1) + (warp & 3));
            float *xs = reinterpret_cast<float *>(sm + Cf::OffX) + 256 * i;  // [half][row]
            uint32_t sph = 0, oph = 0, xph = 0, uph = 1;  // phases of S, O, the exchange and the used P
            // a row's value of the other column half: its warp has read the one before
            // by the time it is written again (S of the next key tile comes after every
            // warp's P; where a key tile has several, a thread writes where it has itself
            // read last)
            int xw = hf;
            auto other = [&](float mine, bool &ok) {
                xs[xw * 128 + r] = mine;
                __syncwarp();
                if (lane == 0) pf_arrive(bx);
                ok = wait(bx, xph);
                xph ^= 1u;
                const float got = xs[(xw ^ 1) * 128 + r];
                if constexpr (Wide) xw ^= 1;
                return got;
            };
            int n_tile = 0;  // Wide: key tiles of the items before
            // fp32: weights from a key tile's own maximum `top` (2^PExp there) in the units of
            // the sums, whose reference is m
            auto own_down = [](float top, float m) {
                return top == -INFINITY ? 0.f : ex2(top - m - PfT<T>::PExp);
            };
            // 32 weights as two f16 parts: the high ones in w, what those leave in place
            auto parts = [](uint32_t *x, uint32_t (&w)[16]) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float a = __uint_as_float(x[2 * e]), b = __uint_as_float(x[2 * e + 1]);
                    w[e] = pack2<M>(a, b);
                    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                    x[e] = pack2<M>(a - h.x, b - h.y);
                }
            };
            bool ok = true;
            PfTile t;
            for (int n = 0; ok; ++n) {
                ok = tile_of(n, t);
                if (!ok || t.seq < 0) break;
                tile_read(n);
                // rows that are not finite are left to the warp that takes them again
                auto post = [&](unsigned rows) {
                    if (lane == 0) {
                        mask_s[(n % kPfItems) * Cf::Soft + warp] = rows;
                        pf_arrive(b_mask + 8 * (n % kPfItems));
                    }
                };
                int k_first, nk, tail, f_tile = 0;
                if constexpr (Wide) {
                    keys_of(t, k_first, nk, tail);
                    f_tile = n_tile;
                    n_tile += nk;
                }
                if (i >= (t.tokens + TQ - 1) / TQ) {
                    post(0u);
                    continue;
                }
                if constexpr (!Wide) keys_of(t, k_first, nk, tail);
                const int tok = i * TQ + r / G, g = r % G;
                const bool live = r < G * TQ && tok < t.tokens;
                const int pos = t.pos0 + (live ? tok : min(i * TQ, t.tokens - 1));
                const int pmin = t.pos0 + i * TQ, pmax = t.pos0 + min((i + 1) * TQ, t.tokens) - 1;
                const int row = t.row0 + tok, head = t.hk * G + g;
                // what brings S to log2 units: in the exponential's own product (c), fp32 when
                // S is read (cq, with K's factor)
                const float c = NP == 2 ? 1.f : p.scale * 1.4426950408889634f;
                float cq = 1.f;
                if constexpr (NP == 2)
                    cq = p.scale * 1.4426950408889634f * (Wide ? 1.f : kPfUsual) * (live ? p.qback[(size_t)row * p.H + head] : 0.f);
                float m = -INFINITY, l = 0.f;
                float back = 1.f;  // fp32: what the last key tile's O (and sum of weights) is in the sums' units
                for (int j = 0; j < nk; ++j) {
                    ok = wait(b_s + 8 * i, sph);
                    sph ^= 1u;
                    if (!ok) break;
                    tc::fence_after_sync();
                    // fp32: the tensor core's accumulation truncates, which over a long chain
                    // of products shows (3e-6 of the output after 2048 positions, 8e-7 with
                    // two key tiles in a chain, 4e-7 so): each key tile's O is added to a
                    // sum beside it.  S came after the product before it: O is complete
                    if (NP == 2 && j > 0) {
#pragma unroll 1
                        for (int q = 0; q < D / (16 * HF); ++q) {
                            uint32_t o[16], a[16];
                            const uint32_t at = (D / HF) * hf + 16 * q;
                            tc::ld16(to + at, o);
                            if (j > 1) {
                                tc::ld16(tsum + at, a);
                                tc::wait_ld16(a);
                            }
                            tc::wait_ld16(o);
                            const uint64_t b2 = pair_f32(back, back);
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const uint64_t y = fma_f32x2(pair_u32(o[e], o[e + 1]), b2, j > 1 ? pair_u32(a[e], a[e + 1]) : 0ull);
                                o[e] = (uint32_t)y;
                                o[e + 1] = (uint32_t)(y >> 32);
                            }
                            tc::st16(tsum + at, o);
                        }
                    }
                    if constexpr (Wide) {
                        const int k0 = k_first + j * KT;
                        const bool masked = k0 + KT - 1 > pmin || (p.window > 0 && k0 <= pmax - p.window);
                        const int hi = pos - k0 - CW * hf, lo = p.window > 0 ? pos - p.window + 1 - k0 - CW * hf : -1;
                        // the positions' factors, and whether all have the same
                        const int at = f_tile + j;
                        ok = wait(b_f + 8 * (at % Cf::NF), (uint32_t)(at / Cf::NF) & 1u);
                        if (!ok) break;
                        const uint32_t f0 = Cf::OffF + (at % Cf::NF) * Cf::FacBytes, fac = sb + f0 + CW * 4 * hf;
                        const uint2 same = *reinterpret_cast<const uint2 *>(sm + f0 + 4 * KT);
                        // each position with its own factor: the scores of 32 columns from q on,
                        // in log2 units (read again in every pass over them: registers for all of
                        // them beside the other path's were not to be had)
                        auto own_scores = [&](int q, uint32_t (&x)[32]) {
                            tc::ld32(ts + CW * hf + q, x);
                            tc::wait_ld32(x);
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const uint4 f = lds128_at<0>(fac + 4 * (q + e));
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    x[e + y] = __float_as_uint(__uint_as_float(x[e + y]) * (__uint_as_float(w_of(f, y) & 0xffff0000u) * cq));
                                    if (masked && (q + e + y > hi || q + e + y < lo)) x[e + y] = 0xff800000u;
                                }
                            }
                        };
                        uint64_t sum[2] = {0ull, 0ull}, mc2 = 0ull;
                        float top = -INFINITY, mc = 0.f, down = 0.f;
                        // the row's maximum with this key tile's, and the sums so far to it
                        auto raise = [&]() {
                            top = fmaxf(top, other(top, ok));
                            if (!ok) return;
                            if (j == 0) {
                                m = top;
                            } else {
                                const bool grew = top > m && (m == -INFINITY || top - m > kPfGrow);
                                if (__any_sync(0xffffffffu, grew)) {  // the same answer in both halves' warps
                                    const float mn = grew ? fmaxf(m, top) : m;
                                    const float alpha = m == -INFINITY ? 0.f : ex2(m - mn);
                                    l *= alpha;
                                    m = mn;
                                    tc::wait_st();  // the sum's columns were stored above
#pragma unroll 1
                                    for (int q = 0; q < QO; ++q) {
                                        uint32_t o[16];
                                        const uint32_t at = tsum + 16 * q + (D / HF) * hf;
                                        tc::ld16(at, o);
                                        tc::wait_ld16(o);
#pragma unroll
                                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                        tc::st16(at, o);
                                    }
                                }
                            }
                            mc = (top == -INFINITY ? 0.f : -top) + PfT<T>::PExp;
                            mc2 = pair_f32(mc, mc);
                            down = own_down(top, m);
                        };
                        if (same.y != 0u) {
                            uint32_t s[CW];
#pragma unroll
                            for (int q = 0; q < CW / 32; ++q) tc::ld32(ts + CW * hf + 32 * q, s + 32 * q);
#pragma unroll
                            for (int q = 0; q < CW / 32; ++q) tc::wait_ld32(s + 32 * q);
                            const float cs = cq * __uint_as_float(same.x & 0xffff0000u);
                            const uint64_t cs2 = pair_f32(cs, cs);
#pragma unroll
                            for (int e = 0; e < CW; e += 2) {
                                const uint64_t y = mul_f32x2(pair_u32(s[e], s[e + 1]), cs2);
                                s[e] = (uint32_t)y;
                                s[e + 1] = (uint32_t)(y >> 32);
                            }
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < CW; ++e)
                                    if (e > hi || e < lo) s[e] = 0xff800000u;
                            }
                            float mx[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) mx[q] = fmaxf(__uint_as_float(s[q]), __uint_as_float(s[4 + q]));
#pragma unroll
                            for (int e = 8; e < CW; e += 8)
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    mx[q] = fmaxf(fmaxf(mx[q], __uint_as_float(s[e + q])), __uint_as_float(s[e + 4 + q]));
                            top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                            raise();
                            if (!ok) break;
                            back = down * __uint_as_float(same.x << 16);
#pragma unroll
                        for (int e = 0; e < CW; e += 2) {
                            const uint64_t x = add_f32x2(pair_u32(s[e], s[e + 1]), mc2);
                            const float a = ex2(lo_f32(x)), b = ex2(hi_f32(x));
                            sum[e / 2 & 1] = add_f32x2(sum[e / 2 & 1], pair_f32(a, b));
                            s[e] = __float_as_uint(a);
                            s[e + 1] = __float_as_uint(b);
                        }
#pragma unroll
                        for (int q = 0; q < CW / 32; ++q) {
                            uint32_t w[16];
                            parts(s + 32 * q, w);
                            tc::st16(ts + CW * hf + 32 * q, w);
                            tc::st16(ts + CW * hf + 32 * q + 16, s + 32 * q);
                        }
                    } else {
#pragma unroll 1
                            for (int q = 0; q < CW; q += 32) {
                                uint32_t x[32];
                                own_scores(q, x);
#pragma unroll
                                for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(x[e]));
                            }
                            raise();
                            if (!ok) break;
                            // the largest of the attended factors of V, of the weights of values that
                            // are not zero, and of their products
                            float big = 0.f, big_v = 0.f, big_w = 0.f;
#pragma unroll 1
                            for (int q = 0; q < CW; q += 32) {
                                uint32_t x[32];
                                own_scores(q, x);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    float v;
                                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(fac + 4 * (q + e)) : "memory");
                                    v = __uint_as_float(__float_as_uint(v) << 16);
                                    if (__uint_as_float(x[e]) > -INFINITY && v > 0.f) {
                                        const float w = ex2(__uint_as_float(x[e]) + mc);
                                        big = fmaxf(big, w * v);
                                        big_v = fmaxf(big_v, v);
                                        big_w = fmaxf(big_w, w);
                                    }
                                }
                            }
                            big = fmaxf(big, other(big, ok));
                            if (!ok) break;
                            big_v = fmaxf(big_v, other(big_v, ok));
                            if (!ok) break;
                            big_w = fmaxf(big_w, other(big_w, ok));
                            if (!ok) break;
                            // The largest factor becomes the one of all, as long as the largest
                            // product is within 2^6 of that weight at it (it is when the attended
                            // factors are the same: the bits are then those of a key tile with one);
                            // else the largest product goes to [2^13, 2^14).  Powers of two, back and
                            // forth below 2^127
                            const uint32_t e_big = __float_as_uint(big) >> 23, e_v = __float_as_uint(big_v) >> 23;
                            const uint32_t ex = min(big < big_w * big_v * 0.015625f ? 267u - e_big : 254u - e_v, 253u);
                            const float up = __uint_as_float(ex << 23);
                            back = down * __uint_as_float((254u - ex) << 23);
#pragma unroll 1
                            for (int q = 0; q < CW; q += 32) {
                                uint32_t x[32], w[16];
                                own_scores(q, x);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float v0, v1;
                                    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v0), "=f"(v1) : "r"(fac + 4 * (q + 2 * e)) : "memory");
                                    const uint64_t y = add_f32x2(pair_u32(x[2 * e], x[2 * e + 1]), mc2);
                                    const float a = ex2(lo_f32(y)), b = ex2(hi_f32(y));
                                    sum[e & 1] = add_f32x2(sum[e & 1], pair_f32(a, b));
                                    x[2 * e] = __float_as_uint(a * (__uint_as_float(__float_as_uint(v0) << 16) * up));
                                x[2 * e + 1] = __float_as_uint(b * (__uint_as_float(__float_as_uint(v1) << 16) * up));
                            }
                            parts(x, w);
                            tc::st16(ts + CW * hf + q, w);
                                tc::st16(ts + CW * hf + q + 16, x);
                            }
                        }
                        const uint64_t s2 = add_f32x2(sum[0], sum[1]);
                        l = fmaf(lo_f32(s2) + hi_f32(s2), down, l);
                    } else {
                        uint32_t s[CW];
#pragma unroll
                        for (int q = 0; q < CW / 32; ++q) tc::ld32(ts + CW * hf + 32 * q, s + 32 * q);
#pragma unroll
                        for (int q = 0; q < CW / 32; ++q) tc::wait_ld32(s + 32 * q);
                        if constexpr (NP == 2) {
                            const uint64_t cq2 = pair_f32(cq, cq);
#pragma unroll
                            for (int e = 0; e < CW; e += 2) {
                                const uint64_t y = mul_f32x2(pair_u32(s[e], s[e + 1]), cq2);
                                s[e] = (uint32_t)y;
                                s[e + 1] = (uint32_t)(y >> 32);
                            }
                        }
                        const int k0 = k_first + j * KT;
                        if (k0 + KT - 1 > pmin || (p.window > 0 && k0 <= pmax - p.window)) {
                            const int hi = pos - k0 - CW * hf, lo = p.window > 0 ? pos - p.window + 1 - k0 - CW * hf : -1;
#pragma unroll
                            for (int e = 0; e < CW; ++e)
                                if (e > hi || e < lo) s[e] = 0xff800000u;
                        }
                        float mx[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(__uint_as_float(s[q]), __uint_as_float(s[4 + q]));
#pragma unroll
                        for (int e = 8; e < CW; e += 8)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mx[q] = fmaxf(fmaxf(mx[q], __uint_as_float(s[e + q])), __uint_as_float(s[e + 4 + q]));
                        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        if constexpr (HF == 2) {
                            top = fmaxf(top, other(top, ok));
                            if (!ok) break;
                        }
                        bool used = !Cf::PS;  // the product before this key tile's is complete
                        auto wait_used = [&]() {
                            if (!used) {
                                ok = wait(b_pe + 8 * i, uph);
                                uph ^= 1u;
                                tc::fence_after_sync();
                                used = true;
                            }
                        };
                        if constexpr (Cf::PS) {  // S (and the other half's maximum) has been read
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) pf_arrive(b_sr + 8 * i);
                        }
                        if (j == 0) {
                            m = top;
                        } else {
                            const bool grew = top > m && (m == -INFINITY || (top - m) * c > kPfGrow);
                            if (__any_sync(0xffffffffu, grew)) {  // the same answer in both halves' warps
                                // (fp32: only the rows that grew, so that none follows its neighbours)
                                const float mn = NP == 1 || grew ? fmaxf(m, top) : m;
                                const float alpha = m == -INFINITY ? 0.f : ex2((m - mn) * c);
                                l *= alpha;
                                m = mn;
                                wait_used();
                                // the sum's columns were stored above: a load is not ordered after
                                // a store of the same columns until the store's wait
                                if constexpr (NP == 2) tc::wait_st();
#pragma unroll 1
                                for (int q = 0; q < QO; ++q) {
                                    uint32_t o[16];
                                    const uint32_t at = (NP == 2 ? tsum : to) + 16 * q + (D / HF) * hf;
                                    tc::ld16(at, o);
                                    tc::wait_ld16(o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tc::st16(at, o);
                                }
                            }
                        }
                        // (fp32: from the key tile's own maximum)
                        const float ref = NP == 2 ? top : m;
                        const float mc = (ref == -INFINITY ? 0.f : -ref * c) + PfT<T>::PExp;
                        const uint64_t c2 = pair_f32(c, c), mc2 = pair_f32(mc, mc);
                        uint64_t sum[2] = {0ull, 0ull};
                        if constexpr (NP == 2) {  // (all, then their parts: 74 us, pair by pair 81)
#pragma unroll
                            for (int e = 0; e < CW; e += 2) {
                                const uint64_t x = add_f32x2(pair_u32(s[e], s[e + 1]), mc2);
                                const float a = ex2(lo_f32(x)), b = ex2(hi_f32(x));
                                sum[e / 2 & 1] = add_f32x2(sum[e / 2 & 1], pair_f32(a, b));
                                s[e] = __float_as_uint(a);
                                s[e + 1] = __float_as_uint(b);
                            }
                        }
                        // (over S's columns: the row's warps have read them)
#pragma unroll
                        for (int q = 0; q < CW / 32; ++q) {
                            uint32_t w[16];
                            if constexpr (NP == 2) {
                                parts(s + 32 * q, w);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const uint64_t x = fma_f32x2(pair_u32(s[32 * q + 2 * e], s[32 * q + 2 * e + 1]), c2, mc2);
                                    const float a = ex2(lo_f32(x)), b = ex2(hi_f32(x));
                                    sum[e & 1] = add_f32x2(sum[e & 1], pair_f32(a, b));
                                    w[e] = pack2<M>(a, b);
                                }
                            }
                            if constexpr (Cf::PS) {
                                wait_used();
                                uint8_t *dst = sm + Cf::OffP + i * Cf::PTile + hf * kPfBlk + r * 128;
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    *reinterpret_cast<uint4 *>(dst + (((4 * q + x) ^ (r & 7)) << 4)) =
                                        make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                            } else {
                                tc::st16(ts + (NP == 2 ? CW * hf + 32 * q : CW / 2 * hf + 16 * q), w);
                            }
                            if constexpr (NP == 2) tc::st16(ts + CW * hf + 32 * q + 16, s + 32 * q);
                        }
                        const uint64_t s2 = add_f32x2(sum[0], sum[1]);
                        if constexpr (NP == 2) {
                            back = own_down(top, m);
                            l = fmaf(lo_f32(s2) + hi_f32(s2), back, l);
                        }
                        else
                            l += lo_f32(s2) + hi_f32(s2);
                    }
                    if (!ok) break;
                    tc::wait_st();
                    tc::fence_before_sync();
                    if constexpr (Cf::PS) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) pf_arrive(b_p + 8 * i);
                }
                ok = ok && wait(b_o + 8 * i, oph);
                oph ^= 1u;
                if (!ok) break;
                tc::fence_after_sync();
                uint32_t o[16 * QO];
                float worst = 0.f;  // NaN where a value is not finite
#pragma unroll
                for (int q = 0; q < QO; ++q) {
                    tc::ld16(to + (D / HF) * hf + 16 * q, o + 16 * q);
                    if (NP == 2 && nk > 1) {
                        uint32_t a[16];
                        tc::ld16(tsum + (D / HF) * hf + 16 * q, a);
                        tc::wait_ld16(a);
                        tc::wait_ld16(o + 16 * q);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[16 * q + e] = __float_as_uint(fmaf(__uint_as_float(o[16 * q + e]), back, __uint_as_float(a[e])));
                    }
                }
#pragma unroll
                for (int q = 0; q < QO; ++q) tc::wait_ld16(o + 16 * q);
                if (NP == 2 && nk == 1)
#pragma unroll
                    for (int e = 0; e < 16 * QO; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * back);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) pf_arrive(b_oe + 8 * i);  // the next item's product may begin
#pragma unroll
                for (int e = 0; e < 16 * QO; ++e) worst = fmaf(__uint_as_float(o[e]), 0.f, worst);
                l += worst;
                if constexpr (HF == 2) {
                    l += other(l, ok);
                    if (!ok) break;
                    __syncwarp();
                    if (lane == 0) pf_arrive(bx);  // read: may be written again
                }
                // (both halves' warps see the same l)
                const bool finite = l > 0.f && l < INFINITY;  // (0: every score is -inf)
                float inv = 1.f / l;
                if constexpr (NP == 2 && !Wide) inv *= kPfUsual;
                // 128 bytes of a row at a time: eight lanes exchange theirs, so that a store
                // fills whole lines (each lane its own row: 7000 cycles an item, not 2000)
                const size_t at = ((size_t)row * p.H + head) * D + (D / HF) * hf;
                const unsigned good = __ballot_sync(0xffffffffu, live && finite);
#pragma unroll
                for (int q = 0; q < D * (int)sizeof(T) / (128 * HF); ++q) {
                    uint32_t w[8][4];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if constexpr (sizeof(T) == 4)
                            w[e / 4][e % 4] = __float_as_uint(__uint_as_float(o[32 * q + e]) * inv);
                        else
                            w[e / 4][e % 4] = pack2<T>(__uint_as_float(o[64 * q + 2 * e]) * inv, __uint_as_float(o[64 * q + 2 * e + 1]) * inv);
                    }
                    pf_transpose8(w, lane);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int src = (lane & 24) + x;
                        const size_t a = __shfl_sync(0xffffffffu, at, src);
                        if ((good >> src) & 1u)
                            *reinterpret_cast<uint4 *>((uint8_t *)((T *)p.out + a) + 128 * q + 16 * (lane & 7)) =
                                make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
                    }
                }
                post(__ballot_sync(0xffffffffu, live && hf == 0 && !finite));
                if constexpr (HF == 2) {
                    ok = wait(bx, xph);
                    xph ^= 1u;
                }
            }
            if (!ok && lane == 0) fail();
        };
        if (wide)
            softmax(std::integral_constant<bool, NP == 2>());
        else
            softmax(std::false_type());
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == Cf::Mma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(taddr, 512);
    }
}

// ---------------------------------------------------------------- fp32 caches
// q4attn_prefill_split_kernel writes the two f16 parts of Q's rows, and of the
// attended positions' K and V into images laid out like the pages ([part][page]
// [kv head][slot][D]), so that the tensor maps of a 16-bit cache fit.  A power of
// two a row puts its largest finite value below 2^14 (of Q, per head, in [2^13,
// 2^14); of K and V, per position and kv head, in steps of 2^12: in [2^2, 2^14)); its
// inverses lie beside (Q's fp32; K's and V's as one word of bf16 halves, laid out like
// the pages).  They follow from the row alone: pages that sequences share get the
// same values from each.  A part's rounding is 2^-25 at least, so a value of K or V
// enters with 22 bits or to 2^-27 of its row's largest.

constexpr int kPfChunk = 64;  // positions of a staging item

// The power of two for a largest magnitude.
__device__ __forceinline__ int pf_exp(float mx) {
    if (!(mx > 0.f)) return 0;
    int e;
    frexpf(mx, &e);
    return min(14 - e, 126);  // at least -114
}
// The same in steps of 12: values of 2^-5 .. 2^7, a cache's usual ones, in one step
__device__ __forceinline__ int pf_exp12(float mx) {
    if (!(mx > 0.f)) return 0;
    int e;
    frexpf(mx, &e);
    return min(7 - ((e + 4 + 156) / 12 - 13) * 12, 126);  // at least -125
}

// hi and lo parts of four values times f
__device__ __forceinline__ void pf_split4(float4 v, float f, uint2 &hi, uint2 &lo) {
    v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    hi = make_uint2(pack2<__half>(v.x, v.y), pack2<__half>(v.z, v.w));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&hi.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi.y));
    lo = make_uint2(pack2<__half>(v.x - a.x, v.y - a.y), pack2<__half>(v.z - b.x, v.w - b.y));
}
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}

// fn(sequence, kv head, first position, end) for this CTA's items: the chunks
// of every sequence's attended positions (rounded down to a multiple of `Align`)
// by kv heads.
template <int Align, class F>
__device__ __forceinline__ void pf_items(const PrefillParams &p, F fn) {
    __shared__ long long prefix[kMaxSeqs + 1];
    __shared__ long long wsum[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto range = [&](int b, int &lo, int &end) {
        const int begin = min(max(p.cu[b], 0), p.rows), rows = max(min(p.cu[b + 1], p.rows) - begin, 0);
        const int first = p.start ? p.start[b] : 0;
        lo = end = 0;
        if (rows == 0 || first < 0 || first >= (long long)p.kv.width * p.kv.page) return;
        end = (int)min((long long)first + rows, (long long)p.kv.width * p.kv.page);
        lo = (p.window > 0 && first + 1 > p.window ? first + 1 - p.window : 0) & ~(Align - 1);
    };
    long long n[4], own = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = 4 * tid + i;
        int lo = 0, end = 0;
        if (b < p.kv.nseq) range(b, lo, end);
        n[i] = (end - lo + kPfChunk - 1) / kPfChunk;
        own += n[i];
    }
    long long inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    long long base = inc - own;
    for (int w = 0; w < warp; ++w) base += wsum[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * tid + i <= p.kv.nseq) prefix[4 * tid + i] = base;
        base += n[i];
    }
    if (tid == 255 && p.kv.nseq == kMaxSeqs) prefix[kMaxSeqs] = base;
    __syncthreads();
    const long long total = prefix[p.kv.nseq] * p.kv.hkv;
    for (long long it = blockIdx.x; it < total; it += gridDim.x) {
        const long long c = it / p.kv.hkv;
        const int hk = (int)(it - c * p.kv.hkv);
        int b = 0, hi = p.kv.nseq;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (prefix[mid] <= c)
                b = mid;
            else
                hi = mid;
        }
        int lo, end;
        range(b, lo, end);
        const int at = lo + (int)(c - prefix[b]) * kPfChunk;
        fn(b, hk, at, min(end, at + kPfChunk));
    }
}

// The K and V values of a staging item that a thread handles: dims 4 (tid % L) ..
// of every 256 / L-th position, all loads at once (ok: bit i, position i is
// attended and its page in range).
template <int D>
struct PfRows {
    static constexpr int L = D / 4, N = kPfChunk * L / 256;
    float4 k[N], v[N];
    size_t off[N], place[N];  // element of (position, this thread's dims); of the position's factors
    unsigned ok = 0;
    __device__ __forceinline__ PfRows(const PrefillParams &p, int b, int hk, int at, int end) {
        const int tid = threadIdx.x;
        int page[N], slot[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int pos = at + tid / L + i * (256 / L), col = page_col(p.kv, pos);
            page[i] = pos < end ? page_at(p.kv, b, col) : -1;
            slot[i] = pos - col * p.kv.page;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            k[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (page[i] < 0) continue;
            ok |= 1u << i;
            off[i] = row_off(p.kv, page[i], hk, slot[i], D) + 4 * (tid % L);
            place[i] = ((size_t)page[i] * p.kv.hkv + hk) * p.fac_stride + slot[i];
            k[i] = *reinterpret_cast<const float4 *>((const float *)p.kv.k + off[i]);
            v[i] = *reinterpret_cast<const float4 *>((const float *)p.kv.v + off[i]);
        }
    }
};
__device__ __forceinline__ float finite_max(float m, float4 v) {
    return fmaxf(fmaxf(m, fmaxf(finite_abs(v.x), finite_abs(v.y))), fmaxf(finite_abs(v.z), finite_abs(v.w)));
}

// The largest of m[0 .. N) over the D / 4 lanes of a row.
template <int D, int N>
__device__ __forceinline__ void row_max(float (&m)[N]) {
#pragma unroll
    for (int o = D / 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
}

template <int D>
__global__ void __launch_bounds__(256, 2) q4attn_prefill_split_kernel(const __grid_constant__ PrefillParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int L = D / 4, U = 4;  // lanes of a row, rows of Q at once
    const int tid = threadIdx.x, j = 4 * (tid % L);
    const size_t part = (size_t)p.kv.num_pages * p.kv.hkv * p.kv.page * D;
    bool met = false;  // a factor that is not the usual one
    pf_items<128>(p, [&](int b, int hk, int at, int end) {  // from a key tile's start
        constexpr int N = PfRows<D>::N;
        const PfRows<D> x(p, b, hk, at, end);
        float mk[N], mv[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            mk[i] = finite_max(0.f, x.k[i]);
            mv[i] = finite_max(0.f, x.v[i]);
        }
        row_max<D>(mk);
        row_max<D>(mv);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (((x.ok >> i) & 1u) == 0) continue;
            const int ek = pf_exp12(mk[i]), ev = pf_exp12(mv[i]);
            uint2 hi, lo;
            pf_split4(x.k[i], ldexpf(1.f, ek), hi, lo);
            *reinterpret_cast<uint2 *>(p.kimg + x.off[i]) = hi;
            *reinterpret_cast<uint2 *>(p.kimg + part + x.off[i]) = lo;
            pf_split4(x.v[i], ldexpf(1.f, ev), hi, lo);
            *reinterpret_cast<uint2 *>(p.vimg + x.off[i]) = hi;
            *reinterpret_cast<uint2 *>(p.vimg + part + x.off[i]) = lo;
            // zeros: 0, so that their weight does not set the others' step
            met = met || (mk[i] > 0.f && ek != 7) || (mv[i] > 0.f && ev != 7);
            if (j == 0)
                p.fac[x.place[i]] = (mk[i] > 0.f ? __float_as_uint(ldexpf(1.f, -ek)) : 0u) |
                                    (mv[i] > 0.f ? __float_as_uint(ldexpf(1.f, -ev)) >> 16 : 0u);
        }
    });
    if (const int any = __syncthreads_or(met); tid == 0) p.met[blockIdx.x] = any;
    const size_t units = (size_t)p.rows * p.H, qpart = units * D;
    for (size_t u0 = (size_t)blockIdx.x * (U * 256 / L); u0 < units; u0 += (size_t)gridDim.x * (U * 256 / L)) {
        float4 q[U];
        float m[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const size_t u = u0 + tid / L + i * (256 / L);
            q[i] = u < units ? *reinterpret_cast<const float4 *>((const float *)p.q + u * D + j)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) m[i] = finite_max(0.f, q[i]);
        row_max<D>(m);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const size_t u = u0 + tid / L + i * (256 / L);
            if (u >= units) continue;
            const int e = pf_exp(m[i]);
            uint2 hi, lo;
            pf_split4(q[i], ldexpf(1.f, e), hi, lo);
            *reinterpret_cast<uint2 *>(p.qimg + u * D + j) = hi;
            *reinterpret_cast<uint2 *>(p.qimg + qpart + u * D + j) = lo;
            if (j == 0) p.qback[u] = ldexpf(1.f, -e);
        }
    }
}

}  // namespace dev

constexpr int kPfStaging = 1024;  // CTAs of the staging at most

// The fp32 form's workspace: the staging CTAs' words, K's and V's factors back, Q's,
// Q's parts, K's and V's.
size_t prefill_workspace(PrefillParams &p, int num_pages, int page, uint8_t *ws) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t q = (size_t)p.rows * p.H, kv = (size_t)num_pages * p.kv.hkv * page * p.D;
    size_t at = 0;
    p.met = (uint32_t *)(ws + at);
    at += up(sizeof(uint32_t) * kPfStaging);
    p.fac = (uint32_t *)(ws + at);
    p.fac_stride = (page + 3) / 4 * 4;  // four positions a load
    at += up(sizeof(uint32_t) * num_pages * p.kv.hkv * p.fac_stride);
    p.qback = (float *)(ws + at);
    at += up(q * sizeof(float));
    p.qimg = (uint16_t *)(ws + at);
    at += up(2 * q * p.D * sizeof(uint16_t));
    p.kimg = (uint16_t *)(ws + at);
    at += up(2 * kv * sizeof(uint16_t));
    p.vimg = (uint16_t *)(ws + at);
    return at + up(2 * kv * sizeof(uint16_t));
}

template <typename T, int D>
static int launch_tc(PrefillParams p, int sms, cudaStream_t stream) {
    constexpr int NP = dev::PfT<T>::Parts;
    using Cf = dev::PfCfg<D, NP>;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    const int G = p.H / p.kv.hkv, TQ = 128 / G;
    // positions a copy box takes: a power of two that divides the page, so
    // that no box crosses a page's end (one page alone: whole key tiles)
    int box_rows = Cf::KT;
    while (p.kv.width > 1 && p.kv.page % box_rows != 0) box_rows /= 2;
    // A scale of zero as the least number there is: times any score it is nothing, and a
    // masked one stays -inf (times 0 it is NaN, and its row would be taken by the
    // definition: 75 ms for 1024 rows of 8 heads, against 25 us)
    p.scale = std::max(p.scale, std::numeric_limits<float>::denorm_min());
    const void *q = p.q, *k = p.kv.k, *v = p.kv.v;
    cudaLaunchAttribute attr;
    if (NP == 2) {  // the parts of Q, K and V
        q = p.qimg;
        k = p.kimg;
        v = p.vimg;
        p.nmet = std::min(4 * sms, kPfStaging);
        const cudaLaunchConfig_t cfg = pdl_config((unsigned)p.nmet, 256, 0, stream, &attr);
        if (cudaLaunchKernelEx(&cfg, dev::q4attn_prefill_split_kernel<D>, p) != cudaSuccess) return -1;
    }
    CUtensorMap mq, mk, mv;
    const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)p.H, (cuuint64_t)p.rows, (cuuint64_t)NP};
    const cuuint32_t qb[4] = {64, (cuuint32_t)G, (cuuint32_t)TQ, 1};
    const cuuint64_t kd[5] = {(cuuint64_t)D, (cuuint64_t)p.kv.page, (cuuint64_t)p.kv.hkv, (cuuint64_t)p.kv.num_pages,
                              (cuuint64_t)NP};
    const cuuint32_t kb[5] = {64, (cuuint32_t)box_rows, 1, 1, 1};
    if (!make_map(&mq, BF, q, 4, qd, qb) || !make_map(&mk, BF, k, 5, kd, kb) || !make_map(&mv, BF, v, 5, kd, kb))
        return -1;
    auto kern = dev::q4attn_prefill_tc_kernel<T, D>;
    static size_t smem_set[64] = {0};
    if (!raise_smem(kern, (size_t)Cf::Smem, smem_set)) return -1;
    // row tiles a CTA: NT, fewer while that leaves the device without a CTA and a
    // half an SM; at most one part-filled item a sequence
    int row_tiles = Cf::NT;
    auto ctas = [&](int n) {
        return (p.rows + std::min<long long>(p.kv.nseq, p.rows) * (n * TQ - 1)) / (n * TQ) * p.kv.hkv;
    };
    while (row_tiles > 1 && 2 * ctas(row_tiles) < 3 * sms) row_tiles /= 2;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)ctas(row_tiles), Cf::Threads, Cf::Smem, stream, &attr);
    const bool more = ctas(row_tiles) > sms;  // than run at once
    return cudaLaunchKernelEx(&cfg, kern, p, mq, mk, mv, box_rows, row_tiles, more) == cudaSuccess ? 0 : -1;
}

int launch_prefill(const PrefillParams &p, int dtype, int sms, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    switch (dtype) {
        case 0: return p.D == 64 ? launch_tc<float, 64>(p, sms, s) : launch_tc<float, 128>(p, sms, s);
        case 1: return p.D == 64 ? launch_tc<__half, 64>(p, sms, s) : launch_tc<__half, 128>(p, sms, s);
        case 2: return p.D == 64 ? launch_tc<__nv_bfloat16, 64>(p, sms, s) : launch_tc<__nv_bfloat16, 128>(p, sms, s);
    }
    return -1;
}

}  // namespace q4
