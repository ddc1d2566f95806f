// kv_append.cu -- new keys and values into a paged KV cache (honeycrisp/
// mod.rs: the RoPE and KV-append part of the fused dispatch of
// forward_decode_fused_layers, for packed rows of several sequences): k and
// optionally q rotated by their position's row of the RoPE tables, k and v
// rounded to the cache's type and written to their pages, q rounded to that
// type into q_out.
//
// A pure stream: 4 bytes read and one cache element written per value.  One
// CTA per packed row; its sequence is the number of sequence ends at or below
// the row, counted by all threads at once (a binary search would be a chain of
// dependent loads).  A thread takes four rotation pairs (j .. j + 3 with j +
// D/2 ..), so every load is 16 bytes and every store 8 or 16; the first loads go
// out before the row's place is known, so the two latencies overlap.  8191 rows
// of 48 heads of 128 (306 MB): 45.8 us, 6.7 TB/s (51.7 with the head size an
// argument, whose divisions were half the instructions; 53.6 with the loads after).
#include "paged.cuh"
#include "tensor_map.h"

namespace q4 {
namespace dev {

constexpr int kAppendThreads = 256;
constexpr int kAppendAhead = 3;  // units a thread loads ahead

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) q4kv_append_kernel(const __grid_constant__ AppendParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.x, tid = threadIdx.x;
    constexpr int half = D / 2, UH = D / 8;
    const int Hq = p.q ? p.H : 0, Hkv = p.kv.hkv;
    const int units = (Hq + 2 * Hkv) * UH;
    // unit u: head u / UH of q, then k, then v, values j .. and half + j ..
    auto load = [&](unsigned u, float4 &a, float4 &b) {
        const int hs = u / UH, j = 4 * (u % UH);
        const float *src = hs < Hq         ? p.q + ((size_t)row * p.H + hs) * D
                           : hs < Hq + Hkv ? p.k + ((size_t)row * Hkv + hs - Hq) * D
                                           : p.v + ((size_t)row * Hkv + hs - Hq - Hkv) * D;
        a = *reinterpret_cast<const float4 *>(src + j);
        b = *reinterpret_cast<const float4 *>(src + j + half);
    };
    float4 a[kAppendAhead], b[kAppendAhead];
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i)
        if (tid + i * kAppendThreads < units) load(tid + i * kAppendThreads, a[i], b[i]);
    int seq = 0;
    for (int b0 = 0; b0 < p.kv.nseq; b0 += kAppendThreads) {
        const int s = b0 + tid;
        seq += __syncthreads_count(s < p.kv.nseq && p.cu[s + 1] <= row);
    }
    if (seq >= p.kv.nseq) return;  // a row behind the last sequence
    const int begin = p.cu[seq], first = p.start ? p.start[seq] : 0;
    const long long pos64 = (long long)first + row - begin;
    const bool in_range = begin >= 0 && begin <= row && first >= 0 &&
                          pos64 < (long long)p.kv.width * p.kv.page && (!p.rope_cos || pos64 < p.rope_rows);
    const int pos = in_range ? (int)pos64 : 0;
    const int col = page_col(p.kv, pos), page = in_range ? page_at(p.kv, seq, col) : -1;
    if (page < 0) {  // recorded, nothing of this row is written
        if (tid == 0) atomicExch(p.err, kErrPaged);
        return;
    }
    const int slot = pos - col * p.kv.page;
    const float *cosr = p.rope_cos ? p.rope_cos + (size_t)pos * half : nullptr;
    const float *sinr = p.rope_cos ? p.rope_sin + (size_t)pos * half : nullptr;
    auto store = [&](unsigned u, float4 x, float4 y) {
        const int hs = u / UH, j = 4 * (u % UH);
        const bool isq = hs < Hq, isv = hs >= Hq + Hkv;
        if (cosr && !isv)
            rotate4(x, y, *reinterpret_cast<const float4 *>(cosr + j), *reinterpret_cast<const float4 *>(sinr + j));
        T *dst = isq ? (T *)p.q_out + ((size_t)row * p.H + hs) * D
                     : (T *)(isv ? p.kv.v : p.kv.k) + row_off(p.kv, page, isv ? hs - Hq - Hkv : hs - Hq, slot, D);
        store4(dst + j, x);
        store4(dst + j + half, y);
    };
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i)
        if (tid + i * kAppendThreads < units) store(tid + i * kAppendThreads, a[i], b[i]);
    for (int u = tid + kAppendAhead * kAppendThreads; u < units; u += kAppendThreads) {
        load(u, a[0], b[0]);
        store(u, a[0], b[0]);
    }
}

}  // namespace dev

template <typename T>
static int launch_append_t(const AppendParams &p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)p.rows, dev::kAppendThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, p.D == 64 ? dev::q4kv_append_kernel<T, 64> : dev::q4kv_append_kernel<T, 128>, p) ==
                   cudaSuccess
               ? 0
               : -1;
}

int launch_append(const AppendParams &p, int dtype, void *stream_) {
    cudaStream_t stream = (cudaStream_t)stream_;
    switch (dtype) {
        case 0: return launch_append_t<float>(p, stream);
        case 1: return launch_append_t<__half>(p, stream);
        case 2: return launch_append_t<__nv_bfloat16>(p, stream);
    }
    return -1;
}

}  // namespace q4
