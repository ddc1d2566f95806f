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
// D/2 ..), so every load is 16 bytes and every store 8 or 16.
#include "paged.cuh"

namespace q4 {
namespace dev {

constexpr int kAppendThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) q4kv_append_kernel(const __grid_constant__ AppendParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.x, tid = threadIdx.x;
    int seq = 0;
    for (int b0 = 0; b0 < p.kv.nseq; b0 += kAppendThreads) {
        const int b = b0 + tid;
        seq += __syncthreads_count(b < p.kv.nseq && p.cu[b + 1] <= row);
    }
    if (seq >= p.kv.nseq) return;  // a row behind the last sequence
    const int D = p.D, half = D / 2, UH = D / 8;
    const int begin = p.cu[seq], first = p.start ? p.start[seq] : 0;
    const long long pos64 = (long long)first + row - begin;
    const bool in_range = begin >= 0 && begin <= row && first >= 0 &&
                          pos64 < (long long)p.kv.width * p.kv.page && (!p.rope_cos || pos64 < p.rope_rows);
    const int pos = in_range ? (int)pos64 : 0;
    const int page = in_range ? page_at(p.kv, seq, pos / p.kv.page) : -1;
    if (page < 0) {  // recorded, nothing of this row is written
        if (tid == 0) atomicExch(p.err, kErrPaged);
        return;
    }
    const int slot = pos % p.kv.page;
    const float *cosr = p.rope_cos ? p.rope_cos + (size_t)pos * half : nullptr;
    const float *sinr = p.rope_cos ? p.rope_sin + (size_t)pos * half : nullptr;
    const int Hq = p.q ? p.H : 0, Hkv = p.kv.hkv;
    const int units = (Hq + 2 * Hkv) * UH;
#pragma unroll 4
    for (int u = tid; u < units; u += kAppendThreads) {
        const int hs = u / UH, j = 4 * (u - hs * UH);
        const bool isq = hs < Hq, isv = hs >= Hq + Hkv;
        const int h = isq ? hs : isv ? hs - Hq - Hkv : hs - Hq;
        const float *src = isq ? p.q + ((size_t)row * p.H + h) * D : (isv ? p.v : p.k) + ((size_t)row * Hkv + h) * D;
        float4 a = *reinterpret_cast<const float4 *>(src + j), b = *reinterpret_cast<const float4 *>(src + j + half);
        if (cosr && !isv)
            rotate4(a, b, *reinterpret_cast<const float4 *>(cosr + j), *reinterpret_cast<const float4 *>(sinr + j));
        T *dst = isq ? (T *)p.q_out + ((size_t)row * p.H + h) * D
                     : (T *)(isv ? p.kv.v : p.kv.k) + row_off(p.kv, page, h, slot, D);
        store4(dst + j, a);
        store4(dst + j + half, b);
    }
}

}  // namespace dev

template <typename T>
static int launch_append_t(const AppendParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows, 1, 1);
    cfg.blockDim = dim3(dev::kAppendThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dev::q4kv_append_kernel<T>, p) == cudaSuccess ? 0 : -1;
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
