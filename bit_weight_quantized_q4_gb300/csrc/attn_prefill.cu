// attn_prefill.cu -- causal attention of packed prompt rows over the pages of
// their sequences (honeycrisp/mod.rs, gpu_attention, for a prompt): a warp per
// row and head.
#include "attn_prefill_row.cuh"

namespace q4 {
namespace dev {

template <typename T, int D>
__global__ void __launch_bounds__(256) q4attn_prefill_rows_kernel(const __grid_constant__ PrefillParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x;
    int seq, pos;
    if (!locate_row(p, row, lane, seq, pos)) return;
    for (int h = threadIdx.x >> 5; h < p.H; h += 8) attn_row<T, D>(p, row, h, seq, pos, lane);
}

}  // namespace dev

template <typename T, int D>
static int launch_rows(const PrefillParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dev::q4attn_prefill_rows_kernel<T, D>, p) == cudaSuccess ? 0 : -1;
}

int launch_prefill(const PrefillParams &p, int dtype, void *stream_) {
    cudaStream_t s = (cudaStream_t)stream_;
    switch (dtype) {
        case 0: return p.D == 64 ? launch_rows<float, 64>(p, s) : launch_rows<float, 128>(p, s);
        case 1: return p.D == 64 ? launch_rows<__half, 64>(p, s) : launch_rows<__half, 128>(p, s);
        case 2: return p.D == 64 ? launch_rows<__nv_bfloat16, 64>(p, s) : launch_rows<__nv_bfloat16, 128>(p, s);
    }
    return -1;
}

}  // namespace q4
